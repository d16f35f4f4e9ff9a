"""Pins the oracles of block-scaled quantisation, of the gated gradient and of
the norms on worked examples and on differences."""
import numpy as np
import torch

from oracle import fp8 as O
from oracle import norms as N


def test_group_codes_worked_example():
    """Largest value 448: the scale is 1, values are coded as they are."""
    v = np.zeros(128)
    v[:6] = [448, -1, 17, 18, 19, 2.0 ** -10]
    c, s = O.group_codes(v)
    assert s == 1 and c[0] == 0x7E and c[1] == 0xB8
    # steps of 2 at 16..32: 17 and 19 are ties, to even codes 16 and 20
    assert O.values(c[:6]).tolist() == [448, -1, 16, 18, 20, 0]
    c, s = O.group_codes(np.zeros(128))
    assert not c.any() and s == np.float32(2.0 ** -100) / np.float32(448)
    for bad in (np.inf, np.nan):
        v[0] = bad
        c, s = O.group_codes(v)
        with np.errstate(invalid="ignore"):
            assert np.isnan(O.values(c) * np.float64(s)).all()


def test_codes_are_the_type_s_own():
    """Every finite code decodes to what the tensor type says."""
    c = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    v = c.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, O.values(c.numpy()), equal_nan=True)


def test_layouts():
    x = np.arange(3 * 130, dtype=np.float64).reshape(3, 130)
    c, s = O.quantise_rows(x)
    assert c.shape == (3, 256) and s.shape == (2, 3) and not c[:, 130:].any()
    assert np.abs(O.row_values(c, s)[:, :130] - x).max() <= 390 * 2.0 ** -4
    c, s = O.quantise_blocks(x)
    assert c.shape == (3, 256) and s.shape == (1, 2)
    assert s[0, 0] == np.float32(387) / np.float32(448) and s[0, 1] == np.float32(389) / np.float32(448)


def difference(f, v, d, h=1e-6):
    """Directional derivative of sum(d * f) by central differences."""
    g = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        e = np.zeros_like(v)
        e[i] = h
        g[i] = np.sum(d * (f(v + e) - f(v - e))) / (2 * h)
    return g


def test_gated_backward_is_the_difference():
    rng = np.random.default_rng(0)
    z, da = rng.standard_normal((3, 10)), rng.standard_normal((3, 5))
    ref = difference(lambda v: O.silu(v[:, :5]) * v[:, 5:], z, da)
    assert np.abs(O.gated_backward(z, da) - ref).max() < 1e-8


def test_norm_gradients_are_the_differences():
    """Each gradient against differences of the forward formulas, for every
    spread of the gate, with and without its parts."""
    rng = np.random.default_rng(1)
    T, n, eps, eps2, alpha = 3, 7, 0.01, 0.02, 0.6
    y, r, dout, dnext = (rng.standard_normal((T, n)) for _ in range(4))
    w, w2 = rng.standard_normal(n), rng.standard_normal(n)
    for gate in (None, rng.standard_normal((T, 1)), rng.standard_normal((1, n)), rng.standard_normal((T, n))):
        for weight in (w, None):
            for dn, do in ((dnext, dout), (None, dout), (dnext, None)):
                def loss(y=y, r=r, weight=weight, gate=gate, w2=w2):
                    h = N.after(y, r, alpha, weight, gate, eps)
                    return (0 if do is None else (do * h).sum()) + (0 if dn is None else (dn * N.before(h, w2, eps2)).sum())
                h = N.after(y, r, alpha, weight, gate, eps)
                dy, dr, dw, dg, dw2 = N.backward(do, dn, y, h, alpha, weight, gate, w2, eps, eps2)

                def near(got, name, v):
                    ref = difference(lambda x: np.array(loss(**{name: x})), v, 1.0)
                    assert np.abs(got - ref).max() < 1e-7, name
                near(dy, "y", y)
                near(dr, "r", r)
                if weight is not None:
                    near(dw, "weight", weight)
                if gate is not None:
                    near(dg, "gate", gate)
                if dn is not None:
                    near(dw2, "w2", w2)


def test_layer_worked_example():
    """One token, three experts of which the ties' lower ids win."""
    x = np.array([[1.0, 2.0]])
    router = np.array([[0.0, 0.0], [1.0, 0.0], [1.0, 0.0]])
    gu = {1: np.array([[1.0, 0.0], [0.0, 1.0]]), 2: np.array([[0.0, 1.0], [1.0, 0.0]])}
    dn = {1: np.array([[1.0], [0.0]]), 2: np.array([[0.0], [4.0]])}
    out, ids, w, z = O.layer(x, router, None, 2, gu.get, dn.get)
    assert ids.tolist() == [[1, 2]] and w.tolist() == [[0.5, 0.5]] and z.tolist() == [[0, 1, 1]]
    s = lambda g: g / (1 + np.exp(-g))
    assert np.allclose(out, [[0.5 * s(1.0) * 2, 0.5 * 4 * s(2.0)]], rtol=1e-15)
    out, ids, _, _ = O.layer(x, router, np.array([2.0, 0, 0]), 1, {0: gu[1]}.get, {0: dn[1]}.get, base=np.ones((1, 2)))
    assert ids.tolist() == [[0]] and np.allclose(out, [[1 + s(1.0) * 2, 1]])
