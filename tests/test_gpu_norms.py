"""GPU parity of the norms around a block, forward and backward, with the
float64 oracle.

Forward: a mean of n squares is off by at most 40 u of itself (u = 2^-24 a
rounding; a thread sums up to 16 squares, waves and their sums add less than 16
more roundings, so 40 cover every width), its root and quotient by 3 more, so a
normed value by N = 32 u of itself; h by 3 roundings of its terms' magnitudes,
and half a step of its type.  The next norm is checked on the h that was
stored.  Backward: the mean of products is off by 44 u of the mean of their
magnitudes; the bounds below count each product and sum."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import fp8, norms
from oracle import fp8 as OF
from oracle import norms as O

pytestmark = pytest.mark.gpu

BF, HF, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
EPS, EPS2 = 1e-5, 1e-3
PAIRS = [(BF, BF), (BF, F32), (HF, HF), (HF, F32), (F32, F32)]
WIDTHS = [(1, 1), (1, 2048), (3, 7), (5, 64), (6, 511), (9, 513), (4, 1000), (5, 1025), (7, 2048), (3, 2500), (2, 4096),
          (3, 4100), (2, 8192), (3, 8200), (2, 16384), (70, 300), (0, 32)]
BACK = [w for w in WIDTHS if w[1] <= 8192]
GATES = ["none", "token", "channel", "full"]


def half(t):
    return torch.finfo(t).eps / 2


def least(t):
    return 2.0 ** -25 if t == HF else 2.0 ** -134


def np64(t):
    return t.double().cpu().numpy()


def dev(v, dt, pad=0):
    v = np.asarray(v, dtype=np.float32)
    if pad:
        v = np.concatenate([v, np.zeros((v.shape[0], pad), dtype=np.float32)], 1)
        return torch.from_numpy(v).to(dt).cuda()[:, :-pad]
    return torch.from_numpy(v).to(dt).cuda()


def gate_of(rng, kind, T, n, dt):
    if kind == "none":
        return None
    shape = dict(token=(T, 1), channel=(1, n), full=(T, n))[kind]
    return dev(rng.standard_normal(shape), dt)


def check_next(nxt, h, w, eps):
    """The next norm of stored rows h."""
    ref = O.before(h, w, eps)
    tol = 40 * U * np.abs(ref)
    tol = tol + half(nxt.dtype) * 1.01 * (np.abs(ref) + tol) + least(nxt.dtype)
    assert (np.abs(np64(nxt) - ref) <= tol).all()


def check_codes(codes, scales, h, w, eps):
    """Codes of the next norm: as of values off by 40 u, 42 u in the scale."""
    T, n = h.shape
    v = np.zeros((T, fp8.padded(n)))
    v[:, :n] = O.before(h, w, eps)
    want = np.maximum(np.abs(v).reshape(T, -1, 128).max(2).T, 2.0 ** -100) / 448
    assert (np.abs(np64(scales) - want) <= 43 * U * want).all()
    got = OF.row_values(codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy())
    step = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * np.repeat(want.T, 128, 1))
    assert (np.abs(got - v) <= step * (1 + 100 * U) + 90 * U * np.abs(v)).all()
    assert (got[:, n:] == 0).all()


@pytest.mark.parametrize("dt,rt", PAIRS)
@pytest.mark.parametrize("T,n", WIDTHS)
def test_before(T, n, dt, rt):
    print(f"before T={T} n={n} {dt} {rt}", flush=True)
    rng = np.random.default_rng(T + n)
    x = dev(rng.standard_normal((T, n)) * np.exp(rng.standard_normal((T, 1))), rt, 3)
    for wt in {dt, F32}:
        w = dev(1 + 0.3 * rng.standard_normal(n), wt)
        out = torch.full((T, n + 1), 9.0, device="cuda", dtype=dt)
        norms.before(x, w, out[:, :n], eps=EPS)
        check_next(out[:, :n], np64(x), np64(w), EPS)
        assert (out[:, n:] == 9.0).all()
        G = fp8.padded(n) // 128
        codes, s = torch.zeros(T, 128 * G, dtype=torch.uint8, device="cuda").view(F8), torch.zeros(G, T, device="cuda")
        if rt == dt or wt == dt:
            norms.before(x, w, codes, scales=s, eps=EPS)
            if T:
                check_codes(codes, s, np64(x), np64(w), EPS)


@pytest.mark.parametrize("dt,rt", PAIRS)
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,n", [w for w in WIDTHS if w[0] != 1 or w[1] in (1, 2048)])
def test_after(T, n, gate, dt, rt):
    print(f"after T={T} n={n} {gate} {dt} {rt}", flush=True)
    rng = np.random.default_rng(T * n)
    y = dev(rng.standard_normal((T, n)) * 2, dt, 2)
    r = dev(rng.standard_normal((T, n)), rt, 5)
    alpha = 0.75
    for wt, gt, with_w in ((dt, dt, True), (F32, F32, True), (dt, F32, False)):
        w = dev(1 + 0.3 * rng.standard_normal(n), wt) if with_w else None
        w2 = dev(1 + 0.3 * rng.standard_normal(n), wt)
        g = gate_of(rng, gate, T, n, gt)
        out = torch.full((T, n + 1), 9.0, device="cuda", dtype=rt)
        nxt = torch.full((T, n + 4), 9.0, device="cuda", dtype=dt)
        norms.after(y, r, out[:, :n], weight=w, gate=g, alpha=alpha, eps=EPS, next_weight=w2, next_out=nxt[:, :n],
                    next_eps=EPS2)
        hw, hg = None if w is None else np64(w), None if g is None else np64(g)
        ref = O.after(np64(y), np64(r), alpha, hw, hg, EPS)
        mag = np.abs(alpha * np64(r)) + np.abs(O.after(np64(y), None, 0, hw, hg, EPS))
        tol = 48 * U * mag
        tol = tol + half(rt) * 1.01 * (np.abs(ref) + tol) + least(rt)
        assert (np.abs(np64(out[:, :n]) - ref) <= tol).all()
        check_next(nxt[:, :n], np64(out[:, :n]), np64(w2), EPS2)
        assert (out[:, n:] == 9.0).all() and (nxt[:, n:] == 9.0).all()
        # alone, in place, and with codes: the same rows
        alone = torch.empty(T, n, device="cuda", dtype=rt)
        norms.after(y, r, alone, weight=w, gate=g, alpha=alpha, eps=EPS)
        assert torch.equal(alone, out[:, :n])
        place = r.clone()
        G = fp8.padded(n) // 128
        codes, s = torch.zeros(T, 128 * G, dtype=torch.uint8, device="cuda").view(F8), torch.zeros(G, T, device="cuda")
        norms.after(y, place, place, weight=w, gate=g, alpha=alpha, eps=EPS, next_weight=w2, next_out=codes,
                    next_scales=s, next_eps=EPS2)
        assert torch.equal(place, alone)
        if T:
            check_codes(codes, s, np64(out[:, :n]), np64(w2), EPS2)
        # and in two calls
        two = torch.empty(T, n, device="cuda", dtype=dt)
        norms.before(alone, w2, two, eps=EPS2)
        assert torch.equal(two, nxt[:, :n])


def through(v, d, eps):
    """Magnitude of the terms of the gradient through v / rms(v)."""
    r = O.rms(v, eps)
    m = np.abs(d) / r + np.abs(v) / r ** 3 * np.mean(np.abs(v * d), axis=1, keepdims=True)
    return m


@pytest.mark.parametrize("dt,rt", PAIRS)
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,n", BACK + [(1500, 40), (1100, 1500), (600, 4100)])
def test_after_backward(T, n, gate, dt, rt):
    print(f"after backward T={T} n={n} {gate} {dt} {rt}", flush=True)
    rng = np.random.default_rng(T * n + 1)
    alpha, forms = 0.75, ((dt, dt, True, True, True), (F32, F32, True, True, False), (dt, dt, False, False, True))
    y, h = dev(rng.standard_normal((T, n)) * 2, dt, 2), dev(rng.standard_normal((T, n)), rt, 1)
    dout, dnext = dev(rng.standard_normal((T, n)), rt), dev(rng.standard_normal((T, n)), dt, 3)
    for wt, gt, with_w, with_next, with_out in forms[:1 if T > 200 else 3]:
        w = dev(1 + 0.3 * rng.standard_normal(n), wt) if with_w else None
        w2 = dev(1 + 0.3 * rng.standard_normal(n), wt) if with_next else None
        g = gate_of(rng, gate, T, n, gt)
        dy = torch.full((T, n + 1), 9.0, device="cuda", dtype=dt)
        dr = torch.full((T, n + 2), 9.0, device="cuda", dtype=rt)
        dw, dw2 = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
        dg = None if g is None else torch.full_like(g, 9.0)
        norms.after_backward(dout if with_out else None, y, dy[:, :n], dr[:, :n], weight=w, dweight=dw if with_w else None,
                             gate=g, dgate=dg, alpha=alpha, eps=EPS, dnext=dnext if with_next else None,
                             out=h if with_next else None, next_weight=w2, dnext_weight=dw2 if with_next else None,
                             next_eps=EPS2)
        hy, hh = np64(y), np64(h)
        hw, hg, hw2 = (None if v is None else np64(v) for v in (w, g, w2))
        do, dn = np64(dout) if with_out else None, np64(dnext) if with_next else None
        ref = O.backward(do, dn, hy, hh, alpha, hw, hg, hw2, EPS, EPS2)
        # magnitudes of the terms, and the error of d = the whole gradient of h
        md = np.zeros((T, n)) if do is None else np.abs(do)
        if with_next:
            md = md + through(hh, np.abs(dn * hw2), EPS2)
        ed = 130 * U * md
        x = hy if hw is None else hy / O.rms(hy, EPS)
        ww, gg = (np.ones(n) if hw is None else hw), (np.ones((1, 1)) if hg is None else hg)
        mv = (md + ed) * np.abs(gg) * np.abs(ww)
        my = mv if hw is None else through(hy, mv, EPS)

        def near(got, want, err, t, name):
            err = err + half(t) * 1.01 * (np.abs(want) + err) + least(t)
            bad = np.abs(np64(got) - want) > err
            assert not bad.any(), (name, np.abs(np64(got) - want).max())
        # 130 u of d, one product with each of gate, weight and 1 / rms, mean and sum: 130 + 90
        near(dy[:, :n], ref[0], 220 * U * my, dt, "dy")
        near(dr[:, :n], ref[1], 132 * U * alpha * md, rt, "dr")
        assert (dy[:, n:] == 9.0).all() and (dr[:, n:] == 9.0).all()
        # sums over up to T rows (a part's rows in turn, then the parts): T roundings at most
        if with_w:
            near(dw, ref[2], (180 + T) * U * np.sum(md * np.abs(gg) * np.abs(x), 0), F32, "dw")
        if with_next:
            near(dw2, ref[4], (40 + T) * U * np.sum(np.abs(dn * hh) / O.rms(hh, EPS2), 0), F32, "dw2")
        if g is not None:
            m = md * np.abs(x * ww)
            for axis in (0, 1):
                if hg.shape[axis] == 1 and m.shape[axis] != 1:
                    m = m.sum(axis, keepdims=True)
            near(dg, ref[3], (230 + T) * U * m, gt, "dgate")


@pytest.mark.parametrize("dt,rt", PAIRS)
@pytest.mark.parametrize("T,n", BACK)
def test_before_backward(T, n, dt, rt):
    print(f"before backward T={T} n={n} {dt} {rt}", flush=True)
    rng = np.random.default_rng(T * n + 2)
    x, base = dev(rng.standard_normal((T, n)) * 3, rt, 2), dev(rng.standard_normal((T, n)), rt)
    dout, w = dev(rng.standard_normal((T, n)), dt), dev(1 + 0.3 * rng.standard_normal(n), dt)
    for b in (base, None):
        dx, dw = torch.full((T, n + 1), 9.0, device="cuda", dtype=rt), torch.full((n,), 9.0, device="cuda")
        norms.before_backward(dout, x, w, dx[:, :n], dw, base=b, eps=EPS)
        hb = None if b is None else np64(b)
        _, ref, _, _, refw = O.backward(hb, np64(dout), None, np64(x), 1.0, None, None, np64(w), EPS, EPS)
        m = through(np64(x), np.abs(np64(dout) * np64(w)), EPS) + (0 if b is None else np.abs(hb))
        err = 130 * U * m
        err = err + half(rt) * 1.01 * (np.abs(ref) + err) + least(rt)
        assert (np.abs(np64(dx[:, :n]) - ref) <= err).all() and (dx[:, n:] == 9.0).all()
        err = (42 + T) * U * np.sum(np.abs(np64(dout) * np64(x)) / O.rms(np64(x), EPS), 0) + 2.0 ** -134
        assert (np.abs(np64(dw) - refw) <= err).all()
        dx2 = torch.empty(T, n, device="cuda", dtype=rt)
        norms.before_backward(dout, x, w, dx2, base=b, eps=EPS)
        assert torch.equal(dx2, dx[:, :n])


def test_rows_are_independent():
    """A row with NaN or an infinity touches no other row; a row of zeros has
    a norm of zeros."""
    print("rows independent", flush=True)
    y = torch.randn(9, 700, device="cuda").to(BF)
    y[2, 5], y[4, 600], y[6] = float("nan"), float("inf"), 0
    w = torch.ones(700, device="cuda", dtype=BF)
    out = torch.empty_like(y)
    norms.before(y, w, out, eps=EPS)
    fine = [0, 1, 3, 5, 6, 7, 8]
    assert out[2].isnan().all() and out[4, 600].isnan() and (out[6] == 0).all()
    check_next(out[fine], np64(y[fine]), np64(w), EPS)


def test_captured_backward_replays_like_eager():
    """Also with a side stream and a workspace of the caller's."""
    print("captured", flush=True)
    T, n = 333, 1000

    def buffers():
        z = lambda *s, dt=BF: torch.zeros(s, device="cuda", dtype=dt)
        return dict(y=z(T, n), r=z(T, n), h=z(T, n), nx=z(T, n), w=z(n), w2=z(n), g=z(1, n), dh=z(T, n), dn=z(T, n),
                    dy=z(T, n), dr=z(T, n), dw=z(n, dt=F32), dw2=z(n, dt=F32), dg=z(1, n, dt=F32),
                    ws=z(norms.backward_workspace_bytes(T, n), dt=torch.uint8))

    def step(b):
        norms.after(b["y"], b["r"], b["h"], weight=b["w"], gate=b["g"], next_weight=b["w2"], next_out=b["nx"])
        norms.after_backward(b["dh"], b["y"], b["dy"], b["dr"], weight=b["w"], dweight=b["dw"], gate=b["g"], dgate=b["dg"],
                             dnext=b["dn"], out=b["h"], next_weight=b["w2"], dnext_weight=b["dw2"], ws=b["ws"])
    b, eager = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for seed in range(4):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        for k in ("y", "r", "w", "w2", "g", "dh", "dn"):
            b[k].copy_(torch.randn(b[k].shape, generator=gen, device="cuda"))
            eager[k].copy_(b[k])
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        for k in ("h", "nx", "dy", "dr", "dw", "dw2", "dg"):
            assert torch.equal(b[k], eager[k]), (seed, k)
