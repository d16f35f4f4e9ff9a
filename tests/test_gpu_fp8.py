"""GPU parity of the block-scaled 8-bit operators with the float64 oracle.

Quantisation is defined to the bit (three fp32 roundings and one to E4M3), so
codes and scales are equal.  Of silu(gate) * up the fp32 value is off by at
most 4 u of itself (u = 2^-23: exp one step, sum, quotient and product half a
step each, with room), hence the scale by 5 u, and a code stands for its value
within half a step: 2^-4 of it, or 2^-10 of the scale where that is larger.

Products: inside a group of 128 the products of codes are exact.  In fp32 sums
(u for a step, the matrix instruction may truncate) a result passes 128 sums in
its group, one product of scales, one with them and one sum per group, all
below m = sum |a| |w| scales: |error| <= (2 * 128 + 2 G + 16) u m.  The 8-bit
matrix instruction, which 16-bit outputs of many rows take, adds 8 neighbouring
products at a time and keeps of each what is over 2^-13 of the largest one's
power of two: at most 8 * 2^-13 * (largest |a w|) per 8, m8 in all.  Half a
step of the output type comes on top.  Small integers and scales of powers of
two pass every sum exactly, on every path."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import dispatch as D
from expert_ffn_execution_router_amd import fp8
from oracle import fp8 as O

pytestmark = pytest.mark.gpu

BF, HF, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -23
TYPES = [BF, HF, F32]


def half(t):
    return torch.finfo(t).eps / 2


def np64(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def empty_codes(*shape, fill=0xAA):
    return torch.full(shape, fill, dtype=torch.uint8, device="cuda").view(F8)


def rows_for(R, K):
    return empty_codes(R, fp8.padded(K)), torch.full((fp8.padded(K) // 128, R), -7.0, device="cuda")


def cols_for(R, K):
    return empty_codes(K, fp8.padded(R)), torch.full((fp8.padded(R) // 128, K), -7.0, device="cuda")


def values_of(rng, R, K, dt, pad=0):
    v = rng.standard_normal((R, K + pad)) * np.exp(rng.standard_normal((R, 1)) * 2)
    return torch.from_numpy(v.astype(np.float32)).to(dt).cuda()[:, :K]


def same_codes(codes, scales, ref):
    """Equal values: the signs of zeros and NaN aside, which the oracle's encoder
    does not give."""
    got, want = (np.where((c & 0x7F) % 0x7F == 0, c & 0x7F, c) for c in (bits(codes), ref[0]))
    assert np.array_equal(got, want), np.argwhere(got != want)[:4]
    assert np.array_equal(scales.cpu().numpy(), ref[1], equal_nan=True)


SIZES = [(1, 1), (1, 128), (1, 4096), (2, 127), (3, 129), (7, 300), (127, 64), (128, 128), (129, 257), (260, 1000),
         (400, 36)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("R,K", SIZES)
def test_quantize(R, K, dt):
    print(f"quantize R={R} K={K} {dt}", flush=True)
    rng = np.random.default_rng(R + K)
    for pad in (0, 5):
        x = values_of(rng, R, K, dt, pad)
        ref, ref_t = O.quantise_rows(np64(x)), O.quantise_rows(np64(x).T)
        c, s = rows_for(R, K)
        ct, st = cols_for(R, K)
        fp8.quantize(x, c, s)
        same_codes(c, s, ref)
        fp8.quantize(x, codes_t=ct, scales_t=st)
        same_codes(ct, st, ref_t)
        c2, s2 = rows_for(R, K)
        ct2, st2 = cols_for(R, K)
        fp8.quantize(x, c2, s2, ct2, st2)
        same_codes(c2, s2, ref)
        same_codes(ct2, st2, ref_t)


@pytest.mark.parametrize("dt", TYPES)
def test_quantize_special_values(dt):
    """Groups of zeros, of the smallest values, of the largest; signed zeros;
    an infinity or NaN spoils its own group alone."""
    print(f"special values {dt}", flush=True)
    tiny, top = float(torch.finfo(dt).tiny), float(torch.finfo(dt).max)
    x = torch.zeros(130, 384, dtype=dt, device="cuda")
    x[0] = -0.0
    x[1, :128] = tiny
    x[1, 128:256] = tiny / 4
    x[2] = top
    x[2, ::3] = -top
    x[3, 5], x[3, 200], x[4, 300] = float("inf"), float("nan"), -float("inf")
    x[5, :128] = torch.linspace(-3, 3, 128)
    x[6, 0], x[6, 1] = 1.0, 2.0 ** -17
    x[7:] = torch.randn(123, 384, device="cuda").to(dt)
    host = np64(x)
    c, s = rows_for(130, 384)
    ct, st = cols_for(130, 384)
    fp8.quantize(x, c, s, ct, st)
    same_codes(c, s, O.quantise_rows(host))
    same_codes(ct, st, O.quantise_rows(host.T))
    a = O.row_values(bits(c), s.cpu().numpy())
    bad = ~np.isfinite(a).reshape(130, 3, 128)
    spoilt = [(3, 0), (3, 1), (4, 2)]
    for r, g in spoilt:
        assert bad[r, g].all() or np.isinf(s[g, r].item())
        bad[r, g] = False
    assert not bad.any()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("k,K", [(1, 200), (3, 384)])
def test_quantize_through_a_map(dt, k, K):
    """Rows gathered through sorted pairs: padding rows become zeros, rows
    behind the last segment (and groups of nothing else) stay."""
    print(f"map k={k} K={K} {dt}", flush=True)
    rng = np.random.default_rng(k)
    x = values_of(rng, 50, K, dt)
    m = rng.integers(0, 50 * k, 400).astype(np.int32)
    m[rng.random(400) < 0.2] = -1
    m[7], m[8] = 50 * k, 2 ** 31 - 1                             # past x: zeros
    m[250:] = -2
    m[300] = -5
    host = np.where(((m >= 0) & (m < 50 * k))[:, None], np64(x)[np.clip(m, 0, 50 * k - 1) // k], 0)
    mt = torch.from_numpy(m).cuda()
    c, s = rows_for(400, K)
    ct, st = cols_for(400, K)
    fp8.quantize(x, c, s, ct, st, row_map=mt, map_div=k)
    ref, ref_t = O.quantise_rows(host), O.quantise_rows(host.T)
    ref[0][250:], ref[1][:, 250:] = 0xAA, -7
    ref_t[0][:, 256:], ref_t[1][2:] = 0xAA, -7
    same_codes(c, s, ref)
    same_codes(ct, st, ref_t)
    # rows that are grouped already: the map only says which there are
    xs = values_of(rng, 400, K, dt)
    xs[torch.from_numpy(m < 0).cuda()] = float("nan")
    host = np.where((m >= 0)[:, None], np64(xs), 0)
    c, s = rows_for(400, K)
    ct, st = cols_for(400, K)
    fp8.quantize(xs, c, s, ct, st, row_map=mt, map_div=0)
    ref, ref_t = O.quantise_rows(host), O.quantise_rows(host.T)
    ref[0][250:], ref[1][:, 250:] = 0xAA, -7
    ref_t[0][:, 256:], ref_t[1][2:] = 0xAA, -7
    same_codes(c, s, ref)
    same_codes(ct, st, ref_t)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("R,K", [(1, 64), (5, 300), (200, 130)])
def test_quantize_gated(R, K, dt):
    print(f"gated R={R} K={K} {dt}", flush=True)
    rng = np.random.default_rng(R * K)
    z = values_of(rng, R, 2 * K, dt, 3)
    h = np64(z)
    v = O.silu(h[:, :K]) * h[:, K:]
    c, s = rows_for(R, K)
    ct, st = cols_for(R, K)
    fp8.quantize(z, c, s, ct, st, gated=True)
    for codes, scales, ref in ((c, s, v), (ct, st, v.T)):
        n, w = ref.shape
        g = np.zeros((n, fp8.padded(w)))
        g[:, :w] = ref
        want = np.maximum(np.abs(g).reshape(n, -1, 128).max(2).T, 2.0 ** -100) / 448
        assert (np.abs(np64(scales) - want) <= 5 * U * want).all()
        got = O.row_values(bits(codes), scales.cpu().numpy())
        step = np.maximum(2.0 ** -4 * np.abs(g), 2.0 ** -10 * np.repeat(want.T, 128, 1))
        assert (np.abs(got - g) <= step * (1 + 16 * U) + 8 * U * np.abs(g)).all()
        assert (got[:, w:] == 0).all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lead,N,K", [((), 1, 1), ((), 128, 128), ((), 130, 300), ((3,), 200, 129), ((2,), 50, 640)])
def test_quantize_weights(lead, N, K, dt):
    print(f"weights {lead} N={N} K={K} {dt}", flush=True)
    rng = np.random.default_rng(N + K)
    w = torch.from_numpy(rng.standard_normal(lead + (N, K)).astype(np.float32)).to(dt).cuda()
    Np, Kp = fp8.padded(N), fp8.padded(K)
    c, s = empty_codes(*lead, N, Kp), torch.zeros(*lead, Np // 128, Kp // 128, device="cuda")
    ct, st = empty_codes(*lead, K, Np), torch.zeros(*lead, Kp // 128, Np // 128, device="cuda")
    fp8.quantize_weights(w, c, s, ct, st)
    one, two = empty_codes(*lead, N, Kp), empty_codes(*lead, K, Np)
    fp8.quantize_weights(w, one, torch.zeros_like(s))
    fp8.quantize_weights(w, codes_t=two, scales_t=torch.zeros_like(st))
    assert np.array_equal(bits(one), bits(c)) and np.array_equal(bits(two), bits(ct))
    for i in range(lead[0] if lead else 1):
        at = (lambda t: t[i]) if lead else (lambda t: t)
        ref = O.quantise_blocks(np64(at(w)))
        same_codes(at(c), at(s), ref)
        full = np.zeros((Np, Kp), dtype=np.uint8)
        full[:N] = ref[0]
        same_codes(at(ct), at(st), (full[:, :K].T, ref[1].T))


@pytest.mark.parametrize("dt", TYPES)
def test_gated_backward(dt):
    """Against the formula: s = 1 / (1 + e^-g) is off by 3 u, s (1 + g (1 - s))
    by 3 u (1 + |g|) + 4 u of its terms' magnitudes, the products by 2 u."""
    print(f"gated backward {dt}", flush=True)
    rng = np.random.default_rng(5)
    for R, I in ((1, 1), (3, 8), (40, 77), (300, 768)):
        z, da = values_of(rng, R, 2 * I, dt, 4), values_of(rng, R, I, dt, 1)
        z[0, 0] = -100.0
        dz = torch.full((R, 2 * I + 2), 3.0, device="cuda", dtype=dt)
        fp8.gated_backward(z, da, dz[:, :2 * I])
        h, d = np64(z), np64(da)
        ref = O.gated_backward(h, d)
        g, u = h[:, :I], h[:, I:]
        s = 1 / (1 + np.exp(-g))
        terms = s * (1 + np.abs(g) * (1 + 8 * U)) * np.abs(d)
        mag = np.concatenate([terms * np.abs(u) * (1 + np.abs(g)), terms], 1)
        tol = 16 * U * mag + half(dt) * 1.01 * np.abs(ref) + (2.0 ** -25 if dt == HF else 1e-37) + 1e-36 * mag.max()
        assert (np.abs(np64(dz[:, :2 * I]) - ref) <= tol).all()
        assert (dz[:, 2 * I:] == 3.0).all()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def random_codes(rng, *shape, small=False):
    """Codes of normal values, or of small integers."""
    v = rng.integers(-4, 5, shape) if small else rng.standard_normal(shape) * 100
    return torch.from_numpy(v.astype(np.float32)).clamp(-448, 448).to(F8).cuda()


def random_scales(rng, *shape, small=False):
    v = 2.0 ** rng.integers(-2, 3, shape) if small else np.exp(rng.standard_normal(shape)) * 1e-2
    return torch.from_numpy(v.astype(np.float32)).cuda()


def check_product(out, p, q, groups, small):
    """out against p [R, K] and q [N, K], scaled values on the device in fp64."""
    ref = p @ q.t().contiguous()
    got = out.double()
    if small:
        want = ref.to(F32)
        assert torch.equal(want.double(), ref)
        assert torch.equal(out, want.to(out.dtype))
        return
    mag = p.abs() @ q.abs().t().contiguous()
    tol = 1.01 * (2 * 128 + 2 * groups + 16) * U * mag
    if out.dtype != F32:
        m8 = torch.zeros_like(ref)
        for k in range(0, p.shape[1], 8):
            m8 += (p[:, None, k:k + 8] * q[None, :, k:k + 8]).abs().amax(2)
        tol += 8 * 2.0 ** -13 * 1.01 * m8
    tol = tol + half(out.dtype) * 1.01 * (ref.abs() + tol) + (2.0 ** -25 if out.dtype == HF else 2.0 ** -134)
    assert ((got - ref).abs() <= tol).all(), float(((got - ref).abs() / tol).max())


def row_val(c, s):
    return c.double() * s.double().t().repeat_interleave(128, 1)


def block_val(c, s):
    return c.double() * s.double().repeat_interleave(128, 0)[:c.shape[0]].repeat_interleave(128, 1)


PRODUCTS = [(1, 1, 128), (1, 300, 1024), (2, 128, 256), (16, 100, 384), (17, 130, 640), (32, 512, 128), (33, 257, 512),
            (64, 64, 1152), (65, 300, 256), (130, 96, 384), (257, 513, 256), (300, 1000, 512), (512, 512, 128)]


@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("ot", TYPES)
@pytest.mark.parametrize("R,N,K", PRODUCTS)
def test_linear(R, N, K, ot, small):
    print(f"linear R={R} N={N} K={K} {ot} small={small}", flush=True)
    rng = np.random.default_rng(R + N + K)
    a, w = random_codes(rng, R, K, small=small), random_codes(rng, N, K, small=small)
    sa = random_scales(rng, K // 128, R, small=small)
    sw = random_scales(rng, fp8.padded(N) // 128, K // 128, small=small)
    out = torch.full((R, N + 3), 7.0, device="cuda", dtype=ot)
    fp8.linear(a, sa, w, sw, out[:, :N])
    check_product(out[:, :N], row_val(a, sa), block_val(w, sw), K // 128, small)
    assert (out[:, N:] == 7.0).all()
    again = torch.empty(R, N, device="cuda", dtype=ot)
    fp8.linear(a, sa, w, sw, again)
    assert torch.equal(again, out[:, :N])


def segments(rng, T, k, E, align, drop=0.0, skew=True, extra=5):
    p = 1.0 / np.arange(1, E + 1) ** (1.5 if skew else 0.0)
    ids = np.argsort(-(np.log(p) + rng.gumbel(size=(T, E))), axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = D.sort_rows(T, k, E, align) + extra
    c, o, perm, pos = (torch.zeros(n, **i32) for n in (E, E + 1, rows, (T, k)))
    D.sort(torch.from_numpy(np.ascontiguousarray(ids)).cuda(), c, o, perm, pos, align=align)
    return ids, c, o, perm, pos


GROUPED = [(1, 1, 1, 40, 128, 1, 0.0), (1, 8, 128, 96, 256, 1, 0.0), (5, 3, 70, 36, 384, 128, 0.2),
           (64, 8, 32, 200, 256, 1, 0.0), (64, 4, 130, 130, 128, 128, 0.3), (300, 2, 5, 300, 256, 16, 0.0),
           (6, 2, 9, 16, 128, 4, 1.0), (700, 3, 4, 520, 384, 128, 0.1), (0, 2, 3, 64, 128, 128, 0.0)]


@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("ot", TYPES)
@pytest.mark.parametrize("T,k,E,N,K,align,drop", GROUPED)
def test_experts(T, k, E, N, K, align, drop, ot, small):
    print(f"experts T={T} k={k} E={E} N={N} K={K} align={align} {ot} small={small}", flush=True)
    rng = np.random.default_rng(T * 7 + E)
    _, c, o, perm, _ = segments(rng, T, k, E, align, drop)
    rows = perm.numel()
    a, w = random_codes(rng, rows, K, small=small), random_codes(rng, E, N, K, small=small)
    sa = random_scales(rng, K // 128, rows, small=small)
    sw = random_scales(rng, E, fp8.padded(N) // 128, K // 128, small=small)
    for counts in (c, None):
        out = torch.full((rows, N + 1), 5.0, device="cuda", dtype=ot)
        fp8.experts(a, sa, o, w, sw, out[:, :N], counts=counts)
        first, many = o.tolist(), c.tolist()
        stays = torch.ones(rows, dtype=torch.bool, device="cuda")
        for e in range(E):
            r = slice(first[e], first[e] + many[e] if counts is not None else first[e + 1])
            stays[r] = False
            if r.stop > r.start:
                check_product(out[r, :N], row_val(a[r], sa[:, r]), block_val(w[e], sw[e]), K // 128, small)
        assert (out[stays] == 5.0).all() and (out[:, N] == 5.0).all()


@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("R,N,K", [(1, 1, 1), (5, 40, 130), (128, 128, 128), (300, 257, 100), (1000, 33, 513),
                                   (130, 300, 520), (0, 7, 9), (5000, 40, 36), (9000, 130, 257)])
def test_weight_gradient(R, N, K, small):
    print(f"weight gradient R={R} N={N} K={K} small={small}", flush=True)
    rng = np.random.default_rng(R + N + K)
    Rp = fp8.padded(R)
    dy, x = random_codes(rng, N, Rp, small=small), random_codes(rng, K, Rp, small=small)
    sy, sx = random_scales(rng, Rp // 128, N, small=small), random_scales(rng, Rp // 128, K, small=small)
    dw = torch.full((N, K), 3.0, device="cuda")
    fp8.weight_gradient(dy, sy, x, sx, dw)
    p, q = row_val(dy, sy), row_val(x, sx)
    check_product(dw, p, q, Rp // 128, small)
    first = dw.clone()
    fp8.weight_gradient(dy, sy, x, sx, dw, add=True)
    assert torch.equal(dw, first + first)
    fp8.weight_gradient(dy, sy, x, sx, dw)
    assert torch.equal(dw, first)


@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("T,k,E,N,K,drop", [(1, 1, 1, 40, 64, 0.0), (64, 2, 9, 130, 200, 0.3), (700, 3, 4, 300, 136, 0.1),
                                            (5, 2, 40, 16, 24, 0.5), (0, 1, 3, 20, 20, 0.0)])
def test_weight_gradient_per_expert(T, k, E, N, K, drop, small):
    print(f"experts' gradient T={T} k={k} E={E} N={N} K={K} small={small}", flush=True)
    rng = np.random.default_rng(T + E)
    _, c, o, perm, _ = segments(rng, T, k, E, 128, drop)
    Rp = fp8.padded(perm.numel())
    dy, x = random_codes(rng, N, Rp, small=small), random_codes(rng, K, Rp, small=small)
    sy, sx = random_scales(rng, Rp // 128, N, small=small), random_scales(rng, Rp // 128, K, small=small)
    dw = torch.full((E, N, K), 3.0, device="cuda")
    fp8.weight_gradient(dy, sy, x, sx, dw, offsets=o)
    p, q, first = row_val(dy, sy), row_val(x, sx), o.tolist()
    for e in range(E):
        r = slice(first[e], first[e + 1])
        if r.stop == r.start:
            assert (dw[e] == 0).all()
        else:
            check_product(dw[e], p[:, r], q[:, r], (r.stop - r.start) // 128, small)
    total = dw.clone()
    fp8.weight_gradient(dy, sy, x, sx, dw, offsets=o, add=True)
    assert torch.equal(dw, total + total)


def test_spoilt_rows_touch_no_other():
    """A NaN or an infinite group gives a row of NaN, the others stay."""
    print("spoilt rows", flush=True)
    rng = np.random.default_rng(3)
    for R in (5, 40, 300):
        x = values_of(rng, R, 512, BF)
        x[2, 77], x[4, 300] = float("nan"), float("inf")
        c, s = rows_for(R, 512)
        fp8.quantize(x, c, s)
        w, sw = random_codes(rng, 150, 512), random_scales(rng, 2, 4)
        out = torch.empty(R, 150, device="cuda")
        fp8.linear(c, s, w, sw, out)
        assert out[[2, 4]].isnan().all()
        fine = [r for r in range(R) if r not in (2, 4)]
        check_product(out[fine], row_val(c[fine], s[:, fine]), block_val(w, sw), 4, False)


# ---------------------------------------------------------------------------
# the calls together
# ---------------------------------------------------------------------------

def training_step(b):
    """Forward and backward of the experts' FFN, as fp8.py's head shows it."""
    D.sort(b["ids"], b["counts"], b["offsets"], b["perm"], b["pos"], align=128)
    k, m = b["ids"].shape[1], dict(row_map=b["perm"])
    fp8.quantize(b["x"], *b["xq"], *b["xt"], map_div=k, **m)
    fp8.experts(*b["xq"], b["offsets"], *b["gu"], b["z"], counts=b["counts"])
    fp8.quantize(b["z"], *b["aq"], *b["at"], map_div=0, gated=True, **m)
    fp8.experts(*b["aq"], b["offsets"], *b["down"], b["y"], counts=b["counts"])
    D.unpermute(b["y"], b["pos"], b["w"], b["out"])
    D.unpermute_backward(b["dout"], b["y"], b["perm"], b["pos"], b["w"], b["dy"], b["dw"])
    fp8.quantize(b["dy"], *b["dq"], *b["dt"], map_div=0, **m)
    fp8.experts(*b["dq"], b["offsets"], *b["down_t"], b["da"], counts=b["counts"])
    fp8.weight_gradient(*b["dt"], *b["at"], b["ddown"], offsets=b["offsets"])
    fp8.gated_backward(b["z"], b["da"], b["dz"])
    fp8.quantize(b["dz"], *b["zq"], *b["zt"], map_div=0, **m)
    fp8.experts(*b["zq"], b["offsets"], *b["gu_t"], b["dxs"], counts=b["counts"])
    fp8.weight_gradient(*b["zt"], *b["xt"], b["dgu"], offsets=b["offsets"])
    D.permute_backward(b["dxs"], b["pos"], b["dx"])


def training_buffers(T, k, E, H, I, seed=0):
    rng = np.random.default_rng(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = D.sort_rows(T, k, E, 128)
    Rp = fp8.padded(rows)

    def codes(R, K):
        return (torch.zeros(R, K, dtype=torch.uint8, device="cuda").view(F8), torch.zeros(K // 128, R, device="cuda"))
    b = dict(ids=torch.zeros(T, k, **i32), counts=torch.zeros(E, **i32), offsets=torch.zeros(E + 1, **i32),
             perm=torch.zeros(rows, **i32), pos=torch.zeros(T, k, **i32), w=torch.zeros(T, k, device="cuda"),
             dw=torch.zeros(T, k, device="cuda"))
    # what no segment holds is never read: NaN there shows if it is
    for n, w in (("z", 2 * I), ("y", H), ("dy", H), ("da", I), ("dz", 2 * I), ("dxs", H)):
        b[n] = torch.full((rows, w), float("nan"), device="cuda", dtype=BF)
    for n in ("x", "out", "dout", "dx"):
        b[n] = torch.zeros(T, H, device="cuda", dtype=BF)
    for n, w in (("x", H), ("a", I), ("d", H), ("z", 2 * I)):
        b[n + "q"], b[n + "t"] = codes(rows, w), codes(w, Rp)
    b["ddown"], b["dgu"] = torch.zeros(E, H, I, device="cuda"), torch.zeros(E, 2 * I, H, device="cuda")
    for n, N, K in (("gu", 2 * I, H), ("down", H, I)):
        w = torch.from_numpy(rng.standard_normal((E, N, K)).astype(np.float32) / K ** 0.5).cuda()
        q = [torch.zeros(E, N, K, dtype=torch.uint8, device="cuda").view(F8),
             torch.zeros(E, N // 128, K // 128, device="cuda"),
             torch.zeros(E, K, N, dtype=torch.uint8, device="cuda").view(F8),
             torch.zeros(E, K // 128, N // 128, device="cuda")]
        fp8.quantize_weights(w, *q)
        b[n], b[n + "_t"] = tuple(q[:2]), tuple(q[2:])
    return b


def fill(b, seed):
    rng = np.random.default_rng(seed)
    T, k = b["ids"].shape
    E, H = b["counts"].numel(), b["x"].shape[1]
    b["ids"].copy_(torch.from_numpy(np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)))
    w = rng.random((T, k)).astype(np.float32) + 0.1
    b["w"].copy_(torch.from_numpy(w / w.sum(1, keepdims=True)))
    for n in ("x", "dout"):
        b[n].copy_(torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)))


def test_training_step_against_the_unquantised_one():
    """Results and gradients of the whole step beside those of the same FFN
    with the dequantised weights in float64.  Each quantisation is off by at
    most 2^-4 of a value, 2^-4 / sqrt(3) in the mean, independent from value to
    value; the input's, the activation's, the gradient's and its second one
    follow each other, so a result is off by at most 4 * 2^-4 / sqrt(3) = 0.15
    of itself in the 2-norm, with room for what they multiply in silu's slope
    (at most 1.1) and for 16-bit rounding: 0.2."""
    print("training step", flush=True)
    T, k, E, H, I = 150, 2, 5, 256, 384
    b = training_buffers(T, k, E, H, I)
    fill(b, 1)
    training_step(b)
    torch.cuda.synchronize()
    ids, w = b["ids"].long(), b["w"].double()
    gu = [block_val(b["gu"][0][e], b["gu"][1][e]) for e in range(E)]
    dn = [block_val(b["down"][0][e], b["down"][1][e]) for e in range(E)]
    x, dout = b["x"].double(), b["dout"].double()
    out, dx, dw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
    ddn, dgu = torch.zeros(E, H, I).double().cuda(), torch.zeros(E, 2 * I, H).double().cuda()
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        z = x[t] @ gu[e].t().contiguous()
        g, u = z[:, :I], z[:, I:]
        s = torch.sigmoid(g)
        a = g * s * u
        y = a @ dn[e].t().contiguous()
        out.index_add_(0, t, y * w[t, j][:, None])
        dw[t, j] = (dout[t] * y).sum(1)
        dy = dout[t] * w[t, j][:, None]
        da = dy @ dn[e]
        ddn[e] = dy.t().contiguous() @ a
        dz = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
        dgu[e] = dz.t().contiguous() @ x[t]
        dx.index_add_(0, t, dz @ gu[e])
    for n, ref in (("out", out), ("dw", dw), ("ddown", ddn), ("dgu", dgu), ("dx", dx)):
        err = float((b[n].double() - ref).norm() / ref.norm())
        print(n, err, flush=True)
        assert err < 0.2, (n, err)


def test_captured_training_step_replays_like_eager():
    print("captured", flush=True)
    b, eager = (training_buffers(90, 3, 6, 128, 256) for _ in range(2))
    fill(b, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        training_step(b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        training_step(b)
    for seed in range(4):
        fill(b, seed)
        fill(eager, seed)
        graph.replay()
        torch.cuda.synchronize()
        training_step(eager)
        torch.cuda.synchronize()
        for n in ("out", "dw", "ddown", "dgu", "dx", "offsets"):
            assert torch.equal(b[n], eager[n]), (seed, n)


def test_two_streams_at_once():
    print("two streams", flush=True)
    rng = np.random.default_rng(9)
    todo = []
    for i in range(2):
        R = 40 + 300 * i
        a, w = random_codes(rng, R, 1024), random_codes(rng, 700, 1024)
        sa, sw = random_scales(rng, 8, R), random_scales(rng, 6, 8)
        todo.append((torch.cuda.Stream(), a, sa, w, sw, torch.zeros(R, 700, device="cuda")))
    torch.cuda.synchronize()
    for s, *args in todo:
        fp8.linear(*args, stream=s)
    torch.cuda.synchronize()
    for _, a, sa, w, sw, out in todo:
        check_product(out, row_val(a, sa), block_val(w, sw), 8, False)


def test_experts_past_32_bits():
    """Codes of the last experts lie past 4 GiB, results past 2^31 values."""
    print("past 32 bits", flush=True)
    rng = np.random.default_rng(8)
    E, N, K, far = 70, 8192, 8192, 2 ** 30
    w = torch.randint(0, 120, (E, N, K), dtype=torch.uint8, device="cuda").view(F8)
    sw = torch.rand(E, N // 128, K // 128, device="cuda") * 0.01
    a, sa = random_codes(rng, 5, K), random_scales(rng, K // 128, 5)
    out = torch.empty(5, far, device="cuda", dtype=BF)[:, :N]
    o = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    o[35:], o[69:], o[70:] = 1, 2, 5
    fp8.experts(a, sa, o, w, sw, out)
    for e, r in ((34, [0]), (68, [1]), (69, [2, 3, 4])):
        n = torch.tensor([0, 1, 777, 4096, N - 1], device="cuda")
        wv = w[e][n].double() * sw[e][n // 128].double().repeat_interleave(128, 1)
        check_product(out[r][:, n], row_val(a[r], sa[:, r]), wv, K // 128, False)
