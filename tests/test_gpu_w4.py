"""GPU parity of the 4-bit group-scaled products with the float64 oracle.

The kernel's products are exact in fp32 (a 16-bit value times an integer up to
15), so only fp32 sums round, each by at most u = 2^-23 of the running
magnitude (the matrix instruction may truncate; nearest would be 2^-24).  A
result passes at most G sums inside its group, with the group's sum of x, then
one zero point and one scale product and one sum per group and wave; all
partial sums are below the magnitude m = sum |x| (q + |zero|) |scale|.  Hence
|error| <= (2 G + 2 K / G + 16) u m, and half a step of the output type on
top.  Where x, zeros and scales are integers and powers of two and m stays
below 2^24 steps of the result, no sum rounds and fp32 outputs are equal."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import dispatch as D
from expert_ffn_execution_router_amd import w4
from oracle import w4 as O

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -23


def half(t):
    return torch.finfo(t).eps / 2


def np64(t):
    return t.double().cpu().numpy()


def matrix(rng, lead, K, group, xt, st, with_zeros, exact=False):
    """Device codes, scales, zeros and their host values."""
    q = rng.integers(0, 16, lead + (K,))
    if exact:
        s = 2.0 ** rng.integers(-3, 3, lead + (K // group,))
        z = rng.integers(0, 16, lead + (K // group,)).astype(np.float64)
    else:
        s = rng.uniform(0.002, 0.02, lead + (K // group,)) * rng.choice([-1, 1, 1, 1], lead + (K // group,))
        z = rng.uniform(3, 12, lead + (K // group,))
    sd = torch.from_numpy(s.astype(np.float32)).to(st).cuda()
    zd = torch.from_numpy(z.astype(np.float32)).to(xt).cuda() if with_zeros else None
    return (torch.from_numpy(O.pack(q)).cuda(), sd, zd), (q, np64(sd), None if zd is None else np64(zd))


def xrows(rng, n, K, xt, exact=False, pad=0):
    v = rng.integers(-4, 5, (n, K + pad)) if exact else rng.standard_normal((n, K + pad))
    return torch.from_numpy(v.astype(np.float32)).to(xt).cuda()[:, :K]


def check(out, x, q, s, z, group, gated):
    """out rows [n, N'] against the oracle on x rows [n, K]; K/G groups."""
    ref, mag = O.product(x, q, s, z, group)
    K = x.shape[1]
    tol = 1.01 * (2 * group + 2 * (K // group) + 16) * U * mag
    if gated:
        n = ref.shape[1] // 2
        g, u, eg, eu = ref[:, :n], ref[:, n:], tol[:, :n], tol[:, n:]
        ref = O.silu(g) * u
        # |silu'| <= 1.1, |silu(g)| <= |g|; exp, sum, quotient and product: 8 roundings
        tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(O.silu(g)) * eu + 8 * U * np.abs(ref) + 1e-36
    got = np64(out)
    tol = tol + half(out.dtype) * 1.01 * (np.abs(ref) + tol) + (2.0 ** -25 if out.dtype == HF else 2.0 ** -134)
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err.max(), (err / tol).max())


SIZES = [(1, 2048, 2048, 128), (1, 16, 32, 32), (3, 1, 64, 64), (5, 1003, 2080, 32), (7, 100, 192, 64),
         (16, 50, 768, 128), (17, 33, 768, 256), (31, 130, 1024, 32), (33, 64, 1088, 64), (64, 260, 2048, 128),
         (65, 20, 512, 512), (150, 34, 96, 32), (0, 8, 64, 32), (2, 48, 4096, 128), (18, 40, 3968, 64),
         (17, 34, 6144, 32), (3, 33, 5120, 1024), (4, 20, 8320, 64), (2, 18, 16384, 128)]


@pytest.mark.parametrize("xt,st,ot", [(BF, BF, BF), (BF, HF, F32), (HF, HF, HF), (HF, BF, F32)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,N,K,group", SIZES)
def test_linear(T, N, K, group, xt, st, ot, zeros):
    print(f"linear T={T} N={N} K={K} group={group} {xt} {st} {ot} zeros={zeros}", flush=True)
    rng = np.random.default_rng(T + N + K)
    dev, host = matrix(rng, (N,), K, group, xt, st, zeros)
    x = xrows(rng, T, K, xt, pad=8)
    out = torch.full((T, N + 3), 7.0, device="cuda", dtype=ot)
    w4.linear(x, out[:, :N], *dev)
    check(out[:, :N], np64(x), *host, group, False)
    assert (out[:, N:] == 7.0).all()
    if N % 2 == 0:
        w4.linear(x, out[:, :N // 2], *dev, gated=True)
        check(out[:, :N // 2], np64(x), *host, group, True)


@pytest.mark.parametrize("xt", [BF, HF])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,N,K,group", [(1, 40, 2048, 128), (9, 40, 1056, 32), (20, 72, 832, 64), (64, 72, 2048, 256),
                                         (130, 17, 160, 32)])
def test_linear_exact_integers(T, N, K, group, xt, zeros):
    """Integer inputs and power-of-two scales: every sum is exact."""
    print(f"exact T={T} N={N} K={K} group={group} {xt} zeros={zeros}", flush=True)
    rng = np.random.default_rng(K)
    dev, host = matrix(rng, (N,), K, group, xt, xt, zeros, exact=True)
    x = xrows(rng, T, K, xt, exact=True)
    ref, mag = O.product(np64(x), *host, group)
    assert mag.max() < 2.0 ** 21                                 # steps of 2^-3
    out = torch.empty(T, N, device="cuda")
    w4.linear(x, out, *dev)
    assert np.array_equal(np64(out), ref)


def test_linear_rows_are_independent():
    """A row with NaN or an infinity touches no other row."""
    print("rows independent", flush=True)
    rng = np.random.default_rng(3)
    dev, host = matrix(rng, (96,), 1024, 64, BF, BF, True)
    x = xrows(rng, 64, 1024, BF)
    x[5, 77] = float("nan")
    x[40, 3] = float("inf")
    for n in (6, 16, 30, 64):
        out = torch.empty(n, 96, device="cuda")
        w4.linear(x[:n], out, *dev)
        fine = [r for r in range(n) if r not in (5, 40)]
        assert all(out[r].isnan().all() for r in (5, 40) if r < n)
        check(out[fine], np64(x)[fine], *host, 64, False)


def test_small_and_large_values():
    """fp16 subnormal inputs and inputs near both types' limits."""
    print("value range", flush=True)
    rng = np.random.default_rng(4)
    for xt, mag in ((HF, 2.0 ** -20), (HF, 3e4), (BF, 2.0 ** -120), (BF, 2.0 ** 100)):
        dev, host = matrix(rng, (32,), 256, 32, xt, BF, False)
        x = (xrows(rng, 4, 256, F32).clamp(-2, 2) * mag).to(xt)
        out = torch.empty(4, 32, device="cuda")
        w4.linear(x, out, *dev)
        check(out, np64(x), *host, 32, False)


def grouped(T, k, E, seed, skew=False, drop=0.0, align=1, extra=0):
    rng = np.random.default_rng(seed)
    p = 1.0 / np.arange(1, E + 1) ** (1.5 if skew else 0.0)
    ids = np.argsort(-(np.log(p) + rng.gumbel(size=(T, E))), axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = D.sort_rows(T, k, E, align) + extra
    c, o, perm, pos = (torch.zeros(n, **i32) for n in (E, E + 1, rows, (T, k)))
    d = torch.from_numpy(np.ascontiguousarray(ids)).cuda()
    D.sort(d, c, o, perm, pos, align=align)
    return ids, c, o, perm, pos


GROUPED = [(1, 8, 128, 96, 256, 128, False, 0.0, 1), (1, 1, 1, 40, 64, 32, False, 0.0, 1),
           (5, 3, 70, 36, 192, 64, False, 0.2, 1), (64, 8, 32, 64, 256, 128, True, 0.0, 1),
           (64, 4, 130, 34, 160, 32, True, 0.3, 16), (300, 2, 5, 48, 128, 64, True, 0.0, 8),
           (6, 2, 9, 16, 64, 32, False, 1.0, 4), (40, 3, 300, 44, 4096, 64, True, 0.1, 1),
         (9, 2, 6, 70, 8448, 128, False, 0.0, 1)]


@pytest.mark.parametrize("xt,ot,zeros", [(BF, BF, False), (HF, F32, True), (BF, F32, True)])
@pytest.mark.parametrize("T,k,E,N,K,group,skew,drop,align", GROUPED)
@pytest.mark.parametrize("gated", [False, True])
def test_experts(T, k, E, N, K, group, skew, drop, align, gated, xt, ot, zeros):
    """Token rows through the sorted pairs, and grouped rows, per expert;
    padding rows, rows behind the last segment and spare columns stay."""
    print(f"experts T={T} k={k} E={E} N={N} K={K} group={group} align={align} gated={gated} {xt} {ot}", flush=True)
    rng = np.random.default_rng(T * 7 + E)
    ids, c, o, perm, pos = grouped(T, k, E, 1, skew, drop, align, extra=5)
    dev, (q, s, z) = matrix(rng, (E, N), K, group, xt, xt, zeros)
    x = xrows(rng, T, K, xt, pad=16)
    rows, cols = perm.numel(), N // 2 if gated else N
    out = torch.full((rows, cols + 1), 5.0, device="cuda", dtype=ot)
    w4.experts(x, o, out[:, :cols], *dev, counts=c, row_map=perm, map_div=k, gated=gated)
    xs = torch.full((rows, K), float("nan"), device="cuda", dtype=xt)
    D.permute(x, None, pos, xs)
    again = torch.full((rows, cols), 5.0, device="cuda", dtype=ot)
    w4.experts(xs, o, again, *dev, counts=c, gated=gated)
    assert torch.equal(again, out[:, :cols])                      # the same arithmetic on the same rows
    pm, tok = perm.cpu().numpy(), np64(x)
    assert (out[torch.from_numpy(pm < 0).cuda()] == 5.0).all() and (out[:, cols] == 5.0).all()
    flat = ids.reshape(-1)
    for e in range(E):
        r = np.nonzero((pm >= 0) & (flat[np.maximum(pm, 0)] == e))[0]
        if len(r):
            check(out[torch.from_numpy(r).cuda(), :cols], tok[pm[r] // k], q[e], s[e], None if z is None else z[e],
                  group, gated)


def test_experts_map_outside_reads_zeros():
    print("map outside", flush=True)
    rng = np.random.default_rng(6)
    dev, (q, s, z) = matrix(rng, (2, 24), 128, 32, BF, BF, True)
    x = xrows(rng, 3, 128, BF)
    i32 = dict(dtype=torch.int32, device="cuda")
    o = torch.tensor([0, 4, 6], **i32)
    m = torch.tensor([2, -1, 3, 0, -7, 2 ** 31 - 1], **i32)
    out = torch.full((6, 24), 5.0, device="cuda")
    w4.experts(x, o, out, *dev, row_map=m)
    assert (out[[1, 2, 4, 5]] == 0).all()
    check(out[[0, 3]], np64(x)[[2, 0]], q[0], s[0], z[0], 32, False)


def test_experts_past_32_bits():
    """Codes of the last experts lie past 4 GiB, their rows and results past
    2^31 values."""
    print("experts past 32 bits", flush=True)
    rng = np.random.default_rng(8)
    E, N, K, group, far = 70, 8192, 16384, 512, 2 ** 30
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.rand(E, N, K // group, device="cuda").mul_(0.01).to(BF)
    x = torch.empty(5, far, device="cuda", dtype=BF)[:, :K]
    x.copy_(xrows(rng, 5, K, BF))
    out = torch.empty(5, far, device="cuda", dtype=BF)[:, :N]
    o = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    o[35:], o[69:], o[70:] = 1, 2, 5
    w4.experts(x, o, out, codes, scales)
    for e, r in ((34, [0]), (68, [1]), (69, [2, 3, 4])):
        n = torch.tensor([0, 1, 777, 4096, N - 1], device="cuda")
        b = codes[e][n].cpu().numpy()
        q = np.stack([b & 15, b >> 4], -1).reshape(len(n), K)
        check(out[r][:, n], np64(x[r]), q, np64(scales[e][n]), None, group, False)


def test_two_streams_at_once():
    """Two products of different weights in flight together, each on its own
    stream."""
    print("two streams", flush=True)
    rng = np.random.default_rng(9)
    todo = []
    for i in range(2):
        dev, host = matrix(rng, (130,), 6144, 64, BF, BF, i == 1)
        todo.append((torch.cuda.Stream(), xrows(rng, 7 + i, 6144, BF), torch.zeros(7 + i, 130, device="cuda"), dev, host))
    torch.cuda.synchronize()
    for s, x, out, dev, _ in todo:
        w4.linear(x, out, *dev, stream=s)
    torch.cuda.synchronize()
    for _, x, out, _, host in todo:
        check(out, np64(x), *host, 64, False)


def layer(b):
    """A MoE layer on 4-bit experts with a gated shared expert."""
    D.sort(b["ids"], b["counts"], b["offsets"], b["perm"], b["pos"])
    w4.experts(b["x"], b["offsets"], b["a"], *b["gu"], row_map=b["perm"], map_div=b["ids"].shape[1], gated=True)
    w4.experts(b["a"], b["offsets"], b["z"], *b["down"])
    w4.linear(b["x"], b["sa"], *b["sgu"], gated=True)
    w4.linear(b["sa"], b["base"], *b["sdown"])
    D.unpermute(b["z"], b["pos"], b["w"], b["out"], base=b["base"])


def layer_buffers(T, k, E, H, I, seed=0):
    rng = np.random.default_rng(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    b = dict(ids=torch.zeros(T, k, **i32), counts=torch.zeros(E, **i32), offsets=torch.zeros(E + 1, **i32),
             perm=torch.zeros(T * k, **i32), pos=torch.zeros(T, k, **i32), w=torch.zeros(T, k, device="cuda"),
             x=torch.zeros(T, H, device="cuda", dtype=BF), a=torch.zeros(T * k, I, device="cuda", dtype=BF),
             z=torch.zeros(T * k, H, device="cuda", dtype=BF), sa=torch.zeros(T, I, device="cuda", dtype=BF),
             base=torch.zeros(T, H, device="cuda"), out=torch.zeros(T, H, device="cuda", dtype=BF))
    host = {}
    for name, lead, K in (("gu", (E, 2 * I), H), ("down", (E, H), I), ("sgu", (2 * I,), H), ("sdown", (H,), I)):
        q = rng.integers(0, 16, lead + (K,))
        s = torch.full(lead + (K // 128,), 2.0 ** -7, device="cuda", dtype=BF)
        b[name], host[name] = (torch.from_numpy(O.pack(q)).cuda(), s, None), q
    return b, host


def test_layer_equals_the_framework_forward():
    """The 4-bit layer against moe_layer_forward on the same weights in
    bf16 (codes times a power of two are exact there) and the same router,
    the shared expert entering both as an fp32 partial: both round A and Z to
    bf16 and the output once, so they differ by the framework's bf16
    tolerance at most."""
    import synth
    from expert_ffn_execution_router_amd.runtime import HostPool, MoeRuntime
    print("layer against the framework forward", flush=True)
    T, k, E, H, I = 24, 4, 16, 256, 128
    b, host = layer_buffers(T, k, E, H, I)
    cfg = synth.MoeShape("w4", L=1, E=E, k=k, H=H, I=I, fmt=0, slot_fraction=1.0)
    pool = HostPool(E * cfg.expert_bytes)
    wgu = (host["gu"] - 8.0) * 2.0 ** -7
    wd = (host["down"] - 8.0) * 2.0 ** -7
    blob = np.concatenate([wgu.reshape(E, -1), wd.reshape(E, -1)], 1).astype(np.float32)
    pool.array()[:] = (blob.view(np.uint32) >> 16).astype(np.uint16).reshape(-1).view(np.uint8)
    rt = MoeRuntime(1, E, k, H, I, 0, E, T, pool, host_threads=2)
    try:
        rt.admit(0, list(range(E)))
        b["x"].copy_(torch.from_numpy(np.random.default_rng(1).standard_normal((T, H)).astype(np.float32)))
        R = torch.from_numpy(np.random.default_rng(2).standard_normal((E, H)).astype(np.float32) * 0.1).cuda()
        rt.route(b["x"], R, None, b["ids"], b["w"])
        layer(b)
        ref = torch.empty(T, H, device="cuda", dtype=BF)
        rt.forward(0, b["x"], R, None, rt.slot_table()[:E], ref, host_partial=b["base"])
        torch.cuda.synchronize()
        assert rt.check_device_error() == 0
        err = (b["out"].float() - ref.float()).abs().max() / ref.float().abs().max()
        assert err <= 1e-2, float(err)
    finally:
        rt.close()
        pool.free()


@pytest.mark.parametrize("T", [1, 40])
def test_layer_captured_replays_like_eager(T):
    print(f"captured layer T={T}", flush=True)
    k, E, H, I = 4, 32, 512, 256
    b, _ = layer_buffers(T, k, E, H, I)
    eager = {n: v.clone() if isinstance(v, torch.Tensor) else v for n, v in b.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(b)
    for seed in range(4):
        rng = np.random.default_rng(seed)
        ids = torch.from_numpy(np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)).cuda()
        x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
        for d in (b, eager):
            d["ids"].copy_(ids)
            d["x"].copy_(x)
            d["w"].copy_(torch.from_numpy(rng.random((T, k)).astype(np.float32)) if d is b else b["w"])
        graph.replay()
        torch.cuda.synchronize()
        layer(eager)
        torch.cuda.synchronize()
        for n in ("offsets", "pos", "a", "z", "base", "out"):
            assert torch.equal(b[n], eager[n]), (seed, n)
