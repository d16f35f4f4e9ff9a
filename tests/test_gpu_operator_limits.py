"""GPU tests of the dispatch and 4-bit operators at the limits of what they
accept, against the float64 oracle."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import binding as B
from expert_ffn_execution_router_amd import dispatch as D
from expert_ffn_execution_router_amd import w4
from oracle import dispatch as O
from oracle import w4 as OW

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def np64(t):
    return t.double().cpu().numpy()


def test_neighbours_and_column_ranges_of_one_buffer():
    """Arrays that touch but do not meet are taken: a sort into one int
    buffer, end to end, and a copy between column ranges of one buffer."""
    print("neighbours", flush=True)
    T, k, E, cols = 700, 3, 16, 72                                # 2100 pairs: the sort over blocks, with a workspace
    ids = np.random.default_rng(0).integers(-1, E, (T, k)).astype(np.int32)
    n, need = T * k, D.sort_workspace_bytes(T, k, E)
    one = torch.zeros(n + E + (E + 1) + n + n + need // 4, dtype=torch.int32, device="cuda")
    d, counts, offsets, perm, pos, ws = torch.split(one, [n, E, E + 1, n, n, need // 4])
    d.copy_(torch.from_numpy(ids.reshape(-1)))
    D.sort(d.view(T, k), counts, offsets, perm, pos.view(T, k), ws=ws.view(torch.uint8))
    ref = O.sort_pairs(ids, E, 1, n)
    for g, r in zip((counts, offsets, perm, pos.view(T, k)), ref):
        assert np.array_equal(g.cpu().numpy(), r)
    assert np.array_equal(d.view(T, k).cpu().numpy(), ids)

    buf = torch.randn(n, 2 * cols, device="cuda").to(BF)
    x, out = buf[:T, cols:], buf[:, :cols]
    rows, want = np64(x), np64(out)
    step = 2 * cols
    rc = B.moe_permute(B.MOE_T_BF16, x.data_ptr(), step, None, pos.data_ptr(), T, k, n, cols, out.data_ptr(), step,
                       torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert np.array_equal(np64(out), O.permute(rows, ref[2], ref[3], want))
    assert np.array_equal(np64(x), rows)


def test_index_and_weight_tensors_are_looked_at():
    """Through the torch layer, with nothing run: results over places,
    weights, counts and scales."""
    print("shared", flush=True)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, counts, offsets, perm, pos = (torch.full(s, -1, **i32) for s in ((4, 2), (8,), (9,), (8,), (4, 2)))
    x, y, w = torch.ones(4, 64, device="cuda"), torch.ones(8, 64, device="cuda"), torch.ones(4, 2, device="cuda")
    codes, scales = torch.zeros(1, 16, 32, device="cuda", dtype=torch.uint8), torch.ones(1, 16, 2, device="cuda", dtype=BF)
    calls = [lambda: D.sort(ids, counts, offsets, perm, ids),
             lambda: D.sort(ids, offsets[1:], offsets, perm, pos),
             lambda: D.sort(ids, counts, offsets, pos.view(-1), pos),
             lambda: D.unpermute_backward(x, y, perm, pos, w, torch.empty_like(y), w),
             lambda: D.unpermute(y[:, :1], pos, w, w[:, :1]),
             lambda: D.permute(x[:, :1], None, pos, pos.view(torch.float32).view(8, 1)),
             lambda: w4.linear(x[:1].to(BF), scales.view(1, 32)[:, :16], codes[0], scales[0])]
    for call in calls:
        with pytest.raises(B.MoeError, match="shares memory"):
            call()
    assert (ids == -1).all() and (pos == -1).all() and (w == 1).all() and (scales == 1).all() and (offsets == -1).all()


# E, N, K, group: as few group values as one load of a step reads, or fewer in
# a matrix of several
FEWEST = [(1, 1, 128, 32), (1, 2, 64, 32), (2, 1, 64, 32), (3, 1, 64, 32), (5, 1, 96, 32), (4, 1, 32, 32), (1, 1, 32, 32),
          (1, 1, 128, 64), (1, 1, 192, 64), (3, 1, 128, 64), (1, 1, 256, 128), (1, 1, 384, 128), (2, 1, 256, 128),
          (1, 1, 512, 256), (1, 1, 64, 64)]


@pytest.mark.parametrize("xt", [BF, HF])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("E,N,K,group", FEWEST)
def test_fewest_group_values(E, N, K, group, zeros, xt):
    """Exact integers; what lies beside the scales and zeros is NaN, so a
    value read from there would show, were its x a zero."""
    print(f"fewest E={E} N={N} K={K} group={group} zeros={zeros} {xt}", flush=True)
    rng = np.random.default_rng(E + N + K)
    q = rng.integers(0, 16, (E, N, K))
    s = 2.0 ** rng.integers(-3, 3, (E, N, K // group))
    z = rng.integers(0, 16, s.shape).astype(np.float64) if zeros else None
    xv = rng.integers(-4, 5, (2 * E + 1, K)).astype(np.float64)

    def among_nan(v):
        b = torch.full((v.size + 32,), float("nan"), dtype=xt, device="cuda")
        b[16:16 + v.size] = torch.from_numpy(v.reshape(-1)).to(xt).cuda()
        return b[16:16 + v.size].view(v.shape)
    sd, zd = among_nan(s), among_nan(z) if zeros else None
    x = torch.from_numpy(xv).to(xt).cuda()
    out = torch.full((2 * E + 1, N), 5.0, device="cuda")
    codes = torch.from_numpy(OW.pack(q)).cuda()
    o = torch.arange(0, 2 * E + 1, 2, dtype=torch.int32, device="cuda")
    w4.experts(x, o, out, codes, sd, zeros=zd)
    for e in range(E):
        ref, _ = OW.product(xv[2 * e:2 * e + 2], q[e], s[e], None if z is None else z[e], group)
        assert np.array_equal(np64(out[2 * e:2 * e + 2]), ref), e
    assert (out[2 * E] == 5.0).all()
    if E == 1:
        dense = torch.empty(2, N, device="cuda")
        w4.linear(x[:2], dense, codes[0], sd[0], zeros=None if zd is None else zd[0])
        assert torch.equal(dense, out[:2])


@pytest.mark.parametrize("zero", [None, -16.0, 16.0])
@pytest.mark.parametrize("K,group", [(256, 32), (256, 64), (640, 128), (1024, 512), (6144, 64), (6144, 2048)])
def test_largest_inputs(K, group, zero):
    """bf16 inputs just below 2^116, all of one sign in a row, against the
    codes that make its sums largest.  x = 15 2^112: q x, zero x and all their
    sums are integers times 2^112, below 31 15 K < 2^22 of them, so no sum
    rounds; the scale is a power of two."""
    print(f"largest K={K} group={group} zero={zero}", flush=True)
    rng = np.random.default_rng(K)
    q = rng.integers(0, 16, (20, K))
    q[:8], q[8:12] = 15, 0
    s = np.full((20, K // group), 2.0 ** -20)
    z = None if zero is None else np.full(s.shape, zero)
    xv = np.full((5, K), 15 * 2.0 ** 112) * np.array([1, -1, 1, -1, 1])[:, None]
    xv[4, ::3] = 0
    sd = torch.from_numpy(s).to(BF).cuda()
    zd = None if zero is None else torch.from_numpy(z).to(BF).cuda()
    out = torch.empty(5, 20, device="cuda")
    w4.linear(torch.from_numpy(xv).to(BF).cuda(), out, torch.from_numpy(OW.pack(q)).cuda(), sd, zeros=zd)
    ref, _ = OW.product(xv, q, s, z, group)
    assert np.array_equal(np64(out), ref)


# ---------------------------------------------------------------------------
# every path through the 4-bit kernel
# ---------------------------------------------------------------------------
# Integer x in [-2, 2], codes and zeros in [0, 15], scales 1/2 or 1: all sums
# are integers and halves below 60 K < 2^19, so fp32 rounds none, in any order,
# and a product equals the float64 one in every value.  A gated result takes
# exp, sum, quotient and two products from exact z: 8 roundings of 2^-23, and
# where exp overflows (gate below -88.7) |silu| < 3e-37 becomes 0.

def integers(g, E, N, K, group, zeros, xt):
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(1, 3, (E, N, K // group), generator=g, device="cuda").to(xt) / 2
    z = torch.randint(0, 16, s.shape, generator=g, device="cuda").to(xt) if zeros else None
    return codes, s, z


def product64(x, codes, s, z, group):
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    z = 8.0 if z is None else z.double().repeat_interleave(group, -1)
    w = (q - z) * s.double().repeat_interleave(group, -1)
    return x.double() @ w.t().contiguous()


def same(out, z, gated):
    if not gated:
        assert torch.equal(out.double(), z)
        return
    n = z.shape[1] // 2
    gate, up = z[:, :n], z[:, n:]
    ref = gate / (1 + torch.exp(-gate)) * up
    assert ((out.double() - ref).abs() <= 8 * 2.0 ** -23 * ref.abs() + 1e-36 * (1 + up.abs())).all()


# tokens, choices, experts (0: dense rows), width of out, inputs.  The launch
# gives each workgroup 2 to 8 tile groups (1 where a form without gate has half
# as many), and where row blocks go in turn it has 170 places for 188 of them
# (gated 87), or 341 (178) for a bound of 362 that the dropped pairs leave
# unfilled.
PATHS = {
    "tile groups in turn": (64, 8, 128, 544, 1024),
    "eight tile groups in turn, the last tile ragged": (64, 8, 128, 1000, 256),
    "tile groups in turn, in passes": (640, 0, 0, 3300, 4224),
    "grouped rows in passes": (64, 8, 128, 400, 2560),
    "row blocks in turn": (3000, 0, 0, 6000, 640),
    "row blocks in turn, in passes": (3000, 0, 0, 6000, 4224),
    "row blocks in turn, fewer than their bound": (700, 4, 200, 2912, 256),
    "four steps held, the last wave's mostly past the inputs": (1040, 0, 0, 2048, 2176),
    "four steps held": (1040, 0, 0, 2048, 4096),
    "four steps held, grouped rows": (64, 8, 128, 1000, 2176),
}


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("kind", [32, 64, 128])
@pytest.mark.parametrize("path", PATHS)
def test_every_path_is_exact(path, kind, zeros, gated):
    T, k, E, width, K = PATHS[path]
    group = kind if kind < 128 else next(n for n in (1024, 512, 256, 128) if K % n == 0)
    xt = HF if kind == 64 else BF
    print(f"{path}: T={T} k={k} E={E} width={width} K={K} group={group} zeros={zeros} gated={gated} {xt}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + K + kind)
    codes, s, z = integers(g, max(E, 1), 2 * width if gated else width, K, group, zeros, xt)
    x = torch.randint(-2, 3, (T, K), generator=g, device="cuda").to(xt)
    if not E:
        out = torch.full((T, width + 1), 5.0, device="cuda")
        w4.linear(x, out[:, :width], codes[0], s[0], zeros=None if z is None else z[0], gated=gated)
        same(out[:, :width], product64(x, codes[0], s[0], None if z is None else z[0], group), gated)
        assert (out[:, width] == 5.0).all()
        return
    i32 = dict(dtype=torch.int32, device="cuda")
    bias = -torch.log(torch.arange(1, E + 1, device="cuda"))       # a few experts take many rows
    score = torch.rand(T, E, generator=g, device="cuda") * 4 + bias
    ids = torch.topk(score, k, dim=1).indices.to(torch.int32)
    ids[torch.rand(T, k, generator=g, device="cuda") < 0.2] = -1
    counts, offsets, perm, pos = (torch.zeros(n, **i32) for n in (E, E + 1, T * k, (T, k)))
    D.sort(ids, counts, offsets, perm, pos)
    out = torch.full((T * k, width + 1), 5.0, device="cuda")
    w4.experts(x, offsets, out[:, :width], codes, s, zeros=z, row_map=perm, map_div=k, gated=gated)
    o = offsets.tolist()
    assert max(b - a for a, b in zip(o, o[1:])) > 16
    for e in range(E):
        if o[e + 1] > o[e]:
            rows = slice(o[e], o[e + 1])
            xe = x[torch.div(perm[rows], k, rounding_mode="floor").long()]
            same(out[rows, :width], product64(xe, codes[e], s[e], None if z is None else z[e], group), gated)
    assert (out[o[E]:] == 5.0).all() and (out[:, width] == 5.0).all()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,N,K,group", [(2, 48, 4096, 128), (19, 40, 6144, 32), (17, 34, 6144, 1024), (4, 20, 8320, 64),
                                         (33, 33, 5120, 1024), (3, 50, 32768, 256)])
def test_long_rows_are_exact(T, N, K, group, zeros):
    """Rows that are taken in passes; K = 32768: sums below 60 K < 2^21, halves
    of them still within 24 bits."""
    print(f"long rows T={T} N={N} K={K} group={group} zeros={zeros}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    for xt in (BF, HF):
        codes, s, z = integers(g, 1, N, K, group, zeros, xt)
        x = torch.randint(-2, 3, (T, K), generator=g, device="cuda").to(xt)
        out = torch.empty(T, N, device="cuda")
        w4.linear(x, out, codes[0], s[0], zeros=None if z is None else z[0])
        same(out, product64(x, codes[0], s[0], None if z is None else z[0], group), False)
