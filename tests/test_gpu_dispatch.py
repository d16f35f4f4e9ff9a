"""GPU parity of expert dispatch (sort, copy, combine, gradients) with the
float64 oracle.

Tolerances count roundings: u = 2^-24 is half a step of an fp32 sum or
product, half(t) half a step of the output type.  A sum of n terms of total
magnitude m, each term rounded once, is off by at most (n + 1) u m up to
second order (n u is below 1e-3 here, covered by the factor 1.01)."""

import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import dispatch as D
from oracle import dispatch as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SUB = {BF: 2.0 ** -134, HF: 2.0 ** -25, F32: 2.0 ** -150}       # half a step among the subnormals


def half(t):
    return torch.finfo(t).eps / 2


def np64(t):
    return t.double().cpu().numpy()


def make_ids(T, k, E, drop, seed):
    """Distinct experts per token (repeats only where k > E), a share of the
    pairs out of range on either side, some tokens dropped whole."""
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, max(E, k))), axis=1)[:, :k].astype(np.int64) % E
    if drop:
        out = np.array([-1, E, E + 7, -5, 2 ** 31 - 1, -2 ** 31], dtype=np.int64)
        ids = np.where(rng.random((T, k)) < drop, out[rng.integers(0, 6, (T, k))], ids)
        ids[T // 3:T // 3 + max(1, T // 9)] = -1
    return ids.astype(np.int32)


def run_sort(ids, E, align, extra=0, **kw):
    T, k = ids.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets = torch.full((E,), 77, **i32), torch.full((E + 1,), 77, **i32)
    perm = torch.full((D.sort_rows(T, k, E, align) + extra,), 77, **i32)
    pos = torch.full((T, k), 77, **i32)
    D.sort(torch.from_numpy(ids).cuda(), counts, offsets, perm, pos, align=align, **kw)
    return counts, offsets, perm, pos


SORTS = [(0, 1, 4, 1, 0.0), (1, 1, 1, 1, 0.0), (1, 8, 128, 1, 0.0), (64, 8, 128, 1, 0.0), (64, 8, 128, 128, 0.3),
         (65, 8, 100, 7, 0.1), (256, 8, 256, 16, 0.0), (257, 8, 256, 16, 0.5), (2048, 1, 1024, 3, 0.0),
         (2049, 1, 1, 1, 0.2), (5, 64, 1000, 2, 0.0), (33, 64, 7, 1, 0.0), (4099, 6, 60, 128, 0.1),
         (70001, 3, 300, 4, 0.05), (300, 5, 257, 1, 1.0)]


@pytest.mark.parametrize("T,k,E,align,drop", SORTS)
def test_sort_bit_exact(T, k, E, align, drop):
    print(f"sort T={T} k={k} E={E} align={align} drop={drop}", flush=True)
    ids = make_ids(T, k, E, drop, seed=T + E)
    got = run_sort(ids, E, align, extra=130)
    ref = O.sort_pairs(ids, E, align, got[2].numel())
    for g, r in zip(got, ref):
        assert np.array_equal(g.cpu().numpy(), r)


def test_sort_one_expert_takes_all():
    """Every pair on one expert: ranks run through every wave and block."""
    print("sort one expert", flush=True)
    ids = np.full((6000, 2), 5, dtype=np.int32)
    got = run_sort(ids, 9, 4)
    for g, r in zip(got, O.sort_pairs(ids, 9, 4, got[2].numel())):
        assert np.array_equal(g.cpu().numpy(), r)


def rows_tensor(rng, n, cols, dt, pad, shift, fill=None):
    """[n, cols] view of a wider buffer: `pad` spare columns, starting
    `shift` values into it."""
    buf = torch.from_numpy(rng.standard_normal((n, cols + pad + shift)).astype(np.float32)).to(dt)
    if fill is not None:
        buf[:] = fill
    return buf.cuda()[:, shift:shift + cols]


SHAPES = [(1, 8, 128, 2048, 1, 0.0, 0, 0), (5, 2, 3, 1, 4, 0.2, 0, 0), (37, 3, 10, 7, 16, 0.2, 0, 0),
          (64, 8, 128, 1001, 1, 0.1, 0, 0), (100, 8, 60, 6144, 16, 0.5, 0, 0), (33, 1, 256, 100, 1, 0.0, 4, 0),
          (50, 6, 16, 264, 8, 0.3, 8, 0), (50, 6, 16, 264, 8, 0.3, 7, 1), (7, 64, 9, 520, 1, 0.1, 0, 0),
          (9, 11, 64, 1536, 2, 0.2, 16, 8), (0, 4, 8, 64, 1, 0.0, 0, 0), (12, 4, 8, 136, 32, 1.0, 0, 0)]


def plan(T, k, E, align, drop, seed, extra=3):
    ids = make_ids(T, k, E, drop, seed)
    c, o, perm, pos = run_sort(ids, E, align, extra=extra)
    return ids, perm, pos


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("T,k,E,cols,align,drop,pad,shift", SHAPES)
def test_permute(T, k, E, cols, align, drop, pad, shift, dt):
    print(f"permute T={T} k={k} E={E} cols={cols} align={align} {dt}", flush=True)
    rng = np.random.default_rng(cols)
    ids, perm, pos = plan(T, k, E, align, drop, 1)
    x = rows_tensor(rng, T, cols, dt, pad, shift)
    dropped = ((ids < 0) | (ids >= E)).all(1)
    x[torch.from_numpy(dropped).cuda()] = float("nan")            # never copied
    out = rows_tensor(rng, perm.numel(), cols, dt, pad, shift)
    before = np64(out)
    D.permute(x, perm, pos, out)
    assert np.array_equal(np64(out), O.permute(np64(x), perm.cpu().numpy(), pos.cpu().numpy(), before))


PAIRS = [(BF, BF), (HF, HF), (F32, F32), (BF, F32), (HF, F32), (F32, BF), (F32, HF)]


def poisoned_rows(rng, perm, cols, dt, pad, shift):
    """Grouped rows whose padding and unused rows hold NaN and infinities."""
    y = rows_tensor(rng, perm.numel(), cols, dt, pad, shift)
    y[perm == -1] = float("nan")
    y[perm == -2] = float("inf")
    return y


@pytest.mark.parametrize("yt,ot", PAIRS)
@pytest.mark.parametrize("T,k,E,cols,align,drop,pad,shift", SHAPES)
@pytest.mark.parametrize("mode", ["w", "base", "ones"])
def test_unpermute(T, k, E, cols, align, drop, pad, shift, yt, ot, mode):
    print(f"unpermute T={T} k={k} E={E} cols={cols} align={align} {yt} {ot} {mode}", flush=True)
    rng = np.random.default_rng(cols + 1)
    ids, perm, pos = plan(T, k, E, align, drop, 2)
    y = poisoned_rows(rng, perm, cols, yt, pad, shift)
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda() if mode != "ones" else None
    base = rows_tensor(rng, T, cols, F32, pad, shift) if mode == "base" else None
    out = rows_tensor(rng, T, cols, ot, pad, shift, fill=3.0)
    if mode == "ones":
        D.permute_backward(y, pos, out)
    else:
        D.unpermute(y, pos, w, out, base=base)
    ref, mag = O.unpermute(np64(y), pos.cpu().numpy(), None if w is None else np64(w),
                           None if base is None else np64(base), cols)
    err = np.abs(np64(out) - ref)
    assert (err <= 1.01 * (k + 1) * U * mag + half(ot) * np.abs(ref) * 1.01 + SUB[ot]).all(), err.max()


def test_unpermute_base_in_place():
    """base may be out itself (fp32): partial sums added up over calls."""
    print("unpermute in place", flush=True)
    rng = np.random.default_rng(5)
    ids, perm, pos = plan(40, 4, 16, 8, 0.2, 3)
    y = poisoned_rows(rng, perm, 512, BF, 0, 0)
    w = torch.from_numpy(rng.random((40, 4)).astype(np.float32)).cuda()
    a = torch.randn(40, 512, device="cuda")
    b = torch.empty_like(a)
    D.unpermute(y, pos, w, b, base=a)
    D.unpermute(y, pos, w, a, base=a)
    assert torch.equal(a, b)


@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("cols", [5, 9, 12, 513, 4100])
def test_base_in_place_of_odd_widths(cols, yt):
    """Units that overlap would add a value's rows twice."""
    print(f"in place cols={cols} {yt}", flush=True)
    rng = np.random.default_rng(cols)
    ids, perm, pos = plan(21, 3, 7, 4, 0.2, 4)
    y = poisoned_rows(rng, perm, cols, yt, 1, 0)
    w = torch.from_numpy(rng.random((21, 3)).astype(np.float32)).cuda()
    a = torch.randn(21, cols + 3, device="cuda")[:, :cols]
    b = torch.empty(21, cols, device="cuda")
    D.unpermute(y, pos, w, b, base=a)
    D.unpermute(y, pos, w, a, base=a)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [BF, F32])
def test_no_tokens_still_clear_padding(dt):
    print(f"no tokens {dt}", flush=True)
    perm = torch.tensor([-1, -2, -1] + [-2] * 40 + [-1], dtype=torch.int32, device="cuda")
    pos, w = torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 2, device="cuda")
    x, want = torch.zeros(0, 67, device="cuda", dtype=dt), torch.full((44, 67), 5.0, device="cuda", dtype=dt)
    out, y = want.clone(), want.clone()
    want[perm == -1] = 0
    D.permute(x, perm, pos, out)
    assert torch.equal(out, want)
    dy = torch.full_like(want, 5.0)
    D.unpermute_backward(x, y, perm, pos, w, dy, w.clone())
    assert torch.equal(dy, want)


def test_offsets_past_32_bits():
    """Rows 2^30 values apart, in each role."""
    print("rows far apart", flush=True)
    cols, far = 264, 2 ** 30
    ids, perm, pos = plan(5, 1, 3, 1, 0.0, 5, extra=0)
    wide = [torch.empty(5, far, device="cuda", dtype=BF)[:, 8:8 + cols] for _ in range(3)]
    x, xs, dy = wide
    x.copy_(torch.randn(5, cols, device="cuda"))
    D.permute(x, perm, pos, xs)
    near, nxs = x.contiguous(), torch.zeros(5, cols, device="cuda", dtype=BF)
    D.permute(near, perm, pos, nxs)
    assert torch.equal(xs, nxs) and torch.equal(nxs[pos[:, 0].long()], near)
    w = torch.rand(5, 1, device="cuda")
    ndy, dw, ndw = torch.zeros_like(nxs), torch.zeros(5, 1, device="cuda"), torch.zeros(5, 1, device="cuda")
    D.unpermute_backward(x, xs, perm, pos, w, dy, dw)
    D.unpermute_backward(near, nxs, perm, pos, w, ndy, ndw)
    assert torch.equal(dy, ndy) and torch.equal(dw, ndw)
    out = torch.zeros(5, cols, device="cuda", dtype=BF)
    D.unpermute(xs, pos, w, x)
    D.unpermute(nxs, pos, w, out)
    assert torch.equal(x, out)


@pytest.mark.parametrize("yt,ot", PAIRS)
@pytest.mark.parametrize("T,k,E,cols,align,drop,pad,shift", SHAPES)
def test_unpermute_backward(T, k, E, cols, align, drop, pad, shift, yt, ot):
    print(f"unpermute_backward T={T} k={k} E={E} cols={cols} align={align} {yt} {ot}", flush=True)
    rng = np.random.default_rng(cols + 2)
    ids, perm, pos = plan(T, k, E, align, drop, 4)
    y = poisoned_rows(rng, perm, cols, yt, pad, shift)
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    dout = rows_tensor(rng, T, cols, ot, pad, shift)
    dy = rows_tensor(rng, perm.numel(), cols, yt, pad, shift)
    dw = torch.full((T, k), 9.0, device="cuda")
    before = np64(dy)
    D.unpermute_backward(dout, y, perm, pos, w, dy, dw)
    rdy, rdw, mag = O.unpermute_backward(np64(dout), np64(y), perm.cpu().numpy(), pos.cpu().numpy(), np64(w), before)
    # a product rounded to fp32, then to the type
    assert (np.abs(np64(dy) - rdy) <= 1.01 * (half(yt) + U) * np.abs(rdy) + SUB[yt]).all()
    assert (np.abs(np64(dw) - rdw) <= 1.01 * (cols + 1) * U * mag + SUB[F32]).all()


@pytest.mark.parametrize("T,k,E", [(0, 2, 8), (1, 1, 1), (1, 8, 128), (37, 3, 65), (64, 8, 256), (301, 64, 1000)])
def test_gate_backward(T, k, E):
    print(f"gate_backward T={T} k={k} E={E}", flush=True)
    rng = np.random.default_rng(E)
    ids = make_ids(T, k, E, 0.2 if T > 30 else 0.0, 6)
    if T > 30:
        ids[5, :2] = 3                                            # the same expert twice
    w = rng.random((T, k)).astype(np.float32)
    w /= np.maximum(w.sum(1, keepdims=True), 1e-6)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dz = torch.full((T, E + 5), 4.0, device="cuda")
    D.gate_backward(torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(dw).cuda(), dz[:, :E])
    ref, mag = O.gate_backward(ids, w.astype(np.float64), dw.astype(np.float64), E)
    # inner sum: k products and sums; then one difference, one product, k sums
    assert (np.abs(np64(dz[:, :E]) - ref) <= 1.01 * (2 * k + 4) * U * mag + SUB[F32]).all()
    assert (dz[:, E:] == 4.0).all()


def test_gate_backward_against_differences():
    """Central differences of <dw, softmax of the chosen logits> in float64:
    off by h^2/6 times a third derivative of at most 6 |dw| plus 2^-52/h, so
    below 1e-8 |dw| at h = 1e-5 (dw is around one, four choices)."""
    print("gate differences", flush=True)
    rng = np.random.default_rng(8)
    T, k, E, h = 6, 4, 12, 1e-5
    z = rng.standard_normal((T, E))
    ids = make_ids(T, k, E, 0.0, 9)
    dw = rng.standard_normal((T, k)).astype(np.float32)

    def soft(z):
        s = np.take_along_axis(z, ids.astype(np.int64), 1)
        s = np.exp(s - s.max(1, keepdims=True))
        return s / s.sum(1, keepdims=True)
    num = np.zeros((T, E))
    for e in range(E):
        d = np.zeros((T, E))
        d[:, e] = h
        num[:, e] = ((soft(z + d) - soft(z - d)) * dw).sum(1) / (2 * h)
    dz = torch.empty(T, E, device="cuda")
    D.gate_backward(torch.from_numpy(ids).cuda(), torch.from_numpy(soft(z).astype(np.float32)).cuda(),
                    torch.from_numpy(dw).cuda(), dz)
    # w rounded to fp32 adds a rounding of each of the formula's terms
    _, mag = O.gate_backward(ids, soft(z), dw.astype(np.float64), E)
    assert (np.abs(np64(dz) - num) <= 1.01 * (4 * k + 8) * U * mag + 1e-8 * np.abs(dw).sum()).all()


def test_step_against_differences():
    """The combine is linear in y and in w, so a difference over a whole
    step is its gradient's inner product, up to the roundings of the two
    forward values."""
    print("combine differences", flush=True)
    rng = np.random.default_rng(10)
    T, k, cols = 30, 3, 200
    ids, perm, pos = plan(T, k, 12, 4, 0.2, 11)
    y = poisoned_rows(rng, perm, cols, F32, 0, 0)
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    dout = torch.from_numpy(rng.standard_normal((T, cols)).astype(np.float32)).cuda()
    live = perm >= 0
    step_y = torch.where(live[:, None], torch.randn(y.shape, device="cuda"), torch.zeros((), device="cuda"))
    step_w = torch.randn(T, k, device="cuda")
    dy, dw = torch.zeros_like(y), torch.zeros(T, k, device="cuda")
    D.unpermute_backward(dout, y, perm, pos, w, dy, dw)

    def loss(y, w):
        out = torch.empty(T, cols, device="cuda")
        D.unpermute(y, pos, w, out)
        _, mag = O.unpermute(np64(y), pos.cpu().numpy(), np64(w), None, cols)
        return (np64(out) * np64(dout)).sum(), 1.01 * (k + 2) * U * (mag * np.abs(np64(dout))).sum()
    l0, e0 = loss(y, w)
    for y1, w1, grad, step in ((y + step_y, w, dy, step_y), (y, w + step_w, dw, step_w)):
        l1, e1 = loss(y1, w1)
        real = np64(y1)[live.cpu().numpy()] - np64(y)[live.cpu().numpy()] if grad is dy else np64(w1) - np64(w)
        g = np64(grad)[live.cpu().numpy()] if grad is dy else np64(grad)
        kept = (g != 0)
        want = (g * np.where(kept, real, 0)).sum()
        slack = e0 + e1 + (cols + 2) * U * (np.abs(g * np.where(kept, real, 0))).sum() * 4 + \
            (cols + 2) * U * k * np.abs(np64(dout)).sum() * np.abs(real).max() * np.nanmax(np.abs(np64(y)[live.cpu().numpy()]))
        assert abs((l1 - l0) - want) <= slack


def test_captured_step_replays_like_eager():
    """sort, copy, combine and the gradients captured once; replayed on new
    inputs with eager work between, every replay equal to the eager calls."""
    print("captured dispatch", flush=True)
    T, k, E, cols, align = 400, 8, 64, 256, 16                   # 3200 pairs: the multi-block sort
    rows = D.sort_rows(T, k, E, align)

    def buffers():
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(ids=torch.zeros(T, k, **i32), counts=torch.zeros(E, **i32), offsets=torch.zeros(E + 1, **i32),
                    perm=torch.zeros(rows, **i32), pos=torch.zeros(T, k, **i32),
                    ws=torch.empty(D.sort_workspace_bytes(T, k, E), dtype=torch.uint8, device="cuda"),
                    x=torch.zeros(T, cols, device="cuda", dtype=BF), xs=torch.zeros(rows, cols, device="cuda", dtype=BF),
                    w=torch.zeros(T, k, device="cuda"), out=torch.zeros(T, cols, device="cuda", dtype=BF),
                    dy=torch.zeros(rows, cols, device="cuda", dtype=BF), dw=torch.zeros(T, k, device="cuda"),
                    dx=torch.zeros(T, cols, device="cuda", dtype=BF), dz=torch.zeros(T, E, device="cuda"))

    def step(b):
        D.sort(b["ids"], b["counts"], b["offsets"], b["perm"], b["pos"], align=align, ws=b["ws"])
        D.permute(b["x"], b["perm"], b["pos"], b["xs"])
        D.unpermute(b["xs"], b["pos"], b["w"], b["out"])
        D.unpermute_backward(b["out"], b["xs"], b["perm"], b["pos"], b["w"], b["dy"], b["dw"])
        D.permute_backward(b["dy"], b["pos"], b["dx"])
        D.gate_backward(b["ids"], b["w"], b["dw"], b["dz"])
    cap, eager = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for seed in range(4):
        ids = torch.from_numpy(make_ids(T, k, E, 0.1, seed)).cuda()
        x = torch.randn(T, cols, device="cuda").to(BF)
        w = torch.rand(T, k, device="cuda")
        for b in (cap, eager):
            b["ids"].copy_(ids)
            b["x"].copy_(x)
            b["w"].copy_(w)
            b["xs"].zero_()
            b["dy"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        for n in ("counts", "offsets", "perm", "pos", "xs", "out", "dy", "dw", "dx", "dz"):
            assert torch.equal(cap[n], eager[n]), (seed, n)


def test_two_streams():
    """Two sorts and copies at once on two streams, each with its own buffers."""
    print("two streams", flush=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    todo = []
    for i in range(2):
        ids = make_ids(3000 + i, 4, 50, 0.1, i)
        d = torch.from_numpy(ids).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        rows = D.sort_rows(*ids.shape, 50)
        todo.append((ids, d, torch.zeros(50, **i32), torch.zeros(51, **i32), torch.zeros(rows, **i32),
                     torch.zeros(ids.shape, **i32), torch.randn(len(ids), 96, device="cuda").to(BF),
                     torch.zeros(rows, 96, device="cuda", dtype=BF)))
    torch.cuda.synchronize()
    for s, (ids, d, c, o, perm, pos, x, xs) in zip(streams, todo):
        D.sort(d, c, o, perm, pos, stream=s)
        D.permute(x, perm, pos, xs, stream=s)
    torch.cuda.synchronize()
    for ids, d, c, o, perm, pos, x, xs in todo:
        ref = O.sort_pairs(ids, 50, 1, perm.numel())
        for g, r in zip((c, o, perm, pos), ref):
            assert np.array_equal(g.cpu().numpy(), r)
        assert np.array_equal(np64(xs), O.permute(np64(x), ref[2], ref[3], np.zeros(xs.shape)))
