"""The 8-bit products and gradients at sizes large enough for each tile shape,
with ragged edges, and the split gradient captured.  The bounds are those of
test_gpu_fp8.py."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import fp8
from test_gpu_fp8 import BF, F32, HF, block_val, check_product, random_codes, random_scales, row_val, segments

pytestmark = pytest.mark.gpu

# tiles of 64 x 128, 128 x 128, 128 x 256, 256 x 256 (fp32: 128 x 256)
DENSE = [(1000, 2000, 256), (1990, 2010, 256), (2300, 2100, 384), (4000, 4090, 256)]
GROUPED = [(2000, 2, 8, 1500, 256), (600, 2, 4, 1500, 256), (2000, 2, 8, 2500, 256), (4000, 2, 8, 1500, 256)]
# and of the gradients; the last two are split
GRADIENTS = [(300, 500, 700), (300, 2000, 2010), (300, 2300, 2100), (9000, 130, 257), (6000, 1500, 700)]


@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("ot", [BF, HF, F32])
@pytest.mark.parametrize("R,N,K", DENSE)
def test_linear_of_many_rows(R, N, K, ot, small):
    print(f"linear R={R} N={N} K={K} {ot} small={small}", flush=True)
    rng = np.random.default_rng(R)
    a, w = random_codes(rng, R, K, small=small), random_codes(rng, N, K, small=small)
    sa = random_scales(rng, K // 128, R, small=small)
    sw = random_scales(rng, fp8.padded(N) // 128, K // 128, small=small)
    out = torch.full((R, N + 3), 7.0, device="cuda", dtype=ot)
    fp8.linear(a, sa, w, sw, out[:, :N])
    check_product(out[:, :N], row_val(a, sa), block_val(w, sw), K // 128, small)
    assert (out[:, N:] == 7.0).all()


@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("T,k,E,N,K", GROUPED)
def test_experts_of_many_rows(T, k, E, N, K, ot, small):
    print(f"experts T={T} k={k} E={E} N={N} K={K} {ot} small={small}", flush=True)
    rng = np.random.default_rng(T + N)
    _, c, o, perm, _ = segments(rng, T, k, E, 128, 0.1, skew=False)
    rows = perm.numel()
    a, w = random_codes(rng, rows, K, small=small), random_codes(rng, E, N, K, small=small)
    sa = random_scales(rng, K // 128, rows, small=small)
    sw = random_scales(rng, E, fp8.padded(N) // 128, K // 128, small=small)
    out = torch.full((rows, N + 1), 5.0, device="cuda", dtype=ot)
    fp8.experts(a, sa, o, w, sw, out[:, :N], counts=c)
    stays = torch.ones(rows, dtype=torch.bool, device="cuda")
    for e, (first, many) in enumerate(zip(o.tolist(), c.tolist())):
        r = slice(first, first + many)
        stays[r] = False
        if many:
            check_product(out[r, :N], row_val(a[r], sa[:, r]), block_val(w[e], sw[e]), K // 128, small)
    assert (out[stays] == 5.0).all() and (out[:, N] == 5.0).all()


@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("R,N,K", GRADIENTS)
def test_weight_gradient_of_large_matrices(R, N, K, small):
    print(f"weight gradient R={R} N={N} K={K} small={small}", flush=True)
    rng = np.random.default_rng(N)
    Rp = fp8.padded(R)
    dy, x = random_codes(rng, N, Rp, small=small), random_codes(rng, K, Rp, small=small)
    sy, sx = random_scales(rng, Rp // 128, N, small=small), random_scales(rng, Rp // 128, K, small=small)
    dw = torch.full((N, K), 3.0, device="cuda")
    fp8.weight_gradient(dy, sy, x, sx, dw)
    check_product(dw, row_val(dy, sy), row_val(x, sx), Rp // 128, small)
    first = dw.clone()
    fp8.weight_gradient(dy, sy, x, sx, dw, add=True)
    assert torch.equal(dw, first + first)


def test_captured_split_gradients_replay_like_eager():
    """Two captured gradients share a workspace, as one stream's calls may."""
    print("captured split gradients", flush=True)
    N, K, R = 130, 257, 9000
    Rp, need = fp8.padded(R), fp8.weight_gradient_workspace_bytes(1, fp8.padded(R), N, K)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)

    def inputs():
        return (random_codes(rng, N, Rp), random_scales(rng, Rp // 128, N), random_codes(rng, K, Rp),
                random_scales(rng, Rp // 128, K))
    sets = [inputs() for _ in range(2)]
    out = [torch.zeros(N, K, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s, o in zip(sets, out):
            fp8.weight_gradient(*s, o, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for s, o in zip(sets, out):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fp8.weight_gradient(*s, o, ws=ws)
    for turn in range(3):
        for s in sets:
            for old, new in zip(s, inputs()):
                old.copy_(new)
        for o in out:
            o.fill_(-1.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, o in zip(sets, out):
            eager = torch.zeros(N, K, device="cuda")
            fp8.weight_gradient(*s, eager)
            torch.cuda.synchronize()
            assert torch.equal(o, eager), turn
