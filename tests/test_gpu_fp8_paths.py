"""The products per expert on the paths that sizes choose: few rows read straight
into registers, 16, 32 and 64 to a workgroup, where segments are looked up on the
device (also past 64 experts), and the tiles of every shape that experts of many
rows take, with whole tiles, stages used in turn and stores left outstanding.
The bounds are those of test_gpu_fp8.py."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import fp8
from test_gpu_fp8 import BF, F32, HF, block_val, check_product, random_codes, random_scales, row_val

pytestmark = pytest.mark.gpu


def run(counts, gap, N, K, ot, small, with_counts=True):
    """Segments of counts rows with gap rows behind each; all rows checked."""
    rng = np.random.default_rng(N + K + len(counts))
    E, held = len(counts), [c + gap for c in counts]
    R = sum(held) + 3
    o = torch.tensor(np.cumsum([0, *held]), dtype=torch.int32, device="cuda")
    many = torch.tensor(counts, dtype=torch.int32, device="cuda")
    a, w = random_codes(rng, R, K, small=small), random_codes(rng, E, N, K, small=small)
    sa = random_scales(rng, K // 128, R, small=small)
    sw = random_scales(rng, E, fp8.padded(N) // 128, K // 128, small=small)
    out = torch.full((R, N + 3), 5.0, device="cuda", dtype=ot)
    fp8.experts(a, sa, o, w, sw, out[:, :N], counts=many if with_counts else None)
    again = torch.full((R, N + 3), 5.0, device="cuda", dtype=ot)
    fp8.experts(a, sa, o, w, sw, again[:, :N], counts=many if with_counts else None)
    stays = torch.ones(R, dtype=torch.bool, device="cuda")
    first = o.tolist()
    for e in range(E):
        r = slice(first[e], first[e] + counts[e] if with_counts else first[e + 1])
        stays[r] = False
        if r.stop > r.start:
            check_product(out[r, :N], row_val(a[r], sa[:, r]), block_val(w[e], sw[e]), K // 128, small)
    assert (out[stays] == 5.0).all() and (out[:, N:] == 5.0).all() and torch.equal(out, again)


# rows to a workgroup: 16, 16 past 64 experts, 32, 64, and 16 with rows between the segments
FEW = [((1, 0, 3, 2), 0, 300, 1024), ((1,) * 40 + (0,) * 30 + (2, 1, 17), 0, 36, 1024), ((45, 19), 0, 900, 1024),
       ((80, 0, 70), 0, 1024, 2048), ((5, 12, 0, 1), 2, 130, 768), ((9,), 0, 40, 4096)]


@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("ot", [BF, HF, F32])
@pytest.mark.parametrize("counts,gap,N,K", FEW)
def test_experts_of_few_rows(counts, gap, N, K, ot, small):
    print(f"few rows {counts} gap={gap} N={N} K={K} {ot} small={small}", flush=True)
    run(counts, gap, N, K, ot, small)
    run(counts, gap, N, K, ot, small, with_counts=False)


# the tiles of bf16 and of fp32 results: 64 x 128, 128 x 128, 128 x 256 (whole columns, then a ragged edge), 256 x
# 256 and 128 x 128, 256 x 256 and 128 x 256
MANY = [((150, 40, 300, 200, 90), 0, 1500, 1024), ((350, 200, 0, 513, 128), 0, 2500, 1024),
        ((512, 700, 384, 256, 0, 1024, 513, 300, 900), 0, 1536, 1024),
        ((512, 512, 130, 640, 640, 640, 512, 512, 500), 0, 1400, 768), ((1500, 0, 2100, 1700, 1300), 0, 1400, 1024),
        ((1500, 2100, 1700, 1300), 0, 2048, 768)]


@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("counts,gap,N,K", MANY)
def test_experts_of_many_rows(counts, gap, N, K, ot, small):
    print(f"many rows {counts} N={N} K={K} {ot} small={small}", flush=True)
    run(counts, gap, N, K, ot, small)


def test_captured_experts_of_few_rows_replay_like_eager():
    """Counts change between replays."""
    print("captured few rows", flush=True)
    rng = np.random.default_rng(4)
    E, R, N, K = 6, 40, 300, 1024
    a, sa = random_codes(rng, R, K), random_scales(rng, K // 128, R)
    w, sw = random_codes(rng, E, N, K), random_scales(rng, E, 3, K // 128)
    o, c = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
    out = torch.zeros(R, N, device="cuda", dtype=BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8.experts(a, sa, o, w, sw, out, counts=c)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.experts(a, sa, o, w, sw, out, counts=c)
    for counts in ([1, 0, 5, 20, 3, 2], [0] * 6, [40, 0, 0, 0, 0, 0], [6, 6, 6, 6, 6, 6]):
        c.copy_(torch.tensor(counts, dtype=torch.int32))
        o.copy_(torch.tensor(np.cumsum([0, *counts]), dtype=torch.int32))
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.full_like(out, 3.0)
        fp8.experts(a, sa, o, w, sw, eager, counts=c)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), counts
        assert (out[sum(counts):] == 3.0).all()
