"""GPU tests of the dispatch and 4-bit operators at the limits of what they
accept, against the float64 oracle."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import binding as B
from expert_ffn_execution_router_amd import dispatch as D
from oracle import dispatch as O

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


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
