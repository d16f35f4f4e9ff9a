"""CPU tests of what the dispatch and 4-bit operators refuse at their limits:
sizes past 32 bits, memory shared with an output, inputs that want a graph.
Every refusal is made on the host, before any device work."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from expert_ffn_execution_router_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from expert_ffn_execution_router_amd.build import build
        build()
    return binding


P = 4096          # stands for a device pointer: refused calls never use it
CUT = 2 ** 32     # added to a size, leaves its low 32 bits as they were


def test_sizes_are_not_cut_to_32_bits(B):
    """A size whose low 32 bits are a valid one is refused."""
    for i in range(4):
        a = [4, 2, 8, 1]
        a[i] += CUT
        assert B.moe_sort_rows(*a) == -1, a
        assert i == 3 or B.moe_sort_workspace_bytes(*a[:3]) == 0, a
    assert B.moe_sort_rows(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) > 0

    def sort(T=0, k=2, E=8, align=1, rows=32):
        return B.moe_sort(P, T, k, E, align, P, P, P, rows, P, None, 0, None)
    assert sort(T=CUT) == B.MOE_E_UNSUPPORTED
    assert sort(T=2 ** 62, k=4) == B.MOE_E_UNSUPPORTED
    assert sort(k=CUT + 2) == sort(E=CUT + 8) == sort(align=CUT + 1) == B.MOE_E_INVAL

    def permute(T=0, k=2, rows=8, cols=64):
        return B.moe_permute(0, P, CUT * 2, None, P, T, k, rows, cols, P, CUT * 2, None)
    assert permute() == 0                                                  # nothing to do
    assert permute(cols=CUT + 64) == permute(T=CUT) == B.MOE_E_UNSUPPORTED
    assert permute(k=CUT + 2) == permute(rows=CUT) == B.MOE_E_INVAL

    def unpermute(T=0, k=2, cols=64):
        return B.moe_unpermute(0, P, CUT * 2, 8, P, P, None, 0, T, k, cols, 0, P, CUT * 2, None)
    assert unpermute() == 0
    assert unpermute(cols=CUT + 64) == unpermute(T=CUT) == B.MOE_E_UNSUPPORTED
    assert unpermute(k=CUT + 2) == B.MOE_E_INVAL

    def backward(T=0, k=2, cols=64):
        return B.moe_unpermute_backward(0, P, CUT * 2, 0, P, CUT * 2, None, 8, P, P, T, k, cols, P, CUT * 2, P, None)
    assert backward() == 0
    assert backward(cols=CUT + 64) == backward(T=CUT) == B.MOE_E_UNSUPPORTED
    assert backward(k=CUT + 2) == B.MOE_E_INVAL

    def gate(T=0, k=2, E=8):
        return B.moe_gate_backward(P, P, P, T, k, E, P, CUT * 2, None)
    assert gate() == 0
    assert gate(T=CUT) == gate(E=CUT + 8) == B.MOE_E_UNSUPPORTED
    assert gate(k=CUT + 2) == B.MOE_E_INVAL

    def mm(E=1, N=32, K=256, group=128, md=1, off=None):
        return B.moe_w4_matmul(0, P, CUT * 2, 4, P, md, off, None, E, 0, P, 0, P, None, N, K, group, 0, 0, P, CUT * 2,
                               None)
    assert mm() == 0
    assert mm(N=CUT + 32) == mm(K=CUT + 256) == B.MOE_E_UNSUPPORTED
    assert mm(N=2 ** 62) == B.MOE_E_UNSUPPORTED
    assert mm(E=CUT + 1) == mm(E=CUT + 8, off=P) == mm(group=CUT + 128) == mm(md=CUT + 1) == B.MOE_E_INVAL


@pytest.mark.parametrize("over", [2 ** 31, CUT, CUT + 1, 2 ** 64 + 1])
def test_torch_layer_sizes_are_not_cut(B, over):
    from expert_ffn_execution_router_amd import dispatch as D
    from expert_ffn_execution_router_amd import w4
    for i in range(4):
        a = [4, 2, 8, 1]
        a[i] = over
        with pytest.raises(ValueError, match="2\\^31"):
            D.sort_rows(*a)
        if i < 3:
            with pytest.raises(ValueError, match="2\\^31"):
                D.sort_workspace_bytes(*a[:3])
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="align"):
        D.sort(torch.zeros(4, 2, **i32), torch.zeros(8, **i32), torch.zeros(9, **i32), torch.zeros(8, **i32),
               torch.zeros(4, 2, **i32), align=over)
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="map_div"):
        w4.experts(torch.zeros(4, 64, **bf), torch.zeros(2, **i32), torch.zeros(4, 16, **bf),
                   torch.zeros(1, 16, 32, dtype=torch.uint8), torch.zeros(1, 16, 2, **bf),
                   row_map=torch.zeros(4, **i32), map_div=over)
