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


# addresses a megabyte apart: arrays of these calls that start there are apart
A = [(i + 1) << 20 for i in range(8)]


def check_shared(B, call, outputs, inputs, sizes):
    """call refuses each output that begins at, or one byte before the end
    of, an input or another output; sizes: bytes of each."""
    for o in outputs:
        for other in inputs + outputs:
            if other == o:
                continue
            at = call.__kwdefaults__[other]
            for p in (at, at + sizes[other] - 1, at - sizes[o] + 1):
                assert call(**{o: p}) == B.MOE_E_INVAL, (o, other, p)
                assert "shares memory" in B.last_error(), (o, other, p)


def test_shared_memory_is_refused(B):
    """A written tensor that meets a read one would be read half old, half
    new; one that meets another written one would hold neither."""
    def sort(*, ids=A[0], counts=A[1], offsets=A[2], perm=A[3], pos=A[4], ws=A[5]):
        return B.moe_sort(ids, 1500, 2, 8, 1, counts, offsets, perm, 3000, pos, ws, 4096, None)
    need = B.moe_sort_workspace_bytes(1500, 2, 8)
    check_shared(B, sort, ["counts", "offsets", "perm", "pos"], ["ids", "ws"],
                 dict(ids=12000, counts=32, offsets=36, perm=12000, pos=12000, ws=need))

    def permute(*, x=A[0], perm=A[1], pos=A[2], out=A[3]):
        return B.moe_permute(0, x, 64, perm, pos, 4, 2, 8, 64, out, 64, None)
    check_shared(B, permute, ["out"], ["x", "perm", "pos"], dict(x=512, perm=32, pos=32, out=1024))

    def unpermute(*, y=A[0], pos=A[1], w=A[2], base=A[3], out=A[4]):
        return B.moe_unpermute(0, y, 64, 8, pos, w, base, 64, 4, 2, 64, 0, out, 64, None)
    check_shared(B, unpermute, ["out"], ["y", "pos", "w"], dict(y=1024, pos=32, w=32, base=1024, out=512))
    assert unpermute(out=A[3] + 2) == unpermute(out=A[3] - 2) == B.MOE_E_INVAL

    def no_rows(*, base=A[3], out=A[4]):
        return B.moe_unpermute(2, None, 64, 0, A[0], None, base, 64, 4, 2, 64, 2, out, 64, None)
    assert no_rows(out=A[3] + 4) == no_rows(base=A[4] + 4) == B.MOE_E_INVAL

    def backward(*, dout=A[0], y=A[1], perm=A[2], pos=A[3], w=A[4], dy=A[5], dw=A[6]):
        return B.moe_unpermute_backward(0, dout, 64, 0, y, 64, perm, 8, pos, w, 4, 2, 64, dy, 64, dw, None)
    check_shared(B, backward, ["dy", "dw"], ["dout", "y", "perm", "pos", "w"],
                 dict(dout=512, y=1024, perm=32, pos=32, w=32, dy=1024, dw=32))

    def gate(*, ids=A[0], w=A[1], dw=A[2], dz=A[3]):
        return B.moe_gate_backward(ids, w, dw, 4, 2, 8, dz, 8, None)
    check_shared(B, gate, ["dz"], ["ids", "w", "dw"], dict(ids=32, w=32, dw=32, dz=128))

    def mm(*, x=A[0], row_map=A[1], offsets=A[2], counts=A[3], codes=A[4], scales=A[5], zeros=A[6], out=A[7]):
        return B.moe_w4_matmul(0, x, 256, 4, row_map, 1, offsets, counts, 2, 4, codes, 0, scales, zeros, 32, 256, 128,
                               0, 0, out, 32, None)
    check_shared(B, mm, ["out"], ["x", "row_map", "offsets", "counts", "codes", "scales", "zeros"],
                 dict(x=2048, row_map=16, offsets=12, counts=8, codes=8192, scales=256, zeros=256, out=256))


def test_rows_that_cross_are_refused(B):
    """Rows of one buffer: columns that meet, and rows of different strides."""
    def permute(x, ldx, out, ldo, rows=8):
        return B.moe_permute(0, x, ldx, None, A[6], 4, 2, rows, 64, out, ldo, None)
    base = A[0]
    assert permute(base, 256, base + 2 * 63, 256) == B.MOE_E_INVAL         # the last column
    assert permute(base, 256, base + 2 * (256 - 63), 256) == B.MOE_E_INVAL  # the first column of the next row
    assert permute(base + 2 * 63, 256, base, 256) == B.MOE_E_INVAL
    assert permute(base, 256, base + 128, 264) == B.MOE_E_INVAL            # other strides: whole ranges
    assert permute(base, 2 ** 60, base + 2 ** 62, 64) == B.MOE_E_INVAL     # no wrap in 64 bits
    assert permute(base, 256, base + 2 * 63, 64, rows=1) == B.MOE_E_INVAL  # one row, across two


def test_workspace_off_its_alignment_is_refused(B):
    """The workspace is any bytes to the caller and ints to the kernels."""
    for off in (1, 2, 3):
        assert B.moe_sort(A[0], 1500, 2, 8, 1, A[1], A[2], A[3], 3000, A[4], A[5] + off, 4096, None) == B.MOE_E_INVAL
        assert "4 bytes" in B.last_error()


def test_tensors_that_want_a_graph_are_refused(B):
    """Results are written past autograd, so a tensor that requires grad would
    lose its gradient without a word; without gradients it is a plain tensor
    (here refused last, for being on the CPU)."""
    from expert_ffn_execution_router_amd import dispatch as D
    from expert_ffn_execution_router_amd import w4
    perm, pos, ids = (torch.zeros(s, dtype=torch.int32) for s in (8, (4, 2), (4, 2)))
    bf = dict(dtype=torch.bfloat16)
    t = dict(x=torch.zeros(4, 64, **bf), xs=torch.zeros(8, 64, **bf), w=torch.zeros(4, 2), base=torch.zeros(4, 64),
             out=torch.zeros(4, 64, **bf), dy=torch.zeros(8, 64, **bf), dw=torch.zeros(4, 2), dz=torch.zeros(4, 8),
             scales=torch.zeros(16, 2, **bf), zeros=torch.zeros(16, 2, **bf), z=torch.zeros(4, 16, **bf))
    codes, eo = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    calls = [("x xs", lambda v: D.permute(v["x"], perm, pos, v["xs"])),
             ("xs w out base", lambda v: D.unpermute(v["xs"], pos, v["w"], v["out"], base=v["base"])),
             ("xs out", lambda v: D.permute_backward(v["xs"], pos, v["out"])),
             ("out xs w dy dw", lambda v: D.unpermute_backward(v["out"], v["xs"], perm, pos, v["w"], v["dy"], v["dw"])),
             ("w dw dz", lambda v: D.gate_backward(ids, v["w"], v["dw"], v["dz"])),
             ("x scales zeros z", lambda v: w4.linear(v["x"], v["z"], codes, v["scales"], zeros=v["zeros"])),
             ("x scales zeros z", lambda v: w4.experts(v["x"], eo, v["z"], codes[None], v["scales"][None],
                                                       zeros=v["zeros"][None]))]
    for names, call in calls:
        for n in names.split():
            v = dict(t, **{n: t[n].clone().requires_grad_()})
            with pytest.raises(ValueError, match="requires grad"):
                call(v)
            with torch.no_grad(), pytest.raises(ValueError, match="on the GPU"):
                call(v)

    class Copy(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            D.permute(x, perm, pos, t["xs"])

    with pytest.raises(ValueError, match="on the GPU"):
        Copy.apply(t["x"].clone().requires_grad_())


def test_fewest_groups(B):
    """Only groups of 32 are too few by themselves (no rows: nothing runs)."""
    def mm(N, K, group, E=1):
        return B.moe_w4_matmul(0, P, K, 4, None, 1, P if E > 1 else None, None, E, 0, P, 0, P, None, N, K, group, 0, 0,
                               P, N, None)
    for shape in ((1, 128, 64), (1, 192, 64), (1, 256, 128), (1, 384, 128), (1, 512, 256), (1, 128, 32), (2, 64, 32),
                  (1, 32, 32), (1, 64, 32, 2)):
        assert mm(*shape) == 0, shape
    assert mm(1, 64, 32) == mm(1, 96, 32) == B.MOE_E_UNSUPPORTED
