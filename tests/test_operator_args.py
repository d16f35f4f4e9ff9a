"""CPU tests of the dispatch and 4-bit operators: every refusal of the C ABI
happens before device work (no GPU here), the torch layer refuses wrong
types, shapes, strides and overlaps, and the sizes are as documented.  Also
pins the oracles on worked examples."""
import os

import numpy as np
import pytest
import torch

from oracle import dispatch as OD
from oracle import w4 as OW


@pytest.fixture(scope="module")
def B():
    from expert_ffn_execution_router_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from expert_ffn_execution_router_amd.build import build
        build()
    return binding


P = 4096          # stands for a device pointer: refused calls never use it


def test_sizes(B):
    assert B.moe_sort_rows(64, 8, 128, 1) == 512
    assert B.moe_sort_rows(64, 8, 128, 16) == 512 + 128 * 15
    assert B.moe_sort_rows(1, 8, 128, 16) == 8 + 8 * 15
    assert B.moe_sort_rows(0, 8, 128, 16) == 0
    assert B.moe_sort_rows(2 ** 30, 64, 4, 2) == 2 ** 36 + 4
    assert B.moe_sort_rows(-1, 8, 128, 16) == -1 and B.moe_sort_rows(1, 8, 128, 0) == -1
    assert B.moe_sort_workspace_bytes(256, 8, 128) == 0
    assert B.moe_sort_workspace_bytes(257, 8, 128) == 3 * 128 * 4
    assert B.moe_sort_workspace_bytes(0, 8, 128) == 0


def test_sort_refusals(B):
    def sort(T=16, k=2, E=8, align=1, rows=32, ids=P, counts=P, offsets=P, perm=P, pos=P, ws=None, wsb=0):
        return B.moe_sort(ids, T, k, E, align, counts, offsets, perm, rows, pos, ws, wsb, None)
    for bad in (dict(T=-1), dict(k=0), dict(k=65, rows=9999), dict(E=0), dict(E=1025), dict(align=0), dict(rows=31),
                dict(align=2, rows=39), dict(ids=None), dict(counts=None), dict(offsets=None), dict(perm=None),
                dict(pos=None), dict(rows=2 ** 31), dict(T=2000, rows=4000),
                dict(T=2000, rows=4000, ws=P, wsb=3 * 8 * 4 - 1)):
        assert sort(**bad) == B.MOE_E_INVAL, bad
    assert sort(T=2 ** 30, k=4, rows=2 ** 31 - 1) == B.MOE_E_UNSUPPORTED
    assert "pairs" in B.last_error()


def test_row_refusals(B):
    def permute(dt=0, x=P, ldx=64, perm=P, pos=P, T=4, k=2, rows=8, cols=64, out=P, ldo=64):
        return B.moe_permute(dt, x, ldx, perm, pos, T, k, rows, cols, out, ldo, None)

    def unpermute(yt=0, y=P, ldy=64, rows=8, pos=P, w=P, base=None, ldb=0, T=4, k=2, cols=64, ot=0, out=P, ldo=64):
        return B.moe_unpermute(yt, y, ldy, rows, pos, w, base, ldb, T, k, cols, ot, out, ldo, None)

    def backward(ot=0, dout=P, ldd=64, yt=0, y=P, ldy=64, perm=P, rows=8, pos=P, w=P, T=4, k=2, cols=64, dy=P,
                 lddy=64, dw=P):
        return B.moe_unpermute_backward(ot, dout, ldd, yt, y, ldy, perm, rows, pos, w, T, k, cols, dy, lddy, dw, None)

    def gate(ids=P, w=P, dw=P, T=4, k=2, E=8, dz=P, ldz=8):
        return B.moe_gate_backward(ids, w, dw, T, k, E, dz, ldz, None)
    for bad in (dict(dt=3), dict(dt=-1), dict(ldx=63), dict(ldo=63), dict(T=-1), dict(k=0), dict(k=65), dict(cols=0),
                dict(rows=-1), dict(x=None), dict(pos=None), dict(out=None)):
        assert permute(**bad) == B.MOE_E_INVAL, bad
    assert permute(rows=0) == 0
    wide = 2 ** 30 + 1
    assert permute(cols=wide, ldx=wide, ldo=wide) == B.MOE_E_UNSUPPORTED
    many = dict(T=2 ** 24, k=1, cols=4096)
    assert permute(ldx=4096, ldo=4096, **many) == B.MOE_E_UNSUPPORTED      # over 2^24 - 1 workgroups
    assert unpermute(ldy=4096, ldo=4096, **many) == B.MOE_E_UNSUPPORTED
    assert unpermute(ldy=4096, ldo=4096, rows=0, **many) == B.MOE_E_UNSUPPORTED
    assert backward(ldd=4096, ldy=4096, lddy=4096, **many) == B.MOE_E_UNSUPPORTED
    assert gate(T=2 ** 26, k=1) == B.MOE_E_UNSUPPORTED
    for bad in (dict(yt=3), dict(ot=9), dict(ldy=63), dict(ldo=1), dict(base=P, ldb=63), dict(T=-1), dict(k=0),
                dict(cols=0), dict(rows=-1), dict(y=None), dict(pos=None), dict(out=None)):
        assert unpermute(**bad) == B.MOE_E_INVAL, bad
    assert unpermute(yt=0, ot=1) == B.MOE_E_UNSUPPORTED
    assert unpermute(base=P, ldb=64) == B.MOE_E_INVAL                      # out itself, but bf16
    assert unpermute(ot=2, base=P, ldb=72, ldo=64) == B.MOE_E_INVAL        # out itself, of another stride
    assert unpermute(T=0) == 0
    for bad in (dict(yt=3), dict(ot=9), dict(ldy=63), dict(ldd=1), dict(lddy=63), dict(T=-1), dict(k=65),
                dict(cols=0), dict(rows=-1), dict(y=None), dict(pos=None), dict(dout=None), dict(dy=None),
                dict(w=None), dict(dw=None)):
        assert backward(**bad) == B.MOE_E_INVAL, bad
    assert backward(yt=1, ot=0) == B.MOE_E_UNSUPPORTED
    assert backward(T=0, rows=0) == 0
    for bad in (dict(T=-1), dict(k=0), dict(k=65), dict(E=0), dict(ldz=7), dict(ids=None), dict(w=None),
                dict(dw=None), dict(dz=None)):
        assert gate(**bad) == B.MOE_E_INVAL, bad
    assert gate(T=0) == 0


def test_w4_refusals(B):
    def mm(xt=0, x=P, ldx=256, xr=4, rm=None, md=1, off=None, cnt=None, E=1, rows=4, codes=P, st=0, scales=P,
           zeros=None, N=32, K=256, group=128, gated=0, ot=0, out=P, ldo=32):
        return B.moe_w4_matmul(xt, x, ldx, xr, rm, md, off, cnt, E, rows, codes, st, scales, zeros, N, K, group,
                               gated, ot, out, ldo, None)
    for bad in (dict(xt=2), dict(xt=5), dict(st=2), dict(ot=1), dict(xt=1, ot=0), dict(N=0), dict(K=0),
                dict(gated=1, N=31), dict(group=16), dict(group=96), dict(group=192), dict(group=0), dict(group=-128),
                dict(K=200), dict(K=320), dict(rows=-1), dict(rows=2 ** 31), dict(E=0), dict(E=2), dict(E=1025, off=P),
                dict(cnt=P), dict(rm=P, md=0, off=P), dict(xr=3), dict(xr=-1), dict(ldx=255), dict(ldx=260),
                dict(ldo=31), dict(gated=1, ldo=15), dict(x=None), dict(codes=None), dict(scales=None),
                dict(out=None), dict(x=P + 8), dict(codes=P + 8)):
        assert mm(**bad) == B.MOE_E_INVAL, bad
    assert mm(K=32896, ldx=32896) == B.MOE_E_UNSUPPORTED
    assert mm(N=1, K=64, group=32, ldx=64) == B.MOE_E_UNSUPPORTED          # fewer than 4 groups in all
    assert mm(N=2 ** 28, group=32, ldo=2 ** 28) == B.MOE_E_UNSUPPORTED
    assert mm(rows=0) == 0


def test_torch_layer_refuses(B):
    """Everything but the device is right or wrong here as on the GPU; CPU
    tensors that pass every other check are refused last."""
    from expert_ffn_execution_router_amd import dispatch as D
    from expert_ffn_execution_router_amd import w4
    i32 = dict(dtype=torch.int32)
    ids, c, o, perm, pos = (torch.zeros(s, **i32) for s in ((4, 2), 8, 9, 8, (4, 2)))
    bf = torch.bfloat16
    x, xs, w, z = torch.zeros(4, 64, dtype=bf), torch.zeros(8, 64, dtype=bf), torch.zeros(4, 2), torch.zeros(4, 8)

    def no(fn, *a, match=None, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)
    no(D.sort, ids, c, o, perm, pos, match="GPU")
    no(D.sort, ids.long(), c, o, perm, pos, match="ids")
    no(D.sort, ids.reshape(-1), c, o, perm, pos, match="ids")
    no(D.sort, ids, c, o[:8], perm, pos, match="offsets")
    no(D.sort, ids, c, o, perm, pos.t(), match="pos")
    no(D.sort, torch.zeros(4, 4, **i32)[:, :2], c, o, perm, pos, match="ids")
    no(D.permute, x, perm, pos, xs, match="GPU")
    no(D.permute, x[:3], perm, pos, xs, match="x")
    no(D.permute, x.t(), perm, pos, xs, match="x")
    no(D.permute, x, perm, pos, xs.float(), match="out")
    no(D.permute, x, perm[:7], pos, xs, match="perm")
    no(D.permute, x.double(), perm, pos, xs.double(), match="x")
    no(D.permute, xs[:4], perm, pos, xs, match="overlaps")
    no(D.permute, x, perm, pos, torch.zeros(1, 64, dtype=bf).expand(8, 64), match="out")
    no(D.unpermute, xs, pos, w, x, match="GPU")
    no(D.unpermute, xs, pos, w.double(), x, match="w")
    no(D.unpermute, xs, pos, w[:3], x, match="w")
    no(D.unpermute, xs, pos, w, x[:3], match="out")
    no(D.unpermute, xs, pos, w, x, base=torch.zeros(4, 63), match="base")
    no(D.unpermute, xs, pos, w, x, base=torch.zeros(4, 64, dtype=bf), match="base")
    no(D.unpermute, xs, pos, w, xs[:4], match="overlaps")
    no(D.unpermute_backward, x, xs, perm, pos, w, xs, w.clone(), match="overlaps")
    no(D.unpermute_backward, x, xs, perm, pos, w, xs[:7].clone(), w.clone(), match="dy")
    no(D.unpermute_backward, x, xs, perm, pos, w, xs.clone(), w.t(), match="dw")
    no(D.unpermute_backward, x, xs, perm, pos, w, xs.clone(), w.clone(), match="GPU")
    no(D.gate_backward, ids, w, w.clone(), z, match="GPU")
    no(D.gate_backward, ids, w, w.clone(), z.double(), match="dlogits")
    no(D.gate_backward, ids, w, w.clone(), z[:3], match="dlogits")
    codes, sc = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=bf)
    out = torch.zeros(4, 16, dtype=bf)
    no(w4.linear, x, out, codes, sc, match="GPU")
    no(w4.linear, x, out, codes[:, :31], sc, match="codes")
    no(w4.linear, x, out, codes[None], sc[None], match="codes")
    no(w4.linear, x, out, codes, sc[:15], match="scales")
    no(w4.linear, x, out, codes, sc.float(), match="scales")
    no(w4.linear, x, out, codes, sc, zeros=sc.half(), match="zeros")
    no(w4.linear, x, out[:3], codes, sc, match="out")
    no(w4.linear, x, out, codes, sc, gated=True, match="out")
    no(w4.linear, x.float(), out, codes, sc, match="x")
    eo = torch.zeros(3, **i32)
    no(w4.experts, xs, eo, torch.zeros(8, 16, dtype=bf), codes[None].repeat(2, 1, 1), sc[None].repeat(2, 1, 1),
       match="GPU")
    no(w4.experts, x, eo, torch.zeros(8, 16, dtype=bf), codes[None].repeat(2, 1, 1), sc[None].repeat(2, 1, 1),
       match="x")
    no(w4.experts, xs, eo[:2], torch.zeros(8, 16, dtype=bf), codes[None].repeat(2, 1, 1), sc[None].repeat(2, 1, 1),
       match="offsets")


def test_oracle_dispatch_worked_example():
    """3 tokens, 2 choices, 3 experts, one dropped pair, segments of 2."""
    ids = np.array([[2, 0], [0, -1], [2, 0]], dtype=np.int32)
    c, o, perm, pos = OD.sort_pairs(ids, 3, 2, 8)
    assert c.tolist() == [3, 0, 2] and o.tolist() == [0, 4, 4, 6]
    assert perm.tolist() == [1, 2, 5, -1, 0, 4, -2, -2]
    assert pos.tolist() == [[4, 0], [1, -1], [5, 2]]
    x = np.array([[1.0], [2.0], [3.0]])
    xs = OD.permute(x, perm, pos, np.full((8, 1), 9.0))
    assert xs[:, 0].tolist() == [1, 2, 3, 0, 1, 3, 9, 9]
    w = np.array([[0.5, 0.5], [1.0, 7.0], [0.25, 0.75]])
    out, _ = OD.unpermute(xs, pos, w, np.ones((3, 1)), 1)
    assert out[:, 0].tolist() == [2, 3, 4]
    dout = np.array([[2.0], [3.0], [4.0]])
    dy, dw, _ = OD.unpermute_backward(dout, xs, perm, pos, w, np.full((8, 1), 9.0))
    assert dy[:, 0].tolist() == [1, 3, 3, 0, 1, 1, 9, 9]
    assert dw.tolist() == [[2, 2], [6, 0], [12, 12]]
    dz, _ = OD.gate_backward(ids, np.array([[0.5, 0.5], [1.0, 0.0], [0.25, 0.75]]), dw, 3)
    assert dz.tolist() == [[0, 0, 0], [0, 0, 0], [0, 0, 0]]
    dz, _ = OD.gate_backward(ids[:1], w[:1], np.array([[1.0, 3.0]]), 3)
    assert dz.tolist() == [[0.5, 0, -0.5]]


def test_oracle_w4_worked_example():
    q = np.array([[0, 15, 8, 9]])
    assert OW.pack(q).tolist() == [[0xF0, 0x98]]
    w = OW.dequantise(q, np.array([[0.5, 2.0]]), None, 2)
    assert w.tolist() == [[-4.0, 3.5, 0.0, 2.0]]
    w = OW.dequantise(q, np.array([[0.5, 2.0]]), np.array([[1.0, 9.0]]), 2)
    assert w.tolist() == [[-0.5, 7.0, -2.0, 0.0]]
    z, mag = OW.product(np.array([[1.0, -1.0, 2.0, 3.0]]), q, np.array([[0.5, 2.0]]), None, 2)
    assert z.tolist() == [[-4.0 - 3.5 + 6.0]]
    assert mag.tolist() == [[4.0 + 11.5 + 2 * 32 + 3 * 34]]
