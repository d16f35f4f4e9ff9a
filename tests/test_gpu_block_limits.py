"""Quantisation, weights' gradients and norms where offsets pass 32 bits: the last
rows and matrices are those of a small call on the same values, to the bit (rows,
tiles and groups do not depend on where they lie)."""
import pytest
import torch

from expert_ffn_execution_router_amd import fp8, norms

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def codes(R, K):
    return (torch.zeros(R, fp8.padded(K), dtype=torch.uint8, device="cuda").view(F8),
            torch.zeros(fp8.padded(K) // 128, R, device="cuda"))


def test_quantize_past_32_bits():
    """4.3 G codes; x rows past 4 GiB."""
    print("quantize past 32 bits", flush=True)
    R, K, n = 525000, 8192, 300
    x = torch.empty(R, K, dtype=BF, device="cuda")
    x[-n:].normal_()
    x[:-n].zero_()
    q, s = codes(R, K)
    fp8.quantize(x, q, s)
    few, fs = codes(n, K)
    fp8.quantize(x[-n:], few, fs)
    assert torch.equal(q[-n:].view(torch.uint8), few.view(torch.uint8)) and torch.equal(s[:, -n:], fs)
    # through a map whose rows come from the end, transposed as well
    m = torch.full((1024,), -1, dtype=torch.int32, device="cuda")
    m[:n] = torch.arange(R - n, R, dtype=torch.int32, device="cuda")
    mq, ms = codes(1024, K)
    mt, mst = codes(K, 1024)
    fp8.quantize(x, mq, ms, mt, mst, row_map=m)
    assert torch.equal(mq[:n].view(torch.uint8), few.view(torch.uint8))
    ft, fst = codes(K, n)
    fp8.quantize(x[-n:], codes_t=ft, scales_t=fst)
    P = fp8.padded(n)
    assert torch.equal(mt[:, :P].view(torch.uint8), ft.view(torch.uint8)) and torch.equal(mst[:P // 128], fst)
    assert (mt[:, P:].view(torch.uint8) == 0).all()


def test_weight_gradient_past_32_bits():
    """70 matrices of 64 M values, 18.8 GB."""
    print("weight gradient past 32 bits", flush=True)
    E, N, K = 70, 8192, 8192
    o = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    o[1:36], o[36:70], o[70] = 128, 256, 512
    dy, dys = torch.randint(0, 120, (N, 512), dtype=torch.uint8, device="cuda").view(F8), torch.rand(4, N, device="cuda")
    x, xs = torch.randint(0, 120, (K, 512), dtype=torch.uint8, device="cuda").view(F8), torch.rand(4, K, device="cuda")
    dw = torch.full((E, N, K), -1.0, device="cuda")
    fp8.weight_gradient(dy, dys, x, xs, dw, offsets=o)
    one = torch.zeros(1, N, K, device="cuda")
    for e, (a, b) in ((0, (0, 128)), (35, (128, 256)), (69, (256, 512))):
        span = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        fp8.weight_gradient(dy[:, a:b].contiguous(), dys[a // 128:b // 128].contiguous(), x[:, a:b].contiguous(),
                            xs[a // 128:b // 128].contiguous(), one, offsets=span)
        assert torch.equal(dw[e], one[0]), e
    assert (dw[1] == 0).all() and (dw[34] == 0).all() and (dw[68] == 0).all()


def test_norms_past_32_bits():
    """Rows past 4 GiB, forward and backward."""
    print("norms past 32 bits", flush=True)
    T, n, few = 530000, 4100, 5
    y, r = (torch.zeros(T, n, dtype=BF, device="cuda") for _ in range(2))
    y[-few:].normal_()
    r[-few:].normal_()
    w = torch.rand(n, device="cuda") + 0.5
    out, nx = torch.empty_like(r), torch.empty_like(r)
    norms.after(y, r, out, weight=w, next_weight=w, next_out=nx)
    so, sn = torch.empty_like(r[-few:]), torch.empty_like(r[-few:])
    norms.after(y[-few:], r[-few:], so, weight=w, next_weight=w, next_out=sn)
    assert torch.equal(out[-few:], so) and torch.equal(nx[-few:], sn)
    assert (out[:-few] == 0).all()
    dy, dr = torch.empty_like(r), torch.empty_like(r)
    sy, sr = torch.empty_like(so), torch.empty_like(so)
    norms.after_backward(r, y, dy, dr, weight=w, dnext=nx, out=out, next_weight=w)
    norms.after_backward(r[-few:], y[-few:], sy, sr, weight=w, dnext=nx[-few:], out=so, next_weight=w)
    assert torch.equal(dy[-few:], sy) and torch.equal(dr[-few:], sr)
