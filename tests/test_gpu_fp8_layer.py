"""GPU parity of the layer of a few tokens with the float64 oracle.

Logits: fp32 sums of H products, rounded to the nearest (u / 2, u = 2^-23), off
by at most ez = (H / 64 + 12) u / 2 sum |x R| + u |z| (a lane adds H / 64
products, a wave 6 sums, then the bias).  A token is compared where its chosen
logits differ from each other and from the rest by more than their two ez: their
order is certain then.  Gate weights move by at most 4 ez + 16 u of themselves.
Gate and up: products of codes and 16-bit rows are exact, up to
(2 * 128 + 2 G + 16) roundings of sums below m = sum |x| |w|.  silu(g) u as in
the 4-bit products; it is kept to 2^-24 of itself.  The down product adds three
exact products a value: (2 * 384 + 2 n + 16) roundings for n groups in all."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import fp8
from oracle import fp8 as O

pytestmark = pytest.mark.gpu

BF, HF, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -23


def np64(t):
    return t.double().cpu().numpy()


def half(t):
    return torch.finfo(t).eps / 2


def weights(rng, E, H, I):
    def codes(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * 100).clamp(-448, 448).to(F8).cuda()

    def scales(s, *shape):
        return torch.from_numpy((np.exp(rng.standard_normal(shape) * 0.5) * s).astype(np.float32)).cuda()
    return dict(router=torch.from_numpy(rng.standard_normal((E, H)).astype(np.float32) / H ** 0.5).cuda(),
                gate_up=codes(E, 2 * I, H), gate_up_scales=scales(0.01 / H ** 0.5, E, I // 64, H // 128),
                down=codes(E, H, I), down_scales=scales(0.01 / I ** 0.5, E, H // 128, I // 128))


def run(x, p, k, ot, **kw):
    T, H = x.shape
    out = torch.full((T, H + 8), 7.0, device="cuda", dtype=ot)
    ids, w = torch.full((T, k), -9, dtype=torch.int32, device="cuda"), torch.full((T, k), -9.0, device="cuda")
    fp8.layer(x, p["router"], p["gate_up"], p["gate_up_scales"], p["down"], p["down_scales"], out[:, :H], ids, w, **kw)
    assert (out[:, H:] == 7.0).all()
    return out[:, :H], ids, w


def check(got, x, p, k, bias=None, base=None, rows=None):
    """Every token whose routing is not too near to call."""
    out, ids, w = got
    T, H = x.shape
    I = p["gate_up"].shape[1] // 2
    hx, R = np64(x), np64(p["router"])
    hb = None if bias is None else np64(bias)
    cache = {}

    def matrix(name, e):
        if (name, e) not in cache:
            cache[name, e] = O.block_values(p[name][e].view(torch.uint8).cpu().numpy(), p[name + "_scales"][e].cpu().numpy())
        return cache[name, e]
    rows = range(T) if rows is None else rows
    z = hx @ R.T + (0 if hb is None else hb)
    ez = (H / 64 + 12) * U / 2 * (np.abs(hx) @ np.abs(R).T) + U * np.abs(z)
    compared = 0
    for t in rows:
        order = np.argsort(-z[t], kind="stable")
        top = order[:k + 1]
        far = [z[t, a] - z[t, b] > ez[t, a] + ez[t, b] for a, b in zip(top, top[1:])]
        if not all(far):
            continue
        compared += 1
        pick = order[:k]
        assert ids[t].tolist() == pick.tolist()
        wt = np.exp(z[t, pick] - z[t, pick[0]])
        wt /= wt.sum()
        ew = wt * (4 * ez[t, pick].max() + 16 * U)
        assert (np.abs(np64(w[t]) - wt) <= ew).all()
        ref, err, mag = np.zeros(H), np.zeros(H), np.zeros(H)
        G = H // 128
        for j, e in enumerate(pick):
            gu, dn = matrix("gate_up", e), matrix("down", e)
            v = gu @ hx[t]
            ev = 1.01 * (2 * 128 + 2 * G + 16) * U * (np.abs(gu) @ np.abs(hx[t]))
            g, u, eg, eu = v[:I], v[I:], ev[:I], ev[I:]
            h = O.silu(g) * u
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(O.silu(g)) * eu + 8 * U * np.abs(h) + 1e-36
            y = dn @ h
            ref += wt[j] * y
            mag += wt[j] * (np.abs(dn) @ (np.abs(h) + eh))
            err += wt[j] * (np.abs(dn) @ eh) + ew[j] * np.abs(y)
        n = k * (I // 128)
        err += (2 * 384 + 2 * n + 16) * U * mag * 1.01
        if base is not None:
            ref = ref + np64(base[t])
            err += U * (np.abs(ref) + np.abs(np64(base[t])))
        err += half(out.dtype) * 1.01 * (np.abs(ref) + err) + (2.0 ** -25 if out.dtype == HF else 2.0 ** -134)
        d = np.abs(np64(out[t]) - ref)
        assert (d <= err).all(), (t, (d / err).max())
    return compared


LAYERS = [(1, 8, 2, 128, 128), (1, 1, 1, 128, 128), (2, 64, 8, 384, 256), (3, 65, 4, 256, 384), (5, 128, 8, 512, 128),
          (16, 200, 6, 640, 256), (16, 256, 8, 256, 256), (9, 4, 4, 128, 640), (16, 2, 1, 2048, 128), (1, 128, 8, 2048, 768),
          (4, 30, 3, 4224, 256)]


@pytest.mark.parametrize("xt,ot", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("T,E,k,H,I", LAYERS)
def test_layer(T, E, k, H, I, xt, ot):
    print(f"layer T={T} E={E} k={k} H={H} I={I} {xt} {ot}", flush=True)
    rng = np.random.default_rng(T + E + H)
    p = weights(rng, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H + 8)).astype(np.float32)).to(xt).cuda()[:, :H]
    bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32)).cuda()
    base = torch.from_numpy(rng.standard_normal((T, H + 4)).astype(np.float32)).cuda()[:, :H]
    plain = run(x, p, k, ot)
    assert check(plain, x, p, k) >= (T + 1) // 2
    more = run(x, p, k, ot, bias=bias, base=base)
    assert check(more, x, p, k, bias, base) >= (T + 1) // 2
    again = run(x, p, k, ot)
    assert all(torch.equal(a, b) for a, b in zip(plain, again))


def test_ties_and_masked_experts():
    """Equal logits go to the lower expert; experts masked by a bias of minus
    infinity are not chosen while others are left."""
    print("ties", flush=True)
    rng = np.random.default_rng(0)
    p = weights(rng, 70, 128, 128)
    x = torch.ones(3, 128, device="cuda", dtype=BF)
    p["router"].zero_()
    _, ids, w = run(x, p, 5, BF)
    assert ids.tolist() == [[0, 1, 2, 3, 4]] * 3 and (w == 0.2).all()
    bias = torch.full((70,), -float("inf"), device="cuda")
    bias[[68, 3, 40]] = torch.tensor([1.0, 1.0, 2.0], device="cuda")
    out, ids, w = run(x, p, 3, F32, bias=bias)
    assert ids.tolist() == [[40, 3, 68]] * 3 and out.isfinite().all()
    out, ids, w = run(x, p, 4, F32, bias=bias)
    assert ids.tolist() == [[40, 3, 68, 0]] * 3 and (w[:, 3] == 0).all() and out.isfinite().all()


def test_spoilt_tokens_touch_no_other():
    """Tokens with NaN and infinities beside others that choose the same
    experts: NaN in their rows, experts in range, nothing in the others."""
    print("spoilt tokens", flush=True)
    rng = np.random.default_rng(1)
    p = weights(rng, 6, 256, 128)
    x = torch.from_numpy(rng.standard_normal((8, 256)).astype(np.float32)).to(BF).cuda()
    x[2, 7], x[5, 100] = float("nan"), float("inf")
    out, ids, w = run(x, p, 4, F32)
    assert out[[2, 5]].isnan().any(1).all()
    assert ((ids >= 0) & (ids < 6)).all()
    assert check((out, ids, w), x, p, 4, rows=[0, 1, 3, 4, 6, 7]) >= 3


def test_two_streams_and_workspaces():
    """Calls in flight together, a workspace each, filled with anything."""
    print("two streams", flush=True)
    rng = np.random.default_rng(2)
    p = weights(rng, 64, 512, 256)
    todo = []
    for T in (16, 3, 1, 8):
        x = torch.from_numpy(rng.standard_normal((T, 512)).astype(np.float32)).to(BF).cuda()
        ws = torch.full((fp8.layer_workspace_bytes(T, 64, 6, 512, 256),), 0xFF, dtype=torch.uint8, device="cuda")
        todo.append((torch.cuda.Stream(), x, ws, run(x, p, 6, BF)))
    torch.cuda.synchronize()
    for _ in range(20):
        got = [run(x, p, 6, BF, ws=ws, stream=s) for s, x, ws, _ in todo]
        torch.cuda.synchronize()
        for g, (_, _, _, ref) in zip(got, todo):
            assert all(torch.equal(a, b) for a, b in zip(g, ref))


def test_captured_layer_replays_like_eager():
    print("captured layer", flush=True)
    rng = np.random.default_rng(3)
    p = weights(rng, 32, 256, 128)
    x = torch.zeros(4, 256, device="cuda", dtype=BF)
    out, ids, w = torch.zeros_like(x), torch.zeros(4, 4, dtype=torch.int32, device="cuda"), torch.zeros(4, 4, device="cuda")
    ws = torch.zeros(fp8.layer_workspace_bytes(4, 32, 4, 256, 128), dtype=torch.uint8, device="cuda")
    args = (p["router"], p["gate_up"], p["gate_up_scales"], p["down"], p["down_scales"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8.layer(x, *args, out, ids, w, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.layer(x, *args, out, ids, w, ws=ws)
    for seed in range(5):
        x.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((4, 256)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        ref = run(x, p, 4, BF)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, ids, w), ref)), seed
        check((out, ids, w), x, p, 4)
