"""The norms at odd widths past 8192 (the bounds are those of test_gpu_norms.py),
and rows that NaN or an infinity spoils beside others, forward and backward."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import fp8, norms
from oracle import norms as O
from test_gpu_norms import BF, EPS, EPS2, F8, F32, GATES, HF, PAIRS, U, check_codes, check_next, dev, gate_of, half, least, np64

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def codes_for(T, n):
    G = fp8.padded(n) // 128
    return torch.zeros(T, 128 * G, dtype=torch.uint8, device="cuda").view(F8), torch.zeros(G, T, device="cuda")


@pytest.mark.parametrize("dt,rt", PAIRS)
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,n", [(3, 8193), (2, 12345), (2, 16383)])
def test_odd_widths_past_8192(T, n, gate, dt, rt):
    print(f"wide T={T} n={n} {gate} {dt} {rt}", flush=True)
    rng = np.random.default_rng(n)
    y, r = dev(rng.standard_normal((T, n)) * 2, dt, 2), dev(rng.standard_normal((T, n)), rt, 1)
    for wt, with_w in ((dt, True), (F32, True), (dt, False)):
        w = dev(1 + 0.3 * rng.standard_normal(n), wt) if with_w else None
        w2 = dev(1 + 0.3 * rng.standard_normal(n), wt)
        g = gate_of(rng, gate, T, n, wt)
        out = torch.full((T, n + 1), 9.0, device="cuda", dtype=rt)
        nxt = torch.full((T, n + 4), 9.0, device="cuda", dtype=dt)
        norms.after(y, r, out[:, :n], weight=w, gate=g, alpha=0.75, eps=EPS, next_weight=w2, next_out=nxt[:, :n],
                    next_eps=EPS2)
        hw, hg = None if w is None else np64(w), None if g is None else np64(g)
        ref = O.after(np64(y), np64(r), 0.75, hw, hg, EPS)
        tol = 48 * U * (np.abs(0.75 * np64(r)) + np.abs(O.after(np64(y), None, 0, hw, hg, EPS)))
        tol = tol + half(rt) * 1.01 * (np.abs(ref) + tol) + least(rt)
        assert (np.abs(np64(out[:, :n]) - ref) <= tol).all()
        check_next(nxt[:, :n], np64(out[:, :n]), np64(w2), EPS2)
        assert (out[:, n:] == 9.0).all() and (nxt[:, n:] == 9.0).all()
        codes, s = codes_for(T, n)
        alone = torch.empty(T, n, device="cuda", dtype=rt)
        norms.after(y, r, alone, weight=w, gate=g, alpha=0.75, eps=EPS, next_weight=w2, next_out=codes, next_scales=s,
                    next_eps=EPS2)
        assert torch.equal(alone, out[:, :n])
        check_codes(codes, s, np64(alone), np64(w2), EPS2)
        two = torch.empty(T, n, device="cuda", dtype=dt)
        norms.before(alone, w2, two, eps=EPS2)
        assert torch.equal(two, nxt[:, :n])


@pytest.mark.parametrize("dt,rt", [(BF, F32), (HF, HF), (F32, F32)])
@pytest.mark.parametrize("n", [40, 700, 1025, 2048, 4100])
def test_spoilt_rows_stay_alone(n, dt, rt):
    """NaN or an infinity in any operand of a row makes that row's results NaN
    (its own values; all of a row that a norm goes over) and leaves the others'
    bits; sums over the rows are NaN."""
    print(f"spoilt n={n} {dt} {rt}", flush=True)
    rng = np.random.default_rng(n)
    T = 9
    fine = dict(y=dev(rng.standard_normal((T, n)), dt), r=dev(rng.standard_normal((T, n)), rt),
                g=dev(rng.standard_normal((T, 1)), dt), dh=dev(rng.standard_normal((T, n)), rt),
                dn=dev(rng.standard_normal((T, n)), dt))
    w, w2 = (dev(1 + 0.3 * rng.standard_normal(n), dt) for _ in range(2))

    def run(b, h=None):
        o = dict(out=torch.empty(T, n, device="cuda", dtype=rt), nxt=torch.empty(T, n, device="cuda", dtype=dt),
                 dy=torch.empty(T, n, device="cuda", dtype=dt), dr=torch.empty(T, n, device="cuda", dtype=rt),
                 dg=torch.empty(T, 1, device="cuda"), dw=torch.empty(n, device="cuda"), dw2=torch.empty(n, device="cuda"))
        codes, s = codes_for(T, n)
        norms.after(b["y"], b["r"], o["out"], weight=w, gate=b["g"], eps=EPS, next_weight=w2, next_out=o["nxt"])
        norms.after(b["y"], b["r"], o["out"], weight=w, gate=b["g"], eps=EPS, next_weight=w2, next_out=codes, next_scales=s)
        norms.after_backward(b["dh"], b["y"], o["dy"], o["dr"], weight=w, dweight=o["dw"], gate=b["g"], dgate=o["dg"],
                             eps=EPS, dnext=b["dn"], out=o["out"] if h is None else h, next_weight=w2,
                             dnext_weight=o["dw2"])
        o["codes"], o["s"] = codes.view(torch.uint8), s.t().contiguous()
        return o
    good = run(fine)
    assert all(v.isfinite().all() for v in good.values())
    bad = {k: v.clone() for k, v in fine.items()}
    bad["y"][1, n - 1], bad["y"][2, 0] = NAN, INF
    bad["r"][3, n // 2], bad["g"][4, 0] = NAN, INF
    bad["dh"][5, 1], bad["dn"][6, n - 2], bad["dn"][7, 0] = NAN, -INF, NAN
    got = run(bad)
    for k in ("out", "nxt", "codes", "s"):
        for t in (0, 5, 6, 7, 8):
            assert torch.equal(got[k][t], good[k][t]), (k, t)
    for k in ("dy", "dr", "dg"):
        for t in (0, 8):
            assert torch.equal(got[k][t], good[k][t]), (k, t)
    for t in (1, 2, 3, 4):
        assert got["nxt"][t].isnan().any() and got["out"][t].isfinite().all() == False      # noqa: E712
    assert got["out"][1].isnan().all() and got["nxt"][1].isnan().all()
    assert got["nxt"][3].isnan().all() and got["out"][3].isnan().sum() == 1
    for t in range(1, 8):
        assert got["dy"][t].isnan().any(), t
    assert got["dw"].isnan().all() and got["dw2"].isnan().any()
    # the first and last rows' share of the sums is what it was: NaN rows taken out
    rest = {k: v[[0, 8]].contiguous() for k, v in fine.items()}
    dw, dw2 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    norms.after_backward(rest["dh"], rest["y"], torch.empty(2, n, device="cuda", dtype=dt), None, weight=w, dweight=dw,
                         gate=rest["g"], eps=EPS, dnext=rest["dn"], out=good["out"][[0, 8]].contiguous(), next_weight=w2,
                         dnext_weight=dw2)
    assert dw.isfinite().all() and dw2.isfinite().all()
