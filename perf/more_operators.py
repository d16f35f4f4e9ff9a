"""Measured cases of the block-scaled 8-bit operators, the norms around a block
and the layer of a few tokens.

Five operators, each with a plain form (elementary torch operations in fp32)
beside the library's calls:

  quantize  values to e4m3 codes with one fp32 scale per 128 of them: rows
            (gathered by the sorted pairs, or silu(gate) * up of them), the
            same transposed (groups of 128 rows), weights in blocks of 128x128
  product   rows times weights of such codes, dense or per expert
  backward  a product's training step: the gradient rows quantised both ways,
            the gradient of the rows (transposed weights) and of the weights
  norm      after a block: alpha r + gate * (norm of y) and the next block's
            norm of it (as 16-bit values or e4m3 codes); and its gradients
  layer     a whole MoE layer for a few tokens: router, top-k, expert FFNs
            with e4m3 weights, weighted sum
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
F8 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # prefill batch to its grouped rows: the fp8 shape's hidden rows, segments aligned to 128
        dict(name="quantize_gather_T4096", op="quantize", kind="gather", T=4096, E=256, k=6, K=4096, dtype="bf16"),
        # activations of a training step, for the down product and its weight gradient; ragged number of rows
        dict(name="quantize_gated_R9001", op="quantize", kind="gated", R=9001, K=768, dtype="f16", both=True),
        # batched decode through a dense projection: the weights are the work
        dict(name="linear_T32", op="product", kind="dense", R=32, N=4096, K=4096, out="bf16"),
        # prefill chunk through a dense projection
        dict(name="linear_T8192", op="product", kind="dense", R=8192, N=4096, K=4096, out="bf16"),
        # gate/up of all experts of the fp8 shape, about 96 rows an expert
        dict(name="experts_T4096", op="product", kind="experts", T=4096, E=256, k=6, N=4096, K=4096, align=128,
             out="bf16"),
        # small dense step, nothing a multiple of anything, fp32 gradients
        dict(name="backward_T777", op="backward", kind="dense", R=777, N=1003, K=1001, dtype="f32", out="f32"),
        # experts of a training step on the prefill shape (gate/up)
        dict(name="backward_experts_T8192", op="backward", kind="experts", T=8192, E=128, k=8, N=1536, K=2048,
             dtype="bf16", out="bf16"),
        # single-token decode: latency, next block's input as codes
        dict(name="norm_T1", op="norm", kind="after", T=1, H=2048, dtype="bf16", res="bf16", gate="none", next="f8"),
        # prefill chunk, fp32 residual stream, a gate per token
        dict(name="norm_T8192", op="norm", kind="after", T=8192, H=4096, dtype="bf16", res="f32", gate="token",
             next="bf16"),
        # training step, a learned gate per channel, ragged number of rows
        dict(name="norm_backward_T4099", op="norm", kind="backward", T=4099, H=4096, dtype="bf16", res="bf16",
             gate="channel", next="bf16"),
        # single-token decode on the decode shape
        dict(name="layer_T1", op="layer", T=1, E=128, k=8, H=2048, I=768, dtype="bf16", out="bf16"),
        # a few sequences on the fp8 shape
        dict(name="layer_T16", op="layer", T=16, E=256, k=6, H=4096, I=2048, dtype="bf16", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log_int(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["quantize", "product", "backward", "norm", "layer"])
    dt = rng.choice(["bf16", "f16", "f32"])
    if op == "quantize":
        kind = rng.choice(["rows", "gather", "gated", "weights"])
        K = _log_int(rng, 64, 6144)
        if rng.random() < 0.6:
            K = max(8, K // 8 * 8)
        c = dict(op=op, kind=kind, K=K, dtype=dt)
        if kind == "gather":
            E = _log_int(rng, 8, 256)
            c.update(E=E, k=rng.randint(1, min(8, E)), T=_log_int(rng, 1, 2048))
        else:
            c.update(R=_log_int(rng, 1, 8192), both=rng.random() < 0.5)
        return c
    if op in ("product", "backward"):
        kind = rng.choice(["dense", "experts"])
        N = _log_int(rng, 100, 4096)
        if rng.random() < 0.6:
            N = N // 16 * 16
        c = dict(op=op, kind=kind, N=N, K=_mult(rng, 128, 4096, 128), out=rng.choice(["bf16", "f16", "f32"]))
        if op == "backward":
            c.update(dtype=dt, K=max(64, c["K"] - rng.choice([0, 0, rng.randint(1, 127)])))
        if kind == "dense":
            c["R"] = _log_int(rng, 1, 4096)
        else:
            E = _log_int(rng, 4, 128)
            k = rng.randint(1, min(8, E))
            align = 128 if op == "backward" else rng.choice([1, 128])
            c.update(E=E, k=k, T=_log_int(rng, 1, 2048), align=align)
        return c
    if op == "norm":
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(8, H // 8 * 8)
        kind = rng.choice(["before", "after", "backward"])
        return dict(op=op, kind=kind, T=_log_int(rng, 1, 8192), H=H, dtype=dt, res=rng.choice([dt, "f32"]),
                    gate=rng.choice(["none", "token", "channel", "full"]),
                    next=dt if kind == "backward" else rng.choice([dt, "f8"]))
    E = _log_int(rng, 8, 256)
    dt = rng.choice(["bf16", "f16"])
    return dict(op=op, T=rng.choice([1, 1, 2, 3, 5, 8, 13, 16]), E=E, k=rng.randint(1, min(8, E)),
                H=_mult(rng, 128, 4096, 128), I=_mult(rng, 128, 2048, 128), dtype=dt, out=rng.choice([dt, "f32"]))


# -- inputs ------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pad(n):
    return (n + 127) // 128 * 128


def _routing(T, E, k, gen, device="cuda"):
    """Distinct experts per token from logits with a Zipf(0.5) bias over a
    random order of the experts."""
    rank = torch.randperm(E, generator=gen, device=device).float() + 1
    z = torch.randn(T, E, generator=gen, device=device) * 2 - 0.5 * torch.log(rank)
    return torch.topk(z, k, dim=1)[1].to(torch.int32)


def _grouping(ids, E, align, rows):
    """Pairs sorted by expert, segments padded to `align` rows.  perm: pair of
    a grouped row, -1 in padding, -2 behind the last segment."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    ends = torch.cumsum((counts + align - 1) // align * align, 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    first = torch.cumsum(counts, 0) - counts
    key = flat[order]
    place = offsets[key] + torch.arange(n, device=ids.device) - first[key]
    perm = torch.where(torch.arange(rows, device=ids.device) < offsets[E], -1, -2)
    perm[place] = order
    return counts.to(torch.int32), offsets.to(torch.int32), perm.to(torch.int32)


def _codes(shape, gen):
    """Codes of bell-shaped values that reach to the type's largest."""
    v = torch.special.ndtri((torch.arange(8192, device="cuda") + 0.5) / 8192) * 115
    v = v.clamp(-448, 448).to(F8).view(torch.uint8).to(torch.int32)
    pair = v[torch.randint(8192, (1 << 16, 2), generator=gen, device="cuda")]
    table = (pair[:, 0] | (pair[:, 1] << 8)).to(torch.int16)
    n = math.prod(shape)
    idx = torch.randint(1 << 16, ((n + 1) // 2,), generator=gen, device="cuda", dtype=torch.int32)
    return table[idx].view(torch.uint8)[:n].view(F8).reshape(shape)


def _scales(shape, gen):
    return torch.exp(torch.randn(shape, generator=gen, device="cuda") * 0.3) * 1e-3


def _values(shape, gen, dt):
    """Rows of different sizes."""
    v = torch.randn(shape, generator=gen, device="cuda")
    v *= torch.exp(torch.randn(shape[0], 1, generator=gen, device="cuda") * 0.5)
    return v.to(dt)


def _f8(*shape):
    return torch.zeros(shape, device="cuda", dtype=torch.uint8).view(F8)


def _zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, device="cuda", dtype=dtype)


def _grouped(case, gen):
    """Grouped rows of an expert case: capacity, and the device's segments."""
    ids = _routing(case["T"], case["E"], case["k"], gen)
    n, align = case["T"] * case["k"], case.get("align", 128)
    rows = n + min(case["E"], n) * (align - 1)
    counts, offsets, perm = _grouping(ids, case["E"], align, rows)
    return dict(rows=rows, counts=counts, offsets=offsets, perm=perm, most=int(counts.max()))


def prepare(case, seed):
    gen = _generator(seed)
    op, s = case["op"], dict(case)
    if op == "quantize":
        K, kind, dt = case["K"], case["kind"], DTYPES[case["dtype"]]
        if kind == "weights":
            R = case["R"]
            s.update(x=(torch.randn(R, K, generator=gen, device="cuda") * 0.02).to(dt), codes=_f8(R, _pad(K)),
                     scales=_zeros(_pad(R) // 128, _pad(K) // 128))
            if case["both"]:
                s.update(codes_t=_f8(K, _pad(R)), scales_t=_zeros(_pad(K) // 128, _pad(R) // 128))
            return s
        if kind == "gather":
            g = _grouped(case, gen)
            R = g["rows"]
            s.update(row_map=g["perm"], x=_values((case["T"], K), gen, dt))
        else:
            R = case["R"]
            s["x"] = _values((R, 2 * K if kind == "gated" else K), gen, dt)
        s.update(R=R, codes=_f8(R, _pad(K)), scales=_zeros(_pad(K) // 128, R))
        if case.get("both"):
            s.update(codes_t=_f8(K, _pad(R)), scales_t=_zeros(_pad(R) // 128, K))
        return s
    if op in ("product", "backward"):
        N, K, experts = case["N"], case["K"], case["kind"] == "experts"
        lead = ()
        R = case.get("R")
        if experts:
            g = _grouped(case, gen)
            R, lead = g["rows"], (case["E"],)
            s.update(g)
        dt = DTYPES[case["out"]]
        if op == "product":
            s.update(a=_codes((R, K), gen), sa=_scales((K // 128, R), gen), w=_codes(lead + (N, K), gen),
                     sw=_scales(lead + (_pad(N) // 128, K // 128), gen), res=_zeros(R, N, dtype=dt))
            return s
        # gradient rows dy [R, N]; the transposed weights [K, N] and rows [K, R] that the forward pass kept
        Np, Rp = _pad(N), _pad(R)
        wt, xt = _codes(lead + (K, Np), gen), _codes((K, Rp), gen)
        wt.view(torch.uint8)[..., N:] = 0
        xt.view(torch.uint8)[:, R:] = 0
        if experts:             # padding rows are zeros
            pad = torch.cat([s["perm"] < 0, torch.zeros(Rp - R, device="cuda", dtype=torch.bool)])
            xt.view(torch.uint8)[:, pad] = 0
        dy = _values((R, N), gen, DTYPES[case["dtype"]])
        if experts:
            dy[s["perm"] < 0] = 0
        s.update(R=R, dy=dy, wt=wt, swt=_scales(lead + (_pad(K) // 128, Np // 128), gen), xt=xt,
                 sxt=_scales((Rp // 128, K), gen), codes=_f8(R, Np), scales=_zeros(Np // 128, R), codes_t=_f8(N, Rp),
                 scales_t=_zeros(Rp // 128, N), dx=_zeros(R, K, dtype=dt), dw=_zeros(*lead, N, K))
        return s
    if op == "norm":
        T, H, dt, rt = case["T"], case["H"], DTYPES[case["dtype"]], DTYPES[case["res"]]

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda")
        s["w2"] = (1 + 0.2 * randn(H)).to(dt)
        if case["kind"] == "before":
            s["y"] = _values((T, H), gen, dt)
        else:
            s.update(y=_values((T, H), gen, dt), r=(2 * randn(T, H)).to(rt), w1=(1 + 0.2 * randn(H)).to(dt),
                     alpha=0.75, res_out=_zeros(T, H, dtype=rt))
            shape = dict(none=None, token=(T, 1), channel=(1, H), full=(T, H))[case["gate"]]
            s["g"] = None if shape is None else (0.5 + 0.3 * randn(*shape)).to(dt)
        if case["kind"] == "backward":
            # the residual rows that the forward pass wrote, gradients of both results
            s.update(out=(2 * randn(T, H)).to(rt), dout=randn(T, H).to(rt), dnext=randn(T, H).to(dt),
                     dy=_zeros(T, H, dtype=dt), dr=_zeros(T, H, dtype=rt), dw1=_zeros(H), dw2=_zeros(H))
            s["dg"] = None if s["g"] is None else _zeros(*s["g"].shape,
                                                         dtype=dt if case["gate"] == "full" else torch.float32)
        elif case["next"] == "f8":
            s.update(nxt=_f8(T, _pad(H)), scales=_zeros(_pad(H) // 128, T))
        else:
            s.update(nxt=_zeros(T, H, dtype=dt), scales=None)
        return s
    T, E, k, H, I = (case[x] for x in ("T", "E", "k", "H", "I"))
    s.update(x=torch.randn(T, H, generator=gen, device="cuda").to(DTYPES[case["dtype"]]),
             router=torch.randn(E, H, generator=gen, device="cuda") / math.sqrt(H),
             gu=_codes((E, 2 * I, H), gen), sgu=_scales((E, 2 * I // 128, H // 128), gen) * (10 / math.sqrt(H)),
             dn=_codes((E, H, I), gen), sdn=_scales((E, H // 128, I // 128), gen) * (10 / math.sqrt(I)),
             res=_zeros(T, H, dtype=DTYPES[case["out"]]), ids=_zeros(T, k, dtype=torch.int32), wts=_zeros(T, k))
    return s


# -- one pass ----------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"quantize": _plain_quantize, "product": _plain_product, "backward": _plain_backward, "norm": _plain_norm,
            "layer": _plain_layer}[s["op"]](s)


_QUANTISED = ("codes", "scales", "codes_t", "scales_t")


def _run_own(s):
    from expert_ffn_execution_router_amd import fp8, norms
    op = s["op"]
    if op == "quantize":
        to = {n: s[n] for n in _QUANTISED if n in s}
        if s["kind"] == "weights":
            fp8.quantize_weights(s["x"], **to)
        elif s["kind"] == "gather":
            fp8.quantize(s["x"], **to, row_map=s["row_map"], map_div=s["k"])
        else:
            fp8.quantize(s["x"], **to, gated=s["kind"] == "gated")
        return to
    if op == "product":
        if s["kind"] == "dense":
            fp8.linear(s["a"], s["sa"], s["w"], s["sw"], s["res"])
        else:
            fp8.experts(s["a"], s["sa"], s["offsets"], s["w"], s["sw"], s["res"], counts=s["counts"])
        return s["res"]
    if op == "backward":
        fp8.quantize(s["dy"], s["codes"], s["scales"], s["codes_t"], s["scales_t"])
        if s["kind"] == "dense":
            fp8.linear(s["codes"], s["scales"], s["wt"], s["swt"], s["dx"])
            fp8.weight_gradient(s["codes_t"], s["scales_t"], s["xt"], s["sxt"], s["dw"])
        else:
            fp8.experts(s["codes"], s["scales"], s["offsets"], s["wt"], s["swt"], s["dx"], counts=s["counts"])
            fp8.weight_gradient(s["codes_t"], s["scales_t"], s["xt"], s["sxt"], s["dw"], offsets=s["offsets"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "norm":
        if s["kind"] == "before":
            norms.before(s["y"], s["w2"], s["nxt"], scales=s["scales"], eps=EPS)
            return {"next": s["nxt"], "scales": s["scales"]}
        if s["kind"] == "after":
            norms.after(s["y"], s["r"], s["res_out"], weight=s["w1"], gate=s["g"], alpha=s["alpha"], eps=EPS,
                        next_weight=s["w2"], next_out=s["nxt"], next_scales=s["scales"])
            return {"out": s["res_out"], "next": s["nxt"], "scales": s["scales"]}
        norms.after_backward(s["dout"], s["y"], s["dy"], s["dr"], weight=s["w1"], dweight=s["dw1"], gate=s["g"],
                             dgate=s["dg"], alpha=s["alpha"], eps=EPS, dnext=s["dnext"], out=s["out"],
                             next_weight=s["w2"], dnext_weight=s["dw2"])
        return {n: s[n] for n in ("dy", "dr", "dw1", "dw2", "dg")}
    fp8.layer(s["x"], s["router"], s["gu"], s["sgu"], s["dn"], s["sdn"], s["res"], s["ids"], s["wts"])
    return {"out": s["res"], "ids": s["ids"], "weights": s["wts"]}


def _to_codes(v, dims):
    """e4m3 codes of v, one scale per group (the axes `dims`): the largest
    value becomes 448, quotients and scales are fp32 numbers."""
    amax = v.abs().amax(dims, keepdim=True).clamp(min=2.0 ** -100)
    top = torch.full_like(amax, 448)
    return (v * (top / amax)).to(F8), amax / top


def _padded(v, rows, cols):
    return torch.nn.functional.pad(v, (0, cols - v.shape[1], 0, rows - v.shape[0]))


def _rows_quantised(v):
    R, K = v.shape
    q, sc = _to_codes(_padded(v, R, _pad(K)).unflatten(1, (-1, 128)), (2,))
    return q.flatten(1), sc[..., 0].t().contiguous()


def _blocks_quantised(v):
    R, K = v.shape
    q, sc = _to_codes(_padded(v, _pad(R), _pad(K)).reshape(_pad(R) // 128, 128, _pad(K) // 128, 128), (1, 3))
    return q.reshape(_pad(R), _pad(K)), sc[:, 0, :, 0]


def _plain_quantize(s):
    x, K = s["x"].float(), s["K"]
    if s["kind"] == "weights":
        codes, scales = _blocks_quantised(x)
        out = {"codes": codes[:x.shape[0]].contiguous(), "scales": scales.contiguous()}
        if "codes_t" in s:
            out.update(codes_t=codes.view(torch.uint8)[:, :K].t().contiguous().view(F8),
                       scales_t=scales.t().contiguous())
        return out
    if s["kind"] == "gated":
        gate, up = x.chunk(2, 1)
        x = gate / (1 + torch.exp(-gate)) * up
    if s["kind"] == "gather":
        m = s["row_map"].long()
        x = torch.where((m >= 0)[:, None], x[torch.div(m.clamp(min=0), s["k"], rounding_mode="floor")],
                        torch.zeros((), device="cuda"))
    codes, scales = _rows_quantised(x)
    if s["kind"] == "gather":           # rows behind the last segment stay as they were
        behind = s["row_map"] < -1
        codes = torch.where(behind[:, None], s["codes"].view(torch.uint8), codes.view(torch.uint8)).view(F8)
        scales = torch.where(behind, s["scales"], scales)
    out = {"codes": codes, "scales": scales}
    if "codes_t" in s:
        out["codes_t"], out["scales_t"] = _rows_quantised(x.t())
    return out


def _row_values(codes, scales):
    """Values of codes [R, K] with scales [K/128, R]."""
    return (codes.float().unflatten(1, (-1, 128)) * scales.t()[..., None]).flatten(1)


def _block_values(codes, scales):
    """Values of codes [.., N, K] with scales [.., ceil(N/128), K/128]."""
    N = codes.shape[-2]
    return codes.float() * scales.repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)


def _segments(s):
    """[E, most] grouped rows of each expert, and which of them there are."""
    i = torch.arange(s["most"], device="cuda")
    at = s["offsets"][:-1, None].long() + i
    real = i < s["counts"][:, None]
    return torch.where(real, at, torch.zeros_like(at)), real


def _expert_product(s, rows, w):
    """[R, N] rows times their expert's matrix (w [E, N, K])."""
    at, real = _segments(s)
    z = torch.bmm(rows[at], w.transpose(1, 2).contiguous())                # [E, most, N]
    res = torch.zeros(rows.shape[0] + 1, w.shape[1], device="cuda")
    res[torch.where(real, at, torch.full_like(at, rows.shape[0])).reshape(-1)] = z.flatten(0, 1)
    return res[:-1]


def _plain_product(s):
    a, w = _row_values(s["a"], s["sa"]), _block_values(s["w"], s["sw"])
    z = a @ w.t() if s["kind"] == "dense" else _expert_product(s, a, w)
    return z.to(DTYPES[s["out"]])


def _plain_backward(s):
    dy = s["dy"].float()
    N, R = s["N"], s["R"]
    rows = _row_values(*_rows_quantised(dy))[:, :N]
    cols = _row_values(*_rows_quantised(dy.t()))[:, :R]                    # [N, R]
    wt, xt = _block_values(s["wt"], s["swt"])[..., :N], _row_values(s["xt"], s["sxt"])[:, :R]
    if s["kind"] == "dense":
        return {"dx": (rows @ wt.t()).to(DTYPES[s["out"]]), "dw": cols @ xt.t()}
    at, real = _segments(s)
    x = torch.where(real[..., None], xt.t().contiguous()[at], torch.zeros((), device="cuda"))   # [E, most, K]
    dw = torch.bmm(cols.t().contiguous()[at].transpose(1, 2).contiguous(), x)
    return {"dx": _expert_product(s, rows, wt).to(DTYPES[s["out"]]), "dw": dw}


def _rms(x):
    return torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)


def _plain_norm(s):
    y = s["y"].float()
    if s["kind"] == "backward":
        return _plain_norm_backward(s, y)
    dt, out = DTYPES[s["dtype"]], {}
    if s["kind"] == "after":
        v = y * _rms(y) * s["w1"].float()
        if s["g"] is not None:
            v = v * s["g"].float()
        out["out"] = (s["alpha"] * s["r"].float() + v).to(s["r"].dtype)
        y = out["out"].float()
    z = y * _rms(y) * s["w2"].float()
    if s["next"] == "f8":
        out["next"], out["scales"] = _rows_quantised(z)
    else:
        out.update(next=z.to(dt), scales=None)
    return out


def _plain_norm_backward(s, y):
    dt, rt = DTYPES[s["dtype"]], s["r"].dtype
    h, dn, w1, w2 = s["out"].float(), s["dnext"].float(), s["w1"].float(), s["w2"].float()
    rs = _rms(h)
    n, dnw = h * rs, dn * w2
    d = s["dout"].float() + rs * (dnw - n * (dnw * n).mean(1, keepdim=True))
    ry = _rms(y)
    yn = y * ry
    dv, dg = d, None
    if s["g"] is not None:
        dv = d * s["g"].float()
        dg = d * (yn * w1)
        dg = dg.sum(1, keepdim=True) if s["gate"] == "token" else dg.sum(0, keepdim=True) if s["gate"] == "channel" \
            else dg.to(dt)
    dvw = dv * w1
    dy = ry * (dvw - yn * (dvw * yn).mean(1, keepdim=True))
    return {"dy": dy.to(dt), "dr": (s["alpha"] * d).to(rt), "dw1": (dv * yn).sum(0), "dw2": (dn * n).sum(0), "dg": dg}


def _plain_layer(s):
    x, k, I = s["x"].float(), s["k"], s["I"]
    z, order = torch.sort(x @ s["router"].t(), dim=1, descending=True, stable=True)
    ids, p = order[:, :k], torch.exp(z[:, :k] - z[:, :1])
    wts = p / p.sum(1, keepdim=True)
    e = ids.reshape(-1)
    gu = torch.bmm(_block_values(s["gu"][e], s["sgu"][e]), x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
    h = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
    y = torch.bmm(_block_values(s["dn"][e], s["sdn"][e]), h[:, :, None])[:, :, 0]
    out = (y.unflatten(0, (-1, k)) * wts[..., None]).sum(1)
    return {"out": out.to(DTYPES[s["out"]]), "ids": ids.to(torch.int32), "weights": wts}


# -- definition in 64 bits -----------------------------------------------------

def _exact_codes(v, amax):
    """Nearest e4m3 values (ties to even) of v in 64 bits under the group's
    largest value: the factor and the product are fp32 numbers."""
    top = amax.clamp(min=2.0 ** -100)
    q = (v * (448 / top).float().double()).float().double()
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(q / step) * step, (top / 448).float().double()


def _exact_rows(v):
    """Per row and 128 columns; values [R, ceil K], scales [G, R]."""
    R, K = v.shape
    g = torch.zeros(R, _pad(K), device="cuda", dtype=torch.float64)
    g[:, :K] = v
    g = g.view(R, -1, 128)
    q, sc = _exact_codes(g, g.abs().amax(2, keepdim=True))
    return q.reshape(R, -1), sc[:, :, 0].t()


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        x, K = s["x"].double(), case["K"]
        if case["kind"] == "weights":
            R = x.shape[0]
            nb, kb = _pad(R) // 128, _pad(K) // 128
            g = torch.zeros(nb * 128, kb * 128, device="cuda", dtype=torch.float64)
            g[:R, :K] = x
            amax = torch.nn.functional.max_pool2d(g.abs()[None, None], 128)[0, 0]
            q, sc = _exact_codes(g, amax.repeat_interleave(128, 0).repeat_interleave(128, 1))
            sc = sc[::128, ::128]
            out = {"codes": q[:R], "scales": sc}
            if case["both"]:
                out.update(codes_t=q[:, :K].t(), scales_t=sc.t())
            return out
        if case["kind"] == "gated":
            x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
        if case["kind"] == "gather":
            m = s["row_map"].long()
            live = torch.nonzero(m >= 0)[:, 0]
            g = torch.zeros(m.numel(), K, device="cuda", dtype=torch.float64)
            g[live] = x[m[live] // case["k"]]
            q, sc = _exact_rows(g)
            sc = sc.masked_fill(m < -1, 0)
            return {"codes": q, "scales": sc}
        out = dict(zip(("codes", "scales"), _exact_rows(x)))
        if case["both"]:
            out.update(zip(("codes_t", "scales_t"), _exact_rows(x.t())))
        return out
    if op in ("product", "backward"):
        N, K, experts = case["N"], case["K"], case["kind"] == "experts"
        R = s["a"].shape[0] if op == "product" else s["R"]
        segs = [(0, 0, R)]
        if experts:
            first, many = s["offsets"].tolist(), s["counts"].tolist()
            segs = [(e, first[e], first[e] + many[e]) for e in range(case["E"]) if many[e]]

        def weight(codes, scales, e):
            c, f = (codes[e], scales[e]) if experts else (codes, scales)
            n = torch.arange(c.shape[0], device="cuda") // 128
            return c.double() * f.double()[n].repeat_interleave(128, 1)
        if op == "product":
            res = torch.zeros(R, N, device="cuda", dtype=torch.float64)
            for e, r0, r1 in segs:
                a = s["a"][r0:r1].double() * s["sa"][:, r0:r1].double().t().repeat_interleave(128, 1)
                res[r0:r1] = torch.matmul(a, weight(s["w"], s["sw"], e).t().contiguous())
            return res
        q, sc = _exact_rows(s["dy"].double())
        qt, sct = _exact_rows(s["dy"].double().t())
        dy = q * sc.t().repeat_interleave(128, 1)
        dyt = (qt * sct.t().repeat_interleave(128, 1))[:, :R]
        dx = torch.zeros(R, K, device="cuda", dtype=torch.float64)
        dw = torch.zeros(s["dw"].shape, device="cuda", dtype=torch.float64)
        for e, r0, r1 in segs:
            dx[r0:r1] = torch.matmul(dy[r0:r1], weight(s["wt"], s["swt"], e).t().contiguous())
            tokens = torch.arange(r0, r1, device="cuda")
            x = s["xt"][:, r0:r1].double() * s["sxt"].double()[tokens // 128].t()
            (dw[e] if experts else dw).copy_(torch.matmul(dyt[:, r0:r1], x.t().contiguous()))
        return {"dx": dx, "dw": dw}
    if op == "norm":
        return _exact_norm(case, s)
    x, k, I = s["x"].double(), case["k"], case["I"]
    z = torch.matmul(x, s["router"].double().t())
    out = torch.zeros(case["T"], case["H"], device="cuda", dtype=torch.float64)
    ids = torch.zeros(case["T"], k, device="cuda", dtype=torch.int32)
    wts = torch.zeros(case["T"], k, device="cuda", dtype=torch.float64)

    def values(c, f):
        return c.double() * torch.kron(f.double(), torch.ones(128, 128, device="cuda", dtype=torch.float64))
    for t in range(case["T"]):
        top = torch.topk(z[t], k)
        w = torch.softmax(top.values, 0)
        for j, e in enumerate(top.indices.tolist()):
            gu = torch.mv(values(s["gu"][e], s["sgu"][e]), x[t])
            h = gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]
            out[t] += w[j] * torch.mv(values(s["dn"][e], s["sdn"][e]), h)
            ids[t, j] = e
        wts[t] = w
    return {"out": out, "ids": ids, "weights": wts}


def _exact_norm(case, s):
    kind = case["kind"]
    y, w2 = s["y"].double(), s["w2"].double()

    def scale_of(v):
        return 1 / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)
    if kind != "backward":
        out = {}
        if kind == "after":
            g = 1.0 if s["g"] is None else s["g"].double()
            h = s["alpha"] * s["r"].double() + g * (y * scale_of(y) * s["w1"].double())
            out["out"] = h
            y = h.float().to(s["r"].dtype).double()         # the next norm reads what is stored
        z = y * scale_of(y) * w2
        if case["next"] == "f8":
            out["next"], out["scales"] = _exact_rows(z)
        else:
            out.update(next=z, scales=None)
        return out
    H = case["H"]

    def jacobian(v, d):
        """Gradient through v / rms(v): r d - r^3 v <v, d> / H."""
        r = scale_of(v)
        return r * d - r ** 3 * v * (v * d).sum(1, keepdim=True) / H
    h, dn, w1 = s["out"].double(), s["dnext"].double(), s["w1"].double()
    d = s["dout"].double() + jacobian(h, dn * w2)
    g = torch.ones_like(d) if s["g"] is None else s["g"].double().expand_as(d)
    yn = y * scale_of(y)
    dg = d * w1 * yn
    dg = {"none": None, "token": dg.sum(1, keepdim=True), "channel": dg.sum(0, keepdim=True), "full": dg}[case["gate"]]
    return {"dy": jacobian(y, d * g * w1), "dr": s["alpha"] * d, "dw1": (d * g * yn).sum(0),
            "dw2": (dn * h * scale_of(h)).sum(0), "dg": dg}


# -- what a pass cannot do without -----------------------------------------------

def work(case):
    op = case["op"]
    if op == "quantize":
        b, K, kind = BYTES[case["dtype"]], case["K"], case["kind"]
        if kind == "weights":
            R = case["R"]
            return {"bytes": R * K * b + (1 + case["both"]) * R * K, "flops": 3 * R * K}
        R = case["T"] * case["k"] if kind == "gather" else case["R"]
        reads = case["T"] * K * b + R * 4 if kind == "gather" else R * K * b * (2 if kind == "gated" else 1)
        sides = 2 if case.get("both") else 1
        return {"bytes": reads + sides * (R * K + R * K // 32), "flops": (8 if kind == "gated" else 3) * sides * R * K}
    if op in ("product", "backward"):
        N, K, E = case["N"], case["K"], 1
        R = case.get("R")
        if case["kind"] == "experts":
            R = case["T"] * case["k"]
            gen = torch.Generator()
            gen.manual_seed(0)
            E = int(torch.unique(_routing(case["T"], case["E"], case["k"], gen, "cpu")).numel())
        weights = E * (N * K + N * K // 4096)
        if op == "product":
            return {"bytes": R * K + R * K // 32 + weights + R * N * BYTES[case["out"]], "flops": 2 * R * N * K}
        # dy in, x in; the weights; dx and dw out
        return {"bytes": R * N * BYTES[case["dtype"]] + R * K + weights + R * K * BYTES[case["out"]] +
                case.get("E", 1) * N * K * 4, "flops": 4 * R * N * K}
    if op == "norm":
        T, H, b, br = case["T"], case["H"], BYTES[case["dtype"]], BYTES[case["res"]]
        gate = {"none": 0, "token": T, "channel": H, "full": T * H}[case["gate"]]
        if case["kind"] == "before":
            return {"bytes": T * H * (b + (1 if case["next"] == "f8" else b)) + H * b, "flops": 6 * T * H}
        if case["kind"] == "after":
            return {"bytes": T * H * (b + 2 * br + (1 if case["next"] == "f8" else b)) + (2 * H + gate) * b,
                    "flops": 12 * T * H}
        return {"bytes": T * H * (3 * b + 3 * br) + 2 * H * (b + 4) + gate * b * 2, "flops": 30 * T * H}
    T, E, k, H, I = (case[x] for x in ("T", "E", "k", "H", "I"))
    gen = torch.Generator()
    gen.manual_seed(0)
    z = torch.randn(T, E, generator=gen)
    active = int(torch.unique(torch.topk(z, k, dim=1)[1]).numel())
    return {"bytes": active * 3 * H * I + E * H * 4 + T * H * 2 * BYTES[case["dtype"]], "flops": 6 * T * k * H * I}
