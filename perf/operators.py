"""Cases and plain forms of the operators that stand around the token dispatch: the residual addition with
the RMS norm (rows out, FP8 codes with block scales out, and the backward), and the whole MoE layer for a few
tokens. ``own`` selects the library's kernels; without it the plain forms run (elementary torch operations)."""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
FP8_MAX = 448.0
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2, "fp8": 1}


def listed():
    return [
        # one decoded token's hidden row: latency only
        dict(name="norm_one_token", op="norm", T=1, H=7168, dtype="bf16", residual=True),
        # a prefill batch at the size of the largest dispatch workload
        dict(name="norm_prefill", op="norm", T=16384, H=7168, dtype="bf16", residual=True),
        # rows that no vector width divides, float32, a ragged batch, the first layer (nothing to add)
        dict(name="norm_f32_odd", op="norm", T=3001, H=1003, dtype="f32", residual=False),
        # a decode batch on its way to the FP8 dispatch
        dict(name="norm_fp8_decode", op="norm_fp8", T=64, H=4096, dtype="bf16", residual=True, block=128),
        # a prefill batch on its way to the FP8 dispatch
        dict(name="norm_fp8_prefill", op="norm_fp8", T=8192, H=7168, dtype="bf16", residual=True, block=128),
        # a training step's backward, with the gradient that arrives along the residual
        dict(name="norm_backward_train", op="norm_backward", T=8192, H=7168, dtype="bf16", residual=True),
        # the same for a small float32 model with odd rows
        dict(name="norm_backward_f32_odd", op="norm_backward", T=1024, H=513, dtype="f32", residual=False),
        # the smallest layer: one token, few small experts, float32
        dict(name="layer_f32_one_token", op="layer", T=1, H=512, I=1024, E=8, K=2, dtype="f32", skew=0.0),
        # one decoded token of a large layer
        dict(name="layer_one_token", op="layer", T=1, H=7168, I=1024, E=256, K=8, dtype="bf16", skew=1.2),
        # a decode batch of a large layer: nearly every expert is used, by a token or two each
        dict(name="layer_decode", op="layer", T=64, H=7168, I=1024, E=256, K=8, dtype="bf16", skew=0.0),
        # a small decode batch with FP8 weights and a skewed router
        dict(name="layer_fp8_decode", op="layer", T=8, H=4096, I=2048, E=128, K=8, dtype="fp8", block=128, skew=1.0),
        # a ragged batch over few experts: many rows an expert, sizes that no tile divides
        dict(name="layer_ragged", op="layer", T=133, H=2056, I=1399, E=64, K=2, dtype="bf16", skew=0.0),
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], spread over its logarithm; some odd, some multiples of 8 or 128."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    m = rng.choice((1, 8, 8, 128))
    return max(lo, min(hi, n // m * m)) if n >= m else n


def draw(rng):
    op = rng.choice(("norm", "norm_fp8", "norm_backward", "layer", "layer"))
    while True:
        if op == "layer":
            dtype = rng.choice(("f32", "bf16", "bf16", "fp8"))
            E = rng.choice((8, 16, 24, 64, 100, 128, 256))
            c = dict(op=op, T=_size(rng, 1, 256), H=_size(rng, 256, 7168), I=_size(rng, 128, 2048), E=E,
                     K=rng.randint(1, 8), dtype=dtype, skew=rng.choice((0.0, 1.0, 1.2)))
            if dtype == "fp8":
                c.update(block=128, H=max(256, c["H"] // 128 * 128), I=max(128, c["I"] // 128 * 128))
            if 3 * E * c["H"] * c["I"] * SIZE[dtype] <= 6e9:
                return c
        else:
            c = dict(op=op, T=_size(rng, 1, 16384), H=_size(rng, 64, 8192), dtype=rng.choice(("f32", "bf16", "bf16")),
                     residual=rng.random() < 0.7)
            if op == "norm_fp8":
                c.update(block=128, H=max(128, c["H"] // 128 * 128))
            if c["T"] * c["H"] * SIZE[c["dtype"]] <= 16384 * 7168 * 2:
                return c


def _rows(g, T, H, dtype):
    return torch.randn(T, H, generator=g, device="cuda").to(DT[dtype])


def _quantized(w, block):
    """E4M3 codes (as bytes) and the scales of blocks of `block` consecutive elements of each row."""
    v = w.float().view(*w.shape[:-1], -1, block)
    amax = v.abs().amax(-1)
    s = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    return (v / s[..., None]).to(torch.float8_e4m3fn).view(w.shape).view(torch.uint8), s


def _weights(g, E, rows, cols, dtype, block):
    """One matrix [rows, cols] for each expert; FP8 ones with their scales."""
    if dtype != "fp8":
        return torch.randn(E, rows, cols, generator=g, device="cuda", dtype=DT[dtype]).mul_(cols ** -0.5), None
    q = torch.empty(E, rows, cols, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, rows, cols // block, device="cuda")
    for e in range(E):
        q[e], s[e] = _quantized(torch.randn(rows, cols, generator=g, device="cuda").mul_(cols ** -0.5), block)
    return q, s


def _zipf_bias(E, s):
    """Logit biases log p_e, p_e proportional to (e + 1)^-s: the low ids are popular (0: none)."""
    r = np.arange(1, E + 1, dtype=np.float64) ** -float(s)
    return np.log(r / r.sum()) * (s > 0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] != "layer":
        T, H, dt = c["T"], c["H"], c["dtype"]
        s = dict(case=c, x=_rows(g, T, H, dt), w=1 + 0.1 * torch.randn(H, generator=g, device="cuda"))
        s["residual"] = _rows(g, T, H, dt) if c["residual"] else None
        if c["op"] == "norm_backward":  # x is the row that the forward normalised, residual the gradient beside it
            s["dout"] = _rows(g, T, H, dt)
            s["rstd"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float()
        return s
    T, H, I, E, dt = c["T"], c["H"], c["I"], c["E"], c["dtype"]
    rows = "bf16" if dt == "fp8" else dt
    # normalised hidden rows with a common direction u, along which the router prefers the popular experts
    u = torch.randint(0, 2, (H,), generator=g, device="cuda").float() * 2 - 1
    bias = torch.from_numpy(_zipf_bias(E, c["skew"])).float().cuda()
    router = torch.randn(E, H, generator=g, device="cuda") * (2 * H) ** -0.5 + bias[:, None] * u / H
    s = dict(case=c, x=(torch.randn(T, H, generator=g, device="cuda") + u).to(DT[rows]), router=router.to(DT[rows]),
             bias=_rows(g, T, H, rows))  # the residual stream, which the layer's output joins
    s["w13"], s["s13"] = _weights(g, E, 2 * I, H, dt, c.get("block"))
    s["w2"], s["s2"] = _weights(g, E, H, I, dt, c.get("block"))
    return s


# ---------------------------------------------------------------- plain forms


def _plain_sum(s):
    return s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()


def _plain_norm(s):
    h = _plain_sum(s)
    rstd = (h.square().mean(1) + EPS).rsqrt()
    return h, rstd, h * rstd[:, None] * s["w"]


def _plain_norm_rows(s):
    h, rstd, n = _plain_norm(s)
    dt = s["x"].dtype
    return {"out": n.to(dt), "sum": h.to(dt) if s["residual"] is not None else None, "rstd": rstd}


def _plain_norm_fp8(s):
    h, _, n = _plain_norm(s)
    q, sc = _quantized(n, s["case"]["block"])
    return {"codes": q.view(torch.float8_e4m3fn), "scales": sc, "sum": h.to(s["x"].dtype) if s["residual"] is not None else None}


def _plain_norm_backward(s):
    h, g, rstd = s["x"].float(), s["dout"].float(), s["rstd"][:, None]
    a, n = g * s["w"], h * rstd
    dx = rstd * (a - n * (a * n).mean(1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (g * n).sum(0)}


def _plain_route(s):
    """Top-k by (logit descending, id ascending) of the logits summed in 64 bits and rounded to 32, and the
    softmax over the k."""
    logits = (s["x"].double() @ s["router"].double().t()).float()
    v, i = torch.sort(logits, dim=1, descending=True, stable=True)
    v, i = v[:, : s["case"]["K"]].double(), i[:, : s["case"]["K"]]
    e = torch.exp(v - v[:, :1])
    return i, (e / e.sum(1, keepdim=True)).float()


def _values(w, scales):
    if scales is None:
        return w.float()
    v = w.view(torch.float8_e4m3fn).float()
    return (v.view(*scales.shape, -1) * scales[..., None]).view(v.shape)


def _plain_layer(s):
    c = s["case"]
    T, K, E, I = c["T"], c["K"], c["E"], c["I"]
    idx, w = _plain_route(s)
    x = s["x"].float()
    if 2 * T * K <= E:  # fewer slots than experts: each slot's own matrices
        e = idx.reshape(-1)
        pick = lambda a: None if a is None else a[e]  # noqa: E731
        xs = x.repeat_interleave(K, 0)[:, :, None]
        gu = torch.bmm(_values(s["w13"][e], pick(s["s13"])), xs)[:, :, 0]
        h = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
        y = torch.bmm(_values(s["w2"][e], pick(s["s2"])), h[:, :, None])[:, :, 0].view(T, K, -1)
        out = (y * w[:, :, None]).sum(1)
    else:  # every expert for every token, weight 0 where the token does not use it
        gu = torch.matmul(x, _values(s["w13"], s["s13"]).transpose(1, 2))
        h = gu[:, :, :I] / (1 + torch.exp(-gu[:, :, :I])) * gu[:, :, I:]
        y = torch.bmm(h, _values(s["w2"], s["s2"]).transpose(1, 2))
        dense = torch.zeros(T, E, device=x.device).scatter_(1, idx, w)
        out = (y * dense.t()[:, :, None]).sum(0)
    return {"out": (out + s["bias"].float()).to(s["x"].dtype), "topk_idx": idx.to(torch.int32), "topk_w": w}


def run(s):
    op = s["case"]["op"]
    if own:
        import unpermute_combine_amd as m

        if op == "norm":
            out, total, rstd = m.add_rmsnorm(s["x"], s["w"], residual=s["residual"], eps=EPS, want_rstd=True)
            return {"out": out, "sum": total, "rstd": rstd}
        if op == "norm_fp8":
            q, sc, total = m.add_rmsnorm_fp8(s["x"], s["w"], residual=s["residual"], eps=EPS, block=s["case"]["block"])[:3]
            return {"codes": q.view(torch.float8_e4m3fn), "scales": sc, "sum": total}
        if op == "norm_backward":
            dx, dw = m.add_rmsnorm_backward(s["dout"], s["x"], s["w"], s["rstd"], d_sum=s["residual"])
            return {"dx": dx, "dw": dw}
        out, idx, w = m.few_token_layer(s["x"], s["router"], s["w13"], s["w2"], s["case"]["K"],
                                        gate_up_scales=s["s13"], down_scales=s["s2"], bias=s["bias"])
        return {"out": out, "topk_idx": idx, "topk_w": w}
    return {"norm": _plain_norm_rows, "norm_fp8": _plain_norm_fp8, "norm_backward": _plain_norm_backward,
            "layer": _plain_layer}[op](s)


def work(case):
    c = case
    T, H, b = c["T"], c["H"], SIZE[c["dtype"]]
    if c["op"] == "norm":
        return {"bytes": T * H * b * (4 if c["residual"] else 2) + 4 * H + 4 * T, "flops": 5 * T * H}
    if c["op"] == "norm_fp8":
        return {"bytes": T * H * (b * (3 if c["residual"] else 1) + 1) + 4 * T * (H // c["block"]) + 4 * H, "flops": 7 * T * H}
    if c["op"] == "norm_backward":
        return {"bytes": T * H * b * (4 if c["residual"] else 3) + 4 * T + 8 * H, "flops": 9 * T * H}
    I, E, K = c["I"], c["E"], c["K"]
    # experts that T tokens use, on the average over routings of these logits
    r = np.random.default_rng(7)
    n = max(1, min(16, 65536 // (T * E)))
    z = r.standard_normal((n, T, E)) + _zipf_bias(E, c["skew"])
    top = np.argpartition(-z, K - 1, axis=2)[:, :, :K] if K < E else np.broadcast_to(np.arange(E), (n, T, E))
    used = np.mean([np.unique(t).size for t in top])
    rb = 2 if c["dtype"] == "fp8" else b
    w = 3 * H * I * b + (12 * H * I // c["block"] if c["dtype"] == "fp8" else 0)
    return {"bytes": int(used * w) + E * H * rb + 3 * T * H * rb + 8 * T * K,
            "flops": 6 * T * K * H * I + 2 * T * E * H}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op, total = case["op"], None
    if op == "layer":
        return _exact_layer(case, s)
    x, w, r = s["x"].double(), s["w"].double(), None if s["residual"] is None else s["residual"].double()
    if op == "norm_backward":
        # out_j = w_j x_j r(x), r = rstd as given: dr/dx_i = -r^3 x_i / H
        g, rstd = s["dout"].double(), s["rstd"].double()
        inner = torch.einsum("th,h,th->t", g, w, x)
        dx = torch.einsum("th,h,t->th", g, w, rstd) - x * (rstd ** 3 * inner / case["H"])[:, None]
        return {"dx": dx if r is None else dx + r, "dw": torch.einsum("th,th,t->h", g, x, rstd)}
    if r is not None:
        total = x = x + r
    rstd = 1 / torch.sqrt(torch.einsum("th,th->t", x, x) / case["H"] + EPS)
    n = torch.einsum("th,t,h->th", x, rstd, w)
    if op == "norm":
        return {"out": n, "sum": total, "rstd": rstd}
    blocks = n.reshape(case["T"], -1, case["block"])
    scales = blocks.abs().max(2).values / FP8_MAX
    scales[scales == 0] = 1
    codes = (blocks / scales[:, :, None]).reshape(n.shape).to(torch.float8_e4m3fn).double()
    return {"codes": codes, "scales": scales, "sum": total}


def _exact_layer(case, s):
    x, K, I = s["x"].double(), case["K"], case["I"]
    logits = torch.einsum("th,eh->te", x, s["router"].double()).float().cpu().numpy()
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :K]
    z = np.exp(np.take_along_axis(logits, ids, 1).astype(np.float64))
    wt = z / z.sum(1, keepdims=True)
    out = s["bias"].double()
    for e in np.unique(ids):
        t, k = np.nonzero(ids == e)
        rows = torch.from_numpy(t).cuda()
        mats = []
        for m, sc in ((s["w13"], s["s13"]), (s["w2"], s["s2"])):
            m = m[e].view(torch.float8_e4m3fn).double() if sc is not None else m[e].double()
            mats.append(m if sc is None else m * sc[e].double().repeat_interleave(case["block"], 1))
        gate, up = (x[rows] @ mats[0].t()).split(I, 1)
        y = (gate * torch.sigmoid(gate) * up) @ mats[1].t()
        out.index_add_(0, rows, y * torch.from_numpy(wt[t, k]).cuda()[:, None])
    return {"out": out, "topk_idx": None, "topk_w": torch.from_numpy(wt).cuda()}
