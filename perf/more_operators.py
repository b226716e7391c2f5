"""Measured cases of the operators around the expert layer's products.

Four operators, each with its plain form (elementary torch operations in fp32, in
fp64 where an order of scores is decided), its calls into the library and its
definition in 64 bits:

  route     router logits to expert ids and weights (softmax or sigmoid scores, a bias
            that only the choice sees, groups, renormalised weights); backward: the
            logits' gradient from the weights'
  norm      a residual's addition, the root-mean-square norm, rows out in 16 bits and in
            8 bits with scales (MXFP8); backward: the rows' and the weight's gradients
  swiglu    silu(gate) * up, out in MXFP8; in training out in the rows' type with the
            gate and up rows kept as MXFP8, and their gradient from those
  product8  rows quantised to MXFP8 times each expert's MXFP4 weight (W4A8)

Sizes are those of the 320-expert layer (d_model 4096, d_ff 1024, top-8, shards of
160 experts) and generic odd ones.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_BLOCK = 32
_EPS = 1e-6


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's choice of experts: latency
        dict(name="route_decode", op="route", backward=False, T=64, E=320, k=8, scores="softmax", bias=False, groups=1,
             top_groups=1, renormalize=True, dtype="fp32"),
        # a prefill batch under a balance bias, eight groups of experts of which four may serve a token
        dict(name="route_prefill_groups", op="route", backward=False, T=16384, E=320, k=8, scores="sigmoid", bias=True,
             groups=8, top_groups=4, renormalize=True, dtype="fp32"),
        # a training batch's gradient to the router, every expert's logit in it
        dict(name="route_grad_train", op="route", backward=True, T=8192, E=320, k=8, scores="softmax", bias=False,
             groups=1, top_groups=1, renormalize=False, dtype="bf16"),
        # one token's hidden state before the layer
        dict(name="norm_one_token", op="norm", backward=False, T=1, d=4096, residual=True, rows=True, mxfp8=True,
             dtype="bf16"),
        # a prefill batch: 16-bit rows for the router, 8-bit rows for the experts
        dict(name="norm_prefill", op="norm", backward=False, T=8192, d=4096, residual=True, rows=True, mxfp8=True,
             dtype="bf16"),
        # a training step's way back through the norm, with the residual's own gradient
        dict(name="norm_grad_train", op="norm", backward=True, T=8192, d=4096, residual=True, dtype="bf16"),
        # a decode step's gate and up rows on one of two expert shards
        dict(name="swiglu_decode", op="swiglu", train=False, T=64, E=320, k=8, offset=0, L=160, F=1024, dtype="bf16"),
        # a training batch there and back, its gate and up rows kept in 8 bits
        dict(name="swiglu_train", op="swiglu", train=True, T=8192, E=320, k=8, offset=0, L=320, F=1024, dtype="bf16"),
        # the same on a small layer of odd sizes, one shard of its experts
        dict(name="swiglu_train_odd", op="swiglu", train=True, T=3001, E=24, k=4, offset=6, L=12, F=1056, dtype="fp16"),
        # a decode step's gate/up product on one expert shard: weight streaming
        dict(name="product8_decode", op="product8", T=64, E=320, k=8, offset=0, L=160, N=2048, K=4096),
        # a prefill batch's gate/up product, all experts
        dict(name="product8_prefill", op="product8", T=8192, E=320, k=8, offset=0, L=320, N=2048, K=4096),
        # odd row counts and widths that end inside every tile
        dict(name="product8_odd", op="product8", T=3001, E=24, k=4, offset=0, L=24, N=1000, K=2080),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_routing(rng, max_tokens, most_experts=320):
    E = _log_int(rng, 1, 320)
    k = rng.randint(1, min(E, 8))
    L = min(most_experts, E if rng.random() < 0.5 else rng.randint(1, E))
    # a narrow shard gets some rows all the same
    return dict(T=max(_log_int(rng, 1, max_tokens), min(max_tokens, 8 * E // (k * L))), E=E, k=k, L=L,
                offset=rng.randint(0, E - L))


def draw(rng):
    op = rng.choice(["route", "norm", "swiglu", "product8"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 5, 8])
        E = groups * _log_int(rng, 4 if groups == 1 else 2, 320 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, E // groups * top_groups))
        return dict(op=op, backward=rng.random() < 0.4, T=_log_int(rng, 1, 16384), E=E, k=k,
                    scores=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups,
                    top_groups=top_groups, renormalize=k > 1 and rng.random() < 0.6,
                    dtype=rng.choice(["bf16", "fp16", "fp32", "fp32"]))
    if op == "norm":
        c = dict(op=op, backward=rng.random() < 0.4, T=_log_int(rng, 1, 8192), d=_log_int(rng, 8, 4096),
                 residual=rng.random() < 0.7, dtype=dtype)
        if not c["backward"]:
            c["mxfp8"] = rng.random() < 0.6
            c["rows"] = not c["mxfp8"] or rng.random() < 0.5
            if c["mxfp8"]:
                c["d"] = max(1, c["d"] // _BLOCK) * _BLOCK
        return c
    if op == "swiglu":
        c = dict(op=op, train=rng.random() < 0.6, dtype=dtype, F=_BLOCK * _log_int(rng, 1, 64), **_draw_routing(rng, 8192))
        c["T"] = max(1, min(c["T"], 8192 * 8 * 1024 // (c["k"] * c["F"])))
        return c
    N, K = _log_int(rng, 1, 4096), _BLOCK * _log_int(rng, 1, 128)
    return dict(op=op, N=N, K=K, **_draw_routing(rng, 4096, 320 * 2048 * 4096 // (N * K)))


# -------------------------------------------------------------------------- inputs
def _hidden(n, d, gen):
    """Hidden rows: N(0, 1) with one channel in 64 eight times as large, as trained layers show."""
    x = torch.randn(n, d, generator=gen, device="cuda")
    x[:, ::64] *= 8.0
    return x


def _offsets(c, gen):
    """int32 [L + 1]: where each local expert's rows begin, under a router that prefers none."""
    ids = torch.topk(torch.randn(c["T"], c["E"], generator=gen, device="cuda"), c["k"], dim=1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=c["E"])[c["offset"]:c["offset"] + c["L"]]
    return torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)


def _power(e):
    """2^e in fp32 for whole e in [-254, 254] as two exact factors: one alone passes the range of fp32."""
    return torch.exp2((e // 2).float()), torch.exp2((e - e // 2).float())


def _mxfp4_plain(x):
    """MXFP4 of fp32 x [..., C]: codes uint8 [..., C/2] (even element in the low nibble), scales uint8 [..., C/32]."""
    b = x.reshape(*x.shape[:-1], -1, _BLOCK)
    scale = (((b.abs().amax(-1).view(torch.int32) >> 23) & 0xFF) - 2).clamp(min=0)
    p, q = _power(127 - scale.unsqueeze(-1))
    v = b * p * q
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8) + 8 * torch.signbit(v).to(torch.uint8)).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.to(torch.uint8)


def _mxfp4_values_plain(codes, scales):
    """fp32 values [..., C] of MXFP4 codes [..., C/2] and scales [..., C/32] below 255."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], dim=-1)
    p, q = _power(scales.int().unsqueeze(-1) - 127)
    return (v.reshape(*scales.shape, _BLOCK) * p * q).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _mxfp8_plain(x):
    """The values that fp32 x [..., C] has as MXFP8: per 32 elements a scale 2^(floor(log2 amax) - 8), not below
    2^-127, and E4M3 elements to nearest, halves to even, at most 448."""
    b = x.reshape(*x.shape[:-1], -1, _BLOCK)
    scale = (((b.abs().amax(-1, keepdim=True).view(torch.int32) >> 23) & 0xFF) - 8).clamp(min=0)
    p, q = _power(127 - scale)
    v = b * p * q
    # E4M3's step at |v|: 2^(exponent - 3), from 2^-9 on
    step = torch.exp2(((((v.view(torch.int32) >> 23) & 0xFF) - 127).clamp(min=-6) - 3).float())
    v = (torch.round(v / step) * step).clamp(-448.0, 448.0)
    p, q = _power(scale - 127)
    return (v * p * q).reshape(x.shape)


def _keys64(logits, c, bias):
    """fp64 scores [T, E] of the logits, and the keys that the choice goes by."""
    x = logits.double()
    if c["scores"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    if bias is not None:
        return s, s + bias.double()
    return s, s


def _choose(keys, c):
    """The k experts of the highest keys, equal ones by the lowest id, among the top_groups groups whose two
    highest keys sum highest."""
    T, E = keys.shape
    G = c["groups"]
    if c["top_groups"] < G:
        grouped = keys.reshape(T, G, E // G)
        best = grouped.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        kept = torch.zeros_like(best).scatter_(1, best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]],
                                               1.0)
        keys = torch.where(kept.unsqueeze(2) > 0, grouped, grouped.new_full((), -math.inf)).reshape(T, E)
    return keys.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]


def _inputs(c, seed):
    """The case's inputs, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    dt = _DTYPES.get(c.get("dtype"))
    if c["op"] == "route":
        # a softmax router's logits spread wider than a sigmoid router's; the bias has settled at a few hundredths
        s = dict(logits=(randn(c["T"], c["E"]) * (2.0 if c["scores"] == "softmax" else 1.0)).to(dt),
                 bias=randn(c["E"]) * 0.05 if c["bias"] else None)
        if c["backward"]:
            s["ids"] = _choose(_keys64(s["logits"], c, s["bias"])[1], c).to(torch.int32)
            s["dweights"] = randn(c["T"], c["k"]) * 1e-2
        return s
    if c["op"] == "norm":
        s = dict(x=_hidden(c["T"], c["d"], gen).to(dt), weight=(1.0 + 0.1 * randn(c["d"])).to(dt))
        if c["backward"]:
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + _EPS).float()
            s["dy"] = (randn(c["T"], c["d"]) * 1e-2).to(dt)
        if c["residual"]:
            s["dh" if c["backward"] else "residual"] = (randn(c["T"], c["d"]) * (1e-2 if c["backward"] else 1.0)).to(dt)
        return s
    s = dict(offsets=_offsets(c, gen))
    rows = c["T"] * c["k"]
    if c["op"] == "swiglu":
        s["u"] = randn(rows, 2 * c["F"]).to(dt)
        if c["train"]:
            s["da"] = (randn(rows, c["F"]) * 1e-2).to(dt)
        return s
    N, K, L = c["N"], c["K"], c["L"]
    s["codes"] = torch.empty(L, N, K // 2, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.empty(L, N, K // _BLOCK, dtype=torch.uint8, device="cuda")
    for g in range(L):
        s["codes"][g], s["scales"][g] = _mxfp4_plain(randn(N, K) * K ** -0.5)
    s["rows"] = _hidden(rows, K, gen).to(torch.bfloat16)
    return s


def prepare(case, seed):
    c = case
    s = dict(case=c, **_inputs(c, seed))
    empty = lambda *shape, t: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
    dt, bf = _DTYPES.get(c.get("dtype")), torch.bfloat16
    # buffers that a program keeps; rows of no expert are left as they were: zeros
    if c["op"] == "route":
        s["out"] = empty(c["T"], c["E"], t=dt) if c["backward"] else \
            [empty(c["T"], c["k"], t=torch.int32), empty(c["T"], c["k"], t=torch.float32)]
    elif c["op"] == "norm" and c["backward"]:
        s["out"] = [empty(c["T"], c["d"], t=dt), empty(c["d"], t=torch.float32)]
    elif c["op"] == "norm":
        s["h"] = empty(c["T"], c["d"], t=dt) if c["residual"] else None
        s["y"] = empty(c["T"], c["d"], t=dt) if c["rows"] else None
        s["rstd"] = empty(c["T"], t=torch.float32)
        s["values"] = empty(c["T"], c["d"], t=bf) if c["mxfp8"] else None
    else:
        rows = c["T"] * c["k"]
        # which rows are whose: a program with its own loop over experts keeps this on the host
        s["bounds"] = s["offsets"].tolist()
        if c["op"] == "product8":
            s["out"] = torch.zeros(rows, c["N"], dtype=bf, device="cuda")
        elif c["train"]:
            s["out"] = [torch.zeros(rows, c["F"], dtype=dt, device="cuda"),
                        torch.zeros(rows, 2 * c["F"], dtype=dt, device="cuda")]
        else:
            s["values"] = torch.zeros(rows, c["F"], dtype=bf, device="cuda")
    if own:
        import nvfp4_expert_layer_amd as nv
        if c["op"] == "route":
            kind = nv.ROUTE_SOFTMAX if c["scores"] == "softmax" else nv.ROUTE_SIGMOID
            s["problem"] = nv.make_route_problem(c["T"], c["E"], c["k"], kind, c["groups"], c["top_groups"],
                                                 renormalize=c["renormalize"], dtype=dt)
        elif c["op"] == "norm":
            s["problem"] = nv.make_norm_problem(c["T"], c["d"], _EPS, dt, weight_dtype=dt)
            if c["backward"]:
                s["workspace"] = nv.alloc_norm_workspace(s["problem"])
            elif c["mxfp8"]:
                s["q"] = nv.MXFP8Rows.empty(c["T"], c["d"])
        elif c["op"] == "swiglu":
            s["problem"] = nv.make_swiglu_problem(rows, c["F"], c["L"], dt)
            s["q"] = nv.MXFP8Rows.empty(rows, 2 * c["F"] if c["train"] else c["F"])
            # rows of no expert stay as they are: codes of 0
            s["q"].codes.zero_()
            s["q"].scales.fill_(127)
        else:
            s["problem"] = nv.make_product_problem(rows, c["N"], c["K"], c["L"])
            s["w"] = nv.MXFP4Weights(s["codes"], s["scales"])
            s["q"] = nv.MXFP8Rows.empty(rows, c["K"])
    return s


# ----------------------------------------------------------------------------- run
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import nvfp4_expert_layer_amd as nv
    c, p = s["case"], s["problem"]
    if c["op"] == "route":
        if c["backward"]:
            return nv.moe_route_backward(p, s["logits"], s["ids"], s["dweights"], s["out"])
        return nv.moe_route(p, s["logits"], s["bias"], *s["out"])
    if c["op"] == "norm":
        if c["backward"]:
            return nv.moe_norm_backward(p, s["x"], s["weight"], s["rstd"], s["dy"], s.get("dh"), *s["out"], s["workspace"])
        q = s.get("q")
        nv.moe_norm(p, s["x"], s.get("residual"), s["weight"], s["h"], s["y"], q, s["rstd"])
        if q is not None:
            nv.moe_mxfp8_dequantize(q.codes, q.scales, s["values"])
        return _norm_outputs(s["h"], s["y"], s["rstd"], s["values"])
    q = s["q"]
    if c["op"] == "swiglu":
        if c["train"]:
            a, du = s["out"]
            nv.moe_swiglu(p, s["u"], s["offsets"], a, None, q)
            nv.moe_swiglu_backward(p, q, s["offsets"], s["da"], du)
            return [a, du]
        nv.moe_swiglu(p, s["u"], s["offsets"], None, q, None)
        return nv.moe_mxfp8_dequantize(q.codes, q.scales, s["values"])
    nv.moe_mxfp8_quantize(s["rows"], q.codes, q.scales)
    return nv.moe_mxfp8_product(p, q, s["w"], s["offsets"], s["out"])


def _norm_outputs(h, y, rstd, values):
    out = dict(rstd=rstd)
    if h is not None:
        out["h"] = h
    if y is not None:
        out["y"] = y
    if values is not None:
        out["values"] = values
    return out


def _run_plain(s):
    return dict(route=_route_plain, norm=_norm_plain, swiglu=_swiglu_plain, product8=_product_plain)[s["case"]["op"]](s)


def _route_plain(s):
    c, x = s["case"], s["logits"].float()
    soft, scores = c["scores"] == "softmax", None
    if not (soft and c["renormalize"]):
        if soft:
            e = torch.exp(x - x.amax(1, keepdim=True))
            scores = e / e.sum(1, keepdim=True)
        else:
            scores = 1.0 / (1.0 + torch.exp(-x))
    ids = s["ids"].long() if c["backward"] else _choose(_keys64(s["logits"], c, s["bias"])[1], c)
    if soft and c["renormalize"]:
        # the sum over all experts cancels: a softmax over the chosen ones
        z = x.gather(1, ids)
        z = torch.exp(z - z.amax(1, keepdim=True))
        w = z / z.sum(1, keepdim=True)
    else:
        w = scores.gather(1, ids)
        if c["renormalize"]:
            total = w.sum(1, keepdim=True)
            w = w / total
    if not c["backward"]:
        return [ids.to(torch.int32), w]
    g = s["dweights"]
    if c["renormalize"]:
        g = g - (w * g).sum(1, keepdim=True)          # through the division by the sum
    if soft and not c["renormalize"]:
        dx = torch.zeros_like(x).scatter_(1, ids, g)
        dx = scores * (dx - (w * g).sum(1, keepdim=True))
    elif soft:
        dx = torch.zeros_like(x).scatter_(1, ids, w * g)
    else:
        score = scores.gather(1, ids)
        if c["renormalize"]:
            g = g / total
        dx = torch.zeros_like(x).scatter_(1, ids, g * score * (1.0 / (1.0 + torch.exp(x.gather(1, ids)))))
    return dx.to(s["out"].dtype)


def _norm_plain(s):
    c, dt = s["case"], s["x"].dtype
    w = s["weight"].float()
    if c["backward"]:
        g, r = s["dy"].float(), s["rstd"].unsqueeze(1)
        n = s["x"].float() * r
        dweight = (g * n).sum(0)
        g = g * w
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        if "dh" in s:
            dx = dx + s["dh"].float()
        return [dx.to(dt), dweight]
    h = s["x"]
    if c["residual"]:
        h = (h.float() + s["residual"].float()).to(dt)
    f = h.float()
    r = 1.0 / torch.sqrt(f.square().mean(1, keepdim=True) + _EPS)
    y = f * r * w
    return _norm_outputs(h if c["residual"] else None, y.to(dt) if c["rows"] else None, r.squeeze(1),
                         _mxfp8_plain(y).to(torch.bfloat16) if c["mxfp8"] else None)


def _swiglu_plain(s):
    c, F, n = s["case"], s["case"]["F"], s["bounds"][-1]
    dt = s["u"].dtype
    u = s["u"][:n].float()
    gate, up = u[:, :F], u[:, F:]
    a = gate / (1.0 + torch.exp(-gate)) * up
    if not c["train"]:
        out = torch.zeros_like(s["values"])
        out[:n] = _mxfp8_plain(a).to(torch.bfloat16)
        return out
    kept = _mxfp8_plain(u)
    gate, up = kept[:, :F], kept[:, F:]
    sig, da = 1.0 / (1.0 + torch.exp(-gate)), s["da"][:n].float()
    out, du = torch.zeros_like(s["out"][0]), torch.zeros_like(s["out"][1])
    out[:n] = a.to(dt)
    du[:n, :F] = (da * up * sig * (1.0 + gate * (1.0 - sig))).to(dt)
    du[:n, F:] = (da * gate * sig).to(dt)
    return [out, du]


def _product_plain(s):
    out = torch.zeros_like(s["out"])
    for g, (b, e) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])):
        if b < e:
            w = _mxfp4_values_plain(s["codes"][g], s["scales"][g])
            out[b:e] = torch.matmul(_mxfp8_plain(s["rows"][b:e].float()), w.t()).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------- work
def work(case):
    c, b = case, _BYTES.get(case.get("dtype"), 2)
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        if c["backward"]:
            read = T * E * b if c["scores"] == "softmax" and not c["renormalize"] else T * k * b
            return {"bytes": read + T * E * b + 8 * T * k, "flops": 4.0 * T * E}
        return {"bytes": T * E * b + 8 * T * k + (4 * E if c["bias"] else 0), "flops": 4.0 * T * E}
    if c["op"] == "norm":
        n = c["T"] * c["d"]
        if c["backward"]:
            return {"bytes": n * b * (4 if c["residual"] else 3) + c["d"] * (b + 4) + 4 * c["T"], "flops": 10.0 * n}
        moved = b * (1 + 2 * c["residual"] + c["rows"])
        if c["mxfp8"]:
            moved += 2 * (1 + 1 / _BLOCK) + 2          # written, read back, its values
        return {"bytes": n * moved + c["d"] * b + 4 * c["T"], "flops": 6.0 * n}
    P = c["T"] * c["k"] * c["L"] / c["E"]
    if c["op"] == "swiglu":
        n, q = P * c["F"], 1 + 1 / _BLOCK
        if c["train"]:
            # there: gate and up, the activation, both kept; back: both kept, its gradient, theirs
            return {"bytes": n * (3 * b + 2 * q + 2 * q + 3 * b), "flops": 30.0 * n}
        return {"bytes": n * (2 * b + q) + c["T"] * c["k"] * c["F"] * (q + 2), "flops": 10.0 * n}
    N, K = c["N"], c["K"]
    touched = c["L"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])
    return {"bytes": touched * N * K * (0.5 + 1 / _BLOCK) + P * (N + K) * 2 + 4 * (c["L"] + 1), "flops": 2.0 * P * N * K}


# --------------------------------------------------------------------------- exact
def _two_to(e):
    """2^e in fp64 for whole e, exactly (a power function is not)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e2m1_exact(codes):
    """fp64 values of E2M1 codes from the format's fields: sign, two exponent bits (bias 1), one fraction bit."""
    c = codes.to(torch.int64)
    sign, e, m = 1.0 - 2.0 * (c >> 3).double(), (c >> 1) & 3, (c & 1).double()
    return sign * torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * _two_to(e - 1))


def _mxfp4_exact(codes, scales):
    """fp64 values of stored MXFP4 tensors."""
    pair = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    return _e2m1_exact(pair) * _two_to(scales.long() - 127).repeat_interleave(_BLOCK, dim=-1)


def _mxfp8_exact(x):
    """fp64 x [..., C] -> the nearest MXFP8 values: E4M3's grid under the block's scale, halves to even."""
    b = x.unflatten(-1, (-1, _BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    power = torch.where(top > 0, torch.frexp(top)[1].long() - 9, -127).clamp(min=-127)
    q = b / _two_to(power)
    step = _two_to((torch.frexp(q)[1].long() - 1).clamp(min=-6) - 3)
    return ((torch.round(q / step) * step).clamp(-448.0, 448.0) * _two_to(power)).flatten(-2)


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "route":
        return _route_exact(c, s)
    if c["op"] == "norm":
        x, w = s["x"].double(), s["weight"].double()
        if c["backward"]:
            g, r = s["dy"].double() * w, s["rstd"].double()
            n = x * r[:, None]
            dx = (g - n * ((g * n).sum(1) / c["d"])[:, None]) * r[:, None]
            return [dx + s["dh"].double() if c["residual"] else dx, torch.einsum("td,td->d", s["dy"].double(), n)]
        h = (x + s["residual"].double()).to(s["x"].dtype).double() if c["residual"] else x
        r = (h.pow(2).sum(1) / c["d"] + _EPS).pow(-0.5)
        y = h * r[:, None] * w
        return _norm_outputs(h if c["residual"] else None, y if c["rows"] else None, r,
                             _mxfp8_exact(y) if c["mxfp8"] else None)
    n = int(s["offsets"][-1])
    if c["op"] == "swiglu":
        F, u = c["F"], s["u"][:n].double()
        held = lambda v: torch.cat([v, v.new_zeros(s["u"].shape[0] - n, v.shape[1])])  # noqa: E731
        a = u[:, :F] * torch.sigmoid(u[:, :F]) * u[:, F:]
        if not c["train"]:
            return held(_mxfp8_exact(a))
        kept = _mxfp8_exact(u)
        gate, up, da = kept[:, :F], kept[:, F:], s["da"][:n].double()
        slope = torch.sigmoid(gate) + gate * torch.sigmoid(gate) * torch.sigmoid(-gate)
        return [held(a), held(torch.cat([da * up * slope, da * gate * torch.sigmoid(gate)], 1))]
    bounds = s["offsets"].tolist()
    out = torch.zeros(c["T"] * c["k"], c["N"], dtype=torch.float64, device="cuda")
    for g, (b, e) in enumerate(zip(bounds[:-1], bounds[1:])):
        if e > b:
            w = _mxfp4_exact(s["codes"][g], s["scales"][g])
            out[b:e] = _mxfp8_exact(s["rows"][b:e].double()) @ w.t().contiguous()
    return out


def _route_exact(c, s):
    """Weights and gradients in fp64, the latter from the score's Jacobian; the choice by repeated maxima."""
    x = s["logits"].double()
    T, E = x.shape
    score = torch.softmax(x, 1) if c["scores"] == "softmax" else torch.sigmoid(x)
    if c["backward"]:
        ids = s["ids"].long()
    else:
        key = score + (s["bias"].double() if c["bias"] else 0.0)
        group = torch.arange(E, device="cuda") // (E // c["groups"])
        best = torch.stack([key[:, group == g].topk(min(2, E // c["groups"]), 1).values.sum(1)
                            for g in range(c["groups"])], 1)
        place = (best[:, None, :] > best[:, :, None]).sum(2)              # groups ahead of each
        place += ((best[:, None, :] == best[:, :, None]).tril(-1)).sum(2)
        key = torch.where((place < c["top_groups"])[:, group], key, -math.inf)
        ids = torch.empty(T, c["k"], dtype=torch.long, device="cuda")
        for j in range(c["k"]):
            ids[:, j] = (key == key.amax(1, keepdim=True)).to(torch.uint8).argmax(1)
            key[torch.arange(T, device="cuda"), ids[:, j]] = -math.inf
    picked = score.gather(1, ids)
    total = picked.sum(1, keepdim=True)
    if not c["backward"]:
        return [ids.to(torch.int32), picked / total if c["renormalize"] else picked]
    g = s["dweights"].double()
    if c["renormalize"]:
        g = (g - (g * (picked / total)).sum(1, keepdim=True)) / total
    ds = torch.zeros_like(x).scatter_(1, ids, g)
    if c["scores"] == "softmax":
        return score * (ds - (score * ds).sum(1, keepdim=True))
    return ds * score * torch.sigmoid(-x)
