"""Workloads of the operators in front of a routed expert FFN and of its
checkpoints: routing from scores with a balance bias and groups of experts, the
root-mean-square norm with the residual's addition, rows held in 8 bits, and
linear layers that leave and read such rows, each with its gradient.

``listed()`` names the workloads, ``draw(rng)`` gives one more of the same
ranges, ``prepare(case, seed)`` makes a call's inputs on the GPU, and
``run(state)`` makes one call: in plain torch operations in 32 bits, or, with
``own`` true, through the library.  ``exact(case, seed)`` is the same result
from the definitions in 64 bits, ``work(case)`` what a call cannot do without.

Rows in 8 bits: a block of a row's columns shares a power of two 2^e, the least
with max |v| < 127.5 2^e ("int8": codes rint(v 2^-e) + 128) or max |v| <= 464 2^e
("e4m3": codes v 2^-e in that type).  What is held so comes back as the values it
stands for, which bfloat16 and float16 hold exactly.

Inputs follow the recipes of the layer workloads: activations and logits
N(0, 1), weights N(0, 1) / sqrt(fan-in), biases N(0, 1) * 0.1; experts are
drawn with probability ~ (rank + 1)^-skew, distinct within a token.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def _route(name, direction, T, E, k, scores, groups=1, kept=1, group_top=2, bias=True, normalize=1, scale=1.0, masked=0.0):
    return {"name": name, "op": "route", "direction": direction, "T": T, "E": E, "k": k, "scores": scores,
            "groups": groups, "kept": kept, "group_top": group_top, "bias": bias, "normalize": normalize,
            "scale": scale, "masked": masked}


def _norm(name, direction, dtype, M, H, residual=True, weight=True, format="", block=128, output=True):
    return {"name": name, "op": "norm", "direction": direction, "dtype": dtype, "M": M, "H": H, "residual": residual,
            "weight": weight, "format": format, "block": block, "output": output}


def _rows8(name, dtype, M, N, format, block=128, k=0):
    return {"name": name, "op": "rows8", "direction": "round", "dtype": dtype, "M": M, "N": N, "format": format,
            "block": block, "k": k}


def _linear8(name, direction, dtype, M, K, N, format, block=128, G=0, activation="silu", bias=True, residual=False,
             skew=0.0, k=0, tail=0):
    return {"name": name, "op": "linear8", "direction": direction, "dtype": dtype, "M": M, "K": K, "N": N,
            "format": format, "block": block, "G": G, "activation": activation, "bias": bias, "residual": residual,
            "skew": skew, "k": k, "tail": tail}


def listed():
    return [
        # the router of one decode step: the smallest call, all latency
        _route("route_decode", "forward", 16, 128, 8, "sigmoid", groups=8, kept=4, scale=2.5),
        # a prompt through the router of a layer of very many experts, one of its groups half masked
        _route("route_prompt", "forward", 16384, 256, 6, "softmax", groups=16, kept=5, group_top=1, normalize=0,
               masked=0.03),
        # training the router of a layer of many experts
        _route("route_train_grad", "backward", 8192, 128, 8, "sigmoid", groups=8, kept=4, scale=2.5),
        # the norm in front of a layer in one decode step: latency
        _norm("norm_decode", "forward", "bf16", 16, 4096),
        # the same in training: rows for the products, and their 8-bit form as the checkpoint
        _norm("norm_train", "forward", "bf16", 8192, 4096, format="int8"),
        # float32 rows of odd length, 8-bit rows alone, small blocks
        _norm("norm_float32_odd", "forward", "f32", 2047, 1411, format="e4m3", block=32, output=False),
        # the norm's gradients, with the gradient that arrives beside it on the residual stream
        _norm("norm_grad", "backward", "bf16", 8192, 4096),
        # a layer's pre-activations into 8 bits and back
        _rows8("rows_preact", "bf16", 4096, 14336, "int8"),
        # 8-bit rows of tokens taken to the places of their experts' slots
        _rows8("rows_to_slots", "f16", 2047, 2048, "e4m3", block=64, k=6),
        # the experts' gated projection over sorted rows, pre-activations left in 8 bits
        _linear8("experts_keep", "forward", "bf16", 12288, 2048, 2816, "int8", G=64, activation="swiglu", bias=False,
                 skew=0.3),
        # its gradients, the input held in 8 bits once a token
        _linear8("experts_keep_grad", "backward", "f16", 12288, 2048, 2816, "e4m3", G=64, activation="swiglu",
                 bias=False, skew=0.3, k=6),
        # the gradients of the largest dense projection from its checkpoints
        _linear8("linear_large_grad", "backward", "bf16", 4096, 4096, 14336, "int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "rows8", "linear8", "linear8"])
    direction = rng.choice(["forward", "backward"])
    dtype, fmt, block = rng.choice(["f32", "f16", "bf16", "bf16"]), rng.choice(["int8", "e4m3"]), rng.choice([16, 32, 64, 128, 128])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16, 5])
        E = groups * _log(rng, 2 if groups > 1 else 4, 256 // groups)
        kept = rng.randint(1, groups)
        c = _route("", direction, _log(rng, 1, 16384), E, rng.randint(1, min(10, kept * (E // groups))),
                   rng.choice(["softmax", "sigmoid"]), groups, kept, rng.choice([1, 2]), rng.random() < 0.7,
                   rng.randint(0, 1), rng.choice([1.0, 2.5]), rng.choice([0.0, 0.0, 0.1]))
    elif op == "norm":
        H = _log(rng, 32, 16384)
        H = H if rng.random() < 0.3 else max(8, H // 8 * 8)
        M = max(1, min(_log(rng, 1, 16384), (1 << 25) // H))
        out8 = rng.choice(["", fmt]) if direction == "forward" else ""
        c = _norm("", direction, dtype, M, H, rng.random() < 0.6, rng.random() < 0.8, out8, block,
                  not out8 or rng.random() < 0.5)
    elif op == "rows8":
        N = _log(rng, 8, 16384)
        N = N if rng.random() < 0.3 else max(8, N // 8 * 8)
        k = rng.choice([0, 0, rng.randint(1, 8)])
        M = max(1, min(_log(rng, 1, 16384), (1 << 25) // (N * max(k, 1))))
        c = _rows8("", dtype, M, N, fmt, block, k)
    else:
        G = rng.choice([0, 0, _log(rng, 1, 64)])
        M, K, N = _log(rng, 1, 8192), _log(rng, 32, 8192), _log(rng, 32, 8192)
        if rng.random() < 0.7:
            K, N = max(8, K // 8 * 8), max(8, N // 8 * 8)
        most = (1 << 35) if dtype == "f32" else (1 << 37)
        M = max(1, min(M, most // (K * N)))
        while max(1, G) * N * K > 1 << 28:
            G //= 2
        k = rng.choice([0, rng.randint(1, 8)]) if G and direction == "backward" else 0
        if k:
            M = max(k, M // k * k)
        activation = rng.choice(["relu", "gelu", "silu", "swiglu"])
        if activation == "swiglu":
            N += N % 2
        c = _linear8("", direction, dtype, M, K, N, fmt, block, G, activation, rng.random() < 0.5,
                     direction == "forward" and rng.random() < 0.3, rng.uniform(0.0, 0.5) if G else 0.0, k,
                     rng.choice([0, M // 4]) if G else 0)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _expert_probs(E, skew):
    p = torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** -skew
    return p / p.sum()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    op, back = case["op"], case["direction"] == "backward"
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # router projections answer in bfloat16 steps, so equal logits occur
        st["logits"] = _normal(g, T, E).bfloat16().float()
        if case["masked"]:
            off = torch.rand(T, E, generator=g, device="cuda") < case["masked"]
            off[: T // 2, : E // (2 * case["groups"])] = True
            st["logits"].masked_fill_(off, -math.inf)
        st["b"] = _normal(g, E, scale=0.02 if case["scores"] == "sigmoid" else 0.002) if case["bias"] else None
        if back:
            st["indices"] = _plain_route(st)[0]
            st["grad_weights"] = _normal(g, T, k)
        return st
    dt = DTYPES[case["dtype"]]
    if op == "norm":
        M, H = case["M"], case["H"]
        st["x"] = _normal(g, M, H, dtype=dt)
        st["w"] = (1.0 + _normal(g, H, scale=0.1)).to(dt) if case["weight"] else None
        st["r"] = _normal(g, M, H, dtype=dt) if case["residual"] else None
        if back:
            st["grad_out"] = _normal(g, M, H, dtype=dt)
        return st
    if op == "rows8":
        M, N, k = case["M"], case["N"], case["k"]
        # activations have columns that are larger than others in every row
        st["x"] = (_normal(g, M, N) * torch.exp(_normal(g, N))).to(dt)
        st["perm"] = torch.randperm(M * k, generator=g, device="cuda").to(torch.int32) if k else None
        return st
    M, K, N, G, k = case["M"], case["K"], case["N"], case["G"], case["k"]
    No = N // 2 if case["activation"] == "swiglu" else N
    st["weight"] = _normal(g, *((G,) if G else ()), N, K, scale=K ** -0.5, dtype=dt)
    st["offsets"], st["group"], st["widest"] = None, None, 0
    if G:
        live = M - case["tail"]
        of = torch.multinomial(_expert_probs(G, case["skew"]), max(live, 1), replacement=True, generator=g)[:live]
        counts = torch.bincount(of, minlength=G)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["widest"] = max(1, int(counts.max()))  # the plan of the padded products
    if back:
        st["grad_out"] = _normal(g, M, No, dtype=dt)
        st["x8"] = _plain_quantize(_normal(g, M // max(k, 1), K, dtype=dt).float(), case["format"], case["block"])
        st["z8"] = _plain_quantize(_normal(g, M, N, dtype=dt).float(), case["format"], case["block"])
        st["perm"] = torch.randperm(M, generator=g, device="cuda").to(torch.int32) if k else None
    else:
        st["x"] = _normal(g, M, K, dtype=dt)
        st["b"] = _normal(g, *((G,) if G else ()), N, scale=0.1, dtype=dt) if case["bias"] else None
        st["r"] = _normal(g, M, No, dtype=dt) if case["residual"] else None
    return st


# ------------------------------------------------------------------ the plain form
def _top(c, k):
    """The k largest of each row, equal ones by ascending place: (values, places)."""
    val, at = torch.sort(c, dim=1, descending=True, stable=True)
    return val[:, :k], at[:, :k]


def _plain_scores(s):
    """Scores in 32 bits from 64 (values next to another one decide the selection), and the masked experts."""
    l = s["logits"].clamp(max=torch.finfo(torch.float32).max).double()
    off = torch.isnan(l) | (l == -math.inf)
    if s["scores"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = torch.where(off, -math.inf, l).max(1, keepdim=True).values
        e = torch.where(off, 0.0, torch.exp(l - m))
        p = e / e.sum(1, keepdim=True)
    return torch.where(off, 0.0, p).float(), off


def _plain_route(s):
    p, off = _plain_scores(s)
    c = p if s["b"] is None else p + s["b"]
    c = torch.where(off, -math.inf, c)
    T, E, G = s["T"], s["E"], s["groups"]
    if s["kept"] < G:
        best = torch.sort(c.reshape(T, G, E // G), dim=2, descending=True).values[:, :, : s["group_top"]]
        group = best[:, :, 0] + (torch.where(best[:, :, 1:] == -math.inf, 0.0, best[:, :, 1:])).sum(2)
        kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, _top(group, s["kept"])[1], True)
        c = torch.where(kept[:, :, None].expand(T, G, E // G).reshape(T, E), c, -math.inf)
    val, at = _top(c, s["k"])
    none = val == -math.inf
    w = torch.where(none, 0.0, p.gather(1, at))
    if s["normalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-37)
    return torch.where(none, -1, at).to(torch.int32), w * s["scale"]


def _plain_route_grad(s):
    p = _plain_scores(s)[0].double()
    at = s["indices"].long()
    held = at >= 0
    at = at.clamp(min=0)
    a = torch.where(held, s["grad_weights"].double() * s["scale"], 0.0)
    chosen = torch.where(held, p.gather(1, at), 0.0)
    if s["normalize"]:
        total = chosen.sum(1, keepdim=True).clamp(min=1e-37)
        a = (a - (a * chosen).sum(1, keepdim=True) / total) / total
    a = torch.zeros_like(p).scatter_add_(1, at, torch.where(held, a, 0.0))
    if s["scores"] == "sigmoid":
        return (a * p * (1.0 - p)).float()
    return (p * (a - (a * p).sum(1, keepdim=True))).float()


def _plain_quantize(v, fmt, block):
    """Codes [M, N] and scales [M, blocks] of the 32-bit rows v."""
    M, N = v.shape
    B = -(-N // block)
    pad = torch.zeros(M, B * block, device=v.device)
    pad[:, :N] = v
    m = pad.reshape(M, B, block).abs().amax(2)
    f, x = torch.frexp(m)
    if fmt == "int8":
        e = torch.where(f < 127.5 / 128, x - 7, x - 6)
    else:
        e = torch.where(f <= 464.0 / 512, x - 9, x - 8)
    e = torch.where(m == 0.0, 0, e).clamp(min=-126).to(torch.int32)
    scale = ((e + 127) << 23).view(torch.float32)
    q = v * ((127 - e) << 23).view(torch.float32).repeat_interleave(block, dim=1)[:, :N]
    return (torch.round(q) + 128.0).to(torch.uint8) if fmt == "int8" else q.to(torch.float8_e4m3fn), scale


def _plain_values(codes, scales, block):
    """The 32-bit values that codes and scales stand for."""
    q = codes.float()
    if codes.dtype == torch.uint8:
        q = q - 128.0
    return q * scales.repeat_interleave(block, dim=1)[:, : codes.shape[1]]


def _plain_norm(s):
    dt, h = s["x"].dtype, s["x"]
    if s["r"] is not None:
        h = (h.float() + s["r"].float()).to(dt)
    v = h.float()
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)
    y = y if s["w"] is None else y * s["w"].float()
    out = {}
    if s["output"]:
        out["output"] = y.to(dt)
    if s["r"] is not None:
        out["sum"] = h
    if s["format"]:
        out["values"] = _plain_values(*_plain_quantize(y, s["format"], s["block"]), s["block"]).bfloat16()
    return out


def _plain_norm_grad(s):
    dt, h, g = s["x"].dtype, s["x"].float(), s["grad_out"].float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6)
    n = h * rstd
    gw = g if s["w"] is None else g * s["w"].float()
    dh = rstd * (gw - n * (gw * n).mean(1, keepdim=True))
    if s["r"] is not None:
        dh = dh + s["r"].float()
    return dh.to(dt) if s["w"] is None else (dh.to(dt), (g * n).double().sum(0).to(dt))


def _plain_rows8(s):
    v = _plain_values(*_plain_quantize(s["x"].float(), s["format"], s["block"]), s["block"])
    if s["perm"] is not None:
        v = v[s["perm"].long() // s["k"]]
    return v.to(s["x"].dtype)


def _plain_act(z, kind):
    if kind == "relu":
        return torch.clamp(z, min=0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z[:, 0::2] * torch.sigmoid(z[:, 0::2]) * z[:, 1::2]


def _plain_act_grad(dy, z, kind):
    if kind == "relu":
        return dy * (z > 0)
    if kind == "gelu":
        return dy * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if kind == "silu":
        t = torch.sigmoid(z)
        return dy * t * (1.0 + z * (1.0 - t))
    g, u = z[:, 0::2], z[:, 1::2]
    t = torch.sigmoid(g)
    return torch.stack([dy * u * t * (1.0 + g * (1.0 - t)), dy * g * t], dim=2).reshape(z.shape)


def _plain_place(s):
    """Rows of groups, and every row's place within its group's padded block (the others in a block of their own)."""
    row = torch.arange(s["M"], device="cuda")
    off = s["offsets"].long()
    group = torch.searchsorted(off[1:], row, right=True)
    live = group < s["G"]
    at = torch.where(live, group * s["widest"] + row - off[group.clamp(max=s["G"] - 1)], s["G"] * s["widest"])
    return live, at


def _plain_pad(a, s, at):
    p = torch.zeros(s["G"] * s["widest"] + 1, a.shape[1], device="cuda")
    p[at] = a.float()
    return p[:-1].reshape(s["G"], s["widest"], -1)


def _plain_linear8(s):
    dt = s["x"].dtype
    w, b, r = s["weight"].float(), s["b"], s["r"]
    if s["G"]:
        live, at = _plain_place(s)
        z = torch.bmm(_plain_pad(s["x"], s, at), w.transpose(1, 2).contiguous())
        z = z if b is None else z + b.float()[:, None]
        z = torch.cat([z.reshape(-1, s["N"]), z.new_zeros(1, s["N"])])[at]
        z = torch.where(live[:, None], z, 0.0)
    else:
        z = torch.mm(s["x"].float(), w.t())
        z = z if b is None else z + b.float()
    y = _plain_act(z, s["activation"])
    if r is not None:
        y = y + r.float()
        y = y if not s["G"] else torch.where(live[:, None], y, 0.0)
    return y.to(dt), _plain_values(*_plain_quantize(z, s["format"], s["block"]), s["block"]).bfloat16()


def _plain_linear8_grad(s):
    w, dt = s["weight"].float(), s["weight"].dtype
    x, z = _plain_values(*s["x8"], s["block"]), _plain_values(*s["z8"], s["block"])
    if s["perm"] is not None:
        x = x[s["perm"].long() // s["k"]]
    dz = _plain_act_grad(s["grad_out"].float(), z, s["activation"])
    if s["G"]:
        live, at = _plain_place(s)
        dzp, xp = _plain_pad(dz, s, at), _plain_pad(x, s, at)
        dx = torch.bmm(dzp, w).reshape(-1, s["K"])
        dx = torch.cat([dx, dx.new_zeros(1, s["K"])])[at]
        dx = torch.where(live[:, None], dx, 0.0)
        dw, db = torch.bmm(dzp.transpose(1, 2).contiguous(), xp), dzp.sum(1)
    else:
        dx, dw, db = torch.mm(dz, w), torch.mm(dz.t(), x), dz.sum(0)
    return (dx.to(dt), dw.to(dt), db.to(dt)) if s["bias"] else (dx.to(dt), dw.to(dt))


def _plain(s):
    op, back = s["op"], s["direction"] == "backward"
    if op == "route":
        return _plain_route_grad(s) if back else _plain_route(s)
    if op == "norm":
        return _plain_norm_grad(s) if back else _plain_norm(s)
    if op == "rows8":
        return _plain_rows8(s)
    return _plain_linear8_grad(s) if back else _plain_linear8(s)


# ------------------------------------------------------------------ the library
def _own(s):
    import quantized_mixture_experts_router_amd as qm
    op, back = s["op"], s["direction"] == "backward"
    if op == "route":
        attrs = {"k": s["k"], "scores": s["scores"], "groups": s["groups"], "kept_groups": s["kept"],
                 "group_top": s["group_top"], "normalize_routing_weights": s["normalize"], "scale": s["scale"]}
        if back:
            return qm.route_scored_backward(s["grad_weights"], s["logits"], s["indices"], attrs)
        return qm.route_scored(s["logits"], s["b"], attrs)
    if op == "norm":
        if back:
            gx, gw = qm.rms_norm_backward(s["grad_out"], s["x"], s["w"], grad_sum=s["r"])
            return gx if s["w"] is None else (gx, gw)
        y, h, codes, scales = qm.rms_norm(s["x"], s["w"], s["r"], format=s["format"] or None, block_size=s["block"],
                                          keep_output=s["output"])
        out = {"output": y} if s["output"] else {}
        if h is not None:
            out["sum"] = h
        if s["format"]:
            out["values"] = qm.dequantize_rows(codes, scales, torch.bfloat16, s["block"])
        return out
    if op == "rows8":
        codes, scales = qm.quantize_rows(s["x"], s["format"], s["block"])
        return qm.dequantize_rows(codes, scales, s["x"].dtype, s["block"], perm=s["perm"])
    attrs = {"activation_type": s["activation"], "swiglu_fusion": int(s["activation"] == "swiglu")}
    if back:
        grads = qm.linear_backward_q8(s["grad_out"], s["x8"], s["weight"], s["z8"], s["offsets"], attrs,
                                      bias=s["bias"], block_size=s["block"], perm=s["perm"])
        return grads if s["bias"] else grads[:2]
    y, codes, scales = qm.linear_q8(s["x"], s["weight"], s["b"], s["r"], s["offsets"], attrs, format=s["format"],
                                    block_size=s["block"])
    return y, qm.dequantize_rows(codes, scales, torch.bfloat16, s["block"])


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------ what a call needs
def work(case):
    back = case["direction"] == "backward"
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * (T * E * (2 if back else 1) + 2 * T * k + E), "flops": 8 * T * E}
    es, block = SIZE[case["dtype"]], case.get("block", 128)
    if case["op"] == "norm":
        n = case["M"] * case["H"]
        if back:
            return {"bytes": es * n * (4 if case["residual"] else 3), "flops": 10 * n}
        held = (1 + 4 / block) * n + 2 * n if case["format"] else 0  # 8-bit rows, and the values read off them
        return {"bytes": int(es * n * ((3 if case["residual"] else 1) + int(case["output"])) + held), "flops": 5 * n}
    if case["op"] == "rows8":
        n = case["M"] * case["N"]
        return {"bytes": int(n * (es + 2 * (1 + 4 / block) + es * max(1, case["k"]))), "flops": 4 * n}
    M, K, N, G = case["M"], case["K"], case["N"], case["G"]
    live = M - case["tail"]
    No = N // 2 if case["activation"] == "swiglu" else N
    used = min(max(G, 1), live) if G else 1
    q = 1 + 4 / block
    if back:
        bytes_ = es * (live * No + used * N * K + M * K + max(G, 1) * N * (K + (1 if case["bias"] else 0)))
        return {"bytes": int(bytes_ + q * (live * N + M // max(1, case["k"]) * K)), "flops": 4 * live * N * K}
    bytes_ = es * (live * K + used * N * K + M * No * (2 if case["residual"] else 1))
    return {"bytes": int(bytes_ + (q + q + 2) * M * N), "flops": 2 * live * N * K}


# ------------------------------------------------------------------ 64 bits
def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_eight(v, fmt, block):
    """The values that 8-bit rows of v hold."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], block):
        part = v[:, c:c + block]
        top = part.abs().max(1, keepdim=True).values
        if fmt == "int8":
            # 2^e > top / 127.5, the least
            e = torch.frexp(top / 127.5).exponent
        else:
            # 2^e >= top / 464, the least
            frac, e = torch.frexp(top / 464.0)
            e = e - (frac == 0.5).to(e.dtype)
        unit = _two_to(e.clamp(min=-126))
        q = part / unit
        if fmt == "int8":
            q = torch.round(q)
        else:
            step = _two_to((torch.frexp(q).exponent - 1).clamp(min=-6) - 3)
            q = torch.round(q / step) * step
        out[:, c:c + block] = q * unit
    return out


def _exact_route(case, s):
    l = s["logits"].double()
    E, per = case["E"], case["E"] // case["groups"]
    if case["scores"] == "sigmoid":
        p = torch.special.expit(l)
    else:
        p = torch.nan_to_num(torch.softmax(l, 1))
    # scores count as float32 where they are ranked
    rank = p.float()
    if s["b"] is not None:
        rank = rank + s["b"][None]
    rank[torch.isinf(l)] = -math.inf
    if case["kept"] < case["groups"]:
        marks = []
        for g in range(case["groups"]):
            part = rank[:, g * per:(g + 1) * per]
            mark = part.max(1).values
            if case["group_top"] == 2 and per > 1:
                second = torch.kthvalue(part, per - 1, dim=1).values
                mark = torch.where(torch.isinf(second), mark, mark + second)
            marks.append(mark)
        marks = torch.stack(marks, 1)
        order = torch.argsort(-marks, dim=1, stable=True)
        place = torch.argsort(order, dim=1)
        rank[(place >= case["kept"]).repeat_interleave(per, dim=1)] = -math.inf
    order = torch.argsort(-rank, dim=1, stable=True)[:, :case["k"]]
    ok = ~torch.isinf(rank.gather(1, order))
    w = p.gather(1, order) * ok
    if case["normalize"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return torch.where(ok, order, -1).to(torch.int32), w * case["scale"]


def _exact_route_grad(case, s):
    with torch.enable_grad():
        l = s["logits"].double().requires_grad_()
        p = torch.special.expit(l) if case["scores"] == "sigmoid" else torch.softmax(l, 1)
        idx = s["indices"].long()
        ok = idx >= 0
        w = torch.where(ok, p.gather(1, idx.clamp(min=0)), 0.0)
        if case["normalize"]:
            some = ok.any(1, keepdim=True)
            w = torch.where(some, w / torch.where(some, w.sum(1, keepdim=True), 1.0), 0.0)
        (w * case["scale"] * s["grad_weights"].double()).sum().backward()
    return torch.nan_to_num(l.grad)


def _exact_norm(case, s):
    h = s["x"].double()
    if case["direction"] == "backward":
        g, w = s["grad_out"].double(), 1.0 if s["w"] is None else s["w"].double()
        q = 1.0 / torch.sqrt(h.square().sum(1, keepdim=True) / case["H"] + 1e-6)
        inner = (g * w * h).sum(1, keepdim=True) / case["H"]
        dh = q * g * w - q ** 3 * inner * h
        if s["r"] is not None:
            dh += s["r"].double()
        return dh if s["w"] is None else (dh, (g * h * q).sum(0))
    if s["r"] is not None:
        h = (h + s["r"].double()).to(s["x"].dtype).double()
    y = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["H"] + 1e-6)
    if s["w"] is not None:
        y = y * s["w"].double()
    out = {"output": y} if case["output"] else {}
    if s["r"] is not None:
        out["sum"] = h
    if case["format"]:
        out["values"] = _exact_eight(y, case["format"], case["block"])
    return out


def _exact_linear8(case, s):
    d = lambda t: None if t is None else t.double()  # noqa: E731
    M, N, K, kind = case["M"], case["N"], case["K"], case["activation"]
    w = d(s["weight"])
    if case["G"]:
        o = s["offsets"].tolist()
        spans = list(zip(o[:-1], o[1:]))
    else:
        spans, w = [(0, M)], w[None]
    live = spans[-1][1]
    if case["direction"] == "forward":
        x, b = d(s["x"]), d(s["b"])
        b = b[None] if b is not None and not case["G"] else b
        z = x.new_zeros(M, N)
        for g, (lo, hi) in enumerate(spans):
            z[lo:hi] = x[lo:hi] @ w[g].T
            if b is not None:
                z[lo:hi] += b[g]
        if kind == "swiglu":
            y = z[:, ::2] / (1 + (-z[:, ::2]).exp()) * z[:, 1::2]
        elif kind == "silu":
            y = z / (1 + (-z).exp())
        else:
            y = z * torch.special.ndtr(z) if kind == "gelu" else z.relu()
        if s["r"] is not None:
            y[:live] += d(s["r"])[:live]
        return y, _exact_eight(z, case["format"], case["block"])

    def held(codes, scales):
        v = codes.to(torch.float64) - (128 if case["format"] == "int8" else 0)
        at = torch.arange(v.shape[1], device="cuda") // case["block"]
        return v * scales.double()[:, at]
    dy, z, x = d(s["grad_out"]), held(*s["z8"]), held(*s["x8"])
    if case["k"]:
        x = x[torch.div(s["perm"].long(), case["k"], rounding_mode="floor")]
    if kind == "relu":
        dz = torch.where(z > 0, dy, torch.zeros_like(dy))
    elif kind == "gelu":
        dz = dy * (torch.special.ndtr(z) + z * (-z.square() / 2).exp() * (2 * math.pi) ** -0.5)
    elif kind == "silu":
        q = 1 / (1 + (-z).exp())
        dz = dy * (q + z * q * (1 - q))
    else:
        q = 1 / (1 + (-z[:, ::2]).exp())
        dz = torch.empty_like(z)
        dz[:, ::2] = dy * z[:, 1::2] * (q + z[:, ::2] * q * (1 - q))
        dz[:, 1::2] = dy * z[:, ::2] * q
    dx, dw, db = x.new_zeros(M, K), torch.zeros_like(w), x.new_zeros(w.shape[0], N)
    for g, (lo, hi) in enumerate(spans):
        dx[lo:hi] = dz[lo:hi] @ w[g]
        dw[g] = dz[lo:hi].T.contiguous() @ x[lo:hi]
        db[g] = dz[lo:hi].sum(0)
    if not case["G"]:
        dw, db = dw[0], db[0]
    return (dx, dw, db) if case["bias"] else (dx, dw)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route_grad(case, s) if case["direction"] == "backward" else _exact_route(case, s)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "rows8":
        v = _exact_eight(s["x"].double(), case["format"], case["block"])
        return v if s["perm"] is None else v[torch.div(s["perm"].long(), case["k"], rounding_mode="floor")]
    return _exact_linear8(case, s)
