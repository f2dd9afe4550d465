"""Workloads of the operators around a routed expert FFN: routing weights,
tokens sorted by expert and back, and linear layers (dense or one weight per
expert), each forward and backward.

``listed()`` names the workloads, ``draw(rng)`` gives one more of the same
ranges, ``prepare(case, seed)`` makes a call's inputs on the GPU, and
``run(state)`` makes one call: in plain torch operations in 32 bits, or, with
``own`` true, through the library.  ``exact(case, seed)`` is the same result
from the definitions in 64 bits, ``work(case)`` what a call cannot do without.

Inputs follow the recipes of the layer workloads: activations and logits
N(0, 1), weights N(0, 1) / sqrt(fan-in), biases N(0, 1) * 0.1; experts are
drawn with probability ~ (rank + 1)^-skew, distinct within a token.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def _route(name, direction, T, E, k, routing="qmoe", normalize=0, masked=0.0):
    return {"name": name, "op": "route", "direction": direction, "T": T, "E": E, "k": k, "routing": routing,
            "normalize": normalize, "masked": masked}


def _rows(name, op, direction, dtype, T, H, E, k, skew, dropped=0.0):
    return {"name": name, "op": op, "direction": direction, "dtype": dtype, "T": T, "H": H, "E": E, "k": k,
            "skew": skew, "dropped": dropped}


def _linear(name, direction, dtype, M, K, N, G=0, activation="identity", bias=True, residual=False, keep=False,
            skew=0.0, tail=0):
    return {"name": name, "op": "linear", "direction": direction, "dtype": dtype, "M": M, "K": K, "N": N, "G": G,
            "activation": activation, "bias": bias, "residual": residual, "keep": keep, "skew": skew, "tail": tail}


def listed():
    return [
        # the router of one decode step: the smallest call, all latency
        _route("route_decode", "forward", 16, 8, 2),
        # training the router of a layer of many experts: softmax over all of them before the selection, some masked
        _route("route_train_grad", "backward", 8192, 128, 8, routing="moe", masked=0.02),
        # a fine-grained layer's tokens to its experts, skewed load
        _rows("dispatch_fine", "dispatch", "forward", "bf16", 2048, 2048, 64, 6, 0.5),
        # the gradient of that step for a layer of many experts on a GPU that holds half of them
        _rows("dispatch_large_grad", "dispatch", "backward", "bf16", 8192, 4096, 128, 8, 0.3, dropped=0.5),
        # one decode step's rows back to their tokens
        _rows("combine_decode", "combine", "forward", "f16", 16, 4096, 8, 2, 0.2),
        # a fine-grained layer's gradient at rows and weights, an odd token count
        _rows("combine_fine_grad", "combine", "backward", "bf16", 2047, 2048, 64, 6, 0.5),
        # one token through a dense gated projection: a read of the weights
        _linear("linear_one_token", "forward", "bf16", 1, 4096, 28672, activation="swiglu", bias=False),
        # the shared expert's output projection, added onto the routed sum
        _linear("linear_shared_out", "forward", "bf16", 4096, 14336, 4096, residual=True, bias=False),
        # a dense projection in float32, odd in every size, pre-activations kept for the backward pass
        _linear("linear_float32_odd", "forward", "f32", 1001, 2047, 1411, activation="gelu", keep=True),
        # training a dense projection: both gradients of the largest layer
        _linear("linear_large_grad", "backward", "bf16", 4096, 4096, 14336, activation="silu"),
        # the experts' gated projection over the sorted rows of a fine-grained layer
        _linear("experts_fine", "forward", "f16", 12288, 2048, 2816, G=64, activation="swiglu", keep=True, skew=0.3),
        # both gradients of the experts' output projection, a GPU's share of the rows
        _linear("experts_grad", "backward", "bf16", 16384, 1536, 4096, G=16, skew=0.3, tail=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "linear", "linear", "linear"])
    direction = rng.choice(["forward", "backward"])
    if op == "route":
        E = _log(rng, 4, 256)
        c = _route("", direction, _log(rng, 4, 16384), E, rng.randint(2, min(E, 10)), rng.choice(["qmoe", "moe"]),
                   rng.randint(0, 1), rng.choice([0.0, 0.0, 0.1]))
    elif op in ("dispatch", "combine"):
        E = _log(rng, 2, 256)
        k = rng.randint(1, min(E, 8))
        H = _log(rng, 32, 8192)
        H = H if rng.random() < 0.3 else max(8, H // 8 * 8)
        T = max(1, min(_log(rng, 1, 8192), (1 << 27) // (k * H)))
        c = _rows("", op, direction, rng.choice(["f32", "f16", "bf16"]), T, H, E, k, rng.uniform(0.0, 0.8),
                  rng.choice([0.0, 0.0, 0.5, 0.9]) if T * k >= 64 else 0.0)
    else:
        dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
        G = rng.choice([0, 0, _log(rng, 1, 64)])
        M, K, N = _log(rng, 1, 8192), _log(rng, 32, 8192), _log(rng, 32, 8192)
        if rng.random() < 0.7:
            K, N = max(8, K // 8 * 8), max(8, N // 8 * 8)
        most = (1 << 35) if dtype == "f32" else (1 << 37)
        M = max(1, min(M, most // (K * N)))
        while max(1, G) * N * K > 1 << 28:
            G //= 2
        activation = rng.choice(["identity", "relu", "gelu", "silu", "swiglu"])
        if activation == "swiglu":
            N += N % 2
        c = _linear("", direction, dtype, M, K, N, G, activation, rng.random() < 0.5, rng.random() < 0.3,
                    rng.random() < 0.5, rng.uniform(0.0, 0.5) if G else 0.0,
                    rng.choice([0, M // 4]) if G else 0)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _expert_probs(E, skew):
    p = torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** -skew
    return p / p.sum()


def _indices(g, case):
    """Distinct experts of each token (int32 [T, k]); a share `dropped` of the experts is held elsewhere."""
    T, E, k = case["T"], case["E"], case["k"]
    # k largest of log p + Gumbel noise: k distinct draws
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-6)))
    idx = (torch.log(_expert_probs(E, case["skew"])) + noise).topk(k, dim=1).indices
    first = int(case["dropped"] * E)  # a share that begins at this expert: the lower ones are held elsewhere
    idx = idx - first
    return torch.where(idx < 0, -1, idx).to(torch.int32), E - first


def _sorted_places(idx, E):
    """Place of each slot in expert order, stable; -1 - place for slots outside [0, E)."""
    flat = idx.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    return torch.where(key == E, -1 - place, place).to(torch.int32).reshape(idx.shape)


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
            st["logits"].masked_fill_(off, -math.inf)
        if back:
            st["indices"] = _plain_select(st["logits"], k)[0]
            st["grad_weights"] = _normal(g, T, k)
        return st
    if op in ("dispatch", "combine"):
        T, H, k, dt = case["T"], case["H"], case["k"], DTYPES[case["dtype"]]
        idx, held = _indices(g, case)
        st["indices"], st["experts"] = idx, held
        st["inverse"] = _sorted_places(idx, held)
        if op == "dispatch":
            st["rows" if back else "x"] = _normal(g, T * k if back else T, H, dtype=dt)
        else:
            st["rows"] = _normal(g, T * k, H, dtype=dt)
            st["weights"] = torch.softmax(_normal(g, T, k), dim=1)
            if back:
                st["grad_out"] = _normal(g, T, H, dtype=dt)
        return st
    M, K, N, G, dt = case["M"], case["K"], case["N"], case["G"], DTYPES[case["dtype"]]
    No = N // 2 if case["activation"] == "swiglu" else N
    lead = (G,) if G else ()
    st["x"] = _normal(g, M, K, dtype=dt)
    st["weight"] = _normal(g, *lead, N, K, scale=K ** -0.5, dtype=dt)
    st["b"] = _normal(g, *lead, N, scale=0.1, dtype=dt) if case["bias"] else None
    st["offsets"], st["group"], st["widest"] = None, None, 0
    if G:
        live = M - case["tail"]
        of = torch.multinomial(_expert_probs(G, case["skew"]), max(live, 1), replacement=True, generator=g)[:live]
        counts = torch.bincount(of, minlength=G)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["widest"] = max(1, int(counts.max()))  # the plan of the padded products
    if back:
        st["grad_out"] = _normal(g, M, No, dtype=dt)
        st["z"] = _normal(g, M, N, dtype=dt) if case["activation"] != "identity" else None
    else:
        st["r"] = _normal(g, M, No, dtype=dt) if case["residual"] else None
    return st


# ------------------------------------------------------------------ the plain form
def _plain_select(logits, k):
    l = torch.where(torch.isnan(logits), -math.inf, logits)
    val, idx = torch.sort(l, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    none = torch.isinf(val) & (val < 0)
    return torch.where(none, -1, idx).to(torch.int32), val, none


def _plain_probs(l, chosen, normalize_over_chosen, m):
    e = torch.exp(chosen - m)
    total = e.sum(1, keepdim=True) if normalize_over_chosen else torch.exp(l - m).sum(1, keepdim=True)
    return e, total


def _plain_route(s):
    l = s["logits"]
    idx, val, none = _plain_select(l, s["k"])
    m = torch.where(none[:, :1], 0.0, val[:, :1])
    e, total = _plain_probs(l, val, s["routing"] == "qmoe" or s["normalize"], m)
    return idx, torch.where(none, 0.0, e / total)


def _plain_route_grad(s):
    l, idx, gw = s["logits"], s["indices"].long(), s["grad_weights"]
    none = idx < 0
    at = idx.clamp(min=0)
    m = l.max(1, keepdim=True).values
    m = torch.where(torch.isinf(m), 0.0, m)
    chosen = torch.where(none, -math.inf, l.gather(1, at))
    over_chosen = s["routing"] == "qmoe" or s["normalize"]
    e, total = _plain_probs(l, chosen, over_chosen, m)
    w = torch.where(none, 0.0, e / total)
    mean = (w * gw).sum(1, keepdim=True)
    hit = torch.zeros_like(l).scatter_add_(1, at, torch.where(none, 0.0, w * (gw - mean) if over_chosen else w * gw))
    if over_chosen:
        return hit
    p = torch.where(torch.isinf(l), 0.0, torch.exp(l - m) / total.clamp(min=1e-38))
    return hit - p * mean


def _plain_dispatch(s):
    x, idx, E = s["x"], s["indices"], s["experts"]
    flat = idx.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= E), E, flat)
    perm = torch.sort(key, stable=True).indices
    ends = (key[None, :] <= torch.arange(E, device=key.device)[:, None]).sum(1)
    offsets = torch.cat([ends.new_zeros(1), ends])
    place = torch.empty_like(perm)
    place[perm] = torch.arange(perm.numel(), device=perm.device)
    inverse = torch.where(key == E, -1 - place, place)
    rows = torch.where((key[perm] < E)[:, None], x[perm // s["k"]], torch.zeros((), dtype=x.dtype, device=x.device))
    return rows, offsets.int(), perm.int(), inverse.int().reshape(idx.shape)


def _plain_slots(s):
    """The sorted rows of every token's slots in 32 bits, [T, k, H], zero where a slot is dropped."""
    inv = s["inverse"].long()
    rows = s["rows"][inv.clamp(min=0).reshape(-1)].float().reshape(*inv.shape, -1)
    return rows * (inv >= 0)[..., None]


def _plain_combine_grad(s):
    inv = s["inverse"].long()
    held = inv >= 0
    d = s["grad_out"].float()
    gw = (_plain_slots(s) * d[:, None]).sum(2)
    w = torch.where(held, s["weights"], 0.0)
    rows = torch.empty_like(s["rows"])
    place = torch.where(held, inv, -1 - inv).reshape(-1)
    rows[place] = (w[..., None] * d[:, None]).reshape(rows.shape).to(rows.dtype)
    return rows, gw


def _plain_act(z, kind):
    if kind == "identity":
        return z
    if kind == "relu":
        return torch.clamp(z, min=0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z[:, 0::2] * torch.sigmoid(z[:, 0::2]) * z[:, 1::2]


def _plain_act_grad(dy, z, kind):
    if kind == "identity":
        return dy
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
    """Group and place within its group's padded block of every row (rows behind the last group in a block of their own)."""
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


def _plain_linear(s):
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
    return (y.to(dt), z.to(dt)) if s["keep"] else y.to(dt)


def _plain_linear_grad(s):
    dt, x, w = s["x"].dtype, s["x"], s["weight"].float()
    dz = _plain_act_grad(s["grad_out"].float(), None if s["z"] is None else s["z"].float(), s["activation"])
    if s["G"]:
        live, at = _plain_place(s)
        dzp, xp = _plain_pad(dz, s, at), _plain_pad(x, s, at)
        dx = torch.bmm(dzp, w).reshape(-1, s["K"])
        dx = torch.cat([dx, dx.new_zeros(1, s["K"])])[at]
        dx = torch.where(live[:, None], dx, 0.0)
        dw, db = torch.bmm(dzp.transpose(1, 2).contiguous(), xp), dzp.sum(1)
    else:
        dx, dw, db = torch.mm(dz, w), torch.mm(dz.t(), x.float()), dz.sum(0)
    return (dx.to(dt), dw.to(dt), db.to(dt)) if s["bias"] else (dx.to(dt), dw.to(dt))


def _plain(s):
    op, back = s["op"], s["direction"] == "backward"
    if op == "route":
        return _plain_route_grad(s) if back else _plain_route(s)
    if op == "dispatch":
        return _plain_slots(s).sum(1).to(s["rows"].dtype) if back else _plain_dispatch(s)
    if op == "combine":
        return _plain_combine_grad(s) if back else (_plain_slots(s) * s["weights"][..., None]).sum(1).to(s["rows"].dtype)
    return _plain_linear_grad(s) if back else _plain_linear(s)


# ------------------------------------------------------------------ the library
def _own(s):
    import quantized_mixture_experts_router_amd as qm
    op, back = s["op"], s["direction"] == "backward"
    if op == "route":
        attrs = {"k": s["k"], "routing": s["routing"], "normalize_routing_weights": s["normalize"]}
        if back:
            return qm.route_backward(s["grad_weights"], s["logits"], s["indices"], attrs)
        return qm.route(s["logits"], attrs)
    if op == "dispatch":
        if back:
            return qm.dispatch_backward(s["rows"], s["inverse"])
        return qm.dispatch(s["x"], s["indices"], s["experts"])
    if op == "combine":
        if back:
            return qm.combine_backward(s["grad_out"], s["rows"], s["inverse"], s["weights"])
        return qm.combine(s["rows"], s["inverse"], s["weights"])
    attrs = {"activation_type": s["activation"], "swiglu_fusion": int(s["activation"] == "swiglu")}
    if back:
        grads = qm.linear_backward(s["grad_out"], s["x"], s["weight"], s["z"], s["offsets"], attrs, bias=s["bias"])
        return grads if s["bias"] else grads[:2]
    return qm.linear(s["x"], s["weight"], s["b"], s["r"], s["offsets"], attrs, keep_preact=s["keep"])


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------ what a call needs
def work(case):
    back = case["direction"] == "backward"
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * (T * E * (2 if back else 1) + 2 * T * k), "flops": 4 * T * E}
    es = SIZE[case["dtype"]]
    if case["op"] in ("dispatch", "combine"):
        T, H, k, E = case["T"], case["H"], case["k"], case["E"]
        S = T * k
        # rows of experts held elsewhere are not read; expected over the inputs
        p = [(i + 1) ** -case["skew"] for i in range(E)]
        held = S * sum(p[int(case["dropped"] * E):]) / sum(p)
        if case["op"] == "dispatch":
            if back:
                return {"bytes": int(es * H * (held + T) + 4 * S), "flops": int(held * H)}
            return {"bytes": int(es * H * (S + T) + 12 * S + 4 * E), "flops": 0}
        if back:
            return {"bytes": int(es * H * (T + held + S) + 12 * S), "flops": int(3 * held * H)}
        return {"bytes": int(es * H * (held + T) + 8 * S), "flops": int(2 * held * H)}
    M, K, N, G = case["M"], case["K"], case["N"], case["G"]
    live = M - case["tail"]
    No = N // 2 if case["activation"] == "swiglu" else N
    used = min(max(G, 1), live) if G else 1
    if back:
        z = 0 if case["activation"] == "identity" else live * N
        bytes_ = es * (live * (No + K) + z + used * N * K + M * K + max(G, 1) * N * (K + (1 if case["bias"] else 0)))
        return {"bytes": bytes_, "flops": 4 * live * N * K}
    bytes_ = es * (live * K + used * N * K + M * No * (2 if case["residual"] else 1) + (M * N if case["keep"] else 0))
    return {"bytes": bytes_, "flops": 2 * live * N * K}


# ------------------------------------------------------------------ 64 bits
def _exact_linear(case, s, back):
    d = lambda t: None if t is None else t.double()  # noqa: E731
    x, w, M, N, K = d(s["x"]), d(s["weight"]), case["M"], case["N"], case["K"]
    kind = case["activation"]
    spans = [(0, M)] if not case["G"] else None
    if spans is None:
        o = s["offsets"].tolist()
        spans = list(zip(o[:-1], o[1:]))
        b = d(s["b"])
    else:
        w, b = w[None], None if s["b"] is None else d(s["b"])[None]
    live = spans[-1][1]
    if not back:
        z = x.new_zeros(M, N)
        for g, (lo, hi) in enumerate(spans):
            z[lo:hi] = x[lo:hi] @ w[g].T
            if b is not None:
                z[lo:hi] += b[g]
        if kind == "swiglu":
            y = z[:, ::2] / (1 + (-z[:, ::2]).exp()) * z[:, 1::2]
        elif kind == "silu":
            y = z / (1 + (-z).exp())
        elif kind == "gelu":
            y = z * torch.special.ndtr(z)
        else:
            y = z.relu() if kind == "relu" else z.clone()
        if s["r"] is not None:
            y[:live] += d(s["r"])[:live]
        return (y, z) if case["keep"] else y
    dy, z = d(s["grad_out"]), d(s["z"])
    if kind == "identity":
        dz = dy
    elif kind == "relu":
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
    op, back = case["op"], case["direction"] == "backward"
    if op == "linear":
        return _exact_linear(case, s, back)
    if op == "route":
        l = s["logits"].double()
        over_all = case["routing"] == "moe" and not case["normalize"]
        # stable order: by falling logit, then by index
        order = torch.argsort(-l, dim=1, stable=True)[:, :case["k"]]
        taken = torch.zeros_like(l, dtype=torch.bool).scatter_(1, order, True) & ~torch.isinf(l)
        if over_all:
            p = torch.softmax(l, 1)
        else:
            p = torch.softmax(torch.where(taken, l, -math.inf), 1)
        p = torch.nan_to_num(p)
        if not back:
            w = p.gather(1, order)
            ok = taken.gather(1, order)
            return torch.where(ok, order, -1).to(torch.int32), torch.where(ok, w, 0.0)
        gw = torch.zeros_like(l)
        idx = s["indices"].long()
        ok = idx >= 0
        gw.scatter_add_(1, idx.clamp(min=0), torch.where(ok, s["grad_weights"].double(), 0.0))
        gp = torch.where(taken, gw, 0.0)
        return p * (gp - (p * gp).sum(1, keepdim=True))
    inv = s["inverse"].long()
    held = inv >= 0
    if op == "dispatch" and not back:
        T, k = inv.shape
        place = torch.where(held, inv, -1 - inv).reshape(-1)
        token = torch.arange(T, device="cuda").repeat_interleave(k)
        rows = torch.zeros(T * k, case["H"], device="cuda", dtype=torch.float64)
        rows[place] = s["x"].double()[token] * held.reshape(-1, 1)
        perm = torch.argsort(place)
        flat = s["indices"].reshape(-1)
        n = torch.bincount(flat[held.reshape(-1)].long(), minlength=s["experts"]).tolist()
        offsets = [0]
        for c in n:
            offsets.append(offsets[-1] + c)
        return rows, torch.tensor(offsets, device="cuda", dtype=torch.int32), perm.int(), s["inverse"]
    rows = s["rows"].double()
    picked = rows[torch.where(held, inv, 0).reshape(-1)].reshape(*inv.shape, -1)
    weight = held.double()
    if op == "dispatch":
        return torch.matmul(weight[:, None], picked)[:, 0]
    weight = weight * s["weights"].double()
    if not back:
        return torch.matmul(weight[:, None], picked)[:, 0]
    dout = s["grad_out"].double()
    grad_rows = torch.zeros_like(rows)
    token = torch.arange(inv.shape[0], device="cuda")[:, None].expand_as(inv)[held]
    grad_rows[inv[held]] = weight[held][:, None] * dout[token]
    return grad_rows, torch.matmul(picked, dout[:, :, None])[..., 0] * held
