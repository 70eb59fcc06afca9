"""The routed-experts operators, as they are measured: their cases, inputs, plain forms and the calls of this package.

Three operators of a mixture-of-experts feed-forward layer:

  route      scores of T tokens over E experts (softmax or sigmoid), a selection bias, expert groups, the k best
             experts of each token and their renormalised weights; and the gradient of the logits
  dispatch   the plan (rows sorted by expert, offsets, the map back), the gather of token rows into that order, the
             weighted combination back to tokens, and the gradients of both
  experts    out = act(A[e] @ B[e] + bias[e]) for every expert's run of rows, the backward epilogue
             dX = (G @ W[e]^T) * act'(X), and the weight and bias gradients

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits (selection keys in 64 bits, since
a choice between two experts is a value next to a border); with ``own`` true it calls this package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases

def _route(name, T, E, k, dtype, score, step, bias=False, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0,
           masked=0.0):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "score": score, "step": step,
            "bias": bias, "groups": groups, "top_groups": top_groups, "group_top": group_top, "renorm": renorm,
            "scale": scale, "masked": masked}


def _plan(name, T, E, k, dropped=0.0):
    return {"name": name, "op": "plan", "T": T, "E": E, "k": k, "dropped": dropped}


def _move(name, T, E, k, H, dtype, step, residual=False):
    return {"name": name, "op": "move", "T": T, "E": E, "k": k, "H": H, "dtype": dtype, "step": step,
            "residual": residual}


def _experts(name, T, E, k, K, N, dtype, act, step, indexed=True):
    return {"name": name, "op": "experts", "T": T, "E": E, "k": k, "K": K, "N": N, "dtype": dtype, "act": act,
            "step": step, "indexed": indexed}


def listed():
    return [
        # one decode step of a small serving batch: the router's launch latency
        _route("route_decode", 32, 64, 6, "bf16", "softmax", "forward"),
        # a prompt through a router with a balance bias and node-limited groups
        _route("route_groups", 4096, 256, 8, "f32", "sigmoid", "forward", bias=True, groups=8, top_groups=4,
               group_top=2, scale=2.5),
        # a training step's router, forward and backward, some experts masked for some tokens
        _route("route_train", 16384, 64, 6, "bf16", "softmax", "train", masked=0.02),
        # the plan of a long training batch, some of its slots dropped
        _plan("plan_long", 65536, 256, 8, dropped=0.05),
        # a decode step's plan and the combination that ends it, with the residual
        _move("dispatch_decode", 32, 64, 6, 2048, "bf16", "decode", residual=True),
        # a training step's gather and combination with their gradients
        _move("move_train", 8192, 8, 2, 4096, "bf16", "train"),
        # decode: few rows spread over many small experts, gated, rows read through the plan
        _experts("experts_decode", 32, 64, 6, 2048, 1408, "bf16", "glu", "forward"),
        # a single token through two large experts
        _experts("experts_token", 1, 8, 2, 4096, 14336, "f16", "gelu_tanh", "forward"),
        # a prompt's tokens through many small experts, gated
        _experts("experts_prompt", 4096, 64, 6, 2048, 1408, "bf16", "glu", "forward"),
        # odd sizes throughout, with the gradients
        _experts("experts_ragged", 1021, 12, 3, 1537, 3071, "bf16", "relu", "train", indexed=False),
        # 32-bit weights: a small model's training step
        _experts("experts_f32", 1000, 6, 2, 768, 1000, "f32", "gelu_tanh", "train", indexed=False),
        # a training step of large experts: forward with the saved pre-activation, backward, weight gradients
        _experts("experts_train", 8192, 8, 2, 4096, 14336, "bf16", "gelu_tanh", "train", indexed=False),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm, odd ones among them."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(("route", "plan", "move", "experts", "experts"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * _log(rng, 2, 256 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, top_groups * (E // groups)))
        T = _log(rng, 1, 16384)
        # one renormalised weight is 1 whatever the logits, so its gradient is zero: no case of it
        return _route("", T, E, k, dtype, rng.choice(("softmax", "sigmoid")), rng.choice(("forward", "train")),
                      bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, group_top=rng.choice((1, 2)),
                      renorm=k > 1 and rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                      masked=0.05 if T >= 64 and rng.random() < 0.5 else 0.0)
    E = _log(rng, 2, 256)
    k = rng.randint(1, min(8, E))
    if op == "plan":
        return _plan("", _log(rng, 1, 65536), E, k, dropped=rng.choice((0.0, 0.1)))
    if op == "move":
        H = _log(rng, 64, 8192)
        T = _log(rng, 1, max(1, min(16384, 200_000_000 // (H * k))))
        return _move("", T, E, k, H, dtype, rng.choice(("decode", "train")), residual=rng.random() < 0.5)
    K, N = _log(rng, 64, 4096), _log(rng, 64, 8192)
    E = _log(rng, 2, max(2, min(64, 400_000_000 // (K * N))))
    k = rng.randint(1, min(6, E))
    step = rng.choice(("forward", "train"))
    T = _log(rng, 1, max(1, min(8192, int(1e12 if dtype == "f32" else 4e12) // (6 * K * N * k))))
    act = rng.choice(("none", "relu", "gelu_tanh", "glu"))
    return _experts("", T, E, k, K, N, dtype, act, step, indexed=step == "forward" and rng.random() < 0.7)


# ----------------------------------------------------------------- inputs

def _pick_experts(g, T, E, k):
    """k different experts of each token, some experts more popular than others: (T,k) int32."""
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    return torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()


def _plan_of(experts, E):
    """(offsets (E+1,), token_of_row (T*k,), row_of_slot (T,k)), int32: the slots sorted by expert, slots of one expert
    in token order; a slot without an expert (-1) has row -1, and the rows left at the end have token -1."""
    T, k = experts.shape
    flat = experts.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.long, device=key.device).scatter_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rank = torch.empty_like(order)
    rank[order] = torch.arange(order.numel(), device=order.device)
    row_of_slot = torch.where(flat < 0, torch.full_like(rank, -1), rank).view(T, k)
    live = torch.arange(order.numel(), device=order.device) < offsets[-1]
    token_of_row = torch.where(live, order // k, torch.full_like(order, -1))
    return offsets.to(torch.int32), token_of_row.to(torch.int32), row_of_slot.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0, dtype=None):
        x = torch.empty(*shape, dtype=torch.float32, device=dev).normal_(0.0, std, generator=g)
        return x if dtype is None else x.to(dtype)

    T, E, k = case["T"], case["E"], case["k"]
    s = {"case": dict(case)}
    if case["op"] == "route":
        dt = DTYPES[case["dtype"]]
        logits = normal(T, E, std=1.5)
        if case["masked"]:
            logits.masked_fill_(torch.rand(T, E, generator=g, device=dev) < case["masked"], -math.inf)
            logits[:: 97] = torch.where(torch.rand(len(logits[::97]), 1, generator=g, device=dev) < 0.5, -math.inf,
                                        logits[::97])  # tokens for which no expert is left
        s["logits"] = logits.to(dt)
        s["bias"] = normal(E, std=0.1) if case["bias"] else None
        if case["step"] == "train":
            s["dweights"] = normal(T, k)
        return s
    experts = _pick_experts(g, T, E, k)
    if case["op"] == "plan":
        if case["dropped"]:
            experts.masked_fill_(torch.rand(T, k, generator=g, device=dev) < case["dropped"], -1)
        s["experts"] = experts
        return s
    offsets, token_of_row, row_of_slot = _plan_of(experts, E)
    S = T * k
    dt = DTYPES[case["dtype"]]
    s |= {"offsets": offsets, "token_of_row": token_of_row, "row_of_slot": row_of_slot}
    if case["op"] == "move":
        H = case["H"]
        s["experts"] = experts
        w = torch.rand(T, k, generator=g, device=dev) + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        s["rows"] = normal(S, H, dtype=dt)
        s["residual"] = normal(T, H, dtype=dt) if case["residual"] else None
        if case["step"] == "train":
            s["x"] = normal(T, H, dtype=dt)
            s["dout"] = normal(T, H, dtype=dt)
            s["drows"] = normal(S, H, dtype=dt)
        return s
    K, N = case["K"], case["N"]
    s["cap"] = int((offsets[1:] - offsets[:-1]).max())  # rows of the fullest expert, for the plain form's padding
    s["A"] = normal(T if case["indexed"] else S, K, dtype=dt)
    s["B"] = torch.empty(E, K, N, dtype=dt, device=dev)
    for e in range(E):  # one expert at a time: the 32-bit draws of all of them need not exist at once
        s["B"][e] = normal(K, N, std=K ** -0.5)
    s["bias"] = normal(E, N, std=0.3, dtype=dt)
    s["Y"] = normal(S, N, dtype=dt) if case["act"] == "glu" else None
    if case["step"] == "train":
        # the backward epilogue of a layer whose output meets the weight of the next product, (E, N, K)
        s["W"] = torch.empty(E, N, K, dtype=dt, device=dev)
        for e in range(E):
            s["W"][e] = normal(N, K, std=N ** -0.5)
        s["G"] = normal(S, K, dtype=dt)       # the gradient at that product's output
        s["X"] = normal(S, N, dtype=dt)       # the saved pre-activation
        s["D"] = normal(S, N, std=0.5, dtype=dt)  # the gradient at this layer's product
    return s


# ------------------------------------------------------------ plain forms

def _scores(x, kind):
    """Scores in x's precision; a masked expert (-inf) scores 0, a row of them 0 throughout."""
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    z = e.sum(1, keepdim=True)
    return e / torch.where(z > 0, z, torch.ones_like(z))


def _first(key, n):
    """Indices of the n largest keys of each row, ties to the lowest index."""
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :n]


def _plain_route(s):
    c, logits, bias = s["case"], s["logits"], s["bias"]
    T, E = logits.shape
    G, k = c["groups"], c["k"]
    x = logits.double()
    live = x > -math.inf
    # with neither a bias nor sums over a group the order of the scores is that of the logits
    score = _scores(x, c["score"])
    key = (x if bias is None else score + bias.double()).masked_fill(~live, -math.inf)
    if G > 1:
        gkey = key if c["group_top"] == 1 else (score if bias is None else key).masked_fill(~live, -math.inf)
        per = gkey.view(T, G, E // G)
        if c["group_top"] == 1:
            of = per.amax(2)
        else:
            two = torch.sort(per, dim=2, descending=True).values[:, :, :2]
            of = torch.where(torch.isinf(two[:, :, 0]), two[:, :, 0],
                             torch.where(torch.isinf(two), torch.zeros_like(two), two).sum(2))
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, _first(of, c["top_groups"]), True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, dim=1), -math.inf)
    sel = _first(key, k)
    ok = key.gather(1, sel) > -math.inf
    w = _scores(logits.float(), c["score"]).gather(1, sel) * ok
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return w * c["scale"], torch.where(ok, sel, torch.full_like(sel, -1)).to(torch.int32)


def _plain_route_bwd(s, experts):
    c, logits = s["case"], s["logits"]
    x = logits.float()
    score = _scores(x, c["score"])
    ok = experts >= 0
    at = experts.clamp(min=0).long()
    picked = score.gather(1, at) * ok
    dw = s["dweights"] * c["scale"] * ok
    if c["renorm"]:
        total = picked.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        ds = (dw - (dw * picked).sum(1, keepdim=True) / total) / total * ok
    else:
        ds = dw
    dscore = torch.zeros_like(x).scatter_add_(1, at, ds)
    if c["score"] == "sigmoid":
        dx = dscore * score * (1.0 - score)
    else:
        dx = score * (dscore - (dscore * score).sum(1, keepdim=True))
    return dx.to(logits.dtype)


def _plain_combine(rows, row_of_slot, weights, residual):
    got = rows.float()[row_of_slot.clamp(min=0).long()] * (row_of_slot >= 0)[..., None]
    out = (got if weights is None else got * weights[..., None]).sum(1)
    return (out if residual is None else out + residual.float()).to(rows.dtype)


def _plain_move(s):
    c, dt = s["case"], s["rows"].dtype
    out = _plain_combine(s["rows"], s["row_of_slot"], s["weights"], s["residual"])
    if c["step"] == "decode":
        offsets, token_of_row, row_of_slot = _plan_of(s["experts"], c["E"])
        return {"offsets": offsets, "token_of_row": token_of_row, "row_of_slot": row_of_slot, "out": out}
    T, k = s["row_of_slot"].shape
    gathered = s["x"][s["token_of_row"].long()]
    at = s["row_of_slot"].long()
    d = s["dout"].float()
    drows = torch.empty_like(s["rows"])
    drows[at.reshape(-1)] = (d[:, None, :] * s["weights"][..., None]).to(dt).view(T * k, -1)
    dweights = (s["rows"].float()[at] * d[:, None, :]).sum(2)
    return {"out": out, "gathered": gathered, "drows": drows, "dweights": dweights,
            "dx": _plain_combine(s["drows"], s["row_of_slot"], None, None)}


def _act(x, y, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x + x * y if act == "glu" else x


def _act_grad(x, y, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * x * x)
    return 1.0 + y if act == "glu" else torch.ones_like(x)


def _padded(s, rows):
    """The rows of every expert, padded with zeros to the fullest one's: (E, cap, width) in 32 bits."""
    at = s["offsets"][:-1, None].long() + torch.arange(s["cap"], device=rows.device)
    live = at < s["offsets"][1:, None]
    return rows.float()[torch.where(live, at, torch.zeros_like(at))] * live[..., None]


def _unpadded(s, x):
    """(S, width): every expert's rows of x (E, cap, width) in their order."""
    S = s["token_of_row"].numel()
    r = torch.arange(S, device=x.device)
    e = (r[:, None] >= s["offsets"][None, 1:]).sum(1)
    return x[e, r - s["offsets"].long()[e]]


def _plain_experts(s):
    c = s["case"]
    dt, act = s["B"].dtype, c["act"]
    y = s["Y"].float() if s["Y"] is not None else None
    rows = s["A"][s["token_of_row"].long()] if c["indexed"] else s["A"]
    a = _padded(s, rows)
    x = _unpadded(s, torch.bmm(a, s["B"].float()) + s["bias"].float()[:, None, :])
    if c["step"] == "forward":
        return {"out": _act(x, y, act).to(dt)}
    d = _unpadded(s, torch.bmm(_padded(s, s["G"]), s["W"].float().transpose(1, 2).contiguous()))
    saved = s["X"].float()
    g = _padded(s, s["D"])
    got = {"out": _act(x, y, act).to(dt), "pre": x.to(dt), "dX": (d * _act_grad(saved, y, act)).to(dt),
           "dW": torch.bmm(a.transpose(1, 2).contiguous(), g).to(dt), "dbias": g.sum(1)}
    return got | ({"dY": (d * saved).to(dt)} if act == "glu" else {})


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    if own:
        return _own(state)
    if c["op"] == "route":
        weights, experts = _plain_route(state)
        got = {"weights": weights, "experts": experts}
        return got | ({"dlogits": _plain_route_bwd(state, experts)} if c["step"] == "train" else {})
    if c["op"] == "plan":
        offsets, token_of_row, row_of_slot = _plan_of(state["experts"], c["E"])
        return {"offsets": offsets, "token_of_row": token_of_row, "row_of_slot": row_of_slot}
    return _plain_move(state) if c["op"] == "move" else _plain_experts(state)


def _own(s):
    import activation_epilogue_amd as fl
    c = s["case"]
    if c["op"] == "route":
        how = {"score": c["score"], "renorm": c["renorm"], "scale": c["scale"]}
        weights, experts = fl.moe_route(s["logits"], c["k"], bias=s["bias"], groups=c["groups"],
                                        top_groups=c["top_groups"], group_top=c["group_top"], **how)
        got = {"weights": weights, "experts": experts}
        return got | ({"dlogits": fl.moe_route_bwd(s["logits"], experts, s["dweights"], **how)}
                      if c["step"] == "train" else {})
    if c["op"] == "plan":
        plan = fl.moe_plan(s["experts"], c["E"])
        return {"offsets": plan.offsets, "token_of_row": plan.token_of_row, "row_of_slot": plan.row_of_slot}
    if c["op"] == "move":
        if c["step"] == "decode":
            plan = fl.moe_plan(s["experts"], c["E"])
            out = fl.moe_combine(s["rows"], plan.row_of_slot, s["weights"], R=s["residual"])
            return {"offsets": plan.offsets, "token_of_row": plan.token_of_row, "row_of_slot": plan.row_of_slot,
                    "out": out}
        out = fl.moe_combine(s["rows"], s["row_of_slot"], s["weights"], R=s["residual"])
        drows, dweights = fl.moe_combine_bwd(s["dout"], s["rows"], s["row_of_slot"], s["weights"])
        return {"out": out, "gathered": fl.moe_gather(s["x"], s["token_of_row"]), "drows": drows,
                "dweights": dweights, "dx": fl.moe_combine(s["drows"], s["row_of_slot"])}
    index = s["token_of_row"] if c["indexed"] else None
    if c["step"] == "forward":
        return {"out": fl.grouped_linear(s["A"], s["B"], s["offsets"], s["bias"], s["Y"], act=c["act"], index=index)}
    out, pre = fl.grouped_linear(s["A"], s["B"], s["offsets"], s["bias"], s["Y"], act=c["act"], index=index, pre=True)
    dX, dY = fl.grouped_linear_bwd(s["G"], s["W"], s["X"], s["offsets"], s["Y"], act=c["act"])
    dW, dbias = fl.grouped_weight_grad(s["A"], s["D"], s["offsets"])
    got = {"out": out, "pre": pre, "dX": dX, "dW": dW, "dbias": dbias}
    return got | ({"dY": dY} if c["act"] == "glu" else {})


# ------------------------------------------------------------------- work

def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    S = T * k
    train = case.get("step") == "train"
    if case["op"] == "route":
        es = SIZES[case["dtype"]]
        b = T * E * es + 8 * S + (4 * E if case["bias"] else 0)
        return {"bytes": b + (T * E * es + 4 * S if train else 0), "flops": (12 if train else 6) * T * E}
    if case["op"] == "plan":
        return {"bytes": 12 * S + 4 * (E + 1), "flops": 0}
    es = SIZES[case["dtype"]]
    if case["op"] == "move":
        H = case["H"]
        row, token = S * H * es, T * H * es
        b = row + token + 8 * S + (token if case["residual"] else 0)
        b += 0 if train else 12 * S + 4 * (E + 1)  # the plan
        if train:  # gather; gradients of the combination (its rows are counted above); gradient of the gather
            b += (token + row + 4 * S) + (token + row + 4 * S) + (row + token)
        return {"bytes": b, "flops": S * H * (6 if train else 2)}
    K, N = case["K"], case["N"]
    met = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token of an even draw meets
    gate = case["act"] == "glu"
    a = (min(T, S) if case["indexed"] else S) * K
    b = es * (a + met * (K * N + N) + S * N * (2 if gate else 1)) + 4 * (E + 1) + (4 * S if case["indexed"] else 0)
    if train:  # the saved pre-activation; the backward epilogue; the weight and bias gradients
        b += es * S * N + es * (S * K + met * K * N + S * N * (4 if gate else 2)) + es * (S * N + E * K * N) + 4 * E * N
    return {"bytes": b, "flops": (6 if train else 2) * S * K * N}


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The operators' definitions in 64 bits, one expert (or one token slot) at a time."""
    op = case["op"]
    if op == "plan":  # whole numbers throughout
        return None
    s = prepare(case, seed)
    if op == "route":
        _, experts = _plain_route(s)  # which experts: whole numbers, compared as such
        x = s["logits"].double()
        z = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
        T, k = experts.shape
        weights = torch.zeros(T, k, dtype=torch.float64, device=x.device)
        for j in range(k):
            has = experts[:, j] >= 0
            weights[has, j] = z[has, experts[has, j].long()]
        raw = weights.clone()
        total = raw.sum(1)
        if case["renorm"]:
            some = total > 0
            weights[some] = raw[some] / total[some, None]
        got = {"weights": weights * case["scale"], "experts": None}
        if case["step"] == "train":
            dw = s["dweights"].double() * case["scale"] * (experts >= 0)
            back = torch.zeros_like(x)
            for j in range(k):  # d w_i / d s_j, one chosen expert j at a time
                has = experts[:, j] >= 0
                to = experts[:, j].clamp(min=0).long()
                d = dw[:, j]
                if case["renorm"]:
                    safe = torch.where(total > 0, total, torch.ones_like(total))
                    d = (d - (dw * raw).sum(1) / safe) / safe
                back[has, to[has]] += d[has]
            if case["score"] == "sigmoid":
                got["dlogits"] = back * z * (1 - z)
            else:
                got["dlogits"] = z * back - z * (z * back).sum(1, keepdim=True)
        return got
    if op == "move":
        rows, at, w = s["rows"].double(), s["row_of_slot"].long(), s["weights"].double()
        T, k = at.shape
        out = torch.zeros(T, case["H"], dtype=torch.float64, device=rows.device)
        for j in range(k):
            out += w[:, j, None] * rows[at[:, j]]
        if s["residual"] is not None:
            out += s["residual"].double()
        if case["step"] == "decode":
            return {"offsets": None, "token_of_row": None, "row_of_slot": None, "out": out}
        d = s["dout"].double()
        drows, dweights, dx = torch.zeros_like(rows), torch.zeros_like(w), torch.zeros_like(out)
        for j in range(k):
            drows[at[:, j]] = w[:, j, None] * d
            dweights[:, j] = (rows[at[:, j]] * d).sum(1)
            dx += s["drows"].double()[at[:, j]]
        return {"out": out, "gathered": s["x"].double()[s["token_of_row"].long()], "drows": drows,
                "dweights": dweights, "dx": dx}
    bounds = s["offsets"].tolist()
    S, N, K, act = case["T"] * case["k"], case["N"], case["K"], case["act"]
    wide = {"dtype": torch.float64, "device": "cuda"}
    names = {"out": (S, N)}
    if case["step"] == "train":
        names |= {"pre": (S, N), "dX": (S, N), "dW": (case["E"], K, N), "dbias": (case["E"], N)}
        names |= {"dY": (S, N)} if act == "glu" else {}
    got = {n: torch.zeros(*shape, **wide) for n, shape in names.items()}
    rows = s["A"][s["token_of_row"].long()] if case["indexed"] else s["A"]
    for e in range(case["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        a, y = rows[lo:hi].double(), s["Y"][lo:hi].double() if act == "glu" else None
        x = a @ s["B"][e].double() + s["bias"][e].double()
        got["out"][lo:hi] = _act(x, y, act)
        if case["step"] == "train":
            got["pre"][lo:hi] = x
            back = s["G"][lo:hi].double() @ s["W"][e].double().t().contiguous()
            saved = s["X"][lo:hi].double()
            got["dX"][lo:hi] = back * _act_grad(saved, y, act)
            if act == "glu":
                got["dY"][lo:hi] = back * saved
            g = s["D"][lo:hi].double()
            got["dW"][e] = a.t().contiguous() @ g
            got["dbias"][e] = g.sum(0)
    return got
