"""The operators around a block's quantized products: routing tokens to experts, products of 8-bit
integers (plain and by expert), the weighted sum of the experts' rows, and the norms before and after
a block with its gate and residual scale.  Each is given in its plain form (elementary tensor
operations in 32 bits) and as the library's own entry points (`own`), over cases a model's serving and
training meet: single tokens, ragged batches, whole prompts."""
import math

import torch

own = False

DEV = "cuda"
F32_MAX = torch.finfo(torch.float32).max
F32_TINY = torch.finfo(torch.float32).tiny
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases ---------------------------------------------------------------------------------------
def _route(T, E, k, score, bias=False, groups=1, group_k=1, group_sum=False, renorm=False, scale=1.0, dtype="f32",
           masked=False, train=False):
    return dict(op="route", T=T, E=E, k=k, score=score, bias=bias, groups=groups, group_k=group_k, group_sum=group_sum,
                renorm=renorm, scale=scale, dtype=dtype, masked=masked, train=train)


def _product(M, N, K, x="bf16", out="bf16"):
    return dict(op="product", M=M, N=N, K=K, x=x, out=out)


def _experts(T, k, E, N, K, skew=1.1, out="bf16"):
    return dict(op="experts", T=T, k=k, E=E, N=N, K=K, skew=skew, out=out)


def _combine(T, k, D, dtype="bf16", train=False):
    return dict(op="combine", T=T, k=k, D=D, dtype=dtype, train=train)


def _norm(T, D, x="bf16", y="bf16", post=True, pre=True, gate="channel", one_plus=False, alpha=1.0, train=False):
    return dict(op="norm", T=T, D=D, x=x, y=y, post=post, pre=pre, gate=gate, one_plus=one_plus, alpha=alpha, train=train)


def listed():
    cases = []

    def add(name, case):
        case["name"] = name
        cases.append(case)

    # one generated token asks for its experts: latency only
    add("route_token", _route(1, 64, 8, "softmax", renorm=True))
    # a prompt's tokens over many experts: sigmoid scores, balance bias, four of eight groups
    add("route_prompt", _route(16384, 256, 8, "sigmoid", bias=True, groups=8, group_k=4, group_sum=True, renorm=True, scale=2.5))
    # a training step's routing with its gradient: softmax scores, a number of experts that is no power of two, padded tokens
    add("route_train", _route(8191, 160, 6, "softmax", groups=8, group_k=3, dtype="bf16", masked=True, train=True, scale=16.0))
    # one generated token through a feed-forward weight: the weight's bytes count
    add("product_token", _product(1, 14336, 4096))
    # a small ragged batch of generated tokens, the way back down
    add("product_batch", _product(37, 4096, 14336))
    # a prompt through the same weight: matrix rate
    add("product_prompt", _product(8192, 14336, 4096))
    # a few generated tokens through their experts: every chosen expert's weight is read once
    add("experts_tokens", _experts(8, 8, 64, 1536, 4096))
    # a prompt through the experts, with unequal loads
    add("experts_prompt", _experts(4096, 8, 64, 1536, 4096))
    # a few tokens gather their experts' rows
    add("combine_tokens", _combine(5, 8, 4096))
    # a training step's weighted sum with its gradients
    add("combine_train", _combine(4096, 8, 4096, train=True))
    # one generated token between two blocks: latency only
    add("norm_token", _norm(1, 4096))
    # a training step's norms, gate and residual between two blocks, with all gradients
    add("norm_train", _norm(8192, 4096, train=True, alpha=0.5))
    return cases


def draw(rng):
    def size(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))) / step)) * step)

    op = rng.choice(["route", "route", "product", "product", "experts", "combine", "norm", "norm"])
    if op == "route":
        k = rng.choice([1, 2, 4, 6, 8, 10])
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, -(-k // groups)), 384 // groups)
        group_k = rng.randint(1, groups)
        while group_k * (E // groups) < k:
            group_k += 1
        score = rng.choice(["softmax", "sigmoid"])
        return _route(size(1, 16384), E, k, score, bias=rng.random() < 0.5, groups=groups, group_k=group_k,
                      group_sum=rng.random() < 0.5, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                      dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.3, train=rng.random() < 0.4)
    if op == "product":
        return _product(size(1, 8192), size(64, 14336), size(64, 4096, 16), x=rng.choice(["bf16", "bf16", "f32"]),
                        out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "experts":
        E = rng.choice([4, 8, 16, 60, 64, 128])
        k = rng.choice([1, 2, 4])
        return _experts(size(1, 4096), k, E, size(64, 1536), size(64, 2048, 16), skew=rng.choice([0.0, 0.7, 1.1]),
                        out=rng.choice(["bf16", "f32"]))
    if op == "combine":
        return _combine(size(1, 4096), rng.choice([1, 2, 4, 6, 8]), size(64, 8192, 8), dtype=rng.choice(["bf16", "f32"]),
                        train=rng.random() < 0.5)
    post = rng.random() < 0.7
    return _norm(size(1, 8192), size(64, 8192, 8), x=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "bf16", "f32"]),
                 post=post, pre=rng.random() < 0.8, gate=rng.choice(["none", "channel", "token"]),
                 one_plus=rng.random() < 0.4, alpha=rng.choice([1.0, 0.5, 0.22]), train=rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    s = dict(case)
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        s["logits"] = normal(T, E, std=1.5, dtype=DTYPES[case["dtype"]])
        if case["masked"]:  # padded tokens have no expert; some experts are closed to some tokens
            closed = (uniform(T, E) < 0.1) | (uniform(T, 1) < 0.05)
            s["logits"] = s["logits"].masked_fill(closed, -math.inf)
        # a balance bias moves by one small step a training step
        s["bias_values"] = torch.round(normal(E, std=20.0)) * 1e-3 if case["bias"] else None
        if case["train"]:
            s["dweights"] = normal(T, case["k"])
    elif op == "product":
        s["x_values"] = normal(case["M"], case["K"], dtype=DTYPES[case["x"]])
        s["w"], s["w_scales"] = _plain_quantize(normal(case["N"], case["K"], std=0.02))
    elif op == "experts":
        T, k, E = case["T"], case["k"], case["E"]
        s["x_values"] = normal(T, case["K"], dtype=torch.bfloat16)
        w = [_plain_quantize(normal(case["N"], case["K"], std=0.02)) for _ in range(E)]
        s["w"], s["w_scales"] = torch.cat([a for a, _ in w]), torch.cat([b for _, b in w])
        # loads fall off as a power of the expert's rank; a token's k experts differ
        load = torch.arange(1, E + 1, device=DEV).float().pow(-case["skew"])
        load = load[torch.randperm(E, generator=g, device=DEV)]
        ids = torch.multinomial(load.expand(T, E), k, generator=g).to(torch.int32)
        s["offsets"], s["rows"], s["pos"] = _plain_plan(ids, E)
    elif op == "combine":
        T, k, D = case["T"], case["k"], case["D"]
        dt = DTYPES[case["dtype"]]
        s["y"] = normal(T * k, D, dtype=dt)
        ids = torch.randint(0, 64, (T, k), generator=g, device=DEV, dtype=torch.int32)
        s["offsets"], s["rows"], s["pos"] = _plain_plan(ids, 64)
        s["weights"] = torch.softmax(normal(T, k), dim=1)
        if case["train"]:
            s["dout"] = normal(T, D, dtype=dt)
    else:
        T, D = case["T"], case["D"]
        xt, yt = DTYPES[case["x"]], DTYPES[case["y"]]
        s["x_values"], s["y_values"] = normal(T, D, std=2.0, dtype=xt), normal(T, D, dtype=yt)
        center = 0.0 if case["one_plus"] else 1.0
        s["w_post"] = normal(D, std=0.2, mean=center) if case["post"] else None
        s["w_pre"] = normal(D, std=0.2, mean=center) if case["pre"] else None
        s["gate_values"] = {"none": lambda: None, "channel": lambda: normal(D, std=0.3, mean=0.5),
                            "token": lambda: normal(T, D, std=0.3, mean=0.5, dtype=yt)}[case["gate"]]()
        if case["train"]:
            s["dx_out"] = normal(T, D, dtype=xt)
            s["dn"] = normal(T, D, dtype=yt) if case["pre"] else None
    return s


# ---- plain forms ---------------------------------------------------------------------------------
def _plain_quantize(x):
    """Rows to 8-bit integers: scale amax / 127, values x / scale to the nearest."""
    x = x.float()
    scale = x.abs().amax(dim=1) / 127.0
    live = scale >= F32_TINY
    scale = torch.where(live, scale, torch.zeros_like(scale))
    inv = torch.where(live, 1.0 / scale, torch.zeros_like(scale))
    return torch.round(x * inv[:, None]).clamp(-127, 127).to(torch.int8), scale


def _plain_plan(ids, E):
    """Slots in order of their expert: offsets of the experts, the slot of each row, the row of each slot."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=ids.device)).to(torch.int32)
    rows = torch.where(key < E, order, torch.full_like(order, -1)).to(torch.int32)
    pos = torch.empty_like(flat)
    pos[order] = torch.where(key < E, torch.arange(flat.numel(), device=ids.device), torch.full_like(flat, -1))
    return offsets, rows, pos.to(torch.int32).reshape(ids.shape)


def _plain_scores(logits, score):
    l = logits.float()
    open_ = ~(torch.isnan(l) | (l == -math.inf))
    l = torch.where(open_, l, torch.full_like(l, -math.inf)).clamp(max=F32_MAX)
    if score == "sigmoid":
        return torch.where(open_, 1.0 / (1.0 + torch.exp(-l)), torch.zeros_like(l)), open_
    top = l.amax(dim=1, keepdim=True)
    e = torch.where(open_, torch.exp(l - top), torch.zeros_like(l))
    total = torch.nn.functional.pad(e, (0, (1 << (l.shape[1] - 1).bit_length()) - l.shape[1]))
    while total.shape[1] > 1:  # neighbours first: a sum of one order
        total = total[:, 0::2] + total[:, 1::2]
    return torch.where(open_, e / total, torch.zeros_like(e)), open_


def _plain_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    scores, open_ = _plain_scores(s["logits"], s["score"])
    key = scores if s["bias_values"] is None else scores + s["bias_values"]
    key = torch.where(open_, key, torch.full_like(key, -math.inf))
    if s["group_k"] < G:
        per = key.view(T, G, E // G)
        best = torch.sort(per, dim=2, descending=True).values
        value = best[:, :, 0]
        if s["group_sum"] and E // G > 1:
            value = value + torch.where(best[:, :, 1] == -math.inf, torch.zeros_like(value), best[:, :, 1])
        keep = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :s["group_k"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, keep, True)
        key = torch.where(kept[:, :, None], per, torch.full_like(per, -math.inf)).reshape(T, E)
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    key, ids = key[:, :k], ids[:, :k]
    chosen = key != -math.inf
    picked = torch.where(chosen, scores.gather(1, ids), torch.zeros_like(key))
    ids = torch.where(chosen, ids, torch.full_like(ids, -1))
    weights = picked / (picked.sum(dim=1, keepdim=True) + 1e-20) if s["renorm"] else picked
    return ids.to(torch.int32), weights * s["scale"]


def _plain_route_backward(s, ids):
    scores, _ = _plain_scores(s["logits"], s["score"])
    chosen = ids >= 0
    at = ids.clamp(min=0).long()
    picked = torch.where(chosen, scores.gather(1, at), torch.zeros_like(s["dweights"]))
    dw = torch.where(chosen, s["dweights"], torch.zeros_like(s["dweights"])) * s["scale"]
    if s["renorm"]:
        total = picked.sum(dim=1, keepdim=True) + 1e-20
        dw = (dw - (dw * picked).sum(dim=1, keepdim=True) / total) / total
        dw = torch.where(chosen, dw, torch.zeros_like(dw))
    ds = torch.zeros_like(scores).scatter_add_(1, at, dw)
    if s["score"] == "sigmoid":
        return (ds * scores * (1.0 - scores)).to(s["logits"].dtype)
    return (scores * (ds - (dw * picked).sum(dim=1, keepdim=True))).to(s["logits"].dtype)


def _plain_product(s):
    q, scale = _plain_quantize(s["x_values"])
    c = (q.float() @ s["w"].float().t()) * scale[:, None] * s["w_scales"]
    return c.to(DTYPES[s["out"]])


def _plain_experts(s):
    q, scale = _plain_quantize(s["x_values"])
    slots = torch.div(s["rows"], s["k"], rounding_mode="floor").long()
    out = torch.empty(slots.numel(), s["N"], dtype=DTYPES[s["out"]], device=q.device)
    bounds = s["offsets"].tolist()
    for e in range(s["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            w = s["w"][e * s["N"]:(e + 1) * s["N"]].float()
            c = (q[slots[lo:hi]].float() @ w.t()) * scale[slots[lo:hi], None] * s["w_scales"][e * s["N"]:(e + 1) * s["N"]]
            out[lo:hi] = c.to(out.dtype)
    return out


def _plain_combine(s):
    rows = s["y"][s["pos"].long()].float()
    out = (rows * s["weights"][:, :, None]).sum(dim=1).to(s["y"].dtype)
    if not s["train"]:
        return out
    dout = s["dout"].float()
    dweights = (rows * dout[:, None, :]).sum(dim=2)
    dy = torch.empty_like(s["y"])
    dy[s["pos"].long()] = (dout[:, None, :] * s["weights"][:, :, None]).to(dy.dtype)
    return out, dy, dweights


def _plain_norm(s):
    x, y, alpha, eps = s["x_values"].float(), s["y_values"].float(), s["alpha"], 1e-6
    shift = 1.0 if s["one_plus"] else 0.0
    gate = None if s["gate_values"] is None else s["gate_values"].float()
    yhat, p, r_post, r_pre = y, y, None, None
    if s["w_post"] is not None:
        w_post = s["w_post"] + shift
        r_post = 1.0 / torch.sqrt((y * y).mean(dim=1) + eps)
        yhat = y * r_post[:, None]
        p = yhat * w_post
    x1 = x + alpha * (p if gate is None else gate * p)
    out = {"x": x1.to(s["x_values"].dtype)}
    if s["w_pre"] is not None:
        w_pre = s["w_pre"] + shift
        r_pre = 1.0 / torch.sqrt((x1 * x1).mean(dim=1) + eps)
        xhat = x1 * r_pre[:, None]
        out["n"] = (xhat * w_pre).to(s["y_values"].dtype)
    if not s["train"]:
        return out
    d = s["dx_out"].float()
    if s["w_pre"] is not None:
        dn = s["dn"].float()
        out["dw_pre"] = (dn * xhat).sum(dim=0)
        t = dn * w_pre
        d = d + r_pre[:, None] * (t - xhat * (t * xhat).mean(dim=1, keepdim=True))
    out["dx"] = d.to(s["x_values"].dtype)
    dp = alpha * d if gate is None else alpha * d * gate
    if gate is not None:
        dgate = alpha * d * p
        out["dgate"] = dgate.sum(dim=0) if gate.dim() == 1 else dgate.to(s["gate_values"].dtype)
    if s["w_post"] is not None:
        out["dw_post"] = (dp * yhat).sum(dim=0)
        t = dp * w_post
        dp = r_post[:, None] * (t - yhat * (t * yhat).mean(dim=1, keepdim=True))
    out["dy"] = dp.to(s["y_values"].dtype)
    return out


# ---- the library's entry points --------------------------------------------------------------------
def _own_route(nv, s):
    flags = nv.NVFP4_ROUTE_SIGMOID if s["score"] == "sigmoid" else 0
    flags |= nv.NVFP4_ROUTE_RENORM if s["renorm"] else 0
    flags |= nv.NVFP4_ROUTE_GROUP_SUM2 if s["group_sum"] else 0
    ids, weights, plan = nv.nvfp4_moe_route(s["logits"], s["k"], flags=flags, bias=s["bias_values"], num_groups=s["groups"],
                                            group_top_k=s["group_k"], scale=s["scale"])
    out = {"ids": ids, "weights": weights, "offsets": plan.offsets, "rows": plan.rows, "pos": plan.pos}
    if s["train"]:
        out["dlogits"] = nv.nvfp4_moe_route_backward(s["logits"], ids, s["dweights"], flags=flags, scale=s["scale"])
    return out


def _own(s):
    import nvfp4_bit_block_quantize_amd as nv
    op = s["op"]
    if op == "route":
        return _own_route(nv, s)
    if op in ("product", "experts"):
        w = nv.Int8Tensor(s["w"], s["w_scales"], s["N"], s["K"], s["E"] if op == "experts" else 1)
        q = nv.nvfp4_int8_quantize(s["x_values"])
        plan = nv.MoEPlan(s["offsets"], s["rows"], s["pos"]) if op == "experts" else None
        return nv.nvfp4_int8_gemm(q, w, out_dtype=DTYPES[s["out"]], plan=plan, gather=plan is not None)
    if op == "combine":
        plan = nv.MoEPlan(s["offsets"], s["rows"], s["pos"])
        out = nv.nvfp4_moe_combine(s["y"], plan, weights=s["weights"])
        if not s["train"]:
            return out
        dy, dweights = nv.nvfp4_moe_combine_backward(s["dout"], s["y"], plan, s["weights"])
        return out, dy, dweights
    flags = nv.NVFP4_NORM_ONE_PLUS if s["one_plus"] else 0
    f = nv.nvfp4_block_norm(s["x_values"], s["y_values"], w_post=s["w_post"], gate=s["gate_values"], w_pre=s["w_pre"],
                            alpha=s["alpha"], eps=1e-6, flags=flags)
    out = {"x": f.x}
    if s["w_pre"] is not None:
        out["n"] = f.n
    if s["train"]:
        b = nv.nvfp4_block_norm_backward(s["dx_out"], s["dn"], s["x_values"], s["y_values"], f.rstd_post, f.rstd_pre,
                                         w_post=s["w_post"], gate=s["gate_values"], w_pre=s["w_pre"], alpha=s["alpha"], flags=flags)
        for name in ("dw_pre", "dx", "dgate", "dw_post", "dy"):
            if getattr(b, name) is not None:
                out[name] = getattr(b, name)
    return out


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "route":
        ids, weights = _plain_route(state)
        offsets, rows, pos = _plain_plan(ids, state["E"])
        out = {"ids": ids, "weights": weights, "offsets": offsets, "rows": rows, "pos": pos}
        if state["train"]:
            out["dlogits"] = _plain_route_backward(state, ids)
        return out
    return {"product": _plain_product, "experts": _plain_experts, "combine": _plain_combine, "norm": _plain_norm}[op](state)


# ---- what a pass cannot do without -------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        es = size[case["dtype"]]
        b = T * E * es + T * k * 16 + (E + 1) * 4 + (4 * E if case["bias"] else 0)
        f = T * E * (6 + k)
        if case["train"]:
            b += T * k * 4 + 2 * T * E * es
            f += 8 * T * E
        return {"bytes": b, "flops": f}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * size[case["x"]] + N * K + 4 * N + M * N * size[case["out"]], "flops": 2 * M * N * K}
    if op == "experts":
        T, k, E, N, K = case["T"], case["k"], case["E"], case["N"], case["K"]
        used = min(E, T * k)  # at most so many experts' weights are read
        return {"bytes": T * K * 2 + used * N * (K + 4) + T * k * (N * size[case["out"]] + 4), "flops": 2 * T * k * N * K}
    if op == "combine":
        T, k, D = case["T"], case["k"], case["D"]
        es = size[case["dtype"]]
        b, f = (T * k * D + T * D) * es + T * k * 8, 2 * T * k * D
        if case["train"]:
            b, f = b + (2 * T * k * D + T * D) * es + T * k * 12, f + 3 * T * k * D
        return {"bytes": b, "flops": f}
    T, D = case["T"], case["D"]
    xs, ys = size[case["x"]], size[case["y"]]
    gate = T * D * ys if case["gate"] == "token" else 4 * D if case["gate"] == "channel" else 0
    n = T * D * ys if case["pre"] else 0
    b, f = T * D * (2 * xs + ys) + n + gate + 8 * D, 14 * T * D
    if case["train"]:
        b, f = b + T * D * (3 * xs + 2 * ys) + n + 2 * gate + 12 * D, f + 40 * T * D
    return {"bytes": b, "flops": f}


# ---- the definition in 64 bits -------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "product": _exact_product, "experts": _exact_experts, "combine": _exact_combine,
            "norm": _exact_norm}[case["op"]](s)


def _exact_scores(logits, kind, dtype):
    """Scores in `dtype`: 32 bits for the keys that decide the choice, 64 for the values."""
    v = torch.nan_to_num(logits.to(dtype), nan=-math.inf, posinf=F32_MAX, neginf=-math.inf)
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    m = v.max(dim=1, keepdim=True).values
    e = torch.exp(v - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    width = 1
    while width < v.shape[1]:
        width *= 2
    tree = torch.zeros(v.shape[0], width, dtype=dtype, device=v.device)
    tree[:, :v.shape[1]] = e
    while tree.shape[1] > 1:
        tree = tree.unflatten(1, (-1, 2))
        tree = tree[..., 0] + tree[..., 1]
    return e / torch.where(tree == 0, torch.ones_like(tree), tree)


def _exact_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    shut = torch.isnan(s["logits"]) | (s["logits"] == -math.inf)
    key = _exact_scores(s["logits"], s["score"], torch.float32)
    if s["bias_values"] is not None:
        key = key + s["bias_values"]
    key[shut] = -math.inf
    if s["group_k"] < G:
        two = key.view(T, G, -1).sort(dim=2, descending=True).values[:, :, :2]
        total = two[:, :, 0].clone()
        if s["group_sum"] and two.shape[2] == 2:
            total += two[:, :, 1].nan_to_num(neginf=0.0)
        # a group's place: how many are before it
        ahead = (total[:, None, :] > total[:, :, None]) | ((total[:, None, :] == total[:, :, None])
                                                           & torch.ones(G, G, device=key.device).tril(-1).bool())
        out_of_it = ahead.sum(dim=2) >= s["group_k"]
        key = key.masked_fill(out_of_it.repeat_interleave(E // G, dim=1), -math.inf)
    place = key.neg().sort(dim=1, stable=True)
    ids = place.indices[:, :k]
    none = place.values[:, :k] == math.inf
    score = _exact_scores(s["logits"], s["score"], torch.float64)
    p = score.gather(1, ids).masked_fill(none, 0.0)
    w = p * s["scale"]
    if s["renorm"]:
        w = w / (p.sum(dim=1, keepdim=True) + 1e-20)
    out = {"ids": None, "weights": w, "offsets": None, "rows": None, "pos": None}
    if s["train"]:
        g = s["dweights"].double().masked_fill(none, 0.0) * s["scale"]
        if s["renorm"]:
            t = p.sum(dim=1, keepdim=True) + 1e-20
            g = (g / t - (g * p).sum(dim=1, keepdim=True) / t ** 2).masked_fill(none, 0.0)
        ds = torch.zeros_like(score).scatter_add_(1, ids, g)
        if s["score"] == "sigmoid":
            out["dlogits"] = (ds * (score - score ** 2)).masked_fill(shut, 0.0)
        else:
            out["dlogits"] = (score * ds - score * (score * ds).sum(dim=1, keepdim=True)).masked_fill(shut, 0.0)
    return out


def _exact_int8(x):
    """The 8-bit rows by the definition: scale and reciprocal are 32-bit numbers."""
    v = x.double()
    scale = (v.abs().max(dim=1).values / 127).float()
    scale[scale < F32_TINY] = 0
    inv = (1 / scale.double()).float().nan_to_num(posinf=0.0).double()
    return torch.round((v * inv[:, None]).float()).double(), scale.double()


def _exact_product(s):
    q, scale = _exact_int8(s["x_values"])
    return scale[:, None] * (q @ s["w"].double().t()) * s["w_scales"].double()[None, :]


def _exact_experts(s):
    q, scale = _exact_int8(s["x_values"])
    token = torch.div(s["rows"].long(), s["k"], rounding_mode="floor")
    w, ws = s["w"].view(s["E"], s["N"], s["K"]), s["w_scales"].view(s["E"], s["N"]).double()
    parts, ends = [], s["offsets"].cpu().numpy()
    for e in range(s["E"]):
        t = token[int(ends[e]):int(ends[e + 1])]
        parts.append(scale[t, None] * (q[t] @ w[e].double().t()) * ws[e])
    return torch.cat(parts)


def _exact_combine(s):
    w = s["weights"].double()
    T, k = w.shape
    out = torch.zeros(T, s["D"], dtype=torch.float64, device=w.device)
    dweights = torch.zeros_like(w)
    dy = torch.zeros(T * k, s["D"], dtype=torch.float64, device=w.device)
    for j in range(k):
        at = s["pos"][:, j].long()
        row = s["y"][at].double()
        out += w[:, j, None] * row
        if s["train"]:
            dweights[:, j] = (row * s["dout"].double()).sum(dim=1)
            dy[at] = w[:, j, None] * s["dout"].double()
    return (out, dy, dweights) if s["train"] else out


def _exact_norm(s):
    """The forward in 64 bits, and its gradients by differentiation."""
    leaves = {}

    def leaf(name, t):
        leaves[name] = t.double().requires_grad_(s["train"])
        return leaves[name]

    with torch.enable_grad():
        x, y = leaf("dx", s["x_values"]), leaf("dy", s["y_values"])
        shift = 1 if s["one_plus"] else 0
        b = y
        if s["post"]:
            b = (y * (y.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt()) * (leaf("dw_post", s["w_post"]) + shift)
        if s["gate"] != "none":
            b = b * leaf("dgate", s["gate_values"])
        x1 = x + s["alpha"] * b
        out = {"x": x1.detach()}
        loss = None
        if s["pre"]:
            n = x1 * (x1.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt() * (leaf("dw_pre", s["w_pre"]) + shift)
            out["n"] = n.detach()
        if s["train"]:
            loss = (x1 * s["dx_out"].double()).sum()
            if s["pre"]:
                loss = loss + (n * s["dn"].double()).sum()
            names = [n for n in ("dw_pre", "dx", "dgate", "dw_post", "dy") if n in leaves]
            out.update(zip(names, torch.autograd.grad(loss, [leaves[n] for n in names])))
    return out
