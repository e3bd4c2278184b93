"""What fine-tuning and serving a block over frozen quantized weights needs beside its products: low-rank
adapters of many requests (or experts) with their gradients, the routing's balance loss with counts and
gradient, and the gradient norm over many tensors with clipping.  Each is given in its plain form (elementary
tensor operations in 32 bits) and as the library's own entry points (`own`), over cases a model's serving and
training meet: single tokens, ragged batches, whole prompts, whole lists of gradients."""
import math

import torch

own = False

DEV = "cuda"
F32_MAX = torch.finfo(torch.float32).max
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases ---------------------------------------------------------------------------------------
def _adapter(T, K, N, R, L, none=0.0, out="bf16", train=False):
    """T tokens of many requests; a request has one of L adapters or none."""
    return dict(op="adapter", T=T, K=K, N=N, R=R, L=L, none=none, out=out, train=train, k=0)


def _experts(T, k, K, N, R, L, out="bf16"):
    """The same by expert: a routed token's k rows in the plan's order, an adapter for each expert."""
    return dict(op="adapter", T=T, K=K, N=N, R=R, L=L, none=0.0, out=out, train=False, k=k)


def _balance(T, E, k, score, sequences=1, dtype="f32", masked=False, train=True, add=False):
    return dict(op="balance", T=T, E=E, k=k, score=score, sequences=sequences, dtype=dtype, masked=masked, train=train,
                add=add)


def _clip(shapes, times, dtype="bf16", kind="two", over=3.0, clip=True):
    """`times` copies of a list of tensors (given by their numbers of elements); the norm is about `over` times
    what is allowed."""
    return dict(op="clip", shapes=",".join(str(n) for n in shapes), times=times, dtype=dtype, kind=kind, over=over, clip=clip)


def listed():
    cases = []

    def add(name, case):
        case["name"] = name
        cases.append(case)

    # one generated token of a fine-tuned model: latency only
    add("adapter_token", _adapter(1, 4096, 14336, 16, 1))
    # a batch of generated tokens, every request with an adapter of its own, a few with none
    add("adapter_batch", _adapter(48, 4096, 14336, 16, 64, none=0.1))
    # a smaller ragged batch on the way back down, adapters of a higher rank, 32-bit outputs
    add("adapter_down", _adapter(37, 14336, 4096, 64, 16, out="f32"))
    # prompts of several requests in one batch: the outputs' bytes count
    add("adapter_prompt", _adapter(8192, 4096, 14336, 16, 8, none=0.1))
    # a prompt routed to experts, an adapter for each expert
    add("adapter_experts", _experts(4096, 8, 4096, 1536, 16, 64))
    # a fine-tuning step of one adapter: forward, and gradients of the inputs and of both factors
    add("adapter_train", _adapter(8192, 4096, 14336, 16, 1, train=True))
    # a step of four tasks' adapters at once, of a higher rank, on the way back down
    add("adapter_tasks", _adapter(2047, 14336, 4096, 64, 4, none=0.05, train=True))
    # a small batch's load over the experts: loss and counts without a gradient
    add("balance_small", _balance(64, 64, 8, "softmax", train=False))
    # a training step over four sequences: sigmoid scores, gradient added to the router's
    add("balance_train", _balance(16384, 256, 8, "sigmoid", sequences=4, add=True))
    # a training step with padded tokens and closed experts, a number of experts that is no power of two
    add("balance_masked", _balance(8191, 160, 6, "softmax", dtype="bf16", masked=True))
    # the gradients of 32 layers' adapters: many small tensors
    add("clip_adapters", _clip([16 * 4096, 14336 * 16, 16 * 14336, 4096 * 16, 4096], 32, dtype="f32"))
    # the gradients of two layers' feed-forward weights and norms: memory rate
    add("clip_layers", _clip([14336 * 4096, 14336 * 4096, 4096 * 14336, 4096], 2))
    return cases


def draw(rng):
    def size(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))) / step)) * step)

    op = rng.choice(["adapter", "adapter", "train", "experts", "balance", "balance", "clip"])
    if op in ("adapter", "train"):
        train = op == "train"
        R = rng.choice([8, 16, 16, 32, 64, 128])
        L = rng.choice([n for n in (1, 2, 4, 8, 32, 64) if n * R <= 1024])
        return _adapter(size(1, 2048 if train else 8192), size(64, 14336, 8), size(64, 4096, 8) if train else size(64, 14336), R, L,
                        none=rng.choice([0.0, 0.1, 0.5]), out=rng.choice(["bf16", "bf16", "f32"]), train=train)
    if op == "experts":
        return _experts(size(1, 2048), rng.choice([1, 2, 4]), size(64, 4096, 8), size(64, 1536), rng.choice([8, 16, 32]),
                        rng.choice([4, 8, 16, 32]), out=rng.choice(["bf16", "f32"]))
    if op == "balance":
        k = rng.choice([1, 2, 4, 6, 8, 10])
        S = rng.choice([1, 1, 2, 4, 8])
        return _balance(S * size(1, 16384 // S), rng.randint(max(4, k), 512), k, rng.choice(["softmax", "sigmoid"]), sequences=S,
                        dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.4, train=rng.random() < 0.7,
                        add=rng.random() < 0.4)
    shapes = [size(1, 1 << 24) for _ in range(rng.randint(1, 8))]
    return _clip(shapes, rng.choice([1, 2, 5, 24]) if sum(shapes) < 1 << 22 else 1, dtype=rng.choice(["f32", "bf16", "mixed"]),
                 kind=rng.choice(["two", "two", "max"]), over=rng.choice([0.5, 3.0]), clip=rng.random() < 0.7)


# ---- inputs --------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    s = dict(case)
    if case["op"] == "adapter":
        T, K, N, R, L, k = (case[n] for n in ("T", "K", "N", "R", "L", "k"))
        s["x_values"] = normal(T, K, dtype=torch.bfloat16)
        s["a_values"] = normal(L * R, K, std=K ** -0.5, dtype=torch.bfloat16)
        s["b_values"] = normal(L * N, R, std=0.05, dtype=torch.bfloat16)
        s["scales"] = 0.5 + 1.5 * uniform(L)
        if k:  # loads fall off with the expert's rank; a token's k experts differ
            load = torch.arange(1, L + 1, device=DEV).float().pow(-0.7)
            ids = torch.multinomial(load.expand(T, L), k, generator=g).to(torch.int32)
        else:
            # requests follow one another: one token each in a small batch, ragged prompts in a large one; each has
            # an adapter of its own while there are enough of them
            requests = T if T <= 64 else min(T, 4 * L)
            ends = torch.sort(torch.randperm(T - 1, generator=g, device=DEV)[:requests - 1]).values + 1
            request = torch.searchsorted(ends, torch.arange(T, device=DEV), right=True)
            of = torch.cat([torch.randperm(L, generator=g, device=DEV) for _ in range(-(-requests // L))])[:requests]
            of = torch.where(uniform(requests) < case["none"], torch.full_like(of, -1), of)
            ids = of[request].to(torch.int32)[:, None]
        s["ids"] = ids
        s["offsets"], s["rows"], s["pos"] = _plain_plan(ids, L)
        rows = T * max(k, 1)
        s["base"] = normal(rows, N, dtype=DTYPES[case["out"]])
        if case["train"]:
            s["dout"] = normal(rows, N, dtype=torch.bfloat16)
            s["dx_base"] = normal(T, K, dtype=torch.bfloat16)
    elif case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        logits = normal(T, E, std=1.5, dtype=DTYPES[case["dtype"]])
        # some experts are liked more than others
        logits += normal(E, std=0.5, dtype=DTYPES[case["dtype"]])
        if case["masked"]:  # padded tokens have no expert; some experts are closed to some tokens
            logits = logits.masked_fill((uniform(T, E) < 0.1) | (uniform(T, 1) < 0.05), -math.inf)
        s["logits"] = logits
        key, ids = torch.sort(logits.float(), dim=1, descending=True, stable=True)
        s["ids"] = torch.where(key[:, :k] == -math.inf, torch.full_like(ids[:, :k], -1), ids[:, :k]).to(torch.int32).contiguous()
        s["coef"] = 0.01
        if case["train"]:
            s["dloss"] = 0.5 + uniform(1)
            s["dlogits"] = normal(T, E, std=1e-6, dtype=DTYPES[case["dtype"]]) if case["add"] else None
    else:
        counts = [int(n) for n in case["shapes"].split(",")] * case["times"]
        types = ["f32", "bf16"] if case["dtype"] == "mixed" else [case["dtype"]]
        # layers' gradients differ in size
        s["grads"] = [normal(n, std=1e-3 * 2.0 ** (i % 5), dtype=DTYPES[types[i % len(types)]]) for i, n in enumerate(counts)]
        if case["clip"]:  # the clipped gradients go to the optimizer's bucket, one tensor behind the other
            s["flat"] = [torch.empty(sum(t.numel() for t in s["grads"] if t.dtype == DTYPES[d]), dtype=DTYPES[d], device=DEV) for d in types]
            parts = {f.dtype: iter(torch.split(f, [t.numel() for t in s["grads"] if t.dtype == f.dtype])) for f in s["flat"]}
            s["out"] = [next(parts[t.dtype]) for t in s["grads"]]
        squares = sum(n * (1e-3 * 2.0 ** (i % 5)) ** 2 for i, n in enumerate(counts))
        s["max_norm"] = (math.sqrt(squares) if case["kind"] == "two" else 0.08) / case["over"]
    return s


# ---- plain forms ---------------------------------------------------------------------------------
def _plain_plan(ids, L):
    """Slots in order of their adapter or expert: offsets, the slot of each row, the row of each slot."""
    flat = ids.reshape(-1).long()
    key, order = torch.sort(torch.where(flat < 0, torch.full_like(flat, L), flat), stable=True)
    offsets = torch.searchsorted(key, torch.arange(L + 1, device=ids.device)).to(torch.int32)
    rows = torch.where(key < L, order, torch.full_like(order, -1)).to(torch.int32)
    pos = torch.empty_like(flat)
    pos[order] = torch.where(key < L, torch.arange(flat.numel(), device=ids.device), torch.full_like(flat, -1))
    return offsets, rows, pos.to(torch.int32).reshape(ids.shape)


def _plain_adapter(s):
    """All adapters' products side by side; of each row only its own adapter's columns are kept."""
    L, R, N, K = s["L"], s["R"], s["N"], s["K"]
    if s["k"]:
        x = s["x_values"].float()[torch.div(s["rows"], s["k"], rounding_mode="floor").long()]
        owner = s["ids"].reshape(-1)[s["rows"].long()]
    else:
        x, owner = s["x_values"].float(), s["ids"][:, 0]
    mine = (owner[:, None] == torch.arange(L, device=DEV)).float() * s["scales"]
    mine = mine.repeat_interleave(R, dim=1)
    a = s["a_values"].float()
    b = s["b_values"].float().view(L, N, R).permute(0, 2, 1).reshape(L * R, N)
    h = (x @ a.t()) * mine
    out = (s["base"].float() + h @ b).to(s["base"].dtype)
    if not s["train"]:
        return {"out": out}
    dout = s["dout"].float()
    dh = (dout @ b.t()) * mine
    db = (dout.t() @ h).view(N, L, R).permute(1, 0, 2).reshape(L * N, R)
    dx = (s["dx_base"].float() + dh @ a).to(s["dx_base"].dtype)
    return {"out": out, "dx": dx, "da": dh.t() @ x, "db": db}


def _plain_balance(s):
    S, E, k = s["sequences"], s["E"], s["k"]
    l = s["logits"].float()
    open_ = ~(torch.isnan(l) | (l == -math.inf))
    l = torch.where(open_, l, torch.full_like(l, -math.inf)).clamp(max=F32_MAX)
    live = (s["ids"] >= 0).any(dim=1, keepdim=True)
    zero = torch.zeros_like(l)
    if s["score"] == "sigmoid":
        score = torch.where(open_, 1.0 / (1.0 + torch.exp(-l)), zero)
        slope = torch.where(open_, 1.0 / (1.0 + torch.exp(l)), zero)
        p = score / (score.sum(dim=1, keepdim=True) + 1e-20)
    else:
        slope = torch.ones_like(l)
        e = torch.where(open_, torch.exp(l - l.amax(dim=1, keepdim=True)), zero)
        p = torch.where(open_, e / e.sum(dim=1, keepdim=True), zero)
    p = torch.where(live, p, zero)
    flat = torch.where(s["ids"] >= 0, s["ids"], torch.full_like(s["ids"], E)).long().view(S, -1)
    counts = torch.zeros(S, E + 1, dtype=torch.int32, device=DEV).scatter_add_(1, flat, torch.ones_like(flat, dtype=torch.int32))[:, :E]
    tokens = live.view(S, -1).sum(dim=1)
    n = tokens.clamp(min=1).float()[:, None]
    probs = p.view(S, -1, E).sum(dim=1) / n
    share = counts.float() * (E / k) / n
    out = {"loss": ((share * probs).sum() * (s["coef"] / S)).reshape(1), "counts": counts.contiguous(), "probs": probs,
           "tokens": tokens.to(torch.int32)}
    if s["train"]:
        g = (share / n * (s["coef"] / S) * s["dloss"]).repeat_interleave(s["T"] // S, dim=0)
        d = p * slope * (g - (p * g).sum(dim=1, keepdim=True))
        d = torch.where(live & open_, d, zero)
        out["dlogits"] = (d if s["dlogits"] is None else d + s["dlogits"].float()).to(s["logits"].dtype)
    return out


def _plain_clip(s):
    if s["kind"] == "max":
        norm = torch.stack([t.float().abs().amax() for t in s["grads"]]).amax()
    else:
        norm = torch.stack([t.double().square().sum() for t in s["grads"]]).sum().sqrt().float()
    if not s["clip"]:
        return {"norm": norm.reshape(1)}
    factor = torch.where(torch.isfinite(norm), (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0), torch.ones_like(norm))
    [o.copy_(t.float() * factor) for o, t in zip(s["out"], s["grads"])]
    return {"norm": norm.reshape(1), "grads": s["flat"]}


# ---- the library's entry points --------------------------------------------------------------------
def _own(s):
    import nvfp4_bit_block_quantize_amd as nv
    if s["op"] == "adapter":
        w = nv.Adapters(s["a_values"], s["b_values"], s["scales"], s["R"], s["K"], s["N"], s["L"])
        plan = nv.MoEPlan(s["offsets"], s["rows"], s["pos"])
        how = dict(gather=True) if s["k"] else dict(by_token=True)
        if not s["train"]:
            return {"out": nv.nvfp4_adapter(s["x_values"], w, s["base"], plan=plan, **how)}
        out, h = nv.nvfp4_adapter(s["x_values"], w, s["base"], plan=plan, with_h=True, **how)
        d = nv.nvfp4_adapter_backward(s["dout"], s["x_values"], w, h, dx_base=s["dx_base"], plan=plan, **how)
        return {"out": out, "dx": d.dx, "da": d.da, "db": d.db}
    if s["op"] == "balance":
        flags = nv.NVFP4_ROUTE_SIGMOID if s["score"] == "sigmoid" else 0
        b = nv.nvfp4_moe_balance(s["logits"], s["ids"], s["coef"], flags=flags, sequences=s["sequences"])
        out = {"loss": b.loss, "counts": b.counts, "probs": b.probs, "tokens": b.tokens}
        if s["train"]:
            out["dlogits"] = nv.nvfp4_moe_balance_backward(s["logits"], s["ids"], b, s["coef"], flags=flags, dloss=s["dloss"],
                                                           dlogits=s["dlogits"])
        return out
    flags = nv.NVFP4_GRAD_MAX if s["kind"] == "max" else 0
    if not s["clip"]:
        return {"norm": nv.nvfp4_grad_norm(s["grads"], flags=flags)}
    norm = nv.nvfp4_grad_clip(s["grads"], s["max_norm"], flags=flags, out=s["out"])
    return {"norm": norm, "grads": s["flat"]}


def run(state):
    if own:
        return _own(state)
    return {"adapter": _plain_adapter, "balance": _plain_balance, "clip": _plain_clip}[state["op"]](state)


# ---- what a pass cannot do without -------------------------------------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2, "mixed": 3}
    if case["op"] == "adapter":
        T, K, N, R, L, k = (case[n] for n in ("T", "K", "N", "R", "L", "k"))
        rows = T * max(k, 1)
        used = min(L, rows)  # at most so many adapters are read
        b = T * K * 2 + 2 * rows * N * size[case["out"]] + used * R * (K + N) * 2 + rows * 4
        f = 2 * rows * R * (K + N)
        if case["train"]:
            b += rows * N * 2 + T * K * 6 + used * R * (K + N) * 2 + 4 * L * R * (K + N)
            f *= 3
        return {"bytes": b, "flops": f}
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["sequences"]
        es = size[case["dtype"]]
        b, f = T * E * es + T * k * 4 + 8 * S * E, 6 * T * E
        if case["train"]:
            b, f = b + T * E * es * (3 if case["add"] else 2) + T * k * 4, f + 10 * T * E
        return {"bytes": b, "flops": f}
    n = sum(int(v) for v in case["shapes"].split(",")) * case["times"]
    return {"bytes": n * size[case["dtype"]] * (3 if case["clip"] else 1), "flops": n * (3 if case["clip"] else 2)}


# ---- the definition in 64 bits -------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"adapter": _exact_adapter, "balance": _exact_balance, "clip": _exact_clip}[case["op"]](s)


def _exact_adapter(s):
    """Adapter by adapter."""
    L, R, N, K, k = (s[n] for n in ("L", "R", "N", "K", "k"))
    rows = s["rows"].long()
    ends = s["offsets"].tolist()
    out = s["base"].double()
    grads = {}
    if s["train"]:
        grads = {"dx": s["dx_base"].double(), "da": torch.zeros(L * R, K, dtype=torch.float64, device=DEV),
                 "db": torch.zeros(L * N, R, dtype=torch.float64, device=DEV)}
    for i in range(L):
        lo, hi = ends[i], ends[i + 1]
        if lo == hi:
            continue
        slots = rows[lo:hi]
        x = s["x_values"][slots // k if k else slots].double()
        at = torch.arange(lo, hi, device=DEV) if k else slots
        a, b = s["a_values"][i * R:(i + 1) * R].double(), s["b_values"][i * N:(i + 1) * N].double()
        scale = s["scales"][i].double()
        h = x @ a.t()
        out[at] += scale * (h @ b.t())
        if s["train"]:
            d = s["dout"][at].double()
            g = scale * (d @ b)
            grads["dx"][slots] += g @ a
            grads["da"][i * R:(i + 1) * R] = g.t() @ x
            grads["db"][i * N:(i + 1) * N] = scale * (d.t() @ h)
    return {"out": out, **grads}


def _exact_balance(s):
    """The loss sequence by sequence, and its gradient by differentiation."""
    S, E, k = s["sequences"], s["E"], s["k"]
    seq = s["T"] // S
    leaf = torch.nan_to_num(s["logits"].double(), nan=-math.inf, posinf=F32_MAX, neginf=-math.inf).requires_grad_()
    total, probs = 0.0, []
    with torch.enable_grad():
        for i in range(S):
            ids = s["ids"][i * seq:(i + 1) * seq].long()
            row = leaf[i * seq:(i + 1) * seq][(ids >= 0).any(dim=1)]
            if row.shape[0] == 0:
                probs.append(torch.zeros(E, dtype=torch.float64, device=DEV))
                continue
            if s["score"] == "sigmoid":
                score = torch.sigmoid(row)
                p = score / (score.sum(dim=1, keepdim=True) + 1e-20)
            else:
                p = torch.softmax(row, dim=1)
            load = torch.bincount(ids[ids >= 0], minlength=E).double() * E / (k * row.shape[0])
            probs.append(p.mean(dim=0))
            total = total + (load * probs[-1]).sum() * s["coef"] / S
    out = {"loss": torch.as_tensor(total, dtype=torch.float64, device=DEV).detach().reshape(1), "counts": None,
           "probs": torch.stack([p.detach() for p in probs]), "tokens": None}
    if s["train"]:
        if torch.is_tensor(total):
            d, = torch.autograd.grad(total * s["dloss"].double()[0], leaf)
            d = torch.nan_to_num(d, nan=0.0)  # (closed experts)
        else:
            d = torch.zeros_like(leaf)
        out["dlogits"] = d if s["dlogits"] is None else d + s["dlogits"].double()
    return out


def _exact_clip(s):
    top = [t.double().abs().max() for t in s["grads"]]
    if s["kind"] == "max":
        norm = max(float(v) for v in top)
    else:
        norm = math.sqrt(math.fsum(float(t.double().pow(2).sum()) for t in s["grads"]))
    out = {"norm": torch.tensor([norm], dtype=torch.float64, device=DEV)}
    if s["clip"]:
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
        out["grads"] = [torch.cat([t for t in s["grads"] if t.dtype == f.dtype] or [f]).double() * factor for f in s["flat"]]
    return out
