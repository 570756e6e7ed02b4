"""Cases of the operators around a worker's gradients: the vocabulary layer's cross entropy without its logits, tokens
sorted by expert and back with the chosen experts' weights, the gradients' global norm and clipping.

Each case runs either in its plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the
package's entry points; ``exact`` computes the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # Vocabulary cross entropy. The loss alone of one short sequence: the weight matrix is read once.
        {"name": "vocab short", "op": "vocab", "rows": 64, "vocab": 32000, "hidden": 1024, "grad": False, "dw": "bf16",
         "accumulate": False},
        # Sizes that fill no tile: loss, then the gradient from its log-sum-exp.
        {"name": "vocab odd", "op": "vocab", "rows": 1003, "vocab": 50001, "hidden": 1000, "grad": True, "dw": "bf16",
         "accumulate": False},
        # One of several batches whose weight gradients add up in f32.
        {"name": "vocab accumulate", "op": "vocab", "rows": 4096, "vocab": 32000, "hidden": 2048, "grad": True,
         "dw": "f32", "accumulate": True},
        # A training batch over a large vocabulary.
        {"name": "vocab large", "op": "vocab", "rows": 4096, "vocab": 131072, "hidden": 4096, "grad": True,
         "dw": "bf16", "accumulate": False},
        # Tokens to their experts' rows and the rows' gradients back to the tokens. A few tokens being generated.
        {"name": "dispatch few tokens", "op": "dispatch", "workers": 1, "tokens": 16, "experts": 8, "k": 2,
         "hidden": 1024, "dtype": "bf16", "align": 1, "capacity": 0},
        # Eight workers' batches over many experts, each expert's rows filled up to whole tiles of 128.
        {"name": "dispatch long batch", "op": "dispatch", "workers": 8, "tokens": 4096, "experts": 256, "k": 8,
         "hidden": 4096, "dtype": "bf16", "align": 128, "capacity": 0},
        # The experts' rows back to their tokens with weights and a residual, and the gradient of that. An odd size,
        # with a capacity that some tokens exceed.
        {"name": "combine odd", "op": "combine", "workers": 4, "tokens": 501, "experts": 60, "k": 4, "hidden": 1001,
         "dtype": "f32", "align": 1, "capacity": 40},
        # Eight workers' batches.
        {"name": "combine long batch", "op": "combine", "workers": 8, "tokens": 4096, "experts": 64, "k": 4,
         "hidden": 4096, "dtype": "bf16", "align": 1, "capacity": 0},
        # The chosen experts' weights and their gradient over the router's logits. A short sequence.
        {"name": "weights short", "op": "weights", "workers": 1, "tokens": 300, "experts": 60, "k": 4, "dtype": "bf16"},
        # Eight workers' long batches.
        {"name": "weights long batch", "op": "weights", "workers": 8, "tokens": 16384, "experts": 256, "k": 8,
         "dtype": "f32"},
        # Norm and clipping. One worker's few small tensors, back to back (starts that are not aligned), both types.
        {"name": "clip small", "op": "clip", "workers": 1, "count": 12, "total": 20011, "dtype": "mixed",
         "shared": False, "below": False, "packed": True},
        # The averaged gradients of many tensors of very different sizes, every worker's copy by one norm.
        {"name": "clip averaged", "op": "clip", "workers": 8, "count": 300, "total": 45000465, "dtype": "f32",
         "shared": True, "below": False, "packed": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["vocab", "vocab", "dispatch", "combine", "weights", "clip"])
    if op == "vocab":
        dw = rng.choice(["f32", "bf16"])
        return {"op": op, "rows": _log_int(rng, 1, 4096 if dw == "bf16" else 2048), "vocab": _log_int(rng, 500, 131072),
                "hidden": 8 * _log_int(rng, 8, 512), "grad": rng.random() < 0.8, "dw": dw,
                "accumulate": rng.random() < 0.4}
    if op in ("dispatch", "combine"):
        experts = _log_int(rng, 4, 256)
        workers, tokens, k, hidden = rng.choice([1, 2, 4, 8]), _log_int(rng, 1, 4096), rng.randint(1, min(8, experts)), \
            _log_int(rng, 64, 4096)
        pairs = workers * tokens * k
        layout = rng.choice(["packed", "aligned", "capacity"])
        return {"op": op, "workers": workers, "tokens": tokens, "experts": experts, "k": k, "hidden": hidden,
                "dtype": "bf16" if pairs * hidden > 1 << 28 else rng.choice(["f32", "bf16"]),
                "align": rng.choice([8, 64, 128]) if layout == "aligned" else 1,
                "capacity": max(1, int(pairs / experts * rng.uniform(0.6, 1.3))) if layout == "capacity" else 0}
    if op == "weights":
        experts = _log_int(rng, 4, 256)
        return {"op": op, "workers": rng.choice([1, 2, 4, 8]), "tokens": _log_int(rng, 1, 16384), "experts": experts,
                "k": rng.randint(1, min(8, experts)), "dtype": rng.choice(["f32", "bf16"])}
    count = _log_int(rng, 1, 300)
    return {"op": op, "workers": rng.choice([1, 2, 4, 8]), "count": count,
            "total": max(count, _log_int(rng, 1000, 45000000)), "dtype": rng.choice(["f32", "bf16", "mixed"]),
            "shared": rng.random() < 0.5, "below": rng.random() < 0.2, "packed": rng.random() < 0.4}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV) * scale


def _rand(shape, g):
    return torch.rand(shape, generator=g, device=DEV)


def _rows(c):
    """Rows of the experts' buffer: as many as any choice can ask for."""
    if c["capacity"]:
        return c["experts"] * c["capacity"]
    return c["workers"] * c["tokens"] * c["k"] + c["experts"] * (c["align"] - 1)


def _choices(c, g):
    """Each token's k distinct experts, some experts preferred, some tokens padding (-1)."""
    p, t, e, k = c["workers"], c["tokens"], c["experts"], c["k"]
    z = _normal((p, t, e), g) + _normal((1, 1, e), g, 0.5)
    choice = z.topk(k, dim=2).indices.to(torch.int32)
    choice[_rand((p, t), g) < 0.03] = -1
    choice[0, 0] = torch.arange(k, device=DEV, dtype=torch.int32)
    return z, choice.contiguous()


def _layout(c):
    """(type, element offset, elements) of each tensor of the list; the two types lie in buffers of their own."""
    r = random.Random("%d %d" % (c["count"], c["total"]))
    raw = [math.exp(r.uniform(math.log(256), math.log(2.4e6))) for _ in range(c["count"])]
    sizes = [max(1, int(x * c["total"] / sum(raw))) for x in raw]
    at, out = {"f32": 0, "bf16": 0}, []
    for i, n in enumerate(sizes):
        kind = c["dtype"] if c["dtype"] != "mixed" else ("bf16" if i % 3 else "f32")
        out.append((kind, at[kind], n))
        at[kind] += n if c["packed"] else -(-n // 8) * 8
    return out, at


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "vocab":
        t, v, h = case["rows"], case["vocab"], case["hidden"]
        s["x"] = _normal((t, h), g).bfloat16()
        s["w"] = _normal((v, h), g, 2.0 / math.sqrt(h)).bfloat16()
        target = torch.randint(0, v, (t,), generator=g, device=DEV)
        s["x"] += s["w"][target] * (2.0 * _rand((t, 1), g)).bfloat16()  # the layer has learned something
        target[_rand(t, g) < 0.05] = -100  # tokens that do not count
        target[0] = v - 1
        s["target"] = target.to(torch.int32)
        s["weight"] = (_rand(t, g) + 0.5) / t
        s["loss"], s["lse"] = torch.empty(t, device=DEV), torch.empty(t, device=DEV)
        if case["grad"]:
            s["dx"] = torch.empty((t, h), dtype=torch.bfloat16, device=DEV)
            s["dw"] = torch.empty((v, h), dtype=DTYPES[case["dw"]], device=DEV)
            # the gradient of the batches before
            s["before"] = _normal((v, h), g, 1e-3).to(DTYPES[case["dw"]]) if case["accumulate"] else None
    elif case["op"] in ("dispatch", "combine"):
        p, t, k, h = case["workers"], case["tokens"], case["k"], case["hidden"]
        dt, rows = DTYPES[case["dtype"]], _rows(case)
        s["choice"] = _choices(case, g)[1]
        if case["op"] == "dispatch":
            s["x"] = _normal((p, t, h), g).to(dt)
            s["dxs"] = _normal((rows, h), g, 1e-2).to(dt)
            s["xs"] = torch.zeros((rows, h), dtype=dt, device=DEV)  # rows behind the last expert stay as they are
            s["dx"] = torch.empty((p, t, h), dtype=dt, device=DEV)
            s["position"] = torch.empty((p, t, k), dtype=torch.int32, device=DEV)
            s["source"] = torch.empty(rows, dtype=torch.int32, device=DEV)
            s["offsets"] = torch.empty(case["experts"] + 1, dtype=torch.int32, device=DEV)
        else:
            s["position"], s["source"], _ = _sorted(case, s["choice"])
            s["ys"] = _normal((rows, h), g).to(dt)
            s["weight"] = torch.softmax(_normal((p, t, k), g), 2)
            s["residual"] = _normal((p, t, h), g).to(dt)
            s["dout"] = _normal((p, t, h), g, 1e-2).to(dt)
            s["out"] = torch.empty((p, t, h), dtype=dt, device=DEV)
            s["dys"] = torch.zeros((rows, h), dtype=dt, device=DEV)
            s["dweight"] = torch.empty((p, t, k), device=DEV)
    elif case["op"] == "weights":
        z, s["choice"] = _choices(case, g)
        s["z"] = z.to(DTYPES[case["dtype"]])
        s["dweight"] = _normal(s["choice"].shape, g, 0.1)
        s["weight"] = torch.empty(s["choice"].shape, device=DEV)
        s["dz"] = torch.empty_like(s["z"])
    else:
        s["tensors"], length = _layout(case)
        p = case["workers"]
        s["grads"] = {k: _normal((p, max(n, 1)), g, 0.01).to(DTYPES[k]) for k, n in length.items()}
        mask = {k: torch.zeros(max(n, 1), dtype=torch.bool) for k, n in length.items()}
        for kind, at, n in s["tensors"]:
            mask[kind][at:at + n] = True
        for k, m in mask.items():
            s["grads"][k] *= m.to(DEV)  # the gaps between the tensors
            if case["shared"]:
                s["grads"][k][1:] = s["grads"][k][:1]  # every worker's copy of the average
        s["out"] = {k: torch.zeros_like(x) for k, x in s["grads"].items()}
        s["norm"] = torch.empty(1 if case["shared"] else p, device=DEV)
        n = sum(n for _, _, n in s["tensors"])
        s["max_norm"] = 0.01 * math.sqrt(n) * (2.0 if case["below"] else 0.25)
    return s


# ------------------------------------------------------------- plain forms
def _plain_vocab(s):
    c = s["case"]
    target, v = s["target"].long(), c["vocab"]
    live = (target >= 0) & (target < v) & (s["weight"] != 0)
    at = target.clamp(0, v - 1)[:, None]
    x, w = s["x"].float(), s["w"].float()
    z = torch.matmul(x, w.t())
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    loss = torch.where(live, (lse - z.gather(1, at))[:, 0], 0.0)
    out = {"loss": loss, "lse": torch.where(live, lse[:, 0], 0.0)}
    if c["grad"]:
        p = torch.exp(z.sub_(lse))
        p.scatter_add_(1, at, torch.full_like(lse, -1.0))
        p *= torch.where(live, s["weight"], 0.0)[:, None]
        dw = torch.matmul(p.t(), x)
        if s["before"] is not None:
            dw += s["before"].float()
        out["dx"] = torch.matmul(p, w).to(s["dx"].dtype)
        out["dw"] = dw.to(s["dw"].dtype)
    return out


def _sorted(c, choice):
    """(position, source, offsets): the pairs (worker, token, choice) sorted by expert, in order within each."""
    e, rows = c["experts"], _rows(c)
    flat = choice.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < e), flat, e)
    counts = torch.bincount(key, minlength=e + 1)
    order = torch.sort(key, stable=True).indices
    first = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(key)
    rank[order] = torch.arange(n, device=DEV) - first[key[order]]
    if c["capacity"]:
        offsets = torch.arange(e + 1, device=DEV) * c["capacity"]
        kept = (key < e) & (rank < c["capacity"])
    else:
        filled = -(-counts[:e] // c["align"]) * c["align"]
        offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(filled, 0)])
        kept = key < e
    position = torch.where(kept, offsets[key.clamp(max=e - 1)] + rank, -1)
    source = torch.where(torch.arange(rows, device=DEV) < offsets[e], -1, -2)
    source = torch.cat([source, source[:1]])  # one more place for what has none
    source[torch.where(kept, position, rows)] = torch.arange(n, device=DEV)
    return position.to(torch.int32).view(choice.shape), source[:rows].to(torch.int32), offsets.to(torch.int32)


def _to_rows(x, source, k, weight=None):
    """[P, tokens, hidden] -> the experts' rows; rows without a token are 0."""
    pair = source.long().clamp(min=0)
    y = x.reshape(-1, x.shape[2])[pair // k].float()
    if weight is not None:
        y = y * weight.reshape(-1)[pair][:, None]
    return torch.where((source >= 0)[:, None], y, 0.0)


def _from_rows(y, position, weight=None):
    at = position.long().clamp(min=0)
    w = torch.where(position >= 0, 1.0 if weight is None else weight, 0.0)
    out = y[at[:, :, 0]].float() * w[:, :, :1]
    for j in range(1, position.shape[2]):
        out += y[at[:, :, j]].float() * w[:, :, j:j + 1]
    return out


def _plain_dispatch(s):
    c = s["case"]
    position, source, offsets = _sorted(c, s["choice"])
    xs = _to_rows(s["x"], source, c["k"]).to(s["xs"].dtype)
    dx = _from_rows(s["dxs"], position).to(s["dx"].dtype)
    return {"position": position, "source": source, "offsets": offsets, "xs": xs, "dx": dx}


def _plain_combine(s):
    c, dt = s["case"], s["out"].dtype
    out = _from_rows(s["ys"], s["position"], s["weight"]).add_(s["residual"].float()).to(dt)
    dys = _to_rows(s["dout"], s["source"], c["k"], s["weight"]).to(dt)
    at = s["position"].long().clamp(min=0)
    dout = s["dout"].float()
    dweight = torch.stack([(s["ys"][at[:, :, j]].float() * dout).sum(2) for j in range(c["k"])], 2)
    return {"out": out, "dys": dys, "dweight": torch.where(s["position"] >= 0, dweight, 0.0)}


def _plain_weights(s):
    choice = s["choice"]
    ok, at = choice >= 0, choice.long().clamp(min=0)
    z = torch.where(ok, s["z"].float().gather(2, at), float("-inf"))
    top = torch.where(ok.any(2, keepdim=True), z.amax(2, keepdim=True), 0.0)
    e = torch.exp(z - top)
    w = e / torch.where(ok.any(2, keepdim=True), e.sum(2, keepdim=True), 1.0)
    d = torch.where(ok, s["dweight"], 0.0)
    g = w * (d - (w * d).sum(2, keepdim=True))
    dz = torch.zeros(s["z"].shape, device=DEV).scatter_add_(2, at, torch.where(ok, g, 0.0))
    return {"weight": w, "dz": dz.to(s["z"].dtype)}


def _plain_clip(s):
    g = {k: x.float() for k, x in s["grads"].items()}
    total = (g["f32"] * g["f32"]).sum(1) + (g["bf16"] * g["bf16"]).sum(1)
    norm = torch.sqrt(total[:1] if s["case"]["shared"] else total)
    c = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0)
    return {"norm": norm, "out": {k: (x * c[:, None]).to(s["out"][k].dtype) for k, x in g.items()}}


# ------------------------------------------------------------ own kernels
def _kept(s, name, make):
    """What a user's program makes once and keeps: a workspace, tables of pointers."""
    if name not in s:
        s[name] = make()
    return s[name]


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


def _own(s):
    import gradient_allreduce_homomorphic_gb300 as g

    c = s["case"]
    if c["op"] == "vocab":
        ws = _kept(s, "workspace", lambda: _bytes(g.gar_vocab_workspace_bytes(c["rows"], c["vocab"], c["hidden"],
                                                                              DTYPES[c["dw"]])))
        g.gar_vocab_loss(s["x"], s["w"], s["target"], s["loss"], s["lse"], ws, weight=s["weight"])
        out = {"loss": s["loss"], "lse": s["lse"]}
        if c["grad"]:
            g.gar_vocab_grad(s["x"], s["w"], s["target"], s["lse"], s["dx"], s["dw"], ws, weight=s["weight"],
                             addend=s["before"])
            out |= {"dx": s["dx"], "dw": s["dw"]}
        return out
    if c["op"] == "dispatch":
        t = _kept(s, "tables", lambda: {k: g.PtrTable(s[k]) for k in ("choice", "position", "x", "dx")})
        ws = _kept(s, "workspace", lambda: _bytes(g.gar_expert_workspace_bytes(c["workers"], c["tokens"], c["k"],
                                                                               c["experts"])))
        g.gar_expert_sort(t["choice"], c["experts"], t["position"], s["source"], s["offsets"], ws, align=c["align"],
                          capacity=c["capacity"])
        g.gar_expert_gather(t["x"], t["position"], s["source"], s["xs"])
        g.gar_expert_combine(s["dxs"], t["position"], t["dx"])
        return {k: s[k] for k in ("position", "source", "offsets", "xs", "dx")}
    if c["op"] == "combine":
        t = _kept(s, "tables", lambda: {k: g.PtrTable(s[k]) for k in ("position", "weight", "residual", "dout", "out",
                                                                      "dweight")})
        g.gar_expert_combine(s["ys"], t["position"], t["out"], weight=t["weight"], addend=t["residual"])
        g.gar_expert_combine_grad(t["dout"], s["ys"], t["position"], s["source"], t["weight"], s["dys"], t["dweight"])
        return {"out": s["out"], "dys": s["dys"], "dweight": s["dweight"]}
    if c["op"] == "weights":
        t = _kept(s, "tables", lambda: {k: g.PtrTable(s[k]) for k in ("z", "choice", "weight", "dweight", "dz")})
        g.gar_expert_weights(t["z"], t["choice"], t["weight"])
        g.gar_expert_weights_grad(t["weight"], t["dweight"], t["choice"], t["dz"])
        return {"weight": s["weight"], "dz": s["dz"]}
    tables = _kept(s, "tables", lambda: g.grad_tables(*([[b[kind][w, at:at + n] for kind, at, n in s["tensors"]]
                                                         for w in range(c["workers"])] for b in (s["grads"], s["out"]))))
    ws = _kept(s, "workspace", lambda: _bytes(g.gar_grad_workspace_bytes(tables)))
    g.gar_grad_clip(tables, s["max_norm"], s["norm"], ws, shared=c["shared"])
    return {"norm": s["norm"], "out": s["out"]}


def run(state):
    if own:
        return _own(state)
    return {"vocab": _plain_vocab, "dispatch": _plain_dispatch, "combine": _plain_combine, "weights": _plain_weights,
            "clip": _plain_clip}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "vocab":
        t, v, h = c["rows"], c["vocab"], c["hidden"]
        if not c["grad"]:
            return {"bytes": (t + v) * h * 2 + t * 16, "flops": 2 * t * v * h}
        out = t * h * 2 + v * h * SIZE[c["dw"]] * (2 if c["accumulate"] else 1)
        return {"bytes": (t + v) * h * 2 + t * 16 + out, "flops": 6 * t * v * h}
    if c["op"] == "clip":
        tensors, _ = _layout(c)
        n = sum(n * SIZE[kind] for kind, _, n in tensors) * c["workers"]
        return {"bytes": 2 * n, "flops": 3 * n // 4}
    p, t, e, k = c["workers"], c["tokens"], c["experts"], c["k"]
    if c["op"] == "weights":
        return {"bytes": p * t * (k * (SIZE[c["dtype"]] + 12) + e * SIZE[c["dtype"]]), "flops": 8 * p * t * k}
    h, b = c["hidden"], SIZE[c["dtype"]]
    # with a capacity each expert has its rows; else the rows filled up to `align` depend on the choices
    rows = e * c["capacity"] if c["capacity"] else p * t * k
    used = min(rows, p * t * k)
    if c["op"] == "dispatch":
        return {"bytes": p * t * (2 * h * b + 8 * k) + (rows + used) * h * b + 4 * rows, "flops": p * t * k * h}
    return {"bytes": p * t * (3 * h * b + 12 * k) + (rows + used) * h * b + 4 * rows, "flops": 5 * p * t * k * h}


# ------------------------------------------------------------------ exact
def _exact_vocab(s):
    """Row by row of blocks: log_softmax of the 64-bit logits and its Jacobian."""
    c = s["case"]
    t, v, h = c["rows"], c["vocab"], c["hidden"]
    if t * v * h * (3 if c["grad"] else 1) > 8e12:  # over about 20 seconds of 64-bit products
        return None
    w = s["w"].double()
    loss, lse = torch.zeros(t, dtype=torch.float64, device=DEV), torch.zeros(t, dtype=torch.float64, device=DEV)
    dx = torch.zeros((t, h), dtype=torch.float64, device=DEV)
    dw = torch.zeros((v, h), dtype=torch.float64, device=DEV) if c["grad"] else None
    for lo in range(0, t, 1024):
        target = s["target"][lo:lo + 1024].long()
        on = torch.nonzero((target >= 0) & (target < v) & (s["weight"][lo:lo + 1024] != 0))[:, 0]
        if not on.numel():
            continue
        x = s["x"][lo + on].double()
        z = x @ w.t()
        n = torch.logsumexp(z, 1)
        lse[lo + on] = n
        loss[lo + on] = n - z[torch.arange(on.numel(), device=DEV), target[on]]
        if c["grad"]:
            q = z.sub_(n[:, None]).exp_()
            q[torch.arange(on.numel(), device=DEV), target[on]] -= 1.0
            q *= s["weight"][lo + on].double()[:, None]
            dx[lo + on] = q @ w
            dw += q.t() @ x
    out = {"loss": loss, "lse": lse}
    if c["grad"]:
        if s["before"] is not None:
            dw += s["before"].double()
        out |= {"dx": dx, "dw": dw}
    return out


def _exact_place(c, choice):
    """Each pair's row by counting the pairs of its expert ahead of it, 64 experts at a time; -1: none."""
    flat = choice.reshape(-1).long()
    where = torch.full_like(flat, -1)
    start = 0
    for lo in range(0, c["experts"], 64):
        hi = min(lo + 64, c["experts"])
        hit = flat[:, None] == torch.arange(lo, hi, device=DEV)
        ahead = torch.cumsum(hit.int(), 0).long() - 1
        for e in range(lo, hi):
            own_pairs, rank = hit[:, e - lo], ahead[:, e - lo]
            if c["capacity"]:
                where = torch.where(own_pairs & (rank < c["capacity"]), e * c["capacity"] + rank, where)
            else:
                where = torch.where(own_pairs, start + rank, where)
                n = int(rank[-1]) + 1
                start += (n + c["align"] - 1) // c["align"] * c["align"]
    return where


def _exact_dispatch(s):
    c = s["case"]
    where = _exact_place(c, s["choice"]).view(-1, c["k"])
    x, dt = s["x"].view(where.shape[0], -1), torch.float64
    if s["xs"].numel() > 1 << 29:  # as f32: a copy is exact, and 64 bits of it too much
        dt = torch.float32
    xs = torch.zeros(s["xs"].shape, dtype=dt, device=DEV)
    dx = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
    for j in range(c["k"]):
        on = torch.nonzero(where[:, j] >= 0)[:, 0]
        xs[where[on, j]] = x[on].to(dt)
        dx[on] += s["dxs"][where[on, j]].double()
    return {"position": None, "source": None, "offsets": None, "xs": xs, "dx": dx.view(s["dx"].shape)}


def _exact_combine(s):
    c = s["case"]
    where = _exact_place(c, s["choice"]).view(-1, c["k"])
    weight, dout = s["weight"].view(-1, c["k"]).double(), s["dout"].view(where.shape[0], -1).double()
    out = s["residual"].view(where.shape[0], -1).double()
    dys = torch.zeros(s["dys"].shape, dtype=torch.float64, device=DEV)
    dweight = torch.zeros(weight.shape, dtype=torch.float64, device=DEV)
    for j in range(c["k"]):
        on = torch.nonzero(where[:, j] >= 0)[:, 0]
        y = s["ys"][where[on, j]].double()
        out[on] += y * weight[on, j, None]
        dys[where[on, j]] = dout[on] * weight[on, j, None]
        dweight[on, j] = torch.einsum("th,th->t", y, dout[on])
    return {"out": out.view(s["out"].shape), "dys": dys, "dweight": dweight.view(s["dweight"].shape)}


def _exact_weights(s):
    """Softmax over all experts with the others shut out, and its Jacobian."""
    p, t, k = s["choice"].shape
    e = s["case"]["experts"]
    choice = s["choice"].view(-1, k).long()
    on = torch.nonzero(choice[:, 0] >= 0)[:, 0]
    z = torch.full((p * t, e), float("-inf"), dtype=torch.float64, device=DEV)
    z[on] = z[on].scatter(1, choice[on], s["z"].view(-1, e)[on].double().gather(1, choice[on]))
    q = torch.softmax(z[on], 1)
    d = torch.zeros(q.shape, dtype=torch.float64, device=DEV).scatter(1, choice[on], s["dweight"].view(-1, k)[on].double())
    weight = torch.zeros((p * t, k), dtype=torch.float64, device=DEV)
    weight[on] = q.gather(1, choice[on])
    dz = torch.zeros((p * t, e), dtype=torch.float64, device=DEV)
    dz[on] = q * d - q * torch.einsum("te,te->t", q, d)[:, None]
    return {"weight": weight.view(p, t, k), "dz": dz.view(p, t, e)}


def _exact_clip(s):
    c = s["case"]
    norm = []
    for w in range(1 if c["shared"] else c["workers"]):
        squares = sum(torch.dot(v, v).item() for v in (s["grads"][kind][w, at:at + n].double()
                                                       for kind, at, n in s["tensors"]))
        norm.append(math.sqrt(squares))
    scale = [s["max_norm"] / x if x > s["max_norm"] else 1.0 for x in norm]
    factor = torch.tensor(scale * (c["workers"] if c["shared"] else 1), dtype=torch.float64, device=DEV)
    return {"norm": torch.tensor(norm, dtype=torch.float64, device=DEV),
            "out": {k: x.double() * factor[:, None] for k, x in s["grads"].items()}}


def exact(case, seed):
    s = prepare(case, seed)
    return {"vocab": _exact_vocab, "dispatch": _exact_dispatch, "combine": _exact_combine, "weights": _exact_weights,
            "clip": _exact_clip}[case["op"]](s)
