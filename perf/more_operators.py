"""The router, the token sort and its way back with their gradients, and gradient clipping, as cases that can be
timed and checked.

Each case names one operator (``op``) and its sizes; ``prepare`` draws its inputs on the GPU from a seed,
``run`` makes one pass (``own`` selects the library's kernels, else plain torch arithmetic in 32 bits), and
``exact`` gives the operator's definition in 64 bits.

Definitions (T tokens of k slots, i = t k + s; E experts; row(i) the row of entry i, none if its expert id is
outside [0, E)):

* ``router``   ids[t] = the k largest logits of a token (ties: the lower expert first); w = their softmax over the
               k (``renorm``) or over all E experts; with ``train`` also the logits' gradient from w's.
* ``permute``  the stable sort of the entries by expert: offsets, both maps, and rows[row(i)] = x[t].
* ``combine``  y[t] = sum_s w_i d[row(i)].
* ``combine_bwd``  its gradient: dd[row(i)] = w_i dy[t], dw_i = sum_h dy[t, h] d[row(i), h].
* ``swiglu_bwd``   gradient of h = w silu(g) u with respect to g, u and w, h[row(i)] from w_i.
* ``clip``     n = sqrt(sum of squares over all tensors), out = x min(1, max_norm / (n + 1e-6)); n alone with
               a ``max_norm`` of 0.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token's router while serving, where the launch is what costs
        {"name": "router_one_token", "op": "router", "T": 1, "E": 128, "k": 8, "dtype": "f32", "renorm": True,
         "train": False},
        # several sequences' router in a training step, probabilities over every expert, an odd count of experts
        {"name": "router_train_wide", "op": "router", "T": 16381, "E": 250, "k": 6, "dtype": "bf16", "renorm": False,
         "train": True},
        # a small serving batch sorted for the experts' products
        {"name": "permute_batch_61", "op": "permute", "T": 61, "k": 8, "E": 128, "H": 2048, "dtype": "bf16",
         "routing": "uniform", "dropped": 0.0},
        # the layer at its training length
        {"name": "permute_train", "op": "permute", "T": 4096, "k": 8, "E": 128, "H": 2048, "dtype": "bf16",
         "routing": "softmax", "dropped": 0.0},
        # float32 rows of few, skewed experts with entries over an expert's capacity dropped
        {"name": "combine_dropped", "op": "combine", "T": 1021, "k": 4, "E": 24, "H": 520, "d": "f32", "y": "f32",
         "weighted": True, "routing": "zipf", "dropped": 0.05},
        # the layer's output at the training length, from bf16 expert outputs
        {"name": "combine_train", "op": "combine", "T": 4096, "k": 8, "E": 128, "H": 2048, "d": "bf16", "y": "bf16",
         "weighted": True, "routing": "softmax", "dropped": 0.0},
        # a small fine-tuning batch, float32 expert outputs
        {"name": "combine_bwd_61", "op": "combine_bwd", "T": 61, "k": 8, "E": 128, "H": 2048, "dy": "bf16",
         "d": "f32", "routing": "uniform", "dropped": 0.0},
        # its gradient at the training length
        {"name": "combine_bwd_train", "op": "combine_bwd", "T": 4096, "k": 8, "E": 128, "H": 2048, "dy": "bf16",
         "d": "bf16", "routing": "softmax", "dropped": 0.0},
        # the SwiGLU's gradient with the router weight's, one token's eight rows
        {"name": "swiglu_bwd_one_token", "op": "swiglu_bwd", "T": 1, "k": 8, "E": 128, "I": 768, "routing": "softmax",
         "dropped": 0.0},
        # the same at the training length
        {"name": "swiglu_bwd_train", "op": "swiglu_bwd", "T": 4096, "k": 8, "E": 128, "I": 768, "routing": "softmax",
         "dropped": 0.0},
        # a model's many small tensors (biases, norms, adapters) of odd sizes and both types
        {"name": "clip_many_small", "op": "clip", "dtype": "mixed", "max_norm": 1.0,
         "sizes": "1,2048,2048,771,128,4099,640,2048,33,2048,5120,768,1536,7,9000,2048,2048,512,129,24,2048,40000,768,64,"
                  "2048,2048,1021,128,4096,640,2048,31,2048,5121,769,1535,8,10000,2048,2049,511,130,25,2047,30000,767,63,1"},
        # the layer's own gradients: gate_up, down, QKV, router and two norm weights
        {"name": "clip_layer", "op": "clip", "dtype": "mixed", "max_norm": 1.0,
         "sizes": "402653184,201326592,10485760,262144,2048,2048"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["router", "permute", "combine", "combine_bwd", "swiglu_bwd", "clip"])
    if op == "clip":
        n = _log(rng, 1, 200)
        most = _log(rng, 16, 40_000_000)
        sizes = [min(_log(rng, 1, most), 200_000_000 // n) for _ in range(n)]
        return {"op": op, "dtype": rng.choice(["mixed", "f32", "bf16"]), "max_norm": rng.choice([0.0, 0.5, 1e9]),
                "sizes": ",".join(map(str, sizes))}
    E = _log(rng, 2, 1024)
    k = rng.randint(1, min(32, E)) if rng.random() < 0.3 else rng.randint(1, min(8, E))
    T = _log(rng, 1, 16384)
    if op == "router":
        return {"op": op, "T": min(T, 8_000_000 // E), "E": E, "k": k, "dtype": rng.choice(["bf16", "f32"]),
                "renorm": rng.random() < 0.5, "train": rng.random() < 0.6}
    case = {"op": op, "T": T, "k": k, "E": E}
    kinds = ["bf16", "f32"]
    if op == "swiglu_bwd":
        case["I"] = _log(rng, 8, 2048, 8)
        case["T"] = max(1, min(T, 30_000_000 // (k * case["I"])))
    else:
        case["H"] = _log(rng, 8, 8192, 8)
        case["T"] = max(1, min(T, 60_000_000 // (k * case["H"])))
    if op == "permute":
        case["dtype"] = rng.choice(kinds)
    if op == "combine":
        case |= {"d": rng.choice(kinds), "y": rng.choice(kinds), "weighted": rng.random() < 0.7}
    if op == "combine_bwd":
        case |= {"dy": rng.choice(kinds), "d": rng.choice(kinds)}
    return case | {"routing": rng.choice(["softmax", "uniform", "zipf"]), "dropped": rng.choice([0.0, 0.0, 0.05, 0.5])}


# ------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _sizes(case):
    """(elements, type) of each tensor; `mixed`: the first float32, then bf16 and float32 in turn."""
    sizes = [int(n) for n in case["sizes"].split(",")]
    kind = case["dtype"]
    return [(n, TYPES[kind] if kind != "mixed" else TYPES["f32" if j % 2 == 0 else "bf16"]) for j, n in enumerate(sizes)]


def _route(gen, case):
    """Expert ids [T, k] (distinct in a token; dropped entries -1) and weights [T, k]."""
    T, k, E = case["T"], case["k"], case["E"]
    score = _normal(gen, T, E)
    if case["routing"] == "uniform":
        score = torch.rand((T, E), generator=gen, device=DEV)
    elif case["routing"] == "zipf":
        u = torch.rand((T, E), generator=gen, device=DEV).clamp(1e-7, 1 - 1e-7)
        score = -torch.log(-torch.log(u)) - 1.2 * torch.log(torch.arange(1, E + 1, device=DEV))
    top, ids = score.topk(k, dim=1)
    lost = torch.rand((T, k), generator=gen, device=DEV) < case["dropped"]
    return torch.where(lost, -1, ids).int(), torch.softmax(top, 1).contiguous()


def prepare(case, seed):
    gen, op = _gen(seed), case["op"]
    st = {"case": case}
    if op == "clip":
        st["grads"] = [(0.01 * _normal(gen, n)).to(dt) for n, dt in _sizes(case)]
        if case["max_norm"]:
            st["out"] = [torch.empty_like(g) for g in st["grads"]]
        return st
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    if op == "router":
        st["logits"] = (2 * _normal(gen, T, E)).to(TYPES[case["dtype"]])
        st["dw"] = _normal(gen, T, k)
        return st
    ids, st["topk_w"] = _route(gen, case)
    if op == "permute":
        st["ids"] = ids
        st["x"] = _normal(gen, T, case["H"]).to(TYPES[case["dtype"]])
        # a training program keeps these buffers from step to step; rows of dropped entries stay as they are
        st["out"] = {"rows": torch.zeros((R, case["H"]), dtype=st["x"].dtype, device=DEV),
                     "row_to_tk": torch.full((R,), -1, dtype=torch.int32, device=DEV)}
        return st
    st["offsets"], st["row_to_tk"], st["tk_to_row"] = _sort(ids.reshape(-1), E)
    if op == "swiglu_bwd":
        st["gu"] = 2 * _normal(gen, R, 2 * case["I"])
        st["dh"] = 0.05 * _normal(gen, R, case["I"])
        st["dgu"] = torch.zeros((R, 2 * case["I"]), dtype=torch.bfloat16, device=DEV)
        return st
    st["d"] = _normal(gen, R, case["H"]).to(TYPES[case["d"]])
    if op == "combine_bwd":
        st["dy"] = (0.1 * _normal(gen, T, case["H"])).to(TYPES[case["dy"]])
        st["dd"] = torch.zeros_like(st["d"])
    return st


# ------------------------------------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    import precision_moe_gemm_amd as pmg
    case = st["case"]
    op = case["op"]
    if op == "router":
        ids, w = pmg.moe_router_topk(st["logits"], case["k"], renorm=case["renorm"])
        if not case["train"]:
            return {"ids": ids, "w": w}
        return {"ids": ids, "w": w,
                "dlogits": pmg.moe_router_topk_backward(st["dw"], ids, w, st["logits"], renorm=case["renorm"])}
    if op == "permute":
        return pmg.moe_permute(st["x"], st["ids"], case["E"], out=st["out"])
    if op == "combine":
        return pmg.moe_combine(st["d"], st["tk_to_row"], case["k"], st["topk_w"] if case["weighted"] else None,
                               out_dtype=TYPES[case["y"]])
    if op == "combine_bwd":
        dd, dw = pmg.moe_combine_backward(st["dy"], st["d"], st["tk_to_row"], case["k"], st["topk_w"], dd=st["dd"])
        return {"dd": dd, "dw": dw}
    if op == "swiglu_bwd":
        dgu, dw = pmg.swiglu_backward_weights(st["gu"], st["dh"], st["offsets"], st["topk_w"], st["row_to_tk"],
                                              st["tk_to_row"], dgu=st["dgu"])
        return {"dgu": dgu, "dw": dw}
    if not case["max_norm"]:
        return pmg.grad_norm(st["grads"])
    norm, out = pmg.grad_clip(st["grads"], case["max_norm"], out=st["out"])
    return {"norm": norm, "out": out}


def _sort(ids, E):
    """ids [T k] -> offsets [E + 1], row_to_tk [T k] (-1 behind the last row), tk_to_row [T k] (-1: no row)."""
    valid = (ids >= 0) & (ids < E)
    order = torch.where(valid, ids, E).argsort(stable=True).int()
    at = torch.arange(ids.numel(), dtype=torch.int32, device=ids.device)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = (ids.view(1, -1) == torch.arange(E, device=ids.device).view(-1, 1)).sum(1).cumsum(0)
    live = at < offsets[E]
    tk_to_row = torch.empty_like(at)
    tk_to_row[order.long()] = torch.where(live, at, -1)
    return offsets, torch.where(live, order, -1), tk_to_row


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "router":
        l, k = st["logits"].float(), case["k"]
        top, ids = torch.sort(l, dim=1, descending=True, stable=True)
        ids = ids[:, :k].contiguous()
        e = torch.exp(l - top[:, :1])
        picked = e.gather(1, ids)
        total = (picked if case["renorm"] else e).sum(1, keepdim=True)
        w = picked / total
        out = {"ids": ids.int(), "w": w}
        if case["train"]:
            mean = (w * st["dw"]).sum(1, keepdim=True)
            if case["renorm"]:
                d = torch.zeros_like(l).scatter_(1, ids, w * (st["dw"] - mean))
            else:
                d = e / total * (torch.zeros_like(l).scatter_(1, ids, st["dw"]) - mean)
            out["dlogits"] = d.to(st["logits"].dtype)
        return out
    if op == "permute":
        offsets, row_to_tk, tk_to_row = _sort(st["ids"].reshape(-1), case["E"])
        rows = st["x"][row_to_tk.clamp(min=0).long() // case["k"]] * (row_to_tk >= 0)[:, None]
        return {"rows": rows, "expert_offsets": offsets, "row_to_tk": row_to_tk, "tk_to_row": tk_to_row}
    if op == "clip":
        squares = [(g.float() ** 2).sum(dtype=torch.float64) for g in st["grads"]]
        norm = torch.sqrt(torch.stack(squares).sum())
        if not case["max_norm"]:
            return norm.float().view(1)
        c = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0).float()
        return {"norm": norm.float().view(1), "out": [(g.float() * c).to(g.dtype) for g in st["grads"]]}
    T, k = case["T"], case["k"]
    w = st["topk_w"].view(T, k, 1)
    row = st["tk_to_row"].long().view(T, k)
    live = (row >= 0).unsqueeze(2)
    row = row.clamp(min=0)
    if op == "combine":
        v = st["d"].float()[row] * live
        return (v * w if case["weighted"] else v).sum(1).to(TYPES[case["y"]])
    if op == "combine_bwd":
        dy = st["dy"].float().view(T, 1, -1)
        dw = (dy * st["d"].float()[row] * live).sum(2)
        src = st["row_to_tk"].clamp(min=0).long()
        dd = st["dy"].float()[src // k] * st["topk_w"].view(-1, 1)[src] * (st["row_to_tk"] >= 0)[:, None]
        return {"dd": dd.to(st["d"].dtype), "dw": dw}
    g, u = st["gu"].split(case["I"], dim=1)
    src = st["row_to_tk"].clamp(min=0).long()
    has = (st["row_to_tk"] >= 0)[:, None]
    sig = 1 / (1 + torch.exp(-g))
    t = st["dh"] * st["topk_w"].view(-1, 1)[src]
    dgu = torch.cat([t * u * (sig * (1 + g * (1 - sig))), t * (g * sig)], 1) * has
    per_row = (st["dh"] * (g * sig) * u).sum(1)
    return {"dgu": dgu.bfloat16(), "dw": per_row[row] * live[:, :, 0]}


# ------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "clip":
        n = sum(m for m, _ in _sizes(case))
        b = sum(m * dt.itemsize for m, dt in _sizes(case))
        clipped = case["max_norm"] > 0
        return {"bytes": b * (2 if clipped else 1) + 4, "flops": n * (3 if clipped else 2)}
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    rows = round(R * (1 - case.get("dropped", 0)))
    if op == "router":
        n = T * E
        return {"bytes": n * size[case["dtype"]] * (2 if case["train"] else 1) + (12 if case["train"] else 8) * R,
                "flops": n * (6 if case["train"] else 3)}
    if op == "permute":
        h = case["H"] * size[case["dtype"]]
        return {"bytes": (T + rows) * h + 12 * R + 4 * (E + 1), "flops": R}
    if op == "combine":
        h = case["H"]
        return {"bytes": rows * h * size[case["d"]] + T * h * size[case["y"]] + (8 if case["weighted"] else 4) * R,
                "flops": 2 * rows * h}
    if op == "combine_bwd":
        h = case["H"]
        return {"bytes": T * h * size[case["dy"]] + 2 * rows * h * size[case["d"]] + 12 * R, "flops": 3 * rows * h}
    return {"bytes": rows * case["I"] * 16 + 16 * R, "flops": 16 * rows * case["I"]}


# ------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "clip":
        total = sum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in st["grads"])
        norm = torch.tensor([math.sqrt(total)], dtype=torch.float64, device=DEV)
        if not case["max_norm"]:
            return norm
        c = min(1.0, case["max_norm"] / (math.sqrt(total) + 1e-6))
        return {"norm": norm, "out": [g.double().mul_(c) for g in st["grads"]]}
    T, k, E = case["T"], case["k"], case["E"]
    if op == "router":
        l = st["logits"].double()
        taken = torch.zeros((T, E), dtype=torch.bool, device=DEV)
        ids = torch.empty((T, k), dtype=torch.int64, device=DEV)
        for s in range(k):      # the largest that is left, the first of equals
            left = l.masked_fill(taken, -math.inf)
            first = (left == left.amax(1, keepdim=True)) & ~taken
            ids[:, s] = first.int().argmax(1)
            taken.scatter_(1, ids[:, s:s + 1], True)
        p = torch.softmax(l.masked_fill(~taken, -math.inf) if case["renorm"] else l, 1)
        out = {"ids": ids.int(), "w": p.gather(1, ids)}
        if case["train"]:
            g = torch.zeros_like(p).scatter_(1, ids, st["dw"].double())
            out["dlogits"] = p * (g - (p * g).sum(1, keepdim=True))
        return out
    if op == "permute":
        flat = st["ids"].reshape(-1).tolist()
        lists = [[] for _ in range(E)]
        for i, e in enumerate(flat):
            if 0 <= e < E:
                lists[e].append(i)
        order = [i for part in lists for i in part]
        offsets = [0]
        for part in lists:
            offsets.append(offsets[-1] + len(part))
        back = [-1] * len(flat)
        for r, i in enumerate(order):
            back[i] = r
        whole = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
        rows = torch.zeros((T * k, case["H"]), dtype=torch.float64, device=DEV)
        rows[:len(order)] = st["x"].double()[torch.div(whole(order), k, rounding_mode="floor").long()]
        return {"rows": rows, "expert_offsets": whole(offsets), "row_to_tk": whole(order + [-1] * (len(flat) - len(order))),
                "tk_to_row": whole(back)}
    R = T * k
    n = int(st["offsets"][-1])
    entry = st["row_to_tk"][:n].long()            # of each row that is there
    w = st["topk_w"].double().reshape(-1)
    if op == "combine":
        y = torch.zeros((T, case["H"]), dtype=torch.float64, device=DEV)
        v = st["d"][:n].double()
        return y.index_add_(0, entry // k, v * w[entry, None] if case["weighted"] else v)
    dw = torch.zeros(R, dtype=torch.float64, device=DEV)
    if op == "combine_bwd":
        dy = st["dy"].double()[entry // k]
        dd = torch.zeros((R, case["H"]), dtype=torch.float64, device=DEV)
        dd[:n] = w[entry, None] * dy
        dw[entry] = (dy * st["d"][:n]).sum(1)
        return {"dd": dd, "dw": dw.view(T, k)}
    I = case["I"]
    g, u, dh = st["gu"][:n, :I].double(), st["gu"][:n, I:].double(), st["dh"][:n].double()
    sig = torch.sigmoid(g)
    dw[entry] = (dh * u * g * sig).sum(1)
    dgu = torch.zeros((R, 2 * I), dtype=torch.float64, device=DEV)
    dgu[:n, :I] = dh * w[entry, None] * u * (sig + g * sig * torch.sigmoid(-g))
    dgu[:n, I:] = dh * w[entry, None] * g * sig
    return {"dgu": dgu, "dw": dw.view(T, k)}
