"""The FP8 operators and the BF16 weight gradient of the MoE layer, as cases that can be timed and checked.

Each case names one operator (``op``) and its sizes; ``prepare`` draws its inputs on the GPU from a seed,
``run`` makes one pass (``own`` selects the library's kernels, else plain torch arithmetic in 32 bits), and
``exact`` gives the operator's definition in 64 bits.

Definitions (e4m3 = E4M3fn, largest value 448; a block is 128 consecutive elements, the last may be shorter):

* ``rows``    FP8 rows: per row and block s = max|x| / 448, code = e4m3(x / s); scales are [blocks, rows].
* ``weights`` FP8 weights: one s per 128 x 128 block of each [N, K] matrix; the transposed matrices too.
* ``swiglu``  h = g / (1 + exp(-g)) * u * w per routed row, quantised like ``rows``, with h in bf16 beside it.
* ``gemm``    c[r, n] = sum_j sa[j, r] sw[e, n / 128, j] sum_(k in j) a[r, k] w[e, n, k] for r in expert e's rows.
* ``wgrad``   dW[e, m, n] = sum over expert e's rows r of g[r, m] x[r, n].
"""
import math

import torch

own = False

BLOCK = 128
F8 = torch.float8_e4m3fn
DEV = "cuda"


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token's activations (the hidden size of the layer), where the launch is what costs
        {"name": "rows_one_token", "op": "rows", "rows": 1, "K": 2048, "dtype": "bf16"},
        # float32 rows of a training batch whose length is no multiple of the block (an odd row count too)
        {"name": "rows_f32_ragged", "op": "rows", "rows": 32771, "K": 784, "dtype": "f32"},
        # the dense QKV projection's weight, quantised after an optimiser step, forward order alone
        {"name": "weights_qkv", "op": "weights", "E": 1, "N": 5120, "K": 2048, "transposed": False},
        # every expert's gate_up weight, both orders: the forward and the input gradient read one each
        {"name": "weights_experts", "op": "weights", "E": 128, "N": 1536, "K": 2048, "transposed": True},
        # one token's eight routed rows
        {"name": "swiglu_one_token", "op": "swiglu", "T": 1, "k": 8, "E": 128, "I": 768, "dtype": "f32",
         "weighted": True, "h_out": False, "routing": "softmax"},
        # a training batch: bf16 gate_up output, router weights, h kept for the weight gradient
        {"name": "swiglu_train", "op": "swiglu", "T": 4096, "k": 8, "E": 128, "I": 768, "dtype": "bf16",
         "weighted": True, "h_out": True, "routing": "softmax"},
        # one token through the experts' gate_up: eight weight matrices read for one row each
        {"name": "gemm_one_token", "op": "gemm", "T": 1, "k": 8, "E": 128, "N": 1536, "K": 2048,
         "gather": True, "out": "bf16", "routing": "softmax"},
        # a small serving batch through the experts' down projection
        {"name": "gemm_batch_61", "op": "gemm", "T": 61, "k": 8, "E": 128, "N": 2048, "K": 768,
         "gather": False, "out": "f32", "routing": "uniform"},
        # the layer's gate_up product at the training length, tokens gathered in the loads
        {"name": "gemm_gate_up", "op": "gemm", "T": 4096, "k": 8, "E": 128, "N": 1536, "K": 2048,
         "gather": True, "out": "bf16", "routing": "softmax"},
        # the dense QKV product
        {"name": "gemm_qkv", "op": "gemm", "T": 4096, "k": 1, "E": 1, "N": 5120, "K": 2048,
         "gather": False, "out": "f32", "routing": "softmax"},
        # the gate_up weight gradient at the training length
        {"name": "wgrad_gate_up", "op": "wgrad", "T": 4096, "k": 8, "E": 128, "M": 1536, "N": 2048,
         "gather": "x", "out": "f32", "routing": "softmax"},
        # a few skewed, odd-sized experts: long and empty contractions side by side
        {"name": "wgrad_skewed", "op": "wgrad", "T": 1021, "k": 4, "E": 24, "M": 520, "N": 328,
         "gather": "g", "out": "bf16", "routing": "zipf"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["rows", "weights", "swiglu", "gemm", "gemm", "wgrad"])
    if op == "rows":
        rows, K = _log(rng, 1, 40000), _log(rng, 16, 8192, 16)
        return {"op": op, "rows": max(1, min(rows, 60_000_000 // K)), "K": K, "dtype": rng.choice(["bf16", "f32"])}
    E = _log(rng, 1, 128)
    if op == "weights":
        N, K = _log(rng, 48, 5120, 16), _log(rng, 48, 5120, 16)
        return {"op": op, "E": max(1, min(E, 400_000_000 // (N * K))), "N": N, "K": K,
                "transposed": rng.random() < 0.5}
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 4096)
    routing = rng.choice(["softmax", "uniform", "zipf"])
    if op == "swiglu":
        return {"op": op, "T": T, "k": k, "E": E, "I": _log(rng, 16, 2048, 16), "dtype": rng.choice(["bf16", "f32"]),
                "weighted": rng.random() < 0.7, "h_out": rng.random() < 0.5, "routing": routing}
    if op == "gemm":
        N, K = _log(rng, 24, 5120), _log(rng, 64, 4096, 16)
        E = max(1, min(E, 400_000_000 // (N * K)))
        k = min(k, E)
        T = max(1, min(T, 90_000_000_000 // (k * N * K)))
        return {"op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "gather": rng.random() < 0.5,
                "out": rng.choice(["bf16", "f32"]), "routing": routing}
    M, N = _log(rng, 24, 2560, 8), _log(rng, 24, 2560, 8)
    E = max(1, min(E, 400_000_000 // (M * N)))
    k = min(k, E)
    T = max(1, min(T, 100_000_000_000 // (k * M * N)))
    return {"op": op, "T": T, "k": k, "E": E, "M": M, "N": N, "gather": rng.choice(["g", "x", "none"]),
            "out": rng.choice(["bf16", "f32"]), "routing": routing}


# ------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _activations(gen, shape, dtype=torch.bfloat16):
    """N(0, 1) with one element in a hundred twenty times larger."""
    x = torch.randn(shape, generator=gen, device=DEV)
    big = torch.rand(shape, generator=gen, device=DEV) < 0.01
    return torch.where(big, 20 * x, x).to(dtype)


def _routing(gen, case):
    """ids -> the expert-grouped order: offsets [E + 1], row_to_tk [T k] (stable), router weights [T k]."""
    T, k, E = case["T"], case["k"], case["E"]
    score = torch.rand((T, E), generator=gen, device=DEV)
    if case["routing"] == "softmax":
        score = torch.randn((T, E), generator=gen, device=DEV)
    elif case["routing"] == "zipf":
        gumbel = -torch.log(-torch.log(score.clamp(1e-7, 1 - 1e-7)))
        score = gumbel - 1.2 * torch.log(torch.arange(1, E + 1, device=DEV))
    top, ids = score.topk(k, dim=1)
    ids = ids.reshape(-1)
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return {"offsets": offsets, "row_to_tk": ids.argsort(stable=True).int(),
            "topk_w": torch.softmax(top, 1).reshape(-1).contiguous(), "most": int(counts.max())}


def _fp8_rows(x):
    """Quantised rows (codes, scales [blocks, rows])."""
    rows, K = x.shape
    nb = -(-K // BLOCK)
    x = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - K)).view(rows, nb, BLOCK)
    s = x.abs().amax(2) / 448.0
    q = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros((), device=x.device))
    codes = q.clamp(-448, 448).to(F8).view(rows, nb * BLOCK)[:, :K].contiguous()
    return codes, s.t().contiguous()


def _fp8_weights(w):
    """Quantised 128 x 128 blocks of [E, N, K] (codes, scales [E, N blocks, K blocks])."""
    E, N, K = w.shape
    nn, nk = -(-N // BLOCK), -(-K // BLOCK)
    w = torch.nn.functional.pad(w.float(), (0, nk * BLOCK - K, 0, nn * BLOCK - N)).view(E, nn, BLOCK, nk, BLOCK)
    s = w.abs().amax((2, 4)) / 448.0
    wide = s[:, :, None, :, None]
    q = torch.where(wide > 0, w / wide, torch.zeros((), device=w.device))
    codes = q.clamp(-448, 448).to(F8).view(E, nn * BLOCK, nk * BLOCK)[:, :N, :K].contiguous()
    return codes, s


def prepare(case, seed):
    gen, op = _gen(seed), case["op"]
    if op == "rows":
        return {"case": case, "x": _activations(gen, (case["rows"], case["K"]), torch.float32 if case["dtype"] == "f32" else torch.bfloat16)}
    if op == "weights":
        w = torch.randn((case["E"], case["N"], case["K"]), generator=gen, device=DEV, dtype=torch.float32)
        return {"case": case, "w": (0.02 * w).bfloat16()}
    st = {"case": case, **_routing(gen, case)}
    R = case["T"] * case["k"]
    if op == "swiglu":
        gu = torch.randn((R, 2 * case["I"]), generator=gen, device=DEV)
        st["gu"] = gu if case["dtype"] == "f32" else gu.bfloat16()
    elif op == "gemm":
        a = _activations(gen, (case["T"] if case["gather"] else R, case["K"]))
        w = 0.02 * torch.randn((case["E"], case["N"], case["K"]), generator=gen, device=DEV)
        ac, st["a_scales"] = _fp8_rows(a)
        wc, st["w_scales"] = _fp8_weights(w.bfloat16())
        st["a_codes"], st["w_codes"] = ac.view(torch.uint8), wc.view(torch.uint8)
    else:
        rows = {n: case["T"] if case["gather"] == n else R for n in ("g", "x")}
        st["g"] = (0.01 * torch.randn((rows["g"], case["M"]), generator=gen, device=DEV)).bfloat16()
        st["x"] = _activations(gen, (rows["x"], case["N"]))
    return st


# ------------------------------------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    import precision_moe_gemm_amd as pmg
    case = st["case"]
    op = case["op"]
    if op == "rows":
        codes, scales = pmg.fp8_quantize_rows(st["x"])
        return {"codes": codes.view(F8), "scales": scales}
    if op == "weights":
        got = pmg.fp8_quantize_weights(st["w"], transposed=case["transposed"])
        out = {"codes": got[0].view(F8), "scales": got[1]}
        if case["transposed"]:
            out |= {"codes_t": got[2].view(F8), "scales_t": got[3]}
        return out
    if op == "swiglu":
        tw, tk = (st["topk_w"], st["row_to_tk"]) if case["weighted"] else (None, None)
        codes, scales, h = pmg.fp8_swiglu_quantize(st["gu"], st["offsets"], tw, tk, h_out=case["h_out"])
        return {"codes": codes.view(F8), "scales": scales, "h": h}
    dt = torch.float32 if case["out"] == "f32" else torch.bfloat16
    if op == "gemm":
        if case["gather"]:
            return pmg.fp8_grouped_gemm_gather(st["a_codes"], st["a_scales"], st["row_to_tk"], case["k"], st["offsets"],
                                               st["w_codes"], st["w_scales"], out_dtype=dt)
        return pmg.fp8_grouped_gemm(st["a_codes"], st["a_scales"], st["offsets"], st["w_codes"], st["w_scales"],
                                    out_dtype=dt)
    if case["gather"] == "none":
        return pmg.bf16_grouped_gemm_wgrad(st["g"], st["x"], st["offsets"], out_dtype=dt)
    return pmg.bf16_grouped_gemm_wgrad(st["g"], st["x"], st["offsets"], row_to_tk=st["row_to_tk"], k=case["k"],
                                       gather=case["gather"], out_dtype=dt)


def _padded(st, x):
    """Expert-grouped rows [R, C] -> [E, most, C], zero past an expert's rows."""
    off = st["offsets"].long()
    at = off[:-1, None] + torch.arange(st["most"], device=x.device)
    live = at < off[1:, None]
    return x[at.clamp(max=x.shape[0] - 1)] * live[..., None]


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "rows":
        codes, scales = _fp8_rows(st["x"])
        return {"codes": codes, "scales": scales}
    if op == "weights":
        codes, scales = _fp8_weights(st["w"])
        out = {"codes": codes, "scales": scales}
        if case["transposed"]:
            out |= {"codes_t": codes.view(torch.uint8).transpose(1, 2).contiguous().view(F8),
                    "scales_t": scales.transpose(1, 2).contiguous()}
        return out
    if op == "swiglu":
        g, u = st["gu"].float().split(case["I"], dim=1)
        h = g / (1 + torch.exp(-g)) * u
        if case["weighted"]:
            h = h * st["topk_w"][st["row_to_tk"].long()][:, None]
        codes, scales = _fp8_rows(h)
        return {"codes": codes, "scales": scales, "h": h.bfloat16() if case["h_out"] else None}
    dt = torch.float32 if case["out"] == "f32" else torch.bfloat16
    token = st["row_to_tk"].long() // case["k"]
    if op == "gemm":
        a = st["a_codes"].view(F8).float() * st["a_scales"].t().repeat_interleave(BLOCK, 1)[:, :case["K"]]
        sw = st["w_scales"].repeat_interleave(BLOCK, 1)[:, :case["N"]]
        w = st["w_codes"].view(F8).float() * sw.repeat_interleave(BLOCK, 2)[:, :, :case["K"]]
        a = _padded(st, a[token] if case["gather"] else a)
        c = torch.bmm(a, w.transpose(1, 2).contiguous())
        row = torch.arange(case["T"] * case["k"], device=a.device)
        off = st["offsets"].long()
        e = torch.searchsorted(off[1:].contiguous(), row, right=True)
        return c[e, row - off[e]].to(dt)
    g, x = st["g"].float(), st["x"].float()
    g = _padded(st, g[token] if case["gather"] == "g" else g)
    x = _padded(st, x[token] if case["gather"] == "x" else x)
    return torch.bmm(g.transpose(1, 2).contiguous(), x).to(dt)


# ------------------------------------------------------------------------------------------- work
def _touched(case):
    """Experts that get rows, about: every draw of a token's k distinct experts touches k of them."""
    E, k, T = case["E"], case["k"], case["T"]
    return min(E, T * k) if T * k <= E else E * (1 - (1 - k / E) ** T)


def work(case):
    op = case["op"]
    size = 4 if "f32" in (case.get("dtype"), case.get("out")) else 2
    if op == "rows":
        n = case["rows"] * case["K"]
        return {"bytes": n * (size + 1) + 4 * case["rows"] * -(-case["K"] // BLOCK), "flops": 3 * n}
    if op == "weights":
        n = case["E"] * case["N"] * case["K"]
        blocks = case["E"] * -(-case["N"] // BLOCK) * -(-case["K"] // BLOCK)
        return {"bytes": 2 * n + (n + 4 * blocks) * (2 if case["transposed"] else 1), "flops": 3 * n}
    R = case["T"] * case["k"]
    if op == "swiglu":
        n = R * case["I"]
        return {"bytes": n * (2 * size + 1 + (2 if case["h_out"] else 0)) + 4 * R * -(-case["I"] // BLOCK)
                + (8 * R if case["weighted"] else 0), "flops": 10 * n}
    if op == "gemm":
        N, K = case["N"], case["K"]
        rows = case["T"] if case["gather"] else R
        return {"bytes": rows * (K + 4 * -(-K // BLOCK)) + _touched(case) * N * K + R * N * size
                + (4 * R if case["gather"] else 0), "flops": 2 * R * N * K}
    M, N = case["M"], case["N"]
    rows = {n: case["T"] if case["gather"] == n else R for n in ("g", "x")}
    return {"bytes": 2 * (rows["g"] * M + rows["x"] * N) + case["E"] * M * N * size, "flops": 2 * R * M * N}


# ------------------------------------------------------------------------------------------- exact
def _e4m3_64(v):
    """The nearest e4m3 value of each float64, ties to the even significand, no larger than 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp(min=-9))
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _blocks_64(v, dims):
    """e4m3 values and scales of float64 blocks laid along `dims`."""
    s = v.abs().amax(dims, keepdim=True) / 448.0
    return _e4m3_64(torch.where(s > 0, v / s, torch.zeros_like(v))), s.squeeze(dims)


def _rows_64(x):
    rows, K = x.shape
    nb = (K + BLOCK - 1) // BLOCK
    v = torch.zeros((rows, nb * BLOCK), dtype=torch.float64, device=x.device)
    v[:, :K] = x
    q, s = _blocks_64(v.reshape(rows, nb, BLOCK), (2,))
    return q.reshape(rows, -1)[:, :K].contiguous(), s.t().contiguous()


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "rows":
        q, s = _rows_64(st["x"].double())
        return {"codes": q, "scales": s}
    if op == "weights":
        E, N, K = st["w"].shape
        codes = torch.empty((E, N, K), dtype=torch.float64, device=DEV)
        scales = torch.empty((E, -(-N // BLOCK), -(-K // BLOCK)), dtype=torch.float64, device=DEV)
        nn, nk = scales.shape[1:]
        for e in range(E):
            v = torch.zeros((nn * BLOCK, nk * BLOCK), dtype=torch.float64, device=DEV)
            v[:N, :K] = st["w"][e]
            q, scales[e] = _blocks_64(v.reshape(nn, BLOCK, nk, BLOCK), (1, 3))
            codes[e] = q.reshape(nn * BLOCK, nk * BLOCK)[:N, :K]
        out = {"codes": codes, "scales": scales}
        if case["transposed"]:
            out |= {"codes_t": codes.transpose(1, 2).contiguous(), "scales_t": scales.transpose(1, 2).contiguous()}
        return out
    if op == "swiglu":
        gu, I = st["gu"].double(), case["I"]
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        if case["weighted"]:
            h *= st["topk_w"].double()[st["row_to_tk"].long()].unsqueeze(1)
        q, s = _rows_64(h)
        return {"codes": q, "scales": s, "h": h if case["h_out"] else None}
    off = st["offsets"].tolist()
    token = torch.div(st["row_to_tk"], case["k"], rounding_mode="floor").long()
    if op == "gemm":
        K, N = case["K"], case["N"]
        kb = torch.arange(K, device=DEV) // BLOCK
        nb = torch.arange(N, device=DEV) // BLOCK
        a = st["a_codes"].view(F8).double() * st["a_scales"].double()[kb].t()
        out = torch.zeros((case["T"] * case["k"], N), dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            r = torch.arange(off[e], off[e + 1], device=DEV)
            if len(r):
                w = st["w_codes"][e].view(F8).double() * st["w_scales"][e].double()[nb][:, kb]
                out[r] = a[token[r] if case["gather"] else r] @ w.t()
        return out
    out = torch.zeros((case["E"], case["M"], case["N"]), dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        r = torch.arange(off[e], off[e + 1], device=DEV)
        if len(r):
            g = st["g"][token[r] if case["gather"] == "g" else r].double()
            x = st["x"][token[r] if case["gather"] == "x" else r].double()
            out[e] = g.t() @ x
    return out
