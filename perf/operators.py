"""The 8-bit floating-point and expert-routing operators: cases, plain forms and exact values.

Four operators, as a layer of routed experts with 8-bit weights uses them one after the other:

  pack     x or W -> e4m3 codes with one fp32 scale for each block of 128 (1 x 128 of activations,
           128 x 128 of weights): scale = max|v| / 448 (0 -> 1), code = e4m3(v / scale). Activations
           may be silu(gate) * up of rows that hold gate and up side by side.
  gemm     y[m, n] = sum over blocks b of k: xs[m, b] * ws[n / 128, b] * sum of x[m, k] * w[n, k]
  grouped  the same product for rows sorted by expert, each expert with weights of its own
  route    tokens sorted by expert (stable), gathered, and back: out[t] = sum over j of
           weight[t, j] * ys[pos[t, j]]; and its gradients by ys, the weights and x

`run` computes them in elementary torch operations, or, where `own` is true, by the calls of the
framework.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
F8 = torch.float8_e4m3fn
MOST = 448.0  # the largest finite e4m3 value


def listed():
    return [
        # a decode step's rows before a projection: latency
        {"name": "pack-16x4096", "op": "pack", "what": "rows", "M": 16, "K": 4096, "x": "bf16", "silu": False},
        # prefill: the hidden rows of a gated MLP, silu(gate) * up, before the down projection
        {"name": "pack-silu-8192x14336", "op": "pack", "what": "rows", "M": 8192, "K": 14336, "x": "bf16", "silu": True},
        # a weight matrix, once when a model is loaded
        {"name": "pack-weights-14336x4096", "op": "pack", "what": "weights", "M": 14336, "K": 4096, "x": "f32", "silu": False},
        # one token through a square projection: latency, and the weights' bytes
        {"name": "gemm-1x4096x4096", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "y": "bf16"},
        # a ragged batch of short prompts through an MLP projection, fp32 out for a residual sum
        {"name": "gemm-333x11008x4096", "op": "gemm", "M": 333, "N": 11008, "K": 4096, "y": "f32"},
        # prefill of a long batch
        {"name": "gemm-8192x14336x4096", "op": "gemm", "M": 8192, "N": 14336, "K": 4096, "y": "bf16"},
        # 16 decoding tokens, two of eight large experts each
        {"name": "grouped-8x14336x4096-t16", "op": "grouped", "T": 16, "k": 2, "E": 8, "N": 14336, "K": 4096, "y": "bf16"},
        # prefill with many small experts, eight a token
        {"name": "grouped-64x1408x2048-t4096", "op": "grouped", "T": 4096, "k": 8, "E": 64, "N": 1408, "K": 2048, "y": "bf16"},
        # routing of a decode step
        {"name": "route-32x4096-k8of64", "op": "route", "what": "forward", "T": 32, "k": 8, "E": 64, "D": 4096, "x": "bf16"},
        # routing of a prefill batch
        {"name": "route-8192x4096-k8of256", "op": "route", "what": "forward", "T": 8192, "k": 8, "E": 256, "D": 4096, "x": "bf16"},
        # the gradients of a training step's routing
        {"name": "route-grad-4096x4096-k8of64", "op": "route", "what": "backward", "T": 4096, "k": 8, "E": 64, "D": 4096, "x": "bf16"},
        # the same in fp32 with an odd hidden size, a small fine-tuning batch
        {"name": "route-grad-1001x1023-k2of8", "op": "route", "what": "backward", "T": 1001, "k": 2, "E": 8, "D": 1023, "x": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pack", "gemm", "grouped", "route"])
    y = rng.choice(["bf16", "f16", "f32"])
    while True:
        if op == "pack":
            what = rng.choice(["rows", "rows", "weights"])
            c = {"op": op, "what": what, "M": _log(rng, 1, 14336), "K": _log(rng, 64, 14336), "x": y,
                 "silu": what == "rows" and rng.random() < 0.5}
            if c["M"] * c["K"] <= 8192 * 14336:
                return c
        elif op == "gemm":
            # rows of codes are whole 16-byte units: the entry point refuses other K
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 14336), "K": 16 * _log(rng, 8, 896), "y": y}
            if c["M"] * c["N"] * c["K"] <= 8192 * 14336 * 4096 and c["N"] * c["K"] <= 14336 * 4096:
                return c
        elif op == "grouped":
            E = _log(rng, 2, 64)
            c = {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, min(8, E)), "E": E, "N": _log(rng, 64, 14336),
                 "K": 16 * _log(rng, 8, 896), "y": y}
            if c["T"] * c["k"] * c["N"] * c["K"] <= 32768 * 1408 * 2048 and E * c["N"] * c["K"] <= 8 * 14336 * 4096:
                return c
        else:
            E = _log(rng, 2, 256)
            c = {"op": op, "what": rng.choice(["forward", "backward"]), "T": _log(rng, 1, 8192), "k": rng.randint(1, min(8, E)),
                 "E": E, "D": _log(rng, 64, 8192), "x": y}
            if c["T"] * c["k"] * c["D"] <= 4096 * 8 * 4096:
                return c


# ---- inputs -----------------------------------------------------------------------------
def _codes(gen, *shape):
    """Codes as normal values come out of a block's rounding: the block's largest is 448."""
    return torch.randn(*shape, device="cuda", generator=gen).mul_(110.0).clamp_(-MOST, MOST).to(F8)


def _scales(gen, typical, *shape):
    return torch.randn(*shape, device="cuda", generator=gen).mul_(0.3).exp_().mul_(typical / 110.0)


def _blocks(n):
    return (n + 127) // 128


def _experts(gen, T, k, E):
    """Top-k experts of each token, some experts liked more than others; the weights sum to 1."""
    logits = torch.randn(T, E, device="cuda", generator=gen) + 0.5 * torch.randn(E, device="cuda", generator=gen)
    top = torch.topk(logits, k, dim=1)
    return top.indices, torch.softmax(top.values, 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "pack":
        M, K = case["M"], case["K"]
        x = torch.randn(M, (2 if case["silu"] else 1) * K, device="cuda", generator=gen)
        if case["what"] == "rows":
            x[:, :: 97] *= 8.0  # the few large channels of real activations
        else:
            x *= 0.02
        s["x"] = x.to(DT[case["x"]])
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"], s["xs"] = _codes(gen, M, K), _scales(gen, 1.0, M, _blocks(K))
        s["w"], s["ws"] = _codes(gen, N, K), _scales(gen, 0.02, _blocks(N), _blocks(K))
    elif op == "grouped":
        E, N, K = case["E"], case["N"], case["K"]
        ids, _ = _experts(gen, case["T"], case["k"], E)
        rows = (ids.reshape(-1, 1) == torch.arange(E, device="cuda")).sum(0)
        s["offsets"] = torch.cat([rows.new_zeros(1), rows.cumsum(0)]).to(torch.int32)
        s["most"] = int(rows.max())  # rows of the fullest expert
        R = case["T"] * case["k"]
        s["x"], s["xs"] = _codes(gen, R, K), _scales(gen, 1.0, R, _blocks(K))
        s["w"], s["ws"] = _codes(gen, E, N, K), _scales(gen, 0.02, E, _blocks(N), _blocks(K))
    else:
        T, k, E, D = case["T"], case["k"], case["E"], case["D"]
        s["ids"], s["weights"] = _experts(gen, T, k, E)
        # the experts' answers and, for the backward pass, the gradients from above and from the experts
        s["ys"] = torch.randn(T * k, D, device="cuda", generator=gen).to(DT[case["x"]])
        s["x"] = torch.randn(T, D, device="cuda", generator=gen).to(DT[case["x"]])
        if case["what"] == "backward":
            s["dxs"] = torch.randn(T * k, D, device="cuda", generator=gen).to(DT[case["x"]])
            flat = s["ids"].reshape(-1)
            order = torch.sort(flat, stable=True).indices
            pos = torch.empty_like(order)
            pos[order] = torch.arange(T * k, device="cuda")
            s["pos"] = pos.reshape(T, k).to(torch.int32)
    return s


# ---- one pass -----------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"pack": _pack, "gemm": _gemm, "grouped": _grouped, "route": _route}[s["case"]["op"]](s)


def _run_own(s):
    import int4_quantized_b200 as q4

    c = s["case"]
    if c["op"] == "pack":
        return q4.fp8_pack(s["x"], silu_mul=c["silu"]) if c["what"] == "rows" else q4.fp8_pack_weights(s["x"])
    if c["op"] == "gemm":
        return q4.fp8_gemm(s["x"], s["xs"], s["w"], s["ws"], out_dtype=DT[c["y"]])
    if c["op"] == "grouped":
        return q4.fp8_gemm_grouped(s["x"], s["xs"], s["w"], s["ws"], s["offsets"], out_dtype=DT[c["y"]])
    if c["what"] == "forward":
        tokens, pos, offsets = q4.moe_sort(s["ids"], c["E"])
        return tokens, pos, offsets, q4.moe_gather(s["x"], tokens), q4.moe_combine(s["ys"], pos, s["weights"])
    dys, dweights = q4.moe_combine_backward(s["x"], s["ys"], s["pos"], s["weights"])
    return dys, dweights, q4.moe_combine(s["dxs"], s["pos"])


def _pack(s):
    c, x = s["case"], s["x"].float()
    K = c["K"]
    if c["silu"]:
        gate, up = x[:, :K], x[:, K:]
        x = gate / (1 + torch.exp(-gate)) * up
    rows = 128 if c["what"] == "weights" else 1
    M, P, Q = c["M"], -(-c["M"] // rows), _blocks(K)
    x = torch.nn.functional.pad(x, (0, Q * 128 - K, 0, P * rows - M)).view(P, rows, Q, 128)
    scales = x.abs().amax(dim=(1, 3)) / MOST
    scales = torch.where(scales == 0, torch.ones_like(scales), scales)
    codes = (x / scales[:, None, :, None]).clamp_(-MOST, MOST).to(F8).view(P * rows, Q * 128)
    return codes[:M, :K].contiguous(), scales


def _spread(scales, n, dim):
    """One scale for each of n values from one for each 128 of them."""
    return scales.repeat_interleave(128, dim=dim).narrow(dim, 0, n)


def _gemm(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    x = s["x"].float() * _spread(s["xs"], K, 1)
    w = s["w"].float() * _spread(_spread(s["ws"], N, 0), K, 1)
    return (x @ w.t()).to(DT[c["y"]])


def _grouped(s):
    c = s["case"]
    E, N, K, most = c["E"], c["N"], c["K"], s["most"]
    x = s["x"].float() * _spread(s["xs"], K, 1)
    first, last = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    row = first + torch.arange(most, device="cuda")
    live = row < last
    w = s["w"].float() * _spread(_spread(s["ws"], N, 1), K, 2)
    y = torch.bmm(x[row.clamp(max=x.shape[0] - 1)], w.transpose(1, 2))  # the experts' rows side by side, padded to the fullest
    return y[live].to(DT[c["y"]])  # the true places, in order: the sorted rows


def _sort(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device="cuda")
    rows = (flat[:, None] == torch.arange(E, device="cuda")).sum(0)
    offsets = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    return (order // k).to(torch.int32), pos.reshape(T, k).to(torch.int32), offsets.to(torch.int32)


def _route(s):
    c, w = s["case"], s["weights"][..., None]
    if c["what"] == "forward":
        tokens, pos, offsets = _sort(s["ids"], c["E"])
        out = (s["ys"][pos].float() * w).sum(1).to(DT[c["x"]])
        return tokens, pos, offsets, s["x"][tokens], out
    pos, dout = s["pos"], s["x"].float()[:, None, :]
    dys = torch.empty_like(s["ys"])
    dys[pos.reshape(-1)] = (w * dout).to(dys.dtype).reshape(-1, c["D"])
    dweights = (s["ys"][pos].float() * dout).sum(2)
    return dys, dweights, s["dxs"][pos].float().sum(1).to(DT[c["x"]])


# ---- what a pass cannot do without --------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "pack":
        M, K, rows = case["M"], case["K"], 128 if case["what"] == "weights" else 1
        n = M * K
        read = n * SIZE[case["x"]] * (2 if case["silu"] else 1)
        return {"bytes": read + n + 4 * -(-M // rows) * _blocks(K), "flops": n * (8 if case["silu"] else 3)}
    if op in ("gemm", "grouped"):
        N, K, kb = case["N"], case["K"], _blocks(case["K"])
        if op == "gemm":
            R, used = case["M"], 1
        else:
            R, used = case["T"] * case["k"], min(case["E"], case["T"] * case["k"])  # experts with rows, at most
        return {"bytes": R * (K + 4 * kb + N * SIZE[case["y"]]) + used * (N * K + 4 * _blocks(N) * kb), "flops": 2 * R * N * K}
    T, k, D, size = case["T"], case["k"], case["D"], SIZE[case["x"]]
    R = T * k
    if case["what"] == "forward":
        # ids, x, ys, weights in; tokens, pos, offsets, the sorted rows, out
        return {"bytes": R * 8 + T * D * size + R * D * size + R * 4 + R * 8 + 4 * case["E"] + R * D * size + T * D * size, "flops": 2 * R * D}
    # dout, ys, dxs, pos, weights in; dys, dweights, dx out
    return {"bytes": T * D * size + 2 * R * D * size + R * 8 + R * D * size + R * 4 + T * D * size, "flops": 4 * R * D}


# ---- the definition in 64 bits --------------------------------------------------------------
def _dequantized(codes, scales, rows):
    """float64 values of codes [.., n, K] whose blocks are rows x 128."""
    n, K = codes.shape[-2:]
    i = torch.arange(n, device="cuda") // rows
    b = torch.arange(K, device="cuda") // 128
    return codes.double() * scales.double()[..., i, :][..., b]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "pack":
        v, K, rows = s["x"].double(), case["K"], 128 if case["what"] == "weights" else 1
        if case["silu"]:
            v = torch.sigmoid(v[:, :K]) * v[:, :K] * v[:, K:]
        M = case["M"]
        i, b = torch.arange(M, device="cuda") // rows, torch.arange(K, device="cuda") // 128
        by_row = torch.stack([part.abs().amax(1) for part in v.split(128, 1)], 1)
        scales = by_row.new_zeros(-(-M // rows), by_row.shape[1]).index_reduce_(0, i, by_row, "amax") / MOST
        scales[scales == 0] = 1.0
        q = v / scales[i][:, b]
        # nearest of the e4m3 values, ties to even: steps of 2^(e - 3), e the exponent, at least -6
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(q / step) * step).clamp(-MOST, MOST), scales
    if op == "gemm":
        return _dequantized(s["x"], s["xs"], 1) @ _dequantized(s["w"], s["ws"], 128).t()
    if op == "grouped":
        at = s["offsets"].tolist()
        parts = [_dequantized(s["x"][a:b], s["xs"][a:b], 1) @ _dequantized(s["w"][e], s["ws"][e], 128).t()
                 for e, (a, b) in enumerate(zip(at, at[1:]))]
        return torch.cat(parts)
    w, T, k, D = s["weights"].double(), case["T"], case["k"], case["D"]
    if case["what"] == "forward":
        # rank of each choice: those of lower experts, then the earlier ones of its own
        flat = s["ids"].reshape(-1)
        R, E = T * k, case["E"]
        mine = flat[:, None] == torch.arange(E, device="cuda")
        rows = mine.sum(0)
        offsets = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
        pos = offsets[flat] + mine.to(torch.int32).cumsum(0).gather(1, flat[:, None])[:, 0] - 1
        tokens = torch.empty(R, dtype=torch.int64, device="cuda")
        tokens[pos] = torch.arange(R, device="cuda") // k
        pos = pos.reshape(T, k)
        out = torch.zeros(T, D, dtype=torch.float64, device="cuda")
        for j in range(k):
            out += w[:, j, None] * s["ys"][pos[:, j]].double()
        return tokens, pos, offsets, s["x"].double()[tokens], out
    dys = torch.zeros(T * k, D, dtype=torch.float64, device="cuda")
    dweights = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    dx = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for j in range(k):
        at = s["pos"][:, j].long()
        dys[at] = w[:, j, None] * s["x"].double()
        dweights[:, j] = (s["ys"][at].double() * s["x"].double()).sum(1)
        dx += s["dxs"][at].double()
    return dys, dweights, dx
