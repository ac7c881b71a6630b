"""The microscaled (MXFP4) and mixture-of-experts operators of the library, as
cases to be measured: the same pass through the library's entry points
(own = True) or in plain torch operations (own = False).

Five operators, told apart by a case's "op":
  quantize  float rows -> 4-bit E2M1 codes with one power-of-two scale per 32
            elements, and back to the values they stand for;
  linear    C = act(A x W^T + bias) with MXFP4 weights W [N][K] and fp16
            activations ("mxfp4") or activations that are quantised to MXFP4
            on the way ("mxfp4a4");
  experts   the same product with ragged groups of rows, each against its own
            expert's weight, the rows gathered through an index;
  plan      the ragged layout (offsets, row index, inverse) of a router's
            choice; an id outside [0, E) is a choice of an expert elsewhere;
  combine   the weighted sum of every token's expert outputs.
"""
import math

import torch

own = False

BLOCK = 32          # elements that share a scale
# the 16 values of a code: sign bit 3, exponent bits 2:1, mantissa bit 0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the export of one 4096 x 4096 layer from float weights
        {"name": "quantize_layer", "op": "quantize", "R": 4096, "K": 4096, "type": "f32"},
        # one token's activations: the smallest call there is
        {"name": "quantize_token", "op": "quantize", "R": 1, "K": 2560, "type": "f16"},
        # decode of one token through a feed-forward layer: the weight stream
        {"name": "linear_decode", "op": "linear", "M": 1, "K": 4096, "N": 11008, "fmt": "mxfp4", "out": "f32",
         "act": "none"},
        # a 512-token prompt with fp16 activations
        {"name": "linear_prefill", "op": "linear", "M": 512, "K": 4096, "N": 4096, "fmt": "mxfp4", "out": "f32",
         "act": "none"},
        # a longer prompt with 4-bit activations, bias and activation fused, fp16 out
        {"name": "linear_prefill_a4", "op": "linear", "M": 2048, "K": 4096, "N": 11008, "fmt": "mxfp4a4",
         "out": "f16", "act": "silu"},
        # eight requests decoding: a row or two on most of 32 experts
        {"name": "experts_decode", "op": "experts", "T": 8, "topk": 4, "E": 32, "K": 2560, "N": 4096, "fmt": "mxfp4",
         "out": "f32", "act": "none"},
        # a prompt of 2000 tokens over 32 experts, ragged and skewed, with bias and SiLU
        {"name": "experts_prefill", "op": "experts", "T": 2000, "topk": 4, "E": 32, "K": 2560, "N": 4096,
         "fmt": "mxfp4", "out": "f16", "act": "silu"},
        # a batch of prompts with 4-bit activations
        {"name": "experts_prefill_a4", "op": "experts", "T": 4096, "topk": 4, "E": 32, "K": 4096, "N": 2560,
         "fmt": "mxfp4a4", "out": "f16", "act": "none"},
        # the layout of 16 decoding requests
        {"name": "plan_decode", "op": "plan", "T": 16, "topk": 8, "E": 128, "drop": 0.0},
        # the layout of a batch of prompts when a quarter of the experts live on another GPU
        {"name": "plan_prefill", "op": "plan", "T": 16384, "topk": 8, "E": 128, "drop": 0.25},
        # back to tokens: 16 decoding requests, and a batch of prompts with some experts elsewhere
        {"name": "combine_decode", "op": "combine", "T": 16, "topk": 8, "E": 128, "N": 2560, "type": "f32",
         "out": "f16", "drop": 0.0},
        {"name": "combine_prefill", "op": "combine", "T": 4099, "topk": 4, "E": 32, "N": 4096, "type": "f16",
         "out": "f16", "drop": 0.1},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "experts", "experts", "plan", "combine"])
    if op == "quantize":
        R, K = _log(rng, 1, 8192), BLOCK * _log(rng, 1, 512)
        while R * K > 4096 * 4096:
            R = (R + 1) // 2
        return {"op": op, "R": R, "K": K, "type": rng.choice(list(TYPES))}
    if op == "linear":
        M, K, N = _log(rng, 1, 2048), 64 * _log(rng, 2, 256), _log(rng, 33, 16384)
        while M * K * N > 2048 * 4096 * 11008 or K * N > 4096 * 16384:
            N = (N + 1) // 2
        return {"op": op, "M": M, "K": K, "N": N, "fmt": rng.choice(["mxfp4", "mxfp4a4"]),
                "out": rng.choice(["f32", "f16"]), "act": rng.choice(["none", "relu", "silu"])}
    topk, E = rng.randint(1, 8), _log(rng, 8, 256)
    drop = rng.choice([0.0, 0.1, 0.5])
    if op == "plan":
        return {"op": op, "T": _log(rng, 1, 16384), "topk": topk, "E": E, "drop": drop}
    if op == "combine":
        T, N = _log(rng, 1, 8192), _log(rng, 64, 8192)
        while T * topk * N > 4099 * 4 * 4096:
            T = (T + 1) // 2
        return {"op": op, "T": T, "topk": topk, "E": E, "N": N, "type": rng.choice(["f32", "f16"]),
                "out": rng.choice(["f32", "f16"]), "drop": drop}
    T, K, N = _log(rng, 1, 4096), 64 * _log(rng, 2, 128), _log(rng, 64, 4096)
    while E * K * N > 32 * 4096 * 2560:
        E, N = max(8, E // 2), (N + 1) // 2
    while T * topk * K * N > 4096 * 4 * 4096 * 2560:
        T = (T + 1) // 2
    return {"op": op, "T": T, "topk": topk, "E": E, "K": K, "N": N, "fmt": rng.choice(["mxfp4", "mxfp4a4"]),
            "out": rng.choice(["f32", "f16"]), "act": rng.choice(["none", "relu", "silu"])}


def work(case):
    op = case["op"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if op == "quantize":     # the floats in, the codes and scales, the values out
        n = case["R"] * case["K"]
        return {"bytes": n * (size[case["type"]] + 4 + 1 / 2 + 1 / BLOCK), "flops": 4 * n}
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": K * N * 17 / 32 + 2 * M * K + M * N * size[case["out"]], "flops": 2 * M * K * N}
    if op == "plan":
        S = case["T"] * case["topk"]
        return {"bytes": 8 * S + 2 * 4 * S + 4 * (case["E"] + 1), "flops": S}
    S = case["T"] * case["topk"]
    if op == "combine":
        kept = S * (1 - case["drop"]) * case["N"]
        return {"bytes": kept * size[case["type"]] + case["T"] * case["N"] * size[case["out"]] + 8 * S,
                "flops": 2 * kept}
    K, N, E = case["K"], case["N"], case["E"]
    reached = E * (1 - (1 - 1 / E) ** S)      # experts that have a row, if every one were as likely
    return {"bytes": reached * K * N * 17 / 32 + 2 * case["T"] * K + S * N * size[case["out"]] + 8 * S,
            "flops": 2 * S * K * N}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normal(shape, seed, salt, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000 + salt)
    return torch.randn(shape, generator=g, device="cuda") * scale


def _activations(rows, K, seed, salt):
    """Activations as a layer sees them: normal, a few channels twenty times the rest."""
    a = _normal((rows, K), seed, salt)
    a[:, _normal((K,), seed, salt + 1).abs() > 2.9] *= 20.0
    return a


def _choice(case, seed):
    """A router's choice: topk different experts for every token, some experts far likelier
    than others, and for a share of the choices an expert that is not here (id E or more)."""
    T, E = case["T"], case["E"]
    liking = _normal((1, E), seed, 1) * 1.5 + _normal((T, E), seed, 2)
    ids = torch.topk(liking, case["topk"], dim=1).indices
    if case.get("drop"):
        g = torch.Generator(device="cuda").manual_seed(seed * 1000 + 3)
        away = torch.rand(ids.shape, generator=g, device="cuda") < case["drop"]
        ids = torch.where(away, ids + E, ids)
    return ids


def _layout(ids, E):
    """offsets [E + 1], rows [S], slots [T][topk] of a choice, all int32."""
    T, topk = ids.shape
    key = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=key.device)
    offsets[1:] = torch.cumsum(counts, 0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=key.device)
    slots = torch.where(key < E, place, -1).reshape(T, topk)
    return offsets, (order // topk).to(torch.int32), slots.to(torch.int32)


def _encode(x):
    """Codes [R][K / 2] (low nibble first) and scale bytes [R][K / 32] of float rows."""
    R, K = x.shape
    v = x.float().reshape(R, K // BLOCK, BLOCK)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, (torch.frexp(top).exponent - 3).clamp(-127, 127), -127)
    y = torch.ldexp(v.abs(), -e)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6.0)
    # 0 .5 1 1.5 | 2 3 | 4 6 -> 0 1 2 3 | 4 5 | 6 7
    code = torch.where(y < 2, y * 2, torch.where(y < 4, y + 2, y / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).reshape(R, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8).reshape(R, K // BLOCK)


def _decode(q, s, dtype=torch.float32):
    """The values of codes and scales."""
    table = torch.tensor(E2M1, dtype=dtype, device=q.device)
    v = torch.stack((table[(q & 15).long()], table[(q >> 4).long()]), -1)
    scale = torch.ldexp(torch.ones((), dtype=dtype, device=q.device), s.to(torch.int32) - 127)
    return (v.reshape(*s.shape, BLOCK) * scale[..., None]).reshape(*q.shape[:-1], 2 * q.shape[-1])


def _weights(case, seed, E):
    """E experts' canonical codes [E][N][K / 2] and scales [E][N][K / 32]."""
    K, N = case["K"], case["N"]
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, N, K // BLOCK), dtype=torch.uint8, device="cuda")
    for e in range(E):
        q[e], s[e] = _encode(_normal((N, K), seed, 100 + e, 0.02))
    return q, s


def prepare(case, seed):
    op = case["op"]
    if op == "quantize":
        return {"case": case, "X": _activations(case["R"], case["K"], seed, 10).to(TYPES[case["type"]])}
    if op == "plan":
        return {"case": case, "ids": _choice(case, seed)}
    if op == "combine":
        T, topk, N = case["T"], case["topk"], case["N"]
        _, _, slots = _layout(_choice(case, seed), case["E"])
        return {"case": case, "Y": _normal((T * topk, N), seed, 20).to(TYPES[case["type"]]), "slots": slots,
                "weights": torch.softmax(_normal((T, topk), seed, 21), 1)}
    E = case.get("E", 1)
    rows = case["M"] if op == "linear" else case["T"]
    state = {"case": case, "A": _activations(rows, case["K"], seed, 30).half(),
             "bias": _normal((E, case["N"]), seed, 31)}
    if op == "experts":
        state["offsets"], state["rows"], _ = _layout(_choice(case, seed), E)
    q, s = _weights(case, seed, E)
    if own:      # the packed weight and the scratch that a serving program holds
        from weight_quantized_gemm_amd import qgemm as Q
        state["Bq"], state["scales"] = Q.qgemm_mx_pack_device(case["K"], case["N"], q, s, E=E)
        if op == "linear":
            need = Q.qgemm_workspace_size(case["M"], case["K"], case["N"], case["fmt"])
        else:
            need = Q.qgemm_grouped_workspace_size(case["T"] * case["topk"], case["T"], case["K"], case["N"], E,
                                                  case["fmt"])
        state["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        state["ws_bytes"] = need
    else:
        state["q"], state["s"] = q, s
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    return x / (1 + torch.exp(-x)) if act == "silu" else x


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "quantize":
        q, s = _encode(state["X"])
        return {"values": _decode(q, s), "scales": s}
    if op == "plan":
        return dict(zip(("offsets", "rows", "slots"), _layout(state["ids"], case["E"])))
    if op == "combine":
        here = state["slots"] >= 0
        y = state["Y"][state["slots"].clamp(min=0).long()].float()
        y = torch.where(here[..., None], y * state["weights"][..., None], 0.0)
        return y.sum(1).to(TYPES[case["out"]])
    A = _decode(*_encode(state["A"])) if case["fmt"] == "mxfp4a4" else state["A"].float()
    dtype = TYPES[case["out"]]
    if op == "linear":
        C = A @ _decode(state["q"][0], state["s"][0]).t() + state["bias"][0]
        return _act(C, case["act"]).to(dtype)
    C = torch.empty((state["rows"].numel(), case["N"]), dtype=dtype, device="cuda")
    bounds = state["offsets"].tolist()
    for e in range(case["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            c = A[state["rows"][lo:hi].long()] @ _decode(state["q"][e], state["s"][e]).t() + state["bias"][e]
            C[lo:hi] = _act(c, case["act"]).to(dtype)
    return C


def _run_own(state):
    from weight_quantized_gemm_amd import qgemm as Q
    case = state["case"]
    op = case["op"]
    if op == "quantize":
        q, s = Q.qgemm_mx_quantize_device(state["X"])
        return {"values": Q.qgemm_mx_dequantize_device(q, s, "f32"), "scales": s}
    if op == "plan":
        return dict(zip(("offsets", "rows", "slots"), Q.qgemm_group_plan(state["ids"], case["E"])))
    if op == "combine":
        C = torch.empty((case["T"], case["N"]), dtype=TYPES[case["out"]], device="cuda")
        Q.qgemm_group_combine(state["Y"], state["slots"], state["weights"], C)
        return C
    dtype = TYPES[case["out"]]
    if op == "linear":
        C = torch.empty((case["M"], case["N"]), dtype=dtype, device="cuda")
        Q.qgemm_run_ex(case["M"], case["K"], case["N"], case["fmt"], state["A"], state["Bq"], state["scales"], C,
                       bias=state["bias"], activation=case["act"], out_type=case["out"],
                       workspace=state["ws"] if state["ws_bytes"] else None, ws_bytes=state["ws_bytes"])
        return C
    C = torch.empty((state["rows"].numel(), case["N"]), dtype=dtype, device="cuda")
    Q.qgemm_run_grouped(case["K"], case["N"], case["E"], case["fmt"], state["A"], state["rows"], state["offsets"],
                        state["Bq"], state["scales"], C, bias=state["bias"], activation=case["act"],
                        out_type=case["out"], workspace=state["ws"] if state["ws_bytes"] else None,
                        ws_bytes=state["ws_bytes"])
    return C


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _nearest(x):
    """Float rows -> (value of every element's nearest code at its block's scale, scale bytes), in 64 bits:
    the scale is the largest power of two not above max |x| / 4, a tie goes to the even code, nothing exceeds 6."""
    R, K = x.shape
    v = x.double().reshape(R, K // BLOCK, BLOCK)
    top = v.abs().amax(-1)
    # the exponent from the bits of the double: exact at powers of two
    e = ((top.view(torch.int64) >> 52) & 2047) - 1023 - 2
    e = torch.where(top > 0, e.clamp(-127, 127), -127)
    scale = torch.pow(torch.full_like(top, 2.0), e.double())[..., None]
    y = v.abs() / scale
    code = ((y > 0.25).long() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    return (torch.where(v < 0, -grid[code], grid[code]) * scale).reshape(R, K), (e + 127).to(torch.uint8)


def exact(case, seed):
    op = case["op"]
    if op == "quantize":
        values, scales = _nearest(_activations(case["R"], case["K"], seed, 10).to(TYPES[case["type"]]))
        return {"values": values, "scales": scales}
    if op == "plan":      # whole numbers only
        return None
    ids = _choice(case, seed) if "topk" in case else None
    if op == "combine":
        T, topk, N = case["T"], case["topk"], case["N"]
        _, _, slots = _layout(ids, case["E"])
        Y = _normal((T * topk, N), seed, 20).to(TYPES[case["type"]])
        w = torch.softmax(_normal((T, topk), seed, 21), 1).double()
        C = torch.zeros((T, N), dtype=torch.float64, device="cuda")
        for j in range(topk):
            at = (slots[:, j] >= 0).nonzero()[:, 0]
            C[at] += w[at, j, None] * Y[slots[at, j].long()].double()
        return C
    E = case.get("E", 1)
    rows = case["M"] if op == "linear" else case["T"]
    A = _activations(rows, case["K"], seed, 30).half()
    A = _nearest(A)[0] if case["fmt"] == "mxfp4a4" else A.double()
    bias = _normal((E, case["N"]), seed, 31).double()
    out = []
    for e in range(E):
        W, _ = _nearest(_normal((case["N"], case["K"]), seed, 100 + e, 0.02))
        if op == "experts":     # this expert's rows: choices in token order
            token = (ids == e).nonzero()[:, 0]
            c = torch.mm(A[token], W.t()) + bias[e]
        else:
            c = torch.mm(A, W.t()) + bias[e]
        if case["act"] == "relu":
            c = c.clamp(min=0)
        elif case["act"] == "silu":
            c = c * torch.sigmoid(c)
        out.append(c)
    return torch.cat(out)
