"""Timed cases of the 4-bit projection and of token log probabilities.

A 4-bit tensor (OCP MXFP4) holds 32 neighbours of a row as E2M1 values (0,
0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times a power of two of their own:

    s = floor(log2(max |x|)) - 2,  x ~ 2^s e,  e = x / 2^s rounded to the
    nearest E2M1 value, ties to the even code, at most 6

The 4-bit projection takes rows of X to that form and multiplies them by a
weight that is kept in it; its backward pass takes the gradient through the
rounding of X as it is:

    Y = q(X) Wq^T,   dX = dY Wq

Token log probabilities: of the given token of every row, with the row's
entropy and its most likely entries, at temperature T:

    log p = z / T - log sum exp(z / T)
    logprob = log p[token],  entropy = - sum_j p_j log p_j
    dz_j = (dlogprob (1[j = token] - p_j) - dentropy p_j (log p_j + entropy)) / T

A token outside the vocabulary has log probability 0 and takes no gradient.
``run`` gives the plain form (``own`` false) or the library's calls (``own``
true).
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32


def _quant(name, rows, K, dtype, trans=False):
    return {"name": name, "op": "quant", "rows": rows, "K": K, "dtype": dtype, "trans": trans}


def _linear(name, M, K, N, dtype, out, back=False):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "dtype": dtype, "out": out, "back": back}


def _tokens(name, rows, V, dtype, T, top, back=False):
    return {"name": name, "op": "tokens", "rows": rows, "V": V, "dtype": dtype, "T": T, "top": top, "back": back}


def listed():
    return [
        # A weight stored as K rows of N taken to 4 bits when a model is loaded, and looked at.
        _quant("quant_weight", 11008, 4096, "f16", trans=True),
        # Rows that are no whole blocks.
        _quant("quant_odd", 2049, 1025, "f32"),
        # One request's next token through one projection: latency counts.
        _linear("linear_token", 1, 4096, 4096, "bf16", "same"),
        # A decode batch.
        _linear("linear_decode", 32, 4096, 11008, "bf16", "same"),
        # The output head of a few requests: FP32 logits over a large vocabulary.
        _linear("linear_head", 4, 4096, 131072, "f16", "f32"),
        # Odd sizes, nothing a whole block or tile.
        _linear("linear_ragged", 513, 1025, 2049, "f16", "f32"),
        # Long prompts.
        _linear("linear_prompt", 4096, 11008, 4096, "bf16", "same"),
        # Training through a frozen 4-bit weight.
        _linear("linear_back", 4096, 4096, 4096, "bf16", "same", back=True),
        # The sampled tokens of a decode batch, with the alternatives a client asks for.
        _tokens("tokens_decode", 16, 131072, "f32", 0.7, 20),
        # A teacher's most likely entries of a training batch.
        _tokens("tokens_teacher", 2048, 32768, "bf16", 1.0, 64),
        # Training on sampled tokens with an entropy term: forward, then the gradient.
        _tokens("tokens_train", 4096, 32768, "bf16", 1.0, 0, back=True),
        # Odd vocabulary.
        _tokens("tokens_odd", 333, 50003, "f16", 1.3, 5, back=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.random()
    if kind < 0.2:
        rows, K = _log(rng, 1, 16384), _log(rng, 32, 16384)
        if rng.random() < 0.6:   # most models' widths are multiples of 64
            K = (K + 63) // 64 * 64
        while rows * K > 4096 * 11008:
            rows = max(1, rows // 2)
        case = _quant("", rows, K, rng.choice(["bf16", "bf16", "f16", "f32"]), rng.random() < 0.4)
    elif kind < 0.6:
        back = rng.random() < 0.25
        M, K, N = _log(rng, 1, 4096), _log(rng, 256, 11008), _log(rng, 256, 16384)
        if rng.random() < 0.6:
            K, N = (K + 63) // 64 * 64, (N + 63) // 64 * 64
        dtype = rng.choice(["bf16", "bf16", "f16"] if back else ["bf16", "bf16", "f16", "f32"])
        while M * K * N * (1 + back) > 4096 * 4096 * 11008:
            M = max(1, M // 2)
        case = _linear("", M, K, N, dtype, rng.choice(["same", "f32"]), back)
    else:
        rows, V = _log(rng, 1, 4096), _log(rng, 1000, 131072)
        while rows * V > 4096 * 32768:
            rows = max(1, rows // 2)
        back = rng.random() < 0.5
        case = _tokens("", rows, V, rng.choice(["bf16", "f16", "f32"]), round(rng.uniform(0.5, 2.0), 2),
                       rng.choice([0, 0, 1, 5, 20, 64, 128]), back)
    del case["name"]
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, by=1.0, to=dt):
        return (torch.randn(*shape, device="cuda", generator=g) * by).to(to)

    if case["op"] == "quant":
        rows, K = case["rows"], case["K"]
        # Rows of different sizes, some blocks of zeros.
        x = torch.randn(rows, K, device="cuda", generator=g) * torch.exp(torch.randn(rows, 1, device="cuda", generator=g))
        x[:, 64:96] *= (torch.arange(rows, device="cuda") % 5 != 0)[:, None]
        s = {"X": (x.t() if case["trans"] else x).to(dt).contiguous()}
    elif case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        codes, scales = _codes(normal(N, K, by=K ** -0.5, to=torch.float32))
        s = {"codes": codes, "scales": scales}
        if case["back"]:
            s["dY"] = normal(M, N, by=0.1)
        else:
            x = torch.randn(M, K, device="cuda", generator=g)
            x *= torch.where(torch.arange(K, device="cuda") % 97 == 5, 8.0, 1.0)   # a few large channels
            s["X"] = x.to(dt)
    else:
        R, V = case["rows"], case["V"]
        z = torch.randn(R, V, device="cuda", generator=g) * 3.0
        hit = torch.randint(V, (R,), device="cuda", generator=g)
        # Half of the tokens are what the model expects; some positions have none.
        z[torch.arange(R, device="cuda"), hit] += torch.where(torch.arange(R, device="cuda") % 2 == 0, 9.0, 0.0)
        s = {"tokens": hit.to(torch.int32)}
        s["tokens"][9::23] = -1
        # Every 8th row may only take every 3rd entry (but for its token).
        z[3::8] = torch.where((torch.arange(V, device="cuda") % 3 == 0) | (torch.arange(V, device="cuda") == hit[3::8, None]),
                              z[3::8], -math.inf)
        s["logits"] = z.to(dt)
        if case["back"]:
            s["dlogprob"] = -(torch.rand(R, device="cuda", generator=g) + 0.5) / R
            s["dlogprob"][13::17] = 0.0   # positions of a prompt, not trained on
            s["dentropy"] = torch.where(s["dlogprob"] != 0.0, -0.01 / R, 0.0)
    s["case"] = case
    return s


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "quant":
        x = s["X"].t() if case["trans"] else s["X"]
        return _rounded(x.float())[:, :case["K"]].to(x.dtype)
    if case["op"] == "linear":
        return _linear_plain(s, case)
    return _tokens_plain(s, case)


def _run_own(s, case):
    import shape_adaptive_matrix_amd as sam

    if case["op"] == "quant":
        codes, scales = sam.quantize_mxfp4(s["X"], trans=case["trans"])
        return sam.dequantize_mxfp4(codes, scales, case["K"], out_dtype=s["X"].dtype)
    if case["op"] == "linear":
        x = s["dY"] if case["back"] else s["X"]
        out = torch.float32 if case["out"] == "f32" else x.dtype
        if case["back"]:
            return sam.linear_mxfp4_backward(x, s["codes"], s["scales"], case["K"], out_dtype=out)
        return sam.linear_mxfp4(x, s["codes"], s["scales"], out_dtype=out)
    got = sam.token_logprobs(s["logits"], s["tokens"], case["T"], top=case["top"])
    if case["back"]:
        logprob, entropy, norm = got[:3]
        got += (sam.token_logprobs_grad(s["logits"], s["tokens"], norm, entropy, s["dlogprob"], s["dentropy"], case["T"]),)
    return got


# -- 4-bit values, plain -------------------------------------------------------
def _blocks(x):
    """[rows, blocks, 32], zeros behind a row's end, and each block's power of two."""
    rows, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % BLOCK)).reshape(rows, -1, BLOCK)
    exponent = torch.frexp(x.abs().amax(dim=2, keepdim=True))[1] - 3   # amax = m 2^(exponent + 3), 0.5 <= m < 1
    exponent = torch.where(x.abs().amax(dim=2, keepdim=True) > 0, exponent, -127).clamp(-127, 127)
    return x, exponent


def _multiples(x):
    """E2M1 values of x's blocks, and the blocks' exponents."""
    x, exponent = _blocks(x)
    y = torch.ldexp(x, -exponent)
    step = torch.where(y.abs() < 2.0, 0.5, torch.where(y.abs() < 4.0, 1.0, 2.0))
    return (torch.round(y / step) * step).clamp(-6.0, 6.0), exponent


def _rounded(x):
    e, exponent = _multiples(x)
    return torch.ldexp(e, exponent).reshape(x.shape[0], -1)


def _codes(x):
    """Packed codes (element 2 i in the low half of byte i) and scale codes."""
    e, exponent = _multiples(x)
    a = e.abs()
    code = torch.where(a < 2.0, a * 2.0, torch.where(a < 4.0, a + 2.0, a / 2.0 + 4.0)).to(torch.uint8)
    code = (code + torch.where(torch.signbit(e), 8, 0).to(torch.uint8)).reshape(x.shape[0], -1)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), (exponent[:, :, 0] + 127).to(torch.uint8)


def _decoded(codes, scales, K):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat((table, -table))
    e = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), dim=2)
    e = e.reshape(codes.shape[0], -1, BLOCK)
    return torch.ldexp(e, scales.int()[:, :, None] - 127).reshape(codes.shape[0], -1)[:, :K]


def _linear_plain(s, case):
    W = _decoded(s["codes"], s["scales"], case["K"])
    x = s["dY"] if case["back"] else s["X"]
    out = torch.float32 if case["out"] == "f32" else x.dtype
    if case["back"]:
        return (x.float() @ W).to(out)
    return (_rounded(x.float())[:, :case["K"]] @ W.t()).to(out)


# -- token log probabilities, plain ----------------------------------------------
def _ordered(z, V):
    """Whole numbers that order a row's entries: by value, the lowest index first among equals."""
    bits = (z.float() + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
    return key * (1 << 20) + (V - 1 - torch.arange(V, device=z.device))


def _tokens_plain(s, case):
    V, T, top = case["V"], case["T"], case["top"]
    z = s["logits"].float()
    best = z.amax(dim=1, keepdim=True)
    d = (z - best) / T
    e = torch.exp(d)
    total = e.sum(dim=1, keepdim=True)
    log_total = torch.log(total)
    p = e / total
    logp = d - log_total
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(dim=1)
    valid = (s["tokens"] >= 0) & (s["tokens"] < V)
    at = torch.where(valid, s["tokens"], 0).long()
    logprob = torch.where(valid, logp.gather(1, at[:, None])[:, 0], 0.0)
    got = (logprob, entropy, torch.cat((best, log_total), dim=1))
    if top:
        index = torch.topk(_ordered(s["logits"], V), top, dim=1).indices
        got += (logp.gather(1, index), index.to(torch.int32))
    if case["back"]:
        take = torch.where(valid, s["dlogprob"], 0.0)[:, None]
        grad = torch.where(p > 0, -p * (take + s["dentropy"][:, None] * (logp + entropy[:, None])), 0.0)
        grad.scatter_add_(1, at[:, None], take)
        got += ((grad / T).to(s["logits"].dtype),)
    return got


# -- in 64 bits, from the definitions ----------------------------------------------
def _exact_rounded(x):
    """Each value to the E2M1 value whose interval it lies in; the intervals' ends belong to the even codes."""
    rows, K = x.shape
    wide = torch.zeros(rows, (K + BLOCK - 1) // BLOCK * BLOCK, dtype=torch.float64, device=x.device)
    wide[:, :K] = x
    wide = wide.reshape(rows, -1, BLOCK)
    largest = wide.abs().amax(dim=2, keepdim=True)
    unit = torch.full_like(largest, 2.0 ** -127)
    low = torch.floor(torch.log2(largest))   # log2 may round up to a whole number just under one
    low = torch.where(torch.exp2(low) > largest, low - 1, low)
    unit = torch.where(largest > 0, torch.exp2(torch.clamp(low - 2, -127, 127)), unit)
    size = wide.abs() / unit
    value = torch.zeros_like(size)
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    for code in range(1, 8):
        middle = (grid[code - 1] + grid[code]) / 2
        value = torch.where(size > middle if code % 2 else size >= middle, grid[code], value)
    return (torch.sign(wide) * value * unit).reshape(rows, -1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = s["X"].double()
        return _exact_rounded(x.t() if case["trans"] else x)
    if case["op"] == "linear":
        grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        W = torch.zeros(case["N"], 2 * s["codes"].shape[1], dtype=torch.float64, device="cuda")
        for half in (0, 1):
            c = s["codes"] >> 4 if half else s["codes"] & 15
            for i in range(1, 8):
                W[:, half::2] += grid[i] * ((c == i).double() - (c == i + 8).double())
        W *= torch.exp2(s["scales"].double() - 127).repeat_interleave(BLOCK, dim=1)
        W = W[:, :case["K"]]
        return s["dY"].double() @ W if case["back"] else _exact_rounded(s["X"].double()) @ W.t()
    R, V, T, top = (case[k] for k in ("rows", "V", "T", "top"))
    parts = []
    for i in range(0, R, 256):
        raw, token = s["logits"][i:i + 256], s["tokens"][i:i + 256].long()
        z = raw.double() / T
        logp = torch.log_softmax(z, dim=1)
        p = torch.exp(logp)
        entropy = torch.special.entr(p).sum(dim=1)
        has = (token >= 0) & (token < V)
        one = torch.zeros_like(p)
        one[has, token[has]] = 1.0
        largest = raw.double().max(dim=1).values
        part = [torch.where(one > 0, logp, 0.0).sum(dim=1), entropy,
                torch.stack((largest, torch.logsumexp(z, dim=1) - largest / T), dim=1)]
        if top:
            order = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :top]
            part += [torch.gather(logp, 1, order), order.to(torch.int32)]
        if case["back"]:
            u, v = s["dlogprob"][i:i + 256, None].double(), s["dentropy"][i:i + 256, None].double()
            inner = torch.where(p > 0, p * (torch.clamp(logp, min=-1e300) + entropy[:, None]), 0.0)
            part.append((torch.where(has[:, None], u * (one - p), 0.0) - v * inner) / T)
        parts.append(part)
    return tuple(torch.cat(x) for x in zip(*parts))


def work(case):
    if case["op"] == "quant":
        n, es = case["rows"] * case["K"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * es * n + n // 2 + n // BLOCK, "flops": 4 * n}
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        es = 4 if case["dtype"] == "f32" else 2
        given, got = (N, K) if case["back"] else (K, N)
        out = 4 if case["out"] == "f32" else es
        return {"bytes": es * M * given + N * K // 2 + N * K // BLOCK + out * M * got, "flops": 2 * M * N * K}
    R, V = case["rows"], case["V"]
    es = 4 if case["dtype"] == "f32" else 2
    return {"bytes": (3 if case["back"] else 1) * es * R * V + R * (20 + 8 * case["top"]), "flops": (12 if case["back"] else 6) * R * V}
