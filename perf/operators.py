"""Timed cases of the adapter projection and of the distillation loss.

The adapter projection gives every row of X the shared weight and the low-rank
pair of the row's own request:

    Y[m] = X[m] W + scale[a] (X[m] A[a]^T) B[a],   a = ids[m]

with A[a] of r rows of K, B[a] of r rows of N, and no second term for rows
whose id names no adapter. Its backward pass gives the gradients of X, A and
B for a given gradient of Y; W is frozen.

The distillation loss compares the student's logits z of a row with the
teacher's k largest ones t at the entries `index`, at temperature T:

    p = softmax(t / T) over the row's valid entries, q = softmax(z / T)
    loss = weight T^2 sum_j p_j (log p_j - log q_j)
    dz = weight T (q - p)

A row without a valid entry has loss 0 and gradient 0. ``run`` gives the
plain form (``own`` false) or the library's calls (``own`` true).
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _adapter(name, M, K, N, rank, adapters, dtype, ids, out, trans_w=False, back=False):
    return {"name": name, "op": "adapter", "M": M, "K": K, "N": N, "rank": rank, "adapters": adapters, "dtype": dtype,
            "ids": ids, "out": out, "trans_w": trans_w, "back": back}


def _distill(name, rows, V, top, dtype, T, form):
    return {"name": name, "op": "distill", "rows": rows, "V": V, "top": top, "dtype": dtype, "T": T, "form": form}


def listed():
    return [
        # One request's next token through one projection: latency counts.
        _adapter("adapter_token", 1, 4096, 4096, 16, 8, "bf16", "rows", "same"),
        # A decode batch: every row a request of its own, some without an adapter.
        _adapter("adapter_decode", 64, 4096, 11008, 16, 32, "bf16", "rows", "same"),
        # A small prefill chunk of a few requests, weight stored as N rows of K, FP32 result.
        _adapter("adapter_chunk", 256, 4096, 11008, 32, 4, "f16", "runs", "f32", trans_w=True),
        # Sizes whose rows are no whole 16-byte pieces.
        _adapter("adapter_ragged", 2049, 1025, 4097, 8, 5, "bf16", "runs", "same"),
        # Long prompts of a few requests, wide adapters.
        _adapter("adapter_prompt", 4096, 11008, 4096, 64, 4, "bf16", "runs", "same"),
        # Training several adapters in one batch: gradients of X, A and B.
        _adapter("adapter_back", 4096, 4096, 4096, 16, 8, "bf16", "runs", "same", back=True),
        # The same with odd sizes, more adapters than sequences, FP32 gradient of X.
        _adapter("adapter_back_ragged", 1025, 768, 2049, 24, 16, "f16", "runs", "f32", back=True),
        # Scoring a few positions: the loss alone.
        _distill("distill_score", 16, 32768, 16, "bf16", 1.0, "loss"),
        # A training batch: loss and gradient in one call.
        _distill("distill_train", 4096, 32768, 64, "bf16", 2.0, "both"),
        # A large vocabulary, with the FP32 logits that the library's products give.
        _distill("distill_wide", 1024, 131072, 32, "f32", 1.0, "both"),
        # Odd vocabulary, loss first and the gradient in a later call.
        _distill("distill_odd", 333, 50003, 20, "f16", 1.5, "steps"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        M, K, N = _log(rng, 1, 4096), _log(rng, 256, 8192), _log(rng, 256, 8192)
        if rng.random() < 0.6:   # most models' widths are multiples of 64
            K, N = (K + 63) // 64 * 64, (N + 63) // 64 * 64
        back = rng.random() < 0.4
        while M * K * N * (1 + back) > 4096 * 4096 * 11008:
            M = max(1, M // 2)
        case = _adapter("", M, K, N, rng.choice([4, 8, 16, 16, 24, 32, 48, 64]), _log(rng, 1, 32),
                        rng.choice(["bf16", "bf16", "f16"]), "rows" if M <= 128 else "runs", rng.choice(["same", "f32"]),
                        rng.random() < 0.5, back)
    else:
        rows, V = _log(rng, 1, 4096), _log(rng, 1000, 131072)
        while rows * V > 4096 * 32768:
            rows = max(1, rows // 2)
        case = _distill("", rows, V, _log(rng, 1, 128), rng.choice(["bf16", "f16", "f32"]), round(rng.uniform(0.5, 4.0), 2),
                        rng.choice(["loss", "both", "both", "steps"]))
    del case["name"]
    return case


def _ids(case, seed):
    """One id a row; -1: no adapter. "rows": any order; "runs": sequences of rows of one request."""
    r = random.Random(seed)
    M, n = case["M"], case["adapters"]
    if case["ids"] == "rows":
        v = [r.randrange(n) if r.random() < 0.9 else -1 for _ in range(M)]
    else:
        cuts = sorted(r.randrange(M + 1) for _ in range(n)) + [M]
        v, at = [], 0
        for i, c in enumerate(cuts):
            v += [(i * 7 + seed) % n if i < n else -1] * (c - at)
            at = c
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, by=1.0, to=dt):
        return (torch.randn(*shape, device="cuda", generator=g) * by).to(to)

    if case["op"] == "adapter":
        M, K, N, r, n = (case[k] for k in ("M", "K", "N", "rank", "adapters"))
        s = {"X": normal(M, K), "W": normal(*((N, K) if case["trans_w"] else (K, N)), by=K ** -0.5),
             "A": normal(n, r, K, by=K ** -0.5), "B": normal(n, r, N, by=0.5 * r ** -0.5), "ids": _ids(case, seed),
             "scale": torch.rand(n, device="cuda", generator=g) + 0.5}
        if case["back"]:
            s["dY"] = normal(M, N, by=0.1)
    else:
        R, V, k = case["rows"], case["V"], case["top"]
        s = {"logits": normal(R, V, by=3.0)}
        # The teacher agrees with the student in part: its best entries are
        # among the student's better ones. Some entries are left empty, and so
        # are all of every 29th row.
        lift = torch.topk(s["logits"].float() + 3.0 * torch.randn(R, V, device="cuda", generator=g), k, dim=1)
        s["t"], s["index"] = (lift.values + 2.0).to(dt), lift.indices.to(torch.int32)
        gone = torch.rand(R, k, device="cuda", generator=g) < 0.03
        gone[28::29] = True
        s["index"][gone] = -1
        s["weight"] = (torch.rand(R, device="cuda", generator=g) + 0.5) / R
        s["weight"][13::17] = 0.0   # positions of a prompt, not trained on
    s["case"] = case
    return s


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "adapter":
        return _adapter_plain(s, case)
    return _distill_plain(s, case)


def _run_own(s, case):
    import shape_adaptive_matrix_amd as sam

    if case["op"] == "adapter":
        out = torch.float32 if case["out"] == "f32" else s["X"].dtype
        if case["back"]:
            return sam.adapter_backward(s["dY"], s["X"], s["W"], s["A"], s["B"], s["ids"], s["scale"],
                                        trans_w=case["trans_w"], out_dtype=out)
        return sam.adapter_gemm(s["X"], s["W"], s["A"], s["B"], s["ids"], s["scale"], trans_w=case["trans_w"],
                                out_dtype=out)
    if case["form"] == "loss":
        return sam.distill_loss(s["logits"], s["t"], s["index"], s["weight"], case["T"])
    if case["form"] == "both":
        return sam.distill(s["logits"], s["t"], s["index"], s["weight"], case["T"])
    loss, lse = sam.distill_loss(s["logits"], s["t"], s["index"], s["weight"], case["T"])
    return loss, lse, sam.distill_grad(s["logits"], lse, s["t"], s["index"], s["weight"], case["T"])


def _adapter_plain(s, case):
    M, K, N, r, n = (case[k] for k in ("M", "K", "N", "rank", "adapters"))
    out = torch.float32 if case["out"] == "f32" else s["X"].dtype
    X, A, B = s["X"].float(), s["A"].float().reshape(n * r, K), s["B"].float().reshape(n * r, N)
    W = s["W"].float().t() if case["trans_w"] else s["W"].float()
    # Which adapter's columns a row keeps, times that adapter's scale.
    own_rows = (s["ids"][:, None] == torch.arange(n, device="cuda")[None, :]).float() * s["scale"][None, :]
    keep = own_rows[:, :, None].expand(M, n, r).reshape(M, n * r)
    T = (X @ A.t()) * keep
    if not case["back"]:
        return (X @ W + T @ B).to(out)
    dY = s["dY"].float()
    dT = (dY @ B.t()) * keep
    dX = dY @ W.t() + dT @ A
    return dX.to(out), (dT.t() @ X).reshape(n, r, K), (T.t() @ dY).reshape(n, r, N)


def _distill_plain(s, case):
    V, T = case["V"], case["T"]
    z = s["logits"].float() / T
    top = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(dim=1, keepdim=True)
    lse = top + torch.log(total)
    valid = (s["index"] >= 0) & (s["index"] < V)
    at = torch.where(valid, s["index"], 0).long()
    t = torch.where(valid, s["t"].float() / T, -math.inf)
    best = t.amax(dim=1, keepdim=True)
    best = torch.where(torch.isfinite(best), best, 0.0)
    pe = torch.exp(t - best)
    psum = pe.sum(dim=1, keepdim=True)
    live = (psum > 0) & (s["weight"][:, None] != 0)
    p = torch.where(live, pe / psum, 0.0)
    logp = t - best - torch.log(psum)
    w = torch.where(live, s["weight"][:, None], 0.0)
    term = torch.where(p > 0, p * (logp - z.gather(1, at) + lse), 0.0)
    loss = (w * (T * T) * term.sum(dim=1, keepdim=True))[:, 0]
    if case["form"] == "loss":
        return loss, lse[:, 0]
    grad = (e / total).scatter_add_(1, at, -p) * (w * T)
    grad = grad.to(s["logits"].dtype)
    return (loss, grad) if case["form"] == "both" else (loss, lse[:, 0], grad)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adapter":
        W, X = s["W"].double(), s["X"].double()
        if case["trans_w"]:
            W = W.t()
        if not case["back"]:
            Y = X @ W
            for a in range(case["adapters"]):
                rows = torch.nonzero(s["ids"] == a)[:, 0]
                Y[rows] += float(s["scale"][a]) * ((X[rows] @ s["A"][a].double().t()) @ s["B"][a].double())
            return Y
        dY = s["dY"].double()
        dX, dA, dB = dY @ W.t(), [], []
        for a in range(case["adapters"]):
            rows, f = torch.nonzero(s["ids"] == a)[:, 0], float(s["scale"][a])
            Aa, Ba = s["A"][a].double(), s["B"][a].double()
            u, v = X[rows] @ Aa.t(), dY[rows] @ Ba.t()
            dX[rows] += f * (v @ Aa)
            dA.append(f * (v.t() @ X[rows]))
            dB.append(f * (u.t() @ dY[rows]))
        return dX, torch.stack(dA), torch.stack(dB)
    T, R, V = case["T"], case["rows"], case["V"]
    loss = torch.zeros(R, dtype=torch.float64, device="cuda")
    lse = torch.empty(R, dtype=torch.float64, device="cuda")
    grad = None if case["form"] == "loss" else torch.zeros(R, V, dtype=torch.float64, device="cuda")
    for i in range(0, R, 256):
        z = s["logits"][i:i + 256].double() / T
        lse[i:i + 256] = torch.logsumexp(z, dim=1)
        logq = z - lse[i:i + 256, None]
        n = z.shape[0]
        # The teacher's logits spread over the whole vocabulary: an entry that
        # is not given is -inf there (one column more takes the empty entries).
        idx = s["index"][i:i + 256].long()
        wide = torch.full((n, V + 1), -math.inf, dtype=torch.float64, device="cuda")
        wide.scatter_(1, torch.where((idx < 0) | (idx >= V), V, idx), s["t"][i:i + 256].double() / T)
        logp = torch.log_softmax(wide[:, :V], dim=1)
        w = s["weight"][i:i + 256].double()
        live = torch.isfinite(wide[:, :V]).any(dim=1) & (w != 0)
        p = torch.where(live[:, None], torch.exp(logp), 0.0)
        kl = torch.where(p > 0, p * (logp - logq), 0.0).sum(dim=1)
        loss[i:i + 256] = torch.where(live, w * T * T * kl, 0.0)
        if grad is not None:
            grad[i:i + 256] = torch.where(live[:, None], (w * T)[:, None] * (torch.exp(logq) - p), 0.0)
    if grad is None:
        return loss, lse
    return (loss, grad) if case["form"] == "both" else (loss, lse, grad)


def work(case):
    if case["op"] == "adapter":
        M, K, N, r = (case[k] for k in ("M", "K", "N", "rank"))
        n = min(case["adapters"], M)   # adapters that some row can use
        y = M * (K if case["back"] else N) * (4 if case["out"] == "f32" else 2)
        bytes_ = 2 * (M * K + K * N + n * r * (K + N)) + 4 * M + y
        flops = 2 * M * N * K + 2 * M * r * (K + N)
        if case["back"]:
            bytes_ += 2 * M * N + 4 * case["adapters"] * r * (K + N)
            flops += 4 * M * r * (K + N) - 2 * M * r * N
        return {"bytes": bytes_, "flops": flops}
    R, V, k = case["rows"], case["V"], case["top"]
    es = 4 if case["dtype"] == "f32" else 2
    passes = {"loss": 1, "both": 2, "steps": 3}[case["form"]]
    return {"bytes": passes * es * R * V + R * (k * (es + 4) + 12), "flops": {"loss": 4, "both": 8, "steps": 8}[case["form"]] * R * V}
