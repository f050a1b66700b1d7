"""Measured cases of the operators around an expert layer: norm, routing, adapters.

A layer adds the residual, normalises the sum (in 16 bits for the router and the adapters, in 8 bits
for the integer products), scores the experts and chooses each token's; requests with adapters of
their own add these beside a projection that all requests share.  The operators:

* ``norm``        root-mean-square norm of the rows of x + residual, as they are and quantised to 8
                  bits per row, and ``norm_grad``, its gradient;
* ``route``       experts and routing weights of each token from its logits: softmax or sigmoid
                  scores, a bias for balance, groups of experts, renormalised weights, and
                  ``route_grad``, its gradient for the logits;
* ``adapt``       low-rank adapters, one per request, over the rows sorted by adapter.

Where ``own`` is false ``run`` computes them with elementary torch operations, where it is true
with the library's kernels.  8-bit codes are whole numbers here (-127 .. 127, the scale is an
output beside them, and the definition rounds exactly), so they are compared as such.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_TYPE_ID = {"bf16": 0, "fp16": 1, "fp32": 2}  # MOE_T_* of the library
_EPS = 1e-6


def listed():
    return [
        # four decode streams of the MXFP4 shape before its 8-bit products: sum and codes
        {"name": "norm_i8_4_streams", "op": "norm", "M": 4, "K": 6144, "type": "bf16",
         "residual": True, "y": False, "codes": True, "pad": 0},
        # one prefill chunk of the 35B shape: rows for the router and codes for the products
        {"name": "norm_prefill", "op": "norm", "M": 16384, "K": 2048, "type": "bf16",
         "residual": True, "y": True, "codes": True, "pad": 0},
        # a ragged training batch, column slices of wider rows
        {"name": "norm_grad_ragged", "op": "norm_grad", "M": 777, "K": 1000, "type": "fp16",
         "residual": False, "pad": 3},
        # a full training batch of the 35B shape
        {"name": "norm_grad_batch", "op": "norm_grad", "M": 16384, "K": 2048, "type": "bf16",
         "residual": True, "pad": 0},
        # eight decode streams of the 35B shape
        {"name": "route_8_streams", "op": "route", "T": 8, "E": 128, "k": 8, "type": "fp32",
         "score": "softmax", "bias": False, "groups": 1, "best": 1, "kept": 1, "renorm": True,
         "scale": 1.0, "masked": 0, "pad": 0},
        # one prefill chunk of the 35B shape, 16-bit logits: many ties
        {"name": "route_prefill", "op": "route", "T": 16384, "E": 128, "k": 8, "type": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "best": 1, "kept": 1, "renorm": True,
         "scale": 1.0, "masked": 0, "pad": 0},
        # a prefill chunk over 256 experts in 8 groups of which 4 are kept, balanced by a bias
        {"name": "route_groups_prefill", "op": "route", "T": 16384, "E": 256, "k": 8,
         "type": "fp32", "score": "sigmoid", "bias": True, "groups": 8, "best": 2, "kept": 4,
         "renorm": True, "scale": 2.5, "masked": 0, "pad": 0},
        # a ragged training batch: weights that are probabilities, so every logit has a gradient
        {"name": "route_grad_ragged", "op": "route_grad", "T": 777, "E": 60, "k": 4,
         "type": "fp32", "score": "softmax", "renorm": False, "scale": 1.0, "pad": 1},
        # a full training batch over 256 experts
        {"name": "route_grad_batch", "op": "route_grad", "T": 16384, "E": 256, "k": 8,
         "type": "fp32", "score": "sigmoid", "renorm": True, "scale": 2.5, "pad": 0},
        # eight decode streams, each with one of 32 adapters of its own
        {"name": "adapt_8_streams", "op": "adapt", "M": 8, "K": 2048, "N": 2048, "rank": 16,
         "adapters": 32, "requests": 8, "none": 0.0, "type": "bf16", "pad": 0},
        # a ragged batch of requests, some without an adapter
        {"name": "adapt_ragged", "op": "adapt", "M": 1003, "K": 1000, "N": 770, "rank": 24,
         "adapters": 8, "requests": 13, "none": 0.25, "type": "fp16", "pad": 3},
        # a prefill chunk of eleven requests over adapters of a high rank
        {"name": "adapt_prefill", "op": "adapt", "M": 16384, "K": 2048, "N": 2048, "rank": 64,
         "adapters": 16, "requests": 11, "none": 0.0, "type": "bf16", "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "route", "route", "route_grad", "adapt",
                     "adapt", "adapt"])
    pad = rng.choice([0, 0, 8, 3])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    size = _BYTES[kind]
    if op in ("norm", "norm_grad"):
        K = _log(rng, 64, 8192)
        K = K if rng.random() < 0.3 else max(8, K // 8 * 8)
        M = _log(rng, 1, min(32768, 66_000_000 // (K * size)))
        case = {"op": op, "M": M, "K": K, "type": kind, "residual": rng.random() < 0.7,
                "pad": pad}
        if op == "norm":
            y, codes = rng.choice([(True, False), (False, True), (True, True)])
            case.update(y=y, codes=codes)
        return case
    if op in ("route", "route_grad"):
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        k = min(rng.choice([1, 2, 4, 6, 8, 8, 10]), E // 2)
        T = _log(rng, 1, min(32768, 16_000_000 // (E * size)))
        case = {"op": op, "T": T, "E": E, "k": k, "type": kind,
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5, 16.0]), "pad": rng.choice([0, 0, 1])}
        if op == "route":
            groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= k])
            case.update(bias=rng.random() < 0.5, groups=groups, best=rng.choice([1, 2]),
                        kept=groups if groups < 3 else rng.randint(2, groups - 1),
                        masked=rng.choice([0, 0, E // 8]))
        return case
    K, N = _log(rng, 64, 8192), _log(rng, 64, 8192)
    if rng.random() < 0.7:
        K, N = max(8, K // 8 * 8), max(8, N // 8 * 8)
    rank = rng.choice([8, 16, 16, 32, 64, 24])
    adapters = rng.choice([1, 4, 16, 32])
    most = min(16384, 200_000_000 // ((K + 2 * N) * size), 4_290_000_000 // (rank * (K + N)))
    M = _log(rng, 1, most)
    return {"op": op, "M": M, "K": K, "N": N, "rank": rank, "adapters": adapters,
            "requests": min(M, rng.choice([1, 3, 8, 40])), "none": rng.choice([0.0, 0.0, 0.3]),
            "type": kind, "pad": pad}


def _matrix(g, rows, cols, pad, kind):
    """A matrix of activations, a column slice of a wider one where `pad` is set."""
    wide = torch.randn(rows, cols + pad, generator=g, device="cuda")
    wide *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    return wide.to(_TYPES[kind])[:, :cols]


def _logits(g, T, E, pad, kind, masked):
    """Logits whose experts are unequally liked; the first `masked` experts of a random order are
    not to be had."""
    wide = 1.5 * torch.randn(T, E + pad, generator=g, device="cuda")
    wide += 0.5 * torch.randn(E + pad, generator=g, device="cuda")
    if masked:
        wide[:, torch.randperm(E, generator=g, device="cuda")[:masked]] = -math.inf
    return wide.to(_TYPES[kind])[:, :E]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, kind = case["op"], case["type"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        M, K = case["M"], case["K"]
        s["weight"] = (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).to(_TYPES[kind])
        s["x"] = _matrix(g, M, K, case["pad"], kind)
        s["residual"] = _matrix(g, M, K, case["pad"], kind) if case["residual"] else None
        if op == "norm":
            s["sum"] = torch.zeros(M, K, dtype=_TYPES[kind], device="cuda") \
                if case["residual"] else None
            s["y"] = torch.zeros(M, K, dtype=_TYPES[kind], device="cuda") if case["y"] else None
            s["codes"] = s["scale"] = None
            if case["codes"]:
                s["codes"] = torch.zeros(M, K, dtype=torch.int8, device="cuda")
                s["scale"] = torch.zeros(M, device="cuda")
            return s
        # x is the sum that the forward pass kept, residual the gradient that reaches the sum
        # past the norm
        s["dy"] = _matrix(g, M, K, case["pad"], kind)
        s["dx"] = torch.zeros(M, K, dtype=_TYPES[kind], device="cuda")
        s["dweight"] = torch.zeros(K, device="cuda")
        return s
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(g, T, E, case["pad"], kind, case.get("masked", 0))
        if op == "route":
            s["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
            s["idx"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
            s["w"] = torch.zeros(T, k, device="cuda")
            return s
        s["idx"] = torch.topk(s["logits"].float(), k, dim=1).indices.to(torch.int32).contiguous()
        s["dw"] = torch.randn(T, k, generator=g, device="cuda")
        s["dlogits"] = torch.zeros(T, E, dtype=_TYPES[kind], device="cuda")
        return s
    M, K, N, R, A = (case[n] for n in ("M", "K", "N", "rank", "adapters"))
    # requests of unequal lengths one after another, each with an adapter or with none (-1)
    cut = torch.randperm(M - 1, generator=g, device="cuda")[:case["requests"] - 1] + 1
    request = torch.zeros(M, dtype=torch.int64, device="cuda")
    request[cut] = 1
    request = torch.cumsum(request, 0)
    ids = torch.randperm(max(A, case["requests"]), generator=g, device="cuda") % A
    none = torch.rand(case["requests"], generator=g, device="cuda") < case["none"]
    ids = torch.where(none, -1, ids[:case["requests"]])[request]
    # the batch's plan, the same for every projection of a step: rows by adapter
    key = torch.where(ids < 0, A, ids)
    counts = torch.bincount(key, minlength=A + 1)[:A]
    s["offsets"] = torch.zeros(A + 1, dtype=torch.int32, device="cuda")
    s["offsets"][1:] = torch.cumsum(counts, 0)
    s["order"] = torch.argsort(key, stable=True).to(torch.int32)
    s["most_rows"] = int(counts.max())
    s["x"] = _matrix(g, M, K, case["pad"], kind)
    s["a"] = (torch.randn(A, R, K, generator=g, device="cuda") / math.sqrt(K)).to(_TYPES[kind])
    s["b"] = (torch.randn(A, N, R, generator=g, device="cuda") / math.sqrt(R)).to(_TYPES[kind])
    s["alpha"] = 0.5 + torch.rand(A, generator=g, device="cuda")
    s["base"] = _matrix(g, M, N, case["pad"], kind)
    s["out"] = torch.zeros(M, N, dtype=_TYPES[kind], device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _plain_norm(s):
    c, out = s["case"], []
    h = s["x"]
    if c["residual"]:
        h = (h.float() + s["residual"].float()).to(_TYPES[c["type"]])
        out.append(h)
    f, w = h.float(), s["weight"].float()
    rstd = 1 / torch.sqrt((f * f).mean(1, keepdim=True) + _EPS)
    if c["y"]:
        out.append((f * rstd * w).to(_TYPES[c["type"]]))
    if c["codes"]:  # in 64 bits: a code next to a border has to be the right one
        p = h.double() * w.double()
        m = p.abs().amax(1, keepdim=True)
        out.append(torch.round(127 * p / torch.where(m > 0, m, 1.0)).to(torch.int8))
        out.append((m.float() * rstd / 127).reshape(-1))
    return out


def _plain_norm_grad(s):
    c = s["case"]
    h, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + _EPS)
    n = h * rstd
    wdy = w * dy
    dx = rstd * (wdy - n * (wdy * n).mean(1, keepdim=True))
    if c["residual"]:
        dx = dx + s["residual"].float()
    dweight = (dy * n).sum(0, dtype=torch.float64)  # a long sum
    return [dx.to(_TYPES[c["type"]]), dweight.float()]


def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    z = s["logits"].double()  # 64 bits: of two experts that are close the right one is chosen
    if c["score"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-z))
    masked = z == -math.inf
    choice = z if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(masked, -math.inf, choice)
    if G > 1:
        value = choice if c["best"] == 1 else torch.where(
            masked, -math.inf, score if s["bias"] is None else choice)
        best = torch.sort(value.reshape(T, G, E // G), dim=2, descending=True).values
        total = best[:, :, 0]
        if c["best"] == 2:  # a second that is not to be had adds nothing
            total = total + torch.where(best[:, :, 1] == -math.inf, 0.0, best[:, :, 1])
        groups = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = (groups[:, :, None] == torch.arange(G, device="cuda")).any(1)
        choice = torch.where(keep.repeat_interleave(E // G, dim=1), choice, -math.inf)
    value, idx = torch.sort(choice, dim=1, descending=True, stable=True)
    have, idx = value[:, :k] > -math.inf, idx[:, :k]
    w = torch.where(have, torch.gather(score, 1, idx), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return [torch.where(have, idx, -1).to(torch.int32), (w * c["scale"]).float()]


def _plain_route_grad(s):
    c = s["case"]
    z, idx, dw = s["logits"].float(), s["idx"].long(), s["dw"]
    if c["score"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-z))
    chosen = torch.gather(score, 1, idx)
    ds = dw * c["scale"]
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        ds = (ds - (ds * chosen).sum(1, keepdim=True) / total) / total
    if c["score"] == "softmax":
        dz = -score * (ds * chosen).sum(1, keepdim=True)
        # renormalised weights depend on the chosen logits alone
        dz = torch.zeros_like(z) if c["renorm"] else dz
        dz = dz.scatter_add(1, idx, ds * chosen)
    else:
        dz = torch.zeros_like(z).scatter(1, idx, ds * chosen * (1 - chosen))
    return [dz.to(_TYPES[c["type"]])]


def _plain_adapt(s):
    c = s["case"]
    M, A = c["M"], c["adapters"]
    place = torch.arange(M, device="cuda")
    adapter = (place[:, None] >= s["offsets"][1:]).sum(1)
    has = adapter < A
    adapter = adapter.clamp(max=A - 1)
    x = s["x"][s["order"]].float()
    if M <= 64:  # few rows: each with its own adapter's weights
        h = s["a"][adapter].float() @ x[:, :, None]
        v = (s["b"][adapter].float() @ h)[:, :, 0]
    else:  # every adapter's rows padded to the fullest adapter's
        first = s["offsets"][:-1, None]
        at = first + torch.arange(s["most_rows"], device="cuda")
        h = torch.bmm(x[at.clamp(max=M - 1)], s["a"].float().transpose(1, 2))
        v = torch.bmm(h, s["b"].float().transpose(1, 2))
        v = v[adapter, (place - s["offsets"][adapter]).clamp(max=s["most_rows"] - 1)]
    v = s["base"][s["order"]].float() + s["alpha"][adapter][:, None] * v
    out = torch.zeros(M, c["N"], dtype=_TYPES[c["type"]], device="cuda")
    # rows without an adapter are left as they were
    out[s["order"]] = torch.where(has[:, None], v, 0.0).to(out.dtype)
    return [out]


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "route": _plain_route,
          "route_grad": _plain_route_grad, "adapt": _plain_adapt}


# ------------------------------------------------------------------ the library's kernels


def _stride(t, cols):
    return cols if t is None else t.stride(0)


def _kernels(s):
    import expert_cache_offload_amd as m
    c = s["case"]
    op, kind = c["op"], _TYPE_ID[c["type"]]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "norm":
        K = c["K"]
        x, residual, total, y, codes = (s[n] for n in ("x", "residual", "sum", "y", "codes"))
        m.moe_norm_rows(x, x.stride(0), residual, _stride(residual, K), kind, c["M"], K,
                        s["weight"], _EPS, total, _stride(total, K), y, _stride(y, K), codes,
                        _stride(codes, K), s["scale"], stream)
        return [t for t in (total, y, codes, s["scale"]) if t is not None]
    if op == "norm_grad":
        if "workspace" not in s:  # kept beside the outputs, as a user's program keeps it
            size = max(16, m.moe_norm_grad_workspace_bytes(c["M"], c["K"]))
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        dy, dsum, x, dx, ws = s["dy"], s["residual"], s["x"], s["dx"], s["workspace"]
        m.moe_norm_rows_grad(dy, dy.stride(0), dsum, _stride(dsum, c["K"]), x, x.stride(0), kind,
                             c["M"], c["K"], s["weight"], _EPS, dx, dx.stride(0), s["dweight"],
                             ws, ws.numel(), stream)
        return [dx, s["dweight"]]
    if op == "adapt":
        x, a, b, base, out = (s[n] for n in ("x", "a", "b", "base", "out"))
        m.moe_adapt_rows(x, x.stride(0), kind, c["M"], c["K"], a, a.stride(1), b, b.stride(1),
                         c["N"], c["rank"], s["alpha"], c["adapters"], s["offsets"], s["order"],
                         base, base.stride(0), out, out.stride(0), stream)
        return [out]
    score = m.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else m.MOE_SCORE_SIGMOID
    z = s["logits"]
    if op == "route":
        m.moe_route_tokens(z, z.stride(0), kind, c["T"], c["E"], score, s["bias"], c["groups"],
                           c["best"], c["kept"], c["k"], c["renorm"], c["scale"], s["idx"],
                           s["w"], stream)
        return [s["idx"], s["w"]]
    dz = s["dlogits"]
    m.moe_route_tokens_grad(z, z.stride(0), kind, c["T"], c["E"], score, s["idx"], c["k"],
                            c["renorm"], c["scale"], s["dw"], dz, dz.stride(0), stream)
    return [dz]


def run(state):
    if own:
        return _kernels(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op, size = case["op"], _BYTES[case["type"]]
    if op == "norm":
        M, K = case["M"], case["K"]
        row = K * size * (1 + 2 * case["residual"] + case["y"]) + (K + 4) * case["codes"]
        return {"bytes": M * row + K * size, "flops": 5 * M * K}
    if op == "norm_grad":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * size * (3 + case["residual"]) + K * (size + 4),
                "flops": 10 * M * K}
    if op == "adapt":
        M, K, N, R = (case[n] for n in ("M", "K", "N", "rank"))
        used = min(case["adapters"], case["requests"])
        rows = M * (1 - case["none"])
        return {"bytes": int(rows * ((K + 2 * N) * size + 4) + used * R * (K + N) * size),
                "flops": int(2 * rows * R * (K + N))}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        return {"bytes": T * (E * size + 8 * k), "flops": 4 * T * E}
    # renormalised or sigmoid weights read the chosen logits alone
    read = E if case["score"] == "softmax" and not case["renorm"] else k
    return {"bytes": T * ((read + E) * size + 8 * k), "flops": 4 * T * E}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_scores(case, z):
    if case["score"] == "sigmoid":
        return torch.sigmoid(z)
    return torch.softmax(z, 1)


def _exact_norm(case, s):
    x = s["x"].to(torch.float64)
    out = []
    if case["residual"]:  # the sum is rounded once, what follows reads it rounded
        total = x + s["residual"].to(torch.float64)
        out.append(total)
        x = (s["x"].float() + s["residual"].float()).to(_TYPES[case["type"]]).to(torch.float64)
    root = torch.sqrt(torch.linalg.vector_norm(x, dim=1) ** 2 / case["K"] + _EPS)
    y = s["weight"].to(torch.float64) * x / root[:, None]
    if case["y"]:
        out.append(y)
    if case["codes"]:
        out += [None, torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127]
    return out


def _exact_norm_grad(case, s):
    h, dy, w = (s[n].to(torch.float64) for n in ("x", "dy", "weight"))
    variance = torch.linalg.vector_norm(h, dim=1) ** 2 / case["K"] + _EPS
    along = torch.mv(dy * h, w) / case["K"]
    dx = dy * w / variance.sqrt()[:, None] - h * (along / variance ** 1.5)[:, None]
    if case["residual"]:
        dx += s["residual"].to(torch.float64)
    return [dx, torch.mv((dy * h).t(), variance ** -0.5)]


def _ranks(value):
    """Each entry's place in its row, by value and then by index, counted over pairs."""
    n = value.shape[1]
    index = torch.arange(n, device="cuda")
    before = value[:, None, :] > value[:, :, None]
    before |= (value[:, None, :] == value[:, :, None]) & (index[None, :] < index[:, None])
    return before.sum(2)


def _exact_route(case, s):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    step = max(1, (1 << 27) // (E * E))
    w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for at in range(0, T, step):
        z = s["logits"][at:at + step].to(torch.float64)
        score = _exact_scores(case, z)
        value = z if s["bias"] is None else score + s["bias"].to(torch.float64)
        value = value.masked_fill(z == -math.inf, -math.inf)
        if G > 1:
            part = value if case["best"] == 1 or s["bias"] is not None else \
                score.masked_fill(z == -math.inf, -math.inf)
            part = part.reshape(-1, G, E // G)
            rank = _ranks(part.reshape(-1, E // G)).reshape(part.shape)
            total = part.masked_fill(rank != 0, 0.0).sum(2)
            if case["best"] == 2:
                total += part.masked_fill((rank != 1) | (part == -math.inf), 0.0).sum(2)
            out = _ranks(total) >= case["kept"]
            value = value.masked_fill(out.repeat_interleave(E // G, dim=1), -math.inf)
        rank = _ranks(value).masked_fill(value == -math.inf, E)
        for j in range(k):
            w[at:at + step, j] = (score * (rank == j)).sum(1)
    if case["renorm"]:
        w /= w.sum(1, keepdim=True)
    return [None, w * case["scale"]]


def _exact_route_grad(case, s):
    z = s["logits"].to(torch.float64).requires_grad_()
    w = _exact_scores(case, z).gather(1, s["idx"].long())
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return list(torch.autograd.grad(w * case["scale"], z, s["dw"].to(torch.float64)))


def _exact_adapt(case, s):
    out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
    ends = s["offsets"].tolist()
    for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if lo == hi:
            continue
        rows = s["order"][lo:hi].long()
        h = torch.mm(s["x"][rows].to(torch.float64), s["a"][g].to(torch.float64).t())
        h *= s["alpha"][g].to(torch.float64)
        out[rows] = torch.mm(h, s["b"][g].to(torch.float64).t()) + s["base"][rows]
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "route": _exact_route,
            "route_grad": _exact_route_grad, "adapt": _exact_adapt}[case["op"]](case, s)
