"""Measured cases of the token and 8-bit integer operators of the expert layer.

An expert layer sorts its tokens by expert, multiplies each expert's rows with that expert's
weights and adds the results back per token with the routing weights.  The operators:

* ``sort``          tokens sorted by expert (counts, order, places, rows; rows as they are or
                    quantised to 8 bits per token), and ``sort_grad``, its gradient;
* ``combine``       rows back to tokens with the routing weights applied, and ``combine_grad``,
                    its gradient for the rows and for the weights;
* ``quantise``      8-bit codes and one scale per row;
* ``product``       product of 8-bit integers with scales per row and per weight channel, for one
                    weight or one weight per expert, plain or with a SwiGLU epilogue.

Where ``own`` is false ``run`` computes them with elementary torch operations, where it is true
with the library's kernels.  8-bit codes are whole numbers here (-127 .. 127, the scale is an
output beside them), so they are compared as such.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "i8": 1}
_TYPE_ID = {"bf16": 0, "fp16": 1, "fp32": 2, "i8": 3}  # MOE_T_* of the library


def listed():
    return [
        # four decode streams of the MXFP4 shape, their rows sorted and quantised for 8-bit experts
        {"name": "sort_i8_4_streams", "op": "sort", "T": 4, "k": 8, "E": 256, "local": 256,
         "H": 6144, "type": "bf16", "rows": "i8", "pad": 0},
        # one prefill chunk of the 35B shape
        {"name": "sort_prefill", "op": "sort", "T": 16384, "k": 8, "E": 128, "local": 128,
         "H": 2048, "type": "bf16", "rows": "bf16", "pad": 0},
        # gradient of the sort in fp32 training, where this rank holds half of the experts
        {"name": "sort_grad_half_experts", "op": "sort_grad", "T": 4099, "k": 8, "E": 256,
         "local": 128, "H": 4096, "type": "fp32", "pad": 0},
        # eight decode streams of the 35B shape: expert outputs back to their tokens
        {"name": "combine_8_streams", "op": "combine", "T": 8, "k": 8, "E": 128, "local": 128,
         "H": 2048, "type": "bf16", "pad": 0},
        # one prefill chunk of the 35B shape
        {"name": "combine_prefill", "op": "combine", "T": 16384, "k": 8, "E": 128, "local": 128,
         "H": 2048, "type": "bf16", "pad": 0},
        # a ragged training batch with a width that is no multiple of a wave's loads
        {"name": "combine_grad_ragged", "op": "combine_grad", "T": 777, "k": 6, "E": 64,
         "local": 64, "H": 1000, "type": "fp16", "pad": 0},
        # a full training batch of the 35B shape
        {"name": "combine_grad_batch", "op": "combine_grad", "T": 16384, "k": 8, "E": 128,
         "local": 128, "H": 2048, "type": "bf16", "pad": 0},
        # the eight SwiGLU rows of one decoded token of the 35B shape, before the down product
        {"name": "quantise_decode", "op": "quantise", "M": 8, "K": 768, "type": "bf16", "pad": 0},
        # the SwiGLU rows of a prefill chunk of the 35B shape
        {"name": "quantise_prefill", "op": "quantise", "M": 131072, "K": 768, "type": "bf16",
         "pad": 0},
        # gate and up of one decoded token: eight experts with one row each (weights are read once)
        {"name": "product_decode", "op": "product", "T": 1, "k": 8, "E": 128, "N": 1536,
         "K": 2048, "out": "bf16", "swiglu": True, "pad": 0},
        # gate and up of a prefill chunk: 131,072 sorted rows over 128 experts
        {"name": "product_prefill", "op": "product", "T": 16384, "k": 8, "E": 128, "N": 1536,
         "K": 2048, "out": "bf16", "swiglu": True, "pad": 0},
        # a plain 8-bit linear layer over a ragged batch, fp32 out
        {"name": "product_linear_ragged", "op": "product", "T": 4001, "k": 1, "E": 1, "N": 5000,
         "K": 4096, "out": "fp32", "swiglu": False, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "sort", "sort_grad", "combine", "combine_grad", "quantise",
                     "product", "product", "product"])
    pad = rng.choice([0, 0, 8, 3])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "quantise":
        K = _log(rng, 100, 8192)
        return {"op": op, "M": _log(rng, 1, min(131072, 100_000_000 // K)), "K": K, "type": kind,
                "pad": pad}
    if op == "product":
        N, K = 2 * _log(rng, 64, 2500), _log(rng, 128, 6144)
        K = K if rng.random() < 0.25 else max(16, K // 16 * 16)
        E = rng.choice([e for e in (1, 1, 8, 64, 128) if e * N * K <= 400_000_000])
        k = min(E, rng.choice([1, 2, 8]))
        most = min(131072, 400_000_000_000 // (N * K), 300_000_000 // N)
        return {"op": op, "T": max(1, _log(rng, 1, most) // k), "k": k, "E": E, "N": N, "K": K,
                "out": kind, "swiglu": rng.random() < 0.5, "pad": rng.choice([0, 0, 16, 1])}
    E = rng.choice([8, 60, 128, 256])
    k = rng.choice([1, 2, 6, 8])
    H = _log(rng, 64, 8192)
    H = H if rng.random() < 0.3 else max(8, H // 8 * 8)
    T = _log(rng, 1, min(16384, 250_000_000 // (H * k)))
    case = {"op": op, "T": T, "k": k, "E": E, "local": rng.choice([E, E, E // 2]), "H": H,
            "type": kind, "pad": pad}
    if op == "sort":
        case["rows"] = rng.choice([kind, "i8"])
    return case


def _routing(g, T, k, E, local):
    """Expert ids and routing weights of T tokens: the k largest of logits whose experts are
    unequally liked; ids of experts that this rank does not hold are -1."""
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits += 0.5 * torch.randn(E, generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    ids = torch.where(ids < local, ids, -1).to(torch.int32)
    return ids.contiguous(), torch.softmax(top, dim=1).contiguous()


def _matrix(g, rows, cols, pad, kind):
    """A matrix of activations, a column slice of a wider one where `pad` is set."""
    wide = torch.randn(rows, cols + pad, generator=g, device="cuda")
    wide *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    return wide.to(_TYPES[kind])[:, :cols]


def _codes(g, rows, cols, pad):
    wide = torch.empty(rows, cols + pad, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 26) // (cols + pad))
    for at in range(0, rows, step):
        part = torch.randn(min(step, rows - at), cols + pad, generator=g, device="cuda")
        wide[at:at + step] = (part * 36).round_().clamp_(-127, 127).to(torch.int8)
    return wide[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quantise":
        s["x"] = _matrix(g, case["M"], case["K"], case["pad"], case["type"])
        s["codes"] = torch.zeros(case["M"], case["K"], dtype=torch.int8, device="cuda")
        s["scale"] = torch.zeros(case["M"], device="cuda")
        return s
    if op == "product":
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        M = T * k
        s["a"] = _codes(g, M, K, case["pad"])
        s["a_scale"] = torch.exp(0.5 * torch.randn(M, generator=g, device="cuda")) / 40
        s["w"] = _codes(g, E * N, K, case["pad"])
        s["w_scale"] = (0.5 + torch.rand(E * N, generator=g, device="cuda")) * 5e-4
        s["offsets"] = None
        if E > 1:  # the counts of a routed batch: rows are sorted by expert already
            counts = torch.bincount(_routing(g, T, k, E, E)[0].reshape(-1), minlength=E)
            s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
            s["offsets"][1:] = torch.cumsum(counts, 0)
            s["most_rows"] = int(counts.max())
        s["out"] = torch.zeros(M, N // 2 if case["swiglu"] else N, dtype=_TYPES[case["out"]],
                               device="cuda")
        return s
    T, k, E, local, H = (case[n] for n in ("T", "k", "E", "local", "H"))
    ids, weights = _routing(g, T, k, E, local)
    A = T * k
    if op == "sort":
        s["ids"], s["x"] = ids, _matrix(g, T, H, case["pad"], case["type"])
        s["offsets"] = torch.zeros(local + 1, dtype=torch.int32, device="cuda")
        s["order"] = torch.full((A,), -1, dtype=torch.int32, device="cuda")
        s["place"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        i8 = case["rows"] == "i8"
        s["rows"] = torch.zeros(A, H, dtype=torch.int8 if i8 else _TYPES[case["rows"]],
                                device="cuda")
        s["row_scale"] = torch.zeros(A, device="cuda") if i8 else None
        return s
    order = torch.argsort(torch.where(ids < 0, E, ids).reshape(-1), stable=True)
    place = torch.empty(A, dtype=torch.int32, device="cuda")
    place[order] = torch.arange(A, dtype=torch.int32, device="cuda")
    s["place"] = torch.where(ids < 0, -1, place.reshape(T, k)).contiguous()
    s["weights"] = weights
    s["rows"] = _matrix(g, A, H, case["pad"], case["type"])
    s["out"] = torch.zeros(T, H, dtype=_TYPES[case["type"]], device="cuda")
    if op == "combine_grad":
        s["dout"] = _matrix(g, T, H, case["pad"], case["type"])
        s["drows"] = torch.zeros(A, H, dtype=_TYPES[case["type"]], device="cuda")
        s["dweights"] = torch.zeros(T, k, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _quantised(x):
    """Codes and scales of rows, in 64 bits: a code next to a border has to be the right one."""
    x = x.double()
    m = x.abs().amax(1, keepdim=True)
    codes = torch.round(127 * x / torch.where(m > 0, m, 1.0))
    return codes.to(torch.int8), (m / 127).float().reshape(-1)


def _plain_sort(s):
    c = s["case"]
    ids, k, local = s["ids"].reshape(-1), c["k"], c["local"]
    key = torch.where((ids >= 0) & (ids < local), ids, local)
    _, order = torch.sort(key, stable=True)
    experts = torch.arange(local + 1, device="cuda", dtype=torch.int32)
    offsets = (key[None, :] < experts[:, None]).sum(1).to(torch.int32)
    place = torch.empty_like(ids)
    place[order] = torch.arange(ids.numel(), device="cuda", dtype=torch.int32)
    place = torch.where(key < local, place, -1).reshape(-1, k)
    placed = torch.arange(ids.numel(), device="cuda") < offsets[-1]
    token = order // k
    if c["rows"] == "i8":
        codes, scale = _quantised(s["x"])
        rows = torch.where(placed[:, None], codes[token], 0)
        return [offsets, torch.where(placed, order, -1).to(torch.int32), place, rows,
                torch.where(placed, scale[token], 0.0)]
    rows = torch.where(placed[:, None], s["x"][token], 0.0)
    return [offsets, torch.where(placed, order, -1).to(torch.int32), place, rows]


def _plain_combine(s, weighted):
    place, kind = s["place"], _TYPES[s["case"]["type"]]
    rows = s["rows"][place.clamp(min=0).reshape(-1)].float().reshape(*place.shape, -1)
    w = torch.where(place < 0, 0.0, s["weights"] if weighted else 1.0)
    return [(rows * w[:, :, None]).sum(1).to(kind)]


def _plain_combine_grad(s):
    place, kind = s["place"], _TYPES[s["case"]["type"]]
    T, k = place.shape
    dout = s["dout"].float()
    rows = s["rows"][place.clamp(min=0).reshape(-1)].float().reshape(T, k, -1)
    dweights = torch.where(place < 0, 0.0, (rows * dout[:, None, :]).sum(2))
    drows = torch.zeros(T * k + 1, dout.shape[1], dtype=kind, device="cuda")
    at = torch.where(place < 0, T * k, place).reshape(-1)  # dropped ones go behind the last row
    drows[at] = (s["weights"][:, :, None] * dout[:, None, :]).reshape(T * k, -1).to(kind)
    return [drows[:-1], dweights]


def _plain_product(s):
    c = s["case"]
    E, N, K = c["E"], c["N"], c["K"]
    a, M = s["a"].float(), s["a"].shape[0]
    w, w_scale = s["w"].reshape(E, N, K), s["w_scale"].reshape(E, N)
    if E == 1:
        v = a @ w[0].float().T * s["a_scale"][:, None] * w_scale
    else:
        row = torch.arange(M, device="cuda")
        expert = (row[:, None] >= s["offsets"][1:]).sum(1)
        if M <= 64:  # few rows: each with its expert's weight
            v = (w[expert].float() @ a[:, :, None])[:, :, 0]
        else:  # every expert's rows padded to the fullest expert's
            first = s["offsets"][:-1, None]
            at = first + torch.arange(s["most_rows"], device="cuda")
            v = torch.bmm(a[at.clamp(max=M - 1)], w.float().transpose(1, 2))
            v = v[expert, row - s["offsets"][expert]]
        v = v * s["a_scale"][:, None] * w_scale[expert]
    if c["swiglu"]:  # channel 2i is the gate of channel 2i + 1
        v = v[:, 0::2] / (1 + torch.exp(-v[:, 0::2])) * v[:, 1::2]
    return [v.to(_TYPES[c["out"]])]


def _plain(s):
    op = s["case"]["op"]
    if op == "sort":
        return _plain_sort(s)
    if op == "quantise":
        return list(_quantised(s["x"]))
    if op == "product":
        return _plain_product(s)
    if op == "combine_grad":
        return _plain_combine_grad(s)
    return _plain_combine(s, weighted=op == "combine")


# ------------------------------------------------------------------ the library's kernels


def _kernels(s):
    import expert_cache_offload_amd as m
    c = s["case"]
    op = c["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "sort":
        if "workspace" not in s:  # kept beside the outputs, as a user's program keeps it
            size = max(16, m.moe_sort_workspace_bytes(c["T"], c["k"], c["local"]))
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        x, rows, ws = s["x"], s["rows"], s["workspace"]
        m.moe_sort_tokens(s["ids"], c["T"], c["k"], c["local"], s["offsets"], s["order"],
                          s["place"], x, x.stride(0), c["H"], _TYPE_ID[c["type"]], rows,
                          rows.stride(0), _TYPE_ID[c["rows"]], s["row_scale"], ws, ws.numel(),
                          stream)
        out = [s["offsets"], s["order"], s["place"], rows]
        return out if s["row_scale"] is None else out + [s["row_scale"]]
    if op == "quantise":
        x, codes = s["x"], s["codes"]
        m.moe_quantise_rows(x, x.stride(0), _TYPE_ID[c["type"]], c["M"], c["K"], codes,
                            codes.stride(0), s["scale"], None, stream)
        return [codes, s["scale"]]
    if op == "product":
        a, w, out = s["a"], s["w"], s["out"]
        m.moe_product_i8(a, a.stride(0), s["a_scale"], a.shape[0], c["K"], w, w.stride(0),
                         s["w_scale"], c["N"], c["E"], s["offsets"], int(c["swiglu"]), out,
                         out.stride(0), _TYPE_ID[c["out"]], stream)
        return [out]
    rows, out, kind = s["rows"], s["out"], _TYPE_ID[c["type"]]
    T, k, H = c["T"], c["k"], c["H"]
    if op == "combine_grad":
        dout, drows = s["dout"], s["drows"]
        m.moe_combine_tokens_grad(dout, dout.stride(0), rows, rows.stride(0), T * k, kind,
                                  s["place"], s["weights"], T, k, H, drows, drows.stride(0),
                                  s["dweights"], stream)
        return [drows, s["dweights"]]
    if op == "sort_grad":
        m.moe_sort_tokens_grad(rows, rows.stride(0), T * k, kind, s["place"], T, k, H, out,
                               out.stride(0), stream)
    else:
        m.moe_combine_tokens(rows, rows.stride(0), T * k, kind, s["place"], s["weights"], T, k,
                             H, out, out.stride(0), stream)
    return [out]


def run(state):
    if own:
        return _kernels(state)
    return _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "quantise":
        return {"bytes": case["M"] * (case["K"] * (_BYTES[case["type"]] + 1) + 4), "flops": 0}
    if op == "product":
        M, N, K = case["T"] * case["k"], case["N"], case["K"]
        with_rows = min(case["E"], M)
        n_out = N // 2 if case["swiglu"] else N
        return {"bytes": M * K + with_rows * N * (K + 4) + M * (n_out * _BYTES[case["out"]] + 4),
                "flops": 2 * M * N * K}
    A = case["T"] * case["k"]
    n, size = A * case["local"] // case["E"], case["H"] * _BYTES[case["type"]]
    if op == "sort":
        rows = n * case["H"] * _BYTES[case["rows"]] + (4 * n if case["rows"] == "i8" else 0)
        return {"bytes": 8 * A + 4 * n + 4 * case["local"] + case["T"] * size + rows, "flops": 0}
    if op == "combine_grad":
        return {"bytes": case["T"] * size + 2 * n * size + 12 * A, "flops": 3 * n * case["H"]}
    return {"bytes": n * size + case["T"] * size + (8 if op == "combine" else 4) * A,
            "flops": 2 * n * case["H"]}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        x = s["x"].to(torch.float64)
        return [None, torch.linalg.vector_norm(x, ord=math.inf, dim=1) / 127]
    if op == "product":
        N, K = case["N"], case["K"]
        M = case["T"] * case["k"]
        ends = [0, M] if s["offsets"] is None else s["offsets"].tolist()
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if lo == hi:
                continue
            w = s["w"][e * N:(e + 1) * N].to(torch.float64) * s["w_scale"][e * N:(e + 1) * N, None]
            c = torch.mm(s["a"][lo:hi].to(torch.float64) * s["a_scale"][lo:hi, None].double(),
                         w.t())
            if case["swiglu"]:
                pair = c.reshape(hi - lo, N // 2, 2)
                c = pair[..., 0] * torch.sigmoid(pair[..., 0]) * pair[..., 1]
            out[lo:hi] = c
        return [out]
    if op == "sort":
        ids, x = s["ids"], s["x"].to(torch.float64)
        at = [torch.nonzero(ids.reshape(-1) == e).reshape(-1) for e in range(case["local"])]
        token = torch.cat(at) // case["k"]
        rows = torch.zeros(ids.numel(), case["H"], dtype=torch.float64, device="cuda")
        if case["rows"] == "i8":
            scale = torch.zeros(ids.numel(), dtype=torch.float64, device="cuda")
            scale[:token.numel()] = x.abs().max(1).values[token] / 127
            return [None, None, None, None, scale]
        rows[:token.numel()] = x[token]
        return [None, None, None, rows]
    place = s["place"]
    kind = torch.float64
    total = torch.zeros(case["T"], case["H"], dtype=kind, device="cuda")
    drows = torch.zeros(case["T"] * case["k"], case["H"], dtype=kind, device="cuda")
    dweights = torch.zeros(case["T"], case["k"], dtype=kind, device="cuda")
    for j in range(case["k"]):  # one choice of every token at a time
        have = torch.nonzero(place[:, j] >= 0).reshape(-1)
        rows = s["rows"][place[have, j].long()].to(kind)
        w = s["weights"][have, j].to(kind)
        if op == "combine_grad":
            dout = s["dout"][have].to(kind)
            drows[place[have, j].long()] = dout * w[:, None]
            dweights[have, j] = (dout * rows).sum(1)
        else:
            total[have] += rows * w[:, None] if op == "combine" else rows
    return [drows, dweights] if op == "combine_grad" else [total]
