"""The norm, routing and adapter operators: the cases of more_ops_variants, which launch every kernel, and
runs of them together with the sort, the 8-bit products and the gradients, eager, captured and side
by side, against plain implementations in 64 bits."""
import pytest

import more_ops_variants as v
from test_gpu_adapt import _check as check_adapt, _ids as adapter_ids, _operands, _plan, \
    _ref as adapt_ref, _run as run_adapt
from test_gpu_norm import _check as check_norm, _check_grad, _run as run_norm, _run_grad, _sum
from test_gpu_ops import KINDS, LAYER_TOL, U32, _gen, _ids, _layer_buffers, _layer_ref, _matrix, \
    _rel, env  # noqa: F401
from test_gpu_route import SIGMOID, SOFTMAX, _check as check_route, _grad_ref, _logits, \
    _ref as route_ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


# ------------------------------------------------------------------ every kernel


@pytest.mark.parametrize("case", range(17))
@pytest.mark.parametrize("kind", KINDS)
def test_norm_kernels(env, kind, case):
    torch, m, types, tid = env
    assert len(v.norms(kind)) == 17
    M, K = v.norms(kind)[case]
    g = _gen(torch, M + K)
    x, r = (_matrix(torch, g, M, K, types[kind]) for _ in "xr")
    w = (1 + 0.5 * torch.randn(K, generator=g, device="cuda")).to(types[kind])
    check_norm(env, x, r, w, kind, run_norm(env, x, r, w, kind))
    _check_grad(env, r, None, x, w, kind, _run_grad(env, r, None, x, w, kind))


@pytest.mark.parametrize("case", range(len(v.ROUTES)))
@pytest.mark.parametrize("kind", KINDS)
def test_route_kernels(env, kind, case):
    torch, m, types, tid = env
    T, E, k, G, best, kept = v.ROUTES[case]
    g = _gen(torch, T + E)
    z = _logits(torch, g, T, E, types[kind])
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    for score in (SOFTMAX, SIGMOID):
        for b in (None, bias):
            check_route(env, z, kind, score, b, G, best, kept, k, True, 1.0)


@pytest.mark.parametrize("case", range(18))
@pytest.mark.parametrize("kind", KINDS)
def test_adapt_kernels(env, kind, case):
    torch, m, types, tid = env
    assert len(v.adapts(kind)) == 18
    M, K, N, rank, adapters = v.adapts(kind)[case]
    x, a, b, base, scale = _operands(env, M + K, M, K, N, rank, adapters, kind)
    ids = adapter_ids(torch, M, M, adapters, 0.1, 37)
    plan = _plan(env, ids, adapters)
    out = run_adapt(env, x, a, b, base, scale, plan, adapters, rank, kind)
    check_adapt(env, *out, *adapt_ref(torch, x, a, b, base, scale, ids, adapters, rank, kind), kind)


def test_offsets_beyond_32_bits(env):
    """Rows more than 2^31 elements apart in every operand that can be that large."""
    torch, m, types, tid = env
    g = _gen(torch, 9)
    wide, M, K = 1 << 20, 2100, 24

    def rows(cols, kind=torch.bfloat16):
        return torch.empty(M, wide, dtype=kind, device="cuda")[:, :cols]
    x, y = rows(K), rows(K)
    x.copy_(torch.randn(M, K, generator=g, device="cuda"))
    w = torch.rand(K, generator=g, device="cuda").bfloat16()
    codes, scale = rows(K, torch.int8), torch.empty(M, device="cuda")
    m.moe_norm_rows(x, wide, None, 0, 0, M, K, w, EPS, None, 0, y, wide, codes, wide, scale)
    near = x.contiguous()
    ref = run_norm(env, near, None, w, "bf16")
    assert torch.equal(y, ref["y"][1]) and torch.equal(codes, ref["codes"][1])
    dx, dw = rows(K), torch.empty(K, device="cuda")
    size = m.moe_norm_grad_workspace_bytes(M, K)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    m.moe_norm_rows_grad(y, wide, x, wide, x, wide, 0, M, K, w, EPS, dx, wide, dw, ws, size)
    _, ref, ref_w = _run_grad(env, y.contiguous(), near, near, w, "bf16")
    assert torch.equal(dx, ref) and torch.equal(dw, ref_w[:K])
    del codes
    idx = torch.empty(M, 4, dtype=torch.int32, device="cuda")
    weights = torch.empty(M, 4, device="cuda")
    m.moe_route_tokens(x, wide, 0, M, K, SIGMOID, None, 1, 1, 1, 4, True, 1.0, idx, weights)
    ref, ref_w = route_ref(torch, near, SIGMOID, None, 1, 1, 1, 4, True, 1.0)
    assert torch.equal(idx, ref)
    m.moe_route_tokens_grad(x, wide, 0, M, K, SIGMOID, idx, 4, True, 1.0, weights, dx, wide)
    ref = _grad_ref(torch, near, SIGMOID, idx, 4, True, 1.0, weights)
    assert bool(((dx.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + U32) + 1e-13).all())
    rank, adapters = 8, M // K  # A's and B's rows 2^20 elements apart too
    a = x[:adapters * rank]
    b = torch.empty(adapters * K, wide, dtype=torch.bfloat16, device="cuda")[:, :rank]
    b.copy_(torch.randn(adapters * K, rank, generator=g, device="cuda"))
    ids = adapter_ids(torch, 5, M, adapters, 0.1, 9)
    plan = _plan(env, ids, adapters)
    y.fill_(77)
    _, out = run_adapt(env, x, a, b, x, None, plan, adapters, rank, "bf16", out=y)
    check_adapt(env, None, out, *adapt_ref(torch, near, a, b, near, None, ids, adapters, rank,
                                           "bf16"), "bf16")


# ------------------------------------------------------------------ a layer for serving

LAYER = dict(score=SIGMOID, groups=4, best=2, kept=2, scale=2.5)


def _serve_buffers(env, seed, T, k, E, H, I, rank, adapters):
    """Weights of a layer and room for a call of it."""
    torch, m, types, tid = env
    g = _gen(torch, seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    wgu, wd = normal(E, 2 * I, H).double() * 0.06, normal(E, H, I).double() * 0.06
    b = _layer_buffers(env, T, k, E, H, I, wgu, wd)
    b["exact"] = wgu, wd
    b["wn"] = (1 + 0.2 * normal(H)).bfloat16()
    b["router"] = normal(E, H) * 0.06
    b["bias"] = 0.05 * normal(E)
    b["wp"] = normal(H, H).double() * 0.06  # a projection that all requests share
    codes = torch.empty(H, H, dtype=torch.int8, device="cuda")
    b["wp_scale"] = torch.empty(H, device="cuda")
    m.moe_quantise_rows(b["wp"].float(), H, 2, H, H, codes, H, b["wp_scale"])
    b["wp_codes"] = codes
    b["rank"], b["adapters"] = rank, adapters
    b["a"] = (normal(adapters * rank, H) * 0.06).bfloat16()
    b["b"] = (normal(adapters * H, rank) * 0.2).bfloat16()
    b["alpha"] = 0.5 + torch.rand(adapters, generator=g, device="cuda")
    dev = dict(device="cuda")
    for n in ("x", "res", "sum", "norm", "shared"):
        b[n] = torch.zeros(T, H, dtype=torch.bfloat16, **dev)
    b["codes"], b["scale"] = torch.zeros(T, H, dtype=torch.int8, **dev), torch.zeros(T, **dev)
    b["logits"] = torch.zeros(T, E, **dev)
    b["ids"] = torch.zeros(T, k, dtype=torch.int32, **dev)
    b["weights"] = torch.zeros(T, k, **dev)
    b["adapter"] = torch.zeros(T, dtype=torch.int32, **dev)
    b["by"] = torch.zeros(adapters + 1, dtype=torch.int32, **dev)
    b["order"], b["by_place"] = (torch.zeros(T, dtype=torch.int32, **dev) for _ in "op")
    b["by_ws"] = torch.empty(max(16, m.moe_sort_workspace_bytes(T, 1, adapters)),
                             dtype=torch.uint8, **dev)
    return b


def _serve(env, b, stream=0):
    """Residual and norm; router, experts in 8 bits; a shared projection in 8 bits with each request's
    adapter beside it."""
    torch, m, types, tid = env
    T, k, E, H, I = (b[n] for n in ("T", "k", "E", "H", "I"))
    A, L = T * k, LAYER
    m.moe_norm_rows(b["x"], H, b["res"], H, 0, T, H, b["wn"], EPS, b["sum"], H, b["norm"], H,
                    b["codes"], H, b["scale"], stream)
    torch.mm(b["norm"].float(), b["router"].t(), out=b["logits"])
    m.moe_route_tokens(b["logits"], E, 2, T, E, L["score"], b["bias"], L["groups"], L["best"],
                       L["kept"], k, True, L["scale"], b["ids"], b["weights"], stream)
    m.moe_sort_tokens(b["ids"], T, k, E, b["offsets"], None, b["place"], b["norm"], H, H, 0, b["xq"],
                      H, 3, b["xs"], b["ws"], b["ws"].numel(), stream)
    m.moe_product_i8(b["xq"], H, b["xs"], A, H, b["wgu"], H, b["sgu"], 2 * I, E, b["offsets"], 1,
                     b["act"], I, 0, stream)
    m.moe_quantise_rows(b["act"], I, 0, A, I, b["aq"], I, b["as"], b["offsets"][E:], stream)
    m.moe_product_i8(b["aq"], I, b["as"], A, I, b["wd"], I, b["sd"], H, E, b["offsets"], 0,
                     b["y_rows"], H, 0, stream)
    m.moe_combine_tokens(b["y_rows"], H, A, 0, b["place"], b["weights"], T, k, H, b["y"], H, stream)
    m.moe_product_i8(b["codes"], H, b["scale"], T, H, b["wp_codes"], H, b["wp_scale"], H, 1, None, 0,
                     b["shared"], H, 0, stream)
    m.moe_sort_tokens(b["adapter"], T, 1, b["adapters"], b["by"], b["order"], b["by_place"],
                      workspace=b["by_ws"], workspace_bytes=b["by_ws"].numel(), stream=stream)
    m.moe_adapt_rows(b["norm"], H, 0, T, H, b["a"], H, b["b"], b["rank"], H, b["rank"], b["alpha"],
                     b["adapters"], b["by"], b["order"], b["shared"], H, b["shared"], H, stream)


def _check_served(env, b):
    """Against 64 bits without any quantisation; the choice of experts exactly, from the logits."""
    torch = env[0]
    L = LAYER
    h = (b["x"].double() + b["res"].double()).bfloat16()
    assert torch.equal(b["sum"], h)
    y = h.double() * (h.double().square().mean(1, keepdim=True) + EPS).rsqrt() * b["wn"].double()
    assert _rel(b["norm"], y) <= 2.0 ** -8
    y = b["norm"].double()
    # fp32 products of H terms: the library's own, off by 2^-24 for each at most
    z = y @ b["router"].double().t()
    assert bool(((b["logits"].double() - z).abs() <=
                 (b["H"] + 8) * U32 * (y.abs() @ b["router"].double().abs().t())).all())
    ids, w = route_ref(torch, b["logits"], L["score"], b["bias"], L["groups"], L["best"], L["kept"],
                       b["k"], True, L["scale"])
    assert torch.equal(b["ids"], ids)
    torch.testing.assert_close(b["weights"].double(), w, rtol=U32 * 1.001, atol=0)
    assert _rel(b["y"], _layer_ref(torch, b["norm"], ids, w, *b["exact"])) <= LAYER_TOL
    shared = y @ b["wp"].t()
    for g in range(b["adapters"]):
        rows = b["adapter"] == g
        low = y[rows] @ b["a"][g * b["rank"]:(g + 1) * b["rank"]].double().t()
        shared[rows] += float(b["alpha"][g]) * low @ b["b"][g * b["H"]:(g + 1) * b["H"]].double().t()
    assert _rel(b["shared"], shared) <= LAYER_TOL


def _requests(env, b, g, none):
    torch = env[0]
    T, H = b["T"], b["H"]
    b["x"].copy_(torch.randn(T, H, generator=g, device="cuda"))
    b["res"].copy_(3 * torch.randn(T, H, generator=g, device="cuda"))
    b["adapter"].copy_(adapter_ids(torch, T, T, b["adapters"], none, max(1, T // 9)))


@pytest.mark.parametrize("T", [1, 8, 700])
def test_serving_layer(env, T):
    """A token, a few streams, a prompt."""
    torch = env[0]
    b = _serve_buffers(env, T, T, 4, 16, 256, 128, 16, 5)
    for none in (0.0, 0.4):
        _requests(env, b, _gen(torch, T + 1), none)
        _serve(env, b)
        _check_served(env, b)


def test_serving_layer_captured_and_on_another_stream(env):
    """Captured once and replayed with new inputs, eager work and synchronisation between the replays;
    and eagerly on a side stream."""
    torch = env[0]
    b, eager = (_serve_buffers(env, 3, 300, 4, 16, 256, 128, 24, 6) for _ in "ab")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):  # torch's product chooses its kernel before the capture
        _serve(env, b, side.cuda_stream)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        _serve(env, b, side.cuda_stream)
    torch.cuda.synchronize()
    for r in range(4):
        _requests(env, eager, _gen(torch, 60 + r), 0.2 * r)
        for n in ("x", "res", "adapter"):
            b[n].copy_(eager[n])
        torch.cuda.synchronize()
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        if r % 2:
            with torch.cuda.stream(side):
                _serve(env, eager, side.cuda_stream)
        else:
            _serve(env, eager)
        torch.cuda.synchronize()
        for n in ("sum", "norm", "codes", "ids", "weights", "y", "shared"):
            assert torch.equal(b[n], eager[n]), (r, n)
        _check_served(env, b)


def test_two_serving_layers_at_once(env):
    """Two layers of different sizes on two streams at the same time, each with its own buffers, give
    what each gives alone, every time."""
    torch = env[0]
    layers, alone = [], []
    for n, size in enumerate([(900, 4, 16, 512, 256, 40, 7), (37, 8, 32, 264, 72, 8, 20)]):
        b = _serve_buffers(env, 71 + n, *size)
        _requests(env, b, _gen(torch, 81 + n), 0.1)
        _serve(env, b)
        torch.cuda.synchronize()
        layers.append(b)
        alone.append({n: b[n].clone() for n in ("y", "shared")})
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        for b in layers:
            b["y"].fill_(3), b["shared"].fill_(3)
        torch.cuda.synchronize()
        for _ in range(3):
            for b, s in zip(layers, streams):
                with torch.cuda.stream(s):
                    _serve(env, b, s.cuda_stream)
        torch.cuda.synchronize()
        for b, was in zip(layers, alone):
            assert torch.equal(b["y"], was["y"]) and torch.equal(b["shared"], was["shared"])


# ------------------------------------------------------------------ a training step


@pytest.mark.parametrize("score,renorm", [(SOFTMAX, True), (SOFTMAX, False), (SIGMOID, True)])
def test_training_step_captured_beside_live_gradients(env, score, renorm):
    """Norm, router, sort, a factor per expert in torch, combine, and every gradient, captured and
    replayed while an eager autograd graph over the same leaves is alive; gradients against
    autograd's of the plain form in 64 bits, at the experts that the kernel chose."""
    torch, m, types, tid = env
    T, H, E, k = 90, 72, 10, 3
    g = _gen(torch, 31)

    def leaf(*shape, by=1.0):
        return (by * torch.randn(*shape, generator=g, device="cuda")).requires_grad_()
    x, r, wr = leaf(T, H), leaf(T, H), leaf(E, H, by=0.2)
    wn = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).requires_grad_()
    dout, dsum = (torch.randn(T, H, generator=g, device="cuda") for _ in "ds")
    factor = torch.randn(E, generator=g, device="cuda")
    dev = dict(device="cuda")
    h, y, out, dy, dx = (torch.zeros(T, H, **dev) for _ in range(5))
    z, dz = torch.zeros(T, E, **dev), torch.zeros(T, E, **dev)
    ids, w, dw = torch.zeros(T, k, dtype=torch.int32, **dev), torch.zeros(T, k, **dev), \
        torch.zeros(T, k, **dev)
    rows, y_rows, drows = (torch.zeros(T * k, H, **dev) for _ in range(3))
    by = torch.zeros(T * k, 1, **dev)
    offsets, order, place = (torch.zeros(n, dtype=torch.int32, **dev)
                             for n in (E + 1, T * k, T * k))
    dwn, dwr = torch.zeros(H, **dev), torch.zeros(E, H, **dev)
    size = m.moe_norm_grad_workspace_bytes(T, H)
    ws = torch.empty(max(16, size, m.moe_sort_workspace_bytes(T, k, E)), dtype=torch.uint8, **dev)
    xd, rd, wrd, wnd = (t.detach() for t in (x, r, wr, wn))
    A = T * k

    def step(s):
        m.moe_norm_rows(xd, H, rd, H, 2, T, H, wnd, EPS, h, H, y, H, stream=s)
        torch.mm(y, wrd.t(), out=z)
        m.moe_route_tokens(z, E, 2, T, E, score, None, 1, 1, 1, k, renorm, 1.5, ids, w, s)
        m.moe_sort_tokens(ids, T, k, E, offsets, order, place, y, H, H, 2, rows, H, 2, None, ws,
                          ws.numel(), s)
        by.copy_(factor[ids.reshape(-1)[order.long()].long()][:, None])
        torch.mul(rows, by, out=y_rows)
        m.moe_combine_tokens(y_rows, H, A, 2, place, w, T, k, H, out, H, s)
        m.moe_combine_tokens_grad(dout, H, y_rows, H, A, 2, place, w, T, k, H, drows, H, dw, s)
        drows.mul_(by)
        m.moe_sort_tokens_grad(drows, H, A, 2, place, T, k, H, dy, H, s)
        m.moe_route_tokens_grad(z, E, 2, T, E, score, ids, k, renorm, 1.5, dw, dz, E, s)
        dy.addmm_(dz, wrd)
        torch.mm(dz.t(), y, out=dwr)
        m.moe_norm_rows_grad(dy, H, dsum, H, h, H, 2, T, H, wnd, EPS, dx, H, dwn, ws, ws.numel(), s)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(side.cuda_stream)
    torch.cuda.synchronize()
    at = ids.long()

    def plain():
        ph = x.double() + r.double()
        py = ph * (ph.square().mean(1, keepdim=True) + EPS).rsqrt() * wn.double()
        pz = py @ wr.double().t()
        s = torch.softmax(pz, 1) if score == SOFTMAX else torch.sigmoid(pz)
        s = s.gather(1, at)
        if renorm:
            s = s / s.sum(1, keepdim=True)
        pout = (1.5 * s * factor.double()[at]).sum(1, keepdim=True) * py
        return ph, pout
    ph, pout = plain()  # alive while the step is captured
    with torch.cuda.graph(graph, stream=side):
        step(side.cuda_stream)
    torch.cuda.synchronize()
    torch.autograd.backward([ph, pout], [dsum.double(), dout.double()])
    for _ in range(3):
        for t in (h, y, out, dy, dx, z, dz, w, dw, rows, y_rows, drows, dwn, dwr, by):
            t.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        # six steps of sums over at most T = 90 terms each, at worst added up one by one, where the
        # differences of the score's gradient cancel to a quarter: norms within 6 * 90 * 4 * 2^-24
        for got, ref in ((out, pout.detach()), (dx, x.grad), (dx, r.grad), (dwn, wn.grad),
                         (dwr, wr.grad)):
            assert _rel(got, ref.double()) <= 6 * 90 * 4 * U32
