"""Routing from logits (softmax or sigmoid scores, bias, groups, top-k, renormalised weights) and its
gradient, against plain implementations in 64 bits.

Experts are compared exactly.  Weights and gradients are computed in 64 bits and rounded to fp32 and
then to their type: U32 = 2^-24 and eps_t / 2 relative to the value."""
import math

import pytest

from test_gpu_ops import KINDS, U32, _gen, _half_ulp, env  # noqa: F401

pytestmark = pytest.mark.gpu
SOFTMAX, SIGMOID = 0, 1


def _scores(torch, z, score):
    if score == SIGMOID:
        return 1 / (1 + torch.exp(-z))
    e = torch.exp(z - z.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _ref(torch, z, score, bias, G, best, kept, k, renorm, scale):
    """Experts and weights in 64 bits; tokens without a NaN among their choice values."""
    z = z.double()
    T, E = z.shape
    inf = math.inf
    s = _scores(torch, z, score)
    out = z == -inf
    if bias is not None:
        out = out | (bias == -inf)
    c = z if bias is None else s + bias.double()
    c = torch.where(out, -inf, c)
    if G > 1 and kept < G:
        v = c if bias is not None or best == 1 else torch.where(out, -inf, s)
        top = torch.sort(v.reshape(T, G, E // G), dim=2, descending=True).values[:, :, :best]
        total = top[:, :, 0]
        if best == 2 and top.shape[2] == 2:
            total = total + torch.where(top[:, :, 1] == -inf, 0.0, top[:, :, 1])
        stay = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, stay, True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, -inf)
    value, idx = torch.sort(c, dim=1, descending=True, stable=True)
    idx, has = idx[:, :k], value[:, :k] > -inf
    w = torch.where(has, s.gather(1, idx), 0.0)
    if renorm:
        if score == SOFTMAX:  # scores far below the largest have left even 64 bits
            zc = torch.where(has, z.gather(1, idx), -inf)
            w = torch.where(has, torch.exp(zc - zc.amax(1, keepdim=True)), 0.0)
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(has, idx, -1).to(torch.int32), w * scale


def _run(env, z, kind, score, bias, G, best, kept, k, renorm, scale, stream=0):
    torch, m, types, tid = env
    T, E = z.shape
    idx = torch.full((T * k + 1,), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T * k + 1,), 77.0, device="cuda")
    m.moe_route_tokens(z, z.stride(0), tid[kind], T, E, score, bias, G, best, kept, k, renorm, scale,
                       idx, w, stream)
    assert int(idx[-1]) == -7 and float(w[-1]) == 77
    return idx[:-1].reshape(T, k), w[:-1].reshape(T, k)


def _check(env, z, kind, *args):
    torch = env[0]
    idx, w = _run(env, z, kind, *args)
    ref, ref_w = _ref(torch, z, *args)
    assert torch.equal(idx, ref), torch.nonzero(idx != ref)[:4].tolist()
    torch.testing.assert_close(w.double(), ref_w, rtol=U32 * 1.001, atol=2.0 ** -126)


def _logits(torch, g, T, E, kind, pad=0, masked=0.0, spread=1.5):
    wide = spread * torch.randn(T, E + pad, generator=g, device="cuda")
    if masked:
        wide[torch.rand(wide.shape, generator=g, device="cuda") < masked] = -math.inf
        wide[::7] = -math.inf  # rows that have no expert
    return wide.to(kind)[:, pad - pad // 2:pad - pad // 2 + E]


ROUTES = [  # T, E, k, groups, kept, padding, share masked
    (1, 1, 1, 1, 1, 0, 0.0), (8, 128, 8, 1, 1, 0, 0.0), (1, 256, 8, 8, 4, 0, 0.0),
    (1000, 60, 4, 6, 2, 1, 0.0), (5, 1024, 16, 16, 3, 0, 0.0), (33, 65, 3, 5, 2, 3, 0.3),
    (700, 257, 8, 1, 1, 0, 0.2), (100, 512, 10, 64, 7, 8, 0.9), (20001, 8, 2, 4, 1, 0, 0.0),
    (300, 384, 6, 3, 1, 0, 0.1), (64, 16, 16, 16, 16, 5, 0.5), (50, 130, 5, 13, 12, 0, 0.0),
    (3, 1000, 7, 50, 9, 1, 0.05), (9000, 128, 8, 2, 1, 0, 0.0),
    (3001, 160, 6, 8, 3, 0, 0.0), (2050, 256, 8, 8, 4, 3, 0.1), (77, 64, 12, 4, 2, 0, 0.2),
    (130, 96, 4, 1, 1, 0, 0.0), (9, 512, 16, 16, 4, 0, 0.0)]


@pytest.mark.parametrize("T,E,k,G,kept,pad,masked", ROUTES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route(env, T, E, k, G, kept, pad, masked, kind, score):
    torch, m, types, tid = env
    g = _gen(torch, T + E)
    z = _logits(torch, g, T, E, types[kind], pad, masked)
    bias = 0.2 * torch.randn(E, generator=g, device="cuda")
    some = torch.where(torch.rand(E, generator=g, device="cuda") < 0.3, -math.inf, bias)
    for b in (None, bias, some):
        for groups, stay, best in ((1, 1, 1), (G, kept, 1), (G, kept, 2)):
            for renorm, scale in ((True, 2.5), (False, 1.0)):
                _check(env, z, kind, score, b, groups, best, stay, k, renorm, scale)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_ties_and_near_ties(env, score):
    """Equal choice values go to the lower expert and the lower group; values that differ by less than
    fp32 holds are ordered as in 64 bits."""
    torch, m, types, tid = env
    g = _gen(torch, 4)
    T, E, k = 400, 256, 8
    z = torch.randint(-2, 3, (T, E), generator=g, device="cuda") / 4.0
    steps = torch.randint(0, 3, (E,), generator=g, device="cuda") / 8.0
    for b in (None, steps, steps * 0):
        for G, best, kept in ((1, 1, 1), (8, 1, 3), (8, 2, 3), (32, 2, 5)):
            _check(env, z.bfloat16(), "bf16", score, b, G, best, kept, k, True, 1.0)
            _check(env, z, "fp32", score, b, G, best, kept, k, True, 1.0)
    z = torch.randn(1, E, generator=g, device="cuda")
    if score == SOFTMAX:
        z = z.expand(T, E).contiguous()
    near = (0.5 - _scores(torch, z.double(), score)[0]).float()
    z = z + 1e-7 * torch.randn(T, E, generator=g, device="cuda")
    for G, best, kept in ((1, 1, 1), (8, 1, 3), (8, 2, 3)):
        _check(env, z.contiguous(), "fp32", score, near, G, best, kept, k, True, 1.0)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_far_values(env, score):
    """Logits far apart and biases that force a choice (also by infinity) or decide alone."""
    torch, m, types, tid = env
    g = _gen(torch, 6)
    T, E, k = 100, 96, 6
    z = 300 * torch.randn(T, E, generator=g, device="cuda")
    force = torch.zeros(E, device="cuda")
    force[[5, 50, 7]] = math.inf
    rank = torch.randperm(E, generator=g, device="cuda").float() * 10
    for b in (None, force, rank, -rank):
        for G, best, kept in ((1, 1, 1), (8, 2, 2)):
            for renorm in (True, False):
                _check(env, z, "fp32", score, b, G, best, kept, k, renorm, 1.0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_nan(env, kind, score):
    """A token with a NaN choice value has experts 0 .. k - 1 and weights NaN; the others keep theirs."""
    torch, m, types, tid = env
    g = _gen(torch, 8)
    T, E, k = 20, 64, 4
    z = _logits(torch, g, T, E, types[kind])
    clean = z.clone()
    z[3, 17] = math.nan
    z[5] = math.nan
    z[9, 0] = math.inf
    bad = [3, 5] + ([9] if score == SOFTMAX else [])
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    bias[17] = -math.inf  # not to be chosen: sigmoid scores do not look at its logit
    for b in (None, bias):
        args = (score, b, 8, 2, 3, k, True, 1.0)
        idx, w = _run(env, z, kind, *args)
        ref, ref_w = _ref(torch, torch.where(torch.isnan(z), -math.inf, z) if score == SIGMOID
                          else clean, *args)
        for t in range(T):
            if t in bad and not (t == 3 and score == SIGMOID and b is not None):
                assert idx[t].tolist() == list(range(k)) and bool(torch.isnan(w[t]).all())
            else:
                assert torch.equal(idx[t], ref[t]), t
                torch.testing.assert_close(w[t].double(), ref_w[t], rtol=U32 * 1.001, atol=0)
    nan_bias = bias.clone()
    nan_bias[1] = math.nan
    idx, w = _run(env, clean, kind, score, nan_bias, 1, 1, 1, k, False, 1.0)
    assert bool(torch.isnan(w).all()) and idx.tolist() == [list(range(k))] * T


def _grad_ref(torch, z, score, idx, k, renorm, scale, dw):
    z = z.double().clone().requires_grad_()
    has = (idx >= 0) & (idx < z.shape[1])
    at = torch.where(has, idx, 0).long()
    if score == SOFTMAX and renorm:
        w = torch.where(has, z.gather(1, at), -math.inf)
        w = torch.softmax(torch.where(has.any(1, keepdim=True), w, 0.0), 1)
    else:
        w = _scores(torch, z, score).gather(1, at)
        w = torch.where(has, w, 0.0)
        if renorm:
            w = w / torch.where(has.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
    loss = (torch.where(has, w * scale, 0.0) * dw.double().nan_to_num()).sum()
    return torch.autograd.grad(loss, z)[0]


@pytest.mark.parametrize("T,E,k,G,kept,pad,masked", ROUTES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_grad(env, T, E, k, G, kept, pad, masked, kind, score):
    torch, m, types, tid = env
    g = _gen(torch, T * 3 + E)
    z = _logits(torch, g, T, E, types[kind], pad)
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    if masked:
        r = torch.rand(T, k, generator=g, device="cuda")
        idx = torch.where(r < masked / 2, -1, torch.where(r < masked, E + 2, idx))
    idx = idx.contiguous()
    dw = torch.randn(T, k, generator=g, device="cuda")
    dw = torch.where((idx < 0) | (idx >= E), math.nan, dw)  # whatever stands beside no expert
    u = _half_ulp(torch, types[kind])
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        wide = torch.full((T + 1, E + 3), 77.0, dtype=types[kind], device="cuda")
        dz = wide[:T, 1:1 + E]
        m.moe_route_tokens_grad(z, z.stride(0), tid[kind], T, E, score, idx, k, renorm, scale, dw,
                                dz, E + 3)
        ref = _grad_ref(torch, z, score, idx, k, renorm, scale, dw)
        tol = ref.abs() * (u + 2 * U32) + 1e-13 * scale + (2.0 ** -25 if kind == "fp16" else 0)
        ok = (dz.double() - ref).abs() <= tol
        assert bool(ok.all()), (renorm, torch.nonzero(~ok)[:4].tolist())
        assert bool((wide[T:] == 77).all()) and bool((wide[:, 0] == 77).all()) and \
            bool((wide[:, 1 + E:] == 77).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("T,E,k", [(1, 5, 2), (33, 64, 8), (700, 257, 4), (50, 1024, 16)])
def test_route_grad_in_place(env, T, E, k, kind, score):
    """The gradient over the logits themselves."""
    torch, m, types, tid = env
    g = _gen(torch, T)
    z = _logits(torch, g, T, E, types[kind])
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    dw = torch.randn(T, k, generator=g, device="cuda")
    for renorm in (True, False):
        args = (tid[kind], T, E, score, idx, k, renorm, 2.5, dw)
        dz, own = torch.full((T, E), 77.0, dtype=types[kind], device="cuda"), z.clone()
        m.moe_route_tokens_grad(z, E, *args, dz, E)
        m.moe_route_tokens_grad(own, E, *args, own, E)
        assert torch.equal(own, dz)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("T,E,scale", [(1, 1, 1.0), (31, 8, 1.0), (612, 60, 16.0), (1749, 64, 2.5)])
def test_route_grad_of_one_renormalised_choice(env, T, E, scale, kind, score):
    """A single score divided by itself is one whatever the logits are: the gradient is zero, exactly,
    and it is written."""
    torch, m, types, tid = env
    g = _gen(torch, T)
    z = _logits(torch, g, T, E, types[kind])
    idx = torch.randint(0, E, (T, 1), generator=g, device="cuda").to(torch.int32)
    dw = torch.randn(T, 1, generator=g, device="cuda")
    dz = torch.full((T, E), 77.0, dtype=types[kind], device="cuda")
    m.moe_route_tokens_grad(z, E, tid[kind], T, E, score, idx, 1, True, scale, dw, dz, E)
    assert not bool(dz.any())


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_against_differences(env, score, renorm):
    """The derivative of a weighted sum of the chosen experts' weights along random directions; the
    choice has no derivative and stays."""
    torch, m, types, tid = env
    g = _gen(torch, 5)
    T, E, k, e = 3, 40, 6, 2.0 ** -7
    z = torch.randn(T, E, generator=g, device="cuda")
    z[:, ::5] += 4
    z = torch.round(z * 256) / 256  # z + e d is exact
    d = torch.sign(torch.randn(T, E, generator=g, device="cuda"))
    dw = torch.randn(T, k, generator=g, device="cuda")
    args = (score, None, 1, 1, 1, k, renorm, 1.0)
    idx, _ = _run(env, z, "fp32", *args)
    dz = torch.empty(T, E, device="cuda")
    m.moe_route_tokens_grad(z, E, tid["fp32"], T, E, score, idx, k, renorm, 1.0, dw, dz, E)
    sums = []
    for sign in (1, -1):
        w = _scores(torch, (z + sign * e * d).double(), score).gather(1, idx.long())
        if renorm:
            w = w / w.sum(1, keepdim=True)
        sums.append((w * dw.double()).sum().item())
    slope = (sums[0] - sums[1]) / (2 * e)
    # third derivatives of order one times e^2 / 6, and the gradient's roundings, of T k terms
    assert abs((dz.double() * d).sum().item() - slope) < T * k * (e * e + U32 / e)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_grad_of_masked_rows(env, score):
    """Rows without an expert have no gradient, a NaN stays one."""
    torch, m, types, tid = env
    T, E, k = 4, 16, 3
    z = torch.randn(T, E, generator=_gen(torch, 1), device="cuda")
    z[1] = -math.inf
    z[2, 3] = math.nan
    dw = torch.ones(T, k, device="cuda")
    dz = torch.full((T, E), 77.0, device="cuda")
    idx, _ = _run(env, z, "fp32", score, None, 1, 1, 1, k, False, 1.0)
    idx[2] = torch.tensor([3, 4, 5], dtype=torch.int32)
    m.moe_route_tokens_grad(z, E, tid["fp32"], T, E, score, idx, k, False, 1.0, dw, dz, E)
    assert not bool(dz[1].any()) and bool(torch.isnan(dz[2, 3])) and bool(
        torch.isfinite(dz[[0, 3]]).all())
