"""Calls that the norm, routing and adapter operators refuse, on the host, before any GPU work (no GPU
needed: the addresses are never dereferenced), and calls of no rows, which return without a launch."""
import math

import pytest

import more_ops_variants as v

BF16, FP16, FP32, I8 = 0, 1, 2, 3
P = 1 << 20  # an address


def _m():
    import expert_cache_offload_amd as m
    return m


def _refused(name, status, **kw):
    m = _m()
    with pytest.raises(m.MoeError) as e:
        getattr(m, name)(**kw)
    assert e.value.status == status, (name, kw, e.value)


Q = 1 << 24  # another one
NORM = {**v.norm_args(16, 64, "bf16"), "x": Q, "residual": 2 * Q, "y": 3 * Q}


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=P + 1), dict(x_stride=63), dict(x_stride=(1 << 40) + 1), dict(type=I8),
    dict(type=-1), dict(M=-1), dict(M=1 << 24), dict(K=0), dict(K=16385), dict(residual_stride=63),
    dict(residual=P + 1), dict(weight=None), dict(weight=P + 1), dict(eps=0.0), dict(eps=-1e-6),
    dict(eps=math.inf), dict(eps=math.nan), dict(sum_stride=63), dict(sum=P + 1),
    dict(residual=None), dict(y_stride=63), dict(y=P + 1), dict(codes_stride=63), dict(scale=None),
    dict(scale=P + 2), dict(y=None, codes=None)])
def test_norm_refuses(bad):
    _refused("moe_norm_rows", _m().MOE_E_INVALID, **{**NORM, **bad})


@pytest.mark.parametrize("over", [
    dict(sum=3 * Q), dict(sum=Q, sum_stride=65), dict(sum=2 * Q, sum_stride=65),
    dict(y=Q, y_stride=65), dict(y=2 * Q, y_stride=65)])
def test_norm_refuses_outputs_over_each_other_or_over_other_rows(over):
    _refused("moe_norm_rows", _m().MOE_E_INVALID, **{**NORM, **over})


@pytest.mark.parametrize("over", [dict(dx=Q, dx_stride=65), dict(dx=2 * Q, dx_stride=65)])
def test_norm_grad_refuses_other_rows(over):
    _refused("moe_norm_rows_grad", _m().MOE_E_INVALID,
             **{**GRAD, "dy": Q, "dsum": 2 * Q, "dsum_stride": 64, **over})


GRAD = v.norm_grad_args(500, 64, "fp32")


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(dy_stride=63), dict(dy=P + 2), dict(dsum=P, dsum_stride=63), dict(sum=None),
    dict(sum_stride=63), dict(type=I8), dict(M=-1), dict(M=1 << 24), dict(K=0), dict(K=16385),
    dict(weight=None), dict(eps=0.0), dict(dx_stride=63), dict(dx=P + 2), dict(dweight=P + 2),
    dict(dx=None, dweight=None), dict(workspace=None), dict(workspace=P + 2)])
def test_norm_grad_refuses(bad):
    _refused("moe_norm_rows_grad", _m().MOE_E_INVALID, **{**GRAD, **bad})


def test_norm_grad_workspace():
    m = _m()
    need = m.moe_norm_grad_workspace_bytes(500, 64)
    assert need > 0
    for M, K in ((-1, 64), (500, 0), (500, 16385), (0, 64), (1, 64)):
        assert m.moe_norm_grad_workspace_bytes(M, K) == 0
    _refused("moe_norm_rows_grad", m.MOE_E_SCRATCH, **{**GRAD, "workspace_bytes": need - 1})
    _refused("moe_norm_rows_grad", m.MOE_E_SCRATCH,
             **{**GRAD, "type": BF16, "workspace_bytes": need - 1})


@pytest.mark.parametrize("K,rows", [(3, 16), (64, 16), (300, 8), (1000, 4), (2000, 1), (16384, 1)])
def test_norm_grad_workspace_of_many_rows(K, rows):
    """A part of the weight's gradient holds 256 rows of each of a workgroup's row groups at most."""
    m = _m()
    for M in (1, 500, 1 << 17, (1 << 24) - 1):
        assert m.moe_norm_grad_workspace_bytes(M, K) >= 4 * K * (-(-M // (256 * rows)) if M > 1 else 0)


ROUTE = v.route_args(16, 64, 8, 8, 2, 4, "fp32")


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=P + 2), dict(logits_stride=63), dict(type=I8), dict(T=-1),
    dict(T=(1 << 20) + 1), dict(experts=0), dict(experts=1025), dict(score=2), dict(score=-1),
    dict(bias=P + 2), dict(groups=0), dict(groups=65), dict(groups=7), dict(group_best=0),
    dict(group_best=3), dict(top_groups=0), dict(top_groups=9), dict(top_k=0), dict(top_k=17),
    dict(experts=4, groups=1, top_groups=1, top_k=5), dict(scale=math.inf), dict(scale=math.nan),
    dict(topk_idx=None), dict(topk_idx=P + 2), dict(topk_w=None), dict(topk_w=P + 1)])
def test_route_refuses(bad):
    _refused("moe_route_tokens", _m().MOE_E_INVALID, **{**ROUTE, **bad})


ROUTE_GRAD = v.route_grad_args(16, 64, 8, "bf16")


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=P + 1), dict(logits_stride=63), dict(type=I8), dict(T=-1),
    dict(experts=1025), dict(score=2), dict(topk_idx=None), dict(topk_idx=P + 2), dict(top_k=17),
    dict(scale=math.nan), dict(dweights=None), dict(dweights=P + 2), dict(dlogits=None),
    dict(dlogits=P + 1), dict(dlogits_stride=63)])
def test_route_grad_refuses(bad):
    _refused("moe_route_tokens_grad", _m().MOE_E_INVALID, **{**ROUTE_GRAD, **bad})


@pytest.mark.parametrize("over", [dict(dx_stride=65), dict(sum_stride=65)])
def test_norm_grad_refuses_other_rows_of_the_sum(over):
    _refused("moe_norm_rows_grad", _m().MOE_E_INVALID,
             **{**GRAD, "dy": Q, "sum": 2 * Q, "dx": 2 * Q, **over})


@pytest.mark.parametrize("over", [dict(dlogits_stride=65), dict(logits_stride=65)])
def test_route_grad_refuses_other_rows(over):
    _refused("moe_route_tokens_grad", _m().MOE_E_INVALID,
             **{**ROUTE_GRAD, "logits": Q, "dlogits": Q, **over})


ADAPT = v.adapt_args(16, 64, 48, 8, 4, "fp16")


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=P + 1), dict(x_stride=63), dict(type=I8), dict(M=-1), dict(M=1 << 24),
    dict(K=0), dict(K=(1 << 20) + 1), dict(a=None), dict(a=P + 1), dict(a_stride=63), dict(b=None),
    dict(b=P + 1), dict(b_stride=7), dict(N=0), dict(N=(1 << 20) + 1), dict(rank=0),
    dict(rank=129, b_stride=129), dict(scale=P + 2), dict(adapters=0), dict(adapters=1025),
    dict(offsets=None), dict(offsets=P + 1), dict(order=P + 2), dict(base=P + 1),
    dict(base_stride=47), dict(out=None), dict(out=P + 1), dict(out_stride=47)])
def test_adapt_refuses(bad):
    _refused("moe_adapt_rows", _m().MOE_E_INVALID, **{**ADAPT, **bad})


def test_adapt_refuses_base_over_other_rows_of_out():
    over = dict(base=2 * Q, out=2 * Q)
    for strides in (dict(out_stride=49), dict(base_stride=49), dict(base_stride=96, out_stride=48)):
        _refused("moe_adapt_rows", _m().MOE_E_INVALID, **{**ADAPT, **over, **strides})


def test_no_rows_with_empty_buffers():
    m = _m()
    m.moe_norm_rows(None, 64, None, 64, BF16, 0, 64, None, 1e-6, None, 64, None, 64)
    m.moe_norm_rows_grad(None, 64, None, 64, None, 64, FP32, 0, 64, None, 1e-6, None, 64)
    m.moe_route_tokens(None, 64, FP32, 0, 64, 0, None, 1, 1, 1, 8, True, 1.0, None, None)
    m.moe_route_tokens_grad(None, 64, FP32, 0, 64, 1, None, 8, False, 1.0, None, None, 64)
    m.moe_adapt_rows(None, 64, FP16, 0, 64, None, 64, None, 8, 48, 8, None, 4, P, None, None, 48,
                     None, 48)


@pytest.mark.parametrize("name,good", [
    ("moe_norm_rows", NORM), ("moe_norm_rows_grad", {**GRAD, "dweight": None}),
    ("moe_route_tokens", ROUTE), ("moe_route_tokens_grad", ROUTE_GRAD), ("moe_adapt_rows", ADAPT)])
def test_no_rows_still_checks_sizes_and_types(name, good):
    rows = "T" if "T" in good else "M"
    getattr(_m(), name)(**{**good, rows: 0})
    for bad in (dict(type=I8), dict(K=0), dict(experts=0), dict(rank=200), dict(eps=0.0),
                dict(top_k=17)):
        if set(bad) <= set(good):
            _refused(name, _m().MOE_E_INVALID, **{**good, rows: 0, **bad})


def test_tensors_that_a_call_would_misread():
    """Tensors whose elements are of another width than the call reads, and tensors in ordinary host
    memory, are refused."""
    import torch
    m = _m()
    wide, half = torch.zeros(64, dtype=torch.int64), torch.zeros(64, dtype=torch.bfloat16)
    word, real = torch.zeros(64, dtype=torch.int32), torch.zeros(64)
    wrong = {  # by the width that is read: another one, and the right one in host memory
        "moe_norm_rows": (NORM, {n: (real, half) for n in ("x", "residual", "weight", "sum", "y")}
                          | {"codes": (half, half.view(torch.int8)), "scale": (half, real)}),
        "moe_norm_rows_grad": (GRAD, {n: (half, real) for n in ("dy", "sum", "weight", "dx",
                                                                "dweight")}
                               | {"workspace": (word, half)}),
        "moe_route_tokens": (ROUTE, {"logits": (half, real), "bias": (half, real),
                                     "topk_idx": (wide, word), "topk_w": (half, real)}),
        "moe_route_tokens_grad": (ROUTE_GRAD, {"logits": (real, half), "topk_idx": (wide, word),
                                               "dweights": (half, real), "dlogits": (real, half)}),
        "moe_adapt_rows": (ADAPT, {n: (real, half) for n in ("x", "a", "b", "base", "out")}
                           | {"scale": (half, real), "offsets": (wide, word),
                              "order": (wide, word)})}
    for name, (good, tensors) in wrong.items():
        for arg, both in tensors.items():
            for t in both:
                _refused(name, m.MOE_E_INVALID, **{**good, arg: t})
