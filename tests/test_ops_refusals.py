"""Calls that the token and 8-bit operators refuse, on the host, before any GPU work (no GPU needed:
the addresses are never dereferenced), and calls of no rows, which return without a launch."""
import pytest

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


SORT = dict(topk_idx=P, T=16, top_k=2, experts=8, offsets=P, order=P, place=P, x=P, x_stride=64,
            hidden=64, x_type=BF16, rows=P, rows_stride=64, rows_type=BF16, row_scale=None,
            workspace=None, workspace_bytes=0, stream=0)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=(1 << 20) + 1), dict(top_k=0), dict(top_k=17), dict(experts=0),
    dict(experts=1025), dict(topk_idx=None), dict(offsets=None), dict(place=None),
    dict(topk_idx=P + 2), dict(offsets=P + 1), dict(place=P + 2), dict(order=P + 2),
    dict(x=None), dict(rows=None), dict(hidden=0), dict(hidden=(1 << 20) + 1),
    dict(x_stride=63), dict(rows_stride=63), dict(x_type=I8, rows_type=I8), dict(x_type=4),
    dict(rows_type=FP16), dict(rows_type=I8), dict(x=P + 1), dict(rows=P + 1),
    dict(rows_type=I8, row_scale=P + 2), dict(x_stride=(1 << 40) + 1)])
def test_sort_refuses(bad):
    _refused("moe_sort_tokens", _m().MOE_E_INVALID, **{**SORT, **bad})


def test_sort_workspace():
    m = _m()
    assert m.moe_sort_workspace_bytes(1, 8, 128) == 0
    need = m.moe_sort_workspace_bytes(16384, 8, 128)
    assert need > 0
    assert m.moe_sort_workspace_bytes(-1, 8, 128) == 0
    assert m.moe_sort_workspace_bytes(16384, 17, 128) == 0
    big = {**SORT, "T": 16384, "top_k": 8, "experts": 128}
    _refused("moe_sort_tokens", m.MOE_E_SCRATCH,
             **{**big, "workspace": P, "workspace_bytes": need - 1})
    _refused("moe_sort_tokens", m.MOE_E_INVALID, **{**big, "workspace_bytes": need})
    _refused("moe_sort_tokens", m.MOE_E_INVALID,
             **{**big, "workspace": P + 2, "workspace_bytes": need})


COMBINE = dict(rows=P, rows_stride=64, n_rows=32, type=BF16, place=P, weights=P, T=16, top_k=2,
               hidden=64, out=P, out_stride=64, stream=0)


@pytest.mark.parametrize("bad", [
    dict(rows=None), dict(rows_stride=63), dict(n_rows=-1), dict(type=I8), dict(type=-1),
    dict(place=None), dict(place=P + 2), dict(weights=None), dict(weights=P + 2), dict(T=-1),
    dict(T=(1 << 20) + 1), dict(top_k=0), dict(top_k=17), dict(hidden=0), dict(out=None),
    dict(out_stride=63), dict(out=P + 1), dict(rows=P + 1)])
def test_combine_refuses(bad):
    _refused("moe_combine_tokens", _m().MOE_E_INVALID, **{**COMBINE, **bad})


@pytest.mark.parametrize("bad", [
    dict(drows=None), dict(drows_stride=63), dict(n_rows=-1), dict(type=I8), dict(place=None),
    dict(T=-1), dict(top_k=0), dict(hidden=0), dict(dx=None), dict(dx_stride=63)])
def test_sort_grad_refuses(bad):
    good = dict(drows=P, drows_stride=64, n_rows=32, type=FP16, place=P, T=16, top_k=2,
                hidden=64, dx=P, dx_stride=64, stream=0)
    _refused("moe_sort_tokens_grad", _m().MOE_E_INVALID, **{**good, **bad})


@pytest.mark.parametrize("bad", [
    dict(dout=None), dict(dout_stride=63), dict(rows=None), dict(rows_stride=63),
    dict(n_rows=-1), dict(type=I8), dict(place=None), dict(weights=None), dict(T=-1),
    dict(top_k=17), dict(hidden=0), dict(drows_stride=63), dict(drows=P + 2),
    dict(dweights=P + 2), dict(drows=None, dweights=None)])
def test_combine_grad_refuses(bad):
    good = dict(dout=P, dout_stride=64, rows=P, rows_stride=64, n_rows=32, type=FP32, place=P,
                weights=P, T=16, top_k=2, hidden=64, drows=P, drows_stride=64, dweights=P,
                stream=0)
    _refused("moe_combine_tokens_grad", _m().MOE_E_INVALID, **{**good, **bad})


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x_stride=63), dict(type=I8), dict(M=-1), dict(M=1 << 24), dict(K=0),
    dict(K=(1 << 20) + 1),
    dict(codes=None), dict(codes_stride=63), dict(scale=None), dict(scale=P + 2),
    dict(rows_end=P + 1), dict(x=P + 1)])
def test_quantise_refuses(bad):
    good = dict(x=P, x_stride=64, type=BF16, M=16, K=64, codes=P, codes_stride=64, scale=P,
                rows_end=None, stream=0)
    _refused("moe_quantise_rows", _m().MOE_E_INVALID, **{**good, **bad})


PRODUCT = dict(a=P, a_stride=64, a_scale=P, M=16, K=64, w=P, w_stride=64, w_scale=P, N=32,
               groups=4, offsets=P, epilogue=0, out=P, out_stride=32, out_type=BF16, stream=0)


@pytest.mark.parametrize("bad", [
    dict(a=None), dict(a_stride=63), dict(a_scale=None), dict(a_scale=P + 2), dict(M=-1),
    dict(M=1 << 24), dict(K=0), dict(K=131072, a_stride=131072, w_stride=131072),
    dict(w=None), dict(w_stride=63), dict(w_scale=None), dict(w_scale=P + 2), dict(N=0),
    dict(N=(1 << 20) + 1), dict(groups=0), dict(groups=1025), dict(offsets=None),
    dict(offsets=P + 2), dict(epilogue=2), dict(epilogue=-1), dict(epilogue=1, N=31),
    dict(out=None), dict(out_stride=31), dict(out_type=I8), dict(out_type=-1), dict(out=P + 1)])
def test_product_refuses(bad):
    _refused("moe_product_i8", _m().MOE_E_INVALID, **{**PRODUCT, **bad})


def test_no_rows_is_no_work():
    m = _m()
    m.moe_combine_tokens(**{**COMBINE, "T": 0})
    m.moe_product_i8(**{**PRODUCT, "M": 0})


def test_no_rows_with_empty_buffers():
    """An empty buffer has no address: calls of no tokens or no rows take null pointers for every
    buffer that is empty then (a rank of an expert-parallel layer that was sent no token)."""
    m = _m()
    none = dict(rows=None, place=None, weights=None, out=None, n_rows=0, T=0)
    m.moe_combine_tokens(**{**COMBINE, **none})
    m.moe_combine_tokens(**{**COMBINE, **none, "rows": P, "n_rows": 5})
    m.moe_sort_tokens_grad(None, 64, 0, BF16, None, 0, 2, 64, None, 64)
    for drows, dweights in ((P, P), (P, None), (None, P), (None, None)):
        m.moe_combine_tokens_grad(None, 64, None, 64, 0, FP32, None, None, 0, 2, 64, drows, 64,
                                  dweights)
    m.moe_quantise_rows(None, 64, FP16, 0, 64, None, 64, None)
    m.moe_product_i8(None, 64, None, 0, 64, P, 64, P, 32, 4, P, 0, None, 32, FP32)
    # tokens of which none was placed: no row to write a gradient to
    m.moe_combine_tokens_grad(P, 64, None, 64, 0, FP32, P, P, 16, 2, 64, None, 64, None)


@pytest.mark.parametrize("name,args", [
    ("moe_combine_tokens", (None, 64, 0, I8, None, None, 0, 2, 64, None, 64)),
    ("moe_combine_tokens", (None, 64, -1, BF16, None, None, 0, 2, 64, None, 64)),
    ("moe_combine_tokens", (None, 64, 0, BF16, None, None, 0, 17, 64, None, 64)),
    ("moe_sort_tokens_grad", (None, 64, 0, BF16, None, 0, 2, 0, None, 64)),
    ("moe_combine_tokens_grad", (None, 64, None, 64, 0, I8, None, None, 0, 2, 64, None, 64, None)),
    ("moe_quantise_rows", (None, 64, I8, 0, 64, None, 64, None)),
    ("moe_quantise_rows", (None, 64, BF16, 0, 0, None, 64, None)),
    ("moe_product_i8", (None, 64, None, 0, 0, P, 64, P, 32, 4, P, 0, None, 32, FP32)),
    ("moe_sort_tokens", (None, 0, 2, 8, None, None, None)),
    ("moe_sort_tokens", (None, 0, 2, 8, P, None, None, P, 64, 64, I8, None, 64, I8))])
def test_no_rows_still_checks_sizes_and_types(name, args):
    m = _m()
    with pytest.raises(m.MoeError) as e:
        getattr(m, name)(*args)
    assert e.value.status == m.MOE_E_INVALID


def test_tensors_that_a_call_would_misread():
    """Tensors whose elements are of another width than the call reads (64-bit expert ids, as
    torch.topk gives them, 16-bit weights) and tensors in ordinary host memory are refused."""
    import torch
    m = _m()
    wide, half = torch.zeros(64, dtype=torch.int64), torch.zeros(64, dtype=torch.bfloat16)
    word, real = torch.zeros(64, dtype=torch.int32), torch.zeros(64)
    for name in ("topk_idx", "offsets", "order", "place"):
        for t in (wide, word):  # another width; host memory
            _refused("moe_sort_tokens", m.MOE_E_INVALID, **{**SORT, name: t})
    for name, t in (("x", real), ("rows", real), ("row_scale", half), ("workspace", word)):
        _refused("moe_sort_tokens", m.MOE_E_INVALID, **{**SORT, name: t})
    for name, t in (("rows", real), ("place", wide), ("weights", half), ("out", real)):
        _refused("moe_combine_tokens", m.MOE_E_INVALID, **{**COMBINE, name: t})
    for name, t in (("a", word), ("a_scale", half), ("w", word), ("w_scale", half),
                    ("offsets", wide), ("out", real)):
        _refused("moe_product_i8", m.MOE_E_INVALID, **{**PRODUCT, name: t})
    grad = dict(dout=P, dout_stride=64, rows=P, rows_stride=64, n_rows=32, type=BF16, place=P,
                weights=P, T=16, top_k=2, hidden=64, drows=P, drows_stride=64, dweights=P)
    for name, t in (("dout", real), ("rows", real), ("place", wide), ("weights", half),
                    ("drows", real), ("dweights", half)):
        _refused("moe_combine_tokens_grad", m.MOE_E_INVALID, **{**grad, name: t})
    grad = dict(drows=P, drows_stride=64, n_rows=32, type=BF16, place=P, T=16, top_k=2, hidden=64,
                dx=P, dx_stride=64)
    for name, t in (("drows", real), ("place", wide), ("dx", real)):
        _refused("moe_sort_tokens_grad", m.MOE_E_INVALID, **{**grad, name: t})
    rows = dict(x=P, x_stride=64, type=BF16, M=16, K=64, codes=P, codes_stride=64, scale=P)
    for name, t in (("x", real), ("codes", word), ("scale", half), ("rows_end", wide)):
        _refused("moe_quantise_rows", m.MOE_E_INVALID, **{**rows, name: t})
