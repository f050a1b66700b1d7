"""The cases of ops_variants, which launch every kernel of the operators, against plain implementations
in 64 bits: rows matrices above 128 MiB, sorts of many chunks, every tile of the 8-bit product going
on to a second tile.  Integers, copies and codes are compared exactly, tolerances count roundings."""
import pytest

import ops_variants as v
from test_gpu_ops import U32, _codes, _gen, _half_ulp, _matrix, _quantised, _scales, env  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ 8-bit product


def _sums(torch, a, w, N, ends):
    """The integer sums in 64 bits, and the group of each row that has one."""
    M = a.shape[0]
    c = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    group = torch.full((M,), -1, dtype=torch.int64)
    for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if lo < hi:
            torch.mm(a[lo:hi].double(), w[g * N:(g + 1) * N].double().t(), out=c[lo:hi])
            group[lo:hi] = g
    return c, group.cuda()


def _check_products(env, counts, N, K, pad, at):
    torch, m, types, tid = env
    one = isinstance(counts, int)
    G = 1 if one else len(counts)
    ends = [0, counts] if one else [v.BEFORE]
    for n in () if one else counts:
        ends.append(ends[-1] + n)
    M = counts if one else ends[-1] + v.BEHIND
    g = _gen(torch, M + N + K)
    a, w = _codes(torch, g, M, K, pad, at), _codes(torch, g, G * N, K, pad, at)
    a_scale, w_scale = _scales(torch, g, M, G * N)
    offsets = None if one else torch.tensor(ends, dtype=torch.int32, device="cuda")
    c, group = _sums(torch, a, w, N, ends)
    has = group >= 0
    c *= a_scale.double()[:, None] * w_scale.reshape(G, N).double()[group.clamp(min=0)]
    for swiglu in (False, True):
        # conversion of the sum and two scales; with SwiGLU these for gate and up, the gate's
        # acting on silu 1 + |gate| times at most, and those of silu itself; a gate whose exp
        # leaves fp32 gives 0 for less than |gate| 2^-128
        ref, steps = c, 3.0 * c.abs()
        if swiglu:
            gate, up = c[:, 0::2], c[:, 1::2]
            ref = gate * torch.sigmoid(gate) * up
            steps = ref.abs() * (16 + 3 * gate.abs()) + (gate * up).abs() * (2.0 ** -128 / U32)
        for kind in v.KINDS:
            args = v.product_args(counts, N, K, pad, at, kind, swiglu)
            out = torch.full(ref.shape, 77.0, dtype=types[kind], device="cuda")
            assert (args["M"], args["a_stride"]) == (M, a.stride(0))
            m.moe_product_i8(**{**args, "a": a, "a_scale": a_scale, "w": w, "w_scale": w_scale,
                                "offsets": offsets, "out": out})
            u = _half_ulp(torch, types[kind])
            tol = steps * (U32 * (1 + u)) + u * ref.abs() + (2.0 ** -25 if kind == "fp16" else 0)
            ok = (out.double() - ref).abs_() <= tol
            ok[~has] = (out == 77)[~has]
            assert bool(ok.all()), (kind, swiglu, torch.nonzero(~ok)[:4].tolist())


@pytest.mark.parametrize("case", range(len(v.TILES)))
def test_product_tiles(env, case):
    """More tiles than workgroups: the next tile is taken up while the last one's outputs are on
    their way; one, an even and an odd number of rounds; groups of all sizes, also more of
    them than a workgroup has threads."""
    _check_products(env, *v.TILES[case][3:])


@pytest.mark.parametrize("case", range(len(v.FEW)))
def test_product_few(env, case):
    _check_products(env, *v.FEW[case])


# ------------------------------------------------------------------ tokens


def _routing(torch, g, T, k, experts, drop):
    ids = torch.randint(0, experts, (T, k), generator=g, device="cuda", dtype=torch.int32)
    if drop:
        r = torch.rand(T, k, generator=g, device="cuda")
        ids = torch.where(r < drop / 2, -1, torch.where(r < drop, experts + 3, ids))
    return ids.contiguous()


def _sorted(torch, ids, experts):
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    n = int(offsets[-1])
    order = torch.sort(key, stable=True).indices[:n]
    place = torch.full_like(flat, -1)
    place[order] = torch.arange(n, dtype=torch.int32, device="cuda")
    return offsets, order, place, n


def _check_sort(env, T, k, experts, drop, H, pad, at, kind, rows_kind):
    torch, m, types, tid = env
    g = _gen(torch, T + k + H)
    ids = _routing(torch, g, T, k, experts, drop)
    A = T * k
    offsets = torch.full((experts + 2,), -7, dtype=torch.int32, device="cuda")
    order, place = (torch.full((A + 1,), -7, dtype=torch.int32, device="cuda") for _ in "ab")
    size = m.moe_sort_workspace_bytes(T, k, experts)
    ws = torch.full((max(size, 16) + 64,), 0x5a, dtype=torch.uint8, device="cuda")
    ints = dict(topk_idx=ids, T=T, top_k=k, experts=experts, offsets=offsets, order=order,
                place=place, workspace=ws, workspace_bytes=max(size, 16))
    if H:
        x = _matrix(torch, g, T, H, types[kind], pad, at)
        rows = torch.full((A + 1, H), 77, dtype=types[rows_kind], device="cuda")
        scale = torch.full((A + 1,), 77.0, device="cuda")
        args = v.sort_args(T, k, experts, H, pad, at, kind, rows_kind)
        assert args["x_stride"] == x.stride(0)
        m.moe_sort_tokens(**{**args, **ints, "x": x, "rows": rows, "row_scale": scale})
    else:
        m.moe_sort_tokens(**ints)
    ref_offsets, ref_order, ref_place, n = _sorted(torch, ids, experts)
    assert torch.equal(offsets[:-1].long(), ref_offsets) and int(offsets[-1]) == -7
    assert torch.equal(order[:n].long(), ref_order) and bool((order[n:] == -7).all())
    assert torch.equal(place[:-1], ref_place) and int(place[-1]) == -7
    assert bool((ws[max(size, 16):] == 0x5a).all())
    if not H:
        return
    token = ref_order // k
    assert bool((rows[n:] == 77).all())
    if rows_kind == "i8":
        codes, want = _quantised(torch, x)
        assert torch.equal(rows[:n], codes[token])
        torch.testing.assert_close(scale[:n].double(), want[token], rtol=U32, atol=0)
        assert bool((scale[n:] == 77).all())
    else:
        assert torch.equal(rows[:n], x[token]) and bool((scale == 77).all())


@pytest.mark.parametrize("case", range(len(v.SORTS)))
@pytest.mark.parametrize("kind", v.KINDS)
@pytest.mark.parametrize("codes", [False, True])
def test_sort(env, case, kind, codes):
    _check_sort(env, *v.SORTS[case], kind, "i8" if codes else kind)


@pytest.mark.parametrize("kind", v.KINDS)
def test_sort_of_short_rows_above_128_mib(env, kind):
    _check_sort(env, *v.SORTS_SHORT_STREAMED[kind == "fp32"], kind, kind)


@pytest.mark.parametrize("T,k,experts,drop", v.SORTS_INTEGERS)
def test_sort_of_many_chunks(env, T, k, experts, drop):
    """Up to 16,384 chunks: the scan's segments hold more of them than it keeps in registers."""
    _check_sort(env, T, k, experts, drop, 0, 0, 0, None, None)


def _places(torch, g, T, k, drop):
    """Distinct places of the kept assignments in a random order, among T * k rows."""
    keep = torch.rand(T * k, generator=g, device="cuda") >= drop
    place = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    return torch.where(keep, place, -1).reshape(T, k).contiguous()


@pytest.mark.parametrize("case", range(len(v.COMBINES)))
@pytest.mark.parametrize("kind", v.KINDS)
def test_combine_and_gradients(env, case, kind):
    torch, m, types, tid = env
    T, k, drop, H, pad, at = v.COMBINES[case]
    g = _gen(torch, T + H)
    place = _places(torch, g, T, k, drop)
    rows = _matrix(torch, g, T * k, H, types[kind], pad, at)
    dout = _matrix(torch, g, T, H, types[kind])
    w = torch.rand(T, k, generator=g, device="cuda") * 2 - 0.5
    args = v.combine_args(T, k, H, pad, at, kind)
    assert args["rows_stride"] == rows.stride(0)
    kept, at_row = place >= 0, place.clamp(min=0).long()
    u, low = _half_ulp(torch, types[kind]), 2.0 ** -25 if kind == "fp16" else 0.0
    r = [torch.where(kept[:, j, None], rows[at_row[:, j]].double(), 0.0) for j in range(k)]
    # sums: k products and k - 1 additions in sequence, then the output's own rounding
    for weights in (w, None):
        out = torch.full((T, H), 77.0, dtype=types[kind], device="cuda")
        f = torch.ones(T, k, dtype=torch.float64, device="cuda") if weights is None else w.double()
        ref = sum(r[j] * f[:, j, None] for j in range(k))
        mag = sum((r[j] * f[:, j, None]).abs() for j in range(k))
        if weights is None:
            m.moe_sort_tokens_grad(rows, rows.stride(0), T * k, tid[kind], place, T, k, H, out, H)
        else:
            m.moe_combine_tokens(**{**args, "rows": rows, "place": place, "weights": w,
                                    "out": out})
        tol = (k + 1) * U32 * (1 + u) * mag + u * ref.abs() + low
        assert bool(((out.double() - ref).abs() <= tol).all())
    drows = torch.full((T * k, H), 77.0, dtype=types[kind], device="cuda")
    dw = torch.full((T, k), 77.0, device="cuda")
    m.moe_combine_tokens_grad(dout, H, rows, rows.stride(0), T * k, tid[kind], place, w, T, k, H,
                              drows, H, dw)
    left = torch.ones(T * k, dtype=torch.bool, device="cuda")
    for j in range(k):
        ref = dout.double() * w[:, j, None].double()
        got = drows[at_row[:, j]].double()
        ok = (got - ref).abs() <= (u + 2 * U32) * ref.abs() + low
        assert bool(ok[kept[:, j]].all())
        left[at_row[kept[:, j], j]] = False
        _check_weight_gradient(torch, dw[:, j], dout.double() * r[j], kind)
    assert bool((drows[left] == 77).all())


def _check_weight_gradient(torch, got, products, kind):
    """Products and sums in fp32 within a chunk of 16 bytes (as many roundings as elements), exact
    but for 2^-53 beyond, rounded once to fp32."""
    ref, mag = products.sum(1), products.abs().sum(1)
    chunk = 4 if kind == "fp32" else 8
    tol = (chunk + 2.0 ** -20) * U32 * mag + U32 * ref.abs()
    assert bool(((got.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("kind", v.KINDS)
@pytest.mark.parametrize("H", [1, 7, 515, 2051, 20001])
def test_weight_gradient_roundings(env, H, kind):
    torch, m, types, tid = env
    g = _gen(torch, H)
    T, k = 40, 3
    place = _places(torch, g, T, k, 0.2)
    rows, dout = (_matrix(torch, g, n, H, types[kind]) for n in (T * k, T))
    dw = torch.full((T, k), 77.0, device="cuda")
    m.moe_combine_tokens_grad(dout, H, rows, H, T * k, tid[kind], place,
                              torch.ones(T, k, device="cuda"), T, k, H, None, H, dw)
    r = torch.where((place >= 0)[:, :, None], rows[place.clamp(min=0).long()].double(), 0.0)
    for j in range(k):
        _check_weight_gradient(torch, dw[:, j], dout.double() * r[:, j], kind)


@pytest.mark.parametrize("kind", v.KINDS)
def test_weight_gradient_of_sums_that_cancel(env, kind):
    """A large part that cancels over a lane's chunks and a small one that stays: every chunk's sum is
    a number of fp32, their sums are not, and the result is exact in 64 bits."""
    torch, m, types, tid = env
    chunk = 4 if kind == "fp32" else 8
    rounds = 8  # chunks of a lane
    H = 64 * chunk * rounds
    big, small = 2.0 ** 15, 2.0 ** -10  # of fp16 too; 25 bits apart
    value = torch.tensor([big, small, -big, small] * (rounds // 4), dtype=torch.float64)
    x = torch.zeros(rounds, 64, chunk, dtype=torch.float64)
    x[:, :, 0] = value[:, None]
    rows = x.reshape(1, H).cuda().to(types[kind])
    want = 64 * rounds // 2 * small
    assert float(rows.double().sum()) == want
    lane = torch.zeros((), dtype=torch.float32)  # what sums held in fp32 over a lane would give
    for c in value:
        lane = lane + c.float()
    assert float(lane) * 64 != want
    one = torch.ones(1, H, device="cuda").to(types[kind])
    dw = torch.full((1, 1), 77.0, device="cuda")
    m.moe_combine_tokens_grad(one, H, rows, H, 1, tid[kind],
                              torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                              torch.ones(1, 1, device="cuda"), 1, 1, H, None, H, dw)
    assert float(dw) == want


@pytest.mark.parametrize("kind,at", [(kind, at) for kind in v.KINDS
                                     for at in range(2 * len(v.QUANTISES))])
def test_quantise(env, kind, at):
    torch, m, types, tid = env
    M, K = v.quantises(kind)[at]
    g = _gen(torch, M + K)
    x = torch.empty(M, K, dtype=types[kind], device="cuda").normal_(generator=g)
    x *= torch.exp(torch.randn(M, 1, generator=g, device="cuda")).to(types[kind])
    codes = torch.full((M + 1, K), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((M + 1,), 99.0, device="cuda")
    m.moe_quantise_rows(**{**v.quantise_args(M, K, kind), "x": x, "codes": codes, "scale": scale})
    ref, want = _quantised(torch, x)
    assert torch.equal(codes[:M], ref) and bool((codes[M] == 99).all())
    torch.testing.assert_close(scale[:M].double(), want, rtol=U32, atol=0)
    assert float(scale[M]) == 99


# ------------------------------------------------------------------ no tokens


def test_layer_of_no_tokens(env):
    """An expert layer's calls on real empty buffers: the offsets are zero, nothing else is
    written."""
    torch, m, types, tid = env
    E, k, H, inter = 6, 4, 64, 32
    z = dict(device="cuda")
    offsets = torch.full((E + 1,), -7, dtype=torch.int32, **z)
    ids, place = (torch.zeros(0, k, dtype=torch.int32, **z) for _ in "ab")
    weights, x, y = torch.zeros(0, k, **z), *(torch.zeros(0, H, **z).bfloat16() for _ in "ab")
    xq, act = torch.zeros(0, H, dtype=torch.int8, **z), torch.zeros(0, inter, **z).bfloat16()
    scale = torch.zeros(0, **z)
    wgu = torch.ones(E * 2 * inter, H, dtype=torch.int8, **z)
    sgu = torch.ones(E * 2 * inter, **z)
    assert x.data_ptr() == 0
    m.moe_sort_tokens(ids, 0, k, E, offsets, None, place, x, H, H, 0, xq, H, 3, scale)
    assert offsets.tolist() == [0] * (E + 1)
    offsets.fill_(-7)
    room = torch.full((8, H), 77.0, **z).bfloat16()  # one of the two buffers is not empty
    m.moe_sort_tokens(ids, 0, k, E, offsets, None, place, x, H, H, 0, room, H, 0)
    assert offsets.tolist() == [0] * (E + 1) and bool((room == 77).all())
    m.moe_product_i8(xq, H, scale, 0, H, wgu, H, sgu, 2 * inter, E, offsets, 1, act, inter, 0)
    m.moe_quantise_rows(act, inter, 0, 0, inter, xq, inter, scale, offsets[E:])
    m.moe_combine_tokens(act, H, 0, 0, place, weights, 0, k, H, y, H)
    m.moe_combine_tokens_grad(y, H, act, H, 0, 0, place, weights, 0, k, H, act, H, weights)
    m.moe_sort_tokens_grad(act, H, 0, 0, place, 0, k, H, x, H)
    torch.cuda.synchronize()
