"""Low-rank adapters over rows sorted by adapter, against a plain implementation in 64 bits.

Tolerances count roundings: U32 = 2^-24 for each fp32 addition relative to the magnitudes it adds, the
parts that x A^T is split into (bf16: 2^-17 relative to each; fp16: 2^-22 of the row's largest), and
eps_t / 2 for the output's own rounding."""
import pytest

import more_ops_variants as v
from test_gpu_ops import KINDS, U32, _gen, _half_ulp, _matrix, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _plan(env, ids, adapters):
    """offsets and order as the sort writes them."""
    torch, m, types, tid = env
    M = ids.numel()
    offsets = torch.full((adapters + 1,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((M,), -7, dtype=torch.int32, device="cuda")
    place = torch.empty(M, dtype=torch.int32, device="cuda")
    size = m.moe_sort_workspace_bytes(M, 1, adapters)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    m.moe_sort_tokens(ids, M, 1, adapters, offsets, order, place, workspace=ws,
                      workspace_bytes=ws.numel())
    return offsets, order


def _operands(env, seed, M, K, N, rank, adapters, kind, pad=0, at=0):
    torch, m, types, tid = env
    g = _gen(torch, seed)
    x = _matrix(torch, g, M, K, types[kind], pad, at)
    a = _matrix(torch, g, adapters * rank, K, types[kind], pad, at)
    b = _matrix(torch, g, adapters * N, rank, types[kind], pad, at)
    base = _matrix(torch, g, M, N, types[kind], pad, at)
    scale = torch.randn(adapters, generator=g, device="cuda")
    return x, a, b, base, scale


def _ref(torch, x, a, b, base, scale, ids, adapters, rank, kind):
    """Output, tolerance before the output's rounding, and which rows have an adapter."""
    M, N = x.shape[0], b.shape[0] // adapters
    K = x.shape[1]
    ref, tol = (torch.zeros(M, N, dtype=torch.float64, device="cuda") for _ in "rt")
    if base is not None:
        ref += base.double()
        tol += base.double().abs() * U32
    has = torch.zeros(M, dtype=torch.bool, device="cuda")
    for g in range(adapters):
        rows = torch.nonzero(ids == g)[:, 0]
        if not rows.numel():
            continue
        has[rows] = True
        s = 1.0 if scale is None else float(scale[g])
        xg, ag = x[rows].double(), a[g * rank:(g + 1) * rank].double()
        bg = b[g * N:(g + 1) * N].double()
        h = xg @ ag.t()
        ref[rows] += s * (h @ bg.t())
        size = (xg.abs() @ ag.abs().t()) @ bg.abs().t() * abs(s)
        split = {"bf16": 2.0 ** -17, "fp16": 2.0 ** -22, "fp32": 0.0}[kind]
        tol[rows] += size * (U32 * (K + 2 * rank + 16) + split)
        if kind == "fp16":
            tol[rows] += 2.0 ** -22 * abs(s) * h.abs().amax(1, keepdim=True) * bg.abs().sum(1)
    return ref, tol, has


def _run(env, x, a, b, base, scale, plan, adapters, rank, kind, stream=0, out=None):
    torch, m, types, tid = env
    M, N = x.shape[0], b.shape[0] // adapters
    wide = None
    if out is None:
        wide = torch.full((M + 1, N + 4), 77.0, dtype=types[kind], device="cuda")
        out = wide[:M, 1:1 + N]
    offsets, order = plan
    m.moe_adapt_rows(x, x.stride(0), tid[kind], M, x.shape[1], a, a.stride(0), b, b.stride(0), N, rank,
                     scale, adapters, offsets, order, base, N if base is None else base.stride(0),
                     out, out.stride(0), stream)
    return wide, out


def _check(env, wide, out, ref, tol, has, kind):
    torch, m, types, tid = env
    u = _half_ulp(torch, types[kind])
    tol = tol * (1 + u) + ref.abs() * u + (2.0 ** -25 if kind == "fp16" else 2.0 ** -126)
    ok = (out.double() - ref).abs() <= tol
    # from the largest number and half a step on, to nearest is infinity (fp16: from 65520)
    ok |= (ref.abs() + tol >= torch.finfo(types[kind]).max) & (out.double() == ref.sign() * torch.inf)
    ok[~has] = (out == 77)[~has]  # left as they were
    assert bool(ok.all()), torch.nonzero(~ok)[:4].tolist()
    if wide is not None:
        N = out.shape[1]
        assert bool((wide[-1] == 77).all()) and bool((wide[:, 0] == 77).all()) and \
            bool((wide[:, 1 + N:] == 77).all())


def _ids(torch, seed, M, adapters, none, run):
    """Adapters of rows, the same for `run` neighbours; some without one, by either kind of id."""
    g = _gen(torch, seed + 1)
    n = -(-M // run)
    ids = torch.randint(0, adapters, (n,), generator=g, device="cuda")
    r = torch.rand(n, generator=g, device="cuda")
    ids = torch.where(r < none / 2, -1, torch.where(r < none, adapters + 1, ids))
    return ids.repeat_interleave(run)[:M].to(torch.int32).contiguous()


ADAPTS = [  # M, K, N, rank, adapters, share without one, rows of a request, padding, start
    (1, 8, 8, 1, 1, 0.0, 1, 0, 0), (1, 2048, 2048, 16, 3, 0.0, 1, 0, 0),
    (8, 2048, 2048, 16, 32, 0.0, 1, 0, 0), (1003, 1000, 770, 24, 8, 0.25, 80, 3, 1),
    (100, 5, 3, 2, 4, 0.2, 3, 1, 0), (257, 129, 65, 7, 3, 0.1, 30, 0, 1),
    (64, 4096, 130, 128, 5, 0.0, 9, 0, 0), (700, 72, 200, 33, 1000, 0.1, 1, 8, 0),
    (33, 3, 70, 100, 2, 0.0, 33, 2, 3), (5000, 264, 96, 64, 4, 0.0, 700, 0, 0),
    (40, 64, 64, 8, 1, 0.5, 1, 0, 0), (90, 520, 1100, 32, 2, 0.0, 45, 8, 8),
    (3000, 96, 61, 12, 70, 0.3, 11, 0, 0), (50, 66, 300, 65, 6, 0.0, 10, 0, 1),
    (20, 40, 40, 16, 4, 1.0, 5, 0, 0),
    # long rows, few of them: one, a tile's, one more; lengths around a step of all waves
    (1, 6145, 100, 16, 1, 0.0, 1, 0, 0), (17, 4104, 1000, 3, 2, 0.0, 16, 8, 0),
    (16, 4099, 66, 24, 1, 0.0, 16, 1, 1), (300, 1088, 130, 17, 5, 0.1, 40, 0, 0),
    (70, 2049, 71, 64, 3, 0.1, 9, 0, 0), (5, 7000, 520, 40, 2, 0.0, 2, 0, 0),
    # a few more tiles than one or two for each CU, whose channels are shared out
    (8300, 40, 1100, 16, 3, 0.0, 900, 0, 0), (4000, 24, 2100, 40, 100, 0.1, 35, 3, 1),
    (16500, 16, 530, 64, 9, 0.0, 1700, 0, 0), (4112, 9, 777, 128, 1, 0.0, 4112, 0, 0)]


@pytest.mark.parametrize("M,K,N,rank,adapters,none,run,pad,at", ADAPTS)
@pytest.mark.parametrize("kind", KINDS)
def test_adapt(env, M, K, N, rank, adapters, none, run, pad, at, kind):
    torch, m, types, tid = env
    x, a, b, base, scale = _operands(env, M + K, M, K, N, rank, adapters, kind, pad, at)
    ids = _ids(torch, M, M, adapters, none, run)
    plan = _plan(env, ids, adapters)
    for add, f in ((base, scale), (None, None)):
        ref, tol, has = _ref(torch, x, a, b, add, f, ids, adapters, rank, kind)
        out = _run(env, x, a, b, add, f, plan, adapters, rank, kind)
        _check(env, *out, ref, tol, has, kind)
    # over a projection's own output: rows without an adapter keep it
    ref, tol, has = _ref(torch, x, a, b, base, scale, ids, adapters, rank, kind)
    own = base.clone()
    _, got = _run(env, x, a, b, own, scale, plan, adapters, rank, kind, out=own)
    assert torch.equal(got[~has], base[~has])
    keep = got.clone()
    keep[~has] = 77
    _check(env, None, keep, ref, tol, has, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_sorted_rows_and_one_adapter(env, kind):
    """Rows that lie sorted need no order; one adapter for all rows no offsets."""
    torch, m, types, tid = env
    M, K, N, rank, adapters = 90, 70, 50, 10, 4
    x, a, b, base, scale = _operands(env, 3, M, K, N, rank, adapters, kind)
    ids = torch.sort(_ids(torch, 5, M, adapters, 0.0, 1))[0]
    offsets, _ = _plan(env, ids, adapters)
    ref = _ref(torch, x, a, b, base, scale, ids, adapters, rank, kind)
    _check(env, *_run(env, x, a, b, base, scale, (offsets, None), adapters, rank, kind), *ref, kind)
    a, b = a[:rank], b[:N]
    ref = _ref(torch, x, a, b, base, scale[:1], ids * 0, 1, rank, kind)
    _check(env, *_run(env, x, a, b, base, scale[:1], (None, None), 1, rank, kind), *ref, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_bad_plans_stay_in_bounds(env, kind):
    """Offsets beyond the rows are cut off, places outside them left out."""
    torch, m, types, tid = env
    M, K, N, rank, adapters = 60, 40, 30, 8, 3
    x, a, b, base, scale = _operands(env, 4, M, K, N, rank, adapters, kind)
    offsets = torch.tensor([-5, 20, 10, 900], dtype=torch.int32, device="cuda")
    order = torch.arange(M, dtype=torch.int32, device="cuda")
    order[::7] = M + 100
    order[3::7] = -9
    wide, out = _run(env, x, a, b, base, scale, (offsets, order), adapters, rank, kind)
    bad = (order < 0) | (order >= M)
    assert bool((out[bad] == 77).all()) and bool((wide[-1] == 77).all())
    ids = torch.zeros(M, dtype=torch.int64, device="cuda")
    ids[10:] = 2  # of rows 10 .. 19, in two adapters, either
    ref, tol, has = _ref(torch, x, a, b, base, scale, ids, adapters, rank, kind)
    clear = ~bad
    clear[10:20] = False
    has &= clear
    got = torch.where(clear[:, None], out, 77.0)
    _check(env, None, got, ref, tol, has, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_values(env, kind):
    """A row's NaN and infinities stay in the row; an adapter's in its rows; large and small h keep
    their accuracy."""
    torch, m, types, tid = env
    M, K, N, rank, adapters = 48, 100, 72, 20, 3
    x, a, b, base, scale = _operands(env, 7, M, K, N, rank, adapters, kind)
    ids = _ids(torch, 8, M, adapters, 0.0, 1)
    x[5, 99] = float("nan")
    x[9, 0] = float("inf")
    x[11] *= 1e-4
    a[2 * rank:] = 1.5  # of adapter 2: h far beyond fp16's range, or its subnormals
    x[ids == 2] = torch.where(x[ids == 2] > 0, 1000.0, 900.0).to(types[kind])
    b[2 * N:] *= 1e-4
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[[5, 9]] = True
    clean = x.clone()
    clean[bad] = 0
    plan = _plan(env, ids, adapters)
    wide, out = _run(env, x, a, b, base, scale, plan, adapters, rank, kind)
    ref, tol, has = _ref(torch, clean, a, b, base, scale, ids, adapters, rank, kind)
    assert not bool(torch.isfinite(out[5]).any()) or int(ids[5]) == 2
    assert not bool(torch.isfinite(out[bad]).all(1).any())
    got = torch.where(bad[:, None], 77.0, out)
    big = ref.abs() > 0.999 * torch.finfo(types[kind]).max  # of fp16: rounded to infinity
    got, ref = torch.where(big, 0.0, got.double()), torch.where(big, 0.0, ref)
    _check(env, None, got, ref, tol, has & ~bad, kind)


def _whole(env, seed, M, K, N, rank, adapters, kind, pad=0):
    """Operands of small whole numbers, whose products and sums are exact in fp32 (and x A^T in the parts
    that it is split into, 16 bits at least): only the output is rounded."""
    torch, m, types, tid = env
    g = _gen(torch, seed)

    def matrix(rows, cols, most):
        wide = torch.randint(-most, most + 1, (rows, cols + pad), generator=g, device="cuda")
        return wide.to(types[kind])[:, :cols]
    scale = 2.0 ** torch.randint(-1, 2, (adapters,), generator=g, device="cuda")
    return (matrix(M, K, 2), matrix(adapters * rank, K, 1), matrix(adapters * N, rank, 1),
            matrix(M, N, 9), scale.float())


def _check_whole(env, x, a, b, base, scale, ids, adapters, rank, kind):
    torch, m, types, tid = env
    ref, _, has = _ref(torch, x, a, b, base, scale, ids, adapters, rank, kind)
    plan = _plan(env, ids, adapters)
    _, out = _run(env, x, a, b, base, scale, plan, adapters, rank, kind)
    want = torch.where(has[:, None], ref.to(types[kind]), 77.0)
    assert torch.equal(out, want), torch.nonzero(out != want)[:4].tolist()
    own = base.clone()
    _run(env, x, a, b, own, scale, plan, adapters, rank, kind, out=own)
    assert torch.equal(own, torch.where(has[:, None], ref.to(types[kind]), base))


@pytest.mark.parametrize("rank", [1, 7, 8, 16, 17, 24, 32, 40, 64, 65, 127, 128])
@pytest.mark.parametrize("kind", KINDS)
def test_every_element_counts(env, kind, rank):
    """Whole numbers, bit for bit: of rows around the steps that a wave or all of them take at a time, no
    element may be left out or taken twice."""
    torch = env[0]
    for K in (1, 7, 9, 31, 33, 64, 65, 127, 255, 257, 520, 1023, 2049, 4099, 6145, 7000):
        M, N, adapters = 19, 133, 2
        ids = _ids(torch, K, M, adapters, 0.1, 4)
        _check_whole(env, *_whole(env, K + rank, M, K, N, rank, adapters, kind, K % 3), ids, adapters,
                     rank, kind)


@pytest.mark.parametrize("tile,rows,none,K,N,rank", v.ADAPT_RESTS)
@pytest.mark.parametrize("kind", KINDS)
def test_tiles_left_over(env, kind, tile, rows, none, K, N, rank):
    """Tiles beyond a multiple of the CUs, whose channels are shared out: whole numbers, bit for bit."""
    torch = env[0]
    adapters = len(rows)
    counts = torch.tensor(rows + [none], device="cuda")
    ids = torch.repeat_interleave(torch.arange(adapters + 1, device="cuda"), counts)
    ids = ids[torch.randperm(ids.numel(), generator=_gen(torch, K), device="cuda")]
    ids = torch.where(ids == adapters, -1, ids).to(torch.int32)
    M = ids.numel()
    _check_whole(env, *_whole(env, M, M, K, N, rank, adapters, kind), ids, adapters, rank, kind)
