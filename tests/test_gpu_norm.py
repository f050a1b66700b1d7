"""The norm of rows with the residual's addition, rounded and in 8 bits, and its gradient, against
plain implementations in 64 bits.

Codes and the rounded sum are compared exactly.  Tolerances count roundings: a value rounded to
type t is off by at most eps_t / 2 relative to it, U32 = 2^-24 a rounding in fp32."""
import pytest

from test_gpu_ops import KINDS, U32, _gen, _half_ulp, _matrix, env  # noqa: F401

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _sum(torch, x, r):
    """x + r rounded once: the sum of two numbers of these types is exact in 64 bits up to a rounding
    far below theirs, except that fp32's own sum rounds the same way in 32."""
    if x.dtype == torch.float32:
        return x + r
    return (x.double() + r.double()).to(x.dtype)


def _codes(torch, h, w):
    p = h.double() * w.double()
    m = p.abs().amax(1, keepdim=True)
    bad = ~torch.isfinite(m)
    codes = torch.round(127 * p / torch.where(m > 0, m, 1.0))
    return torch.where(bad, 0.0, codes).to(torch.int8), torch.where(bad, torch.nan, m)[:, 0]


def _wide(torch, rows, cols, kind):
    """Outputs between marks: a buffer, and its middle columns."""
    wide = torch.full((rows + 1, cols + 4), 77, dtype=kind, device="cuda")
    return wide, wide[:rows, 1:1 + cols]


def _untouched(wide, rows, cols):
    w = wide.double()
    return bool((w[rows:] == 77).all()) and bool((w[:, 0] == 77).all()) and \
        bool((w[:, 1 + cols:] == 77).all())


def _run(env, x, r, w, kind, want=("sum", "y", "codes"), eps=EPS, stream=0):
    torch, m, types, tid = env
    M, K = x.shape
    o = {}
    for name in ("sum", "y", "codes"):
        o[name] = _wide(torch, M, K, torch.int8 if name == "codes" else types[kind]) \
            if name in want and (name != "sum" or r is not None) else (None, None)
    o["scale"] = torch.full((M + 1,), 77.0, device="cuda") if "codes" in want else None
    m.moe_norm_rows(x, x.stride(0), r, 0 if r is None else r.stride(0), tid[kind], M, K, w, eps,
                    o["sum"][1], K + 4, o["y"][1], K + 4, o["codes"][1], K + 4, o["scale"], stream)
    return o


def _check(env, x, r, w, kind, o, eps=EPS):
    torch, m, types, tid = env
    M, K = x.shape
    u = _half_ulp(torch, types[kind])
    h = x if r is None else _sum(torch, x, r)
    q = (h.double().square().mean(1, keepdim=True) + eps).rsqrt()
    wide, got = o["sum"]
    if got is not None:
        assert torch.equal(got.nan_to_num(5.0), h.nan_to_num(5.0))
        assert _untouched(wide, M, K)
    wide, got = o["y"]
    if got is not None:
        ref = h.double() * q * w.double()
        # the factor and two products in fp32, then the output's own rounding (fp16's subnormal step);
        # 16-bit rows add up eight squares at a time in fp32, four additions in sequence of two exact
        # products each: 2^-22 of the sum, half of that of its root
        tol = ref.abs() * (u + 6 * U32) + (2.0 ** -25 if kind == "fp16" else 2.0 ** -126)
        ok = (got.double() - ref).abs() <= tol
        ok |= torch.isnan(ref) & torch.isnan(got)
        assert bool(ok.all()), torch.nonzero(~ok)[:4].tolist()
        assert _untouched(wide, M, K)
    wide, got = o["codes"]
    if got is not None:
        codes, big = _codes(torch, h, w)
        assert torch.equal(got, codes), torch.nonzero(got != codes)[:4].tolist()
        assert _untouched(wide, M, K)
        ref = big * q[:, 0] / 127
        # 64 bits rounded once, and the sum's 2 U32 as above
        torch.testing.assert_close(o["scale"][:M].double(), ref, rtol=4 * U32, atol=2.0 ** -149,
                                   equal_nan=True)
        assert float(o["scale"][M]) == 77


NORMS = [  # M, K, padding, start
    (1, 1, 0, 0), (3, 7, 2, 1), (5, 8, 0, 0), (1, 2048, 0, 0), (4, 6144, 0, 0), (777, 1000, 3, 1),
    (130, 513, 0, 0), (2, 16384, 0, 0), (33, 4097, 1, 3), (65, 257, 8, 0), (40, 65, 0, 5),
    (3, 8193, 0, 0), (9000, 72, 8, 0), (12, 2049, 0, 0), (40000, 33, 0, 1)]


@pytest.mark.parametrize("M,K,pad,at", NORMS)
@pytest.mark.parametrize("kind", KINDS)
def test_norm(env, M, K, pad, at, kind):
    torch, m, types, tid = env
    g = _gen(torch, M + K)
    x, r = (_matrix(torch, g, M, K, types[kind], pad, at) for _ in "xr")
    w = (1 + 0.5 * torch.randn(K, generator=g, device="cuda")).to(types[kind])
    _check(env, x, r, w, kind, _run(env, x, r, w, kind))
    _check(env, x, None, w, kind, _run(env, x, None, w, kind))
    for want in (("y",), ("codes",), ("sum", "codes")):
        _check(env, x, r, w, kind, _run(env, x, r, w, kind, want))


@pytest.mark.parametrize("kind", KINDS)
def test_norm_values(env, kind):
    """Zeros, tiny and huge rows and weights, ties of codes, infinities and NaN."""
    torch, m, types, tid = env
    g = _gen(torch, 9)
    K, t = 300, types[kind]
    big = torch.finfo(t).max
    x = torch.randn(64, K, generator=g, device="cuda").double()
    x[1] = 0
    x[2] *= 1e-30
    x[3] = torch.arange(K, device="cuda") / 2.0 - 63.5
    x[3, 0] = 127
    x[4, 17] = float("inf")
    x[5, K - 1] = float("nan")
    x[6] = 0
    x[6, K - 1] = -torch.finfo(t).smallest_normal / 8
    x[7] = big
    x[8] = torch.linspace(-1, 1, K, device="cuda") * big
    x[9, 0] = -float("inf")
    x[10:40] = torch.round(x[10:40] * 16) / 16
    x[40:44] *= 1e18
    x[44:48] *= 1e-18
    odd = torch.arange(-127, 128, 2, device="cuda").double() / 254
    x[48:56, :128] = odd * torch.randint(1, 1 << 20, (8, 1), generator=g, device="cuda")
    x[48:56, 128:] = x[48:56, :1] * 2
    x = x.to(t)
    ws = [torch.ones(K, device="cuda"), torch.randn(K, generator=g, device="cuda"),
          torch.randn(K, generator=g, device="cuda") * 1e-25,
          torch.randn(K, generator=g, device="cuda") * 1e25]
    ws[1][::3] = 0
    for w in ws:
        w = w.to(t)
        o = _run(env, x, None, w, kind, ("codes",))
        _check(env, x, None, w, kind, o)
    w = ws[0].to(t)
    keep = [i for i in range(64) if i not in (4, 9)]  # an infinite row is 0 but for its infinities
    o = _run(env, x[keep].contiguous(), None, w, kind)
    _check(env, x[keep].contiguous(), None, w, kind, o)


@pytest.mark.parametrize("kind", KINDS)
def test_norm_subnormals(env, kind):
    """Rows whose sum of squares is made of subnormal numbers."""
    torch, m, types, tid = env
    K, t = 512, types[kind]
    tiny = torch.finfo(t).smallest_normal
    g = _gen(torch, 3)
    x = torch.full((6, K), tiny / 2, dtype=torch.float64, device="cuda")
    x[1, 5] = tiny
    x[2] = tiny * torch.rand(K, generator=g, device="cuda")
    x[3, ::2] = -tiny * 2
    x[4, 0] = tiny * 64
    x[5] /= 4
    x = x.to(t)
    w = torch.ones(K, device="cuda", dtype=t)
    for eps in (1e-30, 1e-6):
        _check(env, x, None, w, kind, _run(env, x, None, w, kind, eps=eps), eps)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,K", [(5, 1001), (70, 72), (3, 9001), (9, 5), (300, 2048)])
def test_norm_in_place(env, kind, M, K):
    """The sum written over the residual or x, y over the other: what streaming layers do."""
    torch, m, types, tid = env
    g = _gen(torch, K)
    x, r = (torch.randn(M, K, generator=g, device="cuda").to(types[kind]) for _ in "xr")
    w = torch.rand(K, generator=g, device="cuda").to(types[kind])
    ref = _run(env, x, r, w, kind)
    for first in (True, False):
        a, b = x.clone(), r.clone()
        total, y = (a, b) if first else (b, a)
        m.moe_norm_rows(a, K, b, K, tid[kind], M, K, w, EPS, total, K, y, K)
        assert torch.equal(total, ref["sum"][1]) and torch.equal(y, ref["y"][1])
    a = x.clone()
    m.moe_norm_rows(a, K, None, 0, tid[kind], M, K, w, EPS, None, 0, a, K)
    assert torch.equal(a, _run(env, x, None, w, kind)["y"][1])


def _grad_ref(torch, dy, dsum, h, w, eps=EPS):
    """dx, dweight, and the magnitudes that their roundings are relative to."""
    dy, h, w = dy.double(), h.double(), w.double()
    q = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    along = (w * dy * h).mean(1, keepdim=True)
    dx = q * w * dy - h * q ** 3 * along
    mag = (q * w * dy).abs() + (h * q ** 3).abs() * (w * dy * h).abs().mean(1, keepdim=True)
    if dsum is not None:
        dx = dx + dsum.double()
        mag = mag + dsum.double().abs()
    n = q * dy * h
    return dx, mag, n.sum(0), n.abs().sum(0)


def _run_grad(env, dy, dsum, h, w, kind, want=("dx", "dweight"), stream=0, eps=EPS):
    torch, m, types, tid = env
    M, K = dy.shape
    wide, dx = _wide(torch, M, K, types[kind]) if "dx" in want else (None, None)
    dw = torch.full((K + 1,), 77.0, device="cuda") if "dweight" in want else None
    size = m.moe_norm_grad_workspace_bytes(M, K)
    ws = torch.full((size + 64,), 0x5a, dtype=torch.uint8, device="cuda")
    m.moe_norm_rows_grad(dy, dy.stride(0), dsum, 0 if dsum is None else dsum.stride(0), h,
                         h.stride(0), tid[kind], M, K, w, eps, dx, K + 4, dw, ws, size, stream)
    assert bool((ws[size:] == 0x5a).all())
    return wide, dx, dw


def _check_grad(env, dy, dsum, h, w, kind, out, eps=EPS):
    torch, m, types, tid = env
    M, K = dy.shape
    u = _half_ulp(torch, types[kind])
    dx, mag, dw, dw_mag = _grad_ref(torch, dy, dsum, h, w, eps)
    wide, got, got_w = out
    if got is not None:
        # the factors, their products and sums in fp32 (six roundings on the way to any term), then
        # the output's own rounding
        tol = dx.abs() * u + mag * (8 * U32) + (2.0 ** -25 if kind == "fp16" else 2.0 ** -126)
        ok = (got.double() - dx).abs() <= tol
        assert bool(ok.all()), torch.nonzero(~ok)[:4].tolist()
        assert _untouched(wide, M, K)
    if got_w is not None:
        # the term's three roundings, and fp32 additions over the rows that a lane and then a
        # workgroup adds up (of M rows over at least min(M, 256) workgroups), at last its own
        tol = dw_mag * U32 * (8 + 16 + M / 256) + 2.0 ** -126
        ok = (got_w[:K].double() - dw).abs() <= tol
        assert bool(ok.all()), torch.nonzero(~ok)[:4].tolist()
        assert float(got_w[K]) == 77


@pytest.mark.parametrize("M,K,pad,at", NORMS)
@pytest.mark.parametrize("kind", KINDS)
def test_norm_grad(env, M, K, pad, at, kind):
    torch, m, types, tid = env
    g = _gen(torch, M * 3 + K)
    dy, dsum, h = (_matrix(torch, g, M, K, types[kind], pad, at) for _ in "abc")
    w = (1 + 0.5 * torch.randn(K, generator=g, device="cuda")).to(types[kind])
    _check_grad(env, dy, dsum, h, w, kind, _run_grad(env, dy, dsum, h, w, kind))
    for want in (("dx",), ("dweight",), ("dx", "dweight")):
        _check_grad(env, dy, None, h, w, kind, _run_grad(env, dy, None, h, w, kind, want))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [5, 72, 1001, 9001])
def test_norm_grad_in_place_and_repeated(env, kind, K):
    """dx over dy or dsum; the same bits on every run; zeros for no rows."""
    torch, m, types, tid = env
    M = 300
    g = _gen(torch, K)
    dy, dsum, h = (torch.randn(M, K, generator=g, device="cuda").to(types[kind]) for _ in "abc")
    w = torch.rand(K, generator=g, device="cuda").to(types[kind])
    _, ref, ref_w = _run_grad(env, dy, dsum, h, w, kind)
    size = m.moe_norm_grad_workspace_bytes(M, K)
    ws = torch.empty(size + 16, dtype=torch.uint8, device="cuda")
    for first in (True, False):
        a, b = dy.clone(), dsum.clone()
        dx, dw = (a if first else b), torch.empty(K, device="cuda")
        m.moe_norm_rows_grad(a, K, b, K, h, K, tid[kind], M, K, w, EPS, dx, K, dw, ws, size)
        assert torch.equal(dx, ref) and torch.equal(dw, ref_w[:K])
    m.moe_norm_rows_grad(None, K, None, 0, None, K, tid[kind], 0, K, None, EPS, None, K, dw)
    assert not bool(dw.any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,K", [(1, 3), (300, 5), (5000, 72), (3000, 700), (2500, 2001), (900, 9001),
                                 (600, 16384)])
def test_norm_grad_over_the_sum(env, kind, M, K):
    """dx over the rows that were normalised."""
    torch, m, types, tid = env
    g = _gen(torch, K + M)
    dy, dsum, h = (torch.randn(M, K, generator=g, device="cuda").to(types[kind]) for _ in "abc")
    w = torch.rand(K, generator=g, device="cuda").to(types[kind])
    _, ref, ref_w = _run_grad(env, dy, dsum, h, w, kind)
    size = m.moe_norm_grad_workspace_bytes(M, K)
    ws, dw = torch.empty(size + 16, dtype=torch.uint8, device="cuda"), torch.empty(K, device="cuda")
    m.moe_norm_rows_grad(dy, K, dsum, K, h, K, tid[kind], M, K, w, EPS, h, K, dw, ws, size)
    assert torch.equal(h, ref) and torch.equal(dw, ref_w[:K])


def test_norm_grad_of_the_most_rows(env):
    """The weight's gradient is as exact over many rows as over few: 2^24 - 1 equal terms, which an
    addition in fp32 rounds to the same side each time once some hundreds are summed.  The
    roundings of 256 additions one after the other, those of 16 such sums, the term's own three and
    the result's, however many rows there are."""
    torch, m, types, tid = env
    M, K = (1 << 24) - 1, 3
    term = 1 + 2.0 ** -14 - 2.0 ** -20
    dy, h = torch.full((M, K), term, device="cuda"), torch.ones(M, K, device="cuda")
    w = torch.ones(K, device="cuda")
    size = m.moe_norm_grad_workspace_bytes(M, K)
    ws, dw = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.zeros(K, device="cuda")
    m.moe_norm_rows_grad(dy, K, None, 0, h, K, tid["fp32"], M, K, w, 1e-30, None, K, dw, ws, size)
    off = (dw.double() / (M * term) - 1).abs()
    assert bool((off <= U32 * (256 + 16 + 3 + 1)).all()), off


def test_norm_grad_of_far_rows(env):
    """Rows, and an eps, so small or large that the factor's cube leaves fp32's range."""
    torch, m, types, tid = env
    g = _gen(torch, 12)
    M, K = 8, 300
    dy, h = (torch.randn(M, K, generator=g, device="cuda") for _ in "ab")
    w = torch.rand(K, generator=g, device="cuda")
    h *= torch.tensor([1e-19, 1e-17, 1e-10, 1e-3, 1, 1e5, 1e10, 1e15], device="cuda")[:, None]
    for eps in (1e-37, 1e-6, 1e6):
        _check_grad(env, dy, None, h, w, "fp32", _run_grad(env, dy, None, h, w, "fp32", eps=eps),
                    eps)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("K", [3, 300, 700, 2000, 4097, 16384])
def test_norm_grad_of_far_products(env, kind, K):
    """Rows, gradients and weights whose products leave fp32's range though dx does not: too large, too
    small, all of them lost, some of a row's; and a row without a gradient, which has none."""
    torch, m, types, tid = env
    g = _gen(torch, K)
    #        h     dy
    rows = [(1e20, 1e20), (1e25, 1e14), (1e30, 1e30), (1e-20, 1e-25), (1e-25, 1e-20), (1e-30, 1e-10),
            (1e-12, 1e-33), (1e37, 1e37), (1, 1e-37), (1e-12, 1e-25), (1, 1), (1e-3, 0), (1e5, 0)]
    M = len(rows)
    h, dy = (torch.randn(M, K, generator=g, device="cuda").double() for _ in "ab")
    size = torch.tensor(rows, dtype=torch.float64, device="cuda")
    h, dy = h * size[:, :1], dy * size[:, 1:]
    h[10, 0], dy[10, 0] = 1e20, 1e20  # one term of a row alone
    dsum = torch.randn(M, K, generator=g, device="cuda").to(types[kind])
    h, dy = h.to(types[kind]), dy.to(types[kind])
    for scale in (1.0, 1e12, 1e-20):
        w = (scale * (0.5 + torch.rand(K, generator=g, device="cuda"))).to(types[kind])
        for eps in (1e-6, 1e-37):
            # rows whose dx is a number of the type
            ref = _grad_ref(torch, dy, None, h, w, eps)[0]
            keep = torch.nonzero(ref.abs().amax(1) < torch.finfo(types[kind]).max / 4)[:, 0]
            assert keep.numel() > 6
            args = [t[keep].contiguous() for t in (dy, dsum, h)]
            _check_grad(env, *args, w, kind, _run_grad(env, *args, w, kind, eps=eps), eps)
            args[1] = None
            out = _run_grad(env, *args, w, kind, eps=eps)
            _check_grad(env, *args, w, kind, out, eps)
            assert not bool(out[1][(args[0] == 0).all(1)].any())


def test_norm_grad_against_differences(env):
    """fp32: the directional derivative of a weighted sum of y, and of the sum's own way."""
    torch, m, types, tid = env
    M, K = 6, 700
    g = _gen(torch, 2)
    x, r, dy, dsum, vx = (torch.randn(M, K, generator=g, device="cuda") for _ in "abcde")
    w, vw = (torch.rand(K, generator=g, device="cuda") + 0.5 for _ in "ab")

    def loss(step):
        h = (x + r).double() + step * vx.double()
        y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * (w + step * vw.double())
        return ((y * dy).sum() + (h * dsum).sum()).item()

    e = 1e-4
    slope = (loss(e) - loss(-e)) / (2 * e)
    _, dx, dw = _run_grad(env, dy, dsum, x + r, w, "fp32")
    got = ((dx.double() * vx).sum() + (dw[:K].double() * vw).sum()).item()
    # differences: the third derivative's e^2, of terms of order M K; sums of order sqrt(M K)
    assert abs(got - slope) < 1e-4 * (M * K) ** 0.5, (got, slope)
