"""What the operators launch, and what they answer when a launch fails, seen without a GPU: the
runtime's launches are replaced (hip_stub.py)."""
import re

import pytest

import hip_stub

BF16, FP16, FP32, I8 = 0, 1, 2, 3
P = 1 << 20  # an address
OK, INVALID, HIP, SCRATCH = 0, -1, -4, -7

SORT = dict(topk_idx=P, T=16, top_k=2, experts=8, offsets=P, order=P, place=P, x=P, x_stride=64,
            hidden=64, x_type=BF16, rows=P, rows_stride=64, rows_type=BF16, row_scale=P,
            workspace=P, workspace_bytes=1 << 40, stream=0)


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    lib = hip_stub.build(tmp_path_factory.mktemp("stub"))

    def run(*wanted):
        """Each wanted call as (name, arguments[, settings])."""
        out, kernels = hip_stub.run(lib, [[w[0], w[1], w[2] if len(w) > 2 else {}]
                                          for w in wanted])
        run.kernels = kernels
        return out
    return run


def test_sort_of_no_tokens_writes_offsets(calls):
    """One launch, whichever of the two matrices is an empty buffer (which has no address)."""
    none = dict(T=0, topk_idx=None, place=None)
    for r in calls(*[("moe_sort_tokens", {**SORT, **none, **kw}) for kw in (
            {}, dict(x=None), dict(rows=None), dict(x=None, rows=None),
            dict(x=None, rows_type=I8, row_scale=None))]):
        assert r["status"] == OK and len(r["launches"]) == 1
        assert "sort_small_kernel" in r["launches"][0][0] and r["launches"][0][1] == 1
    refused = calls(("moe_sort_tokens", {**SORT, "x": None}),
                    ("moe_sort_tokens", {**SORT, "rows": None}),
                    ("moe_sort_tokens", {**SORT, **none, "offsets": None}),
                    ("moe_sort_tokens", {**SORT, **none, "x": None, "x_type": I8}))
    assert all(r["status"] == INVALID and not r["launches"] for r in refused)


COMBINE = dict(rows=P, rows_stride=64, n_rows=32, type=BF16, place=P, weights=P, T=16, top_k=2,
               hidden=64, out=P, out_stride=64, stream=0)
PRODUCT = dict(a=P, a_stride=64, a_scale=P, M=16, K=64, w=P, w_stride=64, w_scale=P, N=32,
               groups=4, offsets=P, epilogue=0, out=P, out_stride=32, out_type=BF16, stream=0)
EACH = [  # a call of every operator, of the sort one for each number of launches
    ("moe_sort_tokens", SORT, 1), ("moe_sort_tokens", {**SORT, "T": 4096}, 2),
    ("moe_sort_tokens", {**SORT, "T": 40000}, 3),
    ("moe_sort_tokens_grad", dict(drows=P, drows_stride=64, n_rows=32, type=FP16, place=P, T=16,
                                  top_k=2, hidden=64, dx=P, dx_stride=64, stream=0), 1),
    ("moe_combine_tokens", COMBINE, 1),
    ("moe_combine_tokens_grad", dict(dout=P, dout_stride=64, rows=P, rows_stride=64, n_rows=32,
                                     type=FP32, place=P, weights=P, T=16, top_k=2, hidden=64,
                                     drows=P, drows_stride=64, dweights=P, stream=0), 1),
    ("moe_quantise_rows", dict(x=P, x_stride=64, type=BF16, M=16, K=64, codes=P, codes_stride=64,
                               scale=P, rows_end=None, stream=0), 1),
    ("moe_product_i8", PRODUCT, 1), ("moe_product_i8", {**PRODUCT, "M": 5000, "N": 4096,
                                                        "out_stride": 4096}, 1)]


def test_error_of_another_call_is_neither_reported_nor_taken(calls):
    for (name, args, n), r in zip(EACH, calls(*[(name, args, dict(error=1))
                                                for name, args, _ in EACH])):
        assert r["status"] == OK and len(r["launches"]) == n, (name, r)
        assert r["error"] == 1, name


def test_failed_launch_ends_the_call(calls):
    """Nothing is launched after it: the sort's later kernels would take whatever the workspace
    holds as counts."""
    wanted = [(name, args, at) for name, args, n in EACH for at in range(1, n + 1)]
    for (name, args, at), r in zip(wanted, calls(*[(name, args, dict(launch=at))
                                                   for name, args, at in wanted])):
        assert r["status"] == HIP and len(r["launches"]) == at, (name, at, r)
        assert r["error"] == 0, name  # reported, so no later call finds it


def test_lds_limit_of_a_kernel_is_one_for_all_calls(calls):
    """The limit belongs to the kernel, whichever thread sets it: every call on a device needs at
    most what the first has set, and a limit that cannot be set ends the call before its launch."""
    big = {**PRODUCT, "M": 2_000_000, "N": 4096, "K": 2048, "a_stride": 2048, "w_stride": 2048,
           "out_stride": 4096}
    odd = {**big, "a_stride": 2049}
    wanted = []
    for args in (big, odd):
        wanted += [("moe_product_i8", args, dict(attribute=1)), ("moe_product_i8", args),
                   ("moe_product_i8", {**args, "groups": 500}), ("moe_product_i8", args),
                   ("moe_product_i8", args, dict(device=1)),
                   ("moe_product_i8", args, dict(device=1))]
    out = calls(*wanted)
    limit = {}
    for (_, args, *setting), r in zip(wanted, out):
        setting = setting[0] if setting else {}
        if setting.get("attribute"):
            assert r["status"] == HIP and not r["launches"] and r["error"] == 0
            continue
        assert r["status"] == OK and len(r["launches"]) == 1
        kernel, lds = r["launches"][0][0], r["launches"][0][4]
        assert "product_tile_kernel" in kernel and lds > 1 << 16
        key = kernel, setting.get("device", 0)
        for name, value in r["attributes"]:
            assert name == kernel and key not in limit
            limit[key] = value
        assert lds <= limit[key]
    assert len(limit) == 4  # one kernel for each of the two, whatever the groups, on two devices
    assert len(set(limit.values())) == 2


def _variant_calls():
    """Every case of ops_variants as a call, with the tile it is there for."""
    import ops_variants as v
    for tile, per_gpu, any_, counts, N, K, pad, at in v.TILES:
        for kind in v.KINDS:
            for swiglu in (False, True):
                yield "moe_product_i8", v.product_args(counts, N, K, pad, at, kind, swiglu), \
                    (tile, per_gpu, any_, counts, N)
    for counts, N, K, pad, at in v.FEW:
        for kind in v.KINDS:
            for swiglu in (False, True):
                yield "moe_product_i8", v.product_args(counts, N, K, pad, at, kind, swiglu), None
    for kind in v.KINDS:
        for T, k, E, _, H, pad, at in v.SORTS:
            for rows in (kind, "i8"):
                yield "moe_sort_tokens", v.sort_args(T, k, E, H, pad, at, kind, rows), None
        T, k, E, _, H, pad, at = v.SORTS_SHORT_STREAMED[kind == "fp32"]
        yield "moe_sort_tokens", v.sort_args(T, k, E, H, pad, at, kind, kind), None
        for T, k, _, H, pad, at in v.COMBINES:
            args = v.combine_args(T, k, H, pad, at, kind)
            yield "moe_combine_tokens", args, None
            yield "moe_sort_tokens_grad", dict(
                drows=args["rows"], drows_stride=args["rows_stride"], n_rows=args["n_rows"],
                type=args["type"], place=P, T=T, top_k=k, hidden=H, dx=P, dx_stride=H), None
            yield "moe_combine_tokens_grad", dict(
                dout=P, dout_stride=H, rows=args["rows"], rows_stride=args["rows_stride"],
                n_rows=args["n_rows"], type=args["type"], place=P, weights=P, T=T, top_k=k,
                hidden=H, drows=P, drows_stride=H, dweights=P), None
        for M, K in v.quantises(kind):
            yield "moe_quantise_rows", v.quantise_args(M, K, kind), None


def test_variants_reach_every_kernel(calls):
    """The cases that the GPU tests run launch every kernel of the operators, and every tile kernel
    with more tiles than workgroups, so that a workgroup goes on to a second tile."""
    wanted = list(_variant_calls())
    out = calls(*[(name, args) for name, args, _ in wanted])
    reached, second = set(), set()
    for (name, args, tile), r in zip(wanted, out):
        assert r["status"] == OK, (name, args)
        reached |= {launch[0] for launch in r["launches"]}
        if tile is None:
            continue
        (rows, channels, sets), per_gpu, any_, counts, N = tile
        kernel, grid = r["launches"][0][:2]
        shape = re.search(r"product_tile_kernelI.*Lb[01]ELb([01])ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)"
                          r"ELi(\d+)ELi(\d+)EEE", kernel)
        assert shape, (kernel, args)
        free, wm, wn, mi, ni, ks, per_cu = map(int, shape.groups())
        assert (32 * wm * mi, 32 * wn * ni, ks, 256 * per_cu, bool(free)) == (
            rows, channels, sets, per_gpu, any_), args
        groups = [counts] if isinstance(counts, int) else counts
        tiles = sum(-(-c // rows) for c in groups) * -(-N // channels)
        assert tiles > grid == per_gpu, (args, tiles, grid)
        second.add(kernel)
    kernels = {k for k in calls.kernels if re.search(r"\d(sort|combine|quantise|product)_", k)
               and not k.endswith("7FfnArgsE")}  # the layer step's own combine
    assert len(kernels) > 100
    assert {k for k in kernels if "product_tile_kernel" in k} == second
    missed = sorted(kernels - reached)
    assert not missed, (len(missed), missed)
