"""What the norm, routing and adapter operators launch, and what they answer when a launch fails, seen
without a GPU: the runtime's launches are replaced (hip_stub.py)."""
import re

import pytest

import hip_stub
import more_ops_variants as v

OK, HIP = 0, -4


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    lib = hip_stub.build(tmp_path_factory.mktemp("stub"))

    def run(*wanted):
        out, kernels = hip_stub.run(lib, [[w[0], w[1], w[2] if len(w) > 2 else {}]
                                          for w in wanted])
        run.kernels = kernels
        return out
    return run


EACH = [  # a call of every operator, with its launches
    ("moe_norm_rows", v.norm_args(5, 64, "bf16"), 1),
    ("moe_norm_rows_grad", v.norm_grad_args(3, 2000, "bf16"), 1),  # one workgroup: no parts to join
    ("moe_norm_rows_grad", v.norm_grad_args(500, 64, "fp16"), 2),
    ("moe_norm_rows_grad", {**v.norm_grad_args(500, 64, "fp16"), "dweight": None}, 1),
    ("moe_norm_rows_grad", {**v.norm_grad_args(0, 64, "fp16"), "dy": None, "sum": None}, 1),
    ("moe_route_tokens", v.route_args(9, 64, 4, 1, 1, 1, "fp32"), 1),
    ("moe_route_tokens_grad", v.route_grad_args(9, 64, 4, "fp32"), 1),
    ("moe_adapt_rows", v.adapt_args(9, 64, 64, 8, 4, "bf16"), 1)]


def test_error_of_another_call_is_neither_reported_nor_taken(calls):
    for (name, args, n), r in zip(EACH, calls(*[(name, args, dict(error=1))
                                                for name, args, _ in EACH])):
        assert r["status"] == OK and len(r["launches"]) == n, (name, r)
        assert r["error"] == 1, name


def test_failed_launch_ends_the_call(calls):
    """Nothing is launched after it: the parts of a gradient that was not computed are not joined."""
    wanted = [(name, args, at) for name, args, n in EACH for at in range(1, n + 1)]
    for (name, args, at), r in zip(wanted, calls(*[(name, args, dict(launch=at))
                                                   for name, args, at in wanted])):
        assert r["status"] == HIP and len(r["launches"]) == at, (name, at, r)
        assert r["error"] == 0, name


def test_short_rows_stream_where_their_outputs_start_with_half_a_line(calls):
    """By the addresses and strides of what is written, not by the rows' length."""
    streams = "Lb1E"  # the kernels' last template argument
    codes = {"codes": None, "scale": None}
    at = dict(sum_stride=1024, y_stride=1024, codes_stride=1024)
    wanted = []
    for K in (512, 500, 1000, 1024):
        base = {**v.norm_args(1 << 18, K, "bf16"), "x": 3 * v.P, "x_stride": K + 3,
                "residual": 3 * v.P, "residual_stride": K + 3, **at}
        wanted += [(base, True), ({**base, "y_stride": 1027}, False),
                   ({**base, "sum_stride": 1027}, False),
                   ({**base, "y_stride": 1056}, True),  # 33 half lines
                   ({**base, "sum": v.P + 32}, False), ({**base, "codes_stride": 1027}, K > 512),
                   ({**base, "codes_stride": 1027, **codes}, True),
                   ({**base, "y": None, "y_stride": 1027}, True)]
    for (args, yes), r in zip(wanted, calls(*[("moe_norm_rows", args) for args, _ in wanted])):
        (kernel, *_), = r["launches"]
        assert (streams in kernel) == yes, (args, kernel)


def test_groups_that_all_stay_are_no_groups(calls):
    """The same kernel as without groups, whatever their size."""
    same = calls(("moe_route_tokens", v.route_args(9, 100, 4, 1, 1, 1, "fp32")),
                 ("moe_route_tokens", v.route_args(9, 100, 4, 10, 2, 10, "fp32")))
    assert same[0]["launches"] == same[1]["launches"]


def test_variants_reach_every_kernel(calls):
    wanted = []
    for kind in v.KINDS:
        for M, K in v.norms(kind):
            wanted.append(("moe_norm_rows", v.norm_args(M, K, kind)))
            wanted.append(("moe_norm_rows_grad", v.norm_grad_args(M, K, kind)))
        for case in v.ROUTES:
            wanted.append(("moe_route_tokens", v.route_args(*case, kind)))
            wanted.append(("moe_route_tokens_grad", v.route_grad_args(*case[:3], kind)))
        for case in v.adapts(kind):
            wanted.append(("moe_adapt_rows", v.adapt_args(*case, kind)))
    reached = set()
    for (name, args), r in zip(wanted, calls(*wanted)):
        assert r["status"] == OK, (name, args)
        for kernel, x, y, threads, lds in r["launches"]:
            reached.add(kernel)
            assert 0 < x * threads < 1 << 32 and 0 < y < 1 << 16 and lds <= 1 << 16
    kernels = {k for k in calls.kernels if re.search(r"\d(norm_rows|route_tokens|adapt_rows)_", k)}
    assert len(kernels) > 90
    missed = sorted(kernels - reached)
    assert not missed, (len(missed), missed)


def test_adapters_tiles_left_over(calls):
    """Those cases have one workgroup for all channels of a tile, tiles left over beside those that every
    CU has had, and workgroups for the parts that they are shared out into."""
    wanted = []
    for kind in v.KINDS:
        for tile, rows, none, K, N, rank in v.ADAPT_RESTS:
            M = sum(rows) + none
            wanted.append((tile, rows, M, N, v.adapt_args(M, K, N, rank, len(rows), kind)))
    reached = set()
    for (tile, rows, M, N, args), r in zip(wanted, calls(*[("moe_adapt_rows", w[4])
                                                           for w in wanted])):
        (kernel, x, y, threads, _), = r["launches"]
        RT, MT, UC, W = map(int, re.search(r"Li(\d)ELi(\d)ELi(\d)ELi(\d)E", kernel).groups())
        reached.add((RT, MT, W))
        total = sum(-(-n // tile) for n in rows)
        rest = total % 256
        assert tile == 16 * MT and y == 1 and total > 256 and 1 <= rest <= 128 and N >= 512, args
        parts = min(256 // rest, N // 256)
        # eight dies: whole rounds of them, and every part of a tile on one of them
        assert parts > 1 and x >= total - rest + -(-rest // 8) * 8 * parts, args
    assert reached == {(1, 1, 4), (1, 1, 8), (2, 1, 4), (2, 1, 8), (2, 2, 4), (4, 1, 4), (4, 1, 8),
                       (4, 2, 4), (8, 1, 4)}
