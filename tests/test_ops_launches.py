"""What the operators launch, and what they answer when a launch fails, seen without a GPU: the
runtime's launches are replaced (hip_stub.py)."""
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
        assert len(kernels) > 100
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
