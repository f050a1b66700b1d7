"""Cases that between them launch every kernel of the operators, and each tile kernel of the 8-bit
product with more tiles than workgroups.  test_ops_launches.py shows that they do (without a GPU),
test_gpu_ops_variants.py that the results are right."""

KINDS = ["bf16", "fp16", "fp32"]
TYPE = {"bf16": 0, "fp16": 1, "fp32": 2, "i8": 3}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "i8": 1}
P = 1 << 20  # an address, where nothing is launched

# ------------------------------------------------------------------ 8-bit product

_WEIGHTS = (4, 3, 5, 0, 6, 2, 7, 1)


def even(groups, rows):
    return [rows // groups] * groups


def ragged(groups, rows):
    """Unequal counts, some of them zero, that add up to about `rows`."""
    return [rows * _WEIGHTS[g % 8] * 2 // (7 * groups) for g in range(groups)]


# Tile (rows, channels, sets of waves over K), its workgroups on the GPU at most, whether operands of
# any alignment; rows of each group (a number: one weight); N, K, padding and start of the rows.  Each
# tile with one, an even and an odd number of rounds of its stages.
_256, _320, _128 = (256, 256, 1), (256, 320, 1), (128, 128, 1)
_64, _64x2, _64x4 = (64, 64, 1), (64, 64, 2), (64, 64, 4)
TILES = [
    (_256, 256, False, ragged(60, 10431), 1680, 16, 0, 0),
    (_256, 256, False, ragged(16, 3006), 6180, 144, 0, 0),
    (_256, 256, False, ragged(8, 50086), 392, 288, 16, 0),
    (_320, 256, False, ragged(60, 10965), 2206, 16, 0, 0),
    (_320, 256, False, ragged(9, 2747), 9938, 144, 16, 16),
    (_320, 256, False, ragged(9, 28158), 1036, 272, 0, 0),
    (_320, 256, False, 53935, 524, 16, 0, 0),
    (_128, 512, False, ragged(700, 44466), 66, 16, 0, 0),
    (_128, 512, False, ragged(700, 43761), 70, 144, 0, 0),
    (_128, 512, False, ragged(700, 47783), 72, 272, 0, 16),
    (_128, 512, True, ragged(700, 46600), 66, 1, 0, 0),
    (_128, 512, True, ragged(700, 53769), 68, 133, 3, 1),
    (_128, 512, True, ragged(700, 45205), 78, 258, 0, 0),
    (_128, 512, True, 43784, 136, 200, 1, 0),
    (_64, 1024, False, ragged(700, 2463), 66, 16, 0, 0),
    (_64, 1024, False, ragged(700, 2867), 72, 144, 0, 0),
    (_64, 1024, False, ragged(700, 3723), 66, 272, 0, 0),
    (_64, 1024, True, ragged(1000, 1174), 68, 1, 0, 0),
    (_64, 1024, True, ragged(700, 2834), 66, 134, 0, 3),
    (_64, 1024, True, ragged(700, 2908), 66, 273, 0, 0),
    (_64x2, 512, False, even(300, 22133), 36, 144, 0, 0),
    (_64x2, 512, False, ragged(2, 156), 9320, 432, 0, 0),
    (_64x2, 512, False, even(8, 533), 2450, 528, 0, 0),
    (_64x2, 512, True, ragged(2, 153), 9046, 194, 0, 0),
    (_64x2, 512, True, even(60, 4038), 284, 410, 0, 1),
    (_64x2, 512, True, even(60, 4421), 292, 525, 0, 0),
    (_64x4, 256, False, even(9, 651), 1078, 320, 0, 0),
    (_64x4, 256, False, even(8, 550), 1200, 800, 0, 0),
    (_64x4, 256, False, even(9, 608), 1104, 1472, 0, 0),
    (_64x4, 256, True, even(9, 592), 1052, 372, 0, 0),
    (_64x4, 256, True, even(9, 611), 1152, 904, 5, 0),
    (_64x4, 256, True, ragged(2, 160), 4506, 1350, 0, 0),
]
FEW = [(7, 130, 96, 0, 0), ([0, 3, 0, 1, 16, 17, 0], 130, 200, 0, 0), (40, 66, 333, 0, 1)]
BEFORE, BEHIND = 2, 3  # rows of no group


def product_args(counts, N, K, pad, at, kind, swiglu):
    groups = 1 if isinstance(counts, int) else len(counts)
    M = counts if isinstance(counts, int) else BEFORE + sum(counts) + BEHIND
    n_out = N // 2 if swiglu else N
    stride = K + pad + at
    return dict(a=P + at, a_stride=stride, a_scale=P, M=M, K=K, w=P + at, w_stride=stride,
                w_scale=P, N=N, groups=groups, offsets=None if groups == 1 else P,
                epilogue=int(swiglu), out=P, out_stride=n_out, out_type=TYPE[kind])


# ------------------------------------------------------------------ tokens

# T, top_k, experts, share dropped, hidden, padding and start of the rows; without a hidden size the
# integers alone.
SORTS = [
    (4, 8, 256, 0.0, 96, 0, 0), (30, 5, 9, 0.2, 3, 0, 1),           # one launch
    (2100, 4, 60, 0.1, 72, 0, 0), (1000, 6, 60, 0.1, 72, 1, 3),     # counts added up by the last one,
    (2100, 4, 60, 0.1, 2500, 0, 1),                                 # rows wider than a wave holds,
    (2100, 4, 60, 0.1, 3, 0, 0), (1000, 6, 60, 0.1, 3, 1, 0),       # rows below 16 bytes
    (40000, 1, 3, 0.3, 33, 0, 0), (2000, 16, 1000, 0.1, 40, 0, 0),  # with a launch between
    (2100, 8, 60, 0.0, 2500, 3, 1), (40000, 1, 3, 0.0, 3, 0, 0), (2000, 16, 1000, 0.0, 3, 0, 0),
    (20011, 8, 128, 0.0, 845, 0, 1), (2000, 16, 300, 0.0, 4203, 1, 0),  # rows above 128 MiB
]
SORTS_SHORT_STREAMED = [(1 << 20, 11, 5, 0.0, 7, 0, 0), (1 << 20, 11, 5, 0.0, 3, 0, 0)]
SORTS_INTEGERS = [(1 << 20, 1, 1000, 0.1), (1 << 20, 2, 7, 0.0), (1 << 20, 16, 1000, 0.1),
                  (100000, 3, 1024, 0.5), (70000, 5, 1, 0.0)]


def sort_args(T, k, experts, H, pad, at, kind, rows):
    return dict(topk_idx=P, T=T, top_k=k, experts=experts, offsets=P, order=P, place=P,
                x=P + at * SIZE[kind], x_stride=H + pad + at, hidden=H, x_type=TYPE[kind], rows=P,
                rows_stride=H, rows_type=TYPE[rows], row_scale=P if rows == "i8" else None,
                workspace=P, workspace_bytes=1 << 40)


# T, top_k, share dropped, hidden, padding and start of the rows
COMBINES = [(30, 5, 0.2, 3, 0, 1), (300, 6, 0.1, 72, 0, 0), (40, 8, 0.1, 2101, 0, 0),
            (2000, 16, 0.0, 2101, 0, 1)]  # the last: rows above 128 MiB


def combine_args(T, k, H, pad, at, kind):
    return dict(rows=P + at * SIZE[kind], rows_stride=H + pad + at, n_rows=T * k, type=TYPE[kind],
                place=P, weights=P, T=T, top_k=k, hidden=H, out=P, out_stride=H)


QUANTISES = [(33, K) for K in (3, 101, 501, 1001, 2001, 3001)]


def quantises(kind):
    """M, K: few rows of every width, and rows above 128 MiB."""
    short = 3 if kind == "fp32" else 7
    return QUANTISES + [((128 << 20) // (K * SIZE[kind]) + 1, K)
                        for K in (short, 101, 501, 1001, 2001, 3001)]


def quantise_args(M, K, kind):
    return dict(x=P, x_stride=K, type=TYPE[kind], M=M, K=K, codes=P, codes_stride=K, scale=P)
