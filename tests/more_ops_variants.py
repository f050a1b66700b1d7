"""Cases that between them launch every kernel of the norm, routing and adapter operators.
test_more_ops_launches.py shows that they do (without a GPU), test_gpu_more_ops.py that the results
are right."""

KINDS = ["bf16", "fp16", "fp32"]
TYPE = {"bf16": 0, "fp16": 1, "fp32": 2}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
P = 1 << 20  # an address, where nothing is launched


def norms(kind):
    """M, K: few rows of every width, and of every width that is held in pieces of 16 bytes as many
    rows as make the smallest call of both directions stream."""
    widths = (3, 64, 300, 448, 960, 2000, 3000, 5001, 9000)
    few = [(9, K) for K in widths]
    return few + [((128 << 20) // (2 * K * SIZE[kind]) + 5, K) for K in widths[1:]]


def norm_args(M, K, kind):
    return dict(x=P, x_stride=K, residual=P, residual_stride=K, type=TYPE[kind], M=M, K=K, weight=P,
                eps=1e-6, sum=P, sum_stride=K, y=2 * P, y_stride=K, codes=P, codes_stride=K, scale=P)


def norm_grad_args(M, K, kind):
    return dict(dy=P, dy_stride=K, dsum=None, dsum_stride=K, sum=P, sum_stride=K, type=TYPE[kind],
                M=M, K=K, weight=P, eps=1e-6, dx=P, dx_stride=K, dweight=P, workspace=P,
                workspace_bytes=1 << 40)


# T, experts, top_k, groups, group_best, top_groups: four sizes of either kernel, and one more of the
# kernel that gives a token a wave (16 choices, groups that lanes cannot share, above 512 experts)
ROUTES = [(70, 33, 4, 1, 1, 1), (70, 128, 8, 8, 2, 4), (70, 256, 8, 8, 2, 4), (70, 500, 6, 1, 1, 1),
          (30, 40, 16, 1, 1, 1), (30, 100, 4, 10, 2, 3), (30, 200, 16, 1, 1, 1),
          (30, 450, 5, 50, 1, 7), (30, 1024, 8, 32, 2, 9)]


def route_args(T, E, k, G, best, kept, kind):
    return dict(logits=P, logits_stride=E, type=TYPE[kind], T=T, experts=E, score=1, bias=P,
                groups=G, group_best=best, top_groups=kept, top_k=k, renormalise=1, scale=1.0,
                topk_idx=P, topk_w=P)


def route_grad_args(T, E, k, kind):
    return dict(logits=P, logits_stride=E, type=TYPE[kind], T=T, experts=E, score=0, topk_idx=P,
                top_k=k, renormalise=0, scale=1.0, dweights=P, dlogits=P, dlogits_stride=E)


def adapts(kind):
    """M, K, N, rank, adapters: each range of ranks with few rows an adapter and many, short rows and
    long, below and above what streams."""
    out = []
    for rank in (10, 32, 49, 100):
        out += [(130, 90, 70, rank, 40), (12300, 70, 90, rank, 3)]
        if rank <= 64:
            # rows in tiles of 16, above 80 MiB in whole half lines
            out += [(300, 2100, 130, rank, 40), (30000, 300, 640, rank, 1000)]
        out.append(((80 << 20) // (292 * SIZE[kind]) + 9, 100, 96, rank, 5))
    return out


# Rows to a tile, rows of each adapter, rows without one, K, N, rank: the tiles (each adapter's rounded up)
# are a few more than a multiple of the 256 CUs, and K is long enough beside N that the channels of a
# tile are not shared out otherwise.  Every kernel, and more than 64 adapters
ADAPT_RESTS = [
    (16, [1500, 1300, 1400], 7, 700, 1100, 10), (16, [43] * 100, 40, 500, 800, 16),
    (16, [2] * 300, 100, 2600, 600, 16),
    (16, [700, 900, 1, 1100, 1480], 5, 400, 600, 24), (16, [2] * 300, 100, 2600, 600, 32),
    (32, [3000, 17, 2500, 4000, 3500, 33, 3450], 0, 200, 600, 32),
    (16, [1100, 1000, 900, 1200], 0, 300, 600, 49), (16, [3] * 300, 120, 1000, 520, 64),
    (32, [1000, 900, 1100, 700, 800, 1200, 850, 950, 800], 30, 330, 600, 64),
    (32, [1840] * 9, 80, 1000, 1024, 64),  # above 80 MiB
    (16, [1100, 1000, 900, 1200], 11, 300, 600, 128), (16, [15, 16, 17, 18] * 45, 60, 500, 600, 100)]


def adapt_args(M, K, N, rank, adapters, kind):
    return dict(x=P, x_stride=K, type=TYPE[kind], M=M, K=K, a=P, a_stride=K, b=P, b_stride=rank, N=N,
                rank=rank, scale=P, adapters=adapters, offsets=P, order=P, base=P, base_stride=N,
                out=P, out_stride=N)
