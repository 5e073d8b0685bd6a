"""Every size that a call admits can be launched: HIP takes fewer than 2^32 threads
along x in one launch, and the GPU's limit along y and z is 65536 workgroups."""
import pytest

from launch_util import run

ROWS = """
out = []
for topk in (1, 2, 64):
    for tokens in (1, (1 << 24) - 1, 1 << 24, (1 << 24) + 3, (1 << 30) // topk):
        if tokens * topk > 1 << 30:
            continue
        for K in (8, 1 << 22):
            st = [L.qlora_expert_gather(P, tokens, topk, K, P, P, None),
                  L.qlora_expert_combine(P, tokens, topk, K, P, P, P, None),
                  L.qlora_expert_combine_bwd(P, P, tokens, topk, K, P, P, P, P, None)]
            out.append((tokens, topk, K, st, [l[0] for l in launches()]))
for n in (1, 1 << 24, 1 << 30):
    for E in (1, 1024):
        st = [L.qlora_expert_plan(P, n, E, P, P, P, P, BIG, None)]
        out.append((n, 0, E, st, [l[0] for l in launches()]))
print(json.dumps(out))
"""

DROPOUT = """
out = []
for n in (1, 1 << 24, (1 << 36) - 1, 1 << 36, (1 << 36) + 1, (1 << 37) - 8192, 1 << 37, 3 << 37):
    st = [L.qlora_dropout_apply(P, n, drop(0.1), P, None)]
    out.append((n, st, [l[0] for l in launches()]))
print(json.dumps(out))
"""

# (A group of rows can be launched or is refused with QLORA_ERR_SHAPE, 2, whatever
# memory it would need; 2^30 rows of 64 columns fit one GPU.)
GROUPED = """
out = []
for E, N, K in ((1, 8, 64), (1, 256, 64), (4, 264, 64), (1024, 8, 64), (1, 8, 256), (1, 1 << 20, 64),
                (1, 8, 1 << 22), (64, 4096, 4096)):
    for r in (0, 8, 256):
        for M in (0, 1, 17, 1 << 16, 1 << 20, 1 << 24, 1 << 28, 1 << 30, 3 << 29, 1610613000,
                  (1 << 31) - 1):
            st = [L.qlora_grouped_fwd(P, M, P, E, weight(E * N, K, 0), P, P, r, 1.0, None, P, P, P,
                                      BIG, None),
                  L.qlora_grouped_bwd(P, P, M, P, E, weight(E * N, K, 0), P, P, r, 1.0, drop(0.1), P,
                                      P, P, P, P, BIG, None)]
            if N == 8 and K == 64 and r == 0 and M <= 1 << 30:
                assert st == [0, 0], (M, E, st)
            out.append((M, E, N, K, r, [s for s in st if s != 2], [l[0] for l in launches()]))
print(json.dumps(out))
"""

LAYER = """
out = []
for M in (1, 16, 17, 2048, 1 << 23, (1 << 23) + 200, 1 << 24, 1 << 26, 1 << 28):
    for N, K, r in ((8, 64, 8), (8, 64, 256), (4096, 4096, 64), (8, 1 << 22, 8), (1 << 22, 64, 8)):
        if M * (2 * (N + K) + 8 * r) > 288 << 30:   # (T and its partial sums)
            continue
        for d in (None, drop(0.1)):
            st = [L.qlora_linear_dropout_fwd(P, M, weight(N, K), P, P, r, 1.0, d, P, P, P, BIG, None),
                  L.qlora_linear_dropout_bwd(P, P, M, weight(N, K), P, P, r, 1.0, d, None, P, P, P, P,
                                             BIG, None)]
            yz = max(blocks_yz(), default=0)
            out.append((M, N, K, r, yz, [s for s in st if M < 1 << 26 or s != 2],
                        [l[0] for l in launches()]))
            assert yz <= 65536, (M, N, K, r, yz)
print(json.dumps(out))
"""


@pytest.mark.parametrize("calls", [ROWS, DROPOUT, GROUPED, LAYER], ids=["exchange", "dropout", "grouped", "layer"])
def test_grids_of_admitted_sizes(tmp_path, calls):
    got = run(tmp_path, calls)
    assert len(got) > 7
    for *size, status, threads in got:
        assert all(s == 0 for s in status), size
        assert (len(threads) >= len(status) or size[0] == 0) and max(threads, default=0) < 2 ** 32, (size, threads)
