"""Every size that a call admits can be launched: HIP takes fewer than 2^32 threads
along x in one launch."""
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


@pytest.mark.parametrize("calls", [ROWS, DROPOUT], ids=["exchange", "dropout"])
def test_grids_of_admitted_sizes(tmp_path, calls):
    got = run(tmp_path, calls)
    assert len(got) > 7
    for *size, status, threads in got:
        assert all(s == 0 for s in status), size
        assert len(threads) >= len(status) and max(threads) < 2 ** 32, (size, threads)
