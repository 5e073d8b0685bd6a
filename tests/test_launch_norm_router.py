"""Every size that the norm, the checkpoints and the router admit can be launched:
fewer than 2^32 threads along x, at most 65536 workgroups along y."""
import pytest

from launch_util import run

NORM = """
out = []
for K in (8, 64, 512, 1024, 4096, 16384, 32768, 65536, 65544, 1 << 22):
    for M in (1, 17, 4096, 1 << 22, (1 << 24) + 3, 1 << 31, 1 << 37):
        if M * K > 1 << 40:
            continue
        c8 = ctypes.byref(q._Act8(1 << 20, 1 << 20)) if K % 64 == 0 else None
        st = [L.qlora_rms_norm_fwd(P, P, P, 1, M, K, 1e-5, P, P, P, c8, None)]
        for dg in (None, P):
            st.append(L.qlora_rms_norm_bwd(P, P, P, P, P, 0, M, K, P, dg, P, BIG, None))
        yz = max(blocks_yz(), default=0)
        out.append((M, K, yz, st, [l[0] for l in launches()]))
print(json.dumps(out))
"""

ACT8 = """
out = []
c8 = ctypes.byref(q._Act8(1 << 20, 1 << 20))
for K in (64, 4096, 1 << 22):
    for M in (1, 1 << 16, 1 << 18, 1 << 28, 1 << 34):
        if M * K > 1 << 40:
            continue
        st = [L.qlora_act8_pack(P, M, K, c8, None), L.qlora_act8_unpack(c8, M, K, P, None)]
        yz = max(blocks_yz(), default=0)
        out.append((M, K, yz, st, [l[0] for l in launches()]))
for E in (1, 31, 32, 63, 64):   # 2^32 threads from 64 experts on: refused
    st = [L.qlora_grouped_act8_bwd(P, c8, 64, P, 1, 64, P, E, weight(8 * E, 1 << 22, 0), P, P, 256, 1.0,
                                   None, P, P, P, P, P, BIG, None)]
    out.append((E, 0, max(blocks_yz(), default=0), [0 if s == 2 and E == 64 else s for s in st],
                [l[0] for l in launches()] + [0] * (E == 64)))
for M in (1, 16, 17, 2048, 1 << 22):
    for r in (8, 64, 256):
        for T in (None, P):
            st = [L.qlora_linear_act8_bwd(P, c8, M, weight(4096, 4096), P, P, r, 1.0, drop(0.1), T,
                                          P, P, P, P, BIG, None),
                  L.qlora_grouped_act8_bwd(P, c8, M, P, 1, M, P, 8, weight(8 * 256, 4096), P, P, r,
                                           1.0, None, T, P, P, P, P, BIG, None)]
            yz = max(blocks_yz(), default=0)
            out.append((M, r, yz, st, [l[0] for l in launches()]))
print(json.dumps(out))
"""

ROUTER = """
out = []
for E in (1, 8, 64, 65, 256, 512, 1000, 1024):
    for tokens in (1, 5, 1 << 20, 1 << 25, (1 << 25) + 1, 1 << 30):
        c = ctypes.byref(q._RouterConfig(1, 1, 1, 1, 1, 1, 1.0))
        st = [L.qlora_router_fwd(P, 1, tokens, E, P, c, P, P, None),
              L.qlora_router_fwd(P, 0, tokens, E, None, c, P, P, None),
              L.qlora_router_bwd(P, P, 1, P, tokens, E, c, P, None),
              L.qlora_router_bwd(P, P, 0, P, tokens, E, c, P, None)]
        if E % 8 == 0:
            g = ctypes.byref(q._RouterConfig(0, 1, 8, 1, 2 if E > 8 else 1, 0, 1.0))
            st.append(L.qlora_router_fwd(P, 1, tokens, E, P, g, P, P, None))
        yz = max(blocks_yz(), default=0)
        out.append((tokens, E, yz, st, [l[0] for l in launches()]))
print(json.dumps(out))
"""


@pytest.mark.parametrize("calls", [NORM, ACT8, ROUTER], ids=["norm", "act8", "router"])
def test_grids_of_admitted_sizes(tmp_path, calls):
    got = run(tmp_path, calls)
    assert len(got) > 7
    for *size, yz, status, threads in got:
        assert all(s == 0 for s in status), (size, status)
        assert yz <= 65536, (size, yz)
        assert len(threads) >= len(status) and max(threads) < 2 ** 32, (size, threads)
