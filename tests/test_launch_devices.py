"""Kernels that use more LDS than a launch gets by default have their limit raised
on every device they are launched on, not only on the first."""
from launch_util import run

CALLS = """
def plain(M, N, K, r):
    nf = ctypes.byref(q._Nf4Weight(1 << 20, 1 << 20, 1 << 20, N, K))
    yield L.qlora_linear_fwd(P, M, nf, P, P, r, 1.0, P, P, P, BIG, None)
    yield L.qlora_linear_bwd(P, P, M, nf, P, P, r, 1.0, P, P, P, P, P, BIG, None)
    for dq in (0, 1):
        w = weight(N, K, dq)
        yield L.qlora_q4_linear_fwd(P, M, w, P, P, r, 1.0, P, P, P, BIG, None)
        yield L.qlora_q4_linear_bwd(P, P, M, w, P, P, r, 1.0, P, P, P, P, P, BIG, None)
        yield L.qlora_linear_dropout_fwd(P, M, w, P, P, r, 1.0, drop(0.1), P, P, P, BIG, None)
        yield L.qlora_linear_dropout_bwd(P, P, M, w, P, P, r, 1.0, drop(0.1), P, P, P, P, P, BIG,
                                         None)
    yield L.qlora_lora16_fwd(P, M, P, N, K, P, P, r, 1.0, P, P, P, BIG, None)
    yield L.qlora_lora16_bwd(P, P, M, P, N, K, P, P, r, 1.0, P, P, P, P, P, BIG, None)

def grouped(M, E, N, K, r):
    for dq in (0, 1):
        for d in (None, drop(0.1)):
            w = weight(E * N, K, dq)
            yield L.qlora_grouped_fwd(P, M, P, E, w, P, P, r, 1.0, d, P, P, P, BIG, None)
            yield L.qlora_grouped_bwd(P, P, M, P, E, w, P, P, r, 1.0, d, P, P, P, P, P, BIG, None)

def every_call():
    for M, K in ((1, 8192), (4, 4096), (16, 1024), (16, 22016), (300, 1024)):
        yield from plain(M, 1024, K, 16)
    # few tokens; each tile height, with 128 and 256 weight rows; dX of many tiles
    for M, E, N, K in ((3, 2, 256, 1024), (40, 2, 256, 1024), (60, 2, 256, 1024),
                       (900, 2, 256, 1024), (400, 32, 4096, 256), (900, 32, 4096, 256),
                       (4000, 2, 4096, 4096)):
        yield from grouped(M, E, N, K, 16)
    yield L.qlora_expert_plan(P, 4096, 1024, P, P, P, P, BIG, None)

status, short, seen = [], [], 0
for device in (0, 1, 5, 0):
    rec.recorder_device(device)
    for i, st in enumerate(every_call()):
        status.append(st)
        for threads, lds, allowed in launches():
            seen += lds > 48 * 1024
            if lds > 48 * 1024 and allowed < lds:
                short.append((device, i, lds, allowed))
print(json.dumps(dict(status=sorted(set(status)), seen=seen, short=short)))
"""


def test_every_device_gets_the_kernels_lds(tmp_path):
    got = run(tmp_path, CALLS)
    assert got["status"] == [0]
    assert got["seen"] > 200 and got["short"] == []
