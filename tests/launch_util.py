"""The library in a process of its own with launch_recorder.cpp in the HIP calls'
place: run(body) gives the body q (the package), L (the library), P (a made-up
address for every pointer) and rec, and returns what it prints as JSON."""
import json
import os
import shutil
import subprocess
import sys

import pytest

import bit_quantized_fine_amd as q

HERE = os.path.dirname(os.path.abspath(__file__))

HEAD = """
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
for name in ("threads_x", "blocks_yz", "lds", "allowed"):
    getattr(rec, "recorder_" + name).restype = ctypes.c_uint64
import bit_quantized_fine_amd as q
L = q.lib()
P = ctypes.c_void_p(1 << 20)
BIG = (1 << 63) - 1

def weight(N, K, dq=1, book=0):
    return ctypes.byref(q._Q4Weight(1 << 20, 1 << 20, 1 << 20, N, K, book, dq))

def drop(p):
    return ctypes.byref(q._Dropout(1 << 20, p))

def blocks_yz():
    return [rec.recorder_blocks_yz(i) for i in range(rec.recorder_count())]

def launches():
    n = rec.recorder_count()
    out = [(rec.recorder_threads_x(i), rec.recorder_lds(i), rec.recorder_allowed(i))
           for i in range(n)]
    rec.recorder_clear()
    return out
"""


def run(tmp_path, body):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(q.LIB_PATH):
        pytest.skip("needs g++ and the built library")
    so = str(tmp_path / "recorder.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC",
                    os.path.join(HERE, "launch_recorder.cpp"), "-o", so], check=True)
    script = tmp_path / "body.py"
    script.write_text(HEAD + body)
    p = subprocess.run([sys.executable, str(script), so], capture_output=True, text=True,
                       timeout=120, env={**os.environ, "PYTHONPATH": os.path.dirname(HERE)})
    assert p.returncode == 0, p.stderr
    return json.loads(p.stdout)
