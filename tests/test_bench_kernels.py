"""The benchmark's traffic record and the kernels as they are built: the names that a
profiler reports for them, and the sources that define them (no GPU)."""
import os
import re
import shutil
import subprocess

import pytest

import bench
import bit_quantized_fine_amd as q
from test_bench import _counter_csv

CSRC = os.path.join(bench.ROOT, "bit_quantized_fine_amd", "csrc")
NEG = "void at::native::vectorized_elementwise_kernel<4, at::native::neg_kernel>(int)"


def _built_names(kernel):
    """Names of the kernel's instances in the built library."""
    if shutil.which("nm") is None or not os.path.exists(q.LIB_PATH):
        pytest.skip("needs nm and the built library")
    out = subprocess.run(["nm", "-C", q.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    return sorted(set(re.findall(r"void (qnf4::" + kernel + r"<[^(]*>\(.*\))", out)))


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_the_training_steps_instance_is_recorded(tmp_path, kernel):
    """Of a kernel's instances exactly one is the training step's; its dispatches
    alone make the record."""
    names = ["void " + n for n in _built_names(kernel)]
    mine = [n for n in names if bench.traffic_kernel(n) == kernel]
    assert len(names) > 2 and len(mine) == 1
    for counter, folder in (("FETCH_SIZE", "f"), ("WRITE_SIZE", "w")):
        _counter_csv(str(tmp_path / folder), counter,
                     [(NEG, 1048576.0)] + [(n, 100.0 if n in mine else 7777.0) for n in names])
    out = bench.write_traffic(str(tmp_path / "f"), str(tmp_path / "w"), 1024, "test",
                              path=str(tmp_path / "t.json"))
    assert set(out) == {kernel}
    assert out[kernel]["dispatches"] == 1
    assert out[kernel]["bytes_per_launch"] == pytest.approx(200 * 1024)


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_a_stored_reading_depends_on_every_source_of_its_kernel(kernel):
    """The hash covers the kernel's file and whatever of this library it includes,
    directly or not."""
    files, todo = set(), [bench.KERNEL_SOURCES[kernel][0]]
    while todo:
        f = todo.pop()
        if f in files:
            continue
        files.add(f)
        with open(os.path.join(CSRC, f)) as fh:
            todo += re.findall(r'^#include "(\w+\.hpp)"', fh.read(), re.M)
    assert files == set(bench.KERNEL_SOURCES[kernel])
