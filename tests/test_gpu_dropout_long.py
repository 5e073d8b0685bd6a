"""Dropout of a tensor with more pieces than one row of workgroups takes."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import OFFSET, SEED, state
from gpu_util import dev, need_gpu, say, torch
from oracle import dropout as od

pytestmark = pytest.mark.gpu


def test_positions_past_2_to_the_36():
    """A tensor of 2^36 + 1003 elements (128 GiB) in place, looked at where a row of
    workgroups ends, at its end, and where piece numbers pass 32 bits."""
    need_gpu()
    n, p = 2 ** 36 + 1003, 0.5
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2 * n + 2 ** 34:
        pytest.skip("not enough free GPU memory")
    say(f"dropout n={n}")
    x = torch.ones(n, dtype=torch.bfloat16, device=dev())
    q.qlora_dropout(x, p, state(), out=x)
    torch.cuda.synchronize()
    for first in (0, 2 ** 35 - 100, 2 ** 36 - 500, 2 ** 36 + 5):
        m = min(1000, n - first)
        keep = od.halves(m, SEED, OFFSET, first) >= od.threshold(p)
        np.testing.assert_array_equal(x[first:first + m].cpu().float().numpy(), 2.0 * keep)
    del x
    torch.cuda.empty_cache()
