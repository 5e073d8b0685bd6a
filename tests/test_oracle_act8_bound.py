"""How far a checkpoint's values are from what was packed: half a step of the block and
half a step of bf16, both counted (CPU, over every significand and every value below)."""
import numpy as np

from oracle import act8, bf16_bits_to_f64


def test_error_of_every_value():
    worst = {}
    for top in range(0x3F80, 0x4000):            # largest values from 1 to 2
        v = np.arange(top + 1, dtype=np.uint16)
        v = np.concatenate([v, np.zeros(-len(v) % 63, np.uint16)]).reshape(-1, 63)
        b = np.concatenate([v, np.full((len(v), 1), top, np.uint16)], axis=1)
        codes, c = act8.pack(b)
        x, got = bf16_bits_to_f64(b), bf16_bits_to_f64(act8.value_bits(codes, c))
        amax = bf16_bits_to_f64(np.array([top], np.uint16))[0]
        err, exact = np.abs(x - got), np.abs(codes * c.astype(np.float64))
        # (the constant and the product are rounded to fp32: 2^-22 of the value)
        assert (err <= amax / 254 + (2.0 ** -8 + 2.0 ** -22) * exact).all(), hex(top)
        worst[amax] = err.max() / (amax / 254)
    assert 1.86 < max(worst.values()) < 1.88 and max(worst, key=worst.get) == 1.0625
    assert worst[1.0] < 1.001
