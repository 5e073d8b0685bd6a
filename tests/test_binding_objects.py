"""Weights that the binding takes by their fields, and numbers that a C argument cannot
hold (CPU: the calls end at the check that their tensors are on a GPU)."""
import os
import types

import pytest
import torch

import bit_quantized_fine_amd as q

pytestmark = pytest.mark.skipif(not os.path.exists(q.LIB_PATH),
                                reason="libqlora_nf4.so not built (run __graft_entry__.build())")


def _weight(N=64, K=128):
    return q.NF4Weight(torch.zeros(N * K // 2, dtype=torch.uint8),
                       torch.zeros(N * K // 64, dtype=torch.uint8),
                       torch.zeros((N * K // 64 + 255) // 256, dtype=torch.float32), N, K)


class Kept(torch.nn.Module):
    """A module that holds a weight's fields as buffers."""

    def __init__(self, w):
        super().__init__()
        for name in ("codes", "absmax_q", "absmax_scale"):
            self.register_buffer(name, getattr(w, name))
        self.N, self.K = w.N, w.K


def _calls(w):
    X, dY = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    return [lambda: q.qlora_linear_dropout_fwd(X, w), lambda: q.qlora_linear_dropout_bwd(dY, X, w),
            lambda: q.qlora_grouped_fwd(X, off, w, 1), lambda: q.qlora_grouped_bwd(dY, X, off, w, 1)]


@pytest.mark.parametrize("make", [lambda w: w, lambda w: types.SimpleNamespace(**w._asdict()), Kept],
                         ids=["tuple", "namespace", "module"])
def test_weights_are_taken_by_their_fields(make):
    """Any object with an NF4Weight's fields, as the plain layer's calls take it."""
    for call in _calls(make(_weight())):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


def test_fields_of_other_weights_are_checked():
    w = _weight()
    bad = types.SimpleNamespace(**dict(w._asdict(), absmax_q=w.absmax_q.int()))
    for call in _calls(bad):
        with pytest.raises(TypeError, match="w.absmax_q must be"):
            call()
    w4 = q.Q4Weight(w.codes, None, torch.zeros(128), 64, 128, "int4", False)
    for call in _calls(w4):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


@pytest.mark.parametrize("name", ["topk", "groups", "top_groups", "group_top"])
@pytest.mark.parametrize("wrong", [2 ** 32 + 2, -2 ** 32 + 2, 2 ** 31, -2 ** 31 - 1, 2 ** 70])
def test_router_numbers_past_32_bits(name, wrong):
    """A number that a C int cannot hold is refused, not taken modulo 2^32."""
    kw = {"topk": 2, "groups": 2, "top_groups": 2, "group_top": 2, name: wrong}
    with pytest.raises(ValueError, match=f"{name} .* 32 bits"):
        q.qlora_router_fwd(torch.zeros(4, 8), **kw)


@pytest.mark.parametrize("wrong", [2 ** 32 + 2, 2 ** 31, -2 ** 33])
def test_grouped_numbers_past_32_bits(wrong):
    w = _weight()
    x8 = q.Act8(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="topk .* 32 bits"):
        q.qlora_grouped_act8_bwd(torch.zeros(8, 64, dtype=torch.bfloat16), x8,
                                 torch.zeros(2, dtype=torch.int32), w, 1,
                                 order=torch.zeros(8, dtype=torch.int32), topk=wrong)
