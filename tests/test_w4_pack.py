"""Packing of 4-bit expert weights (torch_utils.w4_quantize), on the CPU."""
import pytest

torch = pytest.importorskip("torch")

import fp8_expert_ffn_b200 as fx  # noqa: E402
from fp8_expert_ffn_b200 import torch_utils as tu  # noqa: E402


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,k", [(32, 1), (32, 33), (64, 100), (128, 512), (128, 1001)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_values_are_the_nearest_codes(group, k, zeros, dt):
    g = torch.Generator().manual_seed(k)
    w = torch.randn(3, 7, k, generator=g)
    w[1, 2] = 0.0                                   # a row of zeros
    w[2, 3, : min(k, 5)] += 2.0                     # an uneven range
    q = tu.w4_quantize(w, group, zeros, dt)
    ng = -(-k // group)
    assert q.codes.shape[:2] == (3, 7) and q.codes.shape[2] % 16 == 0 and q.codes.shape[2] >= (k + 1) // 2
    assert q.scales.shape == (3, 7, ng) and q.scales.dtype == dt
    assert (q.zeros is None) == (not zeros)
    assert q.desc.group == group and q.desc.ld == q.codes.shape[2]
    assert q.desc.scale_type == (fx.MOE_BF16 if dt == torch.bfloat16 else fx.MOE_F32)
    v = tu.w4_values(q, k)
    assert (v[1, 2] == 0).all()
    step = q.scales.float().repeat_interleave(group, -1)[:, :, :k]
    # half a step; the scale's own rounding (2^-8 in bf16) moves the ends of the
    # range by up to 15 steps times that, and a rounded zero point by half a step
    err = (v - w).abs()
    assert (err <= step * (0.5 + (0.5 if zeros else 0.0) + 15 * 2.0 ** -8) + 1e-7).all()


def test_nibble_order():
    w = torch.tensor([[[-7.0, 0.0, 7.0, 1.0]]])
    q = tu.w4_quantize(w, 32, False, torch.float32)
    assert q.codes[0, 0, :2].tolist() == [1 | (8 << 4), 15 | (9 << 4)]   # column 2i low, 2i + 1 high
    assert torch.equal(tu.w4_values(q, 4), w)
