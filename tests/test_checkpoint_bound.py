"""How far an 8-bit checkpoint may be from a value next to a code's boundary: (1/2 + 2^-14) Delta, as
include/quest.h states. With inv = fl(fl(1 / Delta) (1 - 2^-22)), two roundings of 2^-24 around the factor,
v inv lies at most 1.5 2^-22 below v / Delta (relative), which is 1.5 2^-15 of a step at |v| = 128 Delta; the
floor of the fused product is exact, and restoring rounds (q + 1/2) Delta by at most 2^-24 of 128 Delta."""
import numpy as np
import pytest
import torch

import bit_quantization_aware_blockwise_b200 as q
import block_reference as ref

BOUND = 0.5 + 2.0 ** -14


def restored(v, amax):
    """The checkpoint's arithmetic in fp32 (v inv exact in 64 bits: 24 + 24 bits): values and step."""
    delta = (amax * np.float32(2.0 ** -7)).astype(np.float32)
    inv = (np.float32(1) / delta).astype(np.float32) * np.float32(1 - 2.0 ** -22)
    code = np.floor(v.astype(np.float64) * inv.astype(np.float64))
    assert code.min() >= -128 and code.max() <= 127
    return ((code + 0.5).astype(np.float32) * delta).astype(np.float64), delta.astype(np.float64)


def test_bound_of_the_arithmetic():
    # steps of every mantissa class, values a few units in the last place around every boundary
    rng = np.random.default_rng(1)
    worst = 0.0
    for amax in np.concatenate([np.float32(1) + rng.integers(0, 1 << 23, 400).astype(np.float32) * np.float32(2.0 ** -23),
                                np.float32([1, 2 - 2.0 ** -23])]):
        k = np.arange(-128, 129)
        at = (k * (np.float64(amax) / 128)).astype(np.float32)
        ulps = np.arange(-16, 17)
        v = (at.view(np.int32)[:, None] + ulps[None, :]).view(np.float32).astype(np.float32)
        v = v[np.abs(v) <= amax]
        got, delta = restored(v, np.full_like(v, amax))
        worst = max(worst, float((np.abs(got - v.astype(np.float64)) / delta).max()))
    assert 0.5 + 2.0 ** -16 < worst <= BOUND      # more than half a step is reached, and stated


@pytest.mark.gpu
def test_values_next_to_a_boundary(cuda_device):
    # projections w0 + w1 with w0 = k / 128 and w1 a few units of its last place: amax = 1, so Delta = 2^-7
    F, K = 128, 64
    k = torch.arange(F, device="cuda", dtype=torch.float64)
    for ulps in range(9):
        wg = torch.zeros(F, K, device="cuda", dtype=torch.float64)
        wg[:, 0] = k / 128
        wg[:, 1] = ulps * 2.0 ** -24
        wg[0, 0], wg[0, 1] = 1.0, 0.0
        x = torch.zeros(1, K, device="cuda")
        x[0, :2] = 1
        w = wg.to(torch.bfloat16)
        assert torch.equal(w.double(), wg)
        _, kept = q.gated_linear(x.to(torch.bfloat16), w, w, checkpoint=True)
        q.device_status()
        assert (kept["scales"] == 2.0 ** -7).all()
        for got in ref.halves(kept):
            # 2^-23 of the largest term beside it: the two-term sum's own cut
            assert ((got[0] - wg.sum(1)).abs() <= BOUND * 2.0 ** -7 + 2.0 ** -23).all()
