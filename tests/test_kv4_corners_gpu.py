"""Corners of a cache in 4 bits: keys whose rotation passes the largest 32-bit
number."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv4_ref as kv4
from test_kv4_gpu import D, Decode, Store, layer_of

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- past 32 bits

def huge(shape, seed, share=1.0):
    """bf16 values of 2.2e38 to 3.38e38 of either sign (of both ends of a turn the sum is up to
    4.8e38, a 32-bit number at most 3.40e38), a share of them; the others about 1."""
    rng = np.random.default_rng(seed)
    x = rng.uniform(2.2e38, 3.38e38, shape) * rng.choice([-1.0, 1.0], shape)
    x = np.where(rng.uniform(size=shape) < share, x, rng.standard_normal(shape))
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("rot", [16, 48, 64, 256])
@pytest.mark.parametrize("share", [1.0, 0.05])
def test_store_rotations_past_32_bits(cuda, rot, share):
    """They are the largest number there is, with their sign, and so is their block's scale."""
    s = Store([40, 7], [3, 0], H=2, Hkv=2, seed=60 + rot)
    s.pos[:40] = torch.from_numpy(np.random.default_rng(60).integers(0, 3000, 40).astype(np.int32))
    s.qkv.view(47, 6, D)[:, 2:] = huge((47, 4, D), 61 + rot, share)
    layer = layer_of("sliding", rot=rot)
    s.check(layer)
    k = kv4.project(s.qkv, s.pos, 2, 2, layer)[1]
    assert share < 1 or (np.abs(k) > 3.41e38).any()   # (the case is what it says)


def test_decode_rotation_past_32_bits(cuda):
    """The same of a step's new token (its queries are zeros: all scores are)."""
    d = Decode([20, 1000, 37], H=4, Hkv=2, seed=62, layer=layer_of("sliding"))
    x = d.qkv.view(3, 8, D)
    x[:, :4] = 0
    x[:, 4:6] = huge((3, 2, D), 63)
    d.check()
