"""Rotation at positions past 2^32, to both ends of 64 bits: the phase is position * frequency modulo one
turn, in whole numbers from the stored frequency. Tolerance as in test_gpu_rotary."""
import math

import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot,kw", [(64, {}), (48, dict(base=1e6)),
                                    (96, dict(scaling="yarn", factor=40.0))])
@pytest.mark.parametrize("inverse", [False, True])
def test_phase_is_exact_at_far_positions(rot, kw, inverse):
    places = [1 << 32, (1 << 32) + 1, (1 << 40) + 12345, (1 << 62) + 7, (1 << 63) - 1, -(1 << 63), -1,
              -(1 << 32) - 5, -(1 << 55) + 3, 0]
    fr = ds4idx.rotary_freqs(rot, **kw)
    f = [int(v) for v in fr.freqs]
    x = torch.randn(len(places), 3, rot, generator=torch.Generator().manual_seed(rot))
    y = ds4idx.rotary(x.cuda(), torch.tensor(places).cuda(), fr, inverse=inverse).double().cpu().numpy()
    a, b = x.double().numpy()[..., 0::2], x.double().numpy()[..., 1::2]
    angle = np.array([[2 * math.pi * ((p * v) % (1 << 64) / 2 ** 64) for v in f] for p in places])
    if inverse:
        angle = -angle
    c, s = fr.scale * np.cos(angle)[:, None], fr.scale * np.sin(angle)[:, None]
    bound = 8 * 2.0 ** -24 * fr.scale * (np.abs(a) + np.abs(b)) + 1e-37
    assert np.all(np.abs(y[..., 0::2] - (a * c - b * s)) <= bound)
    assert np.all(np.abs(y[..., 1::2] - (a * s + b * c)) <= bound)
