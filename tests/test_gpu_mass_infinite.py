"""Attention mass of columns whose logits are all -infinity (infinite key norms against the
query): they hand out no weight, as their output is zero, and the other columns and rows of the
call are as without them.

Tolerance: the untouched rows' sums as in the other mass tests (6e-5 of the largest weight).
"""
import math

import numpy as np
import pytest
import torch

from packed_cache_decode_b200 import binding as B

from .test_gpu_bounded_cache import MASS_REL, dequantised, dev, make_layouts, random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,h_kv", [(3, 2), (40, 8)])      # the sums inside the merge; a kernel of their own
@pytest.mark.parametrize("G", [4, 8, 12])
def test_columns_of_minus_infinity_weigh_nothing(G, b, h_kv):
    rng = np.random.default_rng(91)
    lay, olay = make_layouts("k4", 2)                       # one key group: a logit is a norm times one dot product
    most = 500
    tiles = random_cache(olay, b, h_kv, 8, rng)
    lens = [1, 2] + [most - r for r in range(b - 2)]
    q = rng.standard_normal((b, h_kv, G, 128))
    code = 64 * (olay.k_record_bytes + olay.v_record_bytes)
    finite = tiles.copy()
    norms = tiles[:2, :, 0, code:].copy().view(np.float32).reshape(2, h_kv, -1, 64)
    norms[:, :, :-1] = np.inf
    tiles[:2, :, 0, code:] = norms.reshape(2, h_kv, -1).view(np.uint8)
    for r in range(2):
        for h in range(h_kv):
            k, _ = dequantised(olay, finite[r, h], lens[r])
            q[r, h] = -k.sum(0)
            assert ((q[r, h] @ k.T) < -1).all()
    mass0 = rng.uniform(0, 1, (b, h_kv, most)).astype(np.float32)
    mass, out = torch.from_numpy(mass0).cuda(), torch.full((b, h_kv * G, 128), 5.0, device="cuda")
    ws = torch.empty(B.mass_workspace_bytes(lay, b, h_kv * G, h_kv, most), dtype=torch.uint8, device="cuda")
    qd = torch.from_numpy(q.reshape(b, h_kv * G, 128)).float()
    B.decode_attention_mass(lay, qd.cuda(), torch.from_numpy(tiles).cuda(), dev(lens), 512, most, mass, out, ws, h_kv, decay=0.5)
    assert lay.status() == 0
    got, o = mass.cpu().double().numpy(), out.cpu().numpy()
    for r in range(2):
        assert (o[r] == 0).all()
        np.testing.assert_array_equal(got[r, :, :lens[r]], 0.5 * mass0[r, :, :lens[r]])
        np.testing.assert_array_equal(got[r, :, lens[r]:], mass0[r, :, lens[r]:])
    for r, h in ((2, 0), (b - 1, h_kv - 1)):
        n = lens[r]
        k, _ = dequantised(olay, tiles[r, h], n)
        s = qd[r].double().numpy().reshape(h_kv, G, 128)[h] @ k.T / math.sqrt(128)
        p = np.exp(s - s.max(1, keepdims=True))
        w = (p / p.sum(1, keepdims=True)).sum(0)
        err = np.abs(got[r, h, :n] - (0.5 * mass0[r, h, :n].astype(np.float64) + w))
        assert (err <= MASS_REL * w.max() + 2.0 ** -23 * (mass0[r, h, :n] + w)).all()
