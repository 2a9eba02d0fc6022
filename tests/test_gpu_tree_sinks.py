"""Tree attention where one token takes most of a column's weight (an attention sink): a first
token of small value and a long tail of values that share a direction, so that the output is the
tail's. Both kernels, contiguous and paged.

Tolerance: the library's 2e-3 relative L2 (fp32 outputs). Weights are fp16 with their value norms.
In the kernel for many columns an entry keeps half a step of 2^-11 down to 2^-18 of the
largest one seen and is lost below 2^-29, so every tail here is within its reach. The kernel for few
columns has the reference of plain decode attention, the largest weight of a warp's tokens at 1:
where the tail's entries are fp16 subnormals next to the sink (step 2^-24) a warp's share of the
tail loses up to 2^-25 / (2^-drop value) of itself, so its tails stop at 2^-18.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from packed_cache_decode_b200 import binding as B

from .parity_util import ATTN_REL_L2, rel_l2
from .test_gpu_bounded_cache import dequantised, make_layouts, random_cache
from .test_gpu_tree import random_tree, run_tree

pytestmark = pytest.mark.gpu

B_ROWS, H_KV, LENGTH = 8, 4, 4096       # 32 units or more of 64 tiles over the SMs: long slices


def sink_inputs(olay, n, G, drop, value, sink_value, at, rng):
    """Tiles and queries: every query puts token `at` 2^drop above a typical other token; value
    norms `value` sqrt(128) (the sink's `sink_value` times that), the value codes of every tile
    alike (a common component)."""
    tiles = random_cache(olay, B_ROWS, H_KV, LENGTH // 64, rng)
    code = 64 * (olay.k_record_bytes + olay.v_record_bytes)
    tiles[..., 64 * olay.k_record_bytes:code] = tiles[:1, :1, :1, 64 * olay.k_record_bytes:code]
    norms = tiles[..., code:].copy().view(np.float32).reshape(B_ROWS, H_KV, LENGTH // 64, -1, 64)
    norms[..., -1, :] *= np.float32(value)
    norms[:, :, at // 64, -1, 8 * (at % 8) + at % 64 // 8] *= np.float32(sink_value)
    tiles[..., code:] = norms.reshape(B_ROWS, H_KV, LENGTH // 64, -1).view(np.uint8)
    q = 0.2 * rng.standard_normal((B_ROWS, n, H_KV, G, 128))
    for r in range(B_ROWS):
        for h in range(H_KV):
            k, _ = dequantised(olay, tiles[r, h, at // 64:at // 64 + 1], 64)
            k = k[at % 64]
            q[r, :, h] += drop * math.log(2) * math.sqrt(128) * k / (k @ k)
    return tiles, torch.from_numpy(q.reshape(B_ROWS, n, H_KV * G, 128)).float()


def check(lay, olay, tiles, q, n, G, use_pages, rng):
    mask = np.stack([random_tree(rng, n) for _ in range(B_ROWS)])
    out = run_tree(lay, q, mask, tiles, [LENGTH] * B_ROWS, torch.float32, use_pages, rng).cpu().double().numpy()
    assert lay.status() == 0
    worst = 0.0
    for r, h in ((0, 0), (3, 1), (B_ROWS - 1, H_KV - 1)):
        k, v = dequantised(olay, tiles[r, h], LENGTH)
        for j in (0, n // 2, n - 1):
            node = np.arange(LENGTH) - (LENGTH - n)
            see = (node < 0) | np.array([x >= 0 and int(mask[r, j]) >> int(x) & 1 for x in node], bool)
            qq = q[r, j, h * G:(h + 1) * G].double().numpy()
            ref = O.attention(qq, k[see], v[see], 1 / math.sqrt(128))
            worst = max([worst] + [rel_l2(out[r, j, h * G + a], ref[a]) for a in range(G)])
    print(f"largest relative error {worst:.2e}")
    assert worst <= ATTN_REL_L2


@pytest.mark.parametrize("use_pages", [False, True])
@pytest.mark.parametrize("drop,value,sink_value", [(10, 1.0, 0.1), (13, 1.0, 0.1), (10, 0.1, 0.1), (13, 0.03, 0.01),
                                                   (20, 1.0, 1e-3), (20, 0.03, 0.1), (10, 300.0, 0.0), (24, 1.0, 0.0)])
def test_sink_many_columns(drop, value, sink_value, use_pages):
    rng = np.random.default_rng(71)
    lay, olay = make_layouts("k2", 2)
    tiles, q = sink_inputs(olay, 32, 4, drop, value, sink_value, 0, rng)
    check(lay, olay, tiles, q, 32, 4, use_pages, rng)


@pytest.mark.parametrize("at", [70, 2000, LENGTH - 70])
def test_sink_many_columns_elsewhere(at):
    """A dominating token that comes after part of the tail: the reference moves."""
    rng = np.random.default_rng(72)
    lay, olay = make_layouts("k3", 3)
    tiles, q = sink_inputs(olay, 40, 8, 20, 0.1, 0.01, at, rng)
    check(lay, olay, tiles, q, 40, 8, False, rng)


@pytest.mark.parametrize("use_pages", [False, True])
@pytest.mark.parametrize("drop,value,sink_value", [(10, 1.0, 0.1), (13, 1.0, 0.1), (10, 0.1, 0.1), (13, 0.03, 0.01),
                                                   (18, 1.0, 1e-3)])
def test_sink_few_columns(drop, value, sink_value, use_pages):
    rng = np.random.default_rng(73)
    lay, olay = make_layouts("k2", 2)
    tiles, q = sink_inputs(olay, 4, 4, drop, value, sink_value, 0, rng)
    check(lay, olay, tiles, q, 4, 4, use_pages, rng)
