"""Tree attention next to tokens of very large (finite) norms: nodes that some queries do not
see must not cost those queries' other tokens any bits, and a large key that everyone sees none
of the small ones' either. Both kernels.

Tolerance: the library's 2e-3 relative L2 (fp32 outputs). In the kernel for many columns a token
keeps 2^-20 of its logits down to 2^-15 of the largest key norm among its 32 tokens where every
query sees them; further down the step of 2^-24 at 2^11 leaves 2^-35 of that norm's logits: at
2^-16 as below 2^-19 of its own (of a size below 32: 1e-4 of a weight).
"""
import numpy as np
import pytest
import torch

from packed_cache_decode_b200 import binding as B

from .parity_util import ATTN_REL_L2, rel_l2
from .test_gpu_bounded_cache import dequantised, make_layouts, random_cache
from .test_gpu_tree import random_tree, reference, run_tree

pytestmark = pytest.mark.gpu


def set_norms(olay, tiles, pos, key=None, value=None):
    """Multiplies token pos's key norms by `key` and sets its value norm to `value`."""
    code = 64 * (olay.k_record_bytes + olay.v_record_bytes)
    h_kv = tiles.shape[1]
    entry = 8 * (pos % 8) + pos % 64 // 8
    norms = tiles[0, :, pos // 64, code:].copy().view(np.float32).reshape(h_kv, -1, 64)
    if key is not None:
        norms[:, :-1, entry] *= np.float32(key)
    if value is not None:
        norms[:, -1, entry] = value
    tiles[0, :, pos // 64, code:] = norms.reshape(h_kv, -1).view(np.uint8)


@pytest.mark.parametrize("length", [200, 256, 1000])
@pytest.mark.parametrize("key,value", [(1e5, None), (1e9, 1e9), (1e25, 1e30)])
@pytest.mark.parametrize("n,h_q", [(4, 8), (24, 16), (64, 16)])
def test_large_norms_of_unseen_nodes(n, h_q, key, value, length):
    rng = np.random.default_rng(81)
    lay, olay = make_layouts("k2", 2)
    h_kv, G = 2, h_q // 2
    tiles = random_cache(olay, 1, h_kv, -(-length // 64), rng)
    bad = sorted({1, n // 2, n - 1})
    for i in bad:
        set_norms(olay, tiles, length - n + i, key, value)
    mask = random_tree(rng, n)
    for j in range(n):
        for i in bad:
            mask[j] = (mask[j] & ~np.uint64(1 << i)) | np.uint64((1 << i) if i == j else 0)
    q = torch.from_numpy(rng.standard_normal((1, n, h_q, 128))).to(torch.bfloat16)
    o = run_tree(lay, q, mask[None], tiles, [length], torch.float32, False, rng).cpu().double().numpy()
    assert lay.status() == 0
    worst = 0.0
    for h in range(h_kv):
        ref = reference(olay, tiles[0, h], q[0, :, h * G:(h + 1) * G].double().numpy(), mask, n, length)
        for j in range(n):
            if j not in bad:
                worst = max([worst] + [rel_l2(o[0, j, h * G + a], ref[j, a]) for a in range(G)])
    print(f"largest relative error {worst:.2e}")
    assert worst <= ATTN_REL_L2


@pytest.mark.parametrize("n,h_q", [(4, 8), (24, 16)])
def test_large_keys_that_all_queries_see(n, h_q):
    """A key 2^16 times the others' in the prefix, in a tile without nodes: queries against it see
    the other tokens alone."""
    rng = np.random.default_rng(82)
    lay, olay = make_layouts("k2", 2)
    h_kv, G, length, at = 2, h_q // 2, 300, 77
    tiles = random_cache(olay, 1, h_kv, 5, rng)
    set_norms(olay, tiles, at, 2.0 ** 16)
    q = rng.standard_normal((1, n, h_kv, G, 128))
    for h in range(h_kv):
        k, _ = dequantised(olay, tiles[0, h], length)
        dot = q[0, :, h] @ k[at]
        q[0, :, h] *= np.where(dot > 0, -1.0, 1.0)[..., None]
    q = torch.from_numpy(q.reshape(1, n, h_q, 128)).float()
    mask = random_tree(rng, n)
    o = run_tree(lay, q, mask[None], tiles, [length], torch.float32, False, rng).cpu().double().numpy()
    assert lay.status() == 0
    for h in range(h_kv):
        ref = reference(olay, tiles[0, h], q[0, :, h * G:(h + 1) * G].double().numpy(), mask, n, length)
        for j in range(n):
            for a in range(G):
                assert rel_l2(o[0, j, h * G + a], ref[j, a]) <= ATTN_REL_L2
