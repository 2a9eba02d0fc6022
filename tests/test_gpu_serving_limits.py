"""Lengths above max_seq_len in the calls whose buffers are sized by it: clipped to it (not to
the end of its tile), flagged, and nothing written past the rows.

The clipped call and the call with lengths that fit run the same kernels on the same tokens:
equal bits.
"""
import numpy as np
import pytest
import torch

from packed_cache_decode_b200 import binding as B

from .parity_util import ATTN_REL_L2, rel_l2
from .test_gpu_bounded_cache import dev, make_layouts, paged, random_cache
from .test_gpu_tree import random_tree, reference, run_tree

pytestmark = pytest.mark.gpu

GUARD = 1024   # entries behind a buffer; more than the 63 of a tile that a length may exceed the limit by


def guarded(shape, value):
    """A contiguous tensor filled with `value` and the guard entries behind it."""
    n = int(np.prod(shape))
    flat = torch.full((n + GUARD,), float(value), device="cuda")
    return flat[:n].view(*shape), flat[n:]


@pytest.mark.parametrize("use_pages", [False, True])
@pytest.mark.parametrize("b,h_kv,most", [(3, 2, 100), (1, 1, 1), (40, 8, 1000)])
def test_mass_of_longer_rows_is_clipped(b, h_kv, most, use_pages):
    """(40 rows of 1000: the sums' own kernel; else inside the merge.)"""
    rng = np.random.default_rng(61)
    lay, olay = make_layouts("k2", 2)
    nt, h_q = -(-most // 64), 4 * h_kv
    tiles = random_cache(olay, b, h_kv, nt, rng)
    cache = paged(tiles, rng) if use_pages else torch.from_numpy(tiles).cuda()
    q = torch.from_numpy(rng.standard_normal((b, h_q, 128))).to(torch.bfloat16).cuda()
    ws = torch.empty(B.mass_workspace_bytes(lay, b, h_q, h_kv, most), dtype=torch.uint8, device="cuda")
    longer = [nt * 64 - r % (nt * 64 - most) for r in range(b)]          # most + 1 .. the tile's end
    res = []
    for lens, status in (([most] * b, 0), (longer, B.STATUS_DECODE_CLAMPED)):
        mass, guard = guarded((b, h_kv, most), 0.25)
        out = torch.empty(b, h_q, 128, device="cuda")
        if use_pages:
            B.decode_attention_mass_paged(lay, q, cache, dev(lens), most, mass, out, ws, h_kv)
        else:
            B.decode_attention_mass(lay, q, cache, dev(lens), nt * 64, most, mass, out, ws, h_kv)
        assert lay.status() == status
        assert (guard == 0.25).all()
        res.append((mass, out))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    total = res[1][0].sum(-1).cpu()      # each of the 4 query heads hands out a weight of 1
    assert torch.allclose(total, torch.full_like(total, 4 + 0.25 * most), rtol=1e-4)


@pytest.mark.parametrize("use_pages", [False, True])
@pytest.mark.parametrize("n,h_q", [(3, 2), (16, 2), (40, 8)])
def test_tree_of_longer_rows_is_clipped(n, h_q, use_pages):
    """A limit inside a tile, both kernels: the nodes are the last ones before the limit."""
    rng = np.random.default_rng(62)
    lay, olay = make_layouts("k2", 2)
    most = 250
    tiles = random_cache(olay, 1, 2, 5, rng)
    q = torch.from_numpy(rng.standard_normal((1, n, h_q, 128))).to(torch.bfloat16)
    mask = random_tree(rng, n)[None]
    a = run_tree(lay, q, mask, tiles, [most], torch.float32, use_pages, rng, most=most)
    assert lay.status() == 0
    for length in (most + 1, 253, 256, 257, 300):
        b = run_tree(lay, q, mask, tiles, [length], torch.float32, use_pages, rng, most=most)
        assert lay.status() == B.STATUS_DECODE_CLAMPED
        assert torch.equal(a, b)
    G = h_q // 2
    for h in range(2):
        ref = reference(olay, tiles[0, h], q[0, :, h * G:(h + 1) * G].double().numpy(), mask[0], n, most)
        for j in range(n):
            for c in range(G):
                assert rel_l2(a[0, j, h * G + c].cpu().double().numpy(), ref[j, c]) <= ATTN_REL_L2


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("b,h_kv,h_q,most", [(3, 2, 8, 100), (1, 1, 12, 1), (2, 4, 64, 1000)])
def test_scores_of_longer_rows_are_clipped(b, h_kv, h_q, most, per_head):
    rng = np.random.default_rng(63)
    lay, olay = make_layouts("k2", 2)
    nt = -(-most // 64)
    cache = torch.from_numpy(random_cache(olay, b, h_kv, nt, rng)).cuda()
    q = torch.from_numpy(rng.standard_normal((b, h_q, 128))).to(torch.bfloat16).cuda()
    ws = torch.empty(B.workspace_bytes(lay, b, h_q, h_kv, most), dtype=torch.uint8, device="cuda")
    owner = B.LayoutSet([lay] * h_kv) if per_head else lay
    longer = [nt * 64 - r for r in range(b)]                             # most + 1 .. the tile's end
    res = []
    for lens, status in (([most] * b, 0), (longer, B.STATUS_DECODE_CLAMPED)):
        scores, guard = guarded((b, h_q, most), 0.25)
        if per_head:
            B.decode_scores_heads(owner, q, cache, dev(lens), nt * 64, most, scores, ws)
        else:
            B.decode_scores(lay, q, cache, dev(lens), nt * 64, most, scores, ws, h_kv)
        assert owner.status() == status
        assert (guard == 0.25).all()
        res.append(scores)
    assert torch.equal(*res)
