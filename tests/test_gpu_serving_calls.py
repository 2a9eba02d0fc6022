"""Tree attention, commit, attention mass and eviction as a server issues them: captured and
replayed, on two streams at once, with many short rows, with one workspace for calls of
different lengths.

Tolerances. A replay and a call on another stream run the same kernels on the same bytes:
equal bits. Two ways to the same attention output: 2e-3 relative L2 each, 4e-3 apart. The mass
of a row computed alone and in a batch: the logits are the same, the sums of up to 1000
weights may be split elsewhere: 1000 x 2^-24 = 6e-5 of the largest weight.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from packed_cache_decode_b200 import binding as B

from .parity_util import ATTN_REL_L2, rel_l2
from .test_gpu_bounded_cache import dequantised, dev, make_layouts, random_cache
from .test_gpu_tree import random_tree, reference, run_tree

pytestmark = pytest.mark.gpu


def queries(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16).cuda()


def test_many_short_rows_equal_multi_token_attention():
    """More units than SMs, so that a CTA goes from unit to unit; rows of every small length."""
    rng = np.random.default_rng(51)
    lay, olay = make_layouts("k2", 2)
    b, n, h_q, h_kv = 60, 8, 16, 4
    tiles = random_cache(olay, b, h_kv, 6, rng)
    lens = [int(x) for x in rng.integers(0, 385, b)]
    lens[:4] = [0, n, n + 1, 384]
    q = torch.from_numpy(rng.standard_normal((b, n, h_q, 128))).to(torch.bfloat16)
    mask = np.tile(np.array([(2 << j) - 1 for j in range(n)], np.uint64), (b, 1))
    fits = np.array([x == 0 or x >= n for x in lens])      # (a row shorter than its nodes has none)
    out = run_tree(lay, q, mask, tiles, lens, torch.float32, False, rng).cpu().double().numpy()
    ref = torch.empty(b, n, h_q, 128, device="cuda")
    ws = torch.empty(B.workspace_bytes(lay, b, h_q * n, h_kv, 384), dtype=torch.uint8, device="cuda")
    B.decode_attention_multi(lay, q.cuda(), torch.from_numpy(tiles).cuda(), dev(lens), 384, 384, ref, ws, h_kv)
    ref = ref.cpu().double().numpy()
    for r in np.flatnonzero(fits):
        if lens[r] == 0:
            assert (out[r] == 0).all()
            continue
        for x, y in zip(out[r].reshape(-1, 128), ref[r].reshape(-1, 128)):
            assert rel_l2(x, y) <= 2 * ATTN_REL_L2


@pytest.mark.parametrize("n,h_q", [(4, 8), (24, 16)])
def test_infinite_and_nan_norms_stay_in_their_branch(n, h_q):
    """Two nodes with infinite and NaN norms that only they themselves see: every other node's
    output is as if they were not there, theirs are not finite."""
    rng = np.random.default_rng(56)
    lay, olay = make_layouts("k2", 2)
    h_kv, G, length = 2, h_q // 2, 200
    tiles = random_cache(olay, 1, h_kv, 4, rng)
    code = 64 * (olay.k_record_bytes + olay.v_record_bytes)
    bad = (1, n - 1)
    for i, kn, vn in ((bad[0], np.nan, np.inf), (bad[1], np.inf, np.nan)):
        pos = length - n + i
        entry = 8 * (pos % 8) + pos % 64 // 8
        norms = tiles[0, :, pos // 64, code:].copy().view(np.float32).reshape(h_kv, -1, 64)
        norms[:, :-1, entry], norms[:, -1, entry] = kn, vn
        tiles[0, :, pos // 64, code:] = norms.reshape(h_kv, -1).view(np.uint8)
    mask = random_tree(rng, n)
    for j in range(n):
        for i in bad:
            mask[j] = (mask[j] & ~np.uint64(1 << i)) | np.uint64((1 << i) if i == j else 0)
    q = torch.from_numpy(rng.standard_normal((1, n, h_q, 128))).to(torch.bfloat16)
    o = run_tree(lay, q, mask[None], tiles, [length], torch.float32, False, rng).cpu().double().numpy()
    assert lay.status() == 0
    for h in range(h_kv):
        ref = reference(olay, tiles[0, h], q[0, :, h * G:(h + 1) * G].double().numpy(), mask, n, length)
        for j in range(n):
            for a in range(G):
                if j in bad:
                    assert not np.isfinite(o[0, j, h * G + a]).all()
                else:
                    assert rel_l2(o[0, j, h * G + a], ref[j, a]) <= ATTN_REL_L2


def test_long_rows_with_moving_maxima_are_repeatable():
    """Rows long enough for the columns' reference maxima to move now and then, one warp at a time,
    which lets a warp run ahead of its group: the same bits every time, and the reference's outputs."""
    rng = np.random.default_rng(57)
    lay, olay = make_layouts("k2", 2)
    b, n, h_q, h_kv, length = 4, 64, 64, 8, 32768
    tiles = random_cache(olay, b, h_kv, length // 64, rng)
    q = torch.from_numpy(1.4 * rng.standard_normal((b, n, h_q, 128))).to(torch.bfloat16)
    mask = np.stack([random_tree(rng, n) for _ in range(b)])
    cache, m, lens = torch.from_numpy(tiles).cuda(), torch.from_numpy(mask.view(np.int64)).cuda(), dev([length] * b)
    qd = q.cuda()
    ws = torch.empty(B.tree_workspace_bytes(lay, b, h_q, h_kv, n, length), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(12):
        out = torch.full((b, n, h_q, 128), float("nan"), device="cuda")
        B.tree_attention(lay, qd, m, cache, lens, length, length, out, ws, h_kv)
        assert torch.isfinite(out).all()
        first = out if first is None else first
        assert torch.equal(out, first)
    assert lay.status() == 0
    o, G = first.cpu().double().numpy(), h_q // h_kv
    r, h, some = b - 1, h_kv - 1, [0, 31, 63]
    k, v = dequantised(olay, tiles[r, h], length)
    for j in some:
        node = np.arange(length) - (length - n)
        see = (node < 0) | np.array([x >= 0 and int(mask[r, j]) >> int(x) & 1 for x in node], bool)
        ref = O.attention(q[r, j, h * G:(h + 1) * G].double().numpy(), k[see], v[see], 1 / math.sqrt(128))
        for a in range(G):
            assert rel_l2(o[r, j, h * G + a], ref[a]) <= ATTN_REL_L2


def test_one_workspace_for_short_and_long_calls():
    """20 query columns take one kernel up to a cache length and another above it; a workspace
    sized for the longest serves both, and they agree."""
    rng = np.random.default_rng(52)
    lay, olay = make_layouts("k2", 2)
    n, h_q, h_kv, nt = 5, 32, 8, 1600
    tiles = torch.from_numpy(random_cache(olay, 1, h_kv, 8, rng)).cuda()
    cache = torch.zeros(1, h_kv, nt, olay.tile_bytes, dtype=torch.uint8, device="cuda")
    cache[:, :, :8] = tiles
    q = queries(rng, 1, n, h_q, 128)
    mask = torch.from_numpy(random_tree(rng, n)[None].view(np.int64)).cuda()
    ws = torch.empty(B.tree_workspace_bytes(lay, 1, h_q, h_kv, n, nt * 64), dtype=torch.uint8, device="cuda")
    out = []
    for most in (500, 64 * 64, nt * 64):
        o = torch.empty(1, n, h_q, 128, device="cuda")
        B.tree_attention(lay, q, mask, cache, dev([500]), nt * 64, most, o, ws, h_kv)
        out.append(o.cpu().double().numpy().reshape(-1, 128))
    assert lay.status() == 0
    for x, y, z in zip(*out):
        assert rel_l2(y, x) <= 2 * ATTN_REL_L2 and rel_l2(z, x) <= 2 * ATTN_REL_L2


def test_mass_of_many_rows_equals_rows_alone():
    """The mass kernel of a large batch against calls of one row."""
    rng = np.random.default_rng(53)
    lay, olay = make_layouts("k3", 2)
    b, h_q, h_kv, cap = 40, 32, 8, 1024
    tiles = torch.from_numpy(random_cache(olay, b, h_kv, cap // 64, rng)).cuda()
    lens = [int(x) for x in rng.integers(1, 1001, b)]
    lens[:3] = [0, 1, 1000]
    q = queries(rng, b, h_q, 128)
    start = torch.rand(b, h_kv, cap, device="cuda")
    mass, out = start.clone(), torch.empty(b, h_q, 128, device="cuda")
    ws = torch.empty(B.mass_workspace_bytes(lay, b, h_q, h_kv, 1000), dtype=torch.uint8, device="cuda")
    B.decode_attention_mass(lay, q, tiles, dev(lens), cap, 1000, mass, out, ws, h_kv, decay=0.5)
    ws1 = torch.empty(B.mass_workspace_bytes(lay, 1, h_q, h_kv, 1000), dtype=torch.uint8, device="cuda")
    for r in range(b):
        m1, o1 = start[r:r + 1].clone(), torch.empty(1, h_q, 128, device="cuda")
        B.decode_attention_mass(lay, q[r:r + 1].contiguous(), tiles[r:r + 1].contiguous(), dev(lens[r:r + 1]), cap, 1000, m1,
                                o1, ws1, h_kv, decay=0.5)
        # (a kept value of up to 0.5 and 4 weights of up to 1: half a step of 8 for the additions)
        assert float((mass[r] - m1[0]).abs().max()) <= 4 * 6e-5 + 2.0 ** -21
        assert torch.equal(mass[r, :, lens[r]:], start[r, :, lens[r]:])
        for x, y in zip(out[r].cpu().double().numpy(), o1[0].cpu().double().numpy()):
            if lens[r]:
                assert rel_l2(x, y) <= 2 * ATTN_REL_L2
            else:
                assert not x.any() and not y.any()
    assert lay.status() == 0


def mass_and_evict(lay, h_q, h_kv, cap, keep, rng):
    """A call that keeps the mass and evicts by it, with buffers and workspace of its own."""
    ws = torch.empty(B.mass_workspace_bytes(lay, 1, h_q, h_kv, cap), dtype=torch.uint8, device="cuda")

    def call(q, cache, lens, mass, out, dst, mass_out, kept, new):
        B.decode_attention_mass(lay, q, cache, lens, cap, cap, mass, out, ws, h_kv)
        B.cache_evict(lay, cache, lens, cap, cap, mass, keep, 2, 30, dst, dst.shape[2] * 64, mass_out, kept, new, h_kv)

    def results(tile_bytes):
        return [torch.zeros(1, h_kv, cap, device="cuda"), torch.empty(1, h_q, 128, device="cuda"),
                torch.zeros(1, h_kv, -(-keep // 64), tile_bytes, dtype=torch.uint8, device="cuda"),
                torch.empty(1, h_kv, keep, device="cuda"), torch.empty(1, h_kv, keep, dtype=torch.int32, device="cuda"),
                dev([0])]

    return call, results


def test_captured_mass_and_eviction_replay():
    """Captured once, replayed on other queries, caches and lengths."""
    rng = np.random.default_rng(54)
    lay, olay = make_layouts("k2", 2)
    h_q, h_kv, cap, keep = 8, 2, 640, 150
    call, results = mass_and_evict(lay, h_q, h_kv, cap, keep, rng)
    inputs = [(queries(rng, 1, h_q, 128), torch.from_numpy(random_cache(olay, 1, h_kv, cap // 64, rng)).cuda(), dev([n]))
              for n in (640, 371, 100)]
    want = []
    for x in inputs:
        r = results(olay.tile_bytes)
        call(*x, *r)
        want.append(r)
    static, r = [t.clone() for t in inputs[0]], results(olay.tile_bytes)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*static, *r)
    for i in (1, 2, 0):
        for a, c in zip(static, inputs[i]):
            a.copy_(c)
        r[0].zero_()
        r[2].zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, c in zip(r, want[i]):
            assert torch.equal(a, c)
    assert lay.status() == 0


def test_two_streams_at_once():
    """Calls of one layout on two streams, each with its own workspace, none waiting for the other."""
    rng = np.random.default_rng(55)
    lay, olay = make_layouts("k2", 2)
    h_q, h_kv, cap, keep, n = 8, 2, 640, 150, 16
    sets = []
    for _ in range(2):
        call, results = mass_and_evict(lay, h_q, h_kv, cap, keep, rng)
        x = (queries(rng, 1, h_q, 128), torch.from_numpy(random_cache(olay, 1, h_kv, cap // 64, rng)).cuda(), dev([600]))
        tq, mask = queries(rng, 1, n, h_q, 128), torch.from_numpy(random_tree(rng, n)[None].view(np.int64)).cuda()
        ws = torch.empty(B.tree_workspace_bytes(lay, 1, h_q, h_kv, n, cap), dtype=torch.uint8, device="cuda")

        def run(x=x, call=call, results=results, tq=tq, mask=mask, ws=ws):
            r = results(olay.tile_bytes)
            o = torch.empty(1, n, h_q, 128, device="cuda")
            for _ in range(3):
                r[0].zero_()
                call(*x, *r)
                B.tree_attention(lay, tq, mask, x[1], x[2], cap, cap, o, ws, h_kv)
            return r + [o]

        sets.append((run, run()))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for s, (run, _) in zip(streams, sets):
        with torch.cuda.stream(s):
            got.append(run())
    torch.cuda.synchronize()
    for g, (_, want) in zip(got, sets):
        for a, c in zip(g, want):
            assert torch.equal(a, c)
    assert lay.status() == 0
