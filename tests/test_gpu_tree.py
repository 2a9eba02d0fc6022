"""Drafted trees through the C ABI: attention under ancestor masks against a plain fp64
reference, and the commit of the accepted path against the oracle's pack of the same tokens.

Tolerance of the attention: the library's 2e-3 relative L2 per (node, head) plus half a step
of the output's type. The commit moves bits: exact.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from packed_cache_decode_b200 import binding as B

from .parity_util import ATTN_REL_L2, rel_l2
from .test_gpu_bounded_cache import HALF_STEP, dequantised, dev, make_layouts, paged, random_cache

pytestmark = pytest.mark.gpu


def random_tree(rng, n, roots=0.2):
    """Ancestor masks (uint64, own bit set) of a random forest, parents before children."""
    mask = np.zeros(n, np.uint64)
    for i in range(n):
        p = -1 if i == 0 or rng.random() < roots else int(rng.integers(0, i))
        mask[i] = (mask[p] if p >= 0 else np.uint64(0)) | np.uint64(1 << i)
    return mask


def reference(olay, tiles, q, mask, n, length):
    """q [n, G, 128] of one KV head; mask [n] words; the nodes are the last n of `length` tokens."""
    k, v = dequantised(olay, tiles, length)
    pos = np.arange(length)
    out = np.zeros_like(q)
    for j in range(n):
        node = pos - (length - n)
        bit = (int(mask[j]) >> np.clip(node, 0, 63).astype(object)) & 1
        see = (node < 0) | (bit.astype(bool) & (node >= 0))
        if see.any():
            out[j] = O.attention(q[j], k[see], v[see], 1 / math.sqrt(128))
    return out


def run_tree(lay, q, mask, tiles, lens, ot, use_pages, rng, n_nodes=None, most=None, fill=float("nan")):
    b, n, h_q, _ = q.shape
    h_kv, nt = tiles.shape[1], tiles.shape[2]
    most = max(lens) if most is None else most
    out = torch.full(q.shape, fill, dtype=ot, device="cuda")
    ws = torch.empty(B.tree_workspace_bytes(lay, b, h_q, h_kv, n, most), dtype=torch.uint8, device="cuda")
    m = torch.from_numpy(np.ascontiguousarray(mask).view(np.int64)).cuda()
    nn = None if n_nodes is None else dev(n_nodes)
    if use_pages:
        B.tree_attention_paged(lay, q.cuda(), m, paged(tiles, rng), dev(lens), most, out, ws, h_kv, n_nodes=nn)
    else:
        B.tree_attention(lay, q.cuda(), m, torch.from_numpy(tiles).cuda(), dev(lens), nt * 64, most, out, ws, h_kv,
                         n_nodes=nn)
    torch.cuda.synchronize()
    return out


TREE_CASES = [  # mix, v_rate, fp16 norms, h_q, h_kv, nodes, lens, q type, out type, paged
    ("k2", 2, False, 8, 2, 1, [1, 64, 200], torch.bfloat16, torch.bfloat16, False),
    ("k2", 2, False, 8, 2, 6, [6, 70, 333], torch.bfloat16, torch.float32, True),
    ("k3", 3, True, 14, 2, 13, [13, 77, 1000, 128], torch.float16, torch.float16, False),
    ("k4", 4, False, 4, 4, 33, [33, 64, 700], torch.float32, torch.float32, True),
    ("k1", 1, True, 5, 1, 64, [64, 129, 65], torch.bfloat16, torch.bfloat16, False),
    ("holes", 2, False, 16, 2, 17, [100, 18], torch.float16, torch.bfloat16, False),
    ("k2", 3, True, 32, 1, 64, [900], torch.bfloat16, torch.bfloat16, True),
    ("k3", 4, False, 16, 2, 25, [4000, 2049], torch.bfloat16, torch.float32, False),
    ("k2", 2, False, 64, 8, 64, [1500], torch.bfloat16, torch.bfloat16, False),
]


@pytest.mark.parametrize("case", TREE_CASES, ids=lambda c: f"{c[0]}v{c[1]}_{c[3]}q{c[4]}_n{c[5]}")
def test_tree_attention_matches_reference(case):
    mix, vr, fp16, h_q, h_kv, n, lens, qt, ot, use_pages = case
    rng = np.random.default_rng(21)
    lay, olay = make_layouts(mix, vr, fp16)
    b, G = len(lens), h_q // h_kv
    nt = -(-max(lens) // 64) + (n % 2)
    tiles = random_cache(olay, b, h_kv, nt, rng)
    q = torch.from_numpy(rng.standard_normal((b, n, h_q, 128))).to(qt)
    mask = np.stack([random_tree(rng, n) for _ in range(b)])
    o = run_tree(lay, q, mask, tiles, lens, ot, use_pages, rng).cpu().double().numpy()
    assert lay.status() == 0
    for r in range(b):
        for h in range(h_kv):
            ref = reference(olay, tiles[r, h], q[r, :, h * G:(h + 1) * G].double().numpy(), mask[r], n, lens[r])
            for j in range(n):
                for a in range(G):
                    assert rel_l2(o[r, j, h * G + a], ref[j, a]) <= ATTN_REL_L2 + HALF_STEP[ot], (r, h, j, a)


@pytest.mark.parametrize("n,h_q", [(5, 4), (40, 16)])
def test_empty_rows_wild_masks_and_node_counts(n, h_q):
    """Masks without the node's own bit, masks that leave nothing, bits past the row's nodes
    (ignored), rows with fewer nodes (the others are not written), rows that do not fit."""
    rng = np.random.default_rng(22)
    lay, olay = make_layouts("k2", 2)
    lens, nodes = [n, 200, 130, 3, 150, 10], [n, n - 2, 0, n, n + 1, -1]
    b, h_kv = len(lens), 2
    G = h_q // h_kv
    tiles = random_cache(olay, b, h_kv, 4, rng)
    q = torch.from_numpy(rng.standard_normal((b, n, h_q, 128))).to(torch.bfloat16)
    mask = rng.integers(0, 2 ** 64, (b, n), dtype=np.uint64)
    mask[0, ::2] = 0                                     # row 0 is all nodes: these queries see nothing
    mask[1, :2] = 0                                      # these see the prefix alone
    o = run_tree(lay, q, mask, tiles, lens, torch.bfloat16, False, rng, n_nodes=nodes).cpu().double().numpy()
    assert lay.status() == B.STATUS_BAD_TREE
    for r in range(b):
        if r >= 3:                                       # 3 < n tokens, too many nodes, a negative count
            assert (o[r] == 0).all()
            continue
        m = nodes[r]
        assert np.isnan(o[r, m:]).all()
        for h in range(h_kv):
            qq = q[r, :m, h * G:(h + 1) * G].double().numpy()
            ref = reference(olay, tiles[r, h], qq, mask[r], m, lens[r])
            for j in range(m):
                for a in range(G):
                    if r == 0 and int(mask[0, j]) & ((1 << n) - 1) == 0:
                        assert (o[r, j, h * G + a] == 0).all()
                    else:
                        assert rel_l2(o[r, j, h * G + a], ref[j, a]) <= ATTN_REL_L2 + HALF_STEP[torch.bfloat16]


def test_causal_mask_equals_multi_token_attention():
    rng = np.random.default_rng(23)
    lay, olay = make_layouts("k3", 3)
    for n, h_q in ((4, 8), (16, 4)):
        tiles = random_cache(olay, 2, 2, 9, rng)
        q = torch.from_numpy(rng.standard_normal((2, n, h_q, 128))).to(torch.bfloat16)
        mask = np.tile(np.array([(2 << j) - 1 for j in range(n)], np.uint64), (2, 1))
        lens = [500, 321]
        out = run_tree(lay, q, mask, tiles, lens, torch.float32, False, rng)
        ref = torch.empty_like(out)
        ws = torch.empty(B.workspace_bytes(lay, 2, h_q * n, 2, 500), dtype=torch.uint8, device="cuda")
        B.decode_attention_multi(lay, q.cuda(), torch.from_numpy(tiles).cuda(), dev(lens), 576, 500, ref, ws, 2)
        for x, y in zip(out.cpu().double().numpy().reshape(-1, 128), ref.cpu().double().numpy().reshape(-1, 128)):
            assert rel_l2(x, y) <= 2 * ATTN_REL_L2


def test_lengths_past_the_limit_are_clamped():
    rng = np.random.default_rng(24)
    lay, olay = make_layouts("k2", 2)
    for n, h_q in ((3, 2), (40, 8)):
        tiles = random_cache(olay, 1, 2, 5, rng)
        q = torch.from_numpy(rng.standard_normal((1, n, h_q, 128))).to(torch.bfloat16)
        mask = random_tree(rng, n)[None]
        a = run_tree(lay, q, mask, tiles, [256], torch.float32, False, rng, most=256)
        assert lay.status() == 0
        b = run_tree(lay, q, mask, tiles, [300], torch.float32, False, rng, most=256)
        assert lay.status() == B.STATUS_DECODE_CLAMPED
        assert torch.equal(a, b)


@pytest.mark.parametrize("n,h_q", [(4, 8), (32, 16)])
def test_bytes_past_the_row_do_not_matter(n, h_q):
    rng = np.random.default_rng(25)
    lay, olay = make_layouts("k2", 2)
    tiles = random_cache(olay, 1, 2, 4, rng)
    dirty = tiles.copy()
    code = 64 * (olay.k_record_bytes + olay.v_record_bytes)
    tok = np.arange(64)
    norms = dirty[0, :, 2, code:].copy().view(np.float32).reshape(2, -1, 64)
    norms[:, :, (8 * (tok % 8) + tok // 8)[150 - 128:]] = np.nan
    dirty[0, :, 2, code:] = norms.reshape(2, -1).view(np.uint8)
    dirty[0, :, 3, code:] = 0xFF
    q = torch.from_numpy(rng.standard_normal((1, n, h_q, 128))).to(torch.bfloat16)
    mask = random_tree(rng, n)[None]
    a, b = (run_tree(lay, q, mask, t, [150], torch.float32, False, rng, most=256) for t in (tiles, dirty))
    assert torch.equal(a, b) and torch.isfinite(a).all()


def test_missing_page_is_left_out():
    rng = np.random.default_rng(26)
    lay, olay = make_layouts("k2", 2)
    for n, h_q in ((3, 4), (33, 16)):
        tiles = random_cache(olay, 1, 2, 6, rng)
        pc = paged(tiles, rng)
        pc.table[0, 2] = -7
        q = torch.from_numpy(rng.standard_normal((1, n, h_q, 128))).to(torch.bfloat16)
        mask = random_tree(rng, n)
        out = torch.empty(1, n, h_q, 128, device="cuda")
        ws = torch.empty(B.tree_workspace_bytes(lay, 1, h_q, 2, n, 384), dtype=torch.uint8, device="cuda")
        B.tree_attention_paged(lay, q.cuda(), torch.from_numpy(mask[None].view(np.int64)).cuda(), pc, dev([384]), 384, out,
                               ws, 2)
        assert lay.status() == B.STATUS_BAD_PAGE
        G = h_q // 2
        keep = [0, 1, 3, 4, 5]
        for h in range(2):
            ref = reference(olay, tiles[0, h][keep], q[0, :, h * G:(h + 1) * G].double().numpy(), mask, n, 320)
            for j in range(n):
                for a in range(G):
                    assert rel_l2(out[0, j, h * G + a].cpu().double().numpy(), ref[j, a]) <= ATTN_REL_L2


# ------------------------------------------------------------------ commit
COMMIT_CASES = [  # mix, v_rate, fp16, h_kv, nodes, lens, paged
    ("k2", 2, False, 2, 6, [6, 64, 67, 130], False),
    ("k3", 3, True, 1, 64, [64, 65, 127, 128, 200], True),
    ("k4", 4, False, 3, 33, [100, 64], False),
    ("k1", 1, True, 2, 1, [1, 129], True),
    ("holes", 2, False, 1, 50, [300, 75], False),
    ("k3", 1, False, 1, 64, [321], False),
]


def expected_commit(olay, tiles, length, n, path):
    u = O.unpack(olay, tiles.reshape(-1), tiles.shape[0] * 64)
    idx = np.arange(tiles.shape[0] * 64)
    idx[length - n:length - n + len(path)] = length - n + np.asarray(path, int)
    return O.pack(olay, {k: x[idx] for k, x in u.items()}, len(idx)).reshape(tiles.shape)


def run_commit(lay, path, count, n_q, tiles, lens, use_pages, rng, n_nodes=None):
    b, h_kv = tiles.shape[:2]
    new = torch.full((b,), -9, dtype=torch.int32, device="cuda")
    nn = None if n_nodes is None else dev(n_nodes)
    if use_pages:
        pc = paged(tiles, rng)
        B.tree_commit_paged(lay, dev(path), dev(count), n_q, pc, dev(lens), new, h_kv, n_nodes=nn)
        got = pc.pool.view(-1, h_kv, tiles.shape[3])[pc.table.long()].transpose(1, 2).cpu().numpy()
    else:
        c = torch.from_numpy(tiles).cuda()
        B.tree_commit(lay, dev(path), dev(count), n_q, c, dev(lens), new, tiles.shape[2] * 64, h_kv, n_nodes=nn)
        got = c.cpu().numpy()
    return got, new.cpu().numpy()


@pytest.mark.parametrize("case", COMMIT_CASES, ids=lambda c: f"{c[0]}v{c[1]}_n{c[4]}")
@pytest.mark.parametrize("kind", ["ascending", "any"])
def test_commit_matches_reference(case, kind):
    mix, vr, fp16, h_kv, n, lens, use_pages = case
    rng = np.random.default_rng(31)
    lay, olay = make_layouts(mix, vr, fp16)
    b = len(lens)
    tiles = random_cache(olay, b, h_kv, -(-max(lens) // 64) + 1, rng)
    path, count = np.full((b, n + 2), 10 ** 6, np.int32), np.zeros(b, np.int32)
    for r in range(b):
        count[r] = rng.integers(0, n + 1) if r else n
        pick = rng.permutation(n)[:count[r]] if kind == "ascending" else rng.integers(0, n, count[r])
        path[r, :count[r]] = np.sort(pick) if kind == "ascending" else pick   # any order, the same node twice
    got, new = run_commit(lay, path, count, n, tiles, lens, use_pages, rng)
    assert lay.status() == 0
    np.testing.assert_array_equal(new, np.asarray(lens) - n + count)
    for r in range(b):
        for h in range(h_kv):
            np.testing.assert_array_equal(got[r, h], expected_commit(olay, tiles[r, h], lens[r], n, path[r, :count[r]]))


def test_commit_rows_that_do_not_fit_keep_their_tokens():
    rng = np.random.default_rng(32)
    lay, olay = make_layouts("k2", 2)
    lens = [100, 100, 100, 3, 129, 100, 100]
    nodes = [8, 8, 9, 8, 8, -1, 5]
    count = [2, 9, 2, 2, 2, 0, 3]
    path = np.tile(np.array([1, 3, 5, 6, 7, 0, 0, 0], np.int32), (7, 1))
    path[0, 1] = 8                                       # not a node; 9 > 8 nodes; 3 < 8 tokens; past the capacity
    tiles = random_cache(olay, 7, 2, 2, rng)
    got, new = run_commit(lay, path, count, 8, tiles, lens, False, rng, n_nodes=nodes)
    assert lay.status() == B.STATUS_BAD_TREE
    np.testing.assert_array_equal(new, lens)             # row 6 (5 nodes, path 1 3 5: no node 5) included
    np.testing.assert_array_equal(got, tiles)
    path[6, 2] = 4
    got, new = run_commit(lay, path[6:], count[6:], 8, tiles[6:], lens[6:], False, rng, n_nodes=nodes[6:])
    assert lay.status() == 0 and new[0] == 98
    np.testing.assert_array_equal(got[0, 0], expected_commit(olay, tiles[6, 0], 100, 5, [1, 3, 4]))


def test_commit_missing_page():
    rng = np.random.default_rng(33)
    lay, olay = make_layouts("k2", 2)
    tiles = random_cache(olay, 1, 2, 3, rng)
    pc = paged(tiles, rng)
    pc.table[0, 1] = 10 ** 6
    before = pc.pool.clone()
    new = dev([0])
    B.tree_commit_paged(lay, dev([[1, 2, 3, 0, 0, 0, 0, 0, 0, 0]]), dev([3]), 10, pc, dev([66]), new, 2)
    assert lay.status() == B.STATUS_BAD_PAGE and int(new[0]) == 59
    assert torch.equal(pc.pool, before)


# ------------------------------------------------------------------ together
def test_draft_verify_commit_decode_run():
    """Speculative decoding as a server does it: append a drafted tree, attend it, commit the
    accepted path, append the next token and decode."""
    rng = np.random.default_rng(41)
    lay, olay = make_layouts("k2", 2)
    b, h_q, h_kv, n0, n, cap = 2, 16, 2, 120, 20, 256
    G = h_q // h_kv
    kv = torch.from_numpy(rng.standard_normal((2, b, 400, h_kv, 128))).to(torch.bfloat16).cuda()
    cache = torch.zeros(lay.cache_bytes(b, h_kv, cap), dtype=torch.uint8, device="cuda")
    lens = dev([0, 0])
    B.encode_append(lay, kv[0, :, :n0].contiguous(), kv[1, :, :n0].contiguous(), lens, cache, cap)
    lens = dev([n0, n0])
    ws = torch.empty(B.tree_workspace_bytes(lay, b, h_q, h_kv, n, cap), dtype=torch.uint8, device="cuda")
    for step in range(3):
        a = 130 + 40 * step
        B.encode_append(lay, kv[0, :, a:a + n].contiguous(), kv[1, :, a:a + n].contiguous(), lens, cache, cap)
        mask = np.stack([random_tree(rng, n) for _ in range(b)])
        q = torch.from_numpy(rng.standard_normal((b, n, h_q, 128))).to(torch.bfloat16).cuda()
        out = torch.empty(b, n, h_q, 128, device="cuda")
        B.tree_attention(lay, q, torch.from_numpy(mask.view(np.int64)).cuda(), cache, lens + n, cap, cap, out, ws, h_kv)
        host = cache.cpu().numpy().reshape(b, h_kv, cap // 64, -1)
        for r in range(b):
            L = int(lens[r]) + n
            ref = reference(olay, host[r, 1], q[r, :, G:].cpu().double().numpy(), mask[r], n, L)
            for j in range(n):
                assert rel_l2(out[r, j, G:].cpu().double().numpy(), ref[j]) <= ATTN_REL_L2
        path, count = np.zeros((b, n), np.int32), np.zeros(b, np.int32)
        for r in range(b):
            leaf = int(rng.integers(0, n))
            line = [i for i in range(n) if int(mask[r, leaf]) >> i & 1]
            path[r, :len(line)], count[r] = line, len(line)
        new = torch.empty_like(lens)
        B.tree_commit(lay, dev(path), dev(count), n, cache, lens + n, new, cap, h_kv)
        for r in range(b):
            for h in range(h_kv):
                want = expected_commit(olay, host[r, h], int(lens[r]) + n, n, path[r, :count[r]])
                np.testing.assert_array_equal(cache.cpu().numpy().reshape(b, h_kv, cap // 64, -1)[r, h], want)
        lens = new
    q1 = torch.from_numpy(rng.standard_normal((b, h_q, 128))).to(torch.bfloat16).cuda()
    o1 = torch.empty(b, h_q, 128, device="cuda")
    dws = torch.empty(B.workspace_bytes(lay, b, h_q, h_kv, cap), dtype=torch.uint8, device="cuda")
    B.decode_step(lay, kv[0, :, 390:391].contiguous(), kv[1, :, 390:391].contiguous(), q1, cache, lens, cap, cap, o1, dws)
    assert lay.status() == 0
    host = cache.cpu().numpy().reshape(b, h_kv, cap // 64, -1)
    for r in range(b):
        for h in range(h_kv):
            k, v = dequantised(olay, host[r, h], int(lens[r]) + 1)
            ref = O.attention(q1[r, h * G:(h + 1) * G].cpu().double().numpy(), k, v, 1 / math.sqrt(128))
            for a in range(G):
                assert rel_l2(o1[r, h * G + a].cpu().double().numpy(), ref[a]) <= ATTN_REL_L2


def test_captured_calls_replay():
    """Attention and commit captured into one CUDA graph and replayed on new inputs."""
    rng = np.random.default_rng(42)
    lay, olay = make_layouts("k2", 2)
    for n, h_q in ((4, 8), (24, 16)):
        tiles = [torch.from_numpy(random_cache(olay, 1, 2, 4, rng)).cuda() for _ in range(2)]
        q = [torch.from_numpy(rng.standard_normal((1, n, h_q, 128))).to(torch.bfloat16).cuda() for _ in range(2)]
        mask = torch.from_numpy(random_tree(rng, n)[None].view(np.int64)).cuda()
        path, count = dev([list(range(1, n)) + [0]]), dev([n - 1])
        ws = torch.empty(B.tree_workspace_bytes(lay, 1, h_q, 2, n, 256), dtype=torch.uint8, device="cuda")

        def call(x, c, lens, out, new):
            B.tree_attention(lay, x, mask, c, lens, 256, 256, out, ws, 2)
            B.tree_commit(lay, path, count, n, c, lens, new, 256, 2)

        lens = [dev([200]), dev([131])]
        want = []
        for i in range(2):
            out, new, c = torch.empty(1, n, h_q, 128, device="cuda"), dev([0]), tiles[i].clone()
            call(q[i], c, lens[i], out, new)
            want.append((out, new, c))
        sq, sc, sl = q[0].clone(), tiles[0].clone(), lens[0].clone()
        out, new = torch.empty(1, n, h_q, 128, device="cuda"), dev([0])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(sq, sc, sl, out, new)
        for i in (1, 0):
            sq.copy_(q[i])
            sc.copy_(tiles[i])
            sl.copy_(lens[i])
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i][0]) and torch.equal(new, want[i][1]) and torch.equal(sc, want[i][2])
    assert lay.status() == 0
