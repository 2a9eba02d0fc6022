"""Attention mass and eviction through the C ABI, against plain fp64 / integer references.

Caches are filled with random code bytes (every bit pattern is a code) and random norms, so
the references see exactly what the kernels read.

Tolerances. Mass (fp32): a weight is 2^(s - M) / l with s the base-2 logit, so its relative
error is ln 2 times the error of s. The matrix products truncate: each of the up to 16 key
products of a group (8 quad pairs, hi and lo parts of q', two half-steps each) may lose one
step, 2^-23, of the running sum, whose size is at most |s| plus the rate-1 correction of the
same order: 32 x 2^-23 x 20 = 7.6e-5 in the worst case at |s| + correction = 20 (the largest
of these inputs), 5.3e-5 of a weight. The rotated query (hi + lo: 2^-22), the centroids
(2.3e-7) and the exponentials add 5e-6. 6e-5 relative to the largest weight is allowed; the
relative 2-norm, where truncations average, is held to 1e-5.
Outputs as every
attention output of the library: 2e-3 relative L2 per head, plus half a step of the output's
type. Eviction moves bits: exact.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from packed_cache_decode_b200 import binding as B

from .parity_util import ATTN_REL_L2, rel_l2

pytestmark = pytest.mark.gpu

MASS_REL = 6e-5
MIXES = {"k2": (27, 22, 3, 12), "k3": (11, 13, 5, 35), "k4": (0, 0, 0, 64), "k1": (64, 0, 0, 0),
         "holes": (20, 20, 8, 4)}      # 12 uncoded blocks


def make_layouts(mix, v_rate, fp16=False, seed=3):
    rates = np.random.default_rng(seed).permutation(
        np.concatenate([np.repeat([1, 2, 3, 4], MIXES[mix]), np.zeros(64 - sum(MIXES[mix]), int)])).astype(int)
    return (B.Layout(rates, v_rate, seed, norm_fp16=fp16).upload(0),
            O.make_layout(rates, v_rate, seed, norm_fp16=fp16))


def random_cache(olay, batch, h_kv, n_tiles, rng):
    """[batch, h_kv, n_tiles, tile_bytes]: random codes, norms of the size real ones have."""
    code = 64 * (olay.k_record_bytes + olay.v_record_bytes)
    out = rng.integers(0, 256, (batch, h_kv, n_tiles, olay.tile_bytes), dtype=np.uint8)
    sizes = [len(c) for _, c in olay.groups] + [128]
    norms = np.stack([math.sqrt(d) * rng.uniform(0.3, 2.0, (batch, h_kv, n_tiles, 64)) for d in sizes], 3)
    out[..., code:] = norms.astype(np.float16 if olay.norm_fp16 else np.float32).reshape(
        batch, h_kv, n_tiles, -1).view(np.uint8)
    return out


def paged(tiles, rng, spare=3):
    b, h, n, tb = tiles.shape
    perm = rng.permutation(b * n + spare)[:b * n].astype(np.int32)
    pool = np.zeros((b * n + spare, h, tb), np.uint8)
    pool[perm] = tiles.transpose(0, 2, 1, 3).reshape(b * n, h, tb)
    return B.PagedCache(torch.from_numpy(pool).cuda().view(-1), torch.from_numpy(perm.reshape(b, n)).cuda())


def dequantised(olay, tiles, n):
    u = O.unpack(olay, tiles.reshape(-1), n)
    return O.reconstruct(olay, u["k_codes"], u["k_norms"], u["v_codes"], u["v_norm"])


def dev(x, dt=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to("cuda", dt)


HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}

MASS_CASES = [  # mix, v_rate, fp16 norms, h_q, h_kv, lens, q type, out type, decay, paged
    ("k2", 2, False, 8, 2, [1, 63, 64, 65], torch.bfloat16, torch.bfloat16, 1.0, False),
    ("k3", 3, True, 14, 2, [0, 700, 333], torch.float16, torch.float16, 0.9, True),
    ("k4", 4, False, 8, 1, [2500, 1, 0], torch.float32, torch.float32, 0.0, False),
    ("k1", 1, True, 20, 1, [129, 640], torch.bfloat16, torch.float32, 1.0, True),
    ("holes", 2, False, 32, 1, [257], torch.float16, torch.bfloat16, 1.0, False),
]


@pytest.mark.parametrize("case", MASS_CASES, ids=lambda c: f"{c[0]}v{c[1]}_{c[3]}q{c[4]}")
def test_mass_and_output_match_reference(case):
    mix, vr, fp16, h_q, h_kv, lens, qt, ot, decay, use_pages = case
    rng = np.random.default_rng(5)
    lay, olay = make_layouts(mix, vr, fp16)
    b, G, most = len(lens), h_q // h_kv, max(lens)
    nt = -(-max(most, 1) // 64) + 1
    tiles = random_cache(olay, b, h_kv, nt, rng)
    q = torch.from_numpy(rng.standard_normal((b, h_q, 128))).to(qt)
    ld = most + 7                                         # not a multiple of 4
    mass0 = rng.uniform(0, 1, (b, h_kv, ld)).astype(np.float32)
    mass, out = torch.from_numpy(mass0).cuda(), torch.full((b, h_q, 128), float("nan"), dtype=ot, device="cuda")
    ws = torch.empty(B.mass_workspace_bytes(lay, b, h_q, h_kv, most), dtype=torch.uint8, device="cuda")
    if use_pages:
        B.decode_attention_mass_paged(lay, q.cuda(), paged(tiles, rng), dev(lens), most, mass, out, ws, h_kv, decay)
    else:
        B.decode_attention_mass(lay, q.cuda(), torch.from_numpy(tiles).cuda(), dev(lens), nt * 64, most, mass, out, ws,
                                h_kv, decay)
    assert lay.status() == 0
    got, o = mass.cpu().double().numpy(), out.cpu().double().numpy()
    for r in range(b):
        for h in range(h_kv):
            n = lens[r]
            np.testing.assert_array_equal(got[r, h, n:], mass0[r, h, n:])
            qq = q[r, h * G:(h + 1) * G].double().numpy()
            if n == 0:
                assert (o[r, h * G:(h + 1) * G] == 0).all()
                continue
            k, v = dequantised(olay, tiles[r, h], n)
            s = qq @ k.T / math.sqrt(128)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            w = p.sum(0)
            err = np.abs(got[r, h, :n] - (decay * mass0[r, h, :n].astype(np.float64) + w))
            # fp32 rounding of the sum itself: half a step of the result
            assert np.linalg.norm(err) <= 1e-5 * np.linalg.norm(decay * mass0[r, h, :n] + w)
            assert (err <= MASS_REL * w.max() + 2.0 ** -23 * (mass0[r, h, :n] + w)).all(), err.max()
            for a in range(G):
                ref = p[a] @ v
                assert rel_l2(o[r, h * G + a], ref) <= ATTN_REL_L2 + HALF_STEP[ot]


def test_mass_steps_add_up():
    """Two steps: the second adds to the first; the outputs are decode_attention's."""
    rng = np.random.default_rng(6)
    lay, olay = make_layouts("k2", 2)
    b, h_q, h_kv, n = 2, 16, 4, 400
    tiles = torch.from_numpy(random_cache(olay, b, h_kv, 7, rng)).cuda()
    lens = dev([n, 399])
    q = torch.from_numpy(rng.standard_normal((2, b, h_q, 128))).to(torch.bfloat16).cuda()
    ws = torch.empty(B.mass_workspace_bytes(lay, b, h_q, h_kv, n), dtype=torch.uint8, device="cuda")
    mass, one = (torch.zeros(b, h_kv, 448, device="cuda") for _ in range(2))
    out, ref = (torch.empty(b, h_q, 128, device="cuda") for _ in range(2))
    for i in range(2):
        B.decode_attention_mass(lay, q[i], tiles, lens, 448, n, mass, out, ws, h_kv)
        B.decode_attention(lay, q[i], tiles, lens, 448, n, ref, ws, h_kv)
        for x, y in zip(out.cpu().double().numpy().reshape(-1, 128), ref.cpu().double().numpy().reshape(-1, 128)):
            assert rel_l2(x, y) <= 2 * ATTN_REL_L2
    for i in range(2):
        B.decode_attention_mass(lay, q[i], tiles, lens, 448, n, one, out, ws, h_kv)
    assert torch.equal(one, mass)          # the same calls give the same bits
    total = mass.sum(-1).cpu()             # every step and query head hands out a weight of 1
    assert torch.allclose(total, torch.full_like(total, 2.0 * h_q / h_kv), rtol=1e-5)


def test_mass_unseen_bytes_and_missing_page():
    """NaN norms past the row's end do not reach the sums; a tile without a page gets no
    weight and is flagged."""
    rng = np.random.default_rng(7)
    lay, olay = make_layouts("k2", 2)
    tiles = random_cache(olay, 1, 2, 4, rng)
    dirty = tiles.copy()
    code = 64 * (olay.k_record_bytes + olay.v_record_bytes)
    nan = np.full((olay.n_kgroups + 1, 64), np.nan, np.float32)
    tok = np.arange(64)
    entry = 8 * (tok % 8) + tok // 8
    norms = dirty[0, :, 2, code:].copy().view(np.float32).reshape(2, -1, 64)
    norms[:, :, entry[150 - 128:]] = np.nan                # tokens 150 .. 191
    dirty[0, :, 2, code:] = norms.reshape(2, -1).view(np.uint8)
    dirty[0, :, 3, code:] = nan.reshape(-1).view(np.uint8)
    q = torch.from_numpy(rng.standard_normal((1, 8, 128))).to(torch.bfloat16).cuda()
    ws = torch.empty(B.mass_workspace_bytes(lay, 1, 8, 2, 256), dtype=torch.uint8, device="cuda")
    res = []
    for t in (tiles, dirty):
        mass, out = torch.zeros(1, 2, 256, device="cuda"), torch.empty(1, 8, 128, device="cuda")
        B.decode_attention_mass(lay, q, torch.from_numpy(t).cuda(), dev([150]), 256, 256, mass, out, ws, 2)
        res.append((mass, out))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert lay.status() == 0
    pc = paged(tiles, rng)
    pc.table[0, 1] = 10 ** 6
    mass, out = torch.zeros(1, 2, 256, device="cuda"), torch.empty(1, 8, 128, device="cuda")
    B.decode_attention_mass_paged(lay, q, pc, dev([256]), 256, mass, out, ws, 2)
    assert lay.status() == B.STATUS_BAD_PAGE
    assert (mass[..., 64:128] == 0).all() and torch.isfinite(mass).all() and torch.isfinite(out).all()
    assert torch.allclose(mass.sum(-1).cpu(), torch.full((1, 2), 4.0), rtol=1e-5)


# ------------------------------------------------------------------ eviction
def reference_keep(mass, n, keep, n_sink, n_recent):
    """Positions kept: forced ones, then by mass (NaN last), ties to the lowest position."""
    if n <= keep:
        return np.arange(n)
    m = mass[:n].astype(np.float64)
    m = np.where(np.isnan(m), -np.inf, m)
    nan = np.isnan(mass[:n])
    mid = np.arange(n_sink, n - n_recent)
    order = mid[np.lexsort((mid, -m[mid], nan[mid]))]
    want = keep - n_sink - n_recent
    return np.sort(np.concatenate([np.arange(n_sink), order[:want], np.arange(n - n_recent, n)]).astype(int))


def reference_tiles(olay, tiles, idx, n_tiles):
    """Tiles of the tokens idx: codes through the oracle, norms as the bits they are (a norm may
    be any bit pattern, NaN among them)."""
    code, rows = 64 * (olay.k_record_bytes + olay.v_record_bytes), olay.n_kgroups + 1
    u = O.unpack(olay, tiles.reshape(-1), tiles.shape[0] * 64)
    kept = {k: np.zeros_like(x[idx]) if "norm" in k else x[idx] for k, x in u.items()}
    out = O.pack(olay, kept, n_tiles * 64).reshape(n_tiles, -1)
    it = np.uint16 if olay.norm_fp16 else np.uint32

    def by_token(t):                     # [tiles, row, 8 g + m] -> [token g + 8 m, row]
        return t[:, code:].copy().view(it).reshape(-1, rows, 8, 8).transpose(0, 3, 2, 1).reshape(-1, rows)

    norms = np.zeros((n_tiles * 64, rows), it)
    norms[:len(idx)] = by_token(tiles.reshape(-1, olay.tile_bytes))[idx]
    out[:, code:] = norms.reshape(n_tiles, 8, 8, rows).transpose(0, 3, 2, 1).reshape(n_tiles, -1).copy().view(np.uint8).reshape(n_tiles, -1)
    return out


EVICT_CASES = [  # mix, v_rate, fp16, h_kv, lens, keep, sink, recent, kind of mass, paged
    ("k2", 2, False, 2, [200, 64, 0, 1], 64, 4, 16, "smooth", False),
    ("k3", 3, True, 2, [1000, 999, 130], 131, 0, 0, "ties", False),
    ("k4", 4, False, 1, [300, 301], 299, 7, 200, "smooth", True),
    ("k1", 1, False, 3, [500], 1, 0, 1, "equal", False),
    ("holes", 2, True, 1, [777, 65, 64], 65, 65, 0, "smooth", True),
    ("k2", 3, False, 2, [2000, 1500], 700, 3, 64, "special", False),
    ("k3", 1, False, 1, [5000], 4000, 16, 1000, "ties", True),
]


def masses(kind, shape, rng):
    m = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        m = np.round(m * 2) / 2
    elif kind == "equal":
        m[:] = 0.25
    elif kind == "special":
        x = rng.random(shape)
        m[x < 0.02] = np.inf
        m[(x > 0.1) & (x < 0.15)] = np.nan
        m[(x > 0.2) & (x < 0.25)] = -np.inf
        m[(x > 0.3) & (x < 0.5)] = 0.0
        m[(x > 0.5) & (x < 0.7)] = -0.0
        m[(x > 0.7) & (x < 0.8)] *= -1
        m[(x > 0.8) & (x < 0.85)] = 1e-42                  # subnormal
    return m.astype(np.float32)


@pytest.mark.parametrize("case", EVICT_CASES, ids=lambda c: f"{c[0]}v{c[1]}_keep{c[5]}_{c[8]}")
def test_evict_matches_reference(case):
    mix, vr, fp16, h_kv, lens, keep, sink, recent, kind, use_pages = case
    rng = np.random.default_rng(8)
    lay, olay = make_layouts(mix, vr, fp16)
    b, most = len(lens), max(lens)
    nt, dt = -(-most // 64), -(-keep // 64) + 1
    tiles = random_cache(olay, b, h_kv, nt, rng)
    mass = masses(kind, (b, h_kv, most + 3), rng)
    ld_out = keep + 5
    mass_out = torch.full((b, h_kv, ld_out), 9.0, device="cuda")
    kept = torch.full((b, h_kv, keep), 77, dtype=torch.int32, device="cuda")
    new = torch.full((b,), -5, dtype=torch.int32, device="cuda")
    fill = rng.integers(0, 256, (b, h_kv, dt, olay.tile_bytes), dtype=np.uint8)
    if use_pages:
        src, dst = paged(tiles, rng), paged(fill, rng)
        B.cache_evict_paged(lay, src, dev(lens), most, torch.from_numpy(mass).cuda(), keep, sink, recent, dst, mass_out,
                            kept, new, h_kv)
        got = dst.pool.view(-1, h_kv, olay.tile_bytes)[dst.table.long()].transpose(1, 2).cpu().numpy()
    else:
        dst = torch.from_numpy(fill).cuda()
        B.cache_evict(lay, torch.from_numpy(tiles).cuda(), dev(lens), nt * 64, most, torch.from_numpy(mass).cuda(),
                      keep, sink, recent, dst, dt * 64, mass_out, kept, new, h_kv)
        got = dst.cpu().numpy()
    assert lay.status() == 0
    np.testing.assert_array_equal(new.cpu().numpy(), np.minimum(lens, keep))
    for r in range(b):
        for h in range(h_kv):
            idx = reference_keep(mass[r, h], lens[r], keep, sink, recent)
            m = len(idx)
            np.testing.assert_array_equal(kept[r, h].cpu().numpy(), np.concatenate([idx, np.full(keep - m, -1)]))
            np.testing.assert_array_equal(mass_out[r, h].cpu().numpy().view(np.uint32),
                                          np.concatenate([mass[r, h][idx], np.zeros(ld_out - m, np.float32)]).view(np.uint32))
            used = -(-m // 64)
            np.testing.assert_array_equal(got[r, h, used:], fill[r, h, used:])
            if used:
                np.testing.assert_array_equal(got[r, h, :used], reference_tiles(olay, tiles[r, h], idx, used))


def test_evict_long_rows_across_clusters():
    """Rows long enough for several CTAs per unit, and for more keys than shared memory holds."""
    rng = np.random.default_rng(9)
    lay, olay = make_layouts("k1", 1, True)
    for n, keep in ((40_000, 9_001), (210_000, 300)):
        nt = -(-n // 64)
        tiles = torch.randint(0, 256, (1, 1, nt, olay.tile_bytes), dtype=torch.uint8, device="cuda")
        mass = masses("ties", (1, 1, n), rng)
        mass[0, 0, rng.permutation(n)[:n // 2]] = 0.5
        mass_out = torch.empty(1, 1, keep, device="cuda")
        kept = torch.empty(1, 1, keep, dtype=torch.int32, device="cuda")
        new, dst = dev([0]), torch.empty(1, 1, -(-keep // 64), olay.tile_bytes, dtype=torch.uint8, device="cuda")
        B.cache_evict(lay, tiles, dev([n]), nt * 64, n, torch.from_numpy(mass).cuda(), keep, 2, 50, dst,
                      dst.shape[2] * 64, mass_out, kept, new, 1)
        idx = reference_keep(mass[0, 0], n, keep, 2, 50)
        np.testing.assert_array_equal(kept[0, 0].cpu().numpy(), idx)
        some = rng.integers(0, dst.shape[2], 3)
        host = tiles.cpu().numpy()
        for t in some:                                     # a few destination tiles, token by token
            part = idx[64 * t:64 * t + 64]
            src = np.unique(part // 64)
            at = np.searchsorted(src, part // 64) * 64 + part % 64
            want = reference_tiles(olay, host[0, 0, src], at, 1)[0]
            np.testing.assert_array_equal(dst[0, 0, t].cpu().numpy(), want)
    assert lay.status() == 0


def test_evict_missing_pages():
    rng = np.random.default_rng(10)
    lay, olay = make_layouts("k2", 2)
    tiles = random_cache(olay, 1, 2, 4, rng)
    fill = np.full((1, 2, 2, olay.tile_bytes), 7, np.uint8)
    src, dst = paged(tiles, rng), paged(fill, rng)
    src.table[0, 1] = -1
    dst_page = int(dst.table[0, 1])
    dst.table[0, 1] = 10 ** 6
    mass = torch.zeros(1, 2, 256, device="cuda")
    mass_out, kept = torch.empty(1, 2, 128, device="cuda"), torch.empty(1, 2, 128, dtype=torch.int32, device="cuda")
    new = dev([0])
    B.cache_evict_paged(lay, src, dev([256]), 256, mass, 128, 0, 0, dst, mass_out, kept, new, 2)
    assert lay.status() == B.STATUS_BAD_PAGE               # tokens 0..127: tile 1 has no page
    pool = dst.pool.view(-1, 2, olay.tile_bytes).cpu().numpy()
    np.testing.assert_array_equal(pool[int(dst.table[0, 0])], tiles[0, :, 0])
    np.testing.assert_array_equal(pool[dst_page], fill[0, :, 1])


def test_decode_evict_decode_run():
    """As a server uses them: decode steps that keep the mass, eviction into a smaller cache,
    more steps there; the outputs after the eviction match attention over the kept tokens."""
    rng = np.random.default_rng(11)
    lay, olay = make_layouts("k2", 2)
    b, h_q, h_kv, n, keep = 2, 8, 2, 300, 100
    G, cap, cap2 = h_q // h_kv, 320, 192
    kv = torch.from_numpy(rng.standard_normal((2, b, n + 8, h_kv, 128))).to(torch.bfloat16).cuda()
    cache = torch.zeros(lay.cache_bytes(b, h_kv, cap), dtype=torch.uint8, device="cuda")
    B.encode_append(lay, kv[0, :, :n].contiguous(), kv[1, :, :n].contiguous(), dev([0, 0]), cache, cap)
    ws = torch.empty(B.mass_workspace_bytes(lay, b, h_q, h_kv, cap), dtype=torch.uint8, device="cuda")
    mass = torch.zeros(b, h_kv, cap, device="cuda")
    out = torch.empty(b, h_q, 128, device="cuda")
    for i in range(4):
        q = torch.from_numpy(rng.standard_normal((b, h_q, 128))).to(torch.bfloat16).cuda()
        lens = dev([n + i] * b)
        B.encode_append(lay, kv[0, :, n + i:n + i + 1].contiguous(), kv[1, :, n + i:n + i + 1].contiguous(), lens, cache, cap)
        B.decode_attention_mass(lay, q, cache, lens + 1, cap, cap, mass, out, ws, h_kv)
    small = torch.zeros(lay.cache_bytes(b, h_kv, cap2), dtype=torch.uint8, device="cuda")
    mass2 = torch.empty(b, h_kv, cap2, device="cuda")
    kept = torch.empty(b, h_kv, keep, dtype=torch.int32, device="cuda")
    lens2 = dev([0, 0])
    B.cache_evict(lay, cache, dev([n + 4] * b), cap, n + 4, mass, keep, 4, 20, small, cap2, mass2, kept, lens2, h_kv)
    B.encode_append(lay, kv[0, :, n + 4:n + 8].contiguous(), kv[1, :, n + 4:n + 8].contiguous(), lens2, small, cap2)
    B.decode_attention_mass(lay, q, small, lens2 + 4, cap2, cap2, mass2, out, ws, h_kv)
    assert lay.status() == 0
    big = cache.cpu().numpy().reshape(b, h_kv, cap // 64, -1)
    new = small.cpu().numpy().reshape(b, h_kv, cap2 // 64, -1)
    o = out.cpu().double().numpy()
    for r in range(b):
        for h in range(h_kv):
            idx = kept[r, h].cpu().numpy()
            np.testing.assert_array_equal(idx, reference_keep(mass[r, h].cpu().numpy(), n + 4, keep, 4, 20))
            k0, v0 = dequantised(olay, big[r, h], n + 4)
            k1, v1 = dequantised(olay, new[r, h], keep + 4)
            np.testing.assert_array_equal(k1[:keep], k0[idx])
            np.testing.assert_array_equal(v1[:keep], v0[idx])
            ref = O.attention(q[r, h * G:(h + 1) * G].cpu().double().numpy(), k1, v1, 1 / math.sqrt(128))
            for a in range(G):
                assert rel_l2(o[r, h * G + a], ref[a]) <= ATTN_REL_L2
