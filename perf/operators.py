"""Measured cases of the operators that serve drafted tokens and a bounded cache over the packed KV cache:

* tree: attention of a tree of drafted tokens (up to 64 per row, each seeing the whole prefix and its own
  ancestors) over the packed cache that already holds their keys and values;
* commit: the accepted path of the tree moved to the end of the prefix inside the packed cache;
* mass: single-token decode attention that also adds every cached token's attention weight (summed over the
  query heads of its KV head) to a running sum;
* evict: the tokens with the largest sums (and the first and the newest ones) kept, their packed codes and
  norms gathered bit for bit into a smaller cache.

``own`` False computes them in plain torch operations on the same packed bytes; True calls the framework.
"""
import math

import numpy as np
import torch

own = False

HEAD_DIM = 128
TILE = 64
SEED = 11          # rotations of the layouts
# Block rates as the allocation gives them for the Llama-shaped (K2), Qwen-shaped (K3) and uniform K4 layers:
# number of 2-D blocks of rate 1, 2, 3, 4.
RATE_MIX = {"k2": (27, 22, 3, 12), "k3": (11, 13, 5, 35), "k4": (0, 0, 0, 64)}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    base = {"name": name, "op": op, "batch": 1, "h_kv": 8, "group": 4, "length": 4096, "mix": "k2", "v_rate": 2,
            "norm16": False, "paged": False, "ragged": False, "dtype": "bf16", "nodes": 0, "keep": 0, "sinks": 0,
            "recent": 0, "decay": 1.0}
    return {**base, **kw}


def listed():
    return [
        # one user, a short chat, a small draft: the call's latency
        _case("tree_1x1k_n6", "tree", length=1024, nodes=6),
        # a serving batch with a drafted tree per row over a paged cache
        _case("tree_8x8k_n16_paged", "tree", batch=8, length=8192, nodes=16, ragged=True, paged=True),
        # odd sizes: 7 query heads per KV head, 13 nodes, fp16 norms and queries, rates of the Qwen-shaped layer
        _case("tree_3x5001_n13_k3", "tree", batch=3, h_kv=4, group=7, length=5001, nodes=13, ragged=True, mix="k3",
              v_rate=3, norm16=True, dtype="f16"),
        # the 70B-shaped layer with a full tree of 64 nodes: matrix products bound it
        _case("tree_4x32k_n64", "tree", batch=4, group=8, length=32768, nodes=64),
        # the accepted path of one user's draft, and of a large batch's
        _case("commit_1_n6", "commit", length=1024, nodes=6),
        _case("commit_64_n64", "commit", batch=64, length=2048, nodes=64, ragged=True),
        # a decode step that keeps the sums: one user, the 70B-shaped batch, an odd paged batch
        _case("mass_1x4k", "mass", length=4096),
        _case("mass_4x128k", "mass", batch=4, group=8, length=131072),
        _case("mass_5x9001_k3_paged", "mass", batch=5, h_kv=2, group=8, length=9001, ragged=True, paged=True, mix="k3",
              v_rate=3, dtype="f16", decay=0.98),
        # a prompt of 4K cut to 1K for one user; long rows of a batch cut to a quarter; an odd paged batch
        _case("evict_1x4k_to_1k", "evict", length=4096, keep=1024, sinks=4, recent=256),
        _case("evict_16x32k_to_8k", "evict", batch=16, length=32768, keep=8192, sinks=16, recent=1024, ragged=True),
        _case("evict_5x20001_k4_paged", "evict", batch=5, h_kv=2, length=20001, keep=4099, sinks=7, recent=513,
              ragged=True, paged=True, mix="k4", v_rate=4, norm16=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    mix = rng.choice(["k2", "k2", "k3", "k4"])
    kw = {"mix": mix, "v_rate": {"k2": 2, "k3": 3, "k4": 4}[mix], "norm16": rng.random() < 0.3,
          "paged": rng.random() < 0.4, "ragged": rng.random() < 0.6, "dtype": rng.choice(["bf16", "bf16", "f16"]),
          "h_kv": rng.choice([1, 2, 4, 8]), "group": rng.choice([1, 2, 4, 5, 7, 8])}
    op = rng.choice(["tree", "tree", "commit", "mass", "mass", "evict", "evict"])
    batch = log(1, 32)
    if op == "tree":
        # rows x heads x tokens x nodes bounded by the largest listed case's
        nodes = rng.choice([2, 3, 5, 8, 12, 16, 25, 31, 48, 64])
        most = 4 * 8 * 32768 * 64 * 8 // (batch * kw["h_kv"] * nodes * kw["group"])
        c = _case("", op, batch=batch, nodes=nodes, length=max(nodes, log(200, min(65536, max(300, most)))), **kw)
    elif op == "commit":
        c = _case("", op, batch=log(1, 64), nodes=rng.randint(2, 64), length=log(100, 2048), **kw)
    elif op == "mass":
        most = 4 * 8 * 131072 // (batch * kw["h_kv"])
        c = _case("", op, batch=batch, length=log(100, min(131072, most)), decay=rng.choice([1.0, 1.0, 0.95]), **kw)
    else:
        most = 16 * 8 * 32768 // (batch * kw["h_kv"])
        length = log(500, min(131072, most))
        keep = max(40, int(length * rng.uniform(0.1, 0.7)))
        c = _case("", op, batch=batch, length=length, keep=keep, sinks=rng.randint(0, 16),
                  recent=rng.randint(0, keep - 20), **kw)
    del c["name"]
    return c


# ------------------------------------------------------------------ the packed format, as tables
def _rates(mix):
    n = RATE_MIX[mix]
    r = np.repeat([1, 2, 3, 4], n)
    return np.random.default_rng(7).permutation(r).astype(np.int32)


def _groups(rates):
    """(rate, coordinates) of every key group: descending rate, blocks ascending, coordinate j before j + 64."""
    return [(r, np.concatenate([[j, j + 64] for j in np.flatnonzero(rates == r)])) for r in (4, 3, 2, 1)
            if (rates == r).any()]


def _philox_normals(seed, stream, count):
    """N(0,1) draws of the published Philox4x32-10 generator and Box-Muller."""
    n = np.arange((count + 1) // 2, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    c = [n & low, n >> np.uint64(32), np.full_like(n, stream), np.zeros_like(n)]
    k0, k1 = np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32)
    for _ in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ k0, p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ k1, p0 & low]
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & low, (k1 + np.uint64(0xBB67AE85)) & low
    u = [((a >> np.uint64(5)).astype(float) * 67108864.0 + (b >> np.uint64(6)).astype(float) + 0.5) / 2.0 ** 53
         for a, b in ((c[0], c[1]), (c[2], c[3]))]
    r = np.sqrt(-2.0 * np.log(u[0]))
    return np.stack([r * np.cos(2 * math.pi * u[1]), r * np.sin(2 * math.pi * u[1])], 1).reshape(-1)[:count]


def _rotation(stream, d):
    q, t = np.linalg.qr(_philox_normals(SEED, stream, d * d).reshape(d, d))
    return q * np.where(np.diag(t) < 0, -1.0, 1.0)[None, :]


def _lloyd_max(bits):
    """Centroids of the MSE-optimal quantiser of N(0,1) with 2^bits levels."""
    n = 1 << (bits - 1)
    pdf = lambda x: math.exp(-0.5 * x * x) / math.sqrt(2 * math.pi) if x < 1e9 else 0.0  # noqa: E731
    tail = lambda x: 0.5 * math.erfc(x / math.sqrt(2)) if x < 1e9 else 0.0  # noqa: E731
    t = [3.0 * i / n for i in range(n)] + [1e9]
    for _ in range(20000):
        c = [(pdf(a) - pdf(b)) / (tail(a) - tail(b)) for a, b in zip(t[:-1], t[1:])]
        new = [0.0] + [0.5 * (a + b) for a, b in zip(c[:-1], c[1:])] + [1e9]
        done = max(abs(a - b) for a, b in zip(t, new)) < 1e-15
        t = new
        if done:
            break
    return np.array([-x for x in reversed(c)] + c)


def _bit_places(groups, v_rate):
    """Bit of a tile's code bytes that holds bit b of the code of (token, dim): [64, 256, 4], -1 where a code has
    no bit b. Dims 0..127 are the packed key dims, 128..255 the value dims."""
    at = np.full((TILE, 256, 4), -1, dtype=np.int64)
    g, m = np.meshgrid(np.arange(8), np.arange(8), indexing="ij")
    off, p = 0, 0
    for r, coords in groups:
        for c0 in range(0, len(coords), 8):
            pairs = min(8, len(coords) - c0) // 2
            for e in range(pairs):
                lane = g * pairs + e
                for half in range(2):
                    for b in range(r):
                        s = 8 * half + m if r == 1 else 2 * r * m + r * half + b
                        place = 16 * r * lane + s
                        if r == 3:
                            place = np.where(s < 32, 32 * lane + s, 256 * pairs + 16 * lane + s - 32)
                        at[g + 8 * m, p + c0 + 2 * e + half, b] = 8 * off + place
            off += 16 * pairs * r
        p += len(coords)
    lane, n = np.meshgrid(np.arange(32), np.arange(32), indexing="ij")
    for chunk in range(4):
        for half in range(2):
            for b in range(v_rate):
                dim = 16 * (lane >> 2) + 2 * (n >> 2) + (n & 1)
                tok = 16 * chunk + 2 * (lane & 3) + 8 * ((n & 3) >> 1) + half
                s = 32 * (n >> 4) + 16 * half + (n & 15) if v_rate == 1 else 2 * v_rate * n + v_rate * half + b
                place = 64 * v_rate * lane + s
                if v_rate > 2:
                    place = np.where(s < 128, 128 * lane + s, 4096 + (64 * v_rate - 128) * lane + s - 128)
                at[tok, 128 + dim, b] = 8 * (off + chunk * 256 * v_rate) + place
    return at


def _layout(case):
    """Everything about the layer's packing that a plain computation needs, on the GPU."""
    rates = _rates(case["mix"])
    groups, vr = _groups(rates), case["v_rate"]
    at = _bit_places(groups, vr)
    code_bytes = TILE * (sum(r * len(c) for r, c in groups) + 128 * vr) // 8
    flat = np.zeros(8 * code_bytes, dtype=np.int64)           # (token, dim, bit) held by each bit of the tile
    flat[at[at >= 0]] = np.flatnonzero(at.reshape(-1) >= 0)
    dev = "cuda"
    table = np.zeros((5, 16))
    for r in (1, 2, 3, 4):
        table[r, :1 << r] = _lloyd_max(r)
    dim_rate = np.concatenate([np.full(len(c), r) for r, c in groups] + [np.full(128, vr)])
    dim_norm = np.concatenate([np.full(len(c), i) for i, (r, c) in enumerate(groups)] + [np.full(128, len(groups))])
    size = np.array([len(c) for _, c in groups] + [128])
    k_rot, p = np.zeros((128, 128)), 0                        # packed (rotated) dims -> coordinates of the head
    for r, c in groups:
        k_rot[p:p + len(c), c] = _rotation(r, len(c))
        p += len(c)
    lay = {
        "code_bytes": code_bytes,
        "norm_bytes": 2 if case["norm16"] else 4,
        "n_norms": len(groups) + 1,
        "byte": torch.from_numpy(np.where(at < 0, 0, at // 8)).to(dev, torch.int32),
        "shift": torch.from_numpy(np.where(at < 0, 0, at % 8)).to(dev, torch.uint8),
        "has": torch.from_numpy((at >= 0)).to(dev, torch.uint8),
        "source": torch.from_numpy(flat // 4).to(dev, torch.int32),
        "source_bit": torch.from_numpy(flat % 4).to(dev, torch.uint8),
        "row16": torch.from_numpy(dim_rate * 16).to(dev, torch.int32),
        "table": torch.from_numpy(table.reshape(-1)).to(dev),
        "dim_norm": torch.from_numpy(dim_norm).to(dev),
        "inv_root": torch.from_numpy(1.0 / np.sqrt(size[dim_norm])).to(dev),
        "k_rot": torch.from_numpy(k_rot).to(dev),
        "v_rot": torch.from_numpy(_rotation(0, 128)).to(dev),
        "rates": rates,
        "groups": [(int(r), len(c)) for r, c in groups],
    }
    lay["tile_bytes"] = code_bytes + TILE * lay["norm_bytes"] * lay["n_norms"]
    return lay


def _pack(lay, codes, norms):
    """Tiles [..., tile_bytes] from codes [..., 64, 256] (uint8) and norms [..., n_norms, 64] (stored type)."""
    lead = codes.shape[:-2]
    bits = torch.index_select(codes.reshape(-1, TILE * 256), 1, lay["source"])
    bits = (bits >> lay["source_bit"]) & 1
    weight = torch.tensor([1, 2, 4, 8, 16, 32, 64, 128], dtype=torch.uint8, device=codes.device)
    code_bytes = (bits.view(-1, lay["code_bytes"], 8) * weight).sum(-1, dtype=torch.uint8)
    rows = norms.reshape(-1, lay["n_norms"], 8, 8).transpose(-1, -2).contiguous().view(torch.uint8)
    return torch.cat([code_bytes, rows.reshape(len(code_bytes), -1)], 1).view(*lead, lay["tile_bytes"])


def _codes(lay, tiles):
    """Codes [..., 64, 256] (uint8) of tiles [..., tile_bytes]."""
    flat = tiles.reshape(-1, lay["tile_bytes"])

    def bit(b):
        x = torch.index_select(flat, 1, lay["byte"][:, :, b].reshape(-1)).view(-1, TILE, 256)
        return ((x >> lay["shift"][:, :, b]) & lay["has"][:, :, b]) << b

    return (bit(0) | bit(1) | bit(2) | bit(3)).view(*tiles.shape[:-1], TILE, 256)


def _norms(lay, tiles):
    """Stored norms [..., n_norms, 64] by token (a row keeps token g + 8 m at entry 8 g + m)."""
    raw = tiles[..., lay["code_bytes"]:].contiguous().view(torch.float16 if lay["norm_bytes"] == 2 else torch.float32)
    return raw.reshape(*tiles.shape[:-1], lay["n_norms"], 8, 8).transpose(-1, -2).reshape(
        *tiles.shape[:-1], lay["n_norms"], TILE)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _random_tiles(lay, case, n_tiles, gen):
    """Tiles as the encoder leaves them: codes of Gaussian coordinates, key norms that grow with a group's rate
    (the rates follow the energy), value norms near sqrt(128)."""
    dev = "cuda"
    codes = torch.empty(n_tiles, TILE, 256, dtype=torch.uint8, device=dev)
    edges = {}
    for r in {r for r, _ in lay["groups"]} | {case["v_rate"]}:
        c = lay["table"].view(5, 16)[r, :1 << r]
        edges[r] = (0.5 * (c[1:] + c[:-1])).float()
    step = 4096
    for a in range(0, n_tiles, step):
        b = min(n_tiles, a + step)
        p = 0
        for r, d in lay["groups"] + [(case["v_rate"], 128)]:
            y = torch.randn(b - a, TILE, d, device=dev, generator=gen)
            codes[a:b, :, p:p + d] = torch.bucketize(y, edges[r], right=True).to(torch.uint8)
            p += d
    norms = torch.empty(n_tiles, lay["n_norms"], TILE, device=dev)
    for i, (r, d) in enumerate(lay["groups"] + [(None, 128)]):
        sigma = 1.0 if r is None else {1: 0.6, 2: 1.1, 3: 1.8, 4: 2.6}[r]
        z = torch.randn(n_tiles, TILE, device=dev, generator=gen)
        norms[:, i] = sigma * math.sqrt(d) * (1.0 + z / math.sqrt(2.0 * d)).clamp(0.2, 2.0)
    tiles = torch.empty(n_tiles, lay["tile_bytes"], dtype=torch.uint8, device=dev)
    kept = norms.to(torch.float16 if case["norm16"] else torch.float32)
    for a in range(0, n_tiles, step):
        tiles[a:a + step] = _pack(lay, codes[a:a + step], kept[a:a + step])
    return tiles


def _lengths(case, rng, most):
    n = np.full(case["batch"], most)
    if case["ragged"]:
        n[1:] = rng.integers(max(case["nodes"], most // 2), most + 1, case["batch"] - 1)
    return n


def _tree(rng, n):
    """Parents of a random tree (or forest: a row may draft several first tokens) of n nodes, parents first."""
    return np.array([-1] + [int(rng.integers(-1 if rng.random() < 0.2 else max(0, i - 6), i)) for i in range(1, n)])


def _paged(case, tiles, rng):
    """A pool of pages [h_kv][tile] in random order, spare pages among them, and its block table."""
    b, h, n, tb = tiles.shape
    pages = b * n + 5
    table = torch.from_numpy(rng.permutation(pages)[:b * n].reshape(b, n)).to("cuda", torch.int32)
    pool = torch.zeros(pages, h, tb, dtype=torch.uint8, device="cuda")
    pool[table.reshape(-1).long()] = tiles.transpose(1, 2).reshape(b * n, h, tb)
    return pool, table


def prepare(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    lay = _layout(case)
    b, h, length = case["batch"], case["h_kv"], case["length"]
    n_tiles = -(-length // TILE)
    s = {"case": case, "lay": lay, "max_len": length, "capacity": n_tiles * TILE, "scale": 1.0 / math.sqrt(HEAD_DIM)}
    tiles = _random_tiles(lay, case, b * h * n_tiles, gen).view(b, h, n_tiles, lay["tile_bytes"])
    s["lens"] = torch.from_numpy(_lengths(case, rng, length)).to("cuda", torch.int32)
    if case["paged"]:
        s["pool"], s["table"] = _paged(case, tiles, rng)
    else:
        s["cache"] = tiles
    dt = DTYPES[case["dtype"]]
    n, h_q = case["nodes"], h * case["group"]
    if case["op"] == "tree":
        s["q"] = (1.4 * torch.randn(b, n, h_q, HEAD_DIM, device="cuda", generator=gen)).to(dt)
        mask = np.zeros((b, n), dtype=np.uint64)
        for row in range(b):
            for i, parent in enumerate(_tree(rng, n)):
                mask[row, i] = (mask[row, parent] if parent >= 0 else np.uint64(0)) | np.uint64(1 << i)
        s["mask"] = torch.from_numpy(mask.view(np.int64)).cuda()
        s["out"] = torch.empty_like(s["q"])
    elif case["op"] == "commit":
        path = np.zeros((b, n), dtype=np.int32)
        count = np.zeros(b, dtype=np.int32)
        for row in range(b):
            parent, i, line = _tree(rng, n), n - 1, []
            while i >= 0:
                line.append(i)
                i = parent[i]
            count[row] = len(line)
            path[row, :len(line)] = line[::-1]
        s["path"], s["count"] = torch.from_numpy(path).cuda(), torch.from_numpy(count).cuda()
        s["new_lens"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    elif case["op"] == "mass":
        s["q"] = (1.4 * torch.randn(b, h_q, HEAD_DIM, device="cuda", generator=gen)).to(dt)
        s["mass"] = torch.rand(b, h, s["capacity"], device="cuda", generator=gen) / length
        s["out"] = torch.empty_like(s["q"])
    else:
        # sums as decoding leaves them: heavy-tailed, many tokens near zero, some exactly equal
        z = torch.randn(b, h, s["capacity"], device="cuda", generator=gen)
        s["mass"] = torch.exp(2.0 * z)
        s["mass"][..., ::5] = torch.round(s["mass"][..., ::5] * 8) / 8
        kt = -(-case["keep"] // TILE)
        s["mass_out"] = torch.zeros(b, h, kt * TILE, device="cuda")
        s["kept"] = torch.zeros(b, h, case["keep"], dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.zeros(b, dtype=torch.int32, device="cuda")
        out = torch.zeros(b, h, kt, lay["tile_bytes"], dtype=torch.uint8, device="cuda")
        if case["paged"]:
            s["out_pool"], s["out_table"] = _paged(case, out, rng)
        else:
            s["out_cache"] = out
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The handle and the workspace that a program of the framework keeps."""
    from packed_cache_decode_b200 import binding as B
    c = s["case"]
    s["B"] = B
    s["handle"] = B.Layout(s["lay"]["rates"], c["v_rate"], SEED, norm_fp16=c["norm16"]).upload(0)
    h_q = c["h_kv"] * c["group"]
    size = 0
    if c["op"] == "tree":
        size = B.tree_workspace_bytes(s["handle"], c["batch"], h_q, c["h_kv"], c["nodes"], s["max_len"])
    elif c["op"] == "mass":
        size = B.mass_workspace_bytes(s["handle"], c["batch"], h_q, c["h_kv"], s["max_len"])
    s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if c["paged"]:
        s["paged"] = B.PagedCache(s["pool"].view(-1), s["table"])
        if c["op"] == "evict":
            s["out_paged"] = B.PagedCache(s["out_pool"].view(-1), s["out_table"])


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s)
    return {"tree": _plain_tree, "commit": _plain_commit, "mass": _plain_mass, "evict": _plain_evict}[op](s)


def _run_own(s):
    B, c, lay, lens = s["B"], s["case"], s["handle"], s["lens"]
    h, cap, most, op = c["h_kv"], s["capacity"], s["max_len"], c["op"]
    if op == "tree":
        if c["paged"]:
            B.tree_attention_paged(lay, s["q"], s["mask"], s["paged"], lens, most, s["out"], s["ws"], h)
        else:
            B.tree_attention(lay, s["q"], s["mask"], s["cache"], lens, cap, most, s["out"], s["ws"], h)
        return {"out": s["out"]}
    if op == "commit":
        if c["paged"]:
            B.tree_commit_paged(lay, s["path"], s["count"], c["nodes"], s["paged"], lens, s["new_lens"], h)
            return {"cache": s["pool"], "lens": s["new_lens"]}
        B.tree_commit(lay, s["path"], s["count"], c["nodes"], s["cache"], lens, s["new_lens"], cap, h)
        return {"cache": s["cache"], "lens": s["new_lens"]}
    if op == "mass":
        if c["paged"]:
            B.decode_attention_mass_paged(lay, s["q"], s["paged"], lens, most, s["mass"], s["out"], s["ws"], h,
                                          decay=c["decay"])
        else:
            B.decode_attention_mass(lay, s["q"], s["cache"], lens, cap, most, s["mass"], s["out"], s["ws"], h,
                                    decay=c["decay"])
        return {"out": s["out"], "mass": s["mass"]}
    if c["paged"]:
        B.cache_evict_paged(lay, s["paged"], lens, most, s["mass"], c["keep"], c["sinks"], c["recent"], s["out_paged"],
                            s["mass_out"], s["kept"], s["new_lens"], h)
    else:
        B.cache_evict(lay, s["cache"], lens, cap, most, s["mass"], c["keep"], c["sinks"], c["recent"], s["out_cache"],
                      s["out_cache"].shape[2] * TILE, s["mass_out"], s["kept"], s["new_lens"], h)
    return {"cache": s["out_pool"] if c["paged"] else s["out_cache"], "mass": s["mass_out"], "kept": s["kept"],
            "lens": s["new_lens"]}


# ------------------------------------------------------------------ plain forms
def _tiles(s):
    if s["case"]["paged"]:
        return s["pool"][s["table"].long()].transpose(1, 2)
    return s["cache"]


def _dequantised(lay, tiles):
    """Keys and values [b, h, tokens, 128] in 32 bits: centroid times norm / sqrt(size), rotated back."""
    codes, norms = _codes(lay, tiles), _norms(lay, tiles).float()
    b, h, n = tiles.shape[:3]
    y = torch.take(lay["table"].float(), (codes.int() + lay["row16"]).long())
    y = y * norms.transpose(-1, -2)[..., lay["dim_norm"]] * lay["inv_root"].float()
    y = y.view(b, h, n * TILE, 256)
    return y[..., :128] @ lay["k_rot"].float(), y[..., 128:] @ lay["v_rot"].float()


def _softmax(s, visible):
    x = torch.where(visible, s, torch.full_like(s, -math.inf))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, torch.zeros_like(p))


def _plain_tree(s):
    c, lay = s["case"], s["lay"]
    b, h, g, n = c["batch"], c["h_kv"], c["group"], c["nodes"]
    k, v = _dequantised(lay, _tiles(s))
    q = s["q"].float().view(b, n, h, g, HEAD_DIM).permute(0, 2, 1, 3, 4).reshape(b, h, n * g, HEAD_DIM)
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    place = torch.arange(k.shape[2], device="cuda")
    first = (s["lens"].long() - n).view(b, 1, 1)
    node = (place - first).clamp(0, 63)
    sees = ((s["mask"].unsqueeze(-1) >> node) & 1).bool()
    visible = torch.where(place < first, True, sees & (place < first + n))
    p = _softmax(x, visible.repeat_interleave(g, 1).unsqueeze(1))
    o = (p @ v).view(b, h, n, g, HEAD_DIM).permute(0, 2, 1, 3, 4).reshape(b, n, h * g, HEAD_DIM)
    return {"out": o.to(s["q"].dtype)}


def _plain_commit(s):
    """The two tiles that a row's drafted tokens may lie in are opened, the accepted tokens put in order and
    packed again; every other token of them keeps its place."""
    c, lay, n = s["case"], s["lay"], s["case"]["nodes"]
    b, h = c["batch"], c["h_kv"]
    first = s["lens"].long() - n
    rows = torch.arange(b, device="cuda")
    t0 = first // TILE
    t1 = ((first + n - 1) // TILE)
    store = s["pool"] if c["paged"] else s["cache"]

    def get(t):
        return store[s["table"][rows, t].long()] if c["paged"] else store[rows, :, t]

    def put(t, x):
        if c["paged"]:
            store[s["table"][rows, t].long()] = x
        else:
            store[rows, :, t] = x

    two = torch.stack([get(t0), get(t1)], 2)
    codes = _codes(lay, two).view(b, h, 2 * TILE, 256)
    norms = _norms(lay, two).transpose(-1, -2).reshape(b, h, 2 * TILE, lay["n_norms"])
    place = torch.arange(2 * TILE, device="cuda").expand(b, -1)
    local = (first - t0 * TILE).view(b, 1)
    i = (place - local).clamp(0, n - 1)
    moved = (place >= local) & (place < local + s["count"].view(b, 1))
    source = torch.where(moved, local + torch.gather(s["path"].long(), 1, i), place)
    at = source.view(b, 1, -1, 1)
    codes = torch.gather(codes, 2, at.expand(b, h, -1, 256)).view(b, h, 2, TILE, 256)
    norms = torch.gather(norms, 2, at.expand(b, h, -1, lay["n_norms"])).view(b, h, 2, TILE, -1).transpose(-1, -2)
    new = _pack(lay, codes, norms.contiguous())
    put(t1, torch.where((t1 > t0).view(b, 1, 1), new[:, :, 1], two[:, :, 1]))
    put(t0, new[:, :, 0])
    s["new_lens"].copy_(first + s["count"])
    return {"cache": store, "lens": s["new_lens"]}


def _plain_mass(s):
    c, lay = s["case"], s["lay"]
    b, h, g = c["batch"], c["h_kv"], c["group"]
    k, v = _dequantised(lay, _tiles(s))
    q = s["q"].float().view(b, h, g, HEAD_DIM)
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    visible = (torch.arange(k.shape[2], device="cuda") < s["lens"].view(b, 1)).view(b, 1, 1, -1)
    p = _softmax(x, visible)
    out = (p @ v).view(b, h * g, HEAD_DIM)
    s["mass"].copy_(torch.where(visible[:, :, 0], c["decay"] * s["mass"] + p.sum(2), s["mass"]))
    return {"out": out.to(s["q"].dtype), "mass": s["mass"]}


def _plain_evict(s):
    c, lay = s["case"], s["lay"]
    b, h, keep = c["batch"], c["h_kv"], c["keep"]
    tiles = _tiles(s)
    n = tiles.shape[2] * TILE
    lens = s["lens"].long().view(b, 1, 1)
    place = torch.arange(n, device="cuda").view(1, 1, n)
    fixed = (place < c["sinks"]) | (place >= lens - c["recent"])
    worth = torch.where(fixed, torch.full_like(s["mass"], math.inf), s["mass"])
    worth = torch.where(place < lens, worth, torch.full_like(worth, -math.inf))
    best = torch.sort(worth, dim=-1, descending=True, stable=True).indices[..., :keep]
    new = torch.minimum(lens, torch.tensor(keep, device="cuda"))
    if n < keep:
        best = torch.cat([best, torch.zeros(b, h, keep - n, dtype=torch.int64, device="cuda")], -1)
    here = torch.arange(keep, device="cuda").view(1, 1, keep) < new
    best = torch.sort(torch.where(here, best, torch.full_like(best, n))).values   # ascending, the unused ones last
    kept = torch.where(here, best, torch.full_like(best, -1))
    kt = -(-keep // TILE)
    pad = kt * TILE - keep
    at = torch.cat([best.clamp(max=n - 1), torch.zeros(b, h, pad, dtype=torch.int64, device="cuda")], -1)
    live = torch.cat([here.expand(b, h, keep), torch.zeros(b, h, pad, dtype=torch.bool, device="cuda")], -1)
    codes = _codes(lay, tiles).view(b, h, n, 256)
    norms = _norms(lay, tiles).transpose(-1, -2).reshape(b, h, n, lay["n_norms"])
    codes = torch.gather(codes, 2, at.unsqueeze(-1).expand(-1, -1, -1, 256)) * live.unsqueeze(-1).to(torch.uint8)
    norms = torch.gather(norms, 2, at.unsqueeze(-1).expand(-1, -1, -1, lay["n_norms"])) * live.unsqueeze(-1)
    packed = _pack(lay, codes.view(b, h, kt, TILE, 256),
                   norms.view(b, h, kt, TILE, -1).transpose(-1, -2).contiguous())
    used = (torch.arange(kt, device="cuda").view(1, 1, kt, 1) * TILE) < new.unsqueeze(-1)
    if c["paged"]:
        old = s["out_pool"][s["out_table"].long()]
        s["out_pool"][s["out_table"].long()] = torch.where(used.transpose(1, 2), packed.transpose(1, 2), old)
    else:
        s["out_cache"].copy_(torch.where(used, packed, s["out_cache"]))
    s["mass_out"].copy_(torch.where(live, torch.gather(s["mass"], 2, at), torch.zeros_like(s["mass_out"])))
    s["kept"].copy_(kept)
    s["new_lens"].copy_(new.view(b))
    return {"cache": s["out_pool"] if c["paged"] else s["out_cache"], "mass": s["mass_out"], "kept": s["kept"],
            "lens": s["new_lens"]}


# ------------------------------------------------------------------ work and exact values
def work(case):
    rates = np.repeat([1, 2, 3, 4], RATE_MIX[case["mix"]])
    n_norms = len(set(rates.tolist())) + 1
    per_token = 2 * int(rates.sum()) / 8 + 16 * case["v_rate"] + (2 if case["norm16"] else 4) * n_norms
    rng = np.random.default_rng(0)
    lens = _lengths(case, rng, case["length"]) if case["ragged"] else np.full(case["batch"], case["length"])
    tokens = float(lens.mean()) * case["batch"] * case["h_kv"]      # (ragged rows: another draw of the same range)
    h_q, units = case["h_kv"] * case["group"], case["batch"] * case["h_kv"]
    if case["op"] == "tree":
        rows = case["batch"] * case["nodes"] * h_q
        return {"bytes": tokens * per_token + 4.0 * rows * HEAD_DIM + 8 * case["batch"] * case["nodes"],
                "flops": 4.0 * tokens * case["nodes"] * case["group"] * HEAD_DIM}
    if case["op"] == "commit":
        moved = units * case["nodes"] / 4.0                          # a path is a fraction of its tree
        return {"bytes": 2.0 * moved * per_token + 4 * case["batch"] * case["nodes"], "flops": 0.0}
    if case["op"] == "mass":
        return {"bytes": tokens * (per_token + 8) + 4.0 * case["batch"] * h_q * HEAD_DIM,
                "flops": 4.0 * tokens * case["group"] * HEAD_DIM}
    kept = float(np.minimum(lens, case["keep"]).sum()) * case["h_kv"]
    return {"bytes": 4.0 * tokens + 2.0 * kept * per_token + 8.0 * kept, "flops": 0.0}


def _exact_codes(raw, kind, groups, v_rate):
    """Codes [tiles, 64, 128] (int) read string by string from tiles' key (kind 0) or value (kind 1) bytes."""
    n = raw.shape[0]
    out = torch.zeros(n, TILE, HEAD_DIM, dtype=torch.int64, device=raw.device)
    r64 = raw.long()

    def word(off, size):
        return sum(r64[:, off + i] << (8 * i) for i in range(size))

    if kind == 0:
        off = p = 0
        for r, d in groups:
            for c0 in range(0, d, 8):
                pairs = min(8, d - c0) // 2
                lanes = torch.arange(8 * pairs, device=raw.device)
                g, e = lanes // pairs, lanes % pairs
                w = word(off + 4 * lanes, 4) | (word(off + 32 * pairs + 2 * lanes, 2) << 32) if r == 3 \
                    else word(off + 2 * r * lanes, 2 * r)
                for m in range(8):
                    lo, hi = ((w >> m) & 1, (w >> (8 + m)) & 1) if r == 1 else \
                        ((w >> (2 * r * m)) & ((1 << r) - 1), (w >> (2 * r * m + r)) & ((1 << r) - 1))
                    out[:, g + 8 * m, p + c0 + 2 * e] = lo
                    out[:, g + 8 * m, p + c0 + 2 * e + 1] = hi
                off += 16 * pairs * r
            p += d
        return out
    lanes = torch.arange(32, device=raw.device)
    for chunk in range(4):
        base = chunk * 256 * v_rate
        for n_ in range(32):
            k = n_ & 3
            if v_rate == 1:
                w = word(base + 8 * lanes + 4 * (n_ >> 4), 4)
                lo, hi = (w >> (n_ & 15)) & 1, (w >> (16 + (n_ & 15))) & 1
            else:
                first = 2 * v_rate * n_
                both = 0
                for b in range(2 * v_rate):
                    s = first + b
                    at = 128 * lanes + s if v_rate == 2 or s < 128 else 4096 + (64 * v_rate - 128) * lanes + s - 128
                    both = both | (((r64[:, base + at // 8] >> (at % 8)) & 1) << b)
                lo, hi = both & ((1 << v_rate) - 1), both >> v_rate
            dim, tok = 16 * (lanes // 4) + 2 * (n_ >> 2) + (k & 1), 16 * chunk + 2 * (lanes % 4) + 8 * (k >> 1)
            out[:, tok, dim] = lo
            out[:, tok + 1, dim] = hi
    return out


def _exact_unit(s, tiles):
    """Keys and values of one (row, KV head)'s tiles in 64 bits, group by group."""
    lay, c = s["lay"], s["case"]
    groups, table = lay["groups"], lay["table"].view(5, 16)
    k_bytes = sum(r * d for r, d in groups) * TILE // 8
    kc = _exact_codes(tiles[:, :k_bytes], 0, groups, c["v_rate"])
    vc = _exact_codes(tiles[:, k_bytes:lay["code_bytes"]], 1, groups, c["v_rate"])
    raw = tiles[:, lay["code_bytes"]:].contiguous()
    rows = raw.view(torch.float16 if c["norm16"] else torch.float32).double().view(len(tiles), -1, TILE)
    tok = torch.arange(TILE, device=tiles.device)
    by_token = rows[:, :, 8 * (tok % 8) + tok // 8]
    k = torch.zeros(len(tiles), TILE, HEAD_DIM, dtype=torch.float64, device=tiles.device)
    p = 0
    for i, (r, d) in enumerate(groups):
        y = table[r][kc[:, :, p:p + d]] * (by_token[:, i] / math.sqrt(d)).unsqueeze(-1)
        k += y @ lay["k_rot"][p:p + d]
        p += d
    v = (table[c["v_rate"]][vc] * (by_token[:, -1] / math.sqrt(128)).unsqueeze(-1)) @ lay["v_rot"]
    return k.view(-1, HEAD_DIM), v.view(-1, HEAD_DIM)


def _exact_kept_sums(case, s):
    """The kept tokens' sums, chosen one (row, KV head) at a time."""
    out = np.zeros(tuple(s["mass_out"].shape))
    sums, lens = s["mass"].cpu().numpy(), s["lens"].tolist()
    for row in range(case["batch"]):
        n = lens[row]
        for head in range(case["h_kv"]):
            x = sums[row, head, :n]
            if n > case["keep"]:
                mid = np.arange(case["sinks"], n - case["recent"])
                want = case["keep"] - case["sinks"] - case["recent"]
                best = mid[np.lexsort((mid, -x[mid]))][:want]
                x = x[np.sort(np.concatenate([np.arange(case["sinks"]), best, np.arange(n - case["recent"], n)]))]
            out[row, head, :len(x)] = x
    return torch.from_numpy(out).cuda()


def exact(case, seed):
    if case["op"] == "commit":
        return None                       # bytes and lengths: nothing is computed
    s = prepare(case, seed)
    if case["op"] == "evict":
        return {"cache": None, "mass": _exact_kept_sums(case, s), "kept": None, "lens": None}
    lens = s["lens"].tolist()
    b, h, g, n = case["batch"], case["h_kv"], case["group"], max(1, case["nodes"])
    q = s["q"].double().view(b, n, h, g, HEAD_DIM)
    out = torch.zeros_like(q)
    mass = s["mass"].double().clone() if case["op"] == "mass" else None
    for row in range(b):
        length = lens[row]
        nt = -(-length // TILE)
        see = torch.ones(n, length, dtype=torch.bool, device="cuda")
        if case["op"] == "tree":
            bits = torch.arange(n, device="cuda")
            see[:, length - n:] = ((s["mask"][row].view(n, 1) >> bits) & 1).bool()
        for head in range(h):
            tiles = s["pool"][s["table"][row, :nt].long(), head] if case["paged"] else s["cache"][row, head, :nt]
            k, v = _exact_unit(s, tiles)
            x = torch.einsum("ngd,td->ngt", q[row, :, head], k[:length]) * s["scale"]
            x = x.masked_fill(~see.unsqueeze(1), -math.inf)
            p = torch.softmax(x, -1)
            out[row, :, head] = torch.einsum("ngt,td->ngd", p, v[:length])
            if mass is not None:
                mass[row, head, :length] = case["decay"] * mass[row, head, :length] + p.sum((0, 1))
    if case["op"] == "tree":
        return {"out": out.view(b, n, h * g, HEAD_DIM)}
    return {"out": out.view(b, h * g, HEAD_DIM), "mass": mass}
