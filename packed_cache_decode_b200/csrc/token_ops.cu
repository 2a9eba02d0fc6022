// Tokens moved inside and between packed caches, codes and norms bit for bit (nothing is
// decoded or re-encoded):
//  * tree commit: the accepted path of a drafted tree to the end of the prefix, in place;
//  * eviction: the `keep` tokens of a (row, KV head) with the largest attention mass (the
//    first and the newest ones always) chosen by a radix selection, then gathered into
//    another cache.
//
// A tile's codes are fragment-major: a token's codes lie in every lane string of its row
// (token % 8) next to those of seven other tokens, so a token cannot be copied as bytes. A
// CTA brings the whole source tiles of one destination tile into shared memory (bulk
// copies), and every destination string is put together by one lane from the source
// strings of its tokens (shift, mask, or): no atomics, every word written once. A value
// field holds the codes of two neighbouring tokens; a source token's codes of a whole
// 16-bit (8 b-bit) field group move with one mask, since token parity and half only shift
// the group.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "async_copy.cuh"
#include "bgtq_internal.h"
#include "kernels.h"

namespace bgtq {

namespace {

namespace cg = cooperative_groups;

constexpr int kMoveThreads = 256;
constexpr int kMoveSlots = 8;  // source tiles a CTA holds at a time

// Destination string `lane` of key quad Q (rate R): ors in the fields of the destination
// tokens whose source is present. info[t]: source tile's byte offset from `src` + source
// token (offsets are multiples of 64), or -1.
template <int R>
__device__ __forceinline__ void key_string(uint8_t* dst, const uint8_t* src, const int* info, int P, int lane) {
  if (lane >= 8 * P) return;
  const int g = lane / P, e = lane - g * P;
  unsigned long long D = 0;
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const int x = info[g + 8 * m];
    if (x < 0) continue;
    const int tok = x & 63, li = (tok & 7) * P + e, mm = tok >> 3;
    const uint8_t* s = src + (x - tok);
    if constexpr (R == 1) {
      const unsigned w = *reinterpret_cast<const unsigned short*>(s + 2 * li);
      D |= ((w >> mm) & 0x0101u) << m;
    } else if constexpr (R == 2) {
      const unsigned w = *reinterpret_cast<const unsigned*>(s + 4 * li);
      D |= ((w >> (4 * mm)) & 0xFu) << (4 * m);
    } else if constexpr (R == 3) {
      const unsigned lo = *reinterpret_cast<const unsigned*>(s + 4 * li);
      const unsigned hi = *reinterpret_cast<const unsigned short*>(s + 32 * P + 2 * li);
      const unsigned long long w = lo | (static_cast<unsigned long long>(hi) << 32);
      D |= ((w >> (6 * mm)) & 0x3Full) << (6 * m);
    } else {
      D |= static_cast<unsigned long long>(s[8 * li + mm]) << (8 * m);
    }
  }
  if constexpr (R == 1) {
    *reinterpret_cast<unsigned short*>(dst + 2 * lane) |= static_cast<unsigned short>(D);
  } else if constexpr (R == 2) {
    *reinterpret_cast<unsigned*>(dst + 4 * lane) |= static_cast<unsigned>(D);
  } else if constexpr (R == 3) {
    *reinterpret_cast<unsigned*>(dst + 4 * lane) |= static_cast<unsigned>(D);
    *reinterpret_cast<unsigned short*>(dst + 32 * P + 2 * lane) |= static_cast<unsigned short>(D >> 32);
  } else {
    *reinterpret_cast<unsigned long long*>(dst + 8 * lane) |= D;
  }
}

// Words of value string `lane` of a chunk block (rates 3-4: two planes).
template <int VR>
__device__ __forceinline__ void load_value_string(const uint8_t* blk, int lane, unsigned (&w)[2 * VR]) {
  if constexpr (VR == 1) {
    const uint2 x = *reinterpret_cast<const uint2*>(blk + 8 * lane);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(blk + 16 * lane);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
    if constexpr (VR == 3) {
      const uint2 y = *reinterpret_cast<const uint2*>(blk + 512 + 8 * lane);
      w[4] = y.x;
      w[5] = y.y;
    } else if constexpr (VR == 4) {
      const uint4 y = *reinterpret_cast<const uint4*>(blk + 512 + 16 * lane);
      w[4] = y.x;
      w[5] = y.y;
      w[6] = y.z;
      w[7] = y.w;
    }
  }
}
template <int VR>
__device__ __forceinline__ void store_value_string(uint8_t* blk, int lane, const unsigned (&w)[2 * VR]) {
  if constexpr (VR == 1) {
    *reinterpret_cast<uint2*>(blk + 8 * lane) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(blk + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (VR == 3) *reinterpret_cast<uint2*>(blk + 512 + 8 * lane) = make_uint2(w[4], w[5]);
    else if constexpr (VR == 4) *reinterpret_cast<uint4*>(blk + 512 + 16 * lane) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Destination string `lane` of value chunk c: tokens 2 t + 8 h + par of the chunk (h, par in
// 0..1), every one's codes of the lane's 16 dims taken from string 4 g + t' of its source
// chunk. dst, src: the tiles' value areas.
template <int VR>
__device__ __forceinline__ void value_string(uint8_t* dst, const uint8_t* src, const int* info, int c, int lane) {
  const int g = lane >> 2, t = lane & 3;
  uint8_t* blk = dst + c * 256 * VR;
  unsigned D[2 * VR];
  load_value_string<VR>(blk, lane, D);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int h = q >> 1, par = q & 1;
    const int x = info[16 * c + 2 * t + 8 * h + par];
    if (x < 0) continue;
    const int tok = x & 63, jj = tok & 15, hs = jj >> 3, ps = jj & 1;
    unsigned w[2 * VR];
    load_value_string<VR>(src + (x - tok) + (tok >> 4) * 256 * VR, 4 * g + ((jj & 7) >> 1), w);
    if constexpr (VR == 1) {
#pragma unroll
      for (int u = 0; u < 2; ++u) D[u] |= ((w[u] >> (16 * ps + 2 * hs)) & 0x3333u) << (16 * par + 2 * h);
    } else if constexpr (VR == 2) {
#pragma unroll
      for (int u = 0; u < 4; ++u) D[u] |= ((w[u] >> (8 * hs + 2 * ps)) & 0x00330033u) << (8 * h + 2 * par);
    } else if constexpr (VR == 3) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        const int wi = 24 * mt >> 5, sh = 24 * mt & 31;
        const unsigned grp = sh <= 8 ? w[wi] >> sh : __funnelshift_r(w[wi], w[wi + 1], sh);
        const unsigned v = ((grp >> (12 * hs + 3 * ps)) & 0x1C7u) << (12 * h + 3 * par);
        D[wi] |= v << sh;
        if (sh > 8) D[wi + 1] |= v >> (32 - sh);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) D[u] |= ((w[u] >> (16 * hs + 4 * ps)) & 0x0F0Fu) << (16 * h + 4 * par);
    }
  }
  store_value_string<VR>(blk, lane, D);
}

// Ors the tokens that info names into the tile at dst (zero where nothing was put yet).
// Warps take key quads and value chunks in turn; the norms follow.
__device__ __forceinline__ void assemble_tile(const DevLayout& L, uint8_t* dst, const uint8_t* src, const int* info) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nq = L.n_kquads;
  for (int it = warp; it < nq + 4; it += kMoveThreads / 32) {
    if (it < nq) {
      int g = 0;
      while (g + 1 < L.n_kgroups && it >= L.group_quad0[g + 1]) ++g;
      const int off = L.quad_off[it], P = L.quad_np[it];
      switch (L.group_rate[g]) {
        case 1: key_string<1>(dst + off, src + off, info, P, lane); break;
        case 2: key_string<2>(dst + off, src + off, info, P, lane); break;
        case 3: key_string<3>(dst + off, src + off, info, P, lane); break;
        default: key_string<4>(dst + off, src + off, info, P, lane); break;
      }
    } else {
      const int off = L.vcode_off;
      switch (L.v_rate) {
        case 1: value_string<1>(dst + off, src + off, info, it - nq, lane); break;
        case 2: value_string<2>(dst + off, src + off, info, it - nq, lane); break;
        case 3: value_string<3>(dst + off, src + off, info, it - nq, lane); break;
        default: value_string<4>(dst + off, src + off, info, it - nq, lane); break;
      }
    }
  }
  // norm rows of the key groups, then of the values: token g + 8 m of a row at entry 8 g + m
  for (int e = tid; e < (L.n_kgroups + 1) * kTile; e += kMoveThreads) {
    const int row = e >> 6, en = e & 63, x = info[(en >> 3) + 8 * (en & 7)];
    if (x < 0) continue;
    const int tok = x & 63, es = row * kTile + (tok & 7) * 8 + (tok >> 3);
    const uint8_t* s = src + (x - tok) + L.knorm_off;
    if (L.norm_fp16)
      reinterpret_cast<unsigned short*>(dst + L.knorm_off)[e] = reinterpret_cast<const unsigned short*>(s)[es];
    else
      reinterpret_cast<unsigned*>(dst + L.knorm_off)[e] = reinterpret_cast<const unsigned*>(s)[es];
  }
}

__device__ __forceinline__ void zero_tile(uint8_t* p, int bytes) {
  for (int i = threadIdx.x; i < bytes / 16; i += kMoveThreads) reinterpret_cast<uint4*>(p)[i] = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void write_tile(uint8_t* out, const uint8_t* p, int bytes) {
  for (int i = threadIdx.x; i < bytes / 16; i += kMoveThreads)
    reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(p)[i];
}

// Tokens of a row that a call may use: its length, clipped to what the caller sized.
__device__ __forceinline__ int row_tokens(const int* seq_lens, int b, long long most) {
  const long long len = seq_lens[b];
  return int(len < 0 ? 0 : len > most ? most : len);
}

// ------------------------------------------------------------------ tree commit
// One CTA per (row, KV head): the one or two tiles that hold the row's drafted tokens come
// into shared memory whole before anything is written, so a path may name its nodes in any
// order. A path that leaves every token in its place writes nothing. Latency bound: one
// round trip to memory for the lengths and the path, one for the tiles.
__global__ void __launch_bounds__(kMoveThreads) commit_kernel(DevLayout L, CacheRef cache, const int* __restrict__ path,
                                                              int path_ld, const int* __restrict__ n_path,
                                                              const int* __restrict__ n_nodes, int n_q,
                                                              const int* __restrict__ seq_lens,
                                                              int* __restrict__ new_lens, int h_kv) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) unsigned long long bar;
  __shared__ int s_path[64], s_info[2][64], s_state;
  const int tid = threadIdx.x, b = blockIdx.x / h_kv, h = blockIdx.x % h_kv, TB = L.tile_bytes;
  if (tid == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
    s_state = 0;
  }
  __syncthreads();
  const long long len = seq_lens[b];
  const int n = n_nodes ? n_nodes[b] : n_q, a = n_path[b];
  const bool fits = n >= 0 && n <= n_q && a >= 0 && a <= n && len >= n && len <= cache.n_tiles * kTile;
  if (fits && tid < a) {
    const int p = path[(size_t)b * path_ld + tid];
    s_path[tid] = p;
    if (p < 0 || p >= n) atomicOr(&s_state, 1);   // a node that the row does not have
    else if (p != tid) atomicOr(&s_state, 2);     // a token moves
  }
  __syncthreads();
  const bool bad = !fits || (s_state & 1);
  if (h == 0 && tid == 0) new_lens[b] = int(bad ? len : len - n + a);
  if (bad) {
    if (tid == 0) atomicOr(L.status, BGTQ_STATUS_BAD_TREE);
    return;
  }
  if (!(s_state & 2)) return;
  const long long base = len - n;
  const int t0 = int(base / kTile), t1 = int((len - 1) / kTile), last = int((base + a - 1) / kTile);
  uint8_t* tile[2] = {tile_ptr(cache, L, b, h, h_kv, t0), t1 > t0 ? tile_ptr(cache, L, b, h, h_kv, t1) : nullptr};
  if (!tile[0] || (t1 > t0 && !tile[1])) return;  // a page outside the pool (flagged): the row keeps its tokens
  uint8_t* in = smem;
  uint8_t* made = smem + 2 * TB;
  if (tid == 0) {
    mbar_expect_tx(&bar, unsigned(TB) * (t1 > t0 ? 2u : 1u));
    bulk_load(in, tile[0], TB, &bar, evict_last_policy());
    if (t1 > t0) bulk_load(in + TB, tile[1], TB, &bar, evict_last_policy());
  }
  if (tid < 128) {
    // token `place` of the two tiles, counted from the first one's start
    const int place = tid, off = int(base - (long long)t0 * kTile);
    const int from = place >= off && place < off + a ? off + s_path[place - off] : place;
    s_info[tid >> 6][tid & 63] = (from >> 6) * TB + (from & 63);
  }
  zero_tile(made, 2 * TB);
  const bool ok = mbar_wait_bounded(&bar, 0);
  if (__syncthreads_or(!ok)) {
    if (tid == 0) {
      atomicOr(L.status, BGTQ_STATUS_TIMEOUT);
      mbar_wait_bounded(&bar, 0);  // the copies may still land: wait (bounded) before leaving
    }
    __syncthreads();
    return;
  }
  assemble_tile(L, made, in, s_info[0]);
  if (last > t0) assemble_tile(L, made + TB, in, s_info[1]);
  __syncthreads();
  write_tile(tile[0], made, TB);
  if (last > t0) write_tile(tile[1], made + TB, TB);
}

// ------------------------------------------------------------------ eviction: selection
// The keep-th largest key of a unit by radix selection (digits of 11, 11 and 10 bits, most
// significant first) over a cluster of CTAs, each holding its share of the unit's keys in
// shared memory (as many as fit; the others are read again): one read of the mass. Every
// CTA adds up the cluster's histograms over distributed shared memory and finds the same
// digit. Then the kept tokens are written in their order: those above the threshold, and
// of those equal to it the first ones.
constexpr int kSelThreads = 512;
constexpr int kBins = 2048;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelSpan = 8;                             // 32-token spans a warp takes at a time
constexpr int kSelStep = kSelThreads * kSelSpan;        // tokens a CTA takes at a time

// Mass as an unsigned key of the same order; -0 is 0, NaN comes last.
__device__ __forceinline__ unsigned mass_key(float x) {
  if (x != x) return 0u;
  const unsigned u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct SelectArgs {
  const float* mass;
  long long mass_ld, most;   // most: tokens a row may have in this call
  const int* seq_lens;
  int h_kv, keep, n_sink, n_recent, cluster, cached;
  int* kept;                 // [units][keep]
  float* mass_out;
  long long mass_out_ld;
  int* new_lens;
  unsigned* status;
};

__global__ void __launch_bounds__(kSelThreads) select_kernel(SelectArgs a) {
  extern __shared__ __align__(16) unsigned s_keys[];   // a.cached keys
  __shared__ __align__(16) int s_hist[kBins];
  __shared__ int s_warp[2][kSelWarps], s_find[2], s_total[2];
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster, b = u / a.h_kv;
  pdl_trigger();
  const int n = row_tokens(a.seq_lens, b, a.most);
  if (tid == 0 && rank == 0 && a.seq_lens[b] > a.most) atomicOr(a.status, BGTQ_STATUS_DECODE_CLAMPED);
  const int n_new = min(n, a.keep);
  const float* mass = a.mass + (size_t)u * a.mass_ld;
  int* kept = a.kept + (size_t)u * a.keep;
  float* mass_out = a.mass_out + (size_t)u * a.mass_out_ld;
  const int all = a.cluster * kSelThreads, me = rank * kSelThreads + tid;
  if (u % a.h_kv == 0 && me == 0) a.new_lens[b] = n_new;
  for (int i = n_new + me; i < a.keep; i += all) kept[i] = -1;
  for (long long i = n_new + me; i < a.mass_out_ld; i += all) mass_out[i] = 0.f;
  if (n <= a.keep) {  // the same for the whole cluster
    for (int i = me; i < n; i += all) {
      kept[i] = i;
      mass_out[i] = mass[i];
    }
    return;
  }
  const int per = ((n + a.cluster - 1) / a.cluster + 31) & ~31;
  const int c0 = min(n, rank * per), c1 = min(n, c0 + per);
  auto make_key = [&](int i) {
    return i < a.n_sink || i >= n - a.n_recent ? 0xffffffffu : mass_key(mass[i]);
  };
  auto key = [&](int i) { return i - c0 < a.cached ? s_keys[i - c0] : make_key(i); };
  for (int i = c0 + tid; i < min(c1, c0 + a.cached); i += kSelThreads) s_keys[i - c0] = make_key(i);

  unsigned prefix = 0;
  int need = a.keep;   // tokens to take among those whose higher digits equal the prefix
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    const unsigned above = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
    reinterpret_cast<int4*>(s_hist)[tid] = make_int4(0, 0, 0, 0);
    __syncthreads();
    for (int i = c0 + tid; i < c1; i += kSelThreads) {
      const unsigned k = key(i);
      if ((k & above) == prefix) atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1u)], 1);
    }
    cl.sync();
    // thread t: bins 4 (511 - t) .. + 3, the highest digits first
    const int at = kSelThreads - 1 - tid;
    int4 s = make_int4(0, 0, 0, 0);
    for (int r = 0; r < a.cluster; ++r) {
      const int4 x = reinterpret_cast<const int4*>(cl.map_shared_rank(s_hist, r))[at];
      s = make_int4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
    }
    const int sum = s.x + s.y + s.z + s.w;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[0][warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < warp; ++w) before += s_warp[0][w];
    if (before < need && before + sum >= need) {  // exactly one thread: the digit is one of its four
      const int d[4] = {s.w, s.z, s.y, s.x};
      int j = 0;
      while (before + d[j] < need) before += d[j++];
      s_find[0] = 4 * at + 3 - j;
      s_find[1] = before;
    }
    cl.sync();  // the histograms are read: they may be cleared (and s_find is written)
    prefix |= unsigned(s_find[0]) << shift;
    need -= s_find[1];
  }
  // prefix: the threshold; need: how many of the tokens equal to it are kept
  int gt = 0, eq = 0;
  for (int i = c0 + tid; i < c1; i += kSelThreads) {
    const unsigned k = key(i);
    gt += k > prefix;
    eq += k == prefix;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if (lane == 0) {
    s_warp[0][warp] = gt;
    s_warp[1][warp] = eq;
  }
  __syncthreads();
  if (tid < 2) {
    int t = 0;
    for (int w = 0; w < kSelWarps; ++w) t += s_warp[tid][w];
    s_total[tid] = t;
  }
  cl.sync();
  int base_gt = 0, base_eq = 0;
  for (int r = 0; r < rank; ++r) {
    const int* t = cl.map_shared_rank(s_total, r);
    base_gt += t[0];
    base_eq += t[1];
  }
  cl.sync();  // no CTA leaves while another reads its totals
  for (int s0 = c0; s0 < c1; s0 += kSelStep) {
    unsigned mg[kSelSpan], me2[kSelSpan];
    int wg = 0, we = 0;
    const int w0 = s0 + warp * 32 * kSelSpan;
#pragma unroll
    for (int j = 0; j < kSelSpan; ++j) {
      const int i = w0 + 32 * j + lane;
      const unsigned k = i < c1 ? key(i) : 0u;
      mg[j] = __ballot_sync(0xffffffffu, i < c1 && k > prefix);
      me2[j] = __ballot_sync(0xffffffffu, i < c1 && k == prefix);
      wg += __popc(mg[j]);
      we += __popc(me2[j]);
    }
    __syncthreads();  // the last step's totals are read
    if (lane == 0) {
      s_warp[0][warp] = wg;
      s_warp[1][warp] = we;
    }
    __syncthreads();
    int g0 = base_gt, e0 = base_eq;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) {
        g0 += s_warp[0][w];
        e0 += s_warp[1][w];
      }
      base_gt += s_warp[0][w];
      base_eq += s_warp[1][w];
    }
    const unsigned lt = (1u << lane) - 1u;
#pragma unroll
    for (int j = 0; j < kSelSpan; ++j) {
      const int i = w0 + 32 * j + lane;
      const int eb = e0 + __popc(me2[j] & lt), gb = g0 + __popc(mg[j] & lt);
      if ((mg[j] >> lane & 1u) || ((me2[j] >> lane & 1u) && eb < need)) {
        const int p = gb + min(eb, need);
        kept[p] = i;
        mass_out[p] = mass[i];
      }
      g0 += __popc(mg[j]);
      e0 += __popc(me2[j]);
    }
  }
}

// ------------------------------------------------------------------ eviction: gather
// One CTA per destination tile. Bound by memory: the tiles that hold kept tokens are read
// once (a tile that serves two destination tiles comes from L2 the second time), the kept
// tokens are written once.
__global__ void __launch_bounds__(kMoveThreads) gather_kernel(DevLayout L, CacheRef src, CacheRef dst,
                                                              const int* __restrict__ kept,
                                                              const int* __restrict__ seq_lens, long long most,
                                                              int keep, int h_kv) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) unsigned long long bar;
  __shared__ int s_tile[64], s_slot[64], s_tok[64], s_info[64], s_cnt[2];
  const int tid = threadIdx.x, lane = tid & 31, j = blockIdx.x, u = blockIdx.y, b = u / h_kv, h = u % h_kv;
  const int TB = L.tile_bytes;
  uint8_t* made = smem;
  uint8_t* in = smem + TB;
  if (tid == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  zero_tile(made, TB);
  pdl_wait();  // the kept tokens come from the selection
  const int n = row_tokens(seq_lens, b, most), n_new = min(n, keep);
  if (j * kTile >= n_new) return;
  // the source tiles in order: slot of a token = distinct tiles before its own
  int idx = -1;
  if (tid < 64) {
    if (j * kTile + tid < n_new) idx = kept[(size_t)u * keep + j * kTile + tid];
    if (idx >= n) idx = -1;
    s_tile[tid] = idx >> 6;  // (-1 stays -1)
    s_tok[tid] = idx & 63;
  }
  __syncthreads();
  unsigned firsts = 0;
  if (tid < 64) {
    const bool first = idx >= 0 && (tid == 0 || s_tile[tid] != s_tile[tid - 1]);
    firsts = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s_cnt[tid >> 5] = __popc(firsts);
  }
  __syncthreads();
  if (tid < 64) {
    const int s = (tid >= 32 ? s_cnt[0] : 0) + __popc(firsts & (0xffffffffu >> (31 - lane))) - 1;
    s_slot[tid] = idx >= 0 ? s : -1;
  }
  __syncthreads();
  const int n_slots = s_cnt[0] + s_cnt[1];
  unsigned phase = 0;
  for (int b0 = 0; b0 < n_slots; b0 += kMoveSlots, phase ^= 1u) {
    const int cnt = min(kMoveSlots, n_slots - b0);
    if (tid < 64) {
      const int s = s_slot[tid] - b0;
      s_info[tid] = s_slot[tid] >= 0 && s >= 0 && s < cnt && tile_present(src, b, s_tile[tid]) ? s * TB + s_tok[tid] : -1;
    }
    if (tid < 32) {
      // lane s: source tile of slot b0 + s (the first token with that slot names it)
      const uint8_t* p = nullptr;
      if (lane < cnt) {
        int i = 0;
        while (s_slot[i] != b0 + lane) ++i;
        p = tile_ptr(src, L, b, h, h_kv, s_tile[i]);
      }
      const int live = __popc(__ballot_sync(0xffffffffu, p != nullptr));
      if (lane == 0) mbar_expect_tx(&bar, unsigned(TB) * unsigned(live));
      __syncwarp();
      if (p) bulk_load(in + lane * TB, p, TB, &bar, evict_first_policy());
    }
    const bool ok = mbar_wait_bounded(&bar, phase);
    if (__syncthreads_or(!ok)) {
      if (tid == 0) {
        atomicOr(L.status, BGTQ_STATUS_TIMEOUT);
        mbar_wait_bounded(&bar, phase);  // the copies may still land: wait (bounded) before leaving
      }
      __syncthreads();
      return;
    }
    assemble_tile(L, made, in, s_info);
    __syncthreads();
  }
  uint8_t* out = tile_ptr(dst, L, b, h, h_kv, j);
  if (out) write_tile(out, made, TB);
}

int optin_smem(int* dev_out) {
  int dev = 0, optin = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
    return 0;
  *dev_out = dev;
  return optin;
}

// Once per device: the kernel's dynamic shared memory limit raised to what a block may use.
template <typename K>
cudaError_t raise_limit(K kernel, bool (&done)[64]) {
  int dev = 0;
  const int optin = optin_smem(&dev);
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  cudaFuncAttributes fa{};
  cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - int(fa.sharedSizeBytes));
  done[dev] = e == cudaSuccess;
  return e;
}

}  // namespace

cudaError_t launch_commit(const DevLayout& L, int batch, int h_kv, const int* path, int path_ld, const int* n_path,
                          const int* n_nodes, int n_q, const CacheRef& cache, const int* seq_lens, int* new_lens,
                          cudaStream_t stream) {
  static bool done[64] = {};
  cudaError_t e = raise_limit(commit_kernel, done);
  if (e != cudaSuccess) return e;
  commit_kernel<<<unsigned(batch * h_kv), kMoveThreads, 4 * L.tile_bytes, stream>>>(
      L, cache, path, path_ld, n_path, n_nodes, n_q, seq_lens, new_lens, h_kv);
  return cudaGetLastError();
}

cudaError_t launch_evict(const DevLayout& L, int batch, int h_kv, const CacheRef& src, const int* seq_lens,
                         long long max_seq_len, const float* mass, long long mass_ld, int keep, int n_sink,
                         int n_recent, const CacheRef& dst, float* mass_out, long long mass_out_ld, int* kept,
                         int* new_lens, int num_sms, cudaStream_t stream) {
  static bool sel_done[64] = {}, gat_done[64] = {};
  cudaError_t e = raise_limit(select_kernel, sel_done);
  if (e == cudaSuccess) e = raise_limit(gather_kernel, gat_done);
  if (e != cudaSuccess) return e;
  const int units = batch * h_kv;
  // CTAs per unit: enough to fill the SMs or to leave each at most 4096 tokens, 8 at most
  int cluster = 1;
  while (cluster < 8 && units * cluster < num_sms && max_seq_len > 4096LL * cluster) cluster *= 2;
  const long long per = (max_seq_len + cluster - 1) / cluster + 31;
  SelectArgs a{mass, mass_ld, max_seq_len, seq_lens, h_kv, keep, n_sink, n_recent, cluster,
               int(std::min<long long>(per, 24 * 1024)), kept, mass_out, mass_out_ld, new_lens, L.status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units * cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = size_t(a.cached) * sizeof(unsigned);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, select_kernel, a);
  if (e != cudaSuccess) return e;
  const long long tiles = (std::min<long long>(keep, max_seq_len) + kTile - 1) / kTile;
  if (!tiles) return cudaSuccess;  // no row holds a token
  cudaLaunchConfig_t gcfg = {};
  gcfg.gridDim = dim3(unsigned(tiles), unsigned(units));
  gcfg.blockDim = dim3(kMoveThreads);
  gcfg.dynamicSmemBytes = size_t(kMoveSlots + 1) * L.tile_bytes;
  gcfg.stream = stream;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  gcfg.attrs = pdl;
  gcfg.numAttrs = 1;
  return cudaLaunchKernelEx(&gcfg, gather_kernel, L, src, dst, (const int*)kept, seq_lens, max_seq_len, keep, h_kv);
}

}  // namespace bgtq
