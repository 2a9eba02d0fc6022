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

constexpr int kCommitThreads = 256, kGatherThreads = 128;
constexpr int kMoveSlots = 5;  // source tiles a CTA holds at a time

// Where the codes of the 64 destination tokens come from, as each part of a tile needs it (byte
// offsets count from the source tiles' start; a token without a source points at a tile of
// zeros, so nothing branches on it):
//  raw: offset of the source tile, row (token % 8) | slot (token / 8) << 8;
//  key[r - 1]: offset of the row's strings in a full quad of rate r, shift of the slot's field
//    (rate 3: | 8 row << 8 for the second plane; rate 4: the byte is in the offset);
//  value: offset of the token's string in its chunk (lane row / 2 of the first four), shift of
//    its half and parity;
//  norm: offset of its entry in the first row of norms.
struct Moves {
  int2 raw[64], key[4][64], value[64];
  int norm[64];
};
__device__ __forceinline__ void set_move(const DevLayout& L, Moves& mv, int t, int off, int tok) {
  const int g = tok & 7, m = tok >> 3, hs = m & 1, ps = g & 1, b = L.v_rate;
  mv.raw[t] = make_int2(off, g | m << 8);
  mv.key[0][t] = make_int2(off + 8 * g, m);
  mv.key[1][t] = make_int2(off + 16 * g, 4 * m);
  mv.key[2][t] = make_int2(off + 16 * g, 6 * m | (8 * g) << 8);
  mv.key[3][t] = make_int2(off + 32 * g + m, 0);
  const int lane = g >> 1;
  mv.value[t] = make_int2(off + L.vcode_off + (m >> 1) * 256 * b + (b == 1 ? 8 : 16) * lane,
                          (b == 1 ? 16 * ps + 2 * hs : 4 * b * hs + b * ps) | (b == 3 ? 8 : 16) * lane << 8);
  mv.norm[t] = off + L.knorm_off + (L.norm_fp16 ? 2 : 4) * (g * 8 + m);
}

// ADD: ors into what was put before, else stores.
template <bool ADD, typename T>
__device__ __forceinline__ void put(T* p, T v) {
  if constexpr (ADD) *p |= v;
  else *p = v;
}

// Destination string `lane` of a key quad with P < 4 pairs (rate R): its 8 tokens' fields.
template <int R, bool ADD>
__device__ __forceinline__ void key_string(uint8_t* dst, const uint8_t* src, const int2* raw, int P, int lane) {
  if (lane >= 8 * P) return;
  const int g = lane / P, e = lane - g * P;
  unsigned long long D = 0;
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const int2 x = raw[g + 8 * m];
    const int li = (x.y & 7) * P + e, mm = x.y >> 8;
    const uint8_t* s = src + x.x;
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
    put<ADD>(reinterpret_cast<unsigned short*>(dst + 2 * lane), static_cast<unsigned short>(D));
  } else if constexpr (R == 2) {
    put<ADD>(reinterpret_cast<unsigned*>(dst + 4 * lane), static_cast<unsigned>(D));
  } else if constexpr (R == 3) {
    put<ADD>(reinterpret_cast<unsigned*>(dst + 4 * lane), static_cast<unsigned>(D));
    put<ADD>(reinterpret_cast<unsigned short*>(dst + 32 * P + 2 * lane), static_cast<unsigned short>(D >> 32));
  } else {
    put<ADD>(reinterpret_cast<unsigned long long*>(dst + 8 * lane), D);
  }
}

// The same for a full quad (lane = 4 row + pair): one or two loads, a shift and a mask per token.
template <int R, bool ADD>
__device__ __forceinline__ void full_key_string(uint8_t* dst, const uint8_t* src, const int2* key, int lane) {
  const int g = lane >> 2, e = lane & 3;
  unsigned D = 0, D1 = 0;
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const int2 x = key[g + 8 * m];
    const uint8_t* s = src + x.x;
    if constexpr (R == 1) {
      const unsigned w = *reinterpret_cast<const unsigned short*>(s + 2 * e);
      D |= ((w >> x.y) & 0x0101u) << m;
    } else if constexpr (R == 2) {
      const unsigned w = *reinterpret_cast<const unsigned*>(s + 4 * e);
      D |= ((w >> x.y) & 0xFu) << (4 * m);
    } else if constexpr (R == 3) {
      const unsigned lo = *reinterpret_cast<const unsigned*>(s + 4 * e);
      const unsigned hi = *reinterpret_cast<const unsigned short*>(s + 128 - (x.y >> 8) + 2 * e);
      const int sh = x.y & 0xff;
      const unsigned f = (sh < 32 ? __funnelshift_r(lo, hi, sh) : hi >> (sh - 32)) & 0x3Fu;
      if (6 * m < 32) D |= f << (6 * m);
      if (6 * m + 6 > 32) D1 |= 6 * m >= 32 ? f << (6 * m - 32) : f >> (32 - 6 * m);
    } else {
      const unsigned f = s[8 * e];
      if (m < 4) D |= f << (8 * m);
      else D1 |= f << (8 * m - 32);
    }
  }
  if constexpr (R == 1) {
    put<ADD>(reinterpret_cast<unsigned short*>(dst + 2 * lane), static_cast<unsigned short>(D));
  } else if constexpr (R == 2) {
    put<ADD>(reinterpret_cast<unsigned*>(dst + 4 * lane), D);
  } else if constexpr (R == 3) {
    put<ADD>(reinterpret_cast<unsigned*>(dst + 4 * lane), D);
    put<ADD>(reinterpret_cast<unsigned short*>(dst + 128 + 2 * lane), static_cast<unsigned short>(D1));
  } else {
    put<ADD>(reinterpret_cast<unsigned long long*>(dst + 8 * lane), D | static_cast<unsigned long long>(D1) << 32);
  }
}

// Words of a value string at s (rates 3-4: the second plane's words at s2).
template <int VR>
__device__ __forceinline__ void load_value_string(const uint8_t* s, const uint8_t* s2, unsigned (&w)[2 * VR]) {
  if constexpr (VR == 1) {
    const uint2 x = *reinterpret_cast<const uint2*>(s);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(s);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
    if constexpr (VR == 3) {
      const uint2 y = *reinterpret_cast<const uint2*>(s2);
      w[4] = y.x;
      w[5] = y.y;
    } else if constexpr (VR == 4) {
      const uint4 y = *reinterpret_cast<const uint4*>(s2);
      w[4] = y.x;
      w[5] = y.y;
      w[6] = y.z;
      w[7] = y.w;
    }
  }
}
template <int VR>
__device__ __forceinline__ void store_value_string(uint8_t* s, uint8_t* s2, const unsigned (&w)[2 * VR]) {
  if constexpr (VR == 1) {
    *reinterpret_cast<uint2*>(s) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(s) = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (VR == 3) *reinterpret_cast<uint2*>(s2) = make_uint2(w[4], w[5]);
    else if constexpr (VR == 4) *reinterpret_cast<uint4*>(s2) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Destination string `lane` of value chunk c: tokens 2 t + 8 h + par of the chunk (h, par in
// 0..1), every one's codes of the lane's 16 dims taken from string 4 g + t' of its source
// chunk. dst: the tile's value area; src: the source tiles.
template <int VR, bool ADD>
__device__ __forceinline__ void value_string(uint8_t* dst, const uint8_t* src, const int2* value, int c, int lane) {
  const int g = lane >> 2, t = lane & 3;
  // bytes per string in each plane
  constexpr int B1 = VR == 1 ? 8 : 16, B2 = VR == 3 ? 8 : 16;
  uint8_t* d1 = dst + c * 256 * VR + B1 * lane;
  uint8_t* d2 = dst + c * 256 * VR + 512 + B2 * lane;
  unsigned D[2 * VR];
  if constexpr (ADD) {
    load_value_string<VR>(d1, d2, D);
  } else {
#pragma unroll
    for (int i = 0; i < 2 * VR; ++i) D[i] = 0u;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int h = q >> 1, par = q & 1;
    const int2 x = value[16 * c + 2 * t + 8 * h + par];
    const int sh = x.y & 0xff, l2 = x.y >> 8;   // l2: the second plane's offset of the lane (row / 2)
    const uint8_t* s = src + x.x + 4 * B1 * g;
    unsigned w[2 * VR];
    load_value_string<VR>(s, VR >= 3 ? src + (x.x - B1 * (l2 / B2)) + 512 + l2 + 4 * B2 * g : s, w);
    if constexpr (VR == 1) {
#pragma unroll
      for (int u = 0; u < 2; ++u) D[u] |= ((w[u] >> sh) & 0x3333u) << (16 * par + 2 * h);
    } else if constexpr (VR == 2) {
#pragma unroll
      for (int u = 0; u < 4; ++u) D[u] |= ((w[u] >> sh) & 0x00330033u) << (8 * h + 2 * par);
    } else if constexpr (VR == 3) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        const int wi = 24 * mt >> 5, b0 = 24 * mt & 31;
        const unsigned grp = b0 <= 8 ? w[wi] >> b0 : __funnelshift_r(w[wi], w[wi + 1], b0);
        const unsigned v = ((grp >> sh) & 0x1C7u) << (12 * h + 3 * par);
        D[wi] |= v << b0;
        if (b0 > 8) D[wi + 1] |= v >> (32 - b0);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) D[u] |= ((w[u] >> sh) & 0x0F0Fu) << (16 * h + 4 * par);
    }
  }
  store_value_string<VR>(d1, d2, D);
}

// The layout's quads as a kernel parameter: byte offset | pairs << 20 | rate << 24.
struct QuadList {
  unsigned q[kMaxQuads];
};
QuadList quad_list(const DevLayout& L) {
  QuadList l{};
  for (int g = 0; g < L.n_kgroups; ++g)
    for (int i = 0; i < L.group_nquads[g]; ++i) {
      const int it = L.group_quad0[g] + i;
      l.q[it] = unsigned(L.quad_off[it]) | unsigned(L.quad_np[it]) << 20 | unsigned(L.group_rate[g]) << 24;
    }
  return l;
}

// Puts the tokens that mv names into the tile at dst (ADD: next to those put there before).
// NT threads: warps take key quads and value chunks in turn; the norms follow.
template <int NT, bool ADD>
__device__ __forceinline__ void assemble_tile(const DevLayout& L, const QuadList& ql, uint8_t* dst, const uint8_t* src,
                                              const Moves& mv) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nq = L.n_kquads;
#pragma unroll 1
  for (int it = warp; it < nq + 4; it += NT / 32) {
    if (it < nq) {
      const unsigned q = ql.q[it];
      const int off = q & 0xfffffu, P = q >> 20 & 15u;
      if (P == 4) {
        switch (q >> 24) {
          case 1: full_key_string<1, ADD>(dst + off, src + off, mv.key[0], lane); break;
          case 2: full_key_string<2, ADD>(dst + off, src + off, mv.key[1], lane); break;
          case 3: full_key_string<3, ADD>(dst + off, src + off, mv.key[2], lane); break;
          default: full_key_string<4, ADD>(dst + off, src + off, mv.key[3], lane); break;
        }
      } else {
        switch (q >> 24) {
          case 1: key_string<1, ADD>(dst + off, src + off, mv.raw, P, lane); break;
          case 2: key_string<2, ADD>(dst + off, src + off, mv.raw, P, lane); break;
          case 3: key_string<3, ADD>(dst + off, src + off, mv.raw, P, lane); break;
          default: key_string<4, ADD>(dst + off, src + off, mv.raw, P, lane); break;
        }
      }
    } else {
      uint8_t* d = dst + L.vcode_off;
      switch (L.v_rate) {
        case 1: value_string<1, ADD>(d, src, mv.value, it - nq, lane); break;
        case 2: value_string<2, ADD>(d, src, mv.value, it - nq, lane); break;
        case 3: value_string<3, ADD>(d, src, mv.value, it - nq, lane); break;
        default: value_string<4, ADD>(d, src, mv.value, it - nq, lane); break;
      }
    }
  }
  // norm rows of the key groups, then of the values: token g + 8 m of a row at entry 8 g + m
  // (a token without a source adds the zeros it points at)
  const int t = tid & 63, en = (t & 7) * 8 + (t >> 3);
  const uint8_t* s = src + mv.norm[t];
#pragma unroll 1
  for (int row = tid >> 6; row <= L.n_kgroups; row += NT / 64) {
    if (L.norm_fp16) put<ADD>(reinterpret_cast<unsigned short*>(dst + L.knorm_off) + row * kTile + en, reinterpret_cast<const unsigned short*>(s)[row * kTile]);
    else put<ADD>(reinterpret_cast<unsigned*>(dst + L.knorm_off) + row * kTile + en, reinterpret_cast<const unsigned*>(s)[row * kTile]);
  }
}

template <int NT>
__device__ __forceinline__ void zero_tile(uint8_t* p, int bytes) {
  for (int i = threadIdx.x; i < bytes / 16; i += NT) reinterpret_cast<uint4*>(p)[i] = make_uint4(0, 0, 0, 0);
}
template <int NT>
__device__ __forceinline__ void write_tile(uint8_t* out, const uint8_t* p, int bytes) {
  for (int i = threadIdx.x; i < bytes / 16; i += NT)
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
// round trip to memory for the lengths and the path, one for the tiles (8 CTAs 4.1 us, 512
// CTAs of two tiles each 6.8 us in a CUDA graph).
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(DevLayout L, const __grid_constant__ QuadList ql, CacheRef cache, const int* __restrict__ path,
                                                              int path_ld, const int* __restrict__ n_path,
                                                              const int* __restrict__ n_nodes, int n_q,
                                                              const int* __restrict__ seq_lens,
                                                              int* __restrict__ new_lens, int h_kv) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) unsigned long long bar;
  __shared__ int s_path[64], s_state;
  __shared__ __align__(8) Moves s_mv[2];
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
    set_move(L, s_mv[tid >> 6], tid & 63, (from >> 6) * TB, from & 63);
  }
  const bool ok = tid < 32 ? mbar_wait_bounded(&bar, 0) : true;  // (one warp polls)
  if (__syncthreads_or(!ok)) {
    if (tid == 0) {
      atomicOr(L.status, BGTQ_STATUS_TIMEOUT);
      mbar_wait_bounded(&bar, 0);  // the copies may still land: wait (bounded) before leaving
    }
    __syncthreads();
    return;
  }
  assemble_tile<kCommitThreads, false>(L, ql, made, in, s_mv[0]);
  if (last > t0) assemble_tile<kCommitThreads, false>(L, ql, made + TB, in, s_mv[1]);
  __syncthreads();
  write_tile<kCommitThreads>(tile[0], made, TB);
  if (last > t0) write_tile<kCommitThreads>(tile[1], made + TB, TB);
}

// ------------------------------------------------------------------ eviction: selection
// The keep-th largest key of a unit by radix selection (digits of 11, 11 and 10 bits, most
// significant first) over a cluster of CTAs, each holding its share of the unit's keys in
// shared memory (as many as fit; the others are read again): one read of the mass. Every
// CTA adds up the cluster's histograms over distributed shared memory and finds the same
// digit. Then the kept tokens are written in their order: those above the threshold, and
// of those equal to it the first ones. Bound by the cluster's round trips (19 us of latency in a
// small call, 47 us for 16 MB of masses in 128 units, cold).
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

__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(SelectArgs a) {
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
  {
    const int ce = min(c1, c0 + a.cached);
    for (int i0 = c0 + tid; i0 < ce; i0 += 8 * kSelThreads) {  // eight loads in flight
      unsigned k[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = i0 + j * kSelThreads < ce ? make_key(i0 + j * kSelThreads) : 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + j * kSelThreads < ce) s_keys[i0 + j * kSelThreads - c0] = k[j];
    }
  }

  // fn(key) for every key of the CTA, the cached ones four at a time
  const int nc = min(c1 - c0, a.cached);
  auto for_keys = [&](auto fn) {
    for (int i = 4 * tid; i < nc; i += 4 * kSelThreads) {
      const uint4 k = *reinterpret_cast<const uint4*>(s_keys + i);
      fn(k.x);
      if (i + 1 < nc) fn(k.y);
      if (i + 2 < nc) fn(k.z);
      if (i + 3 < nc) fn(k.w);
    }
    for (int i = c0 + nc + tid; i < c1; i += kSelThreads) fn(make_key(i));
  };
  unsigned prefix = 0;
  int need = a.keep;   // tokens to take among those whose higher digits equal the prefix
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    const unsigned above = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
    reinterpret_cast<int4*>(s_hist)[tid] = make_int4(0, 0, 0, 0);
    __syncthreads();
    for_keys([&](unsigned k) {
      if ((k & above) == prefix) atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1u)], 1);
    });
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
  for_keys([&](unsigned k) {
    gt += k > prefix;
    eq += k == prefix;
  });
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
// tokens are written once. 16 rows x 8 heads of 25K tokens to 8K (375 MB in all): 107 us, 3.5
// TB/s; what keeps it from 57 is moving codes between bit positions in shared memory.
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(DevLayout L, const __grid_constant__ QuadList ql, CacheRef src, CacheRef dst,
                                                              const int* __restrict__ kept,
                                                              const int* __restrict__ seq_lens, long long most,
                                                              int keep, int h_kv) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) unsigned long long bar;
  __shared__ int s_tile[64], s_src[64], s_cnt[2];
  __shared__ __align__(8) Moves s_mv;
  const int tid = threadIdx.x, lane = tid & 31, j = blockIdx.x, u = blockIdx.y, b = u / h_kv, h = u % h_kv;
  const int TB = L.tile_bytes;
  uint8_t* made = smem;
  uint8_t* in = smem + TB;                        // kMoveSlots source tiles, then one of zeros
  if (tid == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  pdl_wait();  // the kept tokens come from the selection
  const int n = row_tokens(seq_lens, b, most), n_new = min(n, keep);
  if (j * kTile >= n_new) return;
  // the source tiles in order: slot of a token = distinct tiles before its own
  int idx = -1, slot = -1;
  if (tid < 64) {
    if (j * kTile + tid < n_new) idx = kept[(size_t)u * keep + j * kTile + tid];
    if (idx >= n) idx = -1;
    s_tile[tid] = idx >> 6;  // (-1 stays -1)
  }
  __syncthreads();
  unsigned firsts = 0;
  bool first = false;
  if (tid < 64) {
    first = idx >= 0 && (tid == 0 || s_tile[tid] != s_tile[tid - 1]);
    firsts = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s_cnt[tid >> 5] = __popc(firsts);
  }
  __syncthreads();
  const int n_slots = s_cnt[0] + s_cnt[1];
  if (tid < 64 && idx >= 0) {
    slot = (tid >= 32 ? s_cnt[0] : 0) + __popc(firsts & (0xffffffffu >> (31 - lane))) - 1;
    if (first) s_src[slot] = idx >> 6;
  }
  __syncthreads();
  // a token without a source in a batch points at zeros
  if (n_slots > kMoveSlots || j * kTile + kTile > n_new || src.table) zero_tile<kGatherThreads>(in + kMoveSlots * TB, TB);
  unsigned phase = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < n_slots; b0 += kMoveSlots, phase ^= 1u) {
    const int cnt = min(kMoveSlots, n_slots - b0);
    if (tid < 64) {
      const bool here = slot >= b0 && slot < b0 + cnt && tile_present(src, b, idx >> 6);
      set_move(L, s_mv, tid, here ? (slot - b0) * TB : kMoveSlots * TB, here ? idx & 63 : 0);
    }
    bool ok = true;
    if (tid < 32) {  // lane s brings the source tile of slot b0 + s; only this warp waits
      const uint8_t* p = lane < cnt ? tile_ptr(src, L, b, h, h_kv, s_src[b0 + lane]) : nullptr;
      const int live = __popc(__ballot_sync(0xffffffffu, p != nullptr));
      if (lane == 0) mbar_expect_tx(&bar, unsigned(TB) * unsigned(live));
      __syncwarp();
      if (p) bulk_load(in + lane * TB, p, TB, &bar, evict_first_policy());
      ok = mbar_wait_bounded(&bar, phase);
    }
    if (__syncthreads_or(!ok)) {
      if (tid == 0) {
        atomicOr(L.status, BGTQ_STATUS_TIMEOUT);
        mbar_wait_bounded(&bar, phase);  // the copies may still land: wait (bounded) before leaving
      }
      __syncthreads();
      return;
    }
    if (b0 == 0) assemble_tile<kGatherThreads, false>(L, ql, made, in, s_mv);
    else assemble_tile<kGatherThreads, true>(L, ql, made, in, s_mv);
    __syncthreads();
  }
  uint8_t* out = tile_ptr(dst, L, b, h, h_kv, j);
  if (out) write_tile<kGatherThreads>(out, made, TB);
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
  commit_kernel<<<unsigned(batch * h_kv), kCommitThreads, 4 * L.tile_bytes, stream>>>(
      L, quad_list(L), cache, path, path_ld, n_path, n_nodes, n_q, seq_lens, new_lens, h_kv);
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
  // CTAs per unit: enough to fill the SMs or to leave each at most 2048 tokens, 8 at most
  int cluster = 1;
  while (cluster < 8 && units * cluster < num_sms && max_seq_len > 2048LL * cluster) cluster *= 2;
  const long long per = (max_seq_len + cluster - 1) / cluster + 31;
  SelectArgs a{mass, mass_ld, max_seq_len, seq_lens, h_kv, keep, n_sink, n_recent, cluster,
               int(std::min<long long>((per + 3) / 4 * 4, 24 * 1024)), kept, mass_out, mass_out_ld, new_lens, L.status};
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
  gcfg.blockDim = dim3(kGatherThreads);
  gcfg.dynamicSmemBytes = size_t(kMoveSlots + 2) * L.tile_bytes;
  gcfg.stream = stream;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  gcfg.attrs = pdl;
  gcfg.numAttrs = 1;
  return cudaLaunchKernelEx(&gcfg, gather_kernel, L, quad_list(L), src, dst, (const int*)kept, seq_lens, max_seq_len, keep, h_kv);
}

}  // namespace bgtq
