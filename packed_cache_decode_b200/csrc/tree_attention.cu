// Attention of drafted trees over the packed cache for many query columns, on the 5th
// generation tensor cores (tcgen05, sm_100a).
//
// A KV head's query columns (drafted node x query head, up to 2048) all read the same
// cache, so its codes are decoded once per 128 columns instead of once per 8 (the decode
// kernel's column tile) and the products run as M = 128 matrix instructions. With rotated
// queries q' and decoded keys in the rotated space
//   S[col][t] = sum over packed dims q'[col][d] K[t][d],   K = (|k_g| / 2^e) c[code],
//   O[col][n] = sum_t P[col][t] V[t][n],  P = 2^(s - m) |v| / sqrt(128),  V = c[vcode],
// out = R_V^T O / l; softmax_scale, 1 / sqrt(d_g), log2(e) and the codebook scale sit in q'.
//
// Precision. The logits need about 2^-20: q' and K are both split into fp16 hi + lo parts
// and S = hi hi + lo hi + hi lo (fp32 accumulation; lo lo is 2^-22). A centroid is exact in
// fp16 (rates 3-4: hi + lo), so hi = fp16(c n) and lo = fma(c, n_hi, -hi) + c n_lo is the
// product to 2^-21. Powers of two keep both clear of fp16's range: one per query column, one
// per 32 tokens (2^e, the largest norm among them); they come back as one factor of the
// logits. The norms are folded into K because they differ per group: kept apart, every
// group would need an accumulator of its own. P is fp16 (half a step: 2^-11 of a weight) and
// V the fp16 value codebook (exact for rates 1-2), as in the decode kernel: folding |v| into
// V instead would round twice.
//
// One CTA per SM takes an equal slice of the units' tiles (64 tokens) laid end to end, units
// being (row, KV head, 128 columns); rows count by their true lengths, which a prefix sum
// made by the preparation kernel tells. 16 warps:
//  * warp 13: bulk copies of packed tiles into a ring;
//  * warps 14-15: the tile's norms: scaled hi + lo pairs for the keys, fp32 for the values;
//  * warps 4-11: decode codes into K hi, K lo and V operands in shared memory (two
//    buffers). A quad of a lane's code string is exactly one 16-byte row of a K-major core
//    matrix (8 tokens x 8 dims), so every store of a warp is 128 consecutive bytes;
//  * warp 12: issues the matrix instructions, Q' and P from tensor memory, K and V from
//    shared memory: QK of tile i + 1, then PV of tile i;
//  * warps 0-3: softmax, one thread per column: S from tensor memory, P back to it. The
//    reference maximum moves only when a tile exceeds it by 2^3 (fp16 holds P while |v| /
//    sqrt(128) stays below 8000), so O is seldom rescaled; the sums are right either way.
// Q' lives in tensor memory because an M = 128, N = 64 product reading both operands from
// shared memory would need 192 bytes per cycle of it, above the 128 there are.
// Tensor memory columns: Q' hi and lo (up to 160), S 2 x 64, P 2 x 32, O 128.
// Bound by the tensor pipe and shared memory together: per tile and 128 columns 3 x 9 + 8
// instructions of 32-64 cycles each (1100), against some 1250 cycles of shared memory.
//
// Every wait is bounded; a wait that runs out raises a flag that ends all roles, the status
// says BGTQ_STATUS_TIMEOUT and copies and matrix instructions in flight are waited for
// (bounded) before tensor memory is freed.
#include <cuda_runtime.h>

#include <algorithm>

#include "decode_split.cuh"

namespace bgtq {

namespace {

constexpr int kTreeThreads = 512;
constexpr int kCols = 128;                // query columns of a unit (rows of the matrix products)
constexpr int kDecWarp0 = 4, kDecWarps = 8;
constexpr int kMmaWarp = 12, kLoadWarp = 13, kNormWarp0 = 14;
constexpr int kMaxStages = 4;
constexpr int kMetas = 8;                 // tiles between the norm warps and the softmax: stages + 2 at most
constexpr int kMaxDims = 160;             // packed dims as quads: kMaxQuads x 8
constexpr int kTmemS = 160, kTmemP = 288, kTmemO = 352;
constexpr unsigned kTreeWaitLimit = 1u << 20;
// key norms of a tile as the decode warps use them: per group 64 entries (slot-major) of
// (hi, hi, lo, lo) fp16
constexpr int kNormBytes = kMaxGroups * kTile * 8;

struct TreeLaunch {
  CacheRef cache;
  const int* seq_lens;
  TreeArgs tree;
  const long long* prefix;     // [batch + 1] tiles of the rows before, times row_units
  const uint4* q;              // [unit][word group][column]: Q' hi then lo, 4 words a group
  const float* q_scale;        // [unit][column]
  float4* part_o;              // [slot][32][column]
  float2* part_ml;             // [slot][column]
  long long most;              // tokens a row may have in this call
  int batch, h_kv, G, n_q;     // G: query heads per KV head
  int col_tiles, row_units;    // 128-column tiles per KV head; units per row
  int q_words;                 // words per part (hi or lo) of a column: 4 per quad, quads even
  int stages;
};

__device__ __forceinline__ void mbar_arrive(unsigned long long* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(unsigned long long* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
// D[tmem] (+)= A[tmem] B[shared], fp16 operands, fp32 accumulators.
__device__ __forceinline__ void tc_mma(unsigned d, unsigned a, unsigned long long b, unsigned idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(unsigned(acc))
      : "memory");
}
// Instruction descriptor: fp32 D (1 at bit 4), fp16 A and B (0), both K-major, N / 8 at bit
// 17, M / 16 at bit 24.
__host__ __device__ constexpr unsigned tc_idesc(int M, int N) {
  return (1u << 4) | (unsigned(N >> 3) << 17) | (unsigned(M >> 4) << 24);
}
// Shared-memory operand, K-major without swizzle: 8 x 16-byte core matrices; `lead` bytes
// between neighbours along K, `stride` along the rows; descriptor version 1 (bit 46).
__device__ __forceinline__ unsigned long long tc_desc(unsigned addr, unsigned lead, unsigned stride) {
  return (unsigned long long)((addr & 0x3FFFFu) >> 4) | ((unsigned long long)(lead >> 4) << 16) |
         ((unsigned long long)(stride >> 4) << 32) | (1ull << 46);
}

#define BGTQ_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define BGTQ_W8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
// 32 consecutive tensor-memory columns of the warp's lanes (one lane's columns per thread).
__device__ __forceinline__ void tc_ld32(unsigned (&v)[32], unsigned addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : BGTQ_R8(v, 0), BGTQ_R8(v, 8), BGTQ_R8(v, 16), BGTQ_R8(v, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(unsigned addr, const unsigned (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      BGTQ_W8(v, 0), BGTQ_W8(v, 8), BGTQ_W8(v, 16), BGTQ_W8(v, 24)
      : "memory");
}
__device__ __forceinline__ void tc_st4(unsigned addr, const uint4& v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ __half2 as_h2(unsigned x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ unsigned as_u32(__half2 x) { return *reinterpret_cast<unsigned*>(&x); }
__device__ __forceinline__ void st_s32(unsigned a, unsigned v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// A CTA's slice, segment by segment (tiles of one unit); every role walks it alike.
struct TreeWalk {
  long long at, end;   // position in the sequence of all units' tiles
  int b, nt;           // row, its tiles
  int k, lt0, n;       // unit of the row, first tile, tiles of the segment
  __device__ __forceinline__ void start(const TreeLaunch& a) {
    // (fewer tiles than CTAs: the CTAs past the last tile get none, no slice is empty)
    const long long T = a.prefix[a.batch], c = blockIdx.x, C = min((long long)gridDim.x, T);
    at = c < C ? c * T / C : 0;
    end = c < C ? (c + 1) * T / C : 0;
    int lo = 0, hi = a.batch;  // the row whose range holds `at`
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.prefix[mid] <= at) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  __device__ __forceinline__ bool next(const TreeLaunch& a) {
    if (at >= end) return false;
    while (a.prefix[b + 1] <= at) ++b;
    const long long p0 = a.prefix[b];
    nt = int((a.prefix[b + 1] - p0) / a.row_units);
    k = int((at - p0) / nt);
    lt0 = int((at - p0) % nt);
    n = int(min((long long)(nt - lt0), end - at));
    at += n;
    return true;
  }
  __device__ __forceinline__ long long unit(const TreeLaunch& a) const { return (long long)b * a.row_units + k; }
  __device__ __forceinline__ int head(const TreeLaunch& a) const { return k / a.col_tiles; }
};

__device__ __forceinline__ long long tree_row_len(const TreeLaunch& a, int b) {
  const long long len = a.seq_lens[b];
  return len < 0 ? 0 : min(len, a.most);
}

struct TreeShared {
  unsigned long long full[kMaxStages], normed[kMaxStages], empty[kMaxStages];
  unsigned long long kv_full[2], qk_done[2], p_full[2], pv_done[2], q_full, tables;
  unsigned tmem;
  int abort;
  int present[kMetas];
  float scale[kMetas][2];
  int valid[kMetas];
  alignas(16) float vnorm[kMetas][kTile];   // |v| / (sqrt(128) kappa) by token (read four at a time)
};

// Waits (bounded) for the barrier's phase of the given parity; false once the CTA gives up.
__device__ __forceinline__ bool tree_wait(TreeShared& s, unsigned long long* bar, unsigned parity) {
  for (unsigned i = 0; i < kTreeWaitLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&s.abort)) return false;
  }
  *reinterpret_cast<volatile int*>(&s.abort) = 1;
  return false;
}

// K operand words of one quad (rate R) for the lane's eight tokens: hi at kh + 128 m, lo at
// kh + lo_off + 128 m. nrm: the lane's norm entries (4 x 16 bytes) of the quad's group.
template <int R>
__device__ __forceinline__ void decode_quad(unsigned tb, unsigned off, unsigned nrm, unsigned kh, unsigned lo_off,
                                            unsigned t8, unsigned t3, unsigned c8) {
  KCodes<R> c;
  c.load(tb, off, false);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 nn = ld_s128(nrm + 16 * j);  // (hi, lo) of slots 2j and 2j + 1
    uint2 e2 = make_uint2(0u, 0u);
    if constexpr (R == 2) e2 = ld_s64(t8 + row8(c.w, c8, j));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = 2 * j + i;
      const unsigned nh = i ? nn.z : nn.x, nl = i ? nn.w : nn.y;
      unsigned hi, lo;
      if constexpr (R == 1) {
        const unsigned sgn = (~c.w << (15 - m)) & 0x80008000u;  // code 0 is -1
        hi = nh ^ sgn;
        lo = nl ^ sgn;
      } else {
        unsigned ch, cl = 0;
        if constexpr (R == 2) {
          ch = i ? e2.y : e2.x;
        } else {
          uint2 e;
          if constexpr (R == 3) e = ld_s64(t3 + c.row(m, c8));
          else e = ld_s64(t8 + 128 + row8(m < 4 ? c.w.x : c.w.y, c8, m & 3));
          ch = e.x;
          cl = e.y;
        }
        const __half2 h = __hmul2(as_h2(ch), as_h2(nh));
        __half2 l = __hfma2(as_h2(ch), as_h2(nh), __hneg2(h));
        l = __hfma2(as_h2(ch), as_h2(nl), l);
        if constexpr (R >= 3) l = __hfma2(as_h2(cl), as_h2(nh), l);
        hi = as_u32(h);
        lo = as_u32(l);
      }
      st_s32(kh + 128 * m, hi);
      st_s32(kh + lo_off + 128 * m, lo);
    }
  }
}

template <int VR, bool NH>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(DevLayout L, TreeLaunch a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(16) TreeShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int TB = L.tile_bytes, NS = a.stages;
  const int nq = L.n_kquads, steps = (nq + 1) >> 1;
  constexpr int kTbl = kTbl8Bytes + kTbl3Bytes + vtab_bytes<VR>();
  const unsigned k_part = unsigned(steps) * 2048u;   // bytes of a K part (hi or lo) of a buffer
  const unsigned base = smem_addr(smem);
  const unsigned t8a = base, t3a = base + kTbl8Bytes, vta = t3a + kTbl3Bytes;
  const unsigned k_at = (base + kTbl + 127u) & ~127u;      // [2 buffers][hi, lo]
  const unsigned v_at = k_at + 4u * k_part;                // [2 buffers]
  const unsigned n_at = v_at + 2u * 16384u;                // norms [stage]
  const unsigned r_at = n_at + unsigned(NS) * kNormBytes;  // ring [stage]

  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.normed[i], 2);
      mbar_init(&s.empty[i], kDecWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.kv_full[i], kDecWarps);
      mbar_init(&s.qk_done[i], 1);
      mbar_init(&s.p_full[i], 4);
      mbar_init(&s.pv_done[i], 1);
    }
    mbar_init(&s.q_full, 4);
    mbar_init(&s.tables, 1);
    s.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&s.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // an odd last quad's partner stays zero (the products read it; its q' is zero too)
  if (nq & 1)
    for (int i = tid; i < 4 * 256; i += kTreeThreads)
      st_s32(k_at + unsigned(i >> 8) * k_part + unsigned(nq) * 1024u + 4u * (i & 255), 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = s.tmem;
  if (tid == 0) {
    mbar_expect_tx(&s.tables, unsigned(kTbl));
    bulk_load(smem, L.tables, unsigned(kTbl), &s.tables, evict_last_policy());
  }
  pdl_trigger();
  pdl_wait();  // Q' and the rows' prefix come from the preparation kernel

  TreeWalk w;
  w.start(a);
  if (warp == kLoadWarp) {
    if (lane == 0) {
      const unsigned long long pol = evict_first_policy();
      unsigned i = 0;
      bool go = true;
      while (go && w.next(a)) {
        const int h = w.head(a);
        for (int t = 0; t < w.n; ++t, ++i) {
          const unsigned st = i % NS, round = i / NS;
          if (round > 0 && !tree_wait(s, &s.empty[st], (round - 1) & 1u)) {
            go = false;
            break;
          }
          const uint8_t* src = tile_ptr(a.cache, L, w.b, h, a.h_kv, w.lt0 + t);
          s.present[i % kMetas] = src != nullptr;
          mbar_expect_tx(&s.full[st], src ? unsigned(TB) : 0u);
          if (src) bulk_load(smem + (r_at - base) + st * TB, src, unsigned(TB), &s.full[st], pol);
        }
      }
      // copies in flight land before the CTA ends: the last one of each stage
      for (unsigned st = 0; st < unsigned(NS) && st < i; ++st) {
        const unsigned rounds = (i - 1 - st) / NS;
        mbar_wait_bounded(&s.full[st], rounds & 1u);
      }
    }
  } else if (warp >= kNormWarp0) {
    // token 32 half + lane of every tile: key norms scaled by 2^-e (e: the exponent of the
    // largest of the 32 tokens' norms) as fp16 hi + lo, value norms over sqrt(128) kappa
    // for the softmax
    const int half = warp - kNormWarp0, tok = 32 * half + lane, entry = (tok & 7) * 8 + (tok >> 3);
    const int ng = L.n_kgroups;
    const float vscale = rsqrtf(float(kD)) / L.kappa_v;
    unsigned i = 0;
    bool go = true;
    while (go && w.next(a)) {
      const long long len = tree_row_len(a, w.b);
      for (int t = 0; t < w.n; ++t, ++i) {
        const unsigned st = i % NS, round = i / NS;
        if (!__all_sync(0xffffffffu, tree_wait(s, &s.full[st], round & 1u))) {
          go = false;
          break;
        }
        const int present = *reinterpret_cast<volatile int*>(&s.present[i % kMetas]);
        const int valid = present ? int(min(64LL, len - (long long)(w.lt0 + t) * kTile)) : 0;
        const unsigned tb = launder(r_at + st * TB), dst = n_at + st * kNormBytes;
        auto norm = [&](int row) {
          float x = 0.f;
          if (tok < valid) {
            if constexpr (NH) x = __half2float(__ushort_as_half((unsigned short)ld_s16(tb + L.knorm_off + 2 * (row * kTile + entry))));
            else x = __uint_as_float(ld_s32(tb + L.knorm_off + 4 * (row * kTile + entry)));
          }
          return x;
        };
        float n[kMaxGroups], top = 0.f;
#pragma unroll
        for (int g = 0; g < kMaxGroups; ++g) {
          n[g] = g < ng ? norm(g) : 0.f;
          top = fmaxf(top, fabsf(n[g]));
        }
        const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        const int ex = bits == 0u ? 127 : min(227, max(27, int(bits >> 23)));
        const float down = __int_as_float((254 - ex) << 23);
#pragma unroll
        for (int g = 0; g < kMaxGroups; ++g) {
          if (g >= ng) break;
          const float x = n[g] * down;
          const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
          const unsigned hb = __half_as_ushort(hi), lb = __half_as_ushort(lo);
          const unsigned at = dst + (g * kTile + entry) * 8;
          st_s32(at, hb | hb << 16);
          st_s32(at + 4, lb | lb << 16);
        }
        s.vnorm[i % kMetas][tok] = norm(ng) * vscale;
        if (lane == 0) {
          s.scale[i % kMetas][half] = __int_as_float(ex << 23);
          if (half == 0) s.valid[i % kMetas] = valid;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.normed[st]);
      }
    }
  } else if (warp >= kDecWarp0 && warp < kDecWarp0 + kDecWarps) {
    const unsigned c8 = unsigned(lane & 15) << 3, lane4 = unsigned(lane) << 2;
    const int g = lane >> 2, t4 = lane & 3;
    bool go = __all_sync(0xffffffffu, tree_wait(s, &s.tables, 0u));
    const unsigned t8 = launder(t8a), t3 = launder(t3a), vt = launder(vta);
    unsigned i = 0;
    while (go && w.next(a)) {
      for (int t = 0; t < w.n; ++t, ++i) {
        const unsigned st = i % NS, round = i / NS, buf = i & 1u, use = i >> 1;
        bool ok = tree_wait(s, &s.full[st], round & 1u) && tree_wait(s, &s.normed[st], round & 1u);
        if (use > 0) ok = ok && tree_wait(s, &s.qk_done[buf], (use - 1) & 1u) && tree_wait(s, &s.pv_done[buf], (use - 1) & 1u);
        if (!__all_sync(0xffffffffu, ok)) {
          go = false;
          break;
        }
        const unsigned tb = launder(r_at + st * TB), nb = launder(n_at + st * kNormBytes);
        const unsigned kb = k_at + buf * 2u * k_part + lane4, vb = v_at + buf * 16384u + lane4;
        for (int it = warp - kDecWarp0; it < nq + 8; it += kDecWarps) {
          if (it < nq) {
            int gi = 0;
            while (gi + 1 < L.n_kgroups && it >= L.group_quad0[gi + 1]) ++gi;
            const int r = L.group_rate[gi], P = L.quad_np[it];
            const unsigned li = t4 < P ? g * P + t4 : 0u;  // (a lane without a pair: any code, its q' is zero)
            const unsigned qo = unsigned(L.quad_off[it]);
            const unsigned nrm = nb + unsigned(gi * kTile + 8 * g) * 8u, kh = kb + unsigned(it) * 1024u;
            switch (r) {
              case 1: decode_quad<1>(tb, qo + 2u * li, nrm, kh, k_part, t8, t3, c8); break;
              case 2: decode_quad<2>(tb, qo + 4u * li, nrm, kh, k_part, t8, t3, c8); break;
              case 3: decode_quad<3>(tb, (qo + 4u * li) | ((qo + 32u * P + 2u * li) << 16), nrm, kh, k_part, t8, t3, c8); break;
              default: decode_quad<4>(tb, qo + 8u * li, nrm, kh, k_part, t8, t3, c8); break;
            }
          } else {
            const int v = it - nq, c = v >> 1, m0 = 4 * (v & 1);
            ValueLane<VR> vl;
            vl.load(tb + L.vcode_off + c * 256 * VR, lane);
            auto dims = [&](auto first) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int mt = decltype(first)::value + j;
                unsigned x[4];
                vl.regs(mt, t8, vt, c8, lane4, x);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  st_s32(vb + unsigned((2 * c + (q >> 1)) * 16 + 2 * mt + (q & 1)) * 128u, x[q]);
              }
            };
            if (m0 == 0) dims(IntC<0>{});
            else dims(IntC<4>{});
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.empty[st]);
          mbar_arrive(&s.kv_full[buf]);
        }
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      const unsigned id_s = tc_idesc(kCols, kTile), id_o = tc_idesc(kCols, kD);
      const unsigned q_lo = unsigned(a.q_words);
      auto scores = [&](unsigned i) {  // S of tile i
        const unsigned buf = i & 1u, k0 = k_at + buf * 2u * k_part, d = tmem + kTmemS + 64u * buf;
        for (int k = 0; k < steps; ++k) {
          const unsigned long long hi = tc_desc(k0 + 2048u * k, 1024u, 128u), lo = tc_desc(k0 + k_part + 2048u * k, 1024u, 128u);
          tc_mma(d, tmem + 8u * k, hi, id_s, k > 0);
          tc_mma(d, tmem + q_lo + 8u * k, hi, id_s, true);
          tc_mma(d, tmem + 8u * k, lo, id_s, true);
        }
        tc_commit(&s.qk_done[buf]);
      };
      auto values = [&](unsigned i, bool first) {  // O += P V of tile i
        const unsigned buf = i & 1u, v0 = v_at + buf * 16384u, p = tmem + kTmemP + 32u * buf;
        for (int k = 0; k < 4; ++k) tc_mma(tmem + kTmemO, p + 8u * k, tc_desc(v0 + 4096u * k, 2048u, 128u), id_o, !first || k > 0);
        tc_commit(&s.pv_done[buf]);
      };
      unsigned i = 0, seg = 0;
      bool go = true;
      while (go && w.next(a)) {
        go = tree_wait(s, &s.q_full, seg++ & 1u) && tree_wait(s, &s.kv_full[i & 1u], (i >> 1) & 1u);
        if (!go) break;
        tc_fence_after();
        scores(i);
        for (int t = 0; t < w.n; ++t, ++i) {
          if (t + 1 < w.n) {
            if (!tree_wait(s, &s.kv_full[(i + 1) & 1u], ((i + 1) >> 1) & 1u)) {
              go = false;
              break;
            }
            tc_fence_after();
            scores(i + 1);
          }
          if (!tree_wait(s, &s.p_full[i & 1u], (i >> 1) & 1u)) {
            go = false;
            break;
          }
          tc_fence_after();
          values(i, t == 0);
        }
      }
    }
  } else {
    // softmax: thread = query column `tid` (lane `tid` of tensor memory)
    const unsigned row = tmem + (unsigned(warp) << 21);  // lanes 32 warp ..
    auto load_q = [&](long long u) {
      const uint4* q = a.q + (size_t)u * (2 * a.q_words / 4) * kCols + tid;
      for (int j = 0; j < 2 * a.q_words / 4; ++j) tc_st4(row + 4u * j, __ldg(q + (size_t)j * kCols));
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_full);
    };
    unsigned i = 0;
    bool go = true, more = w.next(a);
    if (more) load_q(w.unit(a));
    while (go && more) {
      const long long u = w.unit(a), len = tree_row_len(a, w.b);
      const int nodes = a.tree.n_nodes ? a.tree.n_nodes[w.b] : a.n_q;  // (a row that does not fit has no tiles)
      const long long s0 = len - nodes;
      const int col = (w.k % a.col_tiles) * kCols + tid;
      const bool live = col < a.G * a.n_q;
      const int node = live ? col / a.G : 0;
      unsigned long long mask = live ? a.tree.mask[(size_t)w.b * a.n_q + node] : 0ull;
      if (nodes < 64) mask &= (1ull << nodes) - 1ull;
      const float qs = a.q_scale[(size_t)u * kCols + tid];
      float m = -INFINITY, l = 0.f;
      const int n = w.n, lt0 = w.lt0;
      for (int t = 0; t < n; ++t, ++i) {
        const unsigned buf = i & 1u, use = i >> 1;
        if (!__all_sync(0xffffffffu, tree_wait(s, &s.qk_done[buf], use & 1u))) {
          go = false;
          break;
        }
        tc_fence_after();
        unsigned x[2][32];
        tc_ld32(x[0], row + kTmemS + 64u * buf);
        tc_ld32(x[1], row + kTmemS + 64u * buf + 32u);
        const float f[2] = {s.scale[i % kMetas][0] * qs, s.scale[i % kMetas][1] * qs};
        const int valid = s.valid[i % kMetas];
        const long long t0 = (long long)(lt0 + t) * kTile;
        tc_wait_ld();
        if (valid < kTile || t0 + kTile > s0) {  // the same for the whole CTA
          const long long d = t0 - s0;   // tokens of the tile before the nodes are seen by all
          unsigned long long vis = d <= -64 ? ~0ull : d < 0 ? ~0ull >> (64 + d) | mask << -d : d < 64 ? mask >> d : 0ull;
          if (valid < kTile) vis &= (1ull << valid) - 1ull;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (!(vis >> e & 1ull)) x[e >> 5][e & 31] = 0xff800000u;
        }
        float top[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float t1 = __uint_as_float(x[hf][0]), t2 = __uint_as_float(x[hf][1]);
#pragma unroll
          for (int e = 2; e < 32; e += 2) {
            t1 = fmaxf(t1, __uint_as_float(x[hf][e]));
            t2 = fmaxf(t2, __uint_as_float(x[hf][e + 1]));
          }
          top[hf] = fmaxf(t1, t2) * f[hf];
        }
        const float mx = fmaxf(top[0], top[1]);
        // move the reference maximum when some column's tile exceeds it by 2^3
        if (__any_sync(0xffffffffu, mx > m + 3.f)) {
          const float mn = fmaxf(m, mx);
          const float c = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
          m = mn;
          l *= c;
          if (t > 0) {
            if (!__all_sync(0xffffffffu, tree_wait(s, &s.pv_done[(i - 1) & 1u], ((i - 1) >> 1) & 1u))) {
              go = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int o = 0; o < 4; ++o) {
              unsigned y[32];
              tc_ld32(y, row + kTmemO + 32u * o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * c);
              tc_st32(row + kTmemO + 32u * o, y);
            }
            tc_wait_st();
          }
        }
        const float mb = m == -INFINITY ? 0.f : m;  // a column that has seen nothing: weights of 0
        unsigned p[32];
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          const float ff = f[e >> 5];
          const float4 v = *reinterpret_cast<const float4*>(&s.vnorm[i % kMetas][e]);
          const unsigned* xe = &x[e >> 5][e & 31];
          const float p0 = fast_exp2(fmaf(__uint_as_float(xe[0]), ff, -mb)), p1 = fast_exp2(fmaf(__uint_as_float(xe[1]), ff, -mb));
          const float p2 = fast_exp2(fmaf(__uint_as_float(xe[2]), ff, -mb)), p3 = fast_exp2(fmaf(__uint_as_float(xe[3]), ff, -mb));
          l0 += p0 + p2;
          l1 += p1 + p3;
          p[e >> 1] = pack_h2(p0 * v.x, p1 * v.y);
          p[(e >> 1) + 1] = pack_h2(p2 * v.z, p3 * v.w);
        }
        l += l0 + l1;
        if (use > 0 && !__all_sync(0xffffffffu, tree_wait(s, &s.pv_done[buf], (use - 1) & 1u))) {
          go = false;
          break;
        }
        tc_fence_after();
        tc_st32(row + kTmemP + 32u * buf, p);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[buf]);
      }
      if (!go) break;
      // the next unit's Q' may come in (this unit's last scores are done), then this unit's
      // partial goes out
      more = w.next(a);
      if (more) load_q(w.unit(a));
      const unsigned last = i - 1;
      if (!__all_sync(0xffffffffu, tree_wait(s, &s.pv_done[last & 1u], (last >> 1) & 1u))) break;
      tc_fence_after();
      const long long slot = (long long)blockIdx.x + u;
      float4* po = a.part_o + (size_t)slot * 32 * kCols + tid;
#pragma unroll 1
      for (int o = 0; o < 4; ++o) {
        unsigned y[32];
        tc_ld32(y, row + kTmemO + 32u * o);
        tc_wait_ld();
        if (live)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            po[(size_t)(8 * o + e) * kCols] = make_float4(__uint_as_float(y[4 * e]), __uint_as_float(y[4 * e + 1]),
                                                          __uint_as_float(y[4 * e + 2]), __uint_as_float(y[4 * e + 3]));
      }
      tc_fence_before();
      if (live) a.part_ml[(size_t)slot * kCols + tid] = make_float2(m, l);
    }
  }
  __syncwarp();
  if (lane == 0 && *reinterpret_cast<volatile int*>(&s.abort)) {
    atomicOr(L.status, BGTQ_STATUS_TIMEOUT);
    // matrix instructions in flight end before tensor memory is freed
    if (warp == kMmaWarp) {
      tc_commit(&s.q_full);
      for (unsigned k = 0; k < 4096u; ++k) __nanosleep(256);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // every CTA waits for the tables it asked for before it ends (a CTA without tiles too)
  if (tid == 0) mbar_wait_bounded(&s.tables, 0u);
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  __syncthreads();
}

// Rows' tile prefix (block 0) and Q' of 32 query columns per block (row, KV head): thread
// (packed dim p, half) sums R_g[i][j] q[j] for 16 columns from the transposed rotation
// (coalesced), a power of two per column brings its largest entry near 2^13, then the fp16
// hi and lo words go out in tensor-memory order. Latency bound.
constexpr int kPrepCols = 32;
__global__ void __launch_bounds__(256) tree_prep_kernel(DevLayout L, TreeLaunch a, const void* __restrict__ q, int q_dtype,
                                                        float qscale, long long* __restrict__ prefix,
                                                        unsigned* __restrict__ qt, float* __restrict__ q_scale) {
  __shared__ __align__(16) float s_q[kPrepCols][kD], s_r[kPrepCols][kD + 1];
  __shared__ float s_up[kPrepCols];
  __shared__ short s_pc[kD], s_dim[kMaxDims];
  pdl_trigger();
  const int tid = threadIdx.x, N = a.G * a.n_q, blocks = a.col_tiles * (kCols / kPrepCols);
  if (blockIdx.x == 0 && tid < 32) {
    long long run = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int b = b0 + tid;
      long long v = 0;
      if (b < a.batch) {
        const long long len = tree_row_len(a, b);
        if (a.seq_lens[b] > a.most) atomicOr(L.status, BGTQ_STATUS_DECODE_CLAMPED);
        if (tree_nodes(a.tree, b, a.n_q, len) < 0) atomicOr(L.status, BGTQ_STATUS_BAD_TREE);
        else v = (len + kTile - 1) / kTile * a.row_units;
      }
      long long incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (tid >= o) incl += x;
      }
      if (b < a.batch) prefix[b + 1] = run + incl;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (tid == 0) prefix[0] = 0;
  }
  const int cb = blockIdx.x % blocks, bh = blockIdx.x / blocks, h = bh % a.h_kv, b = bh / a.h_kv;
  const int c0 = cb * kPrepCols;
  const long long u = (long long)b * a.row_units + (long long)h * a.col_tiles + c0 / kCols;
  const int in0 = c0 % kCols;  // first column inside the unit
  if (tid < kD) s_pc[tid] = L.packed_coord[tid];
  // packed dim of every operand dim (quads of 8; -1 where a quad has no pair)
  for (int e = tid; e < 8 * L.n_kquads; e += 256) s_dim[e] = (e & 7) < 2 * L.quad_np[e >> 3] ? short(L.quad_dim0[e >> 3] + (e & 7)) : short(-1);
  __syncthreads();
  for (int e = tid; e < kPrepCols * kD; e += 256) {
    const int c = e >> 7, p = e & (kD - 1), col = c0 + c;
    float x = 0.f;
    if (col < N && p < L.n_packed) {
      const size_t r = ((size_t)b * a.n_q + col / a.G) * (a.G * a.h_kv) + (size_t)h * a.G + col % a.G;
      x = load_q(q, q_dtype, r * kD + s_pc[p]);
    }
    s_q[c][p] = x;
  }
  __syncthreads();
  {
    const int p = tid & (kD - 1), half = tid >> 7;
    float acc[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) acc[c] = 0.f;
    float f = 0.f;
    if (p < L.n_packed) {
      int g = 0;
      while (g + 1 < L.n_kgroups && p >= L.group_off[g + 1]) ++g;
      const int d = L.group_dim[g], off = L.group_off[g];
      const float* R = L.k_rot32t[g] + (p - off);
      f = qscale * rsqrtf(float(d)) * L.inv_kappa_group[g];
#pragma unroll 4
      for (int j = 0; j < d; ++j) {
        const float r = __ldg(R + (size_t)j * d);
#pragma unroll
        for (int c = 0; c < 16; ++c) acc[c] = fmaf(r, s_q[16 * half + c][off + j], acc[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) s_r[16 * half + c][p] = acc[c] * f;
  }
  __syncthreads();
  {
    const int lane = tid & 31, warp = tid >> 5;
    for (int c = warp; c < kPrepCols; c += 8) {
      float top = 0.f;
      for (int p = lane; p < kD; p += 32) {
        const float x = fabsf(s_r[c][p]);
        if (x <= 3.0e38f) top = fmaxf(top, x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) {
        const int ex = top > 0.f ? min(100, max(-100, 13 - (int(__float_as_uint(top) >> 23) - 127))) : 0;
        s_up[c] = __int_as_float((127 + ex) << 23);
        q_scale[(size_t)u * kCols + in0 + c] = __int_as_float((127 - ex) << 23);
      }
    }
  }
  __syncthreads();
  // word w of a column's part = operand dims 2w, 2w + 1; groups of 4 words, columns innermost
  const int qw = a.q_words;
  for (int e = tid; e < kPrepCols * qw; e += 256) {
    const int k = e & 3, c = (e >> 2) % kPrepCols, w = (e >> 2) / kPrepCols * 4 + k;
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int dim = 2 * w + i < 8 * L.n_kquads ? s_dim[2 * w + i] : -1;
      v[i] = dim >= 0 ? s_r[c][dim] * s_up[c] : 0.f;
    }
    const float h0 = __half2float(__float2half_rn(v[0])), h1 = __half2float(__float2half_rn(v[1]));
    const size_t at = ((size_t)u * (2 * qw / 4) + w / 4) * kCols * 4 + (in0 + c) * 4 + k;
    qt[at] = pack_h2(h0, h1);
    qt[at + (size_t)(qw / 4) * kCols * 4] = pack_h2(v[0] - h0, v[1] - h1);
  }
}

// Merge of a unit's partials for 32 query columns per block, then out = R_V^T o' / l:
// thread (output dim, half) sums 16 columns, the rotation read from L2 once per block.
__global__ void __launch_bounds__(256) tree_combine_kernel(DevLayout L, TreeLaunch a, int n_ctas, void* __restrict__ out,
                                                           int out_dtype) {
  __shared__ __align__(16) float s_o[kPrepCols][kD];
  const int tid = threadIdx.x, N = a.G * a.n_q, blocks = a.col_tiles * (kCols / kPrepCols);
  pdl_trigger();
  pdl_wait();
  const int cb = blockIdx.x % blocks, bh = blockIdx.x / blocks, h = bh % a.h_kv, b = bh / a.h_kv;
  const int c0 = cb * kPrepCols, in0 = c0 % kCols;
  const long long k = (long long)h * a.col_tiles + c0 / kCols, u = (long long)b * a.row_units + k;
  const int n_nodes = a.tree.n_nodes ? a.tree.n_nodes[b] : a.n_q;
  const long long T = a.prefix[a.batch], C = min((long long)n_ctas, T), p0 = a.prefix[b], nt = (a.prefix[b + 1] - p0) / a.row_units;
  const int c = tid & 31, wp = tid >> 5;  // merge: column c, float4s wp, wp + 8, ..
  // (a row without tiles has no partials: zeros)
  int first = 0, last = -1;
  if (nt > 0) {
    first = cta_of_tile(p0 + k * nt, T, C);
    last = cta_of_tile(p0 + (k + 1) * nt - 1, T, C);
  }
  float top = -INFINITY;
  const bool live = c0 + c < N;
  if (live)
    for (int ct = first; ct <= last; ++ct) top = fmaxf(top, a.part_ml[(size_t)(ct + u) * kCols + in0 + c].x);
  float l = 0.f;
  float4 o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live && top != -INFINITY)
    for (int ct = first; ct <= last; ++ct) {
      const float2 ml = a.part_ml[(size_t)(ct + u) * kCols + in0 + c];
      if (ml.x == -INFINITY) continue;
      const float f = exp2f(ml.x - top);
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 x = __ldcs(a.part_o + ((size_t)(ct + u) * 32 + wp + 8 * j) * kCols + in0 + c);
        o[j] = make_float4(fmaf(f, x.x, o[j].x), fmaf(f, x.y, o[j].y), fmaf(f, x.z, o[j].z), fmaf(f, x.w, o[j].w));
      }
    }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // accumulator column n = 8 blk + g holds value dim 16 g + blk
    const float x[4] = {o[j].x, o[j].y, o[j].z, o[j].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = 4 * (wp + 8 * j) + e;
      s_o[c][16 * (n & 7) + (n >> 3)] = x[e] * inv;
    }
  }
  __syncthreads();
  const int d = tid & (kD - 1), half = tid >> 7;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 2
  for (int i = 0; i < kD; i += 4) {
    float r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = __ldg(L.v_rot32 + (size_t)(i + e) * kD + d);
#pragma unroll
    for (int cc = 0; cc < 16; ++cc) {
      const float4 x = *reinterpret_cast<const float4*>(&s_o[16 * half + cc][i]);
      acc[cc] = fmaf(r[0], x.x, fmaf(r[1], x.y, fmaf(r[2], x.z, fmaf(r[3], x.w, acc[cc]))));
    }
  }
#pragma unroll
  for (int cc = 0; cc < 16; ++cc) {
    const int col = c0 + 16 * half + cc, node = col / a.G;
    // rows past a row's drafted nodes are not written (a row that does not fit: zeros)
    if (col >= N || (n_nodes >= 0 && node >= n_nodes)) continue;
    store_out(out, out_dtype, (((size_t)b * a.n_q + node) * (a.G * a.h_kv) + (size_t)h * a.G + col % a.G) * kD + d, acc[cc]);
  }
}

int tree_q_words(const DevLayout& L) { return (L.n_kquads + 1) / 2 * 8; }

int tree_smem_bytes(const DevLayout& L, int stages) {
  const int vt = L.v_rate == 3 ? vtab_bytes<3>() : L.v_rate == 4 ? vtab_bytes<4>() : 0;
  return kTbl8Bytes + kTbl3Bytes + vt + 128 + 4 * ((L.n_kquads + 1) / 2) * 2048 + 2 * 16384 +
         stages * (kNormBytes + L.tile_bytes);
}

template <int VR, bool NH>
cudaError_t launch_tree_kernel(const DevLayout& L, const TreeLaunch& a, unsigned grid, int smem, cudaStream_t stream) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    int optin = 0;
    cudaFuncAttributes fa{};
    e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, tree_kernel<VR, NH>);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(tree_kernel<VR, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - int(fa.sharedSizeBytes));
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_kernel<VR, NH>, L, a);
}

}  // namespace

TreePlan plan_tree(int batch, int h_q, int h_kv, int n_q, long long max_seq_len, int num_sms) {
  TreePlan p{};
  const long long N = (long long)(h_q / h_kv) * n_q;
  p.col_tiles = int((N + kCols - 1) / kCols);
  p.units = (long long)batch * h_kv * p.col_tiles;
  const long long tiles = std::max<long long>(1, (max_seq_len + kTile - 1) / kTile);
  p.n_ctas = int(std::min<long long>(num_sms, p.units * tiles));
  const size_t slots = size_t(p.units) + p.n_ctas;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  p.prefix_at = take(size_t(batch + 1) * sizeof(long long));
  p.q_at = take(size_t(p.units) * kMaxDims * kCols * sizeof(unsigned));
  p.scale_at = take(size_t(p.units) * kCols * sizeof(float));
  p.ml_at = take(slots * kCols * sizeof(float2));
  p.o_at = take(slots * kCols * kD * sizeof(float));
  p.workspace_bytes = at;
  return p;
}

cudaError_t launch_tree(const DevLayout& L, const TreePlan& plan, const void* q, int q_dtype, int batch, int h_q,
                        int h_kv, int n_q, const TreeArgs& tree, const CacheRef& cache, const int* seq_lens,
                        long long max_seq_len, float softmax_scale, void* out, int out_dtype, void* workspace,
                        cudaStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  TreeLaunch a{};
  a.cache = cache;
  a.seq_lens = seq_lens;
  a.tree = tree;
  a.prefix = reinterpret_cast<const long long*>(ws + plan.prefix_at);
  a.q = reinterpret_cast<const uint4*>(ws + plan.q_at);
  a.q_scale = reinterpret_cast<const float*>(ws + plan.scale_at);
  a.part_ml = reinterpret_cast<float2*>(ws + plan.ml_at);
  a.part_o = reinterpret_cast<float4*>(ws + plan.o_at);
  a.most = max_seq_len;
  a.batch = batch;
  a.h_kv = h_kv;
  a.G = h_q / h_kv;
  a.n_q = n_q;
  a.col_tiles = plan.col_tiles;
  a.row_units = h_kv * plan.col_tiles;
  a.q_words = tree_q_words(L);
  const int limit = split_smem_limit();
  a.stages = kMaxStages;
  while (a.stages > 2 && tree_smem_bytes(L, a.stages) > limit) --a.stages;
  const int smem = tree_smem_bytes(L, a.stages);
  if (smem > limit) return cudaErrorInvalidValue;
  const unsigned blocks = unsigned((long long)batch * h_kv * plan.col_tiles * (kCols / kPrepCols));
  tree_prep_kernel<<<blocks, 256, 0, stream>>>(L, a, q, q_dtype, softmax_scale * kLog2e,
                                               reinterpret_cast<long long*>(ws + plan.prefix_at),
                                               reinterpret_cast<unsigned*>(ws + plan.q_at),
                                               reinterpret_cast<float*>(ws + plan.scale_at));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(plan.n_ctas);
  auto go = [&](auto vr) {
    constexpr int VR = decltype(vr)::value;
    return L.norm_fp16 ? launch_tree_kernel<VR, true>(L, a, grid, smem, stream)
                       : launch_tree_kernel<VR, false>(L, a, grid, smem, stream);
  };
  switch (L.v_rate) {
    case 1: e = go(IntC<1>{}); break;
    case 2: e = go(IntC<2>{}); break;
    case 3: e = go(IntC<3>{}); break;
    default: e = go(IntC<4>{}); break;
  }
  if (e != cudaSuccess) return e;
  return launch_dependent(tree_combine_kernel, blocks, 256, stream, L, a, plan.n_ctas, out, out_dtype);
}

}  // namespace bgtq
