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
// per 32 tokens, which puts the largest norm among them at 2^11 (a token keeps 2^-20 of its
// logits down to 2^-15 of that norm); they come back as one factor of the logits. In tiles with
// drafted nodes every token has its own, so that a node's norm takes no bits from the logits of
// queries that do not see it. The norms are folded into K because they differ per group: kept
// apart, every group would need an accumulator of its own. P is fp16 (V as fp16 has one product
// per tile; a hi + lo P would need two) and V the fp16 value codebook (exact for rates 1-2, to
// 1.8e-5 and 9.3e-5 for rates 3 and 4), as in the decode kernel: folding |v| into V instead would
// round twice. The columns' reference follows the largest entry of P itself (the weight with its value norm)
// and puts it at 2^4.9 to 2^15.9, so an entry keeps its half step of 2^-11 down to 2^-18 of the
// largest and is lost (while l, in fp32, counts it) below 2^-29: a token that takes nearly all
// of the weight leaves the tail its bits, whatever its value norm.
//
// One CTA per SM takes an equal slice of the units' tiles (64 tokens) laid end to end, units
// being (row, KV head, 128 columns); rows count by their true lengths, which a prefix sum
// made by the preparation kernel tells. 20 warps:
//  * warp 17: bulk copies of packed tiles into a ring;
//  * warps 18-19: the tile's norms: scaled hi + lo pairs for the keys, fp32 for the values;
//  * warps 8-15: decode codes into K hi, K lo and V operands in shared memory, two groups
//    that take tiles in turn (one buffer each). A quad of a lane's code string is exactly one
//    16-byte row of a K-major core matrix (8 tokens x 8 dims), so every store of a warp is 128
//    consecutive bytes;
//  * warp 16: issues the matrix instructions, Q' and P from tensor memory, K and V from
//    shared memory: PV of tile i and QK of tile i + 2, whichever has its operands first;
//  * warps 0-7: softmax, one thread per column, two groups that take tiles in turn: S from
//    tensor memory, P back over it. A column's reference moves only when a tile has an entry of
//    P 2^8 above the largest when it was set, so O is seldom rescaled.
// Q' lives in tensor memory because an M = 128, N = 64 product reading both operands from
// shared memory would need 192 bytes per cycle of it, above the 128 there are.
// Tensor memory columns: Q' hi and lo (up to 160), S 3 x 64 (each P over its own S), O 128.
// Bound: the tensor pipe needs 1100 cycles a tile and 128 columns (3 x 9 + 8 instructions of
// 32-64 cycles), shared memory some 1250; a tile takes 2250. 64 nodes of 8 query heads per KV
// head at 4 x 32K run in 602 us (the call in a CUDA graph over one cache; 681 in a loop of
// calls over three caches in turn), where the products alone (three for the logits) would
// take 341 at full rate. Half of the issue slots are used; what is left is the round trip of a
// tile through the roles (scores, softmax, PV, decode into the freed buffer), each hand-over
// 250-400 cycles under this load. Measured on that case (587 us then) and not kept: score and value
// instructions from two warps 599 us, value codes in registers with keys decoded first 589,
// in either order 620, a third decode group of its own for values 666.
//
// Every wait is bounded; a wait that runs out raises a flag that ends all roles, the status
// says BGTQ_STATUS_TIMEOUT and copies and matrix instructions in flight are waited for
// (bounded) before tensor memory is freed.
#include <cuda_runtime.h>

#include <algorithm>

#include "decode_split.cuh"

namespace bgtq {

namespace {

constexpr int kTreeThreads = 640;
constexpr int kCols = 128;                // query columns of a unit (rows of the matrix products)
constexpr int kSoftWarps = 8, kDecWarp0 = 8, kDecGroup = 4;  // decode: two groups of kDecGroup warps
constexpr int kMmaWarp = kDecWarp0 + 2 * kDecGroup, kLoadWarp = kMmaWarp + 1, kNormWarp0 = kMmaWarp + 2;
static_assert(32 * (kNormWarp0 + 2) == kTreeThreads && kDecGroup == 4, "warps; a decode warp per value chunk");
constexpr int kMaxStages = 4;
constexpr int kMetas = 8;                 // tiles between the norm warps and the softmax: stages + 2 at most
constexpr int kMaxDims = 160;             // packed dims as quads: kMaxQuads x 8
constexpr int kSBufs = 3;                 // score tiles in tensor memory (P takes the place of its own)
constexpr int kTmemS = 160, kTmemO = kTmemS + 64 * kSBufs;
static_assert(kTmemO + kD <= 512, "tensor memory columns");
// P's largest entry: exponent when the reference is set, and at most (fp16 ends at 2^16); the
// reference is set by a bound at most 2^kEvenExp above it
constexpr float kSetExp = 7.875f, kMoveExp = 15.875f;
constexpr int kEvenExp = 3;
constexpr int kNormExp = 11;   // exponent of the largest scaled key norm (times a centroid, below 3, fp16 holds it)
constexpr unsigned kTreeWaitRounds = 1u << 12, kTreeSuspend = 10000u;  // rounds of 256 tries, nanoseconds of a try
// key norms of a tile as the decode warps use them: per group and slot pair (tokens g + 16 p
// and g + 16 p + 8) the rows' (hi, hi, lo, lo) fp16 of both slots, 128 consecutive bytes
constexpr int kNormBytes = kMaxGroups * kTile * 8;
// what a decode lane needs of a key quad: code offset in the tile, norm offset
constexpr int kUnitBytes = kMaxQuads * 32 * 8;

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
  unsigned quad[kMaxQuads];    // key quads: byte offset | pairs << 16 | group << 20 | rate << 24
  unsigned char range[kDecGroup][5][2];  // key quads of each decode warp, by rate
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
__device__ __forceinline__ void tc_ld16(unsigned (&v)[16], unsigned addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : BGTQ_R8(v, 0), BGTQ_R8(v, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tc_st16(unsigned addr, const unsigned (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      BGTQ_W8(v, 0), BGTQ_W8(v, 8)
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
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.prefix[mid] <= at) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  __device__ __forceinline__ bool next(const TreeLaunch& a) {
    if (at >= end) return false;
#pragma unroll 1
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

// p_full has a barrier per score buffer: a warp may be a tile of its group ahead of the others
// (its next scores need PV of the tile between only), and its arrival for that tile must not
// count for the one before.
struct TreeShared {
  unsigned long long full[kMaxStages], normed[kMaxStages], empty[kMaxStages];
  unsigned long long k_full[2], v_full[2], k_free[2], s_full[kSBufs], p_full[kSBufs], pv_done[2], q_full, o_done, o_free, tables;
  unsigned tmem;
  int abort;
  int range[kDecGroup][5][2];   // key quads of each decode warp, by rate
  int present[kMetas];
  // for each half of a tile: what its key norms were divided by (1 where tokens have scales of their
  // own), the logarithm of its largest value norm (infinity where they span more than 2^kEvenExp)
  alignas(16) float half[kMetas][4];
  int valid[kMetas];
  unsigned long long max_done[2][4], sum_done[2][4];  // sums: by unit parity (the second group may be a unit ahead)
  float mref[kCols];            // the columns' reference maximum
  float total[2][kCols];        // the second group's sums at a unit's end (by unit parity)
  alignas(16) float vnorm[kMetas][kTile];   // |v| / (sqrt(128) kappa) by token (read four at a time)
  alignas(16) __half vlog[kMetas][kTile];   // its base-2 logarithm, -64 at least (to 2^-5: a bound's accuracy)
  alignas(4) unsigned char kexp[kMetas][kTile];  // the tokens' key scales as exponent fields (tiles with drafted nodes)
};
static_assert(sizeof(TreeShared) + 64 <= kStaticReserve, "static shared memory");

// A position in the ring of stages: stage and parity of its current round.
struct RingPos {
  unsigned st = 0, round = 0;
  __device__ __forceinline__ void step(unsigned n) {
    if (++st == n) {
      st = 0;
      ++round;
    }
  }
};

// Whether the phase of the given parity is over, without the suspension that a try may bring.
__device__ __forceinline__ bool mbar_test(unsigned long long* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0u;
}

// Waits (bounded) for the barrier's phase of the given parity; false once the CTA gives up.
// The polling loop is kept short: the waiting warps share issue slots with the working ones.
__device__ __forceinline__ bool tree_wait(TreeShared& s, unsigned long long* bar, unsigned parity) {
  if (mbar_test(bar, parity)) return true;
  const unsigned addr = smem_addr(bar);
#pragma unroll 1
  for (unsigned i = 0; i < kTreeWaitRounds; ++i) {
    unsigned left;
    asm volatile(
        "{\n .reg .pred p, q;\n"
        " mov.u32 %0, 256;\n"
        "AGAIN:\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " @p bra DONE;\n"
        " sub.u32 %0, %0, 1;\n"
        " setp.ne.u32 q, %0, 0;\n"
        " @q bra AGAIN;\n"
        "DONE:\n}\n"
        : "=&r"(left)
        : "r"(addr), "r"(parity), "r"(kTreeSuspend)
        : "memory");
    if (left) return true;
    if (*reinterpret_cast<volatile int*>(&s.abort)) return false;
  }
  *reinterpret_cast<volatile int*>(&s.abort) = 1;
  return false;
}
// The same for a role that runs ahead of the others: it sleeps between its tries.
__device__ __forceinline__ bool tree_wait_patient(TreeShared& s, unsigned long long* bar, unsigned parity) {
#pragma unroll 1
  for (unsigned i = 0; i < kTreeWaitRounds * 64u; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&s.abort)) return false;
    __nanosleep(100);
  }
  *reinterpret_cast<volatile int*>(&s.abort) = 1;
  return false;
}

// K operand words of one quad (rate R) from the lane's codes c, for its eight tokens: hi at
// kh + 128 m, lo at kl + 128 m. nn: the lane's norms of the quad's group, (hi, lo) of slots 2j
// and 2j + 1. All loads first, then the arithmetic; `next` runs in between (it fetches the next
// quad's codes).
template <int R, typename Next>
__device__ __forceinline__ void decode_quad(const KCodes<R>& c, const uint4 (&nn)[4], unsigned kh, unsigned kl, unsigned t8,
                                            unsigned t3, unsigned c8, Next&& next) {
  unsigned ch[8], cl[8];
  if constexpr (R == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint2 e = ld_s64(t8 + row8(c.w, c8, j));
      ch[2 * j] = e.x;
      ch[2 * j + 1] = e.y;
    }
  } else if constexpr (R >= 3) {
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      uint2 e;
      if constexpr (R == 3) e = ld_s64(t3 + c.row(m, c8));
      else e = ld_s64(t8 + 128 + row8(m < 4 ? c.w.x : c.w.y, c8, m & 3));
      ch[m] = e.x;
      cl[m] = e.y;
    }
  }
  unsigned sgn0 = 0;
  if constexpr (R == 1) sgn0 = ~c.w;
  next();
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const unsigned nh = m & 1 ? nn[m >> 1].z : nn[m >> 1].x, nl = m & 1 ? nn[m >> 1].w : nn[m >> 1].y;
    unsigned hi, lo;
    if constexpr (R == 1) {
      const unsigned sgn = (sgn0 << (15 - m)) & 0x80008000u;  // code 0 is -1
      hi = nh ^ sgn;
      lo = nl ^ sgn;
    } else {
      const __half2 h = __hmul2(as_h2(ch[m]), as_h2(nh));
      __half2 l = __hfma2(as_h2(ch[m]), as_h2(nh), __hneg2(h));
      l = __hfma2(as_h2(ch[m]), as_h2(nl), l);
      if constexpr (R >= 3) l = __hfma2(as_h2(cl[m]), as_h2(nh), l);
      hi = as_u32(h);
      lo = as_u32(l);
    }
    st_s32(kh + 128 * m, hi);
    st_s32(kl + 128 * m, lo);
  }
}

// Packed pairs of fp32 (one instruction for two lanes of arithmetic).
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ bool elect_one() {
  unsigned r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

template <int VR, bool NH>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(DevLayout L, TreeLaunch a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(16) TreeShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int TB = L.tile_bytes, NS = a.stages, SH = NS >> 1;  // (2 or 4 stages: the shift is 1 or 2)
  const int nq = L.n_kquads, steps = (nq + 1) >> 1;
  constexpr int kTbl = kTbl8Bytes + kTbl3Bytes + vtab_bytes<VR>();
  const unsigned k_part = unsigned(steps) * 2048u;   // bytes of a K part (hi or lo) of a buffer
  const unsigned base = smem_addr(smem);
  const unsigned t8a = base, t3a = base + kTbl8Bytes, vta = t3a + kTbl3Bytes;
  const unsigned k_at = (base + kTbl + 127u) & ~127u;      // [2 buffers][hi, lo]
  const unsigned v_at = k_at + 4u * k_part;                // [2 buffers]
  const unsigned n_at = v_at + 2u * 16384u;                // norms [stage]
  const unsigned u_at = n_at + unsigned(NS) * kNormBytes;  // key quads [quad][lane]
  const unsigned r_at = u_at + kUnitBytes;                 // ring [stage]

  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.normed[i], 2);
      mbar_init(&s.empty[i], kDecGroup);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.k_full[i], kDecGroup);
      mbar_init(&s.v_full[i], kDecGroup);
      mbar_init(&s.k_free[i], 1);
      mbar_init(&s.pv_done[i], 1);
    }
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s.max_done[0][i], 1);
      mbar_init(&s.max_done[1][i], 1);
      mbar_init(&s.sum_done[0][i], 1);
      mbar_init(&s.sum_done[1][i], 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], kSoftWarps / 2);
    }
    mbar_init(&s.q_full, kSoftWarps);
    mbar_init(&s.o_done, 1);
    mbar_init(&s.o_free, kSoftWarps);
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
#pragma unroll 1
    for (int i = tid; i < 4 * 256; i += kTreeThreads)
      st_s32(k_at + unsigned(i >> 8) * k_part + unsigned(nq) * 1024u + 4u * (i & 255), 0u);
#pragma unroll 1
  for (int it = warp; it < nq; it += kTreeThreads / 32) {
    const unsigned qi = a.quad[it], qo = qi & 0xffffu;
    const int r = qi >> 24, P = qi >> 16 & 15u, gi = qi >> 20 & 15u, g = lane >> 2, t4 = lane & 3;
    const unsigned li = t4 < P ? g * P + t4 : 0u;  // (a lane without a pair: any code, its q' is zero)
    const unsigned off = r == 3 ? (qo + 4u * li) | ((qo + 32u * P + 2u * li) << 16) : qo + 2u * r * li;
    st_s32(u_at + 8u * (it * 32 + lane), off);
    st_s32(u_at + 8u * (it * 32 + lane) + 4u, unsigned(gi * kTile * 8 + 16 * g));
  }
  if (tid < kDecGroup * 10) s.range[tid / 10][tid % 10 / 2][tid % 2] = a.range[tid / 10][tid % 10 / 2][tid % 2];
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
#pragma unroll 1
      while (go && w.next(a)) {
        const int h = w.head(a);
#pragma unroll 1
        for (int t = 0; t < w.n; ++t, ++i) {
          const unsigned st = i & (NS - 1u), round = i >> SH;
          if (round > 0 && !tree_wait_patient(s, &s.empty[st], (round - 1) & 1u)) {
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
#pragma unroll 1
      for (unsigned st = 0; st < unsigned(NS) && st < i; ++st) {
        const unsigned rounds = (i - 1 - st) >> SH;
        mbar_wait_bounded(&s.full[st], rounds & 1u);
      }
    }
  } else if (warp >= kNormWarp0) {
    // token 32 half + lane of every tile: key norms scaled by 2^(kNormExp - e) (e: the exponent of
    // the largest of the 32 tokens' norms, or of the token's own where queries may not see it) as
    // fp16 hi + lo, value norms over sqrt(128) kappa for the softmax
    const int half = warp - kNormWarp0, tok = 32 * half + lane, entry = (tok & 7) * 8 + (tok >> 3);
    const int ng = L.n_kgroups;
    const float vscale = rsqrtf(float(kD)) / L.kappa_v;
    unsigned i = 0;
    bool go = true;
#pragma unroll 1
    while (go && w.next(a)) {
      const long long len = tree_row_len(a, w.b);
      const int full = (int(len) - (a.tree.n_nodes ? a.tree.n_nodes[w.b] : a.n_q)) / kTile;  // tiles without nodes
#pragma unroll 1
      for (int t = 0; t < w.n; ++t, ++i) {
        const unsigned st = i & (NS - 1u);
        if (!__all_sync(0xffffffffu, tree_wait_patient(s, &s.full[st], i >> SH & 1u))) {
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
        float kn[kMaxGroups];  // (all loads in flight together)
#pragma unroll
        for (int g = 0; g < kMaxGroups; ++g) kn[g] = g < ng ? norm(g) : 0.f;
        const float vn = norm(ng) * vscale;
        float top = 0.f;
#pragma unroll
        for (int g = 0; g < kMaxGroups; ++g)
          if (fabsf(kn[g]) < INFINITY) top = fmaxf(top, fabsf(kn[g]));  // (an infinite or NaN norm spoils its own token alone)
        const bool masked = valid < kTile || w.lt0 + t >= full;  // (as the softmax has it)
        const unsigned all = __reduce_max_sync(0xffffffffu, __float_as_uint(top)), bits = masked ? __float_as_uint(top) : all;
        const int ex = (bits == 0u ? 127 : min(187, max(67, int(bits >> 23)))) - kNormExp;
        const float down = __int_as_float((254 - ex) << 23);
        s.kexp[i % kMetas][tok] = (unsigned char)ex;
#pragma unroll
        for (int g = 0; g < kMaxGroups; ++g) {
          if (g >= ng) break;
          const float x = kn[g] * down;
          const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
          const unsigned hb = __half_as_ushort(hi), lb = __half_as_ushort(lo);
          const unsigned at = dst + unsigned(g * kTile) * 8u + unsigned((tok >> 4) * 128 + (tok & 7) * 16 + (tok >> 3 & 1) * 8);
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(hb | hb << 16), "r"(lb | lb << 16) : "memory");
        }
        s.vnorm[i % kMetas][tok] = vn;
        // (at least -64: a token of no value still bounds its weight, 2^79 at most in the sum; an
        // infinite or NaN norm leaves the reference finite)
        auto log_of = [](float x) { return fminf(127.f, fmaxf(-64.f, __log2f(x))); };
        s.vlog[i % kMetas][tok] = __float2half_rn(log_of(fabsf(vn)));
        const unsigned va = __float_as_uint(fabsf(vn));  // (as ordered as the norms; NaN above infinity)
        const unsigned vmax = __reduce_max_sync(0xffffffffu, va), vmin = __reduce_min_sync(0xffffffffu, tok < valid ? va : vmax);
        const float top_v = __uint_as_float(vmax);
        const bool even = top_v <= __uint_as_float(vmin) * float(1 << kEvenExp) && top_v < INFINITY;
        if (lane == 0) {
          s.half[i % kMetas][2 * half] = masked ? 1.f : __int_as_float(ex << 23);
          s.half[i % kMetas][2 * half + 1] = even ? log_of(top_v) : INFINITY;
          if (half == 0) s.valid[i % kMetas] = valid;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.normed[st]);
      }
    }
  } else if (warp >= kDecWarp0 && warp < kMmaWarp) {
    const unsigned c8 = unsigned(lane & 15) << 3, lane4 = unsigned(lane) << 2;
    // two groups take the tiles in turn (group = the operand buffer they fill)
    const unsigned dw = (warp - kDecWarp0) % kDecGroup, buf = (warp - kDecWarp0) / kDecGroup;
    // (a timeout of the tables raises the flag that the waits below see)
    tree_wait(s, &s.tables, 0u);
    bool go = true;
    const unsigned t8 = launder(t8a), t3 = launder(t3a), vt = launder(vta), units = launder(u_at) + 8u * lane;
    const unsigned kb = k_at + buf * 2u * k_part + lane4;
    const unsigned vb = v_at + buf * 16384u + lane4 + unsigned(dw) * 4096u, v_off = L.vcode_off + dw * 256 * VR;
    unsigned first = 0;  // the unit's first tile
#pragma unroll 1
    for (; go && w.next(a); first += w.n) {
      const unsigned end = first + w.n;
#pragma unroll 1
      for (unsigned i = first + ((first ^ buf) & 1u); i < end; i += 2) {
        const unsigned st = i & (NS - 1u), before = ((i >> 1) - 1u) & 1u;
        // (the norms came after the tile itself)
        go = tree_wait(s, &s.normed[st], i >> SH & 1u);
        if (i > 1) go = go && tree_wait(s, &s.k_free[buf], before);
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
        const unsigned tb = launder(r_at + st * TB), nb = launder(n_at + st * kNormBytes);
        auto quads = [&](auto rate) {
          constexpr int R = decltype(rate)::value;
          // a quad's code offset has the alignment of its own rate, and the loads are pure: the
          // launder() in here keeps them from being hoisted out of the branch on the rate
          int it = s.range[dw][R][0];
          const int last = s.range[dw][R][1];
          if (it >= last) return;
          KCodes<R> c;
          uint2 q = ld_s64(units + 256u * launder(it));
          c.load(tb, launder(q.x), false);
          uint4 nn[4];  // one rate is one group: its norms serve all its quads
#pragma unroll
          for (int j = 0; j < 4; ++j) nn[j] = ld_s128(nb + q.y + 128 * j);
#pragma unroll 1
          for (; it < last; ++it) {
            const unsigned kh = kb + unsigned(it) * 1024u;
            KCodes<R> cn;
            unsigned qn;
            decode_quad<R>(c, nn, kh, kh + k_part, t8, t3, c8, [&] {
              qn = ld_s32(units + 256u * launder(min(it + 1, last - 1)));
              cn.load(tb, launder(qn), false);
            });
            c = cn;
          }
        };
        quads(IntC<4>{});
        quads(IntC<3>{});
        quads(IntC<2>{});
        quads(IntC<1>{});
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.k_full[buf]);
        if (i > 1) {
          go = __all_sync(0xffffffffu, tree_wait(s, &s.pv_done[buf], before));
          if (!go) break;
        }
        // values: warp dw takes chunk dw of the tile
        ValueLane<VR> vl;
        vl.load(tb + v_off, lane);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          unsigned x[4];
          vl.regs(mt, t8, vt, c8, lane4, x);
#pragma unroll
          for (int k = 0; k < 4; ++k) st_s32(vb + unsigned(k >> 1) * 2048u + unsigned(2 * mt + (k & 1)) * 128u, x[k]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.empty[st]);
          mbar_arrive(&s.v_full[buf]);
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // the whole warp walks and waits, one elected lane issues
    const unsigned id_s = tc_idesc(kCols, kTile), id_o = tc_idesc(kCols, kD);
    const unsigned q_lo = unsigned(a.q_words);
    RingPos ss;                      // score buffer of the next tile to score
    auto scores = [&](unsigned i) {  // S of tile i
      const unsigned buf = i & 1u, d = tmem + kTmemS + 64u * ss.st;
      unsigned long long hi = tc_desc(k_at + buf * 2u * k_part, 1024u, 128u);
      unsigned long long lo = tc_desc(k_at + buf * 2u * k_part + k_part, 1024u, 128u);
      if (elect_one()) {
#pragma unroll 2
        for (int k = 0; k < steps; ++k, hi += 128u, lo += 128u) {  // (2048 bytes per step of 16 dims)
          tc_mma(d, tmem + 8u * k, hi, id_s, k > 0);
          tc_mma(d, tmem + q_lo + 8u * k, hi, id_s, true);
          tc_mma(d, tmem + 8u * k, lo, id_s, true);
        }
        tc_commit(&s.k_free[buf]);
        tc_commit(&s.s_full[ss.st]);
      }
      ss.step(kSBufs);
      __syncwarp();
    };
    RingPos ps;                                  // score buffer that holds the next P
    auto values = [&](unsigned i, bool first, bool last) {  // O += P V of tile i
      const unsigned buf = i & 1u, p = tmem + kTmemS + 64u * ps.st;
      const unsigned long long v = tc_desc(v_at + buf * 16384u, 2048u, 128u);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k) tc_mma(tmem + kTmemO, p + 8u * k, v + 256u * k, id_o, !first || k > 0);
        tc_commit(&s.pv_done[buf]);
        if (last) tc_commit(&s.o_done);
      }
      ps.step(kSBufs);
      __syncwarp();
    };
    auto wait = [&](unsigned long long* bar, unsigned parity) {
      const bool ok = __all_sync(0xffffffffu, tree_wait(s, bar, parity));
      tc_fence_after();
      return ok;
    };
    auto ready = [&](unsigned long long* bar, unsigned parity) {
      const bool ok = __all_sync(0xffffffffu, mbar_test(bar, parity));
      tc_fence_after();
      return ok;
    };
    unsigned i = 0, seg = 0;
    bool go = true;
#pragma unroll 1
    while (go && w.next(a)) {
      // scores run two tiles ahead: QK of tile i + 2 takes the buffer of tile i - 1, whose PV was
      // issued before it
      go = wait(&s.q_full, seg++ & 1u) && wait(&s.k_full[i & 1u], (i >> 1) & 1u);
      if (!go) break;
      scores(i);
      if (w.n > 1) {
        go = wait(&s.k_full[(i + 1) & 1u], ((i + 1) >> 1) & 1u);
        if (!go) break;
        scores(i + 1);
      }
#pragma unroll 1
      for (int t = 0; t < w.n; ++t, ++i) {
        // (both softmax groups have read the last unit's O)
        if (t == 0 && seg > 1 && !wait(&s.o_free, seg & 1u)) {
          go = false;
          break;
        }
        // PV of this tile and the scores two tiles on, in the order in which they become possible
        bool score = t + 2 < w.n, value = true;
#pragma unroll 1
        for (unsigned tries = 0; score || value; ++tries) {
          if (value && ready(&s.p_full[ps.st], ps.round & 1u) && ready(&s.v_full[i & 1u], (i >> 1) & 1u)) {
            values(i, t == 0, t + 1 == w.n);
            value = false;
          }
          if (score && ready(&s.k_full[i & 1u], ((i + 2) >> 1) & 1u)) {
            scores(i + 2);
            score = false;
          }
          if ((tries & 255u) == 255u && *reinterpret_cast<volatile int*>(&s.abort)) break;
          if (tries > kTreeWaitRounds << 14) {
            *reinterpret_cast<volatile int*>(&s.abort) = 1;
            break;
          }
        }
        if (score || value) {
          go = false;
          break;
        }
      }
    }
  } else {
    // softmax: thread = query column; two groups of four warps take the tiles in turn. The
    // reference maximum of a column passes from group to group: a group raises it for its
    // tile only after the other did for the tile before (max_done, warp by warp), then both
    // work on their exponentials at once. A group's sum follows the reference it last saw.
    const unsigned grp = warp >> 2, quad = warp & 3;
    const int c = tid & (kCols - 1);
    const unsigned row = tmem + (quad << 21);  // lanes 32 quad ..
    auto wait = [&](unsigned long long* bar, unsigned parity) {
      return bool(__all_sync(0xffffffffu, tree_wait(s, bar, parity)));
    };
    auto load_q = [&](long long u) {  // this group's part of Q' (hi or lo)
      const uint4* q = a.q + (size_t)(u * (2 * a.q_words / 4) + grp * (a.q_words / 4)) * kCols + c;
      const unsigned at = row + grp * unsigned(a.q_words);
      // q_words is a multiple of 8: groups of 2 x 4 words, their loads in flight together
#pragma unroll 2
      for (int j = 0; j < a.q_words / 4; j += 2) {
        const uint4 v0 = __ldg(q + (size_t)j * kCols), v1 = __ldg(q + (size_t)(j + 1) * kCols);
        tc_st4(at + 4u * j, v0);
        tc_st4(at + 4u * j + 4u, v1);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_full);
    };
    unsigned i = 0, seg = 0;
    RingPos sp;  // score buffer of tile i
    bool go = true, more = w.next(a);
    if (more) load_q(w.unit(a));
#pragma unroll 1
    while (go && more) {
      const long long u = w.unit(a);
      const int nodes = a.tree.n_nodes ? a.tree.n_nodes[w.b] : a.n_q;  // (a row that does not fit has no tiles)
      const int col = (w.k % a.col_tiles) * kCols + c;
      const bool live = col < a.G * a.n_q;
      unsigned long long mask = live ? a.tree.mask[(size_t)w.b * a.n_q + col / a.G] : 0ull;
      if (nodes < 64) mask &= (1ull << nodes) - 1ull;
      const float qs = a.q_scale[(size_t)u * kCols + c];
      float m = -INFINITY, l = 0.f;
      const int n = w.n;
      long long before = tree_row_len(a, w.b) - nodes - (long long)w.lt0 * kTile;  // tokens before the nodes, from the tile on
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++i, sp.step(kSBufs), before -= kTile) {
        if ((i & 1u) != grp) continue;
        if (!wait(&s.s_full[sp.st], sp.round & 1u)) {
          go = false;
          break;
        }
        const unsigned sbuf = row + kTmemS + 64u * sp.st;
        tc_fence_after();
        const int valid = s.valid[i % kMetas];
        const bool masked = valid < kTile || before < kTile;  // the same for the whole CTA
        // bit e: the column sees token e of the half
        auto seen = [&](int h) {
          const int b = int(max(-64LL, min(before - 32 * h, 32LL))), v = valid - 32 * h;
          unsigned vis = b >= 32 ? ~0u : b > 0 ? ~0u >> (32 - b) | unsigned(mask << b) : b > -64 ? unsigned(mask >> -b) : 0u;
          if (v < 32) vis &= v > 0 ? (1u << v) - 1u : 0u;
          return vis;
        };
        // a tile with nodes: the tokens' own scales and the mask go into the scores where they lie
        // (a rolled loop here; as a branch of load_half it was in every tile's code twice: 732 us
        // instead of 677 for the 70B-shaped layer with 64 nodes)
        if (masked) {
          const unsigned* ke = reinterpret_cast<const unsigned*>(s.kexp[i % kMetas]);
#pragma unroll 1
          for (int o = 0; o < 4; ++o) {
            const unsigned vis = seen(o >> 1) >> (16 * (o & 1));
            unsigned y[16];
            tc_ld16(y, sbuf + 16u * o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float k = __int_as_float((ke[4 * o + (e >> 2)] >> (8 * (e & 3)) & 0xffu) << 23);
              y[e] = vis >> e & 1u ? __float_as_uint(__uint_as_float(y[e]) * k) : 0xff800000u;
            }
            tc_st16(sbuf + 16u * o, y);
          }
          tc_wait_st();
        }
        // scores of one half of the tile, 32 tokens at a time (read twice: for the maximum and
        // for the exponentials)
        unsigned x[32];
        auto load_half = [&](int h) {
          tc_ld32(x, sbuf + 32u * h);
          tc_wait_ld();
        };
        // exponent of the tile's largest entry of P, but for the reference: where the value norms of
        // both halves are within 2^kEvenExp of each other a bound at most that far above, else
        // exact, in a second look. (64 nodes at 4 x 32K, K2V2, 64 heads, in a CUDA graph: 602 us; the
        // maximum of the weights alone, which loses the tail's bits, 593; both ways in one
        // loop 605; in a loop of calls exact everywhere 714 where this takes 680. A reference
        // that may rise by 2^5 before it moves, not 2^8, costs 10. Tiles that all need the second
        // look: 7 to 12 % more.)
        float mx = -INFINITY, even = 0.f;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const float2 st = *reinterpret_cast<const float2*>(&s.half[i % kMetas][2 * h]);
          load_half(h);
          float t1 = __uint_as_float(x[0]), t2 = __uint_as_float(x[1]);
#pragma unroll
          for (int e = 2; e < 30; e += 4) {
            t1 = max3(t1, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            t2 = max3(t2, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
          }
          t1 = fmaxf(max3(t1, __uint_as_float(x[30]), __uint_as_float(x[31])), t2);
          mx = fmaxf(mx, fmaf(t1, st.x * qs, st.y));
          even = fmaxf(even, st.y);
        }
        if (!(even < INFINITY)) {  // the same for the whole CTA
          mx = -INFINITY;
#pragma unroll 1
          for (int o = 0; o < 4; ++o) {
            unsigned y[16];
            tc_ld16(y, sbuf + 16u * o);
            tc_wait_ld();
            const float f = s.half[i % kMetas][o & 2] * qs;
            const unsigned* vl = reinterpret_cast<const unsigned*>(&s.vlog[i % kMetas][16 * o]);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 v = __half22float2(as_h2(vl[e >> 1]));
              mx = max3(mx, fmaf(__uint_as_float(y[e]), f, v.x), fmaf(__uint_as_float(y[e + 1]), f, v.y));
            }
          }
        }
        if (i > 0 && !wait(&s.max_done[grp ^ 1u][quad], ((i - 1) >> 1) & 1u)) {
          go = false;
          break;
        }
        // the reference starts where the first tile's largest entry is 2^kSetExp and moves, to the
        // same place, when some column's tile has one above 2^kMoveExp
        const float mo = t > 0 ? s.mref[c] : -INFINITY;
        const bool above = mx > mo + kMoveExp;
        const bool move = __any_sync(0xffffffffu, above) || t == 0;
        const float mn = above ? mx - kSetExp : mo;
        if (move) s.mref[c] = mn;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.max_done[grp][quad]);
        if (move && t > 0) {
          if (!wait(&s.pv_done[grp ^ 1u], ((i - 1) >> 1) & 1u)) {
            go = false;
            break;
          }
          tc_fence_after();
          const float r = mn == -INFINITY ? 1.f : fast_exp2(mo - mn);
#pragma unroll 1
          for (int o = 0; o < 8; ++o) {
            unsigned y[16];
            tc_ld16(y, row + kTmemO + 16u * o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * r);
            tc_st16(row + kTmemO + 16u * o, y);
          }
        }
        if (m != mn) l *= fast_exp2(m - mn);  // (m = -inf: l is 0)
        m = mn;
        const float mb = m == -INFINITY ? 0.f : m;  // a column that has seen nothing: weights of 0
        tc_fence_after();
        const unsigned long long nm = pack2(-mb, -mb);
        unsigned long long l2 = 0ull, l3 = 0ull;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const float f = s.half[i % kMetas][2 * h] * qs;
          load_half(h);
          unsigned p[16];
          const unsigned long long ff = pack2(f, f);
          const float4* vn = reinterpret_cast<const float4*>(&s.vnorm[i % kMetas][32 * h]);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 v = vn[e >> 2];
            const float2 a0 = unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), ff, nm));
            const float2 a1 = unpack2(fma2(pack2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), ff, nm));
            const unsigned long long p0 = pack2(fast_exp2(a0.x), fast_exp2(a0.y)), p1 = pack2(fast_exp2(a1.x), fast_exp2(a1.y));
            l2 = add2(l2, p0);
            l3 = add2(l3, p1);
            const float2 w0 = unpack2(mul2(p0, pack2(v.x, v.y))), w1 = unpack2(mul2(p1, pack2(v.z, v.w)));
            p[e >> 1] = pack_h2(w0.x, w0.y);
            p[(e >> 1) + 1] = pack_h2(w1.x, w1.y);
          }
          if (masked) {
            // a weight of 0 times an infinite or NaN norm (of a node that the column does not see)
            const unsigned vis = seen(h);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              p[e] &= (vis >> (2 * e) & 1u ? 0xffffu : 0u) | (vis >> (2 * e + 1) & 1u ? 0xffff0000u : 0u);
          }
          tc_st16(sbuf + 16u * h, p);  // (over scores that are read)
        }
        const float2 ls = unpack2(add2(l2, l3));
        l += ls.x + ls.y;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[sp.st]);
      }
      if (!go) break;
      // the unit's final reference is the last tile's; its last scores are done then, so the
      // next unit's Q' may come in. Afterwards this unit's partial goes out, each group
      // writing half of O's columns.
      const unsigned last = i - 1;
      if ((last & 1u) != grp && !wait(&s.max_done[grp ^ 1u][quad], (last >> 1) & 1u)) break;
      const float mf = s.mref[c];
      tc_fence_after();
      more = w.next(a);
      if (more) load_q(w.unit(a));
      if (m != mf) l *= fast_exp2(m - mf);
      if (grp) {
        s.total[seg & 1u][c] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.sum_done[seg & 1u][quad]);
      }
      // (a barrier of its own, one phase a unit: pv_done may be two phases behind here, where a
      // parity cannot tell)
      if (!wait(&s.o_done, seg & 1u)) break;
      tc_fence_after();
      const long long slot = (long long)blockIdx.x + u;
      float4* po = a.part_o + (size_t)slot * 32 * kCols + c;
#pragma unroll 1
      for (int o = 4 * grp; o < 4 * int(grp) + 4; ++o) {
        unsigned y[16];
        tc_ld16(y, row + kTmemO + 16u * o);
        tc_wait_ld();
        if (live)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            po[(size_t)(4 * o + e) * kCols] = make_float4(__uint_as_float(y[4 * e]), __uint_as_float(y[4 * e + 1]),
                                                          __uint_as_float(y[4 * e + 2]), __uint_as_float(y[4 * e + 3]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_free);
      if (!grp) {
        if (!wait(&s.sum_done[seg & 1u][quad], (seg >> 1) & 1u)) break;
        if (live) a.part_ml[(size_t)slot * kCols + c] = make_float2(mf, l + s.total[seg & 1u][c]);
      }
      ++seg;
    }
  }
  __syncwarp();
  if (lane == 0 && *reinterpret_cast<volatile int*>(&s.abort)) {
    atomicOr(L.status, BGTQ_STATUS_TIMEOUT);
    // matrix instructions in flight end before tensor memory is freed
    if (warp == kMmaWarp)
#pragma unroll 1
      for (unsigned k = 0; k < 4096u; ++k) __nanosleep(256);
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

// Rows' tile prefix (block 0) and Q' of COLS query columns per block (row, KV head). The key
// rotations come into shared memory whole, their loads in flight together with the queries;
// thread (packed dim p, half) then sums R_g[i][j] q[j] for half of them, a power of two per
// column brings its largest entry near 2^13, and the fp16 hi and lo words go out in
// tensor-memory order. Latency bound: 512 blocks of the 70B-shaped layer with 64 nodes
// take 30 us (cold).
// COLS columns per block: 32, or 16 or 8 where more would leave SMs without one (8 rows
// x 8 KV heads of 64 columns, the whole call: 32 columns 94.8, 16 86.2, 8 88.5 us).
template <int COLS>
constexpr int kColLd = COLS + 4;   // row of columns in shared memory, 16-byte aligned
template <int COLS>
constexpr int kRotSmem = (kD * kD + kD * kColLd<COLS>) * int(sizeof(float));
// Floats of the key rotations of all groups (only what the layout has: five blocks of the
// preparation fit an SM then, instead of two).
__host__ __device__ inline int rot_floats(const DevLayout& L) {
  int n = 0;
  for (int g = 0; g < L.n_kgroups; ++g) n += L.group_dim[g] * L.group_dim[g];
  return n;
}
template <int COLS>
__global__ void __launch_bounds__(256) tree_prep_kernel(DevLayout L, TreeLaunch a, const void* __restrict__ q, int q_dtype,
                                                        float qscale, long long* __restrict__ prefix,
                                                        unsigned* __restrict__ qt, float* __restrict__ q_scale) {
  extern __shared__ __align__(128) unsigned char smem[];
  float* s_rot = reinterpret_cast<float*>(smem);      // the groups' rotations, transposed, one after the other
  float* s_q = s_rot + rot_floats(L);                 // [packed dim][column], then q' likewise
  __shared__ float s_up[COLS];
  __shared__ short s_pc[kD], s_dim[kMaxDims];
  pdl_trigger();
  const int tid = threadIdx.x, N = a.G * a.n_q, blocks = a.col_tiles * (kCols / COLS);
  if (blockIdx.x == 0 && tid < 32) {
    long long run = 0;
#pragma unroll 1
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
  const int c0 = cb * COLS;
  const long long u = (long long)b * a.row_units + (long long)h * a.col_tiles + c0 / kCols;
  const int in0 = c0 % kCols;  // first column inside the unit
  const int qw = a.q_words;
  if (c0 >= N) {  // columns that no query has: zeros
    for (int e = tid; e < COLS * 2 * qw / 4; e += 256)
      reinterpret_cast<uint4*>(qt)[((size_t)u * (2 * qw / 4) + e / COLS) * kCols + in0 + e % COLS] = make_uint4(0, 0, 0, 0);
    if (tid < COLS) q_scale[(size_t)u * kCols + in0 + tid] = 1.f;
    return;
  }
  for (int g = 0, at = 0; g < L.n_kgroups; ++g) {
    const int n = L.group_dim[g] * L.group_dim[g];  // (dimensions are even: a multiple of 4)
    const float4* src = reinterpret_cast<const float4*>(L.k_rot32t[g]);
#pragma unroll 4
    for (int e = tid; e < n / 4; e += 256) reinterpret_cast<float4*>(s_rot + at)[e] = __ldg(src + e);
    at += n;
  }
  if (tid < kD) s_pc[tid] = L.packed_coord[tid];
  // packed dim of every operand dim (quads of 8; -1 where a quad has no pair)
  for (int e = tid; e < 8 * L.n_kquads; e += 256) s_dim[e] = (e & 7) < 2 * L.quad_np[e >> 3] ? short(L.quad_dim0[e >> 3] + (e & 7)) : short(-1);
  __syncthreads();
#pragma unroll 8
  for (int e = tid; e < COLS * kD; e += 256) {
    const int c = e >> 7, p = e & (kD - 1), col = c0 + c;
    float x = 0.f;
    if (col < N && p < L.n_packed) {
      const size_t r = ((size_t)b * a.n_q + col / a.G) * (a.G * a.h_kv) + (size_t)h * a.G + col % a.G;
      x = load_q(q, q_dtype, r * kD + s_pc[p]);
    }
    s_q[p * kColLd<COLS> + c] = x;
  }
  __syncthreads();
  const int p = tid & (kD - 1), half = tid >> 7;
  float acc[COLS / 2];
#pragma unroll
  for (int c = 0; c < COLS / 2; ++c) acc[c] = 0.f;
  float f = 0.f;
  if (p < L.n_packed) {
    int g = 0, at = 0;
    while (g + 1 < L.n_kgroups && p >= L.group_off[g + 1]) {
      at += L.group_dim[g] * L.group_dim[g];
      ++g;
    }
    const int d = L.group_dim[g], off = L.group_off[g];
    const float* R = s_rot + at + (p - off);
    const float* x = s_q + off * kColLd<COLS> + COLS / 2 * half;
    f = qscale * rsqrtf(float(d)) * L.inv_kappa_group[g];
#pragma unroll 4
    for (int j = 0; j < d; ++j) {
      const float r = R[j * d];
#pragma unroll
      for (int k = 0; k < COLS / 8; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(x + j * kColLd<COLS> + 4 * k);
        acc[4 * k] = fmaf(r, v.x, acc[4 * k]);
        acc[4 * k + 1] = fmaf(r, v.y, acc[4 * k + 1]);
        acc[4 * k + 2] = fmaf(r, v.z, acc[4 * k + 2]);
        acc[4 * k + 3] = fmaf(r, v.w, acc[4 * k + 3]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < COLS / 8; ++k)
    *reinterpret_cast<float4*>(s_q + p * kColLd<COLS> + COLS / 2 * half + 4 * k) =
        make_float4(acc[4 * k] * f, acc[4 * k + 1] * f, acc[4 * k + 2] * f, acc[4 * k + 3] * f);
  __syncthreads();
  if (tid < 8 * COLS) {  // eight threads per column
    const int c = tid >> 3;
    float top = 0.f;
    for (int e = tid & 7; e < kD; e += 8) {
      const float x = fabsf(s_q[e * kColLd<COLS> + c]);
      if (x <= 3.0e38f) top = fmaxf(top, x);  // (an infinite or NaN q' keeps its column so)
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 7) == 0) {
      const int ex = top > 0.f ? min(60, max(-60, 13 - (int(__float_as_uint(top) >> 23) - 127))) : 0;
      s_up[c] = __int_as_float((127 + ex) << 23);
      q_scale[(size_t)u * kCols + in0 + c] = __int_as_float((127 - ex) << 23);
    }
  }
  __syncthreads();
  // word w of a column's part = operand dims 2w, 2w + 1; groups of 4 words, columns innermost
  for (int e = tid; e < COLS * qw / 4; e += 256) {
    const int c = e % COLS, w = e / COLS;
    unsigned hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int od = 8 * w + 2 * k + i, dim = od < 8 * L.n_kquads ? s_dim[od] : -1;
        v[i] = dim >= 0 ? s_q[dim * kColLd<COLS> + c] * s_up[c] : 0.f;
      }
      const float h0 = __half2float(__float2half_rn(v[0])), h1 = __half2float(__float2half_rn(v[1]));
      hi[k] = pack_h2(h0, h1);
      lo[k] = pack_h2(v[0] - h0, v[1] - h1);
    }
    uint4* at = reinterpret_cast<uint4*>(qt) + ((size_t)u * (2 * qw / 4) + w) * kCols + in0 + c;
    at[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    at[(size_t)(qw / 4) * kCols] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// Merge of a unit's partials for COLS query columns per block, then out = R_V^T o' / l with the
// rotation in shared memory (fetched before the wait for the partials): thread (output dim,
// half) sums half of the columns. Bound by its shared-memory reads and by latency.
template <int COLS>
__global__ void __launch_bounds__(256) tree_combine_kernel(DevLayout L, TreeLaunch a, int n_ctas, void* __restrict__ out,
                                                           int out_dtype) {
  extern __shared__ __align__(128) unsigned char smem[];
  float* s_rot = reinterpret_cast<float*>(smem);   // R_V [i][d]
  float* s_o = s_rot + kD * kD;                    // [value dim][column]
  const int tid = threadIdx.x, N = a.G * a.n_q, blocks = (N + COLS - 1) / COLS;
  pdl_trigger();
#pragma unroll
  for (int e = 0; e < kD * kD / 4 / 256; ++e)
    reinterpret_cast<float4*>(s_rot)[e * 256 + tid] = __ldg(reinterpret_cast<const float4*>(L.v_rot32) + e * 256 + tid);
  pdl_wait();
  const int cb = blockIdx.x % blocks, bh = blockIdx.x / blocks, h = bh % a.h_kv, b = bh / a.h_kv;
  const int c0 = cb * COLS, in0 = c0 % kCols;
  const long long k = (long long)h * a.col_tiles + c0 / kCols, u = (long long)b * a.row_units + k;
  const int n_nodes = a.tree.n_nodes ? a.tree.n_nodes[b] : a.n_q;
  const long long T = a.prefix[a.batch], C = min((long long)n_ctas, T), p0 = a.prefix[b], nt = (a.prefix[b + 1] - p0) / a.row_units;
  constexpr int kGroups = 256 / COLS, kVecs = 32 / kGroups;  // merge: column c, float4s wp, wp + kGroups, ..
  const int c = tid % COLS, wp = tid / COLS;
  // (a row without tiles has no partials: zeros)
  int first = 0, n = 0;
  if (nt > 0) {
    first = cta_of_tile(p0 + k * nt, T, C);
    n = cta_of_tile(p0 + (k + 1) * nt - 1, T, C) + 1 - first;
  }
  const bool live = c0 + c < N;
  const float2* ml = a.part_ml + (size_t)(first + u) * kCols + in0 + c;
  const float4* po = a.part_o + ((size_t)(first + u) * 32 + wp) * kCols + in0 + c;
  float top = -INFINITY, l = 0.f;
  float4 o[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  // kSlots partials at a time, their loads in flight together; the running maximum as usual
  constexpr int kSlots = COLS == 32 ? 4 : COLS == 16 ? 8 : 16;
#pragma unroll 1
  for (int s0 = 0; live && s0 < n; s0 += kSlots) {
    float2 v[kSlots];
    float4 x[kSlots][kVecs];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int sl = min(s0 + i, n - 1);
      v[i] = ml[(size_t)sl * kCols];
      if (s0 + i >= n) v[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) x[i][j] = __ldcs(po + ((size_t)sl * 32 + kGroups * j) * kCols);
    }
    float m = top;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) m = fmaxf(m, v[i].x);
    if (m == -INFINITY) {  // nothing seen (or NaN alone)
#pragma unroll
      for (int i = 0; i < kSlots; ++i) l += v[i].y;
      continue;
    }
    const float r = exp2f(top - m);
    l *= r;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) o[j] = make_float4(o[j].x * r, o[j].y * r, o[j].z * r, o[j].w * r);
    top = m;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      if (v[i].x == -INFINITY && v[i].y == 0.f) continue;
      const float f = exp2f(v[i].x - m);
      l = fmaf(f, v[i].y, l);
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        o[j] = make_float4(fmaf(f, x[i][j].x, o[j].x), fmaf(f, x[i][j].y, o[j].y), fmaf(f, x[i][j].z, o[j].z),
                           fmaf(f, x[i][j].w, o[j].w));
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    // accumulator column n = 8 blk + g holds value dim 16 g + blk
    const float x[4] = {o[j].x, o[j].y, o[j].z, o[j].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int nn = 4 * (wp + kGroups * j) + e;
      s_o[(16 * (nn & 7) + (nn >> 3)) * kColLd<COLS> + c] = x[e] * inv;
    }
  }
  __syncthreads();
  const int d = tid & (kD - 1), half = tid >> 7;
  unsigned long long acc[COLS / 4];
#pragma unroll
  for (int i = 0; i < COLS / 4; ++i) acc[i] = 0ull;
#pragma unroll 8
  for (int i = 0; i < kD; ++i) {
    const float r = s_rot[i * kD + d];
    const unsigned long long rr = pack2(r, r);
#pragma unroll
    for (int e = 0; e < COLS / 8; ++e) {
      const float4 x = *reinterpret_cast<const float4*>(s_o + i * kColLd<COLS> + COLS / 2 * half + 4 * e);
      acc[2 * e] = fma2(rr, pack2(x.x, x.y), acc[2 * e]);
      acc[2 * e + 1] = fma2(rr, pack2(x.z, x.w), acc[2 * e + 1]);
    }
  }
#pragma unroll
  for (int cc = 0; cc < COLS / 2; ++cc) {
    const int col = c0 + COLS / 2 * half + cc, node = col / a.G;
    // rows past a row's drafted nodes are not written (a row that does not fit: zeros)
    if (col >= N || (n_nodes >= 0 && node >= n_nodes)) continue;
    const float2 y = unpack2(acc[cc >> 1]);
    store_out(out, out_dtype, (((size_t)b * a.n_q + node) * (a.G * a.h_kv) + (size_t)h * a.G + col % a.G) * kD + d,
              cc & 1 ? y.y : y.x);
  }
}

int tree_q_words(const DevLayout& L) { return (L.n_kquads + 1) / 2 * 8; }

// The layout's quads for the decode warps. They lie in descending rate; each warp of a group
// takes a run of about equal cost (instructions per quad of rate 1..4), so that it and its
// partner in the other group, on the same scheduler, stay with the code of one or two rates.
void set_quads(const DevLayout& L, TreeLaunch& a) {
  auto cost = [](int r) { return r == 1 ? 6 : r == 2 ? 7 : 11; };
  int total = 0, run = 0, it = 0;
  for (int g = 0; g < L.n_kgroups; ++g) total += L.group_nquads[g] * cost(L.group_rate[g]);
  for (int g = 0; g < L.n_kgroups; ++g)
    for (int i = 0; i < L.group_nquads[g]; ++i, ++it) {
      const int r = L.group_rate[g], c = cost(r), w = std::min(kDecGroup - 1, (2 * run + c) * kDecGroup / (2 * total));
      a.quad[it] = unsigned(L.quad_off[it]) | unsigned(L.quad_np[it]) << 16 | unsigned(g) << 20 | unsigned(r) << 24;
      if (a.range[w][r][1] == 0) a.range[w][r][0] = (unsigned char)it;
      a.range[w][r][1] = (unsigned char)(it + 1);
      run += c;
    }
}

int tree_smem_bytes(const DevLayout& L, int stages) {
  const int vt = L.v_rate == 3 ? vtab_bytes<3>() : L.v_rate == 4 ? vtab_bytes<4>() : 0;
  return kTbl8Bytes + kTbl3Bytes + vt + 128 + kUnitBytes + 4 * ((L.n_kquads + 1) / 2) * 2048 + 2 * 16384 +
         stages * (kNormBytes + L.tile_bytes);
}

// Once per device: the kernel's dynamic shared memory limit raised to what a block may use.
template <typename K>
cudaError_t raise_smem_limit(K kernel, bool (&done)[64]) {
  int dev = 0, optin = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  cudaFuncAttributes fa{};
  e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - int(fa.sharedSizeBytes));
  done[dev] = e == cudaSuccess;
  return e;
}

template <int VR, bool NH>
cudaError_t launch_tree_kernel(const DevLayout& L, const TreeLaunch& a, unsigned grid, int smem, cudaStream_t stream) {
  static bool done[64] = {};
  cudaError_t e = raise_smem_limit(tree_kernel<VR, NH>, done);
  if (e != cudaSuccess) return e;
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
  set_quads(L, a);
  const int limit = split_smem_limit();
  a.stages = kMaxStages;
  while (a.stages > 2 && tree_smem_bytes(L, a.stages) > limit) a.stages >>= 1;
  const int smem = tree_smem_bytes(L, a.stages);
  if (smem > limit) return cudaErrorInvalidValue;
  const long long heads = (long long)batch * h_kv;
  const int N = a.G * n_q;
  // columns per block of the preparation and the merge: the most that give every SM a block
  const int block_cols = heads * ((N + 31) / 32) >= plan.n_ctas ? 32 : heads * ((N + 15) / 16) >= plan.n_ctas ? 16 : 8;
  auto prep = [&](auto cols) {
    constexpr int COLS = decltype(cols)::value;
    static bool done[64] = {};
    const cudaError_t e = raise_smem_limit(tree_prep_kernel<COLS>, done);
    if (e != cudaSuccess) return e;
    tree_prep_kernel<COLS><<<unsigned(heads * plan.col_tiles * (kCols / COLS)), 256,
                             kRotSmem<COLS> - (kD * kD - rot_floats(L)) * int(sizeof(float)), stream>>>(
        L, a, q, q_dtype, softmax_scale * kLog2e, reinterpret_cast<long long*>(ws + plan.prefix_at),
        reinterpret_cast<unsigned*>(ws + plan.q_at), reinterpret_cast<float*>(ws + plan.scale_at));
    return cudaGetLastError();
  };
  cudaError_t e = block_cols == 32 ? prep(IntC<32>{}) : block_cols == 16 ? prep(IntC<16>{}) : prep(IntC<8>{});
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
  auto combine = [&](auto cols) {
    constexpr int COLS = decltype(cols)::value;
    static bool done[64] = {};
    const cudaError_t e = raise_smem_limit(tree_combine_kernel<COLS>, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(heads * ((N + COLS - 1) / COLS)));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = kRotSmem<COLS>;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_combine_kernel<COLS>, L, a, plan.n_ctas, out, out_dtype);
  };
  return block_cols == 32 ? combine(IntC<32>{}) : block_cols == 16 ? combine(IntC<16>{}) : combine(IntC<8>{});
}

}  // namespace bgtq
