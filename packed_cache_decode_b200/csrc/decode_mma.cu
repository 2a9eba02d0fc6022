// Host launchers of the decode kernels (decode_split.cuh): the launch plan, decode attention,
// the decode step, the logits and the merge of partial records.
#include <cuda_runtime.h>

#include <algorithm>

#include "decode_split.cuh"

namespace bgtq {

DecodePlan plan_decode(int batch, int h_q, int h_kv, long long max_seq_len, int num_sms, int /*ctas_per_sm*/) {
  DecodePlan p{};
  // h_q counts query columns; more than 8 per KV head are split into column tiles
  const int Gt = h_q / h_kv, CT = (Gt + kMaxG - 1) / kMaxG, G = CT == 1 ? Gt : kMaxG;
  p.max_tiles = int((max_seq_len + kTile - 1) / kTile);
  if (p.max_tiles < 1) p.max_tiles = 1;
  const long long units = (long long)batch * h_kv * CT;
  const long long total = units * p.max_tiles;
  // one CTA per SM, slices of equal length (+-1 tile); a slice may span several units
  long long C = std::min<long long>(num_sms, total);
  // a unit meets at most ceil(C / units) + 1 slices; the merge takes up to kMaxParts
  while (C > 1 && (C + units - 1) / units + 1 > kMaxParts) --C;
  p.n_ctas = int(C);
  p.tiles_per_cta = int((total + C - 1) / C);
  p.n_parts = int((C + units - 1) / units + 1);
  p.workspace_bytes = qfrag_bytes(units) +
                      align256(size_t(units) * p.n_parts * G * 2 * sizeof(float)) +
                      size_t(units) * p.n_parts * G * kD * sizeof(float);
  return p;
}

cudaError_t launch_decode(const DevLayout& L, const DecodePlan& plan, const void* q, int q_dtype, int batch,
                          int h_q, int h_kv, int n_q, const CacheRef& cache, const int* seq_lens, float softmax_scale,
                          float* out, void* workspace, cudaStream_t stream, float* rec, const DevLayout* heads) {
  const int Gt = h_q * n_q / h_kv;
  const long long units = (long long)batch * h_kv * ((Gt + kMaxG - 1) / kMaxG);
  // a plain launch: the split kernel, launched as soon as this kernel starts, reads the
  // cache, which the kernel before this one may write
  if (heads)
    qprep_kernel<true, false><<<unsigned(units), kPrepThreads, 0, stream>>>(
        L, heads, q, q_dtype, h_q, h_kv, Gt, n_q, softmax_scale * kLog2e, static_cast<unsigned*>(workspace));
  else
    qprep_kernel<false, false><<<unsigned(units), kPrepThreads, 0, stream>>>(
        L, nullptr, q, q_dtype, h_q, h_kv, Gt, n_q, softmax_scale * kLog2e, static_cast<unsigned*>(workspace));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_attention<false>(L, plan, batch, h_q, h_kv, n_q, cache, seq_lens, out, workspace, 0, false, stream,
                          nullptr, 0, rec, heads);
}

namespace {
// One CTA of 128 threads per (batch row, query column): log-sum-exp merge of n_rec partial
// records (m, l, o') of the same column over disjoint token ranges, then o = R_V^T o'.
__global__ void __launch_bounds__(kD) merge_records_kernel(const float* __restrict__ recs, int n_rec,
                                                           long long rec_stride, const float* __restrict__ v_rot,
                                                           float* __restrict__ out) {
  const int col = blockIdx.x, d = threadIdx.x;
  __shared__ float op[kD];
  const float* r0 = recs + (size_t)col * (kD + 2);
  float M = -INFINITY;
  for (int r = 0; r < n_rec; ++r) M = fmaxf(M, r0[(size_t)r * rec_stride]);
  float den = 0.f, o = 0.f;
  if (M != -INFINITY)
    for (int r = 0; r < n_rec; ++r) {
      const float* x = r0 + (size_t)r * rec_stride;
      const float w = x[0] == -INFINITY ? 0.f : exp2f(x[0] - M) * x[1];
      den += w;
      o = fmaf(w, x[2 + d], o);
    }
  op[d] = den > 0.f ? o / den : 0.f;
  __syncthreads();
  float acc0 = 0.f, acc1 = 0.f;
#pragma unroll 8
  for (int i = 0; i < kD; i += 2) {
    acc0 = fmaf(__ldg(v_rot + (size_t)i * kD + d), op[i], acc0);
    acc1 = fmaf(__ldg(v_rot + (size_t)(i + 1) * kD + d), op[i + 1], acc1);
  }
  out[(size_t)col * kD + d] = acc0 + acc1;
}
}  // namespace

cudaError_t launch_merge_records(const DevLayout& L, const float* recs, int n_rec, long long columns, float* out,
                                 cudaStream_t stream) {
  merge_records_kernel<<<unsigned(columns), kD, 0, stream>>>(recs, n_rec, columns * (kD + 2), L.v_rot32, out);
  return cudaGetLastError();
}

cudaError_t launch_scores(const DevLayout& L, const DecodePlan& plan, const void* q, int q_dtype, int batch, int h_q,
                          int h_kv, const CacheRef& cache, const int* seq_lens, long long max_seq_len,
                          float softmax_scale, float* scores, long long scores_ld, void* workspace,
                          cudaStream_t stream, const DevLayout* heads) {
  const int Gt = h_q / h_kv;
  const long long units = (long long)batch * h_kv * ((Gt + kMaxG - 1) / kMaxG);
  if (heads)
    qprep_kernel<true, false><<<unsigned(units), kPrepThreads, 0, stream>>>(
        L, heads, q, q_dtype, h_q, h_kv, Gt, 1, softmax_scale * kLog2e, static_cast<unsigned*>(workspace));
  else
    qprep_kernel<false, false><<<unsigned(units), kPrepThreads, 0, stream>>>(
        L, nullptr, q, q_dtype, h_q, h_kv, Gt, 1, softmax_scale * kLog2e, static_cast<unsigned*>(workspace));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_attention<false>(L, plan, batch, h_q, h_kv, 1, cache, seq_lens, nullptr, workspace, 0, false, stream,
                          scores, scores_ld, nullptr, heads, BGTQ_F32, MassArgs{}, TreeArgs{}, max_seq_len);
}

cudaError_t launch_decode_step(const DevLayout& L, const DecodePlan& plan, const void* k_new, const void* v_new,
                               int kv_dtype, int n_new, const int* seq_lens_before, const void* q, int q_dtype,
                               int batch, int h_q, int h_kv, int n_q, const CacheRef& cache, float softmax_scale,
                               float* out, void* workspace, cudaStream_t stream, const DevLayout* heads) {
  const int Gt = h_q * n_q / h_kv;
  const long long cache_units = (long long)batch * h_kv;
  const long long units = cache_units * ((Gt + kMaxG - 1) / kMaxG);  // q' units (column tiles)
  const long long n_enc = (long long)n_new * kEncodeParts * cache_units;
  cudaError_t e;
  if (!L.norm_correct) {
    e = launch_dependent(heads ? step_prep_kernel<false, true> : step_prep_kernel<false, false>,
                         unsigned(n_enc + units), kPrepThreads, stream, L, heads, k_new,
                         v_new, kv_dtype, n_new, batch, seq_lens_before, cache, q, q_dtype, h_q, h_kv, Gt, n_q,
                         softmax_scale * kLog2e, static_cast<unsigned*>(workspace), int(n_enc));
  } else {
    // norm correction: clusters of the four encode parts of a token; the q' blocks
    // follow, padded to a whole cluster (the padding blocks return at once)
    const long long n_blocks = (n_enc + units + kEncodeParts - 1) / kEncodeParts * kEncodeParts;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(n_blocks));
    cfg.blockDim = dim3(kPrepThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kEncodeParts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, heads ? step_prep_kernel<true, true> : step_prep_kernel<true, false>, L, heads,
                           k_new, v_new, kv_dtype, n_new, batch, seq_lens_before, cache, q, q_dtype, h_q, h_kv, Gt,
                           n_q, softmax_scale * kLog2e, static_cast<unsigned*>(workspace), int(n_enc));
  }
  if (e != cudaSuccess) return e;
  return launch_attention<false>(L, plan, batch, h_q, h_kv, n_q, cache, seq_lens_before, out, workspace, n_new,
                          n_new > 0, stream, nullptr, 0, nullptr, heads);
}

}  // namespace bgtq
