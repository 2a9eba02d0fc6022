// The decode kernels' extended variants (decode_split.cuh, EX): drafted trees of few query
// columns, and decode attention that keeps an attention mass.
//
// Precision. Logits to 2^-20 and sums in fp32; the outputs' weights (times the value norms) are fp16
// as in plain decode, half a step of 2^-11 of a weight with each warp's largest at 1: 3.1e-4
// from the 64-bit outputs with fp16 queries and outputs over 9001 tokens of K3V3, where fp32 weights
// give 2.1e-4. Weights as hi + lo would double the value products of a kernel bound by issue. The
// attention mass does not pass through them: it is formed from the fp32 logits.
#include <cuda_runtime.h>

#include <algorithm>

#include "decode_split.cuh"

namespace bgtq {

cudaError_t launch_tree_columns(const DevLayout& L, const DecodePlan& plan, const void* q, int q_dtype, int batch,
                                int h_q, int h_kv, int n_q, const TreeArgs& tree, const CacheRef& cache,
                                const int* seq_lens, long long max_seq_len, float softmax_scale, void* out,
                                int out_dtype, void* workspace, cudaStream_t stream) {
  const int Gt = h_q * n_q / h_kv;
  const long long units = (long long)batch * h_kv * ((Gt + kMaxG - 1) / kMaxG);
  qprep_kernel<false, true><<<unsigned(units), kPrepThreads, 0, stream>>>(
      L, nullptr, q, q_dtype, h_q, h_kv, Gt, n_q, softmax_scale * kLog2e, static_cast<unsigned*>(workspace));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_attention<true>(L, plan, batch, h_q, h_kv, n_q, cache, seq_lens, out, workspace, 0, false, stream, nullptr, 0,
                          nullptr, nullptr, out_dtype, MassArgs{}, tree, max_seq_len);
}

size_t mass_logits_bytes(int batch, int h_q, const DecodePlan& plan) {
  return size_t(batch) * h_q * plan.max_tiles * kTile * sizeof(float);
}

cudaError_t launch_decode_mass(const DevLayout& L, const DecodePlan& plan, const void* q, int q_dtype, int batch,
                               int h_q, int h_kv, const CacheRef& cache, const int* seq_lens, long long max_seq_len,
                               float softmax_scale, float decay, float* mass, long long mass_ld, void* out,
                               int out_dtype, void* workspace, cudaStream_t stream) {
  const int Gt = h_q / h_kv;
  const long long units = (long long)batch * h_kv * ((Gt + kMaxG - 1) / kMaxG);
  qprep_kernel<false, true><<<unsigned(units), kPrepThreads, 0, stream>>>(
      L, nullptr, q, q_dtype, h_q, h_kv, Gt, 1, softmax_scale * kLog2e, static_cast<unsigned*>(workspace));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  MassArgs m{};
  m.mass = mass;
  m.ld = mass_ld;
  m.decay = decay;
  m.logits = reinterpret_cast<const float*>(static_cast<char*>(workspace) + align256(plan.workspace_bytes));
  m.logits_ld = (long long)plan.max_tiles * kTile;
  m.seq_lens = seq_lens;
  m.cache = cache;
  m.most = max_seq_len;
  return launch_attention<true>(L, plan, batch, h_q, h_kv, 1, cache, seq_lens, out, workspace, 0, false, stream, nullptr, 0,
                          nullptr, nullptr, out_dtype, m, TreeArgs{}, max_seq_len);
}

}  // namespace bgtq
