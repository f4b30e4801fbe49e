// Selection of the key blocks that each block of 128 queries attends:
//   score(i, j) = mean(valid rows of query block i) . mean(valid rows of key block j)
// and the topk best key blocks of each query block, ties to the lower index.
// The means and the scores are in 64 bits: a list is decided by comparisons, so
// two scores closer than their rounding errors would be listed by accident.
#include "h3b_common.cuh"
#include "h3b_internal.h"

namespace h3b {
namespace {

constexpr int kMaxKeyBlocks = 4096;

__device__ __forceinline__ int clamp_len(const int* lens, int b, int L) {
  return lens ? min(max(lens[b], 0), L) : L;
}

// means[row][block][lane]: a block per (row = batch item x head, block), a thread per lane.
__global__ void __launch_bounds__(128) block_means_kernel(const __nv_bfloat16* __restrict__ x, const int* lens, int heads,
                                                          int L, int DH, int size, int n_blocks, double* means,
                                                          long long n_means, unsigned* err) {
  griddep_wait();
  griddep_launch_dependents();
  const int blk = blockIdx.x, row = blockIdx.y;
  const int n = min(clamp_len(lens, row / heads, L) - blk * size, size);
  const __nv_bfloat16* p = x + ((size_t)row * L + (size_t)blk * size) * DH + threadIdx.x;
  double s = 0.0;
  for (int i = 0; i < n; ++i) s += (double)__bfloat162float(p[(size_t)i * DH]);
  const long long at = ((long long)row * n_blocks + blk) * DH + threadIdx.x;
  if (H3B_IDX_OK(at, n_means, err)) means[at] = n > 0 ? s / n : 0.0;
}

// The order of the scores as unsigned integers: higher is better, -0 equals +0, NaN is last.
__device__ __forceinline__ unsigned long long order_key(double s) {
  if (s != s) return 1ull;
  const unsigned long long u = (unsigned long long)__double_as_longlong(s + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
constexpr unsigned long long kKeyKeep = ~0ull;

// A block per (query block, batch item x head): scores of all key blocks, then each block's rank.
__global__ void __launch_bounds__(256) select_kernel(const SelectArgs a, const double* qm, const double* km) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ unsigned long long keys[];  // [nkb]
  __shared__ double qs[128];
  __shared__ int warp_n[8];
  const int i = blockIdx.x, row = blockIdx.y, DH = a.head_dim;
  const int b = row / a.n_heads, h = row - b * a.n_heads;
  const int kvrow = b * a.n_kv_heads + h / (a.n_heads / a.n_kv_heads);
  const int qn = clamp_len(a.q_lens, b, a.Lq), kn = clamp_len(a.kv_lens, b, a.Lk);
  const int cand = i * kSparseQueries < qn ? (kn + a.block_k - 1) / a.block_k : 0;
  const int want = min(cand, a.topk);
  if (threadIdx.x < DH) qs[threadIdx.x] = qm[((size_t)row * a.nqb + i) * DH + threadIdx.x];
  __syncthreads();
  const int lo = i * kSparseQueries / a.block_k - a.keep_local + 1;
  const int hi = (i * kSparseQueries + kSparseQueries - 1) / a.block_k + a.keep_local - 1;
  for (int j = threadIdx.x; j < cand; j += blockDim.x) {
    const double* kk = km + ((size_t)kvrow * a.nkb + j) * DH;
    double s = 0.0;
    for (int e = 0; e < DH; ++e) s = fma(qs[e], kk[e], s);
    const bool keep = j < a.keep_first || (a.keep_local > 0 && j >= lo && j <= hi);
    keys[j] = keep ? kKeyKeep : order_key(s);
  }
  __syncthreads();
  const long long list = (long long)row * a.nqb + i;
  int* out = a.blocks + list * a.topk;
  int done = 0;
  for (int j0 = 0; j0 < cand; j0 += blockDim.x) {
    const int j = j0 + threadIdx.x;
    bool take = false;
    if (j < cand) {
      const unsigned long long mine = keys[j];
      int rank = 0;
      for (int o = 0; o < cand; ++o) rank += keys[o] > mine || (keys[o] == mine && o < j);
      take = rank < want;
    }
    const unsigned m = __ballot_sync(0xFFFFFFFFu, take);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) warp_n[warp] = __popc(m);
    __syncthreads();
    int at = done + __popc(m & ((1u << lane) - 1u));
    for (int w = 0; w < 8; ++w) {
      if (w < warp) at += warp_n[w];
      done += warp_n[w];
    }
    if (take && H3B_IDX_OK(at, want, a.err)) out[at] = j;
    __syncthreads();
  }
  for (int t = want + threadIdx.x; t < a.topk; t += blockDim.x) out[t] = -1;
  if (threadIdx.x == 0) a.counts[list] = want;
}

}  // namespace

size_t select_ws_bytes(int B, int n_heads, int n_kv_heads, int head_dim, int nqb, int nkb) {
  return sizeof(double) * (size_t)head_dim * B * ((size_t)n_heads * nqb + (size_t)n_kv_heads * nkb);
}

cudaError_t launch_select_blocks(const SelectArgs& a, int sms, cudaStream_t st) {
  (void)sms;
  double* qm = static_cast<double*>(a.ws);
  const long long nq = (long long)a.B * a.n_heads * a.nqb * a.head_dim;
  const long long nk = (long long)a.B * a.n_kv_heads * a.nkb * a.head_dim;
  double* km = qm + nq;
  cudaError_t e = launch_pdl(block_means_kernel, dim3(a.nqb, a.B * a.n_heads), dim3(a.head_dim), 0, st,
                             static_cast<const __nv_bfloat16*>(a.q), a.q_lens, a.n_heads, a.Lq, a.head_dim,
                             kSparseQueries, a.nqb, qm, nq, a.err);
  if (e != cudaSuccess) return e;
  e = launch_pdl(block_means_kernel, dim3(a.nkb, a.B * a.n_kv_heads), dim3(a.head_dim), 0, st,
                 static_cast<const __nv_bfloat16*>(a.k), a.kv_lens, a.n_kv_heads, a.Lk, a.head_dim, a.block_k, a.nkb,
                 km, nk, a.err);
  if (e != cudaSuccess) return e;
  static_assert(kMaxKeyBlocks * 8 <= 48 * 1024, "the keys fit the default shared memory");
  return launch_pdl(select_kernel, dim3(a.nqb, a.B * a.n_heads), dim3(256), (size_t)a.nkb * 8, st, a,
                    (const double*)qm, (const double*)km);
}

}  // namespace h3b
