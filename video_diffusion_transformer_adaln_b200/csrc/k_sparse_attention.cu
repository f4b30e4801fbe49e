// Softmax attention of blocks of 128 queries over listed blocks of keys:
//   O[i] = sum_j softmax_j(Q[i].K[j] / sqrt(head_dim)) V[j],  j in the listed blocks
// One pass over the list with the running maximum and sum of the softmax.
#include "h3b_common.cuh"
#include "h3b_internal.h"
#include "h3b_softmax.cuh"

namespace h3b {
namespace {

__device__ __forceinline__ int clamp_len(const int* lens, int b, int L) {
  return lens ? min(max(lens[b], 0), L) : L;
}

constexpr int kKeys = 32;  // keys staged at a time

// A block per (query block, batch item x head), a thread per query row.
template <int DH>
__global__ void __launch_bounds__(kSparseQueries) sparse_attention_kernel(const SparseAttnArgs a, float scale_log2) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float ks[kKeys][DH], vs[kKeys][DH];
  const int i = blockIdx.x, bh = blockIdx.y;
  const int b = bh / a.n_heads, h = bh - b * a.n_heads;
  const int kvrow = b * a.n_kv_heads + h / (a.n_heads / a.n_kv_heads);
  const int qn = clamp_len(a.q_lens, b, a.Lq), kn = clamp_len(a.kv_lens, b, a.Lk);
  const int l = i * kSparseQueries + threadIdx.x;
  const bool mine = l < qn;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)bh * a.Lq + l) * DH;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + (size_t)kvrow * a.Lk * DH;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + (size_t)kvrow * a.Lk * DH;
  float o[DH], qf[DH];
#pragma unroll
  for (int e = 0; e < DH; ++e) {
    o[e] = 0.0f;
    qf[e] = mine ? __bfloat162float(q[e]) * scale_log2 : 0.0f;
  }
  float m = -INFINITY, sum = 0.0f;
  const long long list = (long long)bh * a.nqb + i;
  const int count = a.counts ? min(max(a.counts[list], 0), a.topk) : a.topk;
  for (int t = 0; t < count; ++t) {
    const int blk = a.blocks[list * a.topk + t];
    if (blk < 0 || blk >= a.nkb) continue;
    const int end = min(kn, (blk + 1) * a.block_k);
    for (int j0 = blk * a.block_k; j0 < end; j0 += kKeys) {
      const int n = min(kKeys, end - j0);
      __syncthreads();
      for (int x = threadIdx.x; x < n * DH; x += kSparseQueries) {
        ks[x / DH][x % DH] = __bfloat162float(k[(size_t)j0 * DH + x]);
        vs[x / DH][x % DH] = __bfloat162float(v[(size_t)j0 * DH + x]);
      }
      __syncthreads();
      for (int j = 0; j < n; ++j) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < DH; ++e) s = fmaf(qf[e], ks[j][e], s);
        if (s > m) {
          const float alpha = exp2f(m - s);
          m = s;
          sum *= alpha;
#pragma unroll
          for (int e = 0; e < DH; ++e) o[e] *= alpha;
        }
        const float p = exp2f(s - m);
        sum += p;
#pragma unroll
        for (int e = 0; e < DH; ++e) o[e] = fmaf(p, vs[j][e], o[e]);
      }
    }
  }
  if (!mine) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  float amax = 0.0f;
  const long long at = ((long long)b * a.Lq + l) * a.n_heads * DH + h * DH;
  if (!H3B_IDX_OK(at + DH - 1, (long long)a.B * a.Lq * a.n_heads * DH, a.err)) return;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + at;
#pragma unroll
  for (int e = 0; e < DH; ++e) {
    dst[e] = __float2bfloat16_rn(o[e] * inv);
    amax = fmaxf(amax, fabsf(__bfloat162float(dst[e])));
  }
  if (a.absmax) atomicMax(reinterpret_cast<unsigned*>(a.absmax) + (size_t)b * a.Lq + l, __float_as_uint(amax));
}

}  // namespace

size_t sparse_attn_ws_bytes(int B, int n_heads, int head_dim, int nqb, int topk, int block_k) {
  (void)B; (void)n_heads; (void)head_dim; (void)nqb; (void)topk; (void)block_k;
  return 0;
}

cudaError_t launch_sparse_attention(const SparseAttnArgs& a, cudaStream_t st) {
  const dim3 grid(a.nqb, a.B * a.n_heads);
  const float scale_log2 = 1.4426950408889634f / sqrtf((float)a.head_dim);
  if (a.head_dim == 128)
    return launch_pdl(sparse_attention_kernel<128>, grid, dim3(kSparseQueries), 0, st, a, scale_log2);
  return launch_pdl(sparse_attention_kernel<64>, grid, dim3(kSparseQueries), 0, st, a, scale_log2);
}

}  // namespace h3b
