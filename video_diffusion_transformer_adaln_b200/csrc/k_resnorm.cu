// Gated residual with a norm on each side of it, in one pass over the rows:
//   x_out = bf16(x + alpha * gate * (post_norm(y) * w_post))
//   h     = bf16(pre_norm(x_out) * (1 + scale) + shift)
// and the per-row int8 quantizer of h. Bound by HBM: y and x are read once,
// x_out and h (or its codes) written once, 8 (7) bytes a channel.
#include "h3b_common.cuh"
#include "h3b_internal.h"
#include "h3b_quant.cuh"

namespace h3b {
namespace {

constexpr int kThreads = 128;

// Sum (or maximum) over the block; every thread gets it.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* slots) {
  v = kMax ? warp_max(v) : warp_sum(v);
  __syncthreads();  // the slots' last readers are done
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = slots[0];
  for (int w = 1; w < kThreads / 32; ++w) r = kMax ? fmaxf(r, slots[w]) : r + slots[w];
  return r;
}

// A block per row, VPT 16-byte vectors per thread.
template <int VPT>
__global__ void __launch_bounds__(kThreads) residual_norm_kernel(const ResNormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float slots[kThreads / 32];
  const int row = blockIdx.x, vpr = a.d / 8;
  const size_t item = (size_t)(row / a.rows_per_item) * a.mod_stride;
  const uint4* y = static_cast<const uint4*>(a.y) + (size_t)row * vpr;
  const uint4* x = static_cast<const uint4*>(a.x) + (size_t)row * vpr;
  const float inv_d = 1.0f / (float)a.d;
  float f[VPT * 8], xf[VPT * 8];
  auto unpack = [](uint4 u, float* o) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[2 * e] = bf16_lo(w[e]);
      o[2 * e + 1] = bf16_hi(w[e]);
    }
  };
  auto has = [&](int i) {
    const int vec = threadIdx.x + kThreads * i;
    return vec < vpr && H3B_IDX_OK((long long)row * vpr + vec, (long long)a.rows * vpr, a.err);
  };
  auto norm = [&](float* v, int kind, float eps) {  // mean and rstd applied in place
    if (kind == 0) return;
    if (kind == 2) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT * 8; ++i) sum += v[i];
      const float mean = block_reduce<false>(sum, slots) * inv_d;
#pragma unroll
      for (int i = 0; i < VPT * 8; ++i)
        if (has(i / 8)) v[i] -= mean;
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT * 8; ++i) sq = fmaf(v[i], v[i], sq);
    const float rstd = 1.0f / sqrtf(block_reduce<false>(sq, slots) * inv_d + eps);
#pragma unroll
    for (int i = 0; i < VPT * 8; ++i) v[i] *= rstd;
  };
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = threadIdx.x + kThreads * i;
    unpack(has(i) ? __ldcs(y + vec) : make_uint4(0, 0, 0, 0), f + 8 * i);
    unpack(has(i) ? __ldcs(x + vec) : make_uint4(0, 0, 0, 0), xf + 8 * i);
  }
  norm(f, a.post_norm, a.post_eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (!has(i)) continue;
    const int vec = threadIdx.x + kThreads * i;
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = vec * 8 + e;
      const float w = a.w_post ? a.w_post[c] : 1.0f, g = a.gate ? a.gate[item + c] : 1.0f;
      xf[8 * i + e] = round_bf16(xf[8 * i + e] + a.alpha * g * (f[8 * i + e] * w));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = pack_bf16x2(xf[8 * i + 2 * e], xf[8 * i + 2 * e + 1]);
    static_cast<uint4*>(a.x_out)[(size_t)row * vpr + vec] = make_uint4(u[0], u[1], u[2], u[3]);
  }
  if (a.absmax_zero && threadIdx.x == 0) a.absmax_zero[row] = 0.0f;
  if (!a.h_out && !a.q) return;
  norm(xf, a.pre_norm, a.pre_eps);
  float am = 0.0f;
  uint4 h[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = threadIdx.x + kThreads * i;
    if (!has(i)) continue;
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = vec * 8 + e;
      const float sc = a.scale ? a.scale[item + c] : 0.0f, sh = a.shift ? a.shift[item + c] : 0.0f;
      f[8 * i + e] = round_bf16(fmaf(xf[8 * i + e], 1.0f + sc, sh));
      am = fmaxf(am, fabsf(f[8 * i + e]));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = pack_bf16x2(f[8 * i + 2 * e], f[8 * i + 2 * e + 1]);
    h[i] = make_uint4(u[0], u[1], u[2], u[3]);
    if (a.h_out) static_cast<uint4*>(a.h_out)[(size_t)row * vpr + vec] = h[i];
  }
  if (!a.q) return;
  const float amax = block_reduce<true>(am, slots);
  const float sc = __fdiv_rn(amax, 127.0f), rcp = __frcp_rn(sc);
  if (threadIdx.x == 0) a.s[row] = sc;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (has(i))
      reinterpret_cast<uint2*>(a.q)[(size_t)row * vpr + threadIdx.x + kThreads * i] = quant8<true>(h[i], sc, rcp, amax);
}

}  // namespace

cudaError_t launch_residual_norm(const ResNormArgs& a, int sms, cudaStream_t st) {
  (void)sms;
  const int vpr = a.d / 8;
  if (vpr <= kThreads) return launch_pdl(residual_norm_kernel<1>, dim3(a.rows), dim3(kThreads), 0, st, a);
  if (vpr <= 2 * kThreads) return launch_pdl(residual_norm_kernel<2>, dim3(a.rows), dim3(kThreads), 0, st, a);
  if (vpr <= 4 * kThreads) return launch_pdl(residual_norm_kernel<4>, dim3(a.rows), dim3(kThreads), 0, st, a);
  return launch_pdl(residual_norm_kernel<8>, dim3(a.rows), dim3(kThreads), 0, st, a);
}

}  // namespace h3b
