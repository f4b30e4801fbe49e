// Per-head RMSNorm of Q and K and rotary positions on three axes given per
// token, from a token-major projection to the head-major layout:
//   y = x * rsqrt(mean(x^2) + eps) * w            (over the head's lanes)
//   (y[2p], y[2p+1]) turned by pos[axis(p)] * theta^(-2j/r)
// Bound by HBM: every element is read and written once, 4 bytes of traffic.
#include "h3b_common.cuh"
#include "h3b_internal.h"

namespace h3b {
namespace {

constexpr int kThreads = 256;

// (cos, sin) of pair p at this token. The angle in half turns is reduced to
// [-1, 1] in 64 bits before it is rounded to 32, so its error is that of a
// value below pi for any position.
__device__ __forceinline__ float2 pair_turn(const QkRopeArgs& a, const float* pos, int p) {
  const int ax = p < a.axis_end[0] ? 0 : p < a.axis_end[1] ? 1 : 2;
  const double t = (double)pos[ax] * a.freq[p];
  float s, c;
  sincospif((float)(t - 2.0 * rint(0.5 * t)), &s, &c);
  return make_float2(c, s);
}

// A block per token; DH / 8 lanes per head row, one 16-byte vector each.
template <int DH>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ QkRopeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int LPR = DH / 8;  // lanes per head row
  __shared__ float2 turn[DH / 2];
  const int tok = blockIdx.x;
  const int b = tok / a.L, l = tok - b * a.L;
  if (threadIdx.x < DH / 2) {
    const int p = threadIdx.x;
    turn[p] = a.pos && p < a.axis_end[2] ? pair_turn(a, a.pos + (size_t)tok * 3, p) : make_float2(1.0f, 0.0f);
  }
  __syncthreads();
  const int sub = threadIdx.x % LPR, H = a.n_heads, KV = a.n_kv_heads;
  const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.qkv) + (size_t)tok * a.row_stride);
  for (int h0 = 0; h0 < H + 2 * KV; h0 += kThreads / LPR) {  // block-uniform: whole warps take part in the shuffles
    const int h = h0 + threadIdx.x / LPR;
    const bool on = h < H + 2 * KV;
    uint4 u = on ? __ldcs(row + h * LPR + sub) : make_uint4(0, 0, 0, 0);
    const int part = h < H ? 0 : h < H + KV ? 1 : 2;
    const float* w = part == 0 ? a.wq : a.wk;
    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
    float f[8];
    float sq = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = bf16_lo(in[e]);
      f[2 * e + 1] = bf16_hi(in[e]);
      sq = fmaf(f[2 * e], f[2 * e], fmaf(f[2 * e + 1], f[2 * e + 1], sq));
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
    if (!on) continue;
    if (part < 2) {
      if (w) {
        const float rstd = 1.0f / sqrtf(sq * (1.0f / DH) + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * w[sub * 8 + e];
      }
      uint32_t out[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = turn[sub * 4 + e];
        out[e] = pack_bf16x2(f[2 * e] * t.x - f[2 * e + 1] * t.y, f[2 * e] * t.y + f[2 * e + 1] * t.x);
      }
      u = make_uint4(out[0], out[1], out[2], out[3]);
    }
    const int heads = part == 0 ? H : KV, hh = h - (part == 0 ? 0 : part == 1 ? H : H + KV);
    uint4* dst = static_cast<uint4*>(part == 0 ? a.q : part == 1 ? a.k : a.v);
    const size_t at = (((size_t)b * heads + hh) * a.L + l) * LPR + sub;
    if (H3B_IDX_OK(at, (long long)a.B * heads * a.L * LPR, a.err)) dst[at] = u;
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkRopeArgs& a, int sms, cudaStream_t st) {
  (void)sms;
  const dim3 grid((unsigned)((long long)a.B * a.L));
  if (a.head_dim == 128) return launch_pdl(qk_norm_rope_kernel<128>, grid, dim3(kThreads), 0, st, a);
  return launch_pdl(qk_norm_rope_kernel<64>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace h3b
