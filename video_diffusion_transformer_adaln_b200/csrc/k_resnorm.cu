// Gated residual with a norm on each side of it, in one pass over the rows:
//   x_out = bf16(x + alpha * gate * (post_norm(y) * w_post))
//   h     = bf16(pre_norm(x_out) * (1 + scale) + shift)
// and the per-row int8 quantizer of h. Bound by HBM: y and x are read once,
// x_out and h (or its codes) written once, 8 (7) bytes a channel. 18432 rows of 5120:
// 122 us, 6.2 TB/s, 0.95 of a copy (137 us when the power limit has lowered the clock);
// two CTAs of 256 threads per SM 128 (141) us, rows two passes ahead (135) us. With codes in
// place of h: 160 us, 4.1 TB/s.
//
// A row is held in registers by tpr threads, VPT 16-byte vectors each; a CTA
// holds several rows at a time and stages its next rows in shared memory with
// cp.async while it works on the current ones. Reductions: warp shuffles, then a
// slot per warp and a named barrier of the row's warps. Variances are taken
// about the mean, in a second pass over the registers. The row absmax is taken
// in fp32 before the bf16 rounding (rounding is monotone, so the rounded absmax
// is that of the rounded row).
#include <algorithm>

#include "h3b_common.cuh"
#include "h3b_internal.h"
#include "h3b_quant.cuh"

namespace h3b {
namespace {

constexpr int kMaxThreads = 512;

__device__ __forceinline__ void row_barrier(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void copy16(void* smem_dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem_dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void unpack8(uint4 u, float2* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = make_float2(bf16_lo(w[e]), bf16_hi(w[e]));
}

// kStaged: the item's vectors lie in shared memory, folded to alpha * gate * w_post, 1 + scale and shift, and
// the rows of a pass are of one item. Otherwise they are read from global memory (cache) row by row.
template <int VPT, bool kStaged>
__global__ void __launch_bounds__(kMaxThreads, 1) residual_norm_kernel(const ResNormArgs a, int tpr) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ uint4 smem_rows[];
  __shared__ float red[2][kMaxThreads / 32];
  const int vpr = a.d / 8;
  const int rpp = blockDim.x / tpr;  // rows per pass
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wpr = tpr >> 5, w0 = sub * wpr;
  const float inv_d = 1.0f / (float)a.d;
  uint4* stage_y = smem_rows + (size_t)(2 * sub) * vpr;
  uint4* stage_x = stage_y + vpr;
  float4* coef = reinterpret_cast<float4*>(smem_rows + (size_t)(2 * rpp) * vpr);  // [6][vpr]
  const bool want_h = a.h_out || a.q;

  int slot = 0;  // alternates, so that no barrier guards a slot's reuse
  auto row_sum = [&](float v) {
    v = warp_sum(v);
    if (wpr == 1) return v;
    if (lane == 0) red[slot][warp] = v;
    row_barrier(1 + sub, tpr);
    v = 0.0f;
    for (int w = 0; w < wpr; ++w) v += red[slot][w0 + w];
    slot ^= 1;
    return v;
  };
  auto row_max = [&](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (wpr == 1) return v;
    if (lane == 0) red[slot][warp] = v;
    row_barrier(1 + sub, tpr);
    v = 0.0f;
    for (int w = 0; w < wpr; ++w) v = max_nan(v, red[slot][w0 + w]);
    slot ^= 1;
    return v;
  };
  auto has = [&](int i) { return t + tpr * i < vpr; };
  // mean and variance of the row in f, applied in place
  auto norm = [&](float2(&f)[VPT * 4], int kind, float eps) {
    if (kind == 0) return;
    if (kind == 2) {
      float2 s = f[0];
#pragma unroll
      for (int e = 1; e < VPT * 4; ++e) s = __fadd2_rn(s, f[e]);
      const float mean = row_sum(s.x + s.y) * inv_d;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const float m = has(i) ? -mean : 0.0f;  // the vectors behind the row stay zero
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * i + e] = __fadd2_rn(f[4 * i + e], make_float2(m, m));
      }
    }
    float2 s = __fmul2_rn(f[0], f[0]);
#pragma unroll
    for (int e = 1; e < VPT * 4; ++e) s = __ffma2_rn(f[e], f[e], s);
    const float rstd = 1.0f / sqrtf(row_sum(s.x + s.y) * inv_d + eps);
#pragma unroll
    for (int e = 0; e < VPT * 4; ++e) f[e] = __fmul2_rn(f[e], make_float2(rstd, rstd));
  };
  auto prefetch = [&](bool on, int row) {
    if (on) {
      const uint4* y = static_cast<const uint4*>(a.y) + (size_t)row * vpr;
      const uint4* x = static_cast<const uint4*>(a.x) + (size_t)row * vpr;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int vec = t + tpr * i;
        if (vec < vpr && H3B_IDX_OK((long long)row * vpr + vec, (long long)a.rows * vpr, a.err)) {
          copy16(stage_y + vec, y + vec);
          copy16(stage_x + vec, x + vec);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // passes of rpp rows; staged: of one item each
  const int rpi = kStaged ? a.rows_per_item : a.rows;
  const unsigned per_item = ((unsigned)rpi + (unsigned)rpp - 1) / (unsigned)rpp;
  const unsigned items = ((unsigned)a.rows + (unsigned)rpi - 1) / (unsigned)rpi;  // rpi <= rows
  const unsigned passes = items * per_item;  // at most rows, so 32 bits suffice
  unsigned item = blockIdx.x / per_item, in = blockIdx.x % per_item;
  auto row_of = [&](unsigned it, unsigned p) { return (long long)it * rpi + (long long)p * rpp + sub; };
  auto row_on = [&](unsigned it, unsigned p) {
    return (long long)p * rpp + sub < rpi && row_of(it, p) < a.rows;
  };
  int cur = -1;
  prefetch(blockIdx.x < passes && row_on(item, in), (int)row_of(item, in));
  for (unsigned pass = blockIdx.x; pass < passes; pass += gridDim.x) {
    if (kStaged && (int)item != cur) {  // block-uniform
      __syncthreads();
      const size_t off = (size_t)item * a.mod_stride;
      for (int c = threadIdx.x; c < 2 * vpr; c += blockDim.x) {  // four channels each
        const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f), zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float4 w = a.w_post ? __ldg(reinterpret_cast<const float4*>(a.w_post) + c) : one;
        const float4 g = a.gate ? __ldg(reinterpret_cast<const float4*>(a.gate + off) + c) : one;
        const float4 sc = a.scale ? __ldg(reinterpret_cast<const float4*>(a.scale + off) + c) : zero;
        const float4 sh = a.shift ? __ldg(reinterpret_cast<const float4*>(a.shift + off) + c) : zero;
        const int k = c & 1, v = c >> 1;
        coef[k * vpr + v] = make_float4(a.alpha * g.x * w.x, a.alpha * g.y * w.y, a.alpha * g.z * w.z, a.alpha * g.w * w.w);
        coef[(2 + k) * vpr + v] = make_float4(1.0f + sc.x, 1.0f + sc.y, 1.0f + sc.z, 1.0f + sc.w);
        coef[(4 + k) * vpr + v] = sh;
      }
      cur = (int)item;
      __syncthreads();
    }
    const bool on = row_on(item, in);  // row-uniform
    const int row = (int)row_of(item, in);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float2 f[VPT * 4], x[VPT * 4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {  // each vector staged and read back by the same thread
      const bool v = on && has(i);
      unpack8(v ? stage_y[t + tpr * i] : make_uint4(0, 0, 0, 0), f + 4 * i);
      unpack8(v ? stage_x[t + tpr * i] : make_uint4(0, 0, 0, 0), x + 4 * i);
    }
    unsigned n_in = in + gridDim.x, n_item = item;
    while (n_in >= per_item) {
      n_in -= per_item;
      ++n_item;
    }
    prefetch(pass + gridDim.x < passes && row_on(n_item, n_in), (int)row_of(n_item, n_in));

    const size_t off = kStaged ? 0 : (size_t)(on ? row / a.rows_per_item : 0) * a.mod_stride;
    norm(f, a.post_norm, a.post_eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = t + tpr * i;
      if (!has(i)) continue;
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float4 c;
        if (kStaged) {
          c = coef[k * vpr + vec];
        } else {
          c = make_float4(a.alpha, a.alpha, a.alpha, a.alpha);
          if (a.gate) {
            const float4 g = __ldg(reinterpret_cast<const float4*>(a.gate + off) + 2 * vec + k);
            c = make_float4(c.x * g.x, c.y * g.y, c.z * g.z, c.w * g.w);
          }
          if (a.w_post) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(a.w_post) + 2 * vec + k);
            c = make_float4(c.x * w.x, c.y * w.y, c.z * w.z, c.w * w.w);
          }
        }
        const int e = 4 * i + 2 * k;
        const float2 p = __ffma2_rn(f[e], make_float2(c.x, c.y), x[e]);
        const float2 q = __ffma2_rn(f[e + 1], make_float2(c.z, c.w), x[e + 1]);
        u[2 * k] = pack_bf16x2(p.x, p.y);
        u[2 * k + 1] = pack_bf16x2(q.x, q.y);
      }
      const uint4 v = make_uint4(u[0], u[1], u[2], u[3]);
      unpack8(v, x + 4 * i);  // the stream as it is held
      if (on && H3B_IDX_OK((long long)row * vpr + vec, (long long)a.rows * vpr, a.err))
        static_cast<uint4*>(a.x_out)[(size_t)row * vpr + vec] = v;
    }
    if (on && a.absmax_zero && t == 0 && H3B_IDX_OK(row, a.rows, a.err)) a.absmax_zero[row] = 0.0f;
    if (want_h) {
      norm(x, a.pre_norm, a.pre_eps);
      float am = 0.0f;
      uint4 h[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int vec = t + tpr * i;
        h[i] = make_uint4(0, 0, 0, 0);
        if (!has(i)) continue;
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float4 sc, sh;
          if (kStaged) {
            sc = coef[(2 + k) * vpr + vec];
            sh = coef[(4 + k) * vpr + vec];
          } else {
            sc = sh = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (a.scale) sc = __ldg(reinterpret_cast<const float4*>(a.scale + off) + 2 * vec + k);
            if (a.shift) sh = __ldg(reinterpret_cast<const float4*>(a.shift + off) + 2 * vec + k);
            sc = make_float4(1.0f + sc.x, 1.0f + sc.y, 1.0f + sc.z, 1.0f + sc.w);
          }
          const int e = 4 * i + 2 * k;
          const float2 p = __ffma2_rn(x[e], make_float2(sc.x, sc.y), make_float2(sh.x, sh.y));
          const float2 q = __ffma2_rn(x[e + 1], make_float2(sc.z, sc.w), make_float2(sh.z, sh.w));
          am = max3_nan(max3_nan(am, fabsf(p.x), fabsf(p.y)), fabsf(q.x), fabsf(q.y));
          u[2 * k] = pack_bf16x2(p.x, p.y);
          u[2 * k + 1] = pack_bf16x2(q.x, q.y);
        }
        h[i] = make_uint4(u[0], u[1], u[2], u[3]);
        if (a.h_out && on && H3B_IDX_OK((long long)row * vpr + vec, (long long)a.rows * vpr, a.err))
          static_cast<uint4*>(a.h_out)[(size_t)row * vpr + vec] = h[i];
      }
      if (a.q) {
        const float amax = round_bf16(row_max(am));
        const float sc = __fdiv_rn(amax, 127.0f), rcp = __frcp_rn(sc);
        if (on && t == 0 && H3B_IDX_OK(row, a.rows, a.err)) a.s[row] = sc;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int vec = t + tpr * i;
          if (!on || !has(i) || !H3B_IDX_OK((long long)row * vpr + vec, (long long)a.rows * vpr, a.err)) continue;
          reinterpret_cast<uint2*>(a.q)[(size_t)row * vpr + vec] = quant8<true>(h[i], sc, rcp, amax);
        }
      }
    }
    item = n_item;
    in = n_in;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int VPT, bool kStaged>
cudaError_t launch(const ResNormArgs& a, int tpr, int rpp, int sms, cudaStream_t st) {
  const int vpr = a.d / 8;
  const size_t smem = (size_t)(2 * rpp + (kStaged ? 6 : 0)) * vpr * 16;
  auto k = residual_norm_kernel<VPT, kStaged>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long rpi = kStaged ? a.rows_per_item : a.rows;
  const long long passes = (a.rows + rpi - 1) / rpi * ((rpi + rpp - 1) / rpp);
  return launch_pdl(k, dim3((unsigned)std::min<long long>(passes, sms)), dim3(rpp * tpr), smem, st, a, tpr);
}

template <int VPT>
cudaError_t launch_vpt(const ResNormArgs& a, int tpr, int sms, cudaStream_t st) {
  // As many rows at a time as 512 threads hold. The item's vectors are worth staging (a barrier of the
  // whole block, 24 bytes a channel) as soon as a pass of rows shares them: at d = 5120, 2000 rows of one
  // item 22 us staged, 40 us read row by row; at 300 rows the same.
  const int rpp = std::max(1, kMaxThreads / tpr);
  const bool staged = a.rows_per_item >= 4 * rpp;
  return staged ? launch<VPT, true>(a, tpr, rpp, sms, st) : launch<VPT, false>(a, tpr, rpp, sms, st);
}

}  // namespace

cudaError_t launch_residual_norm(const ResNormArgs& args, int sms, cudaStream_t st) {
  ResNormArgs a = args;
  a.rows_per_item = std::min(a.rows_per_item, a.rows);  // the passes are counted by it
  // Vectors per thread, and as many warps as the row then needs. A warp's way through a row costs about as much
  // as three vectors besides its own, and the row's barriers the more the more warps it has. At 20000 rows of 3080
  // channels: 5 vectors, 3 warps 103 us; 1 vector, 13 warps, with fewer idle lanes, 257 us. At 8000 rows of 8192:
  // 4 vectors, 8 warps 94 us; 5 vectors, 7 warps 110 us.
  const int vpr = a.d / 8;
  int vpt = 0, tpr = 0;
  for (const int v : {5, 4, 2, 1}) {
    const int t = (vpr + 32 * v - 1) / (32 * v) * 32;
    if (t <= kMaxThreads && (vpt == 0 || t * (v + 3) <= tpr * (vpt + 3))) {
      vpt = v;
      tpr = t;
    }
  }
  switch (vpt) {
    case 5: return launch_vpt<5>(a, tpr, sms, st);
    case 4: return launch_vpt<4>(a, tpr, sms, st);
    case 2: return launch_vpt<2>(a, tpr, sms, st);
    default: return launch_vpt<1>(a, tpr, sms, st);
  }
}

}  // namespace h3b
