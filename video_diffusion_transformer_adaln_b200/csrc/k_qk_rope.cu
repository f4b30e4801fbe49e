// Per-head RMSNorm of Q and K and rotary positions on three axes given per
// token, from a token-major projection to the head-major layout:
//   y = x * rsqrt(mean(x^2) + eps) * w            (over the head's lanes)
//   (y[2p], y[2p+1]) turned by pos[axis(p)] * theta^(-2j/r)
// Bound by HBM: every element is read and written once, 4 bytes of traffic.
//
// The change of layout is TMA's: the projection is viewed as [item][head][token]
// [lane], a box of it is 16 KB of shared memory of 4 heads by 16 (32) tokens of
// head_dim 128 (64), the rows are normalised and turned in place, and each head's
// rows, which lie side by side in the box and in the head-major output, are
// stored by one bulk copy, cut where the tokens or the part's heads end.
//   warp 8      loads the boxes of the CTA's range into a ring of slots
//   warps 0-7   a warp takes 2 (4) tokens of a box, eight lanes of the head in each
//               thread; a thread's four (cos, sin) pairs depend on its token and
//               lanes alone, and stay in registers for all boxes of the tokens
//   warp 9      stores finished boxes and frees their slots
// The boxes, ordered by tokens, then by heads, are dealt out evenly to as many
// CTAs as are resident.
//
// 18432 tokens, 40 heads of 128: 200 us, 5.66 TB/s, 0.86 of a copy (207 us where only a part
// of the lanes is turned). Rows loaded to and stored from registers, with the next ones on
// their way: 218 us. A box stored by one tensor copy instead of a bulk copy per head: 198 us,
// for three more tensor maps that cost the host as much as a small call takes.
#include <algorithm>
#include <type_traits>

#include "h3b_common.cuh"
#include "h3b_internal.h"

namespace h3b {
namespace {

constexpr int kWarps = 8;                    // that compute
constexpr int kThreads = 32 * (kWarps + 2);
constexpr int kHeads = 4;                    // heads per box
constexpr int kSlots = 6;
constexpr int kBoxBytes = 16384;
constexpr size_t kSmem = (size_t)kSlots * kBoxBytes + 3 * kSlots * 8 + 16 + 128;
constexpr int kCtasPerSm = 2;                // by registers and shared memory

// (cos, sin) of pair p at this token. The angle in half turns is reduced to
// [-1, 1] in 64 bits before it is rounded to 32, so its error is that of a
// value below pi for any position.
__device__ __forceinline__ float2 pair_turn(const QkRopeArgs& a, const float* pos, int p) {
  const int ax = p < a.axis_end[0] ? 0 : p < a.axis_end[1] ? 1 : 2;
  const double t = (double)__ldg(pos + ax) * a.freq[p];
  float s, c;
  sincospif((float)(t - 2.0 * rint(0.5 * t)), &s, &c);
  return make_float2(c, s);
}

// d = a b + c, both halves, where `on`; else d stays. One instruction under a predicate, where two results and a select
// take three.
__device__ __forceinline__ void fma2_if(bool on, float2& d, float2 a, float2 b, float2 c) {
  asm("{\n\t.reg .pred p;\n\t.reg .b64 d, a, b, c;\n\t"
      "setp.ne.s32 p, %8, 0;\n\t"
      "mov.b64 d, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "@p fma.rn.f32x2 d, a, b, c;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d.x), "+f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "r"((int)on));
}

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int token, int head, int item) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(token), "r"(head), "r"(item)
      : "memory");
}
// `bytes` (a multiple of 16) of shared memory to global memory, in this thread's bulk group.
__device__ __forceinline__ void store_bytes(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// Boxes per token tile: those of Q, of K, of V.
struct Boxes {
  int q, k, all;        // q: of Q; k: of Q and K
  int tiles_per_item;   // token tiles
  long long total;
};

template <int DH>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ CUtensorMap tm_in,
                                                                const __grid_constant__ QkRopeArgs a, const Boxes n) {
  constexpr int LPR = DH / 8, TPW = 32 / LPR;  // lanes per head row, tokens per warp and head
  constexpr int TT = kWarps * TPW;             // tokens per box
  static_assert(TT * kHeads * DH * 2 == kBoxBytes, "a box fills its slot");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const uint32_t sb = smem_u32(smem);
  auto full = [&](int s) { return sb + kSlots * kBoxBytes + 8u * s; };
  auto done = [&](int s) { return full(kSlots + s); };
  auto empty = [&](int s) { return full(2 * kSlots + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSlots * kBoxBytes + 3 * kSlots * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(full(s), 1);
      mbar_init(done(s), kWarps);
      mbar_init(empty(s), 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_in);
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  const long long first = n.total * blockIdx.x / gridDim.x, last = n.total * (blockIdx.x + 1) / gridDim.x;
  const int H = a.n_heads, KV = a.n_kv_heads;
  // box i of the range: its token tile's item and first token, its box within the tile
  long long tile = first / n.all;
  int box = (int)(first - tile * n.all);
  int item = (int)(tile / n.tiles_per_item), token = (int)(tile - (long long)item * n.tiles_per_item) * TT;
  auto next_box = [&]() {
    if (++box < n.all) return;
    box = 0;
    token += TT;
    if (token >= n.tiles_per_item * TT) {
      token = 0;
      ++item;
    }
  };
  int slot = 0;
  uint32_t ph = 0;
  auto next_slot = [&]() {
    if (++slot == kSlots) {
      slot = 0;
      ph ^= 1u;
    }
  };
  if (warp == kWarps) {
    if (lane == 0) {
      uint32_t filled = 0, phases = 0;
      bool ok = true;
      for (long long i = first; i < last; ++i) {
        if (!mbar_wait_or_abort(empty(slot), ph ^ 1u, abort_flag, a.err, ERR_WAIT_EPI)) { ok = false; break; }
        mbar_arrive_expect_tx(full(slot), kBoxBytes);
        const int head = box < n.q ? box * kHeads : box < n.k ? H + (box - n.q) * kHeads : H + KV + (box - n.k) * kHeads;
        load_box(sb + slot * kBoxBytes, &tm_in, full(slot), token, head, item);
        filled |= 1u << slot;
        phases = (phases & ~(1u << slot)) | (ph << slot);
        next_slot();
        next_box();
      }
      if (!ok) {  // nothing may land after the CTA has ended
        *abort_flag = 1;
        for (int s = 0; s < kSlots; ++s)
          if (filled & (1u << s)) mbar_wait(full(s), (phases >> s) & 1u, a.err, ERR_WAIT_DRAIN, kDrainLimitNs);
      }
    }
  } else if (warp == kWarps + 1) {
    if (lane == 0) {
      int before = -1;  // slot whose store has been started but may not have been read yet
      for (long long i = first; i < last; ++i) {
        if (!mbar_wait_or_abort(done(slot), ph, abort_flag, a.err, ERR_WAIT_EPI)) {
          *abort_flag = 1;
          break;
        }
        // a head's tokens lie side by side in shared and in global memory
        const int head = (box < n.q ? box : box < n.k ? box - n.q : box - n.k) * kHeads;
        const int heads = box < n.q ? H : KV;
        char* to = static_cast<char*>(box < n.q ? a.q : box < n.k ? a.k : a.v);
        const uint32_t bytes = (uint32_t)min(TT, a.L - token) * DH * 2;
        for (int h = 0; h < kHeads && head + h < heads; ++h) {
          const long long at = (((long long)item * heads + head + h) * a.L + token) * DH;
          if (H3B_IDX_OK(at + bytes / 2 - 1, (long long)a.B * heads * a.L * DH, a.err))
            store_bytes(to + at * 2, sb + slot * kBoxBytes + h * (TT * DH * 2), bytes);
        }
        bulk_commit_group();
        if (before >= 0) {
          asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          mbar_arrive(empty(before));
        }
        before = slot;
        next_slot();
        next_box();
      }
      bulk_wait_group0();
    }
  } else {
    const int sub = lane % LPR;
    const int mine = warp * TPW + lane / LPR;  // token of the box
    float2 turn[4], w[4];
    int turn_token = -1, turn_item = -1, w_part = -1;
    // this thread's pairs that an axis turns; the others pass as they are (a turn by zero would make infinity * 0 of an
    // infinite partner, and lose the sign of zeros)
    const int turned = a.pos ? min(max(a.axis_end[2] - 4 * sub, 0), 4) : 0;
    const bool whole_heads = a.pos && 2 * a.axis_end[2] == DH;
    const uint32_t at = (uint32_t)(warp * 512 + lane * 16);
    for (long long i = first; i < last; ++i) {
      const int part = box < n.q ? 0 : box < n.k ? 1 : 2;
      if (part < 2) {  // before the wait: overlaps the load
        if (token != turn_token || item != turn_item) {
          turn_token = token;
          turn_item = item;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            turn[e] = make_float2(1.0f, 0.0f);
            if (token + mine < a.L && e < turned)
              turn[e] = pair_turn(a, a.pos + ((size_t)item * a.L + token + mine) * 3, 4 * sub + e);
          }
        }
        const float* weights = part == 0 ? a.wq : a.wk;
        if (part != w_part && weights) {
          const float4 w0 = __ldg(reinterpret_cast<const float4*>(weights + sub * 8));
          const float4 w1 = __ldg(reinterpret_cast<const float4*>(weights + sub * 8) + 1);
          w[0] = make_float2(w0.x, w0.y); w[1] = make_float2(w0.z, w0.w);
          w[2] = make_float2(w1.x, w1.y); w[3] = make_float2(w1.z, w1.w);
        }
        w_part = part;
      }
      const bool got = mbar_wait_or_abort(full(slot), ph, abort_flag, a.err, ERR_WAIT_TMA);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        *abort_flag = 1;
        break;
      }
      if (part < 2) {
        const bool normed = (part == 0 ? a.wq : a.wk) != nullptr;
        uint4* rows = reinterpret_cast<uint4*>(smem + slot * kBoxBytes + at);
        constexpr int STEP = TT * DH * 2 / 16;  // vectors from one head of the box to the next
        uint4 u[kHeads];
        float rstd[kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) u[h] = rows[h * STEP];
        if (normed) {
          // the sums of squares of all heads first: their shuffles overlap
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            const uint32_t in[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
            float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = make_float2(bf16_lo(in[e]), bf16_hi(in[e]));
              s = __ffma2_rn(f, f, s);
            }
            rstd[h] = s.x + s.y;
          }
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
            for (int h = 0; h < kHeads; ++h) rstd[h] += __shfl_xor_sync(0xFFFFFFFFu, rstd[h], o);
          // rsqrtf is within 2 units in the last place of 32 bits, far below the output's rounding; a
          // root and a division, with their paths for special values, take as long as all the rest
#pragma unroll
          for (int h = 0; h < kHeads; ++h) rstd[h] = rsqrtf(fmaf(rstd[h], 1.0f / DH, a.eps));
        }
        auto turn_heads = [&](auto whole) {
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            const uint32_t in[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
            uint32_t out[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float2 f = make_float2(bf16_lo(in[e]), bf16_hi(in[e]));
              if (normed) f = __fmul2_rn(__fmul2_rn(f, make_float2(rstd[h], rstd[h])), w[e]);
              // (x c - y s, x s + y c)
              const float2 t = __fmul2_rn(make_float2(f.y, f.y), make_float2(-turn[e].y, turn[e].x));
              float2 z = f;
              if (whole.value) z = __ffma2_rn(make_float2(f.x, f.x), turn[e], t);
              else fma2_if(e < turned, z, make_float2(f.x, f.x), turn[e], t);
              out[e] = pack_bf16x2(z.x, z.y);
            }
            rows[h * STEP] = make_uint4(out[0], out[1], out[2], out[3]);
          }
        };
        // Heads whose every lane is turned take a path of their own. 18432 tokens, 40 heads of 128: 199 us there, 207 with
        // half of the lanes turned (209 with selects in place of the predicate).
        if (whole_heads)
          turn_heads(std::true_type{});
        else
          turn_heads(std::false_type{});
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(done(slot));
      next_slot();
      next_box();
    }
  }
}

template <int DH>
cudaError_t launch(const QkRopeArgs& a, int sms, cudaStream_t st) {
  constexpr int TT = kWarps * 256 / DH;
  const uint64_t H = a.n_heads, KV = a.n_kv_heads, L = a.L, B = a.B;
  const uint32_t box[4] = {DH, TT, kHeads, 1};
  const uint64_t dims[4] = {DH, L, H + 2 * KV, B};
  const uint64_t strides[3] = {(uint64_t)a.row_stride * 2, DH * 2, L * (uint64_t)a.row_stride * 2};
  CUtensorMap in;
  if (!make_tmap_4d_bf16(&in, a.qkv, dims, strides, box)) return cudaErrorInvalidValue;
  Boxes n;
  n.q = (a.n_heads + kHeads - 1) / kHeads;
  n.k = n.q + (a.n_kv_heads + kHeads - 1) / kHeads;
  n.all = n.k + (a.n_kv_heads + kHeads - 1) / kHeads;
  n.tiles_per_item = (a.L + TT - 1) / TT;
  n.total = (long long)n.all * n.tiles_per_item * a.B;
  auto kernel = qk_norm_rope_kernel<DH>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min<long long>(n.total, (long long)kCtasPerSm * sms);
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), kSmem, st, in, a, n);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkRopeArgs& a, int sms, cudaStream_t st) {
  return a.head_dim == 128 ? launch<128>(a, sms, st) : launch<64>(a, sms, st);
}

}  // namespace h3b
