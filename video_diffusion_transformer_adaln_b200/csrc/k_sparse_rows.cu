// Softmax attention of one query per head (a new token) over its listed key
// blocks:
//   o = sum_j softmax_j(q.K[j] / sqrt(head_dim)) V[j],  j in the listed blocks
// A tensor core tile would hold one row of 128. What bounds this is reading the
// listed rows of K and V, so they stream through shared memory and the products
// run on the FP32 pipe, two lanes of the head at a time, with fp32 probabilities.
//
// The units of 64 listed keys of all rows (batch item x head), one row after the
// other, are dealt out evenly to one CTA per processor:
//   warp 8      copies the valid rows of a unit, which lie side by side in K and in V,
//               by two bulk copies into a ring of slots, and notes what they are;
//               after the last unit of a row comes a note without rows
//   warps 0-7   eight keys of each unit per warp, four lanes to a key, each with a
//               quarter of the query and of an output of its own, so that a score needs
//               two shuffles and nothing is exchanged between keys; a key's lanes keep
//               their own running maximum and sum. At the end of a row all of these are
//               joined and written to the workspace.
// A second kernel joins the parts of a row that several CTAs have worked on.
//
// 4 streams, 40 heads of 128 over 8 key heads, 72 of 288 blocks of 64: 51 us for 377 MB of
// gathered rows, 7.4 TB/s of HBM and L2 (the whole cache once from HBM: 46 us). Rows loaded
// straight to registers 106 us; consumers in two groups of four warps 55 us.
#include <algorithm>

#include "h3b_common.cuh"
#include "h3b_internal.h"
#include "h3b_softmax.cuh"

namespace h3b {
namespace {

constexpr int kWarps = 8, kThreads = 32 * (kWarps + 1);
constexpr int kUnit = 64;           // keys per unit, 8 per warp
constexpr int kCtas = 148;          // whatever the device has: the workspace's size must not depend on it
constexpr float kNoMax = -3.0e38f;  // running maximum before any key

__device__ __forceinline__ int clamp_len(const int* lens, int b, int L) {
  return lens ? min(max(__ldg(lens + b), 0), L) : L;
}
__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// How the units are dealt out: CTA c of `ctas` works on units [total c / ctas, total (c + 1) / ctas).
struct Deal {
  int ctas, units, most;  // units: per row; most: rows that a CTA can touch
  long long total;
  __host__ __device__ long long first(int c) const { return total * c / ctas; }
};
Deal deal_of(long long rows, int topk, int block_k) {
  Deal d;
  d.units = topk * (block_k / kUnit);
  d.total = rows * d.units;
  d.ctas = (int)std::max<long long>(1, std::min<long long>(kCtas, d.total / 2));
  const long long share = (d.total + d.ctas - 1) / d.ctas;
  d.most = (int)((share + d.units - 2) / d.units + 1);
  return d;
}

template <int DH>
struct Layout {
  static constexpr int HALF = kUnit * DH * 2;  // K or V of a unit
  static constexpr int NS = DH == 128 ? 6 : 12;
  static constexpr int PART_OFF = NS * 2 * HALF;                          // [2][kWarps][DH + 2]
  static constexpr int BAR_OFF = PART_OFF + 2 * kWarps * (DH + 2) * 4;    // full, empty per slot; a row's parts
  static constexpr int NOTE_OFF = BAR_OFF + (2 * NS + 1) * 8;             // [NS]: row, valid keys
  static constexpr int FLAG_OFF = NOTE_OFF + NS * 8;
  static constexpr size_t SMEM = FLAG_OFF + 16 + 128;
};
static_assert(Layout<128>::SMEM <= 232448 && Layout<64>::SMEM <= 232448, "shared memory of one CTA");

// A part: o[DH], maximum (in exponents of 2), sum.
template <int DH>
__global__ void __launch_bounds__(kThreads, 1) sparse_rows_kernel(const SparseAttnArgs a, const Deal d, float scale_log2,
                                                                  float* parts) {
  using Lay = Layout<DH>;
  constexpr int NS = Lay::NS, NV = DH / 32;  // NV: 16-byte pieces of a row per lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const uint32_t sb = smem_u32(smem);
  auto full = [&](int s) { return sb + Lay::BAR_OFF + 8u * s; };
  auto empty = [&](int s) { return sb + Lay::BAR_OFF + 8u * (NS + s); };
  const uint32_t joined = sb + Lay::BAR_OFF + 8u * 2 * NS;
  volatile int2* notes = reinterpret_cast<volatile int2*>(smem + Lay::NOTE_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::FLAG_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kWarps);
    }
    mbar_init(joined, kWarps);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  const long long f0 = d.first(blockIdx.x), f1 = d.first(blockIdx.x + 1);
  const int row0 = (int)(f0 / d.units), row1 = (int)((f1 - 1) / d.units);  // f1 > f0
  const int per = a.block_k / kUnit;
  int slot = 0;
  uint32_t ph = 0;
  auto next_slot = [&]() {
    if (++slot == NS) {
      slot = 0;
      ph ^= 1u;
    }
  };
  if (warp == kWarps) {
    // ---------------- producer (whole warp; lane 0 copies)
    uint32_t filled = 0, phases = 0;
    bool ok = true;
    // A slot with `nv` rows from `first` on (none: the end of the row).
    auto put = [&](int row, int kvrow, int first, int nv) -> bool {
      const bool free_ = mbar_wait_or_abort(empty(slot), ph ^ 1u, abort_flag, a.err, ERR_WAIT_EPI);
      if (!__all_sync(0xFFFFFFFFu, free_)) return false;
      filled |= 1u << slot;
      phases = (phases & ~(1u << slot)) | (ph << slot);
      if (lane == 0) {
        notes[slot].x = row;
        notes[slot].y = nv;
        if (nv > 0) {
          const uint32_t bytes = (uint32_t)nv * DH * 2, dst = sb + slot * 2 * Lay::HALF;
          const long long at = ((long long)kvrow * a.Lk + first) * DH;
          mbar_arrive_expect_tx(full(slot), 2 * bytes);
          copy_bytes(dst, static_cast<const __nv_bfloat16*>(a.k) + at, bytes, full(slot));
          copy_bytes(dst + Lay::HALF, static_cast<const __nv_bfloat16*>(a.v) + at, bytes, full(slot));
        } else {
          mbar_arrive(full(slot));
        }
      }
      __syncwarp();
      next_slot();
      return true;
    };
    for (int row = row0; row <= row1 && ok; ++row) {
      const int b = row / a.n_heads, h = row - b * a.n_heads;
      const int kvrow = b * a.n_kv_heads + h / (a.n_heads / a.n_kv_heads);
      const int kn = clamp_len(a.kv_lens, b, a.Lk);
      const int entries = a.counts ? min(max(__ldg(a.counts + row), 0), a.topk) : a.topk;
      const int all = clamp_len(a.q_lens, b, 1) > 0 ? entries * per : 0;
      const long long start = (long long)row * d.units;
      const int u0 = (int)max(f0 - start, 0LL), u1 = (int)min((long long)all, f1 - start);
      const int* list = a.blocks + (size_t)row * a.topk;
      for (int base = u0; base < u1 && ok; base += 32) {  // 32 units at a time, one per lane
        const int u = base + lane;
        const int blk = u < u1 ? __ldg(list + u / per) : -1;
        int first = 0, nv = 0;
        if ((unsigned)blk < (unsigned)a.nkb) {
          first = blk * a.block_k + u % per * kUnit;
          nv = min(kUnit, kn - first);
        }
        for (int i = 0; i < 32 && ok; ++i) {
          const int n = __shfl_sync(0xFFFFFFFFu, nv, i), from = __shfl_sync(0xFFFFFFFFu, first, i);
          if (n > 0) ok = put(row, kvrow, from, n);
        }
      }
      if (ok) ok = put(row, kvrow, 0, 0);
    }
    if (!ok) {  // nothing may land after the CTA has ended
      *abort_flag = 1;
      for (int s = 0; s < NS; ++s)
        if (filled & (1u << s)) mbar_wait(full(s), (phases >> s) & 1u, a.err, ERR_WAIT_DRAIN, kDrainLimitNs);
    }
    return;
  }
  // ---------------- consumers
  const int quarter = lane & 3, group = lane >> 2;
  // piece i of this lane: lanes of the head [8 p, 8 p + 8), p = 4 (i ^ odd) + quarter. The keys of two
  // neighbouring groups lie 128 or 256 bytes apart; with the order of the pieces swapped in every
  // other one they are read from distinct banks.
  const int odd = group & 1;
  auto unpack = [](uint4 u, float2* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = make_float2(bf16_lo(w[e]), bf16_hi(w[e]));
  };
  float2 q2[NV * 4], o2[NV * 4];
  float m = kNoMax, l = 0.0f;
  auto begin = [&](int row) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (size_t)row * DH);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack(__ldg(src + 4 * (i ^ odd) + quarter), q2 + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q2[4 * i + e] = __fmul2_rn(q2[4 * i + e], make_float2(scale_log2, scale_log2));
        o2[4 * i + e] = make_float2(0.0f, 0.0f);
      }
    }
    m = kNoMax;
    l = 0.0f;
  };
  int row = row0, parity = 0;
  begin(row);
  while (row <= row1) {
    const bool got = mbar_wait_or_abort(full(slot), ph, abort_flag, a.err, ERR_WAIT_TMA);
    if (!__all_sync(0xFFFFFFFFu, got)) {
      *abort_flag = 1;
      return;
    }
    const int nv = notes[slot].y;
    if (nv > 0) {
      const int key = 8 * warp + group;
      const uint4* ks = reinterpret_cast<const uint4*>(smem + slot * 2 * Lay::HALF) + key * (DH / 8) + quarter;
      const uint4* vs = ks + Lay::HALF / 16;
      float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      uint4 raw[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) raw[i] = ks[4 * (i ^ odd)];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float2 f[4];
        unpack(raw[i], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e & 1] = __ffma2_rn(q2[4 * i + e], f[e], acc[e & 1]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) raw[i] = vs[4 * (i ^ odd)];
      const float2 sum = __fadd2_rn(acc[0], acc[1]);
      float s = sum.x + sum.y;
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
      if (key < nv) {  // the rows behind the valid ones are an older unit's
        if (!(s <= m + 8.0f)) {  // also NaN; the first key, and maxima that grow by more than 2^8
          const float alpha = fast_exp2(m - s);
          m = s;
          l *= alpha;
#pragma unroll
          for (int e = 0; e < NV * 4; ++e) o2[e] = __fmul2_rn(o2[e], make_float2(alpha, alpha));
        }
        const float p = fast_exp2(s - m);
        l += p;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float2 f[4];
          unpack(raw[i], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) o2[4 * i + e] = __ffma2_rn(make_float2(p, p), f[e], o2[4 * i + e]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(slot));
      next_slot();
      continue;
    }
    // the end of the row: join the warp's eight keys, then the warps
    __syncwarp();
    if (lane == 0) mbar_arrive(empty(slot));
    next_slot();
    float M = m;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) M = max_nan(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    const float w = fast_exp2(m - M);
    l *= w;
#pragma unroll
    for (int e = 0; e < NV * 4; ++e) o2[e] = __fmul2_rn(o2[e], make_float2(w, w));
    // groups of one parity hold the same pieces in the same order; the other parity's are brought into it
#pragma unroll
    for (int i = 0; i < NV; i += 2)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = o2[4 * i + e], y = o2[4 * i + 4 + e];
        o2[4 * i + e] = odd ? y : x;
        o2[4 * i + 4 + e] = odd ? x : y;
      }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
#pragma unroll
      for (int e = 0; e < NV * 4; ++e) {
        o2[e].x += __shfl_xor_sync(0xFFFFFFFFu, o2[e].x, o);
        o2[e].y += __shfl_xor_sync(0xFFFFFFFFu, o2[e].y, o);
      }
    }
    float* mine = reinterpret_cast<float*>(smem + Lay::PART_OFF) + (parity * kWarps + warp) * (DH + 2);
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(mine + (4 * i + quarter) * 8 + 2 * e) = o2[4 * i + e];
      if (quarter == 0) {
        mine[DH] = M;
        mine[DH + 1] = l;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(joined);
    const bool there = mbar_wait_or_abort(joined, parity, abort_flag, a.err, ERR_WAIT_EPI);
    if (!__all_sync(0xFFFFFFFFu, there)) {
      *abort_flag = 1;
      return;
    }
    if (threadIdx.x < DH + 2) {
      const float* all = reinterpret_cast<const float*>(smem + Lay::PART_OFF) + parity * kWarps * (DH + 2);
      float top = kNoMax, v = 0.0f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) top = max_nan(top, all[x * (DH + 2) + DH]);
      const int at = threadIdx.x < DH ? threadIdx.x : DH + 1;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) v = fmaf(fast_exp2(all[x * (DH + 2) + DH] - top), all[x * (DH + 2) + at], v);
      if (threadIdx.x == DH) v = top;
      const long long to = ((long long)blockIdx.x * d.most + row - row0) * (DH + 2) + threadIdx.x;
      if (H3B_IDX_OK(to, (long long)d.ctas * d.most * (DH + 2), a.err)) parts[to] = v;
    }
    parity ^= 1;  // the next row's parts go elsewhere; every warp waits for those, so the place is free after that
    if (++row <= row1) begin(row);
  }
}

// o = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c over the CTAs that have worked on a row. A warp per row.
template <int DH>
__global__ void __launch_bounds__(128) sparse_rows_join_kernel(const SparseAttnArgs a, const Deal d, const float* parts) {
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= a.B * a.n_heads) return;
  const int b = row / a.n_heads;
  if (clamp_len(a.q_lens, b, 1) < 1) return;
  // the CTA that a unit belongs to: first(c) <= unit < first(c + 1)
  auto cta_of = [&](long long unit) {
    int c = (int)(unit * d.ctas / d.total);
    while (d.first(c + 1) <= unit) ++c;
    while (d.first(c) > unit) --c;
    return c;
  };
  const int c0 = cta_of((long long)row * d.units), c1 = cta_of((long long)(row + 1) * d.units - 1);
  constexpr int V = DH / 32;
  float M = kNoMax, L = 0.0f, o[V] = {};
  for (int base = c0; base <= c1; base += 32) {  // a part per lane: its place, maximum and sum
    const int c = base + lane;
    long long at = 0;
    float pm = kNoMax, pl = 0.0f;
    if (c <= c1) {
      at = ((long long)c * d.most + row - d.first(c) / d.units) * (DH + 2);
      pm = parts[at + DH];
      pl = parts[at + DH + 1];
    }
    float top = max_nan(M, pm);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    const float before = fast_exp2(M - top), w = fast_exp2(pm - top);
    M = top;
    float sum = w * pl;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
    L = fmaf(L, before, sum);
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] *= before;
    const int n = min(32, c1 - base + 1);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float* p = parts + __shfl_sync(0xFFFFFFFFu, at, i);
      const float f = __shfl_sync(0xFFFFFFFFu, w, i);
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(f, p[lane * V + e], o[e]);
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  float amax = 0.0f;
  uint32_t pk[V / 2];
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    pk[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
    amax = max3_nan(amax, fabsf(bf16_lo(pk[e])), fabsf(bf16_hi(pk[e])));
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, x));
  const long long at = (long long)row * DH + lane * V;
  if (H3B_IDX_OK(at + V - 1, (long long)a.B * a.n_heads * DH, a.err)) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.o) + at);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) dst[e] = pk[e];
  }
  if (a.absmax && lane == 0) atomicMax(reinterpret_cast<unsigned*>(a.absmax) + b, __float_as_uint(amax));
}

template <int DH>
cudaError_t launch(const SparseAttnArgs& a, cudaStream_t st) {
  const int rows = a.B * a.n_heads;
  const Deal d = deal_of(rows, a.topk, a.block_k);
  auto k = sparse_rows_kernel<DH>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<DH>::SMEM);
  if (e != cudaSuccess) return e;
  float* parts = static_cast<float*>(a.ws);
  e = launch_pdl(k, dim3(d.ctas), dim3(kThreads), Layout<DH>::SMEM, st, a, d, 1.4426950408889634f / sqrtf((float)DH), parts);
  if (e != cudaSuccess) return e;
  return launch_pdl(sparse_rows_join_kernel<DH>, dim3((rows + 3) / 4), dim3(128), 0, st, a, d, (const float*)parts);
}

}  // namespace

size_t sparse_rows_ws_bytes(long long rows, int head_dim, int topk, int block_k) {
  const Deal d = deal_of(rows, topk, block_k);
  return sizeof(float) * (size_t)d.ctas * d.most * (head_dim + 2);
}

cudaError_t launch_sparse_rows(const SparseAttnArgs& a, cudaStream_t st) {
  return a.head_dim == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace h3b
