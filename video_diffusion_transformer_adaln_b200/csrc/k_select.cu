// Selection of the key blocks that each block of 128 queries attends:
//   score(i, j) = mean(valid rows of query block i) . mean(valid rows of key block j)
// and the topk best key blocks of each query block, ties to the lower index.
// The means and the scores are in 64 bits: a list is decided by comparisons, so
// two scores closer than their rounding errors would be listed by accident.
//
// Two kernels. The means read q and k once, 16 bytes a lane, and are bound by
// HBM. The scores are a product in 64 bits, [16 query blocks] x [all key blocks]
// per CTA, on the FP64 matrix instruction (16 x 8 x 16), whose key means come
// from L2; the topk of a row is found by a warp, by histograms over the scores
// mapped to unsigned integers.
//
// 18432 tokens, 40 heads of 128, 36 of 288 blocks: 105 us; the means 70 (5.6 TB/s, 0.85
// of a copy; conversions take 66% of their pipe), the scores 18 (the means of all keys of a
// head, 295 KB, from L2 for each CTA), the lists 17 (a warp's chain through a row). With means
// of 65 us, that added pairs in 32 bits: scores on the FP64 vector pipe, topk by bisection 143
// us; threads per CTA of 128 to 512 and two or three CTAs per SM 100 to 112 us, these 100.
#include "h3b_common.cuh"
#include "h3b_internal.h"

namespace h3b {
namespace {

__device__ __forceinline__ int clamp_len(const int* lens, int b, int L) {
  return lens ? min(max(__ldg(lens + b), 0), L) : L;
}

constexpr int kMeanThreads = 256;

// Where the means lie in the workspace: [row = batch item x head][block][lane], q before k.
struct Means {
  double *q, *k;
  long long nq, nk;  // elements
};

Means means_of(void* ws, int B, int n_heads, int n_kv_heads, int DH, int nqb, int nkb) {
  Means m;
  m.nq = (long long)B * n_heads * nqb * DH;
  m.nk = (long long)B * n_kv_heads * nkb * DH;
  m.q = static_cast<double*>(ws);
  m.k = m.q + m.nq;
  return m;
}

// A warp per block of rows: DH / 8 lanes per row, so 32 / (DH / 8) rows at a time, kBatch of them in
// flight while the batch before is added. Every value is converted before it is added: pairs added in 32 bits first
// would halve the conversions (100 us in place of 105 at the size above), but lose what is 2^16 below its partner, and
// with it the order of near scores and the ties of blocks that hold the same rows in another order.
constexpr int kBatch = 8;  // loads per lane and batch

template <int DH>
__device__ __forceinline__ void block_mean(const __nv_bfloat16* p, int n, int lane, double* out) {
  constexpr int LPR = DH / 8, RPI = 32 / LPR;
  const int sub = lane % LPR, r0 = lane / LPR;
  const uint4* src = reinterpret_cast<const uint4*>(p) + sub;
  double s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.0;
  auto fetch = [&](int base, uint4(&v)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = base + r0 + i * RPI;
      v[i] = r < n ? __ldg(src + (size_t)r * LPR) : make_uint4(0, 0, 0, 0);
    }
  };
  auto add = [&](const uint4(&v)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[2 * e] += (double)bf16_lo(x[e]);
        s[2 * e + 1] += (double)bf16_hi(x[e]);
      }
    }
  };
  constexpr int STEP = kBatch * RPI;
  uint4 va[kBatch], vb[kBatch];
  fetch(0, va);
#pragma unroll 1
  for (int r = 0; r < n; r += 2 * STEP) {  // warp-uniform
    fetch(r + STEP, vb);
    add(va);
    if (r + 2 * STEP < n) fetch(r + 2 * STEP, va);
    add(vb);
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += __shfl_xor_sync(0xFFFFFFFFu, s[e], o);
  if (lane < LPR && out) {
    double2* to = reinterpret_cast<double2*>(out + sub * 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e] = n > 0 ? make_double2(s[2 * e] / n, s[2 * e + 1] / n) : make_double2(0.0, 0.0);
  }
}

template <int DH>
__global__ void __launch_bounds__(kMeanThreads) block_means_kernel(const SelectArgs a, const Means m) {
  griddep_wait();
  griddep_launch_dependents();
  const int id = blockIdx.x * (kMeanThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int nq = a.B * a.n_heads * a.nqb, nk = a.B * a.n_kv_heads * a.nkb;
  if (id < nq) {
    const int row = id / a.nqb, blk = id - row * a.nqb;
    const int n = min(max(clamp_len(a.q_lens, row / a.n_heads, a.Lq) - blk * kSparseQueries, 0), kSparseQueries);
    const long long at = (long long)id * DH;
    block_mean<DH>(static_cast<const __nv_bfloat16*>(a.q) + ((size_t)row * a.Lq + (size_t)blk * kSparseQueries) * DH, n, lane,
                   H3B_IDX_OK(at + DH - 1, m.nq, a.err) ? m.q + at : nullptr);
  } else if (id - nq < nk) {
    const int row = (id - nq) / a.nkb, blk = id - nq - row * a.nkb;
    const int n = min(max(clamp_len(a.kv_lens, row / a.n_kv_heads, a.Lk) - blk * a.block_k, 0), a.block_k);
    const long long at = (long long)(id - nq) * DH;
    block_mean<DH>(static_cast<const __nv_bfloat16*>(a.k) + ((size_t)row * a.Lk + (size_t)blk * a.block_k) * DH, n, lane,
                   H3B_IDX_OK(at + DH - 1, m.nk, a.err) ? m.k + at : nullptr);
  }
}

// The order of the scores as unsigned integers: higher is better, -0 equals +0, NaN is last. Minus infinity has
// 0x000FFFFF in its upper half. No key's upper half is zero, so the histograms' ranges, which start at a key's upper
// half, start above zero: the threshold of a range taken from its start on can be lowered by one.
constexpr unsigned long long kKeyNan = 1ull << 32;
__device__ __forceinline__ unsigned long long order_key(double s) {
  if (s != s) return kKeyNan;
  const unsigned long long u = (unsigned long long)__double_as_longlong(s + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
constexpr unsigned long long kKeyKeep = ~0ull;

// D (16 x 8) += A (16 x 16) B (16 x 8) in 64 bits. Lane = 4 g + t holds A[g][.], A[g + 8][.] (a even, odd),
// B[.][g] and D[g][2t], D[g][2t + 1], D[g + 8][2t], D[g + 8][2t + 1], with the inner index of entry s of A and
// B at t + 4 s; any other order of the inner index that A and B share gives the same product.
__device__ __forceinline__ void mma_f64(double (&d)[4], const double (&a)[8], const double (&b)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f64.f64.f64.f64 {%0, %1, %2, %3}, {%4, %5, %6, %7, %8, %9, %10, %11}, "
      "{%12, %13, %14, %15}, {%0, %1, %2, %3};"
      : "+d"(d[0]), "+d"(d[1]), "+d"(d[2]), "+d"(d[3])
      : "d"(a[0]), "d"(a[1]), "d"(a[2]), "d"(a[3]), "d"(a[4]), "d"(a[5]), "d"(a[6]), "d"(a[7]), "d"(b[0]), "d"(b[1]),
        "d"(b[2]), "d"(b[3]));
}

constexpr int kSelectThreads = 256;

// A CTA per QR query blocks of one head (QR <= 16: the rest of the product's rows are zero).
template <int DH, int QR>
__global__ void __launch_bounds__(kSelectThreads, 2) select_kernel(const SelectArgs a, const Means m, int stride) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ double2 smem_select[];
  __shared__ __align__(16) unsigned hist[kSelectThreads / 32][256];
  constexpr int QS = DH + 2;  // padded row: 16-byte reads of neighbouring rows fall in distinct banks
  double* qs = reinterpret_cast<double*>(smem_select);  // [16][QS]
  double* score = qs + 16 * QS;                         // [QR][stride], then the scores' order in the same place
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(score);
  const int i0 = blockIdx.x * QR, row = blockIdx.y;
  const int b = row / a.n_heads, h = row - b * a.n_heads;
  const int kvrow = b * a.n_kv_heads + h / (a.n_heads / a.n_kv_heads);
  const int qn = clamp_len(a.q_lens, b, a.Lq), kn = clamp_len(a.kv_lens, b, a.Lk);
  const int cand = (kn + a.block_k - 1) / a.block_k;  // key blocks that hold a valid key
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 2 * threadIdx.x; x < 16 * DH; x += 2 * kSelectThreads) {
    const int i = x / DH, e = x - i * DH;
    const long long at = ((long long)row * a.nqb + i0 + i) * DH + e;
    const bool on = i < QR && i0 + i < a.nqb && H3B_IDX_OK(at + 1, m.nq, a.err);
    *reinterpret_cast<double2*>(qs + i * QS + e) = on ? __ldg(reinterpret_cast<const double2*>(m.q + at)) : make_double2(0.0, 0.0);
  }
  __syncthreads();
  const double* km = m.k + (size_t)kvrow * a.nkb * DH;
  const int g = lane >> 2, t = lane & 3;
  for (int j0 = 8 * warp; j0 < cand; j0 += kSelectThreads / 4) {  // eight keys of this warp
    // the lane's whole column, requested at once: inner index 16 k + 4 t + s
    double bk[DH / 16][4];
    const double* kj = km + (size_t)min(j0 + g, cand - 1) * DH + 4 * t;
#pragma unroll
    for (int k = 0; k < DH / 16; ++k) {
      const double2 u = __ldg(reinterpret_cast<const double2*>(kj + 16 * k));
      const double2 v = __ldg(reinterpret_cast<const double2*>(kj + 16 * k + 2));
      bk[k][0] = u.x; bk[k][1] = u.y; bk[k][2] = v.x; bk[k][3] = v.y;
    }
    double d[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int k = 0; k < DH / 16; ++k) {
      double ak[8];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int s = 0; s < 4; s += 2) {
          const double2 q2 = *reinterpret_cast<const double2*>(qs + (g + 8 * r) * QS + 16 * k + 4 * t + s);
          ak[2 * s + r] = q2.x;
          ak[2 * s + 2 + r] = q2.y;
        }
      mma_f64(d, ak, bk[k]);
    }
    if (g < QR) *reinterpret_cast<double2*>(score + g * stride + j0 + 2 * t) = make_double2(d[0], d[1]);
    if (g + 8 < QR) *reinterpret_cast<double2*>(score + (g + 8) * stride + j0 + 2 * t) = make_double2(d[2], d[3]);
  }
  __syncthreads();
  for (int i = warp; i < QR && i0 + i < a.nqb; i += kSelectThreads / 32) {
    const int n = (i0 + i) * kSparseQueries < qn ? cand : 0;
    const int want = min(n, a.topk);
    const long long list = (long long)row * a.nqb + i0 + i;
    int* out = a.blocks + list * a.topk;
    const int lo_kept = (i0 + i) * kSparseQueries / a.block_k - a.keep_local + 1;
    const int hi_kept = ((i0 + i) * kSparseQueries + kSparseQueries - 1) / a.block_k + a.keep_local - 1;
    auto key_of = [&](int j) {
      const bool keep = j < a.keep_first || (a.keep_local > 0 && j >= lo_kept && j <= hi_kept);
      return keep ? kKeyKeep : order_key(score[i * stride + j]);
    };
    const unsigned below = (1u << lane) - 1u;
    if (n <= 32) {  // a key per lane: its rank by comparison with all
      const unsigned long long mine = lane < n ? key_of(lane) : 0ull;  // every key is above zero
      int rank = 0;
#pragma unroll
      for (int o = 0; o < 32; ++o) {
        const unsigned long long other = __shfl_sync(0xFFFFFFFFu, mine, o);
        rank += other > mine || (other == mine && o < lane);
      }
      const bool take = lane < n && rank < want;
      const unsigned tk = __ballot_sync(0xFFFFFFFFu, take);
      if (take && H3B_IDX_OK(__popc(tk & below), want, a.err)) out[__popc(tk & below)] = lane;
    } else {
      // The threshold T: all keys above it, and the first `ties` of those equal to it, are listed. A
      // histogram of 256 bins over the keys' range finds the bin that the want-th key lies in, which is
      // the next range; done when the bin is taken whole. Kept blocks are counted apart: their key
      // is not a score, and would stretch the range.
      unsigned long long* key = keys + i * stride;
      unsigned top = 0u, bottom = ~0u;
      int kept = 0;
      for (int j = lane; j < n; j += 32) {
        const unsigned long long v = key_of(j);
        key[j] = v;
        if (v == kKeyKeep) {
          ++kept;
        } else {
          top = max(top, (unsigned)(v >> 32));
          bottom = min(bottom, (unsigned)(v >> 32));
        }
      }
      kept = __reduce_add_sync(0xFFFFFFFFu, kept);
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      bottom = __reduce_min_sync(0xFFFFFFFFu, bottom);
      unsigned long long T = kKeyKeep;
      int ties = n, need = want - kept;
      if (need > 0) {
        unsigned long long lo = (unsigned long long)bottom << 32;
        // the range is a power of two above (top - bottom + 1) 2^32, 256 bins of 2^sh
        int sh = max(0, 64 - __clzll((long long)(((unsigned long long)(top - bottom) << 32) | 0xFFFFFFFFull)) - 8);
        unsigned long long range = 256;  // bins that the range has; fewer once a bin is less than 256 keys wide
        unsigned* bins = hist[warp];
        for (;;) {
          for (int x = lane; x < 64; x += 32) reinterpret_cast<uint4*>(bins)[x] = make_uint4(0, 0, 0, 0);
          __syncwarp();
          for (int j = lane; j < n; j += 32) {
            const unsigned long long v = key[j], d = v - lo;
            if (v != kKeyKeep && v >= lo && (d >> sh) < range) atomicAdd(bins + (unsigned)(d >> sh), 1u);
          }
          __syncwarp();
          // this lane's eight bins, and the keys in bins above them
          const uint4 p = reinterpret_cast<const uint4*>(bins)[2 * lane], q = reinterpret_cast<const uint4*>(bins)[2 * lane + 1];
          const unsigned c[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
          unsigned sum = 0;
#pragma unroll
          for (int x = 0; x < 8; ++x) sum += c[x];
          unsigned upto = sum;  // of this lane and those above
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_down_sync(0xFFFFFFFFu, upto, o);
            if (lane + o < 32) upto += u;
          }
          unsigned over = upto - sum;  // in the bins above the one found
          int bin = 0;
          unsigned in = 0;
          const bool here = over < (unsigned)need && (unsigned)need <= upto;  // one lane
          if (here) {
            bool found = false;
#pragma unroll
            for (int x = 7; x >= 0; --x) {
              if (!found && over + c[x] >= (unsigned)need) {
                found = true;
                bin = 8 * lane + x;
                in = c[x];
              }
              if (!found) over += c[x];
            }
          }
          const int src = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
          bin = __shfl_sync(0xFFFFFFFFu, bin, src);
          in = __shfl_sync(0xFFFFFFFFu, in, src);
          need -= (int)__shfl_sync(0xFFFFFFFFu, over, src);
          T = lo + ((unsigned long long)bin << sh);
          if ((int)in == need) break;  // the whole bin: every key >= T
          if (sh == 0) {               // equal keys, more than needed
            ties = need;
            break;
          }
          lo = T;
          range = 1ull << min(sh, 8);
          sh = max(0, sh - 8);
        }
        if (ties == n) T -= 1;  // keys >= T, as keys above T - 1 (T >= lo > 0)
      }
      int at = 0, seen = 0;  // listed, and equal to T, so far
      for (int j0 = 0; j0 < n && at < want; j0 += 32) {
        const int j = j0 + lane;
        const unsigned long long mine = j < n ? key[j] : 0ull;
        const bool equal = ties < n && j < n && mine == T;
        const unsigned eq = __ballot_sync(0xFFFFFFFFu, equal);
        const bool take = j < n && (mine > T || mine == kKeyKeep || (equal && seen + __popc(eq & below) < ties));
        const unsigned tk = __ballot_sync(0xFFFFFFFFu, take);
        const int to = at + __popc(tk & below);
        if (take && H3B_IDX_OK(to, want, a.err)) out[to] = j;
        at += __popc(tk);
        seen += __popc(eq);
      }
    }
    for (int x = want + lane; x < a.topk; x += 32) out[x] = -1;
    if (lane == 0) a.counts[list] = want;
  }
}

template <int DH, int QR>
cudaError_t launch_select(const SelectArgs& a, const Means& m, cudaStream_t st) {
  const int stride = (a.nkb + 7) & ~7;
  const size_t smem = sizeof(double) * (16 * (size_t)(DH + 2) + (size_t)QR * stride);
  auto k = select_kernel<DH, QR>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3((a.nqb + QR - 1) / QR, a.B * a.n_heads), dim3(kSelectThreads), smem, st, a, m, stride);
}

template <int DH>
cudaError_t launch(const SelectArgs& a, cudaStream_t st) {
  const Means m = means_of(a.ws, a.B, a.n_heads, a.n_kv_heads, DH, a.nqb, a.nkb);
  const long long blocks = (long long)a.B * a.n_heads * a.nqb + (long long)a.B * a.n_kv_heads * a.nkb;
  const dim3 grid((unsigned)((blocks + kMeanThreads / 32 - 1) / (kMeanThreads / 32)));
  const cudaError_t e = launch_pdl(block_means_kernel<DH>, grid, dim3(kMeanThreads), 0, st, a, m);
  if (e != cudaSuccess) return e;
  // rows of scores that fit the shared memory
  if (a.nkb <= 1536) return launch_select<DH, 16>(a, m, st);
  return launch_select<DH, 4>(a, m, st);
}

}  // namespace

size_t select_ws_bytes(int B, int n_heads, int n_kv_heads, int head_dim, int nqb, int nkb) {
  const Means m = means_of(nullptr, B, n_heads, n_kv_heads, head_dim, nqb, nkb);
  return sizeof(double) * (size_t)(m.nq + m.nk);
}

cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t st) {
  return a.head_dim == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace h3b
