// Selection of the key blocks that each block of 128 queries attends:
//   score(i, j) = mean(valid rows of query block i) . mean(valid rows of key block j)
// and the topk best key blocks of each query block, ties to the lower index.
// The means and the scores are in 64 bits: a list is decided by comparisons, so
// two scores closer than their rounding errors would be listed by accident.
//
// Two kernels. The means read q and k once, 16 bytes a lane, and are bound by
// HBM. The scores are a product in 64 bits, [16 query blocks] x [all key blocks]
// per CTA, on the FP64 pipe (64 a cycle and SM), whose key means come from L2
// transposed, two keys a thread; the topk of a row is found by a warp, by
// bisection over the bits of the scores mapped to unsigned integers.
#include "h3b_common.cuh"
#include "h3b_internal.h"

namespace h3b {
namespace {

__device__ __forceinline__ int clamp_len(const int* lens, int b, int L) {
  return lens ? min(max(__ldg(lens + b), 0), L) : L;
}

constexpr int kMeanThreads = 256;

// Where the means lie in the workspace: q [row][query block][lane]; k transposed, [row][lane][key block],
// rows of an even number of key blocks.
struct Means {
  double *q, *k;
  long long nq, nk;  // elements
  int nkb_even;
};

Means means_of(void* ws, int B, int n_heads, int n_kv_heads, int DH, int nqb, int nkb) {
  Means m;
  m.nkb_even = (nkb + 1) & ~1;
  m.nq = (long long)B * n_heads * nqb * DH;
  m.nk = (long long)B * n_kv_heads * m.nkb_even * DH;
  m.q = static_cast<double*>(ws);
  m.k = m.q + m.nq;
  return m;
}

// A warp per block of rows: DH / 8 lanes per row, so 32 / (DH / 8) rows at a time, kBatch of them in
// flight while the batch before is added. Rows are added in pairs in 32 bits (two bf16 values of like size
// add exactly) and the pairs in 64, which halves the conversions and additions on the FP64 pipe.
constexpr int kBatch = 8;  // loads per lane and batch

template <int DH>
__device__ __forceinline__ void block_mean(const __nv_bfloat16* p, int n, int lane, double* out, long long out_stride) {
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
    for (int i = 0; i < kBatch; i += 2) {
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      const uint32_t y[4] = {v[i + 1].x, v[i + 1].y, v[i + 1].z, v[i + 1].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[2 * e] += (double)(bf16_lo(x[e]) + bf16_lo(y[e]));
        s[2 * e + 1] += (double)(bf16_hi(x[e]) + bf16_hi(y[e]));
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
#pragma unroll
    for (int e = 0; e < 8; ++e) out[(sub * 8 + e) * out_stride] = n > 0 ? s[e] / n : 0.0;
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
                   H3B_IDX_OK(at + DH - 1, m.nq, a.err) ? m.q + at : nullptr, 1);
  } else if (id - nq < nk) {
    const int row = (id - nq) / a.nkb, blk = id - nq - row * a.nkb;
    const int n = min(max(clamp_len(a.kv_lens, row / a.n_kv_heads, a.Lk) - blk * a.block_k, 0), a.block_k);
    const long long at = (long long)row * DH * m.nkb_even + blk;
    block_mean<DH>(static_cast<const __nv_bfloat16*>(a.k) + ((size_t)row * a.Lk + (size_t)blk * a.block_k) * DH, n, lane,
                   H3B_IDX_OK(at + (long long)(DH - 1) * m.nkb_even, m.nk, a.err) ? m.k + at : nullptr, m.nkb_even);
  }
}

// The order of the scores as unsigned integers: higher is better, -0 equals +0, NaN is last.
__device__ __forceinline__ unsigned long long order_key(double s) {
  if (s != s) return 1ull;
  const unsigned long long u = (unsigned long long)__double_as_longlong(s + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
constexpr unsigned long long kKeyKeep = ~0ull;

// A CTA per QR query blocks of one head. Its warps cover `tiles` times 64 keys; with few keys, `parts`
// warps share a tile's sums over the lanes of the head, and their parts are added in order.
template <int DH, int QR>
__global__ void __launch_bounds__(256, 2) select_kernel(const SelectArgs a, const Means m, int tiles, int parts) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ double2 smem_select[];
  double* qs = reinterpret_cast<double*>(smem_select);  // [DH][QR]
  double* score = qs + DH * QR;                         // [QR][nkb_even], then the scores' order in the same place
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(score);
  const int i0 = blockIdx.x * QR, row = blockIdx.y;
  const int b = row / a.n_heads, h = row - b * a.n_heads;
  const int kvrow = b * a.n_kv_heads + h / (a.n_heads / a.n_kv_heads);
  const int qn = clamp_len(a.q_lens, b, a.Lq), kn = clamp_len(a.kv_lens, b, a.Lk);
  const int cand = (kn + a.block_k - 1) / a.block_k;  // key blocks that hold a valid key
  const int nke = m.nkb_even;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 8
  for (int x = threadIdx.x; x < DH * QR; x += blockDim.x) {
    const int i = x / DH, e = x - i * DH;
    const long long at = ((long long)row * a.nqb + i0 + i) * DH + e;
    qs[e * QR + i] = i0 + i < a.nqb && H3B_IDX_OK(at, m.nq, a.err) ? __ldg(m.q + at) : 0.0;
  }
  __syncthreads();
  const int part = warp / tiles, len = DH / parts, e_first = part * len;
  const double* km = m.k + (size_t)kvrow * DH * nke + (size_t)e_first * nke;
  constexpr int EB = 4;  // lanes of the head per batch; len is a multiple of 2 EB
  for (int base = 0; base < cand; base += 64 * tiles) {
    const int j = base + 64 * (warp - part * tiles) + 2 * lane;  // keys j, j + 1 of this thread
    const bool mine = j < cand;
    double s0[QR], s1[QR];
#pragma unroll
    for (int i = 0; i < QR; ++i) s0[i] = s1[i] = 0.0;
    const double* kj = km + (mine ? j : 0);
    auto fetch = [&](int e0, double2(&kk)[EB]) {
#pragma unroll
      for (int e = 0; e < EB; ++e) kk[e] = __ldg(reinterpret_cast<const double2*>(kj + (size_t)(e0 + e) * nke));
    };
    auto add = [&](int e0, const double2(&kk)[EB]) {
#pragma unroll
      for (int e = 0; e < EB; ++e)
#pragma unroll
        for (int i = 0; i < QR; i += 2) {
          const double2 q2 = *reinterpret_cast<const double2*>(qs + (e_first + e0 + e) * QR + i);
          s0[i] = fma(q2.x, kk[e].x, s0[i]);
          s1[i] = fma(q2.x, kk[e].y, s1[i]);
          s0[i + 1] = fma(q2.y, kk[e].x, s0[i + 1]);
          s1[i + 1] = fma(q2.y, kk[e].y, s1[i + 1]);
        }
    };
    double2 ka[EB], kb[EB];
    fetch(0, ka);
#pragma unroll 1
    for (int e0 = 0; e0 < len; e0 += 2 * EB) {
      fetch(e0 + EB, kb);
      add(e0, ka);
      if (e0 + 2 * EB < len) fetch(e0 + 2 * EB, ka);
      add(e0 + EB, kb);
    }
    for (int r = 0; r < parts; ++r) {
      if (part == r && mine) {
#pragma unroll
        for (int i = 0; i < QR; ++i) {
          double2* to = reinterpret_cast<double2*>(score + i * nke + j);
          double2 v = make_double2(s0[i], s1[i]);
          if (r > 0) {
            const double2 w = *to;
            v = make_double2(w.x + v.x, w.y + v.y);
          }
          *to = v;
        }
      }
      if (parts > 1) __syncthreads();
    }
  }
  __syncthreads();
  for (int i = warp; i < QR && i0 + i < a.nqb; i += blockDim.x >> 5) {
    const int n = (i0 + i) * kSparseQueries < qn ? cand : 0;
    const int want = min(n, a.topk);
    unsigned long long* key = keys + i * nke;
    // the scores' order, and what bits all of it share
    const int lo = (i0 + i) * kSparseQueries / a.block_k - a.keep_local + 1;
    const int hi = ((i0 + i) * kSparseQueries + kSparseQueries - 1) / a.block_k + a.keep_local - 1;
    unsigned long long all_or = 0ull, all_and = ~0ull;
    for (int j = lane; j < n; j += 32) {
      const bool keep = j < a.keep_first || (a.keep_local > 0 && j >= lo && j <= hi);
      const unsigned long long v = keep ? kKeyKeep : order_key(score[i * nke + j]);
      key[j] = v;
      all_or |= v;
      all_and &= v;
    }
    __syncwarp();
    const unsigned long long differ = ((unsigned long long)__reduce_or_sync(0xFFFFFFFFu, (unsigned)((all_or ^ all_and) >> 32)) << 32) |
                                      __reduce_or_sync(0xFFFFFFFFu, (unsigned)(all_or ^ all_and));
    // every lane's own keys may agree among themselves and differ from another lane's
    const unsigned long long any = ((unsigned long long)__reduce_or_sync(0xFFFFFFFFu, (unsigned)(all_or >> 32)) << 32) |
                                   __reduce_or_sync(0xFFFFFFFFu, (unsigned)all_or);
    const unsigned long long every = ((unsigned long long)__reduce_and_sync(0xFFFFFFFFu, (unsigned)(all_and >> 32)) << 32) |
                                     __reduce_and_sync(0xFFFFFFFFu, (unsigned)all_and);
    const unsigned long long mixed = differ | (any ^ every);  // bits in which two keys differ
    const int top = 63 - __clzll((long long)mixed);           // the highest of them, -1: none
    // the largest T with at least `want` keys >= T, bit by bit; done early when exactly `want` are
    unsigned long long T = top < 0 ? any : top == 63 ? 0ull : any & ~((2ull << top) - 1ull);
    int above = n;  // keys >= T
    for (int bit = top; bit >= 0 && above > want; --bit) {
      const unsigned long long c = T | (1ull << bit);
      int cnt = 0;
      for (int j = lane; j < n; j += 32) cnt += key[j] >= c;
      cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
      if (cnt >= want) {
        T = c;
        above = cnt;
      }
    }
    // above > want: the keys equal to T are more than needed; the lowest of them are listed
    int ties = above;
    if (above > want) {
      int more = 0;
      for (int j = lane; j < n; j += 32) more += key[j] > T;
      ties = want - __reduce_add_sync(0xFFFFFFFFu, more);
    }
    const long long list = (long long)row * a.nqb + i0 + i;
    int* out = a.blocks + list * a.topk;
    int at = 0, seen = 0;  // listed, and equal to T, so far
    for (int j0 = 0; j0 < n && at < want; j0 += 32) {
      const int j = j0 + lane;
      const unsigned long long mine = j < n ? key[j] : 0ull;
      const bool equal = j < n && mine == T;
      const unsigned below = (1u << lane) - 1u;
      const unsigned eq = __ballot_sync(0xFFFFFFFFu, equal);
      const bool take = j < n && (mine > T || (equal && seen + __popc(eq & below) < ties));
      const unsigned tk = __ballot_sync(0xFFFFFFFFu, take);
      const int to = at + __popc(tk & below);
      if (take && H3B_IDX_OK(to, want, a.err)) out[to] = j;
      at += __popc(tk);
      seen += __popc(eq);
    }
    for (int t = want + lane; t < a.topk; t += 32) out[t] = -1;
    if (lane == 0) a.counts[list] = want;
  }
}

template <int DH, int QR>
cudaError_t launch_select(const SelectArgs& a, const Means& m, cudaStream_t st) {
  const size_t smem = sizeof(double) * ((size_t)DH * QR + (size_t)QR * m.nkb_even);
  auto k = select_kernel<DH, QR>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int tiles = min((m.nkb_even + 63) / 64, 8);
  const int parts = tiles == 1 ? 8 : tiles == 2 ? 4 : tiles <= 4 ? 2 : 1;
  return launch_pdl(k, dim3((a.nqb + QR - 1) / QR, a.B * a.n_heads), dim3(32 * tiles * parts), smem, st, a, m, tiles, parts);
}

template <int DH>
cudaError_t launch(const SelectArgs& a, int sms, cudaStream_t st) {
  const Means m = means_of(a.ws, a.B, a.n_heads, a.n_kv_heads, DH, a.nqb, a.nkb);
  const long long blocks = (long long)a.B * a.n_heads * a.nqb + (long long)a.B * a.n_kv_heads * a.nkb;
  const dim3 grid((unsigned)((blocks + kMeanThreads / 32 - 1) / (kMeanThreads / 32)));
  const cudaError_t e = launch_pdl(block_means_kernel<DH>, grid, dim3(kMeanThreads), 0, st, a, m);
  if (e != cudaSuccess) return e;
  // 16 query blocks a CTA read each key mean once for 16 products; fewer where that leaves
  // processors without work, or where 16 rows of scores do not fit the shared memory
  const long long ctas16 = (long long)a.B * a.n_heads * ((a.nqb + 15) / 16);
  if (ctas16 >= sms && m.nkb_even <= 1280) return launch_select<DH, 16>(a, m, st);
  return launch_select<DH, 4>(a, m, st);
}

}  // namespace

size_t select_ws_bytes(int B, int n_heads, int n_kv_heads, int head_dim, int nqb, int nkb) {
  const Means m = means_of(nullptr, B, n_heads, n_kv_heads, head_dim, nqb, nkb);
  return sizeof(double) * (size_t)(m.nq + m.nk);
}

cudaError_t launch_select_blocks(const SelectArgs& a, int sms, cudaStream_t st) {
  return a.head_dim == 128 ? launch<128>(a, sms, st) : launch<64>(a, sms, st);
}

}  // namespace h3b
