// Softmax attention of blocks of 128 queries over listed blocks of keys, on
// sm_100a tensor cores (bf16 operands, fp32 accumulation):
//   O[i] = sum_j softmax_j(Q[i].K[j] / sqrt(head_dim)) V[j],  j in the listed blocks
// in one pass over each list with the running maximum and sum of the softmax.
//
// An item is a query block of one head with a range of its list, 128 listed keys
// (a tile: two units of 64, gathered by their own TMA loads) at a time. One CTA
// works on two items, each with its own list, so that one item's products fill
// the tensor core while the other's softmax runs:
//   warp 0     TMA: Q of both items, then the K and V tiles of both lists in the
//              order the MMAs use them, into one ring of slots
//   warp 1     tcgen05.mma from one thread, in the order
//                S0(0) S1(0) | PV0(0) S0(1) PV1(0) S1(1) | PV0(1) S0(2) ...
//              where an item whose list has ended drops out
//   warps 2-3  idle (they complete warpgroup 0 for the register split)
//   warps 4-7  softmax of item 0, warps 8-11 softmax of item 1 (thread = row)
// A warp without a valid query row does no softmax (one new token uses one of
// four). Tensor memory (512 columns): S0 | S1 | O0 | O1; P_g overwrites the first
// half of S_g. When S_g(j) is complete, PV_g(j-1) is too (a commit tracks every
// earlier MMA of its thread), so O_g can be rescaled without another barrier; it
// is rescaled only when a row's maximum grew by more than 2^8. P is rounded to
// bf16, the type of V, for the tensor core; the row sum adds the unrounded fp32
// exponentials.
//
// Units without a valid key (entries outside the key blocks, blocks behind
// kv_len) are loaded from behind the tensor, where TMA fills zeros. In the one
// unit that kv_len cuts, the V rows behind it are zeroed in shared memory, so
// that nothing they hold (NaN, infinities) meets a zero probability.
//
// With few query blocks a list is split over several items, whose unnormalised
// outputs, maxima and sums go to the workspace and are joined by a second kernel.
#include <algorithm>

#include "h3b_common.cuh"
#include "h3b_internal.h"
#include "h3b_softmax.cuh"

namespace h3b {
namespace {

constexpr int kThreads = 384;
constexpr int kUnit = 64;  // keys per TMA box
constexpr int kTile = 128; // keys per MMA tile
// registers per thread after the split (launch: 384 x 168 = 64512 = 128 x 56 + 256 x 224)
constexpr uint32_t kRegsControl = 56, kRegsSoftmax = 224;
constexpr uint32_t kTmemCols = 512;
constexpr int kUnitBox = kUnit * 128;  // bytes of 64 rows x 64 lanes
constexpr int kBox = kTile * 128;      // bytes of 128 rows x 64 lanes
constexpr float kNoMax = -3.0e38f;     // running maximum before any key

struct SparseParams {
  SparseAttnArgs a;
  int nsplit, split_tiles, rows;  // items = rows * nsplit, item = row * nsplit + split
  float scale_log2;
  float* part_o;   // [item][128][DH], nsplit > 1
  float2* part_ml; // [item][128]: maximum (in exponents of 2), sum
};

template <int DH>
struct Layout {
  static constexpr int NBOX = DH / 64;
  static constexpr int TILE = kTile * DH * 2;  // bytes of a slot, and of one item's Q
  static constexpr int NS = DH == 128 ? 5 : 10;
  static constexpr int Q_OFF = 0, RING_OFF = 2 * TILE;
  static constexpr int BAR_OFF = RING_OFF + NS * TILE;
  static constexpr int NBARS = 2 + 2 * NS + 6 + 1;
  static constexpr size_t SMEM = (size_t)BAR_OFF + NBARS * 8 + 16 + 1024;
  static constexpr uint32_t S_COL(int g) { return g * 128u; }
  static constexpr uint32_t O_COL(int g) { return 256u + g * DH; }
};
static_assert(Layout<128>::SMEM <= 232448 && Layout<64>::SMEM <= 232448, "shared memory of one CTA");
static_assert(Layout<64>::SMEM > 116 * 1024, "one CTA per SM: each holds all tensor memory columns");

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ int clamp_len(const int* lens, int b, int L) {
  return lens ? min(max(__ldg(lens + b), 0), L) : L;
}

// What an item works on; the same in every thread.
struct Item {
  int bh, qb;      // batch item x head, query block
  int kvrow;       // batch item x key head
  int qn, kn;      // valid queries and keys of the batch item
  int t0, units;   // first tile of the range, units in it
  int tiles;       // ceil(units / 2)
  const int* list;
  int entries;     // list entries in use
  bool rows;       // holds valid query rows
};

__device__ __forceinline__ Item load_item(const SparseParams& p, int item) {
  const SparseAttnArgs& a = p.a;
  Item it{};
  if (item >= p.rows * p.nsplit) return it;
  const int row = item / p.nsplit, split = item - row * p.nsplit;
  it.bh = row / a.nqb;
  it.qb = row - it.bh * a.nqb;
  const int b = it.bh / a.n_heads, h = it.bh - b * a.n_heads;
  it.kvrow = b * a.n_kv_heads + h / (a.n_heads / a.n_kv_heads);
  it.qn = clamp_len(a.q_lens, b, a.Lq);
  it.kn = clamp_len(a.kv_lens, b, a.Lk);
  it.rows = it.qb * kSparseQueries < it.qn;
  it.list = a.blocks + (size_t)row * a.topk;
  it.entries = a.counts ? min(max(__ldg(a.counts + row), 0), a.topk) : a.topk;
  const int all = it.rows && it.kn > 0 ? it.entries * (a.block_k / kUnit) : 0;
  it.t0 = split * p.split_tiles;
  it.units = min(max(all - 2 * it.t0, 0), 2 * p.split_tiles);
  it.tiles = (it.units + 1) / 2;
  return it;
}

// Walks an item's list in tiles; a warp's lanes hold 32 entries, with the next 32 on their way.
struct ListWalk {
  int cur, nxt, base;  // this lane's entry of the chunk that starts at entry `base`, and of the next
  __device__ __forceinline__ static int fetch(const Item& it, int e) {
    return e < it.entries ? __ldg(it.list + e) : -1;
  }
  __device__ __forceinline__ void start(const Item& it, int per_tile, int lane) {
    base = it.t0 * per_tile & ~31;
    cur = fetch(it, base + lane);
    nxt = fetch(it, base + 32 + lane);
  }
  // First keys of the two units of tile t (from the item's first): `none` where a unit holds no valid key.
  __device__ __forceinline__ int2 tile(const Item& it, int t, int block_k, int nkb, int none, int lane) {
    const bool wide = block_k == kTile;
    const int e0 = wide ? it.t0 + t : 2 * (it.t0 + t);
    if (e0 - base >= 32) {
      base += 32;
      cur = nxt;
      nxt = fetch(it, base + 32 + lane);
    }
    const int a = __shfl_sync(0xFFFFFFFFu, cur, e0 - base);
    const int b = wide ? a : __shfl_sync(0xFFFFFFFFu, cur, e0 - base + 1);
    int2 s;
    s.x = (unsigned)a < (unsigned)nkb ? a * block_k : none;
    s.y = (unsigned)b < (unsigned)nkb ? b * block_k + (wide ? kUnit : 0) : none;
    if (s.x >= it.kn) s.x = none;
    if (s.y >= it.kn || 2 * t + 1 >= it.units) s.y = none;
    return s;
  }
};

template <int DH, int kPolyMod>
__global__ void __launch_bounds__(kThreads, 1)
    sparse_attention_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                            const __grid_constant__ CUtensorMap tmv, const SparseParams p) {
  using Lay = Layout<DH>;
  constexpr int NS = Lay::NS;
  const SparseAttnArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb0 = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
  const uint32_t bar0 = smem_u32(bars);
  auto q_full = [&](int g) { return bar0 + 8u * g; };
  auto full = [&](int s) { return bar0 + 8u * (2 + s); };
  auto empty = [&](int s) { return bar0 + 8u * (2 + NS + s); };
  auto s_full = [&](int g) { return bar0 + 8u * (2 + 2 * NS + g); };
  auto p_full = [&](int g) { return bar0 + 8u * (4 + 2 * NS + g); };
  auto fin = [&](int g) { return bar0 + 8u * (6 + 2 * NS + g); };
  const uint32_t drain = bar0 + 8u * (8 + 2 * NS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Lay::NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t IDESC_S = instr_desc(1, 1, 0, 0, kSparseQueries, kTile);
  constexpr uint32_t IDESC_S_HALF = instr_desc(1, 1, 0, 0, kSparseQueries, kUnit);
  constexpr uint32_t IDESC_PV = instr_desc(1, 1, 0, 1, kSparseQueries, DH);

  if (threadIdx.x == 0) {
    for (int g = 0; g < 2; ++g) {
      mbar_init(q_full(g), 1); mbar_init(s_full(g), 1); mbar_init(p_full(g), 4); mbar_init(fin(g), 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // q, k, v and the lists may be the previous grid's output
  griddep_launch_dependents();

  const int none = a.nkb * a.block_k;  // >= Lk: rows there read as zeros
  const int per_tile = kTile / a.block_k;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      // ---------------- TMA producer (whole warp; lane 0 issues)
      const Item it[2] = {load_item(p, 2 * blockIdx.x), load_item(p, 2 * blockIdx.x + 1)};
      ListWalk walk[2];
      int2 at[2];  // the units of the K tile loaded last, for its V tile
      bool ok = true;
      int slot = 0, used = 0;  // used: loads issued
      uint32_t ph = 0;
      auto load = [&](const CUtensorMap* tm, int g, int t) -> bool {
        if (used >= NS) {  // the warp decides as one: its lanes may see the abort flag at different times
          const bool free_ = mbar_wait_or_abort(empty(slot), ph ^ 1u, abort_flag, a.err, ERR_WAIT_MMA);
          if (!__all_sync(0xFFFFFFFFu, free_)) return false;
        }
        if (lane == 0) {
          const int nu = min(2, it[g].units - 2 * t);
          const uint32_t dst = sb0 + Lay::RING_OFF + slot * Lay::TILE;
          mbar_arrive_expect_tx(full(slot), nu * Lay::NBOX * kUnitBox);
          for (int u = 0; u < nu; ++u)
            for (int b = 0; b < Lay::NBOX; ++b)
              tma_load_3d(dst + b * kBox + u * kUnitBox, tm, full(slot), b * 64, u ? at[g].y : at[g].x, it[g].kvrow);
        }
        ++used;
        if (++slot == NS) {
          slot = 0;
          ph ^= 1u;
        }
        return true;
      };
      auto load_k = [&](int g, int t) -> bool {
        at[g] = walk[g].tile(it[g], t, a.block_k, a.nkb, none, lane);
        return load(&tmk, g, t);
      };
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        walk[g].start(it[g], per_tile, lane);
        if (it[g].tiles > 0) {
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full(g), Lay::TILE);
            for (int b = 0; b < Lay::NBOX; ++b)
              tma_load_3d(sb0 + Lay::Q_OFF + g * Lay::TILE + b * kBox, &tmq, q_full(g), b * 64,
                          it[g].qb * kSparseQueries, it[g].bh);
          }
          ok = ok && load_k(g, 0);
        }
      }
      const int n = max(it[0].tiles, it[1].tiles);
      for (int t = 0; t < n && ok; ++t) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (ok && t < it[g].tiles) ok = load(&tmv, g, t);
          if (ok && t + 1 < it[g].tiles) ok = load_k(g, t + 1);
        }
      }
      // the loads still in flight land before the CTA may end; on the regular path every slot in
      // use has also been consumed
      if (!ok) *abort_flag = 1;
      const int live = min(used, NS);
      for (int k = 0; k < live; ++k) {
        if (--slot < 0) {
          slot = NS - 1;
          ph ^= 1u;
        }
        if (ok) mbar_wait(empty(slot), ph, a.err, ERR_WAIT_MMA);
        else mbar_wait(full(slot), ph, a.err, ERR_WAIT_DRAIN, kDrainLimitNs);
      }
      if (!ok)
        for (int g = 0; g < 2; ++g)
          if (it[g].tiles > 0) mbar_wait(q_full(g), 0, a.err, ERR_WAIT_DRAIN, kDrainLimitNs);
    } else if (warp == 1 && lane == 0) {
      // ---------------- MMA issuer
      int units[2], tiles[2];
      for (int g = 0; g < 2; ++g) {
        const Item it = load_item(p, 2 * blockIdx.x + g);
        units[g] = it.units;
        tiles[g] = it.tiles;
      }
      bool any = false;
      int slot = 0;
      uint32_t ph = 0;
      auto take = [&]() -> bool { return mbar_wait_or_abort(full(slot), ph, abort_flag, a.err, ERR_WAIT_TMA); };
      auto give = [&]() {
        tc_commit(empty(slot));
        if (++slot == NS) {
          slot = 0;
          ph ^= 1u;
        }
      };
      auto issue_s = [&](int g, int t) -> bool {  // S_g(t) = Q_g K_t^T
        if (!take()) return false;
        tc_fence_after();
        const uint32_t q_addr = sb0 + Lay::Q_OFF + g * Lay::TILE;
        const uint32_t k_addr = sb0 + Lay::RING_OFF + slot * Lay::TILE;
        const uint32_t idesc = units[g] - 2 * t > 1 ? IDESC_S : IDESC_S_HALF;
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          const uint64_t ad = smem_desc_sw128(q_addr + (k >> 2) * kBox + (k & 3) * 32, 16, 1024);
          const uint64_t bd = smem_desc_sw128(k_addr + (k >> 2) * kBox + (k & 3) * 32, 16, 1024);
          mma_f16(tmem + Lay::S_COL(g), ad, bd, idesc, k > 0 ? 1u : 0u);
        }
        any = true;
        tc_commit(s_full(g));
        give();
        return true;
      };
      auto issue_pv = [&](int g, int t) -> bool {  // O_g += P_g(t) V_t
        if (!mbar_wait_or_abort(p_full(g), t & 1, abort_flag, a.err, ERR_WAIT_EPI)) return false;
        if (!take()) return false;
        tc_fence_after();
        const uint32_t v_addr = sb0 + Lay::RING_OFF + slot * Lay::TILE;
        const int steps = units[g] - 2 * t > 1 ? kTile / 16 : kUnit / 16;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k) {
          if (k >= steps) break;
          const uint64_t bd = smem_desc_sw128(v_addr + k * 2048, kBox, 1024);
          mma_f16_ts(tmem + Lay::O_COL(g), tmem + Lay::S_COL(g) + k * 8, bd, IDESC_PV, (t > 0 || k > 0) ? 1u : 0u);
        }
        any = true;
        give();
        return true;
      };
      bool ok = true;
      for (int g = 0; g < 2 && ok; ++g)
        if (tiles[g] > 0) ok = mbar_wait_or_abort(q_full(g), 0, abort_flag, a.err, ERR_WAIT_TMA) && issue_s(g, 0);
      const int n = max(tiles[0], tiles[1]);
      for (int t = 0; t < n && ok; ++t)
        for (int g = 0; g < 2 && ok; ++g) {
          if (t >= tiles[g]) continue;
          ok = issue_pv(g, t);
          if (!ok) break;
          if (t + 1 < tiles[g]) ok = issue_s(g, t + 1);
          else tc_commit(fin(g));
        }
      if (!ok) {
        *abort_flag = 1;
        if (any) {
          tc_commit(drain);
          mbar_wait(drain, 0, a.err, ERR_WAIT_DRAIN, kDrainLimitNs);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---------------- softmax warps: 4-7 -> item 0, 8-11 -> item 1 (thread = query row)
    const int g = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
    const uint32_t s_col = tmem + t_lane + Lay::S_COL(g), o_col = tmem + t_lane + Lay::O_COL(g);
    const int item = 2 * blockIdx.x + g;
    const Item it = load_item(p, item);
    const int other = load_item(p, 2 * blockIdx.x + (g ^ 1)).tiles;
    const int q = it.qb * kSparseQueries + row;
    const bool live = it.qb * kSparseQueries + quad * 32 < it.qn;  // warp-uniform: a valid row in this warp
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    ListWalk walk;
    walk.start(it, per_tile, lane);
    float m_run = kNoMax, l_run = 0.0f;
    bool ok = true;
    for (int t = 0; t < it.tiles; ++t) {
      const int2 at = walk.tile(it, t, a.block_k, a.nkb, none, lane);
      const int nv0 = at.x == none ? 0 : min(kUnit, it.kn - at.x);
      const int nv1 = at.y == none ? 0 : min(kUnit, it.kn - at.y);
      const bool s_ok = mbar_wait_or_abort(s_full(g), t & 1, abort_flag, a.err, ERR_WAIT_MMA);
      if (!__all_sync(0xFFFFFFFFu, s_ok)) { ok = false; break; }
      // V rows behind kv_len (in memory, so TMA does not zero them) are zeroed once V_t has landed. S_g(t) is
      // complete, so every load up to K_g(t) has been used, among them the one that held V_g(t)'s
      // slot before (at least five loads earlier): the parity cannot be of an older phase
      const bool cut0 = nv0 > 0 && nv0 < kUnit && it.kn < a.Lk, cut1 = nv1 > 0 && nv1 < kUnit && it.kn < a.Lk;
      if (cut0 || cut1) {
        // place of V_g(t) in the order of loads: the first K tiles, the loads of the rounds
        // before t, and item 0's loads of this round
        const int n0 = g ? other : it.tiles, n1 = g ? it.tiles : other;
        int pos = (n0 > 0) + (n1 > 0) + min(t, n0) + min(t, max(n0 - 1, 0)) + min(t, n1) + min(t, max(n1 - 1, 0));
        if (g == 1) pos += (t < n0) + (t + 1 < n0);
        const int slot = pos % NS;
        const bool v_ok = mbar_wait_or_abort(full(slot), (pos / NS) & 1, abort_flag, a.err, ERR_WAIT_TMA);
        if (!__all_sync(0xFFFFFFFFu, v_ok)) { ok = false; break; }
        for (int u = 0; u < 2; ++u) {
          if (!(u ? cut1 : cut0)) continue;
          for (int x = (u ? nv1 : nv0) * 8 + row; x < kUnit * 8; x += 128)
            for (int b = 0; b < Lay::NBOX; ++b)
              *reinterpret_cast<uint4*>(smem + Lay::RING_OFF + slot * Lay::TILE + b * kBox + u * kUnitBox + x * 16) =
                  make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      if (live) {
        tc_fence_after();
        uint32_t sr[kTile];
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c)
          tmem_ld32(s_col + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c) tmem_reg_fence(*reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
        if (nv0 < kUnit || nv1 < kUnit) {  // warp-uniform
#pragma unroll
          for (int i = 0; i < kTile; ++i)
            if ((i & (kUnit - 1)) >= (i < kUnit ? nv0 : nv1)) sr[i] = __float_as_uint(-INFINITY);
        }
        // row max with 8 independent partial maxima; NaN if a score is (then the row's sum is NaN too,
        // whichever pipe computes that score's exponential)
        float pm[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) pm[e] = __uint_as_float(sr[e]);
#pragma unroll
        for (int i = 8; i < kTile; i += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e) pm[e] = max3_nan(pm[e], __uint_as_float(sr[i + e]), __uint_as_float(sr[i + 8 + e]));
        const float mx = max3_nan(max3_nan(pm[0], pm[1], pm[2]), max3_nan(pm[3], pm[4], pm[5]), max3_nan(pm[6], pm[7], kNoMax));
        // finite also where every key of the tile is masked, so that exp2(-inf - m) is 0; an infinite
        // score makes it NaN, as inf - inf does in the formula
        const float mxs = fmaf(0.0f, mx, mx * p.scale_log2);
        float alpha = 1.0f;
        bool rescale = false;
        if (t == 0) {
          m_run = mxs;  // O is not there yet
        } else if (!(mxs <= m_run + 8.0f)) {  // NaN as well
          alpha = fast_exp2(m_run - mxs);
          m_run = mxs;
          rescale = true;
        }
        // p = exp2(s * c - m), packed to bf16 pairs in place; sum with 4 packed accumulators
        const float2 nm2 = make_float2(-m_run, -m_run);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < kTile; i += 2) {
          const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])), c2, nm2);
          float2 e;
          if (kPolyMod > 0 && (i >> 1) % (kPolyMod > 0 ? kPolyMod : 1) == kPolyMod - 1)
            e = exp2_poly2(x);
          else
            e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          acc[(i >> 1) & 3] = __fadd2_rn(acc[(i >> 1) & 3], e);
          sr[i >> 1] = pack_bf16x2(e.x, e.y);
        }
        const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
        const float2 a03 = __fadd2_rn(a01, a23);
        l_run = fmaf(l_run, alpha, a03.x + a03.y);
        // S_g(t) complete => PV_g(t-1) complete: O_g is stable until P_g(t) is published.
        if (__any_sync(0xFFFFFFFFu, rescale)) {
#pragma unroll
          for (int c = 0; c < DH / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_col + c * 32, o);
            tmem_ld_wait();
            tmem_reg_fence(o);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])),
                                          make_float2(alpha, alpha));
              o[e] = __float_as_uint(v.x);
              o[e + 1] = __float_as_uint(v.y);
            }
            tmem_st32(o_col + c * 32, o);
          }
        }
        // P_g(t) over the first 64 columns of S_g: column c holds keys 2c (low half) and 2c+1.
        tmem_st32(s_col, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_st32(s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(g));
    }
    const bool f_ok =
        ok && (it.tiles == 0 || mbar_wait_or_abort(fin(g), 0, abort_flag, a.err, ERR_WAIT_MMA));
    if (__all_sync(0xFFFFFFFFu, f_ok)) {
      tc_fence_after();
      if (live) {  // warp-uniform
        const bool mine = q < it.qn;
        const bool empty_row = l_run == 0.0f;  // no valid key: O was never written, or only with zeros
        const int b = it.bh / a.n_heads, h = it.bh - b * a.n_heads;
        const int dm = a.n_heads * DH;
        const long long o_at = ((long long)b * a.Lq + q) * dm + h * DH;
        const long long part_at = ((long long)item * kSparseQueries + row) * DH;
        const long long part_n = (long long)p.rows * p.nsplit * kSparseQueries;
        const float inv_l = 1.0f / l_run;
        const float2 il2 = make_float2(inv_l, inv_l);
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < DH / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_col + c * 32, o);
          tmem_ld_wait();
          tmem_reg_fence(o);
          if (p.nsplit > 1) {
            if (mine && !empty_row && H3B_IDX_OK(part_at + c * 32 + 31, part_n * DH, a.err)) {
              uint4* d4 = reinterpret_cast<uint4*>(p.part_o + part_at + c * 32);
#pragma unroll
              for (int e = 0; e < 8; ++e) d4[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          } else {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), il2);
              pk[e] = empty_row ? 0u : pack_bf16x2(v.x, v.y);
              amax = max3f(amax, fabsf(bf16_lo(pk[e])), fabsf(bf16_hi(pk[e])));
            }
            if (mine && H3B_IDX_OK(o_at + c * 32 + 31, (long long)a.B * a.Lq * dm, a.err)) {
              uint4* d4 = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + o_at + c * 32);
#pragma unroll
              for (int e = 0; e < 4; ++e) d4[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
            }
          }
        }
        if (mine) {
          if (p.nsplit > 1) {
            if (H3B_IDX_OK((long long)item * kSparseQueries + row, part_n, a.err))
              p.part_ml[(size_t)item * kSparseQueries + row] = make_float2(m_run, l_run);
          } else if (a.absmax && H3B_IDX_OK((long long)b * a.Lq + q, (long long)a.B * a.Lq, a.err)) {
            atomicMax(reinterpret_cast<unsigned*>(a.absmax) + (size_t)b * a.Lq + q, __float_as_uint(amax));
          }
        }
      }
    } else {
      *abort_flag = 1;
    }
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the items of a split list: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s. A warp per query row.
template <int DH>
__global__ void __launch_bounds__(128) sparse_join_kernel(const SparseParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const SparseAttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int row_item = blockIdx.x / (kSparseQueries / 4), r = (blockIdx.x % (kSparseQueries / 4)) * 4 + (threadIdx.x >> 5);
  const int bh = row_item / a.nqb, qb = row_item - bh * a.nqb;
  const int b = bh / a.n_heads, h = bh - b * a.n_heads;
  const int q = qb * kSparseQueries + r;
  if (q >= clamp_len(a.q_lens, b, a.Lq)) return;
  constexpr int V = DH / 32;  // lanes of the head per thread
  const size_t first = (size_t)row_item * p.nsplit;
  float M = kNoMax;
  for (int s = 0; s < p.nsplit; ++s) M = fmaxf(M, p.part_ml[(first + s) * kSparseQueries + r].x);
  float l = 0.0f, o[V] = {};
  for (int s = 0; s < p.nsplit; ++s) {
    const float2 ml = p.part_ml[(first + s) * kSparseQueries + r];
    if (ml.y == 0.0f) continue;  // no key in this range: its O was not written
    const float w = fast_exp2(ml.x - M);
    l = fmaf(w, ml.y, l);
    const float* src = p.part_o + ((first + s) * kSparseQueries + r) * DH + lane * V;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = fmaf(w, src[e], o[e]);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  float amax = 0.0f;
  uint32_t pk[V / 2];
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    pk[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
    amax = max3f(amax, fabsf(bf16_lo(pk[e])), fabsf(bf16_hi(pk[e])));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
  const long long at = ((long long)b * a.Lq + q) * a.n_heads * DH + h * DH + lane * V;
  if (H3B_IDX_OK(at + V - 1, (long long)a.B * a.Lq * a.n_heads * DH, a.err)) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.o) + at);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) dst[e] = pk[e];
  }
  if (a.absmax && lane == 0) atomicMax(reinterpret_cast<unsigned*>(a.absmax) + (size_t)b * a.Lq + q, __float_as_uint(amax));
}

// Items per list. A CTA works on two items at a time, and its start and end cost
// about as much as three tiles; the rule takes the split with the fewest tile
// times over all waves. 148 SMs, whatever the device has: the workspace's size
// must not depend on the device.
struct Split {
  int n, tiles;  // items per list, tiles per item
};
Split choose_split(long long rows, int topk, int block_k) {
  const int tiles = (topk * (block_k / kUnit) + 1) / 2;
  Split best{1, tiles};
  long long best_cost = -1;
  for (int n = 1; n <= 64 && n <= tiles; ++n) {
    const int per = (tiles + n - 1) / n, used = (tiles + per - 1) / per;
    const long long waves = ((rows * used + 1) / 2 + 147) / 148;
    const long long cost = waves * (per + 3) + (used > 1 ? 3 : 0);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = {used, per};
    }
  }
  return best;
}

template <int DH>
cudaError_t launch(const SparseAttnArgs& a, cudaStream_t st) {
  using Lay = Layout<DH>;
  SparseParams p{};
  p.a = a;
  p.rows = a.B * a.n_heads * a.nqb;
  const Split sp = choose_split(p.rows, a.topk, a.block_k);
  p.nsplit = sp.n;
  p.split_tiles = sp.tiles;
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)DH);
  const size_t items = (size_t)p.rows * p.nsplit;
  if (p.nsplit > 1) {
    p.part_o = static_cast<float*>(a.ws);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + items * kSparseQueries * DH);
  }
  CUtensorMap tmq, tmk, tmv;
  if (!make_tmap_3d(&tmq, a.q, 2, DH, a.Lq, (uint64_t)a.B * a.n_heads, 64, kSparseQueries) ||
      !make_tmap_3d(&tmk, a.k, 2, DH, a.Lk, (uint64_t)a.B * a.n_kv_heads, 64, kUnit) ||
      !make_tmap_3d(&tmv, a.v, 2, DH, a.Lk, (uint64_t)a.B * a.n_kv_heads, 64, kUnit))
    return cudaErrorInvalidValue;
  auto k = sparse_attention_kernel<DH, 4>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3((unsigned)((items + 1) / 2)), dim3(kThreads), Lay::SMEM, st, tmq, tmk, tmv, p);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  return launch_pdl(sparse_join_kernel<DH>, dim3(p.rows * (kSparseQueries / 4)), dim3(128), 0, st, p);
}

}  // namespace

size_t sparse_attn_ws_bytes(int B, int n_heads, int head_dim, int nqb, int topk, int block_k) {
  const long long rows = (long long)B * n_heads * nqb;
  const Split sp = choose_split(rows, topk, block_k);
  return sp.n > 1 ? (size_t)rows * sp.n * kSparseQueries * (head_dim * 4 + 8) : 0;
}

cudaError_t launch_sparse_attention(const SparseAttnArgs& a, cudaStream_t st) {
  return a.head_dim == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace h3b
