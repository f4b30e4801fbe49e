// Softmax attention of blocks of 128 queries over listed blocks of keys, on
// sm_100a tensor cores (bf16 operands, fp32 accumulation):
//   O[i] = sum_j softmax_j(Q[i].K[j] / sqrt(head_dim)) V[j],  j in the listed blocks
// in one pass over each list with the running maximum and sum of the softmax.
//
// An item is a query block of one head with a range of its list, 128 listed keys
// (a tile: two units of 64, gathered by their own TMA loads) at a time. A CTA
// works on pairs of items, each item with its own list, so that one item's
// products fill the tensor core while the other's softmax runs:
//   warps 0, 2  TMA for item 0, 1: Q, then the K and V tiles, each into its place
//               in one ring of slots that all loads share in the order of the MMAs
//   warp 1      tcgen05.mma from one elected thread, in the order
//                 S0(0) S1(0) | PV0(0) S0(1) PV1(0) S1(1) | PV0(1) S0(2) ...
//               where an item whose list has ended drops out; P comes in halves, and the first
//               is multiplied while the second is formed
//   warp 3      the next pair: takes over a CTA of this grid that has not started
//               (clusterlaunchcontrol), reads what its items need into shared
//               memory, and looks through their lists
//   warps 4-7   softmax of item 0, warps 8-11 softmax of item 1 (thread = row)
// The grid has one CTA per pair; the CTAs that run take over the others, so that
// the loads and first products of a pair overlap the end of the pair before it.
// A warp without a valid query row does no softmax (three new tokens use one of
// four). Tensor memory (512 columns): S0 | S1 | O0 | O1; P_g overwrites the first
// half of S_g. When S_g(j) is complete, PV_g(j-1) is too (a commit tracks every
// earlier MMA of its thread), so O_g can be rescaled without another barrier; it
// is rescaled only when a row's maximum grew by more than 2^16. P is rounded to
// bf16, the type of V, for the tensor core; the row sum adds the unrounded fp32
// exponentials.
//
// Bound by the chain of an item's tile: from S to the softmax 350 cycles, the first half of
// the exponentials 800 to 1100, from P to the MMA warp 300, P V and the next S 770. The two
// items of a pair cover that to about 3800 cycles for a tile of each (the slope over lists of
// 12 to 144 blocks, at 1.96 GHz), of which the tensor core works 2048; a pair's start and end
// add about 9000. 18432 tokens, 40 heads of 128, 36 of 288 blocks of 64 keys: 784 us,
// 1109 TFLOP/s; back to back, where the power limit lowers the clock, 868 to 936 us. The
// exponentials all go to the MUFU pipe (a fourth of them as polynomials 8% slower). Tiles of
// 64 keys with S computed one tile ahead: 12% slower.
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
constexpr int kPairs = 2;              // pairs of items in flight in a CTA
constexpr int kSms = 148;               // of a B200
constexpr int kAhead = 3;              // tiles before a pair's end at which the next is asked for
constexpr int kItemBytes = 64;
constexpr float kNoMax = -3.0e38f;     // running maximum before any key
// Exponents of 2 that a row's maximum may grow before it is raised. Scaled by a power of two, sums lose nothing: they
// stay finite for |v| up to 2^90. With 8, neighbouring keys alike and of variance 2 raised it so often that 798 us
// were 882.
constexpr float kGrowth = 16.0f;

struct SparseParams {
  SparseAttnArgs a;
  int nsplit, split_tiles, rows;  // items = rows * nsplit, item = row * nsplit + split
  int per_cta;                    // items of a pair: 2, or 1 where there are processors for all items
  float scale_log2;
  float4* part_o;  // [item][DH / 4][128], nsplit > 1: neighbouring rows side by side, as the threads that write them
  float2* part_ml; // [item][128]: maximum (in exponents of 2), sum
};

template <int DH>
struct Layout {
  static constexpr int NBOX = DH / 64;
  static constexpr int TILE = kTile * DH * 2;  // bytes of a slot, and of one item's Q
  static constexpr int NS = DH == 128 ? 5 : 10;
  static constexpr int Q_OFF = 0, RING_OFF = 2 * TILE;
  static constexpr int BAR_OFF = RING_OFF + NS * TILE;
  // mbarriers, by their place: per item (P: per item and half of a tile), per slot, per pair in flight
  static constexpr int Q_FULL = 0, Q_EMPTY = 2, S_FIRST = 4, P_FULL = 6, FIN = 10, FULL = 12, EMPTY = FULL + NS;
  static constexpr int PAIR_FULL = EMPTY + NS, PAIR_EMPTY = PAIR_FULL + kPairs, CLEAN = PAIR_EMPTY + kPairs;
  static constexpr int ENDING = CLEAN + kPairs, CANCEL = ENDING + 1;
  static constexpr int DRAIN = CANCEL + 1, NBARS = DRAIN + 1;
  static constexpr int FLAG_OFF = BAR_OFF + (NBARS + 1) / 2 * 16;  // tensor memory address, abort flag, loads
  static constexpr int RESPONSE_OFF = FLAG_OFF + 16;               // of the take-over request
  static constexpr int ITEM_OFF = RESPONSE_OFF + 16;               // [kPairs][2]
  static constexpr size_t SMEM = (size_t)ITEM_OFF + kPairs * 2 * kItemBytes + 1024;
  static constexpr uint32_t S_COL(int g) { return g * 128u; }
  static constexpr uint32_t O_COL(int g) { return 256u + g * DH; }
};
static_assert(Layout<128>::SMEM <= 232448 && Layout<64>::SMEM <= 232448, "shared memory of one CTA");
static_assert(Layout<64>::SMEM > 116 * 1024, "one CTA per SM: each holds all tensor memory columns");

__device__ __forceinline__ int clamp_len(const int* lens, int b, int L) {
  return lens ? min(max(__ldg(lens + b), 0), L) : L;
}

// The MMA warp stays converged and one elected thread's predicate `on` is on each of its instructions, so that
// operands live in uniform registers. Issued from a branch of one thread every MMA takes a dozen moves into those,
// which queue for issue slots behind the softmax: 168 cycles per MMA against 66 beside two warps per scheduler that
// issue all the time (128 x 128 x 16 takes 64).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on;
}
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc), "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit_to(uint32_t bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(on)
      : "memory");
}
// A value that all lanes hold, known as such to the compiler.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// A copy of its own for each role. A value that lives in all of them is kept on the stack while the softmax
// needs the registers, and would be reloaded at each of its uses between the MMAs.
__device__ __forceinline__ uint32_t own_copy(uint32_t v) {
  uint32_t r;
  asm volatile("mov.u32 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Each lane of four holds four pieces (4 registers each) of a row of its own; afterwards lane i of the four
// holds piece i of each of the four rows, in the rows' order.
__device__ __forceinline__ void transpose_quad(uint32_t (&v)[16], int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int x = 0; x < 16; ++x) {  // of pieces i (without the bit) and j (with it): keeps one, sends the other
      const int i = x >> 2, j = i | bit, lo = x, hi = 4 * j + (x & 3);
      if (i & bit) continue;
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? v[lo] : v[hi], bit);
      if (up)
        v[lo] = got;
      else
        v[hi] = got;
    }
  }
}

// What an item works on. Kept in shared memory: the softmax threads' registers are the scores'.
struct Item {
  int bh, qb;     // batch item x head, query block
  int kvrow;      // batch item x key head
  int qn, kn;     // valid queries and keys of the batch item
  int t0, units;  // first tile of the range, units in it
  int tiles;      // ceil(units / 2); -1: no further pair
  int clean;      // every unit of the range holds 64 valid keys (written after the rest)
  int pad;
  const int* list;
};
static_assert(sizeof(Item) <= kItemBytes && kItemBytes % 8 == 0, "the items' place in shared memory");

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
  it.list = a.blocks + (size_t)row * a.topk;
  const int entries = a.counts ? min(max(__ldg(a.counts + row), 0), a.topk) : a.topk;
  const int all = it.qb * kSparseQueries < it.qn && it.kn > 0 ? entries * (a.block_k / kUnit) : 0;
  it.t0 = split * p.split_tiles;
  it.units = min(max(all - 2 * it.t0, 0), 2 * p.split_tiles);
  it.tiles = (it.units + 1) / 2;
  return it;
}

// Whether every unit of the item's range holds 64 valid keys. By a whole warp.
__device__ __forceinline__ int all_clean(const SparseAttnArgs& a, const Item& it, int lane) {
  const int per = a.block_k / kUnit;  // units per entry
  bool clean = true;
  for (int u = lane * per; u < it.units; u += 32 * per) {
    const int v = __ldg(it.list + (2 * it.t0 + u) / per);
    clean = clean && (unsigned)v < (unsigned)a.nkb && (v + 1) * a.block_k <= it.kn;
  }
  return __all_sync(0xFFFFFFFFu, clean);
}

// Walks an item's list in tiles; a warp's lanes hold 32 entries as the first keys of their blocks
// (`none` where an entry holds no valid key), with the next 32 on their way.
struct ListWalk {
  const int* list;
  int entries, kn, block_k, nkb, none;  // entries: of the range
  int cur, nxt, base;                   // this lane's entry of the chunk that starts at entry `base`, and of the next
  __device__ __forceinline__ int fetch(int e) const {
    const int v = e < entries ? __ldg(list + e) : -1;
    return (unsigned)v < (unsigned)nkb && v * block_k < kn ? v * block_k : none;
  }
  // First keys of the two units of tile t of a list whose last unit is `units` - 1.
  __device__ __forceinline__ int2 tile(int t, int units, int lane) {
    const bool wide = block_k == kTile;
    const int e0 = wide ? t : 2 * t;
    if (e0 - base >= 32) {
      base += 32;
      cur = nxt;
      nxt = fetch(base + 32 + lane);
    }
    int2 s;
    s.x = __shfl_sync(0xFFFFFFFFu, cur, e0 - base);
    s.y = __shfl_sync(0xFFFFFFFFu, cur, e0 - base + (wide ? 0 : 1));
    if (wide) s.y = s.x + kUnit < kn ? s.x + kUnit : none;
    if (2 * t + 1 >= units) s.y = none;
    return s;
  }
};

// A place in the order of loads: its slot in the ring, the parity of that use of the slot, its number.
template <int NS>
struct Place {
  int slot = 0;
  uint32_t ph = 0, n = 0;
  __device__ __forceinline__ void advance(int by) {  // by <= NS
    n += by;
    slot += by;
    if (slot >= NS) {
      slot -= NS;
      ph ^= 1u;
    }
  }
  __device__ __forceinline__ void advance_any(int by) {
    n += by;
    const int s = slot + by;
    ph ^= (uint32_t)(s / NS) & 1u;
    slot = s % NS;
  }
};

// Waits (a whole warp, which decides as one) until *count, a running number, has reached `n`; bounded
// like every wait of the library.
__device__ __forceinline__ bool wait_reached(const volatile uint32_t* count, uint32_t n, const volatile int* abort,
                                             unsigned* err) {
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xFFFFFFFFu, (int32_t)(*count - n) >= 0)) return true;
    if ((i & 63u) != 0) continue;
    const bool late = globaltimer() - t0 > kWaitLimitNs;
    if (__any_sync(0xFFFFFFFFu, late || *abort)) {
      if (late) atomicOr(err, ERR_WAIT_MMA);
      return false;
    }
  }
}

// The same in one register, for the softmax threads: the number of the load modulo 2 NS.
template <int NS>
struct Turn {
  int c = 0;
  __device__ __forceinline__ int slot() const { return c < NS ? c : c - NS; }
  __device__ __forceinline__ uint32_t ph() const { return c < NS ? 0u : 1u; }
  __device__ __forceinline__ void advance(int by) {  // by <= 2 NS
    c += by;
    if (c >= 2 * NS) c -= 2 * NS;
  }
  __device__ __forceinline__ void advance_any(int by) { c = (c + by) % (2 * NS); }
};

// Asks for the takeover of a CTA of this grid that has not started; the 16-byte response completes on `bar`.
__device__ __forceinline__ void request_cta(uint32_t response, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   response),
               "r"(bar)
               : "memory");
}
// blockIdx.x of the CTA taken over, or -1 when none was left.
__device__ __forceinline__ int taken_cta(uint32_t response) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(response)
      : "memory");
  return ok ? (int)x : -1;
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
    sparse_attention_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                            const __grid_constant__ CUtensorMap tmv, const SparseParams p) {
  using Lay = Layout<DH>;
  constexpr int NS = Lay::NS;
  const SparseAttnArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb_ = smem_u32(smem);
  auto bar = [&](int place) { return sb_ + Lay::BAR_OFF + 8u * place; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + Lay::FLAG_OFF);
  volatile uint32_t* loaded = reinterpret_cast<volatile uint32_t*>(smem + Lay::FLAG_OFF + 8);  // each producer's last load
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t IDESC_S = instr_desc(1, 1, 0, 0, kSparseQueries, kTile);
  constexpr uint32_t IDESC_S_HALF = instr_desc(1, 1, 0, 0, kSparseQueries, kUnit);
  constexpr uint32_t IDESC_PV = instr_desc(1, 1, 0, 1, kSparseQueries, DH);

  static_assert(Lay::NBARS <= kThreads, "a thread per barrier");
  if (threadIdx.x < Lay::NBARS) {
    const int i = threadIdx.x;
    // arrivals: P of an item by its softmax warps; a pair is let go by producers, MMA and softmax warps
    const bool p_full = i >= Lay::P_FULL && i < Lay::P_FULL + 4;
    const bool pair_empty = i >= Lay::PAIR_EMPTY && i < Lay::PAIR_EMPTY + kPairs;
    mbar_init(bar(i), p_full ? 4 : pair_empty ? 2 + 1 + 8 : i == Lay::ENDING ? 2 : 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    *reinterpret_cast<volatile int*>(smem + Lay::FLAG_OFF + 4) = 0;
    loaded[0] = loaded[1] = ~0u;
    tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  if (warp == 1) {
    tmem_alloc(sb_ + Lay::FLAG_OFF, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // q, k, v and the lists may be the previous grid's output
  griddep_launch_dependents();

  auto flag_at = [](uint32_t base) { return static_cast<volatile int*>(__cvta_shared_to_generic(base + Lay::FLAG_OFF + 4)); };
  // Pair k of this CTA, in every role: its items once they are there (nullptr after a failure).
  // `lanes`: those that call it, which decide as one (they may see the abort flag at different times).
  auto pair_items = [&](uint32_t base, int k, unsigned lanes) -> const Item* {
    const bool ok = mbar_wait_or_abort(base + Lay::BAR_OFF + 8u * (Lay::PAIR_FULL + k % kPairs), (k / kPairs) & 1,
                                       flag_at(base), a.err, ERR_WAIT_EPI);
    if (!__all_sync(lanes, ok)) return nullptr;
    return static_cast<const Item*>(__cvta_shared_to_generic(base + Lay::ITEM_OFF + (k % kPairs) * 2 * kItemBytes));
  };
  auto second = [](const Item* it) {
    return reinterpret_cast<const Item*>(reinterpret_cast<const uint8_t*>(it) + kItemBytes);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0 || warp == 2) {
      // ---------------- TMA producer of item g (whole warp; lane 0 issues)
      const uint32_t sb = own_copy(sb_);
      auto bar = [&](int place) { return sb + Lay::BAR_OFF + 8u * place; };
      volatile int* abort_flag = flag_at(sb);
      const int g = warp >> 1;
      Place<NS> place;                  // of the pair's first load
      uint32_t last = ~0u;              // number of this warp's load before; none yet: the one before the first
      uint32_t filled = 0, phases = 0;  // slots this warp has filled, with the parity of the last use
      uint32_t items_done = 0;          // items with keys so far
      bool ok = true;
      auto load = [&](const CUtensorMap* map, Place<NS> at, int2 keys, bool two, int kvrow) -> bool {
        // Wait until the slot's use before this one is released. A parity tells two uses apart, not
        // more, so the use before that must be known to be over: it is once a load at most NS places
        // back has waited (slots are released in order), this warp's own or, where the other item has
        // had more loads since, the other warp's.
        if (at.n - last > NS && !wait_reached(&loaded[g ^ 1], at.n - NS, abort_flag, a.err)) return false;
        const bool free_ = mbar_wait_or_abort(bar(Lay::EMPTY + at.slot), at.ph ^ 1u, abort_flag, a.err, ERR_WAIT_MMA);
        if (!__all_sync(0xFFFFFFFFu, free_)) return false;
        last = at.n;
        if (lane == 0) loaded[g] = at.n;
        filled |= 1u << at.slot;
        phases = (phases & ~(1u << at.slot)) | (at.ph << at.slot);
        if (lane == 0) {
          const uint32_t full = bar(Lay::FULL + at.slot);
          const uint32_t dst = sb + Lay::RING_OFF + at.slot * Lay::TILE;
          mbar_arrive_expect_tx(full, (two ? 2 : 1) * Lay::NBOX * kUnitBox);
#pragma unroll
          for (int b = 0; b < Lay::NBOX; ++b) {
            tma_load_3d(dst + b * kBox, map, full, b * 64, keys.x, kvrow);
            if (two) tma_load_3d(dst + b * kBox + kUnitBox, map, full, b * 64, keys.y, kvrow);
          }
        }
        return true;
      };
      for (int k = 0; ok; ++k) {
        const Item* pair = pair_items(sb, k, 0xFFFFFFFFu);
        if (!pair) { ok = false; break; }
        const int n0 = pair->tiles, n1 = second(pair)->tiles;
        if (n0 < 0) break;
        const Item* it = g ? second(pair) : pair;
        const int n = g ? n1 : n0, units = it->units, kvrow = it->kvrow;
        Place<NS> at = place;
        place.advance_any(2 * (n0 + n1));
        // The next pair is asked for when the loads of this one are kAhead tiles from their end (see warp 3).
        auto ending = [&](int t) {
          if (t == max(n - kAhead, 0) && lane == 0) mbar_arrive(bar(Lay::ENDING));
        };
        if (n == 0) ending(0);
        if (n > 0) {
          // Q, once the item before is done with its S products
          if (items_done > 0) {
            const bool free_ =
                mbar_wait_or_abort(bar(Lay::Q_EMPTY + g), (items_done - 1) & 1, abort_flag, a.err, ERR_WAIT_MMA);
            if (!__all_sync(0xFFFFFFFFu, free_)) { ok = false; break; }
          }
          ++items_done;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(Lay::Q_FULL + g), Lay::TILE);
#pragma unroll
            for (int b = 0; b < Lay::NBOX; ++b)
              tma_load_3d(sb + Lay::Q_OFF + g * Lay::TILE + b * kBox, &tmq, bar(Lay::Q_FULL + g), b * 64,
                          it->qb * kSparseQueries, it->bh);
          }
          ListWalk walk;
          walk.block_k = a.block_k;
          walk.nkb = a.nkb;
          walk.none = a.nkb * a.block_k;  // >= Lk: rows there read as zeros
          walk.kn = it->kn;
          walk.list = it->list + (a.block_k == kTile ? it->t0 : 2 * it->t0);
          walk.entries = a.block_k == kTile ? (units + 1) / 2 : units;
          walk.base = 0;
          walk.cur = walk.fetch(lane);
          walk.nxt = walk.fetch(32 + lane);
          if (g == 1) at.advance(n0 > 0);
          int2 keys = walk.tile(0, units, lane);
          ok = load(&tmk, at, keys, units > 1, kvrow);
          // to this item's first load of round 0: past the other item's first K tile (item 0) or its
          // loads of the round (item 1)
          at.advance(1 + (g == 0 ? (n1 > 0) : (n0 > 0) + (n0 > 1)));
          for (int t = 0; t < n && ok; ++t) {
            ending(t);
            ok = load(&tmv, at, keys, units - 2 * t > 1, kvrow);
            if (!ok || t + 1 == n) break;
            at.advance(1);
            keys = walk.tile(t + 1, units, lane);
            ok = load(&tmk, at, keys, units - 2 * (t + 1) > 1, kvrow);
            // past the other item's loads between: the rest of round t (item 0) or the start of round t + 1 (item 1)
            at.advance(1 + (g == 0 ? (t < n1) + (t + 1 < n1) : (t + 1 < n0) + (t + 2 < n0)));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Lay::PAIR_EMPTY + k % kPairs));
      }
      if (!ok) {  // nothing of this warp's may land after the CTA has ended
        *abort_flag = 1;
        for (int s = 0; s < NS; ++s)
          if (filled & (1u << s)) mbar_wait(bar(Lay::FULL + s), (phases >> s) & 1u, a.err, ERR_WAIT_DRAIN, kDrainLimitNs);
        if (items_done > 0) mbar_wait(bar(Lay::Q_FULL + g), (items_done - 1) & 1, a.err, ERR_WAIT_DRAIN, kDrainLimitNs);
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer (whole warp, converged)
      const uint32_t sb = uniform(sb_), tm = uniform(*tmem_slot), on = elect_one();
      auto bar = [&](int place) { return sb + Lay::BAR_OFF + 8u * place; };
      volatile int* abort_flag = flag_at(sb);
      bool any = false, ok = true;
      Place<NS> at;
      uint32_t tiles_done[2] = {0, 0}, items_done[2] = {0, 0};
      auto wait = [&](int place, uint32_t parity, unsigned code) -> bool {
        return __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(place), parity, abort_flag, a.err, code));
      };
      auto give = [&]() {
        any = true;
        commit_to(bar(Lay::EMPTY + at.slot), on);
        at.advance(1);
      };
      auto issue_s = [&](int g, bool two, bool first, bool last) {  // S_g = Q_g K^T of the item's next tile
        const uint64_t qd = smem_desc_sw128(sb + Lay::Q_OFF + g * Lay::TILE, 16, 1024);
        const uint64_t kd = smem_desc_sw128(sb + Lay::RING_OFF + at.slot * Lay::TILE, 16, 1024);
        if (two) {
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint32_t step = ((k >> 2) * kBox + (k & 3) * 32) >> 4;  // of the address field
            mma_ss(tm + Lay::S_COL(g), qd + step, kd + step, IDESC_S, k > 0 ? 1u : 0u, on);
          }
        } else {  // one unit: a path of its own, since a choice inside the unrolled one slows every tile
#pragma unroll 1
          for (int k = 0; k < DH / 16; ++k) {
            const uint32_t step = ((k >> 2) * kBox + (k & 3) * 32) >> 4;
            mma_ss(tm + Lay::S_COL(g), qd + step, kd + step, IDESC_S_HALF, k > 0 ? 1u : 0u, on);
          }
        }
        if (first) commit_to(bar(Lay::S_FIRST + g), on);
        if (last) commit_to(bar(Lay::Q_EMPTY + g), on);
        give();
      };
      auto issue_pv = [&](int g, int half, bool fresh) {  // O_g (+)= P_g V, 64 of the tile's keys
        const uint64_t vd = smem_desc_sw128(sb + Lay::RING_OFF + at.slot * Lay::TILE + half * kUnitBox, kBox, 1024);
#pragma unroll
        for (int k = 0; k < kUnit / 16; ++k)
          mma_ts(tm + Lay::O_COL(g), tm + Lay::S_COL(g) + half * 32 + k * 8, vd + (k * 2048 >> 4), IDESC_PV,
                 (!fresh || k > 0) ? 1u : 0u, on);
      };
      // the slot of the load `by` places on holds its tile
      auto landed = [&](int by) -> bool {
        Place<NS> x = at;
        x.advance(by);
        return wait(Lay::FULL + x.slot, x.ph, ERR_WAIT_TMA);
      };
      for (int k = 0; ok; ++k) {
        const Item* pair = pair_items(sb, k, 0xFFFFFFFFu);
        if (!pair) { ok = false; break; }
        const int n0 = uniform(pair->tiles), n1 = uniform(second(pair)->tiles);
        if (n0 < 0) break;
        const int units0 = uniform(pair->units), units1 = uniform(second(pair)->units);
        if (on) mbar_arrive(bar(Lay::PAIR_EMPTY + k % kPairs));
        __syncwarp();
        auto first = [&](int g, int units) -> bool {
          if (units == 0) return true;
          if (!wait(Lay::Q_FULL + g, items_done[g] & 1, ERR_WAIT_TMA)) return false;
          ++items_done[g];
          if (!landed(0)) return false;
          tc_fence_after();
          issue_s(g, units > 1, true, units <= 2);
          return true;
        };
        auto round = [&](int g, int units, int n, int t) -> bool {
          if (t >= n) return true;
          // P last: it is what the rounds wait for, and each wait takes some 150 cycles beside the softmax
          const bool more = t + 1 < n;
          const uint32_t parity = tiles_done[g] & 1;
          ++tiles_done[g];
          if (!landed(0) || (more && !landed(1)) || !wait(Lay::P_FULL + 2 * g, parity, ERR_WAIT_EPI)) return false;
          tc_fence_after();
          issue_pv(g, 0, t == 0);
          if (!wait(Lay::P_FULL + 2 * g + 1, parity, ERR_WAIT_EPI)) return false;
          tc_fence_after();
          if (units - 2 * t > 1) issue_pv(g, 1, false);
          give();
          if (more)
            issue_s(g, units - 2 * (t + 1) > 1, false, t + 2 == n);
          else
            commit_to(bar(Lay::FIN + g), on);
          return true;
        };
        ok = first(0, units0) && first(1, units1);
        const int n = max(n0, n1);
        for (int t = 0; t < n && ok; ++t) ok = round(0, units0, n0, t) && round(1, units1, n1, t);
      }
      if (!ok) {
        *abort_flag = 1;
        if (any) {
          commit_to(bar(Lay::DRAIN), on);
          mbar_wait(bar(Lay::DRAIN), 0, a.err, ERR_WAIT_DRAIN, kDrainLimitNs);
        }
      }
    } else {
      // ---------------- the next pair (whole warp)
      const uint32_t sb = own_copy(sb_);
      auto bar = [&](int place) { return sb + Lay::BAR_OFF + 8u * place; };
      volatile int* abort_flag = flag_at(sb);
      int cta = blockIdx.x;
      bool ok = true;
      const bool more = gridDim.x > kSms;  // else every CTA starts by itself
      for (int k = 0; ok && cta >= 0; ++k) {
        // The place's pair before this one has been let go by all, and the pair before this one nears its end:
        // a CTA is taken over no earlier than its loads need, so the last ones go to whoever is free first.
        bool free_ = mbar_wait_or_abort(bar(Lay::PAIR_EMPTY + k % kPairs), ((k / kPairs) & 1) ^ 1, abort_flag, a.err,
                                        ERR_WAIT_EPI);
        if (k > 0 && more) free_ = free_ && mbar_wait_or_abort(bar(Lay::ENDING), (k - 1) & 1, abort_flag, a.err, ERR_WAIT_EPI);
        ok = __all_sync(0xFFFFFFFFu, free_);
        if (!ok) break;
        if (k > 0 && !more) {
          cta = -1;
        } else if (k > 0) {
          if (lane == 0) {
            fence_proxy_async_smem();  // the response before was read from the same place
            mbar_arrive_expect_tx(bar(Lay::CANCEL), 16);
            request_cta(sb + Lay::RESPONSE_OFF, bar(Lay::CANCEL));
          }
          __syncwarp();
          // not given up on an abort: no response may land after the CTA has ended
          const bool answered = mbar_wait(bar(Lay::CANCEL), (k - 1) & 1, a.err, ERR_WAIT_DRAIN);
          ok = __all_sync(0xFFFFFFFFu, answered);
          if (!ok) break;
          cta = taken_cta(sb + Lay::RESPONSE_OFF);
          __syncwarp();
        }
        Item it0{}, it1{};
        it0.tiles = -1;
        if (cta >= 0) {
          it0 = load_item(p, p.per_cta * cta);
          if (p.per_cta == 2) it1 = load_item(p, 2 * cta + 1);
        }
        Item* to = static_cast<Item*>(__cvta_shared_to_generic(sb + Lay::ITEM_OFF + (k % kPairs) * 2 * kItemBytes));
        if (lane == 0) {
          *to = it0;
          *const_cast<Item*>(second(to)) = it1;
          mbar_arrive(bar(Lay::PAIR_FULL + k % kPairs));
        }
        __syncwarp();
        if (cta >= 0) {  // only the softmax asks, and not before the first tile
          const int clean0 = all_clean(a, it0, lane), clean1 = all_clean(a, it1, lane);
          if (lane == 0) {
            to->clean = clean0;
            const_cast<Item*>(second(to))->clean = clean1;
            mbar_arrive(bar(Lay::CLEAN + k % kPairs));
          }
          __syncwarp();
        }
      }
      if (!ok) *abort_flag = 1;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---------------- softmax warps: 4-7 -> item 0, 8-11 -> item 1 (thread = query row)
    const uint32_t sb = own_copy(sb_);
    auto bar = [&](int place) { return sb + Lay::BAR_OFF + 8u * place; };
    volatile int* abort_flag = flag_at(sb);
    const int g = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
    const uint32_t s_col = *tmem_slot + t_lane + Lay::S_COL(g), o_col = *tmem_slot + t_lane + Lay::O_COL(g);
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t items_done = 0;
    Turn<NS> place;  // of the pair's first load
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const volatile Item* pair = pair_items(sb, k, 0xFFFFFFFFu);
      if (!pair) { ok = false; break; }
      if (pair->tiles < 0) break;
      const bool looked = mbar_wait_or_abort(bar(Lay::CLEAN + k % kPairs), (k / kPairs) & 1, abort_flag, a.err, ERR_WAIT_EPI);
      if (!__all_sync(0xFFFFFFFFu, looked)) { ok = false; break; }
      const volatile Item* it = g ? second(const_cast<const Item*>(pair)) : pair;
      const bool live = it->qb * kSparseQueries + quad * 32 < it->qn;  // warp-uniform: a valid row in this warp
      // valid keys of unit u (counted from the item's first): the entry's block ends at kv_len
      auto valid_keys = [&](int u) {
        if (u >= it->units) return 0;
        const bool wide = a.block_k == kTile;
        const int v = __ldg(const_cast<const int*>(it->list) + (wide ? it->t0 + (u >> 1) : 2 * it->t0 + u));
        if ((unsigned)v >= (unsigned)a.nkb) return 0;
        return min(kUnit, max(0, it->kn - v * a.block_k - (wide ? (u & 1) * kUnit : 0)));
      };
      float m_run = kNoMax, l_run = 0.0f;
      // exp2(s * c + nm) of 64 scores, packed to bf16 pairs in their first 32 places; returns the sum
      auto exponentials = [&](uint32_t* s, float nm) -> float {
        const float2 nm2 = make_float2(nm, nm);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < kUnit; i += 2) {
          const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, nm2);
          const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          acc[(i >> 1) & 3] = __fadd2_rn(acc[(i >> 1) & 3], e);
          s[i >> 1] = pack_bf16x2(e.x, e.y);
        }
        const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
        const float2 a03 = __fadd2_rn(a01, a23);
        return a03.x + a03.y;
      };
      const volatile Item* other = g ? pair : second(const_cast<const Item*>(pair));
      Turn<NS> at = place;  // of K_g(t)
      if (g == 1) at.advance(other->tiles > 0);
      for (int t = 0; t < it->tiles; ++t) {
        int nv0 = kUnit, nv1 = kUnit;
        if (!it->clean || 2 * t + 1 >= it->units) {  // a clean list's whole tiles hold 128 valid keys
          nv0 = valid_keys(2 * t);
          nv1 = valid_keys(2 * t + 1);
        }
        // S_g(t) is complete when its K is released: one commit tells both (each costs the tensor core some
        // 40 cycles). The parity is of this use of the slot: K_g(t-1), at most four loads earlier, is released,
        // so the use NS loads earlier is over, and the next one's release comes after P V of this tile, which waits
        // for this warp. The first tile, which has no K_g(t-1) to go by, has a barrier of its own.
        const uint32_t s_bar = t == 0 ? bar(Lay::S_FIRST + g) : bar(Lay::EMPTY + at.slot());
        const bool s_ok = mbar_wait_or_abort(s_bar, t == 0 ? items_done & 1 : at.ph(), abort_flag, a.err, ERR_WAIT_MMA);
        if (!__all_sync(0xFFFFFFFFu, s_ok)) { ok = false; break; }
        // to V_g(t): past the other item's loads between (see the producers)
        const int others = other->tiles;
        at.advance(1 + (g == 0 ? (t > 0 && t - 1 < others) + (t < others) : (t < others) + (t + 1 < others)));
        // V rows behind kv_len (in memory, so TMA does not zero them) are zeroed once V_t has landed. S_g(t) is
        // complete, so every load up to K_g(t) has been used, among them the one that held V_g(t)'s
        // slot before (at least five loads earlier): the parity cannot be of an older phase
        if (((nv0 > 0 && nv0 < kUnit) || (nv1 > 0 && nv1 < kUnit)) && it->kn < a.Lk) {
          const bool v_ok = mbar_wait_or_abort(bar(Lay::FULL + at.slot()), at.ph(), abort_flag, a.err, ERR_WAIT_TMA);
          if (!__all_sync(0xFFFFFFFFu, v_ok)) { ok = false; break; }
          for (int u = 0; u < 2; ++u) {
            const int nv = u ? nv1 : nv0;
            if (nv == 0) continue;
            for (int x = nv * 8 + row; x < kUnit * 8; x += 128)
              for (int b = 0; b < Lay::NBOX; ++b)
                *static_cast<uint4*>(__cvta_shared_to_generic(sb + Lay::RING_OFF + at.slot() * Lay::TILE + b * kBox + u * kUnitBox + x * 16)) =
                    make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        at.advance(1);  // to K_g(t + 1)
        if (live) {
          // The exponentials of the first half are taken with the running maximum as it is, while the maximum of
          // the tile is found. Only where a row's maximum has grown by more than 2^16 (rare after an item's first tile)
          // is that maximum raised, O rescaled, and the half done again.
          uint32_t sr[kTile];
          float alpha = 1.0f, part;
          for (bool again = false;; again = true) {
            tc_fence_after();
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
            // row max with 8 independent partial maxima; NaN if a score is (then the row's sum is NaN too)
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
            if (t == 0) m_run = mxs;
            part = exponentials(sr, -m_run);
            const bool grown = !(mxs <= m_run + kGrowth);  // NaN as well
            if (again || t == 0 || !__any_sync(0xFFFFFFFFu, grown)) break;
            if (grown) {
              alpha = fast_exp2(m_run - mxs);
              m_run = mxs;
            }
            // S_g(t) complete => PV_g(t-1) complete: O_g is stable until P_g(t) is published.
#pragma unroll 1
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
          // P_g(t) over the first 64 columns of S_g: column c holds keys 2c (low half) and 2c+1. Its first half is
          // multiplied while the second is formed.
          tmem_st32(s_col, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Lay::P_FULL + 2 * g));
          part += exponentials(sr + kUnit, -m_run);
          tmem_st32(s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[kUnit]));
          l_run = fmaf(l_run, alpha, part);
          tmem_st_wait();
        }
        tc_fence_before();  // P is there, and O of the item before has been read
        __syncwarp();
        if (lane == 0) {
          if (!live) mbar_arrive(bar(Lay::P_FULL + 2 * g));
          mbar_arrive(bar(Lay::P_FULL + 2 * g + 1));
        }
      }
      if (!ok) break;
      if (it->tiles > 0) {
        const bool f_ok = mbar_wait_or_abort(bar(Lay::FIN + g), items_done & 1, abort_flag, a.err, ERR_WAIT_MMA);
        if (!__all_sync(0xFFFFFFFFu, f_ok)) { ok = false; break; }
        ++items_done;
      }
      tc_fence_after();
      if (live) {  // warp-uniform
        const int item = (it->bh * a.nqb + it->qb) * p.nsplit + it->t0 / p.split_tiles;
        const int q = it->qb * kSparseQueries + row;
        const bool mine = q < it->qn;
        const bool empty_row = l_run == 0.0f;  // no valid key: O was never written, or only with zeros
        const int b = it->bh / a.n_heads, h = it->bh - b * a.n_heads;
        const int dm = a.n_heads * DH;
        // stores go by quads of lanes: 64 bytes of one row at a time (a lane's own row at 16 bytes a time occupies the
        // load-store unit for 32 cycles an instruction: 4500 to 8700 cycles for the two items)
        const int first = q - (lane & 3);
        const long long o_at = ((long long)b * a.Lq + first) * dm + h * DH + (lane & 3) * 8;
        const long long part_at = (long long)item * (DH / 4) * kSparseQueries + row;
        const float inv_l = 1.0f / l_run;
        const float2 il2 = make_float2(inv_l, inv_l);
        float amax = 0.0f;
#pragma unroll 1  // unrolled, most of its time is the fetch of instructions that run once an item
        for (int c = 0; c < DH / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_col + c * 32, o);
          tmem_ld_wait();
          tmem_reg_fence(o);
          if (p.nsplit > 1) {
            if (mine && !empty_row &&
                H3B_IDX_OK(part_at + (c * 8 + 7) * kSparseQueries, (long long)p.rows * p.nsplit * (DH / 4) * kSparseQueries, a.err)) {
              float4* d4 = p.part_o + part_at + c * 8 * kSparseQueries;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                d4[e * kSparseQueries] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                     __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            }
          } else {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), il2);
              pk[e] = empty_row ? 0u : pack_bf16x2(v.x, v.y);
              amax = max3_nan(amax, fabsf(bf16_lo(pk[e])), fabsf(bf16_hi(pk[e])));
            }
            transpose_quad(pk, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // row e of the quad's four, 16 bytes of it per lane
              const long long at = o_at + (long long)e * dm + c * 32;
              if (first + e < it->qn && H3B_IDX_OK(at + 7, (long long)a.B * a.Lq * dm, a.err))
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + at) =
                    make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
            }
          }
        }
        if (mine) {
          if (p.nsplit > 1) {
            if (H3B_IDX_OK((long long)item * kSparseQueries + row, (long long)p.rows * p.nsplit * kSparseQueries, a.err))
              p.part_ml[(size_t)item * kSparseQueries + row] = make_float2(m_run, l_run);
          } else if (a.absmax && H3B_IDX_OK((long long)b * a.Lq + q, (long long)a.B * a.Lq, a.err)) {
            atomicMax(reinterpret_cast<unsigned*>(a.absmax) + (size_t)b * a.Lq + q, __float_as_uint(amax));
          }
        }
      }
      place.advance_any(2 * (max(pair->tiles, 0) + second(const_cast<const Item*>(pair))->tiles));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Lay::PAIR_EMPTY + k % kPairs));
    }
    if (!ok) *abort_flag = 1;
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(*tmem_slot, kTmemCols);
  }
}

// Joins the items of a split list: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s. A CTA per 32 query rows and
// 32 lanes of the head, a thread per row and four lanes. The parts' weights are formed once, in shared memory, so
// that the loads of the parts wait for nothing; the output is turned into rows in shared memory.
constexpr int kMaxSplit = 64;
template <int DH>
__global__ void __launch_bounds__(256) sparse_join_kernel(const SparseParams p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float2 weight[kMaxSplit][32];  // maximum and sum of a part's row; then its weight, and whether it has one
  __shared__ float tile[32][36];
  const SparseAttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int list = blockIdx.x >> 2, r0 = (blockIdx.x & 3) * 32, r = r0 + lane;
  const int bh = list / a.nqb, qb = list - bh * a.nqb;
  const int b = bh / a.n_heads, h = bh - b * a.n_heads;
  const int valid = clamp_len(a.q_lens, b, a.Lq) - qb * kSparseQueries;  // rows of the query block
  if (r0 >= valid) return;                                               // block-uniform
  const size_t first = (size_t)list * p.nsplit;
  const bool mine = r < valid;
  const int n = p.nsplit;
  for (int s = warp; s < n; s += 8)
    weight[s][lane] = mine ? p.part_ml[(first + s) * kSparseQueries + r] : make_float2(kNoMax, 0.0f);
  const float4* src = p.part_o + (first * (DH / 4) + 8 * blockIdx.y + warp) * kSparseQueries + r;
  constexpr size_t step = (size_t)(DH / 4) * kSparseQueries;  // from one part to the next
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v[8];
  auto fetch = [&](int s0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mine && s0 + i < n ? src[(s0 + i) * step] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  fetch(0);
  __syncthreads();
  float M = kNoMax;
  for (int s = 0; s < n; ++s) M = fmaxf(M, weight[s][lane].x);
  float l = 0.0f;
  for (int s0 = 0; s0 < n; s0 += 8) {
    float4 u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = v[i];
    fetch(s0 + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (s0 + i >= n) break;
      const float2 ml = weight[s0 + i][lane];
      if (ml.y == 0.0f) continue;  // no key in its range: its output was not written; a NaN sum counts
      const float w = fast_exp2(ml.x - M);
      l = fmaf(w, ml.y, l);
      o = make_float4(fmaf(w, u[i].x, o.x), fmaf(w, u[i].y, o.y), fmaf(w, u[i].z, o.z), fmaf(w, u[i].w, o.w));
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<float4*>(&tile[lane][4 * warp]) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  __syncthreads();
  // eight threads per row, four lanes of the head each
  const int i = threadIdx.x >> 3, c = 4 * (threadIdx.x & 7);
  const float4 x = *reinterpret_cast<const float4*>(&tile[i][c]);
  const uint2 pk = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
  float amax = max_nan(max3_nan(fabsf(bf16_lo(pk.x)), fabsf(bf16_hi(pk.x)), fabsf(bf16_lo(pk.y))), fabsf(bf16_hi(pk.y)));
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
  if (r0 + i >= valid) return;
  const int q = qb * kSparseQueries + r0 + i;
  const long long at = ((long long)b * a.Lq + q) * a.n_heads * DH + h * DH + 32 * blockIdx.y + c;
  if (H3B_IDX_OK(at + 3, (long long)a.B * a.Lq * a.n_heads * DH, a.err))
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + at) = pk;
  if (a.absmax && c == 0) atomicMax(reinterpret_cast<unsigned*>(a.absmax) + (size_t)b * a.Lq + q, __float_as_uint(amax));
}

// Items per list. In units of a tile of a CTA with one item (1.77 us): a tile of two items at once takes 1.2, an
// item's start and end 1.3 in each round of CTAs; no less than 0.0065 for each tile of all lists, their keys and
// values from HBM at head_dim 128; joining 2.7, and for each part 0.023 with 128 query rows. The rule takes the split
// with the least time. 148 SMs, whatever the device has: the workspace's size must not depend on the device. Measured
// with 100 queries over 36 tiles: 8 lists in one part each 64 us, as the rule splits them (18 parts) 15.4 us; 40 lists
// 66 and (6) 29.8 us, 80 lists 67 and (3) 49.5 us; 160 lists, which it leaves whole, 81 us, in three parts 92 us.
struct Split {
  int n, tiles;  // items per list, tiles per item
};
Split choose_split(long long rows, int Lq, int head_dim, int topk, int block_k) {
  const int tiles = (topk * (block_k / kUnit) + 1) / 2;
  const double memory = 0.0065 * head_dim / 128 * (double)rows * tiles;
  Split best{1, tiles};
  double best_cost = -1.0;
  for (int n = 1; n <= kMaxSplit && n <= tiles; ++n) {
    const int per = (tiles + n - 1) / n, used = (tiles + per - 1) / per;
    const long long items = rows * used;
    const double rounds = items <= kSms ? (double)per : (double)(((items + 1) / 2 + kSms - 1) / kSms) * (1.2 * per + 1.3);
    const double joined = used > 1 ? 2.7 + 0.023 * (double)items * std::min(Lq, kSparseQueries) / kSparseQueries : 0.0;
    const double cost = std::max(rounds, memory) + joined;
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
  const Split sp = choose_split(p.rows, a.Lq, DH, a.topk, a.block_k);
  p.nsplit = sp.n;
  p.split_tiles = sp.tiles;
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)DH);
  const size_t items = (size_t)p.rows * p.nsplit;
  p.per_cta = items <= kSms ? 1 : 2;
  if (p.nsplit > 1) {
    p.part_o = static_cast<float4*>(a.ws);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + items * kSparseQueries * (DH / 4));
  }
  CUtensorMap tmq, tmk, tmv;
  if (!make_tmap_3d(&tmq, a.q, 2, DH, a.Lq, (uint64_t)a.B * a.n_heads, 64, kSparseQueries) ||
      !make_tmap_3d(&tmk, a.k, 2, DH, a.Lk, (uint64_t)a.B * a.n_kv_heads, 64, kUnit))
    return cudaErrorInvalidValue;
  tmv = tmk;  // of the same shape: encoding a third map costs the host a microsecond
  if (!set_tmap_address(&tmv, a.v)) return cudaErrorInvalidValue;
  auto k = sparse_attention_kernel<DH>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3((unsigned)((items + p.per_cta - 1) / p.per_cta)), dim3(kThreads), Lay::SMEM, st, tmq, tmk, tmv, p);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  return launch_pdl(sparse_join_kernel<DH>, dim3(p.rows * (kSparseQueries / 32), DH / 32), dim3(256), 0, st, p);
}

}  // namespace

size_t sparse_attn_ws_bytes(int B, int n_heads, int head_dim, int Lq, int nqb, int topk, int block_k) {
  const long long rows = (long long)B * n_heads * nqb;
  if (Lq == 1) return sparse_rows_ws_bytes(rows, head_dim, topk, block_k);
  const Split sp = choose_split(rows, Lq, head_dim, topk, block_k);
  return sp.n > 1 ? (size_t)rows * sp.n * kSparseQueries * (head_dim * 4 + 8) : 0;
}

cudaError_t launch_sparse_attention(const SparseAttnArgs& a, cudaStream_t st) {
  if (a.Lq == 1) return launch_sparse_rows(a, st);
  return a.head_dim == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace h3b
