// packed.cu -- attention over packed sequences of different lengths, and over a key prefix
// that a whole batch shares, for sm_100a (TMA + tcgen05 + TMEM).
//
// One work item is a tile of up to 128 rows of one key/value head: 128 / G consecutive query
// tokens times the G query heads that share that key/value head (row r: token r / G, head
// r % G), so grouped heads load each key tile once and short sequences fill a tile with
// their heads.  Row i of a sequence with Lq queries and Lk keys sees the keys c < limit(i),
//
//   limit(i) = Lk, or with the causal mask min(Lk, i + Lk - Lq + 1) (<= 0: no key),
//
// and the kernel computes, over the 128-key blocks that any row of the tile sees,
//
//   O_i = sum_c 2^(x_ic - m_i) v_c / l_i,  l_i = sum_c 2^(x_ic - m_i),
//   LSE_i = ln 2 (m_i + log2 l_i),         x_ic = scale log2(e) <q_i, k_c>,
//
// in one pass with a running reference m_i.  Blocks that every row of the tile sees in full
// take a step without mask code; the others (the diagonal of a causal mask, the end of a
// sequence) take the masked step, where an unseen key's weight is exactly zero.  V rows past
// a sequence's end are zeroed in shared memory before they are multiplied, so whatever
// memory holds there (another sequence, NaN) adds nothing.
//
// Shared prefix (p.splits > 0): one "sequence" of all query tokens of the batch against the
// prefix keys, cut along the keys into p.splits parts so that few rows still fill the GPU;
// each part stores its normalised O and its LSE (log2 units) in float32, joined later with
// the parts of the sequences' own caches.
//
// Items: one CTA per SM starts per item until the SMs are full; a CTA that finishes loading an
// item asks the hardware for one that has not started (cluster launch control) and goes on
// with it, so the next item's loads and first Q K^T run under the current one's epilogue,
// items are still handed out one by one in grid order, and nothing has to be counted in
// memory.  The K producer decodes items and passes them to the other roles through a ring of
// four in shared memory.
//
// Long key ranges with few tiles (p.spare > 0): tiles are cut along their key blocks into parts
// of about an equal share, at most one per SM in all, counted from the lengths by every CTA
// alike.  A tile of one part is stored as usual, the parts of the others are left like a
// prefix's and joined by packed_join_kernel.
//
// Pipeline and warp roles are those of the block-sparse kernel (attn.cu): three S buffers in
// TMEM next to O, P over its own S, Q K^T and P V issued by two threads, rings of three K
// and two (d = 64: three) V tiles of 128 rows, Q double, eight softmax warps with half a row
// per thread, exponentials against the current reference while the block's maximum is found
// alongside, O rescaled only when a row's maximum grows by more than 2^8.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace lva {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int kSoftmaxWarp0 = 2;
constexpr int kSoftmaxWarps = 8;
constexpr int kVWarp = kSoftmaxWarp0 + kSoftmaxWarps;
constexpr int kPVWarp = kVWarp + 1;
constexpr int kThreads = 32 * (kPVWarp + 1);
constexpr float kRescaleThreshold = 8.0f;
constexpr uint32_t kTmemCols = 512;
constexpr float kLn2 = 0.69314718055994530942f;

// One pair of exponentials in eight on the FMA pipe.  Under a load that holds the card at its
// power limit the MUFU's exponentials cost less than the polynomial's steps: one causal
// sequence of 16,379 tokens took 790 us with one pair in eight, 797 with one in sixteen, 799
// with none, 822 with one in four, 842 and 872 with three in eight and one in three (on one card,
// in turn; 788 to 804 with one in eight on others).
__device__ __forceinline__ constexpr bool poly_pair(int e) { return e % 8 == 7; }

struct PackedParams {
  int num_seqs;
  int kv_heads, group, tok;        // tok = 128 / group query tokens per tile
  int64_t total_q, total_k;
  int64_t o_token, o_head;         // O strides in elements
  const int32_t* cu_q;             // [num_seqs + 1]; unused for the shared prefix
  const int32_t* cu_k;
  int causal;
  float scale_log2;                // scale * log2(e)
  __nv_bfloat16* o;
  float* lse;                      // [Hq, total_q]
  int o_boxes;                     // 16 rows are whole tokens: O has a map with boxes of them
  int splits;                      // 0: packed; > 0: parts of the shared prefix
  int spare, max_items;            // packed in parts: parts there may be beyond one per tile (0: none), items part_o holds
  // Parts of a prefix [splits, kv_heads, total_q, group, D], or of packed tiles [items, 128, D],
  // and their LSE in log2 units
  float* part_o;
  float* part_lse;
  int* err;
};

// A work item: rows [tok0, tok0 + rows / group) of the query tokens, key blocks [j0, j1) of
// the key rows that start at k_row.
struct Item {
  int kvh;
  int64_t part_row0;       // where the tile's first row goes among the parts; -1: to O and LSE
  int tok0, q_end;         // first query token of the tile, end of its sequence
  int k_row, lk;           // first key row of the sequence, its keys
  int lim0;                // limit of the tile's first token, possibly below zero
  int causal;
  int j0, j_full, j1;      // blocks [j0, j_full) are seen in full by every row of the tile
  int live;                // 0: nothing to do (in the ring: no more items)
  // The key block at step t: the masked ones first, so that an item has one step that must
  // find its maximum before its exponentials (the first) instead of two.
  __device__ __forceinline__ int block(int t) const {
    const int masked = j1 - j_full;
    return t < masked ? j_full + t : j0 + t - masked;
  }
};

constexpr int kItemRing = 4;
constexpr int kAhead = 6;
constexpr int kItemReaders = kSoftmaxWarps + 3;   // every warp but the K producer

template <int D>
struct Cfg {
  static constexpr int KST = 3, VST = D == 128 ? 2 : 3, NSB = 3;
  static constexpr int QST = 2;                    // the next item's Q loads during the current one
  static constexpr int Q_BYTES = BM * D * 2;
  static constexpr int KV_BYTES = BN * D * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + QST * Q_BYTES;
  static constexpr int OFF_V = OFF_K + KST * KV_BYTES;
  static constexpr int OFF_BAR = OFF_V + VST * KV_BYTES;
  // q_full, k_full/k_empty, v_full/v_empty, s_full, p_full, o_done, the two final drains,
  // v_tail (the TMA of a V tile whose last rows are zeroed before v_full), q_empty (an item's
  // Q K^T done and its O stored), o_free (its O read), clc (the next item's answer), item_full/item_empty
  static constexpr int B_Q = 0, B_KF = B_Q + QST, B_KE = B_KF + KST, B_VF = B_KE + KST, B_VE = B_VF + VST,
                       B_SF = B_VE + VST, B_P = B_SF + NSB, B_O = B_P + NSB, B_FIN = B_O + NSB,
                       B_FIN_PV = B_FIN + 1, B_VT = B_FIN_PV + 1, B_QE = B_VT + 1, B_OF = B_QE + QST,
                       B_CLC = B_OF + 1, B_IF = B_CLC + 1, B_IE = B_IF + kItemRing, NUM_BARS = B_IE + kItemRing;
  static constexpr int OFF_MISC = (OFF_BAR + NUM_BARS * 8 + 15) / 16 * 16;
  static constexpr int OFF_CLC = OFF_MISC + 16;
  static constexpr int OFF_ITEMS = OFF_CLC + 16;
  static constexpr int SMEM_RAW = OFF_ITEMS + kItemRing * int(sizeof(Item));
  // at least 120 KB: one CTA, and one 512-column TMEM allocation, per SM
  static constexpr int SMEM_BYTES = SMEM_RAW > 120 * 1024 ? SMEM_RAW : 120 * 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t TM_S = 0, TM_O = 384;
  static constexpr uint32_t IDESC_QK = idesc_bf16_f32(BM, BN, 0, 0);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(BM, D, 0, 1);
};

// Largest s with start(s) <= slot, start(s) = cu[s] / tok + s, found by the whole warp, 32
// probes a round; -1 when there is none.  start is strictly increasing for a valid cu, and
// sequence s needs at most start(s + 1) - start(s) tiles; whatever cu holds, the answer stays
// in [-1, n).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int n, int tok, uint32_t slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, cnt = n;
  for (;;) {
    const int step = (cnt + 31) / 32;
    const int idx = lo + lane * step;
    bool le = false;
    if (lane * int64_t(step) < cnt) {
      const int32_t c = __ldg(cu + idx);
      le = c < 0 || uint32_t(c) / uint32_t(tok) + uint32_t(idx) <= slot;
    }
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    if (k == 0) return lo == 0 ? -1 : lo;
    const int end = lo + cnt;
    lo += (k - 1) * step;
    if (step == 1) return lo;
    cnt = step < end - lo ? step : end - lo;
  }
}

// A sequence's lengths; one whose entries fall or leave the buffers counts as empty.
struct Sequence { int a, lq, ka, lk; };
__device__ __forceinline__ Sequence sequence_at(const PackedParams& p, int s) {
  const int a = __ldg(p.cu_q + s), b = __ldg(p.cu_q + s + 1);
  const int ka = __ldg(p.cu_k + s), kb = __ldg(p.cu_k + s + 1);
  const bool good = a >= 0 && a <= b && b <= p.total_q && ka >= 0 && ka <= kb && kb <= p.total_k;
  return good ? Sequence{a, b - a, ka, kb - ka} : Sequence{0, 0, 0, 0};
}
__device__ __forceinline__ int blocks_of(int keys) { return int((uint32_t(keys) + BN - 1) / BN); }
__device__ __forceinline__ int tiles_of(const PackedParams& p, int lq) { return int((uint32_t(lq) + p.tok - 1) / uint32_t(p.tok)); }

// Key blocks per part of a packed tile (whole warp; the same in every CTA of a call): all tiles'
// blocks, as of their sequences' last tiles, divided by `spare`, so that the parts are at most
// `spare` more than the tiles; at least kLeastPart, which a part's start and end cost, and
// not more than kMostParts parts.
constexpr int kLeastPart = 6;
constexpr int kMostParts = 64;
__device__ __forceinline__ int part_size(const PackedParams& p) {
  unsigned long long work = 0;
  int longest = 0;
  for (int s = threadIdx.x & 31; s < p.num_seqs; s += 32) {
    const Sequence q = sequence_at(p, s);
    const int blocks = blocks_of(q.lk);
    if (q.lq > 0) {
      work += uint64_t(tiles_of(p, q.lq)) * uint32_t(blocks);
      longest = blocks > longest ? blocks : longest;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
  longest = __reduce_max_sync(0xffffffffu, longest);
  work = (work * uint32_t(p.kv_heads) + uint32_t(p.spare) - 1) / uint32_t(p.spare);
  const int even = work < (1u << 24) ? int(work) : 1 << 24, least = (longest + kMostParts - 1) / kMostParts;
  const int size = even > least ? even : least;
  return size > kLeastPart ? size : kLeastPart;
}
// Parts that each tile of a sequence is given in the list (its longest tile's; a causal tile of
// fewer blocks leaves the last ones empty).
__device__ __forceinline__ int parts_for(int blocks, int size) {
  const int parts = int((uint32_t(blocks) + uint32_t(size) - 1) / uint32_t(size));
  return parts > 1 ? parts : 1;
}

// Tile i0 .. i0 + tok - 1 of a sequence: its rows and key blocks.
__device__ __forceinline__ void set_tile(const PackedParams& p, const Sequence& q, int i0, Item& w) {
  const int last = (i0 + p.tok < q.lq ? i0 + p.tok : q.lq) - 1;
  w.tok0 = q.a + i0;
  w.q_end = q.a + q.lq;
  w.k_row = q.ka;
  w.lk = q.lk;
  w.causal = p.causal;
  w.lim0 = p.causal ? i0 + 1 + (q.lk - q.lq) : q.lk;
  int lim_last = p.causal ? last + 1 + (q.lk - q.lq) : q.lk;
  lim_last = lim_last < 0 ? 0 : lim_last;          // at most lk: last < lq
  const int lim_first = w.lim0 < 0 ? 0 : w.lim0;
  w.j0 = 0;
  w.j1 = blocks_of(lim_last);
  w.j_full = lim_first / BN;
  w.part_row0 = -1;
  w.live = 1;
}
// Part `part` of `parts` of an item's blocks.
__device__ __forceinline__ void cut(Item& w, int part, int parts) {
  const int full = w.j_full;
  const uint32_t n = uint32_t(w.j1);
  w.j0 = int(n * uint32_t(part) / uint32_t(parts));            // parts <= 64, blocks < 2^25
  w.j1 = int(n * uint32_t(part + 1) / uint32_t(parts));
  w.j_full = w.j1 < full ? w.j1 : full;
  if (w.j_full < w.j0) w.j_full = w.j0;
}

// All item arithmetic is in 32 bits: tokens, tiles and the grid stay below 2^31.  live is 0
// where there is nothing to do; `size` is used with p.spare.
template <bool PARTS>
__device__ __forceinline__ Item item_at(const PackedParams& p, uint32_t bid, int size) {
  Item w;
  w.live = 0;
  uint32_t rest = bid / uint32_t(p.kv_heads);
  w.kvh = int(bid - rest * p.kv_heads);
  if (PARTS && p.splits > 0) {
    // Shared prefix: parts fastest after the head, so that the parts of a tile run together.
    const uint32_t tile = rest / uint32_t(p.splits);
    const int split = int(rest - tile * p.splits);
    w.tok0 = int(tile * p.tok);
    w.q_end = int(p.total_q);
    w.k_row = 0;
    w.lk = int(p.total_k);
    w.lim0 = int(p.total_k);
    w.causal = 0;
    w.j1 = blocks_of(int(p.total_k));
    w.j_full = int(p.total_k / BN);
    cut(w, split, p.splits);
    w.part_row0 = ((int64_t(split) * p.kv_heads + w.kvh) * p.total_q + w.tok0) * p.group;
    w.live = w.tok0 < w.q_end ? 1 : 0;
    return w;
  }
  if (PARTS && p.spare > 0) {
    // The list: sequence by sequence, the last tile first, its parts in order, heads fastest.
    const int lane = threadIdx.x & 31;
    for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
      Sequence q{0, 0, 0, 0};
      if (s0 + lane < p.num_seqs) q = sequence_at(p, s0 + lane);
      const int parts = parts_for(blocks_of(q.lk), size);
      const uint32_t own = uint32_t(tiles_of(p, q.lq)) * parts;
      uint32_t sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const unsigned past = __ballot_sync(0xffffffffu, sum > rest);
      if (past == 0) {
        rest -= __shfl_sync(0xffffffffu, sum, 31);
        continue;
      }
      const int l = __ffs(past) - 1;
      const Sequence it{__shfl_sync(0xffffffffu, q.a, l), __shfl_sync(0xffffffffu, q.lq, l),
                        __shfl_sync(0xffffffffu, q.ka, l), __shfl_sync(0xffffffffu, q.lk, l)};
      const int given = __shfl_sync(0xffffffffu, parts, l);
      const uint32_t in = rest - __shfl_sync(0xffffffffu, sum - own, l);
      const uint32_t back = in / uint32_t(given);
      const int part = int(in - back * given);
      set_tile(p, it, int(tiles_of(p, it.lq) - 1 - back) * p.tok, w);
      const int mine = parts_for(w.j1, size);
      if (part >= mine) w.live = 0;
      else if (mine > 1) {
        cut(w, part, mine);
        w.part_row0 = int64_t(bid) * BM;
      }
      return w;
    }
    return w;
  }
  // Packed: the last tiles of the last sequence first (a causal tile's work grows with its
  // place, so the shortest tiles fill the tail), the heads of a tile next to one another.  The
  // lengths play no part: six sequences of 60 to 8,000 keys, 1 to 511 of them new, take 62 to 98 us
  // by their order, 66 with the longest last and 98 with it first.
  const uint32_t slot = uint32_t(p.total_q) / uint32_t(p.tok) + uint32_t(p.num_seqs) - 1u - rest;
  const int s = find_sequence(p.cu_q, p.num_seqs, p.tok, slot);
  if (s < 0) return w;
  const Sequence q = sequence_at(p, s);
  const uint32_t first_slot = uint32_t(q.a) / uint32_t(p.tok) + uint32_t(s);
  // first token of the tile in its sequence; slots before the sequence's or past its tiles
  const int64_t i0 = (int64_t(slot) - int64_t(first_slot)) * p.tok;
  if (i0 < 0 || i0 >= q.lq) return w;
  set_tile(p, q, int(i0), w);
  return w;
}

// O *= alpha for this thread's half row, out of line (rare).
template <int DH>
__device__ __noinline__ void rescale_o(uint32_t taddr, float alpha) {
#pragma unroll 1
  for (int q = 0; q < DH / 32; ++q) {
    uint32_t ov[32];
    tmem_ld_16x2_32<DH>(taddr + q * 32, ov);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
    tmem_st_16x2_32<DH>(taddr + q * 32, ov);
  }
}

// PARTS: the call may leave parts to a join (a shared prefix, or tiles cut along the keys); the
// form without them keeps that code out of the loops (it cost them 10 %).
template <int D, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1) packed_attn_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const PackedParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s_base = smem_u32(smem);
  if (s_base & 1023u) {                           // never expected; checked rather than assumed
    if (threadIdx.x == 0) report_fault(p.err, 4, 1023);
    return;
  }
  // The first CTA checks both length lists: a list that falls or leaves its buffer is
  // reported, and the sequences it spoils are skipped where they are met.
  if (blockIdx.x == 0 && (!PARTS || p.splits == 0)) {
    for (int s = threadIdx.x; s < p.num_seqs; s += kThreads) {
      const int64_t a = __ldg(p.cu_q + s), b = __ldg(p.cu_q + s + 1);
      const int64_t ka = __ldg(p.cu_k + s), kb = __ldg(p.cu_k + s + 1);
      if (!(a >= 0 && a <= b && b <= p.total_q && ka >= 0 && ka <= kb && kb <= p.total_k))
        report_fault(p.err, 1, s);
    }
  }
  const uint32_t sQ = s_base + C::OFF_Q, sK = s_base + C::OFF_K, sV = s_base + C::OFF_V;
  const uint32_t bar0 = s_base + C::OFF_BAR;
  auto bar_q = [&](int s) { return bar0 + 8u * (C::B_Q + s); };
  auto bar_k_full = [&](int s) { return bar0 + 8u * (C::B_KF + s); };
  auto bar_k_empty = [&](int s) { return bar0 + 8u * (C::B_KE + s); };
  auto bar_v_full = [&](int s) { return bar0 + 8u * (C::B_VF + s); };
  auto bar_v_empty = [&](int s) { return bar0 + 8u * (C::B_VE + s); };
  auto bar_s_full = [&](int b) { return bar0 + 8u * (C::B_SF + b); };
  auto bar_p_full = [&](int b) { return bar0 + 8u * (C::B_P + b); };
  auto bar_o_done = [&](int b) { return bar0 + 8u * (C::B_O + b); };
  const uint32_t bar_final = bar0 + 8u * C::B_FIN;
  const uint32_t bar_final_pv = bar0 + 8u * C::B_FIN_PV;
  const uint32_t bar_v_tail = bar0 + 8u * C::B_VT;
  auto bar_q_empty = [&](int s) { return bar0 + 8u * (C::B_QE + s); };
  const uint32_t bar_o_free = bar0 + 8u * C::B_OF;
  const uint32_t bar_clc = bar0 + 8u * C::B_CLC;
  auto bar_item_full = [&](int s) { return bar0 + 8u * (C::B_IF + s); };
  auto bar_item_empty = [&](int s) { return bar0 + 8u * (C::B_IE + s); };
  Item* ring = reinterpret_cast<Item*>(smem + C::OFF_ITEMS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* never = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);  // stays zero
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::QST; ++s) { mbar_init(bar_q(s), 1); mbar_init(bar_q_empty(s), 1 + kSoftmaxWarps); }
    for (int s = 0; s < C::KST; ++s) { mbar_init(bar_k_full(s), 1); mbar_init(bar_k_empty(s), 1); }
    for (int s = 0; s < C::VST; ++s) { mbar_init(bar_v_full(s), 1); mbar_init(bar_v_empty(s), 1); }
    for (int b = 0; b < C::NSB; ++b) {
      mbar_init(bar_s_full(b), 1);
      mbar_init(bar_p_full(b), kSoftmaxWarps);
      mbar_init(bar_o_done(b), 1);
    }
    mbar_init(bar_final, 1);
    mbar_init(bar_final_pv, 1);
    mbar_init(bar_v_tail, 1);
    mbar_init(bar_o_free, kSoftmaxWarps);
    mbar_init(bar_clc, 1);
    for (int s = 0; s < kItemRing; ++s) { mbar_init(bar_item_full(s), 1); mbar_init(bar_item_empty(s), kItemReaders); }
    *abort_flag = 0;
    *never = 0;
    mbar_fence_init();
  }
  if (warp == 1) { tmem_alloc(smem_u32(tmem_slot), kTmemCols); tmem_relinquish(); }
  Item w0;                                        // the first item, found while the CTA is set up
  if (warp == 0) w0 = item_at<PARTS>(p, blockIdx.x, PARTS && p.spare > 0 ? part_size(p) : 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (PARTS) launch_dependents();                 // the join gets ready
  const uint32_t tmem = *tmem_slot;

  // The next item of a role warp (every warp but the K producer): 1, or 0 after the last one,
  // or -1 when the wait gave up.  Pipeline positions T count key blocks over all items of this
  // CTA, so ring slots, S buffers and their phases continue from one item to the next.
  uint32_t ni = 0;
  auto next_item = [&](Item& w) -> int {
    const int s = int(ni % kItemRing);
    if (!__all_sync(0xffffffffu, mbar_wait_sleep(bar_item_full(s), (ni / kItemRing) & 1, abort_flag))) return -1;
    w = ring[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_item_empty(s));
    ++ni;
    return w.live;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ items; TMA producer: Q, K
    if (lane == 0) { tma_prefetch_desc(&tm_q); tma_prefetch_desc(&tm_k); }
    const uint32_t resp = s_base + C::OFF_CLC;
    uint32_t T = 0, answers = 0;
    int nq = 0;
    bool ok = true;
    int64_t bid = blockIdx.x;                      // -1: no more items
    Item w;
    while (ok) {
      w.live = -1;
      if (bid == blockIdx.x) w = w0;
      else if (!PARTS && bid >= 0) w = item_at<PARTS>(p, uint32_t(bid), 0);
      if (w.live < 0) {                              // no more items: the end mark
        bid = -1;
        w.live = 0;
      }
      const int n = w.live ? w.j1 - w.j0 : 0;
      int64_t next = -1;
      if (w.live || bid < 0) {
        if (lane == 0) {
          const int s = int(ni % kItemRing);
          ok = ni < kItemRing || mbar_wait_sleep(bar_item_empty(s), ((ni / kItemRing) - 1) & 1, abort_flag);
          if (ok) {
            ring[s] = w;
            mbar_arrive(bar_item_full(s));
          }
        }
        ++ni;
      }
      if (bid < 0) { ok = __shfl_sync(0xffffffffu, ok, 0); break; }
      // The next item is asked for kAhead blocks before this one's end, which hides the answer's
      // latency; asked for earlier, a CTA with a long item would hold on to one that others
      // are free to take (a batch of short and long sequences took 97 us instead of 78).
      if (lane == 0 && ok) {
        const int t_ask = n > kAhead ? n - kAhead : 0;
        bool asked = false;
        auto ask = [&] {
          // Parts are one to a CTA.  Those of packed tiles all run at once; a prefix's find SMs
          // bit by bit, as the caches' kernel ends, and CTAs that started first would take two
          // (a batch of 32: 48 us instead of 36).
          if (PARTS) return;
          mbar_arrive_expect_tx(bar_clc, 16);
          clc_try_cancel(resp, bar_clc);
          asked = true;
        };
        if (n == 0) ask();
        for (int t = 0; ok && t < n; ++t, ++T) {
          if (t == t_ask) ask();
          if (t == 0) {
            // Q's buffer is free once the item before the previous one has been stored.
            const int s = nq % C::QST;
            ok = nq < C::QST || mbar_wait_sleep(bar_q_empty(s), ((nq / C::QST) - 1) & 1, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(bar_q(s), uint32_t(p.group * p.tok * D * 2));
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sQ + s * C::Q_BYTES + c * BM * 128, &tm_q, c * 64, w.kvh * p.group, w.tok0, bar_q(s));
            ++nq;
          }
          const int s = int(T % C::KST);
          if (T >= uint32_t(C::KST) && !mbar_wait_sleep(bar_k_empty(s), int((T / C::KST) - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar_k_full(s), C::KV_BYTES);
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sK + s * C::KV_BYTES + c * BN * 128, &tm_k, c * 64, w.kvh,
                        w.k_row + w.block(t) * BN, bar_k_full(s));
        }
        // The answer is waited for in every case: it is written into this CTA's memory.
        if (asked) {
          if (mbar_wait_sleep(bar_clc, answers & 1, never)) {
            next = clc_answer(resp);
            fence_proxy_async_smem();              // read before the next answer is written
          } else {
            ok = false;
          }
          ++answers;
        }
      }
      bid = __shfl_sync(0xffffffffu, next, 0);
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      if (!ok) { *abort_flag = 1; report_fault(p.err, 5, 21); }
      if (*abort_flag) {                           // every load in flight lands before the CTA ends
        for (uint32_t u = T > uint32_t(C::KST) ? T - C::KST : 0; u < T; ++u)
          mbar_wait(bar_k_full(int(u % C::KST)), int(u / C::KST) & 1, never);
        for (int u = nq > C::QST ? nq - C::QST : 0; u < nq; ++u) mbar_wait(bar_q(u % C::QST), (u / C::QST) & 1, never);
      }
    }
  } else if (warp == kVWarp) {
    // ------------------------------------------------------------ TMA producer: V
    if (lane == 0) tma_prefetch_desc(&tm_v);
    uint32_t T = 0, tails = 0;
    int got = 1;
    Item w;
    while ((got = next_item(w)) == 1) {
      const int n = w.j1 - w.j0;
      bool ok = true;
      for (int t = 0; ok && t < n; ++t) {
        const int s = int(T % C::VST);
        const int j = w.block(t);
        const int left = w.lk - j * BN;                          // keys of the sequence from here on
        const bool tail = left < BN;                             // at most one block of an item
        if (lane == 0) {
          if (T >= uint32_t(C::VST) && !mbar_wait_sleep(bar_v_empty(s), int((T / C::VST) - 1) & 1, abort_flag)) {
            ok = false;
          } else {
            const uint32_t bar = tail ? bar_v_tail : bar_v_full(s);
            mbar_arrive_expect_tx(bar, C::KV_BYTES);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sV + s * C::KV_BYTES + c * BN * 128, &tm_v, c * 64, w.kvh,
                          w.k_row + j * BN, bar);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        ++T;
        if (tail) {
          // Rows past the sequence's end hold other sequences' values, or anything: zeroed,
          // because their weight of zero times NaN or infinity would not be zero.
          ok = __all_sync(0xffffffffu, mbar_wait(bar_v_tail, tails & 1, never));
          ++tails;
          if (!ok) break;
          for (int c = 0; c < D / 64; ++c) {
            uint8_t* rows = smem + C::OFF_V + s * C::KV_BYTES + c * BN * 128;
            for (int x = left * 8 + lane; x < BN * 8; x += 32)
              reinterpret_cast<uint4*>(rows)[x] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_v_full(s));
        }
      }
      if (!ok) { got = -1; break; }
    }
    if (got < 0 && lane == 0) {
      *abort_flag = 1;
      report_fault(p.err, 5, 22);
      for (uint32_t u = T > uint32_t(C::VST) ? T - C::VST : 0; u < T; ++u)
        mbar_wait(bar_v_full(int(u % C::VST)), int(u / C::VST) & 1, never);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer: S = Q K^T
    const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024);
    const uint64_t k_desc = smem_desc_sw128(sK, 16, 1024);
    uint32_t T = 0;
    int nq = 0, got = 1;
    Item w;
    while ((got = next_item(w)) == 1) {
      const int n = w.j1 - w.j0;
      if (n == 0) continue;
      bool ok = true;
      if (lane == 0) {
        ok = mbar_wait_sleep(bar_q(nq % C::QST), (nq / C::QST) & 1, abort_flag);
        const uint64_t qs = q_desc + uint64_t(((nq % C::QST) * C::Q_BYTES) >> 4);
        for (int t = 0; ok && t < n; ++t, ++T) {
          const int s = int(T % C::KST), b = int(T % C::NSB);
          if (!mbar_wait_sleep(bar_k_full(s), int(T / C::KST) & 1, abort_flag)) { ok = false; break; }
          // S_b is free again once the P that went over it has been multiplied
          if (T >= uint32_t(C::NSB) && !mbar_wait_sleep(bar_o_done(b), int((T / C::NSB) - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ks = k_desc + uint64_t((s * C::KV_BYTES) >> 4);
          const uint32_t s_tm = tmem + C::TM_S + 128 * b;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_f16_ss(s_tm, qs + uint64_t(((kk / 4) * BM * 128 + (kk % 4) * 32) >> 4),
                        ks + uint64_t(((kk / 4) * BN * 128 + (kk % 4) * 32) >> 4), C::IDESC_QK, kk > 0 ? 1u : 0u);
          umma_commit(bar_s_full(b));
          umma_commit(bar_k_empty(s));
        }
        if (ok) umma_commit(bar_q_empty(nq % C::QST));   // this Q may be replaced
      }
      ++nq;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) { got = -1; break; }
    }
    if (lane == 0) {
      if (got < 0) { *abort_flag = 1; report_fault(p.err, 5, 24); }
      umma_commit(bar_final);                      // every MMA of this thread before TMEM is released
      mbar_wait(bar_final, 0, never);
    }
  } else if (warp == kPVWarp) {
    // ------------------------------------------------------------ MMA issuer: O += P V
    const uint64_t v_desc = smem_desc_sw128(sV, BN * 128, 1024);
    uint32_t T = 0;
    int nq = 0, got = 1;
    Item w;
    while ((got = next_item(w)) == 1) {
      const int n = w.j1 - w.j0;
      if (n == 0) continue;
      bool ok = true;
      if (lane == 0) {
        // an item's first P V overwrites O: the previous item's must have been read
        if (nq > 0) ok = mbar_wait_sleep(bar_o_free, (nq - 1) & 1, abort_flag);
        for (int t = 0; ok && t < n; ++t, ++T) {
          const int s = int(T % C::VST), b = int(T % C::NSB);
          if (!mbar_wait_sleep(bar_p_full(b), int(T / C::NSB) & 1, abort_flag)) { ok = false; break; }
          if (!mbar_wait_sleep(bar_v_full(s), int(T / C::VST) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint64_t vs = v_desc + uint64_t((s * C::KV_BYTES) >> 4);
          const uint32_t p_tm = tmem + C::TM_S + 128 * b;
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            umma_f16_ts(tmem + C::TM_O, p_tm + kk * 8, vs + uint64_t((kk * 16 * 128) >> 4), C::IDESC_PV,
                        (t > 0 || kk > 0) ? 1u : 0u);
          umma_commit(bar_v_empty(s));
          umma_commit(bar_o_done(b));
        }
      }
      ++nq;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) { got = -1; break; }
    }
    if (lane == 0) {
      if (got < 0) { *abort_flag = 1; report_fault(p.err, 5, 25); }
      umma_commit(bar_final_pv);
      mbar_wait(bar_final_pv, 0, never);
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    // Thread = (row, column half): lane t and t + 16 hold the halves of one row.
    constexpr int HALF = BN / 2, DH = D / 2;
    const int quarter = warp & 3, sel = (warp - kSoftmaxWarp0) >> 2;
    const int hf = lane >> 4;
    const int row = quarter * 32 + sel * 16 + (lane & 15);
    const uint32_t lane_off = uint32_t(quarter * 32 + sel * 16) << 16;
    const float c = p.scale_log2;
    const int tok_in = row / p.group, head_in = row - tok_in * p.group;
    const bool row_used = row < p.tok * p.group;
    uint32_t T = 0;
    int nq = 0;
    bool q_pending = false;                        // O of item nq - 1 may still be read from its Q buffer
    auto release_q = [&] {
      if (q_pending) {
        bulk_wait_read();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_q_empty((nq - 1) % C::QST));
        q_pending = false;
      }
    };
    Item w;
    int got = next_item(w);
    while (got == 1) {
    const int n = w.j1 - w.j0;
    const int64_t token = int64_t(w.tok0) + tok_in;
    const bool store = row_used && token < w.q_end;
    // Keys this row sees, counted from the sequence's first key (a row past the sequence's end
    // counts on past them; it is not stored).
    const int limit = w.causal ? w.lim0 + (store ? tok_in : 0) : w.lim0;
    const bool sees = store && limit > 0;
    bool ok = true;
    float m_ref = -INFINITY;                       // reference max in log2 units
    float l = 0.f;                                 // this half's share of the row sum

    // One key block t, any row's view of it; false when a wait gives up.  An unseen key's weight
    // is zero (the MUFU's 2^-inf; the polynomial would give 2^-125).
    auto step = [&](int t) -> bool {
      const int b = int(T % C::NSB);
      if (!__all_sync(0xffffffffu, mbar_wait(bar_s_full(b), int(T / C::NSB) & 1, abort_flag))) return false;
      tc_fence_after();
      uint32_t sr[HALF];
#pragma unroll
      for (int q = 0; q < HALF / 32; ++q)
        tmem_ld_16x2_32<HALF>(tmem + lane_off + C::TM_S + 128 * b + q * 32,
                              *reinterpret_cast<uint32_t(*)[32]>(sr + q * 32));
      tmem_wait_ld();
      {
        const int left = limit - (w.block(t) * BN + hf * HALF);
        const int vis = left > HALF ? HALF : left < 0 ? 0 : left;
        const uint32_t lo = vis >= 32 ? ~0u : (1u << vis) - 1u, hi = vis >= 64 ? ~0u : vis <= 32 ? 0u : (1u << (vis - 32)) - 1u;
#pragma unroll
        for (int e = 0; e < HALF; ++e)
          if (!(((e < 32 ? lo : hi) >> (e & 31)) & 1u)) sr[e] = __float_as_uint(-INFINITY);
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < HALF / 2; ++e)
        m4[e & 3] = fmax3(m4[e & 3], __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
      float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float m_old = m_ref;
      if (mx > m_ref + kRescaleThreshold || m_ref == -INFINITY) m_ref = fmaxf(mx, m_ref);
      const float alpha = (m_old == m_ref) ? 1.f : ex2_approx(m_old - m_ref);
      const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
      __syncwarp();                                // every lane's S is loaded: P may go over it
      const uint32_t p_tm = tmem + lane_off + C::TM_S + 128 * b;
      uint32_t pk[HALF / 2];
      const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(-m_use, -m_use);
      uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
      for (int e = 0; e < HALF / 2; ++e) {
        const uint64_t x2 = f2_fma(f2_pack_bits(sr[2 * e], sr[2 * e + 1]), c2, nm2);
        float x0, x1;
        f2_unpack(x2, x0, x1);
        const uint64_t p2 = f2_pack(ex2_approx(x0), ex2_approx(x1));
        acc[e & 1] = f2_add(acc[e & 1], p2);
        float p0, p1;
        f2_unpack(p2, p0, p1);
        pk[e] = pack_bf16x2(p0, p1);               // P in bf16: the MMA's operand type
        if (e == 15) tmem_st_16x2_16<HALF / 2>(p_tm, *reinterpret_cast<const uint32_t(*)[16]>(pk));
      }
      tmem_st_16x2_16<HALF / 2>(p_tm + 16, *reinterpret_cast<const uint32_t(*)[16]>(pk + 16));
      float a0, a1, b0, b1;
      f2_unpack(acc[0], a0, a1);
      f2_unpack(acc[1], b0, b1);
      l = l * alpha + ((a0 + a1) + (b0 + b1));
      if (t >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar_o_done(int((T - 1) % C::NSB)), int((T - 1) / C::NSB) & 1, abort_flag)))
          return false;
        tc_fence_after();
        rescale_o<DH>(tmem + lane_off + C::TM_O, alpha);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p_full(b));
      return true;
    };

    // A block that every row sees, after the first: exponentials against the current
    // reference while the block max is found alongside; given up (2) before anything is
    // stored when a row's max outgrows its reference by 2^8, or is NaN: the polynomial's clamp
    // drops a NaN, step() lets it through.
    auto step_spec = [&]() -> int {
      const int b = int(T % C::NSB);
      if (!__all_sync(0xffffffffu, mbar_wait(bar_s_full(b), int(T / C::NSB) & 1, abort_flag))) return 0;
      tc_fence_after();
      uint32_t sr[HALF];
#pragma unroll
      for (int q = 0; q < HALF / 32; ++q)
        tmem_ld_16x2_32<HALF>(tmem + lane_off + C::TM_S + 128 * b + q * 32,
                              *reinterpret_cast<uint32_t(*)[32]>(sr + q * 32));
      tmem_wait_ld();
      const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(-m_ref, -m_ref);
      uint64_t acc[2] = {0ull, 0ull};
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      uint32_t pk[HALF / 2];
#pragma unroll
      for (int e = 0; e < HALF / 2; ++e) {
        m4[e & 3] = fmax3_nan(m4[e & 3], __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
        const uint64_t x2 = f2_fma(f2_pack_bits(sr[2 * e], sr[2 * e + 1]), c2, nm2);
        uint64_t p2;
        if (poly_pair(e)) {
          p2 = exp2_poly_f2(x2);
        } else {
          float x0, x1;
          f2_unpack(x2, x0, x1);
          p2 = f2_pack(ex2_approx(x0), ex2_approx(x1));
        }
        acc[e & 1] = f2_add(acc[e & 1], p2);
        float p0, p1;
        f2_unpack(p2, p0, p1);
        pk[e] = pack_bf16x2(p0, p1);
      }
      float mx = fmax3_nan(fmax3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]) * c;
      const float far = __shfl_xor_sync(0xffffffffu, mx, 16);
      mx = fmax3_nan(mx, far, far);
      if (__any_sync(0xffffffffu, sees && (!(mx <= m_ref + kRescaleThreshold) || m_ref == -INFINITY))) return 2;
      tmem_st_16x2_32<HALF / 2>(tmem + lane_off + C::TM_S + 128 * b, *reinterpret_cast<const uint32_t(*)[32]>(pk));
      tmem_wait_st();
      float a0, a1, b0, b1;
      f2_unpack(acc[0], a0, a1);
      f2_unpack(acc[1], b0, b1);
      l = l + ((a0 + a1) + (b0 + b1));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p_full(b));
      return 1;
    };

    const int n_masked = w.j1 - w.j_full;
    int t = 0;
    const bool idle = !__any_sync(0xffffffffu, store);
    if (idle) {
      // No row of this warp is stored (a tile of few rows): its P may hold anything.
      for (; ok && t < n; ++t, ++T) {
        const int b = int(T % C::NSB);
        ok = __all_sync(0xffffffffu, mbar_wait(bar_s_full(b), int(T / C::NSB) & 1, abort_flag));
        if (ok && lane == 0) mbar_arrive(bar_p_full(b));
      }
    }
    for (; ok && t < n_masked; ++t, ++T) ok = step(t);
    release_q();                                   // the previous item's buffer, by now stored
    for (; ok && t < n; ++t, ++T) {
      int r = 2;
      if (t > 0) r = step_spec();
      if (r == 0) ok = false;
      else if (r == 2) ok = step(t);
    }

    // ---------------------------------------------------------- epilogue
    // The next item is read while the last P V runs.
    Item nw;
    const int next = ok ? next_item(nw) : -1;
    if (ok && n > 0) {
      const uint32_t u = T - 1;
      ok = __all_sync(0xffffffffu, mbar_wait(bar_o_done(int(u % C::NSB)), int(u / C::NSB) & 1, abort_flag));
      tc_fence_after();
    }
    if (!ok) { got = -1; break; }
    const float l_row = l + __shfl_xor_sync(0xffffffffu, l, 16);
    const bool none = !sees || l_row == 0.f;       // a NaN sum goes through as NaN
    const float inv_l = none ? 0.f : __fdividef(1.f, l_row);
    const int head = w.kvh * p.group + head_in;
    const bool partial = PARTS && w.part_row0 >= 0;
    const int64_t part_row = w.part_row0 + row;
    // Rows go out through this item's Q buffer (its Q K^T is done), a warp's 16 rows in the tensor
    // maps' 128-byte swizzle, so staging meets no bank conflict.  When all 16 are rows of the
    // sequence and whole tokens (the group divides 16) one lane stores them as a box per 64
    // columns, asynchronously: an item's epilogue 2,900 -> 1,000 cycles against stores of half
    // rows from registers.  (A copy per row, issued by 32 lanes, took 2,500 cycles to issue.)
    constexpr int UNITS = D / 8, HU = UNITS / 2;    // 16-byte units of a row, of a half row
    const int r16 = lane & 15;
    const uint32_t stage_off = C::OFF_Q + (nq % C::QST) * C::Q_BYTES + (warp - kSoftmaxWarp0) * 16 * D * 2;
    if (n > 0) {
#pragma unroll 1
      for (int q = 0; q < DH / 32; ++q) {
        uint32_t ov[32];
        tmem_ld_16x2_32<DH>(tmem + lane_off + C::TM_O + q * 32, ov);
        tmem_wait_ld();
        if (q == DH / 32 - 1) {
          // O is in registers: the next item's first P V may overwrite it.
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_o_free);
        }
        if (partial) {
          // 64 columns (32 of each half) of the warp's rows as floats, through the same 4 KB
          // (d = 64: half of it a time): stores of whole 128-byte pieces.
          constexpr int COLS = D == 128 ? 32 : 16;
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += COLS) {
#pragma unroll
            for (int u = 0; u < COLS / 4; ++u) {
              float4 f;
              f.x = none ? 0.f : __uint_as_float(ov[c0 + 4 * u]) * inv_l;
              f.y = none ? 0.f : __uint_as_float(ov[c0 + 4 * u + 1]) * inv_l;
              f.z = none ? 0.f : __uint_as_float(ov[c0 + 4 * u + 2]) * inv_l;
              f.w = none ? 0.f : __uint_as_float(ov[c0 + 4 * u + 3]) * inv_l;
              const int unit = hf * (COLS / 4) + u;
              *reinterpret_cast<float4*>(smem + stage_off + r16 * (COLS * 8) + ((unit ^ (r16 & (COLS / 4 - 1))) << 4)) = f;
            }
            __syncwarp();
            constexpr int RU = COLS / 2, RPI = 32 / RU;          // units a row, rows an instruction
            const int unit = lane % RU;
            const int col = (unit / (RU / 2)) * DH + q * 32 + c0 + (unit % (RU / 2)) * 4;
#pragma unroll 1
            for (int r0 = 0; r0 < 16; r0 += RPI) {
              const int r = r0 + lane / RU;
              const int64_t at = __shfl_sync(0xffffffffu, store ? part_row : int64_t(-1), r);
              const float4 f = *reinterpret_cast<const float4*>(smem + stage_off + r * (COLS * 8) + ((unit ^ (r & (COLS / 4 - 1))) << 4));
              if (at >= 0) *reinterpret_cast<float4*>(p.part_o + at * D + col) = f;
            }
            __syncwarp();
          }
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = none ? 0u : pack_bf16x2(__uint_as_float(ov[8 * u + 2 * e]) * inv_l, __uint_as_float(ov[8 * u + 2 * e + 1]) * inv_l);
            const int unit = hf * HU + q * 4 + u;
            *reinterpret_cast<uint4*>(smem + stage_off + (unit / 8) * 2048 + r16 * 128 + (((unit ^ r16) & 7) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      }
      if (!partial) {
        if (__all_sync(0xffffffffu, store) && p.o_boxes) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            for (int c64 = 0; c64 < D / 64; ++c64)
              tma_store_3d(&tm_o, s_base + stage_off + c64 * 2048, c64 * 64, w.kvh * p.group, int32_t(token));
            bulk_commit();
          }
        } else {
          __syncwarp();
          const int64_t off = store ? token * p.o_token + int64_t(head) * p.o_head : int64_t(-1);
          const int unit = lane % UNITS;
#pragma unroll 1
          for (int r0 = 0; r0 < 16; r0 += 32 / UNITS) {
            const int r = r0 + lane / UNITS;
            const int64_t at = __shfl_sync(0xffffffffu, off, r);
            const uint4 v = *reinterpret_cast<const uint4*>(smem + stage_off + (unit / 8) * 2048 + r * 128 + (((unit ^ r) & 7) << 4));
            if (at >= 0) *reinterpret_cast<uint4*>(p.o + at + unit * 8) = v;
          }
          fence_proxy_async_smem();                // read before the buffer's next TMA write
        }
      } else {
        fence_proxy_async_smem();
      }
      ++nq;
      q_pending = true;
    } else if (store && !partial) {
      // No key for any row: O = 0 (this item has no Q buffer; a part of a prefix has keys).
      uint4* dst = reinterpret_cast<uint4*>(p.o + token * p.o_token + int64_t(head) * p.o_head + hf * DH);
#pragma unroll 1
      for (int e = 0; e < DH / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (store && hf == 0) {
      const float lse2 = none ? -INFINITY : m_ref + __log2f(l_row);
      if (partial) p.part_lse[part_row] = lse2;
      else p.lse[int64_t(head) * p.total_q + token] = lse2 * kLn2;
    }
    __syncwarp();                                  // the next item's loads are the whole warp's
    w = nw;
    got = next;
    }
    bulk_wait_read();                              // shared memory outlives the copies from it
    if (got < 0) {
      *abort_flag = 1;
      if (lane == 0) report_fault(p.err, 5, 26);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // Beside the caches' kernel: what waits for this kernel must find that one ended too.
  if (PARTS && p.splits > 0) wait_prerequisites();
}

// Joins the parts of packed tiles: a CTA per 32 rows of a (tile, head) of the unsplit
// numbering, four rows a warp.
//   LSE = log2 sum_j 2^(LSE_j),  O = sum_j 2^(LSE_j - LSE) O_j, in a fixed order.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) packed_join_kernel(const PackedParams p) {
  __shared__ float weight[kJoinRows][kMostParts + 1];
  __shared__ float row_lse[kJoinRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tile = blockIdx.x / (BM / kJoinRows);
  const int first = int(blockIdx.x % (BM / kJoinRows)) * kJoinRows;
  const uint32_t slot = tile / uint32_t(p.kv_heads);
  const int kvh = int(tile - slot * p.kv_heads);
  // Every warp finds the tile and its place in the list of parts by itself.  A CTA with nothing
  // to join waits all the same: this kernel's end stands for the one before it.
  Item w;
  w.live = 0;
  int parts = 1;
  uint32_t item0 = 0;
  const int size = part_size(p);
  const int s = find_sequence(p.cu_q, p.num_seqs, p.tok, slot);
  if (s >= 0) {
    const Sequence q = sequence_at(p, s);
    const int64_t i0 = (int64_t(slot) - int64_t(uint32_t(q.a) / uint32_t(p.tok) + uint32_t(s))) * p.tok;
    if (i0 >= 0 && i0 < q.lq) {
      set_tile(p, q, int(i0), w);
      parts = parts_for(w.j1, size);
      uint32_t before = 0;
      for (int x = lane; x < s; x += 32) {
        const Sequence y = sequence_at(p, x);
        before += uint32_t(tiles_of(p, y.lq)) * parts_for(blocks_of(y.lk), size);
      }
      before = __reduce_add_sync(0xffffffffu, before);
      const uint32_t back = uint32_t(tiles_of(p, q.lq)) - 1u - uint32_t(i0) / uint32_t(p.tok);
      item0 = (before + back * parts_for(blocks_of(q.lk), size)) * p.kv_heads + kvh;
    }
  }
  wait_prerequisites();
  // (the bound on the items fails only for lengths that were refused)
  if (w.live <= 0 || parts == 1 || item0 + uint32_t(parts - 1) * p.kv_heads >= uint32_t(p.max_items)) return;
  const int rows = (w.q_end - w.tok0 < p.tok ? w.q_end - w.tok0 : p.tok) * p.group - first;   // from `first` on
  if (rows <= 0) return;
  const int64_t row0 = int64_t(item0) * BM + first, step = int64_t(p.kv_heads) * BM;
  // A warp's four rows: lanes over the parts for the weights, then over the columns.
  constexpr int V = D / 32, ROWS = kJoinRows / (kJoinThreads / 32);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = warp * ROWS + i;
    if (r >= rows) break;
    const float x = lane < parts ? p.part_lse[row0 + lane * step + r] : -INFINITY;
    const float y = lane + 32 < parts ? p.part_lse[row0 + (lane + 32) * step + r] : -INFINITY;
    float top = fmaxf(x, y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float use = top == -INFINITY ? 0.f : top;
    float sum = ex2_approx(x - use) + ex2_approx(y - use);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float lse = sum == 0.f ? -INFINITY : use + __log2f(sum);
    const float base = lse == -INFINITY ? 0.f : lse;
    weight[r][lane] = ex2_approx(x - base);
    weight[r][lane + 32] = ex2_approx(y - base);
    if (lane == 0) row_lse[r] = lse;
  }
  __syncwarp();
  float acc[ROWS][V] = {};
#pragma unroll 4
  for (int j = 0; j < parts; ++j) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int r = warp * ROWS + i;
      if (r < rows) {
        const float a = weight[r][j];
        const float* src = p.part_o + (row0 + j * step + r) * D + lane * V;
        float v[V];
        if constexpr (V == 4) {
          const float4 f = *reinterpret_cast<const float4*>(src);
          v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(src);
          v[0] = f.x; v[1] = f.y;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) acc[i][e] = fmaf(a, v[e], acc[i][e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = warp * ROWS + i;
    if (r < rows) {
      const int tok_in = (first + r) / p.group, head = kvh * p.group + (first + r) - tok_in * p.group;
      const int64_t token = int64_t(w.tok0) + tok_in;
      __nv_bfloat16* dst = p.o + token * p.o_token + int64_t(head) * p.o_head + lane * V;
      if constexpr (V == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[i][0], acc[i][1]), pack_bf16x2(acc[i][2], acc[i][3]));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[i][0], acc[i][1]);
      if (lane == 0) p.lse[int64_t(head) * p.total_q + token] = row_lse[r] * kLn2;
    }
  }
}

template <int D, bool PARTS>
cudaError_t launch_d(const PackedArgs& a, cudaStream_t stream, const char** why) {
  using C = Cfg<D>;
  const int group = a.q_heads / a.kv_heads, tok = BM / group;
  CUtensorMap tq, tk, tv, to;
  const bool boxes = a.splits == 0 && 16 % group == 0;
  // Without keys nothing is loaded: the maps then describe Q's rows.
  const bool keys = a.total_k > 0;
  if (!make_heads_map(&tq, a.q, a.total_q, a.q_heads, D, a.q_token, a.q_head, group, tok) ||
      !make_heads_map(&tk, keys ? a.k : a.q, keys ? a.total_k : a.total_q, keys ? a.kv_heads : a.q_heads, D,
                      keys ? a.k_token : a.q_token, keys ? a.k_head : a.q_head, 1, BN) ||
      !make_heads_map(&tv, keys ? a.v : a.q, keys ? a.total_k : a.total_q, keys ? a.kv_heads : a.q_heads, D,
                      keys ? a.v_token : a.q_token, keys ? a.v_head : a.q_head, 1, BN) ||
      (boxes && !make_heads_map(&to, a.o, a.total_q, a.q_heads, D, a.o_token, a.o_head, group, 16 / group))) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  if (!boxes) to = tq;                             // not used
  static DeviceFlags attr_set = {};
  cudaError_t e = once_per_device(attr_set, [] {
    return cudaFuncSetAttribute(packed_attn_kernel<D, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  });
  if (e != cudaSuccess) { *why = "cudaFuncSetAttribute(max dynamic smem) failed"; return e; }
  PackedParams p;
  p.num_seqs = a.num_seqs;
  p.kv_heads = a.kv_heads;
  p.group = group;
  p.tok = tok;
  p.total_q = a.total_q;
  p.total_k = a.total_k;
  p.o_token = a.o_token;
  p.o_head = a.o_head;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.causal = a.causal;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.o_boxes = boxes ? 1 : 0;
  p.splits = a.splits;
  p.spare = a.spare;
  p.max_items = a.max_items;
  p.part_o = a.part_o;
  p.part_lse = a.part_lse;
  p.err = a.err;
  const int64_t tiles = a.splits > 0 ? (a.total_q + tok - 1) / tok * a.splits : a.total_q / tok + a.num_seqs;
  const unsigned blocks = unsigned(tiles * a.kv_heads);
  if (a.beside) return launch_dependent(packed_attn_kernel<D, PARTS>, blocks, kThreads, C::SMEM_BYTES, stream, tq, tk, tv, to, p);
  const unsigned grid = a.spare > 0 ? unsigned(a.max_items) : blocks;
  packed_attn_kernel<D, PARTS><<<grid, kThreads, C::SMEM_BYTES, stream>>>(tq, tk, tv, to, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || !PARTS || a.spare == 0) return e;
  *why = "join launch";
  return launch_dependent(packed_join_kernel<D>, blocks * (BM / kJoinRows), kJoinThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_packed(const PackedArgs& a, cudaStream_t stream, const char** why) {
  if (a.d == 128) return a.part_o ? launch_d<128, true>(a, stream, why) : launch_d<128, false>(a, stream, why);
  if (a.d == 64) return a.part_o ? launch_d<64, true>(a, stream, why) : launch_d<64, false>(a, stream, why);
  *why = "unsupported d";
  return cudaErrorInvalidValue;
}

}  // namespace lva
