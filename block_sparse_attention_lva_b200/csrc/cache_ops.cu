// cache_ops.cu -- the append of new tokens to key/value caches, and the eviction from them by
// accumulated attention weight.
//
// Both move rows of 2 d bytes and compute next to nothing: the bound is the bytes read and
// written at the HBM rate (or, for a step's single token, the launch).
//
// Eviction, per (sequence, key/value head) of n > budget live entries: the first `sinks` and
// the last `recent` entries stay, and of the others the budget - sinks - recent of largest
// weight (ties to the lower index), in their order.
//   rank_kernel    one CTA per plane of up to 640 entries: ranks by comparing all pairs.
//   select_kernel  one CTA per longer plane: the k-th largest weight by three radix passes over an
//                  order-preserving 32-bit key (11 + 11 + 10 bits; the first digit is sign,
//                  exponent and two mantissa bits, so a bin holds a quarter octave and few
//                  lanes of a warp meet in one), then one ordered pass with ballots that
//                  writes the kept indices.
//   move_kernel    out of place: a CTA per 64 kept rows, all independent; launched while the
//                  ranking runs, waits for its end (two launches in a row cost 1 to 2 us more).
//   move_in_place_kernel   rows only ever move down (the j-th kept index is >= j).  A CTA owns
//                  a column slice of one plane's K or V and walks the kept rows in ascending
//                  chunks, loads of the next chunks in flight: chunk i's sources are all
//                  loaded before it stores to rows [i C, (i + 1) C), and a later chunk's
//                  sources lie at or above its own rows, so no row is overwritten unread.
//                  Column slices keep CTAs independent.
#include <cstdint>
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace lva {
namespace {

// ---------------------------------------------------------------- append
struct AppendParams {
  const uint8_t* k_new;
  const uint8_t* v_new;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* weight;
  const int32_t* lens;
  int32_t* lens_out;
  int steps, kv_heads, units;        // units: 16-byte units per row, 8 or 16
  uint32_t hop_heads, hop_tokens;    // kAppendThreads / units rows as heads and tokens
  int64_t capacity;
  int64_t k_token, k_head, v_token, v_head;   // bytes
  int write_lens;
  uint32_t blocks;                   // CTAs per sequence
  int* err;
};

constexpr int kAppendThreads = 256;
constexpr int kAppendPer = kAppendUnits / kAppendThreads;

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  const int b = int(blockIdx.x / p.blocks);
  const uint32_t part = blockIdx.x - uint32_t(b) * p.blocks;
  const int32_t n = p.lens[b];       // read before lens_out, which may be lens, is written below
  const bool fits = n >= 0 && int64_t(n) + p.steps <= p.capacity;
  if (!fits && part == 0 && threadIdx.x == 0) report_fault(p.err, 3, b);
  if (fits && p.steps > 0) {
    // units of K, then of V: (head, token, unit), the unit fastest; below 2^31 of them.  A
    // thread's units are kAppendThreads apart: the same unit of rows `hop` apart.
    const uint32_t rows = 2u * p.kv_heads * p.steps;
    const uint32_t first = part * kAppendUnits + threadIdx.x;
    const uint32_t unit = first & uint32_t(p.units - 1), hop = uint32_t(kAppendThreads) / uint32_t(p.units);
    uint32_t row = first / uint32_t(p.units), h = row / uint32_t(p.steps), t = row - h * p.steps;
    uint4 v[kAppendPer];
    uint8_t* dst[kAppendPer];
#pragma unroll
    for (int i = 0; i < kAppendPer; ++i, row += hop) {
      dst[i] = nullptr;
      if (row < rows) {
        const bool is_v = h >= uint32_t(p.kv_heads);
        const uint32_t head = is_v ? h - p.kv_heads : h;
        const uint8_t* src = is_v ? p.v_new + (int64_t(b) * p.steps + t) * p.v_token + head * p.v_head
                                  : p.k_new + (int64_t(b) * p.steps + t) * p.k_token + head * p.k_head;
        v[i] = __ldg(reinterpret_cast<const uint4*>(src) + unit);
        dst[i] = (is_v ? p.v_cache : p.k_cache) +
                 (((int64_t(b) * p.kv_heads + head) * p.capacity + n + t) * p.units + unit) * 16;
      }
      h += p.hop_heads;
      t += p.hop_tokens;
      if (t >= uint32_t(p.steps)) { t -= p.steps; ++h; }
    }
#pragma unroll
    for (int i = 0; i < kAppendPer; ++i)
      if (dst[i] != nullptr) *reinterpret_cast<uint4*>(dst[i]) = v[i];
    if (p.weight != nullptr) {
      const uint32_t count = uint32_t(p.kv_heads) * p.steps;
      for (uint32_t x = part * kAppendThreads + threadIdx.x; x < count; x += p.blocks * kAppendThreads)
        p.weight[(int64_t(b) * p.kv_heads + x / uint32_t(p.steps)) * p.capacity + n + x % uint32_t(p.steps)] = 0.f;
    }
  }
  if (p.write_lens) {
    __syncthreads();                 // in place with one CTA per sequence: every thread has read it
    if (part == 0 && threadIdx.x == 0) p.lens_out[b] = fits ? n + p.steps : n;
  }
}

__global__ void advance_lens_kernel(int32_t* lens, int B, int steps, int64_t capacity) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < B && lens[b] >= 0 && int64_t(lens[b]) + steps <= capacity) lens[b] += steps;
}

// ---------------------------------------------------------------- eviction: which rows stay
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// Larger weight, larger key; NaN below every number; -0 with +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The bin that holds the k-th largest entry (k >= 1) of a histogram, and how many entries lie
// in the bins above it.  Whole CTA; warp_sum is scratch.
__device__ __forceinline__ void find_bin(const uint32_t* hist, uint32_t k, uint32_t* warp_sum, uint32_t* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // thread t takes the bins 2047 - 2t and 2046 - 2t: falling order
  const uint32_t a = hist[kBins - 1 - 2 * tid], b = hist[kBins - 2 - 2 * tid];
  uint32_t sum = a + b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  const uint32_t base = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u);
  const uint32_t before = base + sum - a - b;        // entries in the bins above this thread's
  if (before < k && k <= before + a) { out[0] = kBins - 1 - 2 * tid; out[1] = before; }
  else if (before + a < k && k <= before + a + b) { out[0] = kBins - 2 - 2 * tid; out[1] = before + a; }
  __syncthreads();
}

struct SelectParams {
  const float* weight;
  const int32_t* lens;
  int32_t* kept;
  int kv_heads;
  int64_t capacity, budget, sinks, recent;
  int* err;
};

constexpr int kPer = 4;                              // rounds of 32 entries per warp and tile
constexpr int kTileEntries = kSelThreads * kPer;
constexpr int kKeepTiles = 4;                        // tiles a CTA holds in registers

// Short caches, an entry a thread: an entry's rank is the number of entries before it (larger, or
// equal with a lower index), counted by a walk over all keys in shared memory.  The walk grows
// with the square of the entries; with the move, against the radix passes: 160 entries 5.5 and
// 12.9 us (8 planes), 512 entries 9.1 and 13.0, 768 entries 14.3 and 13.1; 512 planes of 512
// entries 33 and 53, of 768 entries 66 and 63.
constexpr int kRankMost = 640;

__global__ void __launch_bounds__(kRankMost) evict_rank_kernel(const SelectParams p) {
  launch_dependents();                               // the move's CTAs get ready
  __shared__ __align__(16) uint32_t keys[kRankMost];
  __shared__ uint32_t count[kRankMost / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t plane = blockIdx.x;
  const int b = int(plane / p.kv_heads);
  const int32_t len = __ldg(p.lens + b);
  const bool good = len >= 0 && int64_t(len) <= p.capacity;
  const int n = good ? len : 0, threads = int(blockDim.x);
  if (!good && tid == 0) report_fault(p.err, 1, b);
  int32_t* kept = p.kept + plane * p.budget;
  if (n <= p.budget) {
    for (int j = tid; j < p.budget; j += threads) kept[j] = j < n ? j : -1;
    return;
  }
  const int sinks = int(p.sinks), recent = int(p.recent);
  const int middle = n - sinks - recent;
  const uint32_t k = uint32_t(p.budget - p.sinks - p.recent);
  const uint32_t mine = tid < middle ? weight_key(__ldg(p.weight + plane * p.capacity + sinks + tid)) : 0u;
  keys[tid] = mine;
  for (int j = tid; j < sinks; j += threads) kept[j] = j;
  for (int j = tid; j < recent; j += threads) kept[p.budget - recent + j] = n - recent + j;
  __syncthreads();
  // Entries of lower warps come first when equal, of higher warps when larger; a warp's own by
  // both.  keys[] past the last candidate is 0: never larger, and no lower warp's.
  uint32_t rank = 0;
  const uint4* four = reinterpret_cast<const uint4*>(keys);
  const int quads = (middle + 3) / 4;
  if (warp * 32 < middle) {
#pragma unroll 4
    for (int j = 0; j < warp * 8; ++j) {
      const uint4 x = four[j];
      rank += (x.x >= mine) + (x.y >= mine) + (x.z >= mine) + (x.w >= mine);
    }
    for (int j = 0; j < 32; ++j) {
      const uint32_t other = keys[warp * 32 + j];
      rank += other > mine || (other == mine && j < lane);
    }
#pragma unroll 4
    for (int j = warp * 8 + 8; j < quads; ++j) {
      const uint4 x = four[j];
      rank += (x.x > mine) + (x.y > mine) + (x.z > mine) + (x.w > mine);
    }
  }
  const bool stays = tid < middle && rank < k;
  const unsigned mask = __ballot_sync(0xffffffffu, stays);
  if (lane == 0) count[warp] = __popc(mask);
  __syncthreads();
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? count[lane] : 0u);
  if (stays) kept[sinks + before + __popc(mask & ((1u << lane) - 1u))] = sinks + tid;
}

// KEEP: the candidates fit 16 registers a thread (capacity up to 16,384), are read once, with
// all loads in flight, and serve every pass; otherwise each pass reads them again (from L2).
template <bool KEEP>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectParams p) {
  launch_dependents();                               // the move's CTAs get ready
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sum[kSelWarps];
  __shared__ uint2 counts[kKeepTiles * kSelWarps];   // entries above and at the threshold, per tile and warp
  __shared__ uint32_t found[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t plane = blockIdx.x;
  const int b = int(plane / p.kv_heads);
  const int32_t len = __ldg(p.lens + b);
  const bool good = len >= 0 && int64_t(len) <= p.capacity;
  const int n = good ? len : 0;
  if (!good && tid == 0) report_fault(p.err, 1, b);
  int32_t* kept = p.kept + plane * p.budget;
  if (n <= p.budget) {
    for (int64_t j = tid; j < p.budget; j += kSelThreads) kept[j] = j < n ? int32_t(j) : -1;
    return;
  }
  const int sinks = int(p.sinks), recent = int(p.recent);
  const int middle = n - sinks - recent;                       // candidates, > k
  const uint32_t k = uint32_t(p.budget - p.sinks - p.recent);
  const float* w = p.weight + plane * p.capacity + sinks;
  // entry of round i of tile t: warps take 128 consecutive ones
  auto place = [&](int t, int i) { return t * kTileEntries + (warp * kPer + i) * 32 + lane; };
  uint32_t key[KEEP ? kKeepTiles * kPer : 1];
  if constexpr (KEEP) {
    float v[kKeepTiles * kPer];
#pragma unroll
    for (int t = 0; t < kKeepTiles; ++t)
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[t * kPer + i] = place(t, i) < middle ? __ldg(w + place(t, i)) : 0.f;
#pragma unroll
    for (int x = 0; x < kKeepTiles * kPer; ++x) key[x] = weight_key(v[x]);
  }
  for (int j = tid; j < sinks; j += kSelThreads) kept[j] = j;
  for (int j = tid; j < recent; j += kSelThreads) kept[p.budget - recent + j] = n - recent + j;
  if (k == 0) return;
  // k-th largest key: digit by digit, the entries above the digit's bin taken off k
  uint32_t prefix = 0, need = k;
  constexpr int kShift[3] = {21, 10, 0};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    for (int x = tid; x < kBins; x += kSelThreads) hist[x] = 0;
    __syncthreads();
    const int shift = kShift[pass];
    auto count = [&](uint32_t key_x) {
      const bool in = pass == 0 || (key_x >> kShift[pass - (pass > 0)]) == prefix;
      if (in) atomicAdd(&hist[pass == 2 ? (key_x & 1023u) : ((key_x >> shift) & 2047u)], 1u);
    };
    if constexpr (KEEP) {
#pragma unroll
      for (int t = 0; t < kKeepTiles; ++t)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (place(t, i) < middle) count(key[t * kPer + i]);
    } else {
#pragma unroll 4
      for (int x = tid; x < middle; x += kSelThreads) count(weight_key(__ldg(w + x)));
    }
    __syncthreads();
    find_bin(hist, need, warp_sum, found);
    need -= found[1];
    prefix = pass == 2 ? (prefix << 10) | found[0] : (prefix << 11) | found[0];
    __syncthreads();
  }
  // Everything above the threshold key, and the first `need` entries equal to it, in order:
  // kKeepTiles tiles at a time.
  uint32_t gt_base = 0, eq_base = 0;
  for (int t0 = 0; t0 * kTileEntries < middle; t0 += kKeepTiles) {
    uint32_t gt[kKeepTiles * kPer], eq[kKeepTiles * kPer];
#pragma unroll
    for (int t = 0; t < kKeepTiles; ++t) {
      uint32_t n_gt = 0, n_eq = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = place(t0 + t, i);
        uint32_t kx = 0;
        if constexpr (KEEP) kx = key[t * kPer + i];
        else if (x < middle) kx = weight_key(__ldg(w + x));
        gt[t * kPer + i] = __ballot_sync(0xffffffffu, x < middle && kx > prefix);
        eq[t * kPer + i] = __ballot_sync(0xffffffffu, x < middle && kx == prefix);
        n_gt += __popc(gt[t * kPer + i]);
        n_eq += __popc(eq[t * kPer + i]);
      }
      if (lane == 0) counts[t * kSelWarps + warp] = make_uint2(n_gt, n_eq);
    }
    __syncthreads();
    // exclusive sums over (tile, warp): each lane four consecutive places
    uint2 c[kKeepTiles], before[kKeepTiles];
    uint32_t g = 0, e = 0;
#pragma unroll
    for (int x = 0; x < kKeepTiles; ++x) {
      c[x] = counts[lane * kKeepTiles + x];
      before[x] = make_uint2(g, e);
      g += c[x].x;
      e += c[x].y;
    }
    uint32_t sg = g, se = e;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t ug = __shfl_up_sync(0xffffffffu, sg, o), ue = __shfl_up_sync(0xffffffffu, se, o);
      if (lane >= o) { sg += ug; se += ue; }
    }
    const uint32_t all_g = __shfl_sync(0xffffffffu, sg, 31), all_e = __shfl_sync(0xffffffffu, se, 31);
#pragma unroll
    for (int t = 0; t < kKeepTiles; ++t) {
      const int at = t * kSelWarps + warp, owner = at / kKeepTiles, in = at % kKeepTiles;
      uint32_t bg = before[0].x, be = before[0].y;
#pragma unroll
      for (int x = 1; x < kKeepTiles; ++x)
        if (in == x) { bg = before[x].x; be = before[x].y; }
      uint32_t g0 = gt_base + __shfl_sync(0xffffffffu, sg - g + bg, owner), e0 = eq_base + __shfl_sync(0xffffffffu, se - e + be, owner);
      const uint32_t below = (1u << lane) - 1u;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t mg = gt[t * kPer + i], me = eq[t * kPer + i];
        const uint32_t gi = g0 + __popc(mg & below), ei = e0 + __popc(me & below);
        const bool is_gt = (mg >> lane) & 1u, is_eq = (me >> lane) & 1u;
        if (is_gt || (is_eq && ei < need)) kept[sinks + gi + (ei < need ? ei : need)] = sinks + place(t0 + t, i);
        g0 += __popc(mg);
        e0 += __popc(me);
      }
    }
    gt_base += all_g;
    eq_base += all_e;
    __syncthreads();
  }
}

// ---------------------------------------------------------------- eviction: the rows move
struct MoveParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* weight;
  uint8_t* k_out;
  uint8_t* v_out;
  float* weight_out;
  const int32_t* kept;
  const int32_t* lens;
  int32_t* lens_out;
  int B, kv_heads, units;            // units: 16-byte units per row
  int64_t capacity, budget;
  int slices;                        // in place: column slices of a row (K and V each)
};

// lens_out, by one CTA; nothing else of the move kernels reads lens, so it may be lens itself.
__device__ __forceinline__ void write_lens(const MoveParams& p) {
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int32_t n = p.lens[b];
    p.lens_out[b] = n > p.budget && int64_t(n) <= p.capacity ? int32_t(p.budget) : n;
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p) {
  wait_prerequisites();                              // kept is written, lens has been read
  const int64_t blocks = (p.budget + kMoveRows - 1) / kMoveRows;
  const int64_t plane = blockIdx.x / blocks;
  const int64_t j0 = (blockIdx.x - plane * blocks) * kMoveRows;
  if (blockIdx.x == 0) write_lens(p);
  __shared__ int32_t src[kMoveRows];
  if (threadIdx.x < kMoveRows) {
    const int64_t j = j0 + threadIdx.x;
    const int32_t s = j < p.budget ? p.kept[plane * p.budget + j] : -1;
    src[threadIdx.x] = s;
    if (s >= 0) p.weight_out[plane * p.capacity + j] = __ldg(p.weight + plane * p.capacity + s);
  }
  __syncthreads();
  const int per = kMoveRows * p.units;               // units of K (and of V) of this block
  const uint4* k = reinterpret_cast<const uint4*>(p.k) + plane * p.capacity * p.units;
  const uint4* v = reinterpret_cast<const uint4*>(p.v) + plane * p.capacity * p.units;
  uint4* ko = reinterpret_cast<uint4*>(p.k_out) + (plane * p.capacity + j0) * p.units;
  uint4* vo = reinterpret_cast<uint4*>(p.v_out) + (plane * p.capacity + j0) * p.units;
  for (int x = threadIdx.x; x < per; x += 2 * kMoveThreads) {
    const int x1 = x + kMoveThreads;
    const int r0 = x / p.units, r1 = x1 / p.units;
    const int32_t s0 = src[r0], s1 = x1 < per ? src[r1] : -1;
    uint4 a0, a1, b0, b1;
    if (s0 >= 0) {
      const int64_t at = int64_t(s0) * p.units + (x - r0 * p.units);
      a0 = __ldg(k + at);
      b0 = __ldg(v + at);
    }
    if (s1 >= 0) {
      const int64_t at = int64_t(s1) * p.units + (x1 - r1 * p.units);
      a1 = __ldg(k + at);
      b1 = __ldg(v + at);
    }
    if (s0 >= 0) { ko[x] = a0; vo[x] = b0; }
    if (s1 >= 0) { ko[x1] = a1; vo[x1] = b1; }
  }
}

constexpr int kStages = 3;
constexpr int kStageUnits = 4 * kMoveThreads;         // 16 KB a stage

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__global__ void __launch_bounds__(kMoveThreads) move_in_place_kernel(const MoveParams p) {
  __shared__ __align__(16) uint8_t stage[kStages * kStageUnits * 16];
  const int per_plane = 2 * p.slices + 1;             // K slices, V slices, the weights
  const int64_t plane = blockIdx.x / per_plane;
  const int part = int(blockIdx.x - plane * per_plane);
  if (blockIdx.x == 0) write_lens(p);
  const int32_t* kept = p.kept + plane * p.budget;
  const int tid = threadIdx.x;
  // Rows that stay where they are (the sinks, or a plane below its budget) are passed over;
  // kept[j] > j holds from the first moving row on, and kept ends where -1 begins.
  if (part == 2 * p.slices) {
    float* w = p.weight_out + plane * p.capacity;
    for (int64_t j0 = 0; j0 < p.budget; j0 += kMoveThreads) {
      const int64_t j = j0 + tid;
      const int32_t s = j < p.budget ? __ldg(kept + j) : -1;
      const bool move = s > j;
      const float x = move ? w[s] : 0.f;
      __syncthreads();
      if (move) w[j] = x;
      __syncthreads();
    }
    return;
  }
  uint8_t* base = part < p.slices ? p.k_out : p.v_out;
  const int width = p.units / p.slices;               // units of a slice
  uint8_t* rows = base + plane * p.capacity * p.units * 16 + int64_t(part % p.slices) * width * 16;
  const int64_t pitch = int64_t(p.units) * 16;
  const int chunk_rows = kStageUnits / width;
  const int64_t chunks = (p.budget + chunk_rows - 1) / chunk_rows;
  const uint32_t s_base = smem_u32(stage);
  auto load = [&](int64_t i) {
    if (i < chunks) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int x = e * kMoveThreads + tid;
        const int r = x / width;
        const int64_t j = i * chunk_rows + r;
        const int32_t s = j < p.budget ? __ldg(kept + j) : -1;
        if (s > j)
          cp_async16(s_base + uint32_t((i % kStages) * kStageUnits + x) * 16, rows + s * pitch + (x - r * width) * 16);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kStages - 1; ++i) load(i);
  for (int64_t i = 0; i < chunks; ++i) {
    load(i + kStages - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncthreads();                                  // every thread's loads of chunk i have landed
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = e * kMoveThreads + tid;
      const int r = x / width;
      const int64_t j = i * chunk_rows + r;
      const int32_t s = j < p.budget ? __ldg(kept + j) : -1;
      if (s > j)
        *reinterpret_cast<uint4*>(rows + j * pitch + (x - r * width) * 16) =
            *reinterpret_cast<const uint4*>(stage + ((i % kStages) * kStageUnits + x) * 16);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  AppendParams p;
  p.k_new = static_cast<const uint8_t*>(a.k_new);
  p.v_new = static_cast<const uint8_t*>(a.v_new);
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.weight = a.weight;
  p.lens = a.lens;
  p.lens_out = a.lens_out;
  p.steps = a.steps;
  p.kv_heads = a.kv_heads;
  p.units = a.d / 8;
  const int hop = kAppendThreads / p.units;
  p.hop_heads = a.steps > 0 ? uint32_t(hop / a.steps) : 0;
  p.hop_tokens = a.steps > 0 ? uint32_t(hop % a.steps) : 0;
  p.capacity = a.capacity;
  p.k_token = a.k_token * 2;
  p.k_head = a.k_head * 2;
  p.v_token = a.v_token * 2;
  p.v_head = a.v_head * 2;
  p.err = a.err;
  const int64_t units = 2 * int64_t(a.kv_heads) * a.steps * p.units;
  int64_t blocks = (units + kAppendUnits - 1) / kAppendUnits;
  if (blocks < 1) blocks = 1;        // no token: lens_out alone
  // In place with several CTAs per sequence, the lengths advance in a launch of their own.
  const bool later = a.lens_out == a.lens && blocks > 1;
  p.write_lens = later ? 0 : 1;
  p.blocks = uint32_t(blocks);
  append_kernel<<<unsigned(blocks * a.B), kAppendThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !later) return e;
  advance_lens_kernel<<<unsigned((a.B + 255) / 256), 256, 0, stream>>>(a.lens_out, a.B, a.steps, a.capacity);
  return cudaGetLastError();
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t planes = int64_t(a.B) * a.kv_heads;
  const SelectParams s{a.weight, a.lens, a.kept, a.kv_heads, a.capacity, a.budget, a.sinks, a.recent, a.err};
  if (a.capacity <= kRankMost)
    evict_rank_kernel<<<unsigned(planes), unsigned((a.capacity + 31) / 32 * 32), 0, stream>>>(s);
  else if (a.capacity <= kKeepTiles * kTileEntries) evict_select_kernel<true><<<unsigned(planes), kSelThreads, 0, stream>>>(s);
  else evict_select_kernel<false><<<unsigned(planes), kSelThreads, 0, stream>>>(s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  MoveParams p;
  p.k = static_cast<const uint8_t*>(a.k_cache);
  p.v = static_cast<const uint8_t*>(a.v_cache);
  p.weight = a.weight;
  p.k_out = static_cast<uint8_t*>(a.k_out);
  p.v_out = static_cast<uint8_t*>(a.v_out);
  p.weight_out = a.weight_out;
  p.kept = a.kept;
  p.lens = a.lens;
  p.lens_out = a.lens_out;
  p.B = a.B;
  p.kv_heads = a.kv_heads;
  p.units = a.d / 8;
  p.capacity = a.capacity;
  p.budget = a.budget;
  if (a.k_out == a.k_cache) {
    // Slices of at least 32 bytes (a DRAM sector) until there are three CTAs for an SM: 96
    // planes of 8,192 kept rows 268 us whole, 198 with slices of 128 bytes, 193 with 64, 195 with
    // 32; 64 planes of 20,000 rows 643, 401, 293 and 339; 32 planes of 8,192 rows 222, 129, 83 and
    // 79; 230 planes of 4,096 rows 217, 216, 210 and 229 (weights that are new in every call).
    p.slices = 1;
    while (p.slices < p.units / 2 && planes * 2 * p.slices < 3 * sm_count()) p.slices *= 2;
    move_in_place_kernel<<<unsigned(planes * (2 * p.slices + 1)), kMoveThreads, 0, stream>>>(p);
  } else {
    p.slices = 0;
    return launch_dependent(move_kernel, unsigned(planes * ((a.budget + kMoveRows - 1) / kMoveRows)), kMoveThreads, 0, stream, p);
  }
  return cudaGetLastError();
}

}  // namespace lva
