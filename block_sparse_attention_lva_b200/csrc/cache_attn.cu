// cache_attn.cu -- a few query tokens per sequence against each sequence's own key/value
// cache, and the join with the parts of a key prefix that the batch shares (packed.cu).
//
// With n = lens[b] live entries (the T new tokens' own among them), token t sees the cache
// keys c <= n - T + t.  For one (sequence b, key/value head) "plane" the R = T G rows (row
// r = t G + g: token t, query head g of the group) meet every live key once:
//
//   x_rc = scale log2(e) <q_r, k_c>,  m = max_c x_rc,  l = sum_c 2^(x_rc - m),
//   O_r = sum_c 2^(x_rc - m) v_c / l,  LSE_r = m + log2 l   (log2 units)
//
// With up to 8 rows the bound is the cache's bytes from HBM (4 d per key and plane; a row costs
// 4 d flops per key, R <= 64 of them); with more it is the warps' products and softmax, and with
// d = 128 these forms spill 136 to 240 bytes a thread: 16 caches of 3,000 to 6,000 keys, 8 heads of
// 128 (295 MB, 45 us) take 53, 62, 81 and 125 us with 4, 16, 32 and 64 rows.  Work is cut without looking at single sequences: the 64-key tiles
// of all planes form one list, and each worker (a CTA, one per SM) takes an equal run of it,
// so ragged lengths balance by themselves.  A run may begin and end inside a plane; every
// (plane, worker) segment leaves its normalised O and LSE in float32.  Segments of the list,
// walked in order, raise the plane or the worker by one at each step, so plane + worker
// numbers their slots without a table.
//
// With a prefix there are two kinds of work: the prefix parts (packed.cu) are bound by the
// SMs' softmax rate, the caches by HBM.  The caches' kernel goes first, the prefix parts are a
// programmatic dependent launch (neither reads what the other writes), the join waits for
// both.  The parts run on SMs that the caches' workers were not given, or take over the
// workers' one by one as they end; the entry point estimates which is shorter.  A small batch's
// prefix (all its tokens at most 32 rows) can be one more sequence of the list instead, with
// all tokens' rows against its tiles (PREFIX), which saves a launch.
//
//   cache_attn_kernel  the last warp: TMA producer (K and V tiles of 64 keys in one ring, the
//                      plane's Q rows in two slots); the others: mma.sync m16n8k16 on swizzled
//                      tiles, in groups that take tiles in turn.  Keys are the M side (S^T =
//                      K Q^T, O^T = V^T P^T), so up to 8 rows, the usual step of single
//                      tokens, fill the N side of one product: with rows as the M side, 16 at
//                      least, an SM's tensor pipe (16 cycles a product and quarter) held its
//                      rate to 49 GB/s of the 98 that its loads can bring.  P^T needs its
//                      fragments transposed between the products: one movmatrix per 8 x 8.
//                      A warp works on 32 keys a step, so that a step's chain of latencies
//                      (product, maximum, exponentials, product) is paid per 32 keys.
//   join_kernel        LSE = log2 sum_j 2^(LSE_j), O = sum_j 2^(LSE_j - LSE) O_j over the
//                      row's prefix parts and segments, in float32, in a fixed order; and, on
//                      request, weight[c] += sum_r 2^(x_rc - LSE_r) from the scores the first
//                      kernel left (4 R bytes per key against 2 d for reading K again).
//                      Each weight has one writer and a fixed order of additions.
//                      A row of several tokens' step that came out not finite is looked at again
//                      (without_late_keys).
#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace lva {
namespace {

constexpr int kTile = 64;            // keys per tile
constexpr int kStep = 32;            // keys a warp works on at a time
constexpr float kRescaleThreshold = 8.0f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr unsigned kFull = 0xffffffffu;

struct CacheParams {
  int B, steps, kv_heads, group, rows;       // rows = steps * group
  int64_t capacity;
  const int32_t* lens;
  float scale_log2;
  float* own_o;
  float* own_lse;
  float* scores;
  int64_t score_stride;
  int workers;
  // PREFIX: the shared prefix is the list's last sequence, all tokens of the batch its rows
  int prefix_len, prefix_rows;
  float* part_o;                             // [kv_heads + workers, prefix_rows, D]
  float* part_lse;
  int* err;
};

// Live entries of sequence b; a length outside [0, capacity] counts as none.
__device__ __forceinline__ int live_len(const int32_t* lens, int b, int64_t capacity) {
  const int32_t n = __ldg(lens + b);
  return n >= 0 && int64_t(n) <= capacity ? n : 0;
}
__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// A plane counts as its tiles and kSegment more: what a segment's start and end (its first
// loads' latency, the join of its parts) cost beside its tiles, 1.8 us against 0.36 us a tile
// when latency counts.  Without it a worker with many planes of a tile each took three times as
// long as the others (47 us instead of 16).
constexpr int kSegment = 5;
__device__ __forceinline__ int plane_cost(int tiles) { return tiles > 0 ? tiles + kSegment : 0; }

// Cost of one head of all sequences, and of those before `stop` (whole warp).  All planes'
// costs stay below 2^31: the call is refused when B * kv_heads * (capacity / 64 + 6) is not.
__device__ __forceinline__ int count_cost(const int32_t* lens, int B, int64_t capacity, int stop, int* before) {
  const int lane = threadIdx.x & 31;
  int all = 0, part = 0;
  for (int b = lane; b < B; b += 32) {
    const int t = plane_cost(tiles_of(live_len(lens, b, capacity)));
    all += t;
    if (b < stop) part += t;
  }
  *before = __reduce_add_sync(kFull, part);
  return __reduce_add_sync(kFull, all);
}

// A list of `total` places in runs for up to `workers` workers: the first `total` mod n of the
// n = min(workers, total) runs are one place longer, and none of the n is empty.
struct Runs {
  int n, len, longer;
  __device__ __forceinline__ Runs(int total, int workers) {
    n = total < workers ? total : workers;
    len = n > 0 ? int(uint32_t(total) / uint32_t(n)) : 0;
    longer = total - n * len;
  }
  __device__ __forceinline__ int start(int w) const { return w * len + (w < longer ? w : longer); }
  __device__ __forceinline__ int worker(int x) const {           // whose run holds place x (n > 0)
    const int split = longer * (len + 1);
    return x < split ? int(uint32_t(x) / uint32_t(len + 1)) : longer + int(uint32_t(x - split) / uint32_t(len));
  }
};

// Walks a worker's run plane by plane (every warp the same walk).  A plane's tiles come first in
// its part of the list; a run that meets only the rest of it has no tile there.
template <bool PREFIX>
struct Walk {
  const CacheParams& p;
  int left;                  // of the run, not yet handed out
  int b, kvh, n, tiles, t0;  // the current plane, its first tile of the run
  __device__ __forceinline__ Walk(const CacheParams& params, int worker) : p(params) {
    const int lane = threadIdx.x & 31;
    int unused;
    const int shared = PREFIX ? plane_cost(tiles_of(p.prefix_len)) : 0;
    const Runs runs((count_cost(p.lens, p.B, p.capacity, 0, &unused) + shared) * p.kv_heads, p.workers);
    left = 0;
    b = kvh = n = tiles = t0 = 0;
    if (worker >= runs.n) return;
    int at = runs.start(worker);
    left = runs.start(worker + 1) - at;
    // the sequence that holds place `at`: 32 sequences at a time
    for (int b0 = 0; b0 < p.B + (PREFIX ? 1 : 0); b0 += 32) {
      const int mine = keys(b0 + lane);
      const int own = plane_cost(tiles_of(mine)) * p.kv_heads;
      int sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += up;
      }
      const unsigned past = __ballot_sync(kFull, sum > at);
      if (past != 0) {
        const int l = __ffs(past) - 1;
        b = b0 + l;
        n = __shfl_sync(kFull, mine, l);
        const int in = at - __shfl_sync(kFull, sum - own, l);
        tiles = tiles_of(n);
        kvh = int(uint32_t(in) / uint32_t(plane_cost(tiles)));
        t0 = in - kvh * plane_cost(tiles);
        if (t0 >= tiles) next();                   // starts behind this plane's tiles
        return;
      }
      at -= __shfl_sync(kFull, sum, 31);
    }
    left = 0;                // not reached: the run lies inside the list
  }
  __device__ __forceinline__ int keys(int x) const {
    return x < p.B ? live_len(p.lens, x, p.capacity) : PREFIX && x == p.B ? p.prefix_len : 0;
  }
  __device__ __forceinline__ bool in_prefix() const { return PREFIX && b == p.B; }
  // Tiles of the current plane in this run; at least one while left > 0.
  __device__ __forceinline__ int count() const { return left < tiles - t0 ? left : tiles - t0; }
  __device__ __forceinline__ void next() {
    left -= plane_cost(tiles) - t0;
    t0 = 0;
    if (left <= 0) return;
    if (++kvh < p.kv_heads) return;
    kvh = 0;
    do {
      ++b;
      n = keys(b);
    } while (b < p.B && n == 0);
    tiles = tiles_of(n);
    if (n == 0) left = 0;
  }
};

// NT: 8-row tiles a warp holds; WR: row parts, each a warp's.  Up to 8 * NT * WR rows.
template <int D, int NT, int WR>
struct Cfg {
  // consumer warps: with the producer three a scheduler, 168 registers a thread
  static constexpr int WARPS = NT == 1 ? 10 : 8;
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int GROUP_WARPS = WR > 2 ? WR : 2;
  static constexpr int GROUPS = WARPS / GROUP_WARPS;  // they take the tiles in turn
  static constexpr int WK = GROUP_WARPS / WR;         // key parts of a tile
  static constexpr int KW = kTile / WK;               // keys of a tile per warp
  static constexpr int PARTS = GROUPS * WK;           // (m, l, O) of a row to be joined
  static constexpr int WROWS = 8 * NT;
  static constexpr int QROWS = WROWS * WR;
  static constexpr int SLOT = kTile * D * 2;          // one K or V tile
  // Ring: 160 KB in flight per SM (128 KB with more rows, for their join); 64 KB reach the full
  // HBM rate when all SMs load.  A slot's tiles must all go to one group: its parity
  // wait for a tile is then preceded by its own wait for the slot's tile before.  (A group that
  // waits on a slot whose tile before, another group's, has not landed finds the parity of the
  // tile before that and passes.)
  static constexpr int NSLOT = (NT == 1 ? 10 : 8) * (128 / D);
  static_assert(NSLOT / 2 % GROUPS == 0, "a slot belongs to one group");
  static constexpr int Q_SLOT = QROWS * D * 2;
  static constexpr int FRAG = D / 16 * NT * 4;        // O registers per lane
  static constexpr int STAT = 4 * NT;                 // m, l
  static constexpr int JOIN = PARTS * WR * (FRAG + STAT) * 32 * 4;
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_Q = OFF_KV + NSLOT * SLOT;
  static constexpr int QS = WR == 4 ? 1 : 2;          // Q slots
  static constexpr int OFF_JOIN = OFF_Q + QS * Q_SLOT;
  static constexpr int OFF_BAR = OFF_JOIN + JOIN;
  static constexpr int B_F = 0, B_E = NSLOT, B_QF = 2 * NSLOT, B_QE = B_QF + QS, B_GRP = B_QE + QS, NUM_BARS = B_GRP + 2;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16;
  // more than half of an SM, so that the workers spread over the SMs one by one
  static_assert(SMEM_BYTES > 114 * 1024 && SMEM_BYTES <= 227 * 1024, "one CTA per SM");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 matrix of 16-bit elements over the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

struct CacheMaps {
  CUtensorMap q, k, v;                       // a sequence's step of Q rows, the caches' tiles
  CUtensorMap all_q, prefix_k, prefix_v;     // PREFIX: all tokens' rows, the prefix's tiles
};

template <int D, int NT, int WR, bool PREFIX>
__global__ void __launch_bounds__(Cfg<D, NT, WR>::THREADS, 1) cache_attn_kernel(const __grid_constant__ CacheMaps maps,
                                                                                const CacheParams p) {
  using C = Cfg<D, NT, WR>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s_base = smem_u32(smem);
  if (s_base & 1023u) {                           // never expected; checked rather than assumed
    if (threadIdx.x == 0) report_fault(p.err, 4, 1023);
    return;
  }
  const uint32_t bar0 = s_base + C::OFF_BAR;
  auto bar_full = [&](int s) { return bar0 + 8u * (C::B_F + s); };
  auto bar_empty = [&](int s) { return bar0 + 8u * (C::B_E + s); };
  auto bar_q_full = [&](int s) { return bar0 + 8u * (C::B_QF + s); };
  auto bar_q_empty = [&](int s) { return bar0 + 8u * (C::B_QE + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  volatile int* never = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);   // stays zero
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x;

  if (worker == 0)                                // lengths outside their cache: reported once
    for (int b = threadIdx.x; b < p.B; b += C::THREADS) {
      const int32_t n = __ldg(p.lens + b);
      if (n < 0 || int64_t(n) > p.capacity) report_fault(p.err, 1, b);
    }
  // Q rows past the group's are never loaded: zero, so that no stray value is computed with.
  for (int x = threadIdx.x; x < C::QS * C::Q_SLOT / 16; x += C::THREADS)
    reinterpret_cast<uint4*>(smem + C::OFF_Q)[x] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NSLOT; ++s) { mbar_init(bar_full(s), 1); mbar_init(bar_empty(s), C::GROUP_WARPS); }
    for (int s = 0; s < C::QS; ++s) { mbar_init(bar_q_full(s), 1); mbar_init(bar_q_empty(s), C::WARPS); }
    for (int s = 0; s < 2; ++s) mbar_init(bar0 + 8u * (C::B_GRP + s), C::WARPS);
    *abort_flag = 0;
    *never = 0;
    mbar_fence_init();
  }
  launch_dependents();                            // the prefix parts may start beside this kernel
  Walk<PREFIX> walk(p, worker);
  __syncthreads();

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ TMA producer
    uint32_t u = 0;                               // ring position: K of tile T at 2T, V at 2T + 1
    uint32_t seg = 0, loaded_q = 0;
    bool ok = true;
    if (lane == 0 && walk.left > 0) { tma_prefetch_desc(&maps.q); tma_prefetch_desc(&maps.k); tma_prefetch_desc(&maps.v); }
    for (; ok && walk.left > 0; walk.next(), ++seg) {
      if (lane == 0) {
        const int qs = int(seg % C::QS);
        ok = seg < C::QS || mbar_wait_sleep(bar_q_empty(qs), ((seg / C::QS) - 1) & 1, abort_flag);
        if (ok) {
          const bool shared = walk.in_prefix();
          mbar_arrive_expect_tx(bar_q_full(qs), uint32_t((shared ? p.prefix_rows : p.rows) * D * 2));
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(s_base + C::OFF_Q + qs * C::Q_SLOT + c * C::QROWS * 128, shared ? &maps.all_q : &maps.q, c * 64,
                        walk.kvh * p.group, shared ? 0 : walk.b * p.steps, bar_q_full(qs));
          ++loaded_q;
        }
        const int64_t plane_row = (int64_t(walk.b) * p.kv_heads + walk.kvh) * p.capacity;
        const int cnt = walk.count();
        for (int t = 0; ok && t < cnt; ++t) {
          const int32_t row = int32_t(plane_row + int64_t(walk.t0 + t) * kTile);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++u) {
            const int s = int(u % C::NSLOT);
            if (u >= uint32_t(C::NSLOT) && !mbar_wait_sleep(bar_empty(s), ((u / C::NSLOT) - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(bar_full(s), C::SLOT);
            for (int c = 0; c < D / 64; ++c) {
              const uint32_t dst = s_base + C::OFF_KV + s * C::SLOT + c * kTile * 128;
              if (walk.in_prefix())
                tma_load_3d(dst, kv == 0 ? &maps.prefix_k : &maps.prefix_v, c * 64, walk.kvh, (walk.t0 + t) * kTile, bar_full(s));
              else
                tma_load_2d(dst, kv == 0 ? &maps.k : &maps.v, c * 64, row, bar_full(s));
            }
          }
        }
        if (!ok) {
          *abort_flag = 1;
          report_fault(p.err, 5, 31);
        }
      }
      ok = __shfl_sync(kFull, ok, 0);
    }
    if (lane == 0 && *abort_flag) {               // every load in flight lands before the CTA ends
      for (uint32_t x = u > uint32_t(C::NSLOT) ? u - C::NSLOT : 0; x < u; ++x)
        mbar_wait(bar_full(int(x % C::NSLOT)), (x / C::NSLOT) & 1, never);
      for (uint32_t x = loaded_q > C::QS ? loaded_q - C::QS : 0; x < loaded_q; ++x)
        mbar_wait(bar_q_full(int(x % C::QS)), (x / C::QS) & 1, never);
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int group = warp / C::GROUP_WARPS, in_group = warp % C::GROUP_WARPS;
    const int wr = in_group % WR, wk = in_group / WR;
    const int part = group * C::WK + wk;           // of the row's PARTS
    const int g = lane >> 2, q4 = lane & 3;        // fragment row (key, dim) and column pair (rows)
    const float c = p.scale_log2;
    // This lane's rows: 2 q4 + e of each 8-row tile.
    auto row_of = [&](int nt, int e) { return wr * C::WROWS + nt * 8 + q4 * 2 + e; };
    uint32_t T = 0, seg = 0;
    int seq = 0;
    bool ok = true;
    // Bounded barrier over the consumer warps: sync `seq` uses slot seq & 1, and no warp can
    // arrive for seq + 2 before all have left the wait for seq.
    auto group_sync = [&]() -> bool {
      const uint32_t bar = bar0 + 8u * (C::B_GRP + (seq & 1));
      const uint32_t parity = (seq >> 1) & 1;
      ++seq;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      return __all_sync(kFull, mbar_wait(bar, parity, abort_flag));
    };
    // 16-byte unit `unit` of row r of a swizzled [rows, 64-element] chunk
    auto sw = [](uint32_t chunk, int r, int unit) { return chunk + r * 128 + ((unit ^ (r & 7)) << 4); };

    for (; ok && walk.left > 0; walk.next(), ++seg) {
      const int qs = int(seg % C::QS);
      ok = __all_sync(kFull, mbar_wait_sleep(bar_q_full(qs), (seg / C::QS) & 1, abort_flag));
      if (!ok) break;
      uint32_t qf[D / 16][NT][2];                  // Q^T fragments
      {
        const uint32_t qb = s_base + C::OFF_Q + qs * C::Q_SLOT;
#pragma unroll
        for (int k = 0; k < D / 16; k += 2) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t f[4];                         // k .. k + 7, + 8, + 16, + 24 of 8 rows
            ldsm4(sw(qb + (k / 4) * C::QROWS * 128, wr * C::WROWS + nt * 8 + (lane & 7), (k % 4) * 2 + (lane >> 3)), f);
            qf[k][nt][0] = f[0];
            qf[k][nt][1] = f[1];
            qf[k + 1][nt][0] = f[2];
            qf[k + 1][nt][1] = f[3];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_q_empty(qs));
      }
      float of[D / 16][NT][4];                     // O^T: dims x rows
      float m[NT][2], l[NT][2];
      int lim[NT][2];                              // keys each row sees
      // every row sees the whole prefix, a cache's row as far as its token
      const bool shared = walk.in_prefix();
      const int rows = shared ? p.prefix_rows : p.rows;
      const int base = shared ? walk.n : walk.n - p.steps + 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) of[i][nt][0] = of[i][nt][1] = of[i][nt][2] = of[i][nt][3] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = -INFINITY;
          l[nt][e] = 0.f;
          lim[nt][e] = row_of(nt, e) < rows ? base + (shared ? 0 : row_of(nt, e) / p.group) : 0;
        }
      }
      const int64_t plane = int64_t(walk.b) * p.kv_heads + walk.kvh;
      const int cnt = walk.count();
      const int group0 = int(T % C::GROUPS);       // of the segment's first tile
      for (int t = 0; t < cnt; ++t, ++T) {
        if (int(T % C::GROUPS) != group) continue;
        const int tile0 = (walk.t0 + t) * kTile;                   // the tile's first key
        const uint32_t uk = 2 * T, uv = 2 * T + 1;
        const int ks = int(uk % C::NSLOT), vs = int(uv % C::NSLOT);
        const uint32_t kb = s_base + C::OFF_KV + ks * C::SLOT, vb = s_base + C::OFF_KV + vs * C::SLOT;
        ok = __all_sync(kFull, mbar_wait_sleep(bar_full(ks), (uk / C::NSLOT) & 1, abort_flag));
        if (!ok) break;
#pragma unroll 1
        for (int sub = 0; sub < C::KW; sub += kStep) {
          const int first = wk * C::KW + sub;                      // of the tile's rows
          const int key0 = tile0 + first;
          const bool any = key0 < walk.n;                          // warp-uniform
          float sf[kStep / 16][NT][4];
          if (any) {
#pragma unroll
            for (int i = 0; i < kStep / 16; ++i)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) sf[i][nt][0] = sf[i][nt][1] = sf[i][nt][2] = sf[i][nt][3] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
#pragma unroll
              for (int i = 0; i < kStep / 16; ++i) {
                // K fragment: lanes 0-7, 8-15: keys 0-7, 8-15 at k; lanes 16-31: at k + 8
                uint32_t kf[4];
                ldsm4(sw(kb + (k / 4) * kTile * 128, first + i * 16 + (lane & 15), (k % 4) * 2 + (lane >> 4)), kf);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816(sf[i][nt], kf, qf[k][nt][0], qf[k][nt][1]);
              }
            }
          }
          if (sub + kStep == C::KW) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty(ks));
          }
          uint32_t pf[kStep / 16][NT][2];                          // P^T fragments
          if (any) {
            const bool masked = key0 + kStep > base;               // some row does not see every key
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
              for (int i = 0; i < kStep / 16; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  float x = sf[i][nt][e] * c;
                  const int key = key0 + i * 16 + g + (e >> 1) * 8;
                  if (p.scores != nullptr && !shared && row_of(nt, e & 1) < p.rows)
                    p.scores[(plane * p.rows + row_of(nt, e & 1)) * p.score_stride + key] = x;
                  if (masked && key >= lim[nt][e & 1]) x = -INFINITY;
                  sf[i][nt][e] = x;
                }
                mx[nt][0] = fmax3(mx[nt][0], sf[i][nt][0], sf[i][nt][2]);
                mx[nt][1] = fmax3(mx[nt][1], sf[i][nt][1], sf[i][nt][3]);
              }
            }
            // The reference moves only when some maximum outgrows it by 2^8 (weights stay in
            // range): one vote over the lanes' own maxima, and the rows' maxima only then.
            bool out = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) out |= mx[nt][e] > m[nt][e] + kRescaleThreshold || m[nt][e] == -INFINITY;
            if (__any_sync(kFull, out)) {
#pragma unroll
              for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 2; ++e) mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(kFull, mx[nt][e], o));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float old = m[nt][e];
                  if (mx[nt][e] > old + kRescaleThreshold || old == -INFINITY) m[nt][e] = fmaxf(old, mx[nt][e]);
                  const float al = m[nt][e] == old ? 1.f : ex2_approx(old - m[nt][e]);
                  l[nt][e] *= al;
#pragma unroll
                  for (int i = 0; i < D / 16; ++i) { of[i][nt][e] *= al; of[i][nt][e + 2] *= al; }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float u0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], u1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
              for (int i = 0; i < kStep / 16; ++i) {
                const float p0 = ex2_approx(sf[i][nt][0] - u0), p1 = ex2_approx(sf[i][nt][1] - u1);
                const float p2 = ex2_approx(sf[i][nt][2] - u0), p3 = ex2_approx(sf[i][nt][3] - u1);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                pf[i][nt][0] = transpose8(pack_bf16x2(p0, p1));    // P in bf16: the MMA's operand type
                pf[i][nt][1] = transpose8(pack_bf16x2(p2, p3));
              }
            }
          }
          if (sub == 0) {
            ok = __all_sync(kFull, mbar_wait_sleep(bar_full(vs), (uv / C::NSLOT) & 1, abort_flag));
            if (!ok) break;
          }
          if (any) {
            const bool tail = key0 + kStep > walk.n;               // the plane's last live keys
            if (tail) {
              // V rows past the live ones may hold anything: zero, so that 0 * NaN never is
              uint8_t* vt = smem + C::OFF_KV + vs * C::SLOT;
              for (int ch = 0; ch < D / 64; ++ch)
                for (int x = lane; x < kStep * 8; x += 32) {
                  const int r = first + (x >> 3);
                  if (tile0 + r >= walk.n)
                    *reinterpret_cast<uint4*>(vt + ch * kTile * 128 + r * 128 + ((x & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                }
              __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < kStep / 16; ++i) {
#pragma unroll
              for (int x = 0; x < D / 16; ++x) {
                // V^T fragment: lanes 0-7, 8-15: keys 0-7 at dims 0-7, 8-15; lanes 16-31: keys 8-15
                uint32_t vf[4];
                ldsm4_t(sw(vb + (x / 4) * kTile * 128, first + i * 16 + (lane & 7) + ((lane >> 4) << 3),
                           (x % 4) * 2 + ((lane >> 3) & 1)), vf);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816(of[x][nt], vf, pf[i][nt][0], pf[i][nt][1]);
              }
            }
            if (tail) fence_proxy_async_smem();    // the zeros before the slot's next TMA write
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty(vs));
      }
      if (!ok) break;

      // Row sums over the lanes of a column pair; then the parts meet in shared memory: each that
      // had a tile leaves (O, m, l) there, and the parts' warps share out the 16-dim pieces.
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], o);
      auto slot = [&](int i) {
        return reinterpret_cast<float*>(smem + C::OFF_JOIN) + (i * WR + wr) * (C::FRAG + C::STAT) * 32 + lane;
      };
      auto has_tile = [&](int i) {
        const int after = i / C::WK - group0;      // groups take tiles in turn, from group0 on
        return (after < 0 ? after + C::GROUPS : after) < cnt;
      };
      ok = group_sync();                           // the previous segment's pieces have been read
      if (!ok) break;
      if (has_tile(part)) {
        float* s = slot(part);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[((nt * (D / 16) + x) * 4 + e) * 32] = of[x][nt][e];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[(C::FRAG + nt * 4 + e) * 32] = m[nt][e];
            s[(C::FRAG + nt * 4 + 2 + e) * 32] = l[nt][e];
          }
        }
      }
      ok = group_sync();
      if (!ok) break;
      const int64_t at = shared ? int64_t(walk.kvh + worker) * rows : (plane + worker) * rows;
      float* out_o = shared ? p.part_o : p.own_o;
      float* out_lse = shared ? p.part_lse : p.own_lse;
#pragma unroll 1
      for (int piece = part; piece < NT * (D / 16); piece += C::PARTS) {
        const int nt = piece / (D / 16), x = piece - nt * (D / 16);
        float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < C::PARTS; ++i)
          if (has_tile(i)) {
            top[0] = fmaxf(top[0], slot(i)[(C::FRAG + nt * 4) * 32]);
            top[1] = fmaxf(top[1], slot(i)[(C::FRAG + nt * 4 + 1) * 32]);
          }
        const float use[2] = {top[0] == -INFINITY ? 0.f : top[0], top[1] == -INFINITY ? 0.f : top[1]};
#pragma unroll
        for (int i = 0; i < C::PARTS; ++i)
          if (has_tile(i)) {
            const float* s = slot(i);
            const float w0 = ex2_approx(s[(C::FRAG + nt * 4) * 32] - use[0]), w1 = ex2_approx(s[(C::FRAG + nt * 4 + 1) * 32] - use[1]);
            sum[0] = fmaf(w0, s[(C::FRAG + nt * 4 + 2) * 32], sum[0]);
            sum[1] = fmaf(w1, s[(C::FRAG + nt * 4 + 3) * 32], sum[1]);
            acc[0] = fmaf(w0, s[(piece * 4) * 32], acc[0]);
            acc[1] = fmaf(w1, s[(piece * 4 + 1) * 32], acc[1]);
            acc[2] = fmaf(w0, s[(piece * 4 + 2) * 32], acc[2]);
            acc[3] = fmaf(w1, s[(piece * 4 + 3) * 32], acc[3]);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = row_of(nt, e);
          if (row < rows) {
            const bool none = sum[e] == 0.f;       // a NaN sum goes through as NaN
            const float inv = none ? 0.f : __fdividef(1.f, sum[e]);
            float* dst = out_o + (at + row) * D + x * 16 + g;
            dst[0] = none ? 0.f : acc[e] * inv;
            dst[8] = none ? 0.f : acc[e + 2] * inv;
            if (x == 0 && g == 0) out_lse[at + row] = none ? -INFINITY : top[e] + __log2f(sum[e]);
          }
        }
      }
      __syncwarp();
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) report_fault(p.err, 5, 32);
    }
  }
}

struct JoinParams {
  int B, steps, q_heads, kv_heads, group, rows, splits, workers;   // workers: 0 without caches
  int64_t capacity;
  const int32_t* lens;
  const float* part_o;
  const float* part_lse;
  const float* own_o;
  const float* own_lse;
  const float* scores;
  int64_t score_stride;
  float* weight;
  __nv_bfloat16* o;
  int64_t o_token, o_head;
  float* lse;
  int prefix_len;                     // in the caches' list: its keys, else 0
  int row_blocks, chunks;             // blocks of joined rows; weight chunks per plane
  // for rows that are summed up again (without_late_keys)
  const __nv_bfloat16* q;
  int64_t q_token, q_head;
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  float scale_log2;
};

constexpr int kJoinThreads = 128;
constexpr int kChunk = 4 * kJoinThreads;           // keys of a weight block

// Where one row's parts are: the prefix parts, then the segments of workers w0 .. w1.
struct Parts {
  int64_t prefix0, prefix_step, own0;
  int splits, count;
  __device__ __forceinline__ int64_t at(const JoinParams& p, int j) const {
    return j < splits ? prefix0 + j * prefix_step : own0 + int64_t(j - splits) * p.rows;
  }
  __device__ __forceinline__ float lse(const JoinParams& p, int j) const {
    return (j < splits ? p.part_lse : p.own_lse)[at(p, j)];
  }
};

// The list's length, and the cost of the sequences before b (whole warp).
__device__ __forceinline__ int list_length(const JoinParams& p, int b, int* before) {
  const int shared = p.prefix_len > 0 ? plane_cost(tiles_of(p.prefix_len)) : 0;
  return (count_cost(p.lens, p.B, p.capacity, b, before) + shared) * p.kv_heads;
}

__device__ __forceinline__ Parts parts_of(const JoinParams& p, int b, int kvh, int r, int n, int total, int before) {
  const Runs runs(total, p.workers);
  Parts x;
  const int t = r / p.group, g = r - t * p.group;
  const int64_t all = int64_t(p.B) * p.steps * p.group, row = (int64_t(b) * p.steps + t) * p.group + g;
  x.splits = p.splits;
  x.prefix0 = kvh * all + row;
  x.prefix_step = p.kv_heads * all;
  if (p.prefix_len > 0) {
    const int tiles = tiles_of(p.prefix_len), s0 = total - (p.kv_heads - kvh) * plane_cost(tiles);
    const int w0 = runs.worker(s0);
    x.splits = runs.worker(s0 + tiles - 1) - w0 + 1;
    x.prefix0 = (kvh + w0) * all + row;
    x.prefix_step = all;
  }
  x.count = x.splits;
  x.own0 = 0;
  const int tiles = tiles_of(n);
  if (tiles > 0) {
    const int s0 = before * p.kv_heads + kvh * plane_cost(tiles);
    const int w0 = runs.worker(s0), w1 = runs.worker(s0 + tiles - 1);
    x.own0 = (int64_t(b) * p.kv_heads + kvh + w0) * p.rows + r;
    x.count += w1 - w0 + 1;
  }
  return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

// log2 sum_j 2^(LSE_j) over a row's parts (whole warp; mine: part lane's); -inf when none has a key.
__device__ __forceinline__ float join_lse(const JoinParams& p, const Parts& x, float mine) {
  const int lane = threadIdx.x & 31;
  float top = mine;
  for (int j = lane + 32; j < x.count; j += 32) top = fmaxf(top, x.lse(p, j));
  top = warp_max(top);
  const float use = top == -INFINITY ? 0.f : top;
  float sum = ex2_approx(mine - use);
  for (int j = lane + 32; j < x.count; j += 32) sum += ex2_approx(x.lse(p, j) - use);
  sum = warp_sum(sum);
  return sum == 0.f ? -INFINITY : use + __log2f(sum);
}

// A lane's share of a row.
template <int V>
struct Share { float v[V]; };

template <int V>
__device__ __forceinline__ Share<V> load_bf16(const __nv_bfloat16* src) {
  Share<V> x;
#pragma unroll
  for (int e = 0; e < V; e += 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(src + e);
    x.v[e] = __uint_as_float(w << 16);
    x.v[e + 1] = __uint_as_float(w & 0xffff0000u);
  }
  return x;
}
__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

template <int V>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const float (&v)[V]) {
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(v[0], v[1]);
}

// Stores a token's row that came out not finite.  The cache pass multiplies V of whole tiles, and
// where V is not finite at a live key that only the step's later tokens see, zero, this row's
// weight there, times it is NaN.  Such columns are summed up again, in float32: the prefix's
// parts, and the cache keys that the row sees one by one.  Whole warp, a lane its D / 32 columns;
// out of line and last, so that the other rows do not pay for it.
template <int D>
__device__ __noinline__ void without_late_keys(const JoinParams& p, int row, int n, int total, int before, float lse, Share<D / 32> acc) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31, plane = row / p.rows, r = row - plane * p.rows;
  const int b = plane / p.kv_heads, kvh = plane - b * p.kv_heads, t = r / p.group, head = kvh * p.group + r - t * p.group;
  const int seen = n - p.steps + 1 + t > 0 ? n - p.steps + 1 + t : 0;
  const int64_t first = int64_t(plane) * p.capacity * D + lane * V, token = int64_t(b) * p.steps + t;
  bool late[V] = {}, some = false;
  for (int key = seen; key < n; ++key) {
    const Share<V> v = load_bf16<V>(p.v_cache + first + int64_t(key) * D);
#pragma unroll
    for (int e = 0; e < V; ++e) late[e] |= not_finite(v.v[e]) && not_finite(acc.v[e]);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) some |= late[e];
  if (__any_sync(kFull, some)) {
    const Parts x = parts_of(p, b, kvh, r, n, total, before);
    float sum[V] = {};
    for (int j = 0; j < x.splits; ++j) {
      const float a = ex2_approx(x.lse(p, j) - lse);
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] = fmaf(a, p.part_o[x.at(p, j) * D + lane * V + e], sum[e]);
    }
    const Share<V> q = load_bf16<V>(p.q + token * p.q_token + int64_t(head) * p.q_head + lane * V);
    for (int key = 0; key < seen; ++key) {
      const Share<V> k = load_bf16<V>(p.k_cache + first + int64_t(key) * D), v = load_bf16<V>(p.v_cache + first + int64_t(key) * D);
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) dot = fmaf(q.v[e], k.v[e], dot);
      const float a = ex2_approx(warp_sum(dot) * p.scale_log2 - lse);
      // (a weight is positive, if too small for a float)
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] = not_finite(v.v[e]) ? sum[e] + v.v[e] : fmaf(a, v.v[e], sum[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (late[e]) acc.v[e] = sum[e];
  }
  store_bf16<V>(p.o + token * p.o_token + int64_t(head) * p.o_head + lane * V, acc.v);
}

// WEIGHTS: blocks for the weights follow those of the rows.  SMALL: fewer O parts in flight, so that
// eight blocks fit an SM instead of four, for long lists of blocks over few parts (16 caches of
// up to 6,000 keys, 12 heads, 4 tokens: the call takes 77 us, 80 in the other form; 2 tokens over
// 5,448 shared keys in 22 parts take 23 us so, 21 in the other).
// LATE: several tokens a step; a look at the sums, 0 to 0.5 us a call (16 caches of up to 6,000
// keys, 12 heads, 4 tokens, with weights: 80.3 us, 79.9 without it).
template <int D, bool WEIGHTS, bool SMALL, bool LATE>
__global__ void __launch_bounds__(kJoinThreads, SMALL ? 8 : 4) join_kernel(const __grid_constant__ JoinParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!WEIGHTS || int(blockIdx.x) < p.row_blocks) {
    // One warp per row: O and LSE.
    const uint32_t row = blockIdx.x * (kJoinThreads / 32) + warp;
    if (row >= uint32_t(p.B) * p.kv_heads * p.rows) return;
    const uint32_t plane = row / uint32_t(p.rows);
    const int r = int(row - plane * p.rows);
    const int b = int(plane / uint32_t(p.kv_heads)), kvh = int(plane) - b * p.kv_heads;
    int before = 0, total = 0, n = 0;
    if (p.workers > 0) {
      n = live_len(p.lens, b, p.capacity);
      total = list_length(p, b, &before);
    }
    const Parts x = parts_of(p, b, kvh, r, n, total, before);
    const int t = r / p.group, head = kvh * p.group + (r - t * p.group);
    wait_prerequisites();                          // the caller's lengths needed no wait
    constexpr int V = D / 32, AHEAD = SMALL ? 4 : 16;
    auto load = [&](int j, float (&v)[V]) {
      const float* src = (j < x.splits ? p.part_o : p.own_o) + x.at(p, j) * D + lane * V;
      if constexpr (V == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        v[0] = f.x; v[1] = f.y;
      }
    };
    // The first parts' O loads do not wait for the weights.
    float first[AHEAD][V];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (j < x.count) load(j, first[j]);
    const float mine = lane < x.count ? x.lse(p, lane) : -INFINITY;
    float lse;
    if (x.count <= 32) {
      const float top = warp_max(mine), use = top == -INFINITY ? 0.f : top;
      const float sum = warp_sum(ex2_approx(mine - use));
      lse = sum == 0.f ? -INFINITY : use + __log2f(sum);
    } else {
      lse = join_lse(p, x, mine);
    }
    const float use = lse == -INFINITY ? 0.f : lse;
    float acc[V] = {};
    for (int j0 = 0; j0 < x.count; j0 += 32) {
      const int cnt = x.count - j0 < 32 ? x.count - j0 : 32;
      const float a = ex2_approx((j0 == 0 ? mine : lane < cnt ? x.lse(p, j0 + lane) : -INFINITY) - use);
      if (j0 == 0) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
          if (j < cnt) {
            const float w = __shfl_sync(kFull, a, j);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(w, first[j][e], acc[e]);
          }
      }
#pragma unroll 4
      for (int j = j0 == 0 ? AHEAD : 0; j < cnt; ++j) {
        const float w = __shfl_sync(kFull, a, j);
        float v[V];
        load(j0 + j, v);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(w, v[e], acc[e]);
      }
    }
    if (lane == 0) p.lse[(int64_t(b) * p.q_heads + head) * p.steps + t] = lse * kLn2;
    if constexpr (LATE) {
      bool odd = false;
#pragma unroll
      for (int e = 0; e < V; ++e) odd |= not_finite(acc[e]);
      if (__any_sync(kFull, odd)) {
        Share<V> all;
#pragma unroll
        for (int e = 0; e < V; ++e) all.v[e] = acc[e];
        without_late_keys<D>(p, int(row), n, total, before, use, all);
        return;
      }
    }
    store_bf16<V>(p.o + (int64_t(b) * p.steps + t) * p.o_token + int64_t(head) * p.o_head + lane * V, acc);
    return;
  }
  // A chunk of one plane's keys: the weight they collected.
  __shared__ float row_lse[kCacheMaxRows];
  const uint32_t job = blockIdx.x - uint32_t(p.row_blocks);
  const uint32_t plane = job / uint32_t(p.chunks);
  const int chunk = int(job - plane * p.chunks);
  const int b = int(plane / uint32_t(p.kv_heads)), kvh = int(plane) - b * p.kv_heads;
  const int n = live_len(p.lens, b, p.capacity);
  if (chunk * kChunk >= n) return;
  int before = 0;
  const int total = list_length(p, b, &before);
  wait_prerequisites();
  // The weights so far and the first rows' scores are on their way while the rows' LSE is joined.
  constexpr int AHEAD = 4;
  const int key = chunk * kChunk + threadIdx.x * 4;
  float old[4] = {};
  float* w = p.weight + plane * p.capacity + key;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (key + e < n) old[e] = w[e];
  const float* src = p.scores + int64_t(plane) * p.rows * p.score_stride + key;
  float4 next[AHEAD];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (r0 + i < p.rows && key < n) next[i] = *reinterpret_cast<const float4*>(src + (r0 + i) * p.score_stride);
  };
  load(0);
  // Four rows a warp, eight lanes over each row's parts (all rows of a plane have as many).
  for (int r0 = warp * 4; r0 < p.rows; r0 += kJoinThreads / 8) {
    const int r = r0 + lane / 8, l8 = lane % 8;
    const Parts x = parts_of(p, b, kvh, r < p.rows ? r : 0, n, total, before);
    const float mine = l8 < x.count ? x.lse(p, l8) : -INFINITY;
    float top = mine;
    for (int j = l8 + 8; j < x.count; j += 8) top = fmaxf(top, x.lse(p, j));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    const float use = top == -INFINITY ? 0.f : top;
    float sum = ex2_approx(mine - use);
    for (int j = l8 + 8; j < x.count; j += 8) sum += ex2_approx(x.lse(p, j) - use);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    // no weight where no part has a key: every score is -inf
    if (l8 == 0 && r < p.rows) row_lse[r] = sum == 0.f ? 0.f : use + __log2f(sum);
  }
  __syncthreads();
  if (key >= n) return;
  const int base = n - p.steps + 1;
  float sum[4] = {};
  for (int r0 = 0; r0 < p.rows; r0 += AHEAD) {
    float4 f[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) f[i] = next[i];
    load(r0 + AHEAD);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (r0 + i < p.rows) {
        const int lim = base + (r0 + i) / p.group;   // keys this row sees
        const float lse = row_lse[r0 + i];
        if (key < lim) sum[0] += ex2_approx(f[i].x - lse);
        if (key + 1 < lim) sum[1] += ex2_approx(f[i].y - lse);
        if (key + 2 < lim) sum[2] += ex2_approx(f[i].z - lse);
        if (key + 3 < lim) sum[3] += ex2_approx(f[i].w - lse);
      }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (key + e < n) w[e] = old[e] + sum[e];
}

template <int D, int NT, int WR, bool PREFIX>
cudaError_t launch_cfg(const CacheAttnArgs& a, cudaStream_t stream, const char** why) {
  using C = Cfg<D, NT, WR>;
  const int group = a.q_heads / a.kv_heads, tokens = a.B * a.steps;
  const int64_t rows = int64_t(a.B) * a.kv_heads * a.capacity;
  CacheMaps m = {};
  if (!make_heads_map(&m.q, a.q, tokens, a.q_heads, D, a.q_token, a.q_head, group, a.steps) ||
      !make_rows_map(&m.k, a.k_cache, rows, D, kTile) || !make_rows_map(&m.v, a.v_cache, rows, D, kTile) ||
      (PREFIX && (!make_heads_map(&m.all_q, a.q, tokens, a.q_heads, D, a.q_token, a.q_head, group, tokens) ||
                  !make_heads_map(&m.prefix_k, a.prefix_k, a.prefix_len, a.kv_heads, D, a.k_token, a.k_head, 1, kTile) ||
                  !make_heads_map(&m.prefix_v, a.prefix_v, a.prefix_len, a.kv_heads, D, a.v_token, a.v_head, 1, kTile)))) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  static DeviceFlags attr_set = {};
  const cudaError_t e = once_per_device(attr_set, [] {
    return cudaFuncSetAttribute(cache_attn_kernel<D, NT, WR, PREFIX>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  });
  if (e != cudaSuccess) { *why = "cudaFuncSetAttribute(max dynamic smem) failed"; return e; }
  const CacheParams p{a.B, a.steps, a.kv_heads, group, a.steps * group, a.capacity, a.lens,
                      a.scale * 1.4426950408889634f, a.own_o, a.own_lse, a.scores, a.score_stride, a.workers,
                      PREFIX ? int(a.prefix_len) : 0, PREFIX ? tokens * group : 0, a.part_o, a.part_lse, a.err};
  cache_attn_kernel<D, NT, WR, PREFIX><<<a.workers, C::THREADS, C::SMEM_BYTES, stream>>>(m, p);
  return cudaGetLastError();
}

template <int D, bool PREFIX>
cudaError_t launch_rows(const CacheAttnArgs& a, cudaStream_t stream, const char** why) {
  const int rows = (PREFIX ? a.B : 1) * a.steps * (a.q_heads / a.kv_heads);
  if (rows <= 8) return launch_cfg<D, 1, 1, PREFIX>(a, stream, why);
  if (rows <= 16) return launch_cfg<D, 2, 1, PREFIX>(a, stream, why);
  if (PREFIX || rows <= 32) return launch_cfg<D, 2, 2, PREFIX>(a, stream, why);   // PREFIX: at most kListMaxRows
  return launch_cfg<D, 2, 4, false>(a, stream, why);
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t stream, const char** why) {
  if (a.d == 128) return a.with_prefix ? launch_rows<128, true>(a, stream, why) : launch_rows<128, false>(a, stream, why);
  if (a.d == 64) return a.with_prefix ? launch_rows<64, true>(a, stream, why) : launch_rows<64, false>(a, stream, why);
  *why = "unsupported d";
  return cudaErrorInvalidValue;
}

cudaError_t launch_cache_join(const CacheAttnArgs& a, cudaStream_t stream) {
  const int group = a.q_heads / a.kv_heads, rows = a.steps * group;
  JoinParams p{a.B, a.steps, a.q_heads, a.kv_heads, group, rows, a.splits, a.capacity > 0 ? a.workers : 0, a.capacity, a.lens,
               a.part_o, a.part_lse, a.own_o, a.own_lse, a.scores, a.score_stride, a.weight,
               static_cast<__nv_bfloat16*>(a.o), a.o_token, a.o_head, a.lse, a.with_prefix ? int(a.prefix_len) : 0, 0, 0,
               static_cast<const __nv_bfloat16*>(a.q), a.q_token, a.q_head, static_cast<const __nv_bfloat16*>(a.k_cache),
               static_cast<const __nv_bfloat16*>(a.v_cache), a.scale * 1.4426950408889634f};
  const int64_t planes = int64_t(a.B) * a.kv_heads;
  p.row_blocks = int((planes * rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
  p.chunks = a.weight != nullptr ? int((a.capacity + kChunk - 1) / kChunk) : 0;
  const unsigned blocks = unsigned(p.row_blocks + planes * p.chunks);
  // more blocks than the large form has room for at once, and parts within the small one's loads
  const bool small = p.chunks > 0 && blocks > 4u * unsigned(sm_count()) && a.splits <= 4;
  auto launch = [&](auto kernel) { return launch_dependent(kernel, blocks, kJoinThreads, 0, stream, p); };
  auto form = [&](auto late) {
    constexpr bool LATE = decltype(late)::value;
    if (small) return a.d == 128 ? launch(join_kernel<128, true, true, LATE>) : launch(join_kernel<64, true, true, LATE>);
    if (p.chunks > 0) return a.d == 128 ? launch(join_kernel<128, true, false, LATE>) : launch(join_kernel<64, true, false, LATE>);
    return a.d == 128 ? launch(join_kernel<128, false, false, LATE>) : launch(join_kernel<64, false, false, LATE>);
  };
  return a.steps > 1 && a.capacity > 0 ? form(std::true_type{}) : form(std::false_type{});
}

}  // namespace lva
