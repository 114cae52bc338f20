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
// The bound is the cache's bytes from HBM (4 d per key and plane; a row costs 4 d flops per
// key, R <= 64 of them).  Work is cut without looking at single sequences: the 64-key tiles
// of all planes form one list, and each of kCacheWorkers CTAs (two per SM) takes an equal run
// of it, so ragged lengths balance by themselves.  A run may begin and end inside a plane;
// every (plane, worker) segment leaves its normalised O and LSE in float32.  Segments of the
// list, walked in order, raise the plane or the worker by one at each step, so plane + worker
// numbers their slots without a table.
//
//   cache_attn_kernel  warp 4: TMA producer (K and V tiles of 64 keys in one ring, the plane's
//                      Q rows in two slots); warps 0..3: mma.sync m16n8k16 on swizzled tiles.
//                      R <= 16 rows: each warp takes 16 of a tile's 64 keys; <= 32: two row
//                      halves by two key halves; <= 64: a row quarter each.  The tensor work
//                      is a small part of what mma.sync can do here (tcgen05 needs 128 rows).
//   join_kernel        LSE = log2 sum_j 2^(LSE_j), O = sum_j 2^(LSE_j - LSE) O_j over the
//                      row's prefix parts and segments, in float32, in a fixed order; and, on
//                      request, weight[c] += sum_r 2^(x_rc - LSE_r) from the scores the first
//                      kernel left (4 R bytes per key against 2 d for reading K again).
//                      Each weight has one writer and a fixed order of additions.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace lva {
namespace {

constexpr int kTile = 64;            // keys per tile
constexpr int kWarps = 4;            // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);
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
  int* err;
};

// Live entries of sequence b; a length outside [0, capacity] counts as none.
__device__ __forceinline__ int live_len(const int32_t* lens, int b, int64_t capacity) {
  const int32_t n = __ldg(lens + b);
  return n >= 0 && int64_t(n) <= capacity ? n : 0;
}
__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// Tiles of one head of all sequences, and of those before `stop` (whole warp).
__device__ __forceinline__ int64_t count_tiles(const int32_t* lens, int B, int64_t capacity, int stop, int64_t* before) {
  const int lane = threadIdx.x & 31;
  int64_t all = 0, part = 0;
  for (int b = lane; b < B; b += 32) {
    const int t = tiles_of(live_len(lens, b, capacity));
    all += t;
    if (b < stop) part += t;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(kFull, all, o);
    part += __shfl_xor_sync(kFull, part, o);
  }
  if (before != nullptr) *before = part;
  return all;
}

// Workers with a run in a list of `total` tiles (so that no run among them is empty), the
// first tile of worker w's run, and the worker whose run holds tile x: the largest w with
// run_start(w) <= x.
__device__ __forceinline__ int workers_of(int64_t total) { return total < kCacheWorkers ? int(total) : kCacheWorkers; }
__device__ __forceinline__ int64_t run_start(int64_t total, int w) { return total * w / workers_of(total); }
__device__ __forceinline__ int worker_of(int64_t total, int64_t x) {
  return int(((x + 1) * workers_of(total) - 1) / total);
}

// Walks a worker's run plane by plane (every warp the same walk).
struct Walk {
  const CacheParams& p;
  int64_t left;              // tiles of the run not yet handed out
  int b, kvh, n, tiles, t0;  // the current plane, its first tile of the run
  __device__ __forceinline__ Walk(const CacheParams& params, int worker) : p(params) {
    const int lane = threadIdx.x & 31;
    const int64_t total = count_tiles(p.lens, p.B, p.capacity, 0, nullptr) * p.kv_heads;
    left = 0;
    b = kvh = n = tiles = t0 = 0;
    if (worker >= workers_of(total)) return;
    int64_t at = run_start(total, worker);
    left = run_start(total, worker + 1) - at;
    // the sequence that holds tile `at`: 32 sequences at a time
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int mine = b0 + lane < p.B ? live_len(p.lens, b0 + lane, p.capacity) : 0;
      const int64_t own = int64_t(tiles_of(mine)) * p.kv_heads;
      int64_t sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += up;
      }
      const unsigned past = __ballot_sync(kFull, sum > at);
      if (past != 0) {
        const int l = __ffs(past) - 1;
        b = b0 + l;
        n = __shfl_sync(kFull, mine, l);
        const int64_t before = __shfl_sync(kFull, sum - own, l);
        tiles = tiles_of(n);
        const int64_t in = at - before;
        kvh = int(in / tiles);
        t0 = int(in - int64_t(kvh) * tiles);
        return;
      }
      at -= __shfl_sync(kFull, sum, 31);
    }
    left = 0;                // not reached: the run lies inside the list
  }
  // Tiles of the current plane in this run.
  __device__ __forceinline__ int count() const { return int(left < tiles - t0 ? left : tiles - t0); }
  __device__ __forceinline__ void next() {
    left -= count();
    t0 = 0;
    if (left <= 0) return;
    if (++kvh < p.kv_heads) return;
    kvh = 0;
    do {
      ++b;
      n = b < p.B ? live_len(p.lens, b, p.capacity) : 0;
    } while (b < p.B && n == 0);
    tiles = tiles_of(n);
    if (b >= p.B) left = 0;
  }
};

template <int D, int WR>
struct Cfg {
  static constexpr int WK = kWarps / WR;              // key groups
  static constexpr int KW = kTile / WK;               // keys of a tile per warp
  static constexpr int QROWS = 16 * WR;
  static constexpr int SLOT = kTile * D * 2;          // one K or V tile
  // Ring slots: 80 KB (64 KB with more rows, for their Q and join space) in flight per CTA,
  // two CTAs per SM; about 70 KB per SM cover the latency at the full HBM rate.
  static constexpr int NSLOT = (WR == 1 ? 5 : 4) * (128 / D);
  static constexpr int Q_SLOT = QROWS * D * 2;
  static constexpr int FRAG = D / 8 * 4;              // O registers per lane
  static constexpr int JOIN_WARPS = kWarps / 2;
  static constexpr int JOIN = WK > 1 ? JOIN_WARPS * (FRAG + 4) * 32 * 4 : 0;
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_Q = OFF_KV + NSLOT * SLOT;
  static constexpr int OFF_JOIN = OFF_Q + 2 * Q_SLOT;
  static constexpr int OFF_BAR = OFF_JOIN + JOIN;
  static constexpr int B_F = 0, B_E = NSLOT, B_QF = 2 * NSLOT, B_QE = B_QF + 2, B_GRP = B_QE + 2, NUM_BARS = B_GRP + 2;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16;
  static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
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

template <int D, int WR>
__global__ void __launch_bounds__(kThreads, 2) cache_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                                 const __grid_constant__ CUtensorMap tm_k,
                                                                 const __grid_constant__ CUtensorMap tm_v,
                                                                 const CacheParams p) {
  using C = Cfg<D, WR>;
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
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      const int32_t n = __ldg(p.lens + b);
      if (n < 0 || int64_t(n) > p.capacity) report_fault(p.err, 1, b);
    }
  // Q rows past the group's are never loaded: zero, so that no stray value is computed with.
  for (int x = threadIdx.x; x < 2 * C::Q_SLOT / 16; x += kThreads)
    reinterpret_cast<uint4*>(smem + C::OFF_Q)[x] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NSLOT; ++s) { mbar_init(bar_full(s), 1); mbar_init(bar_empty(s), kWarps); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_q_full(s), 1);
      mbar_init(bar_q_empty(s), kWarps);
      mbar_init(bar0 + 8u * (C::B_GRP + s), kWarps);
    }
    *abort_flag = 0;
    *never = 0;
    mbar_fence_init();
  }
  __syncthreads();
  Walk walk(p, worker);

  if (warp == kWarps) {
    // ------------------------------------------------------------ TMA producer
    uint32_t u = 0;                               // ring position: K of tile T at 2T, V at 2T + 1
    uint32_t seg = 0, loaded_q = 0;
    bool ok = true;
    if (lane == 0 && walk.left > 0) { tma_prefetch_desc(&tm_q); tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v); }
    for (; ok && walk.left > 0; walk.next(), ++seg) {
      if (lane == 0) {
        const int qs = int(seg & 1);
        ok = seg < 2 || mbar_wait_sleep(bar_q_empty(qs), ((seg >> 1) - 1) & 1, abort_flag);
        if (ok) {
          mbar_arrive_expect_tx(bar_q_full(qs), uint32_t(p.rows * D * 2));
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(s_base + C::OFF_Q + qs * C::Q_SLOT + c * C::QROWS * 128, &tm_q, c * 64, walk.kvh * p.group,
                        walk.b * p.steps, bar_q_full(qs));
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
            for (int c = 0; c < D / 64; ++c)
              tma_load_2d(s_base + C::OFF_KV + s * C::SLOT + c * kTile * 128, kv == 0 ? &tm_k : &tm_v, c * 64, row,
                          bar_full(s));
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
      for (uint32_t x = loaded_q > 2 ? loaded_q - 2 : 0; x < loaded_q; ++x) mbar_wait(bar_q_full(int(x & 1)), (x >> 1) & 1, never);
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int wr = warp % WR, wk = warp / WR;
    const int g = lane >> 2, q4 = lane & 3;        // fragment row and column group
    const float c = p.scale_log2;
    const int row_a = wr * 16 + g, row_b = row_a + 8;
    const int tok_a = row_a / p.group, tok_b = row_b / p.group;
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
      const int qs = int(seg & 1);
      ok = __all_sync(kFull, mbar_wait(bar_q_full(qs), (seg >> 1) & 1, abort_flag));
      if (!ok) break;
      uint32_t qf[D / 16][4];
      {
        const uint32_t qb = s_base + C::OFF_Q + qs * C::Q_SLOT;
        const int r = wr * 16 + (lane & 15);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ldsm4(sw(qb + (k / 4) * C::QROWS * 128, r, (k % 4) * 2 + (lane >> 4)), qf[k]);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_q_empty(qs));
      }
      float of[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) of[i][0] = of[i][1] = of[i][2] = of[i][3] = 0.f;
      float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
      const int64_t plane = int64_t(walk.b) * p.kv_heads + walk.kvh;
      // keys each of this thread's two rows sees
      const int base = walk.n - p.steps + 1;
      const int lim_a = row_a < p.rows ? base + tok_a : 0, lim_b = row_b < p.rows ? base + tok_b : 0;
      const int cnt = walk.count();
      for (int t = 0; t < cnt; ++t, ++T) {
        const int key0 = (walk.t0 + t) * kTile + wk * C::KW;       // this warp's first key
        const uint32_t uk = 2 * T, uv = 2 * T + 1;
        const int ks = int(uk % C::NSLOT), vs = int(uv % C::NSLOT);
        ok = __all_sync(kFull, mbar_wait(bar_full(ks), (uk / C::NSLOT) & 1, abort_flag));
        if (!ok) break;
        const bool any = key0 < walk.n;                            // warp-uniform
        float sf[C::KW / 8][4];
        if (any) {
          const uint32_t kb = s_base + C::OFF_KV + ks * C::SLOT;
#pragma unroll
          for (int i = 0; i < C::KW / 8; ++i) sf[i][0] = sf[i][1] = sf[i][2] = sf[i][3] = 0.f;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
#pragma unroll
            for (int i = 0; i < C::KW / 16; ++i) {
              // lanes 0-7, 8-15: keys 0-7 at k, k + 8; lanes 16-31: keys 8-15
              const int r = wk * C::KW + i * 16 + (lane & 7) + ((lane >> 4) << 3);
              uint32_t kf[4];
              ldsm4(sw(kb + (k / 4) * kTile * 128, r, (k % 4) * 2 + ((lane >> 3) & 1)), kf);
              mma16816(sf[2 * i], qf[k], kf[0], kf[1]);
              mma16816(sf[2 * i + 1], qf[k], kf[2], kf[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty(ks));
        uint32_t pf[C::KW / 8][2];
        if (any) {
          float mx_a = -INFINITY, mx_b = -INFINITY;
          const bool masked = key0 + C::KW > base;                 // some row does not see every key
#pragma unroll
          for (int i = 0; i < C::KW / 8; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sf[i][e] *= c;
            if (p.scores != nullptr) {
              const int key = key0 + i * 8 + q4 * 2;
              float* dst = p.scores + (plane * p.rows) * p.score_stride + key;
              if (row_a < p.rows) *reinterpret_cast<float2*>(dst + row_a * p.score_stride) = make_float2(sf[i][0], sf[i][1]);
              if (row_b < p.rows) *reinterpret_cast<float2*>(dst + row_b * p.score_stride) = make_float2(sf[i][2], sf[i][3]);
            }
            if (masked) {
              const int key = key0 + i * 8 + q4 * 2;
              if (key >= lim_a) sf[i][0] = -INFINITY;
              if (key + 1 >= lim_a) sf[i][1] = -INFINITY;
              if (key >= lim_b) sf[i][2] = -INFINITY;
              if (key + 1 >= lim_b) sf[i][3] = -INFINITY;
            }
            mx_a = fmaxf(mx_a, fmaxf(sf[i][0], sf[i][1]));
            mx_b = fmaxf(mx_b, fmaxf(sf[i][2], sf[i][3]));
          }
          mx_a = fmaxf(mx_a, __shfl_xor_sync(kFull, mx_a, 1));
          mx_b = fmaxf(mx_b, __shfl_xor_sync(kFull, mx_b, 1));
          mx_a = fmaxf(mx_a, __shfl_xor_sync(kFull, mx_a, 2));
          mx_b = fmaxf(mx_b, __shfl_xor_sync(kFull, mx_b, 2));
          // the reference moves only when a maximum outgrows it by 2^8 (weights stay in range)
          const float old_a = m_a, old_b = m_b;
          if (mx_a > m_a + kRescaleThreshold || m_a == -INFINITY) m_a = fmaxf(m_a, mx_a);
          if (mx_b > m_b + kRescaleThreshold || m_b == -INFINITY) m_b = fmaxf(m_b, mx_b);
          if (__any_sync(kFull, m_a != old_a || m_b != old_b)) {
            const float al_a = m_a == old_a ? 1.f : ex2_approx(old_a - m_a);
            const float al_b = m_b == old_b ? 1.f : ex2_approx(old_b - m_b);
            l_a *= al_a;
            l_b *= al_b;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) { of[i][0] *= al_a; of[i][1] *= al_a; of[i][2] *= al_b; of[i][3] *= al_b; }
          }
          const float u_a = m_a == -INFINITY ? 0.f : m_a, u_b = m_b == -INFINITY ? 0.f : m_b;
#pragma unroll
          for (int i = 0; i < C::KW / 8; ++i) {
            const float p0 = ex2_approx(sf[i][0] - u_a), p1 = ex2_approx(sf[i][1] - u_a);
            const float p2 = ex2_approx(sf[i][2] - u_b), p3 = ex2_approx(sf[i][3] - u_b);
            l_a += p0 + p1;
            l_b += p2 + p3;
            pf[i][0] = pack_bf16x2(p0, p1);        // P in bf16: the MMA's operand type
            pf[i][1] = pack_bf16x2(p2, p3);
          }
        }
        ok = __all_sync(kFull, mbar_wait(bar_full(vs), (uv / C::NSLOT) & 1, abort_flag));
        if (!ok) break;
        const bool tail = (walk.t0 + t + 1) * kTile > walk.n;      // the plane's last, partial tile
        if (any) {
          uint8_t* vt = smem + C::OFF_KV + vs * C::SLOT;
          if (tail) {
            // V rows past the live ones may hold anything: zero, so that 0 * NaN never is
            for (int ch = 0; ch < D / 64; ++ch)
              for (int x = lane; x < C::KW * 8; x += 32) {
                const int r = wk * C::KW + (x >> 3);
                if ((walk.t0 + t) * kTile + r >= walk.n)
                  *reinterpret_cast<uint4*>(vt + ch * kTile * 128 + r * 128 + ((x & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
              }
            __syncwarp();
          }
          const uint32_t vb = s_base + C::OFF_KV + vs * C::SLOT;
#pragma unroll
          for (int k = 0; k < C::KW / 16; ++k) {
            const uint32_t af[4] = {pf[2 * k][0], pf[2 * k][1], pf[2 * k + 1][0], pf[2 * k + 1][1]};
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              // lanes 0-15: keys 0-15 at dims i*16; lanes 16-31: the same keys, dims + 8
              const int r = wk * C::KW + k * 16 + (lane & 15);
              uint32_t vf[4];
              ldsm4_t(sw(vb + (i / 4) * kTile * 128, r, (i % 4) * 2 + (lane >> 4)), vf);
              mma16816(of[2 * i], af, vf[0], vf[1]);
              mma16816(of[2 * i + 1], af, vf[2], vf[3]);
            }
          }
          if (tail) fence_proxy_async_smem();      // the zeros before the slot's next TMA write
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty(vs));
      }
      if (!ok) break;

      // Row sums over the quad; then the key groups meet, upper half into lower half.
      l_a += __shfl_xor_sync(kFull, l_a, 1);
      l_b += __shfl_xor_sync(kFull, l_b, 1);
      l_a += __shfl_xor_sync(kFull, l_a, 2);
      l_b += __shfl_xor_sync(kFull, l_b, 2);
      if constexpr (C::WK > 1) {
        auto slot = [&](int i) { return reinterpret_cast<float*>(smem + C::OFF_JOIN) + i * (C::FRAG + 4) * 32 + lane; };
        auto put = [&](int i) {
          float* s = slot(i);
#pragma unroll
          for (int x = 0; x < D / 8; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[(4 * x + e) * 32] = of[x][e];
          s[C::FRAG * 32] = m_a;
          s[(C::FRAG + 1) * 32] = m_b;
          s[(C::FRAG + 2) * 32] = l_a;
          s[(C::FRAG + 3) * 32] = l_b;
        };
        auto add = [&](int i) {
          const float* s = slot(i);
          const float n_a = s[C::FRAG * 32], n_b = s[(C::FRAG + 1) * 32];
          const float t_a = fmaxf(m_a, n_a), t_b = fmaxf(m_b, n_b);
          const float u_a = t_a == -INFINITY ? 0.f : t_a, u_b = t_b == -INFINITY ? 0.f : t_b;
          const float x_a = ex2_approx(m_a - u_a), x_b = ex2_approx(m_b - u_b);
          const float y_a = ex2_approx(n_a - u_a), y_b = ex2_approx(n_b - u_b);
          l_a = l_a * x_a + s[(C::FRAG + 2) * 32] * y_a;
          l_b = l_b * x_b + s[(C::FRAG + 3) * 32] * y_b;
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            of[x][0] = of[x][0] * x_a + s[(4 * x) * 32] * y_a;
            of[x][1] = of[x][1] * x_a + s[(4 * x + 1) * 32] * y_a;
            of[x][2] = of[x][2] * x_b + s[(4 * x + 2) * 32] * y_b;
            of[x][3] = of[x][3] * x_b + s[(4 * x + 3) * 32] * y_b;
          }
          m_a = t_a;
          m_b = t_b;
        };
        // warps 2, 3 into 0, 1 (their keys two groups on, or one with two row halves)
        if (warp >= 2) put(warp - 2);
        ok = group_sync();
        if (ok && warp < 2) add(warp);
        if constexpr (C::WK == 4) {
          if (ok && warp == 1) put(1);             // its own slot: only this warp has read it
          ok = ok && group_sync();
          if (ok && warp == 0) add(1);
        }
        ok = ok && group_sync();                   // the slots may be written again
        if (!ok) break;
      }
      if (wk == 0) {
        const int64_t at = (plane + worker) * p.rows;
        const bool none_a = l_a == 0.f, none_b = l_b == 0.f;       // a NaN sum goes through as NaN
        const float inv_a = none_a ? 0.f : 1.f / l_a, inv_b = none_b ? 0.f : 1.f / l_b;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          const int col = x * 8 + q4 * 2;
          if (row_a < p.rows)
            *reinterpret_cast<float2*>(p.own_o + (at + row_a) * D + col) =
                none_a ? make_float2(0.f, 0.f) : make_float2(of[x][0] * inv_a, of[x][1] * inv_a);
          if (row_b < p.rows)
            *reinterpret_cast<float2*>(p.own_o + (at + row_b) * D + col) =
                none_b ? make_float2(0.f, 0.f) : make_float2(of[x][2] * inv_b, of[x][3] * inv_b);
        }
        if (q4 == 0) {
          if (row_a < p.rows) p.own_lse[at + row_a] = none_a ? -INFINITY : m_a + __log2f(l_a);
          if (row_b < p.rows) p.own_lse[at + row_b] = none_b ? -INFINITY : m_b + __log2f(l_b);
        }
      }
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) report_fault(p.err, 5, 32);
    }
  }
}

struct JoinParams {
  int B, steps, q_heads, kv_heads, group, rows, splits, has_cache;
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
  int row_blocks, chunks;             // blocks of joined rows; weight chunks per plane
};

constexpr int kJoinThreads = 128;
constexpr int kChunk = 4 * kJoinThreads;           // keys of a weight block

// Where one row's parts are: the prefix parts, then the segments of workers w0 .. w1.
struct Parts {
  int64_t prefix0, prefix_step, own0, own_step;
  int splits, count;
  __device__ __forceinline__ float lse(const JoinParams& p, int j) const {
    return j < splits ? __ldg(p.part_lse + prefix0 + j * prefix_step) : __ldg(p.own_lse + own0 + (j - splits) * own_step);
  }
  __device__ __forceinline__ const float* o(const JoinParams& p, int j, int d) const {
    return j < splits ? p.part_o + (prefix0 + j * prefix_step) * d : p.own_o + (own0 + (j - splits) * own_step) * d;
  }
};

__device__ __forceinline__ Parts parts_of(const JoinParams& p, int b, int kvh, int r, int64_t total, int64_t before) {
  Parts x;
  const int t = r / p.group, g = r - t * p.group;
  x.splits = p.splits;
  x.prefix0 = (int64_t(kvh) * p.B * p.steps + int64_t(b) * p.steps + t) * p.group + g;
  x.prefix_step = int64_t(p.kv_heads) * p.B * p.steps * p.group;
  x.count = p.splits;
  x.own0 = 0;
  x.own_step = p.rows;
  const int tiles = p.has_cache ? tiles_of(live_len(p.lens, b, p.capacity)) : 0;
  if (tiles > 0) {
    const int64_t s0 = (before * p.kv_heads) + int64_t(kvh) * tiles;
    const int w0 = worker_of(total, s0), w1 = worker_of(total, s0 + tiles - 1);
    x.own0 = (int64_t(b) * p.kv_heads + kvh + w0) * p.rows + r;
    x.count += w1 - w0 + 1;
  }
  return x;
}

// log2 sum_j 2^(LSE_j) over a row's parts (whole warp); -inf when none has a key.
__device__ __forceinline__ float join_lse(const JoinParams& p, const Parts& x) {
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int j = lane; j < x.count; j += 32) top = fmaxf(top, x.lse(p, j));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  const float use = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int j = lane; j < x.count; j += 32) sum += ex2_approx(x.lse(p, j) - use);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  return sum == 0.f ? -INFINITY : use + __log2f(sum);
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const JoinParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (int(blockIdx.x) < p.row_blocks) {
    // One warp per row: O and LSE.
    const int64_t row = int64_t(blockIdx.x) * (kJoinThreads / 32) + warp;
    if (row >= int64_t(p.B) * p.kv_heads * p.rows) return;
    const int r = int(row % p.rows);
    const int64_t plane = row / p.rows;
    const int b = int(plane / p.kv_heads), kvh = int(plane - int64_t(b) * p.kv_heads);
    int64_t before = 0, total = 0;
    if (p.has_cache) total = count_tiles(p.lens, p.B, p.capacity, b, &before) * p.kv_heads;
    const Parts x = parts_of(p, b, kvh, r, total, before);
    const float lse = join_lse(p, x);
    const float use = lse == -INFINITY ? 0.f : lse;
    constexpr int V = D / 32;
    float acc[V] = {};
    for (int j0 = 0; j0 < x.count; j0 += 32) {
      const int cnt = x.count - j0 < 32 ? x.count - j0 : 32;
      const float a = lane < cnt ? ex2_approx(x.lse(p, j0 + lane) - use) : 0.f;
#pragma unroll 4
      for (int j = 0; j < cnt; ++j) {
        const float w = __shfl_sync(kFull, a, j);
        const float* src = x.o(p, j0 + j, D) + lane * V;
        float v[V];
        if constexpr (V == 4) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(src));
          v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
          const float2 f = __ldg(reinterpret_cast<const float2*>(src));
          v[0] = f.x; v[1] = f.y;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(w, v[e], acc[e]);
      }
    }
    const int t = r / p.group, head = kvh * p.group + (r - t * p.group);
    __nv_bfloat16* dst = p.o + (int64_t(b) * p.steps + t) * p.o_token + int64_t(head) * p.o_head + lane * V;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
    else
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0], acc[1]);
    if (lane == 0) p.lse[(int64_t(b) * p.q_heads + head) * p.steps + t] = lse * kLn2;
    return;
  }
  // A chunk of one plane's keys: the weight they collected.
  __shared__ float row_lse[kCacheMaxRows];
  const int64_t job = int64_t(blockIdx.x) - p.row_blocks;
  const int64_t plane = job / p.chunks;
  const int chunk = int(job - plane * p.chunks);
  const int b = int(plane / p.kv_heads), kvh = int(plane - int64_t(b) * p.kv_heads);
  const int n = live_len(p.lens, b, p.capacity);
  if (int64_t(chunk) * kChunk >= n) return;
  int64_t before = 0;
  const int64_t total = count_tiles(p.lens, p.B, p.capacity, b, &before) * p.kv_heads;
  for (int r = warp; r < p.rows; r += kJoinThreads / 32) {
    const float lse = join_lse(p, parts_of(p, b, kvh, r, total, before));
    if (lane == 0) row_lse[r] = lse == -INFINITY ? 0.f : lse;      // no weight: every score is -inf
  }
  __syncthreads();
  const int key = chunk * kChunk + threadIdx.x * 4;
  if (key >= n) return;
  const float* src = p.scores + plane * p.rows * p.score_stride + key;
  const int base = n - p.steps + 1;
  float sum[4] = {};
  for (int r = 0; r < p.rows; ++r) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(src + r * p.score_stride));
    const int lim = base + r / p.group;            // keys this row sees
    const float lse = row_lse[r];
    if (key < lim) sum[0] += ex2_approx(f.x - lse);
    if (key + 1 < lim) sum[1] += ex2_approx(f.y - lse);
    if (key + 2 < lim) sum[2] += ex2_approx(f.z - lse);
    if (key + 3 < lim) sum[3] += ex2_approx(f.w - lse);
  }
  float* w = p.weight + plane * p.capacity + key;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (key + e < n) w[e] += sum[e];
}

template <int D, int WR>
cudaError_t launch_cfg(const CacheAttnArgs& a, cudaStream_t stream, const char** why) {
  using C = Cfg<D, WR>;
  const int group = a.q_heads / a.kv_heads;
  const int64_t rows = int64_t(a.B) * a.kv_heads * a.capacity;
  CUtensorMap tq, tk, tv;
  if (!make_heads_map(&tq, a.q, int64_t(a.B) * a.steps, a.q_heads, D, a.q_token, a.q_head, group, a.steps) ||
      !make_rows_map(&tk, a.k_cache, rows, D, kTile) || !make_rows_map(&tv, a.v_cache, rows, D, kTile)) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  static DeviceFlags attr_set = {};
  const cudaError_t e = once_per_device(attr_set, [] {
    return cudaFuncSetAttribute(cache_attn_kernel<D, WR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  });
  if (e != cudaSuccess) { *why = "cudaFuncSetAttribute(max dynamic smem) failed"; return e; }
  const CacheParams p{a.B, a.steps, a.kv_heads, group, a.steps * group, a.capacity, a.lens,
                      a.scale * 1.4426950408889634f, a.own_o, a.own_lse, a.scores, a.score_stride, a.err};
  cache_attn_kernel<D, WR><<<kCacheWorkers, kThreads, C::SMEM_BYTES, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_rows(const CacheAttnArgs& a, cudaStream_t stream, const char** why) {
  const int rows = a.steps * (a.q_heads / a.kv_heads);
  if (rows <= 16) return launch_cfg<D, 1>(a, stream, why);
  if (rows <= 32) return launch_cfg<D, 2>(a, stream, why);
  return launch_cfg<D, 4>(a, stream, why);
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t stream, const char** why) {
  if (a.d == 128) return launch_rows<128>(a, stream, why);
  if (a.d == 64) return launch_rows<64>(a, stream, why);
  *why = "unsupported d";
  return cudaErrorInvalidValue;
}

cudaError_t launch_cache_join(const CacheAttnArgs& a, cudaStream_t stream) {
  const int group = a.q_heads / a.kv_heads, rows = a.steps * group;
  JoinParams p{a.B, a.steps, a.q_heads, a.kv_heads, group, rows, a.splits, a.capacity > 0 ? 1 : 0, a.capacity, a.lens,
               a.part_o, a.part_lse, a.own_o, a.own_lse, a.scores, a.score_stride, a.weight,
               static_cast<__nv_bfloat16*>(a.o), a.o_token, a.o_head, a.lse, 0, 0};
  const int64_t planes = int64_t(a.B) * a.kv_heads;
  p.row_blocks = int((planes * rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
  p.chunks = a.weight != nullptr ? int((a.capacity + kChunk - 1) / kChunk) : 0;
  const int64_t blocks = p.row_blocks + planes * p.chunks;
  if (a.d == 128) join_kernel<128><<<unsigned(blocks), kJoinThreads, 0, stream>>>(p);
  else join_kernel<64><<<unsigned(blocks), kJoinThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace lva
