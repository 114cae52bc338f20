// api.cu -- the C ABI declared in include/lva.h: argument checks, status codes, the
// per-thread error message, the per-device kernel error word, and dispatch to launchers.
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "kernels.h"
#include "lva.h"

namespace lva {
namespace {

thread_local char g_msg[256] = "";

lva_status fail(lva_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

lva_status ok() {
  g_msg[0] = '\0';
  return LVA_OK;
}

lva_status from_cuda(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  return fail(LVA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Kernel-side error word: [0] = status, [1] = detail, read and written as one 64-bit word.
// One copy per device (module global); its device address is looked up once per device (on
// every call past the cache).
__device__ __align__(8) int g_device_error[2];

// Where lva_device_error's exchange kernel leaves the word it took.
__device__ unsigned long long g_device_error_taken;

// Takes the error word and clears it in one atomic exchange, so a fault recorded by a
// kernel on another stream at the same moment is either taken now or left for the next
// read, never lost.
__global__ void take_error_kernel(unsigned long long* word) {
  g_device_error_taken = atomicExch(word, 0ull);
}

// lva_device_error calls are serialised: they share the taken-word slot of a device.
std::mutex g_take_mutex;

std::atomic<int*> g_err_ptr[kMaxCachedDevices] = {};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

lva_status set_error_message(lva_status status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return status;
}

int* device_error_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  const bool cacheable = dev >= 0 && dev < kMaxCachedDevices;
  if (cacheable) {
    int* cached = g_err_ptr[dev].load(std::memory_order_acquire);
    if (cached != nullptr) return cached;
  }
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
  if (cacheable) g_err_ptr[dev].store(static_cast<int*>(p), std::memory_order_release);
  return static_cast<int*>(p);
}

}  // namespace lva

using namespace lva;

extern "C" {

const char* lva_status_string(lva_status s) {
  switch (s) {
    case LVA_OK: return "LVA_OK";
    case LVA_ERR_INVALID_ARG: return "LVA_ERR_INVALID_ARG";
    case LVA_ERR_UNSUPPORTED: return "LVA_ERR_UNSUPPORTED";
    case LVA_ERR_CAPACITY: return "LVA_ERR_CAPACITY";
    case LVA_ERR_CUDA: return "LVA_ERR_CUDA";
    case LVA_ERR_TIMEOUT: return "LVA_ERR_TIMEOUT";
  }
  return "LVA_ERR_UNKNOWN";
}

const char* lva_last_error_message(void) { return g_msg; }

int lva_version(void) { return LVA_VERSION; }

lva_status lva_reorder_tokens(const void* src, void* dst, int64_t planes, int T, int H, int W,
                              int tile_t, int tile_h, int tile_w, int64_t n_pad, int64_t row_elems,
                              int elem_bytes, int inverse, cudaStream_t stream) {
  if (planes < 0) return fail(LVA_ERR_INVALID_ARG, "reorder: planes < 0");
  if (T <= 0 || H <= 0 || W <= 0 || tile_t <= 0 || tile_h <= 0 || tile_w <= 0)
    return fail(LVA_ERR_INVALID_ARG, "reorder: grid and tile sizes must be positive");
  if (elem_bytes != 2 && elem_bytes != 4) return fail(LVA_ERR_INVALID_ARG, "reorder: elem_bytes must be 2 or 4");
  if (row_elems <= 0) return fail(LVA_ERR_INVALID_ARG, "reorder: row_elems must be positive");
  const int64_t n = int64_t(T) * H * W;
  if (n >= (int64_t(1) << 31)) return fail(LVA_ERR_UNSUPPORTED, "reorder: T*H*W must be < 2^31");
  if (n_pad < n || n_pad >= (int64_t(1) << 31)) return fail(LVA_ERR_INVALID_ARG, "reorder: need T*H*W <= n_pad < 2^31");
  const int64_t row_bytes = row_elems * elem_bytes;
  if (row_bytes > (int64_t(1) << 20)) return fail(LVA_ERR_UNSUPPORTED, "reorder: rows above 1 MiB");
  // One thread per (row, chunk); chunks are at least elem_bytes wide, and the launch's
  // blocks of 256 threads must fit gridDim.x.
  if ((n_pad * row_elems + 255) / 256 > int64_t(0x7fffffff))
    return fail(LVA_ERR_UNSUPPORTED, "reorder: n_pad * row_elems too large for one launch");
  if (planes == 0) return ok();
  if (src == nullptr || dst == nullptr) return fail(LVA_ERR_INVALID_ARG, "reorder: null pointer");
  if (!aligned(src, elem_bytes) || !aligned(dst, elem_bytes))
    return fail(LVA_ERR_INVALID_ARG, "reorder: pointers must be aligned to elem_bytes");
  ReorderArgs a{src, dst, planes, T, H, W, tile_t, tile_h, tile_w, n, n_pad, row_bytes, inverse != 0};
  return from_cuda(launch_reorder(a, stream), "reorder launch");
}

static lva_status check_mask_params(const lva_mask_params* p) {
  if (p == nullptr) return fail(LVA_ERR_INVALID_ARG, "mask: null params");
  if (p->block_size != 64 && p->block_size != 128) return fail(LVA_ERR_UNSUPPORTED, "mask: block_size must be 64 or 128");
  if (p->n_pad <= 0 || p->n_pad % p->block_size != 0) return fail(LVA_ERR_INVALID_ARG, "mask: n_pad must be a positive multiple of block_size");
  if (p->n_valid < 1 || p->n_valid > p->n_pad) return fail(LVA_ERR_INVALID_ARG, "mask: need 1 <= n_valid <= n_pad");
  if (p->mask_heads < 1) return fail(LVA_ERR_INVALID_ARG, "mask: mask_heads must be >= 1");
  const int64_t nb = p->n_pad / p->block_size;
  if (int64_t(p->mask_heads) * nb * nb >= (int64_t(1) << 31))
    return fail(LVA_ERR_UNSUPPORTED, "mask: mask_heads*nb*nb must be < 2^31");
  switch (p->kind) {
    case LVA_MASK_WINDOW_ANCHOR:
      if (p->window_unit_tokens < 1 || p->window_radius < 0 || p->num_anchors < 0 || p->step < 0)
        return fail(LVA_ERR_INVALID_ARG, "mask: window needs unit >= 1, radius >= 0, anchors >= 0, step >= 0");
      if (p->num_anchors > nb) return fail(LVA_ERR_INVALID_ARG, "mask: more anchors than blocks");
      if (p->mask_heads != 1) return fail(LVA_ERR_INVALID_ARG, "mask: parametric kinds build one mask head");
      break;
    case LVA_MASK_TWO_STAGE:
      if (p->group_blocks < 1) return fail(LVA_ERR_INVALID_ARG, "mask: group_blocks must be >= 1");
      if (p->mask_heads != 1) return fail(LVA_ERR_INVALID_ARG, "mask: parametric kinds build one mask head");
      break;
    case LVA_MASK_ALL:
      if (p->mask_heads != 1) return fail(LVA_ERR_INVALID_ARG, "mask: parametric kinds build one mask head");
      break;
    case LVA_MASK_LVSA_FRAMES: {
      if (p->window_unit_tokens < 1 || p->num_anchors < 0 || p->step < 0 || p->budget_frames < 1)
        return fail(LVA_ERR_INVALID_ARG, "mask: LVSA frames need unit >= 1, anchors >= 0, step >= 0, budget >= 1");
      const int64_t frames = (p->n_valid + p->window_unit_tokens - 1) / p->window_unit_tokens;
      if (p->num_anchors > frames) return fail(LVA_ERR_INVALID_ARG, "mask: more global frames than frames");
      if (p->mask_heads != 1) return fail(LVA_ERR_INVALID_ARG, "mask: parametric kinds build one mask head");
      break;
    }
    case LVA_MASK_STATIC:
      break;
    default:
      return fail(LVA_ERR_INVALID_ARG, "mask: unknown kind %d", p->kind);
  }
  return ok();
}

int64_t lva_block_mask_max_nnz(const lva_mask_params* p) {
  if (check_mask_params(p) != LVA_OK) return 0;
  const int64_t nb = p->n_pad / p->block_size;
  return int64_t(p->mask_heads) * nb * nb;
}

// Checks shared by both mask-build calls; fills the launcher arguments.
static lva_status mask_args(const lva_mask_params* p, const uint8_t* dense_mask, int32_t* row_ptr,
                            int32_t* col_idx, int64_t col_capacity, int32_t* nnz_out, MaskArgs* a) {
  lva_status s = check_mask_params(p);
  if (s != LVA_OK) return s;
  if (row_ptr == nullptr || col_idx == nullptr || nnz_out == nullptr)
    return fail(LVA_ERR_INVALID_ARG, "mask: null output pointer");
  if (!aligned(row_ptr, 4) || !aligned(col_idx, 4) || !aligned(nnz_out, 4))
    return fail(LVA_ERR_INVALID_ARG, "mask: outputs must be 4-byte aligned");
  if (p->kind == LVA_MASK_STATIC && dense_mask == nullptr)
    return fail(LVA_ERR_INVALID_ARG, "mask: STATIC needs dense_mask");
  const int64_t need = lva_block_mask_max_nnz(p);
  if (col_capacity < need)
    return fail(LVA_ERR_CAPACITY, "mask: col_capacity %lld < %lld", (long long)col_capacity, (long long)need);
  a->kind = p->kind;
  a->mask_heads = p->mask_heads;
  a->block_size = p->block_size;
  a->n_pad = p->n_pad;
  a->n_valid = p->n_valid;
  a->unit_tokens = p->window_unit_tokens;
  a->radius = p->window_radius;
  a->num_anchors = p->num_anchors;
  a->step = p->step;
  a->group_blocks = p->group_blocks;
  a->budget_frames = p->budget_frames;
  a->dense = dense_mask;
  a->row_ptr = row_ptr;
  a->col_idx = col_idx;
  a->nnz_out = nnz_out;
  return LVA_OK;
}

lva_status lva_build_block_mask(const lva_mask_params* p, const uint8_t* dense_mask, int32_t* row_ptr,
                                int32_t* col_idx, int64_t col_capacity, int32_t* nnz_out,
                                cudaStream_t stream) {
  MaskArgs a;
  const lva_status s = mask_args(p, dense_mask, row_ptr, col_idx, col_capacity, nnz_out, &a);
  if (s != LVA_OK) return s;
  return from_cuda(launch_build_mask(a, stream), "mask launch");
}

int64_t lva_block_mask_workspace_bytes(const lva_mask_params* p) {
  if (check_mask_params(p) != LVA_OK) return -1;
  const int64_t nb = p->n_pad / p->block_size;
  return mask_workspace_bytes(p->kind, int64_t(p->mask_heads) * nb, nb);
}

lva_status lva_build_block_mask_ws(const lva_mask_params* p, const uint8_t* dense_mask, int32_t* row_ptr,
                                   int32_t* col_idx, int64_t col_capacity, int32_t* nnz_out, void* workspace,
                                   int64_t workspace_bytes, cudaStream_t stream) {
  MaskArgs a;
  const lva_status s = mask_args(p, dense_mask, row_ptr, col_idx, col_capacity, nnz_out, &a);
  if (s != LVA_OK) return s;
  const int64_t need = lva_block_mask_workspace_bytes(p);
  if (need == 0) return from_cuda(launch_build_mask(a, stream), "mask launch");
  if (workspace == nullptr) return fail(LVA_ERR_INVALID_ARG, "mask: null workspace");
  if (!aligned(workspace, 16)) return fail(LVA_ERR_INVALID_ARG, "mask: workspace must be 16-byte aligned");
  if (workspace_bytes < need)
    return fail(LVA_ERR_CAPACITY, "mask: workspace_bytes %lld < %lld", (long long)workspace_bytes, (long long)need);
  return from_cuda(launch_build_mask_packed(a, workspace, stream), "mask launch");
}

lva_status lva_build_block_mask_noalloc(const lva_mask_params* p, const uint8_t* dense_mask, int32_t* row_ptr,
                                        int32_t* col_idx, int64_t col_capacity, int32_t* nnz_out,
                                        cudaStream_t stream) {
  MaskArgs a;
  const lva_status s = mask_args(p, dense_mask, row_ptr, col_idx, col_capacity, nnz_out, &a);
  if (s != LVA_OK) return s;
  const int64_t need = lva_block_mask_workspace_bytes(p);
  if (need > mask_noalloc_scratch_bytes())
    return fail(LVA_ERR_CAPACITY,
                "mask_noalloc: these parameters need %lld bytes of scratch; the library holds %lld "
                "(use lva_build_block_mask_ws with a workspace, or lva_build_block_mask)",
                (long long)need, (long long)mask_noalloc_scratch_bytes());
  return from_cuda(launch_build_mask_noalloc(a, stream), "mask_noalloc launch");
}

static lva_status attn_common(const char* fn, const void* q, const void* k, const void* v, void* o,
                              float* lse, int B, int H, int64_t n_pad, int64_t n_valid, int d,
                              int block_size, const int32_t* row_ptr, const int32_t* col_idx,
                              int64_t col_len, int mask_heads, float scale, const int32_t* query_src,
                              int src_heads, void* o_raster, int T, int Hg, int Wg, int tile_t,
                              int tile_h, int tile_w, int gather_windows, int gather_window,
                              cudaStream_t stream, int lse_only = 0) {
  if (B < 0 || H < 1) return fail(LVA_ERR_INVALID_ARG, "%s: need B >= 0 and H >= 1", fn);
  if (d != 64 && d != 128) return fail(LVA_ERR_UNSUPPORTED, "%s: head dim must be 64 or 128", fn);
  if (block_size != 64 && block_size != 128) return fail(LVA_ERR_UNSUPPORTED, "%s: block_size must be 64 or 128", fn);
  if (n_pad <= 0 || n_pad % block_size != 0) return fail(LVA_ERR_INVALID_ARG, "%s: n_pad must be a positive multiple of block_size", fn);
  if (n_valid < 0 || n_valid > n_pad) return fail(LVA_ERR_INVALID_ARG, "%s: need 0 <= n_valid <= n_pad", fn);
  if (mask_heads != 1 && mask_heads != H) return fail(LVA_ERR_INVALID_ARG, "%s: mask_heads must be 1 or H", fn);
  if (int64_t(B) * H * n_pad >= (int64_t(1) << 31)) return fail(LVA_ERR_UNSUPPORTED, "%s: B*H*n_pad must be < 2^31", fn);
  if (!(scale == scale)) return fail(LVA_ERR_INVALID_ARG, "%s: scale is NaN", fn);
  if (col_len < 0) return fail(LVA_ERR_INVALID_ARG, "%s: col_len < 0", fn);
  if (query_src != nullptr && src_heads != 1 && src_heads != H)
    return fail(LVA_ERR_INVALID_ARG, "%s: src_heads must be 1 or H", fn);
  if (query_src != nullptr && !aligned(query_src, 4))
    return fail(LVA_ERR_INVALID_ARG, "%s: query_src must be 4-byte aligned", fn);
  if (o_raster != nullptr) {
    if (T < 1 || Hg < 1 || Wg < 1 || tile_t < 1 || tile_h < 1 || tile_w < 1)
      return fail(LVA_ERR_INVALID_ARG, "%s: grid and tile extents must be >= 1", fn);
    if (int64_t(T) * Hg * Wg != n_valid)
      return fail(LVA_ERR_INVALID_ARG, "%s: T*H*W must equal n_valid", fn);
  }
  if (B == 0) return ok();
  if (!q || !k || (!lse_only && (!v || !(o || o_raster))) || !lse || !row_ptr || (!col_idx && col_len > 0))
    return fail(LVA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(q, 16) || !aligned(k, 16) || (v && !aligned(v, 16)) || (o && !aligned(o, 16)) ||
      (o_raster && !aligned(o_raster, 16)))
    return fail(LVA_ERR_INVALID_ARG, "%s: q, k, v, o must be 16-byte aligned", fn);
  if (!aligned(lse, 4) || !aligned(row_ptr, 4) || !aligned(col_idx, 4))
    return fail(LVA_ERR_INVALID_ARG, "%s: lse, row_ptr, col_idx must be 4-byte aligned", fn);
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "%s: cannot locate the device error word", fn);
  AttnArgs a{q, k, v, o, lse, B, H, n_pad, n_valid, d, block_size, row_ptr,
             col_idx, col_len, mask_heads, scale, query_src, src_heads, err,
             o_raster, T, Hg, Wg, tile_t, tile_h, tile_w, gather_windows, gather_window, lse_only};
  const char* why = "launch";
  cudaError_t e = launch_attn(a, stream, &why);
  if (e != cudaSuccess) return fail(LVA_ERR_CUDA, "%s: %s: %s", fn, why, cudaGetErrorString(e));
  return ok();
}

lva_status lva_block_sparse_attn(const void* q, const void* k, const void* v, void* o, float* lse,
                                 int B, int H, int64_t n_pad, int64_t n_valid, int d, int block_size,
                                 const int32_t* row_ptr, const int32_t* col_idx, int64_t col_len,
                                 int mask_heads, float scale, const int32_t* query_src, int src_heads,
                                 cudaStream_t stream) {
  if (o == nullptr && B > 0) return fail(LVA_ERR_INVALID_ARG, "attn: null pointer");
  return attn_common("attn", q, k, v, o, lse, B, H, n_pad, n_valid, d, block_size, row_ptr, col_idx,
                     col_len, mask_heads, scale, query_src, src_heads, nullptr, 0, 0, 0, 0, 0, 0, 0, 0,
                     stream);
}

lva_status lva_block_sparse_lse(const void* q, const void* k, float* lse, int B, int H, int64_t n_pad,
                                int64_t n_valid, int d, int block_size, const int32_t* row_ptr,
                                const int32_t* col_idx, int64_t col_len, int mask_heads, float scale,
                                cudaStream_t stream) {
  return attn_common("lse", q, k, nullptr, nullptr, lse, B, H, n_pad, n_valid, d, block_size, row_ptr,
                     col_idx, col_len, mask_heads, scale, nullptr, 1, nullptr, 0, 0, 0, 0, 0, 0, 0, 0,
                     stream, 1);
}

lva_status lva_block_sparse_attn_raster(const void* q, const void* k, const void* v, void* o_raster,
                                        float* lse, int B, int H, int64_t n_pad, int64_t n_valid,
                                        int d, int block_size, const int32_t* row_ptr,
                                        const int32_t* col_idx, int64_t col_len, int mask_heads,
                                        float scale, int T, int Hg, int Wg, int tile_t, int tile_h,
                                        int tile_w, cudaStream_t stream) {
  if (o_raster == nullptr && B > 0) return fail(LVA_ERR_INVALID_ARG, "attn_raster: null pointer");
  return attn_common("attn_raster", q, k, v, nullptr, lse, B, H, n_pad, n_valid, d, block_size,
                     row_ptr, col_idx, col_len, mask_heads, scale, nullptr, 1, o_raster, T, Hg, Wg,
                     tile_t, tile_h, tile_w, 0, 0, stream);
}

lva_status lva_window_transposed_attn(const void* q, const void* k, const void* v, void* o, float* lse,
                                      int B, int H, int64_t n, int d, int window, int block_size,
                                      const int32_t* row_ptr, const int32_t* col_idx, int64_t col_len,
                                      int mask_heads, float scale, cudaStream_t stream) {
  if (window < 1 || n <= 0 || n % window != 0)
    return fail(LVA_ERR_INVALID_ARG, "window_attn: n must be a positive multiple of window");
  const int64_t m = n / window;
  if (block_size != 64 && block_size != 128)
    return fail(LVA_ERR_UNSUPPORTED, "window_attn: block_size must be 64 or 128");
  if (m % block_size != 0)
    return fail(LVA_ERR_INVALID_ARG, "window_attn: the window count n / window must be a multiple of block_size");
  if (int64_t(B) * H * m >= (int64_t(1) << 31))
    return fail(LVA_ERR_UNSUPPORTED, "window_attn: B*H*(n/window) must be < 2^31");
  if (o == nullptr && B > 0) return fail(LVA_ERR_INVALID_ARG, "window_attn: null pointer");
  // O goes to the original order through the raster epilogue: the window transpose is the
  // tile order of the grid (1, m, window) with tiles (1, m, 1).
  return attn_common("window_attn", q, k, v, nullptr, lse, B, H, n, n, d, block_size, row_ptr, col_idx,
                     col_len, mask_heads, scale, nullptr, 1, o, 1, int(m), window, 1, int(m), 1, int(m),
                     window, stream);
}

lva_status lva_broadcast_blocks(void* o, float* lse, int B, int H, int64_t n_pad, int d, int block_size,
                                const int32_t* query_src, int src_heads, cudaStream_t stream) {
  if (B < 0 || H < 1) return fail(LVA_ERR_INVALID_ARG, "broadcast: need B >= 0 and H >= 1");
  if (d != 64 && d != 128) return fail(LVA_ERR_UNSUPPORTED, "broadcast: head dim must be 64 or 128");
  if (block_size != 64 && block_size != 128) return fail(LVA_ERR_UNSUPPORTED, "broadcast: block_size must be 64 or 128");
  if (n_pad <= 0 || n_pad % block_size != 0) return fail(LVA_ERR_INVALID_ARG, "broadcast: n_pad must be a positive multiple of block_size");
  if (src_heads != 1 && src_heads != H) return fail(LVA_ERR_INVALID_ARG, "broadcast: src_heads must be 1 or H");
  if (int64_t(B) * H * n_pad >= (int64_t(1) << 31)) return fail(LVA_ERR_UNSUPPORTED, "broadcast: B*H*n_pad must be < 2^31");
  if (B == 0) return ok();
  if (!o || !lse || !query_src) return fail(LVA_ERR_INVALID_ARG, "broadcast: null pointer");
  if (!aligned(o, 16) || !aligned(lse, 4) || !aligned(query_src, 4))
    return fail(LVA_ERR_INVALID_ARG, "broadcast: o must be 16-byte, lse and query_src 4-byte aligned");
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "broadcast: cannot locate the device error word");
  BroadcastArgs a{o, lse, B, H, n_pad, d, block_size, query_src, src_heads, err};
  return from_cuda(launch_broadcast(a, stream), "broadcast launch");
}

lva_status lva_block_energy(const void* q, const void* k, const float* lse, float* energy, int B,
                            int H, int64_t n_pad, int64_t n_valid, int d, int block_size,
                            const int32_t* row_ptr, const int32_t* col_idx, int64_t col_len,
                            int mask_heads, float scale, cudaStream_t stream) {
  if (B < 0 || H < 1) return fail(LVA_ERR_INVALID_ARG, "energy: need B >= 0 and H >= 1");
  if (d != 64 && d != 128) return fail(LVA_ERR_UNSUPPORTED, "energy: head dim must be 64 or 128");
  if (block_size != 64 && block_size != 128) return fail(LVA_ERR_UNSUPPORTED, "energy: block_size must be 64 or 128");
  if (n_pad <= 0 || n_pad % block_size != 0) return fail(LVA_ERR_INVALID_ARG, "energy: n_pad must be a positive multiple of block_size");
  if (n_valid < 0 || n_valid > n_pad) return fail(LVA_ERR_INVALID_ARG, "energy: need 0 <= n_valid <= n_pad");
  if (mask_heads != 1 && mask_heads != H) return fail(LVA_ERR_INVALID_ARG, "energy: mask_heads must be 1 or H");
  if (int64_t(B) * H * n_pad >= (int64_t(1) << 31)) return fail(LVA_ERR_UNSUPPORTED, "energy: B*H*n_pad must be < 2^31");
  if (!(scale == scale)) return fail(LVA_ERR_INVALID_ARG, "energy: scale is NaN");
  if (col_len < 0) return fail(LVA_ERR_INVALID_ARG, "energy: col_len < 0");
  if (B == 0) return ok();
  if (!q || !k || !lse || !energy || !row_ptr || (!col_idx && col_len > 0))
    return fail(LVA_ERR_INVALID_ARG, "energy: null pointer");
  if (!aligned(q, 16) || !aligned(k, 16))
    return fail(LVA_ERR_INVALID_ARG, "energy: q, k must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(energy, 4) || !aligned(row_ptr, 4) || !aligned(col_idx, 4))
    return fail(LVA_ERR_INVALID_ARG, "energy: lse, energy, row_ptr, col_idx must be 4-byte aligned");
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "energy: cannot locate the device error word");
  EnergyArgs a{q, k, lse, energy, B, H, n_pad, n_valid, d, block_size, row_ptr, col_idx, col_len,
               mask_heads, scale, err};
  const char* why = "launch";
  cudaError_t e = launch_energy(a, stream, &why);
  if (e != cudaSuccess) return fail(LVA_ERR_CUDA, "energy: %s: %s", why, cudaGetErrorString(e));
  return ok();
}

lva_status lva_select_blocks(const float* energy, uint8_t* mask, int64_t rows, int nb, double eps,
                             cudaStream_t stream) {
  if (rows < 0) return fail(LVA_ERR_INVALID_ARG, "select: rows < 0");
  if (nb < 1) return fail(LVA_ERR_INVALID_ARG, "select: nb must be >= 1");
  if (nb > kSelectMaxBlocks) return fail(LVA_ERR_UNSUPPORTED, "select: nb must be <= %d", kSelectMaxBlocks);
  if (!(eps >= 0.0 && eps <= 1.0)) return fail(LVA_ERR_INVALID_ARG, "select: eps must be in [0, 1]");
  if (rows > (int64_t(1) << 40) / nb) return fail(LVA_ERR_UNSUPPORTED, "select: rows * nb too large");
  if (rows == 0) return ok();
  if (!energy || !mask) return fail(LVA_ERR_INVALID_ARG, "select: null pointer");
  if (!aligned(energy, 4)) return fail(LVA_ERR_INVALID_ARG, "select: energy must be 4-byte aligned");
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "select: cannot locate the device error word");
  SelectArgs a{energy, mask, rows, nb, eps, err};
  return from_cuda(launch_select(a, stream), "select launch");
}

lva_status lva_aggregate_masks(const uint8_t* masks, uint8_t* out, int prompts, int64_t count,
                               double rho, cudaStream_t stream) {
  if (prompts < 1) return fail(LVA_ERR_INVALID_ARG, "aggregate: prompts must be >= 1");
  if (count < 0) return fail(LVA_ERR_INVALID_ARG, "aggregate: count < 0");
  if (!(rho >= 0.0 && rho <= 1.0)) return fail(LVA_ERR_INVALID_ARG, "aggregate: rho must be in [0, 1]");
  if (count == 0) return ok();
  if (!masks || !out) return fail(LVA_ERR_INVALID_ARG, "aggregate: null pointer");
  AggregateArgs a{masks, out, prompts, count, rho * double(prompts)};
  return from_cuda(launch_aggregate(a, stream), "aggregate launch");
}

// A bf16 [tokens, heads, d] view: strides in elements, rows on 16-byte boundaries.  The TMA
// takes strides below 2^40 bytes.
static bool view_ok(int64_t token_stride, int64_t head_stride, int heads, int d) {
  const int64_t most = int64_t(1) << 38;
  if (token_stride < d || token_stride % 8 != 0 || token_stride > most) return false;
  return heads == 1 || (head_stride >= d && head_stride % 8 == 0 && head_stride <= most);
}

// Checks of head counts, head dim and scale that the context calls share.
static lva_status check_heads(const char* fn, int q_heads, int kv_heads, int d, float scale) {
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0)
    return fail(LVA_ERR_INVALID_ARG, "%s: kv_heads must divide q_heads, both >= 1", fn);
  if (d != 64 && d != 128) return fail(LVA_ERR_UNSUPPORTED, "%s: head dim must be 64 or 128", fn);
  if (!(scale > 0.f) || !std::isfinite(scale) || !std::isfinite(scale * 1.4426950408889634f))
    return fail(LVA_ERR_INVALID_ARG, "%s: scale must be positive and finite", fn);
  return LVA_OK;
}

// Parts of packed tiles, when there are tiles for less than half the SMs (an upper bound from the
// totals; the lengths are on the device) and at least 20 key blocks.  The kernel cuts the tiles
// into at most 148 parts, one per SM: 64 tokens of 40 heads against 8,000 keys, 24 tiles, take
// 31 us so, 37 in up to twice as many parts, 60 whole; 512 tokens of 8 heads against 16,384
// keys 47, 52 and 112.  With tiles for most SMs the parts' start, end and join cost what they
// gain: 128 tiles of 32 blocks took 45 us whole and 48 to 61 cut, 264 of 125 blocks 301 and
// 307 to 337.
struct PackedPlan {
  int spare, max_items;              // 0: no parts
  int64_t part_o, part_lse, bytes;   // byte offsets in the workspace
};

static PackedPlan packed_plan(const lva_packed_params* p) {
  PackedPlan w{0, 0, 0, 0, 0};
  const int tok = 128 / (p->q_heads / p->kv_heads);
  const int64_t tiles = (p->total_q / tok + p->num_seqs) * p->kv_heads;
  const int64_t blocks = (p->total_k + 127) / 128;
  if (p->num_seqs == 0 || p->total_q == 0 || tiles >= 74 || blocks < 20) return w;
  w.max_items = 148;
  w.spare = w.max_items - int(tiles);
  w.part_lse = int64_t(w.max_items) * 128 * p->d * 4;
  w.bytes = w.part_lse + int64_t(w.max_items) * 128 * 4;
  return w;
}

static lva_status check_packed(const lva_packed_params* p) {
  if (p == nullptr) return fail(LVA_ERR_INVALID_ARG, "packed: null params");
  const lva_status s = check_heads("packed", p->q_heads, p->kv_heads, p->d, p->scale);
  if (s != LVA_OK) return s;
  const int group = p->q_heads / p->kv_heads;
  if (group > 128) return fail(LVA_ERR_UNSUPPORTED, "packed: at most 128 query heads per key/value head");
  if (p->num_seqs < 0 || p->total_q < 0 || p->total_k < 0)
    return fail(LVA_ERR_INVALID_ARG, "packed: num_seqs and totals must be >= 0");
  if (p->total_q >= (int64_t(1) << 31) || p->total_k >= (int64_t(1) << 31))
    return fail(LVA_ERR_UNSUPPORTED, "packed: totals must be < 2^31 tokens");
  if ((p->total_q / (128 / group) + p->num_seqs) * p->kv_heads > int64_t(0x7fffffff))
    return fail(LVA_ERR_UNSUPPORTED, "packed: too many tiles for one launch");
  return LVA_OK;
}

int64_t lva_packed_workspace_bytes(const lva_packed_params* p) {
  return check_packed(p) == LVA_OK ? packed_plan(p).bytes : -1;
}

lva_status lva_packed_attn(const lva_packed_params* p, const void* q, const void* k, const void* v, void* o,
                           float* lse, const int32_t* cu_q, const int32_t* cu_k, void* workspace,
                           int64_t workspace_bytes, cudaStream_t stream) {
  const lva_status s = check_packed(p);
  if (s != LVA_OK) return s;
  if (!view_ok(p->q_token_stride, p->q_head_stride, p->q_heads, p->d) ||
      !view_ok(p->k_token_stride, p->k_head_stride, p->kv_heads, p->d) ||
      !view_ok(p->v_token_stride, p->v_head_stride, p->kv_heads, p->d) ||
      !view_ok(p->o_token_stride, p->o_head_stride, p->q_heads, p->d))
    return fail(LVA_ERR_INVALID_ARG, "packed: strides must be multiples of 8 elements, at least d");
  if (p->num_seqs == 0 || p->total_q == 0) return ok();
  if (!q || !o || !lse || !cu_q || !cu_k || (p->total_k > 0 && (!k || !v)))
    return fail(LVA_ERR_INVALID_ARG, "packed: null pointer");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(workspace, 16))
    return fail(LVA_ERR_INVALID_ARG, "packed: q, k, v, o and workspace must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(cu_k, 4))
    return fail(LVA_ERR_INVALID_ARG, "packed: lse, cu_q, cu_k must be 4-byte aligned");
  PackedPlan w{0, 0, 0, 0, 0};
  if (workspace != nullptr) {
    w = packed_plan(p);
    if (workspace_bytes < w.bytes)
      return fail(LVA_ERR_CAPACITY, "packed: workspace_bytes %lld < %lld", (long long)workspace_bytes, (long long)w.bytes);
  }
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "packed: cannot locate the device error word");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PackedArgs a{q, k, v, o, lse, p->num_seqs, p->q_heads, p->kv_heads, p->d, p->total_q, p->total_k,
               p->q_token_stride, p->q_head_stride, p->k_token_stride, p->k_head_stride,
               p->v_token_stride, p->v_head_stride, p->o_token_stride, p->o_head_stride,
               cu_q, cu_k, p->causal != 0, p->scale, 0, w.spare, w.max_items,
               w.spare > 0 ? reinterpret_cast<float*>(ws + w.part_o) : nullptr,
               w.spare > 0 ? reinterpret_cast<float*>(ws + w.part_lse) : nullptr, 0, err};
  const char* why = "launch";
  const cudaError_t e = launch_packed(a, stream, &why);
  if (e != cudaSuccess) return fail(LVA_ERR_CUDA, "packed: %s: %s", why, cudaGetErrorString(e));
  return ok();
}

// Parts of the prefix and workers of the cache pass, from estimates in block times (128 rows by
// 128 keys, 0.9 us).  `join` is what a part's rows cost the join, written and read (about
// 7.2 MB a block time).  The caches, taken as half full (the lengths are on the device), cost
// their bytes at 5.9 MB a block time, or a worker its share of the tiles, 0.5 (8 rows) to 1.9
// (64 rows) each and 0.6 of that with d = 64, and of the planes' starts and ends, 1.5 to 2.5 (4
// rows) to 5.5 (16 rows) each, as fitted to 52 to 148 workers alone.
//   In turn: 148 workers, then the parts.  With c = items * parts CTAs the parts take about
//   blocks / parts when c <= 148, or items * blocks / 148 and half a part of tail when there
//   are more, and in either case 3 for a part's start and end; 13 for the launches and the
//   join, up to 8 more when the caches keep the SMs from the parts.
//   (148, and 74 tiles for packed parts above, are a B200's SMs and half of them: what the
//   estimates were fitted to.  Any count is right.)
//   In one list: where all tokens of the batch are at most 32 rows, the prefix can be one more
//   sequence of the cache pass, at the tiles' cost for that many rows, 0.12 for each piece that
//   the join finds of a row, and 12 for two launches instead of three.  It is taken where it is
//   clearly shorter: at 15 and 1.8 times its work.
//   Beside one another: a part's CTA and a worker have an SM each, parts and workers 148 together
//   and at least 52 workers.
// In loops over one state: 8,192 prefix keys and 32 caches of up to 1,024 (8 heads of 128, 32 query
// heads): 35.8 us in turn, 29 to 31 beside with 4 to 6 parts (32 to 33 among other calls); 30,000 keys, 40 query heads: 55.9 and 53; 65,531 keys
// and 96 caches of up to 4,096: 311 and 290; 462 keys, 83 tiny caches of 12 heads: 42 and 66.
// 1,050 prefix keys, one cache, 4 rows: 16.3 us beside, 14.1 in one list; 9 keys, two caches, 2
// rows: 16.4 and 14.0; with 44 to 64 rows 16 to 18 and 17 to 31.
static double tile_cost(int rows, int d) {
  const int padded = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  return (0.35 + 0.024 * padded) * (d == 64 ? 0.6 : 1.0);
}

// A plane's tiles, its start and its end; the start hides behind the tiles when there are several.
static double plane_work(double tiles, double tile, double rows) {
  const double many = tiles * tile + 0.5, few = tile + 1.5;
  return (many > few ? many : few) + 0.25 * rows;
}

static void prefix_split(const lva_shared_prefix_params* p, int* parts, int* workers, int* with_prefix) {
  *workers = kCacheWorkers;
  *parts = 0;
  *with_prefix = 0;
  if (p->prefix_len == 0) return;
  const int group = p->q_heads / p->kv_heads, tok = 128 / group, rows = group * p->steps;
  const double items = double((int64_t(p->B) * p->steps + tok - 1) / tok * p->kv_heads);
  const int64_t blocks = (p->prefix_len + 127) / 128;
  const double join = double(p->B) * p->steps * p->q_heads * (p->d * 8 + 8) / 7.2e6;
  const double planes = p->capacity > 0 ? double(p->B) * p->kv_heads : 0;
  const double bytes = planes * p->capacity * p->d * 2 / 5.9e6;
  const double work = planes * plane_work(double(p->capacity / 128 + 1), tile_cost(rows, p->d), rows);
  auto caches = [&](double n) { return bytes > work / n ? bytes : work / n; };
  const double all = caches(kCacheWorkers), kept = 2 * all < 8 ? 2 * all : 8;
  double best = 0;
  for (int s = 1; s <= 32 && s <= blocks; ++s) {
    const double part = double((blocks + s - 1) / s), load = items * s / 148;
    const double turn = all + (load <= 1 ? part : items * blocks / 148 + part / 2) + 3 * (load > 1 ? load : 1) + join * s + 13 + kept;
    if (s == 1 || turn < best) { best = turn; *parts = s; *workers = kCacheWorkers; }
    const double left = kCacheWorkers - items * s;
    if (p->capacity == 0 || left < 52) continue;
    const double own = caches(left), beside = (part > own ? part : own) + join * s + 18;
    if (beside < best) { best = beside; *parts = s; *workers = int(left); }
  }
  const double all_rows = double(p->B) * rows;
  const double tiles = double(p->prefix_len / 64 + 1), list = planes * (p->capacity / 64 + 6) + p->kv_heads * (tiles + 5);
  if (p->capacity == 0 || all_rows > kListMaxRows || list >= double(int64_t(1) << 31)) return;
  const double wide = tile_cost(int(all_rows), p->d), places = planes * double(p->capacity / 128 + 6) + p->kv_heads * (tiles + 5);
  const double pieces = places > kCacheWorkers ? (tiles + 5) * kCacheWorkers / places : tiles;
  const double one = (planes * plane_work(double(p->capacity / 128 + 1), wide, rows) +
                      p->kv_heads * plane_work(tiles, wide, all_rows)) / kCacheWorkers + 0.12 * pieces;
  if (15 + 1.8 * one < best) { *parts = 0; *workers = kCacheWorkers; *with_prefix = 1; }
}

// Byte offsets of the workspace's pieces (256-byte steps).
struct PrefixWorkspace {
  int parts, workers, with_prefix;
  int64_t part_o, part_lse, own_o, own_lse, scores, score_stride, bytes;
};

static lva_status prefix_plan(const lva_shared_prefix_params* p, bool with_weight, PrefixWorkspace* w) {
  if (p == nullptr) return fail(LVA_ERR_INVALID_ARG, "shared_prefix: null params");
  const lva_status s = check_heads("shared_prefix", p->q_heads, p->kv_heads, p->d, p->scale);
  if (s != LVA_OK) return s;
  if (p->B < 0 || p->steps < 1) return fail(LVA_ERR_INVALID_ARG, "shared_prefix: need B >= 0 and steps >= 1");
  if (p->prefix_len < 0 || p->capacity < 0)
    return fail(LVA_ERR_INVALID_ARG, "shared_prefix: prefix_len and capacity must be >= 0");
  const int64_t group = p->q_heads / p->kv_heads, rows = p->steps * group;
  if (rows > kCacheMaxRows)
    return fail(LVA_ERR_UNSUPPORTED, "shared_prefix: steps * q_heads / kv_heads must be <= %d", kCacheMaxRows);
  const int64_t most = int64_t(1) << 31;
  if (p->prefix_len >= most || p->capacity >= most)
    return fail(LVA_ERR_UNSUPPORTED, "shared_prefix: prefix_len and capacity must be < 2^31");
  const int64_t planes = int64_t(p->B) * p->kv_heads;
  const int64_t chunks = with_weight ? p->capacity / 512 + 1 : 0;
  if (planes >= most || planes * rows >= most || (p->capacity > 0 && planes >= most / p->capacity) ||
      planes * rows / 4 + 1 + planes * chunks >= most || planes * (p->capacity / 64 + 6) >= most)
    return fail(LVA_ERR_UNSUPPORTED, "shared_prefix: B * kv_heads * capacity and B * steps * q_heads must be < 2^31");
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  prefix_split(p, &w->parts, &w->workers, &w->with_prefix);
  const int64_t part_rows = w->with_prefix ? (p->kv_heads + int64_t(kCacheWorkers)) * p->B * rows : int64_t(w->parts) * planes * rows;
  const int64_t own_rows = p->capacity > 0 ? (planes + kCacheWorkers) * rows : 0;
  w->score_stride = (p->capacity + 63) / 64 * 64;
  w->part_o = 0;
  w->part_lse = w->part_o + up(part_rows * p->d * 4);
  w->own_o = w->part_lse + up(part_rows * 4);
  w->own_lse = w->own_o + up(own_rows * p->d * 4);
  w->scores = w->own_lse + up(own_rows * 4);
  w->bytes = w->scores + (with_weight ? up(planes * rows * w->score_stride * 4) : 0);
  return LVA_OK;
}

int64_t lva_shared_prefix_workspace_bytes(const lva_shared_prefix_params* p, int with_weight) {
  PrefixWorkspace w;
  return prefix_plan(p, with_weight != 0, &w) == LVA_OK ? w.bytes : -1;
}

lva_status lva_shared_prefix_plan(const lva_shared_prefix_params* p, int* parts, int* workers, int* in_list) {
  PrefixWorkspace w;
  const lva_status s = prefix_plan(p, false, &w);
  if (s != LVA_OK) return s;
  if (!parts || !workers || !in_list) return fail(LVA_ERR_INVALID_ARG, "shared_prefix_plan: null pointer");
  *parts = w.parts;
  *workers = w.workers;
  *in_list = w.with_prefix;
  return ok();
}

lva_status lva_shared_prefix_attn(const lva_shared_prefix_params* p, const void* q, const void* prefix_k,
                                  const void* prefix_v, const void* k_cache, const void* v_cache,
                                  const int32_t* lens, void* o, float* lse, float* weight, void* workspace,
                                  int64_t workspace_bytes, cudaStream_t stream) {
  PrefixWorkspace w;
  const lva_status s = prefix_plan(p, weight != nullptr, &w);
  if (s != LVA_OK) return s;
  if (!view_ok(p->q_token_stride, p->q_head_stride, p->q_heads, p->d) ||
      !view_ok(p->o_token_stride, p->o_head_stride, p->q_heads, p->d) ||
      (p->prefix_len > 0 && (!view_ok(p->k_token_stride, p->k_head_stride, p->kv_heads, p->d) ||
                             !view_ok(p->v_token_stride, p->v_head_stride, p->kv_heads, p->d))))
    return fail(LVA_ERR_INVALID_ARG, "shared_prefix: strides must be multiples of 8 elements, at least d");
  if (p->B == 0) return ok();
  if (!q || !o || !lse || (p->prefix_len > 0 && (!prefix_k || !prefix_v)) ||
      (p->capacity > 0 && (!k_cache || !v_cache || !lens)) || (w.bytes > 0 && !workspace))
    return fail(LVA_ERR_INVALID_ARG, "shared_prefix: null pointer");
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(prefix_k, 16) || !aligned(prefix_v, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(workspace, 16))
    return fail(LVA_ERR_INVALID_ARG, "shared_prefix: q, k, v, o, caches and workspace must be 16-byte aligned");
  if (!aligned(lens, 4) || !aligned(lse, 4) || !aligned(weight, 4))
    return fail(LVA_ERR_INVALID_ARG, "shared_prefix: lens, lse, weight must be 4-byte aligned");
  if (workspace_bytes < w.bytes)
    return fail(LVA_ERR_CAPACITY, "shared_prefix: workspace_bytes %lld < %lld", (long long)workspace_bytes,
                (long long)w.bytes);
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "shared_prefix: cannot locate the device error word");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* part_o = reinterpret_cast<float*>(ws + w.part_o);
  float* part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  const char* why = "launch";
  CacheAttnArgs c{q, prefix_k, prefix_v, k_cache, v_cache, lens, o, lse, p->capacity > 0 ? weight : nullptr, p->B, p->steps, p->q_heads,
                  p->kv_heads, p->d, p->prefix_len, p->capacity, p->q_token_stride, p->q_head_stride,
                  p->k_token_stride, p->k_head_stride, p->v_token_stride, p->v_head_stride,
                  p->o_token_stride, p->o_head_stride, p->scale, w.parts, w.with_prefix, part_o, part_lse,
                  reinterpret_cast<float*>(ws + w.own_o), reinterpret_cast<float*>(ws + w.own_lse),
                  weight != nullptr ? reinterpret_cast<float*>(ws + w.scores) : nullptr, w.score_stride,
                  w.workers, err};
  if (p->capacity > 0) {
    const cudaError_t e = launch_cache_attn(c, stream, &why);
    if (e != cudaSuccess) return fail(LVA_ERR_CUDA, "shared_prefix: %s: %s", why, cudaGetErrorString(e));
  }
  if (w.parts > 0) {
    PackedArgs a{q, prefix_k, prefix_v, nullptr, nullptr, 1, p->q_heads, p->kv_heads, p->d,
                 int64_t(p->B) * p->steps, p->prefix_len,
                 p->q_token_stride, p->q_head_stride, p->k_token_stride, p->k_head_stride,
                 p->v_token_stride, p->v_head_stride, 0, 0, nullptr, nullptr, 0, p->scale,
                 w.parts, 0, 0, part_o, part_lse, p->capacity > 0 ? 1 : 0, err};
    const cudaError_t e = launch_packed(a, stream, &why);
    if (e != cudaSuccess) return fail(LVA_ERR_CUDA, "shared_prefix: %s: %s", why, cudaGetErrorString(e));
  }
  return from_cuda(launch_cache_join(c, stream), "shared_prefix join launch");
}

// Sizes of [B, kv_heads, capacity, d] caches.
static lva_status check_cache(const char* fn, int B, int kv_heads, int64_t capacity, int d) {
  if (B < 0 || kv_heads < 1 || capacity < 0)
    return fail(LVA_ERR_INVALID_ARG, "%s: need B >= 0, kv_heads >= 1, capacity >= 0", fn);
  if (d != 64 && d != 128) return fail(LVA_ERR_UNSUPPORTED, "%s: head dim must be 64 or 128", fn);
  const int64_t most = int64_t(1) << 31;
  const int64_t planes = int64_t(B) * kv_heads;
  if (planes >= most || capacity >= most || (planes > 0 && capacity >= (int64_t(1) << 40) / planes))
    return fail(LVA_ERR_UNSUPPORTED, "%s: B * kv_heads and capacity must be < 2^31, their product < 2^40", fn);
  return LVA_OK;
}

// Whether [a, a + n) and [b, b + n) share a byte.
static bool overlap(const void* a, const void* b, int64_t n) {
  const intptr_t x = reinterpret_cast<intptr_t>(a), y = reinterpret_cast<intptr_t>(b);
  return x < y + n && y < x + n;
}

lva_status lva_append_cache(const void* k_new, const void* v_new, int64_t k_token_stride, int64_t k_head_stride,
                            int64_t v_token_stride, int64_t v_head_stride, void* k_cache, void* v_cache,
                            float* weight, const int32_t* lens, int32_t* lens_out, int B, int steps, int kv_heads,
                            int64_t capacity, int d, cudaStream_t stream) {
  const lva_status s = check_cache("append", B, kv_heads, capacity, d);
  if (s != LVA_OK) return s;
  if (steps < 0) return fail(LVA_ERR_INVALID_ARG, "append: steps must be >= 0");
  if (!view_ok(k_token_stride, k_head_stride, kv_heads, d) || !view_ok(v_token_stride, v_head_stride, kv_heads, d))
    return fail(LVA_ERR_INVALID_ARG, "append: strides must be multiples of 8 elements, at least d");
  const int64_t most = int64_t(1) << 31;
  const int64_t units = int64_t(kv_heads) * steps;               // rows of one sequence, K or V
  if (units >= most / 32 || units * 32 / kAppendUnits + 1 >= most / (B > 0 ? B : 1))
    return fail(LVA_ERR_UNSUPPORTED, "append: too many rows for one launch");
  if (B == 0) return ok();
  if (!lens || !lens_out || (steps > 0 && (!k_new || !v_new || (capacity > 0 && (!k_cache || !v_cache)))))
    return fail(LVA_ERR_INVALID_ARG, "append: null pointer");
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return fail(LVA_ERR_INVALID_ARG, "append: rows and caches must be 16-byte aligned");
  if (!aligned(weight, 4) || !aligned(lens, 4) || !aligned(lens_out, 4))
    return fail(LVA_ERR_INVALID_ARG, "append: weight and lens must be 4-byte aligned");
  if (lens_out != lens && overlap(lens, lens_out, int64_t(B) * 4))
    return fail(LVA_ERR_INVALID_ARG, "append: lens_out must be lens or apart from it");
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "append: cannot locate the device error word");
  AppendArgs a{k_new, v_new, k_cache, v_cache, weight, lens, lens_out, B, steps, kv_heads, d, capacity,
               k_token_stride, k_head_stride, v_token_stride, v_head_stride, err};
  return from_cuda(launch_append(a, stream), "append launch");
}

lva_status lva_evict_cache(const void* k_cache, const void* v_cache, const float* weight, const int32_t* lens,
                           void* k_out, void* v_out, float* weight_out, int32_t* lens_out, int32_t* kept, int B,
                           int kv_heads, int64_t capacity, int d, int64_t budget, int64_t sinks, int64_t recent,
                           cudaStream_t stream) {
  const lva_status s = check_cache("evict", B, kv_heads, capacity, d);
  if (s != LVA_OK) return s;
  if (budget < 1 || budget > capacity) return fail(LVA_ERR_INVALID_ARG, "evict: need 1 <= budget <= capacity");
  if (sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
    return fail(LVA_ERR_INVALID_ARG, "evict: need sinks, recent >= 0 and sinks + recent <= budget");
  const int64_t planes = int64_t(B) * kv_heads;
  if (planes * 33 >= (int64_t(1) << 31) || (budget + 63) / 64 >= (int64_t(1) << 31) / (planes > 0 ? planes : 1))
    return fail(LVA_ERR_UNSUPPORTED, "evict: too many rows for one launch");
  if (B == 0) return ok();
  if (!k_cache || !v_cache || !weight || !lens || !k_out || !v_out || !weight_out || !lens_out || !kept)
    return fail(LVA_ERR_INVALID_ARG, "evict: null pointer");
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(LVA_ERR_INVALID_ARG, "evict: caches must be 16-byte aligned");
  if (!aligned(weight, 4) || !aligned(weight_out, 4) || !aligned(lens, 4) || !aligned(lens_out, 4) || !aligned(kept, 4))
    return fail(LVA_ERR_INVALID_ARG, "evict: weight, lens and kept must be 4-byte aligned");
  if (lens_out != lens && overlap(lens, lens_out, int64_t(B) * 4))
    return fail(LVA_ERR_INVALID_ARG, "evict: lens_out must be lens or apart from it");
  const int64_t bytes = planes * capacity * d * 2;
  const bool in_k = k_out == k_cache, in_v = v_out == v_cache, in_w = weight_out == weight;
  if (in_k != in_v || in_k != in_w)
    return fail(LVA_ERR_INVALID_ARG, "evict: k, v and weight must be in place together or not at all");
  if (!in_k) {
    const void* in[2] = {k_cache, v_cache};
    for (const void* x : in)
      if (overlap(x, k_out, bytes) || overlap(x, v_out, bytes))
        return fail(LVA_ERR_INVALID_ARG, "evict: outputs must not overlap the caches");
    if (overlap(weight, weight_out, planes * capacity * 4))
      return fail(LVA_ERR_INVALID_ARG, "evict: weight_out must not overlap weight");
  }
  if (overlap(k_out, v_out, bytes)) return fail(LVA_ERR_INVALID_ARG, "evict: k and v must not overlap");
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "evict: cannot locate the device error word");
  EvictArgs a{k_cache, v_cache, weight, lens, k_out, v_out, weight_out, lens_out, kept, B, kv_heads, d,
              capacity, budget, sinks, recent, err};
  return from_cuda(launch_evict(a, stream), "evict launch");
}

lva_status lva_selftest_wait(int mode, cudaStream_t stream) {
  if (mode < 0 || mode > 2) return fail(LVA_ERR_INVALID_ARG, "selftest_wait: mode must be 0, 1 or 2");
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "selftest_wait: cannot locate the device error word");
  return from_cuda(launch_wait_selftest(mode, err, stream), "selftest_wait launch");
}

lva_status lva_device_error(cudaStream_t stream, lva_status* status, int* detail) {
  if (status == nullptr) return fail(LVA_ERR_INVALID_ARG, "device_error: null status");
  int* err = device_error_word();
  if (err == nullptr) return fail(LVA_ERR_CUDA, "device_error: cannot locate the device error word");
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return from_cuda(e, "device_error: stream sync");
  unsigned long long word = 0;
  {
    std::lock_guard<std::mutex> lock(g_take_mutex);
    take_error_kernel<<<1, 1, 0, stream>>>(reinterpret_cast<unsigned long long*>(err));
    e = cudaGetLastError();
    if (e != cudaSuccess) return from_cuda(e, "device_error: exchange launch");
    e = cudaMemcpyFromSymbolAsync(&word, g_device_error_taken, sizeof(word), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return from_cuda(e, "device_error: read");
  }
  *status = static_cast<lva_status>(static_cast<int>(word & 0xffffffffull));
  if (detail) *detail = static_cast<int>(word >> 32);
  return ok();
}

}  // extern "C"
