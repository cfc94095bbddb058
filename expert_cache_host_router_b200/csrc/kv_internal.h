// kv_internal.h -- what the attention operators share: the 4-bit cache tile, the checks of
// the arguments that describe a cache, and small device helpers.
//
// Cache tile: 16 tokens of one KV head, 18 D bytes in a row (D channels, NB = D / 32 Q4_0
// blocks a token), so that a tile is one bulk copy.  A tile holds the canonical Q4_0 bytes
// (byte j of a block: channel j in the low half, j + 16 in the high one) regrouped so that
// every lane of a warp finds its fragment of an m16n8k16 matrix product in consecutive
// bytes:
//   [0, 8D)     key nibbles    [16 tokens][4 words t][NB blocks][bytes 4t..4t+3 of the block]
//   [8D, 16D)   value nibbles  [8 token pairs][8 words g][NB][2 tokens][bytes 2g, 2g+1]
//   [16D, 17D)  key scales     [16 tokens][NB] fp16
//   [17D, 18D)  value scales   [8 token pairs][NB][2 tokens] fp16
// No byte is shared by two tokens, so that tokens are written one by one without reading.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe_cache.h"

namespace moe {

constexpr int kTileTok = 16;

struct KvView {  // a cache pool and its page table, as the kernels take them
  uint8_t* pool;
  int n_pages, heads, dim, tiles_per_page;
  const int32_t* table;
  int n_seqs, width;
  int64_t table_stride;
  int32_t* error;  // or null
};

// Whether a runtime call went well.  One that did not is not left behind as the thread's last
// error, where the next call's launches would find it.
inline bool kv_ok(cudaError_t e) {
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess;
}
inline int kv_status(cudaError_t e) { return kv_ok(e) ? MOE_OK : MOE_ERR_CUDA; }

// Launches a kernel and says how that launch went (the last error may be another call's).
// dependent: the kernel may start up while the one before it in the stream runs.
template <typename... P, typename... A>
inline cudaError_t kv_launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool dependent, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Current device for the length of a call.
struct DeviceScope {
  int was = -1;
  bool ok = false;
  explicit DeviceScope(int dev) {
    ok = kv_ok(cudaGetDevice(&was)) && (was == dev || kv_ok(cudaSetDevice(dev)));
    now = dev;
  }
  ~DeviceScope() {
    if (ok && was != now) cudaSetDevice(was);
  }
  int now = -1;
};

int kv_stall();  // 1 if this call is to run into its waits' limits (moe_debug_stall_attention)

constexpr int kKvMaxDevices = 64;
constexpr int kKvMaxSeqs = 8192;
constexpr int kKvMaxPos = INT32_MAX - 4095;  // positions, lengths and rows: roundings up to whole tiles stay in 32 bits

inline bool kv_dim_ok(int d) { return d == 64 || d == 128; }
inline int kv_align_ok(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Whether n0 x n1 rows with these strides can be written: no two of them on the same place for
// want of a stride.
inline bool kv_apart(int64_t s0, int64_t n0, int64_t s1, int64_t n1) { return (n0 < 2 || s0) && (n1 < 2 || s1); }

// SMs of a device, 0 if it cannot be asked.  (Calls may come from several threads at once.)
inline int kv_sm_count(int dev) {
  static std::atomic<int> known[kKvMaxDevices];
  int n = known[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (!kv_ok(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev))) return 0;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// MOE_OK, or why the description of a pool and its page table cannot be used.
inline int kv_check(const moe_kv_pool* c, const moe_kv_table* t, KvView* out) {
  if (!c || !t || !c->pool_dev || !t->table_dev) return MOE_ERR_INVALID;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->head_dim < 1 || c->page_tokens < 1) return MOE_ERR_INVALID;
  if (c->device < 0 || c->device >= kKvMaxDevices || !kv_align_ok(c->pool_dev, 16)) return MOE_ERR_INVALID;
  if (t->n_seqs < 0 || t->width < 1 || (t->row_stride < t->width && t->row_stride != 0)) return MOE_ERR_INVALID;
  if (!kv_dim_ok(c->head_dim) || c->page_tokens % kTileTok || c->n_kv_heads > 1024) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)t->width * c->page_tokens > kKvMaxPos || t->n_seqs > kKvMaxSeqs) return MOE_ERR_UNSUPPORTED;
  // tiles are numbered in 32 bits: 2^31 of them are 2.4 TB and more
  if ((int64_t)c->n_pages * (c->page_tokens / kTileTok) > INT32_MAX / c->n_kv_heads) return MOE_ERR_UNSUPPORTED;
  *out = {c->pool_dev, c->n_pages, c->n_kv_heads, c->head_dim, c->page_tokens / kTileTok,
          t->table_dev, t->n_seqs, t->width, t->row_stride, c->error_dev};
  return MOE_OK;
}

__device__ __forceinline__ void kv_flag(int32_t* error, int code) {
  if (error) atomicCAS(error, 0, code);
}

// Number in the pool of tile `tile` of sequence b and head h; -1 (with the error word set)
// when the table or the page number does not reach it.
__device__ __forceinline__ int kv_tile_number(const KvView& c, int b, int h, int tile) {
  const int pg = tile / c.tiles_per_page;
  int page = -1;
  if (tile >= 0 && pg < c.width) page = c.table[(int64_t)b * c.table_stride + pg];
  if ((unsigned)page >= (unsigned)c.n_pages) {
    kv_flag(c.error, MOE_DEVERR_PAGE);
    return -1;
  }
  return (page * c.heads + h) * c.tiles_per_page + (tile - pg * c.tiles_per_page);
}
__device__ __forceinline__ uint8_t* kv_tile(const KvView& c, int b, int h, int tile) {
  const int n = kv_tile_number(c, b, h, tile);
  return n < 0 ? nullptr : c.pool + (int64_t)n * (18 * c.dim);
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

__device__ __forceinline__ uint32_t kv_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

}  // namespace moe
