// kv_cache.cu -- the 4-bit key/value cache of libmoe: writing rows into it, reading them
// back, and cutting sequences down to a budget by their accumulated attention weight.
#include "kv_internal.h"

namespace moe {

// Sequence that token i of a packed batch belongs to: the last b with cu[b] <= i (any
// contents of cu end the search with 0 <= b < n).
__device__ __forceinline__ int kv_find_seq(const int32_t* cu, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

struct RowArgs {  // rows of keys and values in the caller's memory, strides in elements
  void *k, *v;
  int64_t k_tok, k_head, v_tok, v_head;
  const int32_t *cu, *start;
  int n_tokens;
};

// Position of the thread's 8 channels: lanes of one token and head take its D key
// channels, then its D value channels, four lanes to a Q4_0 block.
template <int D>
struct Piece {
  static constexpr int kLanes = D / 4;  // lanes of one token and head
  int tok, head, block, j;
  bool value, live;
  uint8_t* tile;
  int row;
  __device__ Piece(const KvView& c, const RowArgs& a) {
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t unit = t / kLanes;
    const int in = (int)(t % kLanes);
    live = unit < (int64_t)a.n_tokens * c.heads;
    tok = live ? (int)(unit / c.heads) : 0;
    head = (int)(unit % c.heads);
    value = in >= kLanes / 2;
    block = (in % (kLanes / 2)) >> 2;
    j = in & 3;
    tile = nullptr;
    row = 0;
    if (live) live = tok >= a.cu[0] && tok < a.cu[c.n_seqs];  // padding on either side is not a token
    if (live) {
      const int b = kv_find_seq(a.cu, c.n_seqs, tok);
      const int64_t pos = (int64_t)(a.start ? a.start[b] : 0) + tok - a.cu[b];
      const int64_t end = (int64_t)c.width * c.tiles_per_page * kTileTok;
      if (pos < 0 || pos >= end) {
        kv_flag(c.error, MOE_DEVERR_PAGE);
      } else {
        tile = kv_tile(c, b, head, (int)(pos / kTileTok));
        row = (int)(pos % kTileTok);
      }
    }
  }
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (VEC) {
    if constexpr (sizeof(T) == 2) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = to_float(e[i]);
    } else {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float(p[i]);
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (VEC) {
    if constexpr (sizeof(T) == 2) {
      uint4 w;
      T* e = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = from_float<T>(x[i]);
      *reinterpret_cast<uint4*>(p) = w;
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = from_float<T>(x[i]);
  }
}

// Quantise and scatter.  Four lanes share a block of 32 channels: its first value of the
// largest magnitude and a NaN flag go round by two shuffles.  q is found by a division
// and not by a product with 1 / d: for 16-bit inputs x / d is then never so near to a
// border m + 1/2 that its fp32 rounding could cross it (the distance of two such quotients
// is at least 2^-17, the error of quotient and sum below 2^-20), so the stored bytes are
// the definition's.
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(256) kv_store_kernel(const KvView c, const RowArgs a) {
  constexpr int NB = D / 32;
  const Piece<D> p(c, a);
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (p.live && p.tile) {
    const T* src = p.value ? static_cast<const T*>(a.v) + p.tok * a.v_tok + p.head * a.v_head
                           : static_cast<const T*>(a.k) + p.tok * a.k_tok + p.head * a.k_head;
    load8<T, VEC>(src + p.block * 32 + p.j * 8, x);
  }
  float m = x[0];
  int nan = x[0] != x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    if (fabsf(x[i]) > fabsf(m)) m = x[i];
    nan |= x[i] != x[i];
  }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, m, off);
    nan |= __shfl_xor_sync(0xffffffffu, nan, off);
    const bool lower = (p.j & off) != 0;  // the other lane's channels come first
    if (fabsf(o) > fabsf(m) || (lower && fabsf(o) == fabsf(m))) m = o;
  }
  float d = fminf(fmaxf(m * -0.125f, -8188.0f), 8188.0f);
  if (nan) d = __int_as_float(0x7fc00000);
  uint32_t lo = 0, hi = 0;  // the 8 codes, a byte each
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = floorf(__fadd_rn(d == 0.0f ? 0.0f : __fdiv_rn(x[i], d), 8.5f));
    const uint32_t q = (uint32_t)fminf(fmaxf(r, 0.0f), 15.0f);
    if (i < 4) lo |= q << (8 * i); else hi |= q << (8 * (i - 4));
  }
  // lanes j and j + 2 hold channels 8j.. and 16 + 8j..: together two words of the block
  const uint32_t got = __shfl_xor_sync(0xffffffffu, p.j < 2 ? hi : lo, 2);
  const uint32_t word = p.j < 2 ? (lo | got << 4) : (got | hi << 4);
  const int t = 2 * (p.j & 1) + (p.j >> 1);
  if (!p.live || !p.tile) return;
  const __half dh = __float2half_rn(d);
  if (!p.value) {
    *reinterpret_cast<uint32_t*>(p.tile + p.row * 16 * NB + t * 4 * NB + p.block * 4) = word;
    if (p.j == 0) reinterpret_cast<__half*>(p.tile + 16 * D)[p.row * NB + p.block] = dh;
  } else {
    const int pair = p.row >> 1, par = p.row & 1;
    uint8_t* at = p.tile + 8 * D + pair * 32 * NB + 2 * t * 4 * NB + p.block * 4 + par * 2;
    *reinterpret_cast<uint16_t*>(at) = (uint16_t)word;
    *reinterpret_cast<uint16_t*>(at + 4 * NB) = (uint16_t)(word >> 16);
    if (p.j == 0) reinterpret_cast<__half*>(p.tile + 17 * D)[(pair * NB + p.block) * 2 + par] = dh;
  }
}

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(256) kv_load_kernel(const KvView c, const RowArgs a) {
  constexpr int NB = D / 32;
  const Piece<D> p(c, a);
  if (!p.live) return;
  float x[8];
  if (p.tile) {
    const int t = 2 * (p.j & 1), sh = (p.j >> 1) * 4;
    uint32_t w[2];
    float d;
    if (!p.value) {
      const uint8_t* at = p.tile + p.row * 16 * NB + t * 4 * NB + p.block * 4;
      w[0] = *reinterpret_cast<const uint32_t*>(at);
      w[1] = *reinterpret_cast<const uint32_t*>(at + 4 * NB);
      d = __half2float(reinterpret_cast<const __half*>(p.tile + 16 * D)[p.row * NB + p.block]);
    } else {
      const int pair = p.row >> 1, par = p.row & 1;
      const uint8_t* at = p.tile + 8 * D + pair * 32 * NB + 2 * t * 4 * NB + p.block * 4 + par * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = *reinterpret_cast<const uint16_t*>(at + 2 * i * 4 * NB) |
               (uint32_t) * reinterpret_cast<const uint16_t*>(at + (2 * i + 1) * 4 * NB) << 16;
      d = __half2float(reinterpret_cast<const __half*>(p.tile + 17 * D)[(pair * NB + p.block) * 2 + par]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)((int)(w[i >> 2] >> (8 * (i & 3) + sh) & 15) - 8) * d;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __int_as_float(0x7fc00000);  // the table does not reach this row
  }
  T* dst = p.value ? static_cast<T*>(a.v) + p.tok * a.v_tok + p.head * a.v_head
                   : static_cast<T*>(a.k) + p.tok * a.k_tok + p.head * a.k_head;
  store8<T, VEC>(dst + p.block * 32 + p.j * 8, x);
}

// ------------------------------------------------------------------ eviction

struct EvictArgs {
  const int32_t* lens;
  int max_len;
  const float* score;  // [n_seqs][heads][max_len], strides in elements
  int64_t s_seq, s_head;
  int keep, recent;
  int32_t* out_lens;  // [n_seqs]
  int32_t* kept;      // [n_seqs][heads][keep]
  float* out_score;   // [n_seqs][heads][keep] or null
};

// Order-preserving code of a score; NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0;
  const uint32_t u = __float_as_uint(s + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;

// One CTA per sequence and head.  The need-th largest code among the older positions is
// found digit by digit (11, 11 and 10 bits, a shared-memory histogram each); a last pass
// writes every position whose code is larger, the first ones that are equal to it, and
// the recent ones, in order (warps own consecutive runs; ranks by ballots).
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const KvView c, const EvictArgs a) {
  __shared__ int hist[kSelBins];
  __shared__ int wsum[32], weq[32];
  __shared__ int s_digit, s_need;
  const int b = blockIdx.x / c.heads, h = blockIdx.x % c.heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len = a.lens[b];
  if (len < 0 || len > a.max_len || len > c.width * c.tiles_per_page * kTileTok) {
    if (tid == 0) kv_flag(c.error, MOE_DEVERR_PAGE);
    len = 0;
  }
  int32_t* kept = a.kept + (int64_t)blockIdx.x * a.keep;
  float* osc = a.out_score ? a.out_score + (int64_t)blockIdx.x * a.keep : nullptr;
  const float* sc = a.score + b * a.s_seq + h * a.s_head;
  const int n_out = min(len, a.keep);
  if (h == 0 && tid == 0) a.out_lens[b] = n_out;
  for (int i = n_out + tid; i < a.keep; i += kSelThreads) {
    kept[i] = -1;
    if (osc) osc[i] = 0.0f;
  }
  if (len <= a.keep) {
    for (int i = tid; i < len; i += kSelThreads) {
      kept[i] = i;
      if (osc) osc[i] = sc[i];
    }
    return;
  }
  const int n_old = len - a.recent;
  int need = a.keep - a.recent;  // of the n_old > need older positions
  uint32_t prefix = 0, mask = 0;
  if (need > 0) {
    const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
    for (int r = 0; r < 3; ++r) {
      const int nb = 1 << bits[r];
      for (int i = tid; i < nb; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n_old; i += kSelThreads) {
        const uint32_t k = score_key(sc[i]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift[r]) & (nb - 1)], 1);
      }
      __syncthreads();
      // thread tid owns bins nb - 1 - 2 tid and the one below it (top bins first)
      const int b0 = nb - 1 - 2 * tid, b1 = b0 - 1;
      const int c0 = b0 >= 0 ? hist[b0] : 0, c1 = b1 >= 0 ? hist[b1] : 0;
      int s = c0 + c1;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += y;
      }
      if (lane == 31) wsum[warp] = s;
      __syncthreads();
      if (warp == 0) {
        int y = wsum[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int z = __shfl_up_sync(0xffffffffu, y, off);
          if (lane >= off) y += z;
        }
        wsum[lane] = y;
      }
      __syncthreads();
      const int before = s - c0 - c1 + (warp ? wsum[warp - 1] : 0);  // codes above bin b0
      if (before < need && before + c0 >= need) {
        s_digit = b0;
        s_need = need - before;
      } else if (before + c0 < need && before + c0 + c1 >= need) {
        s_digit = b1;
        s_need = need - before - c0;
      }
      __syncthreads();
      prefix |= (uint32_t)s_digit << shift[r];
      mask |= (uint32_t)(nb - 1) << shift[r];
      need = s_need;  // how many of the codes equal to the prefix so far
      __syncthreads();
    }
  }
  // codes > prefix are kept, the first `need` codes == prefix too (none of either when
  // every place goes to recent positions)
  const bool any = a.keep > a.recent;
  const int seg = (len + kSelThreads - 1) / kSelThreads * 32;  // positions of one warp
  const int lo = warp * seg, hi = min(len, lo + seg);
  int n_gt = 0, n_eq = 0;
  for (int base = lo; base < hi; base += 32) {
    const int i = base + lane;
    const uint32_t k = i < hi && i < n_old ? score_key(sc[i]) : 0;
    const bool old = i < hi && i < n_old;
    n_gt += __popc(__ballot_sync(0xffffffffu, (old && any && k > prefix) || (i < hi && i >= n_old)));
    n_eq += __popc(__ballot_sync(0xffffffffu, old && any && k == prefix));
  }
  if (lane == 0) {
    wsum[warp] = n_gt;
    weq[warp] = n_eq;
  }
  __syncthreads();
  int gt = 0, eq = 0;
  for (int w = 0; w < warp; ++w) {
    gt += wsum[w];
    eq += weq[w];
  }
  const uint32_t below = (1u << lane) - 1;
  for (int base = lo; base < hi; base += 32) {
    const int i = base + lane;
    const float s = i < hi ? sc[i] : 0.0f;
    const bool old = i < hi && i < n_old;
    const uint32_t k = old ? score_key(s) : 0;
    const bool is_gt = (old && any && k > prefix) || (i < hi && i >= n_old);
    const bool is_eq = old && any && k == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const int my_eq = eq + __popc(be & below);
    const int rank = gt + __popc(bg & below) + min(my_eq, need);
    if (is_gt || (is_eq && my_eq < need)) {
      kept[rank] = i;
      if (osc) osc[rank] = s;
    }
    gt += __popc(bg);
    eq += __popc(be);
  }
}

constexpr int kMoveTiles = 4;  // destination tiles of one CTA

// Copies the kept rows to the destination pages: a row's bytes keep their place within a
// tile row, so 16-byte pieces move whole (keys) or as the halves of two source pairs
// (values).  Only bytes of rows below the new length are written.
template <int D>
__global__ void __launch_bounds__(192) kv_move_kernel(const KvView c, const KvView o, const EvictArgs a) {
  constexpr int NB = D / 32, ROWS = kMoveTiles * kTileTok;
  __shared__ const uint8_t* src[ROWS];  // source tile of each row
  __shared__ int srow[ROWS];
  __shared__ uint8_t* dst[kMoveTiles];
  const int bh = blockIdx.y, b = bh / c.heads, h = bh % c.heads;
  const int tid = threadIdx.x;
  const int r0 = blockIdx.x * ROWS;
  const int n = a.out_lens[b] - r0;  // rows of this CTA, may exceed ROWS
  if (n <= 0) return;
  if (tid < ROWS) {
    const uint8_t* t = nullptr;
    int r = 0;
    if (tid < n) {
      const int i = a.kept[(int64_t)bh * a.keep + r0 + tid];
      t = kv_tile(c, b, h, i >> 4);
      r = i & 15;
    }
    src[tid] = t;
    srow[tid] = r;
  } else if (tid < ROWS + kMoveTiles) {
    const int t = tid - ROWS;
    dst[t] = t * kTileTok < n ? kv_tile(o, b, h, r0 / kTileTok + t) : nullptr;
  }
  __syncthreads();
  constexpr int PC = D / 2;             // 16-byte pieces of a tile's key (and value) nibbles
  constexpr int PIECES = 2 * PC + 16 + 8 * NB;  // + key scales (a row each) + value scales (a word each)
  for (int w = tid; w < kMoveTiles * PIECES; w += blockDim.x) {
    const int t = w / PIECES, p = w % PIECES;
    uint8_t* d = dst[t];
    if (!d) continue;
    if (p < PC) {
      const int row = p / NB, part = p % NB, i = t * kTileTok + row;
      if (src[i])
        *reinterpret_cast<uint4*>(d + p * 16) = *reinterpret_cast<const uint4*>(src[i] + (srow[i] * NB + part) * 16);
    } else if (p < 2 * PC) {
      const int q = p - PC, pair = q / (2 * NB), part = q % (2 * NB), i = t * kTileTok + 2 * pair;
      uint4* to = reinterpret_cast<uint4*>(d + 8 * D + q * 16);
      const bool e0 = src[i] != nullptr, e1 = src[i + 1] != nullptr;
      if (!e0 && !e1) continue;
      uint4 x{}, y{};
      if (e0) x = *reinterpret_cast<const uint4*>(src[i] + 8 * D + ((srow[i] >> 1) * 2 * NB + part) * 16);
      if (e1) y = *reinterpret_cast<const uint4*>(src[i + 1] + 8 * D + ((srow[i + 1] >> 1) * 2 * NB + part) * 16);
      if (!e0 || !e1) {  // the other half of the pair stays as it is
        const uint4 z = *to;
        if (!e0) x = z; else y = z;
      }
      // half of each word that the source (or, for a row that stays, the destination) has
      const uint32_t s0 = e0 && (srow[i] & 1) ? 0x32u : 0x10u;
      const uint32_t s1 = e1 && !(srow[i + 1] & 1) ? 0x5400u : 0x7600u;
      const uint32_t sel = s0 | s1;
      uint4 r;
      r.x = __byte_perm(x.x, y.x, sel);
      r.y = __byte_perm(x.y, y.y, sel);
      r.z = __byte_perm(x.z, y.z, sel);
      r.w = __byte_perm(x.w, y.w, sel);
      *to = r;
    } else if (p < 2 * PC + 16) {
      const int row = p - 2 * PC, i = t * kTileTok + row;
      if (src[i]) {
#pragma unroll
        for (int k = 0; k < NB / 2; ++k)
          reinterpret_cast<uint32_t*>(d + 16 * D)[row * (NB / 2) + k] =
              reinterpret_cast<const uint32_t*>(src[i] + 16 * D)[srow[i] * (NB / 2) + k];
      }
    } else {
      const int q = p - 2 * PC - 16, pair = q / NB, nb = q % NB;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = t * kTileTok + 2 * pair + e;
        if (src[i])
          reinterpret_cast<uint16_t*>(d + 17 * D)[q * 2 + e] =
              reinterpret_cast<const uint16_t*>(src[i] + 17 * D)[((srow[i] >> 1) * NB + nb) * 2 + (srow[i] & 1)];
      }
    }
  }
}

// ------------------------------------------------------------------ entry points

template <typename T, bool VEC>
static void rows_launch(bool store, const KvView& c, const RowArgs& a, unsigned grid, cudaStream_t st) {
  if (c.dim == 64) {
    if (store) kv_store_kernel<T, 64, VEC><<<grid, 256, 0, st>>>(c, a);
    else kv_load_kernel<T, 64, VEC><<<grid, 256, 0, st>>>(c, a);
  } else {
    if (store) kv_store_kernel<T, 128, VEC><<<grid, 256, 0, st>>>(c, a);
    else kv_load_kernel<T, 128, VEC><<<grid, 256, 0, st>>>(c, a);
  }
}

static int rows_call(bool store, const moe_kv_pool* cache, const moe_kv_table* table, const int32_t* cu,
                     const int32_t* start, const moe_rows* k, const moe_rows* v, int32_t n_tokens, int32_t dtype,
                     void* stream) {
  KvView c;
  const int bad = kv_check(cache, table, &c);
  if (bad) return bad;
  if (!cu || !k || !v || !k->data_dev || !v->data_dev || n_tokens < 0) return MOE_ERR_INVALID;
  if (dtype != MOE_BF16 && dtype != MOE_F16 && dtype != MOE_F32) return MOE_ERR_INVALID;
  if (n_tokens == 0 || c.n_seqs == 0) return MOE_OK;
  const int64_t threads = (int64_t)n_tokens * c.heads * (c.dim / 4);
  if ((threads + 255) / 256 > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const int es = dtype == MOE_F32 ? 4 : 2;
  if (!kv_align_ok(k->data_dev, es) || !kv_align_ok(v->data_dev, es)) return MOE_ERR_INVALID;
  bool vec = kv_align_ok(k->data_dev, 16) && kv_align_ok(v->data_dev, 16);
  for (int64_t s : {k->token_stride, k->head_stride, v->token_stride, v->head_stride}) vec = vec && (s * es) % 16 == 0;
  const RowArgs a{k->data_dev, v->data_dev, k->token_stride, k->head_stride, v->token_stride, v->head_stride,
                  cu, start, n_tokens};
  DeviceScope dev(cache->device);
  if (!dev.ok) return MOE_ERR_CUDA;
  const unsigned grid = (unsigned)((threads + 255) / 256);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == MOE_F32) {
    if (vec) rows_launch<float, true>(store, c, a, grid, st); else rows_launch<float, false>(store, c, a, grid, st);
  } else if (dtype == MOE_F16) {
    if (vec) rows_launch<__half, true>(store, c, a, grid, st); else rows_launch<__half, false>(store, c, a, grid, st);
  } else {
    if (vec) rows_launch<__nv_bfloat16, true>(store, c, a, grid, st);
    else rows_launch<__nv_bfloat16, false>(store, c, a, grid, st);
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_kv_store(const moe_kv_pool* cache, const moe_kv_table* table, const int32_t* cu_dev,
                            const int32_t* start_dev, const moe_rows* k, const moe_rows* v, int32_t n_tokens,
                            int32_t dtype, void* stream) {
  return rows_call(true, cache, table, cu_dev, start_dev, k, v, n_tokens, dtype, stream);
}

extern "C" int moe_kv_load(const moe_kv_pool* cache, const moe_kv_table* table, const int32_t* cu_dev,
                           const int32_t* start_dev, const moe_rows* k, const moe_rows* v, int32_t n_tokens,
                           int32_t dtype, void* stream) {
  return rows_call(false, cache, table, cu_dev, start_dev, k, v, n_tokens, dtype, stream);
}

extern "C" int moe_kv_evict(const moe_kv_pool* cache, const moe_kv_table* table, const int32_t* len_dev,
                            int32_t max_len, const moe_kv_score* score, int32_t keep, int32_t recent,
                            const moe_kv_table* out_table, int32_t* out_len_dev, int32_t* kept_dev,
                            float* out_score_dev, void* stream) {
  KvView c, o;
  int bad = kv_check(cache, table, &c);
  if (!bad) bad = kv_check(cache, out_table, &o);
  if (bad) return bad;
  if (!len_dev || !score || !score->data_dev || !out_len_dev || !kept_dev) return MOE_ERR_INVALID;
  if (out_len_dev == len_dev || out_score_dev == score->data_dev) return MOE_ERR_INVALID;
  if (max_len < 0 || keep < 1 || recent < 0 || recent > keep || o.n_seqs != c.n_seqs) return MOE_ERR_INVALID;
  if (table->table_dev == out_table->table_dev) return MOE_ERR_INVALID;
  if ((int64_t)o.width * cache->page_tokens < keep) return MOE_ERR_INVALID;
  if (c.n_seqs == 0) return MOE_OK;
  if ((int64_t)c.n_seqs * c.heads > 65535) return MOE_ERR_UNSUPPORTED;
  const EvictArgs a{len_dev, max_len, score->data_dev, score->seq_stride, score->head_stride,
                    keep, recent, out_len_dev, kept_dev, out_score_dev};
  DeviceScope dev(cache->device);
  if (!dev.ok) return MOE_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  kv_select_kernel<<<c.n_seqs * c.heads, kSelThreads, 0, st>>>(c, a);
  const dim3 grid((keep + kMoveTiles * kTileTok - 1) / (kMoveTiles * kTileTok), c.n_seqs * c.heads);
  if (c.dim == 64) kv_move_kernel<64><<<grid, 192, 0, st>>>(c, o, a);
  else kv_move_kernel<128><<<grid, 192, 0, st>>>(c, o, a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
