// kv_cache.cu -- the 4-bit key/value cache of libmoe: writing rows into it, reading them
// back, and cutting sequences down to a budget by their accumulated attention weight.
#include <type_traits>

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

// The rows of a CTA: up to kMaxTok consecutive tokens of the packed batch, joined to pairs
// that share a pair of tile rows (values interleave two tokens byte by byte, so that both
// together fill whole words).  The page look-ups of a token are made once, by one thread, and not once per
// thread of its rows: a chain of dependent loads (sequence, start, page) is what such a
// kernel waits for.
constexpr int kMaxTok = 16;
struct Entry {
  int64_t at;   // tile of head 0 in the pool, or -1: the table does not reach it
  int tok, row;
  int both;     // the next token is in the next row of the same pair
};
struct Entries {
  Entry e[kMaxTok];
  int n;
};

// Tokens [tok0, tok0 + n_tok) of this CTA.  A token in an odd row belongs to the one before it, if that is in the
// same sequence: perhaps the last of the CTA before.
constexpr int kKnownSeqs = 255;  // bounds of so many sequences are read at once, into shared memory
__device__ __forceinline__ void kv_entries(const KvView& c, const RowArgs& a, int tok0, int n_tok, Entries* out) {
  __shared__ int bounds[kKnownSeqs + 1], first_pos[kKnownSeqs + 1];
  const bool known = c.n_seqs <= kKnownSeqs;
  if (known) {
    if ((int)threadIdx.x <= c.n_seqs) {
      bounds[threadIdx.x] = a.cu[threadIdx.x];
      first_pos[threadIdx.x] = a.start && (int)threadIdx.x < c.n_seqs ? a.start[threadIdx.x] : 0;
    }
    __syncthreads();
  }
  const int32_t* cu = known ? bounds : a.cu;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, tok = tok0 + lane;
    bool lead = lane < n_tok && tok < a.n_tokens && tok >= cu[0] && tok < cu[c.n_seqs];  // padding on either side is not a token
    int seq = 0, first = 0, end = 0;
    int64_t pos = 0;
    if (lead) {
      seq = kv_find_seq(cu, c.n_seqs, tok);
      first = cu[seq];
      end = min(cu[seq + 1], a.n_tokens);
      pos = (int64_t)(known ? first_pos[seq] : a.start ? a.start[seq] : 0) + tok - first;
      if ((pos & 1) && tok > first && tok > 0) lead = false;
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, lead);
    if (lead) {
      Entry e{-1, tok, (int)(pos & (kTileTok - 1)), !(pos & 1) && tok + 1 < end};
      const int64_t last = (int64_t)c.width * c.tiles_per_page * kTileTok;
      if (pos < 0 || pos >= last) {
        kv_flag(c.error, MOE_DEVERR_PAGE);
      } else {
        const uint8_t* t = kv_tile(c, seq, 0, (int)(pos / kTileTok));
        if (t) e.at = t - c.pool;
      }
      out->e[__popc(mask & ((1u << lane) - 1))] = e;
    }
    if (lane == 0) out->n = __popc(mask);
  }
  __syncthreads();
}

// 8 channels as they lie in memory, and their values.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, Raw8<T>& r) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i];
  }
}
template <typename T>
__device__ __forceinline__ void values8(const Raw8<T>& r, float (&x)[8]) {
  const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_float(e[i]);
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

// The 8 codes of a lane (a byte each, lo: channels 0..3), and the block's scale.  Four lanes
// share a block of 32 channels.
//
// fp32 rows: the definition as it stands, with a division.  The first value of the largest
// magnitude and a NaN flag go round by shuffles.
//
// 16-bit rows: magnitude, place and sign fit one 32-bit key (the low 13 bits of such a value
// in fp32 are 0), so that its maximum is the first largest value, NaN above all.  And
// x / d is computed as a product with 1 / d: where x / d is not exactly a border m + 1/2 it
// is at least 2^-13 away from it (both are ratios of 11-bit integers times a power of two), and product
// and sum are off by less than 2^-20, so adding 2^-18 puts exact borders on their upper side
// and moves nothing else across: the codes are the definition's, bit for bit.  A division
// each made the kernel bound by arithmetic (31 us against 23 us for 16383 tokens of 8 heads of 64).
template <typename T>
__device__ __forceinline__ float quantise8(const float (&x)[8], int j, uint32_t lanes, uint32_t* lo_out, uint32_t* hi_out) {
  uint32_t lo = 0, hi = 0;
  float d;
  if constexpr (sizeof(T) == 2) {
    uint32_t key = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = __float_as_uint(x[i]);
      key = max(key, (u & 0x7FFFFFFFu) | (u >> 31) | (uint32_t)((7 - i) << 1));
    }
    key |= (uint32_t)(3 - j) << 4;
    key = max(key, __shfl_xor_sync(lanes, key, 1));
    key = max(key, __shfl_xor_sync(lanes, key, 2));
    const float m = __uint_as_float((key & 0x7FFFE000u) | key << 31);
    const bool nan = (key & 0x7FFFE000u) > 0x7F800000u;
    d = nan ? __int_as_float(0x7fc00000) : fminf(fmaxf(m * -0.125f, -8188.0f), 8188.0f);
    float inv = __frcp_rn(d), y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    if (std::is_same<T, __half>::value) {
      if (d == 0.0f) inv = 0.0f;
    } else if (key < 0x0F000000u) {  // below 2^-97
      // 1 / d may be beyond fp32 here: both sides 2^64 times as large, which changes no code
      inv = d == 0.0f ? 0.0f : __frcp_rn(d * 0x1p64f);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i] * 0x1p64f;
    }
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // round(x / d + 8 + 2^-18) in the low bits of 2^23 + q
      float r = fminf(fmaf(y[i], inv, 8.0f + 3.814697265625e-6f), 15.0f);
      if (!std::is_same<T, __half>::value) r = fmaxf(r, 0.0f);  // only a limited d gives less: |x| > 65504
      q[i] = __float_as_uint(r + 8388608.0f);
    }
    lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
  } else {
    float m = x[0];
    int nan = x[0] != x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      if (fabsf(x[i]) > fabsf(m)) m = x[i];
      nan |= x[i] != x[i];
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      const float o = __shfl_xor_sync(lanes, m, off);
      nan |= __shfl_xor_sync(lanes, nan, off);
      const bool lower = (j & off) != 0;  // the other lane's channels come first
      if (fabsf(o) > fabsf(m) || (lower && fabsf(o) == fabsf(m))) m = o;
    }
    d = nan ? __int_as_float(0x7fc00000) : fminf(fmaxf(m * -0.125f, -8188.0f), 8188.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = floorf(__fadd_rn(d == 0.0f ? 0.0f : __fdiv_rn(x[i], d), 8.5f));
      const uint32_t q = (uint32_t)fminf(fmaxf(r, 0.0f), 15.0f);
      if (i < 4) lo |= q << (8 * i); else hi |= q << (8 * (i - 4));
    }
  }
  *lo_out = lo;
  *hi_out = hi;
  return d;
}

// How a CTA's threads share its entries and heads: a group of D / 8 lanes takes a row of keys
// (even warps) or values (odd warps), 8 channels a lane; groups go round the entries, and
// round the heads where there are fewer entries than groups.
template <int D>
struct Share {
  static constexpr int kLanes = D / 8, kGroups = 4 * 32 / kLanes;
  int j, block, entry, head, head_step;
  bool value;
  uint32_t lanes;  // of the group
  __device__ __forceinline__ explicit Share(int n) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in = lane % kLanes;
    const int group = (warp >> 1) * (32 / kLanes) + lane / kLanes;
    value = warp & 1;
    j = in & 3;
    block = in >> 2;
    lanes = (uint32_t)((1ull << kLanes) - 1) << (lane - in);
    head_step = n < kGroups ? kGroups / n : 1;
    entry = n < kGroups ? group % n : group;
    head = n < kGroups ? group / n : 0;
    if (head >= head_step) entry = n;  // a group too many
  }
};

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(256, 4) kv_store_kernel(const KvView c, const RowArgs a, int n_tok) {
  constexpr int NB = D / 32;
  __shared__ Entries es;
  kv_entries(c, a, blockIdx.x * n_tok, n_tok, &es);
  const int n = es.n;
  if (n == 0) return;
  const Share<D> sh(n);
  const int j = sh.j, block = sh.block, t = 2 * (j & 1) + (j >> 1);
  const T* src = static_cast<const T*>(sh.value ? a.v : a.k) + block * 32 + j * 8;
  const int64_t st_tok = sh.value ? a.v_tok : a.k_tok, st_head = sh.value ? a.v_head : a.k_head;
  for (int e = sh.entry; e < n; e += Share<D>::kGroups) {
    const Entry en = es.e[e];
    if (en.at < 0) continue;
    const T* p = src + en.tok * st_tok + sh.head * st_head;
    const int64_t head_bytes = (int64_t)c.tiles_per_page * (18 * D);
    uint8_t* tile = c.pool + en.at + sh.head * head_bytes;
    const int64_t step = sh.head_step * st_head;
    // the next head's channels are read before this one's are worked on
    Raw8<T> next[2];
    if (sh.head < c.heads) {
      load8<T, VEC>(p, next[0]);
      if (en.both) load8<T, VEC>(p + st_tok, next[1]);
    }
    for (int h = sh.head; h < c.heads; h += sh.head_step, tile += sh.head_step * head_bytes) {
      float x[2][8];
      values8(next[0], x[0]);
      values8(next[1], x[1]);
      p += step;
      if (h + sh.head_step < c.heads) {
        load8<T, VEC>(p, next[0]);
        if (en.both) load8<T, VEC>(p + st_tok, next[1]);
      }
      uint32_t word[2];
      __half d[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 1 && !en.both) break;
        uint32_t lo, hi;
        d[i] = __float2half_rn(quantise8<T>(x[i], j, sh.lanes, &lo, &hi));
        // lanes j and j + 2 hold channels 8j.. and 16 + 8j..: together two words of the block
        const uint32_t got = __shfl_xor_sync(sh.lanes, j < 2 ? hi : lo, 2);
        word[i] = j < 2 ? (lo | got << 4) : (got | hi << 4);
      }
      if (!sh.value) {
        uint8_t* at = tile + en.row * 16 * NB + t * 4 * NB + block * 4;
        __half* sc = reinterpret_cast<__half*>(tile + 16 * D) + en.row * NB + block;
        *reinterpret_cast<uint32_t*>(at) = word[0];
        if (j == 0) sc[0] = d[0];
        if (en.both) {
          *reinterpret_cast<uint32_t*>(at + 16 * NB) = word[1];
          if (j == 0) sc[NB] = d[1];
        }
      } else {
        const int pair = en.row >> 1, par = en.row & 1;
        uint8_t* at = tile + 8 * D + pair * 32 * NB + 2 * t * 4 * NB + block * 4;
        __half* sc = reinterpret_cast<__half*>(tile + 17 * D) + (pair * NB + block) * 2;
        if (en.both) {
          *reinterpret_cast<uint32_t*>(at) = __byte_perm(word[0], word[1], 0x5410);
          *reinterpret_cast<uint32_t*>(at + 4 * NB) = __byte_perm(word[0], word[1], 0x7632);
          if (j == 0) *reinterpret_cast<__half2*>(sc) = __halves2half2(d[0], d[1]);
        } else {
          *reinterpret_cast<uint16_t*>(at + par * 2) = (uint16_t)word[0];
          *reinterpret_cast<uint16_t*>(at + 4 * NB + par * 2) = (uint16_t)(word[0] >> 16);
          if (j == 0) sc[par] = d[0];
        }
      }
    }
  }
}

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(256, 6) kv_load_kernel(const KvView c, const RowArgs a, int n_tok) {
  constexpr int NB = D / 32;
  __shared__ Entries es;
  kv_entries(c, a, blockIdx.x * n_tok, n_tok, &es);
  const int n = es.n;
  if (n == 0) return;
  const Share<D> share(n);
  const int j = share.j, block = share.block, t = 2 * (j & 1), sh = (j >> 1) * 4;
  T* dst = static_cast<T*>(share.value ? a.v : a.k) + block * 32 + j * 8;
  const int64_t st_tok = share.value ? a.v_tok : a.k_tok, st_head = share.value ? a.v_head : a.k_head;
  for (int e = share.entry; e < n; e += Share<D>::kGroups) {
   const Entry en = es.e[e];
   T* p = dst + en.tok * st_tok + share.head * st_head;
   const int64_t head_bytes = (int64_t)c.tiles_per_page * (18 * D);
   const uint8_t* tile = c.pool + en.at + share.head * head_bytes;
   // words and scales of one head; read for the next head before this one's are worked on
   auto fetch = [&](uint32_t(&v)[4], __half(&s2)[2]) {
     if (!share.value) {
       const uint8_t* at = tile + en.row * 16 * NB + t * 4 * NB + block * 4;
       const __half* sc = reinterpret_cast<const __half*>(tile + 16 * D) + en.row * NB + block;
       v[0] = *reinterpret_cast<const uint32_t*>(at);
       v[1] = *reinterpret_cast<const uint32_t*>(at + 4 * NB);
       s2[0] = sc[0];
       if (en.both) {
         v[2] = *reinterpret_cast<const uint32_t*>(at + 16 * NB);
         v[3] = *reinterpret_cast<const uint32_t*>(at + 20 * NB);
         s2[1] = sc[NB];
       }
     } else {
       const int pair = en.row >> 1;
       const uint8_t* at = tile + 8 * D + pair * 32 * NB + 2 * t * 4 * NB + block * 4;
#pragma unroll
       for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint32_t*>(at + i * 4 * NB);
       *reinterpret_cast<__half2*>(s2) = reinterpret_cast<const __half2*>(tile + 17 * D)[pair * NB + block];
     }
   };
   const bool have = en.at >= 0;
   uint32_t v[4] = {0, 0, 0, 0};
   __align__(4) __half s2[2] = {__ushort_as_half(0x7e00), __ushort_as_half(0x7e00)};  // NaN where the table does not reach
   if (have && share.head < c.heads) fetch(v, s2);
   for (int h = share.head; h < c.heads; h += share.head_step, p += share.head_step * st_head) {
    uint32_t w[2][2];
    __half d[2];
    if (!share.value) {
      w[0][0] = v[0], w[0][1] = v[1], w[1][0] = v[2], w[1][1] = v[3];
      d[0] = s2[0], d[1] = s2[1];
    } else {
      const bool odd = en.row & 1;
      const uint32_t s0 = odd ? 0x7632 : 0x5410;
      w[0][0] = __byte_perm(v[0], v[1], s0), w[0][1] = __byte_perm(v[2], v[3], s0);
      w[1][0] = __byte_perm(v[0], v[1], 0x7632), w[1][1] = __byte_perm(v[2], v[3], 0x7632);
      d[0] = odd ? s2[1] : s2[0];
      d[1] = s2[1];
    }
    tile += share.head_step * head_bytes;
    if (have && h + share.head_step < c.heads) fetch(v, s2);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i == 1 && !en.both) break;
      // codes of channels 2k, 2k + 1 as 1024 + q in fp16, by bit operations (the integer
      // converter is a quarter as fast); q - 8 and, for fp16, its product with d are exact to one rounding
      uint32_t c2[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t b2 = __byte_perm(w[i][k >> 1] >> sh, 0, k & 1 ? 0x4342 : 0x4140);
        c2[k] = (b2 & 0x000F000Fu) | 0x64006400u;
      }
      uint32_t r[4];
      float x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 q = __hsub2(*reinterpret_cast<__half2*>(&c2[k]), __half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408)));
        if constexpr (std::is_same<T, __half>::value) {
          const __half2 v = __hmul2(q, __half2(d[i], d[i]));
          r[k] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
          const float df = __half2float(d[i]);
          const float2 v = __half22float2(q);
          x[2 * k] = v.x * df;
          x[2 * k + 1] = v.y * df;
        }
      }
      if constexpr (std::is_same<T, __half>::value) {
        if (VEC) {
          *reinterpret_cast<uint4*>(p + i * st_tok) = make_uint4(r[0], r[1], r[2], r[3]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) reinterpret_cast<uint16_t*>(p + i * st_tok)[k] = (uint16_t)(r[k >> 1] >> (16 * (k & 1)));
        }
      } else {
        store8<T, VEC>(p + i * st_tok, x);
      }
    }
   }
  }
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
  asm volatile("griddepcontrol.launch_dependents;");  // the second kernel starts up meanwhile
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
// (values).  Only bytes of rows below the new length are written.  A row whose page is not
// there gets scales of NaN, so that nobody reads what was in its place before.
template <int D>
__global__ void __launch_bounds__(192) kv_move_kernel(const KvView c, const KvView o, const EvictArgs a) {
  constexpr int NB = D / 32, ROWS = kMoveTiles * kTileTok;
  __shared__ const uint8_t* src[ROWS];  // source tile of each row
  __shared__ int srow[ROWS];
  __shared__ uint8_t* dst[kMoveTiles];
  const int bh = blockIdx.y, b = bh / c.heads, h = bh % c.heads;
  const int tid = threadIdx.x;
  const int r0 = blockIdx.x * ROWS;
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
      if (i < n) {
#pragma unroll
        for (int k = 0; k < NB / 2; ++k)
          reinterpret_cast<uint32_t*>(d + 16 * D)[row * (NB / 2) + k] =
              src[i] ? reinterpret_cast<const uint32_t*>(src[i] + 16 * D)[srow[i] * (NB / 2) + k] : 0x7E007E00u;
      }
    } else {
      const int q = p - 2 * PC - 16, pair = q / NB, nb = q % NB;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = t * kTileTok + 2 * pair + e;
        if (i < n)
          reinterpret_cast<uint16_t*>(d + 17 * D)[q * 2 + e] =
              src[i] ? reinterpret_cast<const uint16_t*>(src[i] + 17 * D)[((srow[i] >> 1) * NB + nb) * 2 + (srow[i] & 1)] : 0x7E00;
      }
    }
  }
}

// ------------------------------------------------------------------ entry points

template <typename T, bool VEC>
static cudaError_t rows_launch(bool store, const KvView& c, const RowArgs& a, int n_tok, cudaStream_t st) {
  const dim3 grid((a.n_tokens + n_tok - 1) / n_tok);
  if (c.dim == 64) return kv_launch(store ? kv_store_kernel<T, 64, VEC> : kv_load_kernel<T, 64, VEC>, grid, 256, 0, st, false, c, a, n_tok);
  return kv_launch(store ? kv_store_kernel<T, 128, VEC> : kv_load_kernel<T, 128, VEC>, grid, 256, 0, st, false, c, a, n_tok);
}

static int rows_call(bool store, const moe_kv_pool* cache, const moe_kv_table* table, const int32_t* cu,
                     const int32_t* start, const moe_rows* k, const moe_rows* v, int32_t n_tokens, int32_t dtype,
                     void* stream) {
  KvView c;
  const int bad = kv_check(cache, table, &c);
  if (bad) return bad;
  if (!cu || !k || !v || !k->data_dev || !v->data_dev || n_tokens < 0) return MOE_ERR_INVALID;
  if (dtype != MOE_BF16 && dtype != MOE_F16 && dtype != MOE_F32) return MOE_ERR_INVALID;
  if (n_tokens > kKvMaxPos) return MOE_ERR_UNSUPPORTED;
  if (!store)
    for (const moe_rows* r : {k, v})
      if (!kv_apart(r->token_stride, n_tokens, r->head_stride, c.heads)) return MOE_ERR_INVALID;
  if (n_tokens == 0 || c.n_seqs == 0) return MOE_OK;
  const int es = dtype == MOE_F32 ? 4 : 2;
  if (!kv_align_ok(k->data_dev, es) || !kv_align_ok(v->data_dev, es)) return MOE_ERR_INVALID;
  bool vec = kv_align_ok(k->data_dev, 16) && kv_align_ok(v->data_dev, 16);
  for (int64_t s : {k->token_stride, k->head_stride, v->token_stride, v->head_stride}) vec = vec && (s * es) % 16 == 0;
  const RowArgs a{k->data_dev, v->data_dev, k->token_stride, k->head_stride, v->token_stride, v->head_stride,
                  cu, start, n_tokens};
  DeviceScope dev(cache->device);
  if (!dev.ok) return MOE_ERR_CUDA;
  // Tokens of a CTA: the fewest, 2 to 16, with which four CTAs an SM take all of them at once.
  // With more, few tokens share few SMs; with fewer, each CTA's look-ups are paid again.
  // Storing 4 heads of 128, us with 2 / 4 / 8 / 16 tokens: 32 tokens 6.2 / 7.4 / 9.9 / 14.6,
  // 2047 12.5 / 9.5 / 10.5 / 13.7, 4096 20.1 / 14.3 / 12.9 / 15.4, 16383 68.8 / 44.8 / 33.2 / 28.9.
  int n_tok = 2;
  for (const int sms = kv_sm_count(cache->device); n_tok < kMaxTok && n_tokens > 4 * sms * n_tok;) n_tok *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == MOE_F32) return kv_status(vec ? rows_launch<float, true>(store, c, a, n_tok, st) : rows_launch<float, false>(store, c, a, n_tok, st));
  if (dtype == MOE_F16) return kv_status(vec ? rows_launch<__half, true>(store, c, a, n_tok, st) : rows_launch<__half, false>(store, c, a, n_tok, st));
  return kv_status(vec ? rows_launch<__nv_bfloat16, true>(store, c, a, n_tok, st) : rows_launch<__nv_bfloat16, false>(store, c, a, n_tok, st));
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
  if (o.n_seqs > 1 && o.table_stride == 0) return MOE_ERR_INVALID;
  if ((int64_t)o.width * cache->page_tokens < keep) return MOE_ERR_INVALID;
  if (max_len > kKvMaxPos) return MOE_ERR_UNSUPPORTED;
  if (c.n_seqs == 0) return MOE_OK;
  if ((int64_t)c.n_seqs * c.heads > 65535) return MOE_ERR_UNSUPPORTED;
  const EvictArgs a{len_dev, max_len, score->data_dev, score->seq_stride, score->head_stride,
                    keep, recent, out_len_dev, kept_dev, out_score_dev};
  DeviceScope dev(cache->device);
  if (!dev.ok) return MOE_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = kv_launch(kv_select_kernel, dim3(c.n_seqs * c.heads), kSelThreads, 0, st, false, c, a);
  const dim3 grid((keep + kMoveTiles * kTileTok - 1) / (kMoveTiles * kTileTok), c.n_seqs * c.heads);
  if (e == cudaSuccess) e = kv_launch(c.dim == 64 ? kv_move_kernel<64> : kv_move_kernel<128>, grid, 192, 0, st, true, c, o, a);
  return kv_status(e);
}
