// attend_prompt.cu -- causal attention of whole prompts for libmoe: grouped heads, sequences
// of different lengths packed into one call, on the 5th-generation tensor cores.
//
//   o_i = sum_{j <= i} p_ij v_j,  p_i = softmax_j(scale q_i . k_j)   inside each sequence
//
// Two products per key tile, S = Q K^T and O += P V, 4 D FLOP per (row, key) pair, bound by
// the tensor rate for long prompts; one exponential per pair is the next bound: a CTA's 256
// rows x 128 keys take 2048 cycles of tensor pipe (D = 128) and 2048 cycles of the
// exponential unit (16 per cycle and SM), so both have to run at the same time.
//
// Work item: 256 query rows of one head, as two tiles of 128 whose softmax and products
// alternate: while one tile's weights are formed, the tensor pipe works for the other.
// Warp roles, joined by mbarriers:
//   warps 0..3, 4..7  softmax of tile 0, 1: a thread owns a row; it reads S from tensor
//                     memory, keeps the row's maximum and sum in registers, writes P (16-bit) to
//                     tensor memory, and rescales O there when the maximum has grown
//   warp 8            TMA of Q, then of K and V tiles (128 keys) into a ring
//   warp 9            tcgen05.mma of S, both operands from shared memory
//   warp 10           tcgen05.mma of O, P from tensor memory and V from shared memory
//   warp 11           which item comes next
// The kernel is persistent, one CTA per SM: the next item's queries, keys and first products
// come while the last one's output is written, and items go out longest first.
// The maximum that a row's exponents refer to moves only when it is exceeded by more than
// 2^8, so most key tiles rescale nothing; P stays below 256, inside either 16-bit type.
// P is rounded to the input type (half a step per weight); sums, S and O are fp32.
#include <cuda.h>

#include <type_traits>

#include "kv_internal.h"

namespace moe {
namespace {

constexpr int kPM = 128;      // query rows of a tile
constexpr int kPN = 128;      // keys of a tile
constexpr int kPThreads = 384;  // three warpgroups, the last with the TMA and MMA warps

struct PromptArgs {
  const int32_t* cu;
  int n_seqs, n_tokens, n_heads, group, n_blocks;
  float scale2;  // scale * log2(e)
  void* out;
  int64_t o_tok, o_head;
  int vec;
  int stall;  // for tests: the first CTA (or pair) is never given its item of this number (0: it is given all)
  int32_t* error;
  const void *q, *k, *v;  // the rows themselves: see mend_rows
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
};

__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(kv_smem(b)), "r"(n) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred q;\n\tmbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(ok)
      : "r"(kv_smem(b)), "r"(parity), "r"(1000u)  // suspended for at most this many ns
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred q;\n\tmbarrier.test_wait.parity.shared::cta.b64 q, [%1], %2;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(ok)
      : "r"(kv_smem(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint32_t now_ns() {  // wraps after 4.3 s
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
// By whole warps.  False after 2 s, or soon after another role gave up.  (An attempt that fails takes
// about 4 us, so a count of attempts is a poor clock.)  Inline: a call here would make the softmax
// warps save their row of products.  Most phases are over when they are asked for: a test and a vote then take some 55
// cycles, an attempt with a time and a loop that each lane leaves by itself 170 (16384 tokens:
// 817 -> 802 us; 4 heads of 64, 8192 tokens: 72 -> 69).
constexpr uint32_t kLimitNs = 2000000000u;
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, bar_test(b, parity))) return true;
  const uint32_t t0 = now_ns();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, bar_try(b, parity))) return true;
    if (i % 256) continue;
    if (__any_sync(0xffffffffu, *abort)) return false;
    if (__any_sync(0xffffffffu, now_ns() - t0 > kLimitNs)) break;
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(kv_smem(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(kv_smem(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(kv_smem(b))
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(kv_smem(b)) : "memory");
}

// Shared-memory operand with 128-byte swizzle.  K-major (Q, K): rows of 64 elements, 8-row
// groups 1024 bytes apart.  MN-major (V): 64 channels of a key in 128 bytes, 8-key groups
// 1024 bytes apart (the stride offset), the next 64 channels lbo bytes on (the leading one).
__device__ __forceinline__ uint64_t op_desc(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

#define R8(v, i) v[i], v[i + 1], v[i + 2], v[i + 3], v[i + 4], v[i + 5], v[i + 6], v[i + 7]
#define O4(c, v, i) c(v[i]), c(v[i + 1]), c(v[i + 2]), c(v[i + 3])
#define O32(c, v)                                                                                                   \
  O4(c, v, 0), O4(c, v, 4), O4(c, v, 8), O4(c, v, 12), O4(c, v, 16), O4(c, v, 20), O4(c, v, 24), O4(c, v, 28)
#define O16(c, v) O4(c, v, 0), O4(c, v, 4), O4(c, v, 8), O4(c, v, 12)
__device__ __forceinline__ void tm_ld32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : O32("=r", r)
      : "r"(at));
}
__device__ __forceinline__ void tm_ld16(uint32_t at, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : O16("=r", r)
               : "r"(at));
}
__device__ __forceinline__ void tm_st16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::O16("r", r),
      "r"(at)
      : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Uses of loaded registers cannot be scheduled before the wait: they pass through here after it.
__device__ __forceinline__ void tm_landed16(uint32_t* r) { asm volatile("" : O16("+r", r)); }
__device__ __forceinline__ void tm_landed32(uint32_t* r) { asm volatile("" : O32("+r", r)); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// The other CTA of a pair: an address of this CTA's shared memory there, stores, arrivals.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(kv_smem(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_store(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool peer_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred q;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 q, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(ok)
      : "r"(kv_smem(b)), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool peer_wait(uint64_t* b, uint32_t parity, volatile int* abort) {
  const uint32_t t0 = now_ns();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, peer_try(b, parity))) return true;
    if (i % 256) continue;
    if (__any_sync(0xffffffffu, *abort)) return false;
    if (__any_sync(0xffffffffu, now_ns() - t0 > kLimitNs)) break;
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// acc + 0 * p of two 16-bit values: no longer 0 once one of them is not finite.
template <typename T>
__device__ __forceinline__ uint32_t odd2(uint32_t p, uint32_t acc);
template <>
__device__ __forceinline__ uint32_t odd2<__half>(uint32_t p, uint32_t acc) {
  asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(p), "r"(0u));
  return acc;
}
template <>
__device__ __forceinline__ uint32_t odd2<__nv_bfloat16>(uint32_t p, uint32_t acc) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(p), "r"(0u));
  return acc;
}

// Pairs of fp32: one instruction for two.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 256 query rows of one head.
struct PromptItem {
  int row0, n, block, head;  // first row and rows of the sequence, number of the 256 rows in it
  // key tiles of query tile w: up to the one on the diagonal; none for a second tile without rows
  __device__ __forceinline__ int tiles(int w) const {
    const int t = 2 * block + 1 + w;
    return w && t > (n + kPN - 1) / kPN ? 0 : t;
  }
  // those of CTA r of CL
  template <int CL>
  __device__ __forceinline__ int share(int w, int r) const {
    return CL == 1 ? tiles(w) : (tiles(w) - r + CL - 1) / CL;
  }
};

// Blocks of 256 rows of sequence b, its first row and its rows; none if its bounds cannot be.
__device__ __forceinline__ int prompt_blocks(const PromptArgs& a, int b, int* row, int* rows) {
  *row = *rows = 0;
  if (b >= a.n_seqs) return 0;
  const int s = a.cu[b], n = a.cu[b + 1] - s;
  if (s < 0 || n < 0 || n > a.n_tokens - s) {
    kv_flag(a.error, MOE_DEVERR_PAGE);
    return 0;
  }
  *row = s;
  *rows = n;
  return (n + 2 * kPM - 1) / (2 * kPM);
}

// Rows of one query tile whose output is not finite because of a value behind them.  On the
// diagonal the weights of later keys are 0, but 0 times an infinity or NaN is NaN in the product: it
// would reach up to 127 rows before that value's.  The warp finds where each channel's first
// value that is not finite stands in the diagonal tile and computes the channels of rows before it
// again, key by key from memory.  (Rows from it on are not finite by definition.)  Nothing of
// this runs while values are finite; a row of 16384 keys takes a warp about a millisecond.
template <typename T, int D, int COLS>
__device__ __forceinline__ void mend_rows(const PromptArgs& a, const PromptItem& it, int tile0, int r, bool odd, float m, float inv, int ch0) {
  constexpr int C = COLS / 32;  // channels of a lane, one after the other
  struct __align__(2 * C) Some { T x[C]; };
  const int lane = threadIdx.x & 31, kh = it.head / a.group;
  const T* v = static_cast<const T*>(a.v) + it.row0 * a.v_tok + kh * a.v_head + ch0 + C * lane;
  const T* k = static_cast<const T*>(a.k) + it.row0 * a.k_tok + kh * a.k_head;
  const int end = min(tile0 + kPN, it.n);
  int first[C];
#pragma unroll
  for (int i = 0; i < C; ++i) first[i] = end;
#pragma unroll 8
  for (int j = end - 1; j >= tile0; --j) {
    const Some y = *reinterpret_cast<const Some*>(v + j * a.v_tok);
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (!isfinite(to_float(y.x[i]))) first[i] = j;
  }
  uint32_t rows = __ballot_sync(0xffffffffu, odd && r < it.n && isfinite(inv));
#pragma unroll 1
  for (; rows; rows &= rows - 1) {
    const int src = __ffs(rows) - 1, row = __shfl_sync(0xffffffffu, r, src);
    bool need[C], any = false;
#pragma unroll
    for (int i = 0; i < C; ++i) any |= need[i] = first[i] > row && first[i] < end;
    if (!__any_sync(0xffffffffu, any)) continue;
    const float mr = __shfl_sync(0xffffffffu, m, src), fr = __shfl_sync(0xffffffffu, inv, src);
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (it.row0 + row) * a.q_tok + it.head * a.q_head);
    float o[C];
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = 0.0f;
#pragma unroll 1
    for (int j0 = row; j0 >= 0; j0 -= 32) {  // 32 keys at a time, the nearest first: a lane's product, then all lanes' values
      const uint4* kj = reinterpret_cast<const uint4*>(k + max(j0 - lane, 0) * a.k_tok);
      float s = 0.0f;
#pragma unroll 8
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = q[c], y = kj[c];
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(to_float(reinterpret_cast<const T*>(&x)[i]), to_float(reinterpret_cast<const T*>(&y)[i]), s);
      }
      const float w = lane <= j0 ? ex2((s - mr) * a.scale2) : 0.0f;  // (behind key 0: its value again, with no weight)
#pragma unroll 16
      for (int e = 0; e < 32; ++e) {
        const float we = __shfl_sync(0xffffffffu, w, e);
        const Some y = *reinterpret_cast<const Some*>(v + max(j0 - e, 0) * a.v_tok);
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = fmaf(we, to_float(y.x[i]), o[i]);
      }
      bool done = true;
#pragma unroll
      for (int i = 0; i < C; ++i) done &= !need[i] || o[i] != o[i];
      if (__all_sync(0xffffffffu, done)) break;  // a NaN before this tile
    }
    T* dst = static_cast<T*>(a.out) + (int64_t)(it.row0 + row) * a.o_tok + it.head * a.o_head + ch0 + C * lane;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (need[i]) dst[i] = from_float<T>(o[i] * fr);
  }
}

// Items of this CTA (or pair), in order, by a whole warp; f says whether to go on.  s, n and mine:
// prompt_blocks of the sequence of this lane's number.
//
// Longest first: blocks by their number within the sequence (the key tiles they need), the
// last ones first; of those with the same number all sequences that have it, of each all
// heads side by side (they share keys and values).  Of every gridDim items in that order a
// CTA takes one, from the front and from the back in turn (from the front alone, the first
// CTA has the longest each time: 880 us against 814 for one prompt of 16384 tokens).
// Up to 32 sequences a lane keeps its own; of more, all bounds are read again for every block
// number: one prompt of 16384 tokens among 31 or 33 short ones takes 790 us, among 1000 1360,
// among 8000 7900 (8000 short ones alone 3300).
template <int CL, typename F>
__device__ __forceinline__ void each_item(const PromptArgs& a, int s, int n, int mine, F&& f) {
  const int lane = threadIdx.x & 31;
  int most = __reduce_max_sync(0xffffffffu, mine);
  for (int b = 32; b < a.n_seqs; b += 32) {
    mine = prompt_blocks(a, b + lane, &s, &n);
    most = max(most, __reduce_max_sync(0xffffffffu, mine));
  }
  int64_t before = 0, want = blockIdx.x / CL;  // items before the sequences looked at; the next one wanted
  const int64_t step = gridDim.x / CL;
  bool ok = true;
  const bool few = a.n_seqs <= 32;  // then every lane keeps its sequence
  for (int q = most - 1; q >= 0 && ok; --q) {
    for (int b = 0; b < a.n_seqs && ok; b += 32) {
      if (!few) mine = prompt_blocks(a, b + lane, &s, &n);
      const uint32_t has = __ballot_sync(0xffffffffu, mine > q);
      const int64_t here = (int64_t)__popc(has) * a.n_heads;
      while (want < before + here && ok) {
        const int k = (int)(want - before) / a.n_heads, head = (int)(want - before) % a.n_heads;
        // the k-th sequence that has this block
        const int src = __ffs(__ballot_sync(0xffffffffu, (has >> lane & 1) && __popc(has & ((1u << lane) - 1)) == k)) - 1;
        ok = f(PromptItem{__shfl_sync(0xffffffffu, s, src), __shfl_sync(0xffffffffu, n, src), q, head});
        const int64_t round = want / step;
        want = (round + 2) * step - 1 - (want - round * step);
      }
      before += here;
    }
  }
}

template <int D>
struct PromptSmem {
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr uint32_t kBox = 128 * 128;             // 128 rows of 64 elements
  static constexpr uint32_t kTileB = (D / 64) * kBox;     // a Q, K or V tile
  static constexpr uint32_t kQ = 0, kK = 2 * kTileB, kV = kK + kStages * kTileB, kEnd = kV + kStages * kTileB;
  static constexpr uint32_t kBars = kEnd, kML = kEnd + 512, kBytes = kML + 2048 + 1024;  // + alignment to 1024
};

// Tensor memory columns.  P has columns of its own, so that S is free as soon as the softmax warps have it in
// registers: with D = 64 each query tile has an S, with D = 128 there is room for one, which
// the two tiles take in turn.
template <int D>
struct PromptTmem {
  static constexpr int kS = D == 64 ? 2 : 1;
  __device__ static constexpr uint32_t s(int w) { return kS == 2 ? 128 * w : 0; }
  __device__ static constexpr uint32_t p(int w) { return 128 * kS + 64 * w; }
  __device__ static constexpr uint32_t o(int w) { return 128 * kS + 128 + D * w; }
};
static_assert(PromptTmem<64>::kS * 128 + 128 + 2 * 64 <= 512 && PromptTmem<128>::kS * 128 + 128 + 2 * 128 <= 512, "512 columns");

// CL = 2: a pair of CTAs (a cluster) shares an item.  CTA r takes key tiles r, r + 2, ..; at the end each
// gives the other its half of the channels of O with the rows' maxima and sums, through
// distributed shared memory (where Q was), and writes the joined other half.  For calls with fewer
// items than SMs, where the longest item alone is the call's time.
template <typename T, int D, int CL>
__global__ void __launch_bounds__(kPThreads, 1)
    attend_prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv) {
  using S = PromptSmem<D>;
  using M = PromptTmem<D>;
  constexpr int ST = S::kStages, NB = D / 64;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (kv_smem(raw) & 1023u)) & 1023u);
  // Barriers.  Those of a query tile, then those of the ring, then the items'.
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + S::kBars);
  uint64_t *q_empty = q_full + 2, *s_full = q_full + 4, *s_free = q_full + 6, *p_half = q_full + 8, *p_full = q_full + 10,
           *o_done = q_full + 12, *o_free = q_full + 14, *fix = q_full + 16;
  uint64_t *k_full = q_full + 17, *k_empty = k_full + ST, *v_full = k_empty + ST, *v_empty = v_full + ST;
  uint64_t *item_full = v_empty + ST, *item_empty = item_full + 2;
  // pairs: S of an item done here; Q's place free at the other CTA; its halves arrived; ours read
  uint64_t *s_all = item_empty + 2, *peer_ready = s_all + 1, *merge_full = s_all + 2, *merged = s_all + 4;
  uint64_t* drained = s_all + 5;  // after a wait that ran out: the products of each MMA warp are through
  PromptItem* items = reinterpret_cast<PromptItem*>(s_all + 7);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(items + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_at + 1);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = CL == 1 ? 0 : blockIdx.x % CL;  // in the pair: clusters are consecutive CTAs

  if (tid == 0) {
    *abort = 0;
    for (int i = 0; i < 2; ++i) {
      bar_init(q_full + i, 1);
      bar_init(q_empty + i, 1);
      bar_init(s_full + i, 1);
      bar_init(s_free + i, 4);
      bar_init(p_half + i, 4);
      bar_init(p_full + i, 4);
      bar_init(o_done + i, 1);
      bar_init(o_free + i, 4);
      bar_init(item_full + i, 1);
      bar_init(item_empty + i, 11);  // softmax, TMA and MMA warps
    }
    bar_init(fix, 1);
    bar_init(s_all, 1);
    bar_init(peer_ready, 1);
    bar_init(merge_full, 4);
    bar_init(merge_full + 1, 4);
    bar_init(merged, 8);
    bar_init(drained, 1);
    bar_init(drained + 1, 1);
    for (int i = 0; i < ST; ++i) {
      bar_init(k_full + i, 1);
      bar_init(k_empty + i, 1);
      bar_init(v_full + i, 1);
      bar_init(v_empty + i, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  int seq_row = 0, seq_rows = 0, seq_blocks = 0;  // of this lane's sequence (warp 11), read while the rest is set up
  if (warp == 11) seq_blocks = prompt_blocks(a, lane, &seq_row, &seq_rows);
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(kv_smem(tmem_at)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  if (CL > 1) cluster_sync();  // the other CTA's barriers are there
  tc_after();
  const uint32_t tmem = *tmem_at;
  const uint32_t qa = kv_smem(sm + S::kQ), ka = kv_smem(sm + S::kK), va = kv_smem(sm + S::kV);

  // The next item of a role, or one without rows when there are no more (or a wait ran out).
  auto take = [&](int turn) {
    PromptItem it{-1, 0, 0, 0};
    if (bar_wait(item_full + (turn & 1), (turn >> 1) & 1, abort)) {
      it = items[turn & 1];
      __syncwarp();
      if (lane == 0) bar_arrive(item_empty + (turn & 1));
    }
    return it;
  };

  // Registers: the softmax warps hold a row of 128 products each; 2 x 208 + 88 are the
  // 3 x 168 that the kernel was launched with.
  if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int w = warp >> 2;
    auto row = [] { return (int)(threadIdx.x & (kPM - 1)); };  // rarely used: not worth a register
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t st = tmem + lanes + M::s(w), pt = tmem + lanes + M::p(w), ot = tmem + lanes + M::o(w);
    bool ok = true;
    int done = 0;  // key tiles of the items before: the barriers' phases go on
    int merges = 0;
    for (int turn = 0; ok; ++turn) {
     // The item stays in its slot until its output is written, so that only its number of key
     // tiles is in registers meanwhile.
     if (!bar_wait(item_full + (turn & 1), (turn >> 1) & 1, abort)) break;
     const volatile PromptItem* slot = items + (turn & 1);
     const int all = slot->row0 < 0 ? -1 : PromptItem{0, slot->n, slot->block, 0}.tiles(w);
     if (all <= 0) {
       __syncwarp();
       if (lane == 0) bar_arrive(item_empty + (turn & 1));
       if (CL > 1 && all == 0) {  // not before the item before is through: the phases count arrivals
         if (turn) ok = bar_wait(merged, (turn - 1) & 1, abort);
         if (lane == 0) bar_arrive(merged);
       }
       if (all) break;
       continue;
     }
     const int nt = CL == 1 ? all : PromptItem{0, slot->n, slot->block, 0}.share<CL>(w, rank);
     const bool diagonal = CL == 1 || (all - 1) % CL == (int)rank;  // the last key tile is this CTA's
     // A tile without keys here waits for no product of this turn, so nothing else keeps it from
     // being through before the item before is: then `merged` would count its arrivals twice.
     if (CL > 1 && nt == 0 && turn) ok = bar_wait(merged, (turn - 1) & 1, abort);
     float m = -INFINITY, l = 0.0f;  // m in units of S
     for (int j = 0; j < nt && ok; ++j) {
      ok = bar_wait(s_full + w, (done + j) & 1, abort);
      if (!ok) break;
      tc_after();
      uint32_t s[128];
      float* f = reinterpret_cast<float*>(s);
#pragma unroll
      for (int c = 0; c < 4; ++c) tm_ld32(st + 32 * c, s + 32 * c);
      tm_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) tm_landed32(s + 32 * c);
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(s_free + w);
      if (j == nt - 1 && diagonal) {  // the diagonal tile: keys behind the row (and so behind the sequence)
#pragma unroll
        for (int c = 0; c < 128; ++c) f[c] = c > row() ? -INFINITY : f[c];
      }
      float mx[4] = {f[0], f[1], f[2], f[3]};
#pragma unroll
      for (int c = 4; c < 124; c += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], f[c + i], f[c + 4 + i]);
      }
      const float top = max3(max3(mx[0], mx[1], f[124]), max3(mx[2], mx[3], f[125]), fmaxf(f[126], f[127]));
      if (__any_sync(0xffffffffu, (top - m) * a.scale2 > 8.0f)) {
        const float mn = fmaxf(m, top);
        const float al = m == mn ? 1.0f : ex2((m - mn) * a.scale2);
        m = mn;
        l *= al;
        if (j > 0) {
          ok = bar_wait(o_done + w, (done + j - 1) & 1, abort);
          if (!ok) break;
          tc_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tm_ld16(ot + c, o);
            tm_wait_ld();
            tm_landed16(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
            tm_st16(ot + c, o);
          }
        }
      }
      // A part of the weights by a polynomial on the FMA pipe instead of the exponential unit was
      // tried (an eighth to a half of them): 1216..1255 against 1255 TFLOP/s, the issue slots being taken as well.
      const float off = m == -INFINITY ? 0.0f : -m * a.scale2;  // products of -inf only, so far: no weight
      const uint64_t sc = f2(a.scale2, a.scale2), of = f2(off, off);
      uint64_t sum[4] = {0, 0, 0, 0};
      auto weights = [&](int c, uint32_t(&p)[16]) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const uint64_t v = fma2(f2(f[c + i], f[c + i + 1]), sc, of);
          float x, y;
          unpack(v, x, y);
          x = ex2(x);
          y = ex2(y);
          sum[(i >> 1) & 3] = add2(sum[(i >> 1) & 3], f2(x, y));
          p[i >> 1] = pack2<T>(x, y);
        }
      };
      uint32_t p[16];
      weights(0, p);
      if (j > 0) {  // P of the tile before must have been used
        ok = bar_wait(o_done + w, (done + j - 1) & 1, abort);
        if (!ok) break;
        tc_after();
      }
      tm_st16(pt, p);
      weights(32, p);
      tm_st16(pt + 16, p);
      tm_wait_st();  // the first half of P V can start
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(p_half + w);
      weights(64, p);
      tm_st16(pt + 32, p);
      weights(96, p);
      tm_st16(pt + 48, p);
      {
        float x, y;
        unpack(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), x, y);
        l += x + y;
      }
      tm_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(p_full + w);
    }
     if (ok && nt) ok = bar_wait(o_done + w, (done + nt - 1) & 1, abort);
     done += nt;
     tc_after();
     const PromptItem it{slot->row0, slot->n, slot->block, slot->head};
     __syncwarp();
     if (lane == 0) bar_arrive(item_empty + (turn & 1));
     const int r = it.block * 2 * kPM + w * kPM + row();
     constexpr int COLS = D / CL;  // channels that this CTA writes
     float f0 = 1.0f, f1 = 0.0f;   // weights of its own partial output and of the other's
     const float* theirs = reinterpret_cast<const float*>(sm + S::kQ) + w * COLS * kPM + row();
     if constexpr (CL > 1) {
       const uint32_t other = rank ^ 1;
       if (ok) ok = peer_wait(peer_ready, turn & 1, abort);
       if (ok) {
         const uint32_t to = peer_addr(theirs, other);
#pragma unroll 1
         for (int c = 0; c < COLS; c += 32) {
           uint32_t o[32];
           if (nt) {
             tm_ld32(ot + other * COLS + c, o);
             tm_wait_ld();
             tm_landed32(o);
           }
#pragma unroll
           for (int i = 0; i < 32; ++i) peer_store(to + (c + i) * (kPM * 4), nt ? __uint_as_float(o[i]) : 0.0f);
         }
         float* ml = reinterpret_cast<float*>(sm + S::kML) + w * 2 * kPM + row();
         peer_store(peer_addr(ml, other), m);
         peer_store(peer_addr(ml + kPM, other), l);
         asm volatile("fence.acq_rel.cluster;" ::: "memory");
         __syncwarp();
         if (lane == 0) peer_arrive(peer_addr(merge_full + w, other));
         ok = peer_wait(merge_full + w, merges & 1, abort);
         const float m1 = ml[0], l1 = ml[kPM], top = fmaxf(m, m1);
         f0 = m == top ? 1.0f : ex2((m - top) * a.scale2);
         f1 = m1 == top ? 1.0f : ex2((m1 - top) * a.scale2);
         l = l * f0 + l1 * f1;
         m = top;
       }
       ++merges;
     }
     const float inv = ok ? 1.0f / l : __int_as_float(0x7fc00000);
     if (!ok && lane == 0) kv_flag(a.error, MOE_DEVERR_TMA);
     T* dst = static_cast<T*>(a.out) + (int64_t)(it.row0 + r) * a.o_tok + it.head * a.o_head + rank * COLS;
     uint32_t odd = 0;
#pragma unroll 1
     for (int c = 0; c < COLS; c += 32) {
       uint32_t o[32];
       if (nt) {
         tm_ld32(ot + rank * COLS + c, o);
         tm_wait_ld();
         tm_landed32(o);
         if (c == COLS - 32) {  // O may be written again
           tc_before();
           __syncwarp();
           if (lane == 0) bar_arrive(o_free + w);
         }
       }
       if constexpr (CL > 1) {
#pragma unroll
         for (int i = 0; i < 32; ++i) {
           const float own = nt ? __uint_as_float(o[i]) * f0 : 0.0f;
           o[i] = __float_as_uint(fmaf(theirs[(c + i) * kPM], f1, own));
         }
       }
       if (r < it.n) {
         uint32_t p[16];
#pragma unroll
         for (int i = 0; i < 16; ++i) p[i] = pack2<T>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
#pragma unroll
         for (int i = 0; i < 16; ++i) odd = odd2<T>(p[i], odd);
         if (a.vec) {
#pragma unroll
           for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(dst + c)[i] = make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
         } else {
#pragma unroll
           for (int i = 0; i < 32; ++i) reinterpret_cast<uint16_t*>(dst + c)[i] = (uint16_t)(p[i >> 1] >> (16 * (i & 1)));
         }
       }
     }
     if (__any_sync(0xffffffffu, odd != 0)) {
       __syncwarp();  // the rows are written: what follows writes some of their channels again
       mend_rows<T, D, COLS>(a, it, it.block * 2 * kPM + w * kPM, r, odd != 0, m, inv, rank * COLS);
     }
     if (CL > 1) {  // Q's place may be loaded again
       asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
       __syncwarp();
       if (lane == 0) bar_arrive(merged);
     }
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------------- TMA
    bool ok = true;
    int kv = 0, ks = 0, fixes = 0, loads[2] = {0, 0};  // tiles of values, of keys, cleared tails and query tiles so far
    int products = 0;                          // items with key tiles of this CTA's so far
    for (int turn = 0; ok; ++turn) {
      const PromptItem it = take(turn);
      if (it.row0 < 0) break;
      const int kh = it.head / a.group, n_kv = it.share<CL>(it.tiles(1) ? 1 : 0, rank);
      if (CL > 1 && turn) ok = bar_wait(merged, (turn - 1) & 1, abort);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!ok || !it.share<CL>(w, rank)) continue;
        if (loads[w]) ok = bar_wait(q_empty + w, (loads[w] - 1) & 1, abort);
        if (ok && lane == 0) {
          bar_expect(q_full + w, S::kTileB);
          for (int c = 0; c < NB; ++c)
            tma3(qa + w * S::kTileB + c * S::kBox, &mq, 64 * c, it.head, it.row0 + it.block * 2 * kPM + w * kPM, q_full + w);
        }
        ++loads[w];
      }
      for (int j = 0; j < n_kv && ok; ++j, ++kv) {
        const int s = kv % ST, round = kv / ST, key0 = it.row0 + (j * CL + rank) * kPN;
        if (round) ok = bar_wait(k_empty + s, (round - 1) & 1, abort);
        if (!ok) break;
        if (lane == 0) {
          bar_expect(k_full + s, S::kTileB);
          for (int c = 0; c < NB; ++c) tma3(ka + s * S::kTileB + c * S::kBox, &mk, 64 * c, kh, key0, k_full + s);
        }
        ++ks;
        if (round) ok = bar_wait(v_empty + s, (round - 1) & 1, abort);
        if (!ok) break;
        const int left = it.n - (j * CL + rank) * kPN;  // keys of this tile that are the sequence's
        uint64_t* vb = left < kPN ? fix : v_full + s;
        if (lane == 0) {
          bar_expect(vb, S::kTileB);
          for (int c = 0; c < NB; ++c) tma3(va + s * S::kTileB + c * S::kBox, &mv, 64 * c, kh, key0, vb);
        }
        if (left < kPN) {
          // Values behind the sequence (another one's, perhaps not finite) meet weights of 0:
          // they are cleared before the product sees them.
          ok = bar_wait(fix, fixes & 1, abort);
          if (!ok) break;
          ++fixes;
          for (int i = lane; i < (kPN - left) * NB * 8; i += 32) {
            const int r = left + i / (NB * 8), c = (i / 8) % NB;
            *reinterpret_cast<uint4*>(sm + S::kV + s * S::kTileB + c * S::kBox + r * 128 + (i % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) bar_arrive(v_full + s);
        }
      }
      if (CL > 1) {  // when S is done here, the other CTA may write where Q was
        // Counted in items that have key tiles here: the other ones (a pair's second CTA has none of a
        // sequence of up to 128 rows) have no Q either, and their commits could complete with
        // those of the item before, two phases at once.  With key tiles, the next commit needs keys that
        // are asked for after this wait.
        if (ok && n_kv) ok = bar_wait(s_all, products++ & 1, abort);
        if (ok && lane == 0) peer_arrive(peer_addr(peer_ready, rank ^ 1));
      }
    }
    if (__any_sync(0xffffffffu, *abort)) {  // what was asked for may still be on its way (each wait ends soon now)
      for (int w = 0; w < 2; ++w) bar_wait(q_full + w, (loads[w] - 1) & 1, abort);
      for (int s = 0; s < ST; ++s) {  // the last round of each stage; -1, a phase that is over, if there was none
        bar_wait(k_full + s, (ks > s ? (ks - 1 - s) / ST : -1) & 1, abort);
        bar_wait(v_full + s, (ks > s ? (ks - 1 - s) / ST : -1) & 1, abort);
      }
      bar_wait(fix, fixes & 1, abort);
    }
  } else if (warp < 11) {
    // ---------------------------------------------------------------- MMA
    // A whole warp walks the loop and one elected lane issues: descriptors and barriers then live in
    // uniform registers, where the instructions take them.  (With a single lane in the branch every
    // product cost some 65 cycles of register moves and every wait 250.)  S and P V are
    // independent but for their barriers, so each has a warp: one warp for both spends half a
    // turn in waits that come one after the other.
    constexpr uint32_t ty = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    constexpr uint32_t base = (1u << 4) | (ty << 7) | (ty << 10) | ((uint32_t)(kPM >> 4) << 24);
    const bool leader = elect_one();
    bool ok = true;
    // Phases of the barriers, in the bits of one word (uniform registers are scarce: counters cost
    // a reload at every product): of the ring, and for query tile w at bits w, w + 2, w + 4.
    int s = 0;
    uint32_t ring = 0, bits = 0;
    if (warp == 9) {
      // S of key tile j, tile 0 then tile 1; the columns are free when the softmax warps have what
      // was in them in registers: the other query tile's S where they share them, else its own.
      constexpr uint32_t id_s = base | ((uint32_t)(kPN >> 3) << 17);
      const uint64_t qd = op_desc(qa, 16), kd = op_desc(ka, 16);
      int last = -1;  // whose S was issued last
      for (int turn = 0; ok; ++turn) {
        const PromptItem it = take(turn);
        if (it.row0 < 0) break;
        const int n0 = it.share<CL>(0, rank), n1 = it.share<CL>(1, rank), n_kv = n1 ? n1 : n0;
        for (int j = 0; j < n_kv && ok; ++j) {
          ok = bar_wait(k_full + s, ring, abort);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int nt = w ? n1 : n0;
            if (!ok || j >= nt) continue;
            if (j == 0) {  // bit w: queries read
              ok = bar_wait(q_full + w, bits >> w & 1, abort);
              bits ^= 1u << w;
            }
            // bit w + 2: the phase of s_free that the last S of tile w completes; bit w + 4: there was one
            if (M::kS == 2) {
              if (ok && (bits >> (4 + w) & 1)) ok = bar_wait(s_free + w, bits >> (2 + w) & 1, abort);
            } else if (ok && last >= 0) {
              ok = bar_wait(s_free + last, bits >> (2 + last) & 1, abort);
            }
            if (!ok) continue;
            tc_after();
            if (leader) {
              const uint64_t q = qd + w * (S::kTileB >> 4), k = kd + s * (S::kTileB >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * S::kBox + (kk & 3) * 32) >> 4;
                mma_ss(tmem + M::s(w), q + o, k + o, id_s, kk > 0);
              }
              commit(s_full + w);
              if (w == 1 || !n1) commit(k_empty + s);
              if (j == nt - 1) commit(q_empty + w);
            }
            __syncwarp();
            if (bits >> (4 + w) & 1) bits ^= 4u << w; else bits |= 16u << w;
            last = w;
          }
          if (++s == ST) s = 0, ring ^= 1;
        }
        if (CL > 1 && n_kv) {
          if (leader && ok) commit(s_all);
          __syncwarp();
        }
      }
    } else {
      constexpr uint32_t id_o = base | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // V is MN-major
      const uint64_t vd = op_desc(va, S::kBox);
      for (int turn = 0; ok; ++turn) {
        const PromptItem it = take(turn);
        if (it.row0 < 0) break;
        const int n0 = it.share<CL>(0, rank), n1 = it.share<CL>(1, rank), n_kv = n1 ? n1 : n0;
        for (int j = 0; j < n_kv && ok; ++j) {
          ok = bar_wait(v_full + s, ring, abort);
          // The two halves of the weights of each query tile in the order in which they come: with an S each
          // (D = 64) the tiles keep step, first halves before second ones (9 packed prompts 50.4 -> 48.3 us);
          // with one S in turn, tile 0 is half a turn ahead.
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int w = M::kS == 2 ? i & 1 : i >> 1, half = M::kS == 2 ? i >> 1 : i & 1;
            if (!ok || j >= (w ? n1 : n0)) continue;
            if (j == 0 && half == 0) {  // bit w + 2: the phase of o_free that the last item of tile w completes; bit w + 4: there was one
              if (bits >> (4 + w) & 1) {
                ok = bar_wait(o_free + w, bits >> (2 + w) & 1, abort);
                bits ^= 4u << w;
              } else {
                bits |= 16u << w;
              }
            }
            // bit w: weights used
            if (ok) ok = bar_wait((half ? p_full : p_half) + w, bits >> w & 1, abort);
            if (!ok) continue;
            tc_after();
            if (leader) {
              const uint64_t v = vd + s * (S::kTileB >> 4);
#pragma unroll
              for (int kk = 0; kk < kPN / 32; ++kk) {
                const int k = half * (kPN / 32) + kk;
                mma_ts(tmem + M::o(w), tmem + M::p(w) + k * 8, v + k * (2048 >> 4), id_o, j > 0 || k > 0);
              }
              if (half) {
                commit(o_done + w);
                if (w == 1 || !n1) commit(v_empty + s);
              }
            }
            __syncwarp();
            if (half) bits ^= 1u << w;
          }
          if (++s == ST) s = 0, ring ^= 1;
        }
      }
    }
    if (__any_sync(0xffffffffu, *abort)) {
      if (leader) commit(drained + warp - 9);
      __syncwarp();
      bar_wait(drained + warp - 9, 0, abort);
    }
  } else {
    // ---------------------------------------------------------------- items
    int turn = 0;
    bool ok = true;
    auto give = [&](const PromptItem& it) {
      if (turn > 1) ok = bar_wait(item_empty + (turn & 1), ((turn >> 1) - 1) & 1, abort);
      if (a.stall && turn == a.stall && blockIdx.x < CL) ok = false;
      if (ok && lane == 0) {
        items[turn & 1] = it;
        bar_arrive(item_full + (turn & 1));
      }
      ++turn;
      return ok;
    };
    each_item<CL>(a, seq_row, seq_rows, seq_blocks, give);
    if (ok) give(PromptItem{-1, 0, 0, 0});
  }
  tc_before();
  __syncwarp();
  __syncthreads();
  if (warp == 11 && *abort) {
    // A wait ran out: what this CTA has to write is not valid, or not there at all.
    kv_flag(a.error, MOE_DEVERR_TMA);
    int s, n;
    const int mine = prompt_blocks(a, lane, &s, &n);
    each_item<CL>(a, s, n, mine, [&](const PromptItem& it) {
      constexpr int COLS = D / CL;
      const int first = it.block * 2 * kPM, rows = min(2 * kPM, it.n - first);
      T* dst = static_cast<T*>(a.out) + (int64_t)(it.row0 + first) * a.o_tok + it.head * a.o_head + rank * COLS;
      for (int i = lane; i < rows * COLS; i += 32) dst[i / COLS * a.o_tok + i % COLS] = from_float<T>(__int_as_float(0x7fc00000));
      return true;
    });
  }
  if (CL > 1) cluster_sync();  // neither leaves while the other may still write to it
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (!kv_ok(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q)) ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Rows [tokens][heads][D] -> boxes of 128 tokens x 64 channels of one head, 128-byte swizzle.
// (The stride of a single head or row means nothing; the map wants one all the same.)
bool rows_map(CUtensorMap* m, const moe_rows* r, int tokens, int heads, int dim, int dtype) {
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? r->head_stride : dim) * 2, (cuuint64_t)(tokens > 1 ? r->token_stride : dim) * 2};
  const cuuint32_t box[3] = {64, 1, 128}, es[3] = {1, 1, 1};
  return encode_tiled()(m, dtype == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                        r->data_dev, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int CL>
cudaError_t prompt_go(const PromptArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int device,
                      int clusters, cudaStream_t st) {
  static std::atomic<bool> ready[kKvMaxDevices];
  if (!ready[device]) {
    const cudaError_t e = cudaFuncSetAttribute(attend_prompt_kernel<T, D, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               PromptSmem<D>::kBytes);
    if (e != cudaSuccess) return e;
    ready[device] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(clusters * CL);
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = PromptSmem<D>::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = CL;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = CL > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attend_prompt_kernel<T, D, CL>, a, mq, mk, mv);
}

template <typename T>
cudaError_t prompt_pick(const PromptArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int dim, int device,
                        cudaStream_t st) {
  const int n_sm = kv_sm_count(device);
  if (!n_sm) return cudaErrorInvalidDevice;
  const int64_t items = (int64_t)a.n_blocks * a.n_heads;  // at most
  // Pairs of CTAs where the longest item decides and is long enough to be worth the exchange at
  // its end.  One prompt of n tokens, us without pairs / with (D = 128): all items on SMs of their
  // own either way, n = 600 13.7 / 14.2, 1024 20.3 / 17.8, 2048 33.4 / 24.5, 8192 111 / 70; two
  // items a pair, n = 2048 34.0 / 34.7, 4096 61.7 / 46.9; more items than SMs, 16384 805 / 927.
  const int64_t each = a.n_tokens / a.n_seqs;
  const bool pairs = (2 * items <= n_sm && each >= 1024) || (items <= n_sm && each >= 4096);
  if (pairs) {
    const int n = (int)(items < n_sm / 2 ? items : n_sm / 2);
    return dim == 64 ? prompt_go<T, 64, 2>(a, mq, mk, mv, device, n, st) : prompt_go<T, 128, 2>(a, mq, mk, mv, device, n, st);
  }
  const int n = (int)(items < n_sm ? items : n_sm);
  return dim == 64 ? prompt_go<T, 64, 1>(a, mq, mk, mv, device, n, st) : prompt_go<T, 128, 1>(a, mq, mk, mv, device, n, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

static std::atomic<int> g_stalls{0};  // calls that are still to run into their waits' limits
int moe::kv_stall() {
  int n = g_stalls.load(std::memory_order_relaxed);
  while (n > 0 && !g_stalls.compare_exchange_weak(n, n - 1)) {
  }
  return n > 0;
}
extern "C" int moe_debug_stall_attention(int32_t n) {
  if (n < 0) return MOE_ERR_INVALID;
  g_stalls = n;
  return MOE_OK;
}

extern "C" int moe_attend_prompt(int32_t device, const moe_rows* q, const moe_rows* k, const moe_rows* v, const moe_rows* out,
                                 const int32_t* cu_dev, int32_t n_seqs, int32_t n_tokens, int32_t n_q_heads,
                                 int32_t n_kv_heads, int32_t head_dim, int32_t dtype, float scale, int32_t* error_dev,
                                 void* stream) {
  if (!q || !k || !v || !out || !cu_dev || !q->data_dev || !k->data_dev || !v->data_dev || !out->data_dev) return MOE_ERR_INVALID;
  if (device < 0 || device >= kKvMaxDevices || n_seqs < 0 || n_tokens < 0 || n_q_heads < 1 || n_kv_heads < 1 ||
      n_q_heads % n_kv_heads)
    return MOE_ERR_INVALID;
  if ((dtype != MOE_BF16 && dtype != MOE_F16) || !(scale > 0.0f) || scale - scale != 0.0f) return MOE_ERR_INVALID;
  if (!kv_dim_ok(head_dim) || n_seqs > kKvMaxSeqs || n_tokens > kKvMaxPos) return MOE_ERR_UNSUPPORTED;
  // The TMA's rules.  It has no documented meaning for a stride of 0.
  auto stride_ok = [](int64_t s, int n) { return n < 2 || (s > 0 && s < (1ll << 38) && s % 8 == 0); };
  for (const moe_rows* r : {q, k, v})
    if (!kv_align_ok(r->data_dev, 16) || !stride_ok(r->token_stride, n_tokens) ||
        !stride_ok(r->head_stride, r == q ? n_q_heads : n_kv_heads))
      return MOE_ERR_UNSUPPORTED;
  if (!kv_align_ok(out->data_dev, 2) || !kv_apart(out->token_stride, n_tokens, out->head_stride, n_q_heads)) return MOE_ERR_INVALID;
  if (n_tokens == 0 || n_seqs == 0) return MOE_OK;
  const int64_t blocks = n_tokens / (2 * kPM) + (n_seqs < n_tokens ? n_seqs : n_tokens);
  if (blocks * n_q_heads > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  DeviceScope dev(device);
  if (!dev.ok) return MOE_ERR_CUDA;
  if (!encode_tiled()) return MOE_ERR_UNSUPPORTED;
  CUtensorMap mq, mk, mv;
  if (!rows_map(&mq, q, n_tokens, n_q_heads, head_dim, dtype) || !rows_map(&mk, k, n_tokens, n_kv_heads, head_dim, dtype) ||
      !rows_map(&mv, v, n_tokens, n_kv_heads, head_dim, dtype))
    return MOE_ERR_UNSUPPORTED;
  PromptArgs a{};
  a.cu = cu_dev;
  a.n_seqs = n_seqs;
  a.n_tokens = n_tokens;
  a.n_heads = n_q_heads;
  a.group = n_q_heads / n_kv_heads;
  a.n_blocks = (int)blocks;
  a.scale2 = scale * 1.4426950408889634f;
  a.out = out->data_dev;
  a.o_tok = out->token_stride;
  a.o_head = out->head_stride;
  a.vec = kv_align_ok(out->data_dev, 16) && out->token_stride % 8 == 0 && out->head_stride % 8 == 0;
  a.error = error_dev;
  a.stall = kv_stall();
  a.q = q->data_dev, a.q_tok = q->token_stride, a.q_head = q->head_stride;
  a.k = k->data_dev, a.k_tok = k->token_stride, a.k_head = k->head_stride;
  a.v = v->data_dev, a.v_tok = v->token_stride, a.v_head = v->head_stride;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MOE_BF16 ? prompt_pick<__nv_bfloat16>(a, mq, mk, mv, head_dim, device, st)
                                          : prompt_pick<__half>(a, mq, mk, mv, head_dim, device, st);
  return kv_status(e);
}
