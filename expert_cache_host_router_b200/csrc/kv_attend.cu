// kv_attend.cu -- attention of one new token per sequence over a 4-bit key/value cache.
//
//   z_j = scale q . k_j,  p = softmax(z) over the sequence's len positions,  o = sum_j p_j v_j
// for every query head; the G query heads of a KV head read the same rows.  Each cached
// byte is used for 2 channels x G heads x 2 FLOP, once: the bound is the cache's bytes
// (18 D per 16 tokens and head) over the HBM rate.
//
// Work split: the tiles (16 tokens) of all sequences and KV heads form one line, cut into
// equal runs, one per CTA, whatever the lengths are: ragged batches and single long
// sequences keep every SM busy alike.  Where a run begins or ends inside a sequence's head
// the CTA writes a partial result (o, running maximum m, sum l), at most two per CTA; the
// second kernel joins those.  Inside a CTA every warp takes every W-th pair of tiles of
// the run with statistics of its own and joins the others at the end of a segment.
//
// Products run on mma.sync m16n8k16 with fp32 accumulation: M is 16 keys (then 16
// channels), N the 8 heads of a group, so 8 query heads cost one instruction.  tcgen05
// would pad N and M to tiles (128 rows) that a decode step does not have, and both
// operands would have to be dequantised into shared memory first.  What limits the kernel
// besides the bytes is the integer pipe (2 warp instructions a cycle), so the nibbles become
// fp16 by few operations: (w & mask) | magic is base + q exactly.  For the keys (base 64) the
// block scale d multiplies the fp32 partial sum, and one more product, of a row's d with
// -72 sum_c q_c of the blocks (split into three fp16 parts), takes the base out.  Values use base 1024 or 64, whichever the
// nibble's place gives without a shift, and become (q - 8) d rounded to fp16 (half a step,
// 2^-11); weights p are fp16 too.  Queries are scaled by a power of two per head to the fp16
// range (exact but for channels 2^-24 below the head's largest); cached values are within
// that range by construction.
#include <cfloat>

#include "kv_internal.h"

namespace moe {

constexpr int kAW = 8;           // warps of a CTA
constexpr int kGT = 2;           // tiles of a group: what a warp takes at a time

struct AttendArgs {
  const void* q;
  int64_t q_seq, q_head;
  void* out;
  int64_t o_seq, o_head;
  const int32_t* lens;
  int max_len, group, n_chunks;  // query heads per KV head; chunks of 8 NT heads that they are split into
  float scale2;                  // scale * log2(e)
  int min_run;                   // tiles a CTA takes at least
  int score_ctas;                // CTAs of a sequence's and KV head's scores
  int vec;                       // rows of q can be read 8 bytes at a time
  uint32_t stall;                // for tests: bytes that every copy is expected to have more than it has
  float* part;                   // [2 CTAs][8 NT][D] partial outputs, unnormalised
  float* ml;                     // [2 CTAs][8 NT][2] their (m, l)
  float* ml_whole;               // [items][8 NT][2] (m, l) of the items that one CTA has whole (scored calls)
  int2* pieces;                  // [items] first CTA and number of CTAs of the items that have positions
  float* z;                      // [items][max_len][8 NT] scaled products in log2 units (scored calls)
  float* score;                  // or null
  int64_t s_seq, s_head;
};

// The line: sequence b starts at pre[b] * items_per_seq and every one of its items (KV head
// and chunk) takes pre[b + 1] - pre[b] places: kItemCost for what an item costs whatever its
// length (queries, joining the warps), then one for each tile.  A CTA takes the tiles that lie
// in its run.  Without the cost, runs over short sequences take longest: 64 sequences of 129
// to 8192 tokens took 64 us with none, 52 with 16, 47 with 40 or 48, 50 with 64; 48
// sequences of 5 to 300 took 11.3 us with 16, 12.7 with 40.  Lengths that cannot be are taken as 0.
constexpr int kItemCost = 40;
__device__ __forceinline__ int attend_len(const KvView& c, const AttendArgs& a, int b) {
  const int len = a.lens[b];
  return len < 0 || len > a.max_len || len > c.width * c.tiles_per_page * kTileTok ? -1 : len;
}

// pre[0..n_seqs], by all threads of the CTA; ends with a barrier.
__device__ __forceinline__ void attend_prefix(const KvView& c, const AttendArgs& a, int* pre, int* tmp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  int carry = 0;
  if (tid == 0) pre[0] = 0;
  for (int base = 0; base < c.n_seqs; base += nt) {
    const int b = base + tid;
    int v = b < c.n_seqs ? (max(attend_len(c, a, b), 0) + kTileTok - 1) / kTileTok : 0;
    if (v) v += kItemCost;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += y;
    }
    if (lane == 31) tmp[warp] = v;
    __syncthreads();
    int sum = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) sum += tmp[w];
      all += tmp[w];
    }
    if (b < c.n_seqs) pre[b + 1] = carry + sum + v;
    carry += all;
    __syncthreads();
  }
  __syncthreads();
}

__device__ __forceinline__ int attend_run(const AttendArgs& a, int total, int n_cta) {
  return max(a.min_run, (total + n_cta - 1) / n_cta);
}

__device__ __forceinline__ void kv_mbar_init(uint64_t* bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(kv_smem(bar)) : "memory");
}
__device__ __forceinline__ bool kv_mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred q;\n\tmbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(ok)
      : "r"(kv_smem(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// False when the copy has not landed within so many ns.
constexpr uint64_t kLimitNs = 2000000000ull;
__device__ __noinline__ bool kv_mbar_spin(uint64_t* bar, uint32_t parity, uint64_t limit) {
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  while (!kv_mbar_try(bar, parity)) {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > limit) return false;
  }
  return true;
}

// One bulk copy into shared memory.
__device__ __forceinline__ void kv_bulk(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(kv_smem(bar))
               : "memory");
}
__device__ __forceinline__ void kv_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(kv_smem(bar)), "r"(bytes) : "memory");
}

template <uint32_t MASK, uint32_t BITS>
__device__ __forceinline__ uint32_t masked(uint32_t w) {  // (w & MASK) | BITS in one instruction
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "n"(BITS));
  return r;
}
constexpr uint32_t kAt0 = 0x000F000Fu, k1024 = 0x64006400u;  // nibble at mantissa bits 0..3: 1024 + q
constexpr uint32_t kAt4 = 0x00F000F0u, k64 = 0x54005400u;    // at bits 4..7: 64 + q

// d += a b and d = a b, 16 x 8 x 16.
__device__ __forceinline__ void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_set(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A run of tiles of one item inside a CTA's part of the line.
struct Segment {
  int b, item, nt, s0, s1;  // sequence, KV head and chunk, tiles of the sequence, tiles [s0, s1) of it
};
struct Line {  // walks the segments of [lin, end)
  int lin, end, b;
  __device__ __forceinline__ bool next(const int* pre, int items, int n_seqs, Segment& s) {
    while (lin < end) {
      while (pre[b + 1] * items <= lin) ++b;  // lin < end <= pre[n_seqs] * items: ends
      const int places = pre[b + 1] - pre[b], off = lin - pre[b] * items;
      s.b = b;
      s.nt = places - kItemCost;
      s.item = off / places;
      const int at = off - s.item * places, to = min(places, at + end - lin);
      lin += to - at;
      s.s0 = max(at - kItemCost, 0);
      s.s1 = to - kItemCost;
      if (s.s1 > s.s0) return true;
    }
    return false;
  }
};

// The groups of one warp, in order: of every segment its share of consecutive groups.
struct Walk {
  Line line;
  Segment s;
  int g, end;  // groups [g, end) of the segment are still to come
  bool more;
  __device__ __forceinline__ void segment(const int* pre, int items, int n_seqs, int warp) {
    more = line.next(pre, items, n_seqs, s);
    const int n = more ? (s.s1 - s.s0 + kGT - 1) / kGT : 0;
    g = n * warp / kAW;
    end = n * (warp + 1) / kAW;
  }
};

template <int D, int NT>
struct AttendSmem {
  static constexpr int kStages = NT == 1 ? 2 : 4;
  static constexpr int kTile = 18 * D, kStage = kGT * kTile;
  static constexpr int kFrag = (D / 4 + 4) * NT;  // floats of a thread's state: o, then m and l of its columns
  static constexpr int kRing = kAW * kStages * kStage;
  // The four-stage ring leaves no room beside it: that kernel joins its warps in two halves.
  static constexpr int kMergeWarps = NT == 1 ? kAW : kAW / 2;
  static constexpr int kBars = kRing + kMergeWarps * 32 * kFrag * 4;
  static constexpr int kWalk = kBars + kAW * kStages * 8;  // two walks a warp: kept here between uses, not in registers
  // prepared queries of a segment: fragments [NT][NB][32 lanes] of 16 bytes, the base's parts
  // [NT][32 lanes] of 8 bytes, scales [8 NT]
  static constexpr int kQuery = (kWalk + kAW * 2 * (int)sizeof(Walk) + 15) / 16 * 16;
  static constexpr int kParts = kQuery + NT * (D / 32) * 512, kScale = kParts + NT * 256;
  static constexpr int kTmp = kScale + 32 * NT;
  static constexpr int kPre = kTmp + 64;
  static int bytes(int n_seqs) { return kPre + (n_seqs + 1) * 4; }
};

template <typename T, int D, int NT, bool SCORED>
__global__ void __launch_bounds__(kAW * 32, NT == 1 ? 2 : 1) kv_attend_kernel(const KvView c, const AttendArgs a) {
  using S = AttendSmem<D, NT>;
  constexpr int NB = D / 32, ST = S::kStages, COLS = 8 * NT;
  extern __shared__ __align__(128) uint8_t sm[];
  int* pre = reinterpret_cast<int*>(sm + S::kPre);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = sm + warp * ST * S::kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBars) + warp * ST;
  float* merge = reinterpret_cast<float*>(sm + S::kRing);
  asm volatile("griddepcontrol.launch_dependents;");
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < ST; ++s) kv_mbar_init(bars + s);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  attend_prefix(c, a, pre, reinterpret_cast<int*>(sm + S::kTmp));
  const int items = c.heads * a.n_chunks;
  const int total = pre[c.n_seqs] * items;
  const int run = attend_run(a, total, gridDim.x);
  const int lin0 = blockIdx.x * run;
  if ((int64_t)blockIdx.x * run >= total) return;
  Walk* walks = reinterpret_cast<Walk*>(sm + S::kWalk) + 2 * warp;  // [0] what is computed, [1] what is looked up
  {
    Walk w{};
    w.line = Line{lin0, min(total, lin0 + run), 0};
    int lo = 0, hi = c.n_seqs - 1;  // first sequence of the run
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * items <= lin0) lo = mid; else hi = mid - 1;
    }
    w.line.b = lo;
    w.segment(pre, items, c.n_seqs, warp);
    if (lane < 2) walks[lane] = w;
    __syncwarp();
  }

  // Look-ahead: every lane holds the two tiles of one of the next 32 groups of this warp (across segment
  // borders), looked up by all lanes at once; a lane issues the copies of its group when
  // its turn comes.
  int tile_a = -1, tile_b = -1;  // numbers in the pool; -1: no such page, -2: no second tile
  int turn = 0, held = 0;
  auto look_up = [&]() {
    Walk w = walks[1];
    turn = held = 0;
    while (held < 32 && w.more) {
      const int n = min(32 - held, w.end - w.g);
      const int k = lane - held;
      if (k >= 0 && k < n) {
        const int h = w.s.item / a.n_chunks, tile = w.s.s0 + (w.g + k) * kGT;
        tile_a = kv_tile_number(c, w.s.b, h, tile);
        tile_b = tile + 1 < w.s.s1 ? kv_tile_number(c, w.s.b, h, tile + 1) : -2;
      }
      held += n;
      w.g += n;
      if (w.g >= w.end) w.segment(pre, items, c.n_seqs, warp);
    }
    __syncwarp();
    if (lane == 0) walks[1] = w;
    __syncwarp();
  };
  auto issue = [&](int stage) {
    if (turn == held) look_up();
    if (lane == turn && turn < held) {
      uint8_t* dst = ring + stage * S::kStage;
      const uint8_t* src = c.pool + (int64_t)tile_a * S::kTile;
      if (tile_a >= 0 && tile_b == tile_a + 1) {
        kv_expect(bars + stage, 2 * S::kTile + a.stall);
        kv_bulk(kv_smem(dst), src, 2 * S::kTile, bars + stage);
      } else {
        // a missing page's keys get NaN scales, which makes the row's output NaN
        if (tile_a < 0 || tile_b == -1)
          for (int i = 0; i < D / 2; ++i) reinterpret_cast<uint16_t*>(dst + 16 * D + (tile_a < 0 ? 0 : S::kTile))[i] = 0x7E00;
        kv_expect(bars + stage, (tile_a >= 0 ? S::kTile : 0) + (tile_b >= 0 ? S::kTile : 0) + a.stall);
        if (tile_a >= 0) kv_bulk(kv_smem(dst), src, S::kTile, bars + stage);
        if (tile_b >= 0) kv_bulk(kv_smem(dst + S::kTile), c.pool + (int64_t)tile_b * S::kTile, S::kTile, bars + stage);
      }
    }
    turn = min(turn + 1, held);
  };
  int stage = 0;
  uint32_t phase = 0;
  bool alive = true, first = true;
  while (walks[0].more) {
    const Segment sg = walks[0].s;
    const int h = sg.item / a.n_chunks, chunk = sg.item - h * a.n_chunks;
    const int n_heads = min(COLS, a.group - chunk * COLS);  // query heads of this item
    const int h0 = h * a.group + chunk * COLS;
    // Queries, prepared once for the CTA: warp w takes heads w, w + 8 of the item, a lane
    // D / 32 consecutive channels (8 or 16 lanes to a block).  As fragments column n = g of
    // each 8 heads; within a block the channels of the two 16-deep steps are 4t + {0, 2, 1, 3}
    // and 16 more, the order that the nibbles come in.
    constexpr int C = D / 32;
    __align__(8) uint16_t raw[NT][C];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool has = n * 8 + warp < n_heads;
      const uint16_t* qp = static_cast<const uint16_t*>(a.q) + sg.b * a.q_seq + (int64_t)(h0 + n * 8 + (has ? warp : 0)) * a.q_head + C * lane;
      if (a.vec) {
        if constexpr (C == 4) *reinterpret_cast<uint2*>(raw[n]) = *reinterpret_cast<const uint2*>(qp);
        else *reinterpret_cast<uint32_t*>(raw[n]) = *reinterpret_cast<const uint32_t*>(qp);
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i) raw[n][i] = qp[i];
      }
    }
    if (first) {  // the first pages are looked up and asked for while the queries come
#pragma unroll 1
      for (int s = 0; s < ST; ++s) issue(s);
      first = false;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool has = n * 8 + warp < n_heads;
      float v[C], top = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        v[i] = has ? to_float(reinterpret_cast<const T*>(raw[n])[i]) : 0.0f;
        top = fmaxf(top, fabsf(v[i]));
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      // 2^-x and 2^x, x the exponent of the largest channel (0 for none, infinity or NaN)
      int x = (int)(__float_as_uint(top) >> 23) - 127;
      if (top == 0.0f || x > 127) x = 0;
      x = max(min(x, 126), -126);  // 2^-x in the fp32 range; subnormal bf16 channels still get 8 bits
      const float down = __uint_as_float((uint32_t)(127 - x) << 23);
      float sum = 0.0f;
      uint16_t* frag = reinterpret_cast<uint16_t*>(sm + S::kQuery);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const __half r = __float2half_rn(v[i] * down);
        sum += __half2float(r);
        // channel c of a block: lane t = (c mod 16) / 4, its word 2 [c >= 16] + [c odd], half [c mod 4 >= 2]
        const int ch = C * lane + i, cc = ch & 31;
        frag[((n * NB + (ch >> 5)) * 32 + warp * 4 + ((cc & 15) >> 2)) * 8 + ((cc >> 4) * 2 + (cc & 1)) * 2 + ((cc >> 1) & 1)] =
            __half_as_ushort(r);
      }
#pragma unroll
      for (int off = 1; off < 32 / C; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      // -72 times the sum of a block's channels in three parts.  Lane t of a column's four has
      // rows 2t, 2t + 1 and 2t + 8, 2t + 9 of that product: blocks 2 (t mod 2), + 1, as its scales lie; the first part in
      // lanes 0 and 1, the second in 2 and 3, the third in the later rows of 0 and 1.
      if (lane % (32 / C) == 0) {
        const int nb = lane / (32 / C);
        const float base = sum * -72.0f;
        const __half p1 = __float2half_rn(base), p2 = __float2half_rn(base - __half2float(p1));
        const __half p3 = __float2half_rn(base - __half2float(p1) - __half2float(p2));
        __half* pt = reinterpret_cast<__half*>(sm + S::kParts) + (n * 32 + warp * 4) * 4;  // [t][2 words][2 blocks]
        const int t0 = nb >> 1, i = nb & 1;
        pt[t0 * 4 + i] = p1;
        pt[(t0 + 2) * 4 + i] = p2;
        pt[t0 * 4 + 2 + i] = p3;
        pt[(t0 + 2) * 4 + 2 + i] = __half(0);
        if (NB == 2) {  // two blocks: the odd lanes have none
          pt[4 + i] = pt[6 + i] = pt[12 + i] = pt[14 + i] = __half(0);
        }
      }
      // Kept between the smallest normal number and the largest: m = -inf, or products that are 0, times the
      // factor must not become NaN, and at these ends no weight depends on the factor's exact value.
      if (lane == 0)
        reinterpret_cast<float*>(sm + S::kScale)[n * 8 + warp] = fminf(fmaxf(a.scale2 * exp2f((float)x), FLT_MIN), FLT_MAX);
    }
    __syncthreads();
    uint32_t qf[NT][NB][4], qb[NT][2];
    float sc[NT][2];  // scale of columns 2t and 2t + 1, with the power of two that the queries were divided by
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        *reinterpret_cast<uint4*>(qf[n][nb]) = reinterpret_cast<const uint4*>(sm + S::kQuery)[(n * NB + nb) * 32 + lane];
      *reinterpret_cast<uint2*>(qb[n]) = reinterpret_cast<const uint2*>(sm + S::kParts)[n * 32 + lane];
      *reinterpret_cast<float2*>(sc[n]) = reinterpret_cast<const float2*>(sm + S::kScale)[n * 4 + t];
    }
    float o[NT][NB][2][4];
    float m[NT][2], l[NT][2];  // m in units of the unscaled products
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < NB * 8; ++i) (&o[n][0][0][0])[i] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    int n_groups = walks[0].end - walks[0].g;
    // keys of the segment from this warp's first group on
    const int key0 = (sg.s0 + walks[0].g * kGT) * kTileTok;
    int left = min(attend_len(c, a, sg.b), sg.s1 * kTileTok) - key0;
    float* zrow = SCORED ? a.z + ((int64_t)(sg.b * items + sg.item) * a.max_len + key0) * COLS + 2 * t : nullptr;
    for (; n_groups > 0; --n_groups, left -= kGT * kTileTok) {
      if (alive && !kv_mbar_try(bars + stage, phase) && !kv_mbar_spin(bars + stage, phase, kLimitNs)) {
        alive = false;  // all that this warp has left becomes NaN; it asks for nothing more
        kv_flag(c.error, MOE_DEVERR_TMA);
        // and lets what it asked for arrive, for up to 10 ms each, before its shared memory may be another CTA's
        for (int s = 0; s < ST; ++s) kv_mbar_spin(bars + s, s >= stage ? phase : phase ^ 1, 10000000ull);
      }
      const uint8_t* base = ring + stage * S::kStage;
      const bool tail = left < kGT * kTileTok;
      float z[NT][kGT][4];
#pragma unroll
      for (int i = 0; i < kGT; ++i) {
        const uint8_t* tl = base + i * S::kTile;
        // keys: lane (g, t) has word t of every block of rows g and g + 8
        uint32_t kw[2][NB];
        __half2 ks[2][NB / 2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (NB == 4) {
            *reinterpret_cast<uint4*>(kw[r]) = *reinterpret_cast<const uint4*>(tl + (g + 8 * r) * 64 + t * 16);
            *reinterpret_cast<uint2*>(ks[r]) = *reinterpret_cast<const uint2*>(tl + 16 * D + (g + 8 * r) * 8);
          } else {
            *reinterpret_cast<uint2*>(kw[r]) = *reinterpret_cast<const uint2*>(tl + (g + 8 * r) * 32 + t * 8);
            *reinterpret_cast<uint32_t*>(ks[r]) = *reinterpret_cast<const uint32_t*>(tl + 16 * D + (g + 8 * r) * 4);
          }
        }
        {
          uint32_t s2[2];  // scales of the lane's two blocks
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const __half2 lo = ks[r][0], hi = ks[r][NB / 2 - 1];
            s2[r] = *reinterpret_cast<const uint32_t*>(t & 1 ? &hi : &lo);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_set(z[n][i], s2[0], s2[1], s2[0], s2[1], qb[n][0], qb[n][1]);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t w0 = kw[0][nb], w1 = kw[1][nb];
          const uint32_t a00 = masked<kAt4, k64>(w0 * 16), a01 = masked<kAt4, k64>(w0), a02 = masked<kAt4, k64>(w0 >> 4),
                         a03 = masked<kAt4, k64>(w0 >> 8);
          const uint32_t a10 = masked<kAt4, k64>(w1 * 16), a11 = masked<kAt4, k64>(w1), a12 = masked<kAt4, k64>(w1 >> 4),
                         a13 = masked<kAt4, k64>(w1 >> 8);
          const float d0 = nb & 1 ? __high2float(ks[0][nb / 2]) : __low2float(ks[0][nb / 2]);
          const float d1 = nb & 1 ? __high2float(ks[1][nb / 2]) : __low2float(ks[1][nb / 2]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float s[4];
            mma_set(s, a00, a10, a02, a12, qf[n][nb][0], qf[n][nb][1]);
            mma_add(s, a01, a11, a03, a13, qf[n][nb][2], qf[n][nb][3]);
            z[n][i][0] = fmaf(s[0], d0, z[n][i][0]);
            z[n][i][1] = fmaf(s[1], d0, z[n][i][1]);
            z[n][i][2] = fmaf(s[2], d1, z[n][i][2]);
            z[n][i][3] = fmaf(s[3], d1, z[n][i][3]);
          }
        }
      }
      if (tail || !alive) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < kGT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (!alive) z[n][i][e] = __int_as_float(0x7fc00000);
              if (i * kTileTok + g + 8 * (e >> 1) >= left) z[n][i][e] = -INFINITY;
            }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (SCORED) {
#pragma unroll
          for (int i = 0; i < kGT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int key = i * kTileTok + g + 8 * r;
              if (key < left)
                *reinterpret_cast<float2*>(zrow + key * COLS + n * 8) =
                    make_float2(z[n][i][2 * r] * sc[n][0], z[n][i][2 * r + 1] * sc[n][1]);
            }
        }
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          mx[e] = fmaxf(fmaxf(z[n][0][e], z[n][0][2 + e]), fmaxf(z[n][1][e], z[n][1][2 + e]));
        // The running maximum moves only when it is exceeded by more than 8 in the exponent (a
        // factor of 256): weights stay below 256, far inside fp16, and most groups rescale
        // nothing, nor do they look for the group's maximum beyond each lane's own products.
        // m = -inf counts as exceeded unless the products are -inf (or NaN) too.
        const bool move = (mx[0] - m[n][0]) * sc[n][0] > 8.0f || (mx[1] - m[n][1]) * sc[n][1] > 8.0f;
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
          }
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m[n][e], mx[e]);
            al[e] = m[n][e] == mn ? 1.0f : exp2_fast((m[n][e] - mn) * sc[n][e]);
            m[n][e] = mn;
            l[n][e] *= al[e];
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[n][nb][x][e] *= al[e & 1];
        }
        const float off0 = -m[n][0] * sc[n][0], off1 = -m[n][1] * sc[n][1];
#pragma unroll
        for (int i = 0; i < kGT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = exp2_fast(fmaf(z[n][i][e], sc[n][e & 1], e & 1 ? off1 : off0));
            z[n][i][e] = p;
            l[n][e & 1] += p;
          }
      }
#pragma unroll
      for (int i = 0; i < kGT; ++i) {
        const uint8_t* tl = base + i * S::kTile + 8 * D;
        // weights: 8 keys x 8 heads at a time, turned so that a lane has two keys of one head
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          pf[n][0] = transpose8x8(half2_of(z[n][i][0], z[n][i][1]));
          pf[n][1] = transpose8x8(half2_of(z[n][i][2], z[n][i][3]));
        }
        uint32_t vw[2][NB], vs[2][NB];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (NB == 4) {
            *reinterpret_cast<uint4*>(vw[r]) = *reinterpret_cast<const uint4*>(tl + (t + 4 * r) * 128 + g * 16);
            *reinterpret_cast<uint4*>(vs[r]) = *reinterpret_cast<const uint4*>(tl + 9 * D + (t + 4 * r) * 16);
          } else {
            *reinterpret_cast<uint2*>(vw[r]) = *reinterpret_cast<const uint2*>(tl + (t + 4 * r) * 64 + g * 8);
            *reinterpret_cast<uint2*>(vs[r]) = *reinterpret_cast<const uint2*>(tl + 9 * D + (t + 4 * r) * 8);
          }
        }
        if (tail) {  // scales of rows behind the end may be anything, NaN too
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int key = i * kTileTok + 2 * t + 8 * r;
            const uint32_t keep = (key < left ? 0xFFFFu : 0u) | (key + 1 < left ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) vs[r][nb] &= keep;
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t va[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t w = vw[r][nb], w8 = w >> 8;
            va[r][0] = hmul2(hsub2(masked<kAt0, k1024>(w), 0x64086408u), vs[r][nb]);   // - 1032
            va[r][1] = hmul2(hsub2(masked<kAt4, k64>(w), 0x54805480u), vs[r][nb]);     // - 72
            va[r][2] = hmul2(hsub2(masked<kAt0, k1024>(w8), 0x64086408u), vs[r][nb]);
            va[r][3] = hmul2(hsub2(masked<kAt4, k64>(w8), 0x54805480u), vs[r][nb]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_add(o[n][nb][0], va[0][0], va[0][1], va[1][0], va[1][1], pf[n][0], pf[n][1]);
            mma_add(o[n][nb][1], va[0][2], va[0][3], va[1][2], va[1][3], pf[n][0], pf[n][1]);
          }
        }
      }
      // Every lane has read the stage; the fence orders those reads before the copy engine's write.
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      alive = __all_sync(0xffffffffu, alive);
      if (alive) issue(stage);
      if (SCORED) zrow += kGT * kTileTok * COLS;
      if (++stage == ST) {
        stage = 0;
        phase ^= 1;
      }
    }

    // Join the warps: each leaves its fragments in shared memory, then thread (warp w, lane)
    // sums fragment entries e4 = w mod 4 of blocks w / 4, w / 4 + 2, .. for its lane.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
        m[n][e] = m[n][e] * sc[n][e];  // in log2 units from here on
      }
    constexpr int MW = S::kMergeWarps;
    float* mine = merge + (warp % MW) * 32 * S::kFrag + lane;
    if constexpr (MW < kAW) {  // the upper half first, taken over by the lower one
      if (warp >= MW) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < NB * 8; ++i) mine[(n * NB * 8 + i) * 32] = (&o[n][0][0][0])[i];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mine[(NT * NB * 8 + 4 * n + e) * 32] = m[n][e];
            mine[(NT * NB * 8 + 4 * n + 2 + e) * 32] = l[n][e];
          }
        }
      }
      __syncthreads();
      if (warp < MW) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float x[2], y[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mo = mine[(NT * NB * 8 + 4 * n + e) * 32], lo = mine[(NT * NB * 8 + 4 * n + 2 + e) * 32];
            const float mn = fmaxf(m[n][e], mo);
            x[e] = m[n][e] == mn ? 1.0f : exp2_fast(m[n][e] - mn);
            y[e] = mo == mn ? 1.0f : exp2_fast(mo - mn);
            m[n][e] = mn;
            l[n][e] = l[n][e] * x[e] + lo * y[e];
          }
#pragma unroll
          for (int i = 0; i < NB * 8; ++i) {
            float* ov = &o[n][0][0][0];
            ov[i] = ov[i] * x[i & 1] + mine[(n * NB * 8 + i) * 32] * y[i & 1];
          }
        }
      }
    }
    if (warp < MW) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < NB * 8; ++i) mine[(n * NB * 8 + i) * 32] = (&o[n][0][0][0])[i];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mine[(NT * NB * 8 + 4 * n + e) * 32] = m[n][e];
          mine[(NT * NB * 8 + 4 * n + 2 + e) * 32] = l[n][e];
        }
      }
    }
    __syncthreads();
    const bool whole = walks[0].s.s0 == 0 && walks[0].s.s1 == walks[0].s.nt;
    if (tid == 0 && sg.s0 == 0) {
      const int end = pre[sg.b] * items + (sg.item + 1) * (sg.nt + kItemCost) - 1;
      a.pieces[sg.b * items + sg.item] = make_int2(blockIdx.x, end / run - (int)blockIdx.x + 1);
    }
    const int slot = 2 * blockIdx.x + (sg.s0 == 0 ? 1 : 0);
    const int e4 = warp & 3, e = e4 & 1;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = n * 8 + 2 * t + e;
      const float* all = merge + lane;
      float f[MW], M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < MW; ++w) {
        f[w] = all[w * 32 * S::kFrag + (NT * NB * 8 + 4 * n + e) * 32];
        M = fmaxf(M, f[w]);
      }
#pragma unroll
      for (int w = 0; w < MW; ++w) {
        f[w] = f[w] == M ? 1.0f : exp2_fast(f[w] - M);
        L = fmaf(all[w * 32 * S::kFrag + (NT * NB * 8 + 4 * n + 2 + e) * 32], f[w], L);
      }
      if (g == 0 && (warp == 0 || warp == 1)) {  // once for each column
        if (!whole) reinterpret_cast<float2*>(a.ml)[(int64_t)slot * COLS + col] = make_float2(M, L);
        else if (SCORED) reinterpret_cast<float2*>(a.ml_whole)[(int64_t)(sg.b * items + sg.item) * COLS + col] = make_float2(M, L);
      }
      const float inv = whole ? 1.0f / L : 1.0f;
#pragma unroll
      for (int nb = warp >> 2; nb < NB; nb += 2) {
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int w = 0; w < MW; ++w) v[x] = fmaf(all[w * 32 * S::kFrag + (n * NB * 8 + nb * 8 + x * 4 + e4) * 32], f[w], v[x]);
        const int ch = nb * 32 + 2 * g + 16 * (e4 >> 1);
        if (!whole) {
          *reinterpret_cast<float2*>(a.part + ((int64_t)slot * COLS + col) * D + ch) = make_float2(v[0], v[1]);
        } else if (col < n_heads) {
          T* op = static_cast<T*>(a.out) + sg.b * a.o_seq + (int64_t)(h0 + col) * a.o_head + ch;
          op[0] = from_float<T>(v[0] * inv);
          op[1] = from_float<T>(v[1] * inv);
        }
      }
    }
    __syncthreads();
    Walk w = walks[0];
    w.segment(pre, items, c.n_seqs, warp);
    __syncwarp();
    if (lane == 0) walks[0] = w;
    __syncwarp();
  }
}

// ------------------------------------------------------------------ second kernel

// The first CTAs join the partial results of items (or write the rows of a sequence without
// positions: zeros, or NaN when its length cannot be).  With few items (each in many pieces)
// a CTA takes one head: the pieces' weights are formed once, one thread each, then every thread
// sums four channels, the pieces in interleaved lines, the first eight of a line read before
// the weights are known.
// With many items (most of them whole or in two pieces) a CTA takes all heads of an item, so that there are
// few CTAs to start; it has the pieces of a long one side by side as well (63 sequences of 300
// positions and one of 65536: 46 us one after the other, 28 so).  Scored
// calls then add the weights of keys to the caller's scores, kJoinThreads keys of a sequence
// and KV head at a time.  A position's weight is summed over its heads in order by one thread: no
// atomics.
constexpr int kJoinMax = 1024;  // most pieces of an item: one per CTA of the first kernel
constexpr int kJoinThreads = 512;
constexpr int kInFlight = 8;     // pieces that a thread has on their way
constexpr int kItemFlight = 2;   // the same where a CTA joins a whole item: with 4, fewer CTAs fit an SM
                                 // (64 sequences of up to 8192 44.8 -> 44.4 us, scored calls 19.1 -> 20.8)

// (m, l) of one column of an item over its pieces, by a warp: right in lane 0.
__device__ __forceinline__ void join_ml(const AttendArgs& a, int item, int cols, int col, float* m_out, float* l_out) {
  const int lane = threadIdx.x & 31;
  const int2 pc = a.pieces[item];
  float M = -INFINITY, L = 0.0f;
  auto add = [&](float m, float l) {
    const float mn = fmaxf(M, m);
    L = L * (M == mn ? 1.0f : exp2_fast(M - mn)) + l * (m == mn ? 1.0f : exp2_fast(m - mn));
    M = mn;
  };
  if (pc.y == 1) {
    const float2 ml = reinterpret_cast<const float2*>(a.ml_whole)[(int64_t)item * cols + col];
    *m_out = ml.x;
    *l_out = ml.y;
    return;
  }
  for (int k = lane; k < pc.y; k += 32) {
    const float2 ml = reinterpret_cast<const float2*>(a.ml)[(2 * (int64_t)(pc.x + k) + (k == 0 ? 1 : 0)) * cols + col];
    add(ml.x, ml.y);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    const float m = __shfl_down_sync(0xffffffffu, M, off), l = __shfl_down_sync(0xffffffffu, L, off);
    add(m, l);
  }
  *m_out = M;
  *l_out = L;
}

template <typename T, int D, int NT, bool HEADS>
__global__ void __launch_bounds__(kJoinThreads) kv_attend_join(const KvView c, const AttendArgs a) {
  constexpr int COLS = 8 * NT, WAYS = kJoinThreads / (D / 4);
  __shared__ float sm_m[kJoinMax], sm_l[kJoinMax];  // pieces of an item; heads of a KV head
  __shared__ float4 red[kJoinThreads];
  __shared__ float red_m[kJoinThreads / 32], red_l[WAYS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = c.heads * a.n_chunks, all = c.n_seqs * items;
  constexpr int PER = HEADS ? COLS : 1;  // joining CTAs of an item
  const int n_join = all * PER;
  const bool joins = (int)blockIdx.x < n_join;
  const int x = (int)blockIdx.x - n_join;
  const int idx = joins ? blockIdx.x / PER : 0;
  const int b = joins ? idx / items : x / a.score_ctas / c.heads;
  const int len = attend_len(c, a, b);  // an argument of the call: not written by the first kernel
  // Every CTA waits for the first kernel, also one without work: this grid's end stands for both.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (joins) {
    const int col = blockIdx.x % PER, item = idx % items;
    const int h = item / a.n_chunks, chunk = item - h * a.n_chunks;
    const int n_heads = min(COLS, a.group - chunk * COLS);
    if (col >= n_heads) return;
    T* out = static_cast<T*>(a.out) + b * a.o_seq + (int64_t)(h * a.group + chunk * COLS + col) * a.o_head;
    if (len <= 0) {
      if (len < 0 && tid == 0) kv_flag(c.error, MOE_DEVERR_PAGE);
      const int n = HEADS ? D : n_heads * D;
      for (int o = tid; o < n; o += kJoinThreads)
        out[(o / D) * a.o_head + o % D] = from_float<T>(len < 0 ? __int_as_float(0x7fc00000) : 0.0f);
      return;
    }
    if constexpr (!HEADS) {
      const int2 pc = a.pieces[idx];
      if (pc.y == 1) return;  // one CTA had it whole
      constexpr int LANES = COLS * (D / 4), IW = kJoinThreads / LANES;  // threads of a piece, pieces side by side
      const int ch4 = tid % (D / 4), hc = tid / (D / 4) % COLS, way = tid / LANES;
      float M = -INFINITY, L = 0.0f;
      float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      auto add = [&](float m, float l, const float4& v) {
        const float mn = fmaxf(M, m);
        const float fo = M == mn ? 1.0f : exp2_fast(M - mn), fk = m == mn ? 1.0f : exp2_fast(m - mn);
        L = L * fo + l * fk;
        O = make_float4(O.x * fo + v.x * fk, O.y * fo + v.y * fk, O.z * fo + v.z * fk, O.w * fo + v.w * fk);
        M = mn;
      };
      if (hc < n_heads) {
        for (int k0 = way; k0 < pc.y; k0 += kItemFlight * IW) {
          float2 ml[kItemFlight];
          float4 v[kItemFlight];
#pragma unroll
          for (int i = 0; i < kItemFlight; ++i) {
            const int k = k0 + i * IW;
            if (k >= pc.y) break;
            const int64_t at = (2 * (int64_t)(pc.x + k) + (k == 0 ? 1 : 0)) * COLS + hc;
            ml[i] = reinterpret_cast<const float2*>(a.ml)[at];
            v[i] = reinterpret_cast<const float4*>(a.part + at * D)[ch4];
          }
#pragma unroll
          for (int i = 0; i < kItemFlight; ++i) {
            if (k0 + i * IW >= pc.y) break;
            add(ml[i].x, ml[i].y, v[i]);
          }
        }
      }
      if (IW > 1) {
        sm_m[tid] = M;
        sm_l[tid] = L;
        red[tid] = O;
        __syncthreads();
#pragma unroll
        for (int w = 1; w < IW; ++w)
          if (way == 0) add(sm_m[tid + w * LANES], sm_l[tid + w * LANES], red[tid + w * LANES]);
      }
      if (way == 0 && hc < n_heads) {
        T* to = out + hc * a.o_head + 4 * ch4;
        to[0] = from_float<T>(L != L ? L : O.x / L);
        to[1] = from_float<T>(L != L ? L : O.y / L);
        to[2] = from_float<T>(L != L ? L : O.z / L);
        to[3] = from_float<T>(L != L ? L : O.w / L);
      }
    } else {
      const int2 pc = a.pieces[idx];
      const int c0 = pc.x, n = pc.y;
      if (n == 1) return;  // one CTA had it whole
      const int ch4 = tid % (D / 4), way = tid / (D / 4);
      auto piece = [&](int k) { return (2 * (int64_t)(c0 + k) + (k == 0 ? 1 : 0)) * COLS + col; };
      auto fetch = [&](int k0, float4(&v)[kInFlight]) {
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
          if (k0 + i * WAYS < n) v[i] = reinterpret_cast<const float4*>(a.part + piece(k0 + i * WAYS) * D)[ch4];
      };
      float4 v[kInFlight];
      fetch(way, v);  // on their way while the weights are formed
      float m = -INFINITY;
      for (int k = tid; k < n; k += kJoinThreads) {
        const float2 ml = reinterpret_cast<const float2*>(a.ml)[piece(k)];
        sm_m[k] = ml.x;
        sm_l[k] = ml.y;
        m = fmaxf(m, ml.x);
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (lane == 0) red_m[warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red_m[w]);
      float L = 0.0f;
      float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k0 = way; k0 < n; k0 += kInFlight * WAYS) {
        if (k0 != way) fetch(k0, v);
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
          const int k = k0 + i * WAYS;
          if (k >= n) break;
          const float f = sm_m[k] == m ? 1.0f : exp2_fast(sm_m[k] - m);
          L = fmaf(sm_l[k], f, L);
          O = make_float4(fmaf(v[i].x, f, O.x), fmaf(v[i].y, f, O.y), fmaf(v[i].z, f, O.z), fmaf(v[i].w, f, O.w));
        }
      }
      red[tid] = O;
      if (ch4 == 0) red_l[way] = L;
      __syncthreads();
      if (tid >= D) return;
      float sum = 0.0f, den = 0.0f;
#pragma unroll
      for (int w = 0; w < WAYS; ++w) {
        sum += reinterpret_cast<const float*>(red)[w * D + tid];
        den += red_l[w];
      }
      out[tid] = from_float<T>(sum / den);  // a NaN of any piece's sum is in den
    }
    return;
  }
  const int h = x / a.score_ctas % c.heads, step = a.score_ctas * kJoinThreads;
  int key = x % a.score_ctas * kJoinThreads + tid;
  if (key - tid >= len) return;
  const float4* z = reinterpret_cast<const float4*>(a.z + ((int64_t)(b * items + h * a.n_chunks) * a.max_len + key) * COLS);
  float* score = a.score + b * a.s_seq + h * a.s_head + key;
  float4 v[COLS / 4];
  auto fetch = [&](int chunk) {
#pragma unroll
    for (int i = 0; i < COLS / 4; ++i) v[i] = z[(int64_t)chunk * a.max_len * (COLS / 4) + i];
  };
  float old = 0.0f;
  if (key < len) {  // on their way while the heads' maxima and sums are joined
    fetch(0);
    old = *score;
  }
  for (int col = warp; col < a.n_chunks * COLS; col += kJoinThreads / 32) {
    float M, L;
    join_ml(a, b * items + h * a.n_chunks + col / COLS, COLS, col % COLS, &M, &L);
    if (lane == 0) {
      sm_m[col] = M;
      sm_l[col] = 1.0f / L;
    }
  }
  __syncthreads();
  while (key < len) {
    float w = 0.0f;
    for (int chunk = 0; chunk < a.n_chunks; ++chunk) {
      const int n = min(COLS, a.group - chunk * COLS);
      if (chunk) fetch(chunk);
#pragma unroll
      for (int i = 0; i < COLS; ++i)
        if (i < n) w += exp2_fast(reinterpret_cast<const float*>(v)[i] - sm_m[chunk * COLS + i]) * sm_l[chunk * COLS + i];
    }
    *score = old + w;
    if (len - key <= step) return;
    key += step;
    z += (int64_t)step * (COLS / 4);
    score += step;
    fetch(0);
    old = *score;
  }
}

// ------------------------------------------------------------------ host

struct AttendPlan {
  int nt, chunks, n_cta, min_run, score_ctas;
  int64_t items;
  size_t part, ml, ml_whole, pieces, z, total;  // byte offsets
};

static int attend_plan(const KvView& c, int device, int n_q_heads, int max_len, bool scored, AttendPlan* p) {
  if (n_q_heads < 1 || max_len < 0) return MOE_ERR_INVALID;
  if (n_q_heads % c.heads) return MOE_ERR_INVALID;
  const int group = n_q_heads / c.heads;
  if (group > 1024 || max_len > kKvMaxPos) return MOE_ERR_UNSUPPORTED;
  // Heads of an item: 16 when there are more than 8, so that a tile is read once for them (us
  // with 8 / 16, 64 sequences of up to 8192, 4 groups of 16 heads of 128: 106 / 94; of 32
  // heads: 197 / 169; one sequence of 700: 9.3 / 10.9); empty columns cost (groups of 8: 60 / 91).
  p->nt = group <= 8 ? 1 : 2;
  p->chunks = (group + 8 * p->nt - 1) / (8 * p->nt);
  p->items = (int64_t)c.n_seqs * c.heads * p->chunks;
  const int64_t tiles = p->items * ((max_len + kTileTok - 1) / kTileTok + kItemCost);
  if (tiles > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  const int sms = kv_sm_count(device);
  if (!sms) return MOE_ERR_CUDA;
  // A run is at least one group a warp, so that short caches are spread no thinner than a
  // CTA's warps.
  p->min_run = kAW * kGT;
  // CTAs for the weights of a sequence's and KV head's keys: one for every 512 that there may be, but no more
  // than 16 an SM in all, which take blocks in turn: sequences are often far shorter than
  // max_len, and each CTA without work costs 2 to 3 ns (63 sequences of 300 positions and one of
  // 65536, 4 KV heads: 111 us with all of them, 39 so; 64 of up to 4096, where all have work: 58 either way).
  const int64_t per = (max_len + kJoinThreads - 1) / kJoinThreads, rows = (int64_t)c.n_seqs * c.heads;
  p->score_ctas = (int)(rows * per <= 16 * sms ? per : rows < 16 * sms ? 16 * sms / rows : 1);
  if (p->items * 8 * p->nt + (scored ? rows * p->score_ctas : 0) > kKvMaxPos) return MOE_ERR_UNSUPPORTED;
  const int64_t most = (tiles + p->min_run - 1) / p->min_run;
  // (Two CTAs an SM fit as long as the starts of the sequences do: up to 471 with heads of 128. From there on
  // they run one after the other: 471 sequences of 1000 positions, 4 groups of 8 heads, 96 us, 472 134.)
  int fill = (p->nt == 1 ? 2 : 1) * sms;
  if (fill > kJoinMax) fill = kJoinMax;
  p->n_cta = (int)(most < fill ? (most ? most : 1) : fill);
  const int cols = 8 * p->nt;
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t r = off;
    off = (off + n + 255) / 256 * 256;
    return r;
  };
  p->part = take((size_t)2 * p->n_cta * cols * c.dim * 4);
  p->ml = take((size_t)2 * p->n_cta * cols * 8);
  p->ml_whole = take(scored ? (size_t)p->items * cols * 8 : 0);
  p->pieces = take((size_t)p->items * 8);
  p->z = take(scored ? (size_t)p->items * max_len * cols * 4 : 0);
  p->total = off;
  return MOE_OK;
}

template <typename T, int D, int NT>
static cudaError_t attend_go(const KvView& c, const AttendArgs& a, const AttendPlan& p, int device, cudaStream_t st) {
  const int smem = AttendSmem<D, NT>::bytes(c.n_seqs);
  static std::atomic<bool> ready[kKvMaxDevices];  // shared-memory limits raised (the same value each time)
  if (!ready[device]) {
    static_assert(AttendSmem<D, NT>::kPre + (kKvMaxSeqs + 1) * 4 <= 227 * 1024, "the prefix of the longest batch fits");
    cudaError_t e = cudaFuncSetAttribute(kv_attend_kernel<T, D, NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv_attend_kernel<T, D, NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    ready[device] = true;
  }
  cudaError_t e = a.score ? kv_launch(kv_attend_kernel<T, D, NT, true>, p.n_cta, kAW * 32, smem, st, false, c, a)
                          : kv_launch(kv_attend_kernel<T, D, NT, false>, p.n_cta, kAW * 32, smem, st, false, c, a);
  if (e != cudaSuccess) return e;
  // Few items have many pieces each: a CTA for every head joins them; of many items each has a
  // piece or two, and a CTA joins all heads.  Us by head / by item, heads of 128: 4 items
  // of 131072 positions 26 / 39, 32 of 8192 16.1 / 17.4, 64 of 4096 19.2 / 17.9, 128 31 / 25, 1024 of 1000
  // 80 / 51; scored calls 38 / 40, 21.3 / 18.4, 24.7 / 20.4, 41 / 32, 98 / 65.
  const bool heads = p.items < 32;  // (scores or not: the same bits)
  const int grid = (int)p.items * (heads ? 8 * NT : 1) + (a.score ? c.n_seqs * c.heads * p.score_ctas : 0);
  return heads ? kv_launch(kv_attend_join<T, D, NT, true>, grid, kJoinThreads, 0, st, true, c, a)
               : kv_launch(kv_attend_join<T, D, NT, false>, grid, kJoinThreads, 0, st, true, c, a);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_kv_attend_workspace(const moe_kv_pool* cache, const moe_kv_table* table, int32_t n_q_heads,
                                       int32_t max_len, int32_t scored, size_t* bytes) {
  KvView c;
  AttendPlan p;
  int bad = kv_check(cache, table, &c);
  if (!bad && !bytes) bad = MOE_ERR_INVALID;
  if (!bad) bad = attend_plan(c, cache->device, n_q_heads, max_len, scored != 0, &p);
  if (!bad) *bytes = p.total;
  return bad;
}

extern "C" int moe_kv_attend(const moe_kv_pool* cache, const moe_kv_table* table, const int32_t* len_dev,
                             int32_t max_len, const moe_rows* q, int32_t n_q_heads, int32_t dtype, float scale,
                             const moe_rows* out, const moe_kv_score* score, void* workspace, size_t workspace_bytes,
                             void* stream) {
  KvView c;
  AttendPlan p;
  int bad = kv_check(cache, table, &c);
  if (bad) return bad;
  if (!len_dev || !q || !out || !q->data_dev || !out->data_dev || (score && !score->data_dev)) return MOE_ERR_INVALID;
  if ((dtype != MOE_BF16 && dtype != MOE_F16) || !(scale > 0.0f) || scale - scale != 0.0f)
    return MOE_ERR_INVALID;
  if (!kv_align_ok(q->data_dev, 2) || !kv_align_ok(out->data_dev, 2)) return MOE_ERR_INVALID;
  if (!kv_apart(out->token_stride, c.n_seqs, out->head_stride, n_q_heads)) return MOE_ERR_INVALID;
  if (score && !kv_apart(score->seq_stride, c.n_seqs, score->head_stride, c.heads)) return MOE_ERR_INVALID;
  bad = attend_plan(c, cache->device, n_q_heads, max_len, score != nullptr, &p);
  if (bad) return bad;
  if (c.n_seqs == 0) return MOE_OK;
  if (!workspace || !kv_align_ok(workspace, 16) || workspace_bytes < p.total) return MOE_ERR_INVALID;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttendArgs a{};
  a.q = q->data_dev;
  a.q_seq = q->token_stride;
  a.q_head = q->head_stride;
  a.out = out->data_dev;
  a.o_seq = out->token_stride;
  a.o_head = out->head_stride;
  a.lens = len_dev;
  a.max_len = max_len;
  a.group = n_q_heads / c.heads;
  a.n_chunks = p.chunks;
  a.scale2 = scale * 1.4426950408889634f;
  a.min_run = p.min_run;
  a.score_ctas = p.score_ctas;
  a.stall = kv_stall();
  a.vec = kv_align_ok(q->data_dev, 8) && q->token_stride % 4 == 0 && q->head_stride % 4 == 0;
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.ml = reinterpret_cast<float*>(ws + p.ml);
  a.ml_whole = reinterpret_cast<float*>(ws + p.ml_whole);
  a.pieces = reinterpret_cast<int2*>(ws + p.pieces);
  a.z = reinterpret_cast<float*>(ws + p.z);
  if (score) {
    a.score = score->data_dev;
    a.s_seq = score->seq_stride;
    a.s_head = score->head_stride;
  }
  DeviceScope dev(cache->device);
  if (!dev.ok) return MOE_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool bf = dtype == MOE_BF16;
#define MOE_GO(D, NT)                                                              \
  (bf ? attend_go<__nv_bfloat16, D, NT>(c, a, p, cache->device, st) : attend_go<__half, D, NT>(c, a, p, cache->device, st))
  if (c.dim == 64) e = p.nt == 1 ? MOE_GO(64, 1) : MOE_GO(64, 2);
  else e = p.nt == 1 ? MOE_GO(128, 1) : MOE_GO(128, 2);
#undef MOE_GO
  return kv_status(e);
}
