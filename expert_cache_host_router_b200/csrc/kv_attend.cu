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
// operands would have to be dequantised into shared memory first.  The nibbles become 16-bit floats
// by bit operations alone: (w & mask) | magic is base + q exactly, and for the keys
// -(base + 8) sum_c q_c is the accumulator's initial value, so the product of the codes
// q - 8 comes out without a subtraction; the block scale multiplies the fp32 partial sum.
// Values are (q - 8) d rounded to fp16 (half a step, 2^-11) and weights p fp16 too, for
// both input types: cached values are within the fp16 range by construction.
#include <type_traits>

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
  int vec;                       // rows of q can be read 8 bytes at a time
  float* part;                   // [2 CTAs][8 NT][D] partial outputs, unnormalised
  float* ml;                     // [2 CTAs][8 NT][2] their (m, l)
  float* ml_whole;               // [items][8 NT][2] (m, l) of the items that one CTA has whole (scored calls)
  float* z;                      // [items][max_len][8 NT] scaled products in log2 units (scored calls)
  float* score;                  // or null
  int64_t s_seq, s_head;
};

// The line of tiles: sequence b starts at pre[b] * items_per_seq and holds pre[b + 1] - pre[b]
// tiles for each of its items (KV head and chunk).  Lengths that cannot be are taken as 0.
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
// False when the copy has not landed within 2 s.
__device__ __noinline__ bool kv_mbar_spin(uint64_t* bar, uint32_t parity) {
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  while (!kv_mbar_try(bar, parity)) {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > 2000000000ull) return false;
  }
  return true;
}

// One bulk copy into shared memory.  Cache rows are read once per step: evict first.
__device__ __forceinline__ void kv_bulk(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(kv_smem(bar))
               : "memory");
}
__device__ __forceinline__ void kv_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(kv_smem(bar)), "r"(bytes) : "memory");
}

// A 16-bit type as the matrix products take it: base + q by bit operations.
template <typename T>
struct Magic;
template <>
struct Magic<__half> {  // 64 + q with q at mantissa bits 4..7
  static constexpr uint32_t mask = 0x00F000F0u, bits = 0x54005400u;
  static constexpr float base = 64.0f;
  static constexpr int at = 4;
};
template <>
struct Magic<__nv_bfloat16> {  // 128 + q with q at mantissa bits 0..3
  static constexpr uint32_t mask = 0x000F000Fu, bits = 0x43004300u;
  static constexpr float base = 128.0f;
  static constexpr int at = 0;
};
template <typename T, int N>  // nibble N of both halves of w
__device__ __forceinline__ uint32_t magic(uint32_t w) {
  constexpr int sh = 4 * N - Magic<T>::at;
  const uint32_t s = sh > 0 ? w >> sh : w << -sh;
  return (s & Magic<T>::mask) | Magic<T>::bits;
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, const float (&c)[4]) {
  if constexpr (sizeof(T) == 2 && Magic<T>::at == 0)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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
    if (lin >= end) return false;
    while (pre[b + 1] * items <= lin) ++b;  // lin < end <= pre[n_seqs] * items: ends
    s.b = b;
    s.nt = pre[b + 1] - pre[b];
    const int off = lin - pre[b] * items;
    s.item = off / s.nt;
    s.s0 = off - s.item * s.nt;
    s.s1 = min(s.nt, s.s0 + end - lin);
    lin += s.s1 - s.s0;
    return true;
  }
};

template <int D, int NT>
struct AttendSmem {
  static constexpr int kStages = NT == 1 ? 2 : 4;
  static constexpr int kTile = 18 * D, kStage = kGT * kTile;
  static constexpr int kFrag = (D / 4) * NT + 4 * NT;  // floats of a thread's state: o, then m and l of its columns
  static constexpr int kRing = kAW * kStages * kStage;
  static constexpr int kMerge = (kAW / 2) * 32 * kFrag * 4;
  static constexpr int kBars = kRing + kMerge;
  static constexpr int kTmp = kBars + kAW * kStages * 8;
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
  Line cons{lin0, min(total, lin0 + run), 0};
  {  // first sequence of the run
    int lo = 0, hi = c.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * items <= lin0) lo = mid; else hi = mid - 1;
    }
    cons.b = lo;
  }

  // Producer side (all lanes keep its state, lane 0 issues): groups of this warp in order,
  // over segment borders.  The page numbers of the group after next are read one step
  // ahead, so that no copy waits for them.
  Line prod = cons;
  Segment ps;
  bool p_more = prod.next(pre, items, c.n_seqs, ps);
  int pk = warp;            // group of the segment
  int pg[kGT], pb[kGT];     // page numbers read ahead, tile within the page
  Segment as{};             // segment and group of the read-ahead
  int ak = -1;
  auto ahead = [&]() {      // next group of this warp: look its pages up
    while (p_more && ps.s0 + pk * kGT >= ps.s1) {
      p_more = prod.next(pre, items, c.n_seqs, ps);
      pk = warp;
    }
    ak = p_more ? pk : -1;
    as = ps;
    if (ak >= 0) {
#pragma unroll
      for (int i = 0; i < kGT; ++i) {
        const int tile = ps.s0 + pk * kGT + i;
        const int p = tile / c.tiles_per_page;
        pb[i] = tile - p * c.tiles_per_page;
        pg[i] = tile < ps.s1 ? c.table[(int64_t)ps.b * c.table_stride + p] : -2;
      }
      pk += kAW;
    }
  };
  uint32_t bad = 0;  // stages whose group names a page that is not there
  auto issue = [&](int stage) {  // copy the group that was looked up, then look up the next
    if (ak >= 0) {
      const int h = as.item / a.n_chunks;
      uint32_t bytes = 0;
      bad &= ~(1u << stage);
#pragma unroll
      for (int i = 0; i < kGT; ++i) {
        if (pg[i] == -2) continue;
        if ((unsigned)pg[i] < (unsigned)c.n_pages) bytes += S::kTile; else bad |= 1u << stage;
      }
      if (lane == 0) {
        kv_expect(bars + stage, bytes);
#pragma unroll
        for (int i = 0; i < kGT; ++i)
          if ((unsigned)pg[i] < (unsigned)c.n_pages)
            kv_bulk(kv_smem(ring + stage * S::kStage + i * S::kTile),
                    c.pool + (((int64_t)pg[i] * c.heads + h) * c.tiles_per_page + pb[i]) * S::kTile, S::kTile,
                    bars + stage);
      }
    }
    ahead();
  };
  ahead();
#pragma unroll
  for (int s = 0; s < ST; ++s) issue(s);

  int stage = 0;
  uint32_t phase = 0;
  bool alive = true;
  Segment sg;
  while (cons.next(pre, items, c.n_seqs, sg)) {
    const int h = sg.item / a.n_chunks, chunk = sg.item - h * a.n_chunks;
    const int len = attend_len(c, a, sg.b);
    const int n_heads = min(COLS, a.group - chunk * COLS);  // query heads of this item
    const int h0 = h * a.group + chunk * COLS;
    // Query fragments: column n = g of each 8 heads; within a block the channels of the two
    // 16-deep steps are 4t + {0, 2, 1, 3} and 16 more, the order that the nibbles come in.
    uint32_t qf[NT][NB][4];
    float qi[NT][NB][2];  // -(base + 8) * sum of a block's channels, for columns 2t and 2t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool has = n * 8 + g < n_heads;
      const T* qp = static_cast<const T*>(a.q) + sg.b * a.q_seq + (int64_t)(h0 + n * 8 + (has ? g : 0)) * a.q_head + 4 * t;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float sum = 0.0f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint16_t e[4] = {0, 0, 0, 0};
          if (has) {
            if (a.vec) {
              *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(qp + nb * 32 + hf * 16);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) e[i] = reinterpret_cast<const uint16_t*>(qp + nb * 32 + hf * 16)[i];
            }
          }
          qf[n][nb][2 * hf] = e[0] | (uint32_t)e[2] << 16;
          qf[n][nb][2 * hf + 1] = e[1] | (uint32_t)e[3] << 16;
#pragma unroll
          for (int i = 0; i < 4; ++i) sum += to_float(*reinterpret_cast<const T*>(&e[i]));
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -(Magic<T>::base + 8.0f);
        qi[n][nb][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
        qi[n][nb][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
      }
    }
    float o[NT][NB][2][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < NB * 8; ++i) (&o[n][0][0][0])[i] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }
    float* zrow = SCORED ? a.z + ((int64_t)(sg.b * items + sg.item) * a.max_len) * COLS : nullptr;

    for (int k = warp; sg.s0 + k * kGT < sg.s1; k += kAW) {
      if (alive && !kv_mbar_try(bars + stage, phase) && !kv_mbar_spin(bars + stage, phase)) {
        alive = false;
        kv_flag(c.error, MOE_DEVERR_TMA);
      }
      const uint8_t* base = ring + stage * S::kStage;
      const int tile0 = sg.s0 + k * kGT;
      const int left = min(len, sg.s1 * kTileTok) - tile0 * kTileTok;  // keys of this group
      float z[NT][kGT][4];
#pragma unroll
      for (int i = 0; i < kGT; ++i) {
        const uint8_t* tl = base + i * S::kTile;
        // keys: lane (g, t) has word t of every block of rows g and g + 8
        uint32_t kw[2][NB];
        __half ks[2][NB];
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
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[n][i][e] = 0.0f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t a0[4], a1[4];
          a0[0] = magic<T, 0>(kw[0][nb]), a0[1] = magic<T, 1>(kw[0][nb]), a0[2] = magic<T, 2>(kw[0][nb]), a0[3] = magic<T, 3>(kw[0][nb]);
          a1[0] = magic<T, 0>(kw[1][nb]), a1[1] = magic<T, 1>(kw[1][nb]), a1[2] = magic<T, 2>(kw[1][nb]), a1[3] = magic<T, 3>(kw[1][nb]);
          const float d0 = __half2float(ks[0][nb]), d1 = __half2float(ks[1][nb]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float s[4];
            const float ini[4] = {qi[n][nb][0], qi[n][nb][1], qi[n][nb][0], qi[n][nb][1]};
            mma16816<T>(s, a0[0], a1[0], a0[2], a1[2], qf[n][nb][0], qf[n][nb][1], ini);
            mma16816<T>(s, a0[1], a1[1], a0[3], a1[3], qf[n][nb][2], qf[n][nb][3], s);
            z[n][i][0] = fmaf(s[0], d0, z[n][i][0]);
            z[n][i][1] = fmaf(s[1], d0, z[n][i][1]);
            z[n][i][2] = fmaf(s[2], d1, z[n][i][2]);
            z[n][i][3] = fmaf(s[3], d1, z[n][i][3]);
          }
        }
      }
      const bool tail = left < kGT * kTileTok, broken = !alive || (bad >> stage & 1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kGT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = z[n][i][e] * a.scale2;
            const int key = i * kTileTok + g + 8 * (e >> 1);
            if (broken) v = __int_as_float(0x7fc00000);
            if (tail && key >= left) v = -INFINITY;
            z[n][i][e] = v;
            mx[e & 1] = fmaxf(mx[e & 1], v);
          }
        if (SCORED) {
#pragma unroll
          for (int i = 0; i < kGT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int key = i * kTileTok + g + 8 * r;
              if (key < left)
                *reinterpret_cast<float2*>(zrow + (int64_t)(tile0 * kTileTok + key) * COLS + n * 8 + 2 * t) =
                    make_float2(z[n][i][2 * r], z[n][i][2 * r + 1]);
            }
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
          mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
        }
        // The running maximum moves only when it is exceeded by more than 8 (a factor of 256):
        // weights stay below 256, far inside fp16, and most groups rescale nothing.
        const bool move = mx[0] > m[n][0] + 8.0f || mx[1] > m[n][1] + 8.0f || m[n][0] == -INFINITY || m[n][1] == -INFINITY;
        if (__any_sync(0xffffffffu, move)) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m[n][e], mx[e]);
            al[e] = m[n][e] == mn ? 1.0f : exp2_fast(m[n][e] - mn);
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
#pragma unroll
        for (int i = 0; i < kGT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = exp2_fast(z[n][i][e] - m[n][e & 1]);
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
          const uint32_t off = 0x54805480u;  // 72 = 64 + 8
          uint32_t va[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            va[r][0] = hmul2(hsub2(magic<__half, 0>(vw[r][nb]), off), vs[r][nb]);
            va[r][1] = hmul2(hsub2(magic<__half, 1>(vw[r][nb]), off), vs[r][nb]);
            va[r][2] = hmul2(hsub2(magic<__half, 2>(vw[r][nb]), off), vs[r][nb]);
            va[r][3] = hmul2(hsub2(magic<__half, 3>(vw[r][nb]), off), vs[r][nb]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816<__half>(o[n][nb][0], va[0][0], va[0][1], va[1][0], va[1][1], pf[n][0], pf[n][1], o[n][nb][0]);
            mma16816<__half>(o[n][nb][1], va[0][2], va[0][3], va[1][2], va[1][3], pf[n][0], pf[n][1], o[n][nb][1]);
          }
        }
      }
      // Every lane has read the stage; the fence orders those reads before the copy engine's write.
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      issue(stage);
      if (++stage == ST) {
        stage = 0;
        phase ^= 1;
      }
    }

    // Join the warps, halves at a time: same lane, same fragment.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
#pragma unroll
    for (int half = kAW / 2; half >= 1; half >>= 1) {
      float* at = merge + (warp & (half - 1)) * 32 * S::kFrag + lane;
      if (warp >= half && warp < 2 * half) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < NB * 8; ++i) at[(n * NB * 8 + i) * 32] = (&o[n][0][0][0])[i];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            at[(NT * NB * 8 + 4 * n + e) * 32] = m[n][e];
            at[(NT * NB * 8 + 4 * n + 2 + e) * 32] = l[n][e];
          }
        }
      }
      __syncthreads();
      if (warp < half) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float x[2], y[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mo = at[(NT * NB * 8 + 4 * n + e) * 32], lo = at[(NT * NB * 8 + 4 * n + 2 + e) * 32];
            const float mn = fmaxf(m[n][e], mo);
            x[e] = m[n][e] == mn || m[n][e] == -INFINITY ? (m[n][e] == mn ? 1.0f : 0.0f) : exp2_fast(m[n][e] - mn);
            y[e] = mo == mn || mo == -INFINITY ? (mo == mn ? 1.0f : 0.0f) : exp2_fast(mo - mn);
            m[n][e] = mn;
            l[n][e] = l[n][e] * x[e] + lo * y[e];
          }
#pragma unroll
          for (int i = 0; i < NB * 8; ++i) {
            float* ov = &o[n][0][0][0];
            ov[i] = ov[i] * x[i & 1] + at[(n * NB * 8 + i) * 32] * y[i & 1];
          }
        }
      }
      __syncthreads();
    }
    if (warp == 0) {
      const bool whole = sg.s0 == 0 && sg.s1 == sg.nt;
      const int slot = 2 * blockIdx.x + (sg.s0 == 0 ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = n * 8 + 2 * t + e;
          if (whole) {
            if (SCORED && g == 0) {
              float* ml = a.ml_whole + ((int64_t)(sg.b * items + sg.item) * COLS + col) * 2;
              ml[0] = m[n][e];
              ml[1] = l[n][e];
            }
            if (col < n_heads) {
              const float inv = 1.0f / l[n][e];
              T* op = static_cast<T*>(a.out) + sg.b * a.o_seq + (int64_t)(h0 + col) * a.o_head + 2 * g;
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                op[nb * 32] = from_float<T>(o[n][nb][0][e] * inv);
                op[nb * 32 + 1] = from_float<T>(o[n][nb][1][e] * inv);
                op[nb * 32 + 16] = from_float<T>(o[n][nb][0][2 + e] * inv);
                op[nb * 32 + 17] = from_float<T>(o[n][nb][1][2 + e] * inv);
              }
            }
          } else {
            if (g == 0) {
              float* ml = a.ml + ((int64_t)slot * COLS + col) * 2;
              ml[0] = m[n][e];
              ml[1] = l[n][e];
            }
            float* pp = a.part + ((int64_t)slot * COLS + col) * D + 2 * g;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              *reinterpret_cast<float2*>(pp + nb * 32) = make_float2(o[n][nb][0][e], o[n][nb][1][e]);
              *reinterpret_cast<float2*>(pp + nb * 32 + 16) = make_float2(o[n][nb][0][2 + e], o[n][nb][1][2 + e]);
            }
          }
        }
    }
  }
}

// ------------------------------------------------------------------ second kernel

// CTA x < items joins the partial results of one item (or writes the rows of a sequence
// without positions: zeros, or NaN when its length cannot be); scored calls then add the
// weights of keys to the caller's scores, 256 keys of an item's sequence and head a CTA.
// A position's weight is summed over its heads in order by one thread: no atomics.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(256) kv_attend_join(const KvView c, const AttendArgs a, int n_cta) {
  constexpr int COLS = 8 * NT;
  __shared__ int tmp[8];
  __shared__ float sm_m[64 * 16], sm_l[64 * 16];  // per head of a KV head's chunks
  extern __shared__ int pre[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  attend_prefix(c, a, pre, tmp);
  const int items = c.heads * a.n_chunks;
  const int total = pre[c.n_seqs] * items;
  const int run = attend_run(a, total, n_cta);
  const int all = c.n_seqs * items;
  if ((int)blockIdx.x < all) {
    const int b = blockIdx.x / items, item = blockIdx.x % items;
    const int h = item / a.n_chunks, chunk = item - h * a.n_chunks;
    const int nt = pre[b + 1] - pre[b];
    const int n_heads = min(COLS, a.group - chunk * COLS), h0 = h * a.group + chunk * COLS;
    const int lo = pre[b] * items + item * nt;
    const int c0 = nt ? lo / run : 0, c1 = nt ? (lo + nt - 1) / run : 0;
    if (nt && c0 == c1) return;  // one CTA had it whole
    const float none = attend_len(c, a, b) < 0 ? __int_as_float(0x7fc00000) : 0.0f;
    if (!nt && none != none && item == 0 && tid == 0) kv_flag(c.error, MOE_DEVERR_PAGE);
    for (int x = tid; x < n_heads * D; x += 256) {
      const int col = x / D, ch = x % D;
      float v = none;
      if (nt) {
        float M = -INFINITY, L = 0.0f, O = 0.0f;
        bool nan = false;
        for (int k = c0; k <= c1; ++k) {
          const int64_t slot = 2 * (int64_t)k + (k == c0 ? 1 : 0);
          const float mk = a.ml[(slot * COLS + col) * 2], lk = a.ml[(slot * COLS + col) * 2 + 1];
          const float ok = a.part[(slot * COLS + col) * D + ch];
          const float mn = fmaxf(M, mk);
          const float fo = M == mn ? 1.0f : exp2_fast(M - mn), fk = mk == mn ? 1.0f : exp2_fast(mk - mn);
          nan = nan || lk != lk;
          L = L * fo + lk * fk;
          O = O * fo + ok * fk;
          M = mn;
        }
        v = nan ? __int_as_float(0x7fc00000) : O / L;
      }
      static_cast<T*>(a.out)[b * a.o_seq + (int64_t)(h0 + col) * a.o_head + ch] = from_float<T>(v);
    }
    return;
  }
  if (!a.score) return;
  const int per = (a.max_len + 255) / 256;
  const int x = blockIdx.x - all, bh = x / per, b = bh / c.heads, h = bh % c.heads;
  const int nt = pre[b + 1] - pre[b], len = attend_len(c, a, b);
  const int key0 = (x % per) * 256;
  if (key0 >= len) return;
  for (int col = tid; col < a.n_chunks * COLS; col += 256) {
    const int chunk = col / COLS, cc = col % COLS, item = h * a.n_chunks + chunk;
    const int lo = pre[b] * items + item * nt;
    const int c0 = lo / run, c1 = (lo + nt - 1) / run;
    float M = -INFINITY, L = 0.0f;
    if (c0 == c1) {
      const float* ml = a.ml_whole + ((int64_t)(b * items + item) * COLS + cc) * 2;
      M = ml[0];
      L = ml[1];
    } else {
      for (int k = c0; k <= c1; ++k) {
        const int64_t slot = 2 * (int64_t)k + (k == c0 ? 1 : 0);
        const float mk = a.ml[(slot * COLS + cc) * 2], lk = a.ml[(slot * COLS + cc) * 2 + 1];
        const float mn = fmaxf(M, mk);
        L = L * (M == mn ? 1.0f : exp2_fast(M - mn)) + lk * (mk == mn ? 1.0f : exp2_fast(mk - mn));
        M = mn;
      }
    }
    sm_m[col] = M;
    sm_l[col] = 1.0f / L;
  }
  __syncthreads();
  const int key = key0 + tid;
  if (key >= len) return;
  float w = 0.0f;
  for (int head = 0; head < a.group; ++head) {
    const int chunk = head / COLS, cc = head % COLS;
    const float zz = a.z[((int64_t)(b * items + h * a.n_chunks + chunk) * a.max_len + key) * COLS + cc];
    w += exp2_fast(zz - sm_m[head]) * sm_l[head];
  }
  a.score[b * a.s_seq + h * a.s_head + key] += w;
}

// ------------------------------------------------------------------ host

struct AttendPlan {
  int nt, chunks, n_cta, min_run;
  int64_t items;
  size_t part, ml, ml_whole, z, total;  // byte offsets
};

static int sm_count(int dev) {
  static int n[kKvMaxDevices];
  if (!n[dev]) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    n[dev] = v;
  }
  return n[dev];
}

static int attend_plan(const KvView& c, int device, int n_q_heads, int max_len, bool scored, AttendPlan* p) {
  if (n_q_heads < 1 || max_len < 0) return MOE_ERR_INVALID;
  if (n_q_heads % c.heads) return MOE_ERR_INVALID;
  const int group = n_q_heads / c.heads;
  if (group > 1024) return MOE_ERR_UNSUPPORTED;
  p->nt = group <= 8 ? 1 : 2;
  p->chunks = (group + 8 * p->nt - 1) / (8 * p->nt);
  p->items = (int64_t)c.n_seqs * c.heads * p->chunks;
  const int64_t tiles = p->items * ((max_len + kTileTok - 1) / kTileTok);
  const int per = (max_len + 255) / 256;
  if (tiles > INT32_MAX / 2 || p->items + (scored ? (int64_t)c.n_seqs * c.heads * per : 0) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const int sms = sm_count(device);
  if (!sms) return MOE_ERR_CUDA;
  // A run is at least one group a warp, so that short caches are spread no thinner than a
  // CTA's warps.
  p->min_run = kAW * kGT;
  const int64_t most = (tiles + p->min_run - 1) / p->min_run;
  const int fill = (p->nt == 1 ? 2 : 1) * sms;
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
  p->z = take(scored ? (size_t)p->items * max_len * cols * 4 : 0);
  p->total = off;
  return MOE_OK;
}

template <typename K>
static cudaError_t launch(K kernel, int grid, int threads, size_t smem, cudaStream_t st, bool dependent,
                          const KvView& c, const AttendArgs& a, int n_cta) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = dependent ? 1 : 0;
  if constexpr (std::is_invocable_v<K, KvView, AttendArgs>) return cudaLaunchKernelEx(&cfg, kernel, c, a);
  else return cudaLaunchKernelEx(&cfg, kernel, c, a, n_cta);
}

template <typename T, int D, int NT>
static cudaError_t attend_go(const KvView& c, const AttendArgs& a, const AttendPlan& p, int device, cudaStream_t st) {
  const int smem = AttendSmem<D, NT>::bytes(c.n_seqs);
  static bool ready[kKvMaxDevices];  // shared-memory limits raised (the same value each time)
  if (!ready[device]) {
    static_assert(AttendSmem<D, NT>::kPre + (kKvMaxSeqs + 1) * 4 <= 227 * 1024, "the prefix of the longest batch fits");
    cudaError_t e = cudaFuncSetAttribute(kv_attend_kernel<T, D, NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv_attend_kernel<T, D, NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    ready[device] = true;
  }
  cudaError_t e = a.score ? launch(kv_attend_kernel<T, D, NT, true>, p.n_cta, kAW * 32, smem, st, false, c, a, 0)
                          : launch(kv_attend_kernel<T, D, NT, false>, p.n_cta, kAW * 32, smem, st, false, c, a, 0);
  if (e != cudaSuccess) return e;
  const int per = (a.max_len + 255) / 256;
  const int grid = (int)p.items + (a.score ? c.n_seqs * c.heads * per : 0);
  return launch(kv_attend_join<T, D, NT>, grid, 256, (size_t)(c.n_seqs + 1) * 4, st, true, c, a, p.n_cta);
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
  a.vec = kv_align_ok(q->data_dev, 8) && q->token_stride % 4 == 0 && q->head_stride % 4 == 0;
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.ml = reinterpret_cast<float*>(ws + p.ml);
  a.ml_whole = reinterpret_cast<float*>(ws + p.ml_whole);
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
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
