// Attention of a chunk of new tokens over a paged cache, bf16, on the tensor
// cores (tcgen05).
//
//   out[t, h] = sum_j softmax_j(scale q.k_j) v_j  over slots j <= p(t)
//
// One online-softmax pass over the keys.  A segment is one (sequence, kv head,
// group of query tokens): two M tiles of 128 rows, each floor(128 / G) tokens
// times their G query heads, against the key tiles its last token can see.
// All segments are laid end to end on an axis of cost (a tile by its M tiles,
// a segment's start and end) and every CTA takes an equal contiguous range of
// it, so prompts, single tokens and anything between fill the machine alike;
// where a range cuts a segment, its pieces are merged by log-sum-exp weights
// inside the kernel by the last piece to arrive.  A range has at most two such
// pieces (its first and its last), so the workspace depends on the number of
// CTAs alone.
//
// Roles (384 threads):
//   warp 0      TMA producer of Q and K.  Key tiles are 128 slots: part of a page of 128
//               or more, or as many whole smaller pages as fit (their boxes
//               land one after another in the tile; page sizes are multiples
//               of the 8-row swizzle atom, any other size takes one page per
//               tile).  Lanes fetch the page table entries and issue one
//               box each.
//   warp 2      the same of V.  K and V share one ring of 32 KB slots (dh =
//               128: 5), K's freed after its scores, V's after its product.
//   warp 1      MMA issuer: S = Q K^T into TMEM, then O += P V with P as bf16
//               in TMEM over the scores' columns.  The whole warp walks the
//               tiles and one elected lane issues; a product waits for its P
//               in a queue while the next scores are issued.
//   warps 4-11  two softmax warpgroups, one query row per thread, each with a
//               score buffer and an O of its own.  A segment of two M tiles
//               gives one to each.  A segment of one M tile (single tokens,
//               short chunks) gives its key tiles to them in turn, two
//               independent chains instead of one; the first warpgroup adds
//               the second's O to its own where the piece ends.
//
// Roundings to fewer bits than fp32: P to bf16, for both operands of a product
// have one type and V is bf16 (relative 2^-8 of each probability, while the sum
// l is of the fp32 values); O to bf16 once, at the end.  Scores, maxima, sums, O
// and the pieces are fp32.
//
// What bounds it, with what it measured (one B200; 6.55 TB/s copy and 1.66
// PFLOP/s bf16 products in a burst, 1.36 sustained):
//   prompts         the chain scores -> maximum -> exponentials -> P of a tile
//                   and, in long runs, the power limit.  8192 tokens, 32 + 8
//                   heads of 128: 485 us a call in a run of 100 (1.13
//                   PFLOP/s), 545 to 560 in runs of a thousand (0.98).
//   short chunks    the same, with M tiles partly empty and segments of a few
//                   tiles: 12 sequences of 1 to 600 tokens that end at 601 to
//                   6000 slots, pages of 16: 157 us in a run of 100, 170 to
//                   183 in long ones.
//   single tokens   HBM: 32 sequences of 30001 to 32768 slots 605 us, 6.8
//                   TB/s (660 to 680 in long runs, under the power limit);
//                   eight of 4096 to 8192 47 us, of which the prologue, the
//                   merge and the launch are a third; one of 6000, all
//                   latency, 19.3 us.
// Tried and slower: tiles of 64 keys with two score buffers a warpgroup (848 us
// where tiles of 128 took 565); some of the exponentials as a polynomial on the
// FMA units (every fourth pair: prompt 498 us, every eighth: 490, none: 480);
// rescaling O at every new maximum (prompt 519); a producer's and an issuer's
// single lane in divergent code (a third slower); one producer for K and V (a V
// waits behind the next K's slot).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "abi_internal.h"
#include "attn_common.cuh"
#include "chunk_attention.cuh"
#include "common.cuh"

namespace medusa {

namespace {

constexpr int kBN = 128;       // keys per tile
constexpr int kMT = 128;       // rows per M tile
constexpr int kRows = 256;     // rows per segment
constexpr int kThreads = 384;
constexpr int kRegsLow = 72;   // registers a thread: producer and MMA warpgroup
constexpr int kRegsHigh = 216;  // softmax warpgroups
constexpr float kLazy = 8.f;   // rescale O only when the maximum grows by 2^8
constexpr uint32_t kTmemCols = 512;
// What a CTA's range is measured in: the cost of a tile of two M tiles, of a
// tile of one, and of a segment's start and end (its Q, its first scores, its
// output).  With 2, 3 and 4 for a tile of one, short chunks took 280, 193 and
// 185 us and the prompt of 8192 tokens 499, 501 and 519; with 4, 8 and 16 for a
// segment 191, 173, 188 and 534, 501, 511.
constexpr int kTwoCost = 4, kOneCost = 3;
constexpr int kSegCost = 8;
// Smallest range a CTA takes: with 8, 16, 24 and 32 a token over 1000 slots of 8
// kv heads took 15.5, 19.5, 20.5 and 16.1 us, a chunk of 100 tokens 25.6, 27.2,
// 30.4 and 34.3.
constexpr int kMinCost = 8;
// The most tiles of a sequence and the longest stretch of a CTA: with them
// seg + (ntiles + 1) * kTwoCost + kSegCost stays below 2^31.
constexpr int kMaxTiles = 1 << 28;
constexpr int kMaxStretch = 1 << 29;
static_assert((long long)kMaxStretch + (kMaxTiles + 1ll) * kTwoCost + kSegCost <= 0x7fffffffll, "");
constexpr int kMaxB = 1024;
constexpr int kFewRows = 8;    // rows of a warp whose pieces the whole warp merges

struct TcParams {
  const int32_t *table, *cu_q, *kv_len;
  int n_pages, page, max_pages;
  int ppt;  // pages per tile (0: pages of 128 or more, tpp tiles each)
  int tpp, kt;  // kt: slots of a full tile
  int max_kv;   // slots of the table's pages, and of no more than kMaxTiles tiles
  int B, T, Hq, Hkv, G, tpt;  // tpt: tokens per M tile
  int q_box;                  // tokens per copy of Q
  float scale_log2;
  __nv_bfloat16* out;
  float* o_part;             // [2 * grid] pieces of [8] warps' rows: groups of 4 columns
                             // [dh / 4][32 rows], or whole rows [32][dh] (kFewRows)
  float* lse_part;           // [2 * grid][256]
  unsigned int* piece_count;  // [grid][8] pieces written, per warp of the segment that
                              // starts in the CTA and leaves it (zeroed per call)
  int32_t* status;
};

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

template <int DH>
struct Smem {
  static constexpr int kPanels = DH / 64;
  static constexpr int kQBytes = kMT * DH * 2;
  static constexpr int kItem = kBN * DH * 2;  // one K or V tile
  static constexpr int kPanel = kBN * 128;
  static constexpr int kRing = 5 * 128 / DH;  // K and V slots
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = 2 * kQBytes;
  static constexpr int kBarOff = kRingOff + kRing * kItem;
  // full[ring], empty[ring], q_full[2], s_full[2], p_full[2][2], pv_done[2], q_empty,
  // half_ready, half_free, drain, exit
  static constexpr int kNumBars = 2 * kRing + 15;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // holder, abort, ok, info[ring]
  static constexpr int kStartOff = kMiscOff + 16 + kRing * 4;
  static constexpr int kHalfOff = (kStartOff + 40 + 7) & ~7;  // float2 {base, sum}[128] of the second half
  static constexpr int kBytes = kHalfOff + kMT * 8;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  static_assert((kMaxB + 1) * 8 <= kRing * kItem, "schedule fits in the ring");
};

// key tiles that cover `vis` slots (at least one, so an empty row is written)
__device__ __forceinline__ int tiles_of(int vis, const TcParams& p) {
  if (p.ppt > 0) return max(1, vis / p.kt + (vis % p.kt != 0 ? 1 : 0));
  const int fp = vis / p.page;
  return max(1, fp * p.tpp + (vis - fp * p.page + kBN - 1) / kBN);
}

// slots the last token of query group qg sees
__device__ __forceinline__ int group_vis(int qlen, int kv, int qg, const TcParams& p) {
  return max(0, kv - qlen + min(qlen, (qg + 1) * 2 * p.tpt));
}

__device__ __forceinline__ int group_mt(int qlen, int qg, const TcParams& p) {
  return qlen - qg * 2 * p.tpt > p.tpt ? 2 : 1;
}
// length of a query group's segment on the axis below (an int: kMaxTiles)
__device__ __forceinline__ int group_cost(int qlen, int kv, int qg, const TcParams& p) {
  return tiles_of(group_vis(qlen, kv, qg, p), p) *
             (group_mt(qlen, qg, p) == 2 ? kTwoCost : kOneCost) +
         kSegCost;
}

// Walks the tiles of a CTA's range.  Segments lie end to end on one axis, each
// tile wt long, kSegCost after its last; a tile belongs to the CTA in whose
// stretch of the axis it starts.  The axis is as long as 64 bits; a cursor
// counts from its CTA's start, where kMaxStretch and kMaxTiles keep everything
// in 32.
struct Cursor {
  int b, kvh, qg, n_qg, q0, qlen, kv;
  int lt, ntiles, vis, n_mt, wt;
  int seg, end;  // from the CTA's start: start of the segment, end of the range
  bool live, first, last;

  __device__ __forceinline__ void sequence(const TcParams& p) {
    q0 = p.cu_q[b];
    qlen = p.cu_q[b + 1] - q0;
    kv = p.kv_len[b];
    n_qg = (qlen + 2 * p.tpt - 1) / (2 * p.tpt);
  }
  __device__ __forceinline__ void group(const TcParams& p) {
    vis = group_vis(qlen, kv, qg, p);
    ntiles = tiles_of(vis, p);
    n_mt = group_mt(qlen, qg, p);
    wt = n_mt == 2 ? kTwoCost : kOneCost;
  }
  // tiles of the segment from lt on that are the CTA's
  __device__ __forceinline__ int piece() const {
    return min(ntiles - lt, (end - seg - lt * wt + wt - 1) / wt);
  }
  // s: {b, kvh, qg, lt, seg, q0, qlen, kv}
  __device__ __forceinline__ void init(const int* s, int end_, const TcParams& p) {
    b = s[0];
    kvh = s[1];
    qg = s[2];
    lt = s[3];
    seg = s[4];
    q0 = s[5];
    qlen = s[6];
    kv = s[7];
    end = end_;
    n_qg = (qlen + 2 * p.tpt - 1) / (2 * p.tpt);
    group(p);
    live = first = true;
    last = piece() == 1;
  }
  __device__ __forceinline__ void advance(const TcParams& p) { skip(1, p); }
  // n tiles on, at most to the first tile of the next segment
  __device__ __forceinline__ void skip(int n, const TcParams& p) {
    lt += n;
    first = false;
    if (lt < ntiles) {
      live = seg + lt * wt < end;
    } else {
      const int next = seg + ntiles * wt + kSegCost;
      live = next < end;
      if (!live) return;
      seg = next;
      lt = 0;
      first = true;
      if (++qg == n_qg) {
        qg = 0;
        if (++kvh == p.Hkv) {
          kvh = 0;
          do {  // a later sequence with new tokens exists: the axis goes on
            ++b;
            sequence(p);
          } while (qlen == 0);
        }
      }
      group(p);
    }
    last = lt == ntiles - 1 || seg + (lt + 1) * wt >= end;
  }
  // first slot of the tile and how many of its slots the segment sees
  __device__ __forceinline__ void span(const TcParams& p, int& key0, int& nv, int& pg, int& r0) const {
    if (p.ppt > 0) {
      pg = lt * p.ppt;
      r0 = 0;
      key0 = lt * p.kt;
      nv = min(p.kt, vis - key0);
    } else {
      pg = lt / p.tpp;
      r0 = (lt - pg * p.tpp) * kBN;
      key0 = pg * p.page + r0;
      nv = min(min(kBN, p.page - r0), vis - key0);
    }
    nv = max(nv, 0);
  }
  // slots of the tile that the copy fills with real rows or zeros, whatever
  // the segment sees (rows nv .. there hold other slots)
  __device__ __forceinline__ int filled(const TcParams& p, int r0) const {
    return p.ppt > 0 ? p.kt : min(kBN, p.page - r0);
  }
};

template <int DH>
__device__ __forceinline__ bool store_row32(__nv_bfloat16* o, const float (&v)[32]) {
  bool finite = true;
  uint4* dst = reinterpret_cast<uint4*>(o);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float a = v[8 * c + 2 * x], b = v[8 * c + 2 * x + 1];
      finite = finite && fabsf(a) < INFINITY && fabsf(b) < INFINITY;
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      w[x] = *reinterpret_cast<const uint32_t*>(&h);
    }
    dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return finite;
}

__global__ void chunk_zero_kernel(unsigned int* __restrict__ cnt, int n) {
  grid_dep_wait();
  grid_dep_launch();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) cnt[i] = 0u;
}

// The workspace has two slots a CTA: the first for a piece at the start of its
// stretch, the second for a segment that starts within it and leaves it.  Slot
// of the k-th piece of a segment whose first is in CTA c0, `within` its stretch.
__device__ __forceinline__ int piece_slot(int c0, int k, bool within) {
  return 2 * (c0 + k) + (k == 0 && within ? 1 : 0);
}

// The merge of the pieces (CTAs c0 .. c0 + n - 1, the first `within` its stretch)
// of a warp's rows by the last to arrive: weights 2^(lse - max lse) over their sum.  `rows`: lanes with a
// row; row0: lane 0's row of the segment.  Partials of other CTAs are read past
// L1 (they were released by a fence before their count).
template <int DH>
__device__ __noinline__ bool merge_rows(const TcParams& p, __nv_bfloat16* out, unsigned int rows,
                                        int c0, int n, bool within, int row0) {
  const int lane = threadIdx.x & 31;
  const bool valid = (rows >> lane) & 1u;
  bool finite = true;
  if (__popc(rows) <= kFewRows) {
    // Few rows (single tokens): the warp takes four rows together, lanes over
    // the pieces for the weights, then over the columns, with 16 loads in
    // flight.  Written to be short: this code runs once a launch, and waiting
    // for its instructions took longer than waiting for the pieces (17 pieces:
    // 17k cycles with the weights worked out in every lane, 31k unrolled
    // twice as far).
    constexpr int kCols = DH / 32;  // columns a lane
    constexpr int kR = 4, kK = 4;   // rows and pieces of a step
    using V = typename std::conditional<kCols == 4, float4, float2>::type;
#pragma unroll 1
    for (unsigned int left = rows; left != 0u;) {
      int src[kR];
      float M[kR], sum[kR], acc[kR][kCols];
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        src[i] = left != 0u ? __ffs(left) - 1 : -1;
        left &= left - 1;
        M[i] = -INFINITY;
        sum[i] = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[i][c] = 0.f;
      }
#pragma unroll 1
      for (int k0 = 0; k0 < n; k0 += 32) {
        const float* lse = p.lse_part + (size_t)piece_slot(c0, k0 + lane, within) * kRows + row0;
        float l[kR], mx[kR], w[kR];  // w: this lane's piece
#pragma unroll
        for (int i = 0; i < kR; ++i)
          mx[i] = l[i] = k0 + lane < n && src[i] >= 0 ? __ldcg(lse + src[i]) : -INFINITY;
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < kR; ++i) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          mx[i] = fmaxf(M[i], mx[i]);
          const float corr = M[i] == -INFINITY ? 0.f : ex2_approx(M[i] - mx[i]);
          w[i] = l[i] == -INFINITY ? 0.f : ex2_approx(l[i] - mx[i]);
          M[i] = mx[i];
          sum[i] = sum[i] * corr + w[i];
#pragma unroll
          for (int c = 0; c < kCols; ++c) acc[i][c] *= corr;
        }
        const int cnt = min(32, n - k0);
#pragma unroll 1
        for (int k = 0; k < cnt; k += kK) {
          V x[kK][kR];
#pragma unroll
          for (int d = 0; d < kK; ++d) {
            const size_t slot = piece_slot(c0, k0 + min(k + d, cnt - 1), within);
            const float* v = p.o_part + (slot * kRows + row0) * DH + lane * kCols;  // whole rows
#pragma unroll
            for (int i = 0; i < kR; ++i)
              x[d][i] = __ldcg(reinterpret_cast<const V*>(v + max(src[i], 0) * DH));
          }
#pragma unroll
          for (int d = 0; d < kK; ++d)
#pragma unroll
            for (int i = 0; i < kR; ++i) {
              // a weight of zero adds nothing, whatever the partial holds
              const float wk = __shfl_sync(0xffffffffu, w[i], k + d);
              const float* f = reinterpret_cast<const float*>(&x[d][i]);
#pragma unroll
              for (int c = 0; c < kCols; ++c) acc[i][c] += wk == 0.f ? 0.f : wk * f[c];
            }
        }
      }
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < kR; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const float inv = sum[i] > 0.f ? 1.f / sum[i] : sum[i];
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(__shfl_sync(
            0xffffffffu, reinterpret_cast<unsigned long long>(out), max(src[i], 0)));
        if (src[i] < 0) continue;
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          const float a = acc[i][c] * inv, b = acc[i][c + 1] * inv;
          finite = finite && fabsf(a) < INFINITY && fabsf(b) < INFINITY;
          *reinterpret_cast<__nv_bfloat162*>(dst + lane * kCols + c) = __floats2bfloat162_rn(a, b);
        }
      }
    }
    return finite;
  }
  // a row per lane
  const int row = row0 + lane;
  float M = -INFINITY;
#pragma unroll 4
  for (int k = 0; k < n; ++k)
    M = fmaxf(M, __ldcg(p.lse_part + (size_t)piece_slot(c0, k, within) * kRows + row));
  float sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const float l = __ldcg(p.lse_part + (size_t)piece_slot(c0, k, within) * kRows + row);
    sum += l == -INFINITY ? 0.f : exp2f(l - M);
  }
  const float inv = sum > 0.f ? 1.f / sum : sum;
#pragma unroll 1
  for (int ch = 0; ch < DH / 32; ++ch) {
    float acc[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) acc[c] = 0.f;
    // (20 tokens over 4000 slots, 12 pieces: 32.5 us one piece at a time, 27.4
    // two, 25.3 four; three or fewer pieces are the same in all)
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const size_t slot = piece_slot(c0, k, within);
      const float l = __ldcg(p.lse_part + slot * kRows + row);
      const float4* src = reinterpret_cast<const float4*>(p.o_part) +
                          (slot * kRows + row0) * (DH / 4) + ch * 8 * 32 + lane;
      float4 v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = __ldcg(src + c * 32);
      const float w = l == -INFINITY ? 0.f : exp2f(l - M) * inv;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        acc[4 * c] += w * v[c].x;
        acc[4 * c + 1] += w * v[c].y;
        acc[4 * c + 2] += w * v[c].z;
        acc[4 * c + 3] += w * v[c].w;
      }
    }
    if (valid) finite = store_row32<DH>(out + ch * 32, acc) && finite;
  }
  return finite;
}

// a / b of numbers not below zero (64-bit divisions take several times as long)
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// One warp finds the CTA's stretch of the axis and the first tile that starts
// in it: out = {b, kvh, qg, lt, seg, q0, qlen, kv, end, length of a stretch},
// seg and end from the stretch's start, end 0 when no tile does or a length is
// out of range (reported).  cum (shared memory, B + 1 words): length of the
// sequences before b.
template <int DH>
__device__ __forceinline__ void schedule(const TcParams& p, long long* cum, int* out, int cta,
                                         int grid) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  long long run = 0;
  int q0 = 0, qlen = 0, kv = 0;  // of this lane's sequence
  if (lane == 0) cum[0] = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    qlen = kv = 0;
    if (b < p.B) {
      const int a1 = p.cu_q[b + 1];
      q0 = p.cu_q[b];
      kv = p.kv_len[b];
      qlen = a1 - q0;
      ok = ok && q0 >= 0 && a1 >= q0 && a1 <= p.T && kv >= 0 &&
           kv <= p.max_kv;
    }
    if (!__all_sync(0xffffffffu, ok)) break;
    const int n_qg = (qlen + 2 * p.tpt - 1) / (2 * p.tpt);
    long long n = 0;
    if (n_qg <= 4)
      for (int g = 0; g < n_qg; ++g) n += group_cost(qlen, kv, g, p);
    // long chunks: the lanes share their query groups
    for (unsigned int todo = __ballot_sync(0xffffffffu, n_qg > 4); todo != 0u; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int q = __shfl_sync(0xffffffffu, qlen, src), k = __shfl_sync(0xffffffffu, kv, src);
      const int groups = __shfl_sync(0xffffffffu, n_qg, src);
      long long s = 0;
      for (int g = lane; g < groups; g += 32) s += group_cost(q, k, g, p);
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == src) n = s;
    }
    n *= p.Hkv;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += a;
    }
    n += run;
    if (b < p.B) cum[b + 1] = n;
    run = __shfl_sync(0xffffffffu, n, 31);
  }
  ok = ok && run <= (long long)grid * kMaxStretch;
  __syncwarp();
  if (!__all_sync(0xffffffffu, ok)) {
    if (lane == 0) {
      if (cta == 0) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
      out[8] = 0;
    }
    return;
  }
  const int per = max(kMinCost, static_cast<int>(divide(run + grid - 1, grid)));
  const long long t0 = (long long)cta * per;
  if (t0 >= run) {
    if (lane == 0) out[8] = 0;
    return;
  }
  const int end = static_cast<int>(min((long long)per, run - t0));
  int lo = 0, hi = p.B;  // cum[lo] <= t0 < cum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= t0) lo = mid;
    else hi = mid;
  }
  const long long per_head = divide(cum[lo + 1] - cum[lo], p.Hkv);
  long long rem = t0 - cum[lo];
  int s[8] = {lo, static_cast<int>(divide(rem, per_head)), 0, 0, 0, 0, 0, 0};
  rem -= s[1] * per_head;
  if (p.B <= 32) {
    s[5] = __shfl_sync(0xffffffffu, q0, lo);
    s[6] = __shfl_sync(0xffffffffu, qlen, lo);
    s[7] = __shfl_sync(0xffffffffu, kv, lo);
  } else {
    s[5] = p.cu_q[lo];
    s[6] = p.cu_q[lo + 1] - s[5];
    s[7] = p.kv_len[lo];
  }
  if (s[6] <= 2 * p.tpt) {
    // one query group (single tokens, short chunks)
    const int wt = group_mt(s[6], 0, p) == 2 ? kTwoCost : kOneCost;
    const int in = static_cast<int>(rem);  // t0 within the segment
    s[3] = (in + wt - 1) / wt;
    s[4] = -in;
  } else {
    for (int g0 = 0;; g0 += 32) {
      // beyond the last group the costs only have to be positive
      const int n = group_cost(s[6], s[7], g0 + lane, p);
      long long c = n;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += a;
      }
      const unsigned int over = __ballot_sync(0xffffffffu, c > rem);
      if (over != 0u) {
        const int at = __ffs(over) - 1;
        const int in = static_cast<int>(__shfl_sync(0xffffffffu, rem - (c - n), at));
        const int wt = group_mt(s[6], g0 + at, p) == 2 ? kTwoCost : kOneCost;
        s[2] = g0 + at;
        s[3] = (in + wt - 1) / wt;
        s[4] = -in;
        break;
      }
      rem -= __shfl_sync(0xffffffffu, c, 31);
    }
  }
  Cursor c;
  c.init(s, end, p);
  if (c.lt >= c.ntiles) {
    c.skip(0, p);  // past the last tile: the next segment, if the stretch has one
  } else {
    c.live = c.seg + c.lt * c.wt < end;
  }
  if (lane == 0) {
    out[0] = c.b;
    out[1] = c.kvh;
    out[2] = c.qg;
    out[3] = c.lt;
    out[4] = c.seg;
    out[5] = c.q0;
    out[6] = c.qlen;
    out[7] = c.kv;
    out[8] = c.live ? end : 0;
    out[9] = per;
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, TcParams p) {
  // The launch before this one is always chunk_zero_kernel, which waited for
  // every earlier grid: the inputs are final already.  Only the piece
  // counters it zeroes (and the writes that must follow it) need its
  // completion, so griddepcontrol.wait comes right before those.  Every CTA
  // also waits before it ends, with or without work: the grid after this one
  // is ordered behind this one alone, and may zero or count again.
  grid_dep_launch();
  using L = Smem<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* full = bars;
  uint64_t* empty = bars + L::kRing;
  uint64_t* q_full = bars + 2 * L::kRing;
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 4;  // p_full[2 * m + half]: keys 0-63, 64-127
  uint64_t* q_empty = pv_done + 2;
  uint64_t* half_ready = q_empty + 1;
  uint64_t* half_free = half_ready + 1;
  uint64_t* drain = half_free + 1;
  uint64_t* exit_bar = drain + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  int* info = reinterpret_cast<int*>(smem + L::kMiscOff + 16);  // per ring slot, with each K
  int* start = reinterpret_cast<int*>(smem + L::kStartOff);     // what schedule() finds
  float2* half_ml = reinterpret_cast<float2*>(smem + L::kHalfOff);

  // ---- barriers, tensor memory and (one warp) the CTA's range ----
  if (warp == 1) {
    tmem_alloc(tmem_holder, kTmemCols);
    tmem_relinquish();
  } else if (warp == 2) {
    schedule<DH>(p, reinterpret_cast<long long*>(smem + L::kRingOff), start, blockIdx.x,
                 gridDim.x);
    fence_proxy_async_smem();  // the ring is the copies' from here on
  } else if (tid == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&q_full[m], 1);
      mbar_init(&s_full[m], 1);
      mbar_init(&p_full[2 * m], 128);
      mbar_init(&p_full[2 * m + 1], 128);
      mbar_init(&pv_done[m], 1);
    }
    mbar_init(q_empty, 1);
    mbar_init(half_ready, 128);
    mbar_init(half_free, 128);
    mbar_init(drain, 1);
    mbar_init(exit_bar, kThreads);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  } else if (warp > 2) {
    // No copy writes the Q rows past a short chunk's tokens: cleared once, for
    // products of zeros draw less power (32 single tokens of 32768 slots hold
    // the card at its limit).
    for (int i = tid - 96; i < L::kRingOff / 16; i += kThreads - 96)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (start[8] == 0) {  // no tile is this CTA's
    if (warp == 1) {
      grid_dep_wait();  // (at the other end, too: no grid ends before the counters are zero)
      tmem_dealloc(*tmem_holder, kTmemCols);
    }
    return;
  }
  const int end = start[8], per = start[9];
  if (p.ppt > 0 && p.kt < kBN) {
    // nor any past a full tile's slots (their weights are zero, but 0 * NaN
    // is not)
    for (int i = L::kRingOff / 16 + tid; i < L::kBarOff / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncthreads();
  }
  const uint32_t tmem_base = *tmem_holder;
  const uint32_t tmem_o = tmem_base;           // O[m]: DH columns each
  const uint32_t tmem_s = tmem_base + 2 * DH;  // S[m], then P[m]: 128 columns each

  // 128 x kRegsLow + 256 x kRegsHigh stays within the launch's 384 x 168
  static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168,
                "register split exceeds the launch's allocation");
  if (warp < 4) {
    warpgroup_regs_dec<kRegsLow>();
    if (warp == 0 || warp == 2) {
      // ---------------- TMA producers: K and Q (warp 0), V (warp 2) ----------------
      const bool is_v = warp == 2;
      // K/V that several query groups read stays in L2, the rest passes by
      const uint64_t keep = l2_policy_evict_last(), pass = l2_policy_evict_first();
      Cursor cur;
      cur.init(start, end, p);
      // A tile's page ids (one per lane) are fetched a tile ahead: the read
      // would otherwise hold up the copies of every tile.
      auto page_id = [&](const Cursor& x) {
        int key0, nv, pg, r0;
        x.span(p, key0, nv, pg, r0);
        const int boxes = p.ppt > 0 ? (nv + p.page - 1) / p.page : (nv > 0 ? 1 : 0);
        return lane < boxes ? p.table[(size_t)x.b * p.max_pages + pg + lane] : INT_MIN;
      };
      int next_id = page_id(cur);
      const int panel_rows = p.ppt > 0 ? p.page : kBN;
      const uint32_t box_bytes = static_cast<uint32_t>(panel_rows) * 128u * L::kPanels;
      const uint32_t q_rows = static_cast<uint32_t>(p.G * p.q_box);
      int slot = is_v ? 1 : 0;
      uint32_t phase = 0, n_pieces = 0;
      uint32_t q_loads0 = 0, q_loads1 = 0;
      bool ok = true, bad_page = false;
      int issued = 0;  // copies of this warp's tiles that were started
      Cursor ahead = cur;
      for (; ok && cur.live; cur = ahead) {
        int key0, nv, pg, r0;
        cur.span(p, key0, nv, pg, r0);
        const int id = next_id;
        ahead.advance(p);
        if (ahead.live) next_id = page_id(ahead);
        bool mine = id != INT_MIN;
        if (mine && (id < 0 || id >= p.n_pages)) {
          bad_page = true;
          mine = false;
        }
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * box_bytes;
        if (lane == 0) {
          ok = mbar_wait_bounded(&empty[slot], phase ^ 1u, abort_flag, p.status);
          if (ok) {
            if (!is_v)
              info[slot] = (cur.first ? 1 : 0) | (cur.n_mt > 1 ? 2 : 0) | (cur.last ? 4 : 0) |
                           (ahead.live ? 0 : 8);
            if (bytes > 0) mbar_arrive_expect_tx(&full[slot], bytes);
            else mbar_arrive(&full[slot]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        ++issued;
        if (mine) {
          const uint64_t pol = cur.n_qg > 1 ? keep : pass;
          uint8_t* dst = smem + L::kRingOff + slot * L::kItem + lane * panel_rows * 128;
#pragma unroll
          for (int pn = 0; pn < L::kPanels; ++pn)
            tma_load_4d(dst + pn * L::kPanel, is_v ? &tmV : &tmK, &full[slot], pn * 64, r0, cur.kvh,
                        id, pol);
        }
        if (!is_v && cur.first) {
          // the piece's Q tiles, once the last piece's scores are done: as many
          // boxes as have tokens
          if (lane == 0 && n_pieces > 0)
            ok = mbar_wait_bounded(q_empty, (n_pieces - 1) & 1, abort_flag, p.status);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          for (int m = 0; ok && m < cur.n_mt; ++m) {
            const int t0 = (cur.qg * 2 + m) * p.tpt;  // of the sequence's new tokens
            const int boxes = (min(p.tpt, cur.qlen - t0) + p.q_box - 1) / p.q_box;
            if (lane == 0) mbar_arrive_expect_tx(&q_full[m], boxes * q_rows * 128u * L::kPanels);
            __syncwarp();
            if (lane < boxes) {
              uint8_t* dst = smem + L::kQOff + m * L::kQBytes + lane * q_rows * 128;
#pragma unroll
              for (int pn = 0; pn < L::kPanels; ++pn)
                tma_load_4d(dst + pn * (kMT * 128), &tmQ, &q_full[m], pn * 64, 0, cur.kvh,
                            cur.q0 + t0 + lane * p.q_box, pass);
            }
            if (m == 0) ++q_loads0;
            else ++q_loads1;
          }
          ++n_pieces;
        }
        slot += 2;
        if (slot >= L::kRing) {
          slot -= L::kRing;
          phase ^= 1u;
        }
      }
      if (bad_page) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
      // every copy started has landed before the CTA may end (the copies of
      // slots that were used again have been consumed)
      if (lane == 0) {
        int no_abort = 0;
        for (int x = max(0, issued - L::kRing); x < issued; ++x) {
          const int item = 2 * x + (is_v ? 1 : 0);
          if (item < 2 * issued - L::kRing) continue;
          mbar_wait_bounded(&full[item % L::kRing], (item / L::kRing) & 1, &no_abort, p.status);
        }
        if (q_loads0 > 0) mbar_wait_bounded(&q_full[0], (q_loads0 - 1) & 1, &no_abort, p.status);
        if (q_loads1 > 0) mbar_wait_bounded(&q_full[1], (q_loads1 - 1) & 1, &no_abort, p.status);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- MMA issuer ----------------
      // A unit is one score buffer m on one key tile: both buffers on every
      // tile (two M tiles), or buffers in turn (one).  A buffer's next QK^T
      // follows its PV, so at most two units wait for their softmax, and
      // while one warpgroup computes the tensor core works for the other.
      // The whole warp walks the loop, so that everything an instruction needs
      // stays warp-uniform; one elected lane issues.
      {
        constexpr uint32_t idesc_qk = umma_idesc_bf16(kMT, kBN, 0);
        constexpr uint32_t idesc_pv = umma_idesc_bf16(kMT, DH, 1);
        const uint64_t dq0 = umma_desc_sw128(smem_u32(smem + L::kQOff));
        const uint64_t dk0 = umma_desc_sw128(smem_u32(smem + L::kRingOff));
        const uint64_t dv0 = umma_desc_sw128_lbo(smem_u32(smem + L::kRingOff), L::kPanel, 1024);
        auto issue_qk = [&](int m, int qm, int st, bool q_done) {
          const uint64_t dq = dq0 + (uint64_t)((qm * L::kQBytes) >> 4);
          const uint64_t dk = dk0 + (uint64_t)((st * L::kItem) >> 4);
          const uint32_t d = tmem_s + m * kBN;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
              constexpr uint32_t qpanel = (kMT * 128) >> 4, kpanel = L::kPanel >> 4;
              umma_bf16(d, dq + (kk >> 2) * qpanel + (kk & 3) * 2,
                        dk + (kk >> 2) * kpanel + (kk & 3) * 2, idesc_qk, kk > 0 ? 1u : 0u);
            }
            umma_commit(&s_full[m]);
            if (q_done) umma_commit(&empty[st]);
          }
          __syncwarp();
        };
        // half of a unit's PV: 64 keys
        auto issue_pv = [&](int m, int st, int half, uint32_t acc0, bool v_done) {
          const uint64_t dv = dv0 + (uint64_t)((st * L::kItem + half * 64 * 128) >> 4);
          const uint32_t d = tmem_o + m * DH;
          const uint32_t pcol = tmem_s + m * kBN + half * 32;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              // 16 keys: 8 columns of packed P, two 8-row groups of V
              umma_bf16_ts(d, pcol + kk * 8, dv + (uint64_t)((kk * 16 * 128) >> 4), idesc_pv,
                           kk > 0 ? 1u : acc0);
            if (half == 1) {
              umma_commit(&pv_done[m]);
              if (v_done) umma_commit(&empty[st]);
            }
          }
          __syncwarp();
        };
        // units whose PV is still to come, oldest first: bit 0 buffer, bit 1
        // O starts over, bit 2 last user of the V tile, bits 8.. ring slot,
        // bit 16 its phase
        int pend0 = -1, pend1 = -1;
        uint32_t np = 0, nq = 0;  // parities of the next waits on p_full / q_full, bit m
        auto pop = [&]() -> bool {
          const int u = pend0;
          pend0 = pend1;
          pend1 = -1;
          const int m = u & 1, vs = (u >> 8) & 0xff;
          if (!mbar_wait_bounded(&full[vs], (u >> 16) & 1, abort_flag, p.status) ||
              !mbar_wait_bounded(&p_full[2 * m], (np >> m) & 1u, abort_flag, p.status))
            return false;
          tc_fence_after();
          issue_pv(m, vs, 0, (u & 2) ? 0u : 1u, false);
          if (!mbar_wait_bounded(&p_full[2 * m + 1], (np >> m) & 1u, abort_flag, p.status))
            return false;
          np ^= 1u << m;
          tc_fence_after();
          issue_pv(m, vs, 1, 1u, (u & 4) != 0);
          return true;
        };
        int ks = 0, at = 0;  // ring slot of K, tile of the piece
        uint32_t kph = 0;
        bool ok = true;
        for (bool more = true; ok && more;) {
          int vs = ks + 1;
          uint32_t vph = kph;
          if (vs == L::kRing) {
            vs = 0;
            vph ^= 1u;
          }
          if (pend1 >= 0 && !pop()) break;
          if (!mbar_wait_bounded(&full[ks], kph, abort_flag, p.status)) break;
          const int word = __shfl_sync(0xffffffffu, info[ks], 0);
          const bool first = (word & 1) != 0, two = (word & 2) != 0;
          more = (word & 8) == 0;
          if (first) at = 0;
          for (int m = two ? 0 : at & 1;; ++m) {
            while (ok && ((pend0 >= 0 && (pend0 & 1) == m) || (pend1 >= 0 && (pend1 & 1) == m)))
              ok = pop();
            if (!ok) break;
            const int qm = two ? m : 0;
            if (first) {
              ok = mbar_wait_bounded(&q_full[qm], (nq >> qm) & 1u, abort_flag, p.status);
              if (!ok) break;
              nq ^= 1u << qm;
            }
            tc_fence_after();
            const bool fresh = two ? first : at < 2, done = !two || m == 1;
            issue_qk(m, qm, ks, done);
            const int u = m | (fresh ? 2 : 0) | (done ? 4 : 0) | (vs << 8) | ((int)vph << 16);
            if (pend0 < 0) pend0 = u;
            else pend1 = u;
            if (done) break;
          }
          if (!ok) break;
          if ((word & 4) && elect_one()) umma_commit(q_empty);
          __syncwarp();
          ++at;
          ks = vs + 1;
          kph = vph;
          if (ks == L::kRing) {
            ks = 0;
            kph ^= 1u;
          }
        }
        while (ok && pend0 >= 0) ok = pop();
        if (elect_one()) umma_commit(drain);
        __syncwarp();
        int no_abort = 0;
        mbar_wait_bounded(drain, 0, &no_abort, p.status);
      }
    }
  } else {
    warpgroup_regs_inc<kRegsHigh>();
    // ---------------- softmax warpgroups (M tile 0: warps 4-7, 1: 8-11) ----------------
    const int m = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int rl = quad * 32 + lane;  // row within the M tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t srow = tmem_s + lane_off + m * kBN;
    const int tok_l = rl / p.G, g = rl - tok_l * p.G;  // token of the M tile, head of the group
    uint32_t tcount = 0;  // units of this warpgroup so far
    uint32_t halves = 0;  // one-tile pieces the second warpgroup took part in
    float m_used = -INFINITY, l_run = 0.f;
    int units = 0;  // this warpgroup's units in the piece
    bool finite = true;
    const uint64_t scale2 = f32x2_pack(p.scale_log2, p.scale_log2);

    // One unit's scores to weights: the row's 128 scores come out of TMEM, the
    // maximum and the sum stay in the thread, P goes back packed over the
    // scores in two halves, so the first half's PV starts under the second.
    // kFull: every slot of the tile is visible to every row of the warp;
    // otherwise the row sees the first `limit`.
    auto unit = [&](auto full_tag, int limit) {
      constexpr bool kFull = decltype(full_tag)::value;
      float sv[kBN];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[2][32];
        tmem_ld32_raw(srow + h * 64, r[0]);
        tmem_ld32_raw(srow + h * 64 + 32, r[1]);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tmem_regs_after_wait(r[q]);
#pragma unroll
          for (int c = 0; c < 32; ++c) sv[h * 64 + q * 32 + c] = __uint_as_float(r[q][c]);
        }
      }
      if (!kFull) {
#pragma unroll
        for (int c = 0; c < kBN; ++c)
          if (c >= limit) sv[c] = -INFINITY;
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < kBN; c += 2) m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], sv[c], sv[c + 1]);
      const float mx = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * p.scale_log2;
      // The exponent base is a running maximum that only moves when a tile
      // exceeds it by more than 2^8 (the stale base cancels in O / l).
      const bool need = (m_used == -INFINITY) ? (mx != -INFINITY) : (mx > m_used + kLazy);
      if (__any_sync(0xffffffffu, need)) {
        const float new_m = need ? mx : m_used;
        const float corr = (need && m_used != -INFINITY) ? ex2_approx(m_used - new_m) : 1.f;
        if (units > 0) {
          // O holds earlier units (their PV precedes this unit's QK)
#pragma unroll 1
          for (int ch = 0; ch < DH / 32; ++ch) {
            float o[32];
            const uint32_t ta = tmem_o + lane_off + m * DH + ch * 32;
            tmem_ld32(ta, o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] *= corr;
            tmem_st32(ta, o);
          }
        }
        l_run *= corr;
        m_used = new_m;
      }
      const float nbase = m_used == -INFINITY ? 0.f : -m_used;
      const uint64_t nbase2 = f32x2_pack(nbase, nbase);
      uint64_t part[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          if (h == 1 && e == 8) {
            // the first half's P is in place
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&p_full[2 * m]);
          }
          const int c = h * 64 + 2 * e;
          const uint64_t x2 = f32x2_fma(f32x2_pack(sv[c], sv[c + 1]), scale2, nbase2);
          float x0, x1;
          f32x2_unpack(x2, x0, x1);
          const uint64_t a2 = f32x2_pack(ex2_approx(x0), ex2_approx(x1));
          part[e & 3] = f32x2_add(part[e & 3], a2);
          float a0, a1;
          f32x2_unpack(a2, a0, a1);
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(a0, a1);
          pk[e] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        tmem_st32_u(srow + h * 32, pk);
      }
      float s0, s1;
      f32x2_unpack(f32x2_add(f32x2_add(part[0], part[1]), f32x2_add(part[2], part[3])), s0, s1);
      l_run += s0 + s1;
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[2 * m + 1]);
    };

    // how many leading tiles are 128 consecutive slots from slot 128 lt on
    // (all, unless pages end inside tiles)
    const int even_lt = p.ppt > 0 ? (p.kt == kBN ? INT_MAX : 0)
                                  : (p.page % kBN == 0 ? INT_MAX : p.page / kBN);
    Cursor cur;
    cur.init(start, end, p);
    int j0 = 0;  // tiles before the piece
    bool ok = true;
    while (ok && cur.live) {
      const int piece_lt0 = cur.lt;
      const int piece_n = cur.piece();
      const bool alt = cur.n_mt == 1;
      const int tok = (cur.qg * 2 + (alt ? 0 : m)) * p.tpt + tok_l;
      const bool valid = tok_l < p.tpt && tok < cur.qlen;
      const int row_vis = cur.kv - cur.qlen + tok + 1;  // slots the row sees
      const bool any = __any_sync(0xffffffffu, valid);
      // leading tiles that every row of the warp sees whole; rows of no query
      // take any score
      const int warp_vis = __reduce_min_sync(0xffffffffu, valid ? max(row_vis, 0) : 0x7fffffff);
      const int lt_full = min(warp_vis / kBN, even_lt);
      m_used = -INFINITY;
      l_run = 0.f;
      units = 0;
      for (int x = alt ? m : 0; x < piece_n; x += alt ? 2 : 1) {
        if (!mbar_wait_bounded(&s_full[m], tcount & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the first PV of a piece overwrites O: the second half's of the last
        // one-tile piece must have been read
        if (m == 1 && units == 0 && halves > 0 &&
            !mbar_wait_bounded(half_free, (halves - 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        cur.lt = piece_lt0 + x;
        if (any && cur.lt < lt_full) {
          unit(std::true_type{}, kBN);
        } else {
          int key0, nv, pg, r0;
          cur.span(p, key0, nv, pg, r0);
          if ((alt || m == 0) && nv < cur.filled(p, r0)) {
            // The tile's V rows from nv on belong to no slot of the segment
            // and may hold anything: cleared once they have landed (the
            // tile's PVs are issued after this warpgroup's arrival).
            const int item = 2 * (j0 + x) + 1, vs = item % L::kRing;
            if (!mbar_wait_bounded(&full[vs], (item / L::kRing) & 1, abort_flag, p.status)) {
              ok = false;
              break;
            }
            uint8_t* vt = smem + L::kRingOff + vs * L::kItem;
            for (int row = nv + quad; row < kBN; row += 4) {
              if (lane < 8 * L::kPanels)
                *reinterpret_cast<uint4*>(vt + (lane >> 3) * L::kPanel + row * 128 +
                                          (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          if (any) {
            unit(std::false_type{}, valid ? min(nv, row_vis - key0) : kBN);
          } else {
            // warps without a query row only keep the pipeline going
            tc_fence_before();
            mbar_arrive(&p_full[2 * m]);
            mbar_arrive(&p_full[2 * m + 1]);
          }
        }
        ++tcount;
        ++units;
      }
      if (!ok) break;
      j0 += piece_n;
      cur.lt = piece_lt0;
      const Cursor done = cur;
      cur.skip(piece_n, p);
      if (units == 0) continue;

      // ---- this warpgroup's share of the piece is complete ----
      if (!mbar_wait_bounded(&pv_done[m], (tcount - 1) & 1, abort_flag, p.status)) break;
      tc_fence_after();
      if (alt && m == 1) {
        half_ml[rl] = make_float2(m_used, l_run);
        ++halves;
        tc_fence_before();
        mbar_arrive(half_ready);
        continue;
      }
      grid_dep_wait();  // the results go where the stream order lets them
      float w0 = 1.f, w1 = 0.f;
      const bool both = alt && piece_n > 1;
      if (both) {
        if (!mbar_wait_bounded(half_ready, halves & 1, abort_flag, p.status)) break;
        ++halves;
        tc_fence_after();
        const float2 h = half_ml[rl];
        const float M = fmaxf(m_used, h.x);
        w0 = l_run == 0.f ? 0.f : ex2_approx(m_used - M);
        w1 = h.y == 0.f ? 0.f : ex2_approx(h.x - M);
        l_run = l_run * w0 + h.y * w1;
        m_used = M;
      }
      // an empty row is zero; a NaN sum is no empty row
      const float inv = l_run == 0.f ? 0.f : l_run > 0.f ? 1.f / l_run : l_run;
      w0 *= inv;
      w1 *= inv;
      auto row32 = [&](int ch, float (&o)[32]) {
        tmem_ld32(tmem_o + lane_off + (both ? 0 : m) * DH + ch * 32, o);
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] *= w0;
        if (both) {
          float x[32];
          tmem_ld32(tmem_o + lane_off + DH + ch * 32, x);
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = fmaf(x[c], w1, o[c]);
        }
      };
      __nv_bfloat16* out = p.out + ((size_t)(done.q0 + tok) * p.Hq + done.kvh * p.G + g) * DH;
      if (!any) {
        // nothing to write
      } else if (piece_lt0 == 0 && piece_n == done.ntiles) {
#pragma unroll 1
        for (int ch = 0; ch < DH / 32; ++ch) {
          float o[32];
          row32(ch, o);
          if (valid) finite = store_row32<DH>(out + ch * 32, o) && finite;
        }
      } else {
        // CTAs before this one that hold earlier pieces, and after it
        const int back = done.seg < 0 ? (per - 1 - done.seg) / per : 0;
        const int ahead = (done.seg + (done.ntiles - 1) * done.wt) / per;
        const bool within = done.seg + back * per != 0;
        const int c0 = blockIdx.x - back, n_pieces = back + ahead + 1;
        const size_t slot = piece_slot(c0, back, within);
        const int row = m * kMT + rl;
        // Many rows in a warp: groups of 4 columns of all rows, so that its
        // lanes write 512 bytes side by side.  Few: whole rows, which the
        // merging warp reads 512 bytes at a time.
        const unsigned int mask = __ballot_sync(0xffffffffu, valid);
        const bool few = __popc(mask) <= kFewRows;
        float4* dst = reinterpret_cast<float4*>(p.o_part) +
                      (slot * kRows + row - lane) * (DH / 4) + (few ? lane * (DH / 4) : lane);
        const int step = few ? 1 : 32;
#pragma unroll 1
        for (int ch = 0; ch < DH / 32; ++ch) {
          float o[32];
          row32(ch, o);
          if (valid) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              dst[(ch * 8 + c) * step] =
                  make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        }
        if (valid)
          p.lse_part[slot * kRows + row] =
              l_run > 0.f ? m_used + log2f(l_run) : l_run == 0.f ? -INFINITY : l_run;
        // release this warp's rows, count them in; the last piece merges
        __threadfence();
        __syncwarp();
        unsigned int before = 0u;
        if (lane == 0) before = atomicAdd(&p.piece_count[c0 * 8 + (warp - 4)], 1u);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before == static_cast<unsigned int>(n_pieces - 1)) {
          __threadfence();
          finite = merge_rows<DH>(p, out, mask, c0, n_pieces, within, row - lane) && finite;
        }
      }
      tc_fence_before();
      if (both) mbar_arrive(half_free);
    }
    if (!finite) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
  }

  // TMEM is released once every thread is past its last TMEM access
  tc_fence_before();
  mbar_arrive(exit_bar);
  if (warp == 1) {
    grid_dep_wait();
    __syncwarp();
    int no_abort = 0;
    mbar_wait_bounded(exit_bar, 0, &no_abort, p.status);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <int DH>
medusa_status_t launch_tc(const ChunkParams& c, void* ws, cudaStream_t stream) {
  using L = Smem<DH>;
  TcParams p{};
  p.table = c.table;
  p.cu_q = c.cu_q;
  p.kv_len = c.kv_len;
  p.n_pages = c.n_pages;
  p.page = c.page_size;
  p.max_pages = c.max_pages;
  if (c.page_size >= kBN) {
    p.ppt = 0;
    p.tpp = (c.page_size + kBN - 1) / kBN;
    p.kt = kBN;
  } else {
    // several pages in a tile need whole swizzle atoms of 8 rows
    p.ppt = c.page_size % 8 == 0 ? kBN / c.page_size : 1;
    p.tpp = 1;
    p.kt = p.ppt * c.page_size;
  }
  // (tiles a page: tpp; or ppt pages a tile)
  const long long slots = (long long)c.max_pages * c.page_size;
  const long long most = p.ppt > 0 ? (long long)kMaxTiles * p.kt
                                   : (long long)(kMaxTiles / p.tpp) * c.page_size;
  const long long bound = slots < most ? slots : most;
  p.max_kv = bound < INT_MAX ? static_cast<int>(bound) : INT_MAX;
  p.B = c.B;
  p.T = c.T;
  p.Hq = c.Hq;
  p.Hkv = c.Hkv;
  p.G = c.G;
  p.tpt = kMT / c.G;
  // copies of Q start on whole swizzle atoms of 8 rows
  p.q_box = c.G % 8 == 0 ? 1 : c.G % 4 == 0 ? 2 : c.G % 2 == 0 ? 4 : 8;
  if (p.q_box > p.tpt) p.q_box = p.tpt;  // one copy
  else p.tpt -= p.tpt % p.q_box;
  p.scale_log2 = c.scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(c.out);
  p.status = c.status;
  const int grid = device_sm_count();  // persistent: one CTA per SM
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  const size_t o_bytes = (size_t)2 * grid * kRows * DH * 4, l_bytes = (size_t)2 * grid * kRows * 4;
  p.o_part = reinterpret_cast<float*>(w8);
  p.lse_part = reinterpret_cast<float*>(w8 + o_bytes);
  p.piece_count = reinterpret_cast<unsigned int*>(w8 + o_bytes + l_bytes);

  CUtensorMap mQ, mK, mV;
  // queries as [T][Hkv][G][DH]: boxes of 64 columns x G heads x q_box tokens
  const uint64_t dq[4] = {DH, (uint64_t)c.G, (uint64_t)c.Hkv, (uint64_t)c.T};
  const uint64_t sq[3] = {DH * 2, (uint64_t)c.G * DH * 2,
                          (uint64_t)(c.T > 1 ? c.q_stride : (long long)c.Hq * DH) * 2};
  const uint32_t bq[4] = {64, (uint32_t)c.G, 1, (uint32_t)p.q_box};
  // pools [n_pages][Hkv][page][DH]: boxes of 64 columns x (a page or 128 rows)
  const uint64_t dk[4] = {DH, (uint64_t)c.page_size, (uint64_t)c.Hkv, (uint64_t)c.n_pages};
  const uint64_t sk[3] = {DH * 2, (uint64_t)c.page_size * DH * 2,
                          (uint64_t)c.Hkv * c.page_size * DH * 2};
  const uint32_t bk[4] = {64, (uint32_t)(c.page_size < kBN ? c.page_size : kBN), 1, 1};
  if (!make_tmap_bf16(&mQ, c.q, 4, dq, sq, bq) || !make_tmap_bf16(&mK, c.K, 4, dk, sk, bk) ||
      !make_tmap_bf16(&mV, c.V, 4, dk, sk, bk))
    return fail(MEDUSA_ERR_CUDA, "chunk_attention: cuTensorMapEncodeTiled failed");
  if (cudaFuncSetAttribute(chunk_attn_tc_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           L::kAlloc) != cudaSuccess)
    return fail(MEDUSA_ERR_CUDA, "cudaFuncSetAttribute(chunk_attention) failed");
  // the register shares must fit in what the launch allocates, or the softmax
  // warpgroups' increase would wait for ever
  static const int regs = [] {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, chunk_attn_tc_kernel<DH>) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (128 * kRegsLow + 256 * kRegsHigh > kThreads * regs)
    return fail(MEDUSA_ERR_UNSUPPORTED, "chunk_attention: register split exceeds the build's");
  launch(chunk_zero_kernel, 1, 1024, 0, stream, p.piece_count, grid * 8);
  const medusa_status_t st = check_launch("chunk_attention_counters");
  if (st != MEDUSA_OK) return st;
  launch(chunk_attn_tc_kernel<DH>, grid, kThreads, L::kAlloc, stream, mQ, mK, mV, p);
  return check_launch("chunk_attention");
}

}  // namespace

size_t chunk_attention_tc_workspace(int dh) {
  const size_t grid = device_sm_count();
  return align256(2 * grid * kRows * dh * 4 + 2 * grid * kRows * 4 + grid * 8 * 4);
}

medusa_status_t chunk_attention_tc(const ChunkParams& p, int dh, void* ws, cudaStream_t stream) {
  if (dh == 128) return launch_tc<128>(p, ws, stream);
  return launch_tc<64>(p, ws, stream);
}

}  // namespace medusa
