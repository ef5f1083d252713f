// Tokens drawn from filtered logits: temperature, top-k, top-p and min-p with
// the caller's uniform numbers.
//
// Every filter keeps a prefix of the row's tokens in the order (logit
// descending, id ascending), so the kept set is a cut: a key (the logit as an
// ordered integer) and the last id that stays among the tokens with exactly
// that key.  The cut is found by selection, never by sorting the row.
//
// bf16: few values occur more than once each, so the tokens are counted by
// value in one pass, and the 4096 values' weights stand for the tokens'.  The
// bound falls on a value; how many of its tokens stay is a division.
//
// fp32 (and the rare bf16 row whose cut lies among its smallest magnitudes):
//   - the top tokens first: those at or above a bound that the threads' maxima
//     give go on a short list.  It holds the cut of a top_k of up to 256, and
//     of most top_p; a row that looks too flat for it is not tried.
//   - otherwise a histogram of the row over 2048 bins of falling logit: counts
//     for top-k, mass for top-p; the bin where the count reaches top_k, or the
//     mass before it reaches top_p of the total, goes on the list, or, too full
//     for it, is split by a histogram over its own keys until it is short or
//     one key is left.
//   - on the list, the 256th of its range that holds the cut until at most 128
//     tokens are left, which are ranked against one another.
// min-p is a bound on the logit and needs no selection.
//
// Masses are exact: w = exp((z - max) / T) is rounded once to 64-bit fixed
// point (units of 2^-42 of the largest weight, which is 1), and integers add
// up the same in any order, so a draw is the same however the row is split
// and a token is decided as in a 64-bit sum up to 2^-42 per token.  A fp32 sum
// over a vocabulary of 128256 decides one draw in about a hundred differently.
//
// A row belongs to a cluster of thread blocks that hold it in shared memory:
// it is read from HBM once, and every later pass runs on the copy.  What the
// blocks tell one another they push into every block's shared memory before a
// cluster barrier and then evaluate redundantly, so a step costs one barrier
// and no broadcast: extremes; group sums of the histogram; the short list;
// kept masses.
//
// Bound by latency: few rows by the chain of three or four cluster barriers
// with a pass between them, many rows by the same chain two blocks at a time
// on an SM and by the shared-memory atomics of the count (about six cycles a
// warp's; computing the bins with half the instructions changed nothing).  One
// row of 32000 (fp32, top-k and top-p) 12 to 18 us, as its list serves at once
// or not; 8 rows of 128256 (bf16, top-p) 16.7 us; 512 of them with settings of
// their own 156 us, 0.84 TB/s.  With the weights of all tokens added into bins,
// as in fp32, the bf16 rows took 44 and 269 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_internal.h"
#include "common.cuh"

namespace cg = cooperative_groups;

namespace medusa {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kGroups = kBins / 32;
constexpr int kList = 1024;  // tokens on the short list, kList / cluster from each block
constexpr int kMaxCluster = 8;
// The largest top_k whose tokens are listed; for top_p alone half as many are
// looked for (the list has room for a few times as many).
constexpr int kTopWanted = 256;
constexpr int kRank = 128;  // tokens of a list that are ranked against one another
// Bytes of a row in a block when there are many rows: a block's barriers cost
// the same whatever its share (512 rows of 128256 bf16: 168 us, with half as
// much 251), and two of this size fit on an SM.
constexpr size_t kManyBytes = 65536;
constexpr int kValues = 4096;  // bins of bf16 logits: 16 octaves of magnitude and a sign
constexpr int kSubs = 4;       // parts of a block's tokens, each with its own counts
constexpr int kExpTable = 256;
constexpr float kMaxTemperature = 1e30f;  // 32 T must stay finite
constexpr uint32_t kLowestKey = 0x00800000u;  // key of the lowest finite float

struct SampleParams {
  const void* logits;
  long long row_stride;
  const int32_t* row_idx;
  int n_rows, R, V, slice;  // slice: elements per block of the cluster
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t *tokens, *kept, *status;
};

// order-preserving integer of a float; -0 counts as +0
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// the largest float below those of key k (-0 has the key of +0)
__device__ __forceinline__ float value_below(uint32_t k) {
  return value_of(k == 0x80000000u ? k - 2u : k - 1u);
}

// A finite float as a double by its bits; zero and subnormals become values
// of that size (below 2^-126), which no logit difference notices.
__device__ __forceinline__ double widen(float z) {
  const int b = __float_as_int(z);
  return __hiloint2double(((b >> 3) & static_cast<int>(0x8fffffffu)) + 0x38000000, b << 29);
}

// NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The row is handled four tokens at a time: a Quad is what holds them.
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  using Quad = uint4;
  static constexpr uint32_t kNegInf = 0xff800000u;  // filler word
  __device__ static void unpack(Quad r, float (&z)[4]) {
    z[0] = __uint_as_float(r.x);
    z[1] = __uint_as_float(r.y);
    z[2] = __uint_as_float(r.z);
    z[3] = __uint_as_float(r.w);
  }
  __device__ static float max_of(Quad r) {
    return max_nan(max_nan(__uint_as_float(r.x), __uint_as_float(r.y)),
                   max_nan(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
  __device__ static float max_of16(uint4 r) { return max_of(r); }
};
template <>
struct Elem<__nv_bfloat16> {
  using Quad = uint2;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  __device__ static void unpack(Quad r, float (&z)[4]) {
    z[0] = __uint_as_float(r.x << 16);
    z[1] = __uint_as_float(r.x & 0xffff0000u);
    z[2] = __uint_as_float(r.y << 16);
    z[3] = __uint_as_float(r.y & 0xffff0000u);
  }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {  // pairs
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ static float max_of_pair(uint32_t m) {
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  __device__ static float max_of(Quad r) { return max_of_pair(max2(r.x, r.y)); }
  __device__ static float max_of16(uint4 r) {
    return max_of_pair(max2(max2(r.x, r.y), max2(r.z, r.w)));
  }
};

// The weight exp((z - max) / T) in units of 2^-42: 2^y with y = (z - max) *
// log2(e) / T split as y = n + j / 256 + r / 256, |r| <= 1/2: a table of
// 2^(j / 256) and the Taylor polynomial of 2^(r / 256) to the third power
// (the fourth term is below 2^-42).  Nine fp64 operations, a table read and
// ten integer ones; the rounding to an integer is the addition of 1.5 * 2^10,
// whose last bit is 2^-42.  Logits are held to `floor` (y = -46) first, where
// the weight rounds to nothing.
struct Weight {
  const double* table;
  double zmax, c;  // c: 256 * log2(e) / T
  float floor;

  __device__ __forceinline__ unsigned long long operator()(float z) const {
    constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52
    constexpr double kRound = 1536.0;              // 1.5 * 2^10: its low word is zero
    constexpr double kL = 2.7076061740622863e-3;   // ln 2 / 256
    const double dz = widen(fmaxf(z, floor)) - zmax;
    const double kd = fma(dz, c, kMagic);
    const int k = __double2loint(kd);
    const double r = fma(dz, c, -(kd - kMagic));
    const double t = table[k & (kExpTable - 1)];
    const double q = fma(fma(kL * kL * kL / 6.0, r, kL * kL / 2.0), r, kL);
    double v = fma(t * r, q, t);
    v = __hiloint2double(__double2hiint(v) + (k & -kExpTable) * (1 << 12), __double2loint(v)) +
        kRound;
    return (static_cast<unsigned long long>(
                static_cast<uint32_t>(__double2hiint(v) - __double2hiint(kRound)))
            << 32) |
           static_cast<uint32_t>(__double2loint(v));
  }
};

// what a block tells the others of its cluster
struct Sums {
  unsigned long long mass;
  unsigned int count;
  int first;  // draw: lowest kept id
};
struct Bin {
  unsigned long long mass;  // before it
  unsigned long long limit;
  unsigned int count;
  uint32_t bin;
};
struct Cut {
  unsigned long long mass;  // of the tokens that stay
  uint32_t key;             // of the last of them
  int id;
};

// the cut among bf16 values
struct ValueCut {
  unsigned long long mass;  // of the tokens that stay
  unsigned int count;       // of them
  uint32_t bin;             // of the last
  unsigned int ties;        // tokens of that value that stay,
  unsigned int before;      // ... of them in the blocks before owner, whose tokens
  int owner;                // of that value are the first that do not all stay
};

struct Shared {
  float hi[kMaxCluster];    // largest logit (NaN: there is one)
  float edge[kMaxCluster];  // a bound below the block's share of the top tokens
  Sums part[kMaxCluster];
  unsigned long long list_mass[kMaxCluster];  // weights of every token of the block
  unsigned int list_n[kMaxCluster];           // tokens the block lists
  uint32_t kmin[kMaxCluster], kmax[kMaxCluster];
  double table[kExpTable];
  unsigned long long word[kRank], word_w[kRank];  // the last words of a list, their weights
  uint32_t cnt[256], lo[256], high[256];          // narrowing a list
  Bin bin;
  Cut cut;
  ValueCut value_cut;
  unsigned int tiny[2][kSubs];  // bf16: weights of the tokens near zero (low, high words)
  unsigned int far;             // finite tokens without weight or bin
  int tie_sub;                  // the part with the last token of the cut's value that stays
  unsigned int tie_n;           // how many of its tokens of that value do
  unsigned int n_local;
  int cut_id, n_th;
  unsigned long long red64[kWarps], red64b[kWarps];
  unsigned int red32[kWarps], red32b[kWarps];
  float redf[kWarps];
  float2 share[kWarps], shares[kMaxCluster];  // mass above and below the edge, a guess
};

// dynamic shared memory after the slice: histogram (counts, low and high words
// of the mass), short lists and group sums of every block
__host__ __device__ constexpr size_t sample_extra_smem(int C) {
  static_assert(3 * kBins * 4 + kList * 8 >= 2 * kValues * 4, "counts of bf16 values");
  return 3 * kBins * 4 + kList * 8 + (size_t)C * kGroups * sizeof(Sums);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_tokens_kernel(SampleParams p) {
  constexpr int VE = 16 / sizeof(T);  // tokens of a 16-byte vector
  using Quad = typename Elem<T>::Quad;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int r = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  extern __shared__ __align__(16) uint8_t dyn[];
  uint4* slice = reinterpret_cast<uint4*>(dyn);
  const Quad* quads = reinterpret_cast<const Quad*>(dyn);
  const int n_vec = p.slice / VE, n_quad = p.slice / 4;
  // this block's histogram of its slice: counts, low and high words of the mass
  uint32_t* h_cnt = reinterpret_cast<uint32_t*>(dyn + (size_t)n_vec * 16);
  uint32_t* h_lo = h_cnt + kBins;
  uint32_t* h_hi = h_lo + kBins;
  // the short lists: words of key and complemented id, cap from each block
  unsigned long long* list = reinterpret_cast<unsigned long long*>(h_hi + kBins);
  Sums* group = reinterpret_cast<Sums*>(list + kList);
  const int cap = kList / C;
  __shared__ Shared sh;

  // the cluster's blocks must all run before one writes to another's memory:
  // the wait is at the first such write
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // what needs no input, while an earlier kernel ends: the table of powers,
  // cleared counts
  if (tid < kExpTable) sh.table[tid] = exp2((double)tid / kExpTable);
  if constexpr (sizeof(T) == 2) {
    for (int i = tid; i < 2 * kValues / 4; i += kThreads)
      reinterpret_cast<uint4*>(h_cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < 2 * kSubs) sh.tiny[tid / kSubs][tid % kSubs] = 0u;
    if (tid == 0) sh.far = 0u;
  }
  grid_dep_wait();
  grid_dep_launch();

  const float temp = p.temperature != nullptr ? p.temperature[r] : 1.f;
  const float u = p.u[r];
  const int top_k = p.top_k != nullptr ? p.top_k[r] : 0;
  const float top_p = p.top_p != nullptr ? p.top_p[r] : 1.f;
  const float min_p = p.min_p != nullptr ? p.min_p[r] : 0.f;
  const int src_row = p.row_idx != nullptr ? p.row_idx[r] : r;
  bool bad = !(u >= 0.f && u < 1.f) || !(temp >= 0.f) || !(top_p >= 0.f) ||
             !(min_p >= 0.f && min_p <= 1.f) || src_row < 0 || src_row >= p.n_rows || temp > kMaxTemperature;

  // ---- the slice into shared memory; its largest logit ----
  // Blocks split the row at 16-byte boundaries of its address: element i of
  // the split is token i - off.
  float hi = -INFINITY;
  int base = 0;
  if (!bad) {
    const T* row = static_cast<const T*>(p.logits) + (size_t)src_row * p.row_stride;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % VE);
    base = rank * p.slice - off;  // token id of the slice's first element
    constexpr int kFetch = 4;     // vectors a thread has in flight
    for (int v0 = tid; v0 < n_vec; v0 += kFetch * kThreads) {
      uint4 raw[kFetch];
#pragma unroll
      for (int f = 0; f < kFetch; ++f) {
        const int v = v0 + f * kThreads, id = base + v * VE;
        raw[f] = make_uint4(Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf);
        if (v < n_vec) {
          if (id >= 0 && id + VE <= p.V) {
            raw[f] = __ldg(reinterpret_cast<const uint4*>(row + id));
          } else {
            uint32_t w[4] = {raw[f].x, raw[f].y, raw[f].z, raw[f].w};
#pragma unroll
            for (int i = 0; i < VE; ++i) {
              if (id + i >= 0 && id + i < p.V) {
                if (sizeof(T) == 4) {
                  w[i % 4] = reinterpret_cast<const uint32_t*>(row)[id + i];
                } else {
                  const uint32_t x = reinterpret_cast<const uint16_t*>(row)[id + i];
                  w[(i / 2) % 4] = (i & 1) ? (w[(i / 2) % 4] & 0xffffu) | (x << 16)
                                           : (w[(i / 2) % 4] & 0xffff0000u) | x;
                }
              }
            }
            raw[f] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
#pragma unroll
      for (int f = 0; f < kFetch; ++f) {
        const int v = v0 + f * kThreads;
        if (v >= n_vec) break;
        slice[v] = raw[f];
        hi = max_nan(hi, Elem<T>::max_of16(raw[f]));
      }
    }
  }
  const float own_hi = hi;  // the largest of this thread's tokens
  for (int o = 16; o > 0; o >>= 1)
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  if (lane == 0) sh.redf[warp] = hi;
  __syncthreads();
  // The share-th largest of the block's threads' largest, to its top 16 bits
  // (found bit by bit): with every block's, at least `want` tokens
  // of the row lie at or above the least of them, and not many more.
  const bool by_k = top_k > 1 && top_k < p.V;
  const bool by_p = top_p < 1.f;
  const bool top_list = sizeof(T) == 4 && (by_k ? top_k <= kTopWanted : by_p);
  float edge = -INFINITY;
  if (top_list) {
    const int want = by_k ? top_k : kTopWanted / 2;
    const int share = (want + C - 1) / C;
    const bool some = own_hi > -INFINITY;
    const uint32_t own = some ? key_of(own_hi) : 0u;
    const uint32_t low = __reduce_min_sync(0xffffffffu, some ? own : 0xffffffffu);
    const uint32_t high = __reduce_max_sync(0xffffffffu, own);
    if (lane == 0) {
      sh.red32[warp] = low;
      sh.red32b[warp] = high;
    }
    const bool enough = __syncthreads_count(some) >= share;
    const uint32_t k0 = __reduce_min_sync(0xffffffffu, sh.red32[lane % kWarps]);
    const uint32_t k1 = __reduce_max_sync(0xffffffffu, sh.red32b[lane % kWarps]);
    // (their common leading bits need no search)
    uint32_t bit = k0 < k1 ? 0x80000000u >> __clz(static_cast<int>(k0 ^ k1)) : 0u;
    uint32_t k = bit > 0u ? k0 & ~(2u * bit - 1u) : k0;
#pragma unroll 1
    for (; bit >= 0x10000u; bit >>= 1)
      if (__syncthreads_count(some && own >= (k | bit)) >= share) k |= bit;
    if (enough) edge = value_of(k);
    if (!by_k) {
      // What share of the mass lies above the edge: the threads' largest there
      // against one of their quads, for all, below it.  (A guess, by which a
      // flat row's list is not tried.)
      const float c = 1.442695f / temp;
      float z[4], above = 0.f, rest = 0.f;
      const Quad raw = tid < n_quad ? quads[tid] : Quad{};
      Elem<T>::unpack(raw, z);
      if (own_hi > edge) above = exp2f((own_hi - hi) * c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (tid < n_quad && z[i] > -INFINITY && !(z[i] > edge)) rest += exp2f((z[i] - hi) * c);
      for (int o = 16; o > 0; o >>= 1) {
        above += __shfl_xor_sync(0xffffffffu, above, o);
        rest += __shfl_xor_sync(0xffffffffu, rest, o);
      }
      if (lane == 0) sh.share[warp] = make_float2(above, rest * max(1.f, (float)n_quad / kThreads));
      __syncthreads();
    }
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (tid < C) {
    hi = sh.redf[0];
    for (int w = 1; w < kWarps; ++w) hi = max_nan(hi, sh.redf[w]);
    *cluster.map_shared_rank(&sh.hi[rank], tid) = hi;
    *cluster.map_shared_rank(&sh.edge[rank], tid) = edge;
    if (top_list && !by_k) {
      float2 t = make_float2(0.f, 0.f);
      for (int w = 0; w < kWarps; ++w) {
        if (!(sh.redf[w] > -INFINITY)) continue;
        const float x = exp2f((sh.redf[w] - hi) * (1.442695f / temp));
        t.x += x * sh.share[w].x;
        t.y += x * sh.share[w].y;
      }
      *cluster.map_shared_rank(&sh.shares[rank], tid) = t;
    }
  }
  cluster.sync();
  hi = sh.hi[0];
  edge = sh.edge[0];
  for (int c = 1; c < C; ++c) {
    hi = max_nan(hi, sh.hi[c]);
    edge = fminf(edge, sh.edge[c]);
  }
  if (!(hi > -INFINITY && hi < INFINITY)) bad = true;  // NaN, +inf, or no finite logit
  if (bad) {
    if (rank == 0 && tid == 0) {
      report(p.status, MEDUSA_ERR_DEVICE_CHECK);
      p.tokens[r] = -1;
      if (p.kept != nullptr) p.kept[r] = 0;
    }
    return;  // the whole cluster takes this branch, after its last exchange
  }
  if (temp == 0.f || top_k == 1) {
    // the lowest id of the largest
    int first = 0x7fffffff;
    for (int v = tid; v < n_quad; v += kThreads) {
      const Quad raw = quads[v];
      if (Elem<T>::max_of(raw) < hi) continue;
      float z[4];
      Elem<T>::unpack(raw, z);
#pragma unroll
      for (int i = 3; i >= 0; --i)
        if (z[i] == hi) first = min(first, base + v * 4 + i);
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.red32[warp] = static_cast<unsigned int>(first);
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kWarps; ++w) first = min(first, static_cast<int>(sh.red32[w]));
      cluster.map_shared_rank(&sh.part[rank], 0)->first = first;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
      for (int c = 0; c < C; ++c) first = min(first, sh.part[c].first);
      p.tokens[r] = first;
      if (p.kept != nullptr) p.kept[r] = 1;
    }
    return;
  }

  // Exponents are bounded on both sides: logits are held to y = -46, and a T
  // far below the distance to the next float under the largest counts as a
  // 64th of it (every other weight is zero either way).  With the lowest
  // float for the largest, T means nothing.
  const float next = value_below(key_of(hi));
  const double zmax = widen(hi);
  const double t_eff =
      fmax(key_of(hi) == kLowestKey ? 1.0 : (double)temp, (zmax - widen(next)) / 64.0);
  const Weight weight{sh.table, zmax, 1.4426950408889634074 / t_eff * kExpTable,
                      fminf(hi - 32.f * temp, next)};
  // bins of level 0: linear in the logit over 16 T below the largest (weights
  // down to 1e-7), the rest of the row in the last
  const float bin_scale = fminf((float)(kBins - 1) / (16.f * temp), 1e30f);
  // (rounded to an integer by the addition of 2^23)
  auto bin0 = [&](float z) -> uint32_t {
    return __float_as_uint(fminf((hi - z) * bin_scale, (float)(kBins - 1)) + 8388608.f) -
           0x4b000000u;
  };
  // The tokens that a bound keeps end in a stretch of the order that is
  // narrowed step by step: all of the row (kTop lists its top tokens, kRow puts
  // them in bins), a bin (kIn lists it), and for a bin too full to be listed a
  // finer histogram of its keys (kRange), until a list holds the stretch.
  enum Stage { kTop, kRow, kIn, kRange };
  int stage = top_list ? kTop : kRow;
  if (top_list && !by_k) {
    float some = 0.f, rest = 0.f;
    for (int c = 0; c < C; ++c) {
      if (!(sh.hi[c] > -INFINITY)) continue;
      const float x = exp2f((sh.hi[c] - hi) * (1.442695f / temp));
      some += x * sh.shares[c].x;
      rest += x * sh.shares[c].y;
    }
    if (some < top_p * (some + rest)) stage = kRow;
  }
  bool by_mass = !by_k;  // the bound looked for; top_k's first
  unsigned long long limit = by_k ? (unsigned long long)top_k : 0ull;  // 0: top_p of the row
  Bin b{0ull, 0ull, 0u, 0u};  // what lies before the stretch
  float below = edge > -INFINITY ? value_below(key_of(edge)) : edge, top = hi;
  int only = -1;                  // the bin of level 0, if the stretch is one
  uint32_t kmin = 0u, kmax = 0u;  // kRange: keys of the stretch, and its bins
  int shift = 0;
  auto within = [&](float z) {
    return z > below && z <= top && (only < 0 || bin0(z) == static_cast<uint32_t>(only));
  };

  // where tokens go by id, warps take contiguous runs of the quads [q0, q1),
  // 32 at a time
  int v_begin, v_end, run;  // run: rows of 32 quads of a warp to a lane
  auto span_of = [&](int q0, int q1) {
    const int seg = (q1 - q0 + kWarps * 32 - 1) / (kWarps * 32) * 32;
    v_begin = min(q1, q0 + warp * seg);
    v_end = min(q1, v_begin + seg);
    run = (seg / 32 + 31) / 32;
  };
  span_of(0, n_quad);

  auto p_limit = [&](unsigned long long total) {
    // kept while the mass before is below top_p * total: an integer limit
    return max(1ull, static_cast<unsigned long long>(ceil((double)top_p * (double)total)));
  };
  // a warp's sum, and the block's from the warps'
  auto warp_sum = [&](unsigned long long m) {
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    return m;
  };
  auto block_sum = [&](const unsigned long long* red) {
    unsigned long long m = 0ull;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) m += red[w];
    return m;
  };

  // inclusive sums over the lanes of a warp
  auto scan = [&](unsigned long long& m, unsigned int& n) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long a = __shfl_up_sync(0xffffffffu, m, o);
      const unsigned int c = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) {
        m += a;
        n += c;
      }
    }
  };

  // The id of the n-th of this block's tokens with logit z (there are as many).
  // Ids rise with the quads' index, of which warps take contiguous runs.
  auto nth_of = [&](float z, unsigned int n) -> int {
    auto count = [&](int v) {
      unsigned int c = 0u;  // one bit per token with the logit
      if (v < v_end) {
        float x[4];
        Elem<T>::unpack(quads[v], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) c |= x[i] == z ? 1u << i : 0u;
      }
      return c;
    };
    unsigned int mine = 0u, before = 0u;
#pragma unroll 4
    for (int v = v_begin + lane; v < v_end; v += 32) mine += __popc(count(v));
    const unsigned int c = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) sh.red32[warp] = c;
    __syncthreads();
#pragma unroll 1
    for (int x = 0; x < warp; ++x) before += sh.red32[x];
    if (before < n && before + c >= n) {
#pragma unroll 1
      for (int vv = v_begin; before < n && vv < v_end; vv += 32) {
        const unsigned int bits = count(vv + lane), x = __popc(bits);
        const unsigned int all = __reduce_add_sync(0xffffffffu, x);
        if (before + all < n) {
          before += all;
          continue;
        }
        unsigned long long none = 0ull;
        unsigned int s = x;
        scan(none, s);
        const unsigned int at = before + s - x;
        if (at < n && at + x >= n) {
          unsigned int left = bits;
          for (unsigned int y = at + 1; y < n; ++y) left &= left - 1;
          sh.n_th = base + (vv + lane) * 4 + __ffs(left) - 1;
        }
        before += all;
      }
    }
    __syncthreads();
    return sh.n_th;
  };

  // ---- pieces of the draw ----
  // larger keys stay, and ids up to cut_id of this one
  uint32_t cut_key = kLowestKey;
  int cut_id = 0x7fffffff;
  auto take = [&](const Cut& c) {
    if (c.key > cut_key || (c.key == cut_key && c.id < cut_id)) {
      cut_key = c.key;
      cut_id = c.id;
    }
  };
  // min_p, w >= min_p: a bound on the logit, rounded up to a float
  auto take_min_p = [&]() {
    if (!(min_p > 0.f)) return;
    const float z_min = __double2float_ru((double)hi + log((double)min_p) * (double)temp);
    if (z_min > -INFINITY && key_of(z_min) > cut_key) {
      cut_key = key_of(z_min);
      cut_id = 0x7fffffff;
    }
  };
  auto stays = [&](float z, int id) {
    const float cut_z = value_of(cut_key);
    return z > cut_z || (z == cut_z && id <= cut_id);
  };
  // four independent weights, then the ones that stay
  auto weights = [&](const float (&z)[4], const bool (&in)[4], unsigned long long (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = weight(z[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = in[i] ? w[i] : 0ull;
  };
  // This warp's tokens that stay, by their weights.  Their mass goes to `mine`
  // by runs of `run` rows of 32 quads, a lane for each.
  unsigned long long mine = 0ull;
  auto kept_of = [&]() -> Sums {
    mine = 0ull;
    unsigned int count = 0u;
    int first = 0x7fffffff;
    int turn = 0, lot = 0;
#pragma unroll 2
    for (int v0 = v_begin; v0 < v_end; v0 += 32) {
      const int v = v0 + lane;
      unsigned long long mass = 0ull;
      const Quad raw = quads[min(v, n_quad - 1)];
      if (v < v_end && Elem<T>::max_of(raw) >= value_of(cut_key)) {
        float z[4];
        Elem<T>::unpack(raw, z);
        bool in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) in[i] = stays(z[i], base + v * 4 + i);
        if (in[0] || in[1] || in[2] || in[3]) {
          unsigned long long w[4];
          weights(z, in, w);
          mass = (w[0] + w[1]) + (w[2] + w[3]);
#pragma unroll
          for (int i = 3; i >= 0; --i) {
            if (in[i]) {
              ++count;
              first = min(first, base + v * 4 + i);
            }
          }
        }
      }
      // below 2^45 a lane: the sum of 32 by 24 bits
      const unsigned int lo = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(mass) & 0xffffffu);
      const unsigned int up = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(mass >> 24));
      if (lane == lot) mine += (static_cast<unsigned long long>(up) << 24) + lo;
      if (++turn == run) {
        turn = 0;
        ++lot;
      }
    }
    return Sums{warp_sum(mine), __reduce_add_sync(0xffffffffu, count),
                __reduce_min_sync(0xffffffffu, first)};
  };
  // the warps' sums, and with them the block's to every block
  auto exchange = [&](const Sums& t) {
    if (lane == 0) {
      sh.red64[warp] = t.mass;
      sh.red32[warp] = t.count;
      sh.red32b[warp] = static_cast<unsigned int>(t.first);
    }
    __syncthreads();
    if (tid < C) {
      Sums t{0ull, 0u, 0x7fffffff};
#pragma unroll 4
      for (int w = 0; w < kWarps; ++w) {
        t.mass += sh.red64[w];
        t.count += sh.red32[w];
        t.first = min(t.first, static_cast<int>(sh.red32b[w]));
      }
      *cluster.map_shared_rank(&sh.part[rank], tid) = t;
    }
    cluster.sync();
  };
  // the row's, and the mass in the blocks before this one
  auto total_of = [&](unsigned long long& before) -> Sums {
    Sums t{0ull, 0u, 0x7fffffff};
#pragma unroll 1
    for (int c = 0; c < C; ++c) {
      if (c == rank) before = t.mass;
      t.mass += sh.part[c].mass;
      t.count += sh.part[c].count;
      t.first = min(t.first, sh.part[c].first);
    }
    return t;
  };
  auto target_of = [&](unsigned long long total) {
    return min(static_cast<unsigned long long>((double)u * (double)total), total - 1);
  };
  // the token that holds the target, if this warp has it: `before` is the mass
  // in front of the block, sh.red64 the warps'
  auto pick = [&](unsigned long long target, unsigned long long before) {
#pragma unroll 1
    for (int w = 0; w < warp; ++w) before += sh.red64[w];
    if (target < before || target >= before + sh.red64[warp]) return;
    // the run that holds it
    unsigned long long s = mine;
    unsigned int none = 0u;
    scan(s, none);
    const int lot = __ffs(__ballot_sync(0xffffffffu, target < before + s)) - 1;
    before += __shfl_sync(0xffffffffu, s - mine, lot);
    const int from = v_begin + lot * run * 32, to = min(v_end, from + run * 32);
#pragma unroll 1
    for (int v0 = from; v0 < to && target >= before; v0 += 32) {
      const int v = v0 + lane;
      unsigned long long w[4] = {0ull, 0ull, 0ull, 0ull};
      if (v < to) {
        float z[4];
        bool in[4];
        Elem<T>::unpack(quads[v], z);
#pragma unroll
        for (int i = 0; i < 4; ++i) in[i] = stays(z[i], base + v * 4 + i);
        weights(z, in, w);
      }
      const unsigned long long n = (w[0] + w[1]) + (w[2] + w[3]);
      unsigned long long s = n;
      scan(s, none);
      unsigned long long at = before + s - n;
      if (target >= at && target < at + n) {
        int id = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (id < 0 && target < at + w[i]) id = base + v * 4 + i;
          at += w[i];
        }
        p.tokens[r] = id;
      }
      before += __shfl_sync(0xffffffffu, s, 31);
    }
  };

  // The group of bins that a bound falls in: the last with tokens before which
  // the count (or the mass) is below the limit, of the given start.  In mass
  // mode limit 0 stands for top_p of the histogram's own total; kGroups if a
  // count limit is above the total.  One warp.
  auto find_group = [&](bool by_mass, Bin b) -> Bin {
    static_assert(kGroups == 64, "two groups per lane");
    Sums s[2];
    for (int x = 0; x < 2; ++x) {
      s[x] = Sums{0ull, 0u, 0};
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        if (c >= C) break;
        const Sums t = group[c * kGroups + 2 * lane + x];
        s[x].mass += t.mass;
        s[x].count += t.count;
      }
    }
    // exclusive prefix over the lanes
    unsigned long long m = s[0].mass + s[1].mass;
    unsigned int n = s[0].count + s[1].count;
    const unsigned long long own_m = m;
    const unsigned int own_n = n;
    scan(m, n);
    if (b.limit == 0ull) b.limit = p_limit(__shfl_sync(0xffffffffu, m, 31));
    if (!by_mass && b.limit > b.count + __shfl_sync(0xffffffffu, n, 31))
      return Bin{0ull, b.limit, 0u, kGroups};
    m += b.mass - own_m;
    n += b.count - own_n;
    // this lane's later qualifying group, if any
    Bin g{0ull, b.limit, 0u, 0u};
    bool some = false;
    for (int x = 0; x < 2; ++x) {
      if ((by_mass ? s[x].mass > 0ull : s[x].count > 0u) &&
          (by_mass ? m : (unsigned long long)n) < b.limit) {
        some = true;
        g = Bin{m, b.limit, n, static_cast<uint32_t>(2 * lane + x)};
      }
      m += s[x].mass;
      n += s[x].count;
    }
    const unsigned int votes = __ballot_sync(0xffffffffu, some);
    const int from = 31 - __clz(votes);  // the first group of all always qualifies
    return Bin{__shfl_sync(0xffffffffu, g.mass, from), b.limit,
               __shfl_sync(0xffffffffu, g.count, from), __shfl_sync(0xffffffffu, g.bin, from)};
  };

  // ---- bf16: tokens counted by value ----
  // Few values occur more than once each, so nothing is weighted token by
  // token: a histogram counts every value of the 16 octaves up to the largest
  // magnitude that has weight, in falling order (magnitudes below share one
  // bin, with the sum of their weights), and 4096 weights serve the row.  The
  // cut is then a value and how many of its tokens stay.  Where it falls among
  // the magnitudes below, the row is cut as one in fp32 is.
  // The block's tokens are counted in kSubs parts (16-bit counts, two to a
  // word): the masses of the parts follow from the counts, and the draw looks
  // at the tokens of one part alone.  Without a cut to find (10 rows of 60000:
  // 13.0 us this way, 7.7 without) the draw below weighs every token once.
  if constexpr (sizeof(T) == 2)
  if (by_k || by_p) {
    const int e = min(254, (__float_as_int(fmaxf(fabsf(hi), fabsf(weight.floor))) >> 23) & 255);
    const int least = max(0, e - 15) << 7;  // magnitude bits of the shared bin's largest
    constexpr int kHalf = kValues / 2, kTiny = kHalf - 1;
    auto value = [&](int bin) {
      const int sign = bin >> 11;
      return __uint_as_float(static_cast<uint32_t>((bin ^ (kTiny + sign)) + least) << 16 |
                             static_cast<uint32_t>(sign) << 31);
    };
    const float z_tiny = __uint_as_float(static_cast<uint32_t>(least) << 16);
    // parts 2 h and 2 h + 1 of a bin: the halves of cnt[h * kValues + bin]
    uint32_t* cnt = h_cnt;
    const int part = (n_vec + kSubs - 1) / kSubs;  // vectors of a part
    static_assert(kSubs == 4, "two words of two counts");
    auto both = [](uint32_t word) { return (word & 0xffffu) + (word >> 16); };
    auto tiny_of = [&](int x) {
      return static_cast<unsigned long long>(sh.tiny[1][x]) << 32 | sh.tiny[0][x];
    };
    {
      unsigned int far = 0u;
#pragma unroll 1
      for (int v = tid; v < n_vec; v += kThreads) {
        const uint4 raw = slice[v];
        const uint32_t word[4] = {raw.x, raw.y, raw.z, raw.w};
        const int sub = (v >= part) + (v >= 2 * part) + (v >= 3 * part);
        uint32_t* counts = cnt + (sub >> 1) * kValues;
        const uint32_t one = sub & 1 ? 0x10000u : 1u;
        unsigned int near = 0u;  // tokens of the shared bin, a bit each
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t bits = i & 1 ? word[i / 2] >> 16 : word[i / 2] & 0xffffu;
          const int mag = static_cast<int>(bits & 0x7fffu) - least;
          if (mag > 0 && mag < kHalf) {
            atomicAdd(&counts[mag ^ (kTiny + (bits >> 15))], one);
          } else if (mag <= 0) {
            near |= 1u << i;
          } else if (bits != 0xff80u) {
            ++far;
          }
        }
        if (near != 0u) {
          unsigned long long w = 0ull;
#pragma unroll 1
          for (int i = 0; i < 8; ++i)
            if ((near >> i) & 1u)
              w += weight(__uint_as_float(reinterpret_cast<const uint16_t*>(slice + v)[i] << 16));
          atomicAdd(&counts[kTiny], __popc(near) * one);
          const uint32_t lo = static_cast<uint32_t>(w);
          const uint32_t carry = atomicAdd(&sh.tiny[0][sub], lo) + lo < lo ? 1u : 0u;
          atomicAdd(&sh.tiny[1][sub], static_cast<uint32_t>(w >> 32) + carry);
        }
      }
      if (far > 0u) atomicAdd(&sh.far, far);
    }
    __syncthreads();
    // the sums of every group of 64 bins to every block
    {
      // eight bins a thread, eight threads a group
      unsigned long long m = 0ull;
      unsigned int k = 0u;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const uint4 a = reinterpret_cast<const uint4*>(cnt)[2 * tid + i / 4];
        const uint4 c = reinterpret_cast<const uint4*>(cnt + kValues)[2 * tid + i / 4];
        const uint32_t n[4] = {both(a.x) + both(c.x), both(a.y) + both(c.y), both(a.z) + both(c.z),
                               both(a.w) + both(c.w)};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int bin = tid * 8 + i + x;
          if (n[x] > 0u)
            m += bin == kTiny ? tiny_of(0) + tiny_of(1) + tiny_of(2) + tiny_of(3)
                              : n[x] * weight(value(bin));
          k += n[x];
        }
      }
#pragma unroll
      for (int o = 1; o < 8; o *= 2) {
        m += __shfl_xor_sync(0xffffffffu, m, o);
        k += __shfl_xor_sync(0xffffffffu, k, o);
      }
      if (tid % 8 < C)
        *cluster.map_shared_rank(&group[rank * kGroups + tid / 8], tid % 8) = Sums{m, k, 0};
    }
    if (tid < C) {
      *cluster.map_shared_rank(&sh.list_mass[rank], tid) =
          tiny_of(0) + tiny_of(1) + tiny_of(2) + tiny_of(3);
      *cluster.map_shared_rank(&sh.list_n[rank], tid) = sh.far;
    }
    cluster.sync();
    unsigned int far = 0u;
#pragma unroll 1
    for (int c = 0; c < C; ++c) far += sh.list_n[c];
    ValueCut cut{0ull, 0u, kValues, 0u, 0u, C};
    bool exact = u > 0.f;
    // the value and the tokens of it that a bound leaves
    auto cut_at = [&](bool by_mass, unsigned long long limit) {
      if (warp == 0) {
        const Bin g = find_group(by_mass, Bin{0ull, limit, 0u, 0u});
        if (lane == 0) sh.value_cut.bin = kValues;
        __syncwarp();
        const int bin = min(g.bin, kGroups - 1u) * 64 + 2 * lane;
        uint2 s = make_uint2(0u, 0u);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint2 n[kMaxCluster];  // reads in flight
#pragma unroll
          for (int c = 0; c < kMaxCluster; ++c)
            n[c] = c < C ? *reinterpret_cast<const uint2*>(cluster.map_shared_rank(cnt, c) +
                                                           half * kValues + bin)
                         : make_uint2(0u, 0u);
#pragma unroll
          for (int c = 0; c < kMaxCluster; ++c) {
            s.x += both(n[c].x);
            s.y += both(n[c].y);
          }
        }
        unsigned long long tiny = 0ull;
        if (bin + 1 == kTiny) {
#pragma unroll 1
          for (int c = 0; c < C; ++c) tiny += sh.list_mass[c];
        }
        unsigned long long w[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) w[x] = weight(value(bin + x));
        const unsigned long long m0 = s.x * w[0], m1 = bin + 1 == kTiny ? tiny : s.y * w[1];
        unsigned long long m = m0 + m1;
        unsigned int k = s.x + s.y;
        scan(m, k);
        m += g.mass - (m0 + m1);
        k += g.count - (s.x + s.y);
        const bool first = (by_mass ? m0 > 0ull : s.x > 0u) &&
                           (by_mass ? m : (unsigned long long)k) < g.limit;
        const bool second = (by_mass ? m1 > 0ull : s.y > 0u) &&
                            (by_mass ? m + m0 : (unsigned long long)(k + s.x)) < g.limit;
        const unsigned int votes = __ballot_sync(0xffffffffu, first || second);
        if (g.bin < kGroups && votes != 0u) {
          const int from = 31 - __clz(votes);
          ValueCut c{};
          c.bin = bin + (second ? 1 : 0);
          const unsigned long long one = second ? w[1] : w[0];
          if (second) {
            m += m0;
            k += s.x;
          }
          const unsigned int here = second ? s.y : s.x;
          if (lane == from) {
            const unsigned long long room = g.limit - (by_mass ? m : (unsigned long long)k);
            c.ties = static_cast<unsigned int>(
                min((unsigned long long)here, by_mass && one > 0ull ? (room + one - 1) / one : room));
          }
          c.mass = m + c.ties * one;
          c.count = k + c.ties;
          // the first block whose tokens of the value do not all stay
          const int cut_bin = __shfl_sync(0xffffffffu, static_cast<int>(c.bin), from);
          const unsigned int ties = __shfl_sync(0xffffffffu, c.ties, from);
          unsigned int y = 0u;
          if (lane < C) {
            const uint32_t* counts = cluster.map_shared_rank(cnt, lane) + cut_bin;
            y = both(counts[0]) + both(counts[kValues]);
          }
          unsigned long long none = 0ull;
          unsigned int sum = y;
          scan(none, sum);
          const unsigned int over = __ballot_sync(0xffffffffu, sum > ties);
          c.owner = over != 0u ? __ffs(over) - 1 : C;
          c.before = __shfl_sync(0xffffffffu, sum - y, over != 0u ? c.owner : 31);
          if (lane == from) sh.value_cut = c;
        }
      }
      __syncthreads();
      const ValueCut c = sh.value_cut;
      __syncthreads();
      // (in the shared bin tokens are not alike)
      exact = exact && c.bin != kTiny;
      if (c.bin == kValues)  // all that are counted stay
        exact = exact && far == 0u;
      else if (c.bin < cut.bin || (c.bin == cut.bin && c.ties < cut.ties)) cut = c;
    };
    if (exact && by_k) cut_at(false, top_k);
    if (exact && by_p) cut_at(true, cut.bin < kValues ? p_limit(cut.mass) : 0ull);
    if (exact) {
      if (cut.bin < kValues) cut_key = key_of(value(cut.bin));
      take_min_p();
      // whether all of the shared bin or nothing of it stays
      exact = !(fabsf(value_of(cut_key)) <= z_tiny);
      // (a min_p below every weight that counts)
      if (far > 0u && cut_key > kLowestKey && value_of(cut_key) < value(kValues - 1)) exact = false;
    }
    if (exact) {
      const float cut_z = value_of(cut_key);
      const bool split = cut.bin < kValues && key_of(value(cut.bin)) == cut_key;
      if (split) cut_id = rank < cut.owner ? 0x7fffffff : -1;
      // this block's tokens that stay, by part
      unsigned long long m[kSubs] = {};
      unsigned int k = 0u;
#pragma unroll 1
      for (int i = 0; i < kValues / kThreads; ++i) {
        const int bin = i * kThreads + tid;
        const float z = value(bin);
        const uint32_t a = cnt[bin], c = cnt[kValues + bin];
        if (z < cut_z || (a | c) == 0u) continue;
        uint32_t n[kSubs] = {a & 0xffffu, a >> 16, c & 0xffffu, c >> 16};
        if (split && z == cut_z) {
          // the first of its tokens stay
          uint32_t left = rank < cut.owner ? 0xffffffffu
                                           : rank == cut.owner ? cut.ties - cut.before : 0u;
          bool cut_here = true;
#pragma unroll
          for (int x = 0; x < kSubs; ++x) {
            if (left < n[x]) {
              if (cut_here) {
                sh.tie_sub = x;
                sh.tie_n = left;
                cut_here = false;
              }
              n[x] = left;
            }
            left -= n[x];
          }
        }
        const unsigned long long w = bin == kTiny ? 0ull : weight(z);
#pragma unroll
        for (int x = 0; x < kSubs; ++x) {
          m[x] += bin == kTiny ? tiny_of(x) : n[x] * w;
          k += n[x];
        }
      }
      exchange(Sums{warp_sum((m[0] + m[1]) + (m[2] + m[3])), __reduce_add_sync(0xffffffffu, k), 0});
      unsigned long long before = 0ull;
      const Sums all = total_of(before);
      if (rank == 0 && tid == 0 && p.kept != nullptr)
        p.kept[r] = static_cast<int>(all.count + (cut_key == kLowestKey ? far : 0u));
      const unsigned long long target = target_of(all.mass);
      if (target < before || target >= before + sh.part[rank].mass) return;
      // This block draws: the part that holds the target, then its token.
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int x = 0; x < kSubs - 1; ++x) m[x] += __shfl_xor_sync(0xffffffffu, m[x], o);
      if (lane == 0) {
#pragma unroll
        for (int x = 0; x < kSubs - 1; ++x) sh.word[x * kWarps + warp] = m[x];
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < kSubs - 1; ++x) m[x] = sh.word[x * kWarps + lane % kWarps];
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1)
#pragma unroll
        for (int x = 0; x < kSubs - 1; ++x) m[x] += __shfl_xor_sync(0xffffffffu, m[x], o);
      int sub = 0;
#pragma unroll
      for (int x = 0; x < kSubs - 1; ++x) {
        if (sub == x && target >= before + m[x]) {
          before += m[x];
          ++sub;
        }
      }
      span_of(min(n_vec, sub * part) * (VE / 4), min(n_vec, (sub + 1) * part) * (VE / 4));
      if (split && rank == cut.owner) {
        if (sub < sh.tie_sub) cut_id = 0x7fffffff;
        else if (sub == sh.tie_sub && sh.tie_n > 0u) cut_id = nth_of(cut_z, sh.tie_n);
      }
      const Sums own = kept_of();
      if (lane == 0) sh.red64[warp] = own.mass;
      __syncthreads();
      pick(target, before);
      return;
    }
    cut_key = kLowestKey;
    cut_id = 0x7fffffff;
    cluster.sync();  // bins and sums will be written again
  }

  // One pass over the slice: the tokens of the stretch onto the list of
  // every block, weights (summed) and counts of tokens into their bins.
  auto pass = [&](bool to_list, bool sum, bool mass_bins, bool count_bins) {
    unsigned long long* mine = list + rank * cap;
    const bool bins = mass_bins || count_bins, weights = sum || mass_bins;
    if (tid == 0) sh.n_local = 0u;
    if (bins) {
#pragma unroll 1
      for (int i = tid; i < 3 * kBins; i += kThreads) h_cnt[i] = 0u;
    }
    __syncthreads();
    unsigned long long m = 0ull;
#pragma unroll 1
    for (int v = tid; v < n_quad; v += kThreads) {
      const Quad raw = quads[v];
      const bool listed = to_list && Elem<T>::max_of(raw) > below;
      if (!listed && !weights && !bins) continue;
      float z[4];
      Elem<T>::unpack(raw, z);
      uint32_t bin[4];
      bool in[4];
      if (bins) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bin[i] = bin0(z[i]);
          in[i] = z[i] > -INFINITY;
          if (stage == kRange) {
            const uint32_t k = key_of(z[i]);
            in[i] = k >= kmin && k <= kmax;
            bin[i] = (kmax - k) >> shift;
          }
          if (count_bins && in[i]) atomicAdd(&h_cnt[bin[i]], 1u);
        }
      }
      if (weights) {
        // four independent weights, then their additions: two 32-bit words
        // with a carry (64-bit shared-memory additions measured 1.5 times
        // slower)
        unsigned long long w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = weight(z[i]);
        m += (w[0] + w[1]) + (w[2] + w[3]);
        if (mass_bins) {
          uint32_t old[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!in[i]) w[i] = 0ull;
            old[i] = w[i] != 0ull ? atomicAdd(&h_lo[bin[i]], static_cast<uint32_t>(w[i])) : 0u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t wl = static_cast<uint32_t>(w[i]);
            const uint32_t wh = static_cast<uint32_t>(w[i] >> 32) + (old[i] + wl < wl ? 1u : 0u);
            if (wh != 0u) atomicAdd(&h_hi[bin[i]], wh);
          }
        }
      }
      if (listed) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (within(z[i])) {
            const unsigned int at = atomicAdd(&sh.n_local, 1u);
            if (at < (unsigned int)cap)
              mine[at] = (static_cast<unsigned long long>(key_of(z[i])) << 32) |
                         (0xffffffffu - static_cast<uint32_t>(base + v * 4 + i));
          }
      }
    }
    if (sum) {
      m = warp_sum(m);
      if (lane == 0) sh.red64[warp] = m;
    }
    __syncthreads();
    if (tid < C && to_list) {
      *cluster.map_shared_rank(&sh.list_n[rank], tid) = sh.n_local;
      *cluster.map_shared_rank(&sh.list_mass[rank], tid) = sum ? block_sum(sh.red64) : 0ull;
    }
    if (to_list) {
      const int n_mine = static_cast<int>(min(sh.n_local, (unsigned int)cap));
      // thread e: entry e / C for block e % C
#pragma unroll 1
      for (int e = tid; e < n_mine * C; e += kThreads)
        if (e % C != rank) *cluster.map_shared_rank(&mine[e / C], e % C) = mine[e / C];
    }
    if (bins) {
      // the sums of every group of 32 bins to every block
#pragma unroll 1
      for (int g = warp; g < kGroups; g += kWarps) {
        const int bin = g * 32 + lane;
        const unsigned int n = __reduce_add_sync(0xffffffffu, h_cnt[bin]);
        const unsigned long long s =
            warp_sum((static_cast<unsigned long long>(h_hi[bin]) << 32) + h_lo[bin]);
        if (lane < C) *cluster.map_shared_rank(&group[rank * kGroups + g], lane) = Sums{s, n, 0};
      }
    }
    cluster.sync();
  };

  // the bin that a bound falls in, likewise
  auto find = [&](bool by_mass, Bin before) -> Bin {
    if (warp == 0) {
      const Bin g = find_group(by_mass, before);
      // its 32 bins over the cluster
      if (g.bin == kGroups) {
        if (lane == 0) sh.bin = Bin{0ull, g.limit, 0u, kBins};
      } else {
      const int bin = g.bin * 32 + lane;
      uint32_t rn[kMaxCluster], rl[kMaxCluster], rh[kMaxCluster];  // all reads in flight
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        rn[c] = c < C ? cluster.map_shared_rank(h_cnt, c)[bin] : 0u;
        rl[c] = c < C ? cluster.map_shared_rank(h_lo, c)[bin] : 0u;
        rh[c] = c < C ? cluster.map_shared_rank(h_hi, c)[bin] : 0u;
      }
      unsigned long long m = 0ull;
      unsigned int n = 0u;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        m += (static_cast<unsigned long long>(rh[c]) << 32) + rl[c];
        n += rn[c];
      }
      const bool some = by_mass ? m > 0ull : n > 0u;
      const unsigned long long bm = m;
      const unsigned int bn = n;
      scan(m, n);
      m += g.mass - bm;
      n += g.count - bn;
      const bool in = some && (by_mass ? m : (unsigned long long)n) < g.limit;
      const unsigned int bins = __ballot_sync(0xffffffffu, in);
      if (lane == 31 - __clz(bins)) sh.bin = Bin{m, g.limit, n, static_cast<uint32_t>(bin)};
      }
    }
    __syncthreads();
    const Bin b = sh.bin;
    __syncthreads();
    return b;
  };


  // The cut among the n listed tokens, which lie after b.count tokens of mass
  // b.mass: the last before which the count (or the mass) is below b.limit.
  // A thread holds up to two of the list's words (key and complemented id, so
  // that larger words come first).  While more than kRank are left, those of
  // the 256th of their range that holds the cut; the rest rank by counting the
  // larger ones and adding up their weights.
  auto list_cut = [&](Bin b, unsigned int n, bool& then_p) -> Cut {
    unsigned long long e[2], w[2];
    bool alive[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int c = (tid + x * kThreads) / cap, i = (tid + x * kThreads) - c * cap;
      alive[x] = c < C && i < (int)sh.list_n[c];
      e[x] = alive[x] ? list[tid + x * kThreads] : 0ull;
    }
    w[0] = w[1] = 0ull;
    if (by_p) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (alive[x]) w[x] = weight(value_of(static_cast<uint32_t>(e[x] >> 32)));
    }
#pragma unroll 1
    while (n > (unsigned int)kRank) {
      then_p = false;
      unsigned long long least = ~0ull, most = 0ull;
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (alive[x]) {
          least = min(least, e[x]);
          most = max(most, e[x]);
        }
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) {
        least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      }
      if (lane == 0) {
        sh.red64[warp] = least;
        sh.red64b[warp] = most;
      }
      if (tid < 256) sh.cnt[tid] = sh.lo[tid] = sh.high[tid] = 0u;
      __syncthreads();
#pragma unroll 1
      for (int x = 0; x < kWarps; ++x) {
        least = min(least, sh.red64[x]);
        most = max(most, sh.red64b[x]);
      }
      // words are distinct: the range is above zero and shrinks 128-fold a turn
      const int sh_r = max(0, 64 - __clzll(static_cast<long long>(most - least)) - 8);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (alive[x]) {
          const uint32_t bin = static_cast<uint32_t>((most - e[x]) >> sh_r);
          atomicAdd(&sh.cnt[bin], 1u);
          const uint32_t wl = static_cast<uint32_t>(w[x]);
          uint32_t wh = static_cast<uint32_t>(w[x] >> 32);
          if (wl != 0u && atomicAdd(&sh.lo[bin], wl) + wl < wl) ++wh;
          if (wh != 0u) atomicAdd(&sh.high[bin], wh);
        }
      __syncthreads();
      if (warp == 0) {
        // eight bins a lane
        unsigned int c = 0u;
        unsigned long long m = 0ull;
#pragma unroll 1
        for (int i = 8 * lane; i < 8 * lane + 8; ++i) {
          c += sh.cnt[i];
          m += (static_cast<unsigned long long>(sh.high[i]) << 32) + sh.lo[i];
        }
        unsigned int sc = c;
        unsigned long long sm = m;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned int y = __shfl_up_sync(0xffffffffu, sc, o);
          const unsigned long long d = __shfl_up_sync(0xffffffffu, sm, o);
          if (lane >= o) {
            sc += y;
            sm += d;
          }
        }
        sc += b.count - c;
        sm += b.mass - m;
        Bin f{};
        bool some = false;
#pragma unroll 1
        for (int i = 8 * lane; i < 8 * lane + 8; ++i) {
          if (sh.cnt[i] > 0u && (by_mass ? sm : (unsigned long long)sc) < b.limit) {
            some = true;
            f = Bin{sm, b.limit, sc, static_cast<uint32_t>(i)};
          }
          sc += sh.cnt[i];
          sm += (static_cast<unsigned long long>(sh.high[i]) << 32) + sh.lo[i];
        }
        const unsigned int votes = __ballot_sync(0xffffffffu, some);
        if (lane == 31 - __clz(votes)) sh.bin = f;
      }
      __syncthreads();
      b = sh.bin;
      n = sh.cnt[b.bin];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        alive[x] = alive[x] && static_cast<uint32_t>((most - e[x]) >> sh_r) == b.bin;
      __syncthreads();
    }
    if (tid == 0) {
      sh.n_local = 0u;
      sh.red32[0] = sh.red32[1] = 0u;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (alive[x]) {
        const unsigned int at = atomicAdd(&sh.n_local, 1u);
        sh.word[at] = e[x];
        sh.word_w[at] = w[x];
      }
    __syncthreads();
    // four threads to a word, each over a quarter of the others
    static_assert(4 * kRank <= kThreads, "");
    const int at = tid / 4;
    unsigned int rk = 0u;
    unsigned long long m = 0ull;
    bool stays = false;
    const unsigned long long own = at < (int)n ? sh.word[at] : 0ull;
    if (warp * 8 < (int)n) {
#pragma unroll 4
      for (int i = tid % 4; i < (int)n; i += 4)
        if (sh.word[i] > own) {
          ++rk;
          m += sh.word_w[i];
        }
      for (int o = 1; o < 4; o *= 2) {
        rk += __shfl_xor_sync(0xffffffffu, rk, o);
        m += __shfl_xor_sync(0xffffffffu, m, o);
      }
      m += b.mass;
      stays = at < (int)n && (by_mass ? m : (unsigned long long)b.count + rk) < b.limit;
      if (stays) atomicMax(&sh.red32[0], rk + 1u);
    }
    __syncthreads();
    if (stays && sh.red32[0] == rk + 1u)
      sh.cut = Cut{m + sh.word_w[at], static_cast<uint32_t>(own >> 32),
                   static_cast<int>(0xffffffffu - static_cast<uint32_t>(own))};
    __syncthreads();
    if (then_p) {
      stays = stays && m < p_limit(sh.cut.mass);
      if (stays) atomicMax(&sh.red32[1], rk + 1u);
      __syncthreads();
      if (stays && sh.red32[1] == rk + 1u)
        sh.cut = Cut{m + sh.word_w[at], static_cast<uint32_t>(own >> 32),
                     static_cast<int>(0xffffffffu - static_cast<uint32_t>(own))};
      __syncthreads();
    }
    const Cut cut = sh.cut;
    __syncthreads();
    return cut;
  };

  // ---- the cut ----
#pragma unroll 1
  while (by_k || by_p) {
    const bool to_list = stage == kTop || stage == kIn;
    pass(to_list, stage == kTop && !by_k, !to_list && by_p,
         stage == kRange || (stage == kRow && by_k));

    if (to_list) {
      unsigned int n = 0u;
      unsigned long long total = 0ull;
      bool fits = true;
#pragma unroll 1
      for (int c = 0; c < C; ++c) {
        fits = fits && sh.list_n[c] <= (unsigned int)cap;
        n += sh.list_n[c];
        total += sh.list_mass[c];
      }
      if (stage == kTop && !by_k) {
        limit = p_limit(total);
        if (fits) {
          // the list serves if its mass reaches the limit
          unsigned long long m = 0ull;
#pragma unroll 1
          for (int e = tid; e < kList; e += kThreads)
            if (e % cap < (int)sh.list_n[e / cap])
              m += weight(value_of(static_cast<uint32_t>(list[e] >> 32)));
          m = warp_sum(m);
          if (lane == 0) sh.red64[warp] = m;
          __syncthreads();
          fits = block_sum(sh.red64) >= limit;
          __syncthreads();
        }
      }
      Cut cut{};
      bool done = fits;
      if (fits) {
        b.limit = limit;
        // both bounds at once if the list is short enough to be ranked whole
        bool then_p = stage == kTop && by_k && by_p;
        const bool both = then_p;
        cut = list_cut(b, n, then_p);
        if (both) {
          by_mass = true;
          if (!then_p) {
            take(cut);
            b.limit = limit = p_limit(cut.mass);
            cut = list_cut(b, n, then_p);
          }
        }
      } else if (stage == kTop) {
        stage = kRow;
        b = Bin{0ull, 0ull, 0u, 0u};
        cluster.sync();  // the lists will be written again
        continue;
      } else {
        // a crowded bin: its key range
        kmin = 0xffffffffu;
        kmax = 0u;
#pragma unroll 1
        for (int v = tid; v < n_quad; v += kThreads) {
          float z[4];
          Elem<T>::unpack(quads[v], z);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (within(z[i])) {
              const uint32_t k = key_of(z[i]);
              kmin = min(kmin, k);
              kmax = max(kmax, k);
            }
        }
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        if (lane == 0) {
          sh.red32[warp] = kmin;
          sh.red32b[warp] = kmax;
        }
        __syncthreads();
        if (tid < C) {
#pragma unroll 1
          for (int w = 0; w < kWarps; ++w) {
            kmin = min(kmin, sh.red32[w]);
            kmax = max(kmax, sh.red32b[w]);
          }
          *cluster.map_shared_rank(&sh.kmin[rank], tid) = kmin;
          *cluster.map_shared_rank(&sh.kmax[rank], tid) = kmax;
        }
        cluster.sync();
        kmin = 0xffffffffu;
        kmax = 0u;
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
          kmin = min(kmin, sh.kmin[c]);
          kmax = max(kmax, sh.kmax[c]);
        }
        if (kmin < kmax) {
          shift = max(0, 32 - __clz(static_cast<int>(kmax - kmin)) - 11);
          stage = kRange;
          continue;
        }
        // one key: how many of its tokens stay, and the last of them
        const unsigned long long w = weight(value_of(kmin));
        const unsigned long long room = limit - (by_mass ? b.mass : (unsigned long long)b.count);
        const unsigned int m = static_cast<unsigned int>(
            min((unsigned long long)n, !by_mass ? room : w == 0ull ? n : (room + w - 1) / w));
        unsigned int before = 0u;
        int owner = 0;
#pragma unroll 1
        for (int c = 0; c < C && before + sh.list_n[c] < m; ++c) {
          before += sh.list_n[c];
          ++owner;
        }
        if (rank == owner) {
          const int id = nth_of(value_of(kmin), m - before);
          if (tid < C) *cluster.map_shared_rank(&sh.cut_id, tid) = id;
        }
        cluster.sync();
        cut = Cut{b.mass + m * w, kmin, sh.cut_id};
        done = true;
      }
      if (done) {
        take(cut);
        if (by_mass || !by_p) break;
        // top_k's cut is found in a bin: the row once more for top_p of the rest
        by_mass = true;
        limit = p_limit(cut.mass);
        stage = kRow;
        b = Bin{0ull, 0ull, 0u, 0u};
        cluster.sync();  // lists and bins will be written again
        continue;
      }
    }
    if (!to_list) {
      b.limit = limit;
      b = find(by_mass, b);
      if (b.bin == kBins) {
        // top_k keeps the whole row
        if (!by_p) break;
        by_mass = true;
        b = find(by_mass, Bin{0ull, 0ull, 0u, 0u});
      }
      limit = b.limit;
      if (stage == kRow) {
        // listed by bin; `below`, half a bin further, leaves out most others
        only = static_cast<int>(b.bin);
        const float lo = hi - (float)(only + 1) / bin_scale;
        below = only == kBins - 1 || !(lo > -INFINITY) ? -INFINITY : value_below(key_of(lo));
        top = hi;
      } else {
        const uint32_t last = kmax - (b.bin << shift), width = (1u << shift) - 1u;
        only = -1;
        top = value_of(last);
        below = value_below(last - kmin > width ? last - width : kmin);
      }
      stage = kIn;
    }
  }
  take_min_p();

  // ---- the draw: kept mass in id order ----
  exchange(kept_of());
  unsigned long long before = 0ull;
  const Sums all = total_of(before);
  if (rank == 0 && tid == 0 && p.kept != nullptr) p.kept[r] = static_cast<int>(all.count);
  if (u == 0.f) {  // the first token that stays, however small its weight
    if (rank == 0 && tid == 0) p.tokens[r] = all.first;
    return;
  }
  pick(target_of(all.mass), before);
}

// a block's share of the row and of its offset in a 16-byte word
template <typename T>
constexpr int sample_slice(int V, int C) {
  constexpr int VE = 16 / sizeof(T);
  return ((V + VE - 1 + C - 1) / C + 32 * VE - 1) / (32 * VE) * (32 * VE);
}

template <typename T>
medusa_status_t launch_sample(SampleParams& p, cudaStream_t stream) {
  // A cluster holds the row in shared memory.  Few rows: more blocks for each
  // while a block still has 4096 tokens.  Many: as few as leave two blocks to
  // an SM (a step's barriers cost a block the same whatever its share).
  const bool few = p.R * kMaxCluster <= 2 * device_sm_count();
  int C = 1;
  while (C < kMaxCluster && (few ? p.V > 4096 * C : (size_t)p.V * sizeof(T) > kManyBytes * C)) C *= 2;
  p.slice = sample_slice<T>(p.V, C);
  const size_t smem = (size_t)p.slice * sizeof(T) + sample_extra_smem(C);
  // What the kernel is allowed is the most that any row needs, not what this one
  // does: the setting is shared by all host threads, and a shorter row's must not
  // lower it between another's setting and its launch.
  constexpr size_t kMaxSmem =
      (size_t)sample_slice<T>(sample_max_vocab(sizeof(T)), kMaxCluster) * sizeof(T) +
      sample_extra_smem(kMaxCluster);
  static_assert(kManyBytes + 1024 + sample_extra_smem(kMaxCluster) <= kMaxSmem,
                "smaller clusters need less");
  static_assert(kMaxSmem + sizeof(Shared) <= 227 * 1024, "shared memory");
  if (cudaFuncSetAttribute(sample_tokens_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kMaxSmem)) != cudaSuccess)
    return fail(MEDUSA_ERR_CUDA, "cudaFuncSetAttribute(sample_tokens) failed");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.R) * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  cudaLaunchKernelEx(&cfg, sample_tokens_kernel<T>, p);
  return check_launch("sample_tokens");
}

}  // namespace

medusa_status_t sample_tokens(const void* logits, medusa_dtype_t dt, long long row_stride,
                              int n_rows, const int32_t* row_idx, int R, int V, const float* u,
                              const float* temperature, const int32_t* top_k, const float* top_p,
                              const float* min_p, int32_t* tokens, int32_t* kept, int32_t* status,
                              cudaStream_t stream) {
  SampleParams p{};
  p.logits = logits;
  p.row_stride = row_stride;
  p.row_idx = row_idx;
  p.n_rows = n_rows;
  p.R = R;
  p.V = V;
  p.u = u;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.tokens = tokens;
  p.kept = kept;
  p.status = status;
  if (dt == MEDUSA_BF16) return launch_sample<__nv_bfloat16>(p, stream);
  return launch_sample<float>(p, stream);
}

}  // namespace medusa
