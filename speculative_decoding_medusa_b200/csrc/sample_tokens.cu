// Tokens drawn from filtered logits: temperature, top-k, top-p and min-p with
// the caller's uniform numbers.
//
// Every filter keeps a prefix of the row's tokens in the order (logit
// descending, id ascending), so the kept set is a cut: a key (the logit as an
// ordered integer) and the last id that stays among the tokens with exactly
// that key.  The cut is found by selection, never by sorting the row:
//   - a histogram of the row over kBins bins of falling logit: token counts
//     for top-k, mass for top-p;
//   - the bin where the count reaches top_k, or the mass before it reaches
//     top_p of the total;
//   - inside that bin the exact cut: its tokens go on a short list and are
//     ranked against one another; a bin that holds too many is split by
//     histograms over its own key range until it is short or one key is left.
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
// Top tokens looked for when only top_p bounds a row; a row whose top_k is at
// most kTopWanted, or whose mass they reach, needs no histogram of its tokens.
constexpr int kTopWanted = 256;
constexpr int kRankBelow = 256;  // lists up to here are ranked by counting, not sorted
constexpr size_t kManyBytes = 65536;  // of a row in a block when there are many rows
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

// A finite float as a double by its bits; zero and subnormals become values
// of that size (below 2^-126), which no logit difference notices.
__device__ __forceinline__ double widen(float z) {
  const int b = __float_as_int(z);
  return __hiloint2double(((b >> 3) & static_cast<int>(0x8fffffffu)) + 0x38000000, b << 29);
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  __device__ static void unpack(uint4 r, float (&z)[4]) {
    z[0] = __uint_as_float(r.x);
    z[1] = __uint_as_float(r.y);
    z[2] = __uint_as_float(r.z);
    z[3] = __uint_as_float(r.w);
  }
  static constexpr uint32_t kNegInf = 0xff800000u;  // filler word
  // NaN if any is
  __device__ static float max2(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
  }
  __device__ static float max_of(uint4 r) {
    return max2(max2(__uint_as_float(r.x), __uint_as_float(r.y)),
                max2(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  __device__ static void unpack(uint4 r, float (&z)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = __uint_as_float(w[i] << 16);
      z[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {  // pairs
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ static float max_of(uint4 r) {
    const uint32_t m = max2(max2(r.x, r.y), max2(r.z, r.w));
    return Elem<float>::max2(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
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

struct Shared {
  float hi[kMaxCluster];    // largest logit (NaN: there is one)
  float edge[kMaxCluster];  // a bound below the block's share of the top tokens
  Sums part[kMaxCluster];
  unsigned long long list_mass[kMaxCluster];  // weights of every token of the block
  unsigned int list_n[kMaxCluster];
  uint32_t kmin[kMaxCluster], kmax[kMaxCluster];
  double table[kExpTable];
  Bin bin;
  Cut cut;
  unsigned int n_local;
  int cut_id;
  unsigned long long red64[kWarps], red64b[kWarps];
  unsigned int red32[kWarps], red32b[kWarps];
  float redf[kWarps];
};

// dynamic shared memory after the slice: histogram (counts, low and high words
// of the mass; the sorted list lies over the mass words), short lists and
// group sums of every block
__host__ __device__ constexpr size_t sample_extra_smem(int C) {
  return 3 * kBins * 4 + kList * 8 + (size_t)C * kGroups * sizeof(Sums);
}
static_assert(kList * 8 <= 2 * kBins * 4, "sorted list over the mass words");

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_tokens_kernel(SampleParams p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int VE = Elem<T>::kVec;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int r = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  extern __shared__ __align__(16) uint8_t dyn[];
  uint4* slice = reinterpret_cast<uint4*>(dyn);
  const int n_vec = p.slice / VE;
  // this block's histogram of its slice: counts, low and high words of the mass
  uint32_t* h_cnt = reinterpret_cast<uint32_t*>(dyn + (size_t)n_vec * 16);
  uint32_t* h_lo = h_cnt + kBins;
  uint32_t* h_hi = h_lo + kBins;
  unsigned long long* sorted = reinterpret_cast<unsigned long long*>(h_lo);
  // the short lists: words of key and complemented id, cap from each block
  unsigned long long* list = reinterpret_cast<unsigned long long*>(h_hi + kBins);
  Sums* group = reinterpret_cast<Sums*>(list + kList);
  const int cap = kList / C;
  __shared__ Shared sh;

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
      // the table of powers, while the first loads are under way
      if (v0 < kExpTable) sh.table[v0] = exp2((double)v0 / kExpTable);
#pragma unroll
      for (int f = 0; f < kFetch; ++f) {
        const int v = v0 + f * kThreads;
        if (v >= n_vec) break;
        slice[v] = raw[f];
        hi = Elem<float>::max2(hi, Elem<T>::max_of(raw[f]));
      }
    }
  }
  if (tid >= n_vec && tid < kExpTable) sh.table[tid] = exp2((double)tid / kExpTable);
  const float own_hi = hi;  // the largest of this thread's tokens
  for (int o = 16; o > 0; o >>= 1)
    hi = Elem<float>::max2(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  if (lane == 0) sh.redf[warp] = hi;
  __syncthreads();
  // The share-th largest of the block's threads' largest, to its top 16 bits
  // (found bit by bit): with every block's, at least `want` tokens of the row
  // lie at or above the least of them, and not many more.
  const bool by_k = top_k > 1 && top_k < p.V;
  const bool by_p = top_p < 1.f;
  const bool top_list = by_k ? top_k <= kTopWanted : by_p;
  float edge = -INFINITY;
  if (top_list) {
    const int want = by_k ? top_k : kTopWanted / 2;
    const int share = (want + C - 1) / C;
    const uint32_t own = own_hi > -INFINITY ? key_of(own_hi) : 0u;
    uint32_t k = 0u;
#pragma unroll 1
    for (uint32_t bit = 0x80000000u; bit >= 0x10000u; bit >>= 1)
      if (__syncthreads_count(own >= (k | bit)) >= share) k |= bit;
    if (k > 0u) edge = value_of(k);
  }
  if (tid < C) {
    hi = sh.redf[0];
    for (int w = 1; w < kWarps; ++w) hi = Elem<float>::max2(hi, sh.redf[w]);
    *cluster.map_shared_rank(&sh.hi[rank], tid) = hi;
    *cluster.map_shared_rank(&sh.edge[rank], tid) = edge;
  }
  cluster.sync();
  hi = sh.hi[0];
  edge = sh.edge[0];
  for (int c = 1; c < C; ++c) {
    hi = Elem<float>::max2(hi, sh.hi[c]);
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
    for (int v = tid; v < n_vec; v += kThreads) {
      const uint4 raw = slice[v];
      if (Elem<T>::max_of(raw) < hi) continue;
      float z[VE];
      Elem<T>::unpack(raw, z);
#pragma unroll
      for (int i = VE - 1; i >= 0; --i)
        if (z[i] == hi) first = min(first, base + v * VE + i);
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
  const float next = value_of(key_of(hi) - 1u);
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
  auto clear_bins = [&]() {
    for (int i = tid; i < kBins; i += kThreads) {
      h_cnt[i] = 0u;
      h_lo[i] = 0u;
      h_hi[i] = 0u;
    }
    __syncthreads();
  };
  // weights to their bins: two 32-bit words with a carry (64-bit shared-memory
  // additions measured 1.5 times slower)
  auto add_mass4 = [&](const uint32_t (&bin)[4], const unsigned long long (&w)[4]) {
    uint32_t old[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      old[i] = w[i] != 0ull ? atomicAdd(&h_lo[bin[i]], static_cast<uint32_t>(w[i])) : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t wl = static_cast<uint32_t>(w[i]);
      const uint32_t wh = static_cast<uint32_t>(w[i] >> 32) + (old[i] + wl < wl ? 1u : 0u);
      if (wh != 0u) atomicAdd(&h_hi[bin[i]], wh);
    }
  };
  // the sums of every group of 32 bins to every block
  auto publish = [&]() {
    __syncthreads();
    for (int g = warp; g < kGroups; g += kWarps) {
      const int bin = g * 32 + lane;
      const unsigned int n = __reduce_add_sync(0xffffffffu, h_cnt[bin]);
      unsigned long long m = (static_cast<unsigned long long>(h_hi[bin]) << 32) + h_lo[bin];
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      if (lane < C) *cluster.map_shared_rank(&group[rank * kGroups + g], lane) = Sums{m, n, 0};
    }
    cluster.sync();
  };
  // One histogram over the cluster: `pick(z, bin)` says whether a finite
  // logit counts and in which bin.  Afterwards every block holds every
  // block's sums of each group of 32 bins, and the blocks' own bins stay in
  // place for find().
  auto histogram = [&](bool counts, bool masses, auto pick) {
    clear_bins();
    for (int v = tid; v < n_vec; v += kThreads) {
      float z[VE];
      Elem<T>::unpack(slice[v], z);
      // four independent weights at a time, then their additions
#pragma unroll
      for (int i0 = 0; i0 < VE; i0 += 4) {
        uint32_t bin[4];
        bool in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) in[i] = z[i0 + i] > -INFINITY && pick(z[i0 + i], bin[i]);
        if (masses) {
          unsigned long long w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = in[i] ? weight(z[i0 + i]) : 0ull;
          add_mass4(bin, w);
        }
        if (counts) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (in[i]) atomicAdd(&h_cnt[bin[i]], 1u);
        }
      }
    }
    publish();
  };

  // The last bin with tokens before which the count (or the mass) is below
  // `limit`, given what lies before the histogram's range.  In mass mode
  // limit 0 stands for top_p of the histogram's own total.
  auto p_limit = [&](unsigned long long total) {
    // kept while the mass before is below top_p * total: an integer limit
    return max(1ull, static_cast<unsigned long long>(ceil((double)top_p * (double)total)));
  };
  auto find = [&](bool by_mass, unsigned long long limit, unsigned int count0,
                  unsigned long long mass0) -> Bin {
    static_assert(kGroups == 64, "two groups per lane");
    if (warp == 0) {
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
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long a = __shfl_up_sync(0xffffffffu, m, o);
        const unsigned int b = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) {
          m += a;
          n += b;
        }
      }
      if (limit == 0ull) limit = p_limit(__shfl_sync(0xffffffffu, m, 31));
      m += mass0 - own_m;
      n += count0 - own_n;
      // this lane's later qualifying group, if any
      int g = -1;
      unsigned long long gm = 0ull;
      unsigned int gn = 0u;
      for (int x = 0; x < 2; ++x) {
        const bool some = by_mass ? s[x].mass > 0ull : s[x].count > 0u;
        if (some && (by_mass ? m : (unsigned long long)n) < limit) {
          g = 2 * lane + x;
          gm = m;
          gn = n;
        }
        m += s[x].mass;
        n += s[x].count;
      }
      const unsigned int votes = __ballot_sync(0xffffffffu, g >= 0);
      const int from = 31 - __clz(votes);  // the first bin of all always qualifies
      g = __shfl_sync(0xffffffffu, g, from);
      gm = __shfl_sync(0xffffffffu, gm, from);
      gn = __shfl_sync(0xffffffffu, gn, from);
      // its 32 bins over the cluster
      const int bin = g * 32 + lane;
      uint32_t rn[kMaxCluster], rl[kMaxCluster], rh[kMaxCluster];  // all reads in flight
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        rn[c] = c < C ? cluster.map_shared_rank(h_cnt, c)[bin] : 0u;
        rl[c] = c < C ? cluster.map_shared_rank(h_lo, c)[bin] : 0u;
        rh[c] = c < C ? cluster.map_shared_rank(h_hi, c)[bin] : 0u;
      }
      m = 0ull;
      n = 0u;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        m += (static_cast<unsigned long long>(rh[c]) << 32) + rl[c];
        n += rn[c];
      }
      const bool some = by_mass ? m > 0ull : n > 0u;
      const unsigned long long bm = m;
      const unsigned int bn = n;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long a = __shfl_up_sync(0xffffffffu, m, o);
        const unsigned int b = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) {
          m += a;
          n += b;
        }
      }
      m += gm - bm;
      n += gn - bn;
      const bool in = some && (by_mass ? m : (unsigned long long)n) < limit;
      const unsigned int bins = __ballot_sync(0xffffffffu, in);
      if (lane == 31 - __clz(bins)) sh.bin = Bin{m, limit, n, static_cast<uint32_t>(bin)};
    }
    __syncthreads();
    const Bin b = sh.bin;
    __syncthreads();
    return b;
  };

  // tokens of one key, n of them with weight w each, that stay
  auto ties_kept = [&](bool by_mass, unsigned long long limit, unsigned int count,
                       unsigned long long mass, unsigned int n, unsigned long long w) {
    if (!by_mass) return static_cast<unsigned int>(min((unsigned long long)n, limit - count));
    if (w == 0ull) return n;
    return static_cast<unsigned int>(min((unsigned long long)n, (limit - mass + w - 1) / w));
  };

  // The tokens for which in(z) holds onto the short list of every block
  // (none(m): no token of a vector whose largest is m); with `masses` also the
  // weights of all tokens, with `bins` these into their bins.  False when a
  // block has too many; n: their number.
  auto gather = [&](auto in, auto none, bool masses, bool bins, unsigned int& n,
                    unsigned long long& mass) -> bool {
    unsigned long long* mine = list + rank * cap;
    if (tid == 0) sh.n_local = 0u;
    if (bins) clear_bins();
    __syncthreads();
    unsigned long long m = 0ull;
    for (int v = tid; v < n_vec; v += kThreads) {
      const uint4 raw = slice[v];
      const bool skip = none(Elem<T>::max_of(raw));
      if (skip && !masses) continue;
      float z[VE];
      Elem<T>::unpack(raw, z);
      if (masses) {
#pragma unroll
        for (int i0 = 0; i0 < VE; i0 += 4) {
          unsigned long long w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = weight(z[i0 + i]);
          m += (w[0] + w[1]) + (w[2] + w[3]);
          if (bins) {
            const uint32_t bin[4] = {bin0(z[i0]), bin0(z[i0 + 1]), bin0(z[i0 + 2]),
                                     bin0(z[i0 + 3])};
            add_mass4(bin, w);
          }
        }
      }
      if (!skip) {
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (in(z[i])) {
            const unsigned int at = atomicAdd(&sh.n_local, 1u);
            if (at < (unsigned int)cap)
              mine[at] = (static_cast<unsigned long long>(key_of(z[i])) << 32) |
                         (0xffffffffu - static_cast<uint32_t>(base + v * VE + i));
          }
      }
    }
    if (masses) {
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      if (lane == 0) sh.red64[warp] = m;
    }
    __syncthreads();
    if (tid < C) {
      *cluster.map_shared_rank(&sh.list_n[rank], tid) = sh.n_local;
      m = 0ull;
      if (masses)
        for (int w = 0; w < kWarps; ++w) m += sh.red64[w];
      *cluster.map_shared_rank(&sh.list_mass[rank], tid) = m;
    }
    const int n_mine = static_cast<int>(min(sh.n_local, (unsigned int)cap));
    for (int e = tid; e < n_mine * C; e += kThreads) {
      const int c = e / n_mine, i = e - c * n_mine;
      if (c != rank) *cluster.map_shared_rank(&mine[i], c) = mine[i];
    }
    cluster.sync();
    bool fits = true;
    n = 0u;
    mass = 0ull;
    for (int c = 0; c < C; ++c) {
      fits = fits && sh.list_n[c] <= (unsigned int)cap;
      n += sh.list_n[c];
      mass += sh.list_mass[c];
    }
    return fits;
  };

  // The lists as one array in the order of the tokens, largest first, and the
  // mass before the thread's two words 2 tid and 2 tid + 1 in it (given what
  // lies before the list).  A long list goes through a bitonic network: thread
  // t holds word t (and t + kThreads when there are more), exchanged by
  // shuffles, and through shared memory for distances of a warp or more.
  bool dirty = false;  // the histogram has been written over
  // the thread's words of the lists and their places in one array (-1: none)
  auto list_words = [&](unsigned long long (&e)[2], int (&at)[2]) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int c = (tid + x * kThreads) / cap, i = (tid + x * kThreads) - c * cap;
      at[x] = -1;
      e[x] = 0ull;
      if (c < C && i < (int)sh.list_n[c]) {
        at[x] = i;
        for (int o = 0; o < c; ++o) at[x] += sh.list_n[o];
        e[x] = list[tid + x * kThreads];
      }
    }
  };
  // Of the listed n tokens of bin b (which lie after b.count tokens of mass
  // b.mass), those of the 256th of their key range that holds the cut, into
  // the array, unsorted: n and what lies before them are updated.
  auto narrow = [&](bool by_mass, Bin& b, unsigned int& n) {
    dirty = true;
    uint32_t* cnt = reinterpret_cast<uint32_t*>(sorted + kList);  // beside the array
    uint32_t *lo = cnt + 256, *high = lo + 256;
    unsigned long long e[2];
    int at[2];
    list_words(e, at);
    uint32_t kmin = 0xffffffffu, kmax = 0u;
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (at[x] >= 0) {
        kmin = min(kmin, static_cast<uint32_t>(e[x] >> 32));
        kmax = max(kmax, static_cast<uint32_t>(e[x] >> 32));
      }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) {
      sh.red32[warp] = kmin;
      sh.red32b[warp] = kmax;
    }
    for (int i = tid; i < 3 * 256; i += kThreads) cnt[i] = 0u;
    if (tid == 0) sh.n_local = 0u;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      kmin = min(kmin, sh.red32[w]);
      kmax = max(kmax, sh.red32b[w]);
    }
    int shift = 0;
    while (((kmax - kmin) >> shift) >= 256u) ++shift;
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (at[x] >= 0) {
        const uint32_t key = static_cast<uint32_t>(e[x] >> 32), bin = (kmax - key) >> shift;
        atomicAdd(&cnt[bin], 1u);
        if (by_p) {
          const unsigned long long w = weight(value_of(key));
          const uint32_t wl = static_cast<uint32_t>(w);
          const uint32_t wh =
              static_cast<uint32_t>(w >> 32) + (atomicAdd(&lo[bin], wl) + wl < wl ? 1u : 0u);
          if (wh != 0u) atomicAdd(&high[bin], wh);
        }
      }
    __syncthreads();
    if (warp == 0) {
      // eight bins a lane
      unsigned int c = 0u;
      unsigned long long m = 0ull;
      for (int i = 8 * lane; i < 8 * lane + 8; ++i) {
        c += cnt[i];
        m += (static_cast<unsigned long long>(high[i]) << 32) + lo[i];
      }
      unsigned int sc = c;
      unsigned long long sm = m;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned int a = __shfl_up_sync(0xffffffffu, sc, o);
        const unsigned long long d = __shfl_up_sync(0xffffffffu, sm, o);
        if (lane >= o) {
          sc += a;
          sm += d;
        }
      }
      sc += b.count - c;
      sm += b.mass - m;
      Bin f{};
      bool some = false;
      for (int i = 8 * lane; i < 8 * lane + 8; ++i) {
        if (cnt[i] > 0u && (by_mass ? sm : (unsigned long long)sc) < b.limit) {
          some = true;
          f = Bin{sm, b.limit, sc, static_cast<uint32_t>(i)};
        }
        sc += cnt[i];
        sm += (static_cast<unsigned long long>(high[i]) << 32) + lo[i];
      }
      const unsigned int votes = __ballot_sync(0xffffffffu, some);
      if (lane == 31 - __clz(votes)) sh.bin = f;
    }
    __syncthreads();
    b = sh.bin;
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (at[x] >= 0 && (kmax - static_cast<uint32_t>(e[x] >> 32)) >> shift == b.bin)
        sorted[atomicAdd(&sh.n_local, 1u)] = e[x];
    __syncthreads();
    n = sh.n_local;
  };
  // listed: the words are the lists' (otherwise the array's first n)
  auto sort_list = [&](bool listed, unsigned int n, unsigned long long mass0, bool masses,
                       unsigned long long (&w)[2]) -> unsigned long long {
    dirty = true;
    unsigned long long e[2];
    int at[2];
    if (listed) {
      list_words(e, at);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (at[x] >= 0) sorted[at[x]] = e[x];
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        at[x] = tid + x * kThreads < (int)n ? tid + x * kThreads : -1;
        e[x] = at[x] >= 0 ? sorted[at[x]] : 0ull;
      }
    }
    if (n <= kRankBelow) {
      // short: every word's rank by counting the larger ones
      __syncthreads();
      int rk[2] = {0, 0};
      if (__any_sync(0xffffffffu, at[0] >= 0 || at[1] >= 0)) {
#pragma unroll 4
        for (int i = 0; i < (int)n; ++i) {
          const unsigned long long o = sorted[i];
          rk[0] += o > e[0] ? 1 : 0;
          rk[1] += o > e[1] ? 1 : 0;
        }
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (at[x] >= 0) sorted[rk[x]] = e[x];
      __syncthreads();
    } else {
      int size = 32;
      while (size < (int)n) size <<= 1;
      for (int i = n + tid; i < size; i += kThreads) sorted[i] = 0ull;
      __syncthreads();
      const bool wide = size > kThreads;
      const bool act = warp * 32 < size;
      unsigned long long e0 = act ? sorted[tid] : 0ull;
      unsigned long long e1 = wide ? sorted[tid + kThreads] : 0ull;
      auto keep = [&](unsigned long long mine, unsigned long long other, int x, int k, int j) {
        const bool larger = ((x & j) == 0) == ((x & k) == 0);
        return (mine > other) == larger ? mine : other;
      };
      for (int k = 2; k <= size; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
          if (j == kThreads) {  // the thread's own two words
            const unsigned long long a = keep(e0, e1, tid, k, j);
            e1 = keep(e1, e0, tid + kThreads, k, j);
            e0 = a;
          } else if (j >= 32) {
            __syncthreads();
            if (act) sorted[tid] = e0;
            if (wide) sorted[tid + kThreads] = e1;
            __syncthreads();
            if (act) e0 = keep(e0, sorted[tid ^ j], tid, k, j);
            if (wide) e1 = keep(e1, sorted[(tid + kThreads) ^ j], tid + kThreads, k, j);
          } else if (act) {
            e0 = keep(e0, __shfl_xor_sync(0xffffffffu, e0, j), tid, k, j);
            if (wide) e1 = keep(e1, __shfl_xor_sync(0xffffffffu, e1, j), tid + kThreads, k, j);
          }
        }
      }
      __syncthreads();
      if (act) sorted[tid] = e0;
      if (wide) sorted[tid + kThreads] = e1;
      __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
      w[x] = masses && 2 * tid + x < (int)n
                 ? weight(value_of(static_cast<uint32_t>(sorted[2 * tid + x] >> 32)))
                 : 0ull;
    unsigned long long m = w[0] + w[1];
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, m, o);
      if (lane >= o) m += y;
    }
    if (lane == 31) sh.red64[warp] = m;
    __syncthreads();
    m += mass0 - w[0] - w[1];
    for (int x = 0; x < warp; ++x) m += sh.red64[x];
    return m;
  };
  // the last of the sorted words for which stay(i, mass before) holds
  auto last_of = [&](unsigned int n, unsigned long long before,
                     const unsigned long long (&w)[2], auto stay) -> Cut {
    int last = -1;
    unsigned long long mass = 0ull;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = 2 * tid + x;
      if (i < (int)n && stay(i, before)) {
        last = i;
        mass = before + w[x];
      }
      before += w[x];
    }
    const unsigned int votes = __ballot_sync(0xffffffffu, last >= 0);
    if (votes != 0u && lane == 31 - __clz(votes)) sh.red32[warp] = last + 1;
    if (votes == 0u && lane == 0) sh.red32[warp] = 0u;
    __syncthreads();
    unsigned int best = 0u;
    for (int x = 0; x < kWarps; ++x) best = max(best, sh.red32[x]);
    if (last >= 0 && (unsigned int)last + 1u == best) {
      const unsigned long long e = sorted[last];
      sh.cut = Cut{mass, static_cast<uint32_t>(e >> 32),
                   static_cast<int>(0xffffffffu - static_cast<uint32_t>(e))};
    }
    __syncthreads();
    const Cut cut = sh.cut;
    __syncthreads();
    return cut;
  };

  // The cut among the n listed tokens, which lie after b.count tokens of mass
  // b.mass: the last before which the count (or the mass) is below b.limit.
  auto list_cut = [&](bool by_mass, Bin b, unsigned int n) -> Cut {
    const bool many = n > kRankBelow / 4;
    if (many) narrow(by_mass, b, n);
    unsigned long long w[2];
    const unsigned long long m = sort_list(!many, n, b.mass, by_p, w);
    return last_of(n, m, w, [&](int i, unsigned long long before) {
      return (by_mass ? before : (unsigned long long)b.count + i) < b.limit;
    });
  };

  // The exact cut inside bin b of the current histogram.
  auto resolve = [&](bool by_mass, Bin b, bool again) -> Cut {
    const unsigned long long limit = b.limit;
    bool level0 = true;
    float below = 0.f, top = 0.f;  // the bin's tokens: below < z <= top (levels >= 1)
    for (;;) {
      auto in_bin = [&](float z) {
        if (level0) return z > -INFINITY && bin0(z) == b.bin;
        return z > below && z <= top;
      };
      auto none = [&](float m) { return level0 ? bin0(m) > b.bin : !(m > below); };
      unsigned int n;
      unsigned long long unused;
      if (gather(in_bin, none, false, false, n, unused)) {
        const Cut cut = list_cut(by_mass, b, n);
        if (again) cluster.sync();  // the lists will be written again
        return cut;
      }
      // a crowded bin: its key range
      uint32_t kmin = 0xffffffffu, kmax = 0u;
      for (int v = tid; v < n_vec; v += kThreads) {
        float z[VE];
        Elem<T>::unpack(slice[v], z);
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (in_bin(z[i])) {
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
      for (int c = 0; c < C; ++c) {
        kmin = min(kmin, sh.kmin[c]);
        kmax = max(kmax, sh.kmax[c]);
      }
      if (kmin == kmax) {
        // one key: the id of the last of its tokens that stay, by counting
        const unsigned long long w = weight(value_of(kmin));
        const unsigned int m = ties_kept(by_mass, limit, b.count, b.mass, n, w);
        unsigned int before = 0u;
        int owner = 0;
        for (int c = 0; c < C; ++c) {
          if (before + sh.list_n[c] >= m) break;
          before += sh.list_n[c];
          ++owner;
        }
        if (rank == owner) {
          // ids rise with the vector index: warps take contiguous runs of it
          const int seg = (n_vec + kWarps * 32 - 1) / (kWarps * 32) * 32;
          const int v0 = warp * seg, v1 = min(n_vec, v0 + seg);
          auto count = [&](int v, float (&z)[VE]) {
            unsigned int c = 0u;
            if (v < v1) {
              Elem<T>::unpack(slice[v], z);
#pragma unroll
              for (int i = 0; i < VE; ++i)
                c += z[i] > -INFINITY && key_of(z[i]) == kmin ? 1u : 0u;
            }
            return c;
          };
          float z[VE];
          unsigned int c = 0u;
          for (int v = v0 + lane; v < v1; v += 32) c += count(v, z);
          c = __reduce_add_sync(0xffffffffu, c);
          if (lane == 0) sh.red32[warp] = c;
          __syncthreads();
          for (int w = 0; w < warp; ++w) before += sh.red32[w];
          if (before < m && before + c >= m) {
            for (int vv = v0; vv < v1; vv += 32) {
              const unsigned int x = count(vv + lane, z);
              unsigned int s = x;
              for (int o = 1; o < 32; o <<= 1) {
                const unsigned int a = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += a;
              }
              unsigned int at = before + s - x;
              if (at < m && at + x >= m) {
#pragma unroll
                for (int i = 0; i < VE; ++i)
                  if (z[i] > -INFINITY && key_of(z[i]) == kmin && ++at == m)
                    for (int c2 = 0; c2 < C; ++c2)
                      *cluster.map_shared_rank(&sh.cut_id, c2) = base + (vv + lane) * VE + i;
              }
              before += __shfl_sync(0xffffffffu, s, 31);
            }
          }
        }
        cluster.sync();
        return Cut{b.mass + m * w, kmin, sh.cut_id};
      }
      dirty = true;
      int shift = 0;
      while (((kmax - kmin) >> shift) >= (uint32_t)kBins) ++shift;
      histogram(true, by_p, [&](float z, uint32_t& bin) {
        const uint32_t k = key_of(z);
        if (k < kmin || k > kmax) return false;
        bin = (kmax - k) >> shift;
        return true;
      });
      b = find(by_mass, limit, b.count, b.mass);  // the same limit
      level0 = false;
      const uint32_t last = kmax - (b.bin << shift), width = (1u << shift) - 1u;
      top = value_of(last);
      below = value_of((last - kmin > width ? last - width : kmin) - 1u);
    }
  };

  // ---- the cut: larger keys stay, and ids up to cut_id of this one ----
  uint32_t cut_key = kLowestKey;
  int cut_id = 0x7fffffff;
  if (by_k || by_p) {
    auto all = [&](float z, uint32_t& bin) {
      bin = bin0(z);
      return true;
    };
    // whether the listed tokens' mass is at least `limit` (before they are sorted)
    auto list_reaches = [&](unsigned long long limit) {
      unsigned long long m = 0ull;
      for (int e = tid; e < C * cap; e += kThreads) {
        const int c = e / cap;
        if (e - c * cap < (int)sh.list_n[c])
          m += weight(value_of(static_cast<uint32_t>(list[e] >> 32)));
      }
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      if (lane == 0) sh.red64[warp] = m;
      __syncthreads();
      m = 0ull;
      for (int w = 0; w < kWarps; ++w) m += sh.red64[w];
      __syncthreads();
      return m >= limit;
    };
    auto group_count = [&]() {
      unsigned int count = 0u;
      for (int i = lane; i < C * kGroups; i += 32) count += group[i].count;
      return __reduce_add_sync(0xffffffffu, count);
    };
    // The top tokens first (from `edge` on): they hold the cut of a top_k, and
    // that of a top_p when they reach it.
    bool found = false, binned = false;
    if (top_list) {
      if (!by_k) {
        // Whether they will is guessed from the block's threads' largest: when
        // those above the edge are short of top_p of all, the weights go into
        // their bins in the same pass.
        const unsigned long long w = own_hi > -INFINITY ? weight(own_hi) : 0ull;
        unsigned long long some = own_hi >= edge ? w : 0ull, whole = w;
        for (int o = 16; o > 0; o >>= 1) {
          some += __shfl_xor_sync(0xffffffffu, some, o);
          whole += __shfl_xor_sync(0xffffffffu, whole, o);
        }
        if (lane == 0) {
          sh.red64[warp] = some;
          sh.red64b[warp] = whole;
        }
        __syncthreads();
        some = whole = 0ull;
        for (int x = 0; x < kWarps; ++x) {
          some += sh.red64[x];
          whole += sh.red64b[x];
        }
        binned = (double)some < (double)top_p * (double)whole;
        __syncthreads();
      }
      unsigned int n;
      unsigned long long total;
      if (gather([&](float z) { return z >= edge && z > -INFINITY; },
                 [&](float m) { return m < edge; }, !by_k, binned, n, total)) {
        const unsigned long long limit = by_k ? (unsigned long long)top_k : p_limit(total);
        if (by_k || list_reaches(limit)) {
          Cut cut = list_cut(!by_k, Bin{0ull, limit, 0u, 0u}, n);
          if (by_k && by_p) {
            const Cut c = list_cut(true, Bin{0ull, p_limit(cut.mass), 0u, 0u}, n);
            if (c.key > cut.key || (c.key == cut.key && c.id < cut.id)) cut = c;
          }
          found = true;
          cut_key = cut.key;
          cut_id = cut.id;
        }
      }
      if (!found) cluster.sync();  // the lists will be written again
    }
    if (!found) {
      if (binned) publish();
      else histogram(by_k, by_p, all);
      dirty = false;
      unsigned long long limit = 0ull;  // top_p of the whole row
      bool k_cut = false;
      if (by_k) {
        k_cut = (unsigned int)top_k < group_count();
      }
      if (k_cut) {
        const Bin b = find(false, (unsigned long long)top_k, 0u, 0ull);
        const Cut cut = resolve(false, b, by_p);
        cut_key = cut.key;
        cut_id = cut.id;
        if (by_p) {
          limit = p_limit(cut.mass);
          if (dirty) histogram(true, true, all);
        }
      }
      if (by_p) {
        const Bin b = find(true, limit, 0u, 0ull);
        const Cut cut = resolve(true, b, false);
        if (cut.key > cut_key || (cut.key == cut_key && cut.id < cut_id)) {
          cut_key = cut.key;
          cut_id = cut.id;
        }
      }
    }
  }
  if (min_p > 0.f) {
    // w >= min_p: a bound on the logit, rounded up to a float
    const float z_min = __double2float_ru((double)hi + log((double)min_p) * (double)temp);
    if (z_min > -INFINITY && key_of(z_min) > cut_key) {
      cut_key = key_of(z_min);
      cut_id = 0x7fffffff;
    }
  }

  // ---- the draw: kept mass in id order ----
  // warp w takes the vectors [w * seg, (w + 1) * seg) of the slice, 32 at a time
  const int seg = (n_vec + kWarps * 32 - 1) / (kWarps * 32) * 32;
  const int v_begin = warp * seg, v_end = min(n_vec, v_begin + seg);
  const float cut_z = value_of(cut_key);
  auto stays = [&](float z, int id) { return z > cut_z || (z == cut_z && id <= cut_id); };
  unsigned long long mass = 0ull;
  unsigned int count = 0u;
  int first = 0x7fffffff;
  for (int v = v_begin + lane; v < v_end; v += 32) {
    const uint4 raw = slice[v];
    if (Elem<T>::max_of(raw) < cut_z) continue;
    float z[VE];
    Elem<T>::unpack(raw, z);
#pragma unroll
    for (int i0 = 0; i0 < VE; i0 += 4) {
      bool in[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) in[i] = stays(z[i0 + i], base + v * VE + i0 + i);
      if (in[0] || in[1] || in[2] || in[3]) {
        // four independent weights, then the ones that stay
        unsigned long long w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = weight(z[i0 + i]);
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          if (in[i]) {
            mass += w[i];
            ++count;
            first = min(first, base + v * VE + i0 + i);
          }
        }
      }
    }
  }
  for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  count = __reduce_add_sync(0xffffffffu, count);
  first = __reduce_min_sync(0xffffffffu, first);
  if (lane == 0) {
    sh.red64[warp] = mass;
    sh.red32[warp] = count;
    sh.red32b[warp] = static_cast<unsigned int>(first);
  }
  __syncthreads();
  if (tid < C) {
    Sums t{0ull, 0u, 0x7fffffff};
    for (int w = 0; w < kWarps; ++w) {
      t.mass += sh.red64[w];
      t.count += sh.red32[w];
      t.first = min(t.first, static_cast<int>(sh.red32b[w]));
    }
    *cluster.map_shared_rank(&sh.part[rank], tid) = t;
  }
  cluster.sync();
  unsigned long long total = 0ull, before = 0ull;
  unsigned int kept = 0u;
  first = 0x7fffffff;
  for (int c = 0; c < C; ++c) {
    if (c == rank) before = total;
    total += sh.part[c].mass;
    kept += sh.part[c].count;
    first = min(first, sh.part[c].first);
  }
  if (rank == 0 && tid == 0 && p.kept != nullptr) p.kept[r] = static_cast<int>(kept);
  if (u == 0.f) {  // the first token that stays, however small its weight
    if (rank == 0 && tid == 0) p.tokens[r] = first;
    return;
  }
  const unsigned long long target =
      min(static_cast<unsigned long long>((double)u * (double)total), total - 1);
  for (int w = 0; w < warp; ++w) before += sh.red64[w];
  if (target < before || target >= before + mass) return;
  // this warp holds the drawn token
  for (int v0 = v_begin; v0 < v_end; v0 += 32) {
    const int v = v0 + lane;
    unsigned long long w[VE], n = 0ull;
    if (v < v_end) {
      float z[VE];
      Elem<T>::unpack(slice[v], z);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        w[i] = stays(z[i], base + v * VE + i) ? weight(z[i]) : 0ull;
        n += w[i];
      }
    }
    unsigned long long s = n;
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long a = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += a;
    }
    unsigned long long at = before + s - n;
    if (target >= at && target < at + n) {
      int id = -1;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        if (id < 0 && target < at + w[i]) id = base + v * VE + i;
        at += w[i];
      }
      p.tokens[r] = id;
    }
    before += __shfl_sync(0xffffffffu, s, 31);
    if (target < before) break;
  }
}

template <typename T>
medusa_status_t launch_sample(SampleParams& p, cudaStream_t stream) {
  constexpr int VE = Elem<T>::kVec;
  // A cluster holds the row in shared memory.  Few rows: more blocks for each
  // while a block still has 4096 tokens.  Many: as few as leave two blocks to
  // an SM (a step's barriers cost a block the same whatever its share).
  const bool few = p.R * kMaxCluster <= 2 * device_sm_count();
  int C = 1;
  while (C < kMaxCluster && (few ? p.V > 4096 * C : (size_t)p.V * sizeof(T) > kManyBytes * C)) C *= 2;
  const int span = p.V + VE - 1;  // the row and its offset in a 16-byte word
  p.slice = ((span + C - 1) / C + 32 * VE - 1) / (32 * VE) * (32 * VE);
  const size_t smem = (size_t)p.slice * sizeof(T) + sample_extra_smem(C);
  if (cudaFuncSetAttribute(sample_tokens_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
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
