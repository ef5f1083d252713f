// Tokens drawn from filtered logits: temperature, top-k, top-p and min-p with
// the caller's uniform numbers.
//
// Every filter keeps a prefix of the row's tokens in the order (logit
// descending, id ascending), so the kept set is a cut: a key and how many of
// the tokens with exactly that key (lowest ids) stay.  The cut is found by
// selection, never by sorting the row:
//   - a histogram of the row over kBins bins of falling logit, with token
//     counts and (for top-p) their mass;
//   - the bin where the count reaches top_k, or the mass before it reaches
//     top_p of the total;
//   - inside that bin the exact key: a short list of its keys ranked against
//     one another, or, when the bin holds too many, histograms over its own
//     key range until it is short or a single key is left.
// min-p is a bound on the exponent and needs no selection.
//
// Masses are exact: w = exp((z - max) / T) is rounded once to 64-bit fixed
// point (units of 2^-42 of the largest weight, which is 1), and integers add
// up the same in any order, so a draw is the same however the row is split
// and a token is decided as in a 64-bit sum up to 2^-43 per token.  A fp32 sum
// over a vocabulary of 128256 decides one draw in about a hundred differently.
//
// A row belongs to a cluster of thread blocks that hold it in shared memory:
// it is read from HBM once, and every later pass runs on the copy.
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
constexpr int kShort = 512;       // keys a bin may hold to be ranked directly
constexpr int kMaxCluster = 8;
constexpr double kUnit = 4398046511104.0;  // 2^42: weight 1 in fixed point

struct SampleParams {
  const void* logits;
  long long row_stride;
  const int32_t* row_idx;
  int n_rows, R, V, slice;  // slice: elements per block of the cluster
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t *tokens, *kept, *status;
};

// order-preserving integer of a finite float or -inf; -0 counts as +0
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
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
};

// what a block tells the others of its cluster
struct Extremes {
  float hi, lo;  // largest logit, smallest finite logit
  int arg;       // lowest id of the largest
  int bad;       // a NaN or +inf
};
struct Totals {
  unsigned long long mass;
  unsigned int count;
  int first;  // lowest kept id
};
struct Found {
  unsigned long long mass;  // before the bin (or key)
  unsigned int count;
  unsigned int n;  // tokens in the bin (or with the key)
  uint32_t bin;    // bin, or cut key
  uint32_t m;      // tokens of the cut key that stay
};

struct Shared {
  Extremes ext[kMaxCluster];
  Totals chunk[kMaxCluster];   // histogram chunk totals
  Totals part[kMaxCluster];    // draw: kept mass of each block
  unsigned int ties[kMaxCluster];
  uint32_t kmin[kMaxCluster], kmax[kMaxCluster];
  Found found;
  unsigned int n_list;
  uint32_t list[kShort];
  unsigned long long list_w[kShort];
  unsigned long long red64[kWarps];
  unsigned int red32[kWarps], red32b[kWarps];
  float redf[kWarps], redg[kWarps];
  uint32_t best_key;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_tokens_kernel(SampleParams p) {
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
  const int per = kBins / C;  // bins of a chunk
  // the cluster's sums over the chunk of bins this block owns
  unsigned long long* c_mass = reinterpret_cast<unsigned long long*>(h_hi + kBins);
  uint32_t* c_cnt = reinterpret_cast<uint32_t*>(c_mass + per);
  __shared__ Shared sh;

  const float temp = p.temperature != nullptr ? p.temperature[r] : 1.f;
  const float u = p.u[r];
  const int top_k = p.top_k != nullptr ? p.top_k[r] : 0;
  const float top_p = p.top_p != nullptr ? p.top_p[r] : 1.f;
  const float min_p = p.min_p != nullptr ? p.min_p[r] : 0.f;
  const int src_row = p.row_idx != nullptr ? p.row_idx[r] : r;
  bool bad = !(u >= 0.f && u < 1.f) || !(temp >= 0.f) || !(top_p >= 0.f) ||
             !(min_p >= 0.f && min_p <= 1.f) ||
             src_row < 0 || src_row >= p.n_rows || isinf(temp);

  // ---- the slice into shared memory; extremes ----
  // Blocks split the row at 16-byte boundaries of its address: element i of
  // the split is token i - off.
  float hi = -INFINITY, lo = INFINITY;
  int arg = 0x7fffffff;
  bool nan = false;
  int base = 0;
  if (!bad) {
    const T* row = static_cast<const T*>(p.logits) + (size_t)src_row * p.row_stride;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % VE);
    base = rank * p.slice - off;  // token id of the slice's first element
    for (int v = tid; v < n_vec; v += kThreads) {
      const int id = base + v * VE;
      uint4 raw;
      if (id >= 0 && id + VE <= p.V) {
        raw = __ldg(reinterpret_cast<const uint4*>(row + id));
      } else {
        raw = make_uint4(Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf);
        T* e = reinterpret_cast<T*>(&raw);
        for (int i = 0; i < VE; ++i)
          if (id + i >= 0 && id + i < p.V) e[i] = row[id + i];
      }
      slice[v] = raw;
      float z[VE];
      Elem<T>::unpack(raw, z);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        if (!(z[i] < INFINITY)) nan = true;
        if (z[i] > hi) {
          hi = z[i];
          arg = id + i;
        }
        if (z[i] > -INFINITY) lo = fminf(lo, z[i]);
      }
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    const float oh = __shfl_xor_sync(0xffffffffu, hi, o);
    const int oa = __shfl_xor_sync(0xffffffffu, arg, o);
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    if (better(oh, oa, hi, arg)) {
      hi = oh;
      arg = oa;
    }
  }
  nan = __any_sync(0xffffffffu, nan);
  if (lane == 0) {
    sh.redf[warp] = hi;
    sh.redg[warp] = lo;
    sh.red32[warp] = static_cast<unsigned int>(arg);
    sh.red32b[warp] = nan ? 1u : 0u;
  }
  __syncthreads();
  if (tid < C) {
    Extremes e{-INFINITY, INFINITY, 0x7fffffff, 0};
    for (int w = 0; w < kWarps; ++w) {
      const int a = static_cast<int>(sh.red32[w]);
      if (better(sh.redf[w], a, e.hi, e.arg)) {
        e.hi = sh.redf[w];
        e.arg = a;
      }
      e.lo = fminf(e.lo, sh.redg[w]);
      e.bad |= static_cast<int>(sh.red32b[w]);
    }
    *cluster.map_shared_rank(&sh.ext[rank], tid) = e;
  }
  cluster.sync();
  float zlo = INFINITY;
  hi = -INFINITY;
  arg = 0x7fffffff;
  for (int c = 0; c < C; ++c) {
    const Extremes e = sh.ext[c];
    if (better(e.hi, e.arg, hi, arg)) {
      hi = e.hi;
      arg = e.arg;
    }
    zlo = fminf(zlo, e.lo);
    if (e.bad) bad = true;
  }
  if (!(hi > -INFINITY)) bad = true;
  if (bad || temp == 0.f || top_k == 1) {
    if (rank == 0 && tid == 0) {
      if (bad) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
      p.tokens[r] = bad ? -1 : arg;
      if (p.kept != nullptr) p.kept[r] = bad ? 0 : 1;
    }
    return;  // the whole cluster takes this branch, after its last exchange
  }

  const double zmax = hi;
  const double c_log2 = 1.4426950408889634074 / (double)temp;  // log2(e) / T
  auto exponent = [&](float z) { return ((double)z - zmax) * c_log2; };
  auto weight = [&](float z) -> unsigned long long {
    const double y = exponent(z);
    return y < -43.5 ? 0ull : __double2ull_rn(exp2(y) * kUnit);
  };
  // bins of level 0: linear in the logit, over the range that can carry mass
  // or, if that is smaller, the row's own
  const float range = fminf(hi - zlo, 32.f * temp);
  const float bin_scale = range > 0.f ? fminf((float)(kBins - 1) / range, 1e30f) : 0.f;
  auto bin0 = [&](float z) -> uint32_t {
    return static_cast<uint32_t>(fminf((hi - z) * bin_scale, (float)(kBins - 1)));
  };
  const bool by_k = top_k > 0 && top_k < p.V;
  const bool by_p = top_p < 1.f;

  // one histogram over the cluster: `pick(z, key, bin)` says whether a token
  // counts and in which bin.  Leaves the chunk sums in c_cnt / c_mass and every
  // chunk's totals in sh.chunk.
  auto histogram = [&](auto pick) {
    for (int i = tid; i < kBins; i += kThreads) {
      h_cnt[i] = 0u;
      h_lo[i] = 0u;
      h_hi[i] = 0u;
    }
    __syncthreads();
    for (int v = tid; v < n_vec; v += kThreads) {
      float z[VE];
      Elem<T>::unpack(slice[v], z);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        uint32_t bin;
        if (z[i] > -INFINITY && pick(z[i], bin)) {
          atomicAdd(&h_cnt[bin], 1u);
          if (by_p) {
            const unsigned long long w = weight(z[i]);
            const uint32_t wl = static_cast<uint32_t>(w);
            uint32_t wh = static_cast<uint32_t>(w >> 32);
            if (wl != 0u && atomicAdd(&h_lo[bin], wl) + wl < wl) ++wh;
            if (wh != 0u) atomicAdd(&h_hi[bin], wh);
          }
        }
      }
    }
    cluster.sync();
    // sum of this block's chunk over the cluster
    unsigned long long mass = 0ull;
    unsigned int count = 0u;
    for (int i = tid; i < per; i += kThreads) {
      const int bin = rank * per + i;
      unsigned int n = 0u;
      unsigned long long m = 0ull;
      for (int c = 0; c < C; ++c) {
        n += cluster.map_shared_rank(h_cnt, c)[bin];
        if (by_p)
          m += (static_cast<unsigned long long>(cluster.map_shared_rank(h_hi, c)[bin]) << 32) +
               cluster.map_shared_rank(h_lo, c)[bin];
      }
      c_cnt[i] = n;
      c_mass[i] = m;
      count += n;
      mass += m;
    }
    for (int o = 16; o > 0; o >>= 1) {
      count += __shfl_xor_sync(0xffffffffu, count, o);
      mass += __shfl_xor_sync(0xffffffffu, mass, o);
    }
    if (lane == 0) {
      sh.red32[warp] = count;
      sh.red64[warp] = mass;
    }
    __syncthreads();
    if (tid < C) {
      Totals t{0ull, 0u, 0};
      for (int w = 0; w < kWarps; ++w) {
        t.count += sh.red32[w];
        t.mass += sh.red64[w];
      }
      *cluster.map_shared_rank(&sh.chunk[rank], tid) = t;
    }
    cluster.sync();
  };

  // the last bin with tokens before which the count (or the mass) is below
  // `limit`, given what lies before the histogram's range; told to every block
  auto find_bin = [&](bool mass_mode, unsigned long long limit, unsigned int count0,
                      unsigned long long mass0) -> Found {
    unsigned int cb = count0, mine_c = 0u;
    unsigned long long mb = mass0, mine_m = 0ull;
    int owner = -1;
    for (int c = 0; c < C; ++c) {
      const Totals t = sh.chunk[c];
      if (t.count > 0u && (mass_mode ? mb : (unsigned long long)cb) < limit) {
        owner = c;
        mine_c = cb;
        mine_m = mb;
      }
      cb += t.count;
      mb += t.mass;
    }
    if (rank == owner) {
      // thread t scans bins t * each .. of the chunk
      const int each = (per + kThreads - 1) / kThreads;
      unsigned int n = 0u;
      unsigned long long m = 0ull;
      for (int i = tid * each; i < min(per, (tid + 1) * each); ++i) {
        n += c_cnt[i];
        m += c_mass[i];
      }
      unsigned int sn = n;
      unsigned long long sm = m;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned int a = __shfl_up_sync(0xffffffffu, sn, o);
        const unsigned long long b = __shfl_up_sync(0xffffffffu, sm, o);
        if (lane >= o) {
          sn += a;
          sm += b;
        }
      }
      if (lane == 31) {
        sh.red32[warp] = sn;
        sh.red64[warp] = sm;
      }
      if (tid == 0) sh.best_key = 0u;
      __syncthreads();
      unsigned int before_n = mine_c + sn - n;
      unsigned long long before_m = mine_m + sm - m;
      for (int w = 0; w < warp; ++w) {
        before_n += sh.red32[w];
        before_m += sh.red64[w];
      }
      int best = -1;
      Found f{};
      for (int i = tid * each; i < min(per, (tid + 1) * each); ++i) {
        if (c_cnt[i] > 0u && (mass_mode ? before_m : (unsigned long long)before_n) < limit) {
          best = i;
          f = Found{before_m, before_n, c_cnt[i], static_cast<uint32_t>(rank * per + i), 0u};
        }
        before_n += c_cnt[i];
        before_m += c_mass[i];
      }
      if (best >= 0) atomicMax(&sh.best_key, static_cast<uint32_t>(best + 1));
      __syncthreads();
      if (best >= 0 && sh.best_key == static_cast<uint32_t>(best + 1))
        for (int c = 0; c < C; ++c) *cluster.map_shared_rank(&sh.found, c) = f;
    }
    cluster.sync();
    const Found f = sh.found;
    cluster.sync();
    return f;
  };

  // tokens of equal key and weight w that stay when `before` lies ahead of them
  auto ties_kept = [&](bool mass_mode, unsigned long long limit, unsigned int count,
                       unsigned long long mass, unsigned int n, unsigned long long w) {
    if (!mass_mode) return static_cast<uint32_t>(min((unsigned long long)n, limit - count));
    if (w == 0ull) return n;
    return static_cast<uint32_t>(min((unsigned long long)n, (limit - mass + w - 1) / w));
  };

  // The exact cut inside bin f of the current histogram; pred(z, key) tells
  // the bin's tokens.  Returns {mass, count before the key, n with the key,
  // key, m kept}.
  auto resolve = [&](bool mass_mode, unsigned long long limit, Found f) -> Found {
    bool level0 = true;
    uint32_t plo = 0u, phi = 0xffffffffu;  // key interval of the bin (levels >= 1)
    for (;;) {
      auto in_bin = [&](float z) {
        if (level0) return bin0(z) == f.bin;
        const uint32_t k = key_of(z);
        return k >= plo && k <= phi;
      };
      if (f.n <= kShort) {
        if (tid == 0) sh.n_list = 0u;
        cluster.sync();
        unsigned int* n_list = cluster.map_shared_rank(&sh.n_list, 0);
        uint32_t* list = cluster.map_shared_rank(sh.list, 0);
        for (int v = tid; v < n_vec; v += kThreads) {
          float z[VE];
          Elem<T>::unpack(slice[v], z);
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (z[i] > -INFINITY && in_bin(z[i])) {
              const unsigned int at = atomicAdd(n_list, 1u);
              if (at < kShort) list[at] = key_of(z[i]);
            }
        }
        cluster.sync();
        if (rank == 0) {
          const int n = static_cast<int>(min(sh.n_list, (unsigned int)kShort));
          for (int i = tid; i < n; i += kThreads) sh.list_w[i] = weight(value_of(sh.list[i]));
          if (tid == 0) sh.best_key = 0xffffffffu;
          __syncthreads();
          Found g{};
          bool ok = false;
          if (tid < n) {  // kShort == kThreads: one key per thread
            const uint32_t k = sh.list[tid];
            unsigned int ahead = 0u, same = 0u;
            unsigned long long ahead_m = 0ull;
            for (int j = 0; j < n; ++j) {
              const uint32_t kj = sh.list[j];
              if (kj > k) {
                ++ahead;
                ahead_m += sh.list_w[j];
              }
              same += kj == k ? 1u : 0u;
            }
            g = Found{f.mass + ahead_m, f.count + ahead, same, k, 0u};
            ok = (mass_mode ? g.mass : (unsigned long long)g.count) < limit;
            if (ok) {
              g.m = ties_kept(mass_mode, limit, g.count, g.mass, same, sh.list_w[tid]);
              atomicMin(&sh.best_key, k);
            }
          }
          __syncthreads();
          if (ok && sh.best_key == g.bin)  // several threads may hold equal copies
            for (int c = 0; c < C; ++c) *cluster.map_shared_rank(&sh.found, c) = g;
        }
        cluster.sync();
        const Found g = sh.found;
        cluster.sync();
        return g;
      }
      // a crowded bin: its key range, then a histogram over that range
      uint32_t kmin = 0xffffffffu, kmax = 0u;
      for (int v = tid; v < n_vec; v += kThreads) {
        float z[VE];
        Elem<T>::unpack(slice[v], z);
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (z[i] > -INFINITY && in_bin(z[i])) {
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
        f.bin = kmin;
        f.m = ties_kept(mass_mode, limit, f.count, f.mass, f.n, weight(value_of(kmin)));
        return f;
      }
      int shift = 0;
      while (((kmax - kmin) >> shift) >= (uint32_t)kBins) ++shift;
      histogram([&](float z, uint32_t& bin) {
        const uint32_t k = key_of(z);
        if (k < kmin || k > kmax) return false;
        bin = (kmax - k) >> shift;
        return true;
      });
      f = find_bin(mass_mode, limit, f.count, f.mass);
      level0 = false;
      phi = kmax - (f.bin << shift);
      const uint32_t width = (1u << shift) - 1u;
      plo = phi - kmin > width ? phi - width : kmin;
    }
  };

  // ---- the cut ----
  uint32_t cut = 0u;            // tokens with a larger key stay
  uint32_t cut_m = 0xffffffffu;  // and the first cut_m with this one
  bool ranked = false;          // some tokens with the cut's key do not stay
  if (by_k || by_p) {
    histogram([&](float z, uint32_t& bin) {
      bin = bin0(z);
      return true;
    });
    unsigned long long total = 0ull;
    unsigned int count = 0u;
    for (int c = 0; c < C; ++c) {
      total += sh.chunk[c].mass;
      count += sh.chunk[c].count;
    }
    Found fp{};
    bool p_cut = false;
    if (by_k && (unsigned int)top_k < count) {
      // find both bins on the level-0 histogram before a crowded bin reuses it
      Found fk = find_bin(false, (unsigned long long)top_k, 0u, 0ull);
      fk = resolve(false, (unsigned long long)top_k, fk);
      cut = fk.bin;
      cut_m = fk.m;
      ranked = fk.m < fk.n;
      if (by_p) {
        total = fk.mass + fk.m * weight(value_of(fk.bin));
        histogram([&](float z, uint32_t& bin) {
          bin = bin0(z);
          return true;
        });
      }
    }
    if (by_p) {
      // kept while the mass before is below top_p * total: an integer limit
      const unsigned long long limit =
          max(1ull, static_cast<unsigned long long>(ceil((double)top_p * (double)total)));
      fp = find_bin(true, limit, 0u, 0ull);
      fp = resolve(true, limit, fp);
      p_cut = fp.bin > cut || (fp.bin == cut && fp.m < cut_m);
    }
    if (p_cut) {
      cut = fp.bin;
      cut_m = fp.m;
      ranked = fp.m < fp.n;
    }
  }

  // ---- the draw: kept mass in id order ----
  // warp w takes the vectors [w * seg, (w + 1) * seg) of the slice, 32 at a time
  const double y_min = min_p > 0.f ? log2((double)min_p) : -INFINITY;
  const int seg = (n_vec + kWarps * 32 - 1) / (kWarps * 32) * 32;
  const int v_begin = warp * seg, v_end = min(n_vec, v_begin + seg);
  unsigned int tie_base = 0u;  // tokens with the cut's key before this warp's
  if (ranked) {
    unsigned int n = 0u;
    for (int v = v_begin + lane; v < v_end; v += 32) {
      float z[VE];
      Elem<T>::unpack(slice[v], z);
#pragma unroll
      for (int i = 0; i < VE; ++i) n += key_of(z[i]) == cut ? 1u : 0u;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sh.red32[warp] = n;
    __syncthreads();
    if (tid < C) {
      unsigned int t = 0u;
      for (int w = 0; w < kWarps; ++w) t += sh.red32[w];
      *cluster.map_shared_rank(&sh.ties[rank], tid) = t;
    }
    cluster.sync();
    for (int c = 0; c < rank; ++c) tie_base += sh.ties[c];
    for (int w = 0; w < warp; ++w) tie_base += sh.red32[w];
    __syncthreads();
  }
  // one vector's kept weights; `tie` counts the cut's key before this warp step
  auto kept_weights = [&](int v, unsigned int& tie, unsigned long long (&w)[VE],
                          bool (&stay)[VE]) {
    float z[VE];
    if (v < v_end) {
      Elem<T>::unpack(slice[v], z);
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) z[i] = -INFINITY;
    }
    unsigned int before = 0u;
    if (ranked) {
      unsigned int n = 0u;
#pragma unroll
      for (int i = 0; i < VE; ++i) n += key_of(z[i]) == cut ? 1u : 0u;
      unsigned int s = n;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned int a = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += a;
      }
      before = tie + s - n;
      tie += __shfl_sync(0xffffffffu, s, 31);
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const uint32_t k = key_of(z[i]);
      bool keep = z[i] > -INFINITY && k >= cut;
      if (ranked && k == cut) keep = before++ < cut_m;
      w[i] = 0ull;
      if (keep) {
        const double y = exponent(z[i]);
        keep = y >= y_min;
        if (keep) w[i] = y < -43.5 ? 0ull : __double2ull_rn(exp2(y) * kUnit);
      }
      stay[i] = keep;
    }
  };
  unsigned long long mass = 0ull;
  unsigned int count = 0u;
  int first = 0x7fffffff;
  {
    unsigned int tie = tie_base;
    for (int v0 = v_begin; v0 < v_end; v0 += 32) {
      unsigned long long w[VE];
      bool stay[VE];
      kept_weights(v0 + lane, tie, w, stay);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        mass += w[i];
        if (stay[i]) {
          ++count;
          first = min(first, base + (v0 + lane) * VE + i);
        }
      }
    }
    for (int o = 16; o > 0; o >>= 1) {
      mass += __shfl_xor_sync(0xffffffffu, mass, o);
      count += __shfl_xor_sync(0xffffffffu, count, o);
      first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
    }
    if (lane == 0) {
      sh.red64[warp] = mass;
      sh.red32[warp] = count;
      sh.red32b[warp] = static_cast<unsigned int>(first);
    }
    __syncthreads();
    if (tid < C) {
      Totals t{0ull, 0u, 0x7fffffff};
      for (int w = 0; w < kWarps; ++w) {
        t.mass += sh.red64[w];
        t.count += sh.red32[w];
        t.first = min(t.first, static_cast<int>(sh.red32b[w]));
      }
      *cluster.map_shared_rank(&sh.part[rank], tid) = t;
    }
    cluster.sync();
  }
  unsigned long long total = 0ull, my_base = 0ull;
  unsigned int all = 0u;
  first = 0x7fffffff;
  for (int c = 0; c < C; ++c) {
    if (c == rank) my_base = total;
    total += sh.part[c].mass;
    all += sh.part[c].count;
    first = min(first, sh.part[c].first);
  }
  if (rank == 0 && tid == 0 && p.kept != nullptr) p.kept[r] = static_cast<int>(all);
  if (u == 0.f) {
    if (rank == 0 && tid == 0) p.tokens[r] = first;
    return;
  }
  const unsigned long long target =
      min(static_cast<unsigned long long>((double)u * (double)total), total - 1);
  for (int w = 0; w < warp; ++w) my_base += sh.red64[w];
  if (target < my_base || target >= my_base + mass) return;
  // this warp holds the drawn token
  unsigned int tie = tie_base;
  for (int v0 = v_begin; v0 < v_end; v0 += 32) {
    unsigned long long w[VE];
    bool stay[VE];
    kept_weights(v0 + lane, tie, w, stay);
    unsigned long long n = 0ull;
#pragma unroll
    for (int i = 0; i < VE; ++i) n += w[i];
    unsigned long long s = n;
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long a = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += a;
    }
    unsigned long long at = my_base + s - n;
    if (target >= at && target < at + n) {
      int id = -1;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        if (id < 0 && target < at + w[i]) id = base + (v0 + lane) * VE + i;
        at += w[i];
      }
      p.tokens[r] = id;
    }
    my_base += __shfl_sync(0xffffffffu, s, 31);
  }
}

template <typename T>
medusa_status_t launch_sample(SampleParams& p, cudaStream_t stream) {
  constexpr int VE = Elem<T>::kVec;
  // a cluster holds the row in shared memory; more blocks than that needs
  // only while a block still has 4096 tokens
  int C = 1;
  while (C < kMaxCluster && p.V > 4096 * C) C *= 2;
  const int span = p.V + VE - 1;  // the row and its offset in a 16-byte word
  p.slice = ((span + C - 1) / C + 32 * VE - 1) / (32 * VE) * (32 * VE);
  const size_t smem = (size_t)p.slice * sizeof(T) + 3 * kBins * sizeof(uint32_t) +
                      (size_t)(kBins / C) * 12;
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
