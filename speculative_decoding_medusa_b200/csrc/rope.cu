// Rotary positions: pairs of head elements rotated by an angle proportional
// to the token's position, alone or with the write of K and V into the cache.
//
//   y0 = s (x0 cos a - x1 sin a),  y1 = s (x0 sin a + x1 cos a),  a = p f_i
//
// The frequency of a pair is kept in full turns per position as a 64-bit
// fraction, so the angle modulo one turn is the low 64 bits of an integer
// product: no range reduction, and the same precision at position 1e6 as at 1
// (a fp32 product p * f would be off by 0.06 rad there).  The top 32 bits,
// taken as a quadrant and a remainder of at most 1/8 turn, go through
// sinpi / cospi in fp32 (angle error below 2^-28 turns).
//
// A token's rot / 2 sine/cosine pairs are computed once into shared memory and
// serve every head (and, in the append, q and k).  The work is units of two
// 16-byte vectors (the two halves of VEC pairs), one per thread at a time.
// Bound by HBM: every byte is read once and written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_internal.h"
#include "attn_common.cuh"
#include "common.cuh"

namespace medusa {

namespace {

constexpr int kChunk = 32;         // tokens whose metadata a block finds at once
constexpr int kSmallB = 256;       // sequences whose lengths fit in shared memory
constexpr int kRopeThreads = 384;  // largest block: several of them fit on an SM

struct RopeParams {
  const void *q, *k, *v;
  void *q_out, *k_out;  // k_out unused in the append
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  const int32_t* positions;
  const uint64_t* turns;
  float scale;
  int rot, interleaved, inverse;
  int T, Hq, Hkv, dh;
  int units, v_units;  // units of two vectors per q or k head, per v head
  // append
  const int32_t *cu_q, *kv_len, *table;
  void *K, *V;
  int B, n_pages, page_size, max_pages;
  int32_t* status;
};

// cosine and sine (times scale) of p * turns / 2^64 turns
__device__ __forceinline__ float2 turn_cos_sin(uint64_t turns, int p, float scale, float sign) {
  const uint64_t t = turns * static_cast<uint64_t>(static_cast<int64_t>(p));
  const uint32_t hi = static_cast<uint32_t>((t + 0x80000000ull) >> 32);  // 2^-32 turns
  const uint32_t quad = (hi + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(hi - (quad << 30))) * 4.656612873077393e-10f;
  const float c = cospif(x), s = sinpif(x);  // x half turns, |x| <= 1/4
  float cc = (quad & 1u) ? -s : c, ss = (quad & 1u) ? c : s;
  if (quad & 2u) {
    cc = -cc;
    ss = -ss;
  }
  return make_float2(cc * scale, ss * scale * sign);
}

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T e[VEC];
};

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }

// one thread's unit: two vectors of a q, k or v head
struct Unit {
  bool is_q, is_v, turns;
  int h, un, o0, o1;  // head, unit of the head, element offsets (o1 < 0: one vector)
};

template <int VEC>
__device__ __forceinline__ Unit unit_of(int w, int nq, int nk, const RopeParams& p) {
  Unit u;
  u.is_q = w < nq;
  u.is_v = w >= nq + nk;
  const int x = u.is_q ? w : u.is_v ? w - nq - nk : w - nq;
  const int per = u.is_v ? p.v_units : p.units;
  u.h = x / per;
  u.un = x - u.h * per;
  const int half = p.rot >> 1, rot_units = half / VEC;
  u.turns = !u.is_v && u.un < rot_units;
  if (u.turns) {
    u.o0 = p.interleaved ? u.un * 2 * VEC : u.un * VEC;
    u.o1 = p.interleaved ? u.o0 + VEC : u.o0 + half;
  } else {
    u.o0 = (u.is_v ? u.un : u.un - rot_units) * 2 * VEC + (u.is_v ? 0 : p.rot);
    u.o1 = u.o0 + VEC < p.dh ? u.o0 + VEC : -1;
  }
  return u;
}

// What a row of the append needs besides its data, found by one warp.
struct Row {
  int state;      // bit 0: the row exists, bit 1: it has a cache slot
  int pos;        // position of the token
  long long dst;  // row of kv head 0 in the pools
};

// The sequences' ends have to ascend up to T: otherwise a row may be counted to
// a sequence whose slots it has no business in, and no row is taken.
__device__ __forceinline__ bool ascends(int first, int end, const RopeParams& p) {
  return first >= 0 && end >= first && end <= p.T;
}

template <bool kAppend>
__device__ __forceinline__ Row row_of(int t, const RopeParams& p) {
  Row r{0, 0, 0};
  if (!kAppend) {
    if (t < p.T) r = Row{1, p.positions[t], 0};
    return r;
  }
  // the sequence of row t: how many sequences end at or before it
  const int lane = threadIdx.x & 31;
  int n = 0;
  bool ok = true;
  for (int b = lane; b < p.B; b += 32) {
    const int end = p.cu_q[b + 1];
    n += end <= t ? 1 : 0;
    ok = ok && ascends(p.cu_q[b], end, p);
  }
  n = __reduce_add_sync(0xffffffffu, n);
  ok = __all_sync(0xffffffffu, ok);
  if (ok && n < p.B) ok = t >= p.cu_q[n];  // (cu_q starts at 0)
  if (!ok) {
    if (lane == 0) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
    return r;
  }
  if (n < p.B) {
    r.state = 1;
    const long long at = (long long)p.kv_len[n] - p.cu_q[n + 1] + t;
    const int slot = static_cast<int>(at);
    r.pos = p.positions != nullptr ? p.positions[t] : slot;
    if (at >= 0) {
      const int pg = slot / p.page_size;
      const int id = pg < p.max_pages ? p.table[(size_t)n * p.max_pages + pg] : -1;
      if (id >= 0 && id < p.n_pages) {
        r.state = 3;
        r.dst = (long long)id * p.Hkv * p.page_size + (slot - pg * p.page_size);
      } else if (lane == 0) {
        report(p.status, MEDUSA_ERR_DEVICE_CHECK);
      }
    }
  }
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void fetch(const Unit& u, int t, const RopeParams& p, Vec<T, VEC>& a,
                                      Vec<T, VEC>& b) {
  const T* s = static_cast<const T*>(u.is_q ? p.q : u.is_v ? p.v : p.k) + (size_t)u.h * p.dh +
               t * (u.is_q ? p.q_stride : u.is_v ? p.v_stride : p.k_stride);
  a = *reinterpret_cast<const Vec<T, VEC>*>(s + u.o0);
  if (u.o1 >= 0) b = *reinterpret_cast<const Vec<T, VEC>*>(s + u.o1);
}

// Rotates the unit and stores it.  c, s: the row's cosines and sines; the
// arithmetic takes two pairs at a time (paired fp32 instructions).
template <typename T, int VEC, bool kInter, bool kAppend>
__device__ __forceinline__ void finish(const Unit& u, int t, const Row& r, const float* cos_t,
                                       const float* sin_t, const RopeParams& p, Vec<T, VEC>& a,
                                       Vec<T, VEC>& b) {
  if (r.state == 0 || (kAppend && !u.is_q && r.state != 3)) return;
  T* dst;
  if (u.is_q)
    dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + (size_t)u.h * p.dh;
  else if (kAppend)
    dst = static_cast<T*>(u.is_v ? p.V : p.K) + (r.dst + (long long)u.h * p.page_size) * p.dh;
  else
    dst = static_cast<T*>(p.k_out) + t * p.k_out_stride + (size_t)u.h * p.dh;
  if (u.turns) {
    const float *fc = cos_t + u.un * VEC, *fs = sin_t + u.un * VEC;
    T z0[VEC], z1[VEC];  // the pairs' two elements
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (kInter) {
        z0[e] = 2 * e < VEC ? a.e[(2 * e) % VEC] : b.e[(2 * e) % VEC];
        z1[e] = 2 * e + 1 < VEC ? a.e[(2 * e + 1) % VEC] : b.e[(2 * e + 1) % VEC];
      } else {
        z0[e] = a.e[e];
        z1[e] = b.e[e];
      }
    }
    if (VEC == 1) {
      const float x0 = to_f(z0[0]), x1 = to_f(z1[0]);
      from_f(z0[0], x0 * fc[0] - x1 * fs[0]);
      from_f(z1[0], x0 * fs[0] + x1 * fc[0]);
    } else {
#pragma unroll
      for (int e = 0; e + 1 < VEC; e += 2) {
        const float2 c = *reinterpret_cast<const float2*>(fc + e);
        const float2 s = *reinterpret_cast<const float2*>(fs + e);
        const uint64_t x0 = f32x2_pack(to_f(z0[e]), to_f(z0[e + 1]));
        const uint64_t x1 = f32x2_pack(to_f(z1[e]), to_f(z1[e + 1]));
        const uint64_t c2 = f32x2_pack(c.x, c.y), s2 = f32x2_pack(s.x, s.y);
        const uint64_t n2 = f32x2_pack(-s.x, -s.y);
        float y0, y1;
        f32x2_unpack(f32x2_fma(x0, c2, f32x2_mul(x1, n2)), y0, y1);
        from_f(z0[e], y0);
        from_f(z0[e + 1], y1);
        f32x2_unpack(f32x2_fma(x0, s2, f32x2_mul(x1, c2)), y0, y1);
        from_f(z1[e], y0);
        from_f(z1[e + 1], y1);
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (kInter) {
        if (2 * e < VEC) a.e[(2 * e) % VEC] = z0[e];
        else b.e[(2 * e) % VEC] = z0[e];
        if (2 * e + 1 < VEC) a.e[(2 * e + 1) % VEC] = z1[e];
        else b.e[(2 * e + 1) % VEC] = z1[e];
      } else {
        a.e[e] = z0[e];
        b.e[e] = z1[e];
      }
    }
  }
  *reinterpret_cast<Vec<T, VEC>*>(dst + u.o0) = a;
  if (u.o1 >= 0) *reinterpret_cast<Vec<T, VEC>*>(dst + u.o1) = b;
}

// A block per token.  The first unit's loads go out before anything else: they
// depend on no metadata, and hide the chain sequence -> slot -> page -> angle
// behind them.
template <typename T, int VEC, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_block_kernel(RopeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ float cs[];  // cosines [rot / 2], then the sines
  __shared__ Row s_row;
  const int t = blockIdx.x, tid = threadIdx.x;
  const int half = p.rot >> 1;
  const int nq = p.q != nullptr ? p.Hq * p.units : 0;
  const int nk = p.k != nullptr ? p.Hkv * p.units : 0;
  const int total = nq + nk + (kAppend ? p.Hkv * p.v_units : 0);
  Vec<T, VEC> a, b;
  int w = tid;
  Unit u{};
  if (w < total) {
    u = unit_of<VEC>(w, nq, nk, p);
    fetch<T, VEC>(u, t, p, a, b);
  }
  if (tid < 32) {
    const Row r = row_of<kAppend>(t, p);
    if (tid == 0) s_row = r;
  }
  __syncthreads();
  const Row r = s_row;
  for (int i = tid; i < half; i += blockDim.x) {
    const float2 f = turn_cos_sin(p.turns[i], r.pos, p.scale, p.inverse ? -1.f : 1.f);
    cs[i] = f.x;
    cs[half + i] = f.y;
  }
  __syncthreads();
  while (w < total) {
    finish<T, VEC, kInter, kAppend>(u, t, r, cs, cs + half, p, a, b);
    w += blockDim.x;
    if (w < total) {
      u = unit_of<VEC>(w, nq, nk, p);
      fetch<T, VEC>(u, t, p, a, b);
    }
  }
}

// What row_of finds, by one thread, with the sequences' lengths in cu and kv
// (shared memory, or global where they do not fit).
template <bool kAppend>
__device__ __forceinline__ Row row_of_thread(uint32_t token, const int* cu, const int* kv,
                                             const RopeParams& p) {
  Row r{0, 0, 0};
  if (token >= static_cast<uint32_t>(p.T)) return r;
  const int t = static_cast<int>(token);
  if (!kAppend) return Row{1, p.positions[t], 0};
  int lo = 0, hi = p.B;  // the first sequence that ends after t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  if (lo >= p.B) return r;
  if (t < cu[lo]) {  // cu_q does not start at 0
    report(p.status, MEDUSA_ERR_DEVICE_CHECK);
    return r;
  }
  r.state = 1;
  const long long at = (long long)kv[lo] - cu[lo + 1] + t;
  const int slot = static_cast<int>(at);
  r.pos = p.positions != nullptr ? p.positions[t] : slot;
  if (at >= 0) {
    const int pg = slot / p.page_size;
    const int id = pg < p.max_pages ? p.table[(size_t)lo * p.max_pages + pg] : -1;
    if (id >= 0 && id < p.n_pages) {
      r.state = 3;
      r.dst = (long long)id * p.Hkv * p.page_size + (slot - pg * p.page_size);
    } else {
      report(p.status, MEDUSA_ERR_DEVICE_CHECK);
    }
  }
  return r;
}

// Many tokens, a thread per unit: resident blocks walk the tokens in chunks of
// kChunk, whose metadata they find at once, with the next token's data and
// angles on their way while they finish the current one; one barrier a token.
// 8192 tokens of 32 + 8 heads written into pages (214 MB): 46.3 us
// (4.6 TB/s of the 6.55 that a copy reaches; 33 us at that), against
// 60 us with a block per token, whose latencies only other blocks cover, and
// 54 us with each token's metadata found two tokens ahead (its chain of three
// reads was as long as a token's turn).  A token of more units than a block has
// threads (64 + 8 or 32 + 32 heads of 128 in bf16, 32 + 8 in fp32) takes a block
// of its own: 80, 90 and 76 us for 8192 of them (4.5, 4.7 and 5.7 TB/s).
template <typename T, int VEC, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_pipe_kernel(RopeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ float cs[];  // two tokens' cosines and sines
  __shared__ Row s_row[kChunk];
  __shared__ int s_cu[kAppend ? kSmallB + 1 : 1], s_kv[kAppend ? kSmallB : 1];
  const int tid = threadIdx.x;
  // (T may lie just below 2^31: tokens ahead of the current one pass it)
  const uint32_t n_tok = static_cast<uint32_t>(p.T), step = gridDim.x;
  const int half = p.rot >> 1;
  const int nq = p.q != nullptr ? p.Hq * p.units : 0;
  const int nk = p.k != nullptr ? p.Hkv * p.units : 0;
  const int total = nq + nk + (kAppend ? p.Hkv * p.v_units : 0);
  const bool works = tid < total;
  const Unit u = unit_of<VEC>(works ? tid : 0, nq, nk, p);
  const float sign = p.inverse ? -1.f : 1.f;
  auto angles = [&](int pos, float* table) {
    for (int i = tid; i < half; i += blockDim.x) {
      const float2 f = turn_cos_sin(p.turns[i], pos, p.scale, sign);
      table[i] = f.x;
      table[half + i] = f.y;
    }
  };
  Vec<T, VEC> a, b, a2, b2;
  uint32_t t = blockIdx.x;
  if (works && t < n_tok) fetch<T, VEC>(u, t, p, a, b);
  const bool small = kAppend && p.B <= kSmallB;
  if (kAppend) {
    bool ok = true;
    for (int i = tid; i < p.B; i += blockDim.x) {
      const int first = p.cu_q[i], end = p.cu_q[i + 1];
      ok = ok && ascends(first, end, p);
      if (small) {
        if (i == 0) s_cu[0] = first;
        s_cu[i + 1] = end;
        s_kv[i] = p.kv_len[i];
      }
    }
    if (!__syncthreads_and(ok)) {
      if (blockIdx.x == 0 && tid == 0) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
      return;
    }
  }
  int parity = 0;
  while (t < n_tok) {
    if (tid < kChunk)
      s_row[tid] = row_of_thread<kAppend>(t + tid * step, small ? s_cu : p.cu_q,
                                          small ? s_kv : p.kv_len, p);
    __syncthreads();
    angles(s_row[0].pos, cs + parity * 2 * half);
    __syncthreads();
    for (int j = 0; j < kChunk && t < n_tok; ++j, t += step) {
      const float* table = cs + parity * 2 * half;
      parity ^= 1;
      if (t + step < n_tok) {
        if (works) fetch<T, VEC>(u, t + step, p, a2, b2);
        if (j + 1 < kChunk) angles(s_row[j + 1].pos, cs + parity * 2 * half);
      }
      if (works) finish<T, VEC, kInter, kAppend>(u, t, s_row[j], table, table + half, p, a, b);
      __syncthreads();
      a = a2;
      b = b2;
    }
  }
}

// A rotated part that whole vectors do not divide (an odd number of pairs, as
// in rot = 34): a block per token holds the token's q, k and v in shared memory,
// read and written by whole vectors whatever the rotation, and every element
// finds its partner there.  8192 tokens of 32 + 8 heads of 128 with rot = 34
// written into pages: 81 us, with vectors as narrow as the pairs allow 154.
template <typename T, int VEC, bool kAppend>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_staged_kernel(RopeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ __align__(16) uint8_t staged[];  // the token, cosines [rot / 2], sines
  __shared__ Row s_row;
  using V = Vec<T, VEC>;
  V* token = reinterpret_cast<V*>(staged);
  const int t = blockIdx.x, tid = threadIdx.x;
  const int half = p.rot >> 1, per = p.dh / VEC;  // vectors of a head
  const int nq = p.q != nullptr ? p.Hq * per : 0;
  const int nk = p.k != nullptr ? p.Hkv * per : 0;
  const int total = nq + nk + (kAppend ? p.Hkv * per : 0);
  float* cs = reinterpret_cast<float*>(token + total);
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + t * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + t * p.v_stride;
  for (int w = tid; w < total; w += blockDim.x)
    token[w] = w < nq        ? reinterpret_cast<const V*>(q)[w]
               : w < nq + nk ? reinterpret_cast<const V*>(k)[w - nq]
                             : reinterpret_cast<const V*>(v)[w - nq - nk];
  if (tid < 32) {
    const Row r = row_of<kAppend>(t, p);
    if (tid == 0) s_row = r;
  }
  __syncthreads();
  const Row r = s_row;
  for (int i = tid; i < half; i += blockDim.x) {
    const float2 f = turn_cos_sin(p.turns[i], r.pos, p.scale, p.inverse ? -1.f : 1.f);
    cs[i] = f.x;
    cs[half + i] = f.y;
  }
  __syncthreads();
  if (r.state == 0) return;
  for (int w = tid; w < total; w += blockDim.x) {
    const bool is_q = w < nq, is_v = w >= nq + nk;
    const int x = is_q ? w : is_v ? w - nq - nk : w - nq;
    const int h = x / per, j0 = (x - h * per) * VEC;
    if (kAppend && !is_q && r.state != 3) continue;
    V a = token[w];
    if (!is_v && j0 < p.rot) {
      const T* head = reinterpret_cast<const T*>(token + (w - j0 / VEC));
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = j0 + e;
        if (j >= p.rot) break;
        const bool second = p.interleaved ? (j & 1) != 0 : j >= half;
        const int i = p.interleaved ? j >> 1 : second ? j - half : j;
        const int partner = p.interleaved ? j ^ 1 : second ? j - half : j + half;
        const float c = cs[i], s = cs[half + i], z = to_f(a.e[e]), y = to_f(head[partner]);
        from_f(a.e[e], second ? fmaf(y, s, z * c) : fmaf(z, c, -(y * s)));
      }
    }
    T* dst;
    if (is_q)
      dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + (size_t)h * p.dh;
    else if (kAppend)
      dst = static_cast<T*>(is_v ? p.V : p.K) + (r.dst + (long long)h * p.page_size) * p.dh;
    else
      dst = static_cast<T*>(p.k_out) + t * p.k_out_stride + (size_t)h * p.dh;
    *reinterpret_cast<V*>(dst + j0) = a;
  }
}

// the widest vector every access allows: VEC elements must divide `part`, the
// head, every stride and (in bytes) every base address
int vector_width(const RopeParams& p, int eb, long long part) {
  uintptr_t addr = 0;
  long long step = part;
  auto take = [&](const void* ptr, long long stride) {
    if (ptr == nullptr) return;
    addr |= reinterpret_cast<uintptr_t>(ptr);
    step |= stride;
  };
  step |= p.dh;
  take(p.q, p.q_stride);
  take(p.q_out, p.q_out_stride);
  take(p.k, p.k_stride);
  take(p.k_out, p.k_out_stride);
  take(p.v, p.v_stride);
  take(p.K, 0);
  take(p.V, 0);
  int vec = 16 / eb;
  while (vec > 1 && (step % vec != 0 || addr % (vec * eb) != 0)) vec >>= 1;
  return vec;
}

template <typename T, int VEC, bool kAppend>
medusa_status_t launch_vec(RopeParams& p, cudaStream_t stream) {
  p.units = p.rot / (2 * VEC) + (p.dh - p.rot + 2 * VEC - 1) / (2 * VEC);
  p.v_units = (p.dh + 2 * VEC - 1) / (2 * VEC);
  const int work = (p.q ? p.Hq * p.units : 0) + (p.k ? p.Hkv * p.units : 0) +
                   (kAppend ? p.Hkv * p.v_units : 0);
  const int rounds = (work + kRopeThreads - 1) / kRopeThreads;
  const int threads = ((work + rounds - 1) / rounds + 31) / 32 * 32;
  const size_t table = (p.rot / 2) * sizeof(float);
  // resident blocks once they have several tokens each (8192 tokens of 1 + 1
  // heads appended: 24 us with three blocks an SM, 10 with as many as fit)
  const int resident = min(3 * kRopeThreads / threads, 32) * device_sm_count();
  if (work <= kRopeThreads && p.T >= 2 * resident) {
    if (p.interleaved)
      launch(rope_pipe_kernel<T, VEC, true, kAppend>, resident, threads, 4 * table, stream, p);
    else
      launch(rope_pipe_kernel<T, VEC, false, kAppend>, resident, threads, 4 * table, stream, p);
  } else if (p.interleaved) {
    launch(rope_block_kernel<T, VEC, true, kAppend>, p.T, threads, 2 * table, stream, p);
  } else {
    launch(rope_block_kernel<T, VEC, false, kAppend>, p.T, threads, 2 * table, stream, p);
  }
  return check_launch(kAppend ? "rope_append" : "rope");
}

template <typename T, int VEC, bool kAppend>
medusa_status_t launch_staged(RopeParams& p, size_t smem, cudaStream_t stream) {
  const int total = ((p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0) + (kAppend ? p.Hkv : 0)) * (p.dh / VEC);
  const int rounds = (total + kRopeThreads - 1) / kRopeThreads;
  const int threads = ((total + rounds - 1) / rounds + 31) / 32 * 32;
  launch(rope_staged_kernel<T, VEC, kAppend>, p.T, threads, smem, stream, p);
  return check_launch(kAppend ? "rope_append" : "rope");
}

template <bool kAppend>
medusa_status_t dispatch(RopeParams& p, medusa_dtype_t dt, cudaStream_t stream) {
  const int eb = dt == MEDUSA_BF16 ? 2 : 4;
  const int width = vector_width(p, eb, p.rot / 2), apart = vector_width(p, eb, 0);
  const size_t smem = ((size_t)(p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0) + (kAppend ? p.Hkv : 0)) *
                          p.dh * eb +
                      (size_t)p.rot * sizeof(float);
  if (width < apart && smem <= 48 * 1024 - 64) {
    if (dt == MEDUSA_BF16) {
      switch (apart) {
        case 8: return launch_staged<__nv_bfloat16, 8, kAppend>(p, smem, stream);
        case 4: return launch_staged<__nv_bfloat16, 4, kAppend>(p, smem, stream);
        default: return launch_staged<__nv_bfloat16, 2, kAppend>(p, smem, stream);
      }
    }
    if (apart == 4) return launch_staged<float, 4, kAppend>(p, smem, stream);
    return launch_staged<float, 2, kAppend>(p, smem, stream);
  }
  if (dt == MEDUSA_BF16) {
    switch (width) {
      case 8: return launch_vec<__nv_bfloat16, 8, kAppend>(p, stream);
      case 4: return launch_vec<__nv_bfloat16, 4, kAppend>(p, stream);
      case 2: return launch_vec<__nv_bfloat16, 2, kAppend>(p, stream);
      default: return launch_vec<__nv_bfloat16, 1, kAppend>(p, stream);
    }
  }
  switch (width) {
    case 4: return launch_vec<float, 4, kAppend>(p, stream);
    case 2: return launch_vec<float, 2, kAppend>(p, stream);
    default: return launch_vec<float, 1, kAppend>(p, stream);
  }
}

}  // namespace

medusa_status_t rope_freqs(int rot, double theta, medusa_rope_scaling_t scaling, double factor,
                           double low_turns, double high_turns, double original_max_position,
                           uint64_t* turns, float* scale) {
  const long double two_pi = 6.283185307179586476925286766559L;
  const long double lt = logl((long double)theta);
  long double lo = 0.0L, hi = 0.0L;
  *scale = 1.f;
  if (scaling == MEDUSA_ROPE_YARN) {
    // the indices whose pairs make high_turns and low_turns full turns over
    // the original length
    const long double lo_len = logl(two_pi * high_turns), hi_len = logl(two_pi * low_turns);
    const long double len = logl((long double)original_max_position);
    lo = fmaxl(floorl(rot * (len - lo_len) / (2.0L * lt)), 0.0L);
    hi = fminl(ceill(rot * (len - hi_len) / (2.0L * lt)), (long double)(rot - 1));
    *scale = (float)(0.1 * log(factor) + 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    long double f = expl(-2.0L * i / rot * lt);
    long double keep = 1.0L;  // share of the unscaled frequency
    if (scaling == MEDUSA_ROPE_LINEAR) {
      keep = 0.0L;
    } else if (scaling == MEDUSA_ROPE_LLAMA3) {
      const long double n = f * original_max_position / two_pi;
      keep = fminl(fmaxl((n - low_turns) / (high_turns - low_turns), 0.0L), 1.0L);
    } else if (scaling == MEDUSA_ROPE_YARN) {
      keep = 1.0L - fminl(fmaxl((i - lo) / fmaxl(hi - lo, 1e-3L), 0.0L), 1.0L);
    }
    f = f * keep + f / factor * (1.0L - keep);
    turns[i] = (uint64_t)(f / two_pi * 18446744073709551616.0L + 0.5L);
  }
  return MEDUSA_OK;
}

medusa_status_t rope(const medusa_rope_t& r, const void* q, long long q_stride, const void* k,
                     long long k_stride, medusa_dtype_t dt, const int32_t* positions, int T,
                     int Hq, int Hkv, int dh, int inverse, void* q_out, long long q_out_stride,
                     void* k_out, long long k_out_stride, cudaStream_t stream) {
  RopeParams p{};
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.positions = positions;
  p.turns = r.turns;
  p.scale = r.scale;
  p.rot = r.rot;
  p.interleaved = r.interleaved;
  p.inverse = inverse;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.dh = dh;
  return dispatch<false>(p, dt, stream);
}

medusa_status_t rope_append(const medusa_rope_t* r, const void* q, long long q_stride,
                            const void* k, long long k_stride, const void* v, long long v_stride,
                            medusa_dtype_t dt, const int32_t* positions, const int32_t* cu_q,
                            const int32_t* kv_len, int B, int T, int Hq, int Hkv, int dh,
                            void* q_out, long long q_out_stride, const medusa_pages_t& pages,
                            int32_t* status, cudaStream_t stream) {
  RopeParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.positions = positions;
  p.scale = 1.f;
  if (r != nullptr) {
    p.turns = r->turns;
    p.scale = r->scale;
    p.rot = r->rot;
    p.interleaved = r->interleaved;
  }
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.dh = dh;
  p.cu_q = cu_q;
  p.kv_len = kv_len;
  p.B = B;
  p.table = pages.table;
  p.K = pages.K;
  p.V = pages.V;
  p.n_pages = pages.n_pages;
  p.page_size = pages.page_size;
  p.max_pages = pages.max_pages;
  p.status = status;
  return dispatch<true>(p, dt, stream);
}

}  // namespace medusa
