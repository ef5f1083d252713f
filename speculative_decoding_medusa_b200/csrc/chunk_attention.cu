// Attention of a chunk of new tokens over a paged cache, fp32.
//
//   out[t, h] = sum_j softmax_j(scale q.k_j) v_j  over slots j <= p(t)
//
// CUDA cores, fp32 throughout.  A unit (a token and up to four query heads of
// one kv head, whose K and V rows it reads once) belongs to S warps of a block,
// which take its keys eight at a time in turn and merge their maxima, sums and
// outputs through shared memory; S is as large as leaves the machine's warps
// enough units (a 128-token prompt of four heads is 512: one warp each would
// leave nine tenths of the machine idle: 27 us against 6.5).  Of a step's eight
// keys the lanes split the head; the eight products are summed over the warp by
// halving (9 exchanges for 8 sums), so that each lane ends with one key's score
// and computes one exponential.  Bound by latency at the smallest sizes, by the
// reads of K and V from L2 at larger ones: 150 tokens of 56 + 8 heads of 128
// over 200 to 300 slots 118 us, with a head to a unit 314.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_internal.h"
#include "chunk_attention.cuh"
#include "common.cuh"

namespace medusa {

namespace {

constexpr int kWarps = 8;

template <int PER, int R>
__global__ void __launch_bounds__(kWarps * 32) chunk_attn_f32_kernel(ChunkParams p, int S) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int DH = PER * 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int units = kWarps / S;  // of a block
  const int split = warp % S;
  __shared__ float s_ml[kWarps][R][2];
  __shared__ float s_acc[kWarps][R][DH];
  // a unit: a token and up to R query heads of one kv head
  const int lots = (p.G + R - 1) / R;
  const long long unit = (long long)blockIdx.x * units + warp / S;
  int visible = 0, n = 0;
  bool live = unit < (long long)p.T * p.Hkv * lots;
  const int t = live ? static_cast<int>(unit / (p.Hkv * lots)) : 0;
  const int in = live ? static_cast<int>(unit - (long long)t * p.Hkv * lots) : 0;
  const int kvh = in / lots, g0 = (in - kvh * lots) * R, hq = kvh * p.G + g0;
  const int nr = min(R, p.G - g0);  // heads of the unit
  // q needs no metadata: its load runs beside the chain lengths -> page -> keys
  float qv[R][PER], acc[R][PER], m[R], l[R];
  const float* qp = static_cast<const float*>(p.q) + t * p.q_stride + (size_t)hq * DH + lane * PER;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < PER; ++e) qv[r][e] = live && r < nr ? qp[r * DH + e] : 0.f;
  if (live) {
    int first = 0, end = 0, kv = 0;  // of sequence `lane`, then of the row's
    // The row's sequence is found by counting the ends at or before it, which
    // says nothing unless they ascend: every warp checks all lengths, and none
    // computes a row of a call that fails.
    const long long slots = (long long)p.max_pages * p.page_size;
    auto in_range = [&](int a, int e, int k) {
      return a >= 0 && e >= a && e <= p.T && k >= 0 && k <= slots;
    };
    bool ok = true;
    if (lane < p.B) {
      first = p.cu_q[lane];
      end = p.cu_q[lane + 1];
      kv = p.kv_len[lane];
      n = end <= t ? 1 : 0;
      ok = in_range(first, end, kv);
    }
    for (int b = lane + 32; b < p.B; b += 32) {
      const int e = p.cu_q[b + 1];
      n += e <= t ? 1 : 0;
      ok = ok && in_range(p.cu_q[b], e, p.kv_len[b]);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    live = n < p.B;  // not behind the last sequence
    if (!__all_sync(0xffffffffu, ok)) {
      if (lane == 0) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
      live = false;
    }
    if (live) {
      if (n < 32) {
        first = __shfl_sync(0xffffffffu, first, n);
        end = __shfl_sync(0xffffffffu, end, n);
        kv = __shfl_sync(0xffffffffu, kv, n);
      } else {
        first = p.cu_q[n];
        end = p.cu_q[n + 1];
        kv = p.kv_len[n];
      }
      if (t < first) {  // cu_q does not start at 0
        if (lane == 0) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
        live = false;
      } else {
        visible = max(0, kv - end + t + 1);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      qv[r][e] *= p.scale;
      acc[r][e] = 0.f;
    }
  }
  const float* Kp = static_cast<const float*>(p.K) + lane * PER;
  const float* Vp = static_cast<const float*>(p.V) + lane * PER;
  const int mine = (lane >> 2) & 7;  // the key whose score this lane ends with
  // (unsigned: a sequence may fill an int with slots)
  const uint32_t n_vis = visible, page_size = p.page_size;
  for (uint32_t j0 = split * 8; j0 < n_vis; j0 += S * 8) {
    const uint32_t nk = min(8u, n_vis - j0);
    size_t at[8];  // element offset of each key's row
    unsigned int have = (1u << nk) - 1u;
    const uint32_t pg0 = j0 / page_size, r0 = j0 - pg0 * page_size;
    if (r0 + nk <= page_size) {  // the eight lie in one page
      const int id = p.table[(size_t)n * p.max_pages + pg0];
      if (id < 0 || id >= p.n_pages) have = 0u;
      const size_t first =
          (((size_t)max(id, 0) * p.Hkv + kvh) * p.page_size + r0) * DH;
#pragma unroll
      for (int x = 0; x < 8; ++x) at[x] = first + (size_t)x * DH;
    } else {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint32_t j = min(j0 + x, n_vis - 1), pg = j / page_size;
        const int id = p.table[(size_t)n * p.max_pages + pg];
        at[x] = 0;
        if (id >= 0 && id < p.n_pages)
          at[x] = (((size_t)id * p.Hkv + kvh) * p.page_size + (j - pg * page_size)) * DH;
        else
          have &= ~(1u << x);
      }
    }
    if (have != (1u << nk) - 1u && lane == 0) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
    float d[R][8], v[8][PER];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      float k[PER];
#pragma unroll
      for (int e = 0; e < PER; ++e) k[e] = v[x][e] = 0.f;
      if ((have >> x) & 1u) {
#pragma unroll
        for (int e = 0; e < PER; ++e) k[e] = Kp[at[x] + e];
#pragma unroll
        for (int e = 0; e < PER; ++e) v[x][e] = Vp[at[x] + e];
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        d[r][x] = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) d[r][x] += qv[r][e] * k[e];
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // lanes with bit 4 set keep keys 4-7, with bit 3 the upper two of those, ...
#pragma unroll
      for (int o = 16, w = 4; o >= 4; o >>= 1, w >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (x >= w) break;
          const float send = up ? d[r][x] : d[r][x + w], keep = up ? d[r][x + w] : d[r][x];
          d[r][x] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
      float s = d[r][0];
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      if (!((have >> mine) & 1u)) s = -INFINITY;
      float mn = s;
#pragma unroll
      for (int o = 16; o >= 4; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mn = fmaxf(mn, m[r]);
      // a NaN score stays NaN; a step without a page adds nothing
      const float w = mn == -INFINITY && s == -INFINITY ? 0.f : expf(s - mn);
      float sum = w;
#pragma unroll
      for (int o = 16; o >= 4; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float corr = m[r] == -INFINITY ? 0.f : expf(m[r] - mn);
      l[r] = l[r] * corr + sum;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[r][e] *= corr;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float wx = __shfl_sync(0xffffffffu, w, x * 4);
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[r][e] += wx * v[x][e];
      }
      m[r] = mn;
    }
  }
  if (S > 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (lane == 0) {
        s_ml[warp][r][0] = m[r];
        s_ml[warp][r][1] = l[r];
      }
#pragma unroll
      for (int e = 0; e < PER; ++e) s_acc[warp][r][lane * PER + e] = acc[r][e];
    }
    __syncthreads();
    if (split != 0) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float M = m[r];
      for (int x = 1; x < S; ++x) M = fmaxf(M, s_ml[warp + x][r][0]);
      const float c0 = m[r] == -INFINITY ? 0.f : expf(m[r] - M);
      l[r] *= c0;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[r][e] *= c0;
      for (int x = 1; x < S; ++x) {
        if (s_ml[warp + x][r][0] == -INFINITY) continue;  // no key
        const float c = expf(s_ml[warp + x][r][0] - M);
        l[r] += c * s_ml[warp + x][r][1];
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[r][e] += c * s_acc[warp + x][r][lane * PER + e];
      }
    }
  }
  if (!live) return;
  float* o = static_cast<float*>(p.out) + ((size_t)t * p.Hq + hq) * DH + lane * PER;
  bool finite = true;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= nr) break;
    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const float y = acc[r][e] * inv;
      finite = finite && isfinite(y);
      o[r * DH + e] = y;
    }
  }
  if (!finite) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
}

template <int PER, int R>
medusa_status_t launch_units(const ChunkParams& p, cudaStream_t stream) {
  const long long units = (long long)p.T * p.Hkv * ((p.G + R - 1) / R);
  int S = kWarps;
  while (S > 1 && units * S > (long long)device_sm_count() * 48) S >>= 1;
  const long long blocks = (units * S + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return fail(MEDUSA_ERR_SHAPE, "chunk_attention: T * Hq too large");
  launch(chunk_attn_f32_kernel<PER, R>, static_cast<int>(blocks), kWarps * 32, 0, stream, p, S);
  return check_launch("chunk_attention");
}

// heads of a unit: four keep a head of 128 in 128 registers, of more than 128
// two do
template <int PER>
medusa_status_t launch_heads(const ChunkParams& p, cudaStream_t stream) {
  if (p.G == 1) return launch_units<PER, 1>(p, stream);
  if (p.G == 2 || PER > 4) return launch_units<PER, 2>(p, stream);
  return launch_units<PER, 4>(p, stream);
}

medusa_status_t launch_f32(const ChunkParams& p, int dh, cudaStream_t stream) {
  switch (dh / 32) {
    case 1: return launch_heads<1>(p, stream);
    case 2: return launch_heads<2>(p, stream);
    case 3: return launch_heads<3>(p, stream);
    case 4: return launch_heads<4>(p, stream);
    case 5: return launch_heads<5>(p, stream);
    case 6: return launch_heads<6>(p, stream);
    case 7: return launch_heads<7>(p, stream);
    default: return launch_heads<8>(p, stream);
  }
}

}  // namespace

size_t chunk_attention_workspace_size(int Hq, int Hkv, int dh, medusa_dtype_t dt) {
  (void)Hq;
  (void)Hkv;
  return dt == MEDUSA_BF16 ? chunk_attention_tc_workspace(dh) : 0;
}

medusa_status_t chunk_attention(const void* q, long long q_stride, const medusa_pages_t& pages,
                                medusa_dtype_t dt, const int32_t* cu_q, const int32_t* kv_len,
                                int B, int T, int Hq, int Hkv, int dh, float scale, void* out,
                                void* ws, int32_t* status, cudaStream_t stream) {
  ChunkParams p{q, q_stride, pages.K, pages.V, pages.table, cu_q, kv_len, pages.n_pages,
                pages.page_size, pages.max_pages, B, T, Hq, Hkv, Hq / Hkv, scale, out, status};
  if (dt == MEDUSA_BF16) return chunk_attention_tc(p, dh, ws, stream);
  return launch_f32(p, dh, stream);
}

}  // namespace medusa
