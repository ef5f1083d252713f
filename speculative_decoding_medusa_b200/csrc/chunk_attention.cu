// Attention of a chunk of new tokens over a paged cache.
//
//   out[t, h] = sum_j softmax_j(scale q.k_j) v_j  over slots j <= p(t)
//
// One warp per (token, query head) on CUDA cores: lanes split the head, eight
// keys are in flight per online-softmax update, fp32 throughout.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_internal.h"
#include "chunk_attention.cuh"
#include "common.cuh"

namespace medusa {

namespace {

__device__ __forceinline__ float ld(const __nv_bfloat16* x) { return __bfloat162float(*x); }
__device__ __forceinline__ float ld(const float* x) { return *x; }
__device__ __forceinline__ void st(__nv_bfloat16* d, float x) { *d = __float2bfloat16_rn(x); }
__device__ __forceinline__ void st(float* d, float x) { *d = x; }

template <typename T, int PER>
__global__ void __launch_bounds__(256) chunk_attn_row_kernel(ChunkParams p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int DH = PER * 32;
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)p.T * p.Hq;
  for (long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); w < rows;
       w += (long long)gridDim.x * 8) {
    const int t = static_cast<int>(w / p.Hq), hq = static_cast<int>(w - (long long)t * p.Hq);
    int n = 0;
    for (int b = lane; b < p.B; b += 32) n += p.cu_q[b + 1] <= t ? 1 : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= p.B) continue;  // behind the last sequence
    const int first = p.cu_q[n], len = p.cu_q[n + 1] - first, kv = p.kv_len[n];
    if (first < 0 || t < first || first + len > p.T || kv < 0 || kv > (long long)p.max_pages * p.page_size) {
      if (lane == 0) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
      continue;
    }
    const int visible = max(0, kv - len + (t - first) + 1);
    const T* qp = static_cast<const T*>(p.q) + t * p.q_stride + (size_t)hq * DH + lane * PER;
    float qv[PER], acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      qv[e] = ld(qp + e) * p.scale;
      acc[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j0 = 0; j0 < visible;) {
      const int pg = j0 / p.page_size, r0 = j0 - pg * p.page_size;
      const int id = p.table[(size_t)n * p.max_pages + pg];
      const int end = min(visible, j0 - r0 + p.page_size);
      if (id < 0 || id >= p.n_pages) {
        if (lane == 0) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
        j0 = end;
        continue;
      }
      const size_t row = ((size_t)id * p.Hkv + hq / p.G) * p.page_size + r0;
      const T* kp = static_cast<const T*>(p.K) + row * DH + lane * PER;
      const T* vp = static_cast<const T*>(p.V) + row * DH + lane * PER;
      for (; j0 < end; j0 += 8) {
        const int nk = min(8, end - j0);
        float s[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          float d = 0.f;
          if (x < nk) {
#pragma unroll
            for (int e = 0; e < PER; ++e) d += qv[e] * ld(kp + (size_t)x * DH + e);
          }
          s[x] = d;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int x = 0; x < 8; ++x) s[x] += __shfl_xor_sync(0xffffffffu, s[x], o);
        float mn = m;
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (x < nk) mn = fmaxf(mn, s[x]);
        const float corr = expf(m - mn);
        l *= corr;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] *= corr;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          if (x < nk) {
            const float pw = expf(s[x] - mn);
            l += pw;
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] += pw * ld(vp + (size_t)x * DH + e);
          }
        }
        m = mn;
        kp += 8 * DH;
        vp += 8 * DH;
      }
      j0 = end;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    T* o = static_cast<T*>(p.out) + (size_t)w * DH + lane * PER;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const float y = acc[e] * inv;
      finite = finite && isfinite(y);
      st(o + e, y);
    }
    if (!finite) report(p.status, MEDUSA_ERR_DEVICE_CHECK);
  }
}

template <typename T>
medusa_status_t launch_rows(const ChunkParams& p, int dh, cudaStream_t stream) {
  const long long blocks = ((long long)p.T * p.Hq + 7) / 8;
  const int grid = (int)(blocks < 148 * 64 ? blocks : 148 * 64);
  switch (dh / 32) {
    case 1: launch(chunk_attn_row_kernel<T, 1>, grid, 256, 0, stream, p); break;
    case 2: launch(chunk_attn_row_kernel<T, 2>, grid, 256, 0, stream, p); break;
    case 3: launch(chunk_attn_row_kernel<T, 3>, grid, 256, 0, stream, p); break;
    case 4: launch(chunk_attn_row_kernel<T, 4>, grid, 256, 0, stream, p); break;
    case 5: launch(chunk_attn_row_kernel<T, 5>, grid, 256, 0, stream, p); break;
    case 6: launch(chunk_attn_row_kernel<T, 6>, grid, 256, 0, stream, p); break;
    case 7: launch(chunk_attn_row_kernel<T, 7>, grid, 256, 0, stream, p); break;
    default: launch(chunk_attn_row_kernel<T, 8>, grid, 256, 0, stream, p); break;
  }
  return check_launch("chunk_attention");
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
  return launch_rows<float>(p, dh, stream);
}

}  // namespace medusa
