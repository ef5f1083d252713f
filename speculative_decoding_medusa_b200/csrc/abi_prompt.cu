// The C entry points of the prompt side (rotary positions, paged chunk
// attention, sampling): argument checks, then the launchers.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_internal.h"

using medusa::fail;

namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool valid_dtype(medusa_dtype_t d) { return d == MEDUSA_BF16 || d == MEDUSA_F32; }

medusa_status_t check_rotation(const medusa_rope_t* r, int dh) {
  if (r->turns == nullptr) return fail(MEDUSA_ERR_INVALID_ARG, "rope: null turns");
  if (r->rot < 2 || r->rot % 2 != 0 || r->rot > 512 || r->rot > dh)
    return fail(MEDUSA_ERR_SHAPE, "rope: rot must be even, in [2, 512] and <= dh");
  if (!aligned(r->turns, 8)) return fail(MEDUSA_ERR_ALIGNMENT, "rope: turns not 8-byte aligned");
  return MEDUSA_OK;
}

// one operand [T, H, dh]
medusa_status_t check_operand(const void* x, long long stride, int T, int H, int dh, size_t eb) {
  if (x == nullptr) return fail(MEDUSA_ERR_INVALID_ARG, "rope: null pointer");
  if (T > 1 && stride < (long long)H * dh)
    return fail(MEDUSA_ERR_SHAPE, "rope: a token stride is below heads * dh");
  if (!aligned(x, eb)) return fail(MEDUSA_ERR_ALIGNMENT, "rope: pointer not aligned to its type");
  return MEDUSA_OK;
}

struct Span {
  const void* p;
  long long stride;  // elements between tokens
  int H;
};

// whether two operands of T tokens share a byte; slices of one buffer with the
// same stride may interleave
bool overlap(const Span& x, const Span& y, int T, int dh, size_t eb) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  const uintptr_t wa = (uintptr_t)x.H * dh * eb, wb = (uintptr_t)y.H * dh * eb;
  const uintptr_t na = (uintptr_t)(T - 1) * x.stride * eb + wa;
  const uintptr_t nb = (uintptr_t)(T - 1) * y.stride * eb + wb;
  if (a + na <= b || b + nb <= a) return false;
  if (T == 1 || x.stride != y.stride) return true;
  const uintptr_t row = (uintptr_t)x.stride * eb;
  const uintptr_t d = b >= a ? (b - a) % row : (row - (a - b) % row) % row;  // of y's row in x's
  return d < wa || d + wb > row;
}

// an output is its input (same stride) or shares no byte with it
medusa_status_t check_in_place(const Span& in, const Span& out, int T, int dh, size_t eb) {
  if (in.p == out.p) {
    if (T > 1 && in.stride != out.stride)
      return fail(MEDUSA_ERR_INVALID_ARG, "rope: in place needs equal strides");
    return MEDUSA_OK;
  }
  if (overlap(in, out, T, dh, eb))
    return fail(MEDUSA_ERR_INVALID_ARG, "rope: an output overlaps its input");
  return MEDUSA_OK;
}

medusa_status_t check_pages(const medusa_pages_t* p, size_t align) {
  if (p == nullptr || p->K == nullptr || p->V == nullptr || p->table == nullptr)
    return fail(MEDUSA_ERR_INVALID_ARG, "pages: null pointer");
  if (p->n_pages < 1 || p->page_size < 1 || p->max_pages < 1)
    return fail(MEDUSA_ERR_SHAPE, "pages: n_pages, page_size and max_pages must be >= 1");
  if (!aligned(p->K, align) || !aligned(p->V, align))
    return fail(MEDUSA_ERR_ALIGNMENT, "pages: pools misaligned");
  return MEDUSA_OK;
}

}  // namespace

extern "C" {

medusa_status_t medusa_rope_freqs(int rot, double theta, medusa_rope_scaling_t scaling,
                                  double factor, double low_turns, double high_turns,
                                  double original_max_position, uint64_t* turns, float* scale) {
  if (turns == nullptr || scale == nullptr)
    return fail(MEDUSA_ERR_INVALID_ARG, "rope_freqs: null pointer");
  if (rot < 2 || rot % 2 != 0 || rot > 512)
    return fail(MEDUSA_ERR_SHAPE, "rope_freqs: rot must be even and in [2, 512]");
  if (scaling < MEDUSA_ROPE_NONE || scaling > MEDUSA_ROPE_YARN)
    return fail(MEDUSA_ERR_INVALID_ARG, "rope_freqs: bad scaling");
  if (!(theta > 1.0) || isinf(theta))
    return fail(MEDUSA_ERR_INVALID_ARG, "rope_freqs: theta must be above 1");
  if (scaling != MEDUSA_ROPE_NONE && (!(factor >= 1.0) || isinf(factor)))
    return fail(MEDUSA_ERR_INVALID_ARG, "rope_freqs: factor must be at least 1");
  if ((scaling == MEDUSA_ROPE_LLAMA3 || scaling == MEDUSA_ROPE_YARN) &&
      (!(low_turns > 0.0) || !(high_turns > low_turns) || isinf(high_turns) ||
       !(original_max_position > 0.0) || isinf(original_max_position)))
    return fail(MEDUSA_ERR_INVALID_ARG,
                "rope_freqs: need 0 < low_turns < high_turns and original_max_position > 0");
  return medusa::rope_freqs(rot, theta, scaling, factor, low_turns, high_turns,
                            original_max_position, turns, scale);
}

medusa_status_t medusa_rope(const medusa_rope_t* rope, const void* q, long long q_stride,
                            const void* k, long long k_stride, medusa_dtype_t dt,
                            const int32_t* positions, int T, int Hq, int Hkv, int dh, int inverse,
                            void* q_out, long long q_out_stride, void* k_out,
                            long long k_out_stride, void* stream) {
  if (rope == nullptr) return fail(MEDUSA_ERR_INVALID_ARG, "rope: null rotation");
  if (!valid_dtype(dt)) return fail(MEDUSA_ERR_INVALID_ARG, "rope: bad dtype");
  if (T < 0 || Hq < 1 || Hq > 65535 || (k != nullptr && (Hkv < 1 || Hkv > 65535)) || dh < 1 ||
      dh > 1024)
    return fail(MEDUSA_ERR_SHAPE, "rope: T, Hq, Hkv or dh out of range");
  medusa_status_t st = check_rotation(rope, dh);
  if (st != MEDUSA_OK) return st;
  if (T == 0) return MEDUSA_OK;
  if (positions == nullptr || (k == nullptr) != (k_out == nullptr))
    return fail(MEDUSA_ERR_INVALID_ARG, "rope: null pointer");
  const size_t eb = dt == MEDUSA_BF16 ? 2 : 4;
  if ((st = check_operand(q, q_stride, T, Hq, dh, eb)) != MEDUSA_OK) return st;
  if ((st = check_operand(q_out, q_out_stride, T, Hq, dh, eb)) != MEDUSA_OK) return st;
  const Span sq{q, q_stride, Hq}, sqo{q_out, q_out_stride, Hq};
  if ((st = check_in_place(sq, sqo, T, dh, eb)) != MEDUSA_OK) return st;
  if (k != nullptr) {
    if ((st = check_operand(k, k_stride, T, Hkv, dh, eb)) != MEDUSA_OK) return st;
    if ((st = check_operand(k_out, k_out_stride, T, Hkv, dh, eb)) != MEDUSA_OK) return st;
    const Span sk{k, k_stride, Hkv}, sko{k_out, k_out_stride, Hkv};
    if ((st = check_in_place(sk, sko, T, dh, eb)) != MEDUSA_OK) return st;
    if (overlap(sqo, sk, T, dh, eb) || overlap(sko, sq, T, dh, eb) || overlap(sqo, sko, T, dh, eb))
      return fail(MEDUSA_ERR_INVALID_ARG, "rope: q's and k's operands overlap");
  }
  return medusa::rope(*rope, q, q_stride, k, k_stride, dt, positions, T, Hq, Hkv, dh,
                      inverse ? 1 : 0, q_out, q_out_stride, k_out, k_out_stride,
                      static_cast<cudaStream_t>(stream));
}

medusa_status_t medusa_rope_append(const medusa_rope_t* rope, const void* q, long long q_stride,
                                   const void* k, long long k_stride, const void* v,
                                   long long v_stride, medusa_dtype_t dt, const int32_t* positions,
                                   const int32_t* cu_q, const int32_t* kv_len, int B, int T, int Hq,
                                   int Hkv, int dh, void* q_out, long long q_out_stride,
                                   const medusa_pages_t* pages, int32_t* dev_status,
                                   void* stream) {
  if (!valid_dtype(dt)) return fail(MEDUSA_ERR_INVALID_ARG, "rope_append: bad dtype");
  const size_t eb = dt == MEDUSA_BF16 ? 2 : 4;
  medusa_status_t st = check_pages(pages, eb);
  if (st != MEDUSA_OK) return st;
  if (B < 1 || T < 0 || (q != nullptr && (Hq < 1 || Hq > 65535)) || Hkv < 1 || Hkv > 65535 ||
      dh < 1 || dh > 1024)
    return fail(MEDUSA_ERR_SHAPE, "rope_append: B, T, Hq, Hkv or dh out of range");
  if (rope == nullptr) {
    if (q != nullptr || q_out != nullptr)
      return fail(MEDUSA_ERR_INVALID_ARG, "rope_append: q without a rotation");
  } else if ((st = check_rotation(rope, dh)) != MEDUSA_OK) {
    return st;
  }
  if (T == 0) return MEDUSA_OK;
  if (cu_q == nullptr || kv_len == nullptr || (q == nullptr) != (q_out == nullptr))
    return fail(MEDUSA_ERR_INVALID_ARG, "rope_append: null pointer");
  if ((st = check_operand(k, k_stride, T, Hkv, dh, eb)) != MEDUSA_OK) return st;
  if ((st = check_operand(v, v_stride, T, Hkv, dh, eb)) != MEDUSA_OK) return st;
  if (q != nullptr) {
    if ((st = check_operand(q, q_stride, T, Hq, dh, eb)) != MEDUSA_OK) return st;
    if ((st = check_operand(q_out, q_out_stride, T, Hq, dh, eb)) != MEDUSA_OK) return st;
    const Span sqo{q_out, q_out_stride, Hq};
    if ((st = check_in_place({q, q_stride, Hq}, sqo, T, dh, eb)) != MEDUSA_OK) return st;
    if (overlap(sqo, {k, k_stride, Hkv}, T, dh, eb) || overlap(sqo, {v, v_stride, Hkv}, T, dh, eb))
      return fail(MEDUSA_ERR_INVALID_ARG, "rope_append: q_out overlaps k or v");
  }
  return medusa::rope_append(rope, q, q_stride, k, k_stride, v, v_stride, dt, positions, cu_q,
                             kv_len, B, T, Hq, Hkv, dh, q_out, q_out_stride, *pages, dev_status,
                             static_cast<cudaStream_t>(stream));
}

size_t medusa_chunk_attention_workspace_size(int Hq, int Hkv, int dh, medusa_dtype_t dt) {
  if (Hq < 1 || Hkv < 1 || dh < 1 || !valid_dtype(dt)) return 0;
  return medusa::chunk_attention_workspace_size(Hq, Hkv, dh, dt);
}

medusa_status_t medusa_chunk_attention(const void* q, long long q_stride,
                                       const medusa_pages_t* pages, medusa_dtype_t dt,
                                       const int32_t* cu_q, const int32_t* kv_len, int B, int T,
                                       int Hq, int Hkv, int dh, float scale, void* out, void* ws,
                                       size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (!valid_dtype(dt)) return fail(MEDUSA_ERR_INVALID_ARG, "chunk_attention: bad dtype");
  medusa_status_t st = check_pages(pages, 16);
  if (st != MEDUSA_OK) return st;
  if (B < 1 || B > 1024 || T < 0 || Hq < 1 || Hkv < 1 || Hkv > 1024 || Hq % Hkv != 0 ||
      Hq / Hkv > 128)
    return fail(MEDUSA_ERR_SHAPE, "chunk_attention: B, T, Hq or Hkv out of range");
  if (dt == MEDUSA_BF16) {
    if (dh != 64 && dh != 128)
      return fail(MEDUSA_ERR_SHAPE, "chunk_attention: bf16 dh must be 64 or 128");
    if (T > 1 && q_stride % 8 != 0)
      return fail(MEDUSA_ERR_ALIGNMENT, "chunk_attention: q_stride must be a multiple of 8");
  } else if (dh < 32 || dh % 32 != 0 || dh > 256) {
    return fail(MEDUSA_ERR_SHAPE, "chunk_attention: f32 dh must be a multiple of 32, <= 256");
  }
  // (dh is above zero here)
  if ((long long)pages->n_pages * pages->page_size > (1LL << 40) / dh / Hkv)
    return fail(MEDUSA_ERR_SHAPE, "chunk_attention: cache too large");
  if (!(scale > 0.f) || isinf(scale))
    return fail(MEDUSA_ERR_INVALID_ARG, "chunk_attention: scale must be > 0");
  if (T == 0) return MEDUSA_OK;
  if (!q || !cu_q || !kv_len || !out)
    return fail(MEDUSA_ERR_INVALID_ARG, "chunk_attention: null pointer");
  if (T > 1 && q_stride < (long long)Hq * dh)
    return fail(MEDUSA_ERR_SHAPE, "chunk_attention: q_stride is below Hq * dh");
  const size_t eb = dt == MEDUSA_BF16 ? 2 : 4;
  const size_t al = dt == MEDUSA_BF16 ? 16 : eb;
  if (!aligned(q, al) || !aligned(out, al))
    return fail(MEDUSA_ERR_ALIGNMENT, "chunk_attention: q or out misaligned");
  if (overlap({q, q_stride, Hq}, {out, (long long)Hq * dh, Hq}, T, dh, eb))
    return fail(MEDUSA_ERR_INVALID_ARG, "chunk_attention: out overlaps q");
  const size_t need = medusa::chunk_attention_workspace_size(Hq, Hkv, dh, dt);
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned(ws, 256)))
    return fail(MEDUSA_ERR_WORKSPACE, "chunk_attention: workspace null, misaligned or too small");
  return medusa::chunk_attention(q, q_stride, *pages, dt, cu_q, kv_len, B, T, Hq, Hkv, dh, scale,
                                 out, ws, dev_status, static_cast<cudaStream_t>(stream));
}

medusa_status_t medusa_sample_tokens(const void* logits, medusa_dtype_t dt, long long row_stride,
                                     int n_rows, const int32_t* row_idx, int R, int V,
                                     const float* u, const float* temperature,
                                     const int32_t* top_k, const float* top_p, const float* min_p,
                                     int32_t* tokens, int32_t* kept, int32_t* dev_status,
                                     void* stream) {
  if (!valid_dtype(dt)) return fail(MEDUSA_ERR_INVALID_ARG, "sample_tokens: bad dtype");
  if (R < 0 || R > 65535 || n_rows < (R > 0 ? 1 : 0) || n_rows > 65535 || V < 1 ||
      V > medusa::sample_max_vocab(dt == MEDUSA_BF16 ? 2 : 4))
    return fail(MEDUSA_ERR_SHAPE, "sample_tokens: R, n_rows or V out of range");
  if (n_rows > 1 && row_stride < V)
    return fail(MEDUSA_ERR_SHAPE, "sample_tokens: row_stride is below V");
  if (row_idx == nullptr && R > n_rows)
    return fail(MEDUSA_ERR_SHAPE, "sample_tokens: more draws than rows need row_idx");
  if (R == 0) return MEDUSA_OK;
  if (!logits || !u || !tokens) return fail(MEDUSA_ERR_INVALID_ARG, "sample_tokens: null pointer");
  if (!aligned(logits, dt == MEDUSA_BF16 ? 2 : 4))
    return fail(MEDUSA_ERR_ALIGNMENT, "sample_tokens: logits not aligned to their type");
  return medusa::sample_tokens(logits, dt, row_stride, n_rows, row_idx, R, V, u, temperature,
                               top_k, top_p, min_p, tokens, kept, dev_status,
                               static_cast<cudaStream_t>(stream));
}

}  // extern "C"
