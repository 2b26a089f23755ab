// qsa_append_api.cu -- C ABI of the KV-cache append with position rotation
// (include/qsa.h): host-side validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "qsa.h"
#include "qsa_append.cuh"
#include "qsa_host.cuh"

namespace {

using namespace qsa::host;
using qsa::ap::AppendParams;

// Whether n0 x n1 rows of `row` elements at strides s0, s1 are disjoint.
bool disjoint(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t row) {
  if (n0 <= 1 && n1 <= 1) return true;
  if (n0 <= 1) return s1 >= row;
  if (n1 <= 1) return s0 >= row;
  // the larger stride must clear the whole run of the smaller one (the
  // product cannot overflow once the smaller stride is at least a row)
  auto clears = [row](int64_t n, int64_t inner, int64_t outer) {
    return inner >= row && outer >= row && (n - 1) <= (outer - row) / inner;
  };
  return clears(n1, s1, s0) || clears(n0, s0, s1);
}

bool misaligned(const int64_t* x, int n, int64_t m) {
  for (int i = 0; i < n; ++i)
    if (x[i] % m != 0) return true;
  return false;
}

// A tensor scale the quantising appends accept: its products and reciprocal
// stay normal FP32 numbers.
bool scale_ok(float s) { return s >= 7.8886091e-31f && s <= 1.2676506e+30f; }   // 2^-100 .. 2^100

qsa_status_t validate(const qsa_append_shape_t* s, int format, const AppendParams& p) {
  if (s == nullptr) return QSA_ERR_NULL;
  if (s->num_tokens < 0 || s->num_q_heads < 0 || s->num_kv_heads <= 0 || s->num_slots < 0 || s->num_positions < 0)
    return QSA_ERR_SHAPE;
  const int R = s->rotary_dim;
  if (s->head_dim != 256 || R < 0 || R > 256 || R % 16 != 0 || s->reserved != 0) return QSA_ERR_UNSUPPORTED;
  if (s->interleaved != 0 && s->interleaved != 1) return QSA_ERR_UNSUPPORTED;
  if (s->num_q_heads > 65535 || s->num_kv_heads > 65535 || s->num_slots > 0x80000000LL ||
      s->num_positions > 0x80000000LL)
    return QSA_ERR_UNSUPPORTED;
  const int64_t rows = s->num_q_heads + 2LL * s->num_kv_heads;
  if (s->num_tokens > 0x7fffffffLL / rows) return QSA_ERR_UNSUPPORTED;
  if (format != qsa::ap::kBf16 && (!scale_ok(p.ts[0]) || !scale_ok(p.ts[1]))) return QSA_ERR_UNSUPPORTED;
  if (s->num_tokens == 0) return QSA_OK;
  const bool q = s->num_q_heads > 0, cache = s->num_slots > 0, codes = format == qsa::ap::kE2m1;
  if (p.k == nullptr || p.v == nullptr || p.slots == nullptr) return QSA_ERR_NULL;
  if (q && (p.q == nullptr || p.q_out == nullptr)) return QSA_ERR_NULL;
  if (R > 0 && (p.table == nullptr || p.positions == nullptr)) return QSA_ERR_NULL;
  if (cache && (p.cache[0] == nullptr || p.cache[1] == nullptr)) return QSA_ERR_NULL;
  if (cache && codes && (p.bscale[0] == nullptr || p.bscale[1] == nullptr)) return QSA_ERR_NULL;
  const int64_t in[] = {s->q_stride_tok, s->q_stride_head, s->qo_stride_tok, s->qo_stride_head,
                        s->k_stride_tok, s->k_stride_head, s->v_stride_tok, s->v_stride_head};
  const int64_t kv[] = {s->kv_stride_slot, s->kv_stride_head}, bs[] = {s->bscale_stride_slot, s->bscale_stride_head};
  for (int i = q ? 0 : 4; i < 8; ++i)
    if (in[i] < 0) return QSA_ERR_SHAPE;
  if (kv[0] < 0 || kv[1] < 0 || (R > 0 && s->table_stride < R)) return QSA_ERR_SHAPE;
  if (codes && (bs[0] < 0 || bs[1] < 0)) return QSA_ERR_SHAPE;
  // rows that are written must not overlap one another
  const int64_t row = codes ? 128 : 256;
  if (q && !disjoint(s->num_tokens, in[2], s->num_q_heads, in[3], 256)) return QSA_ERR_SHAPE;
  if (cache && !disjoint(s->num_slots, kv[0], s->num_kv_heads, kv[1], row)) return QSA_ERR_SHAPE;
  if (cache && codes && !disjoint(s->num_slots, bs[0], s->num_kv_heads, bs[1], 16)) return QSA_ERR_SHAPE;
  if (misaligned(in + (q ? 0 : 4), q ? 8 : 4, 8)) return QSA_ERR_ALIGN;
  if (cache && misaligned(kv, 2, format == qsa::ap::kBf16 ? 8 : 16)) return QSA_ERR_ALIGN;
  if (cache && codes && misaligned(bs, 2, 16)) return QSA_ERR_ALIGN;
  if (q && (!aligned16(p.q) || !aligned16(p.q_out))) return QSA_ERR_ALIGN;
  if (!aligned16(p.k) || !aligned16(p.v)) return QSA_ERR_ALIGN;
  if (R > 0 && (!aligned16(p.table) || s->table_stride % 4 != 0)) return QSA_ERR_ALIGN;
  if (R > 0 && (reinterpret_cast<uintptr_t>(p.positions) & 3u)) return QSA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(p.slots) & 3u) return QSA_ERR_ALIGN;
  for (int i = 0; i < 2; ++i) {
    if (cache && (!aligned16(p.cache[i]) || (codes && !aligned16(p.bscale[i])))) return QSA_ERR_ALIGN;
    if (!aligned16(p.seen[i])) return QSA_ERR_ALIGN;
  }
  // q_out is q itself, row for row, or another buffer
  if (q && p.q == p.q_out && (in[0] != in[2] || in[1] != in[3])) return QSA_ERR_SHAPE;
  return QSA_OK;
}

template <int kFormat>
qsa_status_t run(const qsa_append_shape_t* s, AppendParams& p, void* stream) {
  const qsa_status_t rc = validate(s, kFormat, p);
  if (rc != QSA_OK) return rc;
  if (s->num_tokens == 0) return QSA_OK;
  p.T = s->num_tokens;
  p.S = s->num_slots;
  p.P = s->num_positions;
  p.q_st = s->q_stride_tok;
  p.q_sh = s->q_stride_head;
  p.qo_st = s->qo_stride_tok;
  p.qo_sh = s->qo_stride_head;
  p.k_st = s->k_stride_tok;
  p.k_sh = s->k_stride_head;
  p.v_st = s->v_stride_tok;
  p.v_sh = s->v_stride_head;
  p.table_st = s->table_stride;
  const int64_t elem = kFormat == qsa::ap::kBf16 ? 2 : 1;
  p.c_ss = s->kv_stride_slot * elem;
  p.c_sh = s->kv_stride_head * elem;
  p.b_ss = s->bscale_stride_slot;
  p.b_sh = s->bscale_stride_head;
  p.Hq = s->num_q_heads;
  p.Hkv = s->num_kv_heads;
  p.R = s->rotary_dim;
  p.interleaved = s->interleaved;
  for (int i = 0; i < 2; ++i) {
    const volatile float six = 6.f * p.ts[i];           // FP32, rounded, on every host
    p.inv[i] = 1.f / six;
  }
  const int64_t warps = p.T * ((p.Hq + qsa::ap::kRowsQ - 1) / qsa::ap::kRowsQ +
                               (2LL * p.Hkv + qsa::ap::kRowsKv - 1) / qsa::ap::kRowsKv);
  const unsigned grid = static_cast<unsigned>((warps + qsa::ap::kWarps - 1) / qsa::ap::kWarps);
  qsa::ap::qsa_append_kernel<kFormat><<<grid, 32 * qsa::ap::kWarps, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

AppendParams pointers(const void* q, void* q_out, const void* k, const void* v, const float* cos_sin,
                      const int32_t* positions, const int32_t* slots, int32_t* status) {
  AppendParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.table = cos_sin;
  p.positions = positions;
  p.slots = slots;
  p.status = status;
  p.ts[0] = p.ts[1] = 1.f;
  return p;
}

}  // namespace

extern "C" {

qsa_status_t qsa_kv_append(const qsa_append_shape_t* shape, const void* q, void* q_out, const void* k, const void* v,
                           const float* cos_sin, const int32_t* positions, const int32_t* slots, void* k_cache,
                           void* v_cache, int32_t* status, void* stream) {
  AppendParams p = pointers(q, q_out, k, v, cos_sin, positions, slots, status);
  p.cache[0] = static_cast<char*>(k_cache);
  p.cache[1] = static_cast<char*>(v_cache);
  return run<qsa::ap::kBf16>(shape, p, stream);
}

qsa_status_t qsa_kv_append_fp8(const qsa_append_shape_t* shape, const void* q, void* q_out, const void* k,
                               const void* v, const float* cos_sin, const int32_t* positions, const int32_t* slots,
                               float k_scale, float v_scale, void* k_cache, void* v_cache, void* k_seen,
                               void* v_seen, int32_t* status, void* stream) {
  AppendParams p = pointers(q, q_out, k, v, cos_sin, positions, slots, status);
  p.cache[0] = static_cast<char*>(k_cache);
  p.cache[1] = static_cast<char*>(v_cache);
  p.seen[0] = static_cast<__nv_bfloat16*>(k_seen);
  p.seen[1] = static_cast<__nv_bfloat16*>(v_seen);
  p.ts[0] = k_scale;
  p.ts[1] = v_scale;
  return run<qsa::ap::kE4m3>(shape, p, stream);
}

qsa_status_t qsa_kv_append_fp4(const qsa_append_shape_t* shape, const void* q, void* q_out, const void* k,
                               const void* v, const float* cos_sin, const int32_t* positions, const int32_t* slots,
                               float k_scale, float v_scale, void* k_codes, void* k_bscale, void* v_codes,
                               void* v_bscale, void* k_seen, void* v_seen, int32_t* status, void* stream) {
  AppendParams p = pointers(q, q_out, k, v, cos_sin, positions, slots, status);
  p.cache[0] = static_cast<char*>(k_codes);
  p.cache[1] = static_cast<char*>(v_codes);
  p.bscale[0] = static_cast<char*>(k_bscale);
  p.bscale[1] = static_cast<char*>(v_bscale);
  p.seen[0] = static_cast<__nv_bfloat16*>(k_seen);
  p.seen[1] = static_cast<__nv_bfloat16*>(v_seen);
  p.ts[0] = k_scale;
  p.ts[1] = v_scale;
  return run<qsa::ap::kE2m1>(shape, p, stream);
}

}  // extern "C"
