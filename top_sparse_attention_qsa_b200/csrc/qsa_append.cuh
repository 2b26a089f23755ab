// qsa_append.cuh -- appending new keys and values to the KV cache, with the
// position rotation of Q and K applied on the way (sm_100a).
//
// For every token t at position p = positions[t], with R rotary dims and the
// table row cos_sin[p] = [c_0 .. c_{R/2-1}, s_0 .. s_{R/2-1}], each pair
// (a, b) of rotary dims of every Q and K head becomes
//   y_a = x_a c_i - x_b s_i,   y_b = x_b c_i + x_a s_i
// (pair i: dims (i, i + R/2), or (2i, 2i + 1) in the interleaved form); the
// other dims and V pass through.  K and V rows go to cache row slots[t]:
//   BF16   bf16(y)
//   E4M3   e4m3(y / ts), saturating at 448 (ts: the tensor's FP32 scale)
//   4 bits per 16 dims a block scale e = e4m3(fl32(max |y|) * inv), with inv =
//          fl32(1 / fl32(6 ts)), and codes = the E2M1 value nearest to
//          y / (e ts), ties to the even code, saturating at 6
// The 4-bit code of an element is decided exactly: the products x c and x s of
// a BF16 and an FP32 value have 32 significant bits and are exact in FP64, so
// is the product of an E2M1 midpoint (3 bits), e (4 bits) and ts (24 bits),
// and |y| is compared with those products; a rounded quotient would pick the
// wrong neighbour next to a border.  The other formats rotate in FP32 and
// round once to the cache's type.
//
// One warp per row (one head of Q, K or V of one token), 8 dims per lane, so
// that every global access is 16 bytes per lane and a row is one request; a
// lane's rotation partners are the 16 bytes R/2 dims away, read again from
// the row (an L1 hit).  A block scale's 16 dims belong to two adjacent lanes.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "qsa_ptx.cuh"

namespace qsa {
namespace ap {

constexpr int kWarps = 8;
constexpr uint32_t kStatusOobSlot = 1u, kStatusBadPosition = 4u;

enum Format { kBf16 = 0, kE4m3 = 1, kE2m1 = 2 };

struct AppendParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const float* table;            // cos_sin
  const int32_t* positions;
  const int32_t* slots;
  char* cache[2];                // K, V rows (4-bit: the codes)
  char* bscale[2];               // 4-bit: the block scales
  __nv_bfloat16* seen[2];        // the values as cached, [T][Hkv][256], or nullptr
  int32_t* status;
  int64_t T, S, P;
  int64_t q_st, q_sh, qo_st, qo_sh, k_st, k_sh, v_st, v_sh, table_st;
  int64_t c_ss, c_sh, b_ss, b_sh;   // bytes
  float ts[2], inv[2];
  int32_t Hq, Hkv, R, interleaved;
};

// Four words of BF16 pairs as 8 values, and back (round to nearest even).
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// y_a = a c - b s in FP32 (one rounding of b s, one of the difference) or in
// FP64 (both products exact, one rounding).
__device__ __forceinline__ float rot(float a, float c, float b, float s) { return fmaf(a, c, -__fmul_rn(b, s)); }
__device__ __forceinline__ double rot(double a, double c, double b, double s) {
  return __dsub_rn(__dmul_rn(a, c), __dmul_rn(b, s));
}

// The lane's 8 dims of a row after rotation; `row` are the row's 256 BF16.
template <typename F>
__device__ __forceinline__ void rotate8(const AppendParams& p, const __nv_bfloat16* row, const uint4& own,
                                        const float* cs, int lane, F (&y)[8]) {
  float x[8];
  unpack8(own, x);
  const int d0 = 8 * lane;
  if (d0 >= p.R) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    return;
  }
  const int half = p.R >> 1;
  if (p.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(cs + (d0 >> 1));
    const float4 s = *reinterpret_cast<const float4*>(cs + half + (d0 >> 1));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F a = x[2 * i], b = x[2 * i + 1];
      y[2 * i] = rot(a, F(cc[i]), b, F(ss[i]));
      y[2 * i + 1] = rot(b, F(cc[i]), a, F(-ss[i]));
    }
  } else {
    const bool lo = d0 < half;
    float o[8];
    unpack8(*reinterpret_cast<const uint4*>(row + (lo ? d0 + half : d0 - half)), o);
    const int i0 = lo ? d0 : d0 - half;
    const float4 c0 = *reinterpret_cast<const float4*>(cs + i0), c1 = *reinterpret_cast<const float4*>(cs + i0 + 4);
    const float4 s0 = *reinterpret_cast<const float4*>(cs + half + i0),
                 s1 = *reinterpret_cast<const float4*>(cs + half + i0 + 4);
    const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = rot(F(x[i]), F(cc[i]), F(o[i]), F(lo ? ss[i] : -ss[i]));
  }
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  float lo, hi;
  f16x2_to_f32(e4m3x2_to_f16x2(byte), lo, hi);
  return lo;
}

// 8 codes (element i in bits 4i .. 4i+3) and the block scale byte of the 16
// dims of this lane and its neighbour; `val` gets code * scale (exact in FP32).
__device__ __forceinline__ uint32_t quantise4(const double (&y)[8], float ts, float inv, uint32_t* scale_byte,
                                              float (&val)[8]) {
  double m = 0.0;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m = fmax(m, fabs(y[i]));
    nan |= y[i] != y[i];
  }
  float amax = nan ? __int_as_float(0x7fffffff) : __double2float_rn(m);
  const float other = __shfl_xor_sync(0xffffffffu, amax, 1);
  amax = (amax != amax || other != other) ? __int_as_float(0x7fffffff) : fmaxf(amax, other);
  const uint32_t e = pack_e4m3x2(__fmul_rn(amax, inv), 0.f) & 0xffu;   // saturates at 448; NaN stays NaN
  const float ev = e4m3_value(e);
  const double b = static_cast<double>(ev) * static_cast<double>(ts);
  const bool live = b > 0.0;
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double u = fabs(y[i]);
    int c = 0;
    if (live)
      c = (u > 0.25 * b) + (u >= 0.75 * b) + (u > 1.25 * b) + (u >= 1.75 * b) + (u > 2.5 * b) + (u >= 3.5 * b) +
          (u > 5.0 * b);
    const bool neg = signbit(y[i]);
    // magnitudes 0 .5 1 1.5 2 3 4 6
    const float g = c < 4 ? 0.5f * c : (c < 6 ? c - 2.f : 2.f * c - 8.f);
    val[i] = (neg ? -g : g) * ev;
    w |= static_cast<uint32_t>(c | (neg ? 8 : 0)) << (4 * i);
  }
  *scale_byte = e;
  return w;
}

template <int kFormat>
__global__ void __launch_bounds__(32 * kWarps) qsa_append_kernel(const __grid_constant__ AppendParams p) {
  const int rows = p.Hq + 2 * p.Hkv;
  const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = w / static_cast<uint32_t>(rows);
  const int r = static_cast<int>(w - static_cast<uint32_t>(t) * rows);
  if (t >= p.T) return;
  const float* cs = nullptr;
  if (p.R > 0) {
    const int32_t pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.P) {
      if (r == 0 && lane == 0 && p.status != nullptr) atomicOr(p.status, static_cast<int32_t>(kStatusBadPosition));
      return;
    }
    cs = p.table + pos * p.table_st;
  }
  if (r < p.Hq) {
    const __nv_bfloat16* src = p.q + t * p.q_st + r * p.q_sh;
    __nv_bfloat16* dst = p.q_out + t * p.qo_st + r * p.qo_sh;
    // plain loads: q_out may be q itself, and no lane stores before all have read
    const uint4 own = *reinterpret_cast<const uint4*>(src + 8 * lane);
    float y[8];
    rotate8(p, src, own, cs, lane, y);
    __syncwarp();
    if (8 * lane < p.R || dst != src)
      *reinterpret_cast<uint4*>(dst + 8 * lane) = 8 * lane < p.R ? pack8(y) : own;
    return;
  }
  const int kv = r - p.Hq >= p.Hkv ? 1 : 0;               // K rows, then V rows
  const int g = r - p.Hq - kv * p.Hkv;
  const __nv_bfloat16* src = kv ? p.v + t * p.v_st + g * p.v_sh : p.k + t * p.k_st + g * p.k_sh;
  const uint4 own = *reinterpret_cast<const uint4*>(src + 8 * lane);
  const int32_t slot = __ldg(p.slots + t);
  const bool put = slot >= 0 && slot < p.S;
  if (slot >= p.S && r == p.Hq && lane == 0 && p.status != nullptr)
    atomicOr(p.status, static_cast<int32_t>(kStatusOobSlot));
  char* row = p.cache[kv] + static_cast<int64_t>(put ? slot : 0) * p.c_ss + g * p.c_sh;
  __nv_bfloat16* seen = p.seen[kv] == nullptr ? nullptr : p.seen[kv] + (t * p.Hkv + g) * 256 + 8 * lane;
  if (kFormat == kE2m1) {
    double y[8];
    if (kv) {
      float x[8];
      unpack8(own, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i];
    } else {
      rotate8(p, src, own, cs, lane, y);
    }
    uint32_t e;
    float val[8];
    const uint32_t codes = quantise4(y, p.ts[kv], p.inv[kv], &e, val);
    if (put) {
      *reinterpret_cast<uint32_t*>(row + 4 * lane) = codes;
      if ((lane & 1) == 0)
        p.bscale[kv][static_cast<int64_t>(slot) * p.b_ss + g * p.b_sh + (lane >> 1)] = static_cast<char>(e);
    }
    if (seen != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) val[i] = __fmul_rn(val[i], p.ts[kv]);
      *reinterpret_cast<uint4*>(seen) = pack8(val);
    }
    return;
  }
  float y[8];
  if (kv)
    unpack8(own, y);
  else
    rotate8(p, src, own, cs, lane, y);
  if (kFormat == kBf16) {
    if (put) *reinterpret_cast<uint4*>(row + 16 * lane) = !kv && 8 * lane < p.R ? pack8(y) : own;
    return;
  }
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    b[i] = pack_e4m3x2(__fdiv_rn(y[2 * i], p.ts[kv]), __fdiv_rn(y[2 * i + 1], p.ts[kv]));
  if (put) *reinterpret_cast<uint2*>(row + 8 * lane) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
  if (seen != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f16x2_to_f32(e4m3x2_to_f16x2(b[i]), y[2 * i], y[2 * i + 1]);
      y[2 * i] = __fmul_rn(y[2 * i], p.ts[kv]);
      y[2 * i + 1] = __fmul_rn(y[2 * i + 1], p.ts[kv]);
    }
    *reinterpret_cast<uint4*>(seen) = pack8(y);
  }
}

}  // namespace ap
}  // namespace qsa
