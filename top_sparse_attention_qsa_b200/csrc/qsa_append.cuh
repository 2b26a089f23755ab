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
// A warp takes 8 query rows of one token, or 2 K and V rows; every access is 16
// bytes per lane, and a warp asks for all its rows before the first use.  Query
// rows are mostly dims that do not turn (192 of 256 at R = 64): those are copied
// a row at a time, and a lane turns 8 whole pairs of one row, so that the 8
// rows' rotary dims fill one pass over the lanes.  K and V rows lie 8 dims per
// lane, as the cache rows do; a lane's rotation partners come from the lane
// that holds them, a block scale's 16 dims belong to two adjacent lanes.
//
// Bound by HBM: 236 MB (T = 8192, heads (24,2), R = 64, BF16 cache) move in 38
// us, 6.2 TB/s, 0.95 of the measured copy rate; with a 4-bit cache 242 MB in 44
// us.  Four rows of any kind per warp, 8 dims per lane, took 49 and 61 us (565
// warp instructions per four rows, three quarters of the lanes rotating dims
// that do not turn), one row per warp 90 and 92.  Query rows per warp: 4 take
// 42 us, 6 38, 12 50; K and V rows: 1 take 41 us, 4 as long as 2, but the 4-bit
// cache's 50 against 44.  64 registers spill 8, 12 and 48 bytes a lane (BF16,
// E4M3, 4 bits).  The E4M3 cache (7810 tokens, (12,1), 118 MB) takes 21.9 us, 0.8
// of them the divisions: products with a reciprocal would round otherwise next
// to a border.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "qsa_ptx.cuh"

namespace qsa {
namespace ap {

constexpr int kWarps = 4, kRowsQ = 8, kRowsKv = 2;
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

// a c + b s in FP32 (one rounding of b s, one of the sum) or in FP64 (both
// products exact, one rounding).
__device__ __forceinline__ float rot(float a, float c, float b, float s) { return fmaf(a, c, __fmul_rn(b, s)); }
__device__ __forceinline__ double rot(double a, double c, double b, double s) {
  return __dadd_rn(__dmul_rn(a, c), __dmul_rn(b, s));
}

// The cosines and sines of the lane's pairs: in the interleaved form of its 4
// pairs, else of the pairs its 8 dims belong to (s negated where the lane
// holds the pairs' first halves, so that y = x c + partner * s throughout).
struct Angles {
  float c[8], s[8];
};

__device__ __forceinline__ void load_angles(const AppendParams& p, int64_t pos, int lane, Angles& a) {
  const float* cs = p.table + pos * p.table_st;
  const int half = p.R >> 1, d0 = 8 * lane;
  if (p.interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + (d0 >> 1)));
    const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + (d0 >> 1)));
    a.c[0] = a.c[1] = c.x, a.c[2] = a.c[3] = c.y, a.c[4] = a.c[5] = c.z, a.c[6] = a.c[7] = c.w;
    a.s[0] = -(a.s[1] = s.x), a.s[2] = -(a.s[3] = s.y), a.s[4] = -(a.s[5] = s.z), a.s[6] = -(a.s[7] = s.w);
    return;
  }
  const bool lo = d0 < half;
  const int i0 = lo ? d0 : d0 - half;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + i0 + 4 * q));
    const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + i0 + 4 * q));
    a.c[4 * q] = c.x, a.c[4 * q + 1] = c.y, a.c[4 * q + 2] = c.z, a.c[4 * q + 3] = c.w;
    a.s[4 * q] = lo ? -s.x : s.x, a.s[4 * q + 1] = lo ? -s.y : s.y;
    a.s[4 * q + 2] = lo ? -s.z : s.z, a.s[4 * q + 3] = lo ? -s.w : s.w;
  }
}

// The lane's 8 dims of a row after rotation (all 32 lanes call; lanes past the
// rotary dims return them as they are).
template <typename F>
__device__ __forceinline__ void rotate8(const AppendParams& p, const uint4& own, const Angles& a, int lane, F (&y)[8]) {
  float x[8], o[8];
  unpack8(own, x);
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = x[i ^ 1];
  } else {
    const int step = p.R >> 4;                          // lanes between the halves
    const int from = 8 * lane < (p.R >> 1) ? lane + step : lane - step;
    uint4 w;
    w.x = __shfl_sync(0xffffffffu, own.x, from & 31);
    w.y = __shfl_sync(0xffffffffu, own.y, from & 31);
    w.z = __shfl_sync(0xffffffffu, own.z, from & 31);
    w.w = __shfl_sync(0xffffffffu, own.w, from & 31);
    unpack8(w, o);
  }
  if (8 * lane < p.R) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = rot(F(x[i]), F(a.c[i]), F(o[i]), F(a.s[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
  }
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  float lo, hi;
  f16x2_to_f32(e4m3x2_to_f16x2(byte), lo, hi);
  return lo;
}

// Two FP32 values -> two E2M1 codes (lo in bits 0-3), nearest, saturating at 6.
__device__ __forceinline__ uint32_t pack_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b, z;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tmov.b32 %0, {b, 0, 0, 0};\n\t}\n"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// 8 codes (element i in bits 4i .. 4i+3) and the block scale byte of the 16
// dims of this lane and its neighbour.  The quotient y / (e ts) in FP32 is
// within 2^-22 of its value (four roundings): where codes of the quotient
// moved by 2^-20 either way agree, they are the code; else the element lies
// next to a border and the exact products decide.
// f: the 8 values rounded to FP32; exact(i): |value i| in FP64.
template <typename Exact>
__device__ __forceinline__ uint32_t quantise4(const float (&f)[8], Exact exact, float ts, float inv,
                                              uint32_t* scale_byte) {
  float m = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m = fmaxf(m, fabsf(f[i]));                          // (rounding keeps the order: the largest |y| rounded)
    nan |= f[i] != f[i];
  }
  float amax = nan ? __int_as_float(0x7fffffff) : m;
  const float other = __shfl_xor_sync(0xffffffffu, amax, 1);
  amax = (amax != amax || other != other) ? __int_as_float(0x7fffffff) : fmaxf(amax, other);
  const uint32_t e = pack_e4m3x2(__fmul_rn(amax, inv), 0.f) & 0xffu;   // saturates at 448; NaN stays NaN
  *scale_byte = e;
  const float ev = e4m3_value(e);
  uint32_t neg = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) neg |= (__float_as_uint(f[i]) >> 31) << (4 * i + 3);
  if (!(ev > 0.f)) return neg;                          // zero or NaN scale: code 0
  const float r = __frcp_rn(ev * ts);
  uint32_t lo = 0u, hi = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float u0 = f[2 * i] * r, u1 = f[2 * i + 1] * r;
    constexpr float kDown = 1.f - 9.5367431640625e-7f, kUp = 1.f + 9.5367431640625e-7f;   // 2^-20
    lo |= pack_e2m1x2(u0 * kDown, u1 * kDown) << (8 * i);
    hi |= pack_e2m1x2(u0 * kUp, u1 * kUp) << (8 * i);
  }
  if (lo != hi) {
    const double b = static_cast<double>(ev) * static_cast<double>(ts);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (((lo ^ hi) >> (4 * i)) & 0xfu) {
        const double u = exact(i);
        const uint32_t c = (u > 0.25 * b) + (u >= 0.75 * b) + (u > 1.25 * b) + (u >= 1.75 * b) + (u > 2.5 * b) +
                           (u >= 3.5 * b) + (u > 5.0 * b);
        lo = (lo & ~(0xfu << (4 * i))) | (c << (4 * i));
      }
    }
  }
  return (lo & 0x77777777u) | neg;
}

// The values of 8 codes times the block scale (exact in FP32), times ts.
__device__ __forceinline__ uint4 values4(uint32_t codes, uint32_t scale_byte, float ts) {
  const float ev = e4m3_value(scale_byte);
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f16x2_to_f32(h[i], v[2 * i], v[2 * i + 1]);
    v[2 * i] = __fmul_rn(v[2 * i] * ev, ts);
    v[2 * i + 1] = __fmul_rn(v[2 * i + 1] * ev, ts);
  }
  return pack8(v);
}

// Query rows h0 .. h0 + n - 1 (n <= kRowsQ) of token t.  The dims past R are copied a
// row at a time (not at all in place); of the rotary dims a lane takes 8 pairs
// of one row, with both members, so that nothing is exchanged and lanes whose
// dims do not turn do not go along with those whose do.
__device__ __forceinline__ void append_q(const AppendParams& p, int64_t t, int h0, int n, int32_t pos, bool bad,
                                         int lane) {
  const int half = p.R >> 1;
  // plain loads: q_out may be q itself; a lane stores only what it has read
  const __nv_bfloat16* src = p.q + t * p.q_st + h0 * p.q_sh;
  __nv_bfloat16* dst = p.q_out + t * p.qo_st + h0 * p.qo_sh;
  const bool pass = 8 * lane >= p.R && p.q_out != p.q;
  uint4 own[kRowsQ];
  if (pass) {
#pragma unroll
    for (int i = 0; i < kRowsQ; ++i)
      if (i < n) own[i] = *reinterpret_cast<const uint4*>(src + i * p.q_sh + 8 * lane);
  }
  const uint32_t per_row = p.R >> 4, units = n * per_row;
  struct Unit {
    uint4 a, b;
    int row, at;
  };
  auto ask = [&](uint32_t u) {
    Unit r;
    r.row = u / per_row;
    r.at = 8 * (u - r.row * per_row);
    const __nv_bfloat16* x = src + r.row * p.q_sh + r.at;
    r.a = *reinterpret_cast<const uint4*>(x);
    r.b = *reinterpret_cast<const uint4*>(x + half);
    return r;
  };
  uint32_t u = lane;
  Unit next;
  if (u < units) next = ask(u);
  if (bad) return;
  if (pass) {
#pragma unroll
    for (int i = 0; i < kRowsQ; ++i)
      if (i < n) *reinterpret_cast<uint4*>(dst + i * p.qo_sh + 8 * lane) = own[i];
  }
  const float* cs = p.table + pos * p.table_st;
  for (; u < units; u += 32) {
    const Unit un = next;
    const float* c = cs + (p.interleaved ? un.at >> 1 : un.at);
    const int far = p.interleaved ? half >> 1 : 4;      // the second four angles
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(c)), c1 = __ldg(reinterpret_cast<const float4*>(c + far));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(c + half)),
                 s1 = __ldg(reinterpret_cast<const float4*>(c + half + far));
    if (u + 32 < units) next = ask(u + 32);
    const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    float x[8], z[8], y[8], w[8];
    unpack8(un.a, x);
    unpack8(un.b, z);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p.interleaved) {
        y[2 * i] = rot(x[2 * i], cc[i], x[2 * i + 1], -ss[i]);
        y[2 * i + 1] = rot(x[2 * i + 1], cc[i], x[2 * i], ss[i]);
        w[2 * i] = rot(z[2 * i], cc[4 + i], z[2 * i + 1], -ss[4 + i]);
        w[2 * i + 1] = rot(z[2 * i + 1], cc[4 + i], z[2 * i], ss[4 + i]);
      } else {
#pragma unroll
        for (int k = 2 * i; k < 2 * i + 2; ++k) {
          y[k] = rot(x[k], cc[k], z[k], -ss[k]);
          w[k] = rot(z[k], cc[k], x[k], ss[k]);
        }
      }
    }
    __nv_bfloat16* o = dst + un.row * p.qo_sh + un.at;
    *reinterpret_cast<uint4*>(o) = pack8(y);
    *reinterpret_cast<uint4*>(o + half) = pack8(w);
  }
}

template <int kFormat>
__global__ void __launch_bounds__(32 * kWarps, 8) qsa_append_kernel(const __grid_constant__ AppendParams p) {
  const uint32_t q_warps = (p.Hq + kRowsQ - 1) / kRowsQ;
  const int rows = 2 * p.Hkv, kv_warps = (rows + kRowsKv - 1) / kRowsKv;
  const uint32_t per_tok = q_warps + kv_warps;
  const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t tok = w / per_tok, place = w - tok * per_tok;
  const int64_t t = tok;
  if (t >= p.T) return;
  const int32_t pos = p.R > 0 ? __ldg(p.positions + t) : 0;
  const bool bad = p.R > 0 && (pos < 0 || pos >= p.P);
  if (place < q_warps) {
    const int share = (p.Hq + q_warps - 1) / q_warps;   // the heads evenly: 12 as 6 and 6
    const int h0 = place * share;
    return append_q(p, t, h0, min(share, p.Hq - h0), pos, bad, lane);
  }
  const int r0 = static_cast<int>(place - q_warps);     // K and V rows r0, r0 + kv_warps, ...
  const int32_t slot = __ldg(p.slots + t);
  uint4 own[kRowsKv];
#pragma unroll
  for (int i = 0; i < kRowsKv; ++i) {
    const int r = r0 + i * kv_warps;
    const __nv_bfloat16* src = r < p.Hkv ? p.k + t * p.k_st + r * p.k_sh : p.v + t * p.v_st + (r - p.Hkv) * p.v_sh;
    if (r < rows) own[i] = __ldg(reinterpret_cast<const uint4*>(src + 8 * lane));
  }
  if (bad) {
    if (r0 == 0 && lane == 0 && p.status != nullptr) atomicOr(p.status, static_cast<int32_t>(kStatusBadPosition));
    return;
  }
  Angles an;
  if (8 * lane < p.R) load_angles(p, pos, lane, an);
  const bool put = slot >= 0 && slot < p.S;
  if (slot >= p.S && r0 == 0 && lane == 0 && p.status != nullptr)
    atomicOr(p.status, static_cast<int32_t>(kStatusOobSlot));
#pragma unroll
  for (int i = 0; i < kRowsKv; ++i) {
    const int r = r0 + i * kv_warps;
    if (r >= rows) break;
    const int kv = r >= p.Hkv ? 1 : 0;                    // K rows, then V rows
    const int g = r - kv * p.Hkv;
    char* row = p.cache[kv] + static_cast<int64_t>(put ? slot : 0) * p.c_ss + g * p.c_sh;
    __nv_bfloat16* seen = p.seen[kv] == nullptr ? nullptr : p.seen[kv] + (t * p.Hkv + g) * 256 + 8 * lane;
    if constexpr (kFormat == kE2m1) {
      uint32_t e, codes;
      float f[8];
      if (kv) {
        unpack8(own[i], f);
        codes = quantise4(f, [&](int k) { return static_cast<double>(fabsf(f[k])); }, p.ts[1], p.inv[1], &e);
      } else {
        double y[8];
        rotate8(p, own[i], an, lane, y);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __double2float_rn(y[k]);
        codes = quantise4(f, [&](int k) { return fabs(y[k]); }, p.ts[0], p.inv[0], &e);
      }
      if (put) {
        *reinterpret_cast<uint32_t*>(row + 4 * lane) = codes;
        if ((lane & 1) == 0)
          p.bscale[kv][static_cast<int64_t>(slot) * p.b_ss + g * p.b_sh + (lane >> 1)] = static_cast<char>(e);
      }
      if (seen != nullptr) *reinterpret_cast<uint4*>(seen) = values4(codes, e, p.ts[kv]);
    } else {
      float y[8];
      if (kv)
        unpack8(own[i], y);
      else
        rotate8(p, own[i], an, lane, y);
      if constexpr (kFormat == kBf16) {
        if (put) *reinterpret_cast<uint4*>(row + 16 * lane) = !kv && 8 * lane < p.R ? pack8(y) : own[i];
      } else {
        uint32_t b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          b[k] = pack_e4m3x2(__fdiv_rn(y[2 * k], p.ts[kv]), __fdiv_rn(y[2 * k + 1], p.ts[kv]));
        if (put) *reinterpret_cast<uint2*>(row + 8 * lane) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
        if (seen != nullptr) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f16x2_to_f32(e4m3x2_to_f16x2(b[k]), y[2 * k], y[2 * k + 1]);
            y[2 * k] = __fmul_rn(y[2 * k], p.ts[kv]);
            y[2 * k + 1] = __fmul_rn(y[2 * k + 1], p.ts[kv]);
          }
          *reinterpret_cast<uint4*>(seen) = pack8(y);
        }
      }
    }
  }
}

}  // namespace ap
}  // namespace qsa
