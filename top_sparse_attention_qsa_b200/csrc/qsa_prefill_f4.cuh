// qsa_prefill_f4.cuh -- QSA top-K sparse attention over a 4-bit KV cache:
// cp.async gather + in-SM dequantisation + tcgen05 kind::f16 kernel (sm_100a).
//
// The operation is the one of qsa_prefill_tc.cuh over cache rows of E2M1
// codes with one E4M3 scale per 16 dims and an FP32 scale per tensor:
// element = code * block scale * tensor scale.
//
// An E2M1 value (2 significant bits) times an E4M3 value (4) has at most 6
// significant bits and lies between 2^-10 and 2688, so code * block scale is
// exact in FP16 (11 bits, normal from 2^-14): the gathered codes become FP16
// MMA operands with no rounding.  The tensor scales go into the softmax scale
// and the output.  The query is scaled per head by a power of two that puts
// its largest |q| in [2^14, 2^15) and is then exact in FP16 for every element
// within 2^31 of that (smaller ones are off by at most 2^-25 after scaling,
// 2^-39 of the largest).  Probabilities are rounded to FP16 (11 significant
// bits, three more than BF16 keeps) after scaling by 2^7, which with the lazy
// rescale's p <= 2^8 stays below FP16's largest number and puts the smallest
// step at 2^-31: the sum of all that underflows is below 2^-32 of l per key.
//
// Warps (persistent CTAs, one per SM), in warpgroups:
//   0-3    producers: list entries one tile ahead, 16-byte cp.async of the
//          128-byte code rows (128-byte swizzled) and the 16-byte scale rows
//          into two rings, one of K tiles and one of V tiles
//   4-6    4: the unit's Q as an FP16 tile, one unit ahead; 5: one thread
//          issues the score MMAs; 6: one thread issues the PV MMAs; 7 idles
//   8-11   K dequantisation: thread = key = TMEM lane; 128 dims at a time into
//          TMEM, where the score MMA reads K as its A operand
//   12-15  V dequantisation into the MN-major 128-byte-swizzled FP16 tile the
//          PV MMA reads, one 128-dim half at a time
//   16-23  softmax, two warps per TMEM lane quadrant (8 heads each)
//   24-27  epilogue: O from TMEM (two buffers by unit parity), normalised
// Every wait is bounded (2 s of %globaltimer) as in the other kernels.
#pragma once

#include <cuda_fp16.h>

#include "qsa_prefill_f8.cuh"

namespace qsa {
namespace f4 {

using namespace tc;
using f8::xreduce8;

struct F4Params {
  TcParams t;                     // its kraw / vraw / kv strides / tm_q are unused
  const char* codes[2];           // K, V
  const char* bscale[2];
  int64_t c_ss, c_sh, b_ss, b_sh; // byte strides of the codes and of the scales
};

constexpr int kStages = 2;                          // packed tiles in each ring
constexpr int kCodeBytes = kKeys * 128;             // one packed tile: codes,
constexpr int kStageBytes = kCodeBytes + kKeys * 16;  // then block scales
constexpr int kHalfBytes = 32768;                   // FP16 V half: 128 keys x 128 dims
constexpr int kVHalves = 4;
constexpr int kTkStages = 6;                        // TMEM K stages of 128 dims (64 columns)
constexpr int kMasks = 8;                           // tiles whose key masks are kept
constexpr float kPShift = 7.f;                      // P is stored times 2^7

constexpr int kTmemCols4 = 512;
constexpr int kUS = 0, kUO = 32, kUK = 96;         // S: 2 x 16; O: 2 units x 2 halves x 16; K stages of 64
constexpr int H_K = 0;
constexpr int H_V = H_K + kStages * kStageBytes;
constexpr int H_VH = H_V + kStages * kStageBytes;
constexpr int H_Q = H_VH + kVHalves * kHalfBytes;
constexpr int H_P = H_Q + 2 * kQBytes;
constexpr int H_QSC = H_P + 2 * kPBytes;            // 2 buffers x 16 per-head score factors
constexpr int H_RED = H_QSC + 2 * kGp * 4;          // max[4][16], votes[2][8], sum[2][4][16]
constexpr int H_LM = H_RED + 1024;                  // per unit parity: l[16], m[16]
constexpr int H_MASK = H_LM + 256;                  // kMasks x 4 words: bit = key of the quadrant counts
constexpr int H_BAR = H_MASK + kMasks * 16;
static_assert(kUK + 64 * kTkStages <= kTmemCols4, "TMEM columns");
static_assert(H_VH % 1024 == 0 && H_Q % 1024 == 0 && kStageBytes % 1024 == 0, "swizzle atoms");
constexpr int J_KF = 0, J_KE = J_KF + kStages, J_VF = J_KE + kStages, J_VE = J_VF + kStages, J_TKF = J_VE + kStages,
              J_TKE = J_TKF + kTkStages, J_VHF = J_TKE + kTkStages, J_VHE = J_VHF + kVHalves, J_SF = J_VHE + kVHalves,
              J_SE = J_SF + 2, J_PF = J_SE + 2, J_PE = J_PF + 2, J_QF = J_PE + 2, J_QE = J_QF + 2, J_RMAX = J_QE + 2,
              J_RSUM = J_RMAX + 2, J_RMX2 = J_RSUM + 2, J_OF = J_RMX2 + 1, J_OE = J_OF + 2, J_LF = J_OE + 2,
              J_LE = J_LF + 2, J_DONE = J_LE + 2, J_NUM = J_DONE + 2;
constexpr int H_MISC = H_BAR + J_NUM * 8;           // tmem base, abort flag
constexpr int H_SMEM = H_MISC + 16 + 1024;
static_assert(H_SMEM <= 232448, "shared memory");


// kind::f16 with FP16 A and B (formats 0), FP32 accumulator, M = 128, N = 16.
constexpr uint32_t kIdescQK4 = (1u << 4) | (2u << 17) | (8u << 24);
constexpr uint32_t kIdescPV4 = kIdescQK4 | (1u << 15) | (1u << 16);

constexpr int kWarpMisc4 = 4, kWarpKd4 = 8, kWarpVd4 = 12, kWarpSm4 = 16, kSmWarps4 = 8, kWarpEpi4 = 24;
constexpr int kThreads4 = 28 * 32;
constexpr int kHpw4 = 8;                            // heads per softmax warp
// Registers per thread after setmaxnreg; their sum over the warpgroups stays
// within the launch's 7 x 72.
constexpr int kRegsProd4 = 56, kRegsMisc4 = 48, kRegsKd4 = 80, kRegsVd4 = 64, kRegsSm4 = 96, kRegsEpi4 = 64,
              kRegsLaunch4 = 72;
static_assert(kRegsProd4 + kRegsMisc4 + kRegsKd4 + kRegsVd4 + 2 * kRegsSm4 + kRegsEpi4 <= 7 * kRegsLaunch4,
              "register split");

// ------------------------------------------------------------------ PTX

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Eight E2M1 codes (element i in bits 4i..4i+3) times the FP16 pair s: four
// FP16 pairs, exactly.
__device__ __forceinline__ void dequant8(uint32_t w, __half2 s, uint32_t* out) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __hmul2(*reinterpret_cast<__half2*>(&r[i]), s);
    out[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
}

// Block scales 2 i and 2 i + 1 of a row, each as a pair of equal FP16 values.
__device__ __forceinline__ void scale_pairs(uint32_t two_bytes, __half2& s0, __half2& s1) {
  const uint32_t h = e4m3x2_to_f16x2(two_bytes);
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  s0 = __low2half2(v);
  s1 = __high2half2(v);
}

// ------------------------------------------------------------------ units

// The CTA's units blockIdx.x, + gridDim.x, ... in decode_unit's order, carried
// in 32 bits from one to the next (the host refuses 2^31 - gridDim units or
// more): 64-bit divisions in every warp were a sixth of all instructions.
struct Walk {
  uint32_t per_head, rem, g, left;     // left: units still to do, this one included
  __device__ explicit Walk(const TcParams& p) {
    per_head = static_cast<uint32_t>(p.T) * p.splits;
    const uint32_t units = per_head * p.Hkv;
    g = blockIdx.x / per_head;
    rem = blockIdx.x - g * per_head;
    left = blockIdx.x < units ? (units - blockIdx.x + gridDim.x - 1) / gridDim.x : 0u;
  }
  __device__ bool more() const { return left != 0u; }
  __device__ void next() {
    --left;
    rem += gridDim.x;
    while (rem >= per_head && left != 0u) {
      rem -= per_head;
      ++g;
    }
  }
  __device__ Unit unit(const TcParams& p) const {
    Unit r;
    const uint32_t t = p.splits == 1 ? rem : rem / static_cast<uint32_t>(p.splits);
    r.g = static_cast<int>(g);
    r.t = t;
    r.s = static_cast<int>(rem - t * p.splits);
    int n = p.K;
    if (p.n_valid != nullptr) n = min(n, max(__ldg(p.n_valid + r.t * p.Hkv + r.g), 0));
    r.j0 = r.s * p.chunk;
    r.n_eff = max(0, min((n << p.block_shift) - r.j0, p.chunk));
    r.n_tiles = (r.n_eff + kKeys - 1) / kKeys;
    return r;
  }
};

// ------------------------------------------------------------------ producers

// Warp pw copies rows 32 pw .. 32 pw + 31 of every tile: 8 lanes per code row
// (four rows per instruction), then each lane its own row's scales.
// Which keys count goes to the softmax warps as one ballot word per quadrant,
// in a ring of kMasks tiles: a tile's K stage is refilled only once K tile c -
// kStages is in TMEM, which runs at most kTkStages / 2 tiles ahead of the
// scores, and those at most two ahead of the softmax's reads (with the S it
// has handed back): kStages + kTkStages / 2 + 2 < kMasks.
static_assert(kStages + kTkStages / 2 + 2 < kMasks, "key masks");
template <bool kBlocks>
__device__ void producer4(const F4Params& fp, const Sync& sy, uint32_t sb, uint8_t* sp, int pw, int lane) {
  const TcParams& p = fp.t;
  uint32_t c_tile = 0;
  const int cc = lane & 7, rsel = lane >> 3;
  const int r_own = 32 * pw + lane;
  bool ok = true;
  for (Walk wk(p); wk.more() && ok; wk.next()) {
    const Unit un = wk.unit(p);
    const int32_t* list = p.idx + un.t * p.idx_st + static_cast<int64_t>(un.g) * p.idx_sh;
    const int32_t last = kBlocks ? last_visible(p, un.t) : 0x7fffffff;
    const int64_t hc = static_cast<int64_t>(un.g) * fp.c_sh + cc * 16, hb = static_cast<int64_t>(un.g) * fp.b_sh;
    int32_t entry_next = un.n_tiles > 0 ? key_entry<kBlocks>(p, list, un, r_own) : -1;
    for (int i = 0; i < un.n_tiles && ok; ++i, ++c_tile) {
      int32_t id = key_slot<kBlocks>(p, un, i * kKeys + r_own, entry_next, last);
      entry_next = i + 1 < un.n_tiles ? key_entry<kBlocks>(p, list, un, (i + 1) * kKeys + r_own) : -1;
      if (id == -2) {
        id = -1;
        if (p.status != nullptr) atomicOr(p.status, static_cast<int32_t>(kStatusOob));
      }
      const uint32_t slot = c_tile % kStages, par = ((c_tile / kStages) & 1u) ^ 1u;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {                 // K tile, then V tile
        ok = sy.wait_warp((kv ? J_VE : J_KE) + slot, par);
        if (!ok) break;
        const uint32_t dst = sb + (kv ? H_V : H_K) + slot * kStageBytes;
        const char* src0 = fp.codes[kv] + hc;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = 32 * pw + 4 * k + rsel;
          const int32_t rid = __shfl_sync(0xffffffffu, id, 4 * k + rsel);
          const char* src = src0 + (rid >= 0 ? static_cast<int64_t>(rid) * fp.c_ss : int64_t(0));
          cp_async_16(dst + r * 128 + ((cc ^ (r & 7)) << 4), src, rid >= 0 ? 16 : 0);
        }
        const char* sb0 = fp.bscale[kv] + hb + (id >= 0 ? static_cast<int64_t>(id) * fp.b_ss : int64_t(0));
        cp_async_16(dst + kCodeBytes + r_own * 16, sb0, id >= 0 ? 16 : 0);
        if (kv == 0) {
          const uint32_t mask = __ballot_sync(0xffffffffu, id >= 0);
          if (lane == 0) {
            reinterpret_cast<volatile uint32_t*>(sp + H_MASK)[(c_tile % kMasks) * 4 + pw] = mask;
            mbar_arrive(sy.bar(J_KF + slot));
          }
        }
        cp_async_mbar_arrive(sy.bar((kv ? J_VF : J_KF) + slot));
      }
    }
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");
}

// ------------------------------------------------------------------ dequantisation

// Thread = key row of the tile.  K: the row's FP16 values go to TMEM lane =
// key, two dims per column, 128 dims (64 columns) per stage.
__device__ void k_dequant(const F4Params& fp, const Sync& sy, uint32_t sb, uint32_t tmem, int warp, int lane) {
  const TcParams& p = fp.t;
  uint32_t c_tile = 0, c_half = 0;
  const int row = (warp & 3) * 32 + lane;
  const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kUK;
  bool ok = true;
  for (Walk wk(p); wk.more() && ok; wk.next()) {
    const Unit un = wk.unit(p);
    for (int i = 0; i < un.n_tiles && ok; ++i, ++c_tile) {
      const uint32_t slot = c_tile % kStages;
      ok = sy.wait_warp(J_KF + slot, (c_tile / kStages) & 1u);
      if (!ok) break;
      const uint32_t src = sb + H_K + slot * kStageBytes;
      const uint4 sc = ld_shared_v4(src + kCodeBytes + row * 16);
#pragma unroll 1
      for (int h = 0; h < 2; ++h, ++c_half) {
        const uint32_t st = c_half % kTkStages;
        ok = sy.wait_warp(J_TKE + st, ((c_half / kTkStages) & 1u) ^ 1u);
        if (!ok) break;
        tc_fence_after();
        uint32_t s01 = h ? sc.z : sc.x, s23 = h ? sc.w : sc.y;
        // kept rolled: with every role's loops unrolled the warps waited for
        // instructions more than for anything else
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {                  // 32 dims: one 16-byte chunk, two block scales
          const uint4 w = ld_shared_v4(src + row * 128 + (((4 * h + c) ^ (row & 7)) << 4));
          __half2 s0, s1;
          scale_pairs(s01 & 0xffffu, s0, s1);
          s01 = c == 1 ? s23 : s01 >> 16;
          uint32_t out[16];
          dequant8(w.x, s0, out);
          dequant8(w.y, s0, out + 4);
          dequant8(w.z, s1, out + 8);
          dequant8(w.w, s1, out + 12);
          tmem_st16(tl + st * 64 + c * 16, out);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.bar(J_TKF + st));
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.bar(J_KE + slot));
    }
  }
}

// V: the row's FP16 values into the MN-major 128-byte-swizzled tile.
__device__ void v_dequant(const F4Params& fp, const Sync& sy, uint32_t sb, int warp, int lane) {
  const TcParams& p = fp.t;
  uint32_t c_tile = 0, c_half = 0;
  const int row = (warp & 3) * 32 + lane;
  bool ok = true;
  for (Walk wk(p); wk.more() && ok; wk.next()) {
    const Unit un = wk.unit(p);
    for (int i = 0; i < un.n_tiles && ok; ++i, ++c_tile) {
      const uint32_t slot = c_tile % kStages;
      ok = sy.wait_warp(J_VF + slot, (c_tile / kStages) & 1u);
      if (!ok) break;
      const uint32_t src = sb + H_V + slot * kStageBytes;
      const uint4 sc = ld_shared_v4(src + kCodeBytes + row * 16);
#pragma unroll 1
      for (int h = 0; h < 2; ++h, ++c_half) {
        const uint32_t st = c_half % kVHalves;
        ok = sy.wait_warp(J_VHE + st, ((c_half / kVHalves) & 1u) ^ 1u);
        if (!ok) break;
        const uint32_t dst = sb + H_VH + st * kHalfBytes + row * 128;
        uint32_t s01 = h ? sc.z : sc.x, s23 = h ? sc.w : sc.y;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {                  // 32 dims: FP16 chunks 4 c .. 4 c + 3 of the half
          const uint4 w = ld_shared_v4(src + row * 128 + (((4 * h + c) ^ (row & 7)) << 4));
          __half2 s0, s1;
          scale_pairs(s01 & 0xffffu, s0, s1);
          s01 = c == 1 ? s23 : s01 >> 16;
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
          const uint32_t blk = dst + (c >> 1) * kBlockBytes;
          const int c0 = 4 * (c & 1);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
            dequant8(ws[j], j < 2 ? s0 : s1, o);
            st_shared_v4(blk + (((c0 + j) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.bar(J_VHF + st));
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.bar(J_VE + slot));
    }
  }
}

// ------------------------------------------------------------------ Q

// Lane l takes head l / 2, dims [128 (l & 1), +128): the head's largest |q|
// (with its partner lane), then q * 2^a in FP16, K-major with the 128-byte
// swizzle (four 64-dim blocks of 16 rows x 128 B), and 2^-a * scale_log2.
// Heads past the group are zero.
__device__ __forceinline__ void q_tile(const TcParams& p, const Unit& un, uint32_t qt, float* qsc, int lane) {
  const int h = lane >> 1, half = lane & 1;
  const bool live = h < p.G;
  const uint4* src = reinterpret_cast<const uint4*>(
      reinterpret_cast<const char*>(p.q_ptr) +
      (un.t * p.q_st + (static_cast<int64_t>(un.g) * p.G + (live ? h : 0)) * p.q_sh + half * 128) * 2);
  uint32_t mx = 0u;
  if (live) {
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const uint4 v = __ldg(src + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = max(mx, max((w[j] << 16) & 0x7fffffffu, w[j] & 0x7fff0000u));
    }
  }
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  // a = 14 - floor(log2 max): the largest |q| * 2^a lands in [2^14, 2^15)
  int a = 0;
  if (mx != 0u) a = 14 - (static_cast<int>(mx >> 23) - 127);
  a = min(a, 126);
  const float up = __int_as_float((127 + a) << 23);
  if (half == 0) qsc[h] = p.scale_log2 * __int_as_float((127 - a) << 23);
#pragma unroll 4
  for (int c = 0; c < 16; ++c) {
    const uint4 v = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = pack_f16x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
    const int blk = 2 * half + (c >> 3);
    st_shared_v4(qt + blk * (kQBytes / 4) + h * 128 + (((c & 7) ^ (h & 7)) << 4), o[0], o[1], o[2], o[3]);
  }
}

__device__ void q4(const TcParams& p, const Sync& sy, uint32_t sb, uint8_t* sp, int lane) {
  uint32_t c_unit = 0;
  bool ok = true;
  for (Walk wk(p); wk.more() && ok; wk.next()) {
    const Unit un = wk.unit(p);
    const uint32_t qb = c_unit & 1u;
    ok = sy.wait_warp(J_QE + qb, ((c_unit >> 1) & 1u) ^ 1u);
    if (!ok) break;
    ++c_unit;
    if (un.n_tiles > 0)
      q_tile(p, un, sb + H_Q + qb * kQBytes, reinterpret_cast<float*>(sp + H_QSC) + qb * kGp, lane);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(sy.bar(J_QF + qb));
      if (un.n_tiles == 0) mbar_arrive(sy.bar(J_QE + qb));
    }
  }
}

// ------------------------------------------------------------------ MMA issuers

__device__ void qk4(const TcParams& p, const Sync& sy, uint32_t sb, uint32_t tmem) {
  uint32_t c_tile = 0, c_half = 0, c_unit = 0;
  bool ok = true;
  for (Walk wk(p); wk.more() && ok; wk.next()) {
    const Unit un = wk.unit(p);
    const uint32_t qb = c_unit & 1u;
    if (un.n_tiles > 0) ok = sy.wait(J_QF + qb, (c_unit >> 1) & 1u);
    if (!ok) break;
    ++c_unit;
    const uint32_t qt = sb + H_Q + qb * kQBytes;
    for (int i = 0; i < un.n_tiles && ok; ++i, ++c_tile) {
      const uint32_t sbuf = c_tile & 1u;
      ok = sy.wait(J_SE + sbuf, ((c_tile >> 1) & 1u) ^ 1u);
      for (int h = 0; h < 2 && ok; ++h, ++c_half) {
        const uint32_t st = c_half % kTkStages;
        ok = sy.wait(J_TKF + st, (c_half / kTkStages) & 1u);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          // A: 16 dims are 8 TMEM columns; B: 32 bytes further inside the swizzle atom
          const int ks = 8 * h + kk;
          const uint64_t b = smem_desc(qt + (ks >> 2) * (kQBytes / 4) + (ks & 3) * 32, 16, 1024, 2);
          umma_f16_ts(tmem + kUS + sbuf * 16, tmem + kUK + st * 64 + kk * 8, b, kIdescQK4, ks > 0 ? 1u : 0u);
        }
        umma_commit(sy.bar(J_TKE + st));
      }
      if (!ok) break;
      umma_commit(sy.bar(J_SF + sbuf));
      if (i == un.n_tiles - 1) umma_commit(sy.bar(J_QE + qb));
    }
  }
  umma_commit(sy.bar(J_DONE));
  sy.drain(J_DONE, 0);
}

__device__ void pv4(const TcParams& p, const Sync& sy, uint32_t sb, uint32_t tmem) {
  uint32_t c_tile = 0, c_half = 0, c_unit = 0;
  bool ok = true;
  for (Walk wk(p); wk.more() && ok; wk.next()) {
    const Unit un = wk.unit(p);
    const uint32_t ue = c_unit++;
    const uint32_t ob = ue & 1u;
    ok = sy.wait(J_OE + ob, ((ue >> 1) & 1u) ^ 1u);
    if (!ok) break;
    if (un.n_tiles == 0) {
      mbar_arrive(sy.bar(J_OF + ob));
      continue;
    }
    for (int i = 0; i < un.n_tiles && ok; ++i, ++c_tile) {
      const uint32_t pb = c_tile & 1u;
      ok = sy.wait(J_PF + pb, (c_tile >> 1) & 1u);
      for (int mh = 0; mh < 2 && ok; ++mh, ++c_half) {
        const uint32_t st = c_half % kVHalves;
        ok = sy.wait(J_VHF + st, (c_half / kVHalves) & 1u);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          // as the BF16 kernel's PV: V^T and P^T both MN-major
          const uint64_t a = smem_desc(sb + H_VH + st * kHalfBytes + kk * 2048, kBlockBytes, 1024, 2);
          const uint64_t b = smem_desc(sb + H_P + pb * kPBytes + kk * 256, 128, 2048, 0);
          umma_f16_ss(tmem + kUO + ob * 32 + mh * 16, a, b, kIdescPV4, (i == 0 && kk == 0) ? 0u : 1u);
        }
        umma_commit(sy.bar(J_VHE + st));
      }
      if (!ok) break;
      umma_commit(sy.bar(J_PE + pb));
    }
    if (ok) umma_commit(sy.bar(J_OF + ob));
  }
  umma_commit(sy.bar(J_DONE + 1));
  sy.drain(J_DONE + 1, 0);
}

// ------------------------------------------------------------------ softmax

// Softmax warp w: TMEM lane quadrant w & 3 (thread = key of the tile), heads
// [8 hh, 8 hh + 8).  x = s - mx with mx = m - 7 (m the running max), so that
// p = 2^x is the probability times 2^7 and x > 15 means the lazy rescale's
// bound is passed.  The votes, the exact path and the sums are those of the
// FP8 kernel.  Heads past the group have a score factor 0 and mx = +inf.
__device__ void softmax4(const TcParams& p, const Sync& sy, uint32_t sb, uint8_t* sp, uint32_t tmem, int warp,
                         int lane) {
  const int wq = warp & 3;
  const int hh = (warp - kWarpSm4) >> 2;
  const int h0 = hh * kHpw4;
  const int key = wq * 32 + lane;
  const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  float* red_max = reinterpret_cast<float*>(sp + H_RED);
  uint8_t* votes = sp + H_RED + 256;
  float* red_sum = red_max + 128;
  const float* qsc_all = reinterpret_cast<const float*>(sp + H_QSC);
  const volatile uint32_t* masks = reinterpret_cast<const volatile uint32_t*>(sp + H_MASK) + wq;
  constexpr float kOver = kRescaleLog2 + kPShift;
  uint32_t c_tile = 0, c_unit = 0, c_exact = 0;
  uint32_t vote_par = 0u;
  bool ok = true;
  for (Walk wk(p); wk.more() && ok; wk.next()) {
    const Unit un = wk.unit(p);
    const uint32_t qb = c_unit & 1u;
    ok = sy.wait_warp(J_QF + qb, (c_unit >> 1) & 1u);
    if (!ok) break;
    float qs[kHpw4], mx[kHpw4], l_part[kHpw4];
#pragma unroll
    for (int h = 0; h < kHpw4; ++h) {
      qs[h] = h0 + h < p.G ? qsc_all[qb * kGp + h0 + h] : 0.f;
      mx[h] = h0 + h < p.G ? -INFINITY : INFINITY;     // no key seen; never one
      l_part[h] = 0.f;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(sy.bar(J_QE + qb));
    for (int i = 0; i < un.n_tiles; ++i) {
      const uint32_t c = c_tile + i;
      const uint32_t buf = c & 1u;
      ok = sy.wait_warp(J_SF + buf, (c >> 1) & 1u);
      if (!ok) break;
      tc_fence_after();
      uint32_t r8[8];
      tmem_ld8(tl + kUS + buf * 16 + 8 * hh, r8);
      const bool valid = (masks[(c % kMasks) * 4] >> lane) & 1u;
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.bar(J_SE + buf));
      float x[kHpw4];
      bool exact = true;
      if (i > 0) {
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < kHpw4; ++h) {
          // a head without a key yet has mx = -inf and takes the exact path
          x[h] = valid ? fmaf(__uint_as_float(r8[h]), qs[h], -mx[h]) : -INFINITY;
          top = fmaxf(top, x[h]);
        }
        const bool wover = __any_sync(0xffffffffu, top > kOver);
        uint8_t* vt = votes + buf * 8;
        if (lane == 0) vt[warp - kWarpSm4] = wover ? 1 : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.bar(J_RMAX + buf));
        if (!wover) {
#pragma unroll
          for (int h = 0; h < kHpw4; ++h) x[h] = ex2(x[h]);
        }
        ok = sy.wait_warp(J_RMAX + buf, (vote_par >> buf) & 1u);
        vote_par ^= 1u << buf;
        if (!ok) break;
        const uint2 vw = *reinterpret_cast<const uint2*>(vt);
        exact = (vw.x | vw.y) != 0u;
      }
      if (exact) {
        float s[kHpw4];
#pragma unroll
        for (int h = 0; h < kHpw4; ++h) s[h] = valid && h0 + h < p.G ? __uint_as_float(r8[h]) * qs[h] : -INFINITY;
        const float wmax = xreduce8<true>(s, lane);
        float* rm = red_max;
        if ((lane & 3) == 0) rm[wq * 16 + h0 + ((lane >> 2) & 7)] = wmax;
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.bar(J_RMX2));
        ok = sy.wait_warp(J_RMX2, c_exact & 1u);
        ++c_exact;
        if (!ok) break;
        float tmax[kHpw4];                             // the tile's max, less 7
        bool need = false;
#pragma unroll
        for (int h = 0; h < kHpw4; ++h) {
          tmax[h] = fmaxf(fmaxf(rm[h0 + h], rm[16 + h0 + h]), fmaxf(rm[32 + h0 + h], rm[48 + h0 + h])) - kPShift;
          need |= (mx[h] != -INFINITY) && (tmax[h] > mx[h] + kRescaleLog2);
        }
        if (need) {                                    // (never on a unit's first tile: no head has a max yet)
          const uint32_t cp = c - 1;
          ok = sy.wait_warp(J_PE + (cp & 1u), (cp >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          float alpha[kHpw4];
#pragma unroll
          for (int h = 0; h < kHpw4; ++h) {
            const float mn = fmaxf(mx[h], tmax[h]);
            alpha[h] = mx[h] == mn ? 1.f : ex2(mx[h] - mn);
            mx[h] = mn;
            l_part[h] *= alpha[h];
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t o[8];
            const uint32_t col = kUO + (c_unit & 1u) * 32 + half * 16 + 8 * hh;
            tmem_ld8(tl + col, o);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < kHpw4; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * alpha[h]);
            tmem_st8(tl + col, o);
          }
          tmem_wait_st();
        } else {
#pragma unroll
          for (int h = 0; h < kHpw4; ++h)
            if (mx[h] == -INFINITY) mx[h] = tmax[h];
        }
        // still no key of this head: every s is -inf and p = 0
#pragma unroll
        for (int h = 0; h < kHpw4; ++h) x[h] = ex2(s[h] - (mx[h] == -INFINITY ? 0.f : mx[h]));
      }
      uint32_t pk[4];
#pragma unroll
      for (int h = 0; h < kHpw4; h += 2) pk[h >> 1] = pack_f16x2(x[h], x[h + 1]);
#pragma unroll
      for (int h = 0; h < kHpw4; ++h) l_part[h] += x[h];
      ok = sy.wait_warp(J_PE + buf, ((c >> 1) & 1u) ^ 1u);
      if (!ok) break;
      st_shared_v4(sb + H_P + buf * kPBytes + hh * 2048 + key * 16, pk[0], pk[1], pk[2], pk[3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.bar(J_PF + buf));
    }
    if (!ok) break;
    const float wsum = xreduce8<false>(l_part, lane);
    float* rs = red_sum + (c_unit & 1u) * 64;
    if ((lane & 3) == 0) rs[wq * 16 + h0 + ((lane >> 2) & 7)] = wsum;
    __syncwarp();
    if (lane == 0) mbar_arrive(sy.bar(J_RSUM + (c_unit & 1u)));
    ok = sy.wait_warp(J_RSUM + (c_unit & 1u), (c_unit >> 1) & 1u);
    if (!ok) break;
    const uint32_t lb = c_unit & 1u;
    if (wq == 0) {
      ok = sy.wait_warp(J_LE + lb, ((c_unit >> 1) & 1u) ^ 1u);
      if (!ok) break;
      float* lm = reinterpret_cast<float*>(sp + H_LM) + lb * 32;
      if (lane < kHpw4) {
        float mk = 0.f;
#pragma unroll
        for (int h = 0; h < kHpw4; ++h)
          if (h == lane) mk = mx[h];
        const int h = h0 + lane;
        lm[h] = (rs[h] + rs[16 + h]) + (rs[32 + h] + rs[48 + h]);
        lm[16 + h] = mk;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.bar(J_LF + lb));
    }
    c_tile += un.n_tiles;
    ++c_unit;
  }
}

// Epilogue warp (TMEM lane quadrant w & 3: thread = dim of an output half).
// l = 0 marks an empty row (zeros, lse = -inf); a NaN l stays NaN.
__device__ void epilogue4(const TcParams& p, const Sync& sy, uint8_t* sp, uint32_t tmem, int warp, int lane) {
  const int wq = warp & 3;
  const int key = wq * 32 + lane;
  const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  uint32_t c_unit = 0;
  const int G = p.G;
  bool ok = true;
  for (Walk wk(p); wk.more() && ok; wk.next()) {
    const Unit un = wk.unit(p);
    const uint32_t ub = c_unit & 1u, par = (c_unit >> 1) & 1u;
    ++c_unit;
    ok = sy.wait_warp(J_LF + ub, par);
    if (!ok) break;
    const float* lm = reinterpret_cast<const float*>(sp + H_LM) + ub * 32;
    const int64_t row0 = un.t * static_cast<int64_t>(p.Hkv) * G + static_cast<int64_t>(un.g) * G;
    if (wq == 0 && lane < G && (p.lse != nullptr || p.part_lse != nullptr)) {
      const float lk = lm[lane], mk = lm[16 + lane];
      const float lv = lk == 0.f ? -INFINITY : (mk + lg2(lk)) * 0.69314718055994531f;
      if (p.part_lse != nullptr)
        p.part_lse[(row0 + lane) * p.splits + un.s] = lv;
      else
        p.lse[un.t * p.lse_st + static_cast<int64_t>(un.g) * G + lane] = lv;
    }
    float inv[kGp];
#pragma unroll
    for (int h = 0; h < kGp; ++h) inv[h] = lm[h] == 0.f ? 0.f : p.o_scale / lm[h];
    __syncwarp();
    if (lane == 0) mbar_arrive(sy.bar(J_LE + ub));
    ok = sy.wait_warp(J_OF + ub, par);
    if (!ok) break;
    tc_fence_after();
    __nv_bfloat16* orow = p.out + un.t * p.o_st + static_cast<int64_t>(un.g) * G * p.o_sh;
#pragma unroll
    for (int q = 0; q < 4; ++q) {                     // half q >> 1, heads 8 (q & 1) ..
      uint32_t o[8] = {};
      if (un.n_tiles > 0) {
        tmem_ld8(tl + kUO + ub * 32 + q * 8, o);
        tmem_wait_ld();
      }
      if (q == 3) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.bar(J_OE + ub));
      }
      const int dim = (q >> 1) * 128 + key;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int h = (q & 1) * 8 + j;
        if (h < G) {
          const float v = inv[h] != 0.f ? __uint_as_float(o[j]) * inv[h] : 0.f;
          if (p.part_o != nullptr)
            p.part_o[((row0 + h) * p.splits + un.s) * 256 + dim] = v;
          else
            orow[h * p.o_sh + dim] = __float2bfloat16_rn(v);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ kernel

template <bool kBlocks>
__global__ void __launch_bounds__(kThreads4, 1) qsa_prefill_f4_kernel(const __grid_constant__ F4Params fp) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sp = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const TcParams& p = fp.t;
  Sync sy;
  sy.bars = sb + H_BAR;
  sy.abort_flag = reinterpret_cast<volatile uint32_t*>(sp + H_MISC + 4);
  sy.status = p.status;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(sy.bar(J_KF + s), 128 + 4);         // every lane's copies; each warp's key mask
      mbar_init(sy.bar(J_KE + s), 4);
      mbar_init(sy.bar(J_VF + s), 128);
      mbar_init(sy.bar(J_VE + s), 4);
    }
    for (int s = 0; s < kTkStages; ++s) {
      mbar_init(sy.bar(J_TKF + s), 4);
      mbar_init(sy.bar(J_TKE + s), 1);
    }
    for (int s = 0; s < kVHalves; ++s) {
      mbar_init(sy.bar(J_VHF + s), 4);
      mbar_init(sy.bar(J_VHE + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sy.bar(J_SF + b), 1);
      mbar_init(sy.bar(J_SE + b), kSmWarps4);
      mbar_init(sy.bar(J_PF + b), kSmWarps4);
      mbar_init(sy.bar(J_PE + b), 1);
      mbar_init(sy.bar(J_QF + b), 1);
      mbar_init(sy.bar(J_QE + b), 1 + kSmWarps4);
      mbar_init(sy.bar(J_RMAX + b), kSmWarps4);
      mbar_init(sy.bar(J_RSUM + b), kSmWarps4);
      mbar_init(sy.bar(J_OF + b), 1);
      mbar_init(sy.bar(J_OE + b), 4);
      mbar_init(sy.bar(J_LF + b), 2);
      mbar_init(sy.bar(J_LE + b), 4);
      mbar_init(sy.bar(J_DONE + b), 1);
    }
    mbar_init(sy.bar(J_RMX2), kSmWarps4);
    *sy.abort_flag = 0u;
    mbar_fence_init();
  }
  if (warp == kWarpMisc4 + 1) {
    tmem_alloc(sb + H_MISC, kTmemCols4);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sp + H_MISC);

  if (warp < kWarpMisc4) {
    setmaxnreg_dec<kRegsProd4>();
    producer4<kBlocks>(fp, sy, sb, sp, warp, lane);
  } else if (warp < kWarpKd4) {
    setmaxnreg_dec<kRegsMisc4>();
    if (warp == kWarpMisc4) {
      q4(p, sy, sb, sp, lane);
    } else if (warp == kWarpMisc4 + 1) {
      if (lane == 0) qk4(p, sy, sb, tmem);
      __syncwarp();
    } else if (warp == kWarpMisc4 + 2) {
      if (lane == 0) pv4(p, sy, sb, tmem);
      __syncwarp();
    }
  } else if (warp < kWarpVd4) {
    setmaxnreg_inc<kRegsKd4>();
    k_dequant(fp, sy, sb, tmem, warp, lane);
  } else if (warp < kWarpSm4) {
    setmaxnreg_dec<kRegsVd4>();
    v_dequant(fp, sy, sb, warp, lane);
  } else if (warp < kWarpEpi4) {
    setmaxnreg_inc<kRegsSm4>();
    softmax4(p, sy, sb, sp, tmem, warp, lane);
  } else {
    setmaxnreg_dec<kRegsEpi4>();
    epilogue4(p, sy, sp, tmem, warp, lane);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMisc4 + 1) tmem_dealloc(tmem, kTmemCols4);
}

}  // namespace f4
}  // namespace qsa
