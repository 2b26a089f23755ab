// qsa_prefill_f4.cuh -- QSA top-K sparse attention over a 4-bit KV cache
// (sm_100a): cp.async gather, dequantisation in registers, mma.sync.
//
// The operation is the one of qsa_prefill_tc.cuh over cache rows of E2M1
// codes with one E4M3 scale per 16 dims and an FP32 scale per tensor:
// element = code * block scale * tensor scale.
//
// Numerics.  An E2M1 value (2 significant bits) times an E4M3 value (4) has at
// most 6 significant bits and lies between 2^-10 and 2688, so code * block
// scale is exact in FP16.  The tensor scales go into the softmax scale and the
// output.  The query is scaled per head by a power of two that puts its
// largest |q| in [2^14, 2^15) and is then exact in FP16 for every element
// within 2^31 of that (smaller ones are off by at most 2^-25 after scaling,
// 2^-39 of the largest).  Probabilities are rounded to FP16 (11 significant
// bits) after scaling by 2^7, which with the lazy rescale's p <= 2^8 stays
// below FP16's largest number and puts the smallest step at 2^-31.
//
// Why mma.sync.  A list belongs to one token and one KV head, so the matrices
// have 16 rows (the padded head group).  A tcgen05 MMA with 128 keys or dims
// as its M takes 59 cycles (A from shared memory) or 46 (A from TMEM) for any
// N up to 64 (measured, kind::f16, K = 16): 32 of them per 128 keys are 1500
// to 1900 cycles on the SM, and every dequantised element passes through
// shared memory or TMEM.  m16n8k16 mma.sync fits the 16 rows exactly, takes
// 2.0 cycles on the SM (512 per 128 keys: 1030 cycles) and reads the
// dequantised registers directly.  A warp-specialised tcgen05 version of this
// kernel (K dequantised to TMEM, V to shared memory) ran at 2.85 ms where
// this one takes 2.12 (8192 tokens, 131072 slots, heads (24,2), 2048 entries).
//
// Layout.  A unit is one (token, KV head, chunk of the list); it is worked by
// W warps (1, 2, 4 or 8 of the CTA's 8), each taking every W-th group of 32
// keys with its own running max, sum and output, merged at the unit's end.
// Within a warp (lane = 4 n + j, n = 0..7, j = 0..3) nothing is exchanged but
// the max:
//   S = Q K^T   m16n8k16, rows = heads, columns = keys.  Lane (n, j) reads 32
//               bytes of key n's codes, dims 64 j .. 64 j + 63; MMA step s takes
//               its dims 64 j + 4 s .. + 3 as k = 2j, 2j+1, 2j+8, 2j+9, and Q is
//               read in the same order: the sum does not mind the order of dims.
//   O += P V    rows = heads, columns = dims, k = keys.  The S fragments are
//               the P fragments of the same keys.  Lane (n, j) reads 16 bytes
//               (dims 32 n .. + 31) of keys 2j, 2j+1, 2j+8, 2j+9; nibbles of two
//               keys are interleaved, so that one conversion makes the pair of
//               keys an MMA register holds; output column n of step x is dim
//               32 n + x.
// The code rows sit in shared memory with 16-byte chunk c of row r at place
// c ^ (r & 7): both read patterns and the copies are free of bank conflicts.
//
// What bounds it (that workload, per 128 keys of a list): 2150 cycles, in which
// the MMA pipe is busy 1020, the ALU pipe (conversions, nibbles, addresses) 880
// and half the issue slots are used by 4310 warp instructions.  The 128 output
// accumulators (255 registers, 12 bytes of spills) leave two warps to a
// scheduler, too few to keep three pipes busy at once; splitting a unit between
// warps cost more instructions than the extra warps won.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "qsa_prefill_tc.cuh"

namespace qsa {
namespace f4 {

using tc::key_entry;
using tc::key_slot;
using tc::last_visible;
using tc::TcParams;
using tc::Unit;

struct F4Params {
  TcParams t;                     // its kraw / vraw / kv strides / tm_q are unused
  const char* codes[2];           // K, V
  const char* bscale[2];
  int64_t c_sh, b_sh;             // byte strides of the heads, codes and scales,
  int32_t c_ss, b_ss;             // and of the slots (32 bits: one multiply-add per address)
};

constexpr int kWarps4 = 8, kThreads4 = 32 * kWarps4;
constexpr int kGroup = 32;                          // keys a warp takes at a time
constexpr int kStages = 2;                          // groups in a warp's ring
constexpr int kOffV = kGroup * 128, kOffKs = 2 * kGroup * 128, kOffVs = kOffKs + kGroup * 16;
constexpr int kStageBytes = kOffVs + kGroup * 16;   // K codes, V codes, K scales, V scales
constexpr int kQTile = 16 * 512;                    // FP16 Q of a unit
constexpr int H_RING = 0;
constexpr int H_Q = H_RING + kWarps4 * kStages * kStageBytes;
constexpr int H_QSC = H_Q + kWarps4 * kQTile;       // per unit in work: 16 score factors
constexpr int H_ML = H_QSC + kWarps4 * 16 * 4;      // per warp: mx[16], l[16] (merge)
constexpr int H_SMEM = H_ML + kWarps4 * 32 * 4;
static_assert(H_SMEM <= 232448, "shared memory");
static_assert(kStages * kStageBytes >= 16 * 256 * 4, "a warp's ring holds its output for the merge");
constexpr float kPShift = 7.f;                      // P is formed times 2^7
constexpr float kOver = tc::kRescaleLog2 + kPShift; // x above this: the running max must rise

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];\n" : "=h"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}

// Eight E2M1 codes (element i in bits 4i..4i+3) times the FP16 pair s: four
// FP16 pairs, exactly.
__device__ __forceinline__ void dequant8(uint32_t w, __half2 s, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __hmul2(*reinterpret_cast<__half2*>(&out[i]), s);
    out[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
}

__device__ __forceinline__ uint32_t word(const uint4& v, int w) {
  return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
}

// Two E4M3 scales as FP16.
__device__ __forceinline__ __half2 scales2(uint32_t two_bytes) {
  const uint32_t h = e4m3x2_to_f16x2(two_bytes);
  return *reinterpret_cast<const __half2*>(&h);
}

// ------------------------------------------------------------------ clusters

// A decode list cut into up to 8 chunks can run as one cluster, a CTA per
// chunk: each leaves its chunk's max, sum and unnormalised output in its
// shared memory, and the cluster merges them from there, without a workspace
// and a second launch.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ float cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ float4 cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

// A chunk's result in shared memory: O [16][256], then max - 7 [16] and sum [16].
constexpr int kPartO = 0, kPartM = 16 * 256 * 4, kPartL = kPartM + 64, kPartBytes = kPartL + 64;

// Warp `w` of the cluster's `warps` merges heads w, w + warps, ... of the
// chunks' results at `part` of every CTA; put(h, max, sum, first 4 dims of the
// lane's 8, other 4) gets each, unnormalised.
template <typename Put>
__device__ __forceinline__ void cluster_merge(uint32_t part, int chunks, int G, int w, int warps, int lane, Put put) {
  for (int h = w; h < G; h += warps) {
    // every chunk's numbers at once: one trip through the cluster, not one a chunk
    float m[8], ls[8];
    float4 x[8], y[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      m[c] = -INFINITY;
      if (c < chunks) {
        const uint32_t at = cluster_addr(part, c);
        m[c] = cluster_f32(at + kPartM + 4 * h);
        ls[c] = cluster_f32(at + kPartL + 4 * h);
        x[c] = cluster_f32x4(at + kPartO + h * 1024 + lane * 32);
        y[c] = cluster_f32x4(at + kPartO + h * 1024 + lane * 32 + 16);
      }
    }
    float M = -INFINITY, l = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) M = fmaxf(M, m[c]);
    float4 a = {}, b = {};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c >= chunks) continue;
      const float f = m[c] == M ? 1.f : ex2(m[c] - M);   // a chunk without a key: 0
      l += ls[c] * f;
      a = make_float4(fmaf(x[c].x, f, a.x), fmaf(x[c].y, f, a.y), fmaf(x[c].z, f, a.z), fmaf(x[c].w, f, a.w));
      b = make_float4(fmaf(y[c].x, f, b.x), fmaf(y[c].y, f, b.y), fmaf(y[c].z, f, b.z), fmaf(y[c].w, f, b.w));
    }
    put(h, M, l, a, b);
  }
}

// ------------------------------------------------------------------ units

// The units of slot blockIdx.x + gridDim.x * (warp / W), then every gridDim.x *
// (warps of a CTA / W)-th after it, in decode_unit's order, carried in 32 bits from one to
// the next (the host refuses sizes that reach 2^31 a stride past the end).
struct Walk {
  uint32_t per_head, rem, g, step, left;   // left: units still to do, this one included
  __device__ Walk(const TcParams& p, uint32_t slot, uint32_t stride) : step(stride) {
    per_head = static_cast<uint32_t>(p.T) * p.splits;
    const uint32_t units = per_head * p.Hkv;
    g = slot / per_head;
    rem = slot - g * per_head;
    left = slot < units ? (units - slot + stride - 1) / stride : 0u;
  }
  __device__ void next() {
    --left;
    rem += step;
    while (rem >= per_head && left != 0u) {
      rem -= per_head;
      ++g;
    }
  }
  // The unit's place; n_eff and n_tiles as if the whole list counted.
  __device__ Unit unit(const TcParams& p) const {
    Unit r;
    const uint32_t t = p.splits == 1 ? rem : rem / static_cast<uint32_t>(p.splits);
    r.g = static_cast<int>(g);
    r.t = t;
    r.s = static_cast<int>(rem - t * p.splits);
    r.j0 = r.s * p.chunk;
    r.n_eff = max(0, min((p.K << p.block_shift) - r.j0, p.chunk));
    r.n_tiles = (r.n_eff + kGroup - 1) / kGroup;     // groups of 32 keys
    return r;
  }
  // Cuts the unit to n_valid entries.  The first entries are asked for before
  // this, so that the two loads do not wait for one another.
  __device__ static void cut(const TcParams& p, Unit& r) {
    if (p.n_valid == nullptr) return;
    const int n = min(p.K, max(__ldg(p.n_valid + r.t * p.Hkv + r.g), 0));
    r.n_eff = max(0, min((n << p.block_shift) - r.j0, p.chunk));
    r.n_tiles = (r.n_eff + kGroup - 1) / kGroup;
  }
};

// ------------------------------------------------------------------ gather

// The K or V rows of a group: lane r holds key r's slot; 8 lanes per code row
// (four rows per instruction), then each lane its own row's scales.  Masked
// keys (id < 0) become zeros without a read.
__device__ __forceinline__ void gather(uint32_t codes, uint32_t scales, const char* c0, const char* b0, int32_t c_ss,
                                       int32_t b_ss, int32_t id, uint32_t mask, int lane) {
  const int cc = lane & 7, rsel = lane >> 3;
  // row 4 k + rsel: its swizzle phase is rsel for even k, rsel + 4 for odd k
  const uint32_t d0 = codes + rsel * 128 + ((cc ^ rsel) << 4), d1 = codes + rsel * 128 + 512 + ((cc ^ (rsel + 4)) << 4);
  c0 += cc * 16;
  if (mask == 0xffffffffu) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      cp_async_16(((k & 1) ? d1 : d0) + (k >> 1) * 1024,
                  c0 + static_cast<int64_t>(__shfl_sync(0xffffffffu, id, 4 * k + rsel)) * c_ss, 16);
    cp_async_16(scales + lane * 16, b0 + static_cast<int64_t>(id) * b_ss, 16);
  } else {
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      const int32_t rid = __shfl_sync(0xffffffffu, id, 4 * k + rsel);
      cp_async_16(((k & 1) ? d1 : d0) + (k >> 1) * 1024, c0 + static_cast<int64_t>(max(rid, 0)) * c_ss,
                  rid >= 0 ? 16 : 0);
    }
    cp_async_16(scales + lane * 16, b0 + static_cast<int64_t>(max(id, 0)) * b_ss, id >= 0 ? 16 : 0);
  }
}

// K and V rows of a group at once (one exchange of each row's slot).
__device__ __forceinline__ void gather_kv(const F4Params& fp, uint32_t dst, const char* kc, const char* vc,
                                          const char* kb, const char* vb, int32_t id, uint32_t mask, int lane) {
  if (mask != 0xffffffffu) {
    gather(dst, dst + kOffKs, kc, kb, fp.c_ss, fp.b_ss, id, mask, lane);
    gather(dst + kOffV, dst + kOffVs, vc, vb, fp.c_ss, fp.b_ss, id, mask, lane);
    return;
  }
  const int cc = lane & 7, rsel = lane >> 3;
  const uint32_t d0 = dst + rsel * 128 + ((cc ^ rsel) << 4), d1 = dst + rsel * 128 + 512 + ((cc ^ (rsel + 4)) << 4);
  kc += cc * 16;
  vc += cc * 16;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int32_t rid = __shfl_sync(0xffffffffu, id, 4 * k + rsel);
    const uint32_t d = ((k & 1) ? d1 : d0) + (k >> 1) * 1024;
    cp_async_16(d, kc + static_cast<int64_t>(rid) * fp.c_ss, 16);
    cp_async_16(d + kOffV, vc + static_cast<int64_t>(rid) * fp.c_ss, 16);
  }
  cp_async_16(dst + kOffKs + lane * 16, kb + static_cast<int64_t>(id) * fp.b_ss, 16);
  cp_async_16(dst + kOffVs + lane * 16, vb + static_cast<int64_t>(id) * fp.b_ss, 16);
}

// ------------------------------------------------------------------ Q

// The Q tile is kept as the MMA's A fragments: step s (512 bytes), lane 4 n + j
// (16 bytes): dims 64 j + 4 s, + 1 of heads n and n + 8, then dims + 2, + 3 of
// the same, so that one 16-byte load is one fragment.
// One head's row, 8 dims a lane (heads past the group: zeros).
__device__ __forceinline__ uint4 q_load(const TcParams& p, const Unit& un, int h, int lane) {
  if (h >= p.G) return make_uint4(0u, 0u, 0u, 0u);
  return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q_ptr) + un.t * p.q_st +
                                              (static_cast<int64_t>(un.g) * p.G + h) * p.q_sh) +
               lane);
}

// q * 2^a in FP16 with the row's largest |q| in [2^14, 2^15); returns 2^-a.
__device__ __forceinline__ float q_scale(const uint4& v, uint32_t (&o)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t mx = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) mx = max(mx, max((w[j] << 16) & 0x7fffffffu, w[j] & 0x7fff0000u));
  mx = __reduce_max_sync(0xffffffffu, mx);
  int a = 0;
  if (mx != 0u) a = 14 - (static_cast<int>(mx >> 23) - 127);
  a = min(a, 126);
  const float up = __int_as_float((127 + a) << 23);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = pack_f16x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
  return __int_as_float((127 - a) << 23);
}

// A head's row into the Q tile, and its score factor 2^-a * scale_log2.
__device__ __forceinline__ void q_head(const TcParams& p, const uint4& v, uint32_t qt, float* qsc, int h, int lane) {
  uint32_t o[4];
  const float down = q_scale(v, o);
  // the lane's 8 dims are steps 2 (lane % 8) and + 1 of j = lane / 8
  const uint32_t at = qt + 1024 * (lane & 7) + (4 * (h & 7) + (lane >> 3)) * 16 + (h >> 3) * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) sts32(at + 512 * (j >> 1) + 8 * (j & 1), o[j]);
  if (lane == 0) qsc[h] = h < p.G ? p.scale_log2 * down : 0.f;
}

// ------------------------------------------------------------------ kernel

template <bool kBlocks, int W, bool kCluster = false>
__global__ void __launch_bounds__(kThreads4, 1) qsa_attn_f4_kernel(const __grid_constant__ F4Params fp) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const TcParams& p = fp.t;
  const uint32_t sb = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / W, wi = warp % W;              // the unit slot, this warp's place in it
  const int n = lane >> 2, j = lane & 3;
  const uint32_t ring = sb + H_RING + warp * kStages * kStageBytes;
  const uint32_t qt = sb + H_Q + grp * kQTile;
  float* qsc = reinterpret_cast<float*>(sm + H_QSC) + grp * 16;
  auto sync_unit = [&] {
    if (W == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;\n" ::"r"(1 + grp), "n"(32 * W) : "memory");
  };

  for (Walk wk(p, blockIdx.x + gridDim.x * grp, gridDim.x * (kWarps4 / W)); wk.left != 0u; wk.next()) {
    Unit un = wk.unit(p);
    const int32_t* list = p.idx + un.t * p.idx_st + static_cast<int64_t>(un.g) * p.idx_sh;
    const int32_t e_ask = key_entry<kBlocks>(p, list, un, wi * kGroup + lane);
    // every load of Q at once; where a unit is short (several warps to it, or
    // a chunk of a cluster) with the list's first load, else behind it
    constexpr bool kEarlyQ = kCluster || (W > 1 && W < kWarps4);
    uint4 qv[16 / W];
    auto ask_q = [&] {
#pragma unroll
      for (int h = 0; h < 16 / W; ++h) qv[h] = q_load(p, un, wi + h * W, lane);
    };
    if (kEarlyQ) ask_q();
    Walk::cut(p, un);
    const int32_t e_first = wi * kGroup + lane < un.n_eff ? e_ask : -1;
    const int32_t last = kBlocks ? last_visible(p, un.t) : 0x7fffffff;
    const char* kc = fp.codes[0] + un.g * fp.c_sh;
    const char* vc = fp.codes[1] + un.g * fp.c_sh;
    const char* kb = fp.bscale[0] + un.g * fp.b_sh;
    const char* vb = fp.bscale[1] + un.g * fp.b_sh;
    const int groups = un.n_tiles;

    // the slot of this lane's key of group i, from its entry
    auto entry = [&](int i) { return i < groups ? key_entry<kBlocks>(p, list, un, i * kGroup + lane) : -1; };
    uint32_t mask_next = 0u;
    auto issue = [&](int i, int stage, int32_t e) {
      int32_t id = key_slot<kBlocks>(p, un, i * kGroup + lane, e, last);
      if (id == -2) {
        id = -1;
        if (p.status != nullptr) atomicOr(p.status, static_cast<int32_t>(tc::kStatusOob));
      }
      mask_next = __ballot_sync(0xffffffffu, id >= 0);
      gather_kv(fp, ring + stage * kStageBytes, kc, vc, kb, vb, id, mask_next, lane);
      cp_async_commit();
    };
    int32_t e_next = e_first;
    if (!kEarlyQ && groups > 0) ask_q();
    if (wi < groups) issue(wi, 0, e_next);
    e_next = entry(wi + W);
    // Q, while the first rows are on their way
    if (groups > 0) {
#pragma unroll
      for (int h = 0; h < 16 / W; ++h) q_head(p, qv[h], qt, qsc, wi + h * W, lane);
    }
    sync_unit();

    float o[32][4];
#pragma unroll
    for (int x = 0; x < 32; ++x)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[x][r] = 0.f;
    // heads n and n + 8 of this lane: score factor, mx = running max - 7, sum
    float qs[2], mx[2], l[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool live = n + 8 * r < p.G;
      qs[r] = live && groups > 0 ? qsc[n + 8 * r] : 0.f;
      mx[r] = live ? -INFINITY : INFINITY;              // no key seen; never one
      l[r] = 0.f;
    }

    int stage = 0;
    for (int i = wi; i < groups; i += W, stage ^= 1) {
      const uint32_t mask = mask_next;
      cp_async_wait<0>();
      __syncwarp();
      const uint32_t st = ring + stage * kStageBytes;

      // scores of 32 keys: four tiles of 8
      float s[4][4];
      uint32_t ksc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) s[t][r] = 0.f;
        ksc[t] = lds32(st + kOffKs + (8 * t + n) * 16 + 4 * j);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {                  // 32 of the lane's 64 dims
        uint32_t kw[4][4];
        __half2 sc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint4 v = lds128(st + (8 * t + n) * 128 + (((2 * j + hf) ^ n) << 4));
          kw[t][0] = v.x;
          kw[t][1] = v.y;
          kw[t][2] = v.z;
          kw[t][3] = v.w;
          sc[t] = scales2((ksc[t] >> (16 * hf)) & 0xffffu);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {                   // 8 dims: two MMA steps
          const uint4 qa = lds128(qt + 1024 * (4 * hf + w) + 16 * lane);
          const uint4 qb = lds128(qt + 1024 * (4 * hf + w) + 512 + 16 * lane);
          // a tile's two steps are four MMAs apart: an MMA's result takes about
          // as long, and back to back they stalled the warp
          uint32_t b[4][4];
#pragma unroll
          for (int t = 0; t < 4; ++t)
            dequant8(kw[t][w], w < 2 ? __low2half2(sc[t]) : __high2half2(sc[t]), b[t]);
#pragma unroll
          for (int t = 0; t < 4; ++t) mma_f16(s[t], qa.x, qa.y, qa.z, qa.w, b[t][0], b[t][1]);
#pragma unroll
          for (int t = 0; t < 4; ++t) mma_f16(s[t], qb.x, qb.y, qb.z, qb.w, b[t][2], b[t][3]);
        }
      }

      // the next group's rows, asked for here: ahead of the scores their 18
      // copies and addresses held up the K reads (2.44 against 2.12 ms)
      if (i + W < groups) {
        issue(i + W, stage ^ 1, e_next);
        e_next = entry(i + 2 * W);
      }

      // x = s - mx, p = 2^x; s[t] = {head n: keys 2j, 2j+1; head n + 8: the same} of tile t
      float x[4][4];
      float top = -INFINITY;
      const uint32_t mine = mask >> (2 * j);
      const bool full = mask == 0xffffffffu;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[t][r] = fmaf(s[t][r], qs[r >> 1], -mx[r >> 1]);
          top = fmaxf(top, x[t][r]);
        }
      if (!full) {                                      // some key is masked
        top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[t][r] = (mine >> (8 * t + (r & 1))) & 1u ? x[t][r] : -INFINITY;
            top = fmaxf(top, x[t][r]);
          }
      }
      if (__any_sync(0xffffffffu, top > kOver)) {
        // raise the running max (always for a unit's first keys): sums and
        // output scale by 2^(m_old - m_new)
        float alpha[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float m = -INFINITY;
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if ((mine >> (8 * t + e)) & 1u) m = fmaxf(m, s[t][2 * r + e] * qs[r]);
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const float mn = fmaxf(mx[r], m - kPShift);
          alpha[r] = mx[r] == mn ? 1.f : ex2(mx[r] - mn);
          mx[r] = mn;
          l[r] *= alpha[r];
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          o[y][0] *= alpha[0];
          o[y][1] *= alpha[0];
          o[y][2] *= alpha[1];
          o[y][3] *= alpha[1];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            x[t][r] = (mine >> (8 * t + (r & 1))) & 1u
                          ? fmaf(s[t][r], qs[r >> 1], -(mx[r >> 1] == -INFINITY ? 0.f : mx[r >> 1]))
                          : -INFINITY;
      }
      uint32_t pk[4][2];                                // tile t: head n, head n + 8
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[t][r] = ex2(x[t][r]);
          l[r >> 1] += x[t][r];
        }
        pk[t][0] = pack_f16x2(x[t][0], x[t][1]);
        pk[t][1] = pack_f16x2(x[t][2], x[t][3]);
      }

      // output: two steps of 16 keys
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t vw[4][4];                              // keys 2j, 2j+1, 2j+8, 2j+9 of the step
        uint32_t vs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r7 = 2 * j + (k & 1);               // row & 7
          const uint32_t row = 16 * u + 8 * (k >> 1) + r7;
          const uint4 v = lds128(st + kOffV + row * 128 + ((n ^ r7) << 4));
          vw[k][0] = v.x;
          vw[k][1] = v.y;
          vw[k][2] = v.z;
          vw[k][3] = v.w;
          vs[k] = lds16(st + kOffVs + row * 16 + 2 * n);
        }
        // scales of two keys as a pair, for the lane's two groups of 16 dims
        const __half2 s01a = scales2(__byte_perm(vs[0], vs[1], 0x0040)), s01b = scales2(__byte_perm(vs[0], vs[1], 0x0051));
        const __half2 s23a = scales2(__byte_perm(vs[2], vs[3], 0x0040)), s23b = scales2(__byte_perm(vs[2], vs[3], 0x0051));
#pragma unroll
        for (int w = 0; w < 4; ++w) {                   // dims 8 w .. 8 w + 7 of the lane's 32
          constexpr uint32_t M = 0x0f0f0f0fu;
          const __half2 s01 = w < 2 ? s01a : s01b, s23 = w < 2 ? s23a : s23b;
          uint32_t e01[4], o01[4], e23[4], o23[4];      // even and odd dims, keys (0, 1) and (2, 3)
          dequant8((vw[0][w] & M) | ((vw[1][w] << 4) & ~M), s01, e01);
          dequant8((vw[2][w] & M) | ((vw[3][w] << 4) & ~M), s23, e23);
          dequant8(((vw[0][w] >> 4) & M) | (vw[1][w] & ~M), s01, o01);
          dequant8(((vw[2][w] >> 4) & M) | (vw[3][w] & ~M), s23, o23);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            mma_f16(o[8 * w + 2 * b], pk[2 * u][0], pk[2 * u][1], pk[2 * u + 1][0], pk[2 * u + 1][1], e01[b], e23[b]);
            mma_f16(o[8 * w + 2 * b + 1], pk[2 * u][0], pk[2 * u][1], pk[2 * u + 1][0], pk[2 * u + 1][1], o01[b],
                    o23[b]);
          }
        }
      }
      __syncwarp();                                     // the stage is read
    }

#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    const int64_t row0 = (un.t * p.Hkv + un.g) * p.G;
    // l = 0 marks an empty row (zeros, lse = -inf); a NaN l stays NaN
    auto put_lse = [&](int h, float lt, float m) {
      const float lv = lt == 0.f ? -INFINITY : (m + lg2(lt)) * 0.69314718055994531f;
      if (p.part_lse != nullptr)
        p.part_lse[(row0 + h) * p.splits + un.s] = lv;
      else if (p.lse != nullptr)
        p.lse[un.t * p.lse_st + static_cast<int64_t>(un.g) * p.G + h] = lv;
    };
    if (W == 1) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int h = n + 8 * r;
        if (h >= p.G) continue;
        if (j == 0) put_lse(h, l[r], mx[r]);
        const float inv = l[r] == 0.f ? 0.f : p.o_scale / l[r];
        // lane (n, j): dims 64 j .. + 31 in column 2 r, 64 j + 32 .. + 63 in column 2 r + 1
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (p.part_o != nullptr) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + ((row0 + h) * p.splits + un.s) * 256 + 64 * j + 32 * c);
#pragma unroll
            for (int y = 0; y < 8; ++y)
              dst[y] = make_float4(o[4 * y][2 * r + c] * inv, o[4 * y + 1][2 * r + c] * inv,
                                   o[4 * y + 2][2 * r + c] * inv, o[4 * y + 3][2 * r + c] * inv);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.out + un.t * p.o_st + (static_cast<int64_t>(un.g) * p.G + h) * p.o_sh +
                                                  64 * j + 32 * c);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              dst[y] = make_uint4(pack_bf16x2(o[8 * y][2 * r + c] * inv, o[8 * y + 1][2 * r + c] * inv),
                                  pack_bf16x2(o[8 * y + 2][2 * r + c] * inv, o[8 * y + 3][2 * r + c] * inv),
                                  pack_bf16x2(o[8 * y + 4][2 * r + c] * inv, o[8 * y + 5][2 * r + c] * inv),
                                  pack_bf16x2(o[8 * y + 6][2 * r + c] * inv, o[8 * y + 7][2 * r + c] * inv));
          }
        }
      }
      __syncwarp();                                     // Q is read before the next unit's
      continue;
    }

    // Merge of W warps: out = sum_w 2^(mx_w - M) O_w / sum_w 2^(mx_w - M) l_w
    float* ml = reinterpret_cast<float*>(sm + H_ML) + grp * W * 32;
    if (j == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ml[wi * 32 + n + 8 * r] = mx[r];
        ml[wi * 32 + 16 + n + 8 * r] = l[r];
      }
    }
    sync_unit();
    uint8_t* part = sm + H_Q;                           // (Q is read)
    static_assert(kPartBytes <= kWarps4 * kQTile, "a chunk's result fits where Q was");
    float* slab0 = reinterpret_cast<float*>(sm + H_RING + grp * W * kStages * kStageBytes);
    constexpr int kSlab = kStages * kStageBytes / 4;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int h = n + 8 * r;
      float M = -INFINITY;
      for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w * 32 + h]);
      const float f = mx[r] == M ? 1.f : ex2(mx[r] - M);  // a warp without a key: 0
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          // 16-byte chunk (4 dims) 16 j + 8 c + y of row h, spread over the banks
          const int ch = 16 * j + 8 * c + y;
          float4* dst = reinterpret_cast<float4*>(slab0 + wi * kSlab + h * 256) + (ch ^ (2 * j + (n & 1)));
          *dst = make_float4(o[4 * y][2 * r + c] * f, o[4 * y + 1][2 * r + c] * f, o[4 * y + 2][2 * r + c] * f,
                             o[4 * y + 3][2 * r + c] * f);
        }
    }
    sync_unit();
    for (int h = wi; h < p.G; h += W) {
      float M = -INFINITY, lt = 0.f;
      for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w * 32 + h]);
      for (int w = 0; w < W; ++w) {
        const float m = ml[w * 32 + h];
        lt += ml[w * 32 + 16 + h] * (m == M ? 1.f : ex2(m - M));
      }
      if (lane == 0 && !kCluster) put_lse(h, lt, M);
      const float inv = kCluster ? 1.f : lt == 0.f ? 0.f : p.o_scale / lt;
      float4 acc[2] = {};
#pragma unroll
      for (int c = 0; c < 2; ++c) {                     // chunks 2 lane, 2 lane + 1: dims 8 lane ..
        const int ch = 2 * lane + c;
        for (int w = 0; w < W; ++w) {
          const float4 v = reinterpret_cast<const float4*>(slab0 + w * kSlab + h * 256)[ch ^ (2 * (ch >> 4) + (h & 1))];
          acc[c].x += v.x;
          acc[c].y += v.y;
          acc[c].z += v.z;
          acc[c].w += v.w;
        }
        acc[c].x *= inv;
        acc[c].y *= inv;
        acc[c].z *= inv;
        acc[c].w *= inv;
      }
      if (kCluster) {
        float4* dst = reinterpret_cast<float4*>(part + kPartO + h * 1024) + 2 * lane;
        dst[0] = acc[0];
        dst[1] = acc[1];
        if (lane == 0) {
          *reinterpret_cast<float*>(part + kPartM + 4 * h) = M;
          *reinterpret_cast<float*>(part + kPartL + 4 * h) = lt;
        }
      } else if (p.part_o != nullptr) {
        float4* dst = reinterpret_cast<float4*>(p.part_o + ((row0 + h) * p.splits + un.s) * 256) + 2 * lane;
        dst[0] = acc[0];
        dst[1] = acc[1];
      } else {
        *reinterpret_cast<uint4*>(p.out + un.t * p.o_st + (static_cast<int64_t>(un.g) * p.G + h) * p.o_sh + 8 * lane) =
            make_uint4(pack_bf16x2(acc[0].x, acc[0].y), pack_bf16x2(acc[0].z, acc[0].w),
                       pack_bf16x2(acc[1].x, acc[1].y), pack_bf16x2(acc[1].z, acc[1].w));
      }
    }
    if (kCluster) {                                     // (one unit to a CTA)
      cluster_sync();
      cluster_merge(smem_u32(part), p.splits, p.G, static_cast<int>(cluster_rank()) * W + wi, p.splits * W, lane,
                    [&](int h, float M, float lt, const float4& a, const float4& b) {
                      if (lane == 0) put_lse(h, lt, M);
                      const float inv = lt == 0.f ? 0.f : p.o_scale / lt;
                      *reinterpret_cast<uint4*>(p.out + un.t * p.o_st +
                                                (static_cast<int64_t>(un.g) * p.G + h) * p.o_sh + 8 * lane) =
                          make_uint4(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv),
                                     pack_bf16x2(b.x * inv, b.y * inv), pack_bf16x2(b.z * inv, b.w * inv));
                    });
      cluster_sync();                                   // the other CTAs have read this one's part
      return;
    }
    sync_unit();                                        // slabs and Q are read before the next unit's
  }
}

// ------------------------------------------------------------------ narrow kernel (G <= 8)

// The same with the roles of rows and columns exchanged, for groups of up to
// 8 query heads: heads are the 8 columns of the MMAs and keys (then dims) the
// 16 rows, so that no half of an MMA goes to heads that do not exist.
//   S^T = K Q^T   rows = keys n, n + 8 of a tile of 16, columns = heads; the same
//                 words of K as above, two keys to a fragment
//   O^T += V^T P^T  rows = two dims of a lane's 32, columns = heads.  P^T is
//                 turned from "lane = key" to "lane = head" by movmatrix.
// Half the MMAs and half the accumulators: 12 warps with 168 registers, a unit
// each (W = 1) or W to a unit (16 warps of 128 spilled and were 4 % slower).  Each warp has one buffer for K and one for V: K
// of the next group is asked for once the scores are done, V once the output
// is, which with three warps to a scheduler is long before either is needed.
constexpr int kWarpsN = 12, kThreadsN = 32 * kWarpsN;
constexpr int kQTileN = 8 * 512;
constexpr int N_RING = 0;
constexpr int N_Q = N_RING + kWarpsN * kStageBytes;
constexpr int N_QSC = N_Q + kWarpsN * kQTileN;
constexpr int N_ML = N_QSC + kWarpsN * 8 * 4;       // per warp: mx[8], l[8] (merge)
constexpr int N_SMEM = N_ML + kWarpsN * 16 * 4;
static_assert(N_SMEM <= 232448, "shared memory");
static_assert(kStageBytes >= 8 * 256 * 4, "a warp's buffer holds its output for the merge");

// 8x8 transpose of 16-bit elements: lane 4 r + c holds row r, columns 2c, 2c + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}

template <bool kBlocks, int W, bool kCluster = false>
__global__ void __launch_bounds__(kThreadsN, 1) qsa_attn_f4_narrow_kernel(const __grid_constant__ F4Params fp) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const TcParams& p = fp.t;
  const uint32_t sb = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / W, wi = warp % W;              // the unit slot, this warp's place in it
  const int n = lane >> 2, j = lane & 3;
  const uint32_t st = sb + N_RING + warp * kStageBytes;
  const uint32_t qt = sb + N_Q + grp * kQTileN;
  float* qsc = reinterpret_cast<float*>(sm + N_QSC) + grp * 8;
  auto sync_unit = [&] {
    if (W == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;\n" ::"r"(1 + grp), "n"(32 * W) : "memory");
  };

  for (Walk wk(p, blockIdx.x + gridDim.x * grp, gridDim.x * (kWarpsN / W)); wk.left != 0u; wk.next()) {
    Unit un = wk.unit(p);
    const int32_t* list = p.idx + un.t * p.idx_st + static_cast<int64_t>(un.g) * p.idx_sh;
    const int32_t e_ask = key_entry<kBlocks>(p, list, un, wi * kGroup + lane);
    constexpr int kQ = (8 + W - 1) / W;                 // heads this warp prepares
    uint4 qv[kQ];
#pragma unroll
    for (int h = 0; h < kQ; ++h) qv[h] = q_load(p, un, wi + h * W, lane);
    Walk::cut(p, un);
    const int32_t e_first = wi * kGroup + lane < un.n_eff ? e_ask : -1;
    const int32_t last = kBlocks ? last_visible(p, un.t) : 0x7fffffff;
    const char* kc = fp.codes[0] + un.g * fp.c_sh;
    const char* vc = fp.codes[1] + un.g * fp.c_sh;
    const char* kb = fp.bscale[0] + un.g * fp.b_sh;
    const char* vb = fp.bscale[1] + un.g * fp.b_sh;
    const int groups = un.n_tiles;

    auto entry = [&](int i) { return i < groups ? key_entry<kBlocks>(p, list, un, i * kGroup + lane) : -1; };
    auto resolve = [&](int i, int32_t e) {
      int32_t id = i < groups ? key_slot<kBlocks>(p, un, i * kGroup + lane, e, last) : -1;
      if (id == -2) {
        id = -1;
        if (p.status != nullptr) atomicOr(p.status, static_cast<int32_t>(tc::kStatusOob));
      }
      return id;
    };
    // one commit per call, empty past the last group: K(0), V(0), K(1), V(1), ...
    auto issue_k = [&](int i, int32_t id, uint32_t m) {
      if (i < groups) gather(st, st + kOffKs, kc, kb, fp.c_ss, fp.b_ss, id, m, lane);
      cp_async_commit();
    };
    auto issue_v = [&](int i, int32_t id, uint32_t m) {
      if (i < groups) gather(st + kOffV, st + kOffVs, vc, vb, fp.c_ss, fp.b_ss, id, m, lane);
      cp_async_commit();
    };
    int32_t id = resolve(wi, e_first);
    uint32_t mask = __ballot_sync(0xffffffffu, id >= 0);
    issue_k(wi, id, mask);
    issue_v(wi, id, mask);
    int32_t e_next = entry(wi + W);
    // Q as B fragments: 8 dims (two MMA steps) of head n, lane (n, j), per 512 bytes
    if (groups > 0) {
#pragma unroll
      for (int h = 0; h < kQ; ++h) {
        const int hd = wi + h * W;
        uint32_t o[4];
        const float down = q_scale(qv[h], o);
        if (hd < 8) {
          sts128(qt + 512 * (lane & 7) + (4 * hd + (lane >> 3)) * 16, o[0], o[1], o[2], o[3]);
          if (lane == 0) qsc[hd] = hd < p.G ? p.scale_log2 * down : 0.f;
        }
      }
    }
    sync_unit();

    float o[16][4];
#pragma unroll
    for (int x = 0; x < 16; ++x)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[x][r] = 0.f;
    // heads 2 j and 2 j + 1 of this lane
    float qs[2], mx[2], l[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool live = 2 * j + r < p.G;
      qs[r] = live && groups > 0 ? qsc[2 * j + r] : 0.f;
      mx[r] = live ? -INFINITY : INFINITY;
      l[r] = 0.f;
    }

    for (int i = wi; i < groups; i += W) {
      cp_async_wait<1>();                               // K of this group
      __syncwarp();
      // scores: two tiles of 16 keys; s[t] = {key n: heads 2j, 2j+1; key n + 8: the same}
      float s[2][4];
      uint32_t ksc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        s[t >> 1][2 * (t & 1)] = s[t >> 1][2 * (t & 1) + 1] = 0.f;
        ksc[t] = lds32(st + kOffKs + (8 * t + n) * 16 + 4 * j);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {                  // 32 of the lane's 64 dims
        uint4 kv[4];
        __half2 sc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          kv[t] = lds128(st + (8 * t + n) * 128 + (((2 * j + hf) ^ n) << 4));
          sc[t] = scales2((ksc[t] >> (16 * hf)) & 0xffffu);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {                   // 8 dims: two MMA steps
          const uint4 q = lds128(qt + 512 * (4 * hf + w) + 16 * lane);
#pragma unroll
          for (int t = 0; t < 2; ++t) {                 // 16 keys
            uint32_t b[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
              dequant8(word(kv[2 * t + k], w), w < 2 ? __low2half2(sc[2 * t + k]) : __high2half2(sc[2 * t + k]), b[k]);
            mma_f16(s[t], b[0][0], b[1][0], b[0][1], b[1][1], q.x, q.y);
            mma_f16(s[t], b[0][2], b[1][2], b[0][3], b[1][3], q.z, q.w);
          }
        }
      }
      __syncwarp();                                     // K is read
      const uint32_t cur = mask;
      id = resolve(i + W, e_next);
      mask = __ballot_sync(0xffffffffu, id >= 0);
      e_next = entry(i + 2 * W);
      issue_k(i + W, id, mask);

      float x[2][4];                                    // [t][2 k + r]: key 16 t + 8 k + n, head 2 j + r
      float top = -INFINITY;
      const uint32_t mine = cur >> n;
      const bool full = cur == 0xffffffffu;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[t][r] = fmaf(s[t][r], qs[r & 1], -mx[r & 1]);
          top = fmaxf(top, x[t][r]);
        }
      if (!full) {                                      // some key is masked
        top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[t][r] = (mine >> (16 * t + 8 * (r >> 1))) & 1u ? x[t][r] : -INFINITY;
            top = fmaxf(top, x[t][r]);
          }
      }
      if (__any_sync(0xffffffffu, top > kOver)) {
        float alpha[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float m = -INFINITY;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if ((mine >> (16 * t + 8 * k)) & 1u) m = fmaxf(m, s[t][2 * k + r] * qs[r]);
#pragma unroll
          for (int d = 4; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          const float mn = fmaxf(mx[r], m - kPShift);
          alpha[r] = mx[r] == mn ? 1.f : ex2(mx[r] - mn);
          mx[r] = mn;
          l[r] *= alpha[r];
        }
#pragma unroll
        for (int y = 0; y < 16; ++y)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[y][r] *= alpha[r & 1];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            x[t][r] = (mine >> (16 * t + 8 * (r >> 1))) & 1u
                          ? fmaf(s[t][r], qs[r & 1], -(mx[r & 1] == -INFINITY ? 0.f : mx[r & 1]))
                          : -INFINITY;
      }
      uint32_t pk[2][2];                                // step t: keys 2j, 2j+1 and + 8 of head n
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[t][r] = ex2(x[t][r]);
          l[r & 1] += x[t][r];
        }
        pk[t][0] = transpose8(pack_f16x2(x[t][0], x[t][1]));
        pk[t][1] = transpose8(pack_f16x2(x[t][2], x[t][3]));
      }
      cp_async_wait<1>();                               // V of this group
      __syncwarp();

      // output: two steps of 16 keys
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint4 vw[4];                                    // keys 2j, 2j+1, 2j+8, 2j+9 of the step
        uint32_t vs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r7 = 2 * j + (k & 1);               // row & 7
          const uint32_t row = 16 * u + 8 * (k >> 1) + r7;
          vw[k] = lds128(st + kOffV + row * 128 + ((n ^ r7) << 4));
          vs[k] = lds16(st + kOffVs + row * 16 + 2 * n);
        }
        const __half2 s01a = scales2(__byte_perm(vs[0], vs[1], 0x0040)), s01b = scales2(__byte_perm(vs[0], vs[1], 0x0051));
        const __half2 s23a = scales2(__byte_perm(vs[2], vs[3], 0x0040)), s23b = scales2(__byte_perm(vs[2], vs[3], 0x0051));
#pragma unroll
        for (int w = 0; w < 4; ++w) {                   // dims 8 w .. 8 w + 7 of the lane's 32
          constexpr uint32_t M = 0x0f0f0f0fu;
          const __half2 s01 = w < 2 ? s01a : s01b, s23 = w < 2 ? s23a : s23b;
          const uint32_t v0 = word(vw[0], w), v1 = word(vw[1], w), v2 = word(vw[2], w), v3 = word(vw[3], w);
          uint32_t e01[4], o01[4], e23[4], o23[4];      // even and odd dims, keys (0, 1) and (2, 3)
          dequant8((v0 & M) | ((v1 << 4) & ~M), s01, e01);
          dequant8(((v0 >> 4) & M) | (v1 & ~M), s01, o01);
          dequant8((v2 & M) | ((v3 << 4) & ~M), s23, e23);
          dequant8(((v2 >> 4) & M) | (v3 & ~M), s23, o23);
#pragma unroll
          for (int b = 0; b < 4; ++b) mma_f16(o[4 * w + b], e01[b], o01[b], e23[b], o23[b], pk[u][0], pk[u][1]);
        }
      }
      __syncwarp();                                     // V is read
      issue_v(i + W, id, mask);
    }
    cp_async_wait<0>();

#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
    const int64_t row0 = (un.t * p.Hkv + un.g) * p.G;
    auto put_lse = [&](int h, float lt, float m) {
      const float lv = lt == 0.f ? -INFINITY : (m + lg2(lt)) * 0.69314718055994531f;
      if (p.part_lse != nullptr)
        p.part_lse[(row0 + h) * p.splits + un.s] = lv;
      else if (p.lse != nullptr)
        p.lse[un.t * p.lse_st + static_cast<int64_t>(un.g) * p.G + h] = lv;
    };
    // head 2 j + r: dim 32 n + 2 y in o[y][r], 32 n + 2 y + 1 in o[y][2 + r]
    if (W == 1) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int h = 2 * j + r;
        if (h >= p.G) continue;
        if (n == 0) put_lse(h, l[r], mx[r]);
        const float inv = l[r] == 0.f ? 0.f : p.o_scale / l[r];
        if (p.part_o != nullptr) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + ((row0 + h) * p.splits + un.s) * 256 + 32 * n);
#pragma unroll
          for (int y = 0; y < 8; ++y)
            dst[y] = make_float4(o[2 * y][r] * inv, o[2 * y][2 + r] * inv, o[2 * y + 1][r] * inv,
                                 o[2 * y + 1][2 + r] * inv);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.out + un.t * p.o_st + (static_cast<int64_t>(un.g) * p.G + h) * p.o_sh + 32 * n);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            dst[y] = make_uint4(pack_bf16x2(o[4 * y][r] * inv, o[4 * y][2 + r] * inv),
                                pack_bf16x2(o[4 * y + 1][r] * inv, o[4 * y + 1][2 + r] * inv),
                                pack_bf16x2(o[4 * y + 2][r] * inv, o[4 * y + 2][2 + r] * inv),
                                pack_bf16x2(o[4 * y + 3][r] * inv, o[4 * y + 3][2 + r] * inv));
        }
      }
      __syncwarp();                                     // Q is read before the next unit's
      continue;
    }

    // Merge of W warps, as above
    float* ml = reinterpret_cast<float*>(sm + N_ML) + grp * W * 16;
    if (n == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ml[wi * 16 + 2 * j + r] = mx[r];
        ml[wi * 16 + 8 + 2 * j + r] = l[r];
      }
    }
    sync_unit();
    uint8_t* part = sm + N_Q;                           // (Q is read)
    static_assert(kPartBytes <= kWarpsN * kQTileN, "a chunk's result fits where Q was");
    float* slab0 = reinterpret_cast<float*>(sm + N_RING + grp * W * kStageBytes);
    constexpr int kSlab = kStageBytes / 4;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int h = 2 * j + r;
      float M = -INFINITY;
      for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w * 16 + h]);
      const float f = mx[r] == M ? 1.f : ex2(mx[r] - M);  // a warp without a key: 0
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        // 16-byte chunk (4 dims) 8 n + y of row h, spread over the banks
        float4* dst = reinterpret_cast<float4*>(slab0 + wi * kSlab + h * 256) + (8 * n + (y ^ (4 * (n & 1) + j)));
        *dst = make_float4(o[2 * y][r] * f, o[2 * y][2 + r] * f, o[2 * y + 1][r] * f, o[2 * y + 1][2 + r] * f);
      }
    }
    sync_unit();
    for (int h = wi; h < p.G; h += W) {
      float M = -INFINITY, lt = 0.f;
      for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w * 16 + h]);
      for (int w = 0; w < W; ++w) {
        const float m = ml[w * 16 + h];
        lt += ml[w * 16 + 8 + h] * (m == M ? 1.f : ex2(m - M));
      }
      if (lane == 0 && !kCluster) put_lse(h, lt, M);
      const float inv = kCluster ? 1.f : lt == 0.f ? 0.f : p.o_scale / lt;
      float4 acc[2] = {};
#pragma unroll
      for (int c = 0; c < 2; ++c) {                     // chunks 2 lane, 2 lane + 1: dims 8 lane ..
        const int ch = 2 * lane + c, at = (ch & ~7) + ((ch & 7) ^ (4 * ((ch >> 3) & 1) + (h >> 1)));
        for (int w = 0; w < W; ++w) {
          const float4 v = reinterpret_cast<const float4*>(slab0 + w * kSlab + h * 256)[at];
          acc[c].x += v.x;
          acc[c].y += v.y;
          acc[c].z += v.z;
          acc[c].w += v.w;
        }
        acc[c].x *= inv;
        acc[c].y *= inv;
        acc[c].z *= inv;
        acc[c].w *= inv;
      }
      if (kCluster) {
        float4* dst = reinterpret_cast<float4*>(part + kPartO + h * 1024) + 2 * lane;
        dst[0] = acc[0];
        dst[1] = acc[1];
        if (lane == 0) {
          *reinterpret_cast<float*>(part + kPartM + 4 * h) = M;
          *reinterpret_cast<float*>(part + kPartL + 4 * h) = lt;
        }
      } else if (p.part_o != nullptr) {
        float4* dst = reinterpret_cast<float4*>(p.part_o + ((row0 + h) * p.splits + un.s) * 256) + 2 * lane;
        dst[0] = acc[0];
        dst[1] = acc[1];
      } else {
        *reinterpret_cast<uint4*>(p.out + un.t * p.o_st + (static_cast<int64_t>(un.g) * p.G + h) * p.o_sh + 8 * lane) =
            make_uint4(pack_bf16x2(acc[0].x, acc[0].y), pack_bf16x2(acc[0].z, acc[0].w),
                       pack_bf16x2(acc[1].x, acc[1].y), pack_bf16x2(acc[1].z, acc[1].w));
      }
    }
    if (kCluster) {                                     // (one unit to a CTA)
      cluster_sync();
      cluster_merge(smem_u32(part), p.splits, p.G, static_cast<int>(cluster_rank()) * W + wi, p.splits * W, lane,
                    [&](int h, float M, float lt, const float4& a, const float4& b) {
                      if (lane == 0) put_lse(h, lt, M);
                      const float inv = lt == 0.f ? 0.f : p.o_scale / lt;
                      *reinterpret_cast<uint4*>(p.out + un.t * p.o_st +
                                                (static_cast<int64_t>(un.g) * p.G + h) * p.o_sh + 8 * lane) =
                          make_uint4(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv),
                                     pack_bf16x2(b.x * inv, b.y * inv), pack_bf16x2(b.z * inv, b.w * inv));
                    });
      cluster_sync();                                   // the other CTAs have read this one's part
      return;
    }
    sync_unit();                                        // slabs and Q are read before the next unit's
  }
}

}  // namespace f4
}  // namespace qsa
