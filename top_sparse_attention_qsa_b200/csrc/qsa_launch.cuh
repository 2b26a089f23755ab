// qsa_launch.cuh -- host-side argument checks, parameter set-up and launches
// of the attention kernels, shared by the library's entry points (libqsa.so)
// and its measurement / test-hook library (libqsa_debug.so).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "qsa.h"
#include "qsa_host.cuh"
#include "qsa_prefill_f4.cuh"
#include "qsa_prefill_f8.cuh"
#include "qsa_prefill_mma.cuh"
#include "qsa_prefill_tc.cuh"

namespace qsa {
namespace launch {

using namespace qsa::host;

// Validates `s` and the pointers of a forward call.  Returns QSA_OK or the
// first error found; never touches device memory.
inline qsa_status_t validate(const qsa_shape_t* s, const void* q, const void* k, const void* v,
                             const int32_t* idx, const void* out) {
  if (s == nullptr) return QSA_ERR_NULL;
  if (s->num_tokens < 0 || s->topk < 0 || s->num_slots < 0 || s->num_q_heads <= 0 ||
      s->num_kv_heads <= 0)
    return QSA_ERR_SHAPE;
  if (s->num_q_heads % s->num_kv_heads != 0) return QSA_ERR_SHAPE;
  if (s->head_dim != qsa::kHeadDim) return QSA_ERR_UNSUPPORTED;
  const int G = s->num_q_heads / s->num_kv_heads;
  if (G > 16) return QSA_ERR_UNSUPPORTED;
  if (s->num_kv_heads > 65535 || s->num_tokens > 0x7fffffffLL) return QSA_ERR_UNSUPPORTED;
  if (s->num_tokens == 0) return QSA_OK;
  if (q == nullptr || out == nullptr) return QSA_ERR_NULL;
  const bool reads_cache = s->topk > 0;
  if (reads_cache && (k == nullptr || v == nullptr || idx == nullptr)) return QSA_ERR_NULL;
  // strides: non-negative, rows 16-byte aligned
  const int64_t st[] = {s->q_stride_tok, s->q_stride_head, s->o_stride_tok, s->o_stride_head,
                        s->kv_stride_slot, s->kv_stride_head};
  for (int64_t x : st)
    if (x < 0) return QSA_ERR_SHAPE;
  if (s->idx_stride_tok < 0 || s->idx_stride_head < 0 || s->lse_stride_tok < 0) return QSA_ERR_SHAPE;
  if (reads_cache && s->num_slots > 0 && s->kv_stride_slot == 0) return QSA_ERR_SHAPE;
  for (int64_t x : st)
    if (x % 8 != 0) return QSA_ERR_ALIGN;
  if (!aligned16(q) || !aligned16(out)) return QSA_ERR_ALIGN;
  if (reads_cache && (!aligned16(k) || !aligned16(v))) return QSA_ERR_ALIGN;
  if (reads_cache && (reinterpret_cast<uintptr_t>(idx) & 3u)) return QSA_ERR_ALIGN;
  if (s->num_slots > 0x80000000LL) return QSA_ERR_UNSUPPORTED;  // int32 slot ids
  return QSA_OK;
}

// block_size -> log2 (1, 2, 4, 8, 16), else -1.
inline int block_shift_of(int32_t block_size) {
  for (int b = 0; b <= 4; ++b)
    if (block_size == (1 << b)) return b;
  return -1;
}

template <int NT, bool kDump>
cudaError_t launch_mma(const qsa::PrefillParams& p, cudaStream_t stream) {
  using C = qsa::MmaCfg<NT>;
  static std::atomic<int> done[kMaxDevices];
  auto kernel = qsa::qsa_prefill_mma_kernel<NT, kDump>;
  cudaError_t e = set_smem_once(kernel, C::SMEM, done);
  if (e != cudaSuccess) return e;
  dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>(p.Hkv));
  kernel<<<grid, C::THREADS, C::SMEM, stream>>>(p);
  return cudaGetLastError();
}

// Fills the Q tensor map of the tcgen05 kernels.  Returns false when a TMA
// descriptor cannot express the Q layout or there is nothing to gather.
inline bool make_tc_params(const qsa_shape_t* s, const void* q, qsa::tc::TcParams* tp) {
  using namespace qsa::tc;
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  if (s->topk <= 0 || s->num_slots <= 0 || s->num_slots >= 0x7fffffffLL) return false;
  const cuuint32_t elem_str[3] = {1, 1, 1};
  const uint64_t hq = static_cast<uint64_t>(s->num_q_heads);
  uint64_t st_h = static_cast<uint64_t>(s->q_stride_head) * 2;
  if (hq == 1 || st_h < 512) {
    if (hq > 1) return false;
    st_h = 512;
  }
  uint64_t st_t = static_cast<uint64_t>(s->q_stride_tok) * 2;
  if (s->num_tokens == 1 || st_t < st_h * hq) {
    if (s->num_tokens > 1) return false;
    st_t = st_h * hq;
  }
  const cuuint64_t qdims[3] = {256, hq, static_cast<cuuint64_t>(s->num_tokens)};
  const cuuint64_t qstr[2] = {st_h, st_t};
  const cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(kGp), 1};
  return enc(&tp->tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), qdims, qstr, qbox,
             elem_str, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Every field of the tcgen05 kernels' parameters except the Q tensor map,
// for one unsplit pass over token (shift 0) or microblock lists.
// `score_scale` multiplies the softmax scale (an FP8 cache's k_scale) and
// `o_scale` the normalised output (its v_scale).
inline void fill_tc_params(qsa::tc::TcParams* tp, const qsa_shape_t* s, const void* q, const void* k,
                           const void* v, const int32_t* idx, const int32_t* n_valid, float scale,
                           float score_scale, float o_scale, void* out, float* lse, int32_t* status,
                           int shift, const int32_t* last_slot) {
  const float sc = scale > 0.f ? scale : 0.0625f;  // 1/sqrt(256)
  tp->idx = idx;
  tp->n_valid = n_valid;
  tp->kraw = k;
  tp->vraw = v;
  tp->out = static_cast<__nv_bfloat16*>(out);
  tp->lse = lse;
  tp->status = status;
  tp->gathered = nullptr;
  tp->T = s->num_tokens;
  tp->idx_st = s->idx_stride_tok;
  tp->idx_sh = s->idx_stride_head;
  tp->o_st = s->o_stride_tok;
  tp->o_sh = s->o_stride_head;
  tp->lse_st = s->lse_stride_tok;
  tp->kv_ss = s->kv_stride_slot;
  tp->kv_sh = s->kv_stride_head;
  tp->Hkv = s->num_kv_heads;
  tp->G = s->num_q_heads / s->num_kv_heads;
  tp->K = s->topk;
  tp->S = static_cast<int32_t>(s->num_slots);
  tp->scale_log2 = sc * score_scale * 1.4426950408889634f;
  tp->o_scale = o_scale;
  tp->splits = 1;
  tp->chunk = s->topk << shift;
  tp->part_o = nullptr;
  tp->part_lse = nullptr;
  tp->block_shift = shift;
  tp->last_slot = last_slot;
  tp->q_ptr = q;
  tp->q_st = s->q_stride_tok;
  tp->q_sh = s->q_stride_head;
}

// Persistent grid: one CTA per SM, or one per unit when there are fewer.
inline cudaError_t persistent_grid(const qsa::tc::TcParams& tp, unsigned* grid) {
  const int64_t units = tp.T * tp.Hkv * tp.splits;
  const int nsm = sm_count();
  if (nsm <= 0) return cudaErrorInvalidDevice;
  *grid = static_cast<unsigned>(units < nsm ? units : nsm);
  return cudaSuccess;
}

// The attention kernels rebalance registers between their warpgroups with
// setmaxnreg, which draws on the registers the block was launched with: a
// split larger than that would make a warpgroup wait for registers forever.
// Checked once per kernel against the compiled launch register count;
// `need` = 128 x the sum over the warpgroups of their registers per thread.
template <typename Kernel>
cudaError_t check_register_split(Kernel kernel, int threads, long need, std::atomic<int>* done) {
  if (done->load(std::memory_order_acquire)) return cudaSuccess;
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  if (static_cast<long>(attr.numRegs) * threads < need) return cudaErrorInvalidConfiguration;
  done->store(1, std::memory_order_release);
  return cudaSuccess;
}

template <bool kDump, bool kStall = false, bool kBlocks = false>
cudaError_t launch_tc(const qsa::tc::TcParams& tp, cudaStream_t stream) {
  static std::atomic<int> done[kMaxDevices];
  static std::atomic<int> regs_ok;
  auto kernel = qsa::tc::qsa_prefill_tc_kernel<kDump, kStall, kBlocks>;
  using namespace qsa::tc;
  cudaError_t e = check_register_split(
      kernel, kThreads, 128L * (kRegsSoftmax + long(kProducerGroups) * kRegsProducer + kRegsMma), &regs_ok);
  if (e != cudaSuccess) return e;
  e = set_smem_once(kernel, qsa::tc::SMEM_BYTES, done);
  if (e != cudaSuccess) return e;
  unsigned grid = 0;
  if ((e = persistent_grid(tp, &grid)) != cudaSuccess) return e;
  kernel<<<grid, qsa::tc::kThreads, qsa::tc::SMEM_BYTES, stream>>>(tp);
  return cudaGetLastError();
}

template <bool kBlocks, bool kDump = false>
cudaError_t launch_f8(const qsa::tc::TcParams& tp, cudaStream_t stream) {
  static std::atomic<int> done[kMaxDevices];
  static std::atomic<int> regs_ok;
  auto kernel = qsa::f8::qsa_prefill_f8_kernel<kBlocks, kDump>;
  using namespace qsa::f8;
  cudaError_t e = check_register_split(kernel, kThreads8,
                                       128L * (kRegsProd8 + kRegsMisc8 + 2L * kRegsSm8 + kRegsEpi8), &regs_ok);
  if (e != cudaSuccess) return e;
  e = set_smem_once(kernel, qsa::f8::F_SMEM, done);
  if (e != cudaSuccess) return e;
  unsigned grid = 0;
  if ((e = persistent_grid(tp, &grid)) != cudaSuccess) return e;
  kernel<<<grid, qsa::f8::kThreads8, qsa::f8::F_SMEM, stream>>>(tp);
  return cudaGetLastError();
}

template <typename Kernel>
cudaError_t launch_f4_kernel(Kernel kernel, int threads, int smem, std::atomic<int>* done, const qsa::f4::F4Params& fp,
                             int64_t units, cudaStream_t stream) {
  const cudaError_t e = set_smem_once(kernel, smem, done);
  if (e != cudaSuccess) return e;
  const int nsm = sm_count();
  if (nsm <= 0) return cudaErrorInvalidDevice;
  kernel<<<static_cast<unsigned>(units < nsm ? units : nsm), threads, smem, stream>>>(fp);
  return cudaGetLastError();
}

template <bool kBlocks, int W>
cudaError_t launch_f4_with(const qsa::f4::F4Params& fp, int64_t units, cudaStream_t stream) {
  using namespace qsa::f4;
  static std::atomic<int> done[2][kMaxDevices];
  if (fp.t.G <= 8)   // (12 warps: all of them where the wide kernel has its 8)
    return launch_f4_kernel(qsa_attn_f4_narrow_kernel<kBlocks, W == 8 ? kWarpsN : W>, kThreadsN, N_SMEM, done[1], fp,
                            units, stream);
  return launch_f4_kernel(qsa_attn_f4_kernel<kBlocks, W>, kThreads4, H_SMEM, done[0], fp, units, stream);
}

// Warps per unit: the count with the least time by a model fitted to all four
// counts over 1 to 2368 units of 1 to 64 groups of 32 keys.  In units of the
// time a group takes with every warp of the SM at work, a unit costs its
// slowest warp's groups and `fixed` (Q, output, merge); with at most 4 warps of
// an SM at work, one to a scheduler, all of it takes `alone` of that, and more
// in proportion up to all of them.  Units run in rounds over the SMs' slots, the
// last one as full as it is.  Measured, us (148 units, heads (24,2)): one group
// 7.5, 7.8, 6.4, 7.1 with 1, 2, 4, 8 warps to a unit; two groups 9.0, 7.8, 6.5,
// 7.1; 64 groups 101, 55, 31.5, 26.7; 1184 units of 64 groups 155, 166, 178, 195.
template <bool kBlocks>
cudaError_t launch_f4(const qsa::f4::F4Params& fp, cudaStream_t stream) {
  const int64_t units = fp.t.T * fp.t.Hkv * fp.t.splits;
  const int nsm = sm_count();
  if (nsm <= 0) return cudaErrorInvalidDevice;
  const bool narrow = fp.t.G <= 8;
  const int warps = narrow ? qsa::f4::kWarpsN : qsa::f4::kWarps4;
  static constexpr double kFixed[2][4] = {{3.1, 2.5, 2.0, 1.7}, {2.0, 2.1, 1.5, 0.9}};
  const double alone = narrow ? 0.55 : 0.7;
  const int64_t groups = (fp.t.chunk + qsa::f4::kGroup - 1) / qsa::f4::kGroup;
  int best = 1;
  double best_cost = 0.;
  for (int i = 0; i < 4; ++i) {
    const int w = i == 3 ? warps : 1 << i;
    const int64_t slots = static_cast<int64_t>(nsm) * (warps / w), rest = units % slots;
    const int64_t busy = (rest + nsm - 1) / nsm * w;    // warps at work on an SM in the last round
    const double last = rest == 0 ? 0. : busy <= 4 ? alone : alone + (1. - alone) * (busy - 4) / (warps - 4);
    const double cost = (static_cast<double>(units / slots) + last) *
                        (kFixed[narrow][i] + static_cast<double>((groups + w - 1) / w));
    if (i == 0 || cost < best_cost) {
      best = 1 << i;
      best_cost = cost;
    }
  }
  switch (best) {
    case 1: return launch_f4_with<kBlocks, 1>(fp, units, stream);
    case 2: return launch_f4_with<kBlocks, 2>(fp, units, stream);
    case 4: return launch_f4_with<kBlocks, 4>(fp, units, stream);
    default: return launch_f4_with<kBlocks, 8>(fp, units, stream);
  }
}

// The cluster form of a decode (qsa_prefill_f4.cuh): a CTA per chunk, the
// chunks of a list one cluster.
template <typename Kernel>
cudaError_t f4_cluster_config(Kernel kernel, int threads, int smem, std::atomic<int>* done, int64_t units, int chunks,
                              cudaLaunchConfig_t* cfg, cudaLaunchAttribute* at, cudaStream_t stream) {
  const cudaError_t e = set_smem_once(kernel, smem, done);
  if (e != cudaSuccess) return e;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = chunks;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  cfg->gridDim = dim3(static_cast<unsigned>(units));
  cfg->blockDim = dim3(threads);
  cfg->dynamicSmemBytes = smem;
  cfg->stream = stream;
  cfg->attrs = at;
  cfg->numAttrs = 1;
  return cudaSuccess;
}

constexpr int kMaxCluster = 8;

// Calls f(kernel, threads, shared memory, once-flags) with the kernel for groups of G heads.
template <typename F>
auto with_f4_cluster_kernel(int G, F f) {
  using namespace qsa::f4;
  static std::atomic<int> done[2][kMaxDevices];
  return G <= 8 ? f(qsa_attn_f4_narrow_kernel<false, kWarpsN, true>, kThreadsN, N_SMEM, done[1])
                : f(qsa_attn_f4_kernel<false, kWarps4, true>, kThreads4, H_SMEM, done[0]);
}

// Whether `lists` lists of `chunks` chunks run as clusters that are all
// resident at once (a second wave would cost more than the merge launch).
inline bool f4_cluster_fits(int G, int64_t lists, int chunks) {
  static std::atomic<int> most[2][kMaxCluster + 1][kMaxDevices];   // clusters resident at once, + 1
  int dev = 0;
  if (chunks < 2 || chunks > kMaxCluster || lists * chunks > sm_count()) return false;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  std::atomic<int>& slot = most[G <= 8 ? 1 : 0][chunks][dev];
  int n = slot.load(std::memory_order_relaxed);
  if (n == 0) {
    n = with_f4_cluster_kernel(G, [&](auto kernel, int threads, int smem, std::atomic<int>* done) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute at = {};
      int k = 0;
      if (f4_cluster_config(kernel, threads, smem, done, chunks, chunks, &cfg, &at, nullptr) != cudaSuccess ||
          cudaOccupancyMaxActiveClusters(&k, kernel, &cfg) != cudaSuccess)
        return 1;
      return k + 1;
    });
    slot.store(n, std::memory_order_relaxed);
  }
  return lists <= n - 1;
}

inline cudaError_t launch_f4_cluster(const qsa::f4::F4Params& fp, cudaStream_t stream) {
  return with_f4_cluster_kernel(fp.t.G, [&](auto kernel, int threads, int smem, std::atomic<int>* done) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at = {};
    const cudaError_t e = f4_cluster_config(kernel, threads, smem, done, fp.t.T * fp.t.Hkv * fp.t.splits, fp.t.splits,
                                            &cfg, &at, stream);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kernel, fp);
  });
}

}  // namespace launch
}  // namespace qsa
