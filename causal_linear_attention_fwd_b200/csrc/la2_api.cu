// la2_api.cu -- the C ABI of libla2 (see include/la2.h): argument checks,
// chunk planning, workspace carving, kernel dispatch, device error word and
// per-kernel event timing.  The whole library is this one translation unit.
#include <cuda_runtime.h>

#include <atomic>
#include <initializer_list>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <type_traits>
#include <vector>

#include "../../include/la2.h"
#include "la2_common.cuh"
#include "la2_decode.cuh"
#include "la2_dlam_tc.cuh"
#include "la2_fmap.cuh"
#include "la2_memo.h"
#include "la2_norm.cuh"
#include "la2_norm_plan.h"
#include "la2_pool.cuh"
#include "la2_rotary.cuh"
#include "la2_shard.cuh"
#include "la2_simt.cuh"
#include "la2_tc.cuh"

namespace {

using la2::Geo;

std::atomic<int> g_opt_split{0};
std::atomic<int> g_opt_path{0};
std::atomic<int> g_opt_inject{0};
std::atomic<int> g_opt_variant{0};
std::atomic<int> g_opt_trace{0};
std::atomic<int> g_opt_varlen_order{0};
std::atomic<int> g_opt_decode_block{0};
std::atomic<int> g_opt_bwd_form{0};

// ------------------------------------------------------------ profiling
enum KernelId {
  K_SIMT_FWD_STATE, K_SIMT_FWD_SCAN, K_SIMT_FWD, K_SIMT_DQ, K_SIMT_REV_STATE,
  K_SIMT_REV_SCAN, K_SIMT_DKDV, K_DECODE, K_TC_FWD_STATE, K_TC_FWD, K_TC_DQ,
  K_TC_REV_STATE, K_TC_DV, K_TC_DK, K_SCAN_FWD, K_SCAN_REV, K_SIMT_DLAMBDA,
  K_SIMT_DLAMBDA_STATE, K_SIMT_DLAMBDA_SCAN, K_TC_DECODE_UNITS, K_FMAP, K_FMAP_GRAD, K_TC_DKDV,
  K_TC_DLAMBDA, K_TC_DLAMBDA_STATE, K_STATE_PAD, K_ROTARY, K_ROTARY_GRAD, K_GATED_NORM,
  K_GATED_NORM_GRAD, K_RESIDUAL_NORM, K_RESIDUAL_NORM_GRAD, K_NORM_WEIGHT_SUM, K_POOL_COPY, K_COUNT
};
const char *kKernelName[K_COUNT] = {
    "simt_fwd_chunk_state", "simt_scan_fwd", "simt_fwd", "simt_dq",
    "simt_rev_chunk_state", "simt_scan_rev", "simt_dkdv", "decode_step",
    "tc_fwd_chunk_state", "tc_fwd", "tc_dq", "tc_rev_chunk_state", "tc_dv", "tc_dk",
    "scan_fwd", "scan_rev", "simt_dlambda", "simt_dlambda_chunk_state", "simt_dlambda_scan",
    "tc_decode_units", "feature_map", "feature_map_grad", "tc_dkdv", "tc_dlambda",
    "tc_dlambda_chunk_state", "state_pad", "rotary", "rotary_grad", "gated_norm",
    "gated_norm_grad", "residual_norm", "residual_norm_grad", "norm_weight_sum", "pool_copy"};

struct ProfRec {
  int kid;
  cudaEvent_t a, b;
};
std::mutex g_prof_mu;
std::atomic<int> g_prof_on{0};
std::vector<ProfRec> g_prof;
std::vector<cudaEvent_t> g_ev_pool;
constexpr size_t kMaxProfRecs = 1 << 16;

cudaEvent_t ev_get() {
  if (!g_ev_pool.empty()) {
    cudaEvent_t e = g_ev_pool.back();
    g_ev_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
  return e;
}

// Runs `launch` (which enqueues one kernel on `st`) and, while profiling is
// on, brackets it with events.  Returns the launch error, if any.
// Runs a launch callable: one that returns void (the launch's error is
// then the runtime's last error) or its own cudaError_t.
template <typename F>
cudaError_t run_launch(F &&launch) {
  if constexpr (std::is_same_v<decltype(launch()), cudaError_t>) {
    const cudaError_t e = launch();
    const cudaError_t last = cudaGetLastError();
    return e != cudaSuccess ? e : last;
  } else {
    launch();
    return cudaGetLastError();
  }
}

template <typename F>
cudaError_t timed(int kid, cudaStream_t st, F &&launch) {
  if (!g_prof_on.load(std::memory_order_relaxed)) return run_launch(launch);
  std::lock_guard<std::mutex> lk(g_prof_mu);
  cudaEvent_t a = nullptr, b = nullptr;
  if (g_prof.size() < kMaxProfRecs) {
    a = ev_get();
    b = ev_get();
  }
  if (a) cudaEventRecord(a, st);
  cudaError_t err = run_launch(launch);
  if (a && b) {
    cudaEventRecord(b, st);
    g_prof.push_back({kid, a, b});
  }
  return err;
}

// ------------------------------------------------------------- helpers
int device_sms() {
  static std::atomic<int> known[64];  // by device; 0: not asked yet
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  if (dev < 64 && n > 0) known[dev].store(n, std::memory_order_relaxed);
  return n > 0 ? n : 148;
}

int device_cc() {
  int dev = 0, ma = 0, mi = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  cudaDeviceGetAttribute(&ma, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&mi, cudaDevAttrComputeCapabilityMinor, dev);
  return ma * 10 + mi;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
  const void *p;
  size_t n;
};
bool overlaps(Span x, Span y) {
  if (!x.p || !y.p || x.n == 0 || y.n == 0) return false;
  uintptr_t a0 = reinterpret_cast<uintptr_t>(x.p), a1 = a0 + x.n;
  uintptr_t b0 = reinterpret_cast<uintptr_t>(y.p), b1 = b0 + y.n;
  return a0 < b1 && b0 < a1;
}
// An output sharing any byte with an input (an exact alias included) or
// with another output.
bool any_overlap(const std::vector<Span> &outs, const std::vector<Span> &ins) {
  for (size_t i = 0; i < outs.size(); i++) {
    for (size_t j = 0; j < ins.size(); j++)
      if (overlaps(outs[i], ins[j])) return true;
    for (size_t j = i + 1; j < outs.size(); j++)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}

bool shape_supported(int d, int e, la2_dtype dt) {
  return (d == 64 || d == 128) && (e == 64 || e == 128) &&
         (dt == LA2_F32 || dt == LA2_BF16);
}

size_t esize(la2_dtype dt) { return dt == LA2_F32 ? 4 : 2; }

// Which kernel family serves a call.  any_head: the entry point runs the
// tensor-core passes for head sizes 64 too (its 64-column tensors read with
// zero columns beyond their width, its states padded to 128 x 128 in
// workspace scratch); else bf16 with d = e = 128 only.
enum Path { PATH_SIMT = 0, PATH_TC = 1, PATH_NONE = 2 };
Path choose_path(int d, int e, la2_dtype dt, bool any_head = false) {
  const int opt = g_opt_path.load();
  const bool shape_ok = la2::tc::supports(d, e, dt == LA2_BF16) ||
                        (any_head && dt == LA2_BF16 && shape_supported(d, e, dt));
  const bool tc_ok = shape_ok && device_cc() == 100;
  if (opt == 1) return PATH_SIMT;
  if (opt == 2) return tc_ok ? PATH_TC : PATH_NONE;
  return tc_ok ? PATH_TC : PATH_SIMT;
}

// Chunk plan: split each (b,h) sequence into S chunks of Lc rows (Lc a
// multiple of the block size `blk`) so that B*H*S CTAs fill the GPU.
// slots: how many chunks the GPU runs at once (0: one per SM; the paired
// reverse pass runs one per two SMs).
Geo plan(int B, int H, int64_t L, int blk, Path path, int slots = 0) {
  Geo g;
  g.cu = nullptr;
  g.lpt = 0;
  g.slots = nullptr;
  g.pool = 0;
  g.inject = 0;
  g.variant = g_opt_variant.load();
  g.trace = g_opt_trace.load() - 1;
  g.B = B;
  g.H = H;
  g.L = L;
  const int64_t nblk = (L + blk - 1) / blk;
  int64_t S = g_opt_split.load();
  if (S <= 0) {
    const int64_t BH = (int64_t)B * H;
    const int sms = device_sms();
    S = path == PATH_TC ? la2::tc::auto_split(BH, nblk, slots > 0 ? slots : sms)
                        : (BH >= 2 * sms ? 1 : (2 * sms + BH - 1) / BH);
  }
  if (S > nblk) S = nblk;
  if (S < 1) S = 1;
  const int64_t per = (nblk + S - 1) / S;
  g.Lc = per * blk;
  g.S = (int)((L + g.Lc - 1) / g.Lc);
  if (g.S < 1) g.S = 1;
  // Sub-chunks for the tensor-core chunk-state pre-passes: those passes
  // have B*H*(S-1) chunks, fewer than the SMs when the split exists at all,
  // so each chunk is cut into M sub-chunks, M minimising (waves of CTAs) x
  // (blocks per CTA).  Lc becomes M * Ls with Ls a multiple of the block.
  int64_t M = 1;
  if (path == PATH_TC && g.S > 1) {
    const int sms = device_sms();
    const int64_t work = (int64_t)B * H * (g.S - 1);
    int64_t best = -1;
    for (int64_t m = 1; m <= 8 && m <= per; m++) {
      const int64_t cost = ((work * m + sms - 1) / sms) * ((per + m - 1) / m);
      if (best < 0 || cost < best) {
        best = cost;
        M = m;
      }
    }
    g.Lc = M * (((per + M - 1) / M) * blk);
    g.S = (int)((L + g.Lc - 1) / g.Lc);
    if (g.S <= 1) {
      g.S = 1;
      M = 1;
    }
  }
  g.M = (int)M;
  g.Ls = g.Lc / M;
  g.Ssub = (int)((L + g.Ls - 1) / g.Ls);
  g.wsS = g.Ssub;
  g.nst = g.S - 1;
  g.c0 = 0;
  return g;
}

int block_rows(Path p) { return p == PATH_TC ? la2::tc::BLOCK : la2::simt::C; }

// Whether the tensor-core backward runs dV and dK as one paired launch (two
// CTAs per chunk in clusters of two) rather than as two passes: yes unless
// LA2_OPT_BWD_FORM = 1 or the phase-serial kernel form is forced.
bool rev_paired(Path p) {
  return p == PATH_TC && g_opt_bwd_form.load() != 1 && g_opt_variant.load() != 1;
}

// Chunk plan of the backward's reverse passes.  Paired, each chunk occupies
// two SMs, so the automatic split aims at SMs / 2 chunks at a time: fewer
// chunks per sequence than the forward scan's plan, and so fewer chunk
// boundaries for the reverse chunk-state pre-pass to cover.  A forced split
// (LA2_OPT_SPLIT) applies to both plans alike.
Geo plan_rev(int B, int H, int64_t L, Path p) {
  if (!rev_paired(p)) return plan(B, H, L, block_rows(p), p);
  Geo g = plan(B, H, L, block_rows(p), p, device_sms() / 2);
  g.rev_pair = 1;
  return g;
}

// Chunk plan of the decay gradient (blocks of blk rows: 32 for the fp32-FMA
// kernel, one CTA per chunk; 128 for the tensor-core one, two CTAs per chunk,
// one per half of the e columns): at most one wave, S = floor(slots / (B*H))
// chunks per sequence when B*H is below the slots -- the SMs, or half of them
// for the tensor-core kernel (LA2_OPT_SPLIT overrides) -- Lc a multiple of
// the block.  (Counting a tensor-core chunk as one slot would split B*H = 64
// sequences in two on 148 SMs: 256 CTAs, two waves as long as the one wave of
// 128 unsplit, plus the pre-pass and the scan.)
// The chunk-state pre-pass covers chunks 0..S-2 only, so it runs on M
// sub-chunks of Ls rows per chunk (Lc = M Ls), M filling the slots (at most
// 8); the workspace holds (S-1) M + 1 (KV, W) pairs per (b,h).
Geo plan_dlambda(int B, int H, int64_t L, bool split_ok, int blk_rows) {
  Geo g = plan(B, H, L, blk_rows, PATH_SIMT);
  const int64_t blk = blk_rows, nblk = (L + blk - 1) / blk;
  const int64_t BH = (int64_t)B * H;
  const int slots = blk_rows == la2::tc::BLOCK ? device_sms() / 2 : device_sms();
  int64_t S = g_opt_split.load();
  if (S <= 0) S = BH >= slots ? 1 : slots / BH;
  if (!split_ok || S > nblk) S = split_ok ? nblk : 1;
  if (S < 1) S = 1;
  int64_t per = (nblk + S - 1) / S;  // blocks per chunk
  S = (nblk + per - 1) / per;
  int64_t M = 1;
  if (S > 1) {
    // the largest M <= min(8, slots / (B*H*(S-1))) whose whole sub-chunks
    // keep S chunks
    int64_t want = slots / (BH * (S - 1));
    if (want > 8) want = 8;
    for (int64_t m = want; m > 1; m--) {
      const int64_t p = ((per + m - 1) / m) * m;
      if ((nblk + p - 1) / p == S) {
        M = m;
        per = p;
        break;
      }
    }
  }
  g.S = (int)S;
  g.Lc = per * blk;
  g.M = (int)M;
  g.Ls = g.Lc / M;
  g.nst = (int)((S - 1) * M);
  g.wsS = g.nst + 1;
  g.Ssub = g.wsS;
  return g;
}

// Workspace of a backward: the forward scan's chunk states (plan g) then
// the reverse scan's (plan gr).
size_t ws_bwd_bytes(const Geo &g, const Geo &gr, int d, int e) {
  auto one = [&](const Geo &x) {
    return x.S > 1 ? (size_t)x.B * x.H * x.wsS * d * e * sizeof(float) : (size_t)0;
  };
  return one(g) + one(gr);
}

// A tensor-core call with a 64-column head size keeps its initial and final
// states padded to 128 x 128 fp32 in scratch after the chunk states: n
// states per (b,h).
bool padded(Path p, int d, int e) { return p == PATH_TC && (d != 128 || e != 128); }
size_t pad_bytes(const Geo &g, int n) { return (size_t)g.B * g.H * 128 * 128 * sizeof(float) * n; }

size_t ws_bytes(int op, const Geo &g, int d, int e) {
  if (op == LA2_OP_DLAMBDA)  // (KV, W) per sub-chunk boundary
    return g.S > 1 ? (size_t)g.B * g.H * g.wsS * 2 * d * e * sizeof(float) : 0;
  if (op == LA2_OP_SHARD_STATE)  // one delta per sub-chunk plus one spare slot
    return (size_t)g.B * g.H * (g.Ssub + 1) * d * e * sizeof(float);
  if (g.S <= 1) return 0;
  size_t one = (size_t)g.B * g.H * g.wsS * d * e * sizeof(float);
  return op == LA2_OP_BACKWARD ? 2 * one : one;
}

// ------------------------------------------------------ SIMT dispatch
// A kernel's dynamic shared memory above the default 48 KB needs an opt-in
// attribute; its failure is returned rather than left to the launch.
template <typename K>
cudaError_t opt_in_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int D, int E>
cudaError_t simt_forward(const void *q, const void *k, const void *v,
                         const float *lam, const float *kv0, void *o,
                         float *kv_out, float *ws, const Geo &g, cudaStream_t st) {
  using namespace la2::simt;
  const T *Q = (const T *)q, *K = (const T *)k, *V = (const T *)v;
  cudaError_t err = cudaSuccess;
  const int64_t BH = (int64_t)g.B * g.H;
  if (g.S > 1) {
    auto kst = fwd_kernel<T, D, E, false>;
    if (cudaError_t e = opt_in_smem(kst, fwd_smem<D, E>())) return e;
    err = timed(K_SIMT_FWD_STATE, st, [&] {
      kst<<<(unsigned)(BH * (g.S - 1)), NT, fwd_smem<D, E>(), st>>>(
          Q, K, V, lam, nullptr, nullptr, nullptr, ws, la2::state_geo(g, false));
    });
    if (err) return err;
    err = timed(K_SIMT_FWD_SCAN, st, [&] {
      scan_fwd_kernel<D, E><<<dim3((D * E + NT - 1) / NT, (unsigned)BH), NT, 0, st>>>(
          ws, kv0, lam, la2::state_geo(g, false));
    });
    if (err) return err;
  }
  auto kf = fwd_kernel<T, D, E, true>;
  if (cudaError_t e = opt_in_smem(kf, fwd_smem<D, E>())) return e;
  return timed(K_SIMT_FWD, st, [&] {
    kf<<<(unsigned)(BH * g.S), NT, fwd_smem<D, E>(), st>>>(Q, K, V, lam, kv0, (T *)o, kv_out, ws, g);
  });
}

template <typename T, int D, int E>
cudaError_t simt_backward(const void *q, const void *k, const void *v,
                          const float *lam, const float *kv0, const void *dO,
                          void *dq, void *dk, void *dv, float *dkv0, float *ws,
                          const Geo &g, bool reuse_fwd, cudaStream_t st,
                          const float *dend = nullptr) {
  using namespace la2::simt;
  const T *Q = (const T *)q, *K = (const T *)k, *V = (const T *)v, *G = (const T *)dO;
  const int64_t BH = (int64_t)g.B * g.H;
  float *wsf = ws;
  float *wsr = ws ? ws + (size_t)BH * g.wsS * D * E : nullptr;
  cudaError_t err = cudaSuccess;
  if (g.S > 1 && !reuse_fwd) {
    auto kst = fwd_kernel<T, D, E, false>;
    if (cudaError_t e = opt_in_smem(kst, fwd_smem<D, E>())) return e;
    err = timed(K_SIMT_FWD_STATE, st, [&] {
      kst<<<(unsigned)(BH * (g.S - 1)), NT, fwd_smem<D, E>(), st>>>(
          Q, K, V, lam, nullptr, nullptr, nullptr, wsf, la2::state_geo(g, false));
    });
    if (err) return err;
    err = timed(K_SIMT_FWD_SCAN, st, [&] {
      scan_fwd_kernel<D, E><<<dim3((D * E + NT - 1) / NT, (unsigned)BH), NT, 0, st>>>(
          wsf, kv0, lam, la2::state_geo(g, false));
    });
    if (err) return err;
  }
  if (g.S > 1) {
    auto krs = rev_state_kernel<T, D, E>;
    if (cudaError_t e = opt_in_smem(krs, rev_smem<D, E>())) return e;
    err = timed(K_SIMT_REV_STATE, st, [&] {
      krs<<<(unsigned)(BH * (g.S - 1)), NT, rev_smem<D, E>(), st>>>(Q, G, lam, wsr,
                                                                    la2::state_geo(g, true));
    });
    if (err) return err;
    err = timed(K_SIMT_REV_SCAN, st, [&] {
      scan_rev_kernel<D, E><<<dim3((D * E + NT - 1) / NT, (unsigned)BH), NT, 0, st>>>(
          wsr, lam, dend, la2::state_geo(g, true));
    });
    if (err) return err;
  }
  auto kq = dq_kernel<T, D, E>;
  if (cudaError_t e = opt_in_smem(kq, dq_smem<D, E>())) return e;
  err = timed(K_SIMT_DQ, st, [&] {
    kq<<<(unsigned)(BH * g.S), NT, dq_smem<D, E>(), st>>>(K, V, G, lam, kv0, (T *)dq, wsf, g);
  });
  if (err) return err;
  auto kk = dkdv_kernel<T, D, E>;
  if (cudaError_t e = opt_in_smem(kk, dkdv_smem<D, E>())) return e;
  return timed(K_SIMT_DKDV, st, [&] {
    kk<<<(unsigned)(BH * g.S), NT, dkdv_smem<D, E>(), st>>>(Q, K, V, G, lam, (T *)dk, (T *)dv,
                                                           dkv0, wsr, dend, g);
  });
}

template <typename T, int D, int E>
cudaError_t decode(const void *q, const void *k, const void *v, const float *lam,
                   float *pool, const int *slots, int pool_size, void *o, int B, int H,
                   int ntok, cudaStream_t st) {
  if (ntok == 1)
    return timed(K_DECODE, st, [&] {
      la2::dec::decode_kernel<T, D, E, 1><<<(unsigned)((int64_t)B * H), la2::dec::NT, 0, st>>>(
          (const T *)q, (const T *)k, (const T *)v, lam, pool, slots, pool_size, (T *)o, H, ntok);
    });
  auto kern = la2::dec::tokens_kernel<T, D, E, 4>;
  constexpr size_t smem = la2::dec::tokens_smem<E, 4>();
  if (cudaError_t e = opt_in_smem(kern, smem)) return e;
  return timed(K_DECODE, st, [&] {
    kern<<<(unsigned)((int64_t)B * H), la2::dec::NTT, smem, st>>>(
        (const T *)q, (const T *)k, (const T *)v, lam, pool, slots, pool_size, (T *)o, H, ntok);
  });
}

#define LA2_DISPATCH_DE(d, e, FN, T, ...)                                   \
  ((d) == 64 && (e) == 64     ? FN<T, 64, 64>(__VA_ARGS__)                  \
   : (d) == 64 && (e) == 128  ? FN<T, 64, 128>(__VA_ARGS__)                 \
   : (d) == 128 && (e) == 64  ? FN<T, 128, 64>(__VA_ARGS__)                 \
                              : FN<T, 128, 128>(__VA_ARGS__))

la2_status to_status(cudaError_t e) { return e == cudaSuccess ? LA2_OK : LA2_ERR_CUDA; }

}  // namespace

// Tokens per request from which la2_decode_tokens runs the tensor-core
// block form (one block of the chunk schedule per request) instead of the
// token-by-token register update.  Measured on B200 at batch 256 x 64 heads:
// the decode-unit kernel takes ~0.93 ms per call for any T <= 128 (148 CTAs,
// ~110 units each, set by each unit's state round trip), the token kernel
// 0.40 ms at T = 4, 0.50 at 8, 0.89 at 16 and 1.18 at 24 (~0.05 ms a token).
constexpr int kDecodeBlockTokens = 17;

// ------------------------------------------------------- d lambda helper
// dlam = 0; split: chunk-state pre-pass over the sub-chunks of chunks
// 0..S-2, the scan of the (KV, W) pairs, then the gradient pass over every
// chunk.
template <typename T, int D, int E>
cudaError_t simt_dlambda(const void *q, const void *k, const void *v, const void *dO,
                         const float *lam, const float *kv0, float *dlam, float *ws,
                         const Geo &g, cudaStream_t st) {
  using namespace la2::simt;
  auto kd = dlambda_kernel<T, D, E, false>;
  auto ks = dlambda_kernel<T, D, E, true>;
  cudaError_t e = cudaFuncSetAttribute(kd, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)dlam_smem<T, D, E>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(ks, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dlam_smem<T, D, E>());
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(dlam, 0, (size_t)g.H * sizeof(float), st);
  if (e != cudaSuccess) return e;
  const int64_t BH = (int64_t)g.B * g.H;
  const T *Q = (const T *)q, *K = (const T *)k, *V = (const T *)v, *G = (const T *)dO;
  if (g.S > 1) {
    e = timed(K_SIMT_DLAMBDA_STATE, st, [&] {
      ks<<<(unsigned)(BH * g.nst), NT, dlam_smem<T, D, E>(), st>>>(Q, K, V, G, lam, nullptr, ws,
                                                                  nullptr, g);
    });
    if (e != cudaSuccess) return e;
    e = timed(K_SIMT_DLAMBDA_SCAN, st, [&] {
      dlam_scan_kernel<D, E><<<dim3(D * E / NT, (unsigned)BH), NT, 0, st>>>(ws, kv0, lam, g);
    });
    if (e != cudaSuccess) return e;
  }
  return timed(K_SIMT_DLAMBDA, st, [&] {
    kd<<<(unsigned)(BH * g.S), NT, dlam_smem<T, D, E>(), st>>>(Q, K, V, G, lam, kv0, ws, dlam, g);
  });
}

// ------------------------------------------------------- shard helpers
template <typename T, int D, int E>
cudaError_t simt_shard_state(const void *a, const void *b, const float *lam, float *ws,
                             const Geo &gs, bool reverse, cudaStream_t st) {
  using namespace la2::simt;
  const int64_t BH = (int64_t)gs.B * gs.H;
  if (!reverse) {
    auto kst = fwd_kernel<T, D, E, false>;
    if (cudaError_t e = opt_in_smem(kst, fwd_smem<D, E>())) return e;
    return timed(K_SIMT_FWD_STATE, st, [&] {
      kst<<<(unsigned)(BH * gs.nst), NT, fwd_smem<D, E>(), st>>>(
          nullptr, (const T *)a, (const T *)b, lam, nullptr, nullptr, nullptr, ws, gs);
    });
  }
  auto krs = rev_state_kernel<T, D, E>;
  if (cudaError_t e = opt_in_smem(krs, rev_smem<D, E>())) return e;
  return timed(K_SIMT_REV_STATE, st, [&] {
    krs<<<(unsigned)(BH * gs.nst), NT, rev_smem<D, E>(), st>>>((const T *)a, (const T *)b, lam,
                                                              ws + (size_t)D * E, gs);
  });
}

template <typename T, int D, int E>
cudaError_t combine(const float *ws, const Geo &gs, const float *lam, bool reverse, float *out,
                    cudaStream_t st) {
  const int64_t BH = (int64_t)gs.B * gs.H;
  la2::shard::combine_kernel<D, E>
      <<<dim3((D * E + la2::shard::NT - 1) / la2::shard::NT, (unsigned)BH), la2::shard::NT, 0, st>>>(
          ws, gs.wsS, reverse ? 0 : 1, gs.nst, gs.Lc, gs.L, lam, gs.H, reverse ? 1 : 0, out);
  return cudaGetLastError();
}

template <typename T, int D, int E>
cudaError_t prefix(const float *delta, const float *kv0, const float *lam, int R, int B, int H,
                   int64_t Ls, bool reverse, float *out, cudaStream_t st) {
  const int64_t BH = (int64_t)B * H;
  la2::shard::prefix_kernel<D, E>
      <<<dim3((D * E + la2::shard::NT - 1) / la2::shard::NT, (unsigned)BH), la2::shard::NT, 0, st>>>(
          delta, kv0, lam, H, R, BH, Ls, reverse ? 1 : 0, out);
  return cudaGetLastError();
}


// ------------------------------------------------------------ feature map
namespace {

// The elementwise calls: tensor t's output may be exactly its own `own`
// input (in place); every other pair of arguments shares no byte.
bool fmap_args_ok(const std::vector<Span> &outs, const std::vector<Span> &ins,
                  const std::vector<const void *> &own) {
  for (size_t i = 0; i < outs.size(); i++) {
    if (!outs[i].p) continue;
    for (size_t j = 0; j < ins.size(); j++)
      if (overlaps(outs[i], ins[j]) && !(ins[j].p == outs[i].p && ins[j].p == own[i]))
        return false;
    for (size_t j = i + 1; j < outs.size(); j++)
      if (overlaps(outs[i], outs[j])) return false;
  }
  return true;
}

template <bool GRAD>
la2_status fmap_call(const void *q, const void *k, const void *gq, const void *gk, void *yq,
                     void *yk, int64_t n, la2_dtype dt, cudaStream_t stream) {
  if (n < 0) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (n == 0) return LA2_OK;
  if (!q || !yq || (GRAD && !gq)) return LA2_ERR_INVALID;
  const bool has_k = k != nullptr;
  if ((yk != nullptr) != has_k || (GRAD && (gk != nullptr) != has_k)) return LA2_ERR_INVALID;
  for (const void *p : {q, k, gq, gk, (const void *)yq, (const void *)yk})
    if (p && !aligned16(p)) return LA2_ERR_INVALID;
  const size_t bytes = (size_t)n * esize(dt);
  std::vector<Span> ins = {{q, bytes}, {k, bytes}, {gq, bytes}, {gk, bytes}};
  std::vector<Span> outs = {{yq, bytes}, {yk, bytes}};
  // in place: the map over its input, the gradient over its upstream gradient
  if (!fmap_args_ok(outs, ins, {GRAD ? gq : q, GRAD ? gk : k})) return LA2_ERR_INVALID;
  const int sms = device_sms();
  const int grid = dt == LA2_F32 ? la2::fmap::grid_for<float, GRAD>(n, sms)
                                 : la2::fmap::grid_for<__nv_bfloat16, GRAD>(n, sms);
  cudaError_t err = timed(GRAD ? K_FMAP_GRAD : K_FMAP, stream, [&] {
    if (dt == LA2_F32)
      la2::fmap::enqueue<float, GRAD>(q, gq, yq, k, gk, yk, n, grid, stream);
    else
      la2::fmap::enqueue<__nv_bfloat16, GRAD>(q, gq, yq, k, gk, yk, n, grid, stream);
  });
  return to_status(err);
}

}  // namespace

// ---------------------------------------------- norms, rotary, pool copies
namespace {

using namespace la2::norm_plan;

// Any byte shared by an output with an input or with another output, but for
// an output that is exactly the input named beside it (in place).  Another input
// at that place has to be of the same length: rows of another type would lie
// elsewhere, and one row's output on rows not yet read.
struct OutSpan {
  Span s;
  const void *over;  // the one input whose very buffer it may be, or null
};
bool out_overlap(std::initializer_list<OutSpan> outs, std::initializer_list<Span> ins) {
  for (const OutSpan *o = outs.begin(); o != outs.end(); o++) {
    for (const Span &i : ins)
      if (overlaps(o->s, i) && !(o->over && o->over == i.p && o->s.p == i.p && o->s.n == i.n))
        return true;
    for (const OutSpan *q = o + 1; q != outs.end(); q++)
      if (overlaps(o->s, q->s)) return true;
  }
  return false;
}
bool all_aligned16(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (p && !aligned16(p)) return false;
  return true;
}
bool dtype_ok(la2_dtype dt) { return dt == LA2_F32 || dt == LA2_BF16; }

// Lets a kernel have all the shared memory that its static arrays leave, once
// per device (`done`: a bit for each).  The limit belongs to the kernel, not to
// the call: where calls of one kernel need different sizes and each set its
// own, one thread's could fall between another's set and its launch.
template <typename K>
cudaError_t opt_in_all_smem(K kernel, std::atomic<uint64_t> &done) {
  int dev = 0, most = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  cudaFuncAttributes a;
  if (cudaError_t e = cudaFuncGetAttributes(&a, kernel)) return e;
  if (cudaError_t e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) return e;
  if (cudaError_t e = opt_in_smem(kernel, (size_t)most - a.sharedSizeBytes)) return e;
  if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return cudaSuccess;
}

// CTAs per SM of a kernel with this much dynamic shared memory, on the current
// device.
template <typename K>
int resident(K kernel, int threads, size_t smem, la2::DeviceMemo &memo) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  return memo.get(dev, smem, 1, [&](int *n) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kernel, threads, smem) == cudaSuccess;
  });
}

// Partial rows of weight gradients that a backward may write per SM: its
// CTAs per SM, at most this many.
constexpr int kNormGradPerSm = 4;

// Groups of CTAs (one row of partial sums each) that walk the rows.  Odd rows:
// where a group walks more than one, they lie a multiple of 8 apart.
int64_t norm_groups(int64_t rows, const NormPlan &g, int per_sm) {
  const int64_t need = (rows + g.rpc - 1) / g.rpc;
  const int64_t full = (int64_t)device_sms() * per_sm / (g.slices * g.cl);
  if (need <= full) return need;
  if (g.odd) return full > 8 ? full / 8 * 8 : 8;
  return full > 1 ? full : 1;
}

// Floats of one weight's partial sums, so that another's begin aligned.
size_t partial_floats(int64_t groups, int D) { return ((size_t)groups * D + 7) / 8 * 8; }

size_t norm_ws_bytes(int op, int B, int H, int64_t L, int d, int e, la2_dtype dt) {
  if (!dtype_ok(dt)) return 0;
  if (op == LA2_OP_RESIDUAL_NORM_BACKWARD) {
    if (d < 1 || d > kNormMaxCols) return 0;
    return partial_floats(norm_groups((int64_t)B * H * L, row_plan(d, d % 8 != 0), kNormGradPerSm), d) *
           sizeof(float) * 2;
  }
  if (e != 64 && e != 128) return 0;
  const int64_t rows = (int64_t)B * L, D = (int64_t)H * e;
  if (D > INT32_MAX) return 0;
  // a weight that the heads share has `slices` rows of e per group, which is
  // never more than one row of H * e
  int64_t most = norm_groups(rows, head_plan(H, e), kNormGradPerSm);
  if (D <= kNormMaxCols) {
    const int64_t n = norm_groups(rows, gated_row_plan((int)D, (int)esize(dt)), kNormGradPerSm);
    if (n > most) most = n;
  }
  return (size_t)(most * D) * sizeof(float);
}

cudaError_t colsum(const float *a, const float *b, float *ya, float *yb, int64_t rows, int cols,
                   cudaStream_t st) {
  using namespace la2::norm;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)((cols + kSumCols - 1) / kSumCols), yb ? 2 : 1);
  c.blockDim = dim3(kSumCols * kSumRows);
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return timed(K_NORM_WEIGHT_SUM, st, [&] {
    return cudaLaunchKernelEx(&c, colsum_kernel, a, b, ya, yb, (int)rows, cols);
  });
}

// A launch in clusters of g.cl CTAs along x.
template <typename K, typename P>
cudaError_t launch_groups(K kern, const P &p, const NormPlan &g, int64_t groups, size_t smem,
                          cudaStream_t st) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(groups * g.cl), (unsigned)g.slices);
  c.blockDim = dim3((unsigned)g.nt);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = (unsigned)g.cl;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = g.cl > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&c, kern, p);
}

template <typename T, int E, bool ROW, bool GRAD, la2::norm::Gate GATE, int NT, int TPR, int NV>
cudaError_t gated_launch(la2::norm::Gated p, const NormPlan &g, float *dw, cudaStream_t st) {
  auto kern = la2::norm::gated_kernel<T, E, ROW, GRAD, GATE, NT, TPR, NV>;
  constexpr size_t smem = la2::norm::gated_smem<T, GRAD, GATE, NT, NV>();
  static std::atomic<uint64_t> opted{0};
  if (smem > 32 * 1024)  // 48 KB with the static arrays go without
    if (cudaError_t e = opt_in_all_smem(kern, opted)) return e;
  static la2::DeviceMemo memo;
  const int per_sm = resident(kern, NT, smem, memo);
  const int64_t groups =
      norm_groups(p.rows, g, GRAD && per_sm > kNormGradPerSm ? kNormGradPerSm : per_sm);
  p.cols = g.cols;
  p.cl = g.cl;
  p.tpr_shift = 0;
  while (1 << p.tpr_shift < g.tpr) p.tpr_shift++;
  cudaError_t e = timed(GRAD ? K_GATED_NORM_GRAD : K_GATED_NORM, st,
                        [&] { return launch_groups(kern, p, g, groups, smem, st); });
  if (e != cudaSuccess || !GRAD || !dw) return e;
  return p.shared ? colsum(p.dw, nullptr, dw, nullptr, groups * g.slices, p.e, st)
                  : colsum(p.dw, nullptr, dw, nullptr, groups, p.H * p.e, st);
}

template <typename T, bool GRAD, la2::norm::Gate GATE>
cudaError_t gated_shape(const la2::norm::Gated &p, bool row, float *dw, cudaStream_t st) {
  if (!row) {
    const NormPlan g = head_plan(p.H, p.e);
    return p.e == 64 ? gated_launch<T, 64, false, GRAD, GATE, 256, 32, 1>(p, g, dw, st)
                     : gated_launch<T, 128, false, GRAD, GATE, 256, 32, 1>(p, g, dw, st);
  }
  const NormPlan g = gated_row_plan(p.H * p.e, sizeof(T));
  if (g.tpr == 32) return gated_launch<T, 0, true, GRAD, GATE, 128, 32, 2>(p, g, dw, st);
  if (g.tpr == 128) return gated_launch<T, 0, true, GRAD, GATE, 128, 128, 1>(p, g, dw, st);
  if (g.nv == 1) return gated_launch<T, 0, true, GRAD, GATE, 256, 256, 1>(p, g, dw, st);
  if (g.tpr == 512) return gated_launch<T, 0, true, GRAD, GATE, 512, 512, 2>(p, g, dw, st);
  return gated_launch<T, 0, true, GRAD, GATE, 256, 256, 2>(p, g, dw, st);
}
template <typename T, bool GRAD>
cudaError_t gated_gate(const la2::norm::Gated &p, unsigned flags, float *dw, cudaStream_t st) {
  using namespace la2::norm;
  const bool row = (flags & LA2_NORM_ROW) != 0;
  if (!p.gate) return gated_shape<T, GRAD, GATE_NONE>(p, row, dw, st);
  return flags & LA2_NORM_SILU ? gated_shape<T, GRAD, GATE_SILU>(p, row, dw, st)
                               : gated_shape<T, GRAD, GATE_SIGMOID>(p, row, dw, st);
}
template <bool GRAD>
cudaError_t gated_call(const la2::norm::Gated &p, la2_dtype dt, unsigned flags, float *dw,
                       cudaStream_t st) {
  return dt == LA2_F32 ? gated_gate<float, GRAD>(p, flags, dw, st)
                       : gated_gate<__nv_bfloat16, GRAD>(p, flags, dw, st);
}

// What two residual norm's CTAs on an SM may each have: half of its shared
// memory less what the system and the kernel's static arrays take.
constexpr size_t two_ctas(bool grad, bool odd) {
  return 233472 / 2 - 1024 - (grad ? 1664 : 384) * (odd ? 2 : 1);
}
// Shared memory of such a CTA: the weights and `stages` rows of the streams
// that there are.
template <typename T, typename R, bool POST, bool GRAD>
size_t residual_smem(const la2::norm::Residual &p, int cols, int stages) {
  size_t row = sizeof(R);
  if (GRAD) row += (p.dh_new ? sizeof(R) : 0) + sizeof(T);
  if (GRAD ? POST : p.y != nullptr) row += sizeof(T);
  return la2::norm::kRingHead + (size_t)cols * (sizeof(float) * (POST ? 2 : 1) + stages * row);
}

template <typename T, typename R, bool POST, bool GRAD, bool ODD, int NT, int TPR, int NV>
cudaError_t residual_launch(la2::norm::Residual p, const NormPlan &g, float *dw, float *dpw,
                            cudaStream_t st) {
  auto kern = la2::norm::residual_kernel<T, R, GRAD, POST, ODD, NT, TPR, NV>;
  size_t smem = 0;
  p.stages = 1;
  if (TPR > 32) {
    // two rows where two CTAs on an SM (one of 512 threads) have room for
    // them, else one
    const size_t room = NT == 512 ? 227 * 1024 - 4 * 1024 : two_ctas(GRAD, ODD);
    p.stages = residual_smem<T, R, POST, GRAD>(p, g.cols, 2) <= room ? 2 : 1;
    smem = residual_smem<T, R, POST, GRAD>(p, g.cols, p.stages);
  } else if (GRAD) {
    smem = (size_t)(NT / TPR) * p.D * sizeof(float);
  }
  static std::atomic<uint64_t> opted{0};
  if (smem > 32 * 1024)  // 48 KB with the static arrays go without
    if (cudaError_t e = opt_in_all_smem(kern, opted)) return e;
  static la2::DeviceMemo memo;
  int per_sm = resident(kern, NT, smem, memo);
  if (GRAD && per_sm > kNormGradPerSm) per_sm = kNormGradPerSm;
  const int64_t groups = norm_groups(p.rows, g, per_sm);
  p.cols = g.cols;
  p.cl = g.cl;
  if (GRAD && dpw) p.dpw = p.dw + partial_floats(groups, p.D);
  if (!dw) p.dw = nullptr;
  cudaError_t e = timed(GRAD ? K_RESIDUAL_NORM_GRAD : K_RESIDUAL_NORM, st,
                        [&] { return launch_groups(kern, p, g, groups, smem, st); });
  if (e != cudaSuccess || !GRAD || (!dw && !dpw)) return e;
  return colsum(p.dw, p.dpw, dw, dpw, groups, p.D, st);
}

template <typename T, typename R, bool POST, bool GRAD>
cudaError_t residual_shape(const la2::norm::Residual &p, float *dw, float *dpw, cudaStream_t st) {
  if (p.D % 8 != 0) {
    const NormPlan g = row_plan(p.D, true);
    if (g.tpr == 32) return residual_launch<T, R, POST, GRAD, true, 128, 32, 2>(p, g, dw, dpw, st);
    if (g.nv == 1) return residual_launch<T, R, POST, GRAD, true, 256, 256, 1>(p, g, dw, dpw, st);
    if (g.tpr == 512) return residual_launch<T, R, POST, GRAD, true, 512, 512, 2>(p, g, dw, dpw, st);
    return residual_launch<T, R, POST, GRAD, true, 256, 256, 2>(p, g, dw, dpw, st);
  }
  NormPlan g = row_plan(p.D, false, GRAD ? 2 : 4);
  // 8,192 columns in a CTA only where two such CTAs fit an SM
  if (g.nv == 4 && residual_smem<T, R, POST, GRAD>(p, g.cols, 1) > two_ctas(GRAD, false))
    g = row_plan(p.D, false, 2);
  if (g.tpr == 32) return residual_launch<T, R, POST, GRAD, false, 128, 32, 2>(p, g, dw, dpw, st);
  if (g.tpr == 128) return residual_launch<T, R, POST, GRAD, false, 128, 128, 1>(p, g, dw, dpw, st);
  if (g.nv == 1) return residual_launch<T, R, POST, GRAD, false, 256, 256, 1>(p, g, dw, dpw, st);
  if constexpr (!GRAD)
    if (g.nv == 4) return residual_launch<T, R, POST, GRAD, false, 256, 256, 4>(p, g, dw, dpw, st);
  if (g.tpr == 512) return residual_launch<T, R, POST, GRAD, false, 512, 512, 2>(p, g, dw, dpw, st);
  return residual_launch<T, R, POST, GRAD, false, 256, 256, 2>(p, g, dw, dpw, st);
}

template <bool GRAD>
cudaError_t residual_call(const la2::norm::Residual &p, la2_dtype h_dt, la2_dtype dt, bool post,
                          float *dw, float *dpw, cudaStream_t st) {
  using bf16 = __nv_bfloat16;
  if (dt == LA2_F32)
    return post ? residual_shape<float, float, true, GRAD>(p, dw, dpw, st)
                : residual_shape<float, float, false, GRAD>(p, dw, dpw, st);
  if (h_dt == LA2_F32)
    return post ? residual_shape<bf16, float, true, GRAD>(p, dw, dpw, st)
                : residual_shape<bf16, float, false, GRAD>(p, dw, dpw, st);
  return post ? residual_shape<bf16, bf16, true, GRAD>(p, dw, dpw, st)
              : residual_shape<bf16, bf16, false, GRAD>(p, dw, dpw, st);
}

// ------------------------------------------------------------- rotary
// Bytes from the first to past the last value of a strided tensor.
size_t heads_span(const la2_heads &x, int B, int n, int64_t L, int width, size_t es) {
  return ((size_t)(B - 1) * x.batch + (size_t)(n - 1) * x.head + (size_t)(L - 1) * x.row + width) * es;
}
// Whether values placed with these strides, `inner` of them side by side, are
// at places of their own: each stride steps over all that the smaller ones
// span.
struct Axis {
  int64_t stride, size;
};
bool distinct(std::initializer_list<Axis> axes, int64_t inner) {
  Axis a[3];
  int n = 0;
  for (const Axis &x : axes)
    if (x.size > 1) a[n++] = x;
  for (int i = 0; i < n; i++)
    for (int j = i + 1; j < n; j++)
      if (a[j].stride < a[i].stride) {
        const Axis s = a[i];
        a[i] = a[j];
        a[j] = s;
      }
  for (int i = 0; i < n; i++) {
    if (a[i].stride < inner) return false;
    inner += a[i].stride * (a[i].size - 1);
  }
  return true;
}
// Whether two strided outputs share no value: apart in memory, or slices of
// one buffer side by side in each row (all heads of one, then all of the
// other) or in each head.
bool apart(const la2_heads &x, int nx, int wx, const la2_heads &y, int ny, int wy, int B, int64_t L,
           size_t es) {
  const uintptr_t px = reinterpret_cast<uintptr_t>(x.p), py = reinterpret_cast<uintptr_t>(y.p);
  if (!overlaps({x.p, heads_span(x, B, nx, L, wx, es)}, {y.p, heads_span(y, B, ny, L, wy, es)}))
    return true;
  if ((B > 1 && x.batch != y.batch) || (L > 1 && x.row != y.row)) return false;
  const uintptr_t lo = px < py ? px : py;
  if ((px - lo) % es || (py - lo) % es) return false;
  const int64_t ox = (int64_t)((px - lo) / es), oy = (int64_t)((py - lo) / es);
  // n: values that one tensor spans within a unit (a row's heads, or a head)
  auto side_by_side = [&](int64_t spanx, int64_t spany, std::initializer_list<Axis> axes) {
    if (ox < oy ? ox + spanx > oy : oy + spany > ox) return false;
    const int64_t ex = ox + spanx, ey = oy + spany;
    return distinct(axes, ex > ey ? ex : ey);
  };
  if (side_by_side((nx - 1) * x.head + wx, (ny - 1) * y.head + wy, {{x.batch, B}, {x.row, L}}))
    return true;
  const int n = nx > ny ? nx : ny;
  if (nx > 1 && ny > 1 && x.head != y.head) return false;
  return side_by_side(wx, wy, {{x.batch, B}, {x.row, L}, {nx > 1 ? x.head : y.head, n}});
}

template <typename T, bool GRAD, bool SUMS, bool INTER, int V, int U>
cudaError_t rotary_launch(const la2::rot::Args &a, dim3 grid, cudaStream_t st) {
  using namespace la2::rot;
  auto kern = rotary_kernel<T, GRAD, SUMS, INTER, V, U>;
  const size_t smem = (size_t)TOK * (a.r / 2) * sizeof(float2) + (SUMS ? sums_smem<T, V>() : 0);
  static std::atomic<uint64_t> opted{0};
  if (smem > 32 * 1024)
    if (cudaError_t e = opt_in_all_smem(kern, opted)) return e;
  kern<<<grid, NT, smem, st>>>(a);
  return cudaSuccess;
}
template <typename T, bool GRAD, bool SUMS, bool INTER>
cudaError_t rotary_vec(const la2::rot::Args &a, dim3 grid, bool vec, cudaStream_t st) {
  return vec ? rotary_launch<T, GRAD, SUMS, INTER, 8, sizeof(T) == 2 ? 4 : 2>(a, grid, st)
             : rotary_launch<T, GRAD, SUMS, INTER, 1, 4>(a, grid, st);
}
template <typename T, bool GRAD>
cudaError_t rotary_form(const la2::rot::Args &a, bool inter, dim3 grid, bool vec, cudaStream_t st) {
  if (GRAD && a.rep > 1)
    return inter ? rotary_vec<T, GRAD, GRAD, true>(a, grid, vec, st)
                 : rotary_vec<T, GRAD, GRAD, false>(a, grid, vec, st);
  return inter ? rotary_vec<T, GRAD, false, true>(a, grid, vec, st)
               : rotary_vec<T, GRAD, false, false>(a, grid, vec, st);
}

template <bool GRAD>
la2_status rotary_call(const la2_heads *q, const la2_heads *k, const la2_heads *v,
                       const double *inv_freq, const int64_t *positions, int kind, void *mq,
                       void *mk, void *mv, float scale, unsigned flags, int B, int H, int Hk,
                       int64_t L, int d, int e, int r, la2_dtype dt, cudaStream_t stream) {
  if (B < 0 || H < 0 || Hk < 0 || L < 0 || r < 2 || r > d || r % 2) return LA2_ERR_INVALID;
  if (flags & ~(unsigned)LA2_ROTARY_INTERLEAVED) return LA2_ERR_INVALID;
  if (kind < LA2_POSITIONS_ROW || kind > LA2_POSITIONS_TABLE) return LA2_ERR_INVALID;
  if (!shape_supported(d, v ? e : d, dt)) return LA2_ERR_UNSUPPORTED;
  if (Hk == 0 ? H != 0 : H % Hk) return LA2_ERR_INVALID;
  if ((int64_t)B * H * L == 0) return LA2_OK;
  if (!q || !k || !q->p || !k->p || (v && !v->p) || !mq || !mk || !inv_freq ||
      (v != nullptr) != (mv != nullptr) || (kind != LA2_POSITIONS_ROW) != (positions != nullptr))
    return LA2_ERR_INVALID;
  if (!all_aligned16({mq, mk, mv}) || reinterpret_cast<uintptr_t>(inv_freq) % 8 ||
      reinterpret_cast<uintptr_t>(positions) % 8)
    return LA2_ERR_INVALID;
  const size_t es = esize(dt);
  const la2_heads *in[3] = {q, k, v};
  void *major[3] = {mq, mk, mv};
  const int n[3] = {H, Hk, Hk}, width[3] = {d, d, e}, parts = v ? 3 : 2;
  bool vec = r % 16 == 0;
  Span strided[3] = {{nullptr, 0}, {nullptr, 0}, {nullptr, 0}}, out[3] = {strided[0], strided[0], strided[0]};
  la2::rot::Args a{};
  for (int i = 0; i < parts; i++) {
    const la2_heads &x = *in[i];
    if (x.batch < 0 || x.head < 0 || x.row < 0) return LA2_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(x.p) % es) return LA2_ERR_INVALID;
    if (GRAD && !distinct({{x.batch, B}, {x.head, n[i]}, {x.row, L}}, width[i])) return LA2_ERR_INVALID;
    strided[i] = {x.p, heads_span(x, B, n[i], L, width[i], es)};
    out[i] = {major[i], (size_t)B * H * L * width[i] * es};
    const int64_t odd = (B > 1 ? x.batch : 0) | (n[i] > 1 ? x.head : 0) | (L > 1 ? x.row : 0);
    vec = vec && aligned16(x.p) && (odd * (int64_t)es) % 16 == 0;
    a.part[i] = {x.p, major[i], x.batch, x.head, x.row, n[i], width[i], i < 2 ? r : 0, 0, 0};
  }
  const Span pos = {positions, kind == LA2_POSITIONS_START   ? (size_t)B * 8
                               : kind == LA2_POSITIONS_TABLE ? (size_t)B * L * 8
                                                             : 0};
  const Span freq = {inv_freq, (size_t)r / 2 * 8};
  if (!GRAD) {
    if (out_overlap({{out[0], nullptr}, {out[1], nullptr}, {out[2], nullptr}},
                    {strided[0], strided[1], strided[2], pos, freq}))
      return LA2_ERR_INVALID;
  } else {
    for (int i = 0; i < parts; i++) {
      if (out_overlap({{strided[i], nullptr}}, {out[0], out[1], out[2], pos, freq})) return LA2_ERR_INVALID;
      for (int j = i + 1; j < parts; j++)
        if (!apart(*in[i], n[i], width[i], *in[j], n[j], width[j], B, L, es)) return LA2_ERR_INVALID;
    }
  }
  a.parts = parts;
  a.freq = inv_freq;
  a.pos = positions;
  a.pos_mode = kind;
  a.L = L;
  a.rows = (int64_t)B * L;
  a.rep = H / Hk;
  a.r = r;
  a.scale = scale;
  using namespace la2::rot;
  const int64_t tiles = (a.rows + TOK - 1) / TOK;
  if (tiles > INT32_MAX) return LA2_ERR_UNSUPPORTED;
  for (int i = 0; i < parts; i++) {
    la2::rot::Part &q = a.part[i];
    while (2 * (vec ? 8 : 1) << q.lanes < q.width) q.lanes++;
    // fewer heads than groups of lanes: several groups to a head's sum
    const int groups = LANES >> q.lanes, copies = i ? a.rep : 1;
    while ((q.n << (q.split + 1)) <= groups && (2 << q.split) <= copies) q.split++;
  }
  // few tokens (decode): the tensors and heads of a token are spread over
  // several CTAs (64 tokens 6.8 us against 10.3); many: a CTA takes all of its
  // tokens' (65,536 tokens 526 us against 552 spread)
  const int per = LANES / (d / (vec ? 16 : 2));
  const int64_t groups = (H + per - 1) / per, want = (4 * (int64_t)device_sms() + tiles - 1) / tiles;
  const dim3 grid((unsigned)tiles, (unsigned)(want < groups ? want : groups), want > 1 ? (unsigned)parts : 1u);
  const bool inter = (flags & LA2_ROTARY_INTERLEAVED) != 0;
  return to_status(timed(GRAD ? K_ROTARY_GRAD : K_ROTARY, stream, [&] {
    return dt == LA2_F32 ? rotary_form<float, GRAD>(a, inter, grid, vec, stream)
                         : rotary_form<__nv_bfloat16, GRAD>(a, inter, grid, vec, stream);
  }));
}

// The checks that both directions of the gated norm share.  LA2_OK with
// *empty: nothing to do.
la2_status gated_checks(unsigned flags, int B, int H, int64_t L, int e, float eps, la2_dtype dt,
                        const void *gate, int64_t gate_batch, int64_t gate_row, bool *empty) {
  *empty = false;
  if (B < 0 || H < 0 || L < 0 || !(eps > 0.f) || gate_batch < 0 || gate_row < 0) return LA2_ERR_INVALID;
  if (flags & ~(unsigned)(LA2_NORM_SILU | LA2_NORM_ROW | LA2_NORM_SHARED_WEIGHT)) return LA2_ERR_INVALID;
  if ((flags & LA2_NORM_ROW) && (flags & LA2_NORM_SHARED_WEIGHT)) return LA2_ERR_INVALID;
  if (!dtype_ok(dt) || (e != 64 && e != 128)) return LA2_ERR_UNSUPPORTED;
  if ((flags & LA2_NORM_ROW) && (int64_t)H * e > kNormMaxCols) return LA2_ERR_UNSUPPORTED;
  if ((int64_t)H * e > INT32_MAX || (H > 0 && head_plan(H, e).slices > 65535)) return LA2_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(gate) % esize(dt)) return LA2_ERR_INVALID;
  *empty = (int64_t)B * H * L == 0;
  return LA2_OK;
}
size_t rows_span(int64_t sb, int64_t sl, int B, int64_t L, int64_t D, size_t es) {
  return ((size_t)(B - 1) * sb + (size_t)(L - 1) * sl + D) * es;
}
bool rows_vec(const void *p, int64_t sb, int64_t sl, int B, int64_t L, size_t es) {
  return aligned16(p) && (((B > 1 ? sb : 0) | (L > 1 ? sl : 0)) * (int64_t)es) % 16 == 0;
}

}  // namespace

extern "C" {

const char *la2_status_string(la2_status s) {
  switch (s) {
    case LA2_OK: return "LA2_OK";
    case LA2_ERR_INVALID: return "LA2_ERR_INVALID";
    case LA2_ERR_UNSUPPORTED: return "LA2_ERR_UNSUPPORTED";
    case LA2_ERR_CUDA: return "LA2_ERR_CUDA";
    case LA2_ERR_TIMEOUT: return "LA2_ERR_TIMEOUT";
  }
  return "LA2_ERR_UNKNOWN";
}

const char *la2_version(void) { return "la2 0.1 sm_100a"; }

int la2_set_option(int option, int value) {
  if (option == LA2_OPT_SPLIT) return g_opt_split.exchange(value);
  if (option == LA2_OPT_PATH) return g_opt_path.exchange(value);
  if (option == LA2_OPT_INJECT_TIMEOUT) return g_opt_inject.exchange(value);
  if (option == LA2_OPT_VARIANT) return g_opt_variant.exchange(value);
  if (option == LA2_OPT_TRACE) return g_opt_trace.exchange(value);
  if (option == LA2_OPT_VARLEN_ORDER) return g_opt_varlen_order.exchange(value);
  if (option == LA2_OPT_DECODE_BLOCK_TOKENS) return g_opt_decode_block.exchange(value);
  if (option == LA2_OPT_BWD_FORM) return g_opt_bwd_form.exchange(value);
  return -1;
}

size_t la2_workspace_size(int op, int B, int H, int64_t L, int d, int e, la2_dtype dt) {
  if (B <= 0 || H <= 0 || L <= 0) return 0;
  if (op == LA2_OP_GATED_NORM_BACKWARD || op == LA2_OP_RESIDUAL_NORM_BACKWARD)
    return norm_ws_bytes(op, B, H, L, d, e, dt);
  if (!shape_supported(d, e, dt)) return 0;
  if (op == LA2_OP_DLAMBDA) {
    const Path p = choose_path(d, e, dt);
    if (p == PATH_NONE) return 0;
    return ws_bytes(op, plan_dlambda(B, H, L, true, block_rows(p)), d, e);
  }
  if (op != LA2_OP_FORWARD && op != LA2_OP_BACKWARD && op != LA2_OP_SHARD_STATE) return 0;
  Path p = choose_path(d, e, dt, op != LA2_OP_SHARD_STATE);
  if (p == PATH_NONE) return 0;
  Geo g = plan(B, H, L, block_rows(p), p);
  const int sd = p == PATH_TC ? 128 : d, se = p == PATH_TC ? 128 : e;  // state slot shape
  if (op == LA2_OP_BACKWARD)
    return ws_bwd_bytes(g, plan_rev(B, H, L, p), sd, se) + (padded(p, d, e) ? pad_bytes(g, 2) : 0);
  if (op == LA2_OP_FORWARD) return ws_bytes(op, g, sd, se) + (padded(p, d, e) ? pad_bytes(g, 2) : 0);
  return ws_bytes(op, g, d, e);
}

}  // extern "C"

namespace {

// The argument checks of la2_forward (and of la2_forward_noalloc, which
// passes no workspace).  LA2_OK with *empty set: B*H == 0, nothing to do.
la2_status forward_checks(const void *q, const void *k, const void *v, const float *lambda,
                          const float *kv0, const void *o, const float *kv_out, int B, int H,
                          int64_t L, int d, int e, la2_dtype dt, const void *workspace,
                          size_t workspace_bytes, bool *empty) {
  *empty = false;
  if (B < 0 || H < 0 || L < 0) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (!shape_supported(d, e, dt)) return LA2_ERR_UNSUPPORTED;
  const int64_t BH = (int64_t)B * H;
  const size_t es = esize(dt);
  const size_t nq = (size_t)BH * L * d * es, nv = (size_t)BH * L * e * es;
  const size_t ns = (size_t)BH * d * e * sizeof(float);
  if (BH == 0) {
    *empty = true;
    return LA2_OK;
  }
  if (!lambda || (L > 0 && (!q || !k || !v || !o))) return LA2_ERR_INVALID;
  for (const void *p : std::initializer_list<const void *>{(const void *)q, (const void *)k, (const void *)v, (const void *)lambda,
                        (const void *)kv0, (const void *)o, (const void *)kv_out, workspace})
    if (p && !aligned16(p)) return LA2_ERR_INVALID;
  if (kv_out && kv_out == kv0) return LA2_ERR_INVALID;
  std::vector<Span> ins = {{q, nq}, {k, nq}, {v, nv}, {lambda, (size_t)H * 4}, {kv0, kv0 ? ns : 0}};
  std::vector<Span> outs = {{o, nv}, {kv_out, kv_out ? ns : 0}, {workspace, workspace_bytes}};
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;
  return LA2_OK;
}

}  // namespace

extern "C" {

la2_status la2_forward(const void *q, const void *k, const void *v,
                       const float *lambda, const float *kv0, void *o, float *kv_out,
                       int B, int H, int64_t L, int d, int e, la2_dtype dt,
                       void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  bool empty = false;
  const la2_status chk = forward_checks(q, k, v, lambda, kv0, o, kv_out, B, H, L, d, e, dt,
                                        workspace, workspace_bytes, &empty);
  if (chk != LA2_OK || empty) return chk;
  const int64_t BH = (int64_t)B * H;
  const size_t ns = (size_t)BH * d * e * sizeof(float);

  if (L == 0) {
    if (!kv_out) return LA2_OK;
    cudaError_t err = kv0 ? cudaMemcpyAsync(kv_out, kv0, ns, cudaMemcpyDeviceToDevice, stream)
                          : cudaMemsetAsync(kv_out, 0, ns, stream);
    return to_status(err);
  }
  Path p = choose_path(d, e, dt, true);
  if (p == PATH_NONE) return LA2_ERR_UNSUPPORTED;
  Geo g = plan(B, H, L, block_rows(p), p);
  const bool pad = padded(p, d, e);
  const size_t states = ws_bytes(LA2_OP_FORWARD, g, p == PATH_TC ? 128 : d, p == PATH_TC ? 128 : e);
  const size_t need = states + (pad ? pad_bytes(g, 2) : 0);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LA2_ERR_INVALID;
  float *ws = (float *)workspace;
  cudaError_t err;
  if (p == PATH_TC) {
    g.inject = g_opt_inject.exchange(0);
    g.d = d;
    g.e = e;
    // 64-column heads: the states in and out padded to 128 x 128
    float *scratch = pad ? reinterpret_cast<float *>(reinterpret_cast<char *>(workspace) + states)
                         : nullptr;
    const float *kv0_t = kv0;
    float *kv_out_t = kv_out;
    if (pad) {
      kv0_t = kv0 ? scratch : nullptr;
      kv_out_t = kv_out ? scratch + (size_t)BH * 128 * 128 : nullptr;
      if (kv0) {
        err = timed(K_STATE_PAD, stream, [&] { la2::tc::pad_states(kv0, scratch, BH, d, e, stream); });
        if (err != cudaSuccess) return to_status(err);
      }
    }
    err = la2::tc::forward(q, k, v, lambda, kv0_t, o, kv_out_t, ws, g, stream,
                           [&](int which, auto &&fn) {
                             return timed(which == 0 ? K_TC_FWD_STATE : which == 1 ? K_SCAN_FWD : K_TC_FWD,
                                          stream, fn);
                           });
    if (err == cudaSuccess && pad && kv_out)
      err = timed(K_STATE_PAD, stream,
                  [&] { la2::tc::unpad_states(kv_out_t, kv_out, BH, d, e, stream); });
  } else if (dt == LA2_F32) {
    err = LA2_DISPATCH_DE(d, e, simt_forward, float, q, k, v, lambda, kv0, o, kv_out, ws, g, stream);
  } else {
    err = LA2_DISPATCH_DE(d, e, simt_forward, __nv_bfloat16, q, k, v, lambda, kv0, o, kv_out, ws, g,
                          stream);
  }
  return to_status(err);
}

la2_status la2_backward(const void *q, const void *k, const void *v,
                        const float *lambda, const float *kv0, const void *dO,
                        void *dq, void *dk, void *dv, float *dkv0,
                        int B, int H, int64_t L, int d, int e, la2_dtype dt,
                        void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return la2_backward_ex(q, k, v, lambda, kv0, dO, dq, dk, dv, dkv0, B, H, L, d, e, dt, workspace,
                         workspace_bytes, 0u, stream);
}

la2_status la2_backward_ex(const void *q, const void *k, const void *v,
                           const float *lambda, const float *kv0, const void *dO,
                           void *dq, void *dk, void *dv, float *dkv0,
                           int B, int H, int64_t L, int d, int e, la2_dtype dt,
                           void *workspace, size_t workspace_bytes, unsigned flags,
                           cudaStream_t stream) {
  if (flags & ~(unsigned)LA2_BWD_REUSE_FORWARD_STATES) return LA2_ERR_INVALID;
  const bool reuse = (flags & LA2_BWD_REUSE_FORWARD_STATES) != 0;
  if (B < 0 || H < 0 || L < 0) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (!shape_supported(d, e, dt)) return LA2_ERR_UNSUPPORTED;
  const int64_t BH = (int64_t)B * H;
  const size_t es = esize(dt);
  const size_t nq = (size_t)BH * L * d * es, nv = (size_t)BH * L * e * es;
  const size_t ns = (size_t)BH * d * e * sizeof(float);
  if (BH == 0) return LA2_OK;
  if (!lambda || (L > 0 && (!q || !k || !v || !dO || !dq || !dk || !dv))) return LA2_ERR_INVALID;
  for (const void *p : std::initializer_list<const void *>{(const void *)q, (const void *)k, (const void *)v, (const void *)lambda,
                        (const void *)kv0, (const void *)dO, (const void *)dq, (const void *)dk,
                        (const void *)dv, (const void *)dkv0, workspace})
    if (p && !aligned16(p)) return LA2_ERR_INVALID;
  std::vector<Span> ins = {{q, nq}, {k, nq}, {v, nv}, {dO, nv}, {lambda, (size_t)H * 4},
                           {kv0, kv0 ? ns : 0}};
  std::vector<Span> outs = {{dq, nq}, {dk, nq}, {dv, nv}, {dkv0, dkv0 ? ns : 0},
                            {workspace, workspace_bytes}};
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;

  if (L == 0) {
    if (!dkv0) return LA2_OK;
    return to_status(cudaMemsetAsync(dkv0, 0, ns, stream));
  }
  Path p = choose_path(d, e, dt, true);
  if (p == PATH_NONE) return LA2_ERR_UNSUPPORTED;
  Geo g = plan(B, H, L, block_rows(p), p);
  Geo gr = plan_rev(B, H, L, p);
  const bool pad = padded(p, d, e);
  const size_t states =
      ws_bwd_bytes(g, gr, p == PATH_TC ? 128 : d, p == PATH_TC ? 128 : e);
  const size_t need = states + (pad ? pad_bytes(g, 2) : 0);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LA2_ERR_INVALID;
  float *ws = (float *)workspace;
  cudaError_t err;
  if (p == PATH_TC) {
    g.d = gr.d = d;
    g.e = gr.e = e;
    // 64-column heads: kv0 in and dkv0 out padded to 128 x 128
    float *scratch = pad ? reinterpret_cast<float *>(reinterpret_cast<char *>(workspace) + states)
                         : nullptr;
    const float *kv0_t = kv0;
    float *dkv0_t = dkv0;
    if (pad) {
      kv0_t = kv0 ? scratch : nullptr;
      dkv0_t = dkv0 ? scratch + (size_t)BH * 128 * 128 : nullptr;
      if (kv0) {
        err = timed(K_STATE_PAD, stream, [&] { la2::tc::pad_states(kv0, scratch, BH, d, e, stream); });
        if (err != cudaSuccess) return to_status(err);
      }
    }
    err = la2::tc::backward(q, k, v, lambda, kv0_t, dO, dq, dk, dv, dkv0_t, ws, g, gr, reuse, stream,
                            [&](int which, auto &&fn) {
                              static const int ids[] = {K_TC_FWD_STATE, K_SCAN_FWD, K_TC_DQ,
                                                        K_TC_REV_STATE, K_SCAN_REV, K_TC_DV,
                                                        K_TC_DK, K_TC_DKDV};
                              return timed(ids[which], stream, fn);
                            });
    if (err == cudaSuccess && pad && dkv0)
      err = timed(K_STATE_PAD, stream,
                  [&] { la2::tc::unpad_states(dkv0_t, dkv0, BH, d, e, stream); });
  } else if (dt == LA2_F32) {
    err = LA2_DISPATCH_DE(d, e, simt_backward, float, q, k, v, lambda, kv0, dO, dq, dk, dv, dkv0,
                          ws, g, reuse, stream);
  } else {
    err = LA2_DISPATCH_DE(d, e, simt_backward, __nv_bfloat16, q, k, v, lambda, kv0, dO, dq, dk,
                          dv, dkv0, ws, g, reuse, stream);
  }
  return to_status(err);
}

// ------------------------------------------------------- packed varlen
namespace {

// One CTA per (sequence, head) over the sequence's rows; no chunk split.
Geo plan_varlen(int N, int H, int64_t T, const int64_t *cu) {
  Geo g;
  g.B = N;
  g.H = H;
  g.L = T;
  g.S = 1;
  g.Lc = T;
  g.M = 1;
  g.Ls = T;
  g.Ssub = 1;
  g.wsS = 1;
  g.nst = 0;
  g.c0 = 0;
  g.cu = cu;
  g.lpt = N <= 64 && g_opt_varlen_order.load() == 0;
  g.slots = nullptr;
  g.pool = 0;
  g.inject = 0;
  g.variant = 0;  // the packed form exists in the warp-specialised kernel only
  g.trace = -1;
  return g;
}

// Shared argument checks of the packed entry points: sizes, null and
// alignment rules, and no output overlapping any argument.
la2_status check_varlen(int N, int H, int64_t T, int d, int e, la2_dtype dt, const int64_t *cu,
                        const float *lambda, std::vector<Span> ins, std::vector<Span> outs,
                        bool need_tensors) {
  if (N < 0 || H < 0 || T < 0) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (!shape_supported(d, e, dt)) return LA2_ERR_UNSUPPORTED;
  if (!lambda || !cu || need_tensors) return LA2_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(cu) % 8 != 0) return LA2_ERR_INVALID;
  for (const Span &sp : ins)
    if (sp.p && sp.p != (const void *)cu && !aligned16(sp.p)) return LA2_ERR_INVALID;
  for (const Span &sp : outs)
    if (sp.p && !aligned16(sp.p)) return LA2_ERR_INVALID;
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;
  return LA2_OK;
}

}  // namespace

la2_status la2_forward_varlen(const void *q, const void *k, const void *v, const float *lambda,
                              const int64_t *cu_seqlens, const float *kv0, void *o,
                              float *kv_out, int N, int H, int64_t T, int d, int e,
                              la2_dtype dt, cudaStream_t stream) {
  if (N == 0 || H == 0) return (N < 0 || H < 0 || T < 0) ? LA2_ERR_INVALID : LA2_OK;
  const size_t es = (dt == LA2_F32 || dt == LA2_BF16) ? esize(dt) : 0;
  const size_t nq = (size_t)H * T * d * es, nv = (size_t)H * T * e * es;
  const size_t ns = (size_t)N * H * d * e * sizeof(float);
  if (kv_out && kv_out == kv0) return LA2_ERR_INVALID;
  la2_status st = check_varlen(
      N, H, T, d, e, dt, cu_seqlens, lambda,
      {{q, nq}, {k, nq}, {v, nv}, {lambda, (size_t)H * 4}, {kv0, kv0 ? ns : 0},
       {cu_seqlens, (size_t)(N + 1) * 8}},
      {{o, nv}, {kv_out, kv_out ? ns : 0}}, T > 0 && (!q || !k || !v || !o));
  if (st != LA2_OK) return st;
  if (T == 0) {  // every sequence is empty
    if (!kv_out) return LA2_OK;
    return to_status(kv0 ? cudaMemcpyAsync(kv_out, kv0, ns, cudaMemcpyDeviceToDevice, stream)
                         : cudaMemsetAsync(kv_out, 0, ns, stream));
  }
  Path p = choose_path(d, e, dt);
  if (p == PATH_NONE) return LA2_ERR_UNSUPPORTED;
  Geo g = plan_varlen(N, H, T, cu_seqlens);
  cudaError_t err;
  if (p == PATH_TC) {
    err = la2::tc::forward_varlen(q, k, v, lambda, kv0, o, kv_out, g, stream,
                                  [&](int, auto &&fn) { return timed(K_TC_FWD, stream, fn); });
  } else if (dt == LA2_F32) {
    err = LA2_DISPATCH_DE(d, e, simt_forward, float, q, k, v, lambda, kv0, o, kv_out, nullptr, g,
                          stream);
  } else {
    err = LA2_DISPATCH_DE(d, e, simt_forward, __nv_bfloat16, q, k, v, lambda, kv0, o, kv_out,
                          nullptr, g, stream);
  }
  return to_status(err);
}

la2_status la2_backward_varlen(const void *q, const void *k, const void *v, const float *lambda,
                               const int64_t *cu_seqlens, const float *kv0, const void *dO,
                               void *dq, void *dk, void *dv, float *dkv0, int N, int H,
                               int64_t T, int d, int e, la2_dtype dt, cudaStream_t stream) {
  if (N == 0 || H == 0) return (N < 0 || H < 0 || T < 0) ? LA2_ERR_INVALID : LA2_OK;
  const size_t es = (dt == LA2_F32 || dt == LA2_BF16) ? esize(dt) : 0;
  const size_t nq = (size_t)H * T * d * es, nv = (size_t)H * T * e * es;
  const size_t ns = (size_t)N * H * d * e * sizeof(float);
  la2_status st = check_varlen(
      N, H, T, d, e, dt, cu_seqlens, lambda,
      {{q, nq}, {k, nq}, {v, nv}, {dO, nv}, {lambda, (size_t)H * 4}, {kv0, kv0 ? ns : 0},
       {cu_seqlens, (size_t)(N + 1) * 8}},
      {{dq, nq}, {dk, nq}, {dv, nv}, {dkv0, dkv0 ? ns : 0}},
      T > 0 && (!q || !k || !v || !dO || !dq || !dk || !dv));
  if (st != LA2_OK) return st;
  if (T == 0) return dkv0 ? to_status(cudaMemsetAsync(dkv0, 0, ns, stream)) : LA2_OK;
  Path p = choose_path(d, e, dt);
  if (p == PATH_NONE) return LA2_ERR_UNSUPPORTED;
  Geo g = plan_varlen(N, H, T, cu_seqlens);
  g.rev_pair = p == PATH_TC && g_opt_bwd_form.load() != 1;
  cudaError_t err;
  if (p == PATH_TC) {
    err = la2::tc::backward_varlen(q, k, v, lambda, kv0, dO, dq, dk, dv, dkv0, g, stream,
                                   [&](int which, auto &&fn) {
                                     return timed(which == 2   ? K_TC_DQ
                                                  : which == 5 ? K_TC_DV
                                                  : which == 6 ? K_TC_DK
                                                               : K_TC_DKDV,
                                                  stream, fn);
                                   });
  } else if (dt == LA2_F32) {
    err = LA2_DISPATCH_DE(d, e, simt_backward, float, q, k, v, lambda, kv0, dO, dq, dk, dv, dkv0,
                          nullptr, g, false, stream);
  } else {
    err = LA2_DISPATCH_DE(d, e, simt_backward, __nv_bfloat16, q, k, v, lambda, kv0, dO, dq, dk,
                          dv, dkv0, nullptr, g, false, stream);
  }
  return to_status(err);
}

la2_status la2_forward_pool(const void *q, const void *k, const void *v, const float *lambda,
                            float *kv_pool, const int32_t *slots, int pool_size, void *o,
                            unsigned flags, int B, int H, int64_t L, int d, int e, la2_dtype dt,
                            void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (flags & ~(unsigned)LA2_POOL_CONTINUE) return LA2_ERR_INVALID;
  if (B < 0 || H < 0 || L < 1 || pool_size < 0) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (!shape_supported(d, e, dt)) return LA2_ERR_UNSUPPORTED;
  const int64_t BH = (int64_t)B * H;
  if (BH == 0) return LA2_OK;
  if (!q || !k || !v || !lambda || !kv_pool || !slots || !o) return LA2_ERR_INVALID;
  for (const void *p : std::initializer_list<const void *>{
           (const void *)q, (const void *)k, (const void *)v, (const void *)lambda,
           (const void *)kv_pool, (const void *)o, workspace})
    if (p && !aligned16(p)) return LA2_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(slots) % 4 != 0) return LA2_ERR_INVALID;
  const size_t es = esize(dt);
  const size_t nq = (size_t)BH * L * d * es, nv = (size_t)BH * L * e * es;
  std::vector<Span> ins = {{q, nq}, {k, nq}, {v, nv}, {lambda, (size_t)H * 4},
                           {slots, (size_t)B * 4}};
  std::vector<Span> outs = {{o, nv},
                            {kv_pool, (size_t)pool_size * H * d * e * sizeof(float)},
                            {workspace, workspace_bytes}};
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;
  Path p = choose_path(d, e, dt);
  if (p == PATH_NONE) return LA2_ERR_UNSUPPORTED;
  Geo g = plan(B, H, L, block_rows(p), p);
  g.slots = slots;
  g.pool = pool_size;
  g.variant = 0;  // the slot table exists in the warp-specialised kernel only
  const size_t need = ws_bytes(LA2_OP_FORWARD, g, d, e);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LA2_ERR_INVALID;
  float *ws = (float *)workspace;
  const float *kv0 = (flags & LA2_POOL_CONTINUE) ? kv_pool : nullptr;
  cudaError_t err;
  if (p == PATH_TC) {
    err = la2::tc::forward(q, k, v, lambda, kv0, o, kv_pool, ws, g, stream,
                           [&](int which, auto &&fn) {
                             return timed(which == 0 ? K_TC_FWD_STATE : which == 1 ? K_SCAN_FWD : K_TC_FWD,
                                          stream, fn);
                           });
  } else if (dt == LA2_F32) {
    err = LA2_DISPATCH_DE(d, e, simt_forward, float, q, k, v, lambda, kv0, o, kv_pool, ws, g,
                          stream);
  } else {
    err = LA2_DISPATCH_DE(d, e, simt_forward, __nv_bfloat16, q, k, v, lambda, kv0, o, kv_pool,
                          ws, g, stream);
  }
  return to_status(err);
}

// ------------------------------------------------------------ shards
namespace {

// The chunk-state passes over every sub-chunk of one shard.
Geo shard_geo(const Geo &g) {
  Geo s = g;
  s.S = g.Ssub;
  s.Lc = g.Ls;
  s.M = 1;
  s.nst = g.Ssub;
  s.c0 = 0;
  s.wsS = g.Ssub + 1;
  s.variant = 0;
  return s;
}

}  // namespace

la2_status la2_shard_state(const void *a, const void *b, const float *lambda, float *out,
                           int B, int H, int64_t L, int d, int e, la2_dtype dt, int reverse,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (B < 0 || H < 0 || L < 1) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (!shape_supported(d, e, dt)) return LA2_ERR_UNSUPPORTED;
  const int64_t BH = (int64_t)B * H;
  if (BH == 0) return LA2_OK;
  if (!a || !b || !lambda || !out || !workspace) return LA2_ERR_INVALID;
  for (const void *p : std::initializer_list<const void *>{a, b, (const void *)lambda,
                                                          (const void *)out, workspace})
    if (!aligned16(p)) return LA2_ERR_INVALID;
  const size_t es = esize(dt);
  std::vector<Span> ins = {{a, (size_t)BH * L * d * es}, {b, (size_t)BH * L * e * es},
                           {lambda, (size_t)H * 4}};
  std::vector<Span> outs = {{out, (size_t)BH * d * e * 4}, {workspace, workspace_bytes}};
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;
  Path p = choose_path(d, e, dt);
  if (p == PATH_NONE) return LA2_ERR_UNSUPPORTED;
  const Geo g = plan(B, H, L, block_rows(p), p);
  if (workspace_bytes < ws_bytes(LA2_OP_SHARD_STATE, g, d, e)) return LA2_ERR_INVALID;
  const Geo gs = shard_geo(g);
  float *ws = (float *)workspace;
  cudaError_t err;
  if (p == PATH_TC) {
    err = la2::tc::shard_state(a, b, lambda, ws, gs, reverse != 0, stream,
                               [&](int which, auto &&fn) {
                                 return timed(which == 0 ? K_TC_FWD_STATE : K_TC_REV_STATE, stream, fn);
                               });
  } else if (dt == LA2_F32) {
    err = LA2_DISPATCH_DE(d, e, simt_shard_state, float, a, b, lambda, ws, gs, reverse != 0, stream);
  } else {
    err = LA2_DISPATCH_DE(d, e, simt_shard_state, __nv_bfloat16, a, b, lambda, ws, gs, reverse != 0,
                          stream);
  }
  if (err == cudaSuccess)
    err = LA2_DISPATCH_DE(d, e, combine, float, ws, gs, lambda, reverse != 0, out, stream);
  return to_status(err);
}

la2_status la2_state_prefix(const float *delta, const float *kv0, const float *lambda,
                            float *out, int R, int B, int H, int64_t L_shard, int d, int e,
                            int reverse, cudaStream_t stream) {
  if (R < 0 || B < 0 || H < 0 || L_shard < 0) return LA2_ERR_INVALID;
  if (!shape_supported(d, e, LA2_F32)) return LA2_ERR_UNSUPPORTED;
  const int64_t BH = (int64_t)B * H;
  if (BH == 0 || R == 0) return LA2_OK;
  if (!delta || !lambda || !out) return LA2_ERR_INVALID;
  for (const void *p : std::initializer_list<const void *>{(const void *)delta, (const void *)kv0,
                                                          (const void *)lambda, (const void *)out})
    if (p && !aligned16(p)) return LA2_ERR_INVALID;
  const size_t all_states = (size_t)R * BH * d * e * 4;
  std::vector<Span> ins = {{delta, all_states}, {kv0, kv0 ? (size_t)BH * d * e * 4 : 0},
                           {lambda, (size_t)H * 4}};
  std::vector<Span> outs = {{out, all_states}};
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;
  return to_status(LA2_DISPATCH_DE(d, e, prefix, float, delta, reverse ? nullptr : kv0, lambda, R,
                                   B, H, L_shard, reverse != 0, out, stream));
}

la2_status la2_backward_shard(const void *q, const void *k, const void *v, const float *lambda,
                              const float *kv0, const void *dO, const float *dstate_end,
                              void *dq, void *dk, void *dv, float *dkv0, int B, int H,
                              int64_t L, int d, int e, la2_dtype dt, void *workspace,
                              size_t workspace_bytes, unsigned flags, cudaStream_t stream) {
  if (flags & ~(unsigned)LA2_BWD_REUSE_FORWARD_STATES) return LA2_ERR_INVALID;
  const bool reuse = (flags & LA2_BWD_REUSE_FORWARD_STATES) != 0;
  if (B < 0 || H < 0 || L < 1) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (!shape_supported(d, e, dt)) return LA2_ERR_UNSUPPORTED;
  const int64_t BH = (int64_t)B * H;
  if (BH == 0) return LA2_OK;
  const size_t es = esize(dt);
  const size_t nq = (size_t)BH * L * d * es, nv = (size_t)BH * L * e * es;
  const size_t ns = (size_t)BH * d * e * sizeof(float);
  if (!lambda || !q || !k || !v || !dO || !dq || !dk || !dv) return LA2_ERR_INVALID;
  for (const void *p : std::initializer_list<const void *>{
           (const void *)q, (const void *)k, (const void *)v, (const void *)lambda,
           (const void *)kv0, (const void *)dO, (const void *)dstate_end, (const void *)dq,
           (const void *)dk, (const void *)dv, (const void *)dkv0, workspace})
    if (p && !aligned16(p)) return LA2_ERR_INVALID;
  std::vector<Span> ins = {{q, nq}, {k, nq}, {v, nv}, {dO, nv}, {lambda, (size_t)H * 4},
                           {kv0, kv0 ? ns : 0}, {dstate_end, dstate_end ? ns : 0}};
  std::vector<Span> outs = {{dq, nq}, {dk, nq}, {dv, nv}, {dkv0, dkv0 ? ns : 0},
                            {workspace, workspace_bytes}};
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;
  Path p = choose_path(d, e, dt);
  if (p == PATH_NONE) return LA2_ERR_UNSUPPORTED;
  Geo g = plan(B, H, L, block_rows(p), p);
  const Geo gr = plan_rev(B, H, L, p);
  const size_t need = ws_bwd_bytes(g, gr, d, e);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LA2_ERR_INVALID;
  float *ws = (float *)workspace;
  cudaError_t err;
  if (p == PATH_TC) {
    err = la2::tc::backward(q, k, v, lambda, kv0, dO, dq, dk, dv, dkv0, ws, g, gr, reuse, stream,
                            [&](int which, auto &&fn) {
                              static const int ids[] = {K_TC_FWD_STATE, K_SCAN_FWD, K_TC_DQ,
                                                        K_TC_REV_STATE, K_SCAN_REV, K_TC_DV,
                                                        K_TC_DK, K_TC_DKDV};
                              return timed(ids[which], stream, fn);
                            },
                            dstate_end);
  } else if (dt == LA2_F32) {
    err = LA2_DISPATCH_DE(d, e, simt_backward, float, q, k, v, lambda, kv0, dO, dq, dk, dv, dkv0,
                          ws, g, reuse, stream, dstate_end);
  } else {
    err = LA2_DISPATCH_DE(d, e, simt_backward, __nv_bfloat16, q, k, v, lambda, kv0, dO, dq, dk,
                          dv, dkv0, ws, g, reuse, stream, dstate_end);
  }
  return to_status(err);
}

namespace {
// split: chunk the sequences as la2_workspace_size(LA2_OP_DLAMBDA) planned
// (the workspace must then hold that much); otherwise one chunk per (b,h).
la2_status dlambda_call(const void *q, const void *k, const void *v, const float *lambda,
                        const float *kv0, const void *dO, float *dlambda, int B, int H,
                        int64_t L, int d, int e, la2_dtype dt, void *workspace,
                        size_t workspace_bytes, bool split, cudaStream_t stream) {
  if (B < 0 || H < 0 || L < 0) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (!shape_supported(d, e, dt)) return LA2_ERR_UNSUPPORTED;
  const int64_t BH = (int64_t)B * H;
  if (H == 0) return LA2_OK;
  if (!lambda || !dlambda || (BH > 0 && L > 0 && (!q || !k || !v || !dO))) return LA2_ERR_INVALID;
  for (const void *p : std::initializer_list<const void *>{
           (const void *)q, (const void *)k, (const void *)v, (const void *)lambda,
           (const void *)kv0, (const void *)dO, (const void *)dlambda, workspace})
    if (p && !aligned16(p)) return LA2_ERR_INVALID;
  const size_t es = esize(dt);
  const size_t nq = (size_t)BH * L * d * es, nv = (size_t)BH * L * e * es;
  std::vector<Span> ins = {{q, nq}, {k, nq}, {v, nv}, {dO, nv}, {lambda, (size_t)H * 4},
                           {kv0, kv0 ? (size_t)BH * d * e * 4 : 0}};
  std::vector<Span> outs = {{dlambda, (size_t)H * 4}, {workspace, workspace ? workspace_bytes : 0}};
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;
  if (BH == 0 || L == 0) {  // no token depends on lambda
    return to_status(cudaMemsetAsync(dlambda, 0, (size_t)H * sizeof(float), stream));
  }
  const Path p = choose_path(d, e, dt);
  if (p == PATH_NONE) return LA2_ERR_UNSUPPORTED;
  const Geo g = plan_dlambda(B, H, L, split, block_rows(p));
  const size_t need = ws_bytes(LA2_OP_DLAMBDA, g, d, e);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LA2_ERR_INVALID;
  float *ws = (float *)workspace;
  if (p == PATH_TC)
    return to_status(la2::tcd::dlambda(q, k, v, dO, lambda, kv0, dlambda, ws, g, stream,
                                       [&](int which, auto &&fn) {
                                         static const int ids[] = {K_TC_DLAMBDA_STATE,
                                                                   K_SIMT_DLAMBDA_SCAN,
                                                                   K_TC_DLAMBDA};
                                         return timed(ids[which], stream, fn);
                                       }));
  cudaError_t err =
      dt == LA2_F32
          ? LA2_DISPATCH_DE(d, e, simt_dlambda, float, q, k, v, dO, lambda, kv0, dlambda, ws, g,
                            stream)
          : LA2_DISPATCH_DE(d, e, simt_dlambda, __nv_bfloat16, q, k, v, dO, lambda, kv0, dlambda,
                            ws, g, stream);
  return to_status(err);
}
}  // namespace

la2_status la2_backward_dlambda(const void *q, const void *k, const void *v,
                                const float *lambda, const float *kv0, const void *dO,
                                float *dlambda, int B, int H, int64_t L, int d, int e,
                                la2_dtype dt, cudaStream_t stream) {
  return dlambda_call(q, k, v, lambda, kv0, dO, dlambda, B, H, L, d, e, dt, nullptr, 0, false,
                      stream);
}

la2_status la2_backward_dlambda_ex(const void *q, const void *k, const void *v,
                                   const float *lambda, const float *kv0, const void *dO,
                                   float *dlambda, int B, int H, int64_t L, int d, int e,
                                   la2_dtype dt, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  return dlambda_call(q, k, v, lambda, kv0, dO, dlambda, B, H, L, d, e, dt, workspace,
                      workspace_bytes, true, stream);
}

la2_status la2_decode_step(const void *q, const void *k, const void *v, const float *lambda,
                           float *kv, void *o, int B, int H, int d, int e, la2_dtype dt,
                           cudaStream_t stream) {
  if (B < 0 || H < 0) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (!shape_supported(d, e, dt)) return LA2_ERR_UNSUPPORTED;
  const int64_t BH = (int64_t)B * H;
  if (BH == 0) return LA2_OK;
  if (!q || !k || !v || !lambda || !kv || !o) return LA2_ERR_INVALID;
  for (const void *p : std::initializer_list<const void *>{(const void *)q, (const void *)k, (const void *)v, (const void *)lambda,
                        (const void *)kv, (const void *)o})
    if (!aligned16(p)) return LA2_ERR_INVALID;
  const size_t es = esize(dt);
  std::vector<Span> ins = {{q, BH * d * es}, {k, BH * d * es}, {v, BH * e * es},
                           {lambda, (size_t)H * 4}};
  std::vector<Span> outs = {{kv, BH * d * e * sizeof(float)}, {o, BH * e * es}};
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;
  cudaError_t err =
      dt == LA2_F32
          ? LA2_DISPATCH_DE(d, e, decode, float, q, k, v, lambda, kv, nullptr, B, o, B, H, 1, stream)
          : LA2_DISPATCH_DE(d, e, decode, __nv_bfloat16, q, k, v, lambda, kv, nullptr, B, o, B, H,
                            1, stream);
  return to_status(err);
}

la2_status la2_feature_map(const void *q, const void *k, void *phi_q, void *phi_k, int64_t n,
                           la2_dtype dt, cudaStream_t stream) {
  return fmap_call<false>(q, k, nullptr, nullptr, phi_q, phi_k, n, dt, stream);
}

la2_status la2_feature_map_backward(const void *q, const void *k, const void *dphi_q,
                                    const void *dphi_k, void *dq, void *dk, int64_t n,
                                    la2_dtype dt, cudaStream_t stream) {
  return fmap_call<true>(q, k, dphi_q, dphi_k, dq, dk, n, dt, stream);
}

la2_status la2_rotary(const la2_heads *q, const la2_heads *k, const la2_heads *v,
                      const double *inv_freq, const int64_t *positions, int positions_kind,
                      void *rq, void *rk, void *rv, float scale, unsigned flags, int B, int H,
                      int Hk, int64_t L, int d, int e, int r, la2_dtype dt, cudaStream_t stream) {
  return rotary_call<false>(q, k, v, inv_freq, positions, positions_kind, rq, rk, rv, scale, flags,
                            B, H, Hk, L, d, e, r, dt, stream);
}

la2_status la2_rotary_backward(const void *dq, const void *dk, const void *dv,
                               const double *inv_freq, const int64_t *positions,
                               int positions_kind, const la2_heads *gq, const la2_heads *gk,
                               const la2_heads *gv, float scale, unsigned flags, int B, int H,
                               int Hk, int64_t L, int d, int e, int r, la2_dtype dt,
                               cudaStream_t stream) {
  return rotary_call<true>(gq, gk, gv, inv_freq, positions, positions_kind, const_cast<void *>(dq),
                           const_cast<void *>(dk), const_cast<void *>(dv), scale, flags, B, H, Hk,
                           L, d, e, r, dt, stream);
}

la2_status la2_gated_norm(const void *o, const void *gate, int64_t gate_batch, int64_t gate_row,
                          const float *weight, void *u, float eps, unsigned flags, int B, int H,
                          int64_t L, int e, la2_dtype dt, cudaStream_t stream) {
  bool empty;
  la2_status s = gated_checks(flags, B, H, L, e, eps, dt, gate, gate_batch, gate_row, &empty);
  if (s != LA2_OK || empty) return s;
  if (!o || !u || !all_aligned16({o, u, weight})) return LA2_ERR_INVALID;
  const size_t es = esize(dt), n = (size_t)B * H * L * e * es;
  const int64_t D = (int64_t)H * e;
  const size_t nw = (size_t)(flags & LA2_NORM_SHARED_WEIGHT ? e : D) * 4;
  if (out_overlap({{{u, n}, nullptr}},
                  {{o, n}, {gate, rows_span(gate_batch, gate_row, B, L, D, es)}, {weight, nw}}))
    return LA2_ERR_INVALID;
  la2::norm::Gated p{};
  p.o = o;
  p.gate = gate;
  p.u = u;
  p.weight = weight;
  p.gate_b = gate_batch;
  p.gate_l = gate_row;
  p.L = L;
  p.rows = (int64_t)B * L;
  p.H = H;
  p.e = e;
  p.shared = (flags & LA2_NORM_SHARED_WEIGHT) != 0;
  p.gate_vec = rows_vec(gate, gate_batch, gate_row, B, L, es);
  p.eps = eps;
  return to_status(gated_call<false>(p, dt, flags, nullptr, stream));
}

la2_status la2_gated_norm_backward(const void *du, const void *o, const void *gate,
                                   int64_t gate_batch, int64_t gate_row, const float *weight,
                                   void *d_o, void *dgate, int64_t dgate_batch, int64_t dgate_row,
                                   float *dweight, float eps, unsigned flags, int B, int H,
                                   int64_t L, int e, la2_dtype dt, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream) {
  bool empty;
  la2_status s = gated_checks(flags, B, H, L, e, eps, dt, gate, gate_batch, gate_row, &empty);
  if (s != LA2_OK) return s;
  if (dgate_batch < 0 || dgate_row < 0) return LA2_ERR_INVALID;
  const size_t es = esize(dt), n = (size_t)B * H * L * e * es;
  const int64_t D = (int64_t)H * e;
  const size_t nw = (size_t)(flags & LA2_NORM_SHARED_WEIGHT ? e : D) * 4;
  if (!all_aligned16({du, o, weight, d_o, dweight, workspace}) ||
      reinterpret_cast<uintptr_t>(dgate) % es)
    return LA2_ERR_INVALID;
  if (empty) return dweight ? to_status(cudaMemsetAsync(dweight, 0, nw, stream)) : LA2_OK;
  if (!du || !o || !d_o || (gate != nullptr) != (dgate != nullptr)) return LA2_ERR_INVALID;
  const size_t need = dweight ? norm_ws_bytes(LA2_OP_GATED_NORM_BACKWARD, B, H, L, e, e, dt) : 0;
  if (need && (!workspace || workspace_bytes < need)) return LA2_ERR_INVALID;
  if (dgate && !distinct({{dgate_batch, B}, {dgate_row, L}}, D)) return LA2_ERR_INVALID;
  const Span sg = {gate, gate ? rows_span(gate_batch, gate_row, B, L, D, es) : 0};
  const Span sd = {dgate, dgate ? rows_span(dgate_batch, dgate_row, B, L, D, es) : 0};
  if (out_overlap({{{d_o, n}, nullptr}, {sd, nullptr}, {{dweight, nw}, nullptr},
                   {{workspace, need}, nullptr}},
                  {{du, n}, {o, n}, sg, {weight, nw}}))
    return LA2_ERR_INVALID;
  la2::norm::Gated p{};
  p.o = o;
  p.gate = gate;
  p.du = du;
  p.d_o = d_o;
  p.dgate = dgate;
  p.weight = weight;
  p.dw = dweight ? static_cast<float *>(workspace) : nullptr;
  p.gate_b = gate_batch;
  p.gate_l = gate_row;
  p.dgate_b = dgate_batch;
  p.dgate_l = dgate_row;
  p.L = L;
  p.rows = (int64_t)B * L;
  p.H = H;
  p.e = e;
  p.shared = (flags & LA2_NORM_SHARED_WEIGHT) != 0;
  p.gate_vec = rows_vec(gate, gate_batch, gate_row, B, L, es);
  p.dgate_vec = rows_vec(dgate, dgate_batch, dgate_row, B, L, es);
  p.eps = eps;
  return to_status(gated_call<true>(p, dt, flags, dweight, stream));
}

la2_status la2_residual_norm(const void *h, la2_dtype h_dt, const void *y, const float *weight,
                             const float *post_weight, void *h_new, void *n, float alpha,
                             float beta, float eps, unsigned flags, int64_t N, int D,
                             la2_dtype dt, cudaStream_t stream) {
  if (N < 0 || D < 1 || !(eps > 0.f) || (flags & ~(unsigned)LA2_NORM_POST)) return LA2_ERR_INVALID;
  if (!dtype_ok(dt) || !dtype_ok(h_dt) || (h_dt == LA2_BF16 && dt == LA2_F32) || D > kNormMaxCols)
    return LA2_ERR_UNSUPPORTED;
  const bool post = (flags & LA2_NORM_POST) != 0;
  if (post && !y) return LA2_ERR_INVALID;
  if (N == 0) return LA2_OK;
  if (!h || !n || (y != nullptr) != (h_new != nullptr) || (post_weight && !post)) return LA2_ERR_INVALID;
  if (!all_aligned16({h, y, weight, post_weight, h_new, n})) return LA2_ERR_INVALID;
  const size_t bh = (size_t)N * D * esize(h_dt), by = (size_t)N * D * esize(dt), bw = (size_t)D * 4;
  if (out_overlap({{{h_new, bh}, h}, {{n, by}, y}},
                  {{h, bh}, {y, y ? by : 0}, {weight, bw}, {post_weight, bw}}))
    return LA2_ERR_INVALID;
  la2::norm::Residual p{};
  p.h = h;
  p.y = y;
  p.h_new = h_new;
  p.n = n;
  p.weight = weight;
  p.post_weight = post_weight;
  p.rows = N;
  p.D = D;
  p.alpha = alpha;
  p.beta = beta;
  p.eps = eps;
  return to_status(residual_call<false>(p, h_dt, dt, post, nullptr, nullptr, stream));
}

la2_status la2_residual_norm_backward(const void *dn, const void *dh_new, const void *h_new,
                                      la2_dtype h_dt, const void *y, const float *weight,
                                      const float *post_weight, void *dh, void *dy,
                                      float *dweight, float *dpost_weight, float alpha,
                                      float beta, float eps, unsigned flags, int64_t N, int D,
                                      la2_dtype dt, void *workspace, size_t workspace_bytes,
                                      cudaStream_t stream) {
  if (N < 0 || D < 1 || !(eps > 0.f) || (flags & ~(unsigned)LA2_NORM_POST)) return LA2_ERR_INVALID;
  if (!dtype_ok(dt) || !dtype_ok(h_dt) || (h_dt == LA2_BF16 && dt == LA2_F32) || D > kNormMaxCols)
    return LA2_ERR_UNSUPPORTED;
  const bool post = (flags & LA2_NORM_POST) != 0;
  if (!post && (post_weight || dpost_weight)) return LA2_ERR_INVALID;
  const size_t bh = (size_t)N * D * esize(h_dt), by = (size_t)N * D * esize(dt), bw = (size_t)D * 4;
  if (!all_aligned16({dn, dh_new, h_new, y, weight, post_weight, dh, dy, dweight, dpost_weight, workspace}))
    return LA2_ERR_INVALID;
  if (N == 0) {
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, bw, stream);
    if (e == cudaSuccess && dpost_weight) e = cudaMemsetAsync(dpost_weight, 0, bw, stream);
    return to_status(e);
  }
  if (!dn || !h_new || !dh || (post && !y)) return LA2_ERR_INVALID;
  const size_t need =
      dweight || dpost_weight
          ? norm_ws_bytes(LA2_OP_RESIDUAL_NORM_BACKWARD, 1, 1, N, D, D, dt)
          : 0;
  if (need && (!workspace || workspace_bytes < need)) return LA2_ERR_INVALID;
  if (out_overlap({{{dh, bh}, dh_new}, {{dy, dy ? by : 0}, nullptr}, {{dweight, bw}, nullptr},
                   {{dpost_weight, bw}, nullptr}, {{workspace, need}, nullptr}},
                  {{dn, by}, {dh_new, bh}, {h_new, bh}, {post ? y : nullptr, by}, {weight, bw},
                   {post_weight, bw}}))
    return LA2_ERR_INVALID;
  la2::norm::Residual p{};
  p.h = h_new;
  p.y = y;
  p.dn = dn;
  p.dh_new = dh_new;
  p.dh = dh;
  p.dy = dy;
  p.weight = weight;
  p.post_weight = post_weight;
  p.dw = static_cast<float *>(workspace);
  p.rows = N;
  p.D = D;
  p.alpha = alpha;
  p.beta = beta;
  p.eps = eps;
  return to_status(residual_call<true>(p, h_dt, dt, post, dweight, dpost_weight, stream));
}

la2_status la2_pool_copy(const float *from, int from_size, float *to, int to_size,
                         const int32_t *src, const int32_t *dst, int N, int layers, int H, int d,
                         int e, cudaStream_t stream) {
  if (N < 0 || layers < 0 || H < 0 || from_size < 0 || to_size < 0) return LA2_ERR_INVALID;
  if (!shape_supported(d, e, LA2_F32) || N > la2::pool::MAX_MOVES) return LA2_ERR_UNSUPPORTED;
  if (N == 0 || layers == 0 || H == 0) return LA2_OK;
  if (!from || !to || !src || !dst || !all_aligned16({from, to}) ||
      reinterpret_cast<uintptr_t>(src) % 4 || reinterpret_cast<uintptr_t>(dst) % 4)
    return LA2_ERR_INVALID;
  const int64_t bytes = (int64_t)H * d * e * sizeof(float);
  const size_t nf = (size_t)layers * from_size * bytes, nt = (size_t)layers * to_size * bytes;
  if (from == to && from_size != to_size) return LA2_ERR_INVALID;
  if (out_overlap({{{to, nt}, from}}, {{from, nf}, {src, (size_t)N * 4}, {dst, (size_t)N * 4}}))
    return LA2_ERR_INVALID;
  auto kern = la2::pool::copy_kernel;
  static std::atomic<uint64_t> opted{0};
  if (cudaError_t er = opt_in_all_smem(kern, opted)) return to_status(er);
  return to_status(timed(K_POOL_COPY, stream, [&] {
    kern<<<(unsigned)device_sms(), la2::pool::NT, la2::pool::SMEM, stream>>>(
        reinterpret_cast<const char *>(from), reinterpret_cast<char *>(to), src, dst, N, from_size,
        to_size, layers, bytes);
  }));
}

la2_status la2_decode_tokens(const void *q, const void *k, const void *v, const float *lambda,
                             float *kv_pool, const int32_t *slots, int pool_size, void *o,
                             int B, int H, int T, int d, int e, la2_dtype dt,
                             cudaStream_t stream) {
  if (B < 0 || H < 0 || T < 0 || pool_size < 0) return LA2_ERR_INVALID;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_UNSUPPORTED;
  if (!shape_supported(d, e, dt)) return LA2_ERR_UNSUPPORTED;
  const int64_t BH = (int64_t)B * H;
  if (BH == 0 || T == 0) return LA2_OK;
  if (!slots && pool_size < B) return LA2_ERR_INVALID;
  if (!q || !k || !v || !lambda || !kv_pool || !o) return LA2_ERR_INVALID;
  for (const void *p : std::initializer_list<const void *>{
           (const void *)q, (const void *)k, (const void *)v, (const void *)lambda,
           (const void *)kv_pool, (const void *)o})
    if (!aligned16(p)) return LA2_ERR_INVALID;
  if (slots && reinterpret_cast<uintptr_t>(slots) % 4 != 0) return LA2_ERR_INVALID;
  const size_t es = esize(dt);
  std::vector<Span> ins = {{q, BH * T * d * es}, {k, BH * T * d * es}, {v, BH * T * e * es},
                           {lambda, (size_t)H * 4}, {slots, slots ? (size_t)B * 4 : 0}};
  std::vector<Span> outs = {{kv_pool, (size_t)pool_size * H * d * e * sizeof(float)},
                            {o, BH * T * e * es}};
  if (any_overlap(outs, ins)) return LA2_ERR_INVALID;
  // From kDecodeBlockTokens tokens per request on, one block of the chunk
  // schedule (tensor cores, the state read and written once per call) beats
  // the token-by-token register update; the [B,H,T,.] layout is the
  // forward's.
  const int from = g_opt_decode_block.load() > 0 ? g_opt_decode_block.load() : kDecodeBlockTokens;
  if (T >= from && choose_path(d, e, dt) == PATH_TC) {
    Geo g = plan(B, H, T, block_rows(PATH_TC), PATH_TC);
    g.slots = slots;
    g.pool = pool_size;
    g.variant = 0;
    // up to one block per request: one CTA per SM walks (request, head)
    // units back to back (a range of units spans at most two heads)
    const int64_t P = BH < device_sms() ? BH : device_sms();
    if (T <= la2::tc::BLOCK && (BH + P - 1) / P <= B) {
      g.L = T;
      return to_status(la2::tc::decode_units(q, k, v, lambda, kv_pool, o, g, (int)P, stream,
                                             [&](int, auto &&fn) { return timed(K_TC_DECODE_UNITS, stream, fn); }));
    }
    g.S = 1;  // one chunk per request: no workspace
    g.Lc = g.Ls = T;
    g.M = g.Ssub = g.wsS = 1;
    g.nst = 0;
    return to_status(la2::tc::forward(q, k, v, lambda, kv_pool, o, kv_pool, nullptr, g, stream,
                                      [&](int, auto &&fn) { return timed(K_TC_FWD, stream, fn); }));
  }
  cudaError_t err =
      dt == LA2_F32 ? LA2_DISPATCH_DE(d, e, decode, float, q, k, v, lambda, kv_pool, slots,
                                      pool_size, o, B, H, T, stream)
                    : LA2_DISPATCH_DE(d, e, decode, __nv_bfloat16, q, k, v, lambda, kv_pool, slots,
                                      pool_size, o, B, H, T, stream);
  return to_status(err);
}

la2_status la2_last_device_error(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return LA2_ERR_CUDA;
  unsigned int word = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&word, la2::g_error_word, sizeof(word)) != cudaSuccess)
    return LA2_ERR_CUDA;
  if (word && cudaMemcpyToSymbol(la2::g_error_word, &zero, sizeof(zero)) != cudaSuccess)
    return LA2_ERR_CUDA;
  if (word & la2::ERR_TIMEOUT) return LA2_ERR_TIMEOUT;
  if (word & la2::ERR_BOUNDS) return LA2_ERR_INVALID;  // e.g. bad varlen offsets
  if (word) return LA2_ERR_CUDA;
  return LA2_OK;
}

size_t la2_trace_read(uint64_t *out, size_t n) {
  const size_t total = (size_t)la2::kTraceEvents * la2::kTraceBlocks;
  if (!out || n == 0) return total;
  if (cudaDeviceSynchronize() != cudaSuccess) return 0;
  const size_t m = n < total ? n : total;
  if (cudaMemcpyFromSymbol(out, la2::g_trace, m * sizeof(uint64_t)) != cudaSuccess) return 0;
  static const unsigned long long zeros[la2::kTraceEvents * la2::kTraceBlocks] = {0};
  cudaMemcpyToSymbol(la2::g_trace, zeros, sizeof(zeros));
  return m;
}

void la2_profile_enable(int on) { g_prof_on.store(on ? 1 : 0); }

size_t la2_profile_report(char *buf, size_t buf_bytes) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  double ms[K_COUNT] = {0};
  long n[K_COUNT] = {0};
  for (auto &r : g_prof) {
    float t = 0.f;
    if (cudaEventSynchronize(r.b) == cudaSuccess && cudaEventElapsedTime(&t, r.a, r.b) == cudaSuccess) {
      ms[r.kid] += t;
      n[r.kid] += 1;
    }
    g_ev_pool.push_back(r.a);
    g_ev_pool.push_back(r.b);
  }
  g_prof.clear();
  std::string s = "{";
  bool first = true;
  for (int i = 0; i < K_COUNT; i++) {
    if (!n[i]) continue;
    char tmp[160];
    snprintf(tmp, sizeof(tmp), "%s\"%s\": {\"launches\": %ld, \"ms\": %.6f}", first ? "" : ", ",
             kKernelName[i], n[i], ms[i]);
    s += tmp;
    first = false;
  }
  s += "}";
  if (buf && buf_bytes) {
    size_t m = s.size() < buf_bytes - 1 ? s.size() : buf_bytes - 1;
    memcpy(buf, s.data(), m);
    buf[m] = 0;
  }
  return s.size() + 1;
}

}  // extern "C"

// ------------------------------------------------------------------------
// Forward pass for callers that cannot allocate device memory.
//
// Some callers cannot call cudaMalloc or any allocating routine: plug-ins
// whose host framework owns every byte of device memory through its own
// allocator, latency-critical code paths where cudaMalloc's implicit device
// synchronisation would stall other streams, and callbacks that receive only
// device pointers and have no allocator at hand.  For them la2_forward_noalloc
// takes the chunk-boundary states from the fixed array below instead of a
// caller-provided workspace.  The array is part of the library's device
// image: every GPU that loads the library holds it until the process exits.
namespace {

constexpr size_t kNoallocScratchBytes = size_t(32) << 20;  // 32 MiB
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoallocScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_noalloc_mu;
void *g_noalloc_ptr[kMaxDevices] = {nullptr};

// Device address of the array on the current device; looked up once per
// device (host code cannot use the array's name as a device address).
void *noalloc_scratch_ptr() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_noalloc_mu);
  if (!g_noalloc_ptr[dev]) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess) return nullptr;
    g_noalloc_ptr[dev] = p;
  }
  return g_noalloc_ptr[dev];
}

}  // namespace

extern "C" la2_status la2_forward_noalloc(const void *q, const void *k, const void *v,
                                          const float *lambda, const float *kv0, void *o,
                                          float *kv_out, int B, int H, int64_t L, int d, int e,
                                          la2_dtype dt, cudaStream_t stream) {
  // la2_forward's argument checks first: a call it would refuse touches
  // neither the device nor the array.
  bool empty = false;
  const la2_status chk = forward_checks(q, k, v, lambda, kv0, o, kv_out, B, H, L, d, e, dt,
                                        nullptr, 0, &empty);
  if (chk != LA2_OK || empty) return chk;
  // Same plan as la2_forward; refuse plans whose scratch exceeds the array.
  if (L > 0 && la2_workspace_size(LA2_OP_FORWARD, B, H, L, d, e, dt) > kNoallocScratchBytes)
    return LA2_ERR_UNSUPPORTED;
  void *scratch = noalloc_scratch_ptr();
  if (!scratch) return LA2_ERR_CUDA;
  return la2_forward(q, k, v, lambda, kv0, o, kv_out, B, H, L, d, e, dt, scratch,
                     kNoallocScratchBytes, stream);
}
