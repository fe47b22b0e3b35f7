// la2_norm.cuh -- the norms around the attention in a layer.
//
// gated_norm (after the attention): for token (b,t), head h, column j,
//     u = o * rstd * w * a(g),   rstd = 1 / sqrt(mean(o^2) + eps)
// with the mean over the head's e columns or over the token's whole row of
// H * e, a the sigmoid or x * sigmoid(x) of the gate g, and o read head-major
// [B,H,L,e] while u is written token-major [B,L,H*e] (what the output
// projection takes).  With y = o * rstd and up the gradient of u, its
// backward is
//     dg = up * w * y * a'(g),   dw = sum over tokens of up * a * y,
//     do = rstd * (dy - y * mean(dy * y)),   dy = up * w * a.
//
// residual_norm (between two blocks):
//     h' = alpha h + beta p,   p = y  or  y * rstd_y * pw,
//     n  = h' * rstd * w
// and backward, with hn = h' * rstd, yn = y * rstd_y, s = dn * w:
//     dH = dh' + rstd * (s - hn * mean(s * hn)),   dw = sum dn * hn,
//     dh = alpha dH,   dp = beta dH,   dpw = sum dp * yn,
//     dy = dp  or  rstd_y * (z - yn * mean(z * yn)),  z = dp * pw.
//
// n is formed from the sum before it is rounded to the residual stream's
// type (one rounding instead of two); the backward works from the stored h'.
// Every sum and statistic is held in fp32; each output is rounded once.
// All are streaming passes bound by HBM: each input is read once and kept in
// registers across the row's reductions, and the backward needs no saved
// statistics because the row it must read anyway gives them again.  While a
// row is reduced and written the next one is on its way: the gated norm
// (rows made of 128- or 256-byte pieces of the heads) has each thread copy its
// own next values into shared memory, the residual norm (contiguous rows)
// takes them by bulk copies into a ring of rows there.
//
// A row is held by a warp (up to 512 columns), a CTA (up to 8,192: 512 threads
// of two units from 4,097 on, or in the residual norm's forward 256 of four) or
// a cluster of 2 CTAs (4 for rows of more than 16,377 columns that 8 does not
// divide) that add their partial sums through distributed shared memory: a
// thread's share, and so the registers it takes, stays bounded at every width.
//
// The weights' gradients are column sums over all rows.  A thread keeps its
// columns over all rows its CTA walks, so each CTA (or cluster) writes one row
// of partial sums to the workspace, and colsum_kernel adds those rows in a
// fixed order: no atomics, the same result on every run.
//
// Measured on B200 (bf16 unless named, cold L2, of the copy bandwidth):
//   gated norm    65,536 x 4,096, one norm a row     271 us  (91 %)
//                 8,192 x 8,192 per head, fp32       139 us  (89 %)
//                 256 x 8,192, one token a request   9-10 us (the launch and
//                                                    one trip to memory)
//     backward    8,196 x 4,096 per head             66 us   (78 %: 39
//                 instructions a value, issue slots 68 % busy)
//   residual norm 65,536 x 4,096                     351 us  (94 %)
//                 16,384 x 8,192, fp32 stream, post  271 us  (91 %)
//     backward    16,384 x 4,096, fp32 stream, post  201 us  (92 %)
//                 10,000 x 2,000, post               59 us   (62 %: 56
//                 instructions a value, issue slots 62 % busy)
//                 8,000 x 16,384, fp32 stream, post  631 us  (57 %: one ring stage
//                 and one CTA an SM)
//                 10,000 x 2,001, post               71 us   (52 %)
//                 65,536 x 256, 65,536 x 64, post    61, 52 us (51, 15 %: lanes
//                 or their second units idle, no row ahead in a warp)
#pragma once

#include <type_traits>

#include "la2_bulk.cuh"
#include "la2_common.cuh"
#include "la2_fmap.cuh"
#include "la2_norm_plan.h"
#include "la2_sm100.cuh"

namespace la2 {
namespace norm {

using namespace sm100;

// ------------------------------------------------------------ eight values
// What a thread holds of a row: units of eight neighbours, moved as 16-byte
// pieces and worked on as four pairs (mul2, fma2).
template <typename T> struct Raw {
  static constexpr int N = 8 * sizeof(T) / 16;
  uint4 r[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; i++) r[i] = make_uint4(0, 0, 0, 0);
  }
  // apart: values from one 16-byte piece to the next (fp32: 4 = neighbours)
  __device__ __forceinline__ void load(const T *p, int apart = 4) {
#pragma unroll
    for (int i = 0; i < N; i++) r[i] = fmap::ld_stream(p + i * apart);
  }
  __device__ __forceinline__ void load_shared(const T *p) {
#pragma unroll
    for (int i = 0; i < N; i++) r[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  // values lo <= i < hi alone, from an address with the element's alignment;
  // the others are 0
  __device__ __forceinline__ void load_some(const T *p, int lo, int hi) {
    using W = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
    const W *q = reinterpret_cast<const W *>(p);
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = i >= lo && i < hi ? q[i] : 0u;
    if constexpr (sizeof(T) == 4) {
      r[0] = make_uint4(v[0], v[1], v[2], v[3]);
      r[N - 1] = make_uint4(v[4], v[5], v[6], v[7]);
    } else {
      r[0] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
  }
  // all eight at any alignment, the last four from p + apart on
  __device__ __forceinline__ void load_any(const T *p, int apart) {
    load_some(p, 0, 4);
    Raw<T> q;
    q.load_some(p + apart - 4, 4, 8);
#pragma unroll
    for (int i = 0; i < N; i++)
      r[i] = make_uint4(r[i].x | q.r[i].x, r[i].y | q.r[i].y, r[i].z | q.r[i].z, r[i].w | q.r[i].w);
  }
  // all but the values lo <= i < hi set to 0
  __device__ __forceinline__ void keep(int lo, int hi) {
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; i++) m[i] = i >= lo && i < hi ? 0xffffffffu : 0u;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; i++) {
        r[i].x &= m[4 * i];
        r[i].y &= m[4 * i + 1];
        r[i].z &= m[4 * i + 2];
        r[i].w &= m[4 * i + 3];
      }
    } else {
      r[0].x &= (m[0] & 0xffffu) | m[1] << 16;
      r[0].y &= (m[2] & 0xffffu) | m[3] << 16;
      r[0].z &= (m[4] & 0xffffu) | m[5] << 16;
      r[0].w &= (m[6] & 0xffffu) | m[7] << 16;
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    constexpr int M = 8 / N;
#pragma unroll
    for (int i = 0; i < N; i++) {
      float g[M];
      fmap::vec16<T>::unpack(r[i], g);
#pragma unroll
      for (int j = 0; j < M; j++) f[i * M + j] = g[j];
    }
  }
  __device__ __forceinline__ void get2(float2 (&f)[4]) const {
    float g[8];
    get(g);
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = make_float2(g[2 * i], g[2 * i + 1]);
  }
};

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8], int apart = 4) {
  constexpr int N = fmap::vec16<T>::N;
#pragma unroll
  for (int i = 0; i < 8 / N; i++) {
    float g[N];
#pragma unroll
    for (int j = 0; j < N; j++) g[j] = f[i * N + j];
    fmap::st_stream(p + i * apart, fmap::vec16<T>::pack(g));
  }
}
// the values lo <= i < hi alone
template <typename T>
__device__ __forceinline__ void store_some(T *p, const float2 (&x)[4], int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 8; i++)
    if (i >= lo && i < hi) io<T>::st(p + i, i % 2 ? x[i / 2].y : x[i / 2].x);
}
// apart: from the first to the fifth value (4: neighbours)
template <typename T>
__device__ __forceinline__ void store_pairs(T *p, const float2 (&x)[4], int apart = 4) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = x[i].x;
    f[2 * i + 1] = x[i].y;
  }
  store8(p, f, apart);
}
// vec: the address is 16-byte aligned (else the element's alignment only)
template <typename T>
__device__ __forceinline__ void store_any(T *p, const float2 (&x)[4], bool vec, int apart) {
  if (vec) {
    store_pairs(p, x, apart);
  } else {
    store_some(p, x, 0, 4);
    store_some(p + apart - 4, x, 4, 8);
  }
}
// 16 bytes into shared memory, behind the thread's back.
__device__ __forceinline__ void copy16_async(void *to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
// Weights: fp32 (null: ones), read by every row of a CTA, so through the cache.
__device__ __forceinline__ void weights8(const float *w, float2 (&f)[4], int apart = 4) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = make_float2(1.f, 1.f);
  } else {
    const float4 x = __ldg(reinterpret_cast<const float4 *>(w));
    const float4 y = __ldg(reinterpret_cast<const float4 *>(w + apart));
    f[0] = make_float2(x.x, x.y);
    f[1] = make_float2(x.z, x.w);
    f[2] = make_float2(y.x, y.y);
    f[3] = make_float2(y.z, y.w);
  }
}
// the weights lo <= i < hi alone (the others 0), at any alignment
__device__ __forceinline__ void weights_some(const float *w, float2 (&f)[4], int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float x = i >= lo && i < hi ? (w ? __ldg(w + i) : 1.f) : 0.f;
    if (i % 2) f[i / 2].y = x;
    else f[i / 2].x = x;
  }
}
__device__ __forceinline__ void copy(const float2 (&x)[4], float2 (&y)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i++) y[i] = x[i];
}
// row = b * L + t; a 64-bit division only where the numbers need one.
__device__ __forceinline__ void split_row(int64_t row, int64_t L, int64_t &b, int64_t &t) {
  if ((uint64_t)(row | L) >> 32 == 0) {
    const uint32_t q = (uint32_t)row / (uint32_t)L;
    b = q;
    t = (uint32_t)row - q * (uint32_t)L;
  } else {
    b = row / L;
    t = row - b * L;
  }
}

// ------------------------------------------------------------ pairs
// Two fp32 operations in one instruction (each rounded as the single one is):
// the norms' backward passes come near the rate at which instructions issue.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

// ------------------------------------------------------------ reductions
// Sum of K values over LANES neighbouring lanes of a warp; every lane gets it.
template <int K, int LANES>
__device__ __forceinline__ void lanes_sum(float (&x)[K]) {
#pragma unroll
  for (int m = LANES / 2; m > 0; m /= 2) {
#pragma unroll
    for (int k = 0; k < K; k++) x[k] += __shfl_xor_sync(0xffffffffu, x[k], m);
  }
}
// Sums of K (5 to 8) values over a warp, one to every four lanes: lanes 4 k to
// 4 k + 3 get value k's.  Each of the first three steps hands half of the
// values over, so it takes 9 shuffles instead of 5 K.
template <int K>
__device__ __forceinline__ float warp_sums(const float (&x)[K]) {
  const int lane = threadIdx.x % 32;
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; k++) v[k] = k < K ? x[k] : 0.f;
#pragma unroll
  for (int half = 4; half > 0; half /= 2) {
    const bool upper = lane & (4 * half);
#pragma unroll
    for (int i = 0; i < half; i++) {
      const float give = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * half);
    }
  }
  float y[1] = {v[0]};
  lanes_sum<1, 4>(y);
  return y[0];
}
// and back: every lane gets all K
template <int K>
__device__ __forceinline__ void spread(float (&x)[K], float y) {
#pragma unroll
  for (int k = 0; k < K; k++) x[k] = __shfl_sync(0xffffffffu, y, 4 * k);
}
__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// One value into the shared memory of CTA `rank`, counted by the barrier at
// the same place there.
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, uint32_t rank, float x) {
  asm volatile(
      "{\n\t.reg .b32 a, b;\n\t"
      "mapa.shared::cluster.u32 a, %0, %2;\n\t"
      "mapa.shared::cluster.u32 b, %1, %2;\n\t"
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.f32 [a], %3, [b];\n\t}" ::"r"(to),
      "r"(bar), "r"(rank), "f"(x)
      : "memory");
}

// Sum of K values over the threads that share a row: a warp (TPR = 32), the
// CTA (cl = 1) or the cl CTAs of a cluster, each of which is sent all warps'
// partial sums.  Two generations of partial sums are used in turn, so one
// wait per sum is enough: a thread that runs ahead writes the other
// generation, and cannot come back to this one before it has the sum in
// between, to which every warp contributes only after reading this one.
// Within a cluster the values are counted by an mbarrier of the receiving
// CTA: a barrier of the whole cluster would also wait for the row's stores
// (16,384 columns in fp32 by clusters of two, forward: 430 us so, 358 by
// counting).  A wait that gives up leaves a stale sum; the
// caller's loop runs on, so that no barrier is missed, and the error word
// tells the host.
// HAND_OVER: the form for many values that issues fewer instructions but waits
// longer for each (residual norm's backward: 3 to 5 % faster where a row is
// held by one unit a thread or by 512 threads, 4 % slower with two units and
// 256).
template <int TPR, int K, int MAXCL, bool HAND_OVER = false>
struct RowSum {
  static constexpr int NW = TPR / 32;
  struct Shared {
    uint64_t bars[2];
    float red[2][K][TPR > 32 ? MAXCL * NW : 1];
  };
  uint32_t uses = 0;
  // before the first sum, by all threads; a barrier of the CTA (cl = 1: none
  // is needed) and of the cluster follow
  __device__ __forceinline__ void init(Shared &s, int cl) {
    if (TPR > 32 && cl > 1 && threadIdx.x == 0) {
      for (int g = 0; g < 2; g++) {
        mbar_init(smem_u32(&s.bars[g]), 1);
        fence_mbar_init();
        mbar_expect_tx(smem_u32(&s.bars[g]), (uint32_t)(cl * NW * K * sizeof(float)));
      }
    }
  }
  __device__ __forceinline__ void operator()(float (&x)[K], Shared &s, int cl, int rank,
                                             volatile int *abort) {
    if constexpr (HAND_OVER) {
      float y = warp_sums(x);
      if constexpr (TPR > 32) {
        const int w = threadIdx.x / 32, l = threadIdx.x % 32, turn = uses & 1, k = l / 4, j = l % 4;
        if (cl == 1) {
          if (j == 0 && k < K) s.red[turn][k][w] = y;
          __syncthreads();
        } else {
          const uint32_t bar = smem_u32(&s.bars[turn]);
          // lane j of value k's four sends it to CTAs j and j + 4
          for (int to = j; to < cl; to += 4)
            if (k < K) send(smem_u32(&s.red[turn][k][rank * NW + w]), bar, to, y);
          mbar_wait(bar, (uses >> 1) & 1, abort);
          if (threadIdx.x == 0) mbar_expect_tx(bar, (uint32_t)(cl * NW * K * sizeof(float)));
        }
        float z[1] = {0.f};
        if (k < K)
          for (int i = j; i < cl * NW; i += 4) z[0] += s.red[turn][k][i];
        lanes_sum<1, 4>(z);
        y = z[0];
        uses++;
      }
      spread(x, y);
      return;
    }
    lanes_sum<K, 32>(x);
    if constexpr (TPR > 32) {
      const int w = threadIdx.x / 32, l = threadIdx.x % 32, turn = uses & 1;
      if (cl == 1) {
        if (l == 0) {
#pragma unroll
          for (int k = 0; k < K; k++) s.red[turn][k][w] = x[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; k++) x[k] = s.red[turn][k][l % NW];
        lanes_sum<K, NW>(x);
      } else {
        const uint32_t bar = smem_u32(&s.bars[turn]);
        if (l < cl) {
#pragma unroll
          for (int k = 0; k < K; k++) send(smem_u32(&s.red[turn][k][rank * NW + w]), bar, l, x[k]);
        }
        mbar_wait(bar, (uses >> 1) & 1, abort);
        if (threadIdx.x == 0) mbar_expect_tx(bar, (uint32_t)(cl * NW * K * sizeof(float)));
#pragma unroll
        for (int k = 0; k < K; k++) {
          x[k] = 0.f;
          for (int j = l; j < cl * NW; j += 32) x[k] += s.red[turn][k][j];
        }
        lanes_sum<K, 32>(x);
      }
      uses++;
    }
  }
};

// Lets the kernel after this one be set up (colsum_kernel; it waits for this
// one's end all the same).
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------ gate
// 1 / (1 + e^-g) of a pair, by the approximate exponential (of base 2) and
// reciprocal.  Values of 16 bits: with no more than these, relative error below
// (|g| + 4) 2^-23 down to g = -87, from the exponent's rounding; below that the
// reciprocal is 0 instead of less than 2^-126.  Values of 32 bits:
// e^-|g| = 2^x (1 + y ln 2), x + y = -|g| log2 e with x rounded and y the rest of
// the product (fma) and of the constant; the sigmoid is 1 or that over 1 + e^-|g|,
// a number of [1, 2], whose reciprocal takes one step of Newton's.  Errors in units
// of 2^-24: the power 4, 1 + y ln 2, the sum, the reciprocal and the product
// 1 each, 8 at every g at which the result is normal; subnormals come down to
// the last, 2^-149 (g = -103).  Measured, 8,192 rows of 64 heads x 128 in fp32
// forward, and the largest error for gates of scale 40 in these units: 139 us and
// 6; with no more than the two instructions 137 us and 64; by expf and a division
// 148 us and 5.
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 g) {
  if constexpr (sizeof(T) == 4) {
    // nothing is left of the power below -150; NaN stays
    float2 a, e;
    asm("max.NaN.f32 %0, %1, 0fC3160000;" : "=f"(a.x) : "f"(-fabsf(g.x)));
    asm("max.NaN.f32 %0, %1, 0fC3160000;" : "=f"(a.y) : "f"(-fabsf(g.y)));
    const float2 x = mul2(a, pair(1.44269504f));
    const float2 y = fma2(a, pair(1.92596303e-8f), fma2(a, pair(1.44269504f), make_float2(-x.x, -x.y)));
    asm("ex2.approx.f32 %0, %1;" : "=f"(e.x) : "f"(x.x));
    asm("ex2.approx.f32 %0, %1;" : "=f"(e.y) : "f"(x.y));
    e = fma2(mul2(e, y), pair(0.693147182f), e);
    const float2 d = fma2(e, pair(1.f), pair(1.f));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    r = fma2(r, fma2(make_float2(-d.x, -d.y), r, pair(1.f)), r);
    return mul2(r, make_float2(g.x >= 0.f ? 1.f : e.x, g.y >= 0.f ? 1.f : e.y));
  }
  float2 s = mul2(g, pair(-1.44269504f));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(s.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(s.y));
  s = fma2(s, pair(1.f), pair(1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(s.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(s.y));
  return s;
}

// ------------------------------------------------------------ gated norm
enum Gate { GATE_NONE, GATE_SIGMOID, GATE_SILU };

struct Gated {
  const void *o, *gate, *du;
  void *u, *d_o, *dgate;
  const float *weight;
  float *dw;                 // partial sums of the weight's gradient, or null
  int64_t gate_b, gate_l;    // strides of the gate's batch and row, in values
  int64_t dgate_b, dgate_l;
  int64_t L, rows;           // rows = B * L tokens
  int H, e;
  int shared;                // weight [e], the same for every head
  int gate_vec, dgate_vec;   // rows of the gate (its gradient) 16-byte aligned
  int tpr_shift;             // per head: log2 of the threads side by side in a row
  int cols, cl;              // columns of a CTA; row: CTAs that share a row
  float eps;
};

// Rows on their way per thread, and CTAs on an SM.  (65,536 x 4,096 forward:
// two rows and four CTAs 270 us, three or four rows, so three CTAs, 287; the
// backward per head with three rows and two CTAs 66, with three CTAs, which
// spill, 89.)
template <bool GRAD, Gate GATE>
constexpr int gated_streams() { return 1 + GRAD + (GATE != GATE_NONE); }
template <typename T, int NV>
constexpr int gated_stages() { return NV == 2 ? 2 : 3; }
template <typename T, bool GRAD, int NT>
constexpr int gated_ctas() { return (GRAD || sizeof(T) == 4 ? 2 : 4) / (NT == 512 ? 2 : 1); }
template <typename T, bool GRAD, Gate GATE, int NT, int NV>
constexpr size_t gated_smem() {
  const size_t ring = (size_t)NT * NV * 8 * sizeof(T) * gated_streams<GRAD, GATE>() * gated_stages<T, NV>();
  const size_t sums = GRAD ? (size_t)NT * NV * 8 * sizeof(float) : 0;  // in its place, at the end
  return ring > sums ? ring : sums;
}

// ROW: one norm spans the H * e values of a token (else one per head, of E =
// e columns; a row's kernel takes every e, its E is 0).
// Threads of a CTA: per head, 2^tpr_shift side by side over `cols` columns
// (heads; slice blockIdx.y) and NT >> tpr_shift tokens; ROW, a warp or the
// CTA per row, NV vectors each, slice = the CTA's rank in its cluster.
template <typename T, int E, bool ROW, bool GRAD, Gate GATE, int NT, int TPR, int NV>
__global__ void __launch_bounds__(NT, gated_ctas<T, GRAD, NT>())
gated_kernel(const __grid_constant__ Gated p) {
  constexpr int V = 8, P = V / 2, LPH = ROW ? 32 : E / V;
  // a unit: 8 neighbours, or in fp32 twice 4 of them, 32 columns apart, so that
  // 8 lanes move whole lines.  The second four have neither bounds nor a head of
  // their own: c0 and the CTA's width are multiples of a block (gated_block).
  constexpr int APART = norm_plan::gated_apart(sizeof(T));
  constexpr int S = gated_stages<T, NV>();
  constexpr bool HOLD = !(GRAD && NV == 2);  // the weights, in registers throughout
  using Sum = RowSum<ROW ? TPR : 32, GRAD ? 2 : 1, norm_plan::most_cl(false)>;
  __shared__ typename Sum::Shared red;
  extern __shared__ __align__(128) char dyn[];
  Sum row_sum;
  const int cl = ROW ? p.cl : 1;
  const int rank = ROW && TPR > 32 && cl > 1 ? (int)cluster_rank() : 0;
  const int tpr = ROW ? TPR : 1 << p.tpr_shift, rpc = ROW ? NT / TPR : NT >> p.tpr_shift;
  const int sub = ROW ? threadIdx.x / TPR : threadIdx.x >> p.tpr_shift;
  const int tr = ROW ? threadIdx.x % TPR : threadIdx.x & (tpr - 1);
  const int e = ROW ? p.e : E, D = p.H * e;
  const int c0 = (ROW ? rank : (int)blockIdx.y) * p.cols;
  const int end = c0 + p.cols < D ? c0 + p.cols : D;
  const float inv = 1.f / (float)(ROW ? D : e);
  __shared__ int abort;
  if (ROW && TPR > 32 && cl > 1) {
    if (threadIdx.x == 0) abort = 0;
    row_sum.init(red, cl);
    __syncthreads();
    cluster_arrive_wait();  // every CTA's barriers are there
  }

  int c[NV];
  int64_t at_o[NV];
  float2 held[HOLD ? NV : 1][P], acc[GRAD ? NV : 1][P];
  auto weights = [&](int col, float2 (&w)[P]) {
    if (col < end) {
      weights8(p.weight ? p.weight + (p.shared ? col % e : col) : nullptr, w, APART);
    } else {
#pragma unroll
      for (int i = 0; i < P; i++) w[i] = pair(0.f);
    }
  };
#pragma unroll
  for (int n = 0; n < NV; n++) {
    c[n] = c0 + norm_plan::gated_unit(sizeof(T), n * tpr + tr);
    at_o[n] = (int64_t)(c[n] / e) * p.L * e + c[n] % e;
    if constexpr (HOLD) weights(c[n], held[n]);
    if constexpr (GRAD) {
#pragma unroll
      for (int i = 0; i < P; i++) acc[n][i] = pair(0.f);
    }
  }
  // Where a row's values are.  A thread's rows are `step` apart, so the next
  // row's place is the last one's plus a constant, and another at the end of
  // a batch.
  const int64_t step = (int64_t)(gridDim.x / cl) * rpc;
  const int64_t r0 = (int64_t)(blockIdx.x / cl) * rpc;
  struct Place {
    int64_t row, t, o, g, dg;
  };
  Place at;
  int64_t sb, st;
  {
    int64_t b;
    at.row = r0 + sub;
    split_row(at.row, p.L, b, at.t);
    at.o = (b * p.H * p.L + at.t) * e;
    at.g = b * p.gate_b + at.t * p.gate_l;
    at.dg = b * p.dgate_b + at.t * p.dgate_l;
    split_row(step, p.L, sb, st);
  }
  const int64_t step_o = (sb * p.H * p.L + st) * e, wrap_o = (int64_t)(p.H - 1) * p.L * e;
  const int64_t step_g = sb * p.gate_b + st * p.gate_l, wrap_g = p.gate_b - p.L * p.gate_l;
  const int64_t step_dg = sb * p.dgate_b + st * p.dgate_l, wrap_dg = p.dgate_b - p.L * p.dgate_l;
  auto advance = [&](Place &a) {
    a.row += step;
    a.t += st;
    a.o += step_o;
    a.g += step_g;
    if constexpr (GRAD) a.dg += step_dg;
    if (a.t >= p.L) {
      a.t -= p.L;
      a.o += wrap_o;
      a.g += wrap_g;
      if constexpr (GRAD) a.dg += wrap_dg;
    }
  };
  // The rows ahead: this thread's vectors of each stream (o, the gate, du) in
  // its own places of shared memory, so it alone waits for them and no
  // barrier is needed.  Lanes stand 16 bytes apart.
  constexpr int N = Raw<T>::N, STREAMS = gated_streams<GRAD, GATE>();
  const bool gate_ahead = GATE != GATE_NONE && p.gate_vec;
  auto slot = [&](int stage, int stream, int n, int i) {
    return reinterpret_cast<uint4 *>(dyn) + (((stage * STREAMS + stream) * NV + n) * N + i) * NT + threadIdx.x;
  };
  auto fetch = [&](int stage, const Place &a) {
    if (a.row < p.rows) {
#pragma unroll
      for (int n = 0; n < NV; n++) {
        if (c[n] >= end) continue;
        const T *x = static_cast<const T *>(p.o) + a.o + at_o[n];
        const T *g = static_cast<const T *>(p.gate) + a.g + c[n];
        const T *up = static_cast<const T *>(p.du) + a.row * D + c[n];
#pragma unroll
        for (int i = 0; i < N; i++) {
          copy16_async(slot(stage, 0, n, i), x + i * APART);
          if (GRAD) copy16_async(slot(stage, 1, n, i), up + i * APART);
          if (gate_ahead) copy16_async(slot(stage, STREAMS - 1, n, i), g + i * APART);
        }
      }
    }
    copies_commit();
  };
  struct {
    Raw<T> x[NV], g[GATE != GATE_NONE ? NV : 1], up[GRAD ? NV : 1];
  } cur;
  auto take = [&](int stage, const Place &a) {
#pragma unroll
    for (int n = 0; n < NV; n++) {
      if (a.row < p.rows && c[n] < end) {
#pragma unroll
        for (int i = 0; i < N; i++) {
          cur.x[n].r[i] = *slot(stage, 0, n, i);
          if constexpr (GRAD) cur.up[n].r[i] = *slot(stage, 1, n, i);
          if constexpr (GATE != GATE_NONE)
            if (gate_ahead) cur.g[n].r[i] = *slot(stage, STREAMS - 1, n, i);
        }
        if constexpr (GATE != GATE_NONE)
          if (!gate_ahead) cur.g[n].load_any(static_cast<const T *>(p.gate) + a.g + c[n], APART);
      } else {
        cur.x[n].clear();
        if constexpr (GATE != GATE_NONE) cur.g[n].clear();
        if constexpr (GRAD) cur.up[n].clear();
      }
    }
  };
  Place to = at;  // of the row at hand; `at` is S - 1 rows on
#pragma unroll
  for (int i = 0; i < S - 1; i++) {
    fetch(i, at);
    advance(at);
  }
  int stage = 0, last = S - 1;
  for (int64_t r = r0; r < p.rows; r += step) {
    fetch(last, at);
    advance(at);
    copies_wait<S - 1>();
    take(stage, to);
    last = stage;
    stage = stage + 1 == S ? 0 : stage + 1;
    // statistics of the row or head; in the backward also sum(dy * o)
    float2 s[GRAD && GATE != GATE_NONE ? NV : 1][P];
    float sum[NV][GRAD ? 2 : 1];
#pragma unroll
    for (int n = 0; n < NV; n++) {
      float2 q = pair(0.f), k = pair(0.f), x[P], g[P], up[P], w[P];
      cur.x[n].get2(x);
      if constexpr (GRAD) {
        if constexpr (HOLD) copy(held[n], w);
        else weights(c[n], w);
        cur.up[n].get2(up);
        if constexpr (GATE != GATE_NONE) cur.g[n].get2(g);
      }
#pragma unroll
      for (int i = 0; i < P; i++) {
        q = fma2(x[i], x[i], q);
        if constexpr (GRAD) {
          float2 dy = mul2(up[i], w[i]);
          if constexpr (GATE != GATE_NONE) {
            s[n][i] = sigmoid2<T>(g[i]);
            dy = mul2(dy, s[n][i]);
          }
          if constexpr (GATE == GATE_SILU) dy = mul2(dy, g[i]);
          k = fma2(dy, x[i], k);
        }
      }
      sum[n][0] = q.x + q.y;
      if constexpr (GRAD) sum[n][1] = k.x + k.y;
    }
    if constexpr (ROW) {
#pragma unroll
      for (int n = 1; n < NV; n++)
#pragma unroll
        for (int k = 0; k < (GRAD ? 2 : 1); k++) sum[0][k] += sum[n][k];
      row_sum(sum[0], red, cl, rank, &abort);
#pragma unroll
      for (int n = 1; n < NV; n++)
#pragma unroll
        for (int k = 0; k < (GRAD ? 2 : 1); k++) sum[n][k] = sum[0][k];
    } else {
#pragma unroll
      for (int n = 0; n < NV; n++) lanes_sum<GRAD ? 2 : 1, LPH>(sum[n]);
    }
    if (to.row < p.rows) {
#pragma unroll
      for (int n = 0; n < NV; n++) {
        if (c[n] >= end) continue;
        const float2 rstd = pair(rsqrtf(fmaf(sum[n][0], inv, p.eps)));
        float2 x[P], g[P], w[P];
        cur.x[n].get2(x);
        if constexpr (GATE != GATE_NONE) cur.g[n].get2(g);
        if constexpr (HOLD) copy(held[n], w);
        else weights(c[n], w);
        if constexpr (!GRAD) {
#pragma unroll
          for (int i = 0; i < P; i++) {
            x[i] = mul2(mul2(x[i], rstd), w[i]);
            if constexpr (GATE != GATE_NONE) x[i] = mul2(x[i], sigmoid2<T>(g[i]));
            if constexpr (GATE == GATE_SILU) x[i] = mul2(x[i], g[i]);
          }
          store_pairs(static_cast<T *>(p.u) + to.row * D + c[n], x, APART);
        } else {
          const float2 m = pair(-sum[n][1] * rstd.x * inv);  // -mean(dy * y)
          float2 up[P], dg[P];
          cur.up[n].get2(up);
#pragma unroll
          for (int i = 0; i < P; i++) {
            const float2 y = mul2(x[i], rstd);
            float2 dy = mul2(up[i], w[i]), uy = mul2(up[i], y);
            if constexpr (GATE != GATE_NONE) {
              const float2 sg = s[n][i], rest = fma2(sg, pair(-1.f), pair(1.f));
              dg[i] = mul2(mul2(dy, y), sg);
              dg[i] = mul2(dg[i], GATE == GATE_SILU ? fma2(g[i], rest, pair(1.f)) : rest);
              const float2 a = GATE == GATE_SILU ? mul2(g[i], sg) : sg;
              dy = mul2(dy, a);
              uy = mul2(uy, a);
            }
            acc[n][i] = fma2(uy, pair(1.f), acc[n][i]);
            x[i] = mul2(rstd, fma2(y, m, dy));
          }
          store_pairs(static_cast<T *>(p.d_o) + to.o + at_o[n], x, APART);
          if constexpr (GATE != GATE_NONE)
            store_any(static_cast<T *>(p.dgate) + to.dg + c[n], dg, p.dgate_vec, APART);
        }
      }
    }
    advance(to);
  }
  if (ROW && TPR > 32 && cl > 1) cluster_arrive_wait();  // none leaves while another sends
  if constexpr (GRAD) {
    if (!p.dw) return;
    launch_dependents();
    float *acc_s = reinterpret_cast<float *>(dyn);
    copies_wait<0>();
    __syncthreads();
    // the CTA's partial sums: over the tokens side by side and, for a weight
    // that the heads share, over the heads it covers
#pragma unroll
    for (int n = 0; n < NV; n++)
#pragma unroll
      for (int i = 0; i < P; i++)
        reinterpret_cast<float2 *>(acc_s)[(threadIdx.x * NV + n) * P + i] = acc[n][i];
    __syncthreads();
    const int width = end - c0, out = p.shared ? e : width;
    const int64_t group = blockIdx.x / cl;
    for (int j = threadIdx.x; j < out; j += NT) {
      float sum = 0.f;
      for (int k = j; k < width; k += out) {
        const int vec = sizeof(T) == 2 ? k / V : k / 64 * 8 + k % 32 / 4;
        const int i = sizeof(T) == 2 ? k % V : k % 64 / 32 * 4 + k % 4;
        const int n = vec / tpr, lane = vec % tpr;
        for (int q = 0; q < rpc; q++) sum += acc_s[((q * tpr + lane) * NV + n) * V + i];
      }
      if (p.shared)
        p.dw[(group * gridDim.y + blockIdx.y) * e + j] = sum;
      else
        p.dw[group * D + c0 + j] = sum;
    }
  }
}

// ------------------------------------------------------------ residual norm
struct Residual {
  const void *h, *y;         // forward: the stream and the block's output
  const void *dn, *dh_new;   // backward: gradients of n and (or null) of h'
  void *h_new, *n;           // forward's outputs (h_new null: n = norm(h))
  void *dh, *dy;
  const float *weight, *post_weight;
  float *dw, *dpw;           // partial sums, or null
  int64_t rows;
  int D, cols, cl;           // columns, of a CTA; CTAs that share a row
  int stages;                // rows that the ring holds (1 or 2)
  float alpha, beta, eps;
};

// Rows wider than a warp holds come through a ring of one or two rows in
// shared memory, filled by thread 0 with one bulk copy per stream.  A row's
// stage is given back by the block barrier of its first reduction (in a
// cluster, the one after it), which no thread passes before all have taken
// their values into registers; so even one stage is filled again while its
// last row is worked on.  The weights stand in front of the ring: with two
// CTAs on an SM little is left of the L1 cache, and read from L2 for every row
// they cost as much as a stream.
//
// ODD rows (D not a multiple of 8) begin anywhere between two 16-byte pieces.
// Their units are laid from the piece that a row begins in, so that all but
// the first and the last still move whole: a unit's values stand `lead`
// places before its columns, lead = (row D) mod 8, and values before the row
// or behind it are masked.  The host lets a thread's rows lie a multiple of 8
// apart, so its lead, and with it its columns, its weights and its partial
// sums, stay the same.
constexpr int kRingHead = 128;  // barriers, in front of the ring

// The values of one row that a thread holds: forward h, y; backward h', dn,
// dh', y (dh' and y where they are).
template <typename T, typename R, bool GRAD, bool POST, int NV>
struct RowData {
  Raw<R> h[NV], g[GRAD ? NV : 1];
  Raw<T> s[GRAD ? NV : 1], y[(GRAD && !POST) ? 1 : NV];
};

// TPR threads hold a row, NV units each.
template <typename T, typename R, bool GRAD, bool POST, bool ODD, int NT, int TPR, int NV>
__global__ void __launch_bounds__(NT, NT == 512 ? 1 : 2) residual_kernel(const __grid_constant__ Residual p) {
  constexpr bool RING = TPR > 32;
  constexpr bool HAS_Y = !GRAD || POST;  // y may be read
  constexpr int RPC = NT / TPR, P = 4;
  using Sum = RowSum<TPR, !GRAD ? 1 : POST ? 6 : 2, norm_plan::most_cl(ODD),
                     GRAD && POST && (NV == 1 || NT == 512)>;
  __shared__ typename Sum::Shared red;
  extern __shared__ __align__(128) char dyn[];
  Sum sum;
  const int cl = TPR > 32 ? p.cl : 1, rank = cl > 1 ? (int)cluster_rank() : 0;
  const int sub = threadIdx.x / TPR, tr = threadIdx.x % TPR;
  const float inv = 1.f / (float)p.D;
  const T *y = static_cast<const T *>(p.y);
  const int64_t step = (int64_t)(gridDim.x / cl) * RPC;
  const int64_t first = (int64_t)(blockIdx.x / cl) * RPC;
  // this CTA's places: `cols` of them from c0 on, of which [lo, hi) are columns
  const int lead = ODD ? (int)((first + sub) % 8) * (p.D % 8) % 8 : 0;
  const int c0 = rank * p.cols;
  const int lo = ODD && lead > c0 ? lead - c0 : 0;
  const int hi = lead + p.D - c0 < p.cols ? lead + p.D - c0 : p.cols;
  __shared__ int gave_up;
  volatile int *abort = &gave_up;
  if constexpr (TPR > 32) {
    if (threadIdx.x == 0) gave_up = 0;
    sum.init(red, cl);
    __syncthreads();
    if (cl > 1) cluster_arrive_wait();  // every CTA's barriers are there
  }

  // unit n: its first place; whether it holds columns, and only columns
  auto col = [&](int n) { return (n * TPR + tr) * 8; };
  auto on = [&](int c) { return c < hi && (!ODD || c + 8 > lo); };
  auto whole = [&](int c) { return !ODD || (c >= lo && c + 8 <= hi); };
  auto put = [&](auto *row, int c, const float2 (&x)[P]) {
    if (whole(c)) store_pairs(row + c, x);
    else store_some(row + c, x, lo - c, hi - c);
  };
  auto take_shared = [&](auto &raw, const auto *row, int c) {
    raw.load_shared(row + c);
    if (!whole(c)) raw.keep(lo - c, hi - c);
  };
  auto take = [&](auto &raw, const auto *row, int c) {
    if (whole(c)) raw.load(row + c);
    else raw.load_some(row + c, lo - c, hi - c);
  };
  // the weights (0: w, 1: pw) of a unit from memory
  auto weights_of = [&](int which, int c, float2 (&x)[P]) {
    const float *w = which ? p.post_weight : p.weight;
    if (w) w += c0 + c - lead;
    if (!ODD) weights8(w, x);
    else weights_some(w, x, lo - c, hi - c);
  };
  // and from where they are kept: a warp's in registers; else in shared
  // memory, the first four and the last four of a unit apart, so that a warp
  // reads whole lines
  float2 mine[RING ? 1 : POST ? 2 : 1][RING ? 1 : NV][P];
  float4 *held = reinterpret_cast<float4 *>(dyn + kRingHead);
  const int units = p.cols / 8;
  auto weights = [&](int which, int n, float2 (&x)[P]) {
    if constexpr (RING) {
      const int u = col(n) / 8;
      const float4 a = held[2 * which * units + u], b = held[(2 * which + 1) * units + u];
      x[0] = make_float2(a.x, a.y);
      x[1] = make_float2(a.z, a.w);
      x[2] = make_float2(b.x, b.y);
      x[3] = make_float2(b.z, b.w);
    } else {
      copy(mine[which][n], x);
    }
  };

  // a stage of the ring: h | dh' | dn | y, the ones that are
  const int64_t total = p.rows * p.D;
  const bool has_g = GRAD && p.dh_new, has_y = HAS_Y && y;
  const uint32_t bars = smem_u32(dyn);
  const uint32_t hb = p.cols * sizeof(R), yb = p.cols * sizeof(T);
  const uint32_t at_g = hb, at_s = at_g + (has_g ? hb : 0), at_y = at_s + (GRAD ? yb : 0);
  const uint32_t stage_bytes = at_y + (has_y ? yb : 0);
  char *ring = dyn + kRingHead + (POST ? 2 : 1) * sizeof(float) * p.cols;
  // Whole pieces from place 0 on.  Behind the end of the tensor (the last row
  // of ODD ones) the values of the last piece come one by one instead.
  auto fetch_one = [&](const auto *x, int64_t at, int n, char *to, uint32_t bar) -> uint32_t {
    using X = typename std::remove_const<typename std::remove_pointer<decltype(x)>::type>::type;
    constexpr int PIECE = 16 / sizeof(X);
    if (ODD && at + n > total) {
      n = (int)(total - at) / PIECE * PIECE;
      for (int i = n; i < hi; i++) reinterpret_cast<X *>(to)[i] = x[at + i];
    }
    if (!ODD || n) bulk::load(smem_u32(to), x + at, (uint32_t)(n * sizeof(X)), bar);
    return (uint32_t)(n * sizeof(X));
  };
  auto fetch = [&](int64_t row, int st) {  // thread 0
    const uint32_t bar = bars + st * 8;
    char *to = ring + st * stage_bytes;
    const int64_t at = row * p.D - lead + c0;
    const int n = ODD ? (hi + 7) / 8 * 8 : hi;
    if constexpr (!ODD)
      mbar_expect_tx(bar, (uint32_t)hi * ((has_g ? 2 : 1) * sizeof(R) + (GRAD + has_y) * sizeof(T)));
    uint32_t bytes = fetch_one(static_cast<const R *>(p.h), at, n, to, bar);
    if (has_g) bytes += fetch_one(static_cast<const R *>(p.dh_new), at, n, to + at_g, bar);
    if (GRAD) bytes += fetch_one(static_cast<const T *>(p.dn), at, n, to + at_s, bar);
    if (has_y) bytes += fetch_one(y, at, n, to + at_y, bar);
    if constexpr (ODD) mbar_expect_tx(bar, bytes);
  };
  if constexpr (RING) {
    if (threadIdx.x == 0) {
      mbar_init(bars, 1);
      mbar_init(bars + 8, 1);
      fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      if (first < p.rows) fetch(first, 0);
      if (p.stages > 1 && first + step < p.rows) fetch(first + step, 1);
    }
    for (int i = threadIdx.x; i < (POST ? 2 : 1) * units; i += NT) {
      const int which = i >= units, u = i - which * units;
      if (on(u * 8)) {
        float2 x[P];
        weights_of(which, u * 8, x);
        held[2 * which * units + u] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        held[(2 * which + 1) * units + u] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
      }
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int k = 0; k < (POST ? 2 : 1); k++)
#pragma unroll
      for (int n = 0; n < NV; n++) {
        if (on(col(n))) {
          weights_of(k, col(n), mine[k][n]);
        } else {
#pragma unroll
          for (int i = 0; i < P; i++) mine[k][n][i] = pair(0.f);
        }
      }
  }
  const int shift = p.stages - 1;

  float2 aw[GRAD ? NV : 1][P], ap[GRAD && POST ? NV : 1][P];
  if constexpr (GRAD) {
#pragma unroll
    for (int n = 0; n < NV; n++)
#pragma unroll
      for (int i = 0; i < P; i++) {
        aw[n][i] = pair(0.f);
        if constexpr (POST) ap[n][i] = pair(0.f);
      }
  }

  int64_t it = 0;
  for (int64_t r0 = first; r0 < p.rows; r0 += step, it++) {
    const int64_t row = r0 + sub;
    const bool live = row < p.rows;
    const int64_t at = row * p.D - lead + c0;
    RowData<T, R, GRAD, POST, NV> d;
    const int st = (int)it & shift;
    const char *stage = ring + st * stage_bytes;
    // on a timeout the values are stale, but every thread stays in step with
    // the barriers below; the error word tells the host
    if constexpr (RING) mbar_wait(bars + st * 8, (uint32_t)(it >> shift) & 1, abort);
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int c = col(n);
      if (live && on(c)) {
        if constexpr (RING) {
          take_shared(d.h[n], reinterpret_cast<const R *>(stage), c);
          if constexpr (GRAD) {
            if (has_g) take_shared(d.g[n], reinterpret_cast<const R *>(stage + at_g), c);
            else d.g[n].clear();
            take_shared(d.s[n], reinterpret_cast<const T *>(stage + at_s), c);
          }
          if constexpr (HAS_Y) {
            if (has_y) take_shared(d.y[n], reinterpret_cast<const T *>(stage + at_y), c);
          }
        } else {
          take(d.h[n], static_cast<const R *>(p.h) + at, c);
          if constexpr (GRAD) {
            if (has_g) take(d.g[n], static_cast<const R *>(p.dh_new) + at, c);
            else d.g[n].clear();
            take(d.s[n], static_cast<const T *>(p.dn) + at, c);
          }
          if constexpr (HAS_Y) {
            if (has_y) take(d.y[n], y + at, c);
          }
        }
      } else {
        d.h[n].clear();
        if constexpr (GRAD) {
          d.g[n].clear();
          d.s[n].clear();
        }
        if constexpr (HAS_Y) d.y[n].clear();
      }
    }
    // after the row's first barrier: its stage is free
    auto refill = [&] {
      if constexpr (RING) {
        if (cl > 1) __syncthreads();
        const int64_t later = r0 + p.stages * step;
        if (threadIdx.x == 0 && later < p.rows) fetch(later, st);
      }
    };
    if constexpr (!GRAD) {
      float2 x[NV][P];
      bool refilled = false;
#pragma unroll
      for (int n = 0; n < NV; n++) d.h[n].get2(x[n]);
      if (y) {
        float2 ry = pair(p.beta);
        if constexpr (POST) {
          float2 q2 = pair(0.f);
#pragma unroll
          for (int n = 0; n < NV; n++) {
            float2 z[P];
            d.y[n].get2(z);
#pragma unroll
            for (int i = 0; i < P; i++) q2 = fma2(z[i], z[i], q2);
          }
          float q[1] = {q2.x + q2.y};
          sum(q, red, cl, rank, abort);
          refill();
          refilled = true;
          ry = pair(rsqrtf(fmaf(q[0], inv, p.eps)) * p.beta);
        }
        const float2 al = pair(p.alpha);
#pragma unroll
        for (int n = 0; n < NV; n++) {
          const int c = col(n);
          if (!(live && on(c))) continue;
          float2 z[P], w[P];
          d.y[n].get2(z);
          if constexpr (POST) weights(1, n, w);
#pragma unroll
          for (int i = 0; i < P; i++) {
            if constexpr (POST) z[i] = mul2(z[i], w[i]);
            x[n][i] = fma2(ry, z[i], mul2(al, x[n][i]));
          }
          put(static_cast<R *>(p.h_new) + at, c, x[n]);
        }
      }
      float2 q2 = pair(0.f);
#pragma unroll
      for (int n = 0; n < NV; n++)
#pragma unroll
        for (int i = 0; i < P; i++) q2 = fma2(x[n][i], x[n][i], q2);
      float q[1] = {q2.x + q2.y};
      sum(q, red, cl, rank, abort);
      if (!refilled) refill();
      const float2 rstd = pair(rsqrtf(fmaf(q[0], inv, p.eps)));
#pragma unroll
      for (int n = 0; n < NV; n++) {
        const int c = col(n);
        if (!(live && on(c))) continue;
        float2 w[P];
        weights(0, n, w);
#pragma unroll
        for (int i = 0; i < P; i++) w[i] = mul2(w[i], mul2(x[n][i], rstd));
        put(static_cast<T *>(p.n) + at, c, w);
      }
    } else {
      // Sums of h'^2, s h' and, with a norm on y, of y^2 and pw y times each of
      // dh', s and h': dH is a combination of these three whose factors the
      // first sums give, so the mean that dy needs comes out of the same
      // reduction.
      float2 q2[POST ? 6 : 2];
#pragma unroll
      for (int i = 0; i < (POST ? 6 : 2); i++) q2[i] = pair(0.f);
#pragma unroll
      for (int n = 0; n < NV; n++) {
        if (!on(col(n))) continue;
        float2 w[P], x[P], s[P];
        weights(0, n, w);
        d.h[n].get2(x);
        d.s[n].get2(s);
#pragma unroll
        for (int i = 0; i < P; i++) {
          s[i] = mul2(s[i], w[i]);
          q2[0] = fma2(x[i], x[i], q2[0]);
          q2[1] = fma2(s[i], x[i], q2[1]);
        }
        if constexpr (POST) {
          float2 z[P], g[P];
          d.y[n].get2(z);
          d.g[n].get2(g);
          weights(1, n, w);
#pragma unroll
          for (int i = 0; i < P; i++) {
            const float2 pz = mul2(z[i], w[i]);
            q2[2] = fma2(z[i], z[i], q2[2]);
            q2[3] = fma2(pz, g[i], q2[3]);
            q2[4] = fma2(pz, s[i], q2[4]);
            q2[5] = fma2(pz, x[i], q2[5]);
          }
        }
      }
      float q[POST ? 6 : 2];
#pragma unroll
      for (int i = 0; i < (POST ? 6 : 2); i++) q[i] = q2[i].x + q2[i].y;
      sum(q, red, cl, rank, abort);
      refill();
      const float r = rsqrtf(fmaf(q[0], inv, p.eps)), mean = -q[1] * r * inv;  // -mean(s hn)
      const float2 rstd = pair(r), m = pair(mean);
      const float2 al = pair(p.alpha), be = pair(p.beta);
      float2 ry = pair(1.f), mz = pair(0.f);  // mz: -mean((dp pw) yn) / rms(y)
      if constexpr (POST) {
        const float y1 = rsqrtf(fmaf(q[2], inv, p.eps));
        ry = pair(y1);
        mz = pair(-p.beta * y1 * y1 * inv * fmaf(r, fmaf(mean * r, q[5], q[4]), q[3]));
      }
#pragma unroll
      for (int n = 0; n < NV; n++) {
        const int c = col(n);
        if (!(live && on(c))) continue;
        float2 w[P], x[P], s[P], g[P];
        weights(0, n, w);
        d.h[n].get2(x);
        d.s[n].get2(s);
        d.g[n].get2(g);
#pragma unroll
        for (int i = 0; i < P; i++) {
          const float2 hn = mul2(x[i], rstd);
          aw[n][i] = fma2(s[i], hn, aw[n][i]);
          const float2 dH = fma2(rstd, fma2(hn, m, mul2(s[i], w[i])), g[i]);
          x[i] = mul2(al, dH);
          g[i] = mul2(be, dH);  // dp
        }
        put(static_cast<R *>(p.dh) + at, c, x);
        if constexpr (POST) {
          float2 z[P];
          d.y[n].get2(z);
          weights(1, n, w);
#pragma unroll
          for (int i = 0; i < P; i++) {
            ap[n][i] = fma2(g[i], mul2(z[i], ry), ap[n][i]);
            g[i] = mul2(ry, fma2(z[i], mz, mul2(g[i], w[i])));
          }
        }
        if (p.dy) put(static_cast<T *>(p.dy) + at, c, g);
      }
    }
  }
  if (cl > 1) cluster_arrive_wait();  // none leaves while another sends
  if constexpr (RING) {
    // after a timeout: let the rows in flight land before the ring is released
    if (threadIdx.x == 0 && *abort) {
      volatile int none = 0;
      for (int64_t j = it > p.stages ? it - p.stages : 0; j < it; j++)
        mbar_wait(bars + ((uint32_t)j & shift) * 8, (uint32_t)(j >> shift) & 1, &none);
    }
  }
  if constexpr (GRAD) {
    launch_dependents();
    // one row of partial sums for the CTA's columns; warps that walked rows
    // side by side are added up first
    const int64_t group = blockIdx.x / cl;
    auto flush = [&](float *to, const float2 (&acc)[NV][P]) {
      if (!to) return;
      to += group * p.D;
      if constexpr (RPC == 1) {
#pragma unroll
        for (int n = 0; n < NV; n++) {
          const int c = col(n);
          if (on(c)) put(to + (c0 - lead), c, acc[n]);
        }
      } else {
        float *acc_s = reinterpret_cast<float *>(dyn) + sub * p.D;
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NV; n++) {
          const int c = col(n);
          if (on(c)) store_some(acc_s - lead + c, acc[n], lo - c, hi - c);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.D; c += NT) {
          float a = 0.f;
#pragma unroll
          for (int k = 0; k < RPC; k++) a += reinterpret_cast<float *>(dyn)[k * p.D + c];
          to[c] = a;
        }
      }
    };
    flush(p.dw, aw);
    if constexpr (POST) flush(p.dpw, ap);
  }
}

// Column sums of two arrays of partial sums [rows][cols] (either may be
// null): 32 columns x 32 rows of threads, each thread's rows in order, then
// the 32 sums by one warp per column.  It is launched while the kernel that
// writes the partial sums still runs, and waits for its end.
constexpr int kSumCols = 32, kSumRows = 32;
__global__ void __launch_bounds__(kSumCols *kSumRows)
colsum_kernel(const float *a, const float *b, float *ya, float *yb, int rows, int cols) {
  __shared__ float s[kSumRows][kSumCols + 1];
  const float *x = blockIdx.y ? b : a;
  float *y = blockIdx.y ? yb : ya;
  if (!y) return;
  const int tc = threadIdx.x % kSumCols, tr = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + tc;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float sum = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int r = tr; r < rows; r += kSumRows) sum += __ldcg(x + (int64_t)r * cols + c);
  }
  s[tr][tc] = sum;
  __syncthreads();
  float q[1] = {s[tc][tr]};  // warp tr: the column's 32 sums
  lanes_sum<1, 32>(q);
  if (tc == 0 && blockIdx.x * kSumCols + tr < cols) y[blockIdx.x * kSumCols + tr] = q[0];
}

}  // namespace norm
}  // namespace la2
