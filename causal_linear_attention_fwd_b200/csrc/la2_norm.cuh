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
// (rows made of 128- or 256-byte pieces of the heads) loads it into
// registers, the residual norm (contiguous rows) by bulk copies into a ring
// of rows in shared memory.
//
// A row is held by a warp (up to 512 columns), a CTA (up to 4,096; 2,048 where
// values move one by one) or a cluster of 2 to 8 CTAs that add their partial
// sums through distributed shared memory: a thread's share, and so the
// registers it takes, stays the same at every width.
//
// The weights' gradients are column sums over all rows.  A thread keeps its
// columns over all rows its CTA walks, so each CTA (or cluster) writes one row
// of partial sums to the workspace, and colsum_kernel adds those rows in a
// fixed order: no atomics, the same result on every run.
#pragma once

#include "la2_common.cuh"
#include "la2_fmap.cuh"
#include "la2_sm100.cuh"

namespace la2 {
namespace norm {

using namespace sm100;

// ------------------------------------------------------------ vectors
// V values of T as they are in memory; V = 8 moves 16-byte pieces, V = 1
// single values (rows that no vector divides).
template <typename T, int V> struct Raw;
template <typename T> struct Raw<T, 8> {
  static constexpr int N = 8 * sizeof(T) / 16;
  uint4 r[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; i++) r[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < N; i++) r[i] = fmap::ld_stream(reinterpret_cast<const uint4 *>(p) + i);
  }
  __device__ __forceinline__ void load_shared(const T *p) {
#pragma unroll
    for (int i = 0; i < N; i++) r[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  // from an address with the element's alignment only
  __device__ __forceinline__ void load_any(const T *p, bool vec) {
    if (vec) {
      load(p);
    } else if constexpr (sizeof(T) == 4) {
      const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
#pragma unroll
      for (int i = 0; i < N; i++) r[i] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
    } else {
      const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
      r[0] = make_uint4(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16,
                        q[4] | (uint32_t)q[5] << 16, q[6] | (uint32_t)q[7] << 16);
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
template <typename T> struct Raw<T, 1> {
  T r;
  __device__ __forceinline__ void clear() { r = T(0.f); }
  __device__ __forceinline__ void load(const T *p) { r = *p; }
  __device__ __forceinline__ void load_shared(const T *p) { r = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = io<T>::ld(&r); }
};

template <typename T, int V>
__device__ __forceinline__ void ldv(const T *p, float (&f)[V]) {
  Raw<T, V> r;
  r.load(p);
  r.get(f);
}
template <typename T, int V>
__device__ __forceinline__ void stv(T *p, const float (&f)[V]) {
  if constexpr (V == 1) {
    io<T>::st(p, f[0]);
  } else {
    constexpr int N = fmap::vec16<T>::N;
#pragma unroll
    for (int i = 0; i < V / N; i++) {
      float g[N];
#pragma unroll
      for (int j = 0; j < N; j++) g[j] = f[i * N + j];
      fmap::st_stream(p + i * N, fmap::vec16<T>::pack(g));
    }
  }
}
// vec: the address is 16-byte aligned (else the element's alignment only)
template <typename T>
__device__ __forceinline__ void stv2(T *p, const float2 (&x)[4], bool vec) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = x[i].x;
    f[2 * i + 1] = x[i].y;
  }
  if (vec) {
    stv<T, 8>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) io<T>::st(p + i, f[i]);
  }
}
// Weights: fp32, read by every row of a CTA, so through the cache.
template <int V>
__device__ __forceinline__ void ldw(const float *w, int c, float (&f)[V]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < V; i++) f[i] = 1.f;
  } else if constexpr (V == 1) {
    f[0] = __ldg(w + c);
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; i++) {
      const float4 x = __ldg(reinterpret_cast<const float4 *>(w + c) + i);
      f[4 * i] = x.x;
      f[4 * i + 1] = x.y;
      f[4 * i + 2] = x.z;
      f[4 * i + 3] = x.w;
    }
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
// the backward of the gated norm is bound by the instructions it issues.
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
__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void store_in_cta(float *p, uint32_t rank, float x) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(smem_u32(p)),
      "r"(rank), "f"(x)
      : "memory");
}

// Sum of K values over the threads that share a row: a warp (TPR = 32), the
// CTA (cl = 1) or the cl CTAs of a cluster, each of which is given all warps'
// partial sums.  Two generations of partial sums are used in turn, so one
// barrier per sum is enough: a thread that runs ahead writes the other
// generation, and cannot come back to this one before every thread has
// passed the barrier in between.
constexpr int kMaxCluster = 8;
template <int TPR, int K>
struct RowSum {
  static constexpr int NW = TPR / 32;
  using Shared = float[2][K][TPR > 32 ? kMaxCluster * NW : 1];
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&x)[K], Shared &red, int cl, int rank) {
    lanes_sum<K, 32>(x);
    if constexpr (TPR > 32) {
      const int w = threadIdx.x / 32, l = threadIdx.x % 32;
      if (cl == 1) {
        if (l == 0) {
#pragma unroll
          for (int k = 0; k < K; k++) red[turn][k][w] = x[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; k++) x[k] = red[turn][k][l % NW];
        lanes_sum<K, NW>(x);
      } else {
        if (l < cl) {
#pragma unroll
          for (int k = 0; k < K; k++) store_in_cta(&red[turn][k][rank * NW + w], l, x[k]);
        }
        cluster_arrive_wait();
#pragma unroll
        for (int k = 0; k < K; k++) {
          x[k] = 0.f;
          for (int j = l; j < cl * NW; j += 32) x[k] += red[turn][k][j];
        }
        lanes_sum<K, 32>(x);
      }
      turn ^= 1;
    }
  }
};

// Lets the kernel after this one be set up (colsum_kernel; it waits for this
// one's end all the same).
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------ gate
// 1 / (1 + e^-g) of a pair.  e^-g overflows to infinity for g below -88,
// where the sigmoid is 0 to fp32 (the quotient gives it).  Values that will
// be rounded to bf16 take the approximate exponential (of base 2) and
// reciprocal, a few 2^-23 off against the rounding's 2^-9; fp32 takes the
// exact ones.
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 g) {
  if constexpr (sizeof(T) == 4) {
    return make_float2(1.f / (1.f + expf(-g.x)), 1.f / (1.f + expf(-g.y)));
  } else {
    float2 s = mul2(g, pair(-1.44269504f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(s.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(s.y));
    s = fma2(s, pair(1.f), pair(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(s.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(s.y));
    return s;
  }
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

// ROW: one norm spans the H * e values of a token (else one per head, of E =
// e columns; a row's kernel takes every e, its E is 0).
// Threads of a CTA: per head, 2^tpr_shift side by side over `cols` columns
// (heads; slice blockIdx.y) and NT >> tpr_shift tokens; ROW, a warp or the
// CTA per row, NV vectors each, slice = the CTA's rank in its cluster.
template <typename T, int E, bool ROW, bool GRAD, Gate GATE, int NT, int TPR, int NV>
__global__ void __launch_bounds__(NT, GRAD || sizeof(T) == 4 ? 2 : 3)
gated_kernel(const __grid_constant__ Gated p) {
  constexpr int V = 8, P = V / 2, LPH = ROW ? 32 : E / V;
  // what fits the registers: the next row ahead, the weights held throughout
  constexpr bool AHEAD = !(GRAD && NV == 2 && sizeof(T) == 4), HOLD = !(GRAD && NV == 2);
  using Sum = RowSum<ROW ? TPR : 32, GRAD ? 2 : 1>;
  __shared__ typename Sum::Shared red;
  extern __shared__ float acc_s[];
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
  if (ROW && TPR > 32 && cl > 1) cluster_arrive_wait();  // every CTA's shared memory is there

  int c[NV];
  int64_t at_o[NV];
  float2 held[HOLD ? NV : 1][P], acc[GRAD ? NV : 1][P];
  auto weights = [&](int col, float2 (&w)[P]) {
    float f[V];
    if (col < end) {
      ldw<V>(p.weight, p.shared ? col % e : col, f);
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) f[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < P; i++) w[i] = make_float2(f[2 * i], f[2 * i + 1]);
  };
#pragma unroll
  for (int n = 0; n < NV; n++) {
    c[n] = c0 + (n * tpr + tr) * V;
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
  struct Loaded {
    Raw<T, V> x[NV], g[GATE != GATE_NONE ? NV : 1], up[GRAD ? NV : 1];
  };
  auto load = [&](Loaded &d, const Place &a) {
    const bool live = a.row < p.rows;
#pragma unroll
    for (int n = 0; n < NV; n++) {
      if (live && c[n] < end) {
        d.x[n].load(static_cast<const T *>(p.o) + a.o + at_o[n]);
        if constexpr (GATE != GATE_NONE)
          d.g[n].load_any(static_cast<const T *>(p.gate) + a.g + c[n], p.gate_vec);
        if constexpr (GRAD) d.up[n].load(static_cast<const T *>(p.du) + a.row * D + c[n]);
      } else {
        d.x[n].clear();
        if constexpr (GATE != GATE_NONE) d.g[n].clear();
        if constexpr (GRAD) d.up[n].clear();
      }
    }
  };
  Loaded cur, next;
  Place to = at;  // of the row at hand; `at` is the next one's
  if (AHEAD) load(cur, at);
  for (int64_t r = r0; r < p.rows; r += step) {
    advance(at);
    if constexpr (AHEAD) load(next, at);
    else load(cur, to);
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
      row_sum(sum[0], red, cl, rank);
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
          stv2(static_cast<T *>(p.u) + to.row * D + c[n], x, true);
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
          stv2(static_cast<T *>(p.d_o) + to.o + at_o[n], x, true);
          if constexpr (GATE != GATE_NONE)
            stv2(static_cast<T *>(p.dgate) + to.dg + c[n], dg, p.dgate_vec);
        }
      }
    }
    if constexpr (AHEAD) cur = next;
    to = at;
  }
  if constexpr (GRAD) {
    if (!p.dw) return;
    launch_dependents();
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
        const int vec = k / V, n = vec / tpr, lane = vec % tpr;
        for (int q = 0; q < rpc; q++) sum += acc_s[((q * tpr + lane) * NV + n) * V + k % V];
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
  float alpha, beta, eps;
};

// Rows wider than a warp holds come through a ring of two rows in shared
// memory, filled by thread 0 with one bulk copy per stream.  A row's stage is
// given back by the block barrier of its first reduction, which no thread
// passes before all have taken their values into registers.
constexpr int kRingHead = 128;  // barriers and the flag, in front of the ring

__device__ __forceinline__ void bulk_row(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// The values of one row that a thread holds: forward h, y; backward h', dn,
// dh', y (dh' and y where they are).
template <typename T, typename R, bool GRAD, bool POST, int V, int NV>
struct RowData {
  Raw<R, V> h[NV], g[GRAD ? NV : 1];
  Raw<T, V> s[GRAD ? NV : 1], y[(GRAD && !POST) ? 1 : NV];
};

template <typename T, typename R, bool GRAD, bool POST, int V, int NT, int TPR, int NV>
__global__ void __launch_bounds__(NT, 2) residual_kernel(const __grid_constant__ Residual p) {
  constexpr bool RING = V == 8 && TPR > 32;
  constexpr bool HAS_Y = !GRAD || POST;  // y may be read
  constexpr int RPC = NT / TPR;
  using Sum = RowSum<TPR, GRAD ? 3 : 1>;
  using Sum1 = RowSum<TPR, 1>;
  __shared__ typename Sum::Shared red;
  __shared__ typename Sum1::Shared red1;
  extern __shared__ __align__(128) char dyn[];
  Sum sum;
  Sum1 sum1;
  const int cl = TPR > 32 ? p.cl : 1, rank = cl > 1 ? (int)cluster_rank() : 0;
  const int sub = threadIdx.x / TPR, tr = threadIdx.x % TPR;
  const int c0 = rank * p.cols;
  const int width = p.D - c0 < p.cols ? p.D - c0 : p.cols;  // this CTA's columns
  const float inv = 1.f / (float)p.D;
  const T *y = static_cast<const T *>(p.y);
  const int64_t step = (int64_t)(gridDim.x / cl) * RPC;
  int64_t r0 = (int64_t)(blockIdx.x / cl) * RPC;
  if (cl > 1) cluster_arrive_wait();  // every CTA's shared memory is there

  const uint32_t hb = (uint32_t)width * sizeof(R), yb = (uint32_t)width * sizeof(T);
  const bool has_g = GRAD && p.dh_new, has_y = HAS_Y && y;
  const uint32_t bars = smem_u32(dyn);
  volatile int *abort = reinterpret_cast<volatile int *>(dyn + 64);
  // a stage: h | g | s | y, the ones that are
  const uint32_t at_g = hb, at_s = at_g + (has_g ? hb : 0), at_y = at_s + (GRAD ? yb : 0);
  const uint32_t row_bytes = at_y + (has_y ? yb : 0), stage_bytes = (row_bytes + 127) / 128 * 128;
  char *ring = dyn + kRingHead;
  auto fetch = [&](int64_t row, int st) {  // thread 0
    const uint32_t bar = bars + st * 8, dst = smem_u32(ring) + st * stage_bytes;
    const int64_t at = row * p.D + c0;
    mbar_expect_tx(bar, row_bytes);
    bulk_row(dst, static_cast<const R *>(p.h) + at, hb, bar);
    if (has_g) bulk_row(dst + at_g, static_cast<const R *>(p.dh_new) + at, hb, bar);
    if (GRAD) bulk_row(dst + at_s, static_cast<const T *>(p.dn) + at, yb, bar);
    if (has_y) bulk_row(dst + at_y, y + at, yb, bar);
  };
  if constexpr (RING) {
    if (threadIdx.x == 0) {
      mbar_init(bars, 1);
      mbar_init(bars + 8, 1);
      *abort = 0;
      fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      if (r0 < p.rows) fetch(r0, 0);
      if (r0 + step < p.rows) fetch(r0 + step, 1);
    }
  }

  float aw[GRAD ? NV : 1][V], ap[GRAD && POST ? NV : 1][V];
  if constexpr (GRAD) {
#pragma unroll
    for (int n = 0; n < NV; n++)
#pragma unroll
      for (int i = 0; i < V; i++) {
        aw[n][i] = 0.f;
        if constexpr (POST) ap[n][i] = 0.f;
      }
  }

  for (int64_t it = 0; r0 < p.rows; r0 += step, it++) {
    const int64_t row = r0 + sub;
    const bool live = row < p.rows;
    const int64_t at = row * p.D + c0;
    RowData<T, R, GRAD, POST, V, NV> d;
    const int st = (int)(it & 1);
    const char *stage = ring + st * stage_bytes;
    // on a timeout the values are stale, but every thread stays in step with
    // the barriers below; the error word tells the host
    if constexpr (RING) mbar_wait(bars + st * 8, (uint32_t)(it >> 1) & 1, abort);
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int c = (n * TPR + tr) * V;
      if (live && c < width) {
        if constexpr (RING) {
          d.h[n].load_shared(reinterpret_cast<const R *>(stage) + c);
          if constexpr (GRAD) {
            if (has_g) d.g[n].load_shared(reinterpret_cast<const R *>(stage + at_g) + c);
            else d.g[n].clear();
            d.s[n].load_shared(reinterpret_cast<const T *>(stage + at_s) + c);
          }
          if constexpr (HAS_Y) {
            if (has_y) d.y[n].load_shared(reinterpret_cast<const T *>(stage + at_y) + c);
          }
        } else {
          d.h[n].load(static_cast<const R *>(p.h) + at + c);
          if constexpr (GRAD) {
            if (has_g) d.g[n].load(static_cast<const R *>(p.dh_new) + at + c);
            else d.g[n].clear();
            d.s[n].load(static_cast<const T *>(p.dn) + at + c);
          }
          if constexpr (HAS_Y) {
            if (has_y) d.y[n].load(y + at + c);
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
        if (threadIdx.x == 0 && r0 + 2 * step < p.rows) fetch(r0 + 2 * step, st);
      }
    };
    if constexpr (!GRAD) {
      float x[NV][V];
      bool refilled = false;
#pragma unroll
      for (int n = 0; n < NV; n++) d.h[n].get(x[n]);
      if (y) {
        float ry = 1.f;
        if constexpr (POST) {
          float q[1] = {0.f};
#pragma unroll
          for (int n = 0; n < NV; n++) {
            float z[V];
            d.y[n].get(z);
#pragma unroll
            for (int i = 0; i < V; i++) q[0] = fmaf(z[i], z[i], q[0]);
          }
          sum1(q, red1, cl, rank);
          refill();
          refilled = true;
          ry = rsqrtf(fmaf(q[0], inv, p.eps));
        }
#pragma unroll
        for (int n = 0; n < NV; n++) {
          const int c = (n * TPR + tr) * V;
          if (!(live && c < width)) continue;
          float z[V], w[V];
          d.y[n].get(z);
          if constexpr (POST) ldw<V>(p.post_weight, c0 + c, w);
#pragma unroll
          for (int i = 0; i < V; i++) {
            const float q = POST ? z[i] * ry * w[i] : z[i];
            x[n][i] = fmaf(p.beta, q, p.alpha * x[n][i]);
          }
          stv<R, V>(static_cast<R *>(p.h_new) + at + c, x[n]);
        }
      }
      float q[1] = {0.f};
#pragma unroll
      for (int n = 0; n < NV; n++)
#pragma unroll
        for (int i = 0; i < V; i++) q[0] = fmaf(x[n][i], x[n][i], q[0]);
      sum(q, red, cl, rank);
      if (!refilled) refill();
      const float rstd = rsqrtf(fmaf(q[0], inv, p.eps));
#pragma unroll
      for (int n = 0; n < NV; n++) {
        const int c = (n * TPR + tr) * V;
        if (!(live && c < width)) continue;
        float w[V];
        ldw<V>(p.weight, c0 + c, w);
#pragma unroll
        for (int i = 0; i < V; i++) w[i] *= x[n][i] * rstd;
        stv<T, V>(static_cast<T *>(p.n) + at + c, w);
      }
    } else {
      // sums of h'^2, (dn w) h' and, with a norm on y, y^2
      float q[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < NV; n++) {
        const int c = (n * TPR + tr) * V;
        if (c >= width) continue;
        float w[V], x[V], s[V];
        ldw<V>(p.weight, c0 + c, w);
        d.h[n].get(x);
        d.s[n].get(s);
#pragma unroll
        for (int i = 0; i < V; i++) {
          q[0] = fmaf(x[i], x[i], q[0]);
          q[1] = fmaf(s[i] * w[i], x[i], q[1]);
        }
        if constexpr (POST) {
          float z[V];
          d.y[n].get(z);
#pragma unroll
          for (int i = 0; i < V; i++) q[2] = fmaf(z[i], z[i], q[2]);
        }
      }
      sum(q, red, cl, rank);
      refill();
      const float rstd = rsqrtf(fmaf(q[0], inv, p.eps));
      const float m = q[1] * rstd * inv;  // mean(s hn)
      const float ry = POST ? rsqrtf(fmaf(q[2], inv, p.eps)) : 1.f;
      float k[1] = {0.f};                 // sum of (dp pw) yn
      float dp[NV][V];
#pragma unroll
      for (int n = 0; n < NV; n++) {
        const int c = (n * TPR + tr) * V;
        if (!(live && c < width)) continue;
        float w[V], x[V], s[V], g[V];
        ldw<V>(p.weight, c0 + c, w);
        d.h[n].get(x);
        d.s[n].get(s);
        d.g[n].get(g);
#pragma unroll
        for (int i = 0; i < V; i++) {
          const float hn = x[i] * rstd;
          aw[n][i] = fmaf(s[i], hn, aw[n][i]);
          const float dH = fmaf(rstd, fmaf(-hn, m, s[i] * w[i]), g[i]);
          x[i] = p.alpha * dH;
          dp[n][i] = p.beta * dH;
        }
        stv<R, V>(static_cast<R *>(p.dh) + at + c, x);
        if constexpr (POST) {
          float z[V];
          d.y[n].get(z);
          ldw<V>(p.post_weight, c0 + c, w);
#pragma unroll
          for (int i = 0; i < V; i++) {
            const float yn = z[i] * ry;
            ap[n][i] = fmaf(dp[n][i], yn, ap[n][i]);
            dp[n][i] *= w[i];
            k[0] = fmaf(dp[n][i], yn, k[0]);
          }
        }
      }
      if (p.dy) {
        if constexpr (POST) sum1(k, red1, cl, rank);
        const float mz = k[0] * inv;
#pragma unroll
        for (int n = 0; n < NV; n++) {
          const int c = (n * TPR + tr) * V;
          if (!(live && c < width)) continue;
          if constexpr (POST) {
            float z[V];
            d.y[n].get(z);
#pragma unroll
            for (int i = 0; i < V; i++) dp[n][i] = ry * fmaf(-z[i] * ry, mz, dp[n][i]);
          }
          stv<T, V>(static_cast<T *>(p.dy) + at + c, dp[n]);
        }
      }
    }
  }
  if constexpr (RING) {
    // after a timeout: let the rows in flight land before the ring is released
    if (threadIdx.x == 0 && *abort) {
      volatile int none = 0;
      const int64_t n = (p.rows - (int64_t)(blockIdx.x / cl) + step - 1) / step;  // rows fetched
      for (int64_t j = n > 2 ? n - 2 : 0; j < n; j++)
        mbar_wait(bars + (uint32_t)(j & 1) * 8, (uint32_t)(j >> 1) & 1, &none);
    }
  }
  if constexpr (GRAD) {
    launch_dependents();
    // one row of partial sums for the CTA's columns; warps that walked rows
    // side by side are added up first
    float *out[2] = {p.dw, POST ? p.dpw : nullptr};
    const int64_t group = blockIdx.x / cl;
#pragma unroll
    for (int j = 0; j < (POST ? 2 : 1); j++) {
      if (!out[j]) continue;
      float *to = out[j] + group * p.D + c0;
      if constexpr (RPC == 1) {
#pragma unroll
        for (int n = 0; n < NV; n++) {
          const int c = (n * TPR + tr) * V;
          if (c < width) {
#pragma unroll
            for (int i = 0; i < V; i++) to[c + i] = j ? ap[POST ? n : 0][i] : aw[n][i];
          }
        }
      } else {
        float *acc_s = reinterpret_cast<float *>(dyn);
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NV; n++)
#pragma unroll
          for (int i = 0; i < V; i++)
            acc_s[sub * (TPR * NV * V) + (n * TPR + tr) * V + i] = j ? ap[POST ? n : 0][i] : aw[n][i];
        __syncthreads();
        for (int c = threadIdx.x; c < width; c += NT) {
          float a = 0.f;
#pragma unroll
          for (int r = 0; r < RPC; r++) a += acc_s[r * (TPR * NV * V) + c];
          to[c] = a;
        }
      }
    }
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
