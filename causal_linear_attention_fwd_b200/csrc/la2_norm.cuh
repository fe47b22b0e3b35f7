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
// statistics because the row it must read anyway gives them again.
//
// The weights' gradients are column sums over all rows.  A thread keeps its
// columns over all rows its CTA walks, so each CTA writes one row of partial
// sums to the workspace, and colsum_kernel adds those rows in a fixed order:
// no atomics, the same result on every run.
#pragma once

#include "la2_common.cuh"
#include "la2_fmap.cuh"

namespace la2 {
namespace norm {

// ------------------------------------------------------------ vectors
// V consecutive values as fp32: V = 8 moves 16-byte pieces (the address is
// 16-byte aligned), V = 1 single values (rows that no vector divides).
template <typename T, int V>
__device__ __forceinline__ void ldv(const T *p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = io<T>::ld(p);
  } else {
    constexpr int N = fmap::vec16<T>::N;
#pragma unroll
    for (int i = 0; i < V / N; i++) {
      float g[N];
      fmap::vec16<T>::unpack(fmap::ld_stream(p + i * N), g);
#pragma unroll
      for (int j = 0; j < N; j++) f[i * N + j] = g[j];
    }
  }
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
// V = 8 values from an address with the element's alignment only.
template <typename T, int V>
__device__ __forceinline__ void ldu(const T *p, float (&f)[V], bool vec) {
  if (vec) {
    ldv<T, V>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) f[i] = io<T>::ld(p + i);
  }
}
template <typename T, int V>
__device__ __forceinline__ void stu(T *p, const float (&f)[V], bool vec) {
  if (vec) {
    stv<T, V>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) io<T>::st(p + i, f[i]);
  }
}
// Weights: fp32, read by every row of a CTA, so through the cache.
template <int V>
__device__ __forceinline__ void ldw(const float *w, int64_t c, float (&f)[V]) {
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

// ------------------------------------------------------------ reductions
// Sum of K values over the LANES neighbouring lanes of a warp; every lane
// gets it.
template <int K>
__device__ __forceinline__ void lanes_sum(float (&x)[K], int lanes) {
  for (int m = lanes / 2; m > 0; m /= 2) {
#pragma unroll
    for (int k = 0; k < K; k++) x[k] += __shfl_xor_sync(0xffffffffu, x[k], m);
  }
}
// Sum of K values over the TPR threads that share a row: a warp, or the
// whole CTA (TPR threads).  `red` holds two generations of partial sums, used
// in turn, so one barrier per sum is enough: a thread that runs ahead writes
// the other half, and cannot come back to this one before every thread has
// passed the barrier in between.
template <int TPR, int K>
__device__ __forceinline__ void row_sum(float (&x)[K], float (*red)[K][32], int &turn) {
  lanes_sum<K>(x, 32);
  if constexpr (TPR > 32) {
    constexpr int NW = TPR / 32;
    const int w = threadIdx.x / 32, l = threadIdx.x % 32;
    if (l == 0) {
#pragma unroll
      for (int k = 0; k < K; k++) red[turn][k][w] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; k++) x[k] = l < NW ? red[turn][k][l] : 0.f;
    lanes_sum<K>(x, 32);
    turn ^= 1;
  }
}

// ------------------------------------------------------------ gate
struct Act {
  float a, da;
};
// The activated gate and its slope.  e^-g overflows to infinity for g below
// -88, where the sigmoid is 0 to fp32 (the quotient gives it).  Values that
// will be rounded to bf16 take the approximate exponential and quotient (a
// few 2^-23 off, against the rounding's 2^-9); fp32 takes the exact ones.
template <typename T>
__device__ __forceinline__ Act activate(float g, bool silu) {
  float s;
  if constexpr (sizeof(T) == 4) s = 1.f / (1.f + expf(-g));
  else s = __fdividef(1.f, 1.f + __expf(-g));
  Act r;
  if (silu) {
    r.a = g * s;
    r.da = s * fmaf(g, 1.f - s, 1.f);
  } else {
    r.a = s;
    r.da = s * (1.f - s);
  }
  return r;
}

// ------------------------------------------------------------ gated norm
struct Gated {
  const void *o, *gate, *du;
  void *u, *d_o, *dgate;
  const float *weight;
  float *dw;                 // partial sums of the weight's gradient, or null
  int64_t gate_b, gate_l;    // strides of the gate's batch and row, in values
  int64_t dgate_b, dgate_l;
  int64_t L, rows;           // rows = B * L tokens
  int H, e;
  int silu, shared;          // shared: weight [e], the same for every head
  int gate_vec, dgate_vec;   // rows of the gate (its gradient) 16-byte aligned
  float eps;
};

// Row: whether one norm spans the H * e values of a token (else one per
// head).  A CTA covers, for one token at a time, TPR threads x NV vectors of
// columns (from column blockIdx.y * TPR * NV * V on, per head only) and walks
// tokens with a stride; TPR < NT: several tokens side by side.
template <typename T, bool ROW, bool GRAD, int NT, int NV>
__global__ void __launch_bounds__(NT) gated_kernel(const Gated p, int TPR, int cols) {
  constexpr int V = 8;
  __shared__ float red[2][2][32];
  extern __shared__ float acc_s[];
  const int rpc = NT / TPR, sub = threadIdx.x / TPR, tr = threadIdx.x % TPR;
  const int64_t D = (int64_t)p.H * p.e;
  const int64_t c0 = (int64_t)blockIdx.y * cols;
  const int lph = p.e / V;   // lanes of one head
  const float inv = 1.f / (ROW ? (float)D : (float)p.e);
  const T *o = static_cast<const T *>(p.o), *gate = static_cast<const T *>(p.gate);
  const T *du = static_cast<const T *>(p.du);
  int turn = 0;
  float acc[GRAD ? NV : 1][V];
#pragma unroll
  for (int n = 0; n < (GRAD ? NV : 1); n++)
#pragma unroll
    for (int i = 0; i < V; i++) acc[n][i] = 0.f;

  for (int64_t r0 = (int64_t)blockIdx.x * rpc; r0 < p.rows; r0 += (int64_t)gridDim.x * rpc) {
    const int64_t row = r0 + sub;
    const bool live = row < p.rows;
    const int64_t b = live ? row / p.L : 0, t = live ? row - b * p.L : 0;
    float x[NV][V], g[NV][V], up[GRAD ? NV : 1][V];
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int64_t c = c0 + (int64_t)(n * TPR + tr) * V;
      const bool on = live && c < D && c < c0 + cols;
      if (on) {
        ldv<T, V>(o + ((b * p.H + c / p.e) * p.L + t) * p.e + c % p.e, x[n]);
        if (gate) ldu<T, V>(gate + b * p.gate_b + t * p.gate_l + c, g[n], p.gate_vec);
        if constexpr (GRAD) ldv<T, V>(du + row * D + c, up[n]);
      } else {
#pragma unroll
        for (int i = 0; i < V; i++) {
          x[n][i] = 0.f;
          g[n][i] = 0.f;
          if constexpr (GRAD) up[n][i] = 0.f;
        }
      }
    }
    // per-row (ROW) or per-head statistics; in the backward also sum(dy * o)
    float st[NV][2];
#pragma unroll
    for (int n = 0; n < NV; n++) {
      st[n][0] = st[n][1] = 0.f;
      const int64_t c = c0 + (int64_t)(n * TPR + tr) * V;
      float w[V];
      if constexpr (GRAD) {
        if (c < D) {
          ldw<V>(p.weight, p.shared ? c % p.e : c, w);
        } else {
#pragma unroll
          for (int i = 0; i < V; i++) w[i] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < V; i++) {
        st[n][0] = fmaf(x[n][i], x[n][i], st[n][0]);
        if constexpr (GRAD) {
          const float a = gate ? activate<T>(g[n][i], p.silu).a : 1.f;
          st[n][1] = fmaf(up[n][i] * w[i] * a, x[n][i], st[n][1]);
        }
      }
    }
    if constexpr (ROW) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < NV; n++) {
        s[0] += st[n][0];
        s[1] += st[n][1];
      }
      if (TPR == 32) row_sum<32, 2>(s, red, turn);
      else row_sum<NT, 2>(s, red, turn);
#pragma unroll
      for (int n = 0; n < NV; n++) {
        st[n][0] = s[0];
        st[n][1] = s[1];
      }
    } else {
#pragma unroll
      for (int n = 0; n < NV; n++) lanes_sum<2>(st[n], lph);
    }
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int64_t c = c0 + (int64_t)(n * TPR + tr) * V;
      if (!(live && c < D && c < c0 + cols)) continue;
      const float rstd = rsqrtf(fmaf(st[n][0], inv, p.eps));
      float w[V];
      ldw<V>(p.weight, p.shared ? c % p.e : c, w);
      if constexpr (!GRAD) {
        float y[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
          const float a = gate ? activate<T>(g[n][i], p.silu).a : 1.f;
          y[i] = x[n][i] * rstd * w[i] * a;
        }
        stv<T, V>(static_cast<T *>(p.u) + row * D + c, y);
      } else {
        const float m = st[n][1] * rstd * inv;  // mean(dy * y)
        float dx[V], dg[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
          const float y = x[n][i] * rstd;
          const Act a = gate ? activate<T>(g[n][i], p.silu) : Act{1.f, 0.f};
          const float uy = up[n][i] * y;
          dg[i] = uy * w[i] * a.da;
          acc[n][i] = fmaf(uy, a.a, acc[n][i]);
          dx[i] = rstd * fmaf(-y, m, up[n][i] * w[i] * a.a);
        }
        stv<T, V>(static_cast<T *>(p.d_o) + ((b * p.H + c / p.e) * p.L + t) * p.e + c % p.e, dx);
        if (gate)
          stu<T, V>(static_cast<T *>(p.dgate) + b * p.dgate_b + t * p.dgate_l + c, dg, p.dgate_vec);
      }
    }
  }
  if constexpr (GRAD) {
    if (!p.dw) return;
    // the CTA's partial sums: over the tokens side by side and, for a weight
    // that the heads share, over the heads it covers
    float *mine = acc_s + (int64_t)threadIdx.x * NV * V;  // [sub][tr][n][i]
#pragma unroll
    for (int n = 0; n < NV; n++)
#pragma unroll
      for (int i = 0; i < V; i++) mine[n * V + i] = acc[n][i];
    __syncthreads();
    const int64_t left = D - c0;
    const int w = (int)(left < cols ? left : cols);
    const int out = p.shared ? p.e : w;
    for (int j = threadIdx.x; j < out; j += NT) {
      float s = 0.f;
      for (int c = j; c < w; c += out) {
        const int vec = c / V, n = vec / TPR, lane = vec % TPR;
        for (int k = 0; k < rpc; k++) s += acc_s[((k * TPR + lane) * NV + n) * V + c % V];
      }
      if (p.shared)
        p.dw[((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * p.e + j] = s;
      else
        p.dw[(int64_t)blockIdx.x * D + c0 + j] = s;
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
  int D;
  float alpha, beta, eps;
};

template <typename T, typename R, bool POST, int V, int NT, int TPR, int NV>
__global__ void __launch_bounds__(NT) residual_kernel(const Residual p) {
  __shared__ float red[2][1][32];
  constexpr int RPC = NT / TPR;
  const int sub = threadIdx.x / TPR, tr = threadIdx.x % TPR;
  const float inv = 1.f / (float)p.D;
  const T *y = static_cast<const T *>(p.y);
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * RPC; r0 < p.rows; r0 += (int64_t)gridDim.x * RPC) {
    const int64_t row = r0 + sub;
    const bool live = row < p.rows;
    const int64_t at = live ? row * p.D : 0;
    float x[NV][V], z[NV][V];
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int c = (n * TPR + tr) * V;
      if (live && c < p.D) {
        ldv<R, V>(static_cast<const R *>(p.h) + at + c, x[n]);
        if (y) ldv<T, V>(y + at + c, z[n]);
      } else {
#pragma unroll
        for (int i = 0; i < V; i++) x[n][i] = z[n][i] = 0.f;
      }
    }
    if (y) {
      float ry = 1.f;
      if constexpr (POST) {
        float s[1] = {0.f};
#pragma unroll
        for (int n = 0; n < NV; n++)
#pragma unroll
          for (int i = 0; i < V; i++) s[0] = fmaf(z[n][i], z[n][i], s[0]);
        row_sum<TPR, 1>(s, red, turn);
        ry = rsqrtf(fmaf(s[0], inv, p.eps));
      }
#pragma unroll
      for (int n = 0; n < NV; n++) {
        const int c = (n * TPR + tr) * V;
        if (!(live && c < p.D)) continue;
        float w[V];
        if constexpr (POST) ldw<V>(p.post_weight, c, w);
#pragma unroll
        for (int i = 0; i < V; i++) {
          const float q = POST ? z[n][i] * ry * w[i] : z[n][i];
          x[n][i] = fmaf(p.beta, q, p.alpha * x[n][i]);
        }
        stv<R, V>(static_cast<R *>(p.h_new) + at + c, x[n]);
      }
    }
    float s[1] = {0.f};
#pragma unroll
    for (int n = 0; n < NV; n++)
#pragma unroll
      for (int i = 0; i < V; i++) s[0] = fmaf(x[n][i], x[n][i], s[0]);
    row_sum<TPR, 1>(s, red, turn);
    const float rstd = rsqrtf(fmaf(s[0], inv, p.eps));
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int c = (n * TPR + tr) * V;
      if (!(live && c < p.D)) continue;
      float w[V];
      ldw<V>(p.weight, c, w);
#pragma unroll
      for (int i = 0; i < V; i++) w[i] *= x[n][i] * rstd;
      stv<T, V>(static_cast<T *>(p.n) + at + c, w);
    }
  }
}

// The weights' partial sums live in shared memory, [RPC][D] each (a thread
// touches its own columns only, so no barrier is needed until the end).
template <typename T, typename R, bool POST, int V, int NT, int TPR, int NV>
__global__ void __launch_bounds__(NT) residual_grad_kernel(const Residual p) {
  __shared__ float red[2][3][32];
  extern __shared__ float acc_s[];
  constexpr int RPC = NT / TPR;
  constexpr int COLS = TPR * NV * V;
  const int sub = threadIdx.x / TPR, tr = threadIdx.x % TPR;
  const float inv = 1.f / (float)p.D;
  float *aw = acc_s + sub * COLS, *ap = acc_s + (RPC + sub) * COLS;
#pragma unroll
  for (int n = 0; n < NV; n++)
#pragma unroll
    for (int i = 0; i < V; i++) {
      aw[(n * TPR + tr) * V + i] = 0.f;
      if constexpr (POST) ap[(n * TPR + tr) * V + i] = 0.f;
    }
  int turn = 0, turn1 = 0;
  __shared__ float red1[2][1][32];
  for (int64_t r0 = (int64_t)blockIdx.x * RPC; r0 < p.rows; r0 += (int64_t)gridDim.x * RPC) {
    const int64_t row = r0 + sub;
    const bool live = row < p.rows;
    const int64_t at = live ? row * p.D : 0;
    float x[NV][V], s[NV][V], g[NV][V], z[POST ? NV : 1][V];
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int c = (n * TPR + tr) * V;
      const bool on = live && c < p.D;
#pragma unroll
      for (int i = 0; i < V; i++) {
        x[n][i] = s[n][i] = g[n][i] = 0.f;
        if constexpr (POST) z[n][i] = 0.f;
      }
      if (on) {
        ldv<R, V>(static_cast<const R *>(p.h) + at + c, x[n]);
        ldv<T, V>(static_cast<const T *>(p.dn) + at + c, s[n]);
        if (p.dh_new) ldv<R, V>(static_cast<const R *>(p.dh_new) + at + c, g[n]);
        if constexpr (POST) ldv<T, V>(static_cast<const T *>(p.y) + at + c, z[n]);
      }
    }
    // sums of h'^2, (dn w) h' and, with a norm on y, y^2
    float q[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int c = (n * TPR + tr) * V;
      if (c >= p.D) continue;
      float w[V];
      ldw<V>(p.weight, c, w);
#pragma unroll
      for (int i = 0; i < V; i++) {
        q[0] = fmaf(x[n][i], x[n][i], q[0]);
        q[1] = fmaf(s[n][i] * w[i], x[n][i], q[1]);
        if constexpr (POST) q[2] = fmaf(z[n][i], z[n][i], q[2]);
      }
    }
    row_sum<TPR, 3>(q, red, turn);
    const float rstd = rsqrtf(fmaf(q[0], inv, p.eps));
    const float m = q[1] * rstd * inv;  // mean(s hn)
    const float ry = POST ? rsqrtf(fmaf(q[2], inv, p.eps)) : 1.f;
    float k[1] = {0.f};                 // sum of (dp pw) yn
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int c = (n * TPR + tr) * V;
      if (!(live && c < p.D)) continue;
      float w[V], pw[V], dh[V];
      ldw<V>(p.weight, c, w);
      if constexpr (POST) ldw<V>(p.post_weight, c, pw);
#pragma unroll
      for (int i = 0; i < V; i++) {
        const float hn = x[n][i] * rstd;
        aw[c + i] = fmaf(s[n][i], hn, aw[c + i]);
        const float dH = fmaf(rstd, fmaf(-hn, m, s[n][i] * w[i]), g[n][i]);
        dh[i] = p.alpha * dH;
        g[n][i] = p.beta * dH;          // dp
        if constexpr (POST) {
          const float yn = z[n][i] * ry;
          ap[c + i] = fmaf(g[n][i], yn, ap[c + i]);
          k[0] = fmaf(g[n][i] * pw[i], yn, k[0]);
        }
      }
      stv<R, V>(static_cast<R *>(p.dh) + at + c, dh);
    }
    if (p.dy) {
      if constexpr (POST) {
        row_sum<TPR, 1>(k, red1, turn1);
        const float mz = k[0] * inv;
#pragma unroll
        for (int n = 0; n < NV; n++) {
          const int c = (n * TPR + tr) * V;
          if (!(live && c < p.D)) continue;
          float pw[V];
          ldw<V>(p.post_weight, c, pw);
#pragma unroll
          for (int i = 0; i < V; i++)
            g[n][i] = ry * fmaf(-z[n][i] * ry, mz, g[n][i] * pw[i]);
        }
      }
#pragma unroll
      for (int n = 0; n < NV; n++) {
        const int c = (n * TPR + tr) * V;
        if (live && c < p.D) stv<T, V>(static_cast<T *>(p.dy) + at + c, g[n]);
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.D; c += NT) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int j = 0; j < RPC; j++) {
      a += acc_s[j * COLS + c];
      if constexpr (POST) b += acc_s[(RPC + j) * COLS + c];
    }
    if (p.dw) p.dw[(int64_t)blockIdx.x * p.D + c] = a;
    if constexpr (POST) {
      if (p.dpw) p.dpw[(int64_t)blockIdx.x * p.D + c] = b;
    }
  }
}

// Column sums of two arrays of partial sums [rows][cols] (either may be
// null): 32 columns x 8 rows of threads, each thread's rows in order, then
// the 8 sums in order.
constexpr int kSumCols = 32, kSumRows = 8;
__global__ void __launch_bounds__(kSumCols *kSumRows)
colsum_kernel(const float *a, const float *b, float *ya, float *yb, int rows, int cols) {
  __shared__ float s[kSumRows][kSumCols];
  const float *x = blockIdx.y ? b : a;
  float *y = blockIdx.y ? yb : ya;
  if (!y) return;
  const int tc = threadIdx.x % kSumCols, tr = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + tc;
  float sum = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int r = tr; r < rows; r += kSumRows) sum += x[(int64_t)r * cols + c];
  }
  s[tr][tc] = sum;
  __syncthreads();
  if (tr == 0 && c < cols) {
#pragma unroll
    for (int j = 1; j < kSumRows; j++) sum += s[j][tc];
    y[c] = sum;
  }
}

}  // namespace norm
}  // namespace la2
