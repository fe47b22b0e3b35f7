// la2_rotary.cuh -- rotary positions on q and k, between a fused projection
// and the attention.
//
// Pair i of a head's first r columns (i and i + r/2, or 2i and 2i + 1) at
// position p turns by the angle p f_i:
//     a' = s (a cos - b sin),   b' = s (a sin + b cos);
// the other columns, and v, pass through.  The projection is token-major (row
// t holds all heads), the attention head-major with one k and v head for
// every q head, so the same pass changes the layout and repeats the k and v
// heads that several q heads share.  Backward: the gradients of a shared
// head's copies are added in fp32, turned by the opposite angle and written
// through the caller's strides (the fused projection's gradient).
//
// Bound by HBM: every value is read once and written once (a shared head
// `rep` times).  The angle is formed in fp64 -- position times frequency has
// up to 53 digits that count at far positions, and fp32 would lose the
// position modulo 2 pi from about 2^20 on -- but only once per (token, pair):
// a CTA takes TOK tokens, its threads fill a table of (s cos, s sin) in
// shared memory, and all heads of the token read it.
//
// Measured on B200 (cold L2, of the copy bandwidth): q, k, v of 65,536 tokens x
// 32 heads x 128 in bf16 522 us (94 %), 32,768 in fp32 535 us (92 %); 8,192
// tokens 76 us (81 %, of which the launch is some 6); one token of 64 requests x
// 16 heads 6.1 us; 16,384 tokens with 20 or 62 columns turned, one by one, 268 us
// (46 %).  The backward of 16,388 tokens with 32 heads each 140 us (88 %), fp32
// 270 us (91 %); with 32 q heads on 8 k, v heads of 64 columns 115 us (69 %: bound
// by the latency of a CTA's loads, 16 warps an SM at 127 registers), on one of
// 128 127 us (66 %).
#pragma once

#include "la2_common.cuh"
#include "la2_norm.cuh"

namespace la2 {
namespace rot {

constexpr int NT = 256;   // threads per CTA
constexpr int TOK = 4;    // tokens per CTA
constexpr int LANES = NT / TOK;

// V values of T as they are in memory.
template <typename T, int V> struct Unit : norm::Raw<T> {};
template <typename T> struct Unit<T, 1> {
  T r;
  __device__ __forceinline__ void load(const T *p, int) { r = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = io<T>::ld(&r); }
};
template <typename T, int V>
__device__ __forceinline__ void put(T *p, const float (&f)[V], int apart) {
  if constexpr (V == 1) io<T>::st(p, f[0]);
  else norm::store8(p, f, apart);
}

// One tensor: `n` heads of `width` columns on the strided side (strides in
// values, unit column stride), n * rep heads on the head-major side.
struct Part {
  void *strided;       // [B, n, L, width] through sb, sh, sl
  void *major;         // [B, n * rep, L, width] contiguous
  int64_t sb, sh, sl;
  int n, width, turn;  // turn: columns that are rotated (r, or 0 for v)
  int lanes, split;    // log2 of the lanes of a head, of the groups of lanes
                       // that share a head's sum
};
struct Args {
  Part part[3];
  int parts;
  const double *freq;
  const int64_t *pos;
  int pos_mode;        // 0: the row index; 1: pos[b] + row; 2: pos[b][row]
  int64_t L, rows;     // rows = B * L
  int rep, r;
  float scale;
};

// Copies of a shared head on their way per thread (128 bytes).
template <typename T, int V>
constexpr int sums_ahead() { return V == 8 ? 8 / (int)sizeof(T) : 0; }
template <typename T, int V>
constexpr size_t sums_smem() {
  return NT * (2 * V * sizeof(float) + 2 * sums_ahead<T, V>() * 2 * V * sizeof(T));
}

// V = 8: a lane moves 2 x 8 columns of one head, both members of 8 pairs; V =
// 1: 2 columns, for widths, alignments or strides that 16-byte pieces do not
// fit.  The lanes of a head share its turned columns and then the rest: lane c
// of n takes 8 from 8 c on in each half of them (fp32: 4 from 4 c on and 4 n
// further, in each half), so that every load and store of the lanes is one run
// of bytes (a 32-byte stride between lanes moves every sector twice).  U heads'
// loads are issued before any of them is turned, and the first ones before the
// table is made.  SUMS: the backward where heads are shared.
template <typename T, bool GRAD, bool SUMS, bool INTER, int V, int U>
__global__ void __launch_bounds__(NT, SUMS ? 2 : 3) rotary_kernel(const __grid_constant__ Args a) {
  extern __shared__ float2 table[];  // [TOK][r / 2]
  const int64_t row0 = (int64_t)blockIdx.x * TOK;
  const int half = a.r / 2;
  const int sub = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int64_t row = row0 + sub;
  const bool live = row < a.rows;
  int64_t b = 0, t = 0;
  if (live) norm::split_row(row, a.L, b, t);
  // where this lane's values of a tensor are
  struct View {
    int per, cc, n_lanes, c0, c1;
    bool turned;
    int64_t hstep;
    T *strided, *major;
  };
  constexpr int W = V == 8 && sizeof(T) == 4 ? 4 : V;
  auto view = [&](const Part &p, int rep) {
    View w;
    w.per = LANES >> p.lanes;  // heads at a time
    const int c = lane & ((1 << p.lanes) - 1);
    w.turned = c * 2 * V < p.turn;
    w.n_lanes = (w.turned ? p.turn : p.width - p.turn) / (2 * V);
    w.cc = w.turned ? c : c - p.turn / (2 * V);
    // the lane's columns: x0 from c0, x1 from c1
    const bool neighbours = V == 1 && INTER && w.turned;
    w.c0 = neighbours ? 2 * w.cc : (w.turned ? 0 : p.turn) + w.cc * W;
    w.c1 = neighbours ? w.c0 + 1 : w.c0 + w.n_lanes * V;
    w.hstep = a.L * p.width;
    w.strided = static_cast<T *>(p.strided) + b * p.sb + t * p.sl;
    w.major = static_cast<T *>(p.major) + (b * p.n * rep * a.L + t) * p.width;
    return w;
  };
  // SUMS: the first copies of the first heads of k and v are on their way into
  // the thread's own places of shared memory while q is worked on.
  constexpr int AHEAD = SUMS ? sums_ahead<T, V>() : 0, PIECES = 2 * sizeof(T) / 2;
  float *partial = reinterpret_cast<float *>(table + TOK * half);  // [2 V][NT]
  auto ahead = [&](int q, int copy, int piece) {
    return reinterpret_cast<uint4 *>(partial + 2 * V * NT) +
           (((q - 1) * AHEAD + copy) * PIECES + piece) * NT + threadIdx.x;
  };
  if constexpr (AHEAD > 0) {
    for (int q = blockIdx.z; q < a.parts; q += gridDim.z) {
      const Part &p = a.part[q];
      const View w = view(p, a.rep);
      const int group = lane >> p.lanes, s = group & ((1 << p.split) - 1);
      const int h = blockIdx.y * (w.per >> p.split) + (group >> p.split);
      if (q > 0 && live && h < p.n) {
        const int begin = s * a.rep >> p.split, end = (s + 1) * a.rep >> p.split;
        const T *m = w.major + (int64_t)(h * a.rep + begin) * w.hstep;
#pragma unroll
        for (int j = 0; j < AHEAD; j++, m += w.hstep)
          if (begin + j < end) {
#pragma unroll
            for (int k = 0; k < PIECES / 2; k++) {
              norm::copy16_async(ahead(q, j, k), m + w.c0 + k * w.n_lanes * 4);
              norm::copy16_async(ahead(q, j, PIECES / 2 + k), m + w.c1 + k * w.n_lanes * 4);
            }
          }
      }
    }
    norm::copies_commit();
  }
#pragma unroll 1
  for (int q = blockIdx.z; q < a.parts; q += gridDim.z) {
    const Part &p = a.part[q];
    const int rep = q == 0 ? 1 : a.rep;
    const View at = view(p, rep);
    const int per = at.per, cc = at.cc, n_lanes = at.n_lanes, c0 = at.c0, c1 = at.c1;
    const int apart = n_lanes * 4;  // between fp32's pieces
    const bool turned = at.turned;
    const int64_t hstep = at.hstep;
    T *strided = at.strided, *major = at.major;
    const int h0 = blockIdx.y * per + (lane >> p.lanes), stride = gridDim.y * per;
    const int n = live ? p.n : 0;
    Unit<T, V> x0[U], x1[U];
    auto fetch = [&](int h) {
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int hu = h + u * stride;
        if (hu < n) {
          const T *s = GRAD ? major + (int64_t)hu * hstep : strided + hu * p.sh;
          x0[u].load(s + c0, apart);
          x1[u].load(s + c1, apart);
        }
      }
    };
    const bool sums = SUMS && q > 0;  // a head's gradients come from several
    if (!sums) fetch(h0);
    if (q == (int)blockIdx.z && p.turn) {
      const int64_t pos = !live ? 0 : a.pos_mode == 0 ? t : a.pos_mode == 1 ? a.pos[b] + t : a.pos[row];
#pragma unroll 1
      for (int i = lane; i < half; i += LANES) {
        // the angle less its whole turns, in fp64; what is left fits fp32
        const double turns = (double)pos * a.freq[i] * 0.15915494309189533577;
        float sn, cs;
        sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
        table[sub * half + i] = make_float2(cs * a.scale, (GRAD ? -sn : sn) * a.scale);
      }
      __syncthreads();
    }
    // the pairs of x0's values (and x1's, which are the same ones); pairs of
    // neighbours: x0's four, then x1's four
    auto angles = [&](float2 (&w)[V]) {
#pragma unroll
      for (int i = 0; i < V; i++) {
        int pr;
        if (V == 8 && INTER) {
          const int k = i % 4;
          pr = (W == 4 ? k / 2 * n_lanes * 2 + cc * 2 + k % 2 : cc * 4 + k) + i / 4 * n_lanes * 4;
        } else {
          pr = W == 4 ? i / 4 * apart + cc * 4 + i % 4 : cc * V + i;
        }
        if (turned) w[i] = table[sub * half + pr];
      }
    };
    auto turn = [&](float (&f)[V], float (&g)[V], const float2 (&w)[V]) {
      if (!turned) return;
      if (V > 1 && INTER) {
        // pairs are neighbours: f holds the first V / 2 pairs, g the rest
#pragma unroll
        for (int i = 0; i + 1 < V; i += 2) {
          const float2 u = w[i / 2], v = w[V / 2 + i / 2];
          const float f0 = f[i], g0 = g[i];
          f[i] = f0 * u.x - f[i + 1] * u.y;
          f[i + 1] = f0 * u.y + f[i + 1] * u.x;
          g[i] = g0 * v.x - g[i + 1] * v.y;
          g[i + 1] = g0 * v.y + g[i + 1] * v.x;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; i++) {
          const float f0 = f[i];
          f[i] = f0 * w[i].x - g[i] * w[i].y;
          g[i] = f0 * w[i].y + g[i] * w[i].x;
        }
      }
    };
    if (!sums) {
      float2 w[V];
      angles(w);
      for (int h = h0; h < n; h += U * stride) {
        if (h != h0) fetch(h);
#pragma unroll
        for (int u = 0; u < U; u++) {
          const int hu = h + u * stride;
          if (hu >= n) break;
          float f[V], g[V];
          x0[u].get(f);
          x1[u].get(g);
          turn(f, g, w);
          if constexpr (GRAD) {
            put<T, V>(strided + hu * p.sh + c0, f, apart);
            put<T, V>(strided + hu * p.sh + c1, g, apart);
          } else {
            T *m = major + (int64_t)hu * rep * hstep;
#pragma unroll 1
            for (int j = 0; j < rep; j++, m += hstep) {
              put<T, V>(m + c0, f, apart);
              put<T, V>(m + c1, g, apart);
            }
          }
        }
      }
    } else if constexpr (SUMS) {
      // `split` groups of lanes share a head's copies where there are fewer
      // heads than groups; their partial sums meet in shared memory
      const int split = 1 << p.split, heads = per >> p.split, group = lane >> p.lanes;
      const int s = group & (split - 1), begin = s * rep >> p.split;
      for (int hb = blockIdx.y * heads; hb < p.n; hb += gridDim.y * heads) {
        const int h = hb + (group >> p.split);
        const T *m = major + (int64_t)h * rep * hstep;
        const int end = h < n ? (s + 1) * rep >> p.split : 0;
        float f[V], g[V];
#pragma unroll
        for (int i = 0; i < V; i++) f[i] = g[i] = 0.f;
        int j = begin;
        if constexpr (AHEAD > 0) {
          if (hb == (int)blockIdx.y * heads) {
            norm::copies_wait<0>();
#pragma unroll
            for (int u = 0; u < AHEAD; u++, j++) {
              if (j < end) {
                norm::Raw<T> r0, r1;
#pragma unroll
                for (int k = 0; k < PIECES / 2; k++) {
                  r0.r[k] = *ahead(q, u, k);
                  r1.r[k] = *ahead(q, u, PIECES / 2 + k);
                }
                float y0[8], y1[8];
                r0.get(y0);
                r1.get(y1);
#pragma unroll
                for (int i = 0; i < V; i++) {
                  f[i] += y0[i];
                  g[i] += y1[i];
                }
              }
            }
          }
        }
        for (; j < end; j += U) {
#pragma unroll
          for (int u = 0; u < U; u++) {
            if (j + u < end) {
              x0[u].load(m + (j + u) * hstep + c0, apart);
              x1[u].load(m + (j + u) * hstep + c1, apart);
            }
          }
#pragma unroll
          for (int u = 0; u < U; u++) {
            if (j + u < end) {
              float y0[V], y1[V];
              x0[u].get(y0);
              x1[u].get(y1);
#pragma unroll
              for (int i = 0; i < V; i++) {
                f[i] += y0[i];
                g[i] += y1[i];
              }
            }
          }
        }
        if (split > 1) {
          __syncthreads();  // the last round's are read
          if (s) {
#pragma unroll
            for (int i = 0; i < V; i++) {
              partial[i * NT + threadIdx.x] = f[i];
              partial[(V + i) * NT + threadIdx.x] = g[i];
            }
          }
          __syncthreads();
          if (s) continue;
          for (int k = 1; k < split; k++) {
#pragma unroll
            for (int i = 0; i < V; i++) {
              f[i] += partial[i * NT + threadIdx.x + (k << p.lanes)];
              g[i] += partial[(V + i) * NT + threadIdx.x + (k << p.lanes)];
            }
          }
        }
        if (h >= n) continue;
        float2 w[V];  // not held while the sums are made
        angles(w);
        turn(f, g, w);
        put<T, V>(strided + h * p.sh + c0, f, apart);
        put<T, V>(strided + h * p.sh + c1, g, apart);
      }
    }
  }
}

}  // namespace rot
}  // namespace la2
