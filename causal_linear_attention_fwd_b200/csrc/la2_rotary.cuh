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
#pragma once

#include "la2_common.cuh"
#include "la2_norm.cuh"

namespace la2 {
namespace rot {

constexpr int NT = 256;   // threads per CTA
constexpr int TOK = 4;    // tokens per CTA
constexpr int LANES = NT / TOK;

// One tensor: `n` heads of `width` columns on the strided side (strides in
// values, unit column stride), n * rep heads on the head-major side.
struct Part {
  void *strided;       // [B, n, L, width] through sb, sh, sl
  void *major;         // [B, n * rep, L, width] contiguous
  int64_t sb, sh, sl;
  int n, width, turn;  // turn: columns that are rotated (r, or 0 for v)
};
struct Args {
  Part part[3];
  int parts;
  const double *freq;
  const int64_t *pos;
  int pos_mode;        // 0: the row index; 1: pos[b] + row; 2: pos[b][row]
  int64_t L, rows;     // rows = B * L
  int rep, r, inter;
  float scale;
};

// V = 8: a lane moves 2 x 8 columns of one head (both members of 8 pairs);
// V = 1: 2 columns, for widths, alignments or strides that 16-byte pieces do
// not fit.
template <typename T, bool GRAD, int V>
__global__ void __launch_bounds__(NT) rotary_kernel(const __grid_constant__ Args a) {
  extern __shared__ float2 table[];  // [TOK][r / 2]
  const int64_t row0 = (int64_t)blockIdx.x * TOK;
  const int half = a.r / 2;
  for (int i = threadIdx.x; i < TOK * half; i += NT) {
    const int64_t row = row0 + i / half;
    if (row >= a.rows) break;
    const int64_t b = row / a.L, t = row - b * a.L;
    const int64_t pos = a.pos_mode == 0 ? t : a.pos_mode == 1 ? a.pos[b] + t : a.pos[row];
    // the angle less its whole turns, in fp64; what is left fits fp32
    const double turns = (double)pos * a.freq[i % half] * 0.15915494309189533577;
    float sn, cs;
    sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
    table[i] = make_float2(cs * a.scale, (GRAD ? -sn : sn) * a.scale);
  }
  __syncthreads();
  const int sub = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int64_t row = row0 + sub;
  if (row >= a.rows) return;
  const int64_t b = row / a.L, t = row - b * a.L;
  const float2 *cs = table + sub * half;
#pragma unroll
  for (int q = 0; q < 3; q++) {
    if (q >= a.parts) break;
    const Part &p = a.part[q];
    const int rep = q == 0 ? 1 : a.rep;
    const int chunks = p.width / (2 * V);      // lanes of one head
    const int per = LANES / chunks;            // heads at a time
    if (lane >= per * chunks) continue;
    const int c = lane % chunks;
    // the lane's columns: x0 from c0, x1 from c1
    const bool turned = c * 2 * V < p.turn;
    const int c0 = turned && !a.inter ? c * V : c * 2 * V;
    const int c1 = turned && !a.inter ? c0 + half : c0 + V;
    T *strided = static_cast<T *>(p.strided) + b * p.sb + t * p.sl;
    T *major = static_cast<T *>(p.major) + (b * p.n * rep * a.L + t) * p.width;
    const int64_t hstep = a.L * p.width;
    for (int h = blockIdx.y * per + lane / chunks; h < p.n; h += gridDim.y * per) {
      float x0[V], x1[V];
      T *s = strided + h * p.sh;
      T *m = major + (int64_t)h * rep * hstep;
      if constexpr (!GRAD) {
        norm::ldv<T, V>(s + c0, x0);
        norm::ldv<T, V>(s + c1, x1);
      } else {
        norm::ldv<T, V>(m + c0, x0);
        norm::ldv<T, V>(m + c1, x1);
        for (int j = 1; j < rep; j++) {
          float y0[V], y1[V];
          norm::ldv<T, V>(m + j * hstep + c0, y0);
          norm::ldv<T, V>(m + j * hstep + c1, y1);
#pragma unroll
          for (int i = 0; i < V; i++) {
            x0[i] += y0[i];
            x1[i] += y1[i];
          }
        }
      }
      if (turned) {
        const float2 *w = cs + c * V;
        if (V > 1 && a.inter) {
          // pairs are neighbours: x0 holds the first V / 2 pairs, x1 the rest
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float2 u = w[i / 2], v = w[V / 2 + i / 2];
            float f = x0[i], g = x0[i + (V > 1)];
            x0[i] = f * u.x - g * u.y;
            x0[i + (V > 1)] = f * u.y + g * u.x;
            f = x1[i];
            g = x1[i + (V > 1)];
            x1[i] = f * v.x - g * v.y;
            x1[i + (V > 1)] = f * v.y + g * v.x;
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; i++) {
            const float2 u = w[i];
            const float f = x0[i], g = x1[i];
            x0[i] = f * u.x - g * u.y;
            x1[i] = f * u.y + g * u.x;
          }
        }
      }
      if constexpr (!GRAD) {
        for (int j = 0; j < rep; j++) {
          norm::stv<T, V>(m + j * hstep + c0, x0);
          norm::stv<T, V>(m + j * hstep + c1, x1);
        }
      } else {
        norm::stv<T, V>(s + c0, x0);
        norm::stv<T, V>(s + c1, x1);
      }
    }
  }
}

}  // namespace rot
}  // namespace la2
