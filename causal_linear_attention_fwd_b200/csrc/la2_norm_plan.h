// la2_norm_plan.h -- how the norms' CTAs cover rows and columns, and where a
// thread's values stand in a row.  Plain C++ for the launcher, the kernels and
// host programs alike.
#pragma once

namespace la2 {
namespace norm_plan {

constexpr int kNormMaxCols = 16384;  // widest row

struct NormPlan {
  int nt, tpr, nv, cols, slices, cl, rpc;
  bool odd;
};

// The gated norm's units of eight values: unit u of a CTA begins at column
// gated_unit(.., u) of it and has its second four gated_apart(..) columns after
// its first.  In 32 bits eight units fill a block of 64 columns, so that eight
// lanes move whole lines; in 16 a unit is a block of its own.
constexpr int gated_block(int value_bytes) { return value_bytes == 2 ? 8 : 64; }
constexpr int gated_apart(int value_bytes) { return value_bytes == 2 ? 4 : 32; }
constexpr int gated_unit(int value_bytes, int u) {
  return value_bytes == 2 ? u * 8 : u / 8 * gated_block(value_bytes) + u % 8 * 4;
}

// The row's width decides who holds it (see la2_norm.cuh): a warp, a CTA of 128
// or 256 threads with up to `most_units` units of eight values each, 512
// threads, or a cluster of CTAs.  odd: rows that begin anywhere between two
// 16-byte pieces (up to 7 places more).  Measured at the borders: 128 threads
// against 256 half of which idle, 1,000 columns backward 92 us against 102;
// 512 threads against a cluster of two, 5,000 columns backward 150 us against
// 219; four units (the residual norm's forward, whose rows leave the registers
// for it) against a cluster of two, 8,192 columns 182 us against 207.
// block: columns that a unit's eight values come from; no CTA of a cluster
// begins inside one.
constexpr NormPlan row_plan(int D, bool odd, int most_units = 2, int block = 8) {
  NormPlan g{};
  g.slices = 1;
  g.odd = odd;
  const int places = odd ? D + 7 : D;
  // 256 threads to a CTA, or 512 where that saves a cluster (two units each)
  const int threads = most_units == 2 && places > 4096 ? 512 : 256, most = 8 * threads * most_units;
  g.cl = 1;
  while (g.cl * most < places) g.cl *= 2;
  g.cols = ((places + block - 1) / block + g.cl - 1) / g.cl * block;
  if (places <= 512) {
    g.nt = 128;
    g.tpr = 32;
    g.nv = 2;
  } else if (!odd && places <= 1024) {
    g.nt = g.tpr = 128;
    g.nv = 1;
  } else {
    g.nt = g.tpr = threads;
    g.nv = g.cols <= 2048 ? 1 : g.cols <= 16 * threads ? 2 : 4;
  }
  g.rpc = g.nt / g.tpr;
  return g;
}
// The most CTAs that share a row: the widest one's (up to 4,096 columns, or
// 8,192 with 512 threads or four units, stay with one).
constexpr int most_cl(bool odd) {
  return odd ? row_plan(kNormMaxCols - 1, true).cl
             : row_plan(kNormMaxCols, false, 2).cl > row_plan(kNormMaxCols, false, 4).cl
                   ? row_plan(kNormMaxCols, false, 2).cl
                   : row_plan(kNormMaxCols, false, 4).cl;
}
// The gated norm's rows of H * e columns: every CTA begins at a block and holds
// whole ones, so no unit leaves its head or meets another CTA's columns.
inline NormPlan gated_row_plan(int D, int value_bytes) {
  return row_plan(D, false, 2, gated_block(value_bytes));
}
// Per head: the most heads side by side that divide H, so no lane is idle.
inline NormPlan head_plan(int H, int e) {
  NormPlan g;
  g.odd = false;
  g.nt = 256;
  g.nv = 1;
  g.cl = 1;
  int heads = g.nt * 8 / e;
  while (H % heads) heads /= 2;
  g.cols = heads * e;
  g.tpr = g.cols / 8;
  g.slices = H / heads;
  g.rpc = g.nt / g.tpr;
  return g;
}

}  // namespace norm_plan
}  // namespace la2
