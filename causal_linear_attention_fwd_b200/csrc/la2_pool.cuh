// la2_pool.cuh -- states copied between the slots of a pool.
//
// For n = 0..N-1 at once: to[dst[n]] = from[src[n]] as it was before the
// call (src[n] < 0: zeros; dst[n] < 0: nothing).  `to` and `from` may be one
// pool, with any slot a source, a destination or both: a fork (one source,
// several destinations), a beam reorder (a permutation with repeats), a
// compaction.
//
// Bound by HBM: each source read once, each destination written once.  A
// state's bytes move independently of one another, so no copy of the
// states is staged in memory: a CTA takes a slab -- the same W bytes of every
// state -- reads that slab of all sources into shared memory, waits, and only
// then writes the destinations.  Slabs share no byte, so CTAs need no order
// among themselves.  The copies are bulk copies between global and shared
// memory (16-byte granules, no data through registers); a ring of
// slabs keeps loads in flight while older slabs are being stored.  Thread i
// issues the load and the store of the moves i, i + NT, ..., so a slab buffer
// is refilled by the very thread whose stores read it.
//
// Measured on B200 (states of 4 MiB, cold L2, of the copy bandwidth): a cycle
// through 200 slots 270 us (95 %), 256 beams 268 us (87 %); cycles through 512 and
// 1,000 states of 256 KiB 78 and 180 us (53 and 45 %: pieces of 128 and 96
// bytes).
#pragma once

#include "la2_bulk.cuh"
#include "la2_common.cuh"
#include "la2_sm100.cuh"

namespace la2 {
namespace pool {

using namespace sm100;

constexpr int NT = 256;
constexpr int MAX_MOVES = 4096;
constexpr int MAX_W = 4096;       // widest slab
constexpr int MAX_STAGES = 8;
constexpr int SMEM = 227 * 1024;  // what a CTA may have
constexpr int HEAD = 256;         // barriers, counters
// shared memory: HEAD, then MAX_W zero bytes, the list of moves, the ring
constexpr int ring_bytes(int n) { return (SMEM - HEAD - MAX_W - (n * 8 + 127) / 128 * 128) / 128 * 128; }

// from [layers, from_size, bytes], to [layers, to_size, bytes]; `bytes` a
// multiple of 16.
__global__ void __launch_bounds__(NT)
copy_kernel(const char *from, char *to, const int *src, const int *dst, int n, int from_size,
            int to_size, int layers, int64_t bytes) {
  extern __shared__ __align__(128) char smem[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + MAX_STAGES * 8);
  int *count = reinterpret_cast<int *>(smem + MAX_STAGES * 8 + 4);
  char *zeros = smem + HEAD;
  int2 *list = reinterpret_cast<int2 *>(zeros + MAX_W);
  char *ring = zeros + MAX_W + (n * 8 + 127) / 128 * 128;
  const int tid = threadIdx.x;

  if (tid == 0) {
    *count = 0;
    *abort = 0;
  }
  for (int i = tid; i < MAX_W / 16; i += NT)
    reinterpret_cast<uint4 *>(zeros)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    const int s = src[i], d = dst[i];
    if (d < 0) continue;
    if (d >= to_size || s >= from_size) {
      if (blockIdx.x == 0) raise_error(ERR_BOUNDS);
      continue;
    }
    if (s == d && from == to) continue;  // stays where it is
    list[atomicAdd(count, 1)] = make_int2(s, d);
  }
  __syncthreads();
  const int m = *count;
  if (m == 0) return;

  // The slab's width: four slabs of all moves in the ring, or three or two
  // where that would leave less than 768 or 256 bytes of each state, and no
  // wider than gives every CTA a slab.  (Narrow pieces cost: 200 moves of
  // 4 MiB took 512 us at 128 bytes each, 313 with two slabs of 512, 274 with
  // three of 256.)
  const int room = ring_bytes(n);
  int w = room / 4 / m;
  if (w < 768) w = room / 3 / m;
  if (w < 256) w = room / 2 / m;
  const int64_t share = (bytes * layers + gridDim.x - 1) / gridDim.x;
  if (w > share) w = (int)share;
  if (w > MAX_W) w = MAX_W;
  w = w >= 128 ? w / 128 * 128 : w / 16 * 16;
  if (w < 16) w = 16;
  int stages = room / (w * m);
  if (stages > MAX_STAGES) stages = MAX_STAGES;
  const int users = m < NT ? m : NT;  // threads that have a move
  if (tid == 0) {
    for (int i = 0; i < stages; i++) mbar_init(smem_u32(bars + i), users);
    fence_mbar_init();
  }
  fence_proxy_async_smem();  // the zeros, for the stores
  __syncthreads();
  if (tid >= users) return;

  // Slab s of layer l is bytes [s w, s w + w) of every state of that layer;
  // this CTA's are gridDim.x apart, counted through the layers.
  const int slabs_row = (int)((bytes + w - 1) / w);
  struct Place {
    int slab, layer, stage;
  };
  auto next = [&](Place &p) {
    p.slab += gridDim.x;
    while (p.slab >= slabs_row && p.layer < layers) {
      p.slab -= slabs_row;
      p.layer++;
    }
    if (++p.stage == stages) p.stage = 0;
  };
  auto length = [&](const Place &p) {
    const int64_t left = bytes - (int64_t)p.slab * w;
    return (uint32_t)(left < w ? left : w);
  };
  auto load = [&](const Place &p) {
    const uint32_t len = length(p), bar = smem_u32(bars + p.stage);
    const char *base = from + (int64_t)p.layer * from_size * bytes + (int64_t)p.slab * w;
    uint32_t total = 0;
    for (int i = tid; i < m; i += NT) total += list[i].x >= 0 ? len : 0;
    mbar_expect_tx(bar, total);
    for (int i = tid; i < m; i += NT) {
      const int s = list[i].x;
      if (s >= 0) bulk::load(smem_u32(ring) + (uint32_t)(p.stage * m + i) * w, base + s * bytes, len, bar);
    }
  };
  Place at{(int)blockIdx.x, 0, 0}, ahead;
  at.slab -= gridDim.x;
  at.stage = -1;
  next(at);
  ahead = at;
  for (int i = 0; i < stages && ahead.layer < layers; i++, next(ahead)) load(ahead);
  bool ok = true;
  uint32_t phase = 0;
  for (int it = 0; at.layer < layers; it++) {
    ok = mbar_wait(smem_u32(bars + at.stage), phase, abort);
    if (!ok) break;
    const uint32_t len = length(at);
    char *base = to + (int64_t)at.layer * to_size * bytes + (int64_t)at.slab * w;
    for (int i = tid; i < m; i += NT)
      bulk::store(base + list[i].y * bytes,
                 list[i].x >= 0 ? smem_u32(ring) + (uint32_t)(at.stage * m + i) * w : smem_u32(zeros), len);
    tma_store_commit();
    next(at);
    if (at.stage == 0) phase ^= 1;
    // refill the slab before this one, whose stores are an iteration old
    // (waiting for older ones instead leaves fewer slabs on their way: 200
    // moves 287 us against 274)
    if (it >= 1 && ahead.layer < layers) {
      bulk::wait_read1();
      load(ahead);
      next(ahead);
    }
  }
  if (!ok) {
    // gave up: let this CTA's own loads land before its memory is released
    volatile int none = 0;
    for (; at.stage != ahead.stage || at.slab != ahead.slab || at.layer != ahead.layer;) {
      mbar_wait(smem_u32(bars + at.stage), phase, &none);
      next(at);
      if (at.stage == 0) phase ^= 1;
    }
  }
  tma_store_wait0();
}

}  // namespace pool
}  // namespace la2
