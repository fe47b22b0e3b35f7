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
// memory (16-byte granules, no data through registers); a ring of STAGES
// slabs keeps loads in flight while older slabs are being stored.  Thread i
// issues the load and the store of the moves i, i + NT, ..., so a slab buffer
// is refilled by the very thread whose stores read it.
#pragma once

#include "la2_common.cuh"
#include "la2_sm100.cuh"

namespace la2 {
namespace pool {

using namespace sm100;

constexpr int NT = 256;
constexpr int MAX_MOVES = 4096;
constexpr int MAX_W = 8192;       // widest slab
constexpr int MAX_STAGES = 8;
constexpr int SMEM = 227 * 1024;  // what a CTA may have
constexpr int HEAD = 256;         // barriers, counters
// shared memory: HEAD, then MAX_W zero bytes, the list of moves, the ring
constexpr int ring_bytes(int n) { return (SMEM - HEAD - MAX_W - (n * 8 + 127) / 128 * 128) / 128 * 128; }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(src), "r"(bytes)
               : "memory");
}
// all but this thread's newest group of bulk stores have read their source
__device__ __forceinline__ void bulk_wait_read1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

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

  // The slab's width: three slabs of all moves in the ring (two where that
  // would leave less than 512 bytes of each state), and no wider than gives
  // every CTA a slab.
  const int room = ring_bytes(n);
  int w = room / 3 / m;
  if (w < 512) w = room / 2 / m;
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

  const int64_t slabs_row = (bytes + w - 1) / w, slabs = slabs_row * layers;
  const int64_t mine = (slabs - blockIdx.x + gridDim.x - 1) / gridDim.x;  // this CTA's slabs
  auto place = [&](int64_t it, int64_t &layer, int64_t &off, uint32_t &len) {
    const int64_t s = blockIdx.x + it * gridDim.x;
    layer = s / slabs_row;
    off = (s - layer * slabs_row) * w;
    len = (uint32_t)(bytes - off < w ? bytes - off : w);
  };
  auto load = [&](int64_t it) {
    int64_t layer, off;
    uint32_t len, total = 0;
    place(it, layer, off, len);
    const int st = (int)(it % stages);
    for (int i = tid; i < m; i += NT) total += list[i].x >= 0 ? len : 0;
    mbar_expect_tx(smem_u32(bars + st), total);
    for (int i = tid; i < m; i += NT) {
      const int s = list[i].x;
      if (s >= 0)
        bulk_load(smem_u32(ring + ((int64_t)st * m + i) * w),
                  from + (layer * from_size + s) * bytes + off, len, smem_u32(bars + st));
    }
  };
  const int ahead = stages - 1;
  for (int64_t it = 0; it < ahead && it < mine; it++) load(it);
  int64_t it = 0;
  bool ok = true;
  for (; it < mine; it++) {
    if (it + ahead < mine && it == 0) load(ahead);  // the one buffer not yet used
    const int st = (int)(it % stages);
    ok = mbar_wait(smem_u32(bars + st), (uint32_t)(it / stages) & 1, abort);
    if (!ok) break;
    int64_t layer, off;
    uint32_t len;
    place(it, layer, off, len);
    for (int i = tid; i < m; i += NT)
      bulk_store(to + (layer * to_size + list[i].y) * bytes + off,
                 list[i].x >= 0 ? smem_u32(ring + ((int64_t)st * m + i) * w) : smem_u32(zeros), len);
    tma_store_commit();
    // refill the slab before this one, whose stores are an iteration old
    if (it >= 1 && it + ahead < mine) {
      bulk_wait_read1();
      load(it + ahead);
    }
  }
  if (!ok) {
    // gave up: let this CTA's own loads land before its memory is released
    volatile int none = 0;
    for (int64_t j = it; j <= it + ahead && j < mine; j++)
      mbar_wait(smem_u32(bars + j % stages), (uint32_t)(j / stages) & 1, &none);
  }
  tma_store_wait0();
}

}  // namespace pool
}  // namespace la2
