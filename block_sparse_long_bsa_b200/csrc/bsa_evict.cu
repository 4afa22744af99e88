// Cutting a paged key/value cache to a budget by accumulated attention weight
// (sm_100a): every key/value head of every sequence keeps its `budget` cached
// tokens, the `recent` newest and then those of largest weight, moved into
// its first slots.
//
// A kept token that lies below the budget stays where it is; the kept ones
// behind it move into the holes, the i-th hole taking the i-th of them.  So a
// row is read only behind the budget and written only below it: every move is
// independent of the others, and as few as possible are made (attention does
// not ask for the order of its keys; `tokens` says which token a slot holds).
//
// Kernel 1 (select_kernel), a cluster of blocks per (sequence, key/value
// head): weights become 32-bit keys whose unsigned order is theirs (protected
// tokens above all), held in shared memory; the budget-th largest is found
// digit by digit (11, 11 and 10 bits, a histogram each, summed over the
// cluster); ties at it go to the lowest slots; ranks of holes and movers come
// from ballots and scans over warps and blocks.
// Kernel 2 (move_kernel), a warp per 32 slots: new weights, tokens and
// lengths, and the moved rows, 16 bytes a lane.  Small cuts have this done by
// kernel 1's block instead.  Its bound is memory: 4 d
// bytes read and written a moved token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>
#include <string>

#include "bsa_device.cuh"
#include "bsa_internal.h"

namespace bsa {
namespace evict {

using ptx::grid_release;
using ptx::grid_wait;
using ptx::cluster_arrive;
using ptx::cluster_sync;
using ptx::cluster_wait;
using ptx::ld_peer;
using ptx::peer_addr;

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kBins = 4 * kSelThreads;          // of an 11-bit digit, four a thread
static_assert(kBins == 2048, "11-bit digits");
constexpr int kBatch = 8;                       // loads of a thread in flight
constexpr int kMaxCluster = 8, kSlotsPerBlock = kBatch * kSelThreads;
constexpr int kKeysInSmem = 48 * 1024;          // a block with more slots recomputes its keys in every pass
constexpr int kMoveThreads = 256;
constexpr int kMaxSlots = 1 << 30;              // of a layout: a thread's next slots stay inside 32 bits

struct Params {
  __nv_bfloat16* kc;
  __nv_bfloat16* vc;
  const int32_t* page_table;
  const int32_t* lengths;
  const float* weights;
  const int32_t* tokens;      // null: slot s holds token s
  float* weights_out;
  int32_t* tokens_out;
  int32_t* lengths_out;
  int32_t* src;               // [rows][cap]: s for a kept slot s, -1 - i for the i-th hole
  int32_t* movers;            // [rows][cap]: the kept slots behind the budget
  int4* meta;                 // [rows]: kept, newest token, 1 if refused, 1 if nothing moves
  uint32_t* status;
  size_t stride;              // of weights, tokens and their outputs
  int n, B, max_blocks, num_pages, hkv, budget, recent, cap;
};

// Order-preserving key of a weight; a NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t b = w == 0.f ? 0u : __float_as_uint(w);
  return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return int(r);
}
__device__ __forceinline__ void add_peer(uint32_t a, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Slot s of a row after the cut (a thread each, warps whole): its weight and
// token, and the row that moves into it.  m: kept, newest token, -, 1 if nothing moves.
template <int HD>
__device__ __forceinline__ void move_slot(const Params& p, int row, int s, int4 m) {
  constexpr int LPR = HD / 8;            // lanes of a row, 16 bytes each
  constexpr int SPI = 32 / (2 * LPR);    // tokens a warp moves at once (key and value)
  const int b = row / p.hkv, hk = row - b * p.hkv;
  const int lane = threadIdx.x & 31;
  const size_t at = size_t(row) * p.stride;
  int from = s;
  if (s < p.n) {
    float wt = 0.f;
    int t = int(int64_t(m.y) + 1 + (s - m.x));               // a slot behind takes the next token to come
    if (s < m.x) {
      if (!m.w) from = p.src[size_t(row) * p.cap + s];
      if (from < 0) from = p.movers[size_t(row) * p.cap + (-1 - from)];
      wt = p.weights[at + from];
      t = p.tokens ? p.tokens[at + from] : from;
    }
    p.weights_out[at + s] = wt;
    p.tokens_out[at + s] = t;
  }
  unsigned todo = __ballot_sync(0xffffffffu, from != s);
  if (!todo) return;
  // rows of the caches, counted in d-element rows (64-bit: long caches pass 2^31 elements)
  int64_t to_row = 0, from_row = 0;
  if (from != s) {
    const int32_t* pt = p.page_table + size_t(b) * p.max_blocks;
    to_row = (int64_t(pt[s / p.B]) * p.hkv + hk) * p.B + s % p.B;
    from_row = (int64_t(pt[from / p.B]) * p.hkv + hk) * p.B + from % p.B;
  }
  const int sub = lane / (2 * LPR), in = lane % (2 * LPR);
  uint4* const base = reinterpret_cast<uint4*>(in < LPR ? p.kc : p.vc) + in % LPR;
  while (todo) {
    constexpr int U = 4;                 // tokens in flight, times SPI
    uint4 v[U];
    int64_t dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // SPI tokens of the ballot: one for each part of the warp
      int x = -1;
#pragma unroll
      for (int y = 0; y < SPI; ++y) {
        const int first = todo ? __ffs(todo) - 1 : -1;
        if (todo) todo &= todo - 1;
        if (y == sub) x = first;
      }
      const int64_t f = __shfl_sync(0xffffffffu, from_row, x & 31);
      dst[u] = __shfl_sync(0xffffffffu, to_row, x & 31);
      if (x < 0) dst[u] = -1;
      else v[u] = base[f * LPR];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] >= 0) base[dst[u] * LPR] = v[u];
  }
}

// A cluster of C blocks per row; block r owns the slots [r per, (r + 1) per).
// Each block adds the bins that it has keys in (few: the keys under one prefix
// share their upper bits) to every block's sum of histograms; the newest
// token, ties, holes and movers before it a block reads from the others' shared
// memory after a barrier.  Nothing read so is written again.  The loops are not
// unrolled: a block runs through them once or a few times, and fetching their
// instructions is what it would wait for.
// HD > 0: C is 1, the block goes on to move the rows, and no second kernel runs.
template <int HD>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const Params p, int C) {
  extern __shared__ uint32_t s_keys[];
  __shared__ __align__(16) int hist[kBins];       // this block's
  __shared__ __align__(16) int sums[3][kBins];    // the cluster's, a digit each
  __shared__ int s_scan[3][kSelWarps];
  __shared__ int s_bad, s_newest, s_digit, s_left, s_equal, s_holes, s_movers;
  const int row = blockIdx.x / C, rank = cluster_rank();
  const int b = row / p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  reinterpret_cast<int4*>(hist)[tid] = make_int4(0, 0, 0, 0);
#pragma unroll
  for (int d = 0; d < 3; ++d) reinterpret_cast<int4*>(sums[d])[tid] = make_int4(0, 0, 0, 0);
  if (tid == 0) {
    s_bad = 0;
    s_newest = INT32_MIN;
  }
  cluster_sync();                                // every block's sums are zero
  grid_wait();                                   // nothing of the caller's is read or written before this
  grid_release();
  const int len = p.lengths[b];
  const float* w = p.weights + size_t(row) * p.stride;
  const int32_t* tok = p.tokens ? p.tokens + size_t(row) * p.stride : nullptr;
  auto refuse = [&]() {
    if (tid == 0 && rank == 0) {
      if (HD == 0) p.meta[row] = make_int4(0, 0, 1, 1);
      else if (row % p.hkv == 0) p.lengths_out[b] = -1;
      atomicOr(p.status, kStatusBadIndex);
    }
  };
  // the end of a row that is not refused
  auto finish = [&](int4 m) {
    if constexpr (HD > 0) {
      if (tid == 0 && row % p.hkv == 0) p.lengths_out[b] = m.x;
#pragma unroll 1
      for (int s0 = 0; s0 < p.n; s0 += kSelThreads) move_slot<HD>(p, row, s0 + tid, m);
    } else if (tid == 0 && rank == 0) {
      p.meta[row] = m;
    }
  };
  if (len < 0 || len > p.n) {
    refuse();
    return;
  }
  if (len > p.budget) {
    // every block of the cluster looks at all pages, so all agree; the answer
    // is read once the keys are there
    bool bad = false;
    for (int j = tid; j < (len + p.B - 1) / p.B; j += kSelThreads) {
      const int pg = p.page_table[size_t(b) * p.max_blocks + j];
      bad |= pg < 0 || pg >= p.num_pages;
    }
    if (bad) s_bad = 1;
  }
  const int per = (len + C * 32 - 1) / (C * 32) * 32;
  const int first = min(len, rank * per), end = min(len, first + per);
  // the newest token, from which the protected ones are counted back
  int newest = len - 1;
  if (tok) {
    int m = INT32_MIN;
    for (int s0 = first + tid; s0 < end; s0 += kBatch * kSelThreads) {
      int t[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) t[i] = s0 + i * kSelThreads < end ? tok[s0 + i * kSelThreads] : INT32_MIN;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) m = max(m, t[i]);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) atomicMax(&s_newest, m);
    cluster_sync();
    newest = INT32_MIN;
#pragma unroll 1
    for (int r = 0; r < C; ++r) newest = max(newest, ld_peer(peer_addr(&s_newest, r)));
    if (len == 0) newest = -1;
  }
  if (len <= p.budget) {
    cluster_sync();                      // the others may still be reading s_newest here
    finish(make_int4(len, newest, 0, 1));
    return;
  }
  const int64_t floor_tok = int64_t(newest) - p.recent;      // tokens above it are protected
  auto key_from = [&](int t, float x) -> uint32_t { return int64_t(t) > floor_tok ? 0xffffffffu : key_of(x); };
  auto make_key = [&](int s) -> uint32_t { return key_from(tok ? tok[s] : s, w[s]); };
  const bool held = per <= kKeysInSmem;
  if (held) {
    for (int s0 = first + tid; s0 < end; s0 += kBatch * kSelThreads) {
      float x[kBatch];
      int t[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int s = s0 + i * kSelThreads;
        x[i] = s < end ? w[s] : 0.f;
        t[i] = tok && s < end ? tok[s] : s;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (s0 + i * kSelThreads < end) s_keys[s0 - first + i * kSelThreads] = key_from(t[i], x[i]);
    }
  }
  auto key_at = [&](int s) -> uint32_t { return held ? s_keys[s - first] : make_key(s); };
  __syncthreads();
  if (s_bad) {
    refuse();
    if (C > 1) cluster_sync();           // the others may still be reading s_newest here
    return;
  }

  // ---- the budget-th largest key, from the highest digit down
  uint32_t prefix = 0, mask = 0;
  int left = p.budget;                   // how many of the keys under the prefix are kept
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
    const uint32_t dm = d == 2 ? 1023u : 2047u;
#pragma unroll 1
    for (int s0 = first; s0 < end; s0 += kSelThreads) {
      const int s = s0 + tid;            // a thread reads the keys that it wrote
      const uint32_t k = s < end ? key_at(s) : 0u;
      const bool in = s < end && (k & mask) == prefix;
      const int bin = in ? int(k >> shift & dm) : -1;
      // one bin for the whole warp (a run of equal weights) is one addition
      int same;
      __match_all_sync(0xffffffffu, bin, &same);
      if (same) {
        if (lane == 0 && bin >= 0) atomicAdd(&hist[bin], 32);
      } else if (in) {
        atomicAdd(&hist[bin], 1);
      }
    }
    __syncthreads();
    // each thread owns four bins, thread 0 the highest ones
    const int top = kBins - 4 - 4 * tid;
    int4 c = *reinterpret_cast<const int4*>(&hist[top]);
    if (C > 1) {
      const int own4[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (own4[x])
#pragma unroll 1
          for (int r = 0; r < C; ++r) add_peer(peer_addr(&sums[d][top + x], r), own4[x]);
      cluster_sync();
      c = *reinterpret_cast<const int4*>(&sums[d][top]);
    }
    // the last digit's own counts are read by the other blocks
    if (d < 2) *reinterpret_cast<int4*>(&hist[top]) = make_int4(0, 0, 0, 0);
    // the digit whose keys, counted from above, reach `left`
    const int own = c.x + c.y + c.z + c.w;
    int sum = own;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += y;
    }
    if (lane == 31) s_scan[d][warp] = sum;
    __syncthreads();
    // sums of the warps before, by the lanes
    sum += __reduce_add_sync(0xffffffffu, lane < warp ? s_scan[d][lane & (kSelWarps - 1)] : 0);
    int above = sum - own;               // keys in higher bins than the thread's
    if (above < left && left <= sum) {
      const int bin[4] = {c.w, c.z, c.y, c.x};
      int x = 0;
      while (above + bin[x] < left) above += bin[x++];
      s_digit = top + 3 - x;
      s_left = left - above;
      s_equal = bin[x];
    }
    __syncthreads();
    prefix |= uint32_t(s_digit) << shift;
    mask |= dm << shift;
    left = s_left;
    if (s_equal == left) break;          // all keys under the prefix stay: its lower bits do not matter
  }
  const bool split = s_equal > left;     // some keys equal to the last one stay, some go
  // keys above `prefix` are kept, and of those equal to it the first `left`

  // ---- ranks: each warp owns a run of the block's slots
  const int wper = (end - first + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
  const int lo = min(end, first + warp * wper), hi = min(end, lo + wper);
  // how many of a count come before this warp in the block
  auto before = [&](int* scan, int count, int& total) -> int {
    if (lane == 0) scan[warp] = count;
    __syncthreads();
    const int v = scan[lane & (kSelWarps - 1)];
    total = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? v : 0);
    return __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
  };
  int total = 0, ties = 0;
  if (split) {
#pragma unroll 1
    for (int r = 0; r < rank; ++r) ties += ld_peer(peer_addr(&hist[prefix & 1023u], r));
    int count = 0;
#pragma unroll 1
    for (int s0 = lo; s0 < hi; s0 += 32) {
      const int s = s0 + lane;
      count += __popc(__ballot_sync(0xffffffffu, s < hi && key_at(s) == prefix));
    }
    ties += before(s_scan[0], count, total);
  }
  // kept slots of a ballot, with the ties seen so far
  auto kept_of = [&](int s0, int& seen) -> unsigned {
    const int s = s0 + lane;
    const uint32_t k = s < hi ? key_at(s) : 0u;
    const unsigned eq = __ballot_sync(0xffffffffu, s < hi && k == prefix);
    const bool take = s < hi && (k > prefix || (k == prefix && seen + __popc(eq & ((1u << lane) - 1u)) < left));
    seen += __popc(eq);
    return __ballot_sync(0xffffffffu, take);
  };
  int holes = 0, movers = 0, seen = ties;
#pragma unroll 4
  for (int s0 = lo; s0 < hi; s0 += 32) {
    const unsigned kept = kept_of(s0, seen);
    // slots of this ballot that lie below the budget
    const int below = min(32, max(0, min(p.budget, hi) - s0));
    const unsigned low = below == 32 ? 0xffffffffu : (1u << below) - 1u;
    holes += __popc(~kept & low);
    movers += __popc(kept & ~low);
  }
  int hole0 = before(s_scan[1], holes, total);
  if (tid == 0) s_holes = total;
  int mover0 = before(s_scan[2], movers, total);
  if (tid == 0) s_movers = total;
  cluster_sync();
#pragma unroll 1
  for (int r = 0; r < rank; ++r) {
    hole0 += ld_peer(peer_addr(&s_holes, r));
    mover0 += ld_peer(peer_addr(&s_movers, r));
  }
  cluster_arrive();
  int32_t* const mv = p.movers + size_t(row) * p.cap;
  int32_t* const src = p.src + size_t(row) * p.cap;
  seen = ties;
#pragma unroll 1
  for (int s0 = lo; s0 < hi; s0 += 32) {
    const unsigned kept = kept_of(s0, seen);
    const int s = s0 + lane;
    const bool is = kept >> lane & 1u, low = s < p.budget && s < hi;
    const unsigned mb = __ballot_sync(0xffffffffu, is && !low), hb = __ballot_sync(0xffffffffu, low && !is);
    const unsigned under = (1u << lane) - 1u;
    if (is && !low) mv[mover0 + __popc(mb & under)] = s;
    if (low) src[s] = is ? s : -1 - (hole0 + __popc(hb & under));
    mover0 += __popc(mb);
    hole0 += __popc(hb);
  }
  cluster_wait();                        // no block ends while another may still read its shared memory
  if (HD > 0) __syncthreads();           // the lists are written
  finish(make_int4(p.budget, newest, 0, 0));
}

template <int HD>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const Params p, int tiles) {
  const int row = blockIdx.x / tiles, tile = blockIdx.x - row * tiles;
  const int b = row / p.hkv, hk = row - b * p.hkv;
  // (no early start for the kernel after this one: the next cut's blocks took
  // room from the moves, 47 us a call against 49)
  grid_wait();
  const int4 m = p.meta[row];
  if (m.z) {                             // refused: left as it was
    if (tile == 0 && threadIdx.x == 0 && hk == 0) p.lengths_out[b] = -1;
    return;
  }
  if (tile == 0 && threadIdx.x == 0 && hk == 0) p.lengths_out[b] = m.x;
  move_slot<HD>(p, row, tile * kMoveThreads + threadIdx.x, m);
}

bool aligned(const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) % a) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int check_sizes(const bsa_layout* layout, int batch, int kv_heads, int budget) {
  if (!layout) return set_error(BSA_ERR_INVALID_ARG, "layout is NULL");
  if (layout->B != 64 && layout->B != 128) return set_error(BSA_ERR_UNSUPPORTED, "B must be 64 or 128");
  if (batch < 1 || kv_heads < 1) return set_error(BSA_ERR_SHAPE, "batch and kv_heads must be >= 1");
  if (kv_heads % batch) return set_error(BSA_ERR_SHAPE, "kv_heads must be a multiple of batch");
  if (budget < 1) return set_error(BSA_ERR_SHAPE, "budget must be >= 1");
  if (layout->n > kMaxSlots) return set_error(BSA_ERR_SHAPE, "n must be at most 2^30");
  if (int64_t(kv_heads) * std::max<int64_t>(kMaxCluster, (int64_t(layout->n) + kMoveThreads - 1) / kMoveThreads) >
      INT32_MAX)
    return set_error(BSA_ERR_SHAPE, "too many slots");
  return BSA_OK;
}

size_t bytes_of(const bsa_layout* layout, int kv_heads, int budget, size_t* movers, size_t* meta) {
  const size_t list = up256(size_t(kv_heads) * std::min(budget, layout->n) * 4);
  *movers = list;
  *meta = 2 * list;
  return 2 * list + size_t(kv_heads) * sizeof(int4);
}

int launch(const Params& p, int rows, int d, cudaStream_t stream) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return set_error(BSA_ERR_CUDA, "cannot query the device");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      for (auto kern : {select_kernel<0>, select_kernel<64>, select_kernel<128>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysInSmem * 4);
      if (e != cudaSuccess) return set_error(BSA_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
      done[dev] = true;
    }
  }
  // blocks per row: one for each kSlotsPerBlock slots, so that a thread has one
  // batch of them, while the GPU holds them two to an SM (a figure for speed
  // alone: any number of blocks is right on any GPU)
  int C = 1;
  while (C < kMaxCluster && p.n > C * kSlotsPerBlock && rows * C <= 148) C *= 2;
  const int per = (p.n + C * 32 - 1) / (C * 32) * 32;
  // One kernel where a row has one block and few slots or moves, of which there
  // are at most min(budget, n - budget), n being what the host knows: a launch
  // less, but a row's own block takes its slots 512 at a time.  (us on the GPU
  // alone, in graphs, one kernel and two.  Slots, cut to a half: 256 rows of
  // 1024 15.1 and 19.2, of 1100 21.1 and 21.4, of 1300 24.2 and 23.0; 8 rows of
  // 1024 9.7 and 9.7, of 1100 13.4 and 11.0.  Moves, all slots full: 256 rows
  // cut to 4096 by 100 24.9 and 27.8, by 128 26.1 and 28.6, by 256 32.3 and
  // 33.8; 8 rows of 2000 cut by 64 10.6 and 9.9, by 128 11.1 and 10.4, by 256
  // 12.9 and 10.4, launched one by one 11.9 and 13.4 by 128, 13.6 and 13.6 by 256.)
  const bool alone = C == 1 && (p.n <= 2 * kSelThreads || std::min(p.budget, p.n - p.budget) <= kSelThreads / 4);
  const auto select = !alone ? select_kernel<0> : d == 128 ? select_kernel<128> : select_kernel<64>;
  int st = launch_dependent("eviction select launch", select, unsigned(rows) * unsigned(C), kSelThreads,
                            size_t(std::min(per, kKeysInSmem)) * 4, unsigned(C), stream, p, C);
  if (st != BSA_OK || alone) return st;
  const int tiles = (p.n + kMoveThreads - 1) / kMoveThreads;
  const unsigned grid = unsigned(rows) * unsigned(tiles);
  return d == 128 ? launch_dependent("eviction move launch", move_kernel<128>, grid, kMoveThreads, 0, 1, stream, p, tiles)
                  : launch_dependent("eviction move launch", move_kernel<64>, grid, kMoveThreads, 0, 1, stream, p, tiles);
}

}  // namespace evict
}  // namespace bsa

extern "C" {

size_t bsa_evict_workspace_bytes(const bsa_layout* layout, int batch, int kv_heads, int budget) {
  if (bsa::evict::check_sizes(layout, batch, kv_heads, budget) != BSA_OK) return 0;
  size_t a, b;
  return bsa::evict::bytes_of(layout, kv_heads, budget, &a, &b);
}

int bsa_evict(void* k_cache, void* v_cache, const int32_t* page_table, int max_blocks, int num_pages,
              const int32_t* lengths, const float* weights, const int32_t* tokens, const bsa_layout* layout, int batch,
              int kv_heads, int d, int budget, int recent, size_t stride, float* weights_out, int32_t* tokens_out,
              int32_t* lengths_out, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace bsa;
  if (!layout) return set_error(BSA_ERR_INVALID_ARG, "layout is NULL");
  int st = evict::check_sizes(layout, batch, kv_heads, budget);
  if (st != BSA_OK) return st;
  if (d != 64 && d != 128) return set_error(BSA_ERR_UNSUPPORTED, "d must be 64 or 128");
  if (recent < 0 || recent > budget) return set_error(BSA_ERR_SHAPE, "recent must lie in [0, budget]");
  if (max_blocks < layout->nb) return set_error(BSA_ERR_SHAPE, "max_blocks is smaller than the layout's blocks");
  if (num_pages < 1) return set_error(BSA_ERR_SHAPE, "num_pages must be >= 1");
  if (stride < size_t(layout->n)) return set_error(BSA_ERR_SHAPE, "stride is smaller than the layout's n");
  if (!k_cache || !v_cache || !page_table || !lengths || !weights || !weights_out || !tokens_out || !lengths_out ||
      !workspace)
    return set_error(BSA_ERR_INVALID_ARG, "null pointer");
  if (!evict::aligned(k_cache, 16) || !evict::aligned(v_cache, 16) || !evict::aligned(workspace, 16))
    return set_error(BSA_ERR_INVALID_ARG, "k_cache, v_cache and workspace must be 16-byte aligned");
  for (const void* x : {static_cast<const void*>(page_table), static_cast<const void*>(lengths),
                        static_cast<const void*>(weights), static_cast<const void*>(tokens),
                        static_cast<const void*>(weights_out), static_cast<const void*>(tokens_out),
                        static_cast<const void*>(lengths_out)})
    if (!evict::aligned(x, 4)) return set_error(BSA_ERR_INVALID_ARG, "arrays must be 4-byte aligned");
  if (weights_out == weights || tokens_out == tokens || lengths_out == lengths)
    return set_error(BSA_ERR_INVALID_ARG, "weights_out, tokens_out and lengths_out must not be the inputs");
  size_t movers = 0, meta = 0;
  const size_t need = evict::bytes_of(layout, kv_heads, budget, &movers, &meta);
  if (workspace_bytes < need)
    return set_error(BSA_ERR_SHAPE, "workspace too small: " + std::to_string(need) + " bytes needed");
  st = check_layout_device(layout);
  if (st != BSA_OK) return st;
  evict::Params p{};
  p.kc = static_cast<__nv_bfloat16*>(k_cache);
  p.vc = static_cast<__nv_bfloat16*>(v_cache);
  p.page_table = page_table;
  p.lengths = lengths;
  p.weights = weights;
  p.tokens = tokens;
  p.weights_out = weights_out;
  p.tokens_out = tokens_out;
  p.lengths_out = lengths_out;
  char* w = static_cast<char*>(workspace);
  p.src = reinterpret_cast<int32_t*>(w);
  p.movers = reinterpret_cast<int32_t*>(w + movers);
  p.meta = reinterpret_cast<int4*>(w + meta);
  p.status = layout->d_status;
  p.stride = stride;
  p.n = layout->n;
  p.B = layout->B;
  p.max_blocks = max_blocks;
  p.num_pages = num_pages;
  p.hkv = kv_heads / batch;
  p.budget = budget;
  p.recent = recent;
  p.cap = std::min(budget, layout->n);
  return evict::launch(p, kv_heads, d, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
