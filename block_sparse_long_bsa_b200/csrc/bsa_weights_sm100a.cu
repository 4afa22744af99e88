// The attention weight that every key of a prompt has received (sm_100a):
//   w[g][u] += sum over the query heads f of key/value head g and the tokens t
//              whose layout row keeps u's block (u <= t) of
//              exp(scale <q_t, k_u> - lse_t),
// the column sums of the forward's probabilities, rebuilt from its lse as the
// gradients rebuild them; no n x n matrix exists.
//
// One work item is a run of at most 16 query blocks of a key block's column of
// the transposed layout (the segments of the key/value gradients) against one
// 64-key chunk of that block.  The chunk's keys stay in shared memory for the
// whole run; the query rows that read them stream past in 128-row tiles (two
// blocks of 64, or one of 128):
//   S = Q K^T                 (tcgen05.mma, bf16 x bf16 -> fp32 in TMEM)
//   acc[c] += exp2(S[r][c] scale log2 e - lse_r log2 e)
// A thread owns one tile row and keeps the 64 running sums of its row slot in
// registers, so the sum over rows is taken once per run, not per tile: a
// transposing butterfly inside each warp, then the four warps in order.  All
// sums are fp32 and their order is fixed by the layout alone, so results do
// not change from run to run: runs leave partial sums in the caller's
// workspace and a second kernel adds each column's runs in order.
//
// Roles (192 threads, two CTAs per SM): warp 0 issues the TMA loads, warp 1
// the products, warps 2-5 hold the rows.  Every wait is bounded as in the
// forward.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <string>

#include "bsa_device.cuh"
#include "bsa_internal.h"
#include "bsa_tmap.h"

namespace bsa {
namespace wts {

using namespace ptx;

constexpr int kThreads = 192;
constexpr int kTileM = 128;
constexpr int kChunk = 64;           // keys of a work item
constexpr int kQSlots = 2, kKSlots = 2, kSBufs = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kWaitNs = 1000000000ull, kDrainNs = 200000000ull;

struct Params {
  const int32_t* col_ptr;
  const int32_t* row_idx;
  const int32_t* seg_ptr;
  const int32_t* segs;
  const float* lse;
  float* part;               // [head group][slot][B]
  float* weights;
  size_t weights_stride;
  uint32_t* status;
  int n, nb, L, g, kv_heads;
  int hpg;                   // query heads of a head group: a key/value head's, or one when routes differ by head
  int groups;                // head groups
  int max_segs, slots;
  int64_t items;             // groups * max_segs * chunks of a block
  float scale_log2;
};

template <int BLK, int HD>
struct Shape {
  static constexpr int kCPB = BLK / kChunk;
  static constexpr int kSubs = kTileM / BLK;                  // query blocks of a tile
  static constexpr int kQBytes = kTileM * HD * 2;
  static constexpr int kKBytes = kChunk * HD * 2;
  static constexpr int kAtomQ = kTileM * 128, kAtomK = kChunk * 128;
  static constexpr int kOffK = kQSlots * kQBytes;
  static constexpr int kOffRed = kOffK + kKSlots * kKBytes;   // [2][4 warps][64] partial column sums
  static constexpr int kOffBar = kOffRed + 2 * 4 * kChunk * 4;
  // q_full, q_free, k_full, k_free, s_full, s_free, drain
  static constexpr int kNumBars = 2 * kQSlots + 2 * kKSlots + 2 * kSBufs + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 16;
  static constexpr uint32_t kTmemCols = kSBufs * kChunk;      // 256
  static constexpr uint32_t kIdesc = idesc_bf16(kTileM, kChunk, 0, 0);
};

// A work item, decoded the same way by every role.
struct Item {
  int j, e0, units;          // key block, first entry of the run, (query block, head) pairs
  int kv, f0, chunk;         // key/value head, first query head, 64-key chunk of the block
  size_t slot;               // row of the partial sums
};

template <int BLK>
__device__ __forceinline__ bool decode(const Params& p, int64_t it, Item& x) {
  constexpr int CPB = BLK / kChunk;
  const int per = p.max_segs * CPB;
  const int grp = int(it / per), rest = int(it - int64_t(grp) * per);
  const int seg = rest / CPB;
  x.chunk = rest - seg * CPB;
  x.f0 = grp * p.hpg;
  x.kv = x.f0 / p.g;
  const int lh = x.f0 % p.L;
  const int s0 = p.seg_ptr[lh];
  if (seg >= p.seg_ptr[lh + 1] - s0) return false;
  const int32_t* s = p.segs + 3 * size_t(s0 + seg);
  x.j = s[0];
  x.e0 = s[1];
  x.units = s[2] * p.hpg;
  // entry / 16 + block grows by at least one from run to run (a column's runs
  // start 16 entries apart, a new column adds its block), so it names the run
  x.slot = size_t(grp) * p.slots + (x.e0 / kColumnSegment - p.col_ptr[size_t(lh) * p.nb] / kColumnSegment) + x.j;
  return true;
}

__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
  asm("{\n\t.reg .b64 ra, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rd, {%0, %1};\n\t"
      "add.rn.f32x2 rd, rd, ra;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}

template <int BLK, int HD>
__global__ void __launch_bounds__(kThreads, 2)
    prompt_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const Params p) {
  using S = Shape<BLK, HD>;
  constexpr int SUBS = S::kSubs;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_addr(smem);
  if (base & 1023u) {                // never expected: the swizzle needs 1024-byte aligned tiles
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t sQ = base, sK = base + S::kOffK, bar0 = base + S::kOffBar;
  const uint32_t bQFull0 = bar0, bQFree0 = bQFull0 + 8u * kQSlots, bKFull0 = bQFree0 + 8u * kQSlots,
                 bKFree0 = bKFull0 + 8u * kKSlots, bSFull0 = bKFree0 + 8u * kKSlots, bSFree0 = bSFull0 + 8u * kSBufs,
                 bDrain = bSFree0 + 8u * kSBufs;
  float* red = reinterpret_cast<float*>(smem + S::kOffRed);
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(smem + S::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Ctl ctl{abort_flag, p.status, kWaitNs};
  if (threadIdx.x == 0) {
    for (int s = 0; s < kQSlots; ++s) {
      mbar_init(bQFull0 + 8u * s, 1);
      mbar_init(bQFree0 + 8u * s, 1);
    }
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(bKFull0 + 8u * s, 1);
      mbar_init(bKFree0 + 8u * s, 1);
    }
    for (int s = 0; s < kSBufs; ++s) {
      mbar_init(bSFull0 + 8u * s, 1);
      mbar_init(bSFree0 + 8u * s, 128);
    }
    mbar_init(bDrain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch(&tmQ);
    tma_prefetch(&tmK);
  }
  if (warp == 1) {
    tmem_alloc(base + S::kOffMisc, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  // Tiles are counted over all items of the CTA (t), items with k: tile t uses
  // Q slot t % 2 and S buffer t % 4, item k the K slot k % 2.
  if (warp == 0) {
    // ================================================================ loads
    if (lane == 0) {
      int t = 0, k = 0;
      bool ok = true;
      for (int64_t it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
        Item x;
        if (!decode<BLK>(p, it, x)) continue;
        if (k >= kKSlots && !(ok = ctl.wait(bKFree0 + 8u * (k % kKSlots), uint32_t(k / kKSlots - 1) & 1u))) break;
        const uint32_t bk = bKFull0 + 8u * (k % kKSlots);
        mbar_expect_tx(bk, S::kKBytes);
        tma_load_kv<HD>(sK + (k % kKSlots) * S::kKBytes, &tmK, bk, x.j * BLK + x.chunk * kChunk, x.kv);
        ++k;
        const int tiles = (x.units + SUBS - 1) / SUBS;
        for (int y = 0; y < tiles && ok; ++y) {
          if (t >= kQSlots && !(ok = ctl.wait(bQFree0 + 8u * (t % kQSlots), uint32_t(t / kQSlots - 1) & 1u))) break;
          const uint32_t bq = bQFull0 + 8u * (t % kQSlots), dst = sQ + (t % kQSlots) * S::kQBytes;
          mbar_expect_tx(bq, S::kQBytes);
#pragma unroll
          for (int sub = 0; sub < SUBS; ++sub) {
            // a tile without a second block repeats the first; its rows are left out
            const int u = min(y * SUBS + sub, x.units - 1);
            const int i = p.row_idx[x.e0 + u / p.hpg], f = x.f0 + u % p.hpg;
#pragma unroll
            for (int a = 0; a < HD / 64; ++a)
              tma_load_3d(dst + a * S::kAtomQ + sub * BLK * 128, &tmQ, bq, a * 64, i * BLK, f);
          }
          ++t;
        }
      }
      // never leave the CTA with copies in flight into its shared memory
      for (int y = t > kQSlots ? t - kQSlots : 0; y < t; ++y)
        wait_drain(bQFull0 + 8u * (y % kQSlots), uint32_t(y / kQSlots) & 1u, kDrainNs);
      for (int y = k > kKSlots ? k - kKSlots : 0; y < k; ++y)
        wait_drain(bKFull0 + 8u * (y % kKSlots), uint32_t(y / kKSlots) & 1u, kDrainNs);
    }
  } else if (warp == 1) {
    // ================================================================ products
    if (lane == 0) {
      constexpr uint64_t kFix = sw128_fixed(16, 1024);
      constexpr uint32_t kHi = uint32_t(kFix >> 32);
      const uint32_t q_lo = uint32_t(kFix) + (sQ >> 4), k_lo = uint32_t(kFix) + (sK >> 4);
      int t = 0, k = 0;
      bool ok = true;
      for (int64_t it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
        Item x;
        if (!decode<BLK>(p, it, x)) continue;
        if (!(ok = ctl.wait(bKFull0 + 8u * (k % kKSlots), uint32_t(k / kKSlots) & 1u))) break;
        const uint32_t kb = k_lo + uint32_t(k % kKSlots) * (S::kKBytes >> 4);
        const int tiles = (x.units + SUBS - 1) / SUBS;
        for (int y = 0; y < tiles; ++y) {
          if (!(ok = ctl.wait(bQFull0 + 8u * (t % kQSlots), uint32_t(t / kQSlots) & 1u))) break;
          if (t >= kSBufs && !(ok = ctl.wait(bSFree0 + 8u * (t % kSBufs), uint32_t(t / kSBufs - 1) & 1u))) break;
          tc_fence_after();
          const uint32_t qb = q_lo + uint32_t(t % kQSlots) * (S::kQBytes >> 4);
          const uint32_t d = tmem + (t % kSBufs) * kChunk;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            mma_ss(d, desc_from(qb + ((kk >> 2) * S::kAtomQ + (kk & 3) * 32) / 16, kHi),
                   desc_from(kb + ((kk >> 2) * S::kAtomK + (kk & 3) * 32) / 16, kHi), S::kIdesc, kk > 0 ? 1u : 0u);
          tc_commit(bSFull0 + 8u * (t % kSBufs));
          tc_commit(bQFree0 + 8u * (t % kQSlots));
          ++t;
        }
        if (!ok) break;
        tc_commit(bKFree0 + 8u * (k % kKSlots));
        ++k;
      }
      tc_commit(bDrain);
      wait_drain(bDrain, 0, kDrainNs);
    }
  } else {
    // ================================================================ rows
    const int q4 = warp & 3;
    const int row = q4 * 32 + lane;
    const int sub = row / BLK, rl = row - sub * BLK;
    const uint32_t lane_base = tmem + (uint32_t(q4 * 32) << 16);
    const float sl2 = p.scale_log2;
    int t = 0, k = 0;
    bool ok = true;
    for (int64_t it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
      Item x;
      if (!decode<BLK>(p, it, x)) continue;
      const int tiles = (x.units + SUBS - 1) / SUBS;
      float acc[kChunk];
#pragma unroll
      for (int c = 0; c < kChunk; ++c) acc[c] = 0.f;
      // this thread's row of tile y: its query block and -lse log2 e; -inf for
      // a row that is none or that has no weight to give
      auto row_of = [&](int y, int& i) -> float {
        const int u = y * SUBS + sub;
        i = 0;
        if (y >= tiles || u >= x.units) return -INFINITY;
        i = p.row_idx[x.e0 + u / p.hpg];
        const int tok = i * BLK + rl;
        if (tok >= p.n) return -INFINITY;
        const float lse = p.lse[size_t(x.f0 + u % p.hpg) * p.n + tok];
        return lse == -INFINITY ? -INFINITY : -lse * kLog2e;
      };
      int i = 0;
      float neg = row_of(0, i);
      for (int y = 0; y < tiles; ++y) {
        int i_next = 0;
        const float neg_next = row_of(y + 1, i_next);      // fetched while this tile is worked on
        ok = __all_sync(0xffffffffu, ctl.wait(bSFull0 + 8u * (t % kSBufs), uint32_t(t / kSBufs) & 1u));
        if (!ok) break;
        tc_fence_after();
        float sv[kChunk];
        const uint32_t s_col = lane_base + (t % kSBufs) * kChunk;
        tmem_ld32(s_col, sv);
        tmem_ld32(s_col + 32, sv + 32);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(bSFree0 + 8u * (t % kSBufs));
        ++t;
        if (neg != -INFINITY) {
          if (i == x.j) {
            // the diagonal block: keys up to the row's own token
            const int lim = rl - x.chunk * kChunk;
#pragma unroll
            for (int c = 0; c < kChunk; ++c)
              if (c <= lim) acc[c] += ex2(fmaf(sv[c], sl2, neg));
          } else {
#pragma unroll
            for (int c = 0; c < kChunk; c += 2) {
              float x0, x1;
              fma2(x0, x1, sv[c], sv[c + 1], sl2, neg);
              add2(acc[c], acc[c + 1], ex2(x0), ex2(x1));
            }
          }
        }
        neg = neg_next;
        i = i_next;
      }
      if (!ok) break;
      // 64 sums over the warp's 32 rows: lanes hand half of their columns over
      // at each step, and end with the sums of columns 2 lane and 2 lane + 1
#pragma unroll
      for (int half = kChunk / 2, off = 16; off > 0; half /= 2, off /= 2) {
        const bool high = lane & off;
#pragma unroll
        for (int c = 0; c < kChunk / 2; ++c) {
          if (c < half) {
            const float give = high ? acc[c] : acc[c + half];
            const float keep = high ? acc[c + half] : acc[c];
            acc[c] = keep + __shfl_xor_sync(0xffffffffu, give, off);
          }
        }
      }
      float* to = red + (k & 1) * 4 * kChunk;
      *reinterpret_cast<float2*>(to + q4 * kChunk + 2 * lane) = make_float2(acc[0], acc[1]);
      // two buffers in turn: a warp that writes one again has passed the
      // barrier of the item between, after every read of it
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (row < kChunk)
        p.part[x.slot * BLK + x.chunk * kChunk + row] =
            (to[row] + to[kChunk + row]) + (to[2 * kChunk + row] + to[3 * kChunk + row]);
      ++k;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// w[kv][u] += the runs of u's block, query head by query head and run by run.
template <int BLK>
__global__ void __launch_bounds__(BLK) add_runs_kernel(const Params p) {
  const int kv = blockIdx.x / p.nb, j = blockIdx.x - kv * p.nb;
  const int u = j * BLK + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (u >= p.n) return;
  // a wait that ran out left runs unwritten: nothing is added then
  if (*reinterpret_cast<volatile uint32_t*>(p.status) & kStatusTimeout) return;
  float sum = 0.f;
  for (int h = 0; h < p.g; h += p.hpg) {
    const int f = kv * p.g + h, lh = f % p.L;
    const int c0 = p.col_ptr[size_t(lh) * p.nb + j], c1 = p.col_ptr[size_t(lh) * p.nb + j + 1];
    const int runs = (c1 - c0 + kColumnSegment - 1) / kColumnSegment;
    const size_t slot = size_t(f / p.hpg) * p.slots +
                        (c0 / kColumnSegment - p.col_ptr[size_t(lh) * p.nb] / kColumnSegment) + j;
    const float* src = p.part + slot * BLK + threadIdx.x;
#pragma unroll 8
    for (int r = 0; r < runs; ++r) sum += src[size_t(r) * BLK];
  }
  p.weights[size_t(kv) * p.weights_stride + u] += sum;
}

// Partial-sum rows of a head group: the most that a layout head's runs name.
int slots_of(const bsa_layout* L) {
  int most = 1;
  for (int h = 0; h < L->L; ++h) {
    const int a = L->col_ptr[size_t(h) * L->nb], b = L->col_ptr[size_t(h + 1) * L->nb];
    most = std::max(most, b / kColumnSegment - a / kColumnSegment + L->nb + 1);
  }
  return most;
}

template <int BLK, int HD>
int launch(const void* q, const void* k, int heads, Params p, cudaStream_t stream) {
  using S = Shape<BLK, HD>;
  auto kern = prompt_weights_kernel<BLK, HD>;
  // enough shared memory that no third CTA shares an SM: TMEM holds two
  constexpr int smem = S::kSmem < 77 * 1024 ? 77 * 1024 : S::kSmem;
  static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs per SM");
  static std::mutex mu;
  static int sms[64] = {};
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return set_error(BSA_ERR_CUDA, "cannot query the device");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!sms[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return set_error(BSA_ERR_CUDA, std::string("weights attributes: ") + cudaGetErrorString(e));
      sms[dev] = n_sm;
    }
    n_sm = sms[dev];
  }
  CUtensorMap mq, mk;
  int st = tmap::encode_atoms(&mq, q, heads, p.n, HD, BLK);
  if (st == BSA_OK) st = tmap::encode_kv(&mk, k, p.kv_heads, p.n, HD);
  if (st != BSA_OK) return st;
  p.items = int64_t(p.groups) * p.max_segs * S::kCPB;
  const unsigned grid = unsigned(std::min<int64_t>(p.items, 2 * n_sm));
  kern<<<grid, kThreads, smem, stream>>>(mq, mk, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(BSA_ERR_CUDA, std::string("prompt weights launch: ") + cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.kv_heads) * unsigned(p.nb), 1, 1);
  cfg.blockDim = dim3(BLK, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, add_runs_kernel<BLK>, p);
  if (e != cudaSuccess) return set_error(BSA_ERR_CUDA, std::string("weights sum launch: ") + cudaGetErrorString(e));
  return BSA_OK;
}

bool aligned(const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) % a) == 0; }

int check_sizes(const bsa_layout* layout, int heads, int kv_heads) {
  if (!layout) return set_error(BSA_ERR_INVALID_ARG, "layout is NULL");
  if (layout->B != 64 && layout->B != 128) return set_error(BSA_ERR_UNSUPPORTED, "B must be 64 or 128");
  if (heads < 1 || kv_heads < 1) return set_error(BSA_ERR_SHAPE, "heads and kv_heads must be >= 1");
  if (heads % kv_heads) return set_error(BSA_ERR_SHAPE, "heads must be a multiple of kv_heads");
  if (heads % layout->L) return set_error(BSA_ERR_SHAPE, "heads must be a multiple of layout_heads");
  if (int64_t(heads) * layout->nb > INT32_MAX) return set_error(BSA_ERR_SHAPE, "too many (head, block) work items");
  return BSA_OK;
}

size_t bytes_of(const bsa_layout* layout, int heads, int kv_heads) {
  return size_t(layout->L == 1 ? kv_heads : heads) * slots_of(layout) * layout->B * sizeof(float);
}

}  // namespace wts
}  // namespace bsa

extern "C" {

size_t bsa_attention_weights_workspace_bytes(const bsa_layout* layout, int heads, int kv_heads) {
  if (bsa::wts::check_sizes(layout, heads, kv_heads) != BSA_OK) return 0;
  return bsa::wts::bytes_of(layout, heads, kv_heads);
}

int bsa_attention_weights(const void* q, const void* k, const float* lse, const bsa_layout* layout, int B, int n,
                          int heads, int kv_heads, int d, float scale, float* weights, size_t weights_stride,
                          void* workspace, size_t workspace_bytes, void* stream) {
  using namespace bsa;
  if (!layout) return set_error(BSA_ERR_INVALID_ARG, "layout is NULL");
  if (B != layout->B || n != layout->n) return set_error(BSA_ERR_SHAPE, "B/n differ from the layout's");
  int st = wts::check_sizes(layout, heads, kv_heads);
  if (st != BSA_OK) return st;
  if (d != 64 && d != 128) return set_error(BSA_ERR_UNSUPPORTED, "d must be 64 or 128");
  if (!(std::isfinite(scale) && scale > 0.f)) return set_error(BSA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!q || !k || !lse || !weights || !workspace) return set_error(BSA_ERR_INVALID_ARG, "null pointer");
  if (!wts::aligned(q, 16) || !wts::aligned(k, 16) || !wts::aligned(workspace, 16))
    return set_error(BSA_ERR_INVALID_ARG, "q, k and workspace must be 16-byte aligned");
  if (!wts::aligned(lse, 4) || !wts::aligned(weights, 4))
    return set_error(BSA_ERR_INVALID_ARG, "lse and weights must be 4-byte aligned");
  if (weights_stride < size_t(n)) return set_error(BSA_ERR_SHAPE, "weights_stride is smaller than n");
  const size_t need = wts::bytes_of(layout, heads, kv_heads);
  if (workspace_bytes < need)
    return set_error(BSA_ERR_SHAPE, "workspace too small: " + std::to_string(need) + " bytes needed");
  st = check_layout_device(layout);
  if (st != BSA_OK || layout->max_segs < 1) return st;   // no runs: an explicit mask that keeps no block
  st = tmap::get_encoder();
  if (st != BSA_OK) return st;
  wts::Params p{};
  p.col_ptr = layout->d_col_ptr;
  p.row_idx = layout->d_row_idx;
  p.seg_ptr = layout->d_seg_ptr;
  p.segs = layout->d_segs;
  p.lse = lse;
  p.part = static_cast<float*>(workspace);
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.status = layout->d_status;
  p.n = n;
  p.nb = layout->nb;
  p.L = layout->L;
  p.g = heads / kv_heads;
  p.kv_heads = kv_heads;
  p.hpg = layout->L == 1 ? p.g : 1;
  p.groups = heads / p.hpg;
  p.max_segs = layout->max_segs;
  p.slots = wts::slots_of(layout);
  p.scale_log2 = float(double(scale) * 1.4426950408889634);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 64) return d == 128 ? wts::launch<64, 128>(q, k, heads, p, s) : wts::launch<64, 64>(q, k, heads, p, s);
  return d == 128 ? wts::launch<128, 128>(q, k, heads, p, s) : wts::launch<128, 64>(q, k, heads, p, s);
}

}  // extern "C"
