// The attention weight that every key of a prompt has received (sm_100a):
//   w[g][u] += sum over the query heads f of key/value head g and the tokens t
//              whose layout row keeps u's block (u <= t) of
//              exp(scale <q_t, k_u> - lse_t),
// the column sums of the forward's probabilities, rebuilt from its lse as the
// gradients rebuild them; no n x n matrix exists.
//
// One work item is a query block row (for B = 64 of two query heads that share
// a key/value head and a route, else of one): its NQ <= 128 query rows stay in
// shared memory while the row's kept key blocks stream past, 128 keys at a
// time.  The product is taken with the keys as its rows,
//   S^T = K Q^T               (tcgen05.mma, bf16 x bf16 -> fp32 in TMEM)
// so that a TMEM lane is a key and the sum over queries, of
// exp2(S^T[u][t] scale log2 e - lse_t log2 e), stays inside a thread: no value
// crosses lanes, and a tile costs its exponentials, one fused multiply-add and
// one addition each.  The exponentials, 16 a clock and SM, keep their unit 76 to
// 78 % busy (32K dyadic route, 16 query heads: 124 us a call, 136 to 141 at the
// power limit); a quarter of them elsewhere takes off 5 %, so a second limit is near.
//
// Each kept block leaves its B sums in the caller's workspace, and a second
// kernel adds each key's sums up in row order, so all sums are fp32 in an
// order that the layout alone fixes.  Key/value heads whose kept blocks need
// more than kStripBytes together are worked off in turns that share the workspace.
//
// Roles (480 threads, one CTA per SM): warp 0 looks items up and loads their
// query rows, warp 2 their keys (one warp for both issued a tile per 1300
// cycles, with the products and sums waiting for it), warp 1 issues the
// products; warps 3-14 take the sums in three groups, each a tile of its own
// with a thread per key, so that on every scheduler one group waits, loads and
// stores while the others' exponentials run.  (Sixteen warps
// on one tile, four threads a key, met at a barrier per tile and left the
// exponential unit idle in between: 175 us for the 32K dyadic route.)  Every
// wait is bounded as in the forward.
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

constexpr int kGroups = 3;           // groups of four key warps, a tile each
constexpr int kThreads = 96 + 128 * kGroups;
constexpr int kTileM = 128;          // keys of a tile
constexpr int kQSlots = 2, kKSlots = 4;
constexpr int kSBufs = 4;            // S buffers, one more than groups: the next product is ready in time
// Items in use at once, where every item is one tile: a group gives the S
// buffer of tile t back before it reads the last of its item's lse, and what
// holds the products back then is the group's next tile, t + kGroups, whose
// buffer they need at t + kGroups + kSBufs.  So they may have ended item
// t + kGroups + kSBufs - 1, and the first warp writes kQSlots items further.
constexpr int kItems = 16;
static_assert(kItems >= kGroups + kSBufs + kQSlots, "an item's entry is written again only after its last reader");
static_assert(kKSlots == kSBufs, "a finished product releases its K slot and fills its S buffer");
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kWaitNs = 1000000000ull, kDrainNs = 200000000ull;
constexpr size_t kStripBytes = size_t(64) << 20;

struct Params {
  const int32_t* row_ptr;
  const int32_t* col_idx;
  const int32_t* col_ptr;
  const int32_t* csr_pos;
  const float* lse;
  float* part;               // [unit][slots][B]
  float* weights;
  size_t weights_stride;
  uint32_t* status;
  int n, nb, L, g, heads;
  int pack;                  // query heads of a unit
  int upk;                   // units of a key/value head
  int kv0, kvs;              // the strip's key/value heads
  int64_t slots;             // kept blocks that a unit has room for
  uint32_t items;            // units of the strip * nb
  float scale_log2;
};

template <int BLK, int HD, int PACK>
struct Shape {
  static constexpr int kNQ = BLK * PACK;                      // query rows of an item
  static constexpr int kBPT = kTileM / BLK;                   // key blocks of a tile
  static constexpr int kQBytes = kNQ * HD * 2;
  static constexpr int kKBytes = kTileM * HD * 2;
  static constexpr int kAtomQ = kNQ * 128, kAtomK = kTileM * 128;
  static constexpr int kOffK = kQSlots * kQBytes;
  static constexpr int kOffNeg = kOffK + kKSlots * kKBytes;   // [kItems][128] -lse log2 e
  static constexpr int kOffCols = kOffNeg + kItems * 128 * 4; // [kItems][32] the row's first key blocks
  static constexpr int kOffItem = kOffCols + kItems * 32 * 4;
  static constexpr int kOffBar = kOffItem + kItems * 32;
  // q_full, q_free, k_full, s_full, s_free, item, drain
  static constexpr int kNumBars = 2 * kQSlots + kKSlots + 2 * kSBufs + kItems + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kUsed = kOffMisc + 16;
  // more than half of an SM's shared memory, so that no second CTA shares it:
  // an item's S buffers take up to all of TMEM
  static constexpr int kSmem = kUsed < 116 * 1024 ? 116 * 1024 : kUsed;
  static constexpr uint32_t kTmemCols = kSBufs * kNQ;         // 256 or 512
  static constexpr uint32_t kIdesc = idesc_bf16(kTileM, kNQ, 0, 0);
  static_assert(kNQ == 64 || kNQ == 128, "query rows of an item");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// A work item as the first warp announces it; tiles 0 ends the stream.
struct Item {
  int tiles, blocks;         // tiles and kept blocks of the row
  int diag;                  // the last kept block is the diagonal one
  int dead;                  // a query row of the item has lse = -inf
  int64_t slot;              // first row of partial sums
  int e0, kv;                // first entry in col_idx; key/value head
};
static_assert(sizeof(Item) == 32, "item ring");

__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %6};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
  asm("{\n\t.reg .b64 ra, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rd, {%0, %1};\n\t"
      "add.rn.f32x2 rd, rd, ra;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}
// Waits for the loads of TMEM into v; the registers are operands so that no
// use of them is moved before it while other loads are in flight.
__device__ __forceinline__ void wait_ld32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

template <int BLK, int HD, int PACK>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const Params p) {
  using S = Shape<BLK, HD, PACK>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_addr(smem);
  // rounds of one item per CTA, every other one the other way round, so that
  // no CTA has the longer row of each
  auto item = [&](uint32_t round) -> uint32_t {
    return round * gridDim.x + (round & 1u ? gridDim.x - 1u - blockIdx.x : blockIdx.x);
  };
  const uint32_t rounds = (p.items + gridDim.x - 1) / gridDim.x;
  // an item's unit, query block and first query head, and its place in row_ptr:
  // unit by unit, last row first (rows grow with their index, and a unit's keys stay in L2)
  auto place = [&](uint32_t it, int& unit, int& i, int& f0) -> size_t {
    unit = int(it / uint32_t(p.nb));
    i = p.nb - 1 - int(it - uint32_t(unit) * uint32_t(p.nb));
    f0 = (p.kv0 * p.upk + unit) * PACK;
    return size_t(f0 % p.L) * p.nb + i;
  };
  // The sums of a CTA that gives up are not whole: all of them become -inf,
  // which no sum of exponentials is, and the second kernel leaves their keys as they were.
  auto spoil = [&]() {
    for (uint32_t round = 0; round < rounds; ++round) {
      const uint32_t it = item(round);
      if (it >= p.items) continue;
      int unit, i, f0;
      const size_t at = place(it, unit, i, f0);
      const int e0 = p.row_ptr[at], floats = (p.row_ptr[at + 1] - e0) * BLK;
      float* const out = p.part + (int64_t(unit) * p.slots + (e0 - p.row_ptr[size_t(f0 % p.L) * p.nb])) * BLK;
      for (int x = threadIdx.x; x < floats; x += kThreads) out[x] = -INFINITY;
    }
  };
  if (base & 1023u) {                // never expected: the swizzle needs 1024-byte aligned tiles
    grid_wait();
    spoil();
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  const uint32_t sQ = base, sK = base + S::kOffK, bar0 = base + S::kOffBar;
  const uint32_t bQFull0 = bar0, bQFree0 = bQFull0 + 8u * kQSlots, bKFull0 = bQFree0 + 8u * kQSlots,
                 bSFull0 = bKFull0 + 8u * kKSlots, bSFree0 = bSFull0 + 8u * kSBufs, bItem0 = bSFree0 + 8u * kSBufs,
                 bDrain = bItem0 + 8u * kItems;
  float* negs = reinterpret_cast<float*>(smem + S::kOffNeg);
  volatile int* colss = reinterpret_cast<volatile int*>(smem + S::kOffCols);
  volatile Item* ring = reinterpret_cast<volatile Item*>(smem + S::kOffItem);
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(smem + S::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Ctl ctl{abort_flag, p.status, kWaitNs};
  // phase x / depth of the barrier x % depth of a ring
  auto wait = [&](uint32_t first, int depth, int x) -> bool {
    return ctl.wait(first + 8u * (x % depth), uint32_t(x / depth) & 1u);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * kQSlots + kKSlots + kSBufs; ++s) mbar_init(bQFull0 + 8u * s, 1);
    for (int s = 0; s < kSBufs; ++s) mbar_init(bSFree0 + 8u * s, 4);
    for (int s = 0; s < kItems; ++s) mbar_init(bItem0 + 8u * s, 1);
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
  grid_wait();                                   // nothing of the caller's is read or written before this
  grid_release();

  // Items with kept blocks are counted by k, their tiles over all of them by t:
  // item k uses Q slot k % 2 and ring entry k % 8, tile t K slot and S buffer t % 4.
  if (warp == 0) {
    // ================================================================ items and query rows
    // An item is looked up in two steps, its row's place in the layout and then
    // its key blocks and lse, each of them an item's time ahead of its use: done
    // one after the other when the item comes up they take 4 us, which is the
    // time of four tiles.
    const bool leader = elect_one();
    int k = 0;
    bool ok = true;
    struct Row {
      int unit, i, f0, e0, len;          // e0, len: still in flight until the next step
    };
    auto find_row = [&](uint32_t it) -> Row {
      Row r{0, 0, 0, 0, -1};
      if (it < p.items) {
        const size_t at = place(it, r.unit, r.i, r.f0);
        r.e0 = p.row_ptr[at];
        r.len = p.row_ptr[at + 1];
      }
      return r;
    };
    constexpr int NQ32 = S::kNQ / 32;
    struct Found {
      int cols, last, base;              // lane x holds entry x; the last entry; the layout head's first
      float lse[NQ32];
    };
    auto find_keys = [&](const Row& r) -> Found {
      Found w{0, -1, 0, {}};
      const int len = r.len - r.e0;
      if (r.len >= 0 && len > 0) {
        w.cols = lane < len ? p.col_idx[r.e0 + lane] : 0;
        w.last = p.col_idx[r.e0 + len - 1];
        w.base = p.row_ptr[size_t(r.f0 % p.L) * p.nb];
#pragma unroll
        for (int x = 0; x < NQ32; ++x) {
          const int c = x * 32 + lane, tok = r.i * BLK + c % BLK;
          w.lse[x] = tok < p.n ? p.lse[size_t(r.f0 + c / BLK) * p.n + tok] : -INFINITY;
        }
      }
      return w;
    };
    Row cur = find_row(item(0)), next = find_row(item(1));
    Found mine = find_keys(cur);
    for (uint32_t round = 0; round < rounds && ok; ++round) {
      const Row after = find_row(item(round + 2));
      const Found theirs = find_keys(next);
      const int e0 = cur.e0, len = cur.len - cur.e0, i = cur.i;
      const Found w = mine;
      const Row row = cur;
      cur = next;
      next = after;
      mine = theirs;
      if (len <= 0) continue;
      // -lse log2 e of the item's query rows.  One past the sequence's end counts as
      // one without weight: its scores are 0 or, with an infinite key, NaN.
      float neg[NQ32];
      bool dead = false;
#pragma unroll
      for (int x = 0; x < NQ32; ++x) {
        dead |= w.lse[x] == -INFINITY;
        neg[x] = w.lse[x] == -INFINITY ? -INFINITY : -w.lse[x] * kLog2e;
      }
      dead = __any_sync(0xffffffffu, dead);
      if (k >= kQSlots && !(ok = __all_sync(0xffffffffu, wait(bQFree0, kQSlots, k - kQSlots)))) break;
#pragma unroll
      for (int x = 0; x < NQ32; ++x) negs[(k % kItems) * 128 + x * 32 + lane] = neg[x];
      colss[(k % kItems) * 32 + lane] = w.cols;
      __syncwarp();
      const uint32_t bq = bQFull0 + 8u * (k % kQSlots), dst = sQ + (k % kQSlots) * S::kQBytes;
      if (leader) {
        volatile Item* e = ring + k % kItems;
        e->tiles = (len + S::kBPT - 1) / S::kBPT;
        e->blocks = len;
        e->diag = w.last == i;
        e->dead = dead;
        e->slot = int64_t(row.unit) * p.slots + (e0 - w.base);
        e->e0 = e0;
        e->kv = row.f0 / p.g;
        mbar_arrive(bItem0 + 8u * (k % kItems));
        mbar_expect_tx(bq, S::kQBytes);
        // one box: the block of one head, or of two heads stacked
        if constexpr (BLK == 64 && PACK == 1) tma_load_kv<HD>(dst, &tmQ, bq, i * BLK, row.f0);
        else tma_load_q<BLK, HD>(dst, &tmQ, bq, i * BLK, row.f0);
      }
      __syncwarp();
      ++k;
    }
    // the end of the stream, in an entry that the sums are done with
    if (ok && k >= kQSlots) ok = __all_sync(0xffffffffu, wait(bQFree0, kQSlots, k - kQSlots));
    if (leader) {
      if (ok) {
        ring[k % kItems].tiles = 0;
        mbar_arrive(bItem0 + 8u * (k % kItems));
      }
      // never leave the CTA with copies in flight into its shared memory
      for (int x = k > kQSlots ? k - kQSlots : 0; x < k; ++x)
        wait_drain(bQFull0 + 8u * (x % kQSlots), uint32_t(x / kQSlots) & 1u, kDrainNs);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ================================================================ keys
    const bool leader = elect_one();
    bool ok = true;
    int t = 0;
    for (int k = 0; ok; ++k) {
      if (!(ok = __all_sync(0xffffffffu, wait(bItem0, kItems, k)))) break;
      volatile Item* e = ring + k % kItems;
      const int tiles = e->tiles;
      if (tiles == 0) break;
      const int len = e->blocks, e0 = e->e0, kv = e->kv;
      int have = 0, cols = colss[(k % kItems) * 32 + lane];   // lane x holds entry have + x
      for (int y = 0; y < tiles; ++y, ++t) {
        if (y * S::kBPT - have >= 32) {
          have = y * S::kBPT;
          cols = have + lane < len ? p.col_idx[e0 + have + lane] : 0;
        }
        // the product that filled this tile's S buffer last has read its K slot
        if (t >= kKSlots && !(ok = __all_sync(0xffffffffu, wait(bSFull0, kSBufs, t - kKSlots)))) break;
        // a last tile without a second block leaves that half as it was: its sums are not stored
        const int blocks = min(S::kBPT, len - y * S::kBPT);
        const uint32_t bk = bKFull0 + 8u * (t % kKSlots), dst = sK + (t % kKSlots) * S::kKBytes;
        const int j0 = __shfl_sync(0xffffffffu, cols, y * S::kBPT - have);
        const int j1 = __shfl_sync(0xffffffffu, cols, (y * S::kBPT + S::kBPT - 1 - have) & 31);
        if (leader) {
          mbar_expect_tx(bk, uint32_t(blocks) * (S::kKBytes / S::kBPT));
#pragma unroll
          for (int a = 0; a < HD / 64; ++a) tma_load_3d(dst + a * S::kAtomK, &tmK, bk, a * 64, j0 * BLK, kv);
          if (S::kBPT == 2 && blocks == 2) {
#pragma unroll
            for (int a = 0; a < HD / 64; ++a)
              tma_load_3d(dst + a * S::kAtomK + BLK * 128, &tmK, bk, a * 64, j1 * BLK, kv);
          }
        }
        __syncwarp();
      }
    }
    if (leader)
      for (int x = t > kKSlots ? t - kKSlots : 0; x < t; ++x)
        wait_drain(bKFull0 + 8u * (x % kKSlots), uint32_t(x / kKSlots) & 1u, kDrainNs);
    __syncwarp();
  } else if (warp == 1) {
    // ================================================================ products
    // The whole warp goes through the loop, so that what a product is given
    // stays in uniform registers; one elected thread issues.
    constexpr uint64_t kFix = sw128_fixed(16, 1024);
    constexpr uint32_t kHi = uint32_t(kFix >> 32);
    const uint32_t q_lo = uint32_t(kFix) + (sQ >> 4), k_lo = uint32_t(kFix) + (sK >> 4);
    const bool leader = elect_one();
    bool ok = true;
    int t = 0;
    for (int k = 0; ok; ++k) {
      if (!(ok = __all_sync(0xffffffffu, wait(bItem0, kItems, k)))) break;
      const int tiles = ring[k % kItems].tiles;
      if (tiles == 0) break;
      if (!(ok = __all_sync(0xffffffffu, wait(bQFull0, kQSlots, k)))) break;
      const uint32_t qb = q_lo + uint32_t(k % kQSlots) * (S::kQBytes >> 4);
      for (int y = 0; y < tiles; ++y, ++t) {
        ok = wait(bKFull0, kKSlots, t) && (t < kSBufs || wait(bSFree0, kSBufs, t - kSBufs));
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t kb = k_lo + uint32_t(t % kKSlots) * (S::kKBytes >> 4);
        const uint32_t d = tmem + (t % kSBufs) * S::kNQ;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            mma_ss(d, desc_from(kb + ((kk >> 2) * S::kAtomK + (kk & 3) * 32) / 16, kHi),
                   desc_from(qb + ((kk >> 2) * S::kAtomQ + (kk & 3) * 32) / 16, kHi), S::kIdesc, kk > 0 ? 1u : 0u);
          tc_commit(bSFull0 + 8u * (t % kSBufs));
          if (y == tiles - 1) tc_commit(bQFree0 + 8u * (k % kQSlots));
        }
        __syncwarp();
      }
    }
    if (leader) {
      tc_commit(bDrain);
      wait_drain(bDrain, 0, kDrainNs);
    }
    __syncwarp();
  } else {
    // ================================================================ sums
    // Group t % 3 of four warps takes tile t, a key per thread; warp w reaches
    // TMEM lanes 32 (w % 4) .., so each scheduler has a warp of every group.
    const int q4 = warp & 3, group = (warp - 3) >> 2;
    const int key = q4 * 32 + lane;
    const int half = key / BLK, kl = key - half * BLK;         // key block of the tile, key in it
    const uint32_t lane_base = tmem + (uint32_t(q4 * 32) << 16);
    const float sl2 = p.scale_log2;
    bool ok = true;
    int t = 0;
    for (int k = 0; ok; ++k) {
      if (!(ok = __all_sync(0xffffffffu, wait(bItem0, kItems, k)))) break;
      volatile Item* e = ring + k % kItems;
      const int tiles = e->tiles;
      if (tiles == 0) break;
      const int y0 = (group + kGroups - t % kGroups) % kGroups;   // the item's first tile of this group
      t += tiles;
      if (y0 >= tiles) continue;
      const int blocks = e->blocks, diag = e->diag ? blocks - 1 : -1, dead = e->dead;
      float* const out = p.part + size_t(e->slot) * BLK + kl;
      const float* const neg = negs + (k % kItems) * 128;
      for (int y = y0; y < tiles; y += kGroups) {
        const int tt = t - tiles + y;
        const uint32_t s_col = lane_base + (tt % kSBufs) * S::kNQ;
        if (!(ok = __all_sync(0xffffffffu, wait(bSFull0, kSBufs, tt)))) break;
        tc_fence_after();
        const int blk = y * S::kBPT + half;                    // the thread's kept block
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
        float sv[2][32];
        tmem_ld32(s_col, sv[0]);
#pragma unroll
        for (int c0 = 0; c0 < S::kNQ; c0 += 32) {
          float* const v = sv[c0 / 32 & 1];
          wait_ld32(v);
          if (c0 + 32 < S::kNQ) {
            tmem_ld32(s_col + c0 + 32, sv[(c0 / 32 & 1) ^ 1]);   // while these columns are worked on
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bSFree0 + 8u * (tt % kSBufs));
          }
          // In the diagonal block a key takes queries from its own token on: of
          // these 32 all, none, or (where they are the warp's own tokens) some.
          const int first = blk == diag ? kl - lane : -32;
          if (c0 % BLK < first) {
          } else if (dead || c0 % BLK == first) {
            // a query row without weight gives nothing, whatever its scores are
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float n = neg[c0 + c];
              const bool use = (blk != diag || (c0 + c) % BLK >= kl) && n != -INFINITY;
              const float x = ex2(fmaf(v[c], sl2, n));
              s0 += use ? x : 0.f;
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 n = *reinterpret_cast<const float4*>(neg + c0 + c);
              float x0, x1, x2, x3;
              fma2(x0, x1, v[c], v[c + 1], sl2, n.x, n.y);
              fma2(x2, x3, v[c + 2], v[c + 3], sl2, n.z, n.w);
              add2(s0, s1, ex2(x0), ex2(x1));
              add2(s2, s3, ex2(x2), ex2(x3));
            }
          }
        }
        if (blk < blocks) out[size_t(blk) * BLK] = (s0 + s1) + (s2 + s3);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
  if (*abort_flag) spoil();
}

// w[kv][u] += the sums of u's block, unit by unit and row by row.  A block of
// 1024 threads takes the SL = 1024 / B key blocks j0 .. j0 + SL - 1, B threads
// for each: four slices of the column's rows, four keys a thread.  A column of
// more than kLong rows (a global first block's) is shared out over the whole
// block instead.  What this costs is the latency of its loads, so those of the
// layout and the weights so far are made before the wait for the first kernel, and those of the sums
// four at a time: 23.4 us a call at 2500 random tokens against 25.0 with eight,
// and 29.3 with a thread to every key and one slice.
constexpr int kAddThreads = 1024, kLong = 64, kStaged = 4096, kUnits = 8, kInFlight = 4;
template <int BLK>
__global__ void __launch_bounds__(kAddThreads) add_rows_kernel(const Params p) {
  constexpr int SL = kAddThreads / BLK, RL = kAddThreads / (BLK / 4);
  __shared__ int s_col[kUnits][SL + 1];          // where the block's columns begin, for each unit
  __shared__ int s_pos[kStaged];                 // csr_pos of the block's columns, if they fit
  __shared__ float4 s_sum[kAddThreads];
  const int per = (p.nb + SL - 1) / SL;
  const int kvl = blockIdx.x / per, j0 = (blockIdx.x - kvl * per) * SL;
  const int sl = threadIdx.x / BLK, kl = threadIdx.x % BLK;
  const int rl = threadIdx.x / (BLK / 4), k4 = threadIdx.x % (BLK / 4);   // slice of the block, four keys
  const int u = (j0 + sl) * BLK + kl;
  float* const f = reinterpret_cast<float*>(s_sum);
  grid_release();
  float* const out = p.weights + size_t(p.kv0 + kvl) * p.weights_stride + u;
  const float old = u < p.n ? __ldcg(out) : 0.f;     // (the kernel ahead has waited for what wrote them)
  float4 t4 = make_float4(0.f, 0.f, 0.f, 0.f);   // this thread's slice of column sl
  float sum = 0.f;                               // of key kl of a long column sl
#pragma unroll 1
  for (int x0 = 0; x0 < p.upk; x0 += kUnits) {
    const int units = min(kUnits, p.upk - x0);
    __syncthreads();
    for (int x = threadIdx.x; x < units * (SL + 1); x += kAddThreads) {
      const int lh = (p.kv0 * p.upk + kvl * p.upk + x0 + x / (SL + 1)) * p.pack % p.L;
      s_col[x / (SL + 1)][x % (SL + 1)] = p.col_ptr[size_t(lh) * p.nb + min(j0 + x % (SL + 1), p.nb)];
    }
    __syncthreads();
    int total = 0;
    for (int x = 0; x < units; ++x) total += s_col[x][SL] - s_col[x][0];
    const bool staged = total <= kStaged;
    if (staged) {
      int off = 0;
      for (int x = 0; x < units; ++x) {
        const int e0 = s_col[x][0], n = s_col[x][SL] - e0;
        for (int y = threadIdx.x; y < n; y += kAddThreads) s_pos[off + y] = p.csr_pos[e0 + y];
        off += n;
      }
    }
    __syncthreads();
    if (x0 == 0) grid_wait();              // the sums are in memory from here on
    int off = 0;
#pragma unroll 1
    for (int x = 0; x < units; ++x) {
      const int unit = kvl * p.upk + x0 + x;
      const int lh = (p.kv0 * p.upk + unit) * p.pack % p.L;
      const float4* const src =
          reinterpret_cast<const float4*>(p.part + (int64_t(unit) * p.slots - p.row_ptr[size_t(lh) * p.nb]) * BLK) + k4;
      const int shift = off - s_col[x][0];       // entry c is s_pos[c + shift]
      off += s_col[x][SL] - s_col[x][0];
      // t += the sums of entries c, c + step, .. below c1, in this order
      auto add = [&](float4& t, int c, int c1, int step) {
#pragma unroll 1
        for (; c < c1; c += kInFlight * step) {
          float4 v[kInFlight];
#pragma unroll
          for (int z = 0; z < kInFlight; ++z) {
            const int e = min(c + z * step, c1 - 1);
            v[z] = src[int64_t(staged ? s_pos[e + shift] : p.csr_pos[e]) * (BLK / 4)];
          }
#pragma unroll
          for (int z = 0; z < kInFlight; ++z) {
            if (c + z * step < c1) {
              t.x += v[z].x;
              t.y += v[z].y;
              t.z += v[z].z;
              t.w += v[z].w;
            }
          }
        }
      };
      const int c0 = s_col[x][sl], c1 = s_col[x][sl + 1];
      const bool mine = c1 - c0 <= kLong;
      if (mine) add(t4, c0 + rl % 4, c1, 4);
      if (__syncthreads_and(mine)) continue;
#pragma unroll 1
      for (int y = 0; y < SL; ++y) {
        const int d0 = s_col[x][y], d1 = s_col[x][y + 1];
        if (d1 - d0 <= kLong) continue;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        add(t, d0 + rl, d1, RL);
        __syncthreads();
        s_sum[threadIdx.x] = t;                  // [RL][BLK] floats
        __syncthreads();
        float part = 0.f;
        for (int z = sl; z < RL; z += SL) part += f[z * BLK + kl];
        __syncthreads();
        f[threadIdx.x] = part;
        __syncthreads();
        if (sl == y)
          for (int z = 0; z < SL; ++z) sum += f[z * BLK + kl];
      }
    }
  }
  __syncthreads();
  s_sum[threadIdx.x] = t4;                       // [SL][4][BLK] floats
  __syncthreads();
  if (u >= p.n) return;
  const float* const mine = f + sl * 4 * BLK + kl;
  const float all = ((mine[0] + mine[BLK]) + (mine[2 * BLK] + mine[3 * BLK])) + sum;
  if (all == -INFINITY) return;          // a wait ran out: see the first kernel
  *out = old + all;
}

// Query heads of a unit: two for B = 64 when a group's heads pair off on one route.
int pack_of(const bsa_layout* L, int g) { return L->B == 64 && g % 2 == 0 && L->L == 1 ? 2 : 1; }

// Kept blocks that a unit needs room for: the most of any layout head.
int64_t kept_of(const bsa_layout* L) {
  int64_t most = 1;
  for (int h = 0; h < L->L; ++h)
    most = std::max<int64_t>(most, L->row_ptr[size_t(h + 1) * L->nb] - L->row_ptr[size_t(h) * L->nb]);
  return most;
}

// Key/value heads of a strip: as many as kStripBytes hold, at least one.
int strip_of(const bsa_layout* L, int heads, int kv_heads) {
  const int upk = heads / kv_heads / pack_of(L, heads / kv_heads);
  const size_t one = size_t(kept_of(L)) * upk * L->B * sizeof(float);
  return int(std::max<size_t>(1, std::min<size_t>(kv_heads, kStripBytes / one)));
}

size_t bytes_of(const bsa_layout* L, int heads, int kv_heads) {
  const int upk = heads / kv_heads / pack_of(L, heads / kv_heads);
  return size_t(strip_of(L, heads, kv_heads)) * upk * size_t(kept_of(L)) * L->B * sizeof(float);
}

template <int BLK, int HD, int PACK>
int launch(const void* q, const void* k, int kv_heads, Params p, const bsa_layout* layout, cudaStream_t stream) {
  using S = Shape<BLK, HD, PACK>;
  auto kern = prompt_weights_kernel<BLK, HD, PACK>;
  static std::mutex mu;
  static int sms[64] = {};
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return set_error(BSA_ERR_CUDA, "cannot query the device");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!sms[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return set_error(BSA_ERR_CUDA, std::string("weights attributes: ") + cudaGetErrorString(e));
      sms[dev] = n_sm;
    }
    n_sm = sms[dev];
  }
  CUtensorMap mq, mk;
  int st = BLK == 64 && PACK == 1 ? tmap::encode_kv(&mq, q, p.heads, p.n, HD) : tmap::encode_q(&mq, q, p.heads, p.n, HD, BLK);
  if (st == BSA_OK) st = tmap::encode_atoms(&mk, k, kv_heads, p.n, HD, BLK);
  if (st != BSA_OK) return st;
  const int strip = strip_of(layout, p.heads, kv_heads);
  for (p.kv0 = 0; p.kv0 < kv_heads; p.kv0 += strip) {
    p.kvs = std::min(strip, kv_heads - p.kv0);
    p.items = uint32_t(p.kvs) * uint32_t(p.upk) * uint32_t(p.nb);
    st = launch_dependent("prompt weights launch", kern, std::min(p.items, unsigned(n_sm)), kThreads, S::kSmem, 1, stream,
                          mq, mk, p);
    if (st != BSA_OK) return st;
    constexpr int SL = kAddThreads / BLK;
    st = launch_dependent("weights sum launch", add_rows_kernel<BLK>, unsigned(p.kvs) * unsigned((p.nb + SL - 1) / SL),
                          kAddThreads, 0, 1, stream, p);
    if (st != BSA_OK) return st;
  }
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
  if (st != BSA_OK || layout->col_idx.empty()) return st;   // no kept block, no weight
  st = tmap::get_encoder();
  if (st != BSA_OK) return st;
  wts::Params p{};
  p.row_ptr = layout->d_row_ptr;
  p.col_idx = layout->d_col_idx;
  p.col_ptr = layout->d_col_ptr;
  p.csr_pos = layout->d_csr_pos;
  p.lse = lse;
  p.part = static_cast<float*>(workspace);
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.status = layout->d_status;
  p.n = n;
  p.nb = layout->nb;
  p.L = layout->L;
  p.g = heads / kv_heads;
  p.heads = heads;
  p.pack = wts::pack_of(layout, p.g);
  p.upk = p.g / p.pack;
  p.slots = wts::kept_of(layout);
  p.scale_log2 = float(double(scale) * 1.4426950408889634);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 128) {
    return d == 128 ? wts::launch<128, 128, 1>(q, k, kv_heads, p, layout, s)
                    : wts::launch<128, 64, 1>(q, k, kv_heads, p, layout, s);
  }
  if (p.pack == 2) {
    return d == 128 ? wts::launch<64, 128, 2>(q, k, kv_heads, p, layout, s)
                    : wts::launch<64, 64, 2>(q, k, kv_heads, p, layout, s);
  }
  return d == 128 ? wts::launch<64, 128, 1>(q, k, kv_heads, p, layout, s)
                  : wts::launch<64, 64, 1>(q, k, kv_heads, p, layout, s);
}

}  // extern "C"
