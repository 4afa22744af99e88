// Attention over the paged key/value cache with the reads of one call split
// over the GPU (sm_100a): the decode step that also adds up the weights it
// gives to the cached keys (bsa_decode_weights), and the attention of a tree
// of drafted tokens over the cache and their own ancestors (bsa_decode_tree).
//
// Both have a few query rows per key/value head (the group's query heads times
// the tree's tokens) against all the cached keys that the rows' layout row
// keeps, so what bounds them is the read of the kept pages, 4 d bytes a key.
// A unit is (sequence, key/value head or query head, 128-row tile, layout
// row): the rows of a tile that share a layout row read the same keys, and no
// key of another route ever meets them, so nothing but the end of the cache
// has to be masked.  The unit's list of 64-key chunks is cut into S runs, one
// CTA each.
//
// Kernel 1 (paged_attention_kernel), per 64-key chunk of a run:
//   S = Q K^T                  (tcgen05.mma, bf16 x bf16 -> fp32 in TMEM)
//   m' = max(m, rowmax S), P = exp2((S - m') scale log2 e)
//   O += P V                   (tcgen05.mma, A = P from TMEM)
// with P written as two bf16 numbers (its upper 16 bits and the rounding of what
// they leave, within 2^-15 of P together) over the 64 columns of S, and two
// products: a step is bound by the cache's bytes, so the second product costs
// nothing that shows there (10 % of a call where full tiles of tree rows run at
// the power limit), and o is then rounded once, at its end.  A run
// leaves its unnormalised O, m and l in the caller's workspace; the step
// leaves the scores too.
// Kernel 2 joins the runs of each row.  The tree's rows add their ancestors
// there (before its wait for kernel 1, as far as its blocks find room beside
// that), at most T keys each, on the plain cores in fp32: an ancestor's key
// and value are read by the rows that descend from it and by no others, so a
// branch's infinity cannot reach another branch.  The step's kernel 2 also
// turns the scores into weights, p = exp2(s scale log2 e - M) / L.  Short steps
// have no kernel 2: their runs are a cluster's, which does this itself.
//
// At most 8 rows (every step of a grouped-query model, short trees) take the
// products the other way round, keys as the rows of a tile:
//   S^T = K Q^T,   O^T += V^T [P^T upper bits | rest]      (N = 16 both)
// where more rows take 128 x 64 and twice 128 x d tiles for the same keys.  A
// step is bound by memory either way, but the large tiles, nearly all of them
// empty, kept the tensor cores 60 % busy, and a server's GPU runs at its power
// limit: 16 x 16K steps that follow each other for seconds took 181 to 193 us
// each with the clocks at 1.45 to 1.6 GHz, and take 158 to 162 at 1.8; a few at
// a time 164 and 160.  (128 rows of S^T are 64 keys and whatever lies behind
// them in shared memory, which nobody reads.)  With 8 rows this way and the
// other take 41.1 and 42.0 us over 2 x 131K, 82.8 and 83.1 over 8 x 16K; with 1
// row 28.0 and 29.2, 80.9 and 81.5.
//
// Roles of kernel 1 (192 threads, two CTAs per SM): warp 0 looks the pages up
// and issues the TMA loads, warp 1 issues the products, warps 2-5 hold one
// query row per thread (few rows: two of them one key per thread, all four a
// lane of O^T).  Every wait is bounded, as in the forward.
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
namespace paged {

using namespace ptx;

constexpr int kThreads = 192;
constexpr int kTileM = 128;            // query rows of a tile (tcgen05 M = 128)
constexpr int kChunk = 64;             // keys per chunk
constexpr int kVS = 3;                 // V slots in shared memory
constexpr int kFew = 8;                // query rows that the keys' side of a product can take
constexpr int kMaxT = 128;             // drafted tokens at most
constexpr float kRescaleThreshold = 8.0f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr uint64_t kWaitNs = 1000000000ull, kDrainNs = 200000000ull;

// Runs of a unit: as many CTAs as the GPU holds at once (two on each of 148
// SMs: a figure for speed alone, fixed so that a host-only layout gives the same
// workspace) shared out over the units, rounded down (twice as many: 64-token
// trees over 8 x 16K 136 us for 130, 2 x 131K steps with a route a head 33.6 for
// 28.4, chains 47.2 for 38.4), and no run longer than kRunChunks, so that
// sequences of other lengths level out (16 x 16K step: 2 runs of 128 chunks 171
// us, 4 of 64 162.6, 8 of 32 164.4; 32 x 8K 169, 158, 160; the trees 130, 130 and 137).
constexpr int kSlots = 2 * 148;
// A step of at most 8 query rows a unit and few chunks is one kernel, a
// cluster of up to 8 CTAs per unit that joins its runs through shared memory:
// a launch less.  (A step of the dyadic route at 32K 11.1 us for 13.1 through
// the binding, 8.0 for 8.8 in a graph; whole caches of 2000 tokens, the most
// chunks there are, 11.0 for 13.1 and 9.5 for 10.9; four sequences 11.5 for 13.1
// and 11.1 for 12.4.)
constexpr int kAloneChunks = 4;        // chunks of a run at most
constexpr int kRunChunks = 64;

struct Plan {
  int hg;          // head groups of a sequence: key/value heads, or query heads when routes differ by head
  int hpt;         // query heads that share a tile
  int rows;        // query rows of a head group
  int mtiles;      // 128-row tiles of them
  int groups;      // layout rows that a tree's positions can fall in
  int units;       // batch * hg * mtiles * groups
  int S;           // runs of a unit
  int cap;         // rows of a partial result
  bool alone;      // one kernel, S CTAs of a cluster a unit
};

Plan plan_of(const bsa_layout* L, int batch, int heads, int kv_heads, int T, bool step) {
  Plan p{};
  const int H = heads / batch, hkv = kv_heads / batch;
  p.hpt = L->L == 1 ? H / hkv : 1;
  p.hg = H / p.hpt;
  p.rows = p.hpt * T;
  p.mtiles = (p.rows + kTileM - 1) / kTileM;
  p.groups = (T + L->B - 2) / L->B + 1;
  const int64_t busy = int64_t(batch) * p.hg * p.mtiles;
  p.units = int(std::min<int64_t>(busy * p.groups, INT32_MAX));
  const int chunks = std::max(1, L->max_row * (L->B / kChunk));
  const int fill = int(std::min<int64_t>(chunks, std::max<int64_t>(1, kSlots / busy)));
  p.S = std::max(fill, (chunks + kRunChunks - 1) / kRunChunks);
  p.cap = std::min(kTileM, p.rows);
  // (a key/value head's query heads are one unit, so that one thread adds a key's weight)
  if (step && p.rows <= kFew && (L->L == 1 || H == hkv)) {
    int C = 8;
    while (C > chunks) C /= 2;
    if (chunks <= C * kAloneChunks && busy * C <= kSlots) {
      p.alone = true;
      p.S = C;
    }
  }
  return p;
}

struct Offsets {
  size_t ml, flag, scores, total;      // bytes; O starts at 0
};
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
Offsets offsets_of(const Plan& p, const bsa_layout* L, int heads, int d, bool scores) {
  Offsets o{};
  const size_t runs = size_t(p.units) * p.S, rows = runs * p.cap;
  o.ml = up256(rows * d * 4);
  o.flag = o.ml + up256(rows * 8);
  o.scores = o.flag + up256(runs * 4);
  o.total = o.scores + (scores ? up256(size_t(heads) * L->max_row * L->B * 4) : 0);
  return o;
}

struct Params {
  const int32_t* page_table;
  const int32_t* lengths;      // step: the new token's position; tree: cached tokens
  const int32_t* parents;      // tree: [batch][T]
  const int32_t* row_ptr;
  const int32_t* col_idx;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_tree;
  const __nv_bfloat16* v_tree;
  __nv_bfloat16* o;
  float* lse;
  float* weights;
  size_t weights_stride;
  float* part_o;               // [unit][run][cap][d]
  float2* part_ml;             // [unit][run][cap]
  int* part_flag;              // [unit][run]
  float* scores;               // step: [heads][max_row * B]
  uint32_t* status;
  size_t score_stride;
  int n, nb, L, H, hkv, max_blocks, num_pages;
  int hg, hpt, rows, mtiles, per_group, S, cap, T, tiles;   // per_group: units of a layout row
  float scale_log2;
};

template <int BLK, int HD, bool FEW>
struct Shape {
  static constexpr int kCPB = BLK / kChunk;
  static constexpr int kKS = FEW ? 3 : 2;                    // K slots, S buffers and P buffers
  static constexpr int kRowsQ = FEW ? 2 * kFew : kTileM;
  static constexpr int kQBytes = kRowsQ * HD * 2;
  static constexpr int kTileBytes = kChunk * HD * 2;
  static constexpr int kAtomQ = kRowsQ * 128, kAtomKV = kChunk * 128;
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffV = kOffK + kKS * kTileBytes;
  // Few rows: P^T as the second product's B operand, N-major and unswizzled:
  // cores of 8 keys by 8 rows, 16 bytes a key; for 8 keys a core of P's upper
  // bits, one of its rest and 32 bytes that keep a warp's writes off each other's banks.
  static constexpr int kKeysP = 2 * 128 + 32, kPBytes = FEW ? kChunk / 8 * kKeysP : 0;
  static constexpr int kOffP = kOffV + kVS * kTileBytes;
  static constexpr int kOffMax = kOffP + kKS * kPBytes;      // row maxima [2][2][kFew], sums [2][kFew], moves [2][2]
  static constexpr int kOffBar = kOffMax + (FEW ? 6 * kFew * 4 + 16 : 0);
  // q_full, k_full[KS], v_full[VS], s_full[KS], p_full[KS], o_done[VS], drain; few rows: max moves[2], maxima[2], sums
  static constexpr int kNumBars = 1 + kKS + kVS + kKS + kKS + kVS + 1 + (FEW ? 5 : 0);
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;   // TMEM address, abort flag, page flag, deepest token
  static constexpr int kOffRun = kOffMisc + 16;
  static constexpr int kOffJump = kOffRun + 32;              // the tree's walk, a byte a token
  static constexpr int kOffDepth = kOffJump + kMaxT;
  static constexpr int kSmem = kOffDepth + kMaxT;
  static constexpr int kSCols = FEW ? 2 * kFew : kChunk;
  static constexpr int kColS = 0, kColO = kKS * kSCols;
  static constexpr uint32_t kTmemCols = FEW ? 64 : 256;
  static constexpr uint32_t kIdescQK = idesc_bf16(kTileM, kSCols, 0, 0);
  static constexpr uint32_t kIdescPV = FEW ? idesc_bf16(kTileM, 2 * kFew, 1, 1) : idesc_bf16(kTileM, HD, 0, 1);
  static_assert(kColO + (FEW ? 2 * kFew : HD) <= int(kTmemCols), "TMEM budget");
  static_assert(!FEW || kKS == kVS, "P buffers and V slots are released by the same products");
  static_assert(kOffBar % 8 == 0 && kOffP % 16 == 0, "alignment");
  // Few rows: a product of 128 rows reads 8 KB past a 64-row operand (the next slot, or what follows the last)
  static_assert(!FEW || kOffV + kVS * kTileBytes + kAtomKV <= 77 * 1024 || HD == 128, "inside the CTA's shared memory");
};

// Two fp32 lanes at once, each rounded as the scalar instruction would.
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The largest of a warp's values, a NaN counting for nothing.
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
__device__ __forceinline__ void bf16x2_to_f32(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}

// Eight consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
// Fixed fields of a shared-memory descriptor without swizzle: `k_bytes` from
// core to core along K, `row_bytes` along the rows.
__host__ __device__ constexpr uint64_t flat_fixed(uint32_t k_bytes, uint32_t row_bytes) {
  return (uint64_t((k_bytes >> 4) & 0x3FFFu) << 16) | (uint64_t((row_bytes >> 4) & 0x3FFFu) << 32) | (uint64_t(1) << 46);
}

// Two probabilities as two bf16 numbers each: their upper 16 bits and the
// rounding of what those leave, at least 2^-20 of P: an infinite value that
// the row reads then has the same sign in both products (a rounded first part
// could leave a negative rest, and 0 * inf is NaN).  2^-20 P is far inside the
// 2^-15 that the rounding may be off by, and a P of 0 gets nothing.  (Below
// 2^-113 the rest may end as 0, below 2^-119 its rounding is that of the
// smallest bf16 number, 2^-134.)
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  float la, lb;
  fma2(la, lb, a, b, 0x1p-20f, 0.f);
  hi = __byte_perm(ua, ub, 0x7632);
  lo = pack_bf16(fmaxf(a - __uint_as_float(ua & 0xffff0000u), la), fmaxf(b - __uint_as_float(ub & 0xffff0000u), lb));
}

// What a CTA of kernel 1 works on, found by one thread and shared.
struct Run {
  int start;       // first list entry of the unit's layout row
  int c0, c1;      // the run's chunks, counted in the unit's list
  int tail;        // valid keys of the list's last chunk
  int last;        // index of the list's last chunk
  int go;          // 0: nothing to do and nothing will be read
};

// A short step's end: what the cluster's CTAs join.
struct End {
  float2 ml[kFew];         // read by the others, as is `state`
  int state;
  int flag[kFew];          // joined
  float M[kFew], L[kFew], w[kFew][8];
};

// Depth of every drafted token by pointer jumping: after round k a token
// points 2^k ancestors up.  A parent that is not an earlier token ends the
// walk (kernel 2 refuses such a token).  Called by all threads.
__device__ __forceinline__ int deepest(const int32_t* parents, int T, volatile int8_t* jump, volatile int8_t* depth,
                                       int* most) {
  const int i = threadIdx.x;
  static_assert(kMaxT <= 128, "a token's index and depth fit a signed byte");
  if (i < kMaxT) {
    const int par = i < T ? parents[i] : -1;
    const bool up = par >= 0 && par < i;
    jump[i] = int8_t(up ? par : -1);
    depth[i] = int8_t(up ? 1 : 0);
  }
  if (i == 0) *most = 0;
  __syncthreads();
  for (int step = 1; step < T; step *= 2) {
    int to = -1, add = 0;
    if (i < kMaxT && jump[i] >= 0) {
      to = jump[jump[i]];
      add = depth[jump[i]];
    }
    __syncthreads();
    if (i < kMaxT && jump[i] >= 0) {
      jump[i] = int8_t(to);
      depth[i] = int8_t(depth[i] + add);
    }
    __syncthreads();
  }
  if (i < T) atomicMax(most, int(depth[i]));
  __syncthreads();
  return *most;
}

// Does row `at` of the layout keep all of the first `blocks` key blocks?  Its
// columns ascend, so one entry tells.
__device__ __forceinline__ bool keeps_all(const Params& p, size_t at, int blocks) {
  const int start = p.row_ptr[at];
  return blocks == 0 || (p.row_ptr[at + 1] - start >= blocks && p.col_idx[start + blocks - 1] == blocks - 1);
}

template <int BLK, int HD, bool TREE, bool FEW, bool ALONE>
__global__ void __launch_bounds__(kThreads, 2)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const Params p) {
  using S = Shape<BLK, HD, FEW>;
  constexpr int CPB = S::kCPB, kKS = S::kKS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_addr(smem);
  if (base & 1023u) {                    // never expected: the swizzle needs 1024-byte aligned tiles
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  // the later layout rows' units last: most of them have nothing to do
  const int run = blockIdx.x % p.S;
  const int unit = blockIdx.x / p.S;
  const int grp = unit / p.per_group;
  const int mt = unit % p.per_group % p.mtiles;
  const int bh = unit % p.per_group / p.mtiles;   // (sequence, head group)
  const int b = bh / p.hg, hg = bh - b * p.hg;
  const int f0 = b * p.H + hg * p.hpt;            // first query head of the tile
  const int hk = p.L == 1 ? hg : hg / (p.H / p.hkv);
  const int vr = min(kTileM, p.rows - mt * kTileM);   // rows of the tile
  const int warps = (vr + 31) / 32;               // softmax warps that hold any

  const uint32_t sQ = base, sK = base + S::kOffK, sV = base + S::kOffV;
  const uint32_t bar0 = base + S::kOffBar;
  const uint32_t bQFull = bar0, bK0 = bar0 + 8u, bV0 = bK0 + 8u * kKS, bS0 = bV0 + 8u * kVS, bP0 = bS0 + 8u * kKS,
                 bO0 = bP0 + 8u * kKS, bDrain = bO0 + 8u * kVS, bMax = bDrain + 8u, bTop = bMax + 16u, bSum = bTop + 16u;
  auto bKFull = [&](int c) { return bK0 + 8u * (c % kKS); };
  auto bVFull = [&](int c) { return bV0 + 8u * (c % kVS); };
  auto bSFull = [&](int c) { return bS0 + 8u * (c % kKS); };
  auto bPFull = [&](int c) { return bP0 + 8u * (c % kKS); };
  auto bODone = [&](int c) { return bO0 + 8u * (c % kVS); };
  auto parK = [](int c) { return uint32_t(c / kKS) & 1u; };
  auto parV = [](int c) { return uint32_t(c / kVS) & 1u; };
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(smem + S::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
  volatile int* s_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 8);
  Run* s_run = reinterpret_cast<Run*>(smem + S::kOffRun);
  End* const s_end = reinterpret_cast<End*>(smem + S::kOffK);   // ALONE, once the products are done
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Ctl ctl{abort_flag, p.status, kWaitNs};
  if (threadIdx.x == 0) {
    mbar_init(bQFull, 1);
    for (int s = 0; s < kKS; ++s) mbar_init(bK0 + 8u * s, 1);
    for (int s = 0; s < kVS; ++s) mbar_init(bV0 + 8u * s, 1);
    for (int s = 0; s < kKS; ++s) {
      mbar_init(bS0 + 8u * s, 1);
      mbar_init(bP0 + 8u * s, FEW ? 128 : 32 * warps);
    }
    for (int s = 0; s < kVS; ++s) mbar_init(bO0 + 8u * s, 1);
    mbar_init(bDrain, 1);
    if constexpr (FEW)
      for (int s = 0; s < 5; ++s) mbar_init(bMax + 8u * s, 2);
    *abort_flag = 0;
    *s_flag = 0;
    fence_barrier_init();
    tma_prefetch(&tmQ);
    tma_prefetch(&tmK);
    tma_prefetch(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(base + S::kOffMisc, S::kTmemCols);
    tmem_relinquish();
  }
  grid_wait();                                    // nothing of the caller's is read or written before this
  // Only now may kernel 2 start: it reads the caller's arrays before its own
  // wait, and what wrote them has ended only from here on.
  grid_release();

  bool skip = false;
  if constexpr (TREE) {
    // a later layout row has rows only if the tree is deep enough to reach it
    if (grp > 0) {
      const int len = p.lengths[b];
      const int need = grp * BLK - len % BLK;     // depth at which the layout row begins
      skip = len < 0 || len > p.n || len / BLK + grp >= p.nb || need > p.T - 1;
      if (!skip)
        skip = need > deepest(p.parents + size_t(b) * p.T, p.T, reinterpret_cast<volatile int8_t*>(smem + S::kOffJump),
                              reinterpret_cast<volatile int8_t*>(smem + S::kOffDepth),
                              reinterpret_cast<int*>(smem + S::kOffMisc + 12));
      // Where this layout row and the tree's first both keep all cached blocks,
      // their rows read the same keys: the first one's runs serve both (a
      // whole cache that a tree straddles two blocks of is read once, not twice).
      if (!skip) {
        const size_t at = size_t(f0 % p.L) * p.nb + len / BLK;
        const int blocks = len / BLK + (len % BLK != 0);
        skip = keeps_all(p, at, blocks) && keeps_all(p, at + grp, blocks);
      }
    }
  }
  // The run's place in its list, found by the warp that loads it: runs are cut
  // from the row's length as the layout has it, so that the entries of a run
  // are fetched at the same time as the row's last ones, which say how many
  // blocks lie before the end of the cache.
  int cols = 0, have = 0;                         // lane x holds list entry have + x
  if (warp == 0) {
    Run r{};
    const int t = p.lengths[b];
    const int row = t / BLK + grp;
    if (!skip && (TREE ? t >= 0 && t <= p.n : t >= 0 && t < p.n) && row < p.nb) {
      const int ctx = TREE ? t : t + 1;           // cached keys that exist
      const size_t at = size_t(f0 % p.L) * p.nb + row;
      r.start = p.row_ptr[at];
      const int full = p.row_ptr[at + 1] - r.start;
      r.c0 = int(int64_t(full) * CPB * run / p.S);
      have = r.c0 / CPB;
      cols = have + lane < full ? p.col_idx[r.start + have + lane] : 0;
      // a row's blocks ascend to its own: at most `groups` of them, the last, lie at or past the end
      const int end = lane < full ? p.col_idx[r.start + full - 1 - lane] : -1;
      const int len = full - __popc(__ballot_sync(0xffffffffu, end >= 0 && end * BLK >= ctx));
      if (len > 0) {
        const int col = __shfl_sync(0xffffffffu, end, full - len);
        const int rem = min(BLK, ctx - col * BLK);
        const int in_last = (rem + kChunk - 1) / kChunk;
        r.last = (len - 1) * CPB + in_last - 1;
        r.tail = rem - (in_last - 1) * kChunk;
        r.c1 = min(int(int64_t(full) * CPB * (run + 1) / p.S), r.last + 1);
      }
      r.go = 1;
    }
    if (lane == 0) *s_run = r;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const Run r = *s_run;
  const int nch = r.c1 - r.c0;
  const size_t part = (size_t(unit) * p.S + run) * p.cap;
  if (!ALONE && nch <= 0) {
    // an empty run: l = 0 tells kernel 2 that its O was not written
    if (r.go) {
      for (int x = threadIdx.x; x < vr; x += kThreads) p.part_ml[part + x] = make_float2(-INFINITY, 0.f);
      if (threadIdx.x == 0) p.part_flag[size_t(unit) * p.S + run] = 0;
    }
    if (warp == 1) tmem_dealloc(tmem, S::kTmemCols);
    return;
  }

  if (ALONE && nch <= 0) {
  } else if (warp == 0) {
    // ================================================================ loads
    const bool leader = elect_one();
    if (leader) {
      mbar_expect_tx(bQFull, S::kQBytes);
#pragma unroll
      for (int a = 0; a < HD / 64; ++a) tma_load_3d(sQ + a * S::kAtomQ, &tmQ, bQFull, a * 64, mt * kTileM, bh);
    }
    const int e1 = (r.c1 - 1) / CPB + 1;          // past the run's last list entry
    int page_of = 0, flag = 0;                    // lane x holds the page of entry have + x
    auto pages = [&]() {
      page_of = 0;
      if (have + lane < e1) {
        const int pg = p.page_table[size_t(b) * p.max_blocks + cols];
        if (pg >= 0 && pg < p.num_pages) page_of = pg;
        else flag = 1;                   // page 0 is read in its place and the rows are refused
      }
    };
    pages();
    int kc = 0, vc = 0;
    auto page_at = [&](int q) -> int {
      const int e = (r.c0 + q) / CPB;
      if (e - have >= 32) {
        have = e;
        cols = have + lane < e1 ? p.col_idx[r.start + have + lane] : 0;
        pages();
      }
      return __shfl_sync(0xffffffffu, page_of, e - have);
    };
    auto load_k = [&](int q, int page) -> bool {
      if (q >= kKS && !__all_sync(0xffffffffu, ctl.wait(bSFull(q), parK(q - kKS)))) return false;
      if (leader) {
        mbar_expect_tx(bKFull(q), S::kTileBytes);
        tma_load_kv<HD>(sK + (q % kKS) * S::kTileBytes, &tmK, bKFull(q), ((r.c0 + q) % CPB) * kChunk,
                        page * p.hkv + hk);
      }
      ++kc;
      return true;
    };
    auto load_v = [&](int q, int page) -> bool {
      if (q >= kVS && !__all_sync(0xffffffffu, ctl.wait(bODone(q), parV(q - kVS)))) return false;
      if (leader) {
        mbar_expect_tx(bVFull(q), S::kTileBytes);
        tma_load_kv<HD>(sV + (q % kVS) * S::kTileBytes, &tmV, bVFull(q), ((r.c0 + q) % CPB) * kChunk,
                        page * p.hkv + hk);
      }
      ++vc;
      return true;
    };
    int page = page_at(0);
    bool ok = load_k(0, page);
    for (int q = 0; q < nch && ok; ++q) {
      const int next = q + 1 < nch ? page_at(q + 1) : 0;
      if (q + 1 < nch) ok = load_k(q + 1, next);
      if (ok) ok = load_v(q, page);
      page = next;
    }
    if (__any_sync(0xffffffffu, flag) && lane == 0) *s_flag = 1;
    // never leave the CTA with copies in flight into its shared memory
    if (lane == 0) {
      wait_drain(bQFull, 0, kDrainNs);
      for (int c = max(0, kc - kKS); c < kc; ++c) wait_drain(bKFull(c), parK(c), kDrainNs);
      for (int c = max(0, vc - kVS); c < vc; ++c) wait_drain(bVFull(c), parV(c), kDrainNs);
    }
  } else if (warp == 1) {
    // ================================================================ products
    const bool leader = elect_one();
    constexpr uint64_t kFixK = sw128_fixed(16, 1024), kFixV = sw128_fixed(S::kAtomKV, 1024);
    // (in a cluster an address's upper bits name the CTA; a descriptor's has 18 bits)
    auto field = [](uint32_t addr) { return (addr & 0x3FFFFu) >> 4; };
    const uint32_t q_lo = uint32_t(kFixK) + field(sQ), k_lo = uint32_t(kFixK) + field(sK);
    const uint32_t v_lo = uint32_t(kFixV) + field(sV);
    constexpr uint32_t kHiK = uint32_t(kFixK >> 32), kHiV = uint32_t(kFixV >> 32);
    constexpr uint64_t kFixP = flat_fixed(S::kKeysP, 128);
    const uint32_t p_lo = uint32_t(kFixP) + field(base + S::kOffP);
    constexpr uint32_t kHiP = uint32_t(kFixP >> 32);
    auto issue_qk = [&](int c) -> bool {
      if (!__all_sync(0xffffffffu, ctl.wait(bKFull(c), parK(c)))) return false;
      tc_fence_after();
      const uint32_t d = tmem + S::kColS + (c % kKS) * S::kSCols;
      const uint32_t kb = k_lo + uint32_t(c % kKS) * (S::kTileBytes >> 4);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint64_t qd = desc_from(q_lo + ((kk >> 2) * S::kAtomQ + (kk & 3) * 32) / 16, kHiK);
          const uint64_t kd = desc_from(kb + ((kk >> 2) * S::kAtomKV + (kk & 3) * 32) / 16, kHiK);
          mma_ss(d, FEW ? kd : qd, FEW ? qd : kd, S::kIdescQK, kk > 0 ? 1u : 0u);
        }
        tc_commit(bSFull(c));
      }
      __syncwarp();
      return true;
    };
    auto issue_pv = [&](int c) -> bool {
      if (!__all_sync(0xffffffffu, ctl.wait(bVFull(c), parV(c)) && ctl.wait(bPFull(c), parK(c)))) return false;
      tc_fence_after();
      const uint32_t pa = tmem + S::kColS + (c % kKS) * S::kSCols;
      const uint32_t vb = v_lo + uint32_t(c % kVS) * (S::kTileBytes >> 4);
      if constexpr (FEW) {
        const uint32_t pb = p_lo + uint32_t(c % kKS) * (S::kPBytes >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk)
            mma_ss(tmem + S::kColO, desc_from(vb + kk * 16 * 128 / 16, kHiV),
                   desc_from(pb + kk * 2 * S::kKeysP / 16, kHiP), S::kIdescPV, (c > 0 || kk > 0) ? 1u : 0u);
          tc_commit(bODone(c));
        }
      } else if (leader) {
#pragma unroll
        for (int part2 = 0; part2 < 2; ++part2)            // P's upper bits, then the rest of it
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk)
            mma_ts(tmem + S::kColO, pa + part2 * 32 + kk * 8, desc_from(vb + kk * 16 * 128 / 16, kHiV), S::kIdescPV,
                   (c > 0 || part2 > 0 || kk > 0) ? 1u : 0u);
        tc_commit(bODone(c));
      }
      __syncwarp();
      return true;
    };
    bool ok = __all_sync(0xffffffffu, ctl.wait(bQFull, 0));
    tc_fence_after();
    if (ok) ok = issue_qk(0);
    for (int c = 0; c < nch && ok; ++c) {
      if (c + 1 < nch) ok = issue_qk(c + 1);
      if (ok) ok = issue_pv(c);
    }
    if (leader) {
      tc_commit(bDrain);
      wait_drain(bDrain, 0, kDrainNs);
    }
    __syncwarp();
  } else if constexpr (FEW) {
    // ================================================================ softmax, one key per thread
    // Lanes 0-63 of S^T are the chunk's keys; all four warps hold O^T, a lane
    // for each of d.  The two warps with keys exchange a bit a chunk, whether a
    // row's max has to move, and its maxima only then.  What they exchange is
    // kept twice, by the chunk's parity: chunk c + 2 is not in TMEM before
    // every warp has passed chunk c.
    const int q4 = warp & 3, key = q4 * 32 + lane;
    const bool keyed = q4 < 2;
    const uint32_t lane_base = tmem + (uint32_t(q4 * 32) << 16);
    const float sl2 = p.scale_log2;
    float* const s_max = reinterpret_cast<float*>(smem + S::kOffMax);
    volatile int* const s_need = reinterpret_cast<volatile int*>(smem + S::kOffMax + 6 * kFew * 4);
    float neg[kFew], l[kFew];                    // -m (0 while a row has no finite score), l
    unsigned fresh = (1u << vr) - 1u;            // rows without a finite score so far
    unsigned moved = 0;                          // parity of the exchanges of maxima, a bit for each parity of the chunk
#pragma unroll
    for (int x = 0; x < kFew; ++x) neg[x] = l[x] = 0.f;
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      const int odd = c & 1;
      float sv[kFew], pr[kFew];
      const bool ends = r.c0 + c == r.last && r.tail < kChunk;
      if (keyed) {
        ok = __all_sync(0xffffffffu, ctl.wait(bSFull(c), parK(c)));
        if (!ok) break;
        tc_fence_after();
        tmem_ld8(lane_base + S::kColS + (c % kKS) * S::kSCols, sv);
        tmem_wait_ld();
        const bool past = ends && key >= r.tail;
        bool need = false;
#pragma unroll
        for (int x = 0; x < kFew; ++x) {
          pr[x] = 0.f;
          if (x >= vr) continue;
          if (past) sv[x] = -INFINITY;
          if constexpr (!TREE) p.scores[size_t(f0 + x) * p.score_stride + size_t(r.c0 + c) * kChunk + key] = sv[x];
          pr[x] = fmaf(sv[x], sl2, neg[x]);
          // the row moves its max only by more than 2^8; the first finite score always moves it
          need |= pr[x] > (fresh >> x & 1u ? -INFINITY : kRescaleThreshold);
        }
        need = __any_sync(0xffffffffu, need);
        if (lane == 0) {
          s_need[odd * 2 + q4] = need;
          mbar_arrive(bMax + 8u * odd);
        }
        // the product that read this P buffer last
        if (c >= kKS) ok = __all_sync(0xffffffffu, ctl.wait(bODone(c - kKS), parV(c - kKS)));
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < kFew; ++x)
          if (x < vr) pr[x] = ex2(pr[x]);
      }
      ok = __all_sync(0xffffffffu, ctl.wait(bMax + 8u * odd, uint32_t(c >> 1) & 1u));
      if (!ok) break;
      if (s_need[odd * 2] | s_need[odd * 2 + 1]) {     // the same in every thread
        float* const mine = s_max + odd * 2 * kFew;
        if (keyed) {
          float top = -INFINITY;                 // lane x's own: row x's max in this warp
#pragma unroll
          for (int x = 0; x < kFew; ++x) {
            if (x >= vr) continue;
            const float v = warp_max(sv[x]);
            if (lane == x) top = v;
          }
          if (lane < kFew) mine[q4 * kFew + lane] = top;
          __syncwarp();
          if (lane == 0) mbar_arrive(bTop + 8u * odd);
        }
        ok = __all_sync(0xffffffffu, ctl.wait(bTop + 8u * odd, moved >> odd & 1u));
        if (!ok) break;
        moved ^= 1u << odd;
        float alpha[kFew];
#pragma unroll
        for (int x = 0; x < kFew; ++x) {
          alpha[x] = 1.f;
          if (x >= vr) continue;
          const float mb = fmaxf(mine[x], mine[kFew + x]) * sl2;
          const float old = fresh >> x & 1u ? -INFINITY : -neg[x];
          if (mb > old + kRescaleThreshold) {
            alpha[x] = ex2(old - mb);
            neg[x] = -mb;
            fresh &= ~(1u << x);
          }
          l[x] *= alpha[x];
          if (keyed) pr[x] = ex2(fmaf(sv[x], sl2, neg[x]));
        }
        if (c > 0) {
          ok = __all_sync(0xffffffffu, ctl.wait(bODone(c - 1), parV(c - 1)));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float ov[kFew];
            tmem_ld8(lane_base + S::kColO + half * kFew, ov);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < kFew; ++x) ov[x] *= alpha[x];
            tmem_st8(lane_base + S::kColO + half * kFew, ov);
          }
          tmem_wait_st();
        }
      }
      if (keyed) {
        const uint32_t to = base + S::kOffP + (c % kKS) * S::kPBytes + (key >> 3) * S::kKeysP + (key & 7) * 16;
        uint32_t hi[kFew / 2], lo[kFew / 2];
#pragma unroll
        for (int x = 0; x < kFew; x += 2) {
          split2(pr[x], pr[x + 1], hi[x / 2], lo[x / 2]);
          l[x] += pr[x];
          l[x + 1] += pr[x + 1];
        }
        st_shared_v4(to, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(to + 128, lo[0], lo[1], lo[2], lo[3]);
        if (ends) {
          // values behind the cached tokens, as below
          ok = __all_sync(0xffffffffu, ctl.wait(bVFull(c), parV(c)));
          if (!ok) break;
          const uint32_t v0 = sV + (c % kVS) * S::kTileBytes;
          const int total = (kChunk - r.tail) * (HD / 8);
          for (int x = key; x < total; x += 64) {
            const int at = r.tail + x / (HD / 8), piece = x % (HD / 8);
            st_shared_v4(v0 + (piece >> 3) * S::kAtomKV + at * 128 + (piece & 7) * 16, 0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async();
      }
      tc_fence_before();
      mbar_arrive(bPFull(c));
    }
    if (ok) ok = __all_sync(0xffffffffu, ctl.wait(bODone(nch - 1), parV(nch - 1)));
    if (ok) {
      tc_fence_after();
      float hi[kFew], lo[kFew];
      tmem_ld8(lane_base + S::kColO, hi);
      tmem_ld8(lane_base + S::kColO + kFew, lo);
      tmem_wait_ld();
      if (key < HD) {
#pragma unroll
        for (int x = 0; x < kFew; ++x)
          if (x < vr) (ALONE ? reinterpret_cast<float*>(smem) + x * HD : p.part_o + (part + x) * HD)[key] = hi[x] + lo[x];
      }
      // the rows' sums over the two warps with keys
      float* const s_sum = s_max + 4 * kFew;
      if (keyed) {
        float mine = 0.f;
#pragma unroll
        for (int x = 0; x < kFew; ++x) {
          float v = l[x];
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
          if (lane == x) mine = v;
        }
        if (lane < kFew) s_sum[q4 * kFew + lane] = mine;
        __syncwarp();
        if (lane == 0) mbar_arrive(bSum);
      }
      if (q4 == 0 && __all_sync(0xffffffffu, ctl.wait(bSum, 0))) {
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < kFew; ++x)
          if (lane == x && !(fresh >> x & 1u)) top = -neg[x];
        if (lane < vr) (ALONE ? s_end->ml : p.part_ml + part)[lane] = make_float2(top, s_sum[lane] + s_sum[kFew + lane]);
      }
    }
  } else if ((warp & 3) < warps) {
    // ================================================================ softmax, one row per thread
    const int q4 = warp & 3;
    const int row = q4 * 32 + lane;
    const bool mine = row < vr;
    const uint32_t lane_base = tmem + (uint32_t(q4 * 32) << 16);
    const float sl2 = p.scale_log2;
    float m2 = -INFINITY, l = 0.f;
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      ok = __all_sync(0xffffffffu, ctl.wait(bSFull(c), parK(c)));
      if (!ok) break;
      tc_fence_after();
      float sv[kChunk];
      const uint32_t s_col = lane_base + S::kColS + (c % kKS) * kChunk;
      tmem_ld32(s_col, sv);
      tmem_ld32(s_col + 32, sv + 32);
      tmem_wait_ld();
      const bool ends = r.c0 + c == r.last && r.tail < kChunk;
      if (ends) {
#pragma unroll
        for (int x = 0; x < kChunk; ++x)
          if (x >= r.tail) sv[x] = -INFINITY;
      }
      if constexpr (!TREE) {
        if (mine) {
          float4* to = reinterpret_cast<float4*>(p.scores + size_t(f0 + mt * kTileM + row) * p.score_stride +
                                                 size_t(r.c0 + c) * kChunk);
#pragma unroll
          for (int x = 0; x < kChunk; x += 4) to[x / 4] = make_float4(sv[x], sv[x + 1], sv[x + 2], sv[x + 3]);
        }
      }
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int x = 0; x < kChunk; x += 4) {
        mx0 = max3(mx0, sv[x], sv[x + 1]);
        mx1 = max3(mx1, sv[x + 2], sv[x + 3]);
      }
      const float mb = fmaxf(mx0, mx1) * sl2;
      // the row moves its max only by more than 2^8; -inf (no finite score yet) always moves
      float alpha = 1.f;
      const bool need = mb > m2 + kRescaleThreshold;
      if (need) {
        alpha = ex2(m2 - mb);
        m2 = mb;
      }
      // (a row that the tile only has room for gets P = 0, not the 1 of its zero
      // scores, which would cost the tensor cores power)
      const float neg_m = !mine ? -INFINITY : m2 == -INFINITY ? 0.f : -m2;
      float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
      for (int x = 0; x < kChunk; x += 4) {
        float x0, x1, x2, x3;
        fma2(x0, x1, sv[x], sv[x + 1], sl2, neg_m);
        fma2(x2, x3, sv[x + 2], sv[x + 3], sl2, neg_m);
        sv[x] = ex2(x0);
        sv[x + 1] = ex2(x1);
        sv[x + 2] = ex2(x2);
        sv[x + 3] = ex2(x3);
        add2(s0, s1, sv[x], sv[x + 1]);
        add2(s2, s3, sv[x + 2], sv[x + 3]);
      }
      l = l * alpha + ((s0 + s1) + (s2 + s3));
      if (c > 0 && __any_sync(0xffffffffu, need && mine)) {
        ok = __all_sync(0xffffffffu, ctl.wait(bODone(c - 1), parV(c - 1)));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < HD / 32; ++x) {
          float ov[32];
          tmem_ld32(lane_base + S::kColO + x * 32, ov);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] *= alpha;
          tmem_st32(lane_base + S::kColO + x * 32, ov);
        }
      }
#pragma unroll
      for (int x = 0; x < kChunk / 32; ++x) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          split2(sv[x * 32 + 2 * e], sv[x * 32 + 2 * e + 1], hi[e], lo[e]);
        }
        tmem_st16(s_col + x * 16, hi);
        tmem_st16(s_col + 32 + x * 16, lo);
      }
      tmem_wait_st();
      if (ends) {
        // Values behind the cached tokens are whatever the page holds, and
        // 0 * NaN is NaN: they are cleared before the product reads them.
        ok = __all_sync(0xffffffffu, ctl.wait(bVFull(c), parV(c)));
        if (!ok) break;
        const uint32_t v0 = sV + (c % kVS) * S::kTileBytes;
        const int total = (kChunk - r.tail) * (HD / 8);
        for (int x = row; x < total; x += 32 * warps) {
          const int key = r.tail + x / (HD / 8), piece = x % (HD / 8);
          st_shared_v4(v0 + (piece >> 3) * S::kAtomKV + key * 128 + (piece & 7) * 16, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
      }
      tc_fence_before();
      mbar_arrive(bPFull(c));
    }
    if (ok) ok = __all_sync(0xffffffffu, ctl.wait(bODone(nch - 1), parV(nch - 1)));
    if (ok) {
      tc_fence_after();
      float4* to = reinterpret_cast<float4*>(p.part_o + (part + row) * HD);
#pragma unroll
      for (int x = 0; x < HD / 32; ++x) {
        float ov[32];
        tmem_ld32(lane_base + S::kColO + x * 32, ov);
        tmem_wait_ld();
        if (mine) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) to[x * 8 + e / 4] = make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
        }
      }
    }
    if (mine) p.part_ml[part + row] = make_float2(m2, l);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
  // 1: a page was out of range, 2: a wait ran out (the partial result is not whole)
  const int state = *s_flag | (*abort_flag ? 2 : 0);
  if constexpr (!ALONE) {
    if (threadIdx.x == 0) p.part_flag[size_t(unit) * p.S + run] = state;
  } else {
    // ================================================================ the step's end, by the unit's cluster
    // Each CTA has its O in its query tile's place, and m and l behind it; a row's
    // are joined by the CTA whose turn it is, and each CTA adds the weights of
    // its own keys, a thread those whose scores it wrote.
    const int tid = threadIdx.x;
    if (tid == 0) s_end->state = state;
    if (nch <= 0 && tid < kFew) s_end->ml[tid] = make_float2(-INFINITY, 0.f);
    const int key = (warp & 3) * 32 + lane;
    const bool keyed = warp >= 2 && key < kChunk;
    int u[kAloneChunks];
    float old[kAloneChunks];
    float* const w = p.weights + size_t(b * p.hkv + (p.L == 1 ? hg : hg / (p.H / p.hkv))) * p.weights_stride;
#pragma unroll
    for (int c = 0; c < kAloneChunks; ++c) {
      const int x = r.c0 + c;
      u[c] = -1;
      if (keyed && c < nch && !(x == r.last && key >= r.tail))
        u[c] = p.col_idx[r.start + x / CPB] * BLK + x % CPB * kChunk + key;
    }
#pragma unroll
    for (int c = 0; c < kAloneChunks; ++c) old[c] = u[c] >= 0 ? w[u[c]] : 0.f;
    cluster_sync();
    if (tid < kFew * 8) {                         // row tid / 8, run tid % 8
      const int x = tid >> 3, peer = tid & 7;
      float m = -INFINITY, l = 0.f;
      int flag = 0;
      if (peer < p.S && x < vr) {
        m = ld_peer_f32(peer_addr(&s_end->ml[x].x, peer));
        l = ld_peer_f32(peer_addr(&s_end->ml[x].y, peer));
        flag = ld_peer(peer_addr(&s_end->state, peer));
      }
      float M = l != 0.f ? m : -INFINITY;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      const float wt = l == 0.f ? 0.f : M == -INFINITY ? 1.f : ex2(m - M);
      float L = wt * l;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) flag |= __shfl_xor_sync(0xffffffffu, flag, off);
      s_end->w[x][peer] = wt;
      if (peer == 0) {
        s_end->M[x] = M;
        s_end->L[x] = L;
        s_end->flag[x] = flag;
      }
    }
    __syncthreads();
    const bool refuse = !r.go || s_end->flag[0];
    if (tid < HD) {
      for (int x = run; x < vr; x += p.S) {
        float o = 0.f;
        for (int peer = 0; peer < p.S; ++peer) {
          const float wt = s_end->w[x][peer];
          if (wt != 0.f) o = fmaf(wt, ld_peer_f32(peer_addr(reinterpret_cast<float*>(smem) + x * HD + tid, peer)), o);
        }
        const float L = s_end->L[x];
        const bool none = refuse || L == 0.f;
        p.o[size_t(f0 + x) * HD + tid] = __float2bfloat16_rn(none ? 0.f : o / L);
        if (tid == 0) p.lse[f0 + x] = none ? -INFINITY : (s_end->M[x] + __log2f(L)) * kLn2;
      }
    }
    if (tid == 0 && run == 0 && (!r.go || (s_end->flag[0] & 1))) atomicOr(p.status, kStatusBadIndex);
    if (!refuse) {
      float sum[kAloneChunks] = {};
      for (int x = 0; x < vr; ++x) {
        const float L = s_end->L[x], M = s_end->M[x];
        if (L == 0.f) continue;                   // a row without any weight adds nothing
        const float neg = M == -INFINITY ? 0.f : -M, inv = 1.f / L;
        const float* const sc = p.scores + size_t(f0 + x) * p.score_stride + size_t(r.c0) * kChunk + key;
#pragma unroll
        for (int c = 0; c < kAloneChunks; ++c)
          if (u[c] >= 0) sum[c] = fmaf(ex2(fmaf(sc[c * kChunk], p.scale_log2, neg)), inv, sum[c]);
      }
#pragma unroll
      for (int c = 0; c < kAloneChunks; ++c)
        if (u[c] >= 0) w[u[c]] = old[c] + sum[c];
    }
    cluster_sync();                               // no CTA ends while another may still read its shared memory
  }
}

// ------------------------------------------------------------ kernel 2

constexpr int kJoinWarps = 8;

// The runs of one row joined: M, L and, per lane, HD / 32 columns of O.
template <int HD>
__device__ __forceinline__ int join_runs(const Params& p, int unit, int row, float& M, float& L, float* acc) {
  const int lane = threadIdx.x & 31;
  constexpr int DPL = HD / 32;
  int flag = 0;
  M = -INFINITY;
  for (int s = lane; s < p.S; s += 32) {
    flag |= p.part_flag[size_t(unit) * p.S + s];
    const float2 ml = p.part_ml[(size_t(unit) * p.S + s) * p.cap + row];
    if (ml.y != 0.f) M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  flag = __reduce_or_sync(0xffffffffu, flag);
  L = 0.f;
#pragma unroll
  for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
  for (int s0 = 0; s0 < p.S; s0 += 32) {
    const int s = s0 + lane;
    float w = 0.f;                       // this lane's run's weight
    if (s < p.S) {
      const float2 ml = p.part_ml[(size_t(unit) * p.S + s) * p.cap + row];
      if (ml.y != 0.f) {
        w = M == -INFINITY ? 1.f : ex2(ml.x - M);
        L += w * ml.y;
      }
    }
    const unsigned live = __ballot_sync(0xffffffffu, w != 0.f);
    const int n = min(32, p.S - s0);
    const float* src = p.part_o + ((size_t(unit) * p.S + s0) * p.cap + row) * HD + lane * DPL;
    const size_t step = size_t(p.cap) * HD;
    constexpr int U = 4;                 // runs in flight; one that wrote nothing is not read
    for (int x0 = 0; x0 < n; x0 += U) {
      float v[U][DPL];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool on = x0 + u < n && (live >> (x0 + u) & 1u);
        if constexpr (DPL == 4) {
          const float4 t = on ? *reinterpret_cast<const float4*>(src + (x0 + u) * step) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[u][0] = t.x;
          v[u][1] = t.y;
          v[u][2] = t.z;
          v[u][3] = t.w;
        } else {
          const float2 t = on ? *reinterpret_cast<const float2*>(src + (x0 + u) * step) : make_float2(0.f, 0.f);
          v[u][0] = t.x;
          v[u][1] = t.y;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float wx = __shfl_sync(0xffffffffu, w, (x0 + u) & 31);
#pragma unroll
        for (int e = 0; e < DPL; ++e) acc[e] = fmaf(x0 + u < n ? wx : 0.f, v[u][e], acc[e]);
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  return flag;
}

template <int HD>
__device__ __forceinline__ void store_row(const Params& p, size_t row, bool refuse, float M, float L, const float* acc) {
  const int lane = threadIdx.x & 31;
  constexpr int DPL = HD / 32;
  const bool none = refuse || L == 0.f;
  float v[DPL];
#pragma unroll
  for (int e = 0; e < DPL; ++e) v[e] = none ? 0.f : acc[e] / L;
  uint32_t* to = reinterpret_cast<uint32_t*>(p.o + row * HD + lane * DPL);
  if constexpr (DPL == 4) *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  else *to = pack_bf16(v[0], v[1]);
  if (lane == 0) p.lse[row] = none ? -INFINITY : (M + __log2f(L)) * kLn2;
}

// Block j's place in row `at` of the layout, -1 if the row does not keep it.
__device__ __forceinline__ int find_block(const Params& p, size_t at, int j) {
  int lo = p.row_ptr[at], hi = p.row_ptr[at + 1];
  const int first = lo;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.col_idx[mid] < j) lo = mid + 1;
    else hi = mid;
  }
  return lo < p.row_ptr[at + 1] && p.col_idx[lo] == j ? lo - first : -1;
}

// The step: blocks [0, row_blocks) join one row per warp; the others turn the
// scores of kTileKeys list keys of a key/value head into weights, kGroups
// times four keys a thread.  (With 256 keys a block the 16 x 16K step spent
// 82 us here, most of it on finding M and L again.)
constexpr int kGroups = 4, kGroupKeys = 4 * kJoinWarps * 32, kTileKeys = kGroups * kGroupKeys;

template <int BLK, int HD>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) join_step_kernel(const Params p, int heads, int row_blocks) {
  __shared__ float s_m[32], s_l[32];
  __shared__ int s_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_release();
  if (int(blockIdx.x) < row_blocks) {
    const int f = blockIdx.x * kJoinWarps + warp;
    const int b = min(f, heads - 1) / p.H, t = p.lengths[b];
    grid_wait();
    if (f >= heads) return;
    const bool in = t >= 0 && t < p.n;
    float M = -INFINITY, L = 0.f, acc[HD / 32] = {};
    int flag = 0;
    if (in) {
      const int hh = f - b * p.H;
      const int unit = (b * p.hg + hh / p.hpt) * p.mtiles + hh % p.hpt / kTileM;
      flag = join_runs<HD>(p, unit, hh % p.hpt % kTileM, M, L, acc);
    }
    store_row<HD>(p, f, !in || flag, M, L, acc);
    if (lane == 0 && (!in || (flag & 1))) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  // ---- weights.  With one route for all heads a block takes list keys of a
  // key/value head and sums its query heads; with a route per head it takes
  // list keys of one query head, and of the key blocks that several heads of
  // the group keep each is summed by the first of them.
  const int x = blockIdx.x - row_blocks;
  const int tile = x % p.tiles, hg = x / p.tiles;           // hg over batch * head groups
  const int g = p.H / p.hkv;
  const int b = hg / p.hg, h0 = (hg - b * p.hg) * p.hpt;    // the block's query head(s) in the sequence
  // A refused position counts as -1, below every key: the keys that a thread
  // does not have are INT32_MAX, which a position of that value would reach.
  const int pos = p.lengths[b];
  const bool in = pos >= 0 && pos < p.n;
  const int t = in ? pos : -1;
  const size_t at0 = size_t((b * p.H + h0) % p.L) * p.nb + (in ? t / BLK : 0);
  const int start = p.row_ptr[at0], list = in ? (p.row_ptr[at0 + 1] - start) * BLK : 0;
  const int kv = h0 / g, first = p.L == 1 ? h0 : kv * g;    // first query head of the group
  float* const w = p.weights + size_t(b * p.hkv + kv) * p.weights_stride;
  // What needs no result of kernel 1 comes before the wait for it: kernel 1
  // lets this one start only once its own wait is over, so whatever the stream
  // held before it has ended.  The running weights are read at L2, past any
  // piece of them that this SM kept from the step before.
  int u[kGroups];                                           // first of four keys; INT32_MAX if there are none
  float old[kGroups][4];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int k = tile * kTileKeys + i * kGroupKeys + int(threadIdx.x) * 4;
    u[i] = k < list ? p.col_idx[start + k / BLK] * BLK + k % BLK : INT32_MAX;
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) old[i][e] = u[i] <= t && u[i] + e <= t ? __ldcg(w + u[i] + e) : 0.f;
  grid_wait();
  if (tile * kTileKeys >= list) return;
  float sum[kGroups][4] = {};
  // up to 32 query heads of the group at a time: their M and L, then their scores
#pragma unroll 1
  for (int h1 = 0; h1 < g; h1 += 32) {
    const int count = min(32, g - h1);
    __syncthreads();
    if (threadIdx.x == 0) s_flag = 0;
    __syncthreads();
#pragma unroll 1
    for (int h = warp; h < count; h += kJoinWarps) {
      const int hh = first + h1 + h;
      const int unit = (b * p.hg + hh / p.hpt) * p.mtiles + hh % p.hpt / kTileM, row = hh % p.hpt % kTileM;
      float M = -INFINITY, L = 0.f;
      int flag = 0;
      for (int s = lane; s < p.S; s += 32) {
        flag |= p.part_flag[size_t(unit) * p.S + s];
        const float2 ml = p.part_ml[(size_t(unit) * p.S + s) * p.cap + row];
        if (ml.y == 0.f) continue;
        const float m = fmaxf(M, ml.x);
        // L stays under the running max; -inf only while every l seen is a NaN's
        L = (M == -INFINITY ? L : L * ex2(M - m)) + (ml.x == -INFINITY ? ml.y : ml.y * ex2(ml.x - m));
        M = m;
      }
      const float mine = M;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      if (mine != -INFINITY) L *= ex2(mine - M);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
      flag = __reduce_or_sync(0xffffffffu, flag);
      if (lane == 0) {
        s_m[h] = M == -INFINITY ? 0.f : -M;
        s_l[h] = L;
        if (flag) atomicOr(&s_flag, 1 << h);
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int h = 0; h < count; ++h) {
      const int hh = first + h1 + h;
      // a refused row and a row without any weight add nothing
      const float l = s_l[h], neg = s_m[h], inv = 1.f / l;
      const bool adds = !(s_flag >> h & 1) && l != 0.f;
      const float* const sc = p.scores + size_t(b * p.H + hh) * p.score_stride;
      const size_t at = size_t((b * p.H + hh) % p.L) * p.nb + t / BLK;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        if (u[i] > t) continue;
        int k = tile * kTileKeys + i * kGroupKeys + int(threadIdx.x) * 4;
        if (p.L > 1 && hh != h0) {
          const int e = find_block(p, at, u[i] / BLK);
          if (e < 0) continue;
          if (hh < h0) {                 // an earlier head of the group keeps the block and sums it
            u[i] = INT32_MAX;
            continue;
          }
          k = e * BLK + u[i] % BLK;
        }
        if (!adds) continue;
        const float4 v = *reinterpret_cast<const float4*>(sc + k);
        sum[i][0] = fmaf(ex2(fmaf(v.x, p.scale_log2, neg)), inv, sum[i][0]);
        sum[i][1] = fmaf(ex2(fmaf(v.y, p.scale_log2, neg)), inv, sum[i][1]);
        sum[i][2] = fmaf(ex2(fmaf(v.z, p.scale_log2, neg)), inv, sum[i][2]);
        sum[i][3] = fmaf(ex2(fmaf(v.w, p.scale_log2, neg)), inv, sum[i][3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (u[i] <= t && u[i] + e <= t) w[u[i] + e] = old[i][e] + sum[i][e];
}

// The tree: one row (query head, drafted token) per warp, its runs joined with
// its ancestors' keys.
template <int BLK, int HD>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) join_tree_kernel(const Params p) {
  constexpr int DPL = HD / 32, CPL = HD / 8;
  __shared__ int s_par[kMaxT];
  __shared__ int s_path[kJoinWarps][kMaxT];       // ancestors from the token up to its root
  __shared__ float s_sc[kJoinWarps][kMaxT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_release();
  const int tb = (p.T + kJoinWarps - 1) / kJoinWarps;
  const int f = blockIdx.x / tb, i = blockIdx.x % tb * kJoinWarps + warp;
  const int b = f / p.H, hh = f - b * p.H;
  for (int x = threadIdx.x; x < p.T; x += blockDim.x) s_par[x] = p.parents[size_t(b) * p.T + x];
  __syncthreads();
  const int len = p.lengths[b];
  const bool live = i < p.T && s_par[i] != -2;    // an unused row is left as it was
  // the path to the root; every parent is an earlier token, so the walk ends
  int count = 0;
  bool bad = len < 0 || len > p.n;
  if (live) {
    for (int x = i;;) {
      if (lane == 0) s_path[warp][count] = x;
      ++count;
      const int up = s_par[x];
      if (up == -1) break;
      if (up < 0 || up >= x) {
        bad = true;
        break;
      }
      x = up;
    }
  }
  __syncwarp();
  if (!bad && live && count > p.n - len) bad = true;   // past the layout's last position
  const int pos = bad ? 0 : len + count - 1;
  // the layout row of the token, and which of the blocks that its path lies in it keeps
  const int blk = pos / BLK, blk0 = bad ? 0 : len / BLK;
  const size_t at = size_t(f % p.L) * p.nb + blk;
  // (they are the row's last entries: its columns ascend up to the row itself)
  unsigned keeps = 0;
  if (live && !bad && lane <= blk - blk0) {
    const int e = p.row_ptr[at + 1] - 1 - lane;
    const int j = e >= p.row_ptr[at] ? p.col_idx[e] : -1;
    if (j >= blk0) keeps = 1u << (j - blk0);
  }
  keeps = __reduce_or_sync(0xffffffffu, keeps);
  int grp = blk - blk0;                           // whose runs the row reads: see kernel 1
  if (live && !bad && grp > 0) {
    const int blocks = len / BLK + (len % BLK != 0);
    if (keeps_all(p, at, blocks) && keeps_all(p, at - grp, blocks)) grp = 0;
  }
  // scores of the ancestors: 8 lanes a key, four keys at a time
  const int sub = lane >> 3, pc = lane & 7;
  const int kvh = b * p.hkv + hh / (p.H / p.hkv);
  float top = -INFINITY, sum = 0.f, anc[DPL] = {};   // the ancestors' part, under its own max
  if (live && !bad) {
    float qr[CPL];
    const uint4* qs = reinterpret_cast<const uint4*>(p.q + (size_t(f) * p.T + i) * HD + pc * CPL);
#pragma unroll
    for (int c = 0; c < CPL / 8; ++c) {
      const uint4 w = qs[c];
      bf16x2_to_f32(w.x, qr[c * 8], qr[c * 8 + 1]);
      bf16x2_to_f32(w.y, qr[c * 8 + 2], qr[c * 8 + 3]);
      bf16x2_to_f32(w.z, qr[c * 8 + 4], qr[c * 8 + 5]);
      bf16x2_to_f32(w.w, qr[c * 8 + 6], qr[c * 8 + 7]);
    }
    for (int x0 = 0; x0 < count; x0 += 4) {
      const int x = x0 + sub;
      const bool use = x < count && (keeps >> ((len + count - 1 - x) / BLK - blk0) & 1u);
      float dot = 0.f;
      if (use) {
        const uint4* ks = reinterpret_cast<const uint4*>(p.k_tree + (size_t(kvh) * p.T + s_path[warp][x]) * HD + pc * CPL);
#pragma unroll
        for (int c = 0; c < CPL / 8; ++c) {
          const uint4 w = ks[c];
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float k0, k1;
            bf16x2_to_f32(ws[e], k0, k1);
            dot = fmaf(k0, qr[c * 8 + 2 * e], dot);
            dot = fmaf(k1, qr[c * 8 + 2 * e + 1], dot);
          }
        }
      }
      dot += __shfl_xor_sync(0xffffffffu, dot, 1);
      dot += __shfl_xor_sync(0xffffffffu, dot, 2);
      dot += __shfl_xor_sync(0xffffffffu, dot, 4);
      const float s = use ? dot * p.scale_log2 : -INFINITY;
      if (pc == 0 && x < count) s_sc[warp][x] = s;
      top = fmaxf(top, s);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
    __syncwarp();
    for (int x = lane; x < count; x += 32) {
      const float s = s_sc[warp][x];
      // one that is not read gets 0 and, as 0 times its value may be NaN, is left out below
      const bool use = keeps >> ((len + count - 1 - x) / BLK - blk0) & 1u;
      const float w = use ? ex2(s - (top == -INFINITY ? 0.f : top)) : 0.f;
      s_sc[warp][x] = w;
      sum += w;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    __syncwarp();
#pragma unroll 4
    for (int x = 0; x < count; ++x) {
      if (!(keeps >> ((len + count - 1 - x) / BLK - blk0) & 1u)) continue;
      const float w = s_sc[warp][x];
      const uint32_t* vs = reinterpret_cast<const uint32_t*>(p.v_tree + (size_t(kvh) * p.T + s_path[warp][x]) * HD + lane * DPL);
#pragma unroll
      for (int e = 0; e < DPL; e += 2) {
        float v0, v1;
        bf16x2_to_f32(vs[e / 2], v0, v1);
        anc[e] = fmaf(w, v0, anc[e]);
        anc[e + 1] = fmaf(w, v1, anc[e + 1]);
      }
    }
  }
  grid_wait();                                    // the runs of kernel 1 are in memory from here on
  if (!live) return;
  float M = -INFINITY, L = 0.f, acc[DPL] = {};
  int flag = 0;
  if (!bad) {
    const int row = hh % p.hpt * p.T + i;
    const int unit = grp * p.per_group + (b * p.hg + hh / p.hpt) * p.mtiles + row / kTileM;
    flag = join_runs<HD>(p, unit, row % kTileM, M, L, acc);
    // the cache's part and the path's under one max
    const float all = fmaxf(M, top);
    const float a = M == -INFINITY ? (L == 0.f ? 0.f : 1.f) : ex2(M - all);
    const float c = top == -INFINITY ? 1.f : ex2(top - all);
    L = fmaf(L, a, sum * c);
#pragma unroll
    for (int e = 0; e < DPL; ++e) acc[e] = fmaf(acc[e], a, anc[e] * c);
    M = all;
  }
  store_row<HD>(p, size_t(f) * p.T + i, bad || flag, M, L, acc);
  if (lane == 0 && (bad || (flag & 1))) atomicOr(p.status, kStatusBadIndex);
}

// ------------------------------------------------------------ host side

struct Call {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  int batch, heads, kv_heads;
  Plan plan;
  cudaStream_t stream;
};

template <int BLK, int HD, bool TREE, bool FEW, bool ALONE>
int launch_rows(const Call& c, const Params& p) {
  using S = Shape<BLK, HD, FEW>;
  auto kern = paged_attention_kernel<BLK, HD, TREE, FEW, ALONE>;
  // enough shared memory that no third CTA shares an SM: TMEM holds two
  constexpr int smem = S::kSmem < 77 * 1024 ? 77 * 1024 : S::kSmem;
  static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs per SM");
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return set_error(BSA_ERR_CUDA, "cannot query the device");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return set_error(BSA_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
      done[dev] = true;
    }
  }
  CUtensorMap mq, mk, mv;
  int st = tmap::encode_atoms(&mq, c.q, c.batch * c.plan.hg, c.plan.rows, HD, S::kRowsQ);
  if (st == BSA_OK) st = tmap::encode_rows(&mk, c.k_cache, p.num_pages * p.hkv, BLK, HD, kChunk);
  if (st == BSA_OK) st = tmap::encode_rows(&mv, c.v_cache, p.num_pages * p.hkv, BLK, HD, kChunk);
  if (st != BSA_OK) return st;
  st = launch_dependent("paged attention launch", kern, unsigned(c.plan.units) * unsigned(c.plan.S), kThreads, smem,
                        ALONE ? unsigned(c.plan.S) : 1u, c.stream, mq, mk, mv, p);
  if (st != BSA_OK || ALONE) return st;
  if constexpr (TREE) {
    const unsigned tb = unsigned(p.T + kJoinWarps - 1) / kJoinWarps;
    return launch_dependent("tree join launch", join_tree_kernel<BLK, HD>, unsigned(c.heads) * tb, kJoinWarps * 32, 0, 1,
                            c.stream, p);
  } else {
    const int row_blocks = (c.heads + kJoinWarps - 1) / kJoinWarps;
    const unsigned grid = unsigned(row_blocks) + unsigned(c.batch * c.plan.hg) * unsigned(p.tiles);
    return launch_dependent("step join launch", join_step_kernel<BLK, HD>, grid, kJoinWarps * 32, 0, 1, c.stream, p,
                            c.heads, row_blocks);
  }
}

template <int BLK, int HD, bool TREE>
int launch(const Call& c, const Params& p) {
  if constexpr (!TREE)
    if (c.plan.alone) return launch_rows<BLK, HD, false, true, true>(c, p);
  return p.rows <= kFew ? launch_rows<BLK, HD, TREE, true, false>(c, p) : launch_rows<BLK, HD, TREE, false, false>(c, p);
}

bool aligned(const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) % a) == 0; }

// What both entry points check of the sizes; workspace sizes are 0 where it fails.
int check_sizes(const bsa_layout* layout, int batch, int heads, int kv_heads, int T, int d, bool step) {
  if (!layout) return set_error(BSA_ERR_INVALID_ARG, "layout is NULL");
  if (layout->B != 64 && layout->B != 128) return set_error(BSA_ERR_UNSUPPORTED, "B must be 64 or 128");
  if (d != 64 && d != 128) return set_error(BSA_ERR_UNSUPPORTED, "d must be 64 or 128");
  if (batch < 1 || heads < 1 || kv_heads < 1) return set_error(BSA_ERR_SHAPE, "batch, heads and kv_heads must be >= 1");
  if (heads % batch || kv_heads % batch)
    return set_error(BSA_ERR_SHAPE, "heads and kv_heads must be multiples of batch");
  const int H = heads / batch, hkv = kv_heads / batch;
  if (H % hkv) return set_error(BSA_ERR_SHAPE, "query heads per sequence must be a multiple of its kv heads");
  if (H % layout->L) return set_error(BSA_ERR_SHAPE, "query heads per sequence must be a multiple of layout_heads");
  if (T < 1 || T > kMaxT) return set_error(BSA_ERR_UNSUPPORTED, "the tree must have 1 to 128 tokens");
  if (int64_t(H / hkv) * T > INT32_MAX / 2) return set_error(BSA_ERR_SHAPE, "too many query rows");
  const Plan p = plan_of(layout, batch, heads, kv_heads, T, step);
  if (int64_t(p.units) * p.S > INT32_MAX || int64_t(heads) * ((T + kJoinWarps - 1) / kJoinWarps) > INT32_MAX / 2)
    return set_error(BSA_ERR_SHAPE, "too many query rows");
  return BSA_OK;
}

int check_call(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table, int max_blocks,
               int num_pages, const int32_t* lengths, const bsa_layout* layout, int batch, int heads, int kv_heads,
               int T, int d, float scale, const void* o, const float* lse, bool step) {
  if (!layout) return set_error(BSA_ERR_INVALID_ARG, "layout is NULL");
  const int st = check_sizes(layout, batch, heads, kv_heads, T, d, step);
  if (st != BSA_OK) return st;
  if (max_blocks < layout->nb) return set_error(BSA_ERR_SHAPE, "max_blocks is smaller than the layout's blocks");
  if (num_pages < 1 || int64_t(num_pages) * (kv_heads / batch) > INT32_MAX)
    return set_error(BSA_ERR_SHAPE, "num_pages must be >= 1 and num_pages * kv heads below 2^31");
  if (!(std::isfinite(scale) && scale > 0.f)) return set_error(BSA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!q || !k_cache || !v_cache || !page_table || !lengths || !o || !lse)
    return set_error(BSA_ERR_INVALID_ARG, "null pointer");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16))
    return set_error(BSA_ERR_INVALID_ARG, "q, k_cache, v_cache and o must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(page_table, 4) || !aligned(lengths, 4))
    return set_error(BSA_ERR_INVALID_ARG, "lse, page_table and positions or lengths must be 4-byte aligned");
  return BSA_OK;
}

int run(bool tree, const void* q, const void* k_tree, const void* v_tree, const void* k_cache, const void* v_cache,
        const int32_t* page_table, int max_blocks, int num_pages, const int32_t* lengths, const int32_t* parents,
        const bsa_layout* layout, int T, int batch, int heads, int kv_heads, int d, float scale, void* o, float* lse,
        float* weights, size_t weights_stride, void* workspace, size_t workspace_bytes, void* stream) {
  const Plan pl = plan_of(layout, batch, heads, kv_heads, T, !tree);
  const Offsets of = offsets_of(pl, layout, heads, d, !tree);
  if (!workspace || !aligned(workspace, 16))
    return set_error(BSA_ERR_INVALID_ARG, "workspace must be non-null and 16-byte aligned");
  if (workspace_bytes < of.total)
    return set_error(BSA_ERR_SHAPE, "workspace too small: " + std::to_string(of.total) + " bytes needed");
  int st = check_layout_device(layout);
  if (st == BSA_OK) st = tmap::get_encoder();
  if (st != BSA_OK) return st;
  char* w = static_cast<char*>(workspace);
  Params p{};
  p.page_table = page_table;
  p.lengths = lengths;
  p.parents = parents;
  p.row_ptr = layout->d_row_ptr;
  p.col_idx = layout->d_col_idx;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_tree = static_cast<const __nv_bfloat16*>(k_tree);
  p.v_tree = static_cast<const __nv_bfloat16*>(v_tree);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.part_o = reinterpret_cast<float*>(w);
  p.part_ml = reinterpret_cast<float2*>(w + of.ml);
  p.part_flag = reinterpret_cast<int*>(w + of.flag);
  p.scores = reinterpret_cast<float*>(w + of.scores);
  p.score_stride = size_t(layout->max_row) * layout->B;
  p.status = layout->d_status;
  p.n = layout->n;
  p.nb = layout->nb;
  p.L = layout->L;
  p.H = heads / batch;
  p.hkv = kv_heads / batch;
  p.max_blocks = max_blocks;
  p.num_pages = num_pages;
  p.hg = pl.hg;
  p.hpt = pl.hpt;
  p.rows = pl.rows;
  p.mtiles = pl.mtiles;
  p.per_group = pl.units / pl.groups;
  p.S = pl.S;
  p.cap = pl.cap;
  p.T = T;
  p.tiles = std::max(1, (layout->max_row * layout->B + kTileKeys - 1) / kTileKeys);
  p.scale_log2 = float(double(scale) * 1.4426950408889634);
  const Call c{q, k_cache, v_cache, batch, heads, kv_heads, pl, static_cast<cudaStream_t>(stream)};
  const int B = layout->B;
  if (tree) {
    if (B == 64) return d == 128 ? launch<64, 128, true>(c, p) : launch<64, 64, true>(c, p);
    return d == 128 ? launch<128, 128, true>(c, p) : launch<128, 64, true>(c, p);
  }
  if (B == 64) return d == 128 ? launch<64, 128, false>(c, p) : launch<64, 64, false>(c, p);
  return d == 128 ? launch<128, 128, false>(c, p) : launch<128, 64, false>(c, p);
}

}  // namespace paged
}  // namespace bsa

extern "C" {

size_t bsa_decode_weights_workspace_bytes(const bsa_layout* layout, int batch, int heads, int kv_heads, int d) {
  using namespace bsa::paged;
  if (check_sizes(layout, batch, heads, kv_heads, 1, d, true) != BSA_OK) return 0;
  return offsets_of(plan_of(layout, batch, heads, kv_heads, 1, true), layout, heads, d, true).total;
}

size_t bsa_decode_tree_workspace_bytes(const bsa_layout* layout, int batch, int heads, int kv_heads, int T, int d) {
  using namespace bsa::paged;
  if (check_sizes(layout, batch, heads, kv_heads, T, d, false) != BSA_OK) return 0;
  return offsets_of(plan_of(layout, batch, heads, kv_heads, T, false), layout, heads, d, false).total;
}

int bsa_decode_weights(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                       int max_blocks, int num_pages, const int32_t* positions, const bsa_layout* layout, int batch,
                       int heads, int kv_heads, int d, float scale, void* o, float* lse, float* weights,
                       size_t weights_stride, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace bsa;
  const int st = paged::check_call(q, k_cache, v_cache, page_table, max_blocks, num_pages, positions, layout, batch,
                                   heads, kv_heads, 1, d, scale, o, lse, true);
  if (st != BSA_OK) return st;
  if (!weights || !paged::aligned(weights, 4))
    return set_error(BSA_ERR_INVALID_ARG, "weights must be non-null and 4-byte aligned");
  if (weights_stride < size_t(layout->n)) return set_error(BSA_ERR_SHAPE, "weights_stride is smaller than the layout's n");
  return paged::run(false, q, nullptr, nullptr, k_cache, v_cache, page_table, max_blocks, num_pages, positions, nullptr,
                    layout, 1, batch, heads, kv_heads, d, scale, o, lse, weights, weights_stride, workspace,
                    workspace_bytes, stream);
}

int bsa_decode_tree(const void* q, const void* k_tree, const void* v_tree, const void* k_cache, const void* v_cache,
                    const int32_t* page_table, int max_blocks, int num_pages, const int32_t* lengths,
                    const int32_t* parents, const bsa_layout* layout, int T, int batch, int heads, int kv_heads, int d,
                    float scale, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace bsa;
  const int st = paged::check_call(q, k_cache, v_cache, page_table, max_blocks, num_pages, lengths, layout, batch, heads,
                                   kv_heads, T, d, scale, o, lse, false);
  if (st != BSA_OK) return st;
  if (!k_tree || !v_tree || !parents) return set_error(BSA_ERR_INVALID_ARG, "null pointer");
  if (!paged::aligned(k_tree, 16) || !paged::aligned(v_tree, 16))
    return set_error(BSA_ERR_INVALID_ARG, "k_tree and v_tree must be 16-byte aligned");
  if (!paged::aligned(parents, 4)) return set_error(BSA_ERR_INVALID_ARG, "parents must be 4-byte aligned");
  return paged::run(true, q, k_tree, v_tree, k_cache, v_cache, page_table, max_blocks, num_pages, lengths, parents,
                    layout, T, batch, heads, kv_heads, d, scale, o, lse, nullptr, 0, workspace, workspace_bytes, stream);
}

}  // extern "C"
