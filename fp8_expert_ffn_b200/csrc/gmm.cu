// Products grouped by expert over ragged rows, in bf16 or fp16 with fp32
// accumulation: the forward product of an expert's weight and its two
// gradients. With group g's rows r in [offsets[g], offsets[g+1]):
//   forward  y[r, n]     = sum_k x[r, k] w[g, n, k]
//   dgrad    dx[r, k]    = sum_n dy[r, n] w[g, n, k]
//   wgrad    dw[g, n, k] = sum_r dy[r, n] x[r, k]   (+ dw when accumulating)
//
// All three are one tile product D[c, r] = sum_i A[i, c] B[i, r]: c is the
// output's contiguous dimension, r its rows, i the contraction. The output's
// columns sit on the MMA's M dimension (TMEM lanes) and its rows on N, so
//   - a ragged group costs only the MMA columns of its own rows (N is the
//     number of rows rounded up to 32, 256 at most) where rows on M would
//     always pay for 128 or 256;
//   - rows past the group's end are other columns of D that are never
//     stored: whatever they hold (NaN included) cannot reach a result.
// The operands are read as they lie in memory: forward, both K-major; dgrad,
// A = w with the contraction n as its slow dimension (MN-major); wgrad, both
// MN-major over the group's rows. A wgrad block that passes the group's end
// (a tail) must not see the rows past it, in either operand: a NaN there would
// not vanish by a zero in the other one. It is loaded by boxes of 32, 8, 2 and
// 1 rows that end with the group, the MMA takes only as many 16-row slices as
// hold its rows, and what is left of the last slice comes from boxes past the
// operand's last row, which the copies fill with zeros.
//
// Kernel layout: CTA pairs (cluster of 2, tcgen05 cta_group::2, M 256 x N up
// to 256 x K 16 per instruction), persistent over a device-side tile list.
// Each CTA holds its own 128 columns of A and half of B's rows, so a
// 256 x 256 tile moves 32 KB per CTA and 64-deep K block from L2 where two
// independent 128 x 256 tiles would move 48 KB.
//   warp 0      TMA producer into a ring of 6 stages (16 KB of A, up to 16 KB of B)
//   warp 1      TMEM allocation; in the leading CTA the MMA issuer
//   warp 2      in the other CTA: hands accumulators back to the leading one
//   warp 3      idle
//   warps 4-11  epilogue, two warpgroups with 128 output rows each: TMEM lanes
//               32*(w%4).., one output column per lane; two 256-column TMEM
//               buffers overlap it with the next tile. Outputs go through
//               shared memory to bulk tensor stores (16-byte aligned rows), or
//               straight to memory where they cannot.
// Bound: the tensor cores, at the power limit, for more than about 250 rows
// per group. A training batch of 36,864 rows over 33 uneven experts,
// 1536 x 5120: 508 us back to back (1.14 PFLOP/s; 993 W, SM clock 1177 of 1965
// MHz) and 402 us one at a time; one group of as many rows 458 and 358 us
// where cuBLAS takes 437 and 352. HBM below (one decode step of 65 experts:
// 170 us, 6.1 TB/s).
// Hand-over between the CTAs: the leading CTA's MMA reads stages that lie in
// the other one, so both CTAs' copies complete on the leading CTA's barrier
// (the cta_group::2 form of the loads; a completion releases what its copy
// wrote at cluster scope), where each CTA has announced its own. Waits on
// barriers that the other CTA signals acquire, and arrivals by threads release,
// at cluster scope. The other CTA's epilogue leaves the release of an
// accumulator to warp 2 (a release by its own warps held the wgrad over 512
// rows per group up by 7 of 101 us).
// No TMA multicast; commits signal both CTAs. Every wait is bounded (1 s): on
// a timeout the status word is set, all roles leave, copies in flight are
// waited for (bounded) and the TMEM is released.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "groups.cuh"
#include "internal.h"
#include "pair.cuh"

namespace moe {

namespace {

constexpr int BC = 256;                 // output columns per tile (128 per CTA)
constexpr int BK = 64;                  // contraction per stage (128 bytes)
constexpr int A_BYTES = 128 * BK * 2;   // 16 KB
constexpr int BOX_BYTES = 64 * 64 * 2;  // one MN-major box: 64 contraction rows x 64 columns
constexpr int FIRST_EPI_WARP = 4;
constexpr int RCHUNK = 8;               // row tiles per chunk of the tile order
constexpr uint32_t TMEM_COLS = 512;
constexpr int STG_BYTES = 8192;         // one staged chunk of output rows: 32 rows x 128 columns of 16 bits, or 16 of fp32
constexpr int TMEM_BUF = 256;           // TMEM columns of one of the two accumulators

// BR: output rows per tile, at most. 256 fill the MMA; 64 are for a few rows
// per group, where the stages hold little but weights and more of them can be
// on their way (10 stages of 20 KB instead of 6 of 32 KB: one decode step of
// 65 experts, 1 GB of weights, 178 -> 170 us).
constexpr int stage_bytes(int BR) { return A_BYTES + BR * BK; }   // each CTA holds half of the rows

// PROMOTE: a contraction too long for one accumulator. The MMA adds to its
// fp32 accumulator by truncation, so a sum's error grows with its length: for
// terms of one sign by 0.85 2^-23 of the result per 16 terms (measured to
// 65,536 fp16 terms, where it was 0.86 of half a step of the output). These
// tiles hand the accumulator over every segment of K blocks and the epilogue
// adds the parts in registers, rounding to nearest: 8 warps with 128 rows of a
// column each, their registers taken from the other warps as in the FP8 GEMMs.
// The segment follows from the output's type: 512 terms for fp32 (2.3e-6 of
// the result after 2,600 terms in one sum, 4.7e-7 so), and where the
// truncation is at most 0.08 of half a step, 6,144 terms for fp16 and
// 49,152 for bf16. A tile's own length decides where its sum is cut, so its
// bits do not depend on the rest of the launch.
constexpr int segment(moe_dtype out) { return out == MOE_F32 ? 8 : out == MOE_F16 ? 96 : 768; }

// Epilogue warps: two warpgroups with 128 rows each, or one where tiles have
// 64 rows (with one for 256 rows, a weight gradient over 512 rows per group
// waited for its stores: 11.7 thousand cycles per tile, 4.1 of them MMA).
constexpr int epi_warps(int BR, bool promote) { return BR == 256 || promote ? 8 : 4; }
constexpr int threads(int BR, bool promote) { return 32 * (FIRST_EPI_WARP + epi_warps(BR, promote)); }
constexpr int stages(int BR, bool promote) { return BR == 256 ? 6 : 10; }
// Two staged chunks: one per warpgroup, or two of the only one.
constexpr int smem_dyn(int BR, bool promote) { return stages(BR, promote) * stage_bytes(BR) + 2 * STG_BYTES + 1024; }
constexpr int LAUNCH_REGS = 168;     // 384 threads, one CTA per SM
constexpr int PRODUCER_REGS = 40;
constexpr int EPILOGUE_REGS = 232;
static_assert(128 * PRODUCER_REGS + 256 * EPILOGUE_REGS <= 384 * LAUNCH_REGS, "register split exceeds launch");

struct GmmArgs {
  const int32_t* offsets;   // [ngroups + 1]
  int ngroups, nweights;    // groups of the offsets; groups that have weights
  int rows;                 // rows of the row operands
  int nr, nc;               // wgrad: output rows (n) per group; all: output columns
  int ntc;                  // column tiles
  int nk;                   // forward, dgrad: K blocks of a tile
  void* out;
  long long ld;             // output row stride, elements
  int out_type;             // moe_dtype
  int segment;              // PROMOTE: K blocks of one accumulator
  int accumulate;           // wgrad: add to what `out` holds
  int bulk;                 // the output takes bulk tensor stores (aligned base and stride),
  int bulk_edge;            // also of boxes that reach past its last column: they write whole
                            // 16-byte pieces, so its rows have to end with one
  uint32_t idesc;           // instruction descriptor without N
  uint32_t* status;
  unsigned long long wait_ns;
  int withhold;             // test only: the first CTA's producer skips its first stage
};

// Tensor maps of the row operand K-major: boxes of 128, 64, 32 and 16 rows,
// so that a tile of few rows moves few bytes.
struct RowMaps {
  CUtensorMap m[4];
};
// wgrad: dy by boxes of 64 rows, and the boxes of a tail (32, 8, 2 and 1 rows)
// of x and dy.
struct WgradMaps {
  CUtensorMap m;
  CUtensorMap a[4], b[4];
};
constexpr int tail_rows(int i) { return i == 0 ? 32 : i == 1 ? 8 : i == 2 ? 2 : 1; }
template <int MODE>
using BMaps = typename std::conditional<MODE == MOE_MM_WGRAD, WgradMaps, RowMaps>::type;

struct Tile {
  int g, col0, row0, nrows, r_first, terms, nk;
  // row0: first output row (global for forward/dgrad, within the group's
  // weight for wgrad); nrows: valid rows; wgrad: the group's first row and its
  // rows; nk: K blocks
};

// The tile list. Forward and dgrad keep the groups' order: a group's weights
// and rows are in use by all pairs at one time and come from HBM once. (Full
// tiles first and the groups' partial ones behind them, largest first, would
// end the busiest pair 1.5% behind the mean instead of 10%, and still took
// 417 us instead of 396 on the training batch: the tensor cores run at the
// power limit, where a second reading of the weights costs more than idle
// pairs.) wgrad takes the groups by falling rows, so that the tiles of one
// round cost the same (FFN 1500 case 408 -> 394 us).
struct TileList {
  GroupPlan plan;                 // prefix: of the tiles (not for wgrad)
  int key[kMaxGroups];            // wgrad: rows of the groups
  uint16_t order[kMaxGroups];     // and the groups by falling rows
  int total;
};

template <int MODE, int BR, int THREADS>
__device__ __forceinline__ void build_tiles(TileList& s, const GmmArgs& p) {
  int n = build_plan<THREADS>(s.plan, p.offsets, p.ngroups, p.nweights, p.rows, p.status, [&](int n_g) -> int {
    return MODE == MOE_MM_WGRAD ? 0 : (n_g + BR - 1) / BR * p.ntc;
  });
  if (MODE == MOE_MM_WGRAD && n >= 0) {
    n = p.nweights * ((p.nr + BR - 1) / BR) * p.ntc;   // groups without rows too
    for (int g = threadIdx.x; g < p.nweights; g += THREADS) s.key[g] = s.plan.off[g + 1] - s.plan.off[g];
    __syncthreads();
    for (int g = threadIdx.x; g < p.nweights; g += THREADS) {
      const int key = s.key[g];
      int rank = 0;
      for (int j = 0; j < p.nweights; ++j) rank += s.key[j] > key || (s.key[j] == key && j < g);
      s.order[rank] = uint16_t(g);
    }
  }
  if (threadIdx.x == 0) s.total = n < 0 ? 0 : n;
}

// The tile that pair `pair` of `npairs` takes in round w (the direction
// alternates, so that the first pairs do not get the larger of every round).
__device__ __forceinline__ int tile_at(int w, int pair, int npairs) {
  return w * npairs + ((w & 1) ? npairs - 1 - pair : pair);
}

template <int MODE, int BR>
__device__ __forceinline__ Tile decode_tile(int i, const TileList& s, const GmmArgs& p) {
  Tile t;
  if (MODE == MOE_MM_WGRAD) {
    const int ct = i / p.ntc;                       // (group, row tile)
    const int rts = (p.nr + BR - 1) / BR;
    t.g = s.order[ct / rts];
    t.col0 = (i - ct * p.ntc) * BC;
    t.row0 = (ct % rts) * BR;
    t.nrows = min(BR, p.nr - t.row0);
    t.r_first = s.plan.off[t.g];
    t.terms = s.plan.off[t.g + 1] - t.r_first;
    t.nk = (t.terms + BK - 1) / BK;
    return t;
  }
  t.r_first = t.terms = 0;
  t.nk = p.nk;
  // chunks of up to 8 row tiles, then the column tiles, then the row tiles:
  // the row tiles that share a weight tile run side by side
  t.g = find_group(s.plan.prefix, p.ngroups, i);
  const int local = i - s.plan.prefix[t.g];
  const int g0 = s.plan.off[t.g], n_g = s.plan.off[t.g + 1] - g0;
  const int rts = (n_g + BR - 1) / BR;
  const int per_chunk = RCHUNK * p.ntc;
  const int chunk = local / per_chunk;
  const int within = local - chunk * per_chunk;
  const int rc = min(RCHUNK, rts - chunk * RCHUNK);
  const int ct = within / rc;
  const int rt = chunk * RCHUNK + (within - ct * rc);
  t.col0 = ct * BC;
  t.row0 = g0 + rt * BR;
  t.nrows = min(BR, n_g - rt * BR);
  return t;
}

// MMA columns of a tile: its rows rounded up to 32 (each CTA holds half).
__device__ __forceinline__ int tile_n(const Tile& t) { return (t.nrows + 31) & ~31; }

// Stores a lane's 32 (or the first m) output rows of one column, from `at`
// on; one rounding, to nearest even, of the fp32 sum.
template <typename T>
__device__ __forceinline__ float load_as_f32(const T* o);
template <>
__device__ __forceinline__ float load_as_f32<float>(const float* o) { return *o; }
template <>
__device__ __forceinline__ float load_as_f32<__nv_bfloat16>(const __nv_bfloat16* o) { return __bfloat162float(*o); }
template <>
__device__ __forceinline__ float load_as_f32<__half>(const __half* o) { return __half2float(*o); }
__device__ __forceinline__ void store_f32(float* o, float v) { *o = v; }
__device__ __forceinline__ void store_f32(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_f32(__half* o, float v) { *o = __float2half_rn(v); }

template <typename T>
__device__ __forceinline__ void store_rows(T* o, long long ld, const float (&v)[32], int m, int accumulate) {
  if (accumulate) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < m) store_f32(o + j * ld, load_as_f32(o + j * ld) + v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < m) store_f32(o + j * ld, v[j]);
  }
}

__device__ __forceinline__ void store_chunk(const GmmArgs& p, size_t at, const float (&v)[32], int m) {
  if (p.out_type == MOE_F32)
    store_rows(static_cast<float*>(p.out) + at, p.ld, v, m, p.accumulate);
  else if (p.out_type == MOE_BF16)
    store_rows(static_cast<__nv_bfloat16*>(p.out) + at, p.ld, v, m, p.accumulate);
  else
    store_rows(static_cast<__half*>(p.out) + at, p.ld, v, m, p.accumulate);
}

// Barrier of the four warps of epilogue warpgroup wg, and whether `ok` holds
// in every thread of them (a barrier too).
__device__ __forceinline__ void epilogue_sync(int wg) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
}
__device__ __forceinline__ bool epilogue_all(int wg, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(ok)), "r"(1 + wg)
      : "memory");
  return r != 0;
}

template <int MODE, int BR, bool PROMOTE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads(BR, PROMOTE), 1)
    grouped_mm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ BMaps<MODE> tmB,
                      const __grid_constant__ CUtensorMap tmO, const GmmArgs p) {
  constexpr bool A_MN = MODE != MOE_MM_FORWARD;   // A's contraction is its slow dimension
  constexpr bool B_MN = MODE == MOE_MM_WGRAD;
  constexpr int STAGES = stages(BR, PROMOTE), STAGE_BYTES = stage_bytes(BR);
  constexpr int THREADS = threads(BR, PROMOTE), EPI_WARPS = epi_warps(BR, PROMOTE);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[STAGES];    // leading CTA: both CTAs' parts of a stage
  __shared__ __align__(8) uint64_t empty_bar[STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tread_bar[2];        // this CTA's epilogue has read the accumulator
  __shared__ __align__(8) uint64_t tempty_bar[2];       // leading CTA: the other one's has
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ TileList s_tiles;
  __shared__ uint32_t tmem_base_s;
  __shared__ int s_abort_store;
  __shared__ uint32_t s_issued, s_withheld, s_drain;
  volatile int* s_abort = &s_abort_store;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 2);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tread_bar[b], EPI_WARPS);
      mbar_init(&tempty_bar[b], 1);
    }
    mbar_init(&done_bar, 1);
    s_abort_store = 0;
    s_issued = 0;
    s_drain = 0;
    s_withheld = 0xFFFFFFFFu;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    if constexpr (B_MN)
      tma_prefetch_desc(&tmB.m);
    else
      for (int j = 0; j < 4; ++j) tma_prefetch_desc(&tmB.m[j]);
  }
  if (warp == 1) tmem_alloc_pair(&tmem_base_s, TMEM_COLS);
  // the set-up above overlaps the previous kernel; offsets, operands and
  // outputs are touched only below
  pdl_wait();
  pdl_launch_dependents();

  build_tiles<MODE, BR, THREADS>(s_tiles, p);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the peer's barriers are initialised and its TMEM is allocated
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_s;
  const int total = s_tiles.total;

  if (warp < FIRST_EPI_WARP) {
  if (PROMOTE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PRODUCER_REGS));
  if (warp == 0) {
    // -------------------------------------------------------------- producer
    if (elect_one()) {
      const uint32_t full = map_rank(full_bar, 0);
      uint32_t it = 0;
      bool ok = true;
      for (int w = 0, i; ok && (i = tile_at(w, pair, npairs)) < total; ++w) {
        const Tile t = decode_tile<MODE, BR>(i, s_tiles, p);
        const int half = tile_n(t) >> 1;
        const int acol = t.col0 + int(rank) * 128;
        const int brow = t.row0 + int(rank) * half;
        const int boxes = 2 + (half > 64 ? 2 : 1);   // wgrad: of 64 columns, A's and B's
        for (int kb = 0; kb < t.nk; ++kb) {
          const int s = it % STAGES;
          if (!mbar_wait_stage<true>(&empty_bar[s], ((it / STAGES) & 1u) ^ 1u, s_abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          if (p.withhold && blockIdx.x == 0 && it == 0) {   // test only: this stage never arrives
            s_withheld = it++;
            continue;
          }
          uint8_t* a = smem + s * STAGE_BYTES;
          const uint32_t fb = full + s * 8;
          if constexpr (MODE == MOE_MM_WGRAD) {
            const int k0 = t.r_first + kb * BK;
            const int valid = min(BK, t.terms - kb * BK), taken = (valid + 15) & ~15;
            mbar_expect_pair(fb, uint32_t(boxes * taken) * 128u);
            if (valid == BK) {
              tma_load_2d_pair(a, &tmA, fb, acol, k0);
              tma_load_2d_pair(a + BOX_BYTES, &tmA, fb, acol + 64, k0);
              tma_load_2d_pair(a + A_BYTES, &tmB.m, fb, brow, k0);
              if (half > 64) tma_load_2d_pair(a + A_BYTES + BOX_BYTES, &tmB.m, fb, brow + 64, k0);
            } else {
              // A tail. The copies' swizzle goes by the shared-memory address,
              // so a box may start at any row of a 1024-byte atom. Each issue
              // names its map (from a map chosen at run time a copy took 170
              // cycles to issue: 1,151 rows per group 619 us against 454).
              int r = 0;
              auto rows_by = [&](const CUtensorMap* ma, const CUtensorMap* mb, int h, int end, int y) {
                for (; end - r >= h; r += h, y += h) {
                  uint8_t* dst = a + r * 128;
                  tma_load_2d_pair(dst, ma, fb, acol, y);
                  tma_load_2d_pair(dst + BOX_BYTES, ma, fb, acol + 64, y);
                  tma_load_2d_pair(dst + A_BYTES, mb, fb, brow, y);
                  if (half > 64) tma_load_2d_pair(dst + A_BYTES + BOX_BYTES, mb, fb, brow + 64, y);
                }
              };
#pragma unroll
              for (int j = 0; j < 4; ++j) rows_by(&tmB.a[j], &tmB.b[j], tail_rows(j), valid, k0 + r);
#pragma unroll
              for (int j = 1; j < 4; ++j) rows_by(&tmB.a[j], &tmB.b[j], tail_rows(j), taken, p.rows);
            }
          } else {
            uint8_t* b = a + A_BYTES;
            const int k0 = kb * BK;
            mbar_expect_pair(fb, A_BYTES + half * BK * 2);
            if (MODE == MOE_MM_FORWARD) {
              tma_load_3d_pair(a, &tmA, fb, k0, acol, t.g);
            } else {
              tma_load_3d_pair(a, &tmA, fb, acol, k0, t.g);
              tma_load_3d_pair(a + BOX_BYTES, &tmA, fb, acol + 64, k0, t.g);
            }
            int r = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // 128, 64, 32, 16 rows: half is a multiple of 16, 128 at most
              const int h = 128 >> j;
              if (half & h) {
                tma_load_2d_pair(b + r * (BK * 2), &tmB.m[j], fb, k0, brow + r);
                r += h;
              }
            }
          }
          ++it;
        }
      }
      s_issued = it;
      // the MMAs' arrivals on this CTA's barriers, which come from the leading
      // CTA, are all in before it may end
      for (uint32_t j = it > STAGES ? it - STAGES : 0; ok && j < it; ++j)
        ok = mbar_wait_stage<true>(&empty_bar[j % STAGES], (j / STAGES) & 1u, s_abort, p.status, p.wait_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0 && elect_one()) {
      uint32_t it = 0, tb = 0;
      bool ok = true;
      for (int w = 0, i; ok && (i = tile_at(w, pair, npairs)) < total; ++w) {
        const Tile t = decode_tile<MODE, BR>(i, s_tiles, p);
        if (t.nk == 0) continue;
        int part = 0;   // K blocks in the accumulator
        const uint32_t idesc = p.idesc | (uint32_t(tile_n(t) >> 3) << 17);
        for (int kb = 0; kb < t.nk; ++kb) {
          const uint32_t buf = tb & 1u;
          if (part == 0 &&
              !(mbar_wait_stage(&tread_bar[buf], ((tb >> 1) & 1u) ^ 1u, s_abort, p.status, p.wait_ns) &&
                mbar_wait_stage<true>(&tempty_bar[buf], ((tb >> 1) & 1u) ^ 1u, s_abort, p.status, p.wait_ns))) {
            ok = false;
            break;
          }
          const uint32_t d = tmem_base + buf * TMEM_BUF;
          const int s = it % STAGES;
          if (!mbar_wait_stage<true>(&full_bar[s], (it / STAGES) & 1u, s_abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + s * STAGE_BYTES);
          const uint64_t ad = A_MN ? smem_desc_mn_sw128(a_addr, BOX_BYTES) : smem_desc_sw128(a_addr);
          const uint64_t bd = B_MN ? smem_desc_mn_sw128(a_addr + A_BYTES, BOX_BYTES) : smem_desc_sw128(a_addr + A_BYTES);
          const int left = MODE == MOE_MM_WGRAD ? t.terms - kb * BK : BK;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            // 16 of the contraction: 32 bytes along a K-major row, two 8-row
            // atoms (2048 bytes) of an MN-major box (address field in 16 bytes)
            if (MODE != MOE_MM_WGRAD || k * 16 < left)
              mma_f16_pair(d, ad + uint64_t(k * (A_MN ? 128 : 2)), bd + uint64_t(k * (B_MN ? 128 : 2)), idesc,
                           (part | k) ? 1u : 0u);
          tc_commit_pair(&empty_bar[s]);
          ++it;
          ++part;
          if (kb == t.nk - 1 || (PROMOTE && part == p.segment)) {
            tc_commit_pair(&tfull_bar[buf]);
            ++tb;
            part = 0;
          }
        }
      }
      tc_commit_pair_self(&done_bar);   // all MMAs issued above have completed
      int never = 0;
      mbar_wait_stage(&done_bar, 0, &never, p.status, p.wait_ns);
    }
  } else if (warp == 2 && rank == 1) {
    // ----------------------------------------------- accumulators handed back
    if (elect_one()) {
      const uint32_t tempty = map_rank(tempty_bar, 0);
      uint32_t tb = 0;
      bool ok = true;
      for (int w = 0, i; ok && (i = tile_at(w, pair, npairs)) < total; ++w) {
        const int nk = decode_tile<MODE, BR>(i, s_tiles, p).nk;
        for (int kb = 0; ok && kb < nk; kb += PROMOTE ? p.segment : nk) {
          ok = mbar_wait_stage(&tread_bar[tb & 1u], (tb >> 1) & 1u, s_abort, p.status, p.wait_ns);
          if (ok) mbar_arrive_pair(tempty + (tb & 1u) * 8);
          ++tb;
        }
      }
    }
  }
  // ------------------------------------------------ teardown (warps 0 to 3)
  __syncwarp();
  asm volatile("bar.sync 0;" ::: "memory");
  if (warp == 0 && lane == 0 && *s_abort) {
    store_rank(&s_drain, 0, 1);
    store_rank(&s_drain, 1, 1);
  }
  __syncwarp();
  tc_fence_before();
  asm volatile("bar.sync 0;" ::: "memory");
  cluster_sync();   // both CTAs are past their last arrival, copy issue and MMA
  if (warp == 0 && lane == 0 && s_drain) {
    // After an abort, copies issued but not waited for must land before the
    // CTAs end. A stage that only one CTA issued gets the other's arrival
    // here, so that its barrier completes with the copies that there are.
    const uint32_t own = s_issued, other = load_rank(&s_issued, rank ^ 1u), last = max(own, other);
    int never = 0;
    for (uint32_t j = last > STAGES ? last - STAGES : 0; j < last; ++j) {
      const uint32_t s = j % STAGES;
      if (j >= own || j == s_withheld) mbar_arrive_pair(map_rank(&full_bar[s], 0));
      if (rank == 0) mbar_wait_stage<true>(&full_bar[s], (j / STAGES) & 1u, &never, p.status, p.wait_ns);
    }
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
  __syncwarp();
  cluster_sync();
  } else {
    // -------------------------------------------------------------- epilogue
    // (its own copy of the teardown, so that both register limits hold on
    // every instruction that they meet)
    if (PROMOTE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPILOGUE_REGS));
    const int q = warp & 3;                           // TMEM lane quarter this warp may access
    const int wg = (warp - FIRST_EPI_WARP) >> 2;      // rows [128 wg, 128 wg + 128) of a tile
    constexpr int STG_BUFS = EPI_WARPS == 8 ? 1 : 2;  // staging buffers of a warpgroup
    uint8_t* staging = smem + STAGES * STAGE_BYTES + wg * STG_BYTES;
    uint32_t tb = 0, sb = 0;
    for (int w = 0, i; (i = tile_at(w, pair, npairs)) < total; ++w) {
      const Tile t = decode_tile<MODE, BR>(i, s_tiles, p);
      const int x = t.col0 + int(rank) * 128;
      const int col = x + q * 32 + lane;
      const bool cv = col < p.nc;
      size_t at = size_t(t.row0) * size_t(p.ld) + size_t(col);
      if (MODE == MOE_MM_WGRAD) at += size_t(t.g) * size_t(p.nr) * size_t(p.ld);
      // rows [c, c + 32) of the tile
      auto put = [&](int c, const float (&v)[32]) {
        const int m = min(32, t.nrows - c);
        // Bulk stores for whole chunks; a ragged group's last rows are stored
        // one by one, so that no row behind them is touched (a weight's last
        // rows are cut off by the tensor map).
        if (p.bulk && (MODE == MOE_MM_WGRAD || m == 32) && (p.bulk_edge || x + 128 <= p.nc)) {
          const int parts = p.out_type == MOE_F32 ? 2 : 1;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == parts) break;
            // the last store from the buffer that is written now has read it
            // (elect_one: always the same thread issues and waits)
            if (q == 0 && elect_one()) {
              if (STG_BUFS == 1)
                bulk_wait_read0();
              else
                bulk_wait_read1();
            }
            epilogue_sync(wg);
            uint8_t* stg = staging + (sb % STG_BUFS) * STG_BYTES;
            if (p.out_type == MOE_F32) {
              float* o = reinterpret_cast<float*>(stg) + q * 32 + lane;
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j * 128] = v[16 * h + j];
            } else if (p.out_type == MOE_BF16) {
              __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(stg) + q * 32 + lane;
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j * 128] = __float2bfloat16_rn(v[j]);
            } else {
              __half* o = reinterpret_cast<__half*>(stg) + q * 32 + lane;
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j * 128] = __float2half_rn(v[j]);
            }
            fence_proxy_async_smem();
            epilogue_sync(wg);
            if (q == 0 && elect_one()) {
              const int y = t.row0 + c + 16 * h;
              if (MODE == MOE_MM_WGRAD) {
                if (x < p.nc && y < p.nr) {
                  if (p.accumulate)
                    tma_add_3d(&tmO, stg, x, y, t.g);
                  else
                    tma_store_3d(&tmO, stg, x, y, t.g);
                }
              } else if (x < p.nc) {
                tma_store_2d(&tmO, stg, x, y);
              }
              bulk_commit();
            }
            ++sb;
          }
        } else if (cv) {
          store_chunk(p, at + size_t(c) * size_t(p.ld), v, m);
        }
      };
      const int c0 = wg * 128, c1 = min(t.nrows, c0 + 128);   // this warpgroup's rows
      if (t.nk == 0) {   // wgrad of a group without rows
        if (!p.accumulate) {
          float z[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = 0.0f;
          for (int c = c0; c < c1; c += 32) put(c, z);
        }
        continue;
      }
      // the accumulator of the tile's next part, or false: give up (all warps
      // of the warpgroup together, since they share barriers)
      auto accumulator = [&](uint32_t& tbase) {
        const uint32_t buf = tb & 1u;
        // one warp polls, the others sleep in the barrier
        const bool got =
            q != 0 || mbar_wait_stage<true>(&tfull_bar[buf], (tb >> 1) & 1u, s_abort, p.status, p.wait_ns);
        if (!epilogue_all(wg, got)) return false;
        tc_fence_after();
        tbase = tmem_base + (uint32_t(q * 32) << 16) + buf * TMEM_BUF;
        return true;
      };
      auto release = [&]() {   // its values are in registers: hand it back
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tread_bar[tb & 1u]);
        ++tb;
      };
      uint32_t tbase;
      if constexpr (!PROMOTE) {
        if (!accumulator(tbase)) break;
        if (c0 >= c1) release();
        for (int c = c0; c < c1; c += 32) {
          float v[32];
          tmem_ld32(tbase + uint32_t(c), v);
          tmem_ld_wait();
          if (c + 32 >= c1) release();
          put(c, v);
        }
      } else {
        float acc[4][32];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[cc][j] = -0.0f;   // the first part as it is, -0 too
        bool ok = true;
        for (int kb = 0; kb < t.nk; kb += p.segment) {
          if (!accumulator(tbase)) { ok = false; break; }
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            if (c0 + cc * 32 < c1) {
              float v[32];
              tmem_ld32(tbase + uint32_t(c0 + cc * 32), v);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) acc[cc][j] += v[j];
            }
          }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
          if (c0 + cc * 32 < c1) put(c0 + cc * 32, acc[cc]);
      }
    }
    if (q == 0 && elect_one()) bulk_wait0();   // stores complete before the CTA exits
    // ------------------------------------------------ teardown (epilogue side)
    __syncwarp();
    asm volatile("bar.sync 0;" ::: "memory");
    tc_fence_before();
    asm volatile("bar.sync 0;" ::: "memory");
    cluster_sync();
    cluster_sync();
  }
}

template <int MODE, int BR, bool PROMOTE>
cudaError_t launch_variant(const moe_layer_s* L, const CUtensorMap& tmA, const BMaps<MODE>& tmB, GmmArgs a, long long tiles,
                        cudaStream_t st) {
  // bulk stores want the base and the row stride in 16-byte units; 16-bit
  // accumulation rounds once, which a bulk add to the 16-bit values would not
  const int es = a.out_type == MOE_F32 ? 4 : 2;
  CUtensorMap tmO = tmA;
  a.bulk = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.ld * es % 16 == 0 && !(a.accumulate && es == 2);
  a.bulk_edge = a.nc * es % 16 == 0;
  if (a.bulk && !encode_tmap_out(&tmO, static_cast<moe_dtype>(a.out_type), a.out, a.nc,
                                 MODE == MOE_MM_WGRAD ? a.nr : a.rows, MODE == MOE_MM_WGRAD ? a.nweights : 0, a.ld,
                                 128, STG_BYTES / 128 / es))
    return cudaErrorInvalidValue;
  static std::atomic<bool> configured[kMaxDevices];   // the attribute is per device
  cudaError_t ce = once_per_device(configured, []() {
    // setmaxnreg.inc waits for registers that come only from this CTA's
    // launch allocation: refuse a build whose count cannot fund the split
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, grouped_mm_kernel<MODE, BR, PROMOTE>);
    if (e != cudaSuccess) return e;
    if (PROMOTE && fa.numRegs * threads(BR, PROMOTE) < 128 * PRODUCER_REGS + 256 * EPILOGUE_REGS)
      return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(grouped_mm_kernel<MODE, BR, PROMOTE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem_dyn(BR, PROMOTE));
  });
  if (ce != cudaSuccess) return ce;
  a.wait_ns = kWaitLimitNs;
  if (L->test_stall_ns) {   // a test armed a stall for this one launch
    a.wait_ns = L->test_stall_ns;
    a.withhold = 1;
    L->test_stall_ns = 0;
  }
  const long long pairs = tiles < L->num_sms / 2 ? tiles : L->num_sms / 2;
  if (pairs <= 0) return cudaSuccess;
  return launch_pdl(grouped_mm_kernel<MODE, BR, PROMOTE>, dim3(unsigned(2 * pairs)), dim3(threads(BR, PROMOTE)),
                    smem_dyn(BR, PROMOTE), st, tmA, tmB, tmO, a);
}

// `terms`: the longest contraction that the launch may hold.
template <int MODE, int BR>
cudaError_t launch_mode(const moe_layer_s* L, const CUtensorMap& tmA, const BMaps<MODE>& tmB, const GmmArgs& a, int terms,
                        long long tiles, cudaStream_t st) {
  if (terms > a.segment * BK)
    return launch_variant<MODE, BR, true>(L, tmA, tmB, a, tiles, st);
  return launch_variant<MODE, BR, false>(L, tmA, tmB, a, tiles, st);
}

// A row operand [rows][cols] whose rows are the tile's N (K-major boxes).
bool encode_row_maps(RowMaps* m, moe_dtype t, const void* base, int cols, int rows, long long ld) {
  for (int j = 0; j < 4; ++j)
    if (!encode_tmap_16(&m->m[j], t, base, cols, rows, 0, ld, 64, 128u >> j)) return false;
  return true;
}

}  // namespace

cudaError_t launch_grouped_mm(const moe_layer_s* L, int mode, moe_dtype t, const void* a, long long lda, const void* b,
                              long long ldb, const int32_t* offsets, int rows, int n, int k, moe_dtype out_t, void* out,
                              long long ldo, int accumulate, cudaStream_t st) {
  const int G = L->E + L->S;
  GmmArgs p = {};
  p.offsets = offsets;
  p.ngroups = L->E + 1;
  p.nweights = G;
  p.rows = rows;
  p.out = out;
  p.ld = ldo;
  p.out_type = out_t;
  p.segment = segment(out_t);
  p.accumulate = accumulate;
  p.status = L->status;
  p.idesc = idesc_16(t, 256, mode != MOE_MM_FORWARD, mode == MOE_MM_WGRAD);
  CUtensorMap tmA;
  if (mode == MOE_MM_WGRAD) {
    // a = dy [rows][n], b = x [rows][k]; output rows n, columns k
    p.nr = n;
    p.nc = k;
    p.ntc = (k + BC - 1) / BC;
    WgradMaps tmB;
    if (!encode_tmap_16(&tmA, t, b, k, rows, 0, ldb, 64, 64) || !encode_tmap_16(&tmB.m, t, a, n, rows, 0, lda, 64, 64))
      return cudaErrorInvalidValue;
    for (int j = 0; j < 4; ++j)
      if (!encode_tmap_16(&tmB.a[j], t, b, k, rows, 0, ldb, 64, tail_rows(j)) ||
          !encode_tmap_16(&tmB.b[j], t, a, n, rows, 0, lda, 64, tail_rows(j)))
        return cudaErrorInvalidValue;
    return launch_mode<MOE_MM_WGRAD, 256>(L, tmA, tmB, p, rows,
                                           static_cast<long long>(G) * ((n + 255) / 256) * p.ntc, st);
  }
  // a = the rows, b = w [G][n][k]
  RowMaps tmB;
  const int contraction = mode == MOE_MM_FORWARD ? k : n;
  p.nc = mode == MOE_MM_FORWARD ? n : k;
  p.ntc = (p.nc + BC - 1) / BC;
  p.nk = (contraction + BK - 1) / BK;
  if (!encode_tmap_16(&tmA, t, b, k, n, G, ldb, 64, mode == MOE_MM_FORWARD ? 128 : 64) ||
      !encode_row_maps(&tmB, t, a, contraction, rows, lda))
    return cudaErrorInvalidValue;
  // Few rows per group on average: narrow tiles (larger groups take several).
  // 64 groups of 1536 x 5120 with 8, 32, 64 and 128 rows in each take 175,
  // 179, 185 and 235 us by tiles of 64 rows and 184, 187, 189 and 201 by tiles
  // of 256; by a Zipf law over the groups 172, 188, 227 and 293 against 182,
  // 182, 185 and 215.
  const int br = rows <= 32ll * G ? 64 : 256;
  // upper bound on the tiles: every group may add one partial row tile
  const long long tiles = (static_cast<long long>(rows) / br + (rows < G ? rows : G)) * p.ntc;
  if (mode == MOE_MM_FORWARD)
    return br == 64 ? launch_mode<MOE_MM_FORWARD, 64>(L, tmA, tmB, p, contraction, tiles, st)
                    : launch_mode<MOE_MM_FORWARD, 256>(L, tmA, tmB, p, contraction, tiles, st);
  return br == 64 ? launch_mode<MOE_MM_DGRAD, 64>(L, tmA, tmB, p, contraction, tiles, st)
                  : launch_mode<MOE_MM_DGRAD, 256>(L, tmA, tmB, p, contraction, tiles, st);
}

}  // namespace moe
