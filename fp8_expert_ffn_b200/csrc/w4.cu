// Products with 4-bit expert weights for few rows per expert (decode):
//   y[r, j] = sum_groups s[g, j, c] * sum_{i in c} x[perm[r], i] (q[g, j, i] - z[g, j, c])
// and the gate/up form h = silu(gate) * up. A weight is read once for up to 8
// (or 16, see launch_w4) rows, half a byte each, so HBM would bound the kernel
// if unpacking kept up: 6.5 TB/s is 46 codes per SM and cycle, or 45 issue
// slots per scheduler for 512 codes, and the kernel takes 38 instructions for
// them. It runs at 4.0 TB/s (a decode batch of 64 tokens over 257 experts,
// 1.84 GB: 450 to 460 us back to back, 433 one at a time, where the same copies
// without the arithmetic took 311): three warps per scheduler issue 0.55
// instructions per cycle.
//
// Unpacking is exact and short (the mantissa trick of Kim, Henry, Fahim and
// Awadalla, "Who Says Elephants Can't Run", 2022): code nibbles i and i + 4 of
// a 32-bit word are masked out together and OR-ed into the mantissas of the
// 16-bit pair (128, 128) in bf16 or (1024, 1024) in fp16; subtracting (128 + z)
// or (1024 + z) leaves q - z exactly. The pairs go to mma.sync m16n8k16 (weights
// as A, up to 8 rows of x as one B) with fp32 sums per scale group; the scale
// multiplies that sum in fp32, so nothing is rounded between the codes and the
// output. The order of the contraction inside a word (0,4,1,5,...) is the
// same for x, whose 8 consecutive values are shuffled with four byte
// permutes. tcgen05 would need the unpacked weights back in shared or tensor
// memory, a second trip per code that the memory-bound case has no use for.
//
// Layout: 4 warps per CTA, 3 CTAs per SM (2 for units of 16 rows), persistent
// over (group, column tile, rows chunk). A warp owns 64 weight rows (32 gate
// and 32 up) and every wk-th stage of the contraction, and streams its codes
// through its own ring of two TMA boxes (64 rows x 128 bytes = 256 codes,
// 128-byte swizzle: lane (g, t) reads word t of a chunk of row g without bank
// conflicts), so no warp waits for another until a unit's partial sums meet in
// shared memory, added in warp order. The warps of a CTA split the contraction
// 4, 2 or 1 ways and the columns by the rest (see launch_w4). Measured and
// dropped: 16 warps per SM with 128-code stages (465 against 418 us) and 128
// rows per warp (500 against 439), both for their 64-byte boxes; 24 warps of
// 80 registers (no gain at 64 tokens, 102 against 86 us for the down
// projection).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "groups.cuh"
#include "internal.h"
#include "pair.cuh"
#include "silu.cuh"

namespace moe {

namespace {

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
// For units of 8 nt rows. Held to the registers of 3 CTAs, the kernels for 16
// rows spill 250 to 810 bytes (32 rows in each of 64 groups, gate/up of
// 1536 x 5120: 585 us against 407).
constexpr int ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }
constexpr int KB = 256;                    // codes per row of a stage
constexpr int KH = KB / 2;                 // and of the half that is worked on at a time
constexpr int STAGES = 2;
constexpr int BOX_ROWS = 64;
constexpr int STAGE_BYTES = BOX_ROWS * KB / 2;   // 8 KB
constexpr int RING_BYTES = WARPS * STAGES * STAGE_BYTES;
constexpr int RED_ROWS = BOX_ROWS / 2;                // weight rows joined at a time
constexpr int RED_BYTES = WARPS * RED_ROWS * 8 * 4;   // their partial sums for 8 rows of x
constexpr int SMEM_DYN = RING_BYTES + RED_BYTES + 1024;

struct W4Args {
  const int32_t* offsets;
  int ngroups, nweights, rows;
  const void* x;
  long long ldx;
  int x_rows;
  const int32_t* perm;
  const void* scales[2];      // gate (or the only weight), up
  const uint8_t* zeros[2];
  int scale_type;
  int vec;                    // a row's scales of a stage are one aligned vector of 16-bit values
  int n, k, ng;               // ng: scale groups of a weight row
  int dual;                   // gate/up form
  int wk;                     // warps along the contraction
  int ntn, nkb;
  void* y;
  long long ldy;
  int y_type;
  uint32_t* status;
  unsigned long long wait_ns;
  int withhold;
  uint32_t mask;              // 0x000F000F (see unpack_pair)
};

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Nibbles i and i + 4 of w, less the zero point, as a 16-bit pair;
// bias = (128 + z, twice) in bf16 or (1024 + z, twice) in fp16. mask is
// 0x000F000F in a register: lop3 takes one immediate, and as a second one the
// mask costs an instruction of its own in every pair.
template <bool BF16>
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w, int i, uint32_t bias, uint32_t mask) {
  uint32_t v, d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * i)), "r"(mask), "n"(BF16 ? 0x43004300 : 0x64006400));
  if (BF16)
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(bias));
  else
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(bias));
  return d;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Read-only loads that stay where they are written (ahead of the wait that
// their latency hides under), which the compiler would not leave __ldg to do.
__device__ __forceinline__ uint4 ldg128(const void* a) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(a));
  return v;
}
__device__ __forceinline__ void ldg128_if(uint4& v, const void* a, bool there) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@p ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
      : "l"(a), "r"(int(there)));
}
__device__ __forceinline__ uint2 ldg64(const void* a) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(a));
  return v;
}
__device__ __forceinline__ uint32_t ldg32(const void* a) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(a));
  return v;
}
__device__ __forceinline__ uint32_t ldg16(const void* a) {
  uint32_t v;
  asm volatile("{\n\t.reg .u16 h;\n\tld.global.nc.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "l"(a));
  return v;
}
__device__ __forceinline__ uint32_t ldg8(const void* a) {
  uint32_t v;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(a));
  return v;
}

struct Unit {
  int g, nt, r0, nr;   // group, column tile, first row, rows (at most 8 NT)
};

template <int RMAX>
__device__ __forceinline__ Unit decode_unit(int i, const GroupPlan& s, const W4Args& p) {
  Unit u;
  u.g = find_group(s.prefix, p.ngroups, i);
  const int local = i - s.prefix[u.g];
  const int n_g = s.off[u.g + 1] - s.off[u.g];
  const int chunks = (n_g + RMAX - 1) / RMAX;
  u.nt = chunks == 1 ? local : local / chunks;   // the chunks that share codes run side by side
  const int c = local - u.nt * chunks;
  u.r0 = s.off[u.g] + c * RMAX;
  u.nr = min(RMAX, n_g - c * RMAX);
  return u;
}

// 8 values of a row of x from column i on; columns past k, and rows that are
// not there, are zero.
template <typename T>
__device__ __forceinline__ uint4 load_x8_edge(const T* row, int i, int k) {
  if (row == nullptr || i >= k) return make_uint4(0u, 0u, 0u, 0u);
  if (i + 8 <= k) return __ldg(reinterpret_cast<const uint4*>(row + i));
  uint32_t v[4] = {0u, 0u, 0u, 0u};
  const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < k) v[j >> 1] |= uint32_t(r[i + j]) << (16 * (j & 1));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void store_y(const W4Args& p, size_t at, float v) {
  if (p.y_type == MOE_F32)
    static_cast<float*>(p.y)[at] = v;
  else if (p.y_type == MOE_BF16)
    static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p.y)[at] = __float2half_rn(v);
}

// A lane's part of a stage's scales and zero points (rows 16 t + g and
// 16 t + 8 + g of the warp's 64, t = lane % 4; the lanes of a quad exchange
// them by shuffles). They are kept as loaded until their use: converting them
// at the load would wait for it. 16-bit scales are packed in pairs.
template <int GPS>
struct Scales {
  uint32_t raw[2][GPS];
  uint32_t zero[2][GPS / 2 < 1 ? 1 : GPS / 2];   // byte pairs
};

// Where every row's scales of a stage are one aligned vector (p.vec), they
// come in one load: 64 rows are as many cache lines, and a load per scale
// spends its time there (T = 64 gate/up: 39 of 455 us).
template <bool ZEROS, int GPS>
__device__ __forceinline__ void load_scales(const W4Args& p, const void* sp, const uint8_t* zp, const int (&srow)[2],
                                            int kb, Scales<GPS>& o) {
  const int g0 = kb * GPS;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (p.vec) {
      const uint16_t* a = static_cast<const uint16_t*>(sp) + (srow[h] + g0);
      if (GPS == 2) {
        o.raw[h][0] = ldg32(a);
      } else if (GPS == 4) {
        const uint2 v = ldg64(a);
        o.raw[h][0] = v.x;
        o.raw[h][1] = v.y;
      } else {
        const uint4 v = ldg128(a);
        o.raw[h][0] = v.x;
        o.raw[h][1] = v.y;
        o.raw[h][2] = v.z;
        o.raw[h][3] = v.w;
      }
      if (ZEROS) {
        const uint8_t* z = zp + (srow[h] + g0);
        if (GPS == 2) {
          o.zero[h][0] = ldg16(z);
        } else if (GPS == 4) {
          o.zero[h][0] = ldg32(z);
        } else {
          const uint2 v = ldg64(z);
          o.zero[h][0] = v.x;
          o.zero[h][1] = v.y;
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < GPS; ++q) {
        // groups past the row's end meet zero x: their scale is zero (an
        // infinite one would make them NaN)
        const int at = srow[h] + g0 + q;
        o.raw[h][q] = 0u;
        if (g0 + q < p.ng)
          o.raw[h][q] = p.scale_type == MOE_F32 ? ldg32(static_cast<const uint32_t*>(sp) + at)
                                                : ldg16(static_cast<const uint16_t*>(sp) + at);
      }
      if (ZEROS) {
#pragma unroll
        for (int q = 0; q < GPS; q += 2)
          o.zero[h][q / 2] = ldg8(zp + srow[h] + min(g0 + q, p.ng - 1)) |
                             (ldg8(zp + srow[h] + min(g0 + q + 1, p.ng - 1)) << 8);
      }
    }
  }
}

// Half H of a stage's scales as floats and zero points as nibbles of a word.
template <bool ZEROS, int GPS, int H>
__device__ __forceinline__ void unpack_scales(const W4Args& p, const Scales<GPS>& s, float (&f)[GPS / 2][2],
                                              uint32_t& zp) {
  constexpr int GPB = GPS / 2;
  zp = 0u;
#pragma unroll
  for (int q = 0; q < GPB; ++q)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = H * GPB + q;
      uint32_t v = p.vec ? s.raw[h][i / 2] >> (16 * (i & 1)) : s.raw[h][i];
      if (p.scale_type == MOE_BF16)
        v <<= 16;
      else if (p.scale_type == MOE_F16)
        v = __float_as_uint(__half2float(__ushort_as_half(uint16_t(v))));
      f[q][h] = __uint_as_float(v);
      if (ZEROS) {
        // vec: four bytes a word; else a byte pair a word
        const uint32_t z = p.vec ? s.zero[h][i / 4] >> (8 * (i & 3)) : s.zero[h][i / 2] >> (8 * (i & 1));
        zp |= (z & 15u) << (4 * (2 * q + h));
      }
    }
}

// A lane's 8-column pieces of NT x 8 rows of x in NC 32-column chunks from
// column `at` on. Rows that are not there keep what x holds (zeros).
template <typename T, int NT, int NC>
__device__ __forceinline__ void load_x(const T* const (&xrow)[NT], bool edge, int at, int k, uint4 (&x)[NT][NC]) {
  if (!edge) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < NC; ++c) ldg128_if(x[j][c], xrow[j] + at + c * 32, xrow[j] != nullptr);
  } else {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < NC; ++c) x[j][c] = load_x8_edge(xrow[j], at + c * 32, k);
  }
}

// Half H of a stage, four chunks of 32 codes x 64 weight rows, against 8 NT
// rows of x.
template <bool BF16, int GS, bool ZEROS, int NT, int H>
__device__ __forceinline__ void half_mma(const W4Args& p, uint32_t st, float (&acc)[4][NT][4],
                                         const Scales<KB / GS>& cur, const uint4 (&x)[NT][4], int lane) {
  constexpr int GPB = KH / GS;   // scale groups of a half
  constexpr int CPG = GS / 32;   // 32-code chunks per scale group
  constexpr uint32_t BASE = BF16 ? 0x43004300u : 0x64006400u;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t mask = p.mask;
  float sc[GPB][2];
  uint32_t zp;
  unpack_scales<ZEROS, KB / GS, H>(p, cur, sc, zp);
  uint32_t xp[NT][4][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      xp[j][c][0] = __byte_perm(x[j][c].x, x[j][c].z, 0x5410);
      xp[j][c][1] = __byte_perm(x[j][c].x, x[j][c].z, 0x7632);
      xp[j][c][2] = __byte_perm(x[j][c].y, x[j][c].w, 0x5410);
      xp[j][c][3] = __byte_perm(x[j][c].y, x[j][c].w, 0x7632);
    }
  // 16-byte chunk c of row r sits at chunk c ^ (r % 8)
  const uint32_t row = st + g * 128 + t * 4;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int src = (lane & ~3) | m;   // the lane that holds this m's scales
    float part[NT][4];
    uint32_t zm = 0x88888888u;
    if (ZEROS) zm = __shfl_sync(0xFFFFFFFFu, zp, src);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int q = c / CPG;
      if (c % CPG == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[j][e] = 0.0f;
      }
      const uint32_t b0 = BASE + ((zm >> (8 * q)) & 15u) * 0x00010001u;
      const uint32_t b1 = BASE + ((zm >> (8 * q + 4)) & 15u) * 0x00010001u;
      const uint32_t at = row + m * 2048 + (((4 * H + c) ^ g) << 4);
      const uint32_t w0 = lds32(at), w1 = lds32(at + 1024);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t a0 = unpack_pair<BF16>(w0, 2 * s, b0, mask), a1 = unpack_pair<BF16>(w1, 2 * s, b1, mask);
        const uint32_t a2 = unpack_pair<BF16>(w0, 2 * s + 1, b0, mask);
        const uint32_t a3 = unpack_pair<BF16>(w1, 2 * s + 1, b1, mask);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_16816<BF16>(part[j], a0, a1, a2, a3, xp[j][c][2 * s], xp[j][c][2 * s + 1]);
      }
      if (c % CPG == CPG - 1) {
        const float s0 = __shfl_sync(0xFFFFFFFFu, sc[q][0], src);
        const float s1 = __shfl_sync(0xFFFFFFFFu, sc[q][1], src);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[m][j][0] = fmaf(part[j][0], s0, acc[m][j][0]);
          acc[m][j][1] = fmaf(part[j][1], s0, acc[m][j][1]);
          acc[m][j][2] = fmaf(part[j][2], s1, acc[m][j][2]);
          acc[m][j][3] = fmaf(part[j][3], s1, acc[m][j][3]);
        }
      }
    }
  }
}

// Barrier of the wk warps that share columns (number nw of the block).
__device__ __forceinline__ void column_sync(int nw, int wk) {
  if (wk == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(nw + 1), "r"(wk * 32) : "memory");
}

template <bool BF16, int GS, bool ZEROS, int NT>
__global__ void __launch_bounds__(THREADS, ctas_per_sm(NT))
    w4_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1, const W4Args p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int RMAX = 8 * NT;   // rows of a unit
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[WARPS][STAGES];
  __shared__ GroupPlan s_plan;
  __shared__ int s_abort_store;
  volatile int* s_abort = &s_abort_store;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(smem + RING_BYTES);   // [WARPS][RED_ROWS][8]
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wn = WARPS / p.wk;                 // warps along the columns
  const int kw = warp % p.wk, nw = warp / p.wk;
  const int wrows = p.dual ? BOX_ROWS / 2 : BOX_ROWS;   // output columns of a warp

  if (threadIdx.x == 0) {
    for (int w = 0; w < WARPS; ++w)
      for (int s = 0; s < STAGES; ++s) mbar_init(&s_bar[w][s], 1);
    s_abort_store = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm0);
    if (p.dual) tma_prefetch_desc(&tm1);
  }
  // the set-up above overlaps the previous kernel; nothing it reads or writes
  // is touched before this point
  pdl_wait();
  pdl_launch_dependents();
  const int total = build_plan<THREADS>(s_plan, p.offsets, p.ngroups, p.nweights, p.rows, p.status,
                                        [&](int n_g) -> int { return ((n_g + RMAX - 1) / RMAX) * p.ntn; });

  // This warp's stages of a unit: every wk-th, so that the warps along the
  // contraction read neighbouring pieces of the same rows at one time.
  const int kb0 = kw, kb1 = p.nkb;
  // The ring runs STAGES stages ahead of use, across units; every lane keeps
  // its state and one of them issues the copies.
  const uint32_t ring = smem_u32(smem) + warp * (STAGES * STAGE_BYTES);
  uint64_t* bar = s_bar[warp];
  uint32_t used = 0, issued = 0;
  const uint32_t withheld = p.withhold && blockIdx.x == 0 ? 0u : 0xFFFFFFFFu;
  int i_unit = int(blockIdx.x), i_kb = kb0, i_g = 0, i_row = 0;
  bool ok = true;
  auto place = [&]() {   // the group and first weight row of i_unit
    if (i_unit < total) {
      const Unit u = decode_unit<RMAX>(i_unit, s_plan, p);
      i_g = u.g;
      i_row = (u.nt * wn + nw) * wrows;
    }
  };
  auto issue = [&]() {   // the next stage, if there is one
    if (i_unit >= total || kb0 >= kb1) return;
    const uint32_t s = issued % STAGES;
    if (issued == withheld) {
      // test only: this stage never arrives
    } else if (elect_one()) {
      uint8_t* dst = smem + (warp * STAGES + s) * STAGE_BYTES;
      mbar_arrive_expect_tx(&bar[s], STAGE_BYTES);
      tma_load_3d(dst, &tm0, &bar[s], i_kb * (KB / 2), i_row, i_g);
      if (p.dual) tma_load_3d(dst + STAGE_BYTES / 2, &tm1, &bar[s], i_kb * (KB / 2), i_row, i_g);
    }
    ++issued;
    if ((i_kb += p.wk) >= kb1) {
      i_kb = kb0;
      i_unit += gridDim.x;
      place();
    }
  };
  place();
  for (int s = 0; s < STAGES; ++s) issue();
  __syncwarp();

  for (int i = blockIdx.x; i < total; i += gridDim.x) {
    const Unit u = decode_unit<RMAX>(i, s_plan, p);
    const int nbase = (u.nt * wn + nw) * wrows;
    // this lane's scale rows within the group (rows past n: the last one's, not stored)
    int srow[2];
    const int which = p.dual ? t >> 1 : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) srow[h] = min(nbase + (p.dual ? (t & 1) : t) * 16 + h * 8 + g, p.n - 1) * p.ng;
    const size_t gofs = size_t(u.g) * size_t(p.n) * size_t(p.ng);
    const void* sp = static_cast<const uint8_t*>(p.scales[which]) + gofs * (p.scale_type == MOE_F32 ? 4 : 2);
    const uint8_t* zp = p.zeros[which] ? p.zeros[which] + gofs : nullptr;
    // rows of x; rows that are not there (past the unit's, or a perm outside
    // x) read as zero
    const T* xrow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      xrow[j] = nullptr;
      if (8 * j + g < u.nr) {
        const int r = u.r0 + 8 * j + g;
        const int tok = p.perm ? __ldg(p.perm + r) : r;
        if (tok >= 0 && tok < p.x_rows)
          xrow[j] = static_cast<const T*>(p.x) + size_t(tok) * size_t(p.ldx);
        else
          set_status(p.status, STATUS_BAD_ROW);
      }
    }
    float acc[4][NT][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
    // x runs one half ahead of its use, the scales one stage
    uint4 x[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[i][j][c] = make_uint4(0u, 0u, 0u, 0u);
    Scales<KB / GS> sc, sn;
    const int hend = min(2 * kb1, (p.k + KH - 1) / KH);   // halves past the row's end hold nothing
    auto ahead = [&](int hk, uint4 (&xx)[NT][4]) {
      if (hk < hend) load_x<T, NT, 4>(xrow, (hk + 1) * KH > p.k, hk * KH + t * 8, p.k, xx);
    };
    if (kb0 < kb1) {
      ahead(2 * kb0, x[0]);
      load_scales<ZEROS>(p, sp, zp, srow, kb0, sn);
    }
    for (int kb = kb0; kb < kb1; kb += p.wk) {
      ahead(2 * kb + 1, x[1]);
      sc = sn;
      if (kb + p.wk < kb1) load_scales<ZEROS>(p, sp, zp, srow, kb + p.wk, sn);
      if (ok) {
        const bool got = mbar_wait_stage(&bar[used % STAGES], (used / STAGES) & 1u, s_abort, p.status, p.wait_ns);
        ok = __all_sync(0xFFFFFFFFu, got);
      }
      const uint32_t st = ring + (used % STAGES) * STAGE_BYTES;
      if (ok) half_mma<BF16, GS, ZEROS, NT, 0>(p, st, acc, sc, x[0], lane);
      if (kb + p.wk < kb1) ahead(2 * (kb + p.wk), x[0]);
      if (ok) {
        if (2 * kb + 1 < hend) half_mma<BF16, GS, ZEROS, NT, 1>(p, st, acc, sc, x[1], lane);
        ++used;
        __syncwarp();   // every lane has read the stage
        issue();
      }
    }
    // partial sums of the warps along the contraction, in warp order; in
    // halves of the warp's rows: m = 0 and 2 (in the gate/up form 16 gate rows
    // and the up rows that go with them), then m = 1 and 3
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float* mine = red + warp * (RED_ROWS * 8) + g * 8 + 2 * t;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const float(&c)[4] = acc[hh + 2 * v][j];
          *reinterpret_cast<float2*>(mine + v * 128) = make_float2(c[0], c[1]);
          *reinterpret_cast<float2*>(mine + v * 128 + 64) = make_float2(c[2], c[3]);
        }
        column_sync(nw, p.wk);
        const int nr = min(8, u.nr - 8 * j);
        const int half = wrows >> 1;   // output columns of this half: 16 or 32
        for (int e = kw * 32 + lane; e < half * nr; e += p.wk * 32) {
          const int r = p.dual ? e >> 4 : e >> 5, cc = e & (half - 1);
          // weight row of cc: row cc of m = hh, or (plain form, cc >= 16) of m = hh + 2
          const int col = nbase + hh * 16 + cc + (cc & 16);
          if (col < p.n) {
            const float* src = red + nw * p.wk * (RED_ROWS * 8) + cc * 8 + r;
            float a = 0.0f, b = 0.0f;
            for (int q = 0; q < p.wk; ++q) a += src[q * (RED_ROWS * 8)];
            if (p.dual) {
              for (int q = 0; q < p.wk; ++q) b += src[q * (RED_ROWS * 8) + 128];
              a = silu_mul<false>(a, b);
            }
            store_y(p, size_t(u.r0 + 8 * j + r) * size_t(p.ldy) + size_t(col), a);
          }
        }
        column_sync(nw, p.wk);   // the partial sums are rewritten
      }
    }
  }
  // copies issued but never used (only after an abort) must land first
  if (lane == 0) {
    int never = 0;
    for (uint32_t j = used; j < issued; ++j)
      if (j != withheld) mbar_wait_stage(&bar[j % STAGES], (j / STAGES) & 1u, &never, p.status, p.wait_ns);
  }
}

template <bool BF16, int GS, bool ZEROS, int NT>
cudaError_t launch(const moe_layer_s* L, const CUtensorMap& tm0, const CUtensorMap& tm1, W4Args a, long long units,
                   cudaStream_t st) {
  static std::atomic<bool> configured[kMaxDevices];   // the attribute is per device
  cudaError_t ce = once_per_device(configured, []() {
    return cudaFuncSetAttribute(w4_kernel<BF16, GS, ZEROS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_DYN);
  });
  if (ce != cudaSuccess) return ce;
  a.wait_ns = kWaitLimitNs;
  if (L->test_stall_ns) {   // a test armed a stall for this one launch
    a.wait_ns = L->test_stall_ns;
    a.withhold = 1;
    L->test_stall_ns = 0;
  }
  const long long cap = static_cast<long long>(ctas_per_sm(NT)) * L->num_sms;
  const dim3 grid(unsigned(units < cap ? units : cap));
  return launch_pdl(w4_kernel<BF16, GS, ZEROS, NT>, grid, dim3(THREADS), SMEM_DYN, st, tm0, tm1, a);
}

template <bool BF16, bool ZEROS, int NT>
cudaError_t launch_group(const moe_layer_s* L, int group, const CUtensorMap& tm0, const CUtensorMap& tm1,
                         const W4Args& a, long long units, cudaStream_t st) {
  if (group == 32) return launch<BF16, 32, ZEROS, NT>(L, tm0, tm1, a, units, st);
  if (group == 64) return launch<BF16, 64, ZEROS, NT>(L, tm0, tm1, a, units, st);
  return launch<BF16, 128, ZEROS, NT>(L, tm0, tm1, a, units, st);
}

template <int NT>
cudaError_t launch_type(const moe_layer_s* L, moe_dtype t, bool zeros, int group, const CUtensorMap& tm0,
                        const CUtensorMap& tm1, const W4Args& a, long long units, cudaStream_t st) {
  if (t == MOE_BF16)
    return zeros ? launch_group<true, true, NT>(L, group, tm0, tm1, a, units, st)
                 : launch_group<true, false, NT>(L, group, tm0, tm1, a, units, st);
  return zeros ? launch_group<false, true, NT>(L, group, tm0, tm1, a, units, st)
               : launch_group<false, false, NT>(L, group, tm0, tm1, a, units, st);
}

}  // namespace

cudaError_t launch_w4(const moe_layer_s* L, moe_dtype t, const void* x, int x_rows, long long ldx, const int32_t* perm,
                      const moe_w4_weights* w, const moe_w4_weights* up, const int32_t* offsets, int rows, int n,
                      int k, moe_dtype out_t, void* y, long long ldy, cudaStream_t st) {
  const int G = L->E + L->S;
  W4Args p = {};
  p.offsets = offsets;
  p.ngroups = L->E + 1;
  p.nweights = G;
  p.rows = rows;
  p.x = x;
  p.ldx = ldx;
  p.x_rows = x_rows;
  p.perm = perm;
  p.scales[0] = w->scales;
  p.zeros[0] = w->zeros;
  p.scales[1] = up ? up->scales : w->scales;
  p.zeros[1] = up ? up->zeros : w->zeros;
  p.scale_type = w->scale_type;
  p.n = n;
  p.k = k;
  p.ng = (k + w->group - 1) / w->group;
  p.dual = up != nullptr;
  const int gps = KB / w->group;
  p.vec = w->scale_type != MOE_F32 && p.ng % gps == 0;
  for (int i = 0; i < 2; ++i)
    p.vec = p.vec && reinterpret_cast<uintptr_t>(p.scales[i]) % (2 * gps) == 0 &&
            reinterpret_cast<uintptr_t>(p.zeros[i]) % gps == 0;
  p.nkb = (k + KB - 1) / KB;
  // Rows of a unit: 8, or 16 when groups hold more than 8 on average (the
  // codes are then unpacked half as often, on two thirds of the warps). With
  // 64 groups and 8, 10, 16, 24, 32 and 64 rows in each, gate/up of
  // 1536 x 5120 takes 148, 268, 259, 367, 492 and 963 us by units of 8 and
  // 208, 219, 229, 412, 407 and 766 by units of 16; with the same means
  // spread unevenly 178, 211, 319, 419, 536 and 1002 against 213, 218, 288,
  // 380, 504 and 851.
  const int nt = rows > 8ll * G ? 2 : 1;
  // units per column tile, at most: a group adds at most one that is not full
  long long groups = rows / (8 * nt) + (rows < G ? rows : G);
  if (groups > rows) groups = rows;
  // Warps along the contraction. More of them give more, smaller units (the
  // only way to fill the machine with few experts), fewer leave more stages
  // per unit to pay for its fixed cost (finding it, joining the partial sums:
  // 0.4 of a stage's time). The split with the least expected time of a CTA,
  // from the groups that evenly spread rows would touch: 4 ways for one token
  // (24.4 us against 31 two ways and 47 one way) or one matrix (20.2 against
  // 30.3 and 54), 2 ways for a decode batch of 64 (456 to 465 against 462 to
  // 471 one way and 480 four ways) and for the down projection of 16 tokens
  // (77 against 87 and 91 to 98).
  const double ctas = double(ctas_per_sm(nt)) * L->num_sms;
  const double touched = G * (1.0 - exp(-double(rows) / G)) + double(rows) / (16 * nt);
  double best = 0.0;
  for (int wk = WARPS; wk >= 1; wk /= 2) {
    const int cols = (WARPS / wk) * (p.dual ? BOX_ROWS / 2 : BOX_ROWS);
    const double rounds = (touched < double(groups) ? touched : double(groups)) * ((n + cols - 1) / cols) / ctas + 0.5;
    const double cost = (rounds > 1.0 ? rounds : 1.0) * (2 * ((p.nkb + wk - 1) / wk) + 0.8);
    if (best == 0.0 || cost < best) {
      best = cost;
      p.wk = wk;
    }
  }
  const int cols = (WARPS / p.wk) * (p.dual ? BOX_ROWS / 2 : BOX_ROWS);
  p.ntn = (n + cols - 1) / cols;
  p.y = y;
  p.ldy = ldy;
  p.y_type = out_t;
  p.status = L->status;
  p.mask = 0x000F000Fu;
  CUtensorMap tm0, tm1;
  const uint32_t box = p.dual ? BOX_ROWS / 2 : BOX_ROWS;
  if (!encode_tmap_codes(&tm0, w->codes, (k + 1) / 2, n, G, w->ld, box)) return cudaErrorInvalidValue;
  tm1 = tm0;
  if (up && !encode_tmap_codes(&tm1, up->codes, (k + 1) / 2, n, G, up->ld, box)) return cudaErrorInvalidValue;
  const long long units = groups * p.ntn;
  return nt == 1 ? launch_type<1>(L, t, w->zeros != nullptr, w->group, tm0, tm1, p, units, st)
                 : launch_type<2>(L, t, w->zeros != nullptr, w->group, tm0, tm1, p, units, st);
}

}  // namespace moe
