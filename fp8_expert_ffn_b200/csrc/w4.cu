// Products with 4-bit expert weights for few rows per expert (decode):
//   y[r, j] = sum_groups s[g, j, c] * sum_{i in c} x[perm[r], i] (q[g, j, i] - z[g, j, c])
// and the gate/up form h = silu(gate) * up. A weight is read once for up to 16
// rows, half a byte each, so HBM bounds the kernel as long as unpacking keeps
// up: 6.5 TB/s is 46 codes per SM and cycle, which leaves about 45
// instructions per warp for 512 codes.
//
// Unpacking is exact and short: code nibbles i and i + 4 of a 32-bit word are
// masked out together and OR-ed into the mantissas of the 16-bit pair
// (128, 128) in bf16 or (1024, 1024) in fp16; subtracting (128 + z) or
// (1024 + z) leaves q - z exactly. The pairs go to mma.sync m16n8k16 (weights
// as A, up to 8 rows of x as one B) with fp32 sums per scale group; the scale
// multiplies that sum in fp32, so nothing is rounded between the codes and the
// output. The order of the contraction inside a word (0,4,1,5,...) is the
// same for x, whose 8 consecutive values are shuffled with four byte
// permutes. tcgen05 would need the unpacked weights back in shared or tensor
// memory, a second trip per code that the memory-bound case has no use for.
//
// Layout: 8 warps per CTA, 2 CTAs per SM, persistent over (group, column tile,
// rows chunk). A warp owns 64 weight rows (32 gate and 32 up) and a contiguous
// part of the contraction, and streams its codes through its own ring of TMA
// boxes (64 rows x 64 bytes = 128 codes, 64-byte swizzle: lane (g, t) reads
// word t of row g without bank conflicts), so no warp waits for another until
// a tile's partial sums meet in shared memory, added in warp order. The warps
// of a CTA split the contraction 8, 4, 2 or 1 ways (and the columns by the
// rest), whichever leaves the fewest idle.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "groups.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int KB = 128;                    // codes per row of a block
constexpr int STAGES = 2;
constexpr int BOX_ROWS = 64;
constexpr int STAGE_BYTES = BOX_ROWS * KB / 2;   // 4 KB
constexpr int RMAX = 16;                   // rows of a chunk
constexpr int RING_BYTES = WARPS * STAGES * STAGE_BYTES;
constexpr int RED_BYTES = WARPS * BOX_ROWS * 8 * 4;   // partial sums of 8 rows
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
// bias = (128 + z, twice) in bf16 or (1024 + z, twice) in fp16.
template <bool BF16>
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w, int i, uint32_t bias) {
  uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | (BF16 ? 0x43004300u : 0x64006400u);
  uint32_t d;
  if (BF16)
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(bias));
  else
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(bias));
  return d;
}

__device__ __forceinline__ float load_scale(const void* s, int type, size_t i) {
  if (type == MOE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(s)[i]);
  if (type == MOE_F16) return __half2float(static_cast<const __half*>(s)[i]);
  return static_cast<const float*>(s)[i];
}

struct Unit {
  int g, nt, r0, nr;   // group, column tile, first row, rows (at most RMAX)
};

__device__ __forceinline__ Unit decode_unit(int i, const GroupPlan& s, const W4Args& p) {
  Unit u;
  u.g = find_group(s.prefix, p.ngroups, i);
  const int local = i - s.prefix[u.g];
  const int n_g = s.off[u.g + 1] - s.off[u.g];
  const int chunks = (n_g + RMAX - 1) / RMAX;
  u.nt = local / chunks;   // the chunks that share codes run side by side
  const int c = local - u.nt * chunks;
  u.r0 = s.off[u.g] + c * RMAX;
  u.nr = min(RMAX, n_g - c * RMAX);
  return u;
}

// 8 values of a row of x from column i on; columns past k are zero.
template <typename T>
__device__ __forceinline__ uint4 load_x8(const T* row, int i, int k) {
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

// One warp's ring: issues run STAGES blocks ahead of use, across tiles.
struct Ring {
  uint8_t* base;        // this warp's stages
  uint64_t* bar;        // [STAGES]
  uint32_t used;        // blocks consumed so far
  uint32_t issued;      // lane 0 only
  int unit, kb, kb1;    // lane 0 only: next block to issue
  int g, row;           // lane 0 only: its group and first weight row
};

template <bool BF16, int GS, int NT>
__device__ __forceinline__ void block_mma(const W4Args& p, const uint8_t* st, float (&acc)[4][NT][4],
                                          const uint4 (&xr)[NT][4], const size_t (&srow)[4][2], int kb, int lane) {
  constexpr int GPB = KB / GS;   // scale groups per block
  constexpr int CPG = GS / 32;   // 32-code chunks per scale group
  const int g = lane >> 2, t = lane & 3;
  uint32_t xp[NT][4][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      xp[j][c][0] = __byte_perm(xr[j][c].x, xr[j][c].z, 0x5410);
      xp[j][c][1] = __byte_perm(xr[j][c].x, xr[j][c].z, 0x7632);
      xp[j][c][2] = __byte_perm(xr[j][c].y, xr[j][c].w, 0x5410);
      xp[j][c][3] = __byte_perm(xr[j][c].y, xr[j][c].w, 0x7632);
    }
  constexpr uint32_t BASE = BF16 ? 0x43004300u : 0x64006400u;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int which = p.dual ? m >> 1 : 0;
    float sc[GPB][2];
    uint32_t bias[GPB][2];
#pragma unroll
    for (int q = 0; q < GPB; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int grp = kb * GPB + q;
        const bool in = grp < p.ng;   // groups past the row's end meet zero x
        sc[q][h] = in ? load_scale(p.scales[which], p.scale_type, srow[m][h] + grp) : 0.0f;
        bias[q][h] = BASE + (p.zeros[which] && in ? uint32_t(p.zeros[which][srow[m][h] + grp] & 15) : 8u) * 0x00010001u;
      }
    float part[NT][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c % CPG == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[j][e] = 0.0f;
      }
      // 16-byte chunk c of row r sits at chunk c ^ ((r / 2) % 4)
      const int r0 = m * 16 + g;
      const int o = ((c ^ ((g >> 1) & 3)) << 4) + t * 4;
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(st + r0 * 64 + o);
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(st + (r0 + 8) * 64 + o);
      const uint32_t b0 = bias[c / CPG][0], b1 = bias[c / CPG][1];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t a0 = unpack_pair<BF16>(w0, 2 * s, b0), a1 = unpack_pair<BF16>(w1, 2 * s, b1);
        const uint32_t a2 = unpack_pair<BF16>(w0, 2 * s + 1, b0), a3 = unpack_pair<BF16>(w1, 2 * s + 1, b1);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_16816<BF16>(part[j], a0, a1, a2, a3, xp[j][c][2 * s], xp[j][c][2 * s + 1]);
      }
      if (c % CPG == CPG - 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[m][j][0] = fmaf(part[j][0], sc[c / CPG][0], acc[m][j][0]);
          acc[m][j][1] = fmaf(part[j][1], sc[c / CPG][0], acc[m][j][1]);
          acc[m][j][2] = fmaf(part[j][2], sc[c / CPG][1], acc[m][j][2]);
          acc[m][j][3] = fmaf(part[j][3], sc[c / CPG][1], acc[m][j][3]);
        }
      }
    }
  }
}

template <bool BF16, int GS>
__global__ void __launch_bounds__(THREADS, 2)
    w4_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1, const W4Args p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[WARPS][STAGES];
  __shared__ GroupPlan s_plan;
  __shared__ int s_abort_store;
  volatile int* s_abort = &s_abort_store;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(smem + RING_BYTES);   // [WARPS][64][8]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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

  const int kb0 = kw * p.nkb / p.wk, kb1 = (kw + 1) * p.nkb / p.wk;   // this warp's blocks of a tile
  Ring ring;
  ring.base = smem + warp * (STAGES * STAGE_BYTES);
  ring.bar = s_bar[warp];
  ring.used = 0;
  ring.issued = 0;
  ring.unit = int(blockIdx.x);
  ring.kb = kb0;
  ring.kb1 = kb1;
  bool ok = true;
  uint32_t withheld = 0xFFFFFFFFu;

  auto place = [&]() {   // lane 0: the group and weight row of ring.unit
    if (ring.unit < total) {
      const Unit u = decode_unit(ring.unit, s_plan, p);
      ring.g = u.g;
      ring.row = (u.nt * wn + nw) * wrows;
    }
  };
  auto issue = [&]() {   // lane 0: the next block, if there is one
    if (ring.unit >= total || kb0 == kb1) return;
    const uint32_t s = ring.issued % STAGES;
    if (p.withhold && blockIdx.x == 0 && warp == 0 && ring.issued == 0) {
      withheld = 0;   // test only: this block never arrives
    } else {
      uint8_t* dst = ring.base + s * STAGE_BYTES;
      mbar_arrive_expect_tx(&ring.bar[s], STAGE_BYTES);
      tma_load_3d(dst, &tm0, &ring.bar[s], ring.kb * (KB / 2), ring.row, ring.g);
      if (p.dual) tma_load_3d(dst + STAGE_BYTES / 2, &tm1, &ring.bar[s], ring.kb * (KB / 2), ring.row, ring.g);
    }
    ++ring.issued;
    if (++ring.kb == kb1) {
      ring.kb = kb0;
      ring.unit += gridDim.x;
      place();
    }
  };
  if (lane == 0) {
    place();
    for (int s = 0; s < STAGES; ++s) issue();
  }
  __syncwarp();

  for (int i = blockIdx.x; i < total; i += gridDim.x) {
    const Unit u = decode_unit(i, s_plan, p);
    const int g = lane >> 2, t = lane & 3;
    const int nbase = (u.nt * wn + nw) * wrows;
    // scale rows of this lane's weight rows (rows past n: the last one's, not stored)
    size_t srow[4][2];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = nbase + (p.dual ? (m & 1) : m) * 16 + h * 8 + g;
        srow[m][h] = (size_t(u.g) * p.n + min(r, p.n - 1)) * size_t(p.ng);
      }
    const T* xrow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      xrow[j] = nullptr;
      const int r = 8 * j + g;
      if (r < u.nr) {
        const int tok = p.perm ? __ldg(p.perm + u.r0 + r) : u.r0 + r;
        if (tok >= 0 && tok < p.x_rows)
          xrow[j] = static_cast<const T*>(p.x) + size_t(tok) * size_t(p.ldx);
        else
          set_status(p.status, STATUS_BAD_ROW);
      }
    }
    auto tile = [&](auto nt_c) {
      constexpr int NT = decltype(nt_c)::value;
      float acc[4][NT][4];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
      for (int kb = kb0; kb < kb1; ++kb) {
        uint4 xr[NT][4];   // in flight while the codes arrive
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) xr[j][c] = load_x8(xrow[j], kb * KB + c * 32 + t * 8, p.k);
        const uint32_t s = ring.used % STAGES;
        if (ok) {
          const bool got = mbar_wait_stage(&ring.bar[s], (ring.used / STAGES) & 1u, s_abort, p.status, p.wait_ns);
          ok = __all_sync(0xFFFFFFFFu, got);
        }
        if (ok) {
          block_mma<BF16, GS, NT>(p, ring.base + s * STAGE_BYTES, acc, xr, srow, kb, lane);
          ++ring.used;
          __syncwarp();   // every lane has read the stage
          if (lane == 0) issue();
        }
      }
      // partial sums of the warps along the contraction, in warp order
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float* mine = red + warp * (BOX_ROWS * 8);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          *reinterpret_cast<float2*>(mine + (m * 16 + g) * 8 + 2 * t) = make_float2(acc[m][j][0], acc[m][j][1]);
          *reinterpret_cast<float2*>(mine + (m * 16 + g + 8) * 8 + 2 * t) = make_float2(acc[m][j][2], acc[m][j][3]);
        }
        __syncthreads();
        const int cols = wrows * wn;   // output columns of the tile
        for (int e = threadIdx.x; e < cols * 8; e += THREADS) {
          const int r = e / cols, c = e - r * cols;
          const int w = c / wrows, cc = c - w * wrows;
          const int col = (u.nt * wn + w) * wrows + cc;
          if (8 * j + r < u.nr && col < p.n) {
            const float* src = red + size_t(w) * p.wk * (BOX_ROWS * 8) + cc * 8 + r;
            float a = 0.0f, b = 0.0f;
            for (int q = 0; q < p.wk; ++q) a += src[q * (BOX_ROWS * 8)];
            if (p.dual) {
              for (int q = 0; q < p.wk; ++q) b += src[q * (BOX_ROWS * 8) + wrows * 8];
              a = a / (1.0f + expf(-a)) * b;
            }
            store_y(p, size_t(u.r0 + 8 * j + r) * size_t(p.ldy) + col, a);
          }
        }
        __syncthreads();   // the partial sums are rewritten
      }
    };
    if (u.nr > 8)
      tile(std::integral_constant<int, 2>());
    else
      tile(std::integral_constant<int, 1>());
  }
  // copies issued but never used (only after an abort) must land first
  if (lane == 0) {
    int never = 0;
    for (uint32_t j = ring.used; j < ring.issued; ++j)
      if (j != withheld) mbar_wait_stage(&ring.bar[j % STAGES], (j / STAGES) & 1u, &never, p.status, p.wait_ns);
  }
}

template <bool BF16, int GS>
cudaError_t launch(const moe_layer_s* L, const CUtensorMap& tm0, const CUtensorMap& tm1, W4Args a, long long units,
                   cudaStream_t st) {
  static std::atomic<bool> configured[kMaxDevices];   // the attribute is per device
  cudaError_t ce = once_per_device(configured, []() {
    return cudaFuncSetAttribute(w4_kernel<BF16, GS>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_DYN);
  });
  if (ce != cudaSuccess) return ce;
  a.wait_ns = kWaitLimitNs;
  if (L->test_stall_ns) {   // a test armed a stall for this one launch
    a.wait_ns = L->test_stall_ns;
    a.withhold = 1;
    L->test_stall_ns = 0;
  }
  const long long cap = 2ll * L->num_sms;
  const dim3 grid(unsigned(units < cap ? units : cap));
  return launch_pdl(w4_kernel<BF16, GS>, grid, dim3(THREADS), SMEM_DYN, st, tm0, tm1, a);
}

template <bool BF16>
cudaError_t launch_group(const moe_layer_s* L, int group, const CUtensorMap& tm0, const CUtensorMap& tm1,
                         const W4Args& a, long long units, cudaStream_t st) {
  if (group == 32) return launch<BF16, 32>(L, tm0, tm1, a, units, st);
  if (group == 64) return launch<BF16, 64>(L, tm0, tm1, a, units, st);
  return launch<BF16, 128>(L, tm0, tm1, a, units, st);
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
  p.nkb = (k + KB - 1) / KB;
  // warps along the contraction: the split that leaves the fewest of their
  // block slots idle (the widest of equals)
  p.wk = WARPS;
  for (int wk = WARPS / 2; wk >= 1; wk /= 2) {
    const int idle = (p.nkb + wk - 1) / wk * wk - p.nkb, best = (p.nkb + p.wk - 1) / p.wk * p.wk - p.nkb;
    if (idle < best) p.wk = wk;
  }
  const int cols = (WARPS / p.wk) * (p.dual ? BOX_ROWS / 2 : BOX_ROWS);
  p.ntn = (n + cols - 1) / cols;
  p.y = y;
  p.ldy = ldy;
  p.y_type = out_t;
  p.status = L->status;
  CUtensorMap tm0, tm1;
  const uint32_t box = p.dual ? BOX_ROWS / 2 : BOX_ROWS;
  if (!encode_tmap_codes(&tm0, w->codes, (k + 1) / 2, n, G, w->ld, box)) return cudaErrorInvalidValue;
  tm1 = tm0;
  if (up && !encode_tmap_codes(&tm1, up->codes, (k + 1) / 2, n, G, up->ld, box)) return cudaErrorInvalidValue;
  const long long units = (static_cast<long long>(rows) / RMAX + (rows < G ? rows : G)) * p.ntn;
  return t == MOE_BF16 ? launch_group<true>(L, w->group, tm0, tm1, p, units, st)
                       : launch_group<false>(L, w->group, tm0, tm1, p, units, st);
}

}  // namespace moe
