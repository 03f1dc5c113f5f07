// SwiGLU over the grouped rows and its gradient, element by element in fp32:
//   h = g s u,  s = 1 / (1 + exp(-g))
//   dh/du = g s,  dh/dg = u s (1 + g (1 - s)),  1 - s = 1 / (1 + exp(g))
// Both are bound by HBM (3 and 5 streams of the operands, 6 with h again; no
// reuse): one 16-byte vector of each operand per thread and trip, 4 CTAs of
// 256 threads per SM (the gradient over 36,864 rows of 1,536 in bf16, 566 MB:
// 94 to 97 us back to back, 5.8 to 6.0 TB/s; with 6 CTAs 8 us more, with two
// vectors in flight per thread 37 for the registers they take).
//
// The arithmetic is silu.cuh's. Its short form holds for gates from kLowGate
// on with a product dh u inside fp32; a vector with others is noticed here
// and done again by careful_elements (3 to 6 of the 97 us are the notice; a
// branch per element in its place took 115 us in all).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "silu.cuh"

namespace moe {

namespace {

constexpr int THREADS = 256;
constexpr int CTAS_PER_SM = 4;

template <typename T>
struct Cvt;
template <>
struct Cvt<float> {
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
};
template <>
struct Cvt<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Cvt<__half> {
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
};

// N consecutive elements as one access (16 bytes at most).
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

struct SwigluArgs {
  const void* dh;
  const void* gate;
  const void* up;
  void* o0;   // h, or dgate
  void* o1;   // dup
  void* o2;   // h of the gradient, or null
  long long ld_dh, ld_gate, ld_up, ld0, ld1, ld2;
  const int32_t* offsets;   // [ngroups + 1], or null: all rows
  int ngroups, nweights;
  int rows, f;
  uint32_t* status;
};

// The launch's rows [r0, r1): those of the groups. False: a bad plan.
__device__ __forceinline__ bool group_rows(const SwigluArgs& p, int& r0, int& r1) {
  r0 = 0;
  r1 = p.rows;
  if (!p.offsets) return true;
  int bad = 0;
  for (int g = threadIdx.x; g < p.ngroups; g += THREADS) {
    const int a = p.offsets[g], b = p.offsets[g + 1];
    bad |= a < 0 || b < a || b > p.rows || (g >= p.nweights && b != a);
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, STATUS_BAD_PLAN);
    return false;
  }
  r0 = p.offsets[0];
  r1 = p.offsets[p.ngroups];
  return true;
}

// N elements from (row, c) on, one by one from memory (in registers, the
// second copy of the arithmetic would spill): right for all values.
template <typename T, int N, bool BACKWARD>
__device__ __forceinline__ void careful_elements(const SwigluArgs& p, size_t row, int c) {
  constexpr bool FAST = sizeof(T) == 2;
#pragma unroll 1
  for (int j = c; j < c + N; ++j) {
    const float g = Cvt<T>::to(static_cast<const T*>(p.gate)[row * p.ld_gate + j]);
    const float u = Cvt<T>::to(static_cast<const T*>(p.up)[row * p.ld_up + j]);
    const T h = Cvt<T>::from(silu_mul<FAST>(g, u));
    if (BACKWARD) {
      const float d = Cvt<T>::to(static_cast<const T*>(p.dh)[row * p.ld_dh + j]);
      static_cast<T*>(p.o0)[row * p.ld0 + j] = Cvt<T>::from(dgate_mul<FAST>(g, u, d));
      static_cast<T*>(p.o1)[row * p.ld1 + j] = Cvt<T>::from(silu_mul<FAST>(g, d));
      if (p.o2) static_cast<T*>(p.o2)[row * p.ld2 + j] = h;
    } else {
      static_cast<T*>(p.o0)[row * p.ld0 + j] = h;
    }
  }
}

template <typename T, int N, bool BACKWARD>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) swiglu_kernel(const SwigluArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  int r0, r1;
  if (!group_rows(p, r0, r1)) return;
  using V = Vec<T, N>;
  constexpr bool FAST = sizeof(T) == 2;
  // fp16: below kLowGate every result is zero, and products stay inside fp32
  constexpr bool RANGE = !std::is_same<T, __half>::value;
  const uint32_t per_row = uint32_t(p.f / N);   // the host picks N = 1 unless it divides f
  const uint64_t total = uint64_t(r1 - r0) * per_row;
  const uint64_t step = uint64_t(gridDim.x) * THREADS;
  for (uint64_t i = uint64_t(blockIdx.x) * THREADS + threadIdx.x; i < total; i += step) {
    // 32-bit division where it will do (a 64-bit one takes as long as the rest)
    const uint64_t r = (total >> 32) ? i / per_row : uint32_t(i) / per_row;
    const size_t row = size_t(r) + size_t(r0);
    const int c = int(i - r * per_row) * N;
    const V g = *reinterpret_cast<const V*>(static_cast<const T*>(p.gate) + row * p.ld_gate + c);
    const V u = *reinterpret_cast<const V*>(static_cast<const T*>(p.up) + row * p.ld_up + c);
    V a, b, d, h;
    if (BACKWARD) d = *reinterpret_cast<const V*>(static_cast<const T*>(p.dh) + row * p.ld_dh + c);
    bool rare = false;   // a gate below kLowGate, or a product dh u beyond fp32
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float gv = Cvt<T>::to(g.v[j]), uv = Cvt<T>::to(u.v[j]);
      rare |= RANGE && gv < kLowGate;
      float s, m;
      sigmoid_pair<FAST>(gv, s, m);
      const float silu = gv * s;
      h.v[j] = Cvt<T>::from(silu * uv);
      if (BACKWARD) {
        const float dv = Cvt<T>::to(d.v[j]);
        const float du = dv * uv;
        rare |= RANGE && fabsf(du) > FLT_MAX;
        a.v[j] = Cvt<T>::from(du * (s + silu * m));
        b.v[j] = Cvt<T>::from(dv * silu);
      }
    }
    if (rare) {
      careful_elements<T, N, BACKWARD>(p, row, c);
      continue;
    }
    if (BACKWARD) {
      *reinterpret_cast<V*>(static_cast<T*>(p.o0) + row * p.ld0 + c) = a;
      *reinterpret_cast<V*>(static_cast<T*>(p.o1) + row * p.ld1 + c) = b;
      if (p.o2) *reinterpret_cast<V*>(static_cast<T*>(p.o2) + row * p.ld2 + c) = h;
    } else {
      *reinterpret_cast<V*>(static_cast<T*>(p.o0) + row * p.ld0 + c) = h;
    }
  }
}

template <typename T, bool BACKWARD>
cudaError_t launch(const moe_layer_s* L, const SwigluArgs& p, cudaStream_t st) {
  constexpr int N = 16 / int(sizeof(T));
  const void* ptr[] = {p.dh, p.gate, p.up, p.o0, p.o1, p.o2};
  const long long ld[] = {p.ld_dh, p.ld_gate, p.ld_up, p.ld0, p.ld1, p.ld2};
  bool wide = p.f % N == 0;
  for (int i = 0; i < 6; ++i)
    if (ptr[i]) wide = wide && reinterpret_cast<uintptr_t>(ptr[i]) % 16 == 0 && ld[i] % N == 0;
  const long long items = static_cast<long long>(p.rows) * (wide ? p.f / N : p.f);
  const long long blocks = (items + THREADS - 1) / THREADS;
  const long long cap = static_cast<long long>(L->num_sms) * CTAS_PER_SM;
  const dim3 grid(unsigned(blocks < cap ? blocks : cap));
  if (wide) return launch_pdl(swiglu_kernel<T, N, BACKWARD>, grid, dim3(THREADS), 0, st, p);
  return launch_pdl(swiglu_kernel<T, 1, BACKWARD>, grid, dim3(THREADS), 0, st, p);
}

template <bool BACKWARD>
cudaError_t launch_type(const moe_layer_s* L, moe_dtype t, const SwigluArgs& p, cudaStream_t st) {
  if (t == MOE_BF16) return launch<__nv_bfloat16, BACKWARD>(L, p, st);
  if (t == MOE_F16) return launch<__half, BACKWARD>(L, p, st);
  return launch<float, BACKWARD>(L, p, st);
}

SwigluArgs args(const moe_layer_s* L, const int32_t* offsets, int rows, int f) {
  SwigluArgs p = {};
  p.offsets = offsets;
  p.ngroups = L->E + 1;
  p.nweights = L->E + L->S;
  p.rows = rows;
  p.f = f;
  p.status = L->status;
  return p;
}

}  // namespace

cudaError_t launch_swiglu(const moe_layer_s* L, moe_dtype t, const void* gate, long long ldg, const void* up,
                          long long ldu, const int32_t* offsets, int rows, int f, void* h, long long ldh,
                          cudaStream_t st) {
  SwigluArgs p = args(L, offsets, rows, f);
  p.gate = gate;
  p.ld_gate = ldg;
  p.up = up;
  p.ld_up = ldu;
  p.o0 = h;
  p.ld0 = ldh;
  return launch_type<false>(L, t, p, st);
}

cudaError_t launch_swiglu_backward(const moe_layer_s* L, moe_dtype t, const void* dh, long long lddh, const void* gate,
                                   long long ldg, const void* up, long long ldu, const int32_t* offsets, int rows,
                                   int f, void* dgate, long long lddg, void* dup, long long lddu, void* h,
                                   long long ldh, cudaStream_t st) {
  SwigluArgs p = args(L, offsets, rows, f);
  p.dh = dh;
  p.ld_dh = lddh;
  p.gate = gate;
  p.ld_gate = ldg;
  p.up = up;
  p.ld_up = ldu;
  p.o0 = dgate;
  p.ld0 = lddg;
  p.o1 = dup;
  p.ld1 = lddu;
  p.o2 = h;
  p.ld2 = ldh;
  return launch_type<true>(L, t, p, st);
}

}  // namespace moe
