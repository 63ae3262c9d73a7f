// What the operators around the token mixer share: their dims in the kernels' form, vector loads and stores of
// any supported type as fp32 values, the gate's two halves, the launchers.  Internal to libswimba.
#pragma once
#include "common.cuh"

namespace swimba {

struct NormDims {
  int M, D, dtype, grad_dtype;
  long long x_stride;
  float eps;
};

struct GatedDims {
  int B, T, W, dtype, grad_dtype;
  long long x_stride, gate_stride;
};

struct FfnDims {
  int M, D, F, dtype, act;
};

// VEC consecutive values as fp32, by 16-byte (or one 8-byte, or element) accesses; p is aligned to the access.
template <class T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  constexpr int kBytes = VEC * (int)sizeof(T);
  if constexpr (kBytes % 16 == 0) {
#pragma unroll
    for (int b = 0; b < kBytes / 16; ++b) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[b];
      T t[16 / sizeof(T)];
      memcpy(t, &u, 16);
#pragma unroll
      for (int j = 0; j < 16 / (int)sizeof(T); ++j) v[b * (16 / sizeof(T)) + j] = to_f32(t[j]);
    }
  } else if constexpr (kBytes == 8) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    T t[8 / sizeof(T)];
    memcpy(t, &u, 8);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = to_f32(t[j]);
  } else if constexpr (kBytes == 4 && VEC > 1) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    T t[4 / sizeof(T)];
    memcpy(t, &u, 4);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = to_f32(t[j]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = to_f32(p[j]);
  }
}

// Two values rounded to a 16-bit type by one conversion, a in the lower half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &r, 4);
  return u;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 r = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &r, 4);
  return u;
}

template <class T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  constexpr int kBytes = VEC * (int)sizeof(T);
  T t[VEC];
  if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const uint32_t u = pack2<T>(v[j], v[j + 1]);
      memcpy(t + j, &u, 4);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) t[j] = from_f32<T>(v[j]);
  }
  if constexpr (kBytes % 16 == 0) {
#pragma unroll
    for (int b = 0; b < kBytes / 16; ++b) {
      uint4 u;
      memcpy(&u, t + b * (16 / sizeof(T)), 16);
      reinterpret_cast<uint4*>(p)[b] = u;
    }
  } else if constexpr (kBytes == 8) {
    uint2 u;
    memcpy(&u, t, 8);
    *reinterpret_cast<uint2*>(p) = u;
  } else if constexpr (kBytes == 4 && VEC > 1) {
    uint32_t u;
    memcpy(&u, t, 4);
    *reinterpret_cast<uint32_t*>(p) = u;
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) p[j] = t[j];
  }
}

// e^x and 1 / x by the hardware's approximations alone, where __expf and __fdividef add instructions for subnormals
// (results and operands that are subnormal are 0 here).  The approximations are good to 2 ulp and 1 ulp; the product with
// log2(e) rounds twice more, which adds 2 |x| u to e^x.
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// f = sigmoid(g) and q = sigmoid(-g) = 1 - f.  The smaller of the two comes from exp(-|g|) in (0, 1], the larger as
// its complement to 1: neither overflows, the small one keeps its relative accuracy, and a gate near 1 is rounded
// once (a bias there would grow with the length of the memory).
__device__ __forceinline__ void gate_pair(float g, float& f, float& q) {
  const float e = exp_fast(-fabsf(g));
  const float small = e * rcp_fast(1.f + e), large = 1.f - small;
  f = g >= 0.f ? large : small;
  q = g >= 0.f ? small : large;
}

// Launchers (each defined beside its kernels).
size_t layer_norm_bwd_ws(const NormDims& d);
cudaError_t launch_layer_norm(const NormDims& d, const void* x, const void* residual, const float* gamma,
                              const float* beta, void* y, void* r_out, cudaStream_t s);
cudaError_t launch_layer_norm_bwd(const NormDims& d, const void* r, const float* gamma, const void* dy, const void* dr,
                                  void* dx, float* dgamma, float* dbeta, float* part, cudaStream_t s);

cudaError_t launch_gated_scan(const GatedDims& d, const void* x, const void* gate, const float* init, void* h,
                              float* final_state, unsigned* st, cudaStream_t s);
cudaError_t launch_gated_scan_bwd(const GatedDims& d, const void* x, const void* gate, const void* h, const float* init,
                                  const void* dh, const float* dfinal, void* dx, void* dgate, float* dinit,
                                  unsigned* st, cudaStream_t s);
cudaError_t launch_gated_step(const GatedDims& d, const void* x, const void* gate, float* state, void* h,
                              cudaStream_t s);

// The feed-forward block.  bwd writes dgate and dup [M][F] each (dtype) to `dgu`.
size_t gated_ffn_ws(const FfnDims& d);
size_t gated_ffn_bwd_ws(const FfnDims& d);
cudaError_t launch_gated_ffn(const FfnDims& d, const void* x, const void* w_gate, const void* w_up, const void* w_down,
                             void* gate, void* up, void* h, void* out, char* ws, unsigned* st, cudaStream_t s);
cudaError_t launch_gated_ffn_bwd(const FfnDims& d, const void* x, const void* gate, const void* up, const void* h,
                                 const void* w_gate, const void* w_up, const void* w_down, const void* dout, void* dx,
                                 void* dw_gate, void* dw_up, void* dw_down, char* ws, unsigned* st, cudaStream_t s);

}  // namespace swimba
