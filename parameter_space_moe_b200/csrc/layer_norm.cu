// Layer norm over the rows of a [M][D] matrix, with the residual sum in front of it, and its gradients.
//
//   r = x (+ residual),  mu = mean(r),  v = mean((r - mu)^2),  y = (r - mu) / sqrt(v + eps) * gamma + beta
//   gradients at the stored r, for an upstream dy (g = dy * gamma, xhat = (r - mu) * rstd):
//   dr = rstd (g - mean(g) - xhat mean(g xhat)) (+ the gradient that reaches r past the norm),
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy.
//
// Both passes read each row once into registers and take the mean first and the centred squares second, so
// no difference of large sums is formed.  Everything between the loads and the stores is fp32; y is
// normalised from the fp32 sum, not from the rounded r.  The backward pass takes the statistics again from
// the stored r: two more sums per row cost nothing next to the row's bytes, and no statistics are kept.
#include "block_common.cuh"

namespace swimba {

namespace {

constexpr int kMaxThreads = 512;  // per row; with at most 32 columns a thread that is 16384 columns

// Sum of two values over the block, the same in every thread.  `red` holds 2 x 32 float2; `which` alternates
// between calls so that one barrier per call is enough.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2 (*red)[32], int which) {
  a = warp_sum(a);
  b = warp_sum(b);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return make_float2(a, b);
  if ((threadIdx.x & 31) == 0) red[which][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 s = red[which][0];
  for (int w = 1; w < nw; ++w) {
    const float2 t = red[which][w];
    s.x += t.x;
    s.y += t.y;
  }
  return s;
}

// One row per block and iteration; thread i holds the vectors i, i + blockDim, ... of VEC columns.
template <class T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads)
layer_norm_kernel(int M, int D, long long xs, float eps, const T* __restrict__ x, const T* residual,
                  const float* __restrict__ gamma, const float* __restrict__ beta, T* y, T* r_out) {
  __shared__ float2 red[2][32];
  int which = 0;
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    float v[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
      if (c < D) {
        load_vec<T, VEC>(x + (size_t)m * xs + c, v[i]);
        if (residual) {
          float q[VEC];
          load_vec<T, VEC>(residual + (size_t)m * D + c, q);
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[i][j] += q[j];
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) s += v[i][j];
      }
    }
    const float mu = block_sum2(s, 0.f, red, which).x / D;
    which ^= 1;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * blockDim.x + threadIdx.x) * VEC < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) sq += (v[i][j] - mu) * (v[i][j] - mu);
      }
    const float rstd = rsqrtf(block_sum2(sq, 0.f, red, which).x / D + eps);
    which ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
      if (c < D) {
        if (r_out) store_vec<T, VEC>(r_out + (size_t)m * D + c, v[i]);
        float g[VEC], b[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) { g[j] = 1.f; b[j] = 0.f; }
        if (gamma) load_vec<float, VEC>(gamma + c, g);
        if (beta) load_vec<float, VEC>(beta + c, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = (v[i][j] - mu) * rstd * g[j] + b[j];
        store_vec<T, VEC>(y + (size_t)m * D + c, v[i]);
      }
    }
  }
}

// Gradients of rows blockIdx.x, blockIdx.x + gridDim.x, ...; the block's sums of dy xhat and dy go to
// part[blockIdx.x][2][D] when `part` is given.
template <class T, class G, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads)
layer_norm_bwd_kernel(int M, int D, float eps, const T* __restrict__ r, const float* __restrict__ gamma, const G* dy,
                      const G* dr, G* dx, float* __restrict__ part) {
  __shared__ float2 red[2][32];
  int which = 0;
  float ag[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) ag[i][j] = ab[i][j] = 0.f;
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    float v[NV][VEC], d[NV][VEC], gm[NV][VEC];
    float s = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) { v[i][j] = d[i][j] = 0.f; gm[i][j] = 1.f; }
      if (c < D) {
        load_vec<T, VEC>(r + (size_t)m * D + c, v[i]);
        load_vec<G, VEC>(dy + (size_t)m * D + c, d[i]);
        if (gamma) load_vec<float, VEC>(gamma + c, gm[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) { s += v[i][j]; sg += d[i][j] * gm[i][j]; }
      }
    }
    const float2 t1 = block_sum2(s, sg, red, which);
    which ^= 1;
    const float mu = t1.x / D, mg = t1.y / D;
    float sq = 0.f, sgc = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * blockDim.x + threadIdx.x) * VEC < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] -= mu;
          sq += v[i][j] * v[i][j];
          sgc += d[i][j] * gm[i][j] * v[i][j];
        }
      }
    const float2 t2 = block_sum2(sq, sgc, red, which);
    which ^= 1;
    const float rstd = rsqrtf(t2.x / D + eps), mgx = t2.y / D * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
      if (c < D) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = 0.f;
        if (dr) load_vec<G, VEC>(dr + (size_t)m * D + c, o);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = v[i][j] * rstd;
          o[j] += rstd * (d[i][j] * gm[i][j] - mg - xh * mgx);
          ag[i][j] += d[i][j] * xh;
          ab[i][j] += d[i][j];
        }
        store_vec<G, VEC>(dx + (size_t)m * D + c, o);
      }
    }
  }
  if (part) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
      if (c < D) {
        store_vec<float, VEC>(part + (size_t)blockIdx.x * 2 * D + c, ag[i]);
        store_vec<float, VEC>(part + (size_t)blockIdx.x * 2 * D + D + c, ab[i]);
      }
    }
  }
}

// dgamma and dbeta: sums over the P partial rows, in a fixed order.  A block covers 32 of the 2 D columns with 32
// threads for each.
__global__ void __launch_bounds__(1024)
layer_norm_params_kernel(int P, int D, const float* __restrict__ part, float* dgamma, float* dbeta) {
  __shared__ float sm[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < 2 * D)
    for (int p = threadIdx.y; p < P; p += 32) s += part[(size_t)p * 2 * D + c];
  sm[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < 2 * D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sm[i][threadIdx.x];
    if (c < D) {
      if (dgamma) dgamma[c] = t;
    } else if (dbeta) {
      dbeta[c - D] = t;
    }
  }
}

// Vectors per thread and threads per row for D columns in vectors of `vec`.
struct RowShape {
  int nv, threads;
};
RowShape row_shape(int D, int vec) {
  const int n = ceil_div(D, vec);
  int nv = 1;
  while (n > 128 * nv && nv * vec < 16) nv *= 2;
  while (n > kMaxThreads * nv) nv *= 2;
  return {nv, ceil_div(ceil_div(n, nv), 32) * 32};
}

// f(integral constant nv) for the vectors per thread that row_shape can choose (at most 32 columns).
template <int VEC, class F>
void with_nv(int nv, F f) {
  switch (nv) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: if constexpr (VEC <= 4) return f(std::integral_constant<int, 8>{}); break;
    case 16: if constexpr (VEC == 1) return f(std::integral_constant<int, 16>{}); break;
    case 32: if constexpr (VEC == 1) return f(std::integral_constant<int, 32>{}); break;
  }
}

// Row vectors are 16 bytes of the widest type that is read in them: D must keep every row aligned.
template <class T>
constexpr int full_vec() { return 16 / (int)sizeof(T); }
int bwd_vec(const NormDims& d) {
  const int v = d.dtype == SWIMBA_F32 ? 4 : 8;
  return d.D % v == 0 ? v : 1;
}
int bwd_blocks(const NormDims& d) {
  const RowShape s = row_shape(d.D, bwd_vec(d));
  int per_sm = 1024 / s.threads;
  per_sm = per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm;
  const int cap = 148 * per_sm;
  return d.M < cap ? d.M : cap;
}

template <class T, int VEC>
cudaError_t fwd_t(const NormDims& d, const void* x, const void* residual, const float* gamma, const float* beta, void* y,
                  void* r_out, cudaStream_t s) {
  const RowShape sh = row_shape(d.D, VEC);
  const int grid = d.M < (1 << 20) ? d.M : (1 << 20);
  auto go = [&](auto kernel) {
    kernel<<<grid, sh.threads, 0, s>>>(d.M, d.D, d.x_stride, d.eps, (const T*)x, (const T*)residual, gamma, beta, (T*)y,
                                       (T*)r_out);
  };
  with_nv<VEC>(sh.nv, [&](auto nv) { go(layer_norm_kernel<T, VEC, decltype(nv)::value>); });
  count_launches(1);
  return cudaGetLastError();
}

template <class T, class G, int VEC>
cudaError_t bwd_t(const NormDims& d, const void* r, const float* gamma, const void* dy, const void* dr, void* dx,
                  float* dgamma, float* dbeta, float* part, cudaStream_t s) {
  const RowShape sh = row_shape(d.D, VEC);
  const int grid = bwd_blocks(d);
  if (!dgamma && !dbeta) part = nullptr;
  auto go = [&](auto kernel) {
    kernel<<<grid, sh.threads, 0, s>>>(d.M, d.D, d.eps, (const T*)r, gamma, (const G*)dy, (const G*)dr, (G*)dx, part);
  };
  with_nv<VEC>(sh.nv, [&](auto nv) { go(layer_norm_bwd_kernel<T, G, VEC, decltype(nv)::value>); });
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (part) {
    layer_norm_params_kernel<<<ceil_div(2 * d.D, 32), dim3(32, 32), 0, s>>>(grid, d.D, part, dgamma, dbeta);
    count_launches(1);
  }
  return cudaGetLastError();
}

template <class T, class G>
cudaError_t bwd_v(const NormDims& d, const void* r, const float* gamma, const void* dy, const void* dr, void* dx,
                  float* dgamma, float* dbeta, float* part, cudaStream_t s) {
  constexpr int V = full_vec<T>();
  return bwd_vec(d) == V ? bwd_t<T, G, V>(d, r, gamma, dy, dr, dx, dgamma, dbeta, part, s)
                         : bwd_t<T, G, 1>(d, r, gamma, dy, dr, dx, dgamma, dbeta, part, s);
}

template <class T>
cudaError_t fwd_v(const NormDims& d, const void* x, const void* residual, const float* gamma, const float* beta, void* y,
                  void* r_out, cudaStream_t s) {
  constexpr int V = full_vec<T>();
  return d.D % V == 0 && d.x_stride % V == 0 ? fwd_t<T, V>(d, x, residual, gamma, beta, y, r_out, s)
                                             : fwd_t<T, 1>(d, x, residual, gamma, beta, y, r_out, s);
}

}  // namespace

size_t layer_norm_bwd_ws(const NormDims& d) { return align_up((size_t)bwd_blocks(d) * 2 * d.D * 4, 256); }

cudaError_t launch_layer_norm(const NormDims& d, const void* x, const void* residual, const float* gamma,
                              const float* beta, void* y, void* r_out, cudaStream_t s) {
  switch (d.dtype) {
    case SWIMBA_F32: return fwd_v<float>(d, x, residual, gamma, beta, y, r_out, s);
    case SWIMBA_BF16: return fwd_v<__nv_bfloat16>(d, x, residual, gamma, beta, y, r_out, s);
    default: return fwd_v<__half>(d, x, residual, gamma, beta, y, r_out, s);
  }
}

cudaError_t launch_layer_norm_bwd(const NormDims& d, const void* r, const float* gamma, const void* dy, const void* dr,
                                  void* dx, float* dgamma, float* dbeta, float* part, cudaStream_t s) {
  const bool g32 = d.grad_dtype == SWIMBA_F32;
  switch (d.dtype) {
    case SWIMBA_F32: return bwd_v<float, float>(d, r, gamma, dy, dr, dx, dgamma, dbeta, part, s);
    case SWIMBA_BF16:
      return g32 ? bwd_v<__nv_bfloat16, float>(d, r, gamma, dy, dr, dx, dgamma, dbeta, part, s)
                 : bwd_v<__nv_bfloat16, __nv_bfloat16>(d, r, gamma, dy, dr, dx, dgamma, dbeta, part, s);
    default:
      return g32 ? bwd_v<__half, float>(d, r, gamma, dy, dr, dx, dgamma, dbeta, part, s)
                 : bwd_v<__half, __half>(d, r, gamma, dy, dr, dx, dgamma, dbeta, part, s);
  }
}

}  // namespace swimba
