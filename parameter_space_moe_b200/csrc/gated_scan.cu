// The per-channel gated linear recurrence over a sequence, its gradients, and its single-token step.
//
//   f_t = sigmoid(gate_t),  h_t = f_t h_{t-1} + (1 - f_t) x_t          (every channel by itself; h_{-1} = init or 0)
//   gradients for an upstream dh (and dfinal on the last state), with the adjoint lambda:
//   lambda_t = dh_t + f_{t+1} lambda_{t+1},  dx_t = (1 - f_t) lambda_t,
//   dgate_t = lambda_t (h_{t-1} - x_t) f_t (1 - f_t),  dinit = f_0 lambda_0.
//
// A step is the linear map c -> a c + b of the carried value c (forward: a = f, b = (1 - f) x, c = h; backward,
// from the last token: a = f, b = f dh, c = f_{t+1} lambda_{t+1}), and maps compose: (a2, b2) after (a1, b1) is
// (a2 a1, a2 b1 + b2).  A cluster of CTAs owns 32 V columns of one sequence.  Per round it covers
// (CTAs x 8 warps x S) consecutive tokens: each warp composes the maps of its S tokens in registers, the warps'
// maps meet in shared memory, the CTAs' in distributed shared memory, and every warp then replays its tokens
// from its true carried value.  So each input is read once, the split along time needs no pass over memory, no
// workspace and no waiting between clusters, and sums run in a fixed order.  All in fp32.
#include "block_common.cuh"
#include "tc_common.cuh"

namespace swimba {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxCluster = 8;

// The maps of a round: this CTA's warps and, by CTA rank, the cluster's CTAs.  Two copies, used in turn, so that
// one barrier separates a round's writes from its reads.
template <int V>
struct Maps {
  float2 warp[2][kWarps][32 * V];
  float2 cta[2][kMaxCluster][32 * V];
};

// 16 bytes global -> shared, zeros where !ok.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void compose(float2& m, float2 later) {
  m.y = fmaf(later.x, m.y, later.y);
  m.x *= later.x;
}

// Given this warp's map `mine` of the round, returns the carried value in front of the warp's first token and
// advances `carry` over the whole round.
template <int V>
__device__ __forceinline__ void exchange(Maps<V>& sm, int buf, int warp, int lane, uint32_t rank, uint32_t nrank,
                                         const float2 (&mine)[V], float (&carry)[V], float (&start)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) sm.warp[buf][warp][32 * v + lane] = mine[v];
  __syncthreads();
  float2 before[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float2 m = make_float2(1.f, 0.f);
    before[v] = m;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) before[v] = m;
      compose(m, sm.warp[buf][w][32 * v + lane]);
    }
    if (nrank == 1) {
      start[v] = fmaf(before[v].x, carry[v], before[v].y);
      carry[v] = fmaf(m.x, carry[v], m.y);
    } else if (warp < (int)nrank) {  // warp w tells CTA w this CTA's map
      const uint32_t to = tc::map_shared(tc::smem_u32(&sm.cta[buf][rank][32 * v + lane]), (uint32_t)warp);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m.x), "f"(m.y) : "memory");
    }
  }
  if (nrank == 1) return;
  tc::cluster_sync();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float c = carry[v];
    for (uint32_t r = 0; r < nrank; ++r) {
      if (r == rank) start[v] = fmaf(before[v].x, c, before[v].y);
      const float2 m = sm.cta[buf][r][32 * v + lane];
      c = fmaf(m.x, c, m.y);
    }
    carry[v] = c;
  }
}

// One warp's tokens of one input, from a stage in shared memory or from registers: 32 V columns of S rows.
template <class T, int V, int S, bool kAsync>
struct Rows {
  static constexpr int kRowBytes = 32 * V * (int)sizeof(T);
  static constexpr int kBytes = S * kRowBytes;
  T raw[kAsync ? 1 : S][V];

  // Starts reading rows first, first + dir, ... (those inside [0, n) and in live columns); row r at p + r * stride.
  __device__ __forceinline__ void fetch(uint8_t* stage, const T* p, size_t stride, int first, int dir, int n, int col0,
                                        int W, int lane) {
    if constexpr (kAsync) {
      constexpr int kChunks = kRowBytes / 16, kPer = 16 / (int)sizeof(T);
      const int c = lane % kChunks, col = col0 + c * kPer;
#pragma unroll
      for (int k = 0; k < S * kChunks / 32; ++k) {
        const int row = k * (32 / kChunks) + lane / kChunks, t = first + dir * row;
        const bool ok = t >= 0 && t < n && col < W;
        cp_async16(stage + row * kRowBytes + c * 16, ok ? p + t * stride + col : p, ok);
      }
    } else {
      const int col = col0 + V * lane;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int t = first + dir * i;
        if (t >= 0 && t < n && col < W) {
#pragma unroll
          for (int v = 0; v < V; ++v) raw[i][v] = p[t * stride + col + v];
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) raw[i][v] = from_f32<T>(0.f);
        }
      }
    }
  }
  __device__ __forceinline__ void get(const uint8_t* stage, int i, int lane, float (&out)[V]) const {
    if constexpr (kAsync) {
      load_vec<T, V>(reinterpret_cast<const T*>(stage + i * kRowBytes) + V * lane, out);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = to_f32(raw[i][v]);
    }
  }
};

template <class T, int V, int S, bool kAsync>
__global__ void __launch_bounds__(32 * kWarps, 2)
gated_scan_kernel(int T_, int W, int ngrp, long long xs, long long gs, const T* __restrict__ x,
                  const T* __restrict__ gate, const float* init, T* __restrict__ h, float* final_state) {
  using R = Rows<T, V, S, kAsync>;
  extern __shared__ __align__(16) uint8_t dyn[];
  Maps<V>& sm = *reinterpret_cast<Maps<V>*>(dyn);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* stages = dyn + sizeof(Maps<V>) + warp * (2 * R::kBytes);
  constexpr int kStride = kWarps * 2 * R::kBytes;  // between stages
  uint32_t rank, nrank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nrank));
  const int grp = blockIdx.x / (int)nrank;
  const int b = grp / ngrp, col0 = (grp % ngrp) * 32 * V, col = col0 + V * lane;
  const bool live = col < W;  // V divides W where V > 1
  const size_t row0 = (size_t)b * T_;
  x += row0 * xs;
  gate += row0 * gs;
  h += row0 * W;
  const int span = (int)nrank * kWarps * S;
  R rx, rg;
  auto fetch = [&](int t0, int st) {
    const int t = t0 + ((int)rank * kWarps + warp) * S;
    rx.fetch(stages + st * kStride, x, xs, t, 1, T_, col0, W, lane);
    rg.fetch(stages + st * kStride + R::kBytes, gate, gs, t, 1, T_, col0, W, lane);
    cp_async_commit();
  };
  fetch(0, 0);
  if (kAsync) fetch(span, 1);
  float carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = init && live ? init[(size_t)b * W + col + v] : 0.f;
  if (nrank > 1) tc::cluster_sync();  // every CTA runs before another writes to its shared memory
  int buf = 0, st = 0;
  for (int t0 = 0; t0 < T_; t0 += span, buf ^= 1) {
    const int t = t0 + ((int)rank * kWarps + warp) * S;
    if (kAsync) {
      // the stage read in the last round (a block barrier ago) takes the round after next
      fetch(t0 + 2 * span, st == 0 ? 2 : st - 1);
      cp_async_wait<2>();
      __syncwarp();
    }
    float f[S][V], q[S][V];
    float2 mine[V];
#pragma unroll
    for (int v = 0; v < V; ++v) mine[v] = make_float2(1.f, 0.f);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float xv[V], gv[V];
      rx.get(stages + st * kStride, i, lane, xv);
      rg.get(stages + st * kStride + R::kBytes, i, lane, gv);
      const bool in = t + i < T_;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gate_pair(gv[v], f[i][v], q[i][v]);
        f[i][v] = in ? f[i][v] : 1.f;
        q[i][v] = in ? q[i][v] * xv[v] : 0.f;
        compose(mine[v], make_float2(f[i][v], q[i][v]));
      }
    }
    if (!kAsync) fetch(t0 + span, 0);
    float c[V];
    exchange<V>(sm, buf, warp, lane, rank, nrank, mine, carry, c);
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = fmaf(f[i][v], c[v], q[i][v]);
      if (live && t + i < T_) store_vec<T, V>(h + (size_t)(t + i) * W + col, c);
    }
    st = st == 2 ? 0 : st + 1;
  }
  cp_async_wait<0>();
  if (final_state && live && rank == 0 && warp == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) final_state[(size_t)b * W + col + v] = carry[v];
  }
}

// Token index tau counts from the last token: t = T - 1 - tau.
template <class T, class G, int V, int S, bool kAsync>
__global__ void __launch_bounds__(32 * kWarps, 2)
gated_scan_bwd_kernel(int T_, int W, int ngrp, long long xs, long long gs, const T* __restrict__ x,
                      const T* __restrict__ gate, const T* __restrict__ h, const float* init, const G* __restrict__ dh,
                      const float* dfinal, G* __restrict__ dx, G* __restrict__ dgate, float* dinit) {
  using R = Rows<T, V, S, kAsync>;
  using RG = Rows<G, V, S, kAsync>;
  constexpr int kWarpBytes = 3 * R::kBytes + RG::kBytes, kStride = kWarps * kWarpBytes;
  extern __shared__ __align__(16) uint8_t dyn[];
  Maps<V>& sm = *reinterpret_cast<Maps<V>*>(dyn);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* stages = dyn + sizeof(Maps<V>) + warp * kWarpBytes;
  uint32_t rank, nrank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nrank));
  const int grp = blockIdx.x / (int)nrank;
  const int b = grp / ngrp, col0 = (grp % ngrp) * 32 * V, col = col0 + V * lane;
  const bool live = col < W;
  const size_t row0 = (size_t)b * T_;
  x += row0 * xs;
  gate += row0 * gs;
  h += row0 * W;
  dh += row0 * W;
  dx += row0 * W;
  dgate += row0 * W;
  const int span = (int)nrank * kWarps * S;
  R rx, rg, rh;
  RG rd;
  auto fetch = [&](int u0, int st) {
    const int t = T_ - 1 - (u0 + ((int)rank * kWarps + warp) * S);
    uint8_t* p = stages + st * kStride;
    rg.fetch(p, gate, gs, t, -1, T_, col0, W, lane);
    rx.fetch(p + R::kBytes, x, xs, t, -1, T_, col0, W, lane);
    rh.fetch(p + 2 * R::kBytes, h, W, t - 1, -1, T_, col0, W, lane);
    rd.fetch(p + 3 * R::kBytes, dh, W, t, -1, T_, col0, W, lane);
    cp_async_commit();
  };
  fetch(0, 0);
  if (kAsync) fetch(span, 1);
  float carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = dfinal && live ? dfinal[(size_t)b * W + col + v] : 0.f;
  if (nrank > 1) tc::cluster_sync();  // every CTA runs before another writes to its shared memory
  int buf = 0, st = 0;
  for (int u0 = 0; u0 < T_; u0 += span, buf ^= 1) {
    const int u = u0 + ((int)rank * kWarps + warp) * S;
    if (kAsync) {
      fetch(u0 + 2 * span, st == 0 ? 2 : st - 1);
      cp_async_wait<2>();
      __syncwarp();
    }
    const uint8_t* p = stages + st * kStride;
    float f[S][V], q[S][V], d[S][V], e[S][V];  // e = h_{t-1} - x_t
    float2 mine[V];
#pragma unroll
    for (int v = 0; v < V; ++v) mine[v] = make_float2(1.f, 0.f);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int t = T_ - 1 - (u + i);
      float xv[V], gv[V], hv[V];
      rg.get(p, i, lane, gv);
      rx.get(p + R::kBytes, i, lane, xv);
      rh.get(p + 2 * R::kBytes, i, lane, hv);
      rd.get(p + 3 * R::kBytes, i, lane, d[i]);
      if (t == 0 && init && live) {
#pragma unroll
        for (int v = 0; v < V; ++v) hv[v] = init[(size_t)b * W + col + v];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gate_pair(gv[v], f[i][v], q[i][v]);
        f[i][v] = t >= 0 ? f[i][v] : 1.f;
        d[i][v] = t >= 0 ? d[i][v] : 0.f;
        e[i][v] = hv[v] - xv[v];
        compose(mine[v], make_float2(f[i][v], f[i][v] * d[i][v]));
      }
    }
    if (!kAsync) fetch(u0 + span, 0);
    float c[V];
    exchange<V>(sm, buf, warp, lane, rank, nrank, mine, carry, c);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int t = T_ - 1 - (u + i);
      float ox[V], og[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float lam = d[i][v] + c[v];
        c[v] = f[i][v] * lam;
        ox[v] = q[i][v] * lam;
        og[v] = c[v] * q[i][v] * e[i][v];
      }
      if (live && t >= 0) {
        store_vec<G, V>(dx + (size_t)t * W + col, ox);
        store_vec<G, V>(dgate + (size_t)t * W + col, og);
      }
    }
    st = st == 2 ? 0 : st + 1;
  }
  cp_async_wait<0>();
  if (dinit && live && rank == 0 && warp == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) dinit[(size_t)b * W + col + v] = carry[v];
  }
}

// One token of every sequence: state <- f state + (1 - f) x, h = state.
template <class T, int V>
__global__ void __launch_bounds__(256)
gated_step_kernel(int B, int W, long long xs, long long gs, const T* __restrict__ x, const T* __restrict__ gate,
                  float* __restrict__ state, T* __restrict__ h) {
  const int per_row = W / V;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < (long long)B * per_row;
       i += (long long)gridDim.x * blockDim.x) {
    const int b = (int)(i / per_row), col = (int)(i % per_row) * V;
    float xv[V], gv[V], sv[V];
    load_vec<T, V>(x + b * xs + col, xv);
    load_vec<T, V>(gate + b * gs + col, gv);
    load_vec<float, V>(state + (size_t)b * W + col, sv);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f, q;
      gate_pair(gv[v], f, q);
      sv[v] = fmaf(f, sv[v], q * xv[v]);
    }
    store_vec<float, V>(state + (size_t)b * W + col, sv);
    store_vec<T, V>(h + (size_t)b * W + col, sv);
  }
}

// CTAs per cluster: as many as the resident CTAs (two per SM) allow all columns' clusters at once, but none without a
// round of its own.
int cluster_size(const GatedDims& d, int groups, int round_tokens) {
  const int c = 2 * 148 / groups, most = ceil_div(d.T, round_tokens);
  return c < 1 ? 1 : (c < most ? c : most) < kMaxCluster ? (c < most ? c : most) : kMaxCluster;
}

template <class K, class... A>
cudaError_t launch_cluster(K kernel, int groups, int c, size_t smem, cudaStream_t s, A... a) {
  cudaError_t e = set_max_dynamic_smem((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * c));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a...);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <class T, int V, int S, bool kAsync>
cudaError_t fwd_t(const GatedDims& d, const void* x, const void* gate, const float* init, void* h, float* fin,
                  cudaStream_t s) {
  const int ngrp = ceil_div(d.W, 32 * V), groups = d.B * ngrp;
  const size_t smem = sizeof(Maps<V>) + (kAsync ? 3 * kWarps * 2 * Rows<T, V, S, kAsync>::kBytes : 0);
  return launch_cluster(gated_scan_kernel<T, V, S, kAsync>, groups, cluster_size(d, groups, kWarps * S), smem, s, d.T, d.W,
                        ngrp, d.x_stride, d.gate_stride, (const T*)x, (const T*)gate, init, (T*)h, fin);
}

template <class T, class G, int V, int S, bool kAsync>
cudaError_t bwd_t(const GatedDims& d, const void* x, const void* gate, const void* h, const float* init, const void* dh,
                  const float* dfinal, void* dx, void* dgate, float* dinit, cudaStream_t s) {
  const int ngrp = ceil_div(d.W, 32 * V), groups = d.B * ngrp;
  const size_t smem = sizeof(Maps<V>) + (kAsync ? 3 * kWarps * (3 * Rows<T, V, S, kAsync>::kBytes + Rows<G, V, S, kAsync>::kBytes) : 0);
  return launch_cluster(gated_scan_bwd_kernel<T, G, V, S, kAsync>, groups, cluster_size(d, groups, kWarps * S), smem, s,
                        d.T, d.W, ngrp, d.x_stride, d.gate_stride, (const T*)x, (const T*)gate, (const T*)h, init,
                        (const G*)dh, dfinal, (G*)dx, (G*)dgate, dinit);
}

// Rows whose 16-byte chunks are aligned in every tensor: they are copied to shared memory, three rounds deep.
bool aligned_rows(const GatedDims& d) {
  const int q = d.dtype == SWIMBA_F32 ? 4 : 8;
  return d.W % q == 0 && d.x_stride % q == 0 && d.gate_stride % q == 0;
}

#ifndef SF
#define SF 16
#define SB 8
#endif
template <class T>
cudaError_t fwd_v(const GatedDims& d, const void* x, const void* gate, const float* init, void* h, float* fin,
                  cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? SF : SF / 2;
  return aligned_rows(d) ? fwd_t<T, 2, S, true>(d, x, gate, init, h, fin, s) : fwd_t<T, 1, 16, false>(d, x, gate, init, h, fin, s);
}

template <class T, class G>
cudaError_t bwd_v(const GatedDims& d, const void* x, const void* gate, const void* h, const float* init, const void* dh,
                  const float* dfinal, void* dx, void* dgate, float* dinit, cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? SB : SB / 2;
  return aligned_rows(d) ? bwd_t<T, G, 2, S, true>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, s)
                         : bwd_t<T, G, 1, 8, false>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, s);
}

template <class T>
cudaError_t step_t(const GatedDims& d, const void* x, const void* gate, float* state, void* h, cudaStream_t s) {
  const bool vec = d.W % 4 == 0 && d.x_stride % 4 == 0 && d.gate_stride % 4 == 0;
  const long long n = (long long)d.B * d.W / (vec ? 4 : 1);
  const long long want = (n + 255) / 256;
  const int grid = (int)(want < 148 * 8 ? want : 148 * 8);
  if (vec)
    gated_step_kernel<T, 4><<<grid, 256, 0, s>>>(d.B, d.W, d.x_stride, d.gate_stride, (const T*)x, (const T*)gate,
                                                 state, (T*)h);
  else
    gated_step_kernel<T, 1><<<grid, 256, 0, s>>>(d.B, d.W, d.x_stride, d.gate_stride, (const T*)x, (const T*)gate,
                                                 state, (T*)h);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_scan(const GatedDims& d, const void* x, const void* gate, const float* init, void* h,
                              float* fin, cudaStream_t s) {
  switch (d.dtype) {
    case SWIMBA_F32: return fwd_v<float>(d, x, gate, init, h, fin, s);
    case SWIMBA_BF16: return fwd_v<__nv_bfloat16>(d, x, gate, init, h, fin, s);
    default: return fwd_v<__half>(d, x, gate, init, h, fin, s);
  }
}

cudaError_t launch_gated_scan_bwd(const GatedDims& d, const void* x, const void* gate, const void* h, const float* init,
                                  const void* dh, const float* dfinal, void* dx, void* dgate, float* dinit,
                                  cudaStream_t s) {
  const bool g32 = d.grad_dtype == SWIMBA_F32;
  switch (d.dtype) {
    case SWIMBA_F32: return bwd_v<float, float>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, s);
    case SWIMBA_BF16:
      return g32 ? bwd_v<__nv_bfloat16, float>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, s)
                 : bwd_v<__nv_bfloat16, __nv_bfloat16>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, s);
    default:
      return g32 ? bwd_v<__half, float>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, s)
                 : bwd_v<__half, __half>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, s);
  }
}

cudaError_t launch_gated_step(const GatedDims& d, const void* x, const void* gate, float* state, void* h,
                              cudaStream_t s) {
  switch (d.dtype) {
    case SWIMBA_F32: return step_t<float>(d, x, gate, state, h, s);
    case SWIMBA_BF16: return step_t<__nv_bfloat16>(d, x, gate, state, h, s);
    default: return step_t<__half>(d, x, gate, state, h, s);
  }
}

}  // namespace swimba
