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
// (CTAs x kWarps x S) consecutive tokens: each warp composes the maps of its S tokens in registers, the warps'
// maps meet in shared memory, the CTAs' in distributed shared memory (asynchronous stores counted on an mbarrier: a
// cluster barrier would first wait for the round's stores of h), and every warp then replays its tokens from its true
// carried value.  So each input is read once, the split along time needs no pass over memory, no workspace and no
// waiting between clusters, and sums run in a fixed order.  All in fp32, pairs of columns by two-wide instructions.
#include <atomic>

#include "block_common.cuh"
#include "tc_common.cuh"

namespace swimba {

namespace {

#ifndef KW
#define KW 4
#define KST 3
#endif
constexpr int kWarps = KW, kStages = KST;
constexpr int kMaxCluster = 8;

// Two-wide fp32 arithmetic for pairs of columns.
__device__ __forceinline__ unsigned long long f2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void un2(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
template <int V>
struct Vec {
  float v[V];
};
template <int V>
__device__ __forceinline__ Vec<V> operator*(const Vec<V>& a, const Vec<V>& b) {
  Vec<V> r;
  if constexpr (V == 2) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2(a.v[0], a.v[1])), "l"(f2(b.v[0], b.v[1])));
    un2(d, r.v[0], r.v[1]);
  } else {
    r.v[0] = a.v[0] * b.v[0];
  }
  return r;
}
template <int V>
__device__ __forceinline__ Vec<V> operator+(const Vec<V>& a, const Vec<V>& b) {
  Vec<V> r;
  if constexpr (V == 2) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2(a.v[0], a.v[1])), "l"(f2(b.v[0], b.v[1])));
    un2(d, r.v[0], r.v[1]);
  } else {
    r.v[0] = a.v[0] + b.v[0];
  }
  return r;
}
template <int V>
__device__ __forceinline__ Vec<V> fma(const Vec<V>& a, const Vec<V>& b, const Vec<V>& c) {
  Vec<V> r;
  if constexpr (V == 2) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(f2(a.v[0], a.v[1])), "l"(f2(b.v[0], b.v[1])), "l"(f2(c.v[0], c.v[1])));
    un2(d, r.v[0], r.v[1]);
  } else {
    r.v[0] = fmaf(a.v[0], b.v[0], c.v[0]);
  }
  return r;
}
template <int V>
__device__ __forceinline__ Vec<V> all(float x) {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = x;
  return r;
}

// gate_pair for V columns.
template <int V>
__device__ __forceinline__ void gates(const Vec<V>& g, Vec<V>& f, Vec<V>& q) {
  Vec<V> e, r;
#pragma unroll
  for (int i = 0; i < V; ++i) e.v[i] = exp_fast(-fabsf(g.v[i]));
  const Vec<V> d = e + all<V>(1.f);
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = rcp_fast(d.v[i]);
  const Vec<V> small = e * r, large = fma(small, all<V>(-1.f), all<V>(1.f));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool open = g.v[i] >= 0.f;
    f.v[i] = open ? large.v[i] : small.v[i];
    q.v[i] = open ? small.v[i] : large.v[i];
  }
}

// The map of some consecutive steps, for a lane's V columns.
template <int V>
struct Map {
  Vec<V> a, b;
};
template <int V>
__device__ __forceinline__ void then(Map<V>& m, const Vec<V>& a, const Vec<V>& b) {
  m.b = fma(a, m.b, b);
  m.a = a * m.a;
}

// A round's maps: this CTA's warps and, by CTA rank, the cluster's CTAs.  Two copies, used in turn: a warp writes a copy
// again two rounds later, after a block barrier (or, from another CTA, after this CTA's map of the round between) that
// follows every read of it.
template <int V>
struct alignas(16) Maps {
  Map<V> warp[2][kWarps][32];
  Map<V> cta[2][kMaxCluster][32];
  uint64_t bar[2];
};

// Waits for the mbarrier's phase with acquire at cluster scope; false if it gave up.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < tc::kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}

// Every thread, before the first round.
template <int V>
__device__ __forceinline__ void exchange_init(Maps<V>& sm, uint32_t nrank) {
  if (nrank == 1) return;
  if (threadIdx.x == 0) {
    tc::mbar_init(&sm.bar[0], 1);
    tc::mbar_init(&sm.bar[1], 1);
    tc::fence_barrier_init();
  }
  tc::cluster_sync();  // every CTA runs, its barriers initialised, before another stores to its shared memory
}

// Given this warp's map of round `round`, returns the carried value in front of the warp's first token and advances
// `carry` over the whole round.
template <int V>
__device__ __forceinline__ Vec<V> exchange(Maps<V>& sm, int round, int warp, int lane, uint32_t rank, uint32_t nrank,
                                           const Map<V>& mine, Vec<V>& carry, unsigned* st) {
  const int buf = round & 1;
  sm.warp[buf][warp][lane] = mine;
  if (nrank > 1 && threadIdx.x == 0) tc::mbar_arrive_expect_tx(&sm.bar[buf], nrank * 32 * (uint32_t)sizeof(Map<V>));
  __syncthreads();
  Map<V> before;
  before.a = all<V>(1.f);
  before.b = all<V>(0.f);
#pragma unroll
  for (int w = 0; w < kWarps - 1; ++w)
    if (w < warp) {
      const Map<V> m = sm.warp[buf][w][lane];
      then(before, m.a, m.b);
    }
  if (nrank == 1) {
    const Vec<V> start = fma(before.a, carry, before.b);
    carry = fma(mine.a, start, mine.b);
#pragma unroll
    for (int w = 1; w < kWarps; ++w)
      if (w > warp) {
        const Map<V> m = sm.warp[buf][w][lane];
        carry = fma(m.a, carry, m.b);
      }
    return start;
  }
  if (warp == kWarps - 1) {
    Map<V> whole = before;
    then(whole, mine.a, mine.b);
    const uint32_t at = tc::smem_u32(&sm.cta[buf][rank][lane]), bar = tc::smem_u32(&sm.bar[buf]);
    for (uint32_t r = 0; r < nrank; ++r) {
      const uint32_t to = tc::map_shared(at, r), on = tc::map_shared(bar, r);
      if constexpr (V == 2)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                     "f"(whole.a.v[0]), "f"(whole.a.v[1]), "f"(whole.b.v[0]), "f"(whole.b.v[1]), "r"(on)
                     : "memory");
      else
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
                     "f"(whole.a.v[0]), "f"(whole.b.v[0]), "r"(on)
                     : "memory");
    }
  }
  if (!wait_cluster(&sm.bar[buf], (uint32_t)(round >> 1) & 1u)) atomicOr(st, ST_TIMEOUT);
  Vec<V> c = carry, start = carry;
  for (uint32_t r = 0; r < nrank; ++r) {
    if (r == rank) start = fma(before.a, c, before.b);
    const Map<V> m = sm.cta[buf][r][lane];
    c = fma(m.a, c, m.b);
  }
  carry = c;
  return start;
}

// 16 bytes global -> shared.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// One warp's tokens of one input, from a stage in shared memory or from registers: 32 V columns of S rows.
template <class T, int V, int S, bool kAsync>
struct Rows {
  static constexpr int kRowBytes = 32 * V * (int)sizeof(T);
  static constexpr int kBytes = S * kRowBytes;
  [[maybe_unused]] static constexpr int kChunks = kRowBytes / 16, kStep = 32 / kChunks;  // lanes per row, rows per copy
  T raw[kAsync ? 1 : S][V];

  // Starts reading rows first, first + dir, ..., those inside [0, n); row r's columns at p + r * stride.
  __device__ __forceinline__ void fetch(uint8_t* stage, const T* p, long long stride, int first, int dir, int n, int col0,
                                        int W, int lane) {
    if constexpr (kAsync) {
      const int c = lane % kChunks, row = lane / kChunks, col = col0 + c * (16 / (int)sizeof(T));
      uint8_t* to = stage + row * kRowBytes + c * 16;
      const int t = first + dir * row, last = first + dir * (S - 1);
      const T* from = p + t * stride + col;
      const long long step = dir * kStep * stride;
      if (col >= W) return;
      if (first >= 0 && first < n && last >= 0 && last < n) {
#pragma unroll
        for (int k = 0; k < S / kStep; ++k) cp_async16(to + k * kStep * kRowBytes, from + k * step);
      } else {
#pragma unroll
        for (int k = 0; k < S / kStep; ++k)
          if (t + dir * k * kStep >= 0 && t + dir * k * kStep < n) cp_async16(to + k * kStep * kRowBytes, from + k * step);
      }
    } else {
      const int col = col0 + V * lane;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int t = first + dir * i;
#pragma unroll
        for (int v = 0; v < V; ++v) raw[i][v] = t >= 0 && t < n && col < W ? p[t * stride + col + v] : from_f32<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ Vec<V> get(const uint8_t* stage, int i, int lane) const {
    Vec<V> out;
    if constexpr (kAsync) {
      load_vec<T, V>(reinterpret_cast<const T*>(stage + i * kRowBytes) + V * lane, out.v);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) out.v[v] = to_f32(raw[i][v]);
    }
    return out;
  }
};

template <int V>
__device__ __forceinline__ Vec<V> load_state(const float* p, size_t at, bool live) {
  Vec<V> r = all<V>(0.f);
  if (p && live) {
#pragma unroll
    for (int v = 0; v < V; ++v) r.v[v] = p[at + v];
  }
  return r;
}

template <class T, int V, int S, bool kAsync>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps)
gated_scan_kernel(int T_, int W, int ngrp, long long xs, long long gs, const T* __restrict__ x,
                  const T* __restrict__ gate, const float* init, T* __restrict__ h, float* final_state, unsigned* status) {
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
  const size_t row0 = (size_t)b * T_, state = (size_t)b * W + col;
  x += row0 * xs;
  gate += row0 * gs;
  h += row0 * W + col;
  const int span = (int)nrank * kWarps * S;
  R rx, rg;
  int t = ((int)rank * kWarps + warp) * S;
  auto fetch = [&](int t, int st) {
    rx.fetch(stages + st * kStride, x, xs, t, 1, T_, col0, W, lane);
    rg.fetch(stages + st * kStride + R::kBytes, gate, gs, t, 1, T_, col0, W, lane);
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < (kAsync ? kStages - 1 : 1); ++k) fetch(t + k * span, k);
  Vec<V> carry = load_state<V>(init, state, live);
  exchange_init(sm, nrank);
  int st = 0;
  for (int round = 0; round * span < T_; ++round, t += span) {
    if (kAsync) {
      // the stage that the last round read (a block barrier ago) is filled next
      fetch(t + (kStages - 1) * span, st == 0 ? kStages - 1 : st - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
    }
    Vec<V> f[S], q[S];
    Map<V> mine;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      gates(rg.get(stages + st * kStride + R::kBytes, i, lane), f[i], q[i]);
      q[i] = q[i] * rx.get(stages + st * kStride, i, lane);
    }
    if (t + S > T_) {
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (t + i >= T_) { f[i] = all<V>(1.f); q[i] = all<V>(0.f); }
    }
    mine.a = f[0];
    mine.b = q[0];
#pragma unroll
    for (int i = 1; i < S; ++i) then(mine, f[i], q[i]);
    if (!kAsync) fetch(t + span, 0);
    Vec<V> c = exchange(sm, round, warp, lane, rank, nrank, mine, carry, status);
    T* out = h + (size_t)t * W;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      c = fma(f[i], c, q[i]);
      if (live && t + i < T_) store_vec<T, V>(out + (size_t)i * W, c.v);
    }
    st = st == kStages - 1 ? 0 : st + 1;
  }
  cp_async_wait<0>();
  if (final_state && live && rank == 0 && warp == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) final_state[state + v] = carry.v[v];
  }
  if (nrank > 1) tc::cluster_sync();  // no CTA leaves while another may still store to it
}

// Token index tau counts from the last token: t = T - 1 - tau.
template <class T, class G, int V, int S, bool kAsync>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps)
gated_scan_bwd_kernel(int T_, int W, int ngrp, long long xs, long long gs, const T* __restrict__ x,
                      const T* __restrict__ gate, const T* __restrict__ h, const float* init, const G* __restrict__ dh,
                      const float* dfinal, G* __restrict__ dx, G* __restrict__ dgate, float* dinit, unsigned* status) {
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
  const size_t row0 = (size_t)b * T_, state = (size_t)b * W + col;
  x += row0 * xs;
  gate += row0 * gs;
  h += row0 * W;
  dh += row0 * W;
  dx += row0 * W + col;
  dgate += row0 * W + col;
  const int span = (int)nrank * kWarps * S;
  R rx, rg, rh;
  RG rd;
  int t = T_ - 1 - ((int)rank * kWarps + warp) * S;  // the warp's first (last) token
  auto fetch = [&](int t, int st) {
    uint8_t* p = stages + st * kStride;
    rg.fetch(p, gate, gs, t, -1, T_, col0, W, lane);
    rx.fetch(p + R::kBytes, x, xs, t, -1, T_, col0, W, lane);
    rh.fetch(p + 2 * R::kBytes, h, W, t - 1, -1, T_, col0, W, lane);
    rd.fetch(p + 3 * R::kBytes, dh, W, t, -1, T_, col0, W, lane);
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < (kAsync ? kStages - 1 : 1); ++k) fetch(t - k * span, k);
  Vec<V> carry = load_state<V>(dfinal, state, live);
  exchange_init(sm, nrank);
  int st = 0;
  for (int round = 0; round * span < T_; ++round, t -= span) {
    if (kAsync) {
      fetch(t - (kStages - 1) * span, st == 0 ? kStages - 1 : st - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
    }
    const uint8_t* p = stages + st * kStride;
    Vec<V> f[S], q[S], d[S], e[S];  // e = h_{t-1} - x_t
    Map<V> mine;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      gates(rg.get(p, i, lane), f[i], q[i]);
      d[i] = rd.get(p + 3 * R::kBytes, i, lane);
      e[i] = fma(rx.get(p + R::kBytes, i, lane), all<V>(-1.f), rh.get(p + 2 * R::kBytes, i, lane));
    }
    if (t - S < 0) {  // the sequence's first token, whose state before it is init, and what would lie in front of it
#pragma unroll
      for (int i = 0; i < S; ++i) {
        if (t - i == 0) e[i] = fma(rx.get(p + R::kBytes, i, lane), all<V>(-1.f), load_state<V>(init, state, live));
        if (t - i < 0) { f[i] = all<V>(1.f); d[i] = all<V>(0.f); }
      }
    }
    mine.a = f[0];
    mine.b = f[0] * d[0];
#pragma unroll
    for (int i = 1; i < S; ++i) then(mine, f[i], f[i] * d[i]);
    if (!kAsync) fetch(t - span, 0);
    Vec<V> c = exchange(sm, round, warp, lane, rank, nrank, mine, carry, status);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const Vec<V> lam = d[i] + c;
      c = f[i] * lam;
      const Vec<V> ox = q[i] * lam, og = c * q[i] * e[i];
      if (live && t - i >= 0) {
        store_vec<G, V>(dx + (size_t)(t - i) * W, ox.v);
        store_vec<G, V>(dgate + (size_t)(t - i) * W, og.v);
      }
    }
    st = st == kStages - 1 ? 0 : st + 1;
  }
  cp_async_wait<0>();
  if (dinit && live && rank == 0 && warp == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) dinit[state + v] = carry.v[v];
  }
  if (nrank > 1) tc::cluster_sync();
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

// CTAs per cluster: of the sizes that leave no CTA without a round, the one with the fewest rounds in a row, counting
// the clusters that can be resident at once (asked once per kernel: GPCs of uneven size hold fewer CTAs in larger
// clusters, and one cluster too many takes as long as a second set).
struct Resident {
  std::atomic<int> clusters[kMaxCluster + 1];
};
template <class K>
int cluster_size(K kernel, Resident& seen, const GatedDims& d, int groups, int round_tokens, size_t smem) {
  const int rounds = ceil_div(d.T, round_tokens);
  int best = 1;
  long long best_cost = 0;
  for (int c = 1; c <= kMaxCluster && c <= rounds; ++c) {
    int n = seen.clusters[c].load(std::memory_order_relaxed);
    if (n == 0) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)c * 1024);
      cfg.blockDim = dim3(32 * kWarps);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)c;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = 1;
      }
      seen.clusters[c].store(n, std::memory_order_relaxed);
    }
    const long long cost = (long long)ceil_div(groups, n) * ceil_div(rounds, c);
    if (c == 1 || cost < best_cost) { best = c; best_cost = cost; }
  }
  return best;
}

template <class K, class... A>
cudaError_t launch_cluster(K kernel, Resident& seen, const GatedDims& d, int groups, int round_tokens, size_t smem,
                           cudaStream_t s, A... a) {
  cudaError_t e = set_max_dynamic_smem((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  const int c = cluster_size(kernel, seen, d, groups, round_tokens, smem);
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
cudaError_t fwd_t(const GatedDims& d, const void* x, const void* gate, const float* init, void* h, float* fin, unsigned* st,
                  cudaStream_t s) {
  static Resident seen;
  const int ngrp = ceil_div(d.W, 32 * V);
  const size_t smem = sizeof(Maps<V>) + (kAsync ? kStages * kWarps * 2 * Rows<T, V, S, kAsync>::kBytes : 0);
  return launch_cluster(gated_scan_kernel<T, V, S, kAsync>, seen, d, d.B * ngrp, kWarps * S, smem, s, d.T, d.W, ngrp,
                        d.x_stride, d.gate_stride, (const T*)x, (const T*)gate, init, (T*)h, fin, st);
}

template <class T, class G, int V, int S, bool kAsync>
cudaError_t bwd_t(const GatedDims& d, const void* x, const void* gate, const void* h, const float* init, const void* dh,
                  const float* dfinal, void* dx, void* dgate, float* dinit, unsigned* st, cudaStream_t s) {
  static Resident seen;
  const int ngrp = ceil_div(d.W, 32 * V);
  constexpr int kWarpBytes = 3 * Rows<T, V, S, kAsync>::kBytes + Rows<G, V, S, kAsync>::kBytes;
  const size_t smem = sizeof(Maps<V>) + (kAsync ? kStages * kWarps * kWarpBytes : 0);
  return launch_cluster(gated_scan_bwd_kernel<T, G, V, S, kAsync>, seen, d, d.B * ngrp, kWarps * S, smem, s, d.T, d.W, ngrp,
                        d.x_stride, d.gate_stride, (const T*)x, (const T*)gate, (const T*)h, init, (const G*)dh, dfinal,
                        (G*)dx, (G*)dgate, dinit, st);
}

// Rows whose 16-byte chunks are aligned in every tensor: they are copied to shared memory, some rounds deep.
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
                  unsigned* st, cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? SF : SF / 2;
  return aligned_rows(d) ? fwd_t<T, 2, S, true>(d, x, gate, init, h, fin, st, s) : fwd_t<T, 1, 16, false>(d, x, gate, init, h, fin, st, s);
}

template <class T, class G>
cudaError_t bwd_v(const GatedDims& d, const void* x, const void* gate, const void* h, const float* init, const void* dh,
                  const float* dfinal, void* dx, void* dgate, float* dinit, unsigned* st, cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? SB : SB / 2;
  return aligned_rows(d) ? bwd_t<T, G, 2, S, true>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, st, s)
                         : bwd_t<T, G, 1, 8, false>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, st, s);
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
                              float* fin, unsigned* st, cudaStream_t s) {
  switch (d.dtype) {
    case SWIMBA_F32: return fwd_v<float>(d, x, gate, init, h, fin, st, s);
    case SWIMBA_BF16: return fwd_v<__nv_bfloat16>(d, x, gate, init, h, fin, st, s);
    default: return fwd_v<__half>(d, x, gate, init, h, fin, st, s);
  }
}

cudaError_t launch_gated_scan_bwd(const GatedDims& d, const void* x, const void* gate, const void* h, const float* init,
                                  const void* dh, const float* dfinal, void* dx, void* dgate, float* dinit,
                                  unsigned* st, cudaStream_t s) {
  const bool g32 = d.grad_dtype == SWIMBA_F32;
  switch (d.dtype) {
    case SWIMBA_F32: return bwd_v<float, float>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, st, s);
    case SWIMBA_BF16:
      return g32 ? bwd_v<__nv_bfloat16, float>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, st, s)
                 : bwd_v<__nv_bfloat16, __nv_bfloat16>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, st, s);
    default:
      return g32 ? bwd_v<__half, float>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, st, s)
                 : bwd_v<__half, __half>(d, x, gate, h, init, dh, dfinal, dx, dgate, dinit, st, s);
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
