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
// (CTAs x warps x S) consecutive tokens: each warp composes the maps of its S tokens in registers, the warps'
// maps meet in shared memory, the CTAs' in distributed shared memory (asynchronous stores counted on an mbarrier: a
// cluster barrier would first wait for the round's stores of h), and every warp then replays its tokens from its true
// carried value.  So each input is read once, the split along time needs no pass over memory, no workspace and no
// waiting between clusters, and sums run in a fixed order.  All in fp32, pairs of columns by two-wide instructions.
//
// Bounds.  Not HBM alone: a round is loads, maps, the exchange across the cluster and the replay, and the registers that
// hold its tokens leave 8 to 16 warps an SM to hide one behind another.  bf16: 1 x 32768 x 2048 (403 MB) 104 us, 0.59 of a
// copy's rate with 42 % of the issue slots used (21 instructions an element); 4 x 2048 x 1536 (75 MB) 23 us; its gradients
// (151 MB) 38 us; captured passes over sets of inputs in turn, larger than L2 together, a user's calls on new inputs 1 to
// 9 % more.  The step reads and writes the state once: 256 x 4096 bf16 4.6 us so, 3.6 us with state and rows in L2.
#include <atomic>

#include "block_common.cuh"
#include "tc_common.cuh"

namespace swimba {

namespace {

constexpr int kWarps = 4, kStages = 2;
// CTAs whose registers fit an SM, by the tokens of a warp's round: the long rounds take twice as many.  The ways below cap
// them by shared memory: three where 16-bit inputs meet fp32 gradients in short rounds, 61 KB a CTA (planned as four, a
// launch of 512 CTAs took two turns: 1 x 2048 x 4096 44 us, 32 us so).
constexpr int fwd_resident(int S, int lane_bytes) { return S * lane_bytes > 64 ? 2 : 4; }
constexpr int bwd_resident(int S, int lane_bytes) { return S * lane_bytes > 32 ? 2 : 4; }

// fp32 arithmetic on a lane's V columns; a pair of columns lives in one 64-bit register pair, where the two-wide
// instructions take it.
template <int V>
struct Vec;
template <>
struct Vec<1> {
  float p;
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ explicit Vec(const float (&v)[1]) : p(v[0]) {}
  __device__ __forceinline__ void out(float (&v)[1]) const { v[0] = p; }
};
template <>
struct Vec<2> {
  unsigned long long p;
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ explicit Vec(const float (&v)[2]) { asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(v[0]), "f"(v[1])); }
  __device__ __forceinline__ void out(float (&v)[2]) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(p)); }
};
__device__ __forceinline__ Vec<1> operator*(Vec<1> a, Vec<1> b) { a.p *= b.p; return a; }
__device__ __forceinline__ Vec<1> operator+(Vec<1> a, Vec<1> b) { a.p += b.p; return a; }
__device__ __forceinline__ Vec<1> fma(Vec<1> a, Vec<1> b, Vec<1> c) { a.p = fmaf(a.p, b.p, c.p); return a; }
__device__ __forceinline__ Vec<2> operator*(Vec<2> a, Vec<2> b) {
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.p) : "l"(b.p));
  return a;
}
__device__ __forceinline__ Vec<2> operator+(Vec<2> a, Vec<2> b) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.p) : "l"(b.p));
  return a;
}
__device__ __forceinline__ Vec<2> fma(Vec<2> a, Vec<2> b, Vec<2> c) {
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a.p) : "l"(b.p), "l"(c.p));
  return a;
}
template <int V>
__device__ __forceinline__ Vec<V> all(float x) {
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = x;
  return Vec<V>(v);
}

// gate_pair for V columns.
template <int V>
__device__ __forceinline__ void gates(const float (&g)[V], Vec<V>& f, Vec<V>& q) {
  float e[V], r[V], s[V], l[V];
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = exp_fast(-fabsf(g[i]));
  const Vec<V> ev(e);
  (ev + all<V>(1.f)).out(r);
#pragma unroll
  for (int i = 0; i < V; ++i) r[i] = rcp_fast(r[i]);
  const Vec<V> small = ev * Vec<V>(r), large = fma(small, all<V>(-1.f), all<V>(1.f));
  small.out(s);
  large.out(l);
  float fo[V], qo[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool open = g[i] >= 0.f;
    fo[i] = open ? l[i] : s[i];
    qo[i] = open ? s[i] : l[i];
  }
  f = Vec<V>(fo);
  q = Vec<V>(qo);
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

// A round's maps: this CTA's warps and, by CTA rank, the cluster's CTAs.  Two copies, used in turn: a warp writes one
// again two rounds later, after a block barrier (another CTA: after this CTA's map of the round between, sent behind one)
// that follows every read of it.
constexpr int kMaxCluster = 16;
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
__device__ __forceinline__ void exchange_init(Maps<V>& sm) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) tc::mbar_init(&sm.bar[i], 1);
    tc::fence_barrier_init();
  }
  tc::cluster_sync();  // every CTA runs, its barriers initialised, before another stores to its shared memory
}

// Sends round `round`'s maps on their way, given the map `mine` of this warp's tokens.  Returns the map of the CTA's tokens
// in front of them.
template <int V>
__device__ __forceinline__ Map<V> send(Maps<V>& sm, int round, int warp, int lane, uint32_t rank, uint32_t nrank,
                                       const Map<V>& mine) {
  const int buf = round & 1;
  sm.warp[buf][warp][lane] = mine;
  if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(&sm.bar[buf], nrank * 32 * (uint32_t)sizeof(Map<V>));
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
  if (warp == kWarps - 1) {
    Map<V> cta = before;
    then(cta, mine.a, mine.b);
    const uint32_t at = tc::smem_u32(&sm.cta[buf][rank][lane]), bar = tc::smem_u32(&sm.bar[buf]);
    float a[V], b[V];
    cta.a.out(a);
    cta.b.out(b);
    for (uint32_t r = 0; r < nrank; ++r) {
      const uint32_t to = tc::map_shared(at, r), on = tc::map_shared(bar, r);
      if constexpr (V == 2)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                     "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "r"(on)
                     : "memory");
      else
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
                     "f"(a[0]), "f"(b[0]), "r"(on)
                     : "memory");
    }
  }
  return before;
}

// Takes round `round`'s maps: returns the carried value in front of this warp's tokens and advances `carry` over the
// round.  A thread whose wait gave up waits no more (`waits`): all its rounds together are bounded like one.
template <int V>
__device__ __forceinline__ Vec<V> receive(Maps<V>& sm, int round, int lane, uint32_t rank, uint32_t nrank,
                                          const Map<V>& before, Vec<V>& carry, bool& waits, unsigned* st) {
  const int buf = round & 1;
  if (waits && !wait_cluster(&sm.bar[buf], (uint32_t)(round >> 1) & 1u)) {
    waits = false;
    atomicOr(st, ST_TIMEOUT);
  }
  Vec<V> c = carry, at = carry;
  const Map<V>* m = sm.cta[buf][0] + lane;
  for (uint32_t r = 0; r < nrank; ++r, m += 32) {
    if (r == rank) at = c;
    c = fma(m->a, c, m->b);
  }
  carry = c;
  return fma(before.a, at, before.b);
}

// 16 bytes global -> shared.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// One warp's tokens of one input, from a stage in shared memory or from registers: S rows of 32 V columns.
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
          if (t + dir * k * kStep >= 0 && t + dir * k * kStep < n)
            cp_async16(to + k * kStep * kRowBytes, from + k * step);
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
  __device__ __forceinline__ void get(const uint8_t* stage, int i, int lane, float (&out)[V]) const {
    if constexpr (kAsync) {
      load_vec<T, V>(reinterpret_cast<const T*>(stage + i * kRowBytes) + V * lane, out);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = to_f32(raw[i][v]);
    }
  }
  __device__ __forceinline__ Vec<V> get(const uint8_t* stage, int i, int lane) const {
    float v[V];
    get(stage, i, lane, v);
    return Vec<V>(v);
  }
};

template <int V>
__device__ __forceinline__ Vec<V> load_state(const float* p, size_t at, bool live) {
  float r[V];
#pragma unroll
  for (int v = 0; v < V; ++v) r[v] = p && live ? p[at + v] : 0.f;
  return Vec<V>(r);
}

template <class T, int V, int S, bool kAsync>
__global__ void __launch_bounds__(32 * kWarps, fwd_resident(S, V * sizeof(T)))
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
  int t = ((int)rank * kWarps + warp) * S;  // the warp's first token
  auto fetch = [&](int t, int st) {
    rx.fetch(stages + st * kStride, x, xs, t, 1, T_, col0, W, lane);
    rg.fetch(stages + st * kStride + R::kBytes, gate, gs, t, 1, T_, col0, W, lane);
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < (kAsync ? kStages - 1 : 1); ++k) fetch(t + k * span, k);
  Vec<V> carry = load_state<V>(init, state, live);
  exchange_init(sm);
  bool waits = true;
  int st = 0;
  for (int round = 0; round * span < T_; ++round, t += span) {
    if (kAsync) {
      // the stage that the last round read (a block barrier ago) is filled next
      fetch(t + (kStages - 1) * span, st == 0 ? kStages - 1 : st - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
    }
    // a token's state is P c + H for the value c carried to the warp's tokens
    Vec<V> P[S], H[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float g[V];
      rg.get(stages + st * kStride + R::kBytes, i, lane, g);
      gates(g, P[i], H[i]);
      H[i] = H[i] * rx.get(stages + st * kStride, i, lane);
    }
    if (t + S > T_) {
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (t + i >= T_) { P[i] = all<V>(1.f); H[i] = all<V>(0.f); }
    }
#pragma unroll
    for (int i = 1; i < S; ++i) {
      H[i] = fma(P[i], H[i - 1], H[i]);
      P[i] = P[i] * P[i - 1];
    }
    if (!kAsync) fetch(t + span, 0);
    Map<V> mine;
    mine.a = P[S - 1];
    mine.b = H[S - 1];
    const Map<V> before = send(sm, round, warp, lane, rank, nrank, mine);
    const Vec<V> c = receive(sm, round, lane, rank, nrank, before, carry, waits, status);
    T* out = h + (size_t)t * W;
    auto put = [&](int n) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        float o[V];
        fma(P[i], c, H[i]).out(o);
        if (i < n) store_vec<T, V>(out, o);
        out += W;
      }
    };
    if (live) {
      if (t + S <= T_) put(S);
      else put(T_ - t);
    }
    st = st == kStages - 1 ? 0 : st + 1;
  }
  cp_async_wait<0>();
  if (final_state && live && rank == 0 && warp == 0) {
    float o[V];
    carry.out(o);
#pragma unroll
    for (int v = 0; v < V; ++v) final_state[state + v] = o[v];
  }
  tc::cluster_sync();  // no CTA leaves while another may still store to it
}

// Token index tau counts from the last token: t = T - 1 - tau.
template <class T, class G, int V, int S, bool kAsync>
__global__ void __launch_bounds__(32 * kWarps, bwd_resident(S, V * sizeof(T)))
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
  int t = T_ - 1 - ((int)rank * kWarps + warp) * S;  // the warp's last token
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
  exchange_init(sm);
  bool waits = true;
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
      float g[V];
      rg.get(p, i, lane, g);
      gates(g, f[i], q[i]);
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
    const Map<V> before = send(sm, round, warp, lane, rank, nrank, mine);
    Vec<V> c = receive(sm, round, lane, rank, nrank, before, carry, waits, status);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const Vec<V> lam = d[i] + c;
      c = f[i] * lam;
      float ox[V], og[V];
      (q[i] * lam).out(ox);
      (c * q[i] * e[i]).out(og);
      if (live && t - i >= 0) {
        store_vec<G, V>(dx + (size_t)(t - i) * W, ox);
        store_vec<G, V>(dgate + (size_t)(t - i) * W, og);
      }
    }
    st = st == kStages - 1 ? 0 : st + 1;
  }
  cp_async_wait<0>();
  if (dinit && live && rank == 0 && warp == 0) {
    float o[V];
    carry.out(o);
#pragma unroll
    for (int v = 0; v < V; ++v) dinit[state + v] = o[v];
  }
  tc::cluster_sync();
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

void set_cluster(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& attr, int c, int groups, size_t smem) {
  cfg.gridDim = dim3((unsigned)(groups * c));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = smem;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)c;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
}

// CTAs per cluster, a power of two, and CTAs per SM.  The cluster size is the one with the least estimated time: for every
// set of clusters that is resident together 2.5 us and its rounds in a row, a round being a fixed part, one for every CTA
// on the fullest SM, and 0.02 us for every CTA of the cluster (fitted to sweeps of 1 .. 16 CTAs over 1 x 32768 x 2048,
// 4 x 2048 x 1536, 1 x 30000 x 64, 1 x 20000 x 512 and odd widths; the parts stand beside the kernels' ways below).  At 16
// sizes outside those sweeps (1 x 12000 x 512 to 16 x 256 x 768, every type, odd widths, forward and gradients) it takes
// at most 2 % more than the best of all cluster sizes and both ways.
// Clusters are placed as densely as they fit, so the launch asks for as much shared memory as lets only its share fit an
// SM (at 4 x 2048 x 1536, 384 CTAs: 23 us with three per SM, 30 us where four fitted and SMs stayed empty); while the scan
// runs, kernels of other streams that use shared memory stay off the SMs it holds.  kFit: CTAs
// that fit at 1 .. 4 per SM by cluster size; GPCs of uneven size hold fewer of the larger ones.
struct Split {
  int c, per_sm;
  double cost;
};
Split best_split(int groups, int rounds, int resident, double fixed, double each) {
  constexpr int kFit[5][4] = {
      {148, 296, 444, 592}, {148, 296, 444, 592}, {132, 284, 416, 568}, {120, 264, 384, 568}, {112, 224, 336, 496}};
  Split best{1, 1, 0};
  for (int c = 1, i = 0; c <= kMaxCluster && (c == 1 || c < 2 * rounds); c *= 2, ++i) {
    int k = 1;
    while (k < resident && (long long)groups * c > kFit[i][k - 1]) ++k;
    const double sets = ceil_div(groups * c, kFit[i][k - 1]);
    const double cost = sets * (2.5 + ceil_div(rounds, c) * (fixed + each * k + 0.02 * c));
    if (best.cost == 0 || cost < best.cost) best = {c, k, cost};
  }
  return best;
}
// Dynamic shared memory of which `per_sm` CTAs, and no more, fit an SM's 228 KB (1 KB of each CTA is the system's).
constexpr size_t kSmSmem = 233472;
constexpr int fitting(int ctas, size_t smem) {
  return ctas * (smem + 1024) <= kSmSmem ? ctas : (int)(kSmSmem / (smem + 1024));
}
size_t smem_for(int per_sm, size_t need) {
  const size_t share = (kSmSmem / (size_t)per_sm - 1024) / 128 * 128;
  return share > need ? share : need;
}

// One way of laying out a scan: its kernel, the columns and tokens of a CTA's round, its shared memory.
template <class K>
struct Way {
  K kernel;
  int cols, tokens, resident;
  double fixed, each;  // of a round's time
  size_t smem;
  std::atomic<unsigned long long>& wide;  // devices (bits) on which clusters of more than 8 CTAs are allowed
};
template <class K>
Split split_of(const Way<K>& w, const GatedDims& d) {
  return best_split(d.B * ceil_div(d.W, w.cols), ceil_div(d.T, w.tokens), w.resident, w.fixed, w.each);
}
template <class K, class... A>
cudaError_t launch_way(const Way<K>& w, const Split& split, const GatedDims& d, cudaStream_t s, A... a) {
  const size_t smem = smem_for(split.per_sm, w.smem);
  cudaError_t e = set_max_dynamic_smem((const void*)w.kernel, smem);
  if (e == cudaSuccess && split.c > 8) {
    int dev = 0;
    e = cudaGetDevice(&dev);
    const unsigned long long bit = 1ULL << (dev & 63);
    if (e == cudaSuccess && !(w.wide.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(w.kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e == cudaSuccess) w.wide.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  const int ngrp = ceil_div(d.W, w.cols);
  set_cluster(cfg, attr, split.c, d.B * ngrp, smem);
  cfg.stream = s;
  e = cudaLaunchKernelEx(&cfg, w.kernel, d.T, d.W, ngrp, d.x_stride, d.gate_stride, a...);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <class T, int V, int S, bool kAsync>
auto fwd_way() {
  constexpr bool kLong = fwd_resident(S, V * sizeof(T)) == 2;
  constexpr double kFixed = V == 1 ? (sizeof(T) == 2 ? 1.5 : 0.5) : kLong ? 0.8 : 0.62;
  constexpr double kEach = V == 1 ? (sizeof(T) == 2 ? 0.5 : 1.25) : kLong ? 1.15 : 0.6;
  static std::atomic<unsigned long long> wide{0};
  auto kernel = gated_scan_kernel<T, V, S, kAsync>;
  using R = Rows<T, V, S, kAsync>;
  constexpr size_t kSmem = sizeof(Maps<V>) + (kAsync ? (size_t)kStages * kWarps * 2 * R::kBytes : 0);
  constexpr int kResident = fitting(fwd_resident(S, V * sizeof(T)), kSmem);
  static_assert(kResident * (kSmem + 1024) <= kSmSmem, "the planned CTAs fit an SM's shared memory");
  return Way<decltype(kernel)>{kernel, 32 * V, kWarps * S, kResident, kFixed, kEach, kSmem, wide};
}
template <class T, class G, int V, int S, bool kAsync>
auto bwd_way() {
  constexpr bool kLong = bwd_resident(S, V * sizeof(T)) == 2;
  constexpr double kFixed = V == 1 ? 1.25 : kLong ? 1.3 : 0.95;
  constexpr double kEach = V == 1 ? 0.45 : kLong ? 0.77 : 0.4;
  static std::atomic<unsigned long long> wide{0};
  auto kernel = gated_scan_bwd_kernel<T, G, V, S, kAsync>;
  constexpr size_t kWarpBytes = 3 * Rows<T, V, S, kAsync>::kBytes + Rows<G, V, S, kAsync>::kBytes;
  constexpr size_t kSmem = sizeof(Maps<V>) + (kAsync ? kStages * kWarps * kWarpBytes : 0);
  constexpr int kResident = fitting(bwd_resident(S, V * sizeof(T)), kSmem);
  static_assert(kResident * (kSmem + 1024) <= kSmSmem, "the planned CTAs fit an SM's shared memory");
  return Way<decltype(kernel)>{kernel, 32 * V, kWarps * S, kResident, kFixed, kEach, kSmem, wide};
}
template <class K, class... A>
cudaError_t launch(const Way<K>& w, const GatedDims& d, cudaStream_t s, A... a) {
  return launch_way(w, split_of(w, d), d, s, a...);
}

// Of two ways, the cheaper: long rounds spread a round's fixed part over twice the tokens where the columns are few.
template <class K1, class K2, class... A>
cudaError_t launch(const Way<K1>& w1, const Way<K2>& w2, const GatedDims& d, cudaStream_t s, A... a) {
  const Split s1 = split_of(w1, d), s2 = split_of(w2, d);
  return s2.cost < s1.cost ? launch_way(w2, s2, d, s, a...) : launch_way(w1, s1, d, s, a...);
}

// Rows whose 16-byte chunks are aligned in every tensor: they are copied to shared memory, a round ahead.
bool aligned_rows(const GatedDims& d) {
  const int q = d.dtype == SWIMBA_F32 ? 4 : 8;
  return d.W % q == 0 && d.x_stride % q == 0 && d.gate_stride % q == 0;
}

template <class T>
cudaError_t fwd_v(const GatedDims& d, const void* x, const void* gate, const float* init, void* h, float* fin,
                  unsigned* st, cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? 16 : 8;
  if (aligned_rows(d))
    return launch(fwd_way<T, 2, S, true>(), fwd_way<T, 2, 2 * S, true>(), d, s, (const T*)x, (const T*)gate, init,
                         (T*)h, fin, st);
  return launch(fwd_way<T, 1, 16, false>(), d, s, (const T*)x, (const T*)gate, init, (T*)h, fin, st);
}

template <class T, class G>
cudaError_t bwd_v(const GatedDims& d, const void* x, const void* gate, const void* h, const float* init, const void* dh,
                  const float* dfinal, void* dx, void* dgate, float* dinit, unsigned* st, cudaStream_t s) {
  constexpr int S = sizeof(T) == 2 ? 8 : 4;
  auto go = [&](auto launch) {
    return launch(d, s, (const T*)x, (const T*)gate, (const T*)h, init, (const G*)dh, dfinal, (G*)dx, (G*)dgate, dinit, st);
  };
  if (aligned_rows(d))
    return go([](auto... a) { return launch(bwd_way<T, G, 2, S, true>(), bwd_way<T, G, 2, 2 * S, true>(), a...); });
  return go([](auto... a) { return launch(bwd_way<T, G, 1, 8, false>(), a...); });
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
