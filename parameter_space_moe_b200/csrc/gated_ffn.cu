// The gated feed-forward block and its gradients on CUDA cores.
//
//   gate = x W_gate^T,  up = x W_up^T,  h = act(gate) * up,  out = h W_down^T
//   dh = dout W_down,  dgate = dh up act'(gate),  dup = dh act(gate),
//   dx = dgate W_gate + dup W_up,  dW_gate = dgate^T x,  dW_up = dup^T x,  dW_down = dout^T h.
//
// One register-tiled product, 128 x 128 outputs per 256-thread CTA and 8 x 8 per thread, with fp32 operands in
// shared memory as [k][row] and the next slice prefetched into registers.  Either operand is read along K or
// along its rows, so no transposed copy is made.  Products:
//   kGlu    A = x, B = 64 rows of W_gate and the same 64 of W_up: a thread's columns c and c + 4 are the gate and
//           the up value of one feature, and the epilogue forms h
//   kDglu   A = dout, B = W_down read across: the epilogue turns dh into dgate and dup
//   kStore  out, dx (two summands of K), and the weight gradients (K = rows of x)
#include <math.h>

#include "block_common.cuh"
#include "ffn_act.cuh"
#include "ffn_tc.cuh"

namespace swimba {

namespace {

constexpr int BT = 128, BK = 16, kThreads = 256;
enum Epi { kGlu, kDglu, kStore };

// Operand tile source: element (row r, k) at p[r * ld + k] (kc) or p[k * ld + r].
template <class T>
struct Operand {
  const T* p;
  const T* p2;  // second summand of K (kStore), or the up rows (kGlu)
  long long ld;
  int rows;
};

template <class T>
struct Out {
  T* a;            // kGlu: h, kDglu: dgate, kStore: the product
  T* b;            // kGlu: gate or null, kDglu: dup
  T* c;            // kGlu: up or null
  const T* gate;   // kDglu
  const T* up;
  long long ld;
};

// Four consecutive values of the tile's slice k0..: along K for one row (KC) or along the rows for one k.
template <class T, bool KC>
__device__ __forceinline__ void fetch(const T* p, long long ld, int rows, int K, int r, int k, float (&v)[4]) {
  v[0] = v[1] = v[2] = v[3] = 0.f;
  if (r < rows && k < K) load_vec<T, 4>(KC ? p + (size_t)r * ld + k : p + (size_t)k * ld + r, v);
}

template <class T, bool AKC, bool BKC, int EPI, int kAct>
__global__ void __launch_bounds__(kThreads)
ffn_simt_kernel(int M, int N, int K, int nsum, Operand<T> A, Operand<T> B, Out<T> o) {
  __shared__ float As[2][BK][BT + 4], Bs[2][BK][BT + 4];
  const int tid = threadIdx.x;
  constexpr int kCols = EPI == kGlu ? BT / 2 : BT;  // features per tile
  const int m0 = blockIdx.x * BT, n0 = blockIdx.y * kCols;
  const int ty = tid >> 4, tx = tid & 15;
  float acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  float ra[2][4], rb[2][4];
  const int nk = ceil_div(K, BK), steps = nk * nsum;
  // each thread moves two groups of four values of either tile
  auto place = [&](bool kc, int g, int& r, int& k) {
    const int id = tid + g * kThreads;
    if (kc) { r = id >> 2; k = (id & 3) * 4; } else { k = id >> 5; r = (id & 31) * 4; }
  };
  auto load = [&](int s) {
    const int k0 = (s % nk) * BK;
    const bool second = s >= nk;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      int r, k;
      place(AKC, g, r, k);
      fetch<T, AKC>(second ? A.p2 : A.p, A.ld, A.rows, K, m0 + r, k0 + k, ra[g]);
      place(BKC, g, r, k);
      if (EPI == kGlu) {
        // columns 8 q .. 8 q + 3 of the tile are gate rows 4 q .., columns 8 q + 4 .. the same up rows
        const int fr = (r >> 3) * 4 + (r & 3);
        fetch<T, BKC>((r & 4) ? B.p2 : B.p, B.ld, B.rows, K, n0 + fr, k0 + k, rb[g]);
      } else {
        fetch<T, BKC>(second ? B.p2 : B.p, B.ld, B.rows, K, n0 + r, k0 + k, rb[g]);
      }
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      int r, k;
      place(AKC, g, r, k);
#pragma unroll
      for (int j = 0; j < 4; ++j) { if (AKC) As[buf][k + j][r] = ra[g][j]; else As[buf][k][r + j] = ra[g][j]; }
      place(BKC, g, r, k);
#pragma unroll
      for (int j = 0; j < 4; ++j) { if (BKC) Bs[buf][k + j][r] = rb[g][j]; else Bs[buf][k][r + j] = rb[g][j]; }
    }
  };
  load(0);
  put(0);
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    const int buf = s & 1;
    if (s + 1 < steps) load(s + 1);
#pragma unroll
    for (int k = 0; k < BK; ++k) {
      float a[8], b[8];
      load_vec<float, 8>(&As[buf][k][ty * 8], a);
      load_vec<float, 8>(&Bs[buf][k][tx * 8], b);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    if (s + 1 < steps) put(buf ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + ty * 8 + i;
    if (m >= M) break;
    if (EPI == kGlu) {
      const int n = n0 + tx * 4;
      if (n >= N) break;
      float g[4], u[4], h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) { g[j] = acc[i][j]; u[j] = acc[i][j + 4]; h[j] = act_value<kAct>(g[j]) * u[j]; }
      store_vec<T, 4>(o.a + (size_t)m * o.ld + n, h);
      if (o.b) store_vec<T, 4>(o.b + (size_t)m * o.ld + n, g);
      if (o.c) store_vec<T, 4>(o.c + (size_t)m * o.ld + n, u);
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int n = n0 + tx * 8 + 4 * q;
        if (n >= N) break;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = acc[i][4 * q + j];
        if (EPI == kDglu) {
          float g[4], u[4], dg[4], du[4];
          load_vec<T, 4>(o.gate + (size_t)m * o.ld + n, g);
          load_vec<T, 4>(o.up + (size_t)m * o.ld + n, u);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float slope;
            const float a = act_both<kAct>(g[j], slope);
            dg[j] = v[j] * u[j] * slope;
            du[j] = v[j] * a;
          }
          store_vec<T, 4>(o.a + (size_t)m * o.ld + n, dg);
          store_vec<T, 4>(o.b + (size_t)m * o.ld + n, du);
        } else {
          store_vec<T, 4>(o.a + (size_t)m * o.ld + n, v);
        }
      }
    }
  }
}

template <class T, bool AKC, bool BKC, int EPI>
cudaError_t product(int M, int N, int K, int nsum, int act, Operand<T> A, Operand<T> B, Out<T> o, cudaStream_t s) {
  const dim3 grid(ceil_div(M, BT), ceil_div(N, EPI == kGlu ? BT / 2 : BT));
  if (EPI == kStore || act == SWIMBA_SILU)
    ffn_simt_kernel<T, AKC, BKC, EPI, SWIMBA_SILU><<<grid, kThreads, 0, s>>>(M, N, K, nsum, A, B, o);
  else
    ffn_simt_kernel<T, AKC, BKC, EPI, SWIMBA_GELU><<<grid, kThreads, 0, s>>>(M, N, K, nsum, A, B, o);
  count_launches(1);
  return cudaGetLastError();
}

#define FFN_TRY(x)                     \
  do {                                 \
    const cudaError_t e_ = (x);        \
    if (e_ != cudaSuccess) return e_;  \
  } while (0)

template <class T>
cudaError_t fwd_t(const FfnDims& d, const T* x, const T* wg, const T* wu, const T* wd, T* gate, T* up, T* h, T* out,
                  cudaStream_t s) {
  FFN_TRY((product<T, true, true, kGlu>(d.M, d.F, d.D, 1, d.act, {x, nullptr, d.D, d.M}, {wg, wu, d.D, d.F},
                                        {h, gate, up, nullptr, nullptr, d.F}, s)));
  return product<T, true, true, kStore>(d.M, d.D, d.F, 1, d.act, {h, nullptr, d.F, d.M}, {wd, nullptr, d.F, d.D},
                                        {out, nullptr, nullptr, nullptr, nullptr, d.D}, s);
}

template <class T>
cudaError_t bwd_t(const FfnDims& d, const T* x, const T* gate, const T* up, const T* h, const T* wg, const T* wu,
                  const T* wd, const T* dout, T* dx, T* dwg, T* dwu, T* dwd, T* dgate, T* dup, cudaStream_t s) {
  FFN_TRY((product<T, true, false, kDglu>(d.M, d.F, d.D, 1, d.act, {dout, nullptr, d.D, d.M}, {wd, nullptr, d.F, d.F},
                                          {dgate, dup, nullptr, gate, up, d.F}, s)));
  FFN_TRY((product<T, true, false, kStore>(d.M, d.D, d.F, 2, d.act, {dgate, dup, d.F, d.M}, {wg, wu, d.D, d.D},
                                           {dx, nullptr, nullptr, nullptr, nullptr, d.D}, s)));
  FFN_TRY((product<T, false, false, kStore>(d.F, d.D, d.M, 1, d.act, {dgate, nullptr, d.F, d.F}, {x, nullptr, d.D, d.D},
                                            {dwg, nullptr, nullptr, nullptr, nullptr, d.D}, s)));
  FFN_TRY((product<T, false, false, kStore>(d.F, d.D, d.M, 1, d.act, {dup, nullptr, d.F, d.F}, {x, nullptr, d.D, d.D},
                                            {dwu, nullptr, nullptr, nullptr, nullptr, d.D}, s)));
  return product<T, false, false, kStore>(d.D, d.F, d.M, 1, d.act, {dout, nullptr, d.D, d.D}, {h, nullptr, d.F, d.F},
                                          {dwd, nullptr, nullptr, nullptr, nullptr, d.F}, s);
}

}  // namespace

namespace {

// The tensor-core launches of the block: operands by number, one problem per product.
FfnProblem problem(int M, int N, int K, int a, bool a_mn, int b, bool b_mn, void* out) {
  FfnProblem q{};
  q.M = M; q.N = N; q.K = K; q.a_mn = a_mn; q.b_mn = b_mn; q.nseg = 1;
  q.a[0] = (unsigned char)a; q.b[0] = (unsigned char)b;
  q.out = out;
  return q;
}

FfnLaunch launch_of(const FfnDims& d, int epi, int nop) {
  FfnLaunch l{};
  l.epi = epi; l.act = d.act; l.dtype = l.op_dtype = d.dtype; l.nop = nop;
  return l;
}

// h (and gate and up) = x, the two weights.
FfnLaunch glu_launch(const FfnDims& d, const void* x, const void* wg, const void* wu, void* gate, void* up, void* h) {
  FfnLaunch l = launch_of(d, kFfnGlu, 3);
  l.op[0] = {x, d.M, d.D, 1}; l.op[1] = {wg, d.F, d.D, 1}; l.op[2] = {wu, d.F, d.D, 1};
  l.nprob = 1;
  l.prob[0] = problem(d.M, d.F, d.D, 0, false, 1, false, h);
  l.prob[0].b_up[0] = 2;
  l.out2 = gate; l.out3 = up;
  return l;
}

FfnLaunch down_launch(const FfnDims& d, const void* h, const void* wd, void* out) {
  FfnLaunch l = launch_of(d, kFfnStore, 2);
  l.op[0] = {h, d.M, d.F, 1}; l.op[1] = {wd, d.D, d.F, 1};
  l.nprob = 1;
  l.prob[0] = problem(d.M, d.D, d.F, 0, false, 1, false, out);
  return l;
}

FfnLaunch dglu_launch(const FfnDims& d, const void* dout, const void* wd, const void* gate, const void* up, void* dgate,
                      void* dup) {
  FfnLaunch l = launch_of(d, kFfnDglu, 2);
  l.op[0] = {dout, d.M, d.D, 1}; l.op[1] = {wd, d.D, d.F, 1};
  l.nprob = 1;
  l.prob[0] = problem(d.M, d.F, d.D, 0, false, 1, true, dgate);
  l.out2 = dup; l.in1 = gate; l.in2 = up;
  return l;
}

// dx (K = both halves of the features) and the three weight gradients (K = the tokens) in one launch.
FfnLaunch grads_launch(const FfnDims& d, const void* x, const void* h, const void* wg, const void* wu, const void* dout,
                       const void* dgate, const void* dup, void* dx, void* dwg, void* dwu, void* dwd) {
  FfnLaunch l = launch_of(d, kFfnStore, 7);
  l.op[0] = {dgate, d.M, d.F, 1}; l.op[1] = {dup, d.M, d.F, 1}; l.op[2] = {wg, d.F, d.D, 1}; l.op[3] = {wu, d.F, d.D, 1};
  l.op[4] = {x, d.M, d.D, 1}; l.op[5] = {dout, d.M, d.D, 1}; l.op[6] = {h, d.M, d.F, 1};
  l.nprob = 4;
  l.prob[0] = problem(d.M, d.D, d.F, 0, false, 2, true, dx);
  l.prob[0].nseg = 2; l.prob[0].a[1] = 1; l.prob[0].b[1] = 3;
  l.prob[1] = problem(d.F, d.D, d.M, 0, true, 4, true, dwg);
  l.prob[2] = problem(d.F, d.D, d.M, 1, true, 4, true, dwu);
  l.prob[3] = problem(d.D, d.F, d.M, 5, true, 6, true, dwd);
  return l;
}

bool tensor_cores(const FfnDims& d) { return d.dtype != SWIMBA_F32; }
size_t half_bytes(const FfnDims& d) { return align_up((size_t)d.M * d.F * elem_bytes(d.dtype), 256); }

}  // namespace

size_t gated_ffn_ws(const FfnDims& d) {
  return 256 + (tensor_cores(d) ? ffn_tc_partial_bytes(down_launch(d, nullptr, nullptr, nullptr)) : 0);
}
size_t gated_ffn_bwd_ws(const FfnDims& d) {
  size_t n = 2 * half_bytes(d);
  if (tensor_cores(d))
    n += ffn_tc_partial_bytes(grads_launch(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                           nullptr, nullptr, nullptr));
  return n;
}

cudaError_t launch_gated_ffn(const FfnDims& d, const void* x, const void* wg, const void* wu, const void* wd, void* gate,
                             void* up, void* h, void* out, char* ws, unsigned* st, cudaStream_t s) {
  if (tensor_cores(d)) {
    FFN_TRY(launch_ffn_tc(glu_launch(d, x, wg, wu, gate, up, h), nullptr, st, s));
    return launch_ffn_tc(down_launch(d, h, wd, out), (float*)ws, st, s);
  }
  return fwd_t<float>(d, (const float*)x, (const float*)wg, (const float*)wu, (const float*)wd, (float*)gate, (float*)up,
                      (float*)h, (float*)out, s);
}

cudaError_t launch_gated_ffn_bwd(const FfnDims& d, const void* x, const void* gate, const void* up, const void* h,
                                 const void* wg, const void* wu, const void* wd, const void* dout, void* dx, void* dwg,
                                 void* dwu, void* dwd, char* ws, unsigned* st, cudaStream_t s) {
  char* dgate = ws;
  char* dup = ws + half_bytes(d);
  if (tensor_cores(d)) {
    FFN_TRY(launch_ffn_tc(dglu_launch(d, dout, wd, gate, up, dgate, dup), nullptr, st, s));
    return launch_ffn_tc(grads_launch(d, x, h, wg, wu, dout, dgate, dup, dx, dwg, dwu, dwd),
                         (float*)(ws + 2 * half_bytes(d)), st, s);
  }
  return bwd_t<float>(d, (const float*)x, (const float*)gate, (const float*)up, (const float*)h, (const float*)wg,
                      (const float*)wu, (const float*)wd, (const float*)dout, (float*)dx, (float*)dwg, (float*)dwu,
                      (float*)dwd, (float*)dgate, (float*)dup, s);
}

}  // namespace swimba
