// The gated feed-forward block and its gradients, as launches of the tensor-core products (ffn_tc.cu).
//
//   gate = x W_gate^T,  up = x W_up^T,  h = act(gate) * up,  out = h W_down^T
//   dh = dout W_down,  dgate = dh up act'(gate),  dup = dh act(gate),
//   dx = dgate W_gate + dup W_up,  dW_gate = dgate^T x,  dW_up = dup^T x,  dW_down = dout^T h.
//
// Forward: one launch for gate, up and h, one for out.  Gradients: one launch for dgate and dup, one for the four other
// products together, so that their tiles fill the SMs' last turn.
#include "block_common.cuh"
#include "ffn_tc.cuh"

namespace swimba {

#define FFN_TRY(x)                     \
  do {                                 \
    const cudaError_t e_ = (x);        \
    if (e_ != cudaSuccess) return e_;  \
  } while (0)

namespace {

// Operands of the block's launches are 16-bit tensors as they are, or an fp32 tensor's three bf16 planes; a product of two
// fp32 tensors is then the six products of planes i and j with i + j <= 2, as six segments of K.  The planes are below
// 2^-8 and 2^-17 of the value, so a pair left out is below 2^-25 of the product and all three together below 2^-24.  On
// CUDA cores the same products took five to seven times as long from 16 x 512 x 1024 on.
void add_segments(FfnProblem& q, int a, int b, int b_up, int planes) {
  for (int i = planes - 1; i >= 0; --i)  // the small terms first
    for (int j = planes - 1 - i; j >= 0; --j) {
      q.a[q.nseg] = (unsigned char)a; q.a_plane[q.nseg] = (unsigned char)i;
      q.b[q.nseg] = (unsigned char)b; q.b_plane[q.nseg] = (unsigned char)j;
      q.b_up[q.nseg] = (unsigned char)b_up;
      ++q.nseg;
    }
}

FfnProblem problem(int M, int N, int K, int a, bool a_mn, int b, bool b_mn, void* out, int planes, int b_up = 0) {
  FfnProblem q{};
  q.M = M; q.N = N; q.K = K; q.a_mn = a_mn; q.b_mn = b_mn;
  q.out = out;
  add_segments(q, a, b, b_up, planes);
  return q;
}

int planes_of(const FfnDims& d) { return d.dtype == SWIMBA_F32 ? 3 : 1; }

FfnLaunch launch_of(const FfnDims& d, int epi, int nop, int nprob) {
  FfnLaunch l{};
  l.epi = epi; l.act = d.act; l.dtype = d.dtype; l.op_dtype = d.dtype == SWIMBA_F32 ? SWIMBA_BF16 : d.dtype;
  l.nop = nop; l.nprob = nprob;
  return l;
}

// h (and gate and up) = x, the two weights.
FfnLaunch glu_launch(const FfnDims& d, const void* x, const void* wg, const void* wu, void* gate, void* up, void* h) {
  const int pl = planes_of(d);
  FfnLaunch l = launch_of(d, kFfnGlu, 3, 1);
  l.op[0] = {x, d.M, d.D, pl}; l.op[1] = {wg, d.F, d.D, pl}; l.op[2] = {wu, d.F, d.D, pl};
  l.prob[0] = problem(d.M, d.F, d.D, 0, false, 1, false, h, pl, 2);
  l.out2 = gate; l.out3 = up;
  return l;
}

FfnLaunch down_launch(const FfnDims& d, const void* h, const void* wd, void* out) {
  const int pl = planes_of(d);
  FfnLaunch l = launch_of(d, kFfnStore, 2, 1);
  l.op[0] = {h, d.M, d.F, pl}; l.op[1] = {wd, d.D, d.F, pl};
  l.prob[0] = problem(d.M, d.D, d.F, 0, false, 1, false, out, pl);
  return l;
}

FfnLaunch dglu_launch(const FfnDims& d, const void* dout, const void* wd, const void* gate, const void* up, void* dgate,
                      void* dup) {
  const int pl = planes_of(d);
  FfnLaunch l = launch_of(d, kFfnDglu, 2, 1);
  l.op[0] = {dout, d.M, d.D, pl}; l.op[1] = {wd, d.D, d.F, pl};
  l.prob[0] = problem(d.M, d.F, d.D, 0, false, 1, true, dgate, pl);
  l.out2 = dup; l.in1 = gate; l.in2 = up;
  return l;
}

// dx (K = both halves of the features) and the three weight gradients (K = the tokens) in one launch.
FfnLaunch grads_launch(const FfnDims& d, const void* x, const void* h, const void* wg, const void* wu, const void* dout,
                       const void* dgate, const void* dup, void* dx, void* dwg, void* dwu, void* dwd) {
  const int pl = planes_of(d);
  FfnLaunch l = launch_of(d, kFfnStore, 7, 4);
  l.op[0] = {dgate, d.M, d.F, pl}; l.op[1] = {dup, d.M, d.F, pl}; l.op[2] = {wg, d.F, d.D, pl}; l.op[3] = {wu, d.F, d.D, pl};
  l.op[4] = {x, d.M, d.D, pl}; l.op[5] = {dout, d.M, d.D, pl}; l.op[6] = {h, d.M, d.F, pl};
  l.prob[0] = problem(d.M, d.D, d.F, 0, false, 2, true, dx, pl);
  add_segments(l.prob[0], 1, 3, 0, pl);
  l.prob[1] = problem(d.F, d.D, d.M, 0, true, 4, true, dwg, pl);
  l.prob[2] = problem(d.F, d.D, d.M, 1, true, 4, true, dwu, pl);
  l.prob[3] = problem(d.D, d.F, d.M, 5, true, 6, true, dwd, pl);
  return l;
}

size_t half_bytes(const FfnDims& d) { return align_up((size_t)d.M * d.F * elem_bytes(d.dtype), 256); }

// An fp32 tensor's planes in the workspace, and the launch that fills several.
struct Planes {
  char* at;
  int n = 0;
  const float* src[kFfnMaxOperands];
  void* dst[kFfnMaxOperands];
  long long count[kFfnMaxOperands];
  const void* add(const void* p, long long count_) {
    void* d = at;
    at += align_up((size_t)count_ * 6, 256);
    src[n] = (const float*)p; dst[n] = d; count[n] = count_;
    ++n;
    return d;
  }
  cudaError_t launch(cudaStream_t s) {
    const cudaError_t e = launch_ffn_split(n, src, dst, count, s);
    n = 0;
    return e;
  }
};
size_t planes_bytes(long long count) { return align_up((size_t)count * 6, 256); }

}  // namespace

size_t gated_ffn_ws(const FfnDims& d) {
  size_t n = 256 + ffn_tc_partial_bytes(down_launch(d, nullptr, nullptr, nullptr));
  if (d.dtype == SWIMBA_F32)
    n += planes_bytes((long long)d.M * d.D) + 3 * planes_bytes((long long)d.F * d.D) + planes_bytes((long long)d.M * d.F);
  return n;
}
size_t gated_ffn_bwd_ws(const FfnDims& d) {
  size_t n = 2 * half_bytes(d);
  n += align_up(ffn_tc_partial_bytes(grads_launch(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                  nullptr, nullptr, nullptr)), 256);
  if (d.dtype == SWIMBA_F32)
    n += 2 * planes_bytes((long long)d.M * d.D) + 3 * planes_bytes((long long)d.F * d.D) + 3 * planes_bytes((long long)d.M * d.F);
  return n;
}

cudaError_t launch_gated_ffn(const FfnDims& d, const void* x, const void* wg, const void* wu, const void* wd, void* gate,
                             void* up, void* h, void* out, char* ws, unsigned* st, cudaStream_t s) {
  const void* h_in = h;
  Planes pl{ws + align_up(ffn_tc_partial_bytes(down_launch(d, nullptr, nullptr, nullptr)), 256)};
  if (d.dtype == SWIMBA_F32) {
    x = pl.add(x, (long long)d.M * d.D);
    wg = pl.add(wg, (long long)d.F * d.D);
    wu = pl.add(wu, (long long)d.F * d.D);
    wd = pl.add(wd, (long long)d.F * d.D);
    FFN_TRY(pl.launch(s));
  }
  FFN_TRY(launch_ffn_tc(glu_launch(d, x, wg, wu, gate, up, h), nullptr, st, s));
  if (d.dtype == SWIMBA_F32) {
    h_in = pl.add(h, (long long)d.M * d.F);
    FFN_TRY(pl.launch(s));
  }
  return launch_ffn_tc(down_launch(d, h_in, wd, out), (float*)ws, st, s);
}

cudaError_t launch_gated_ffn_bwd(const FfnDims& d, const void* x, const void* gate, const void* up, const void* h,
                                 const void* wg, const void* wu, const void* wd, const void* dout, void* dx, void* dwg,
                                 void* dwu, void* dwd, char* ws, unsigned* st, cudaStream_t s) {
  char* dgate = ws;
  char* dup = ws + half_bytes(d);
  char* partial = ws + 2 * half_bytes(d);
  const void* dg_in = dgate;
  const void* du_in = dup;
  Planes pl{partial + align_up(ffn_tc_partial_bytes(grads_launch(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                                 nullptr, nullptr, nullptr, nullptr, nullptr)), 256)};
  if (d.dtype == SWIMBA_F32) {
    dout = pl.add(dout, (long long)d.M * d.D);
    wd = pl.add(wd, (long long)d.F * d.D);
    x = pl.add(x, (long long)d.M * d.D);
    wg = pl.add(wg, (long long)d.F * d.D);
    wu = pl.add(wu, (long long)d.F * d.D);
    h = pl.add(h, (long long)d.M * d.F);
    FFN_TRY(pl.launch(s));
  }
  FFN_TRY(launch_ffn_tc(dglu_launch(d, dout, wd, gate, up, dgate, dup), nullptr, st, s));
  if (d.dtype == SWIMBA_F32) {
    dg_in = pl.add(dgate, (long long)d.M * d.F);
    du_in = pl.add(dup, (long long)d.M * d.F);
    FFN_TRY(pl.launch(s));
  }
  return launch_ffn_tc(grads_launch(d, x, h, wg, wu, dout, dg_in, du_in, dx, dwg, dwu, dwd), (float*)partial, st, s);
}

}  // namespace swimba
