// Interface of the feed-forward block's tensor-core products (ffn_tc.cu).  Internal to libswimba.
#pragma once
#include "block_common.cuh"

namespace swimba {

constexpr int kFfnMaxProblems = 4, kFfnMaxOperands = 8;

// What a product's epilogue does with its fp32 accumulators.
enum FfnEpi {
  kFfnGlu,    // columns are pairs (gate, up) of one feature: h = act(gate) * up, and gate and up where wanted
  kFfnDglu,   // the product is dh: dgate and dup from the stored gate and up
  kFfnStore,  // the product itself, or a split's partial sum of it
};

// An operand in memory: `planes` matrices of rows x cols, row-major, 16-bit.
struct FfnOperand {
  const void* p;
  long long rows, cols;
  int planes;
};

// out = sum over segments of A_s B_s^T: segment s reads plane a_plane[s] of operand a[s] and the same of b.
struct FfnProblem {
  int M, N, K;       // K of one segment
  int a_mn, b_mn;    // the operand's rows are K (its columns M or N), not M or N
  int nseg;
  unsigned char a[12], a_plane[12], b[12], b_plane[12];
  unsigned char b_up[12];  // kFfnGlu: the up weights, where b is the gate's (operand 0 is x)
  void* out;         // [M][N] (kFfnGlu: h, kFfnDglu: dgate)
};

struct FfnLaunch {
  int epi, act, dtype;  // dtype of what is stored
  int nop, nprob;
  FfnOperand op[kFfnMaxOperands];
  int op_dtype;         // SWIMBA_BF16 or SWIMBA_F16
  FfnProblem prob[kFfnMaxProblems];
  void* out2;           // kFfnGlu: gate or null, kFfnDglu: dup
  void* out3;           // kFfnGlu: up or null
  const void* in1;      // kFfnDglu: gate
  const void* in2;      // kFfnDglu: up
};

// Bytes of partial sums that the launch needs (a function of the sizes alone).
size_t ffn_tc_partial_bytes(const FfnLaunch& l);
// fp32 tensors of `count` values (a multiple of 8) as three bf16 planes each, whose sum they are.
cudaError_t launch_ffn_split(int n, const float* const* src, void* const* dst, const long long* count, cudaStream_t s);
cudaError_t launch_ffn_tc(const FfnLaunch& l, float* partial, unsigned* st, cudaStream_t s);

}  // namespace swimba
