// The products of the gated feed-forward block and of its gradients on the 5th-generation tensor cores, with the
// activation (or its gradient) in the epilogue: 16-bit operands, fp32 accumulation in TMEM.
//
// One kernel serves all of them.  Every operand is fetched in boxes of 64 columns x 128 rows (128-byte swizzle): two
// boxes along K for an operand stored along K, two along M or N for one stored across, which the MMA then reads
// MN-major.  So no operand is ever transposed in memory and one tensor map per tensor serves every role.
//   tile        256 x 256 by a CTA pair (cta_group::2, M256 N256 K16: each CTA loads 128 rows of A and 128 of B), or
//               128 x 128 by one CTA where all of them then run in one turn (make_plan)
//   warp 0      TMA producer: A 32 KB + B 32 KB per 128-wide K slice, a ring of kStages
//   warp 1      TMEM owner and MMA issuer, two accumulators in TMEM
//   warps 2..9  epilogue from TMEM: a thread holds one row, 32 columns at a time; each warp stages its 32 x 32 block
//               in shared memory (64-byte swizzle: no bank conflicts) and stores it with TMA, two blocks in flight.
//               Stored from registers, a warp's 16-byte stores touched 32 rows each and held the epilogue of the
//               8192 x 768 x 2048 forward to 10 us a tile, twice the tile's MMAs
// fp32 products (six segments of bf16 planes) leave the accumulator every 256 of K and are added up in registers: the
// tensor cores cut what an addition shifts out.  Over one chain of 12 x 2816 that put the gradient of x 2.5e-5 off, over
// chains of 1024 2.0e-6, of 512 1.0e-6, of 256 5e-7 (fp32 FMAs: 1.1e-6); 256 takes 4 % longer than 512.
// Bounds, bf16.  Many rows: the tensor pipe under the power cap (8192 x 2048 x 5632, the gradients of x and the weights:
// 640 us, pipe 87 % active at the 1.43 GHz that the cap leaves), the epilogue's loads and stores where a tile's K is short
// (gate and up at K = 768: 46 us, pipe 56 %; dgate and dup with their two more inputs: 159 us, 63 %), and
// turns that do not fill the SMs (8192 x 768 from K = 2048: 96 tiles on 74 pairs, 30.7 us, 41 %).  256 rows: the weights'
// bytes and each launch's start and end (256 x 2048 x 5632, 74 MB: 21 + 14 + 5 us alone, 32 us together).
// Persistent over the units (problem, tile, split of K); a product with few tiles is split along K into fp32
// partial sums, added in a fixed order by a second kernel.
#include <math.h>

#include <type_traits>

#include "ffn_act.cuh"
#include "ffn_tc.cuh"
#include "tc_common.cuh"

namespace swimba {

namespace {

constexpr int BK = 128, kStages = 3;
// Epilogue warps, and staged blocks of each.  16 warps with one block each measured 1060 us for the 8192 x 2048 x 5632
// gradients against 915 us (their registers spill), with no gain elsewhere.
constexpr int kEpiWarps = 8, kBlocks = 2;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kBox = 64 * 2 * 128;             // 64 columns of 128 rows, 16-bit
constexpr uint32_t kStageBytes = 4 * kBox;          // two boxes of A, two of B
constexpr uint32_t kBlock = 32 * 64;                // an epilogue warp's staged block: 32 rows of 64 bytes
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + kEpiWarps * kBlocks * kBlock + 256;
constexpr int kSms = 148;                           // what the plan fills; the launch asks the device
constexpr int kMaxSplit = 16;                       // of a product with few tiles
// K blocks of one accumulation of 16-bit operands, at most (kFfnStore; the others sum over the model's width alone).  The
// tensor cores cut what an addition shifts out: 1.1e-7 of the sum for every 16 of K when all terms have one sign.  Over
// 2^20 rows in one chain the weights' gradients came out 6.5e-3 small; 65536 of K leave 4.3e-4, a ninth of bf16's half
// step, 16384 1.1e-4, a quarter of fp16's.  Longer sums leave the accumulator as often and are added up in registers, in
// a kernel of their own, since the registers cost shorter ones up to 5 % (17000 x 2048 x 5632, the gradients: 1.83 and
// 1.93 ms at best).  32768 x 768 x 2048 fp16, the gradients: 588 us in one chain and so, 617 us as split sums, which take
// workspace besides.
constexpr int longest(bool bf16) { return bf16 ? 512 : 128; }

struct Prob {
  int M, N, kbs, nkb, a_mn, b_mn;  // kbs: K blocks of a segment, nkb: of all
  unsigned char a[12], a_plane[12], b[12], b_plane[12], b_up[12];
  int tiles_m, tiles_n, split, begin;  // first unit
  void* dst;    // the output itself, and
  float* part;  // its partial sums [split][M][N] where split > 1
};

struct Args {
  int nprob, units, ab_bf16;
  int out2, out3;  // numbers of the maps, -1 without
  const void* in1;
  const void* in2;
  unsigned* st;
  Prob prob[kFfnMaxProblems];
};

struct Maps {
  CUtensorMap m[kFfnMaxOperands];
  CUtensorMap o[kFfnMaxProblems + 2];  // one per problem (its output, or its partial sums), then out2 and out3
};

struct Unit {
  int p, tm, tn, s, kb0, kb1;
};

__device__ __forceinline__ Unit unit_of(const Args& a, int u) {
  Unit r;
  r.p = 0;
  while (r.p + 1 < a.nprob && a.prob[r.p + 1].begin <= u) ++r.p;
  const Prob& q = a.prob[r.p];
  const int t = u - q.begin;
  r.s = t % q.split;
  const int tile = t / q.split;
  r.tm = tile % q.tiles_m;
  r.tn = tile / q.tiles_m;
  r.kb0 = (int)((long long)q.nkb * r.s / q.split);
  r.kb1 = (int)((long long)q.nkb * (r.s + 1) / q.split);
  return r;
}

template <bool kPair>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  if (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5}], [%2];" ::"r"(tc::smem_u32(dst)),
        "l"((uint64_t)map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            tc::smem_u32(dst)),
        "l"((uint64_t)map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Stores a warp's 32 x 32 block, lane i holding row i, at (row m, column n, plane) of the output behind `map`.  The
// warp's two staging blocks are used in turn; `lane` 0 owns the copies.
template <class T>
__device__ __forceinline__ void store_block(const CUtensorMap* map, uint8_t* stage, int& turn, int lane, const float (&v)[32],
                                            int n, int m, int plane) {
  constexpr int kCols = 64 / (int)sizeof(T);
#pragma unroll
  for (int h = 0; h < 32 / kCols; ++h) {
    uint8_t* b = stage + turn * kBlock;
    turn = turn + 1 == kBlocks ? 0 : turn + 1;
    if (lane == 0) tc::bulk_wait_read<kBlocks - 1>();  // this block's last copy has read it
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float w[kCols / 4];
#pragma unroll
      for (int j = 0; j < kCols / 4; ++j) w[j] = v[h * kCols + c * (kCols / 4) + j];
      store_vec<T, kCols / 4>(reinterpret_cast<T*>(b + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)), w);
    }
    tc::fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      tc::tma_store_3d(map, b, n + h * kCols, m, plane);
      tc::bulk_commit();
    }
  }
}

// The 32 values at p as vectors of 16 bytes; those from `left` on (a multiple of a vector), or all of a dead row, are 0.
template <class T>
struct RowOf {
  static constexpr int kPer = 16 / (int)sizeof(T), kVecs = 32 / kPer;
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const T* p, bool live, int left) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      v[i] = live && kPer * i < left ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ float get(int j) const {
    T t[kPer];
    memcpy(t, &v[j / kPer], 16);
    return to_f32(t[j % kPer]);
  }
};

template <bool kPair, int kEpi, int kAct, class T, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
ffn_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  constexpr int TM = kPair ? 256 : 128, TN = kPair ? 256 : 128;
  constexpr int kFeat = kEpi == kFfnGlu ? TN / 2 : TN;  // output columns of a tile
  constexpr uint32_t kTmemCols = 2 * TN;
  constexpr bool kChains = sizeof(T) == 4 || kLong;     // several accumulations, added up in registers
  constexpr int kChain = sizeof(T) == 4 ? 2 : kLong ? longest(std::is_same<T, __nv_bfloat16>::value) : 1 << 30;  // K blocks of one accumulation
  constexpr int kPart = kFeat / (kEpiWarps / 4);        // columns of a tile that one warp drains
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes + kEpiWarps * kBlocks * kBlock);
  uint64_t* full = bars;
  uint64_t* empty = bars + kStages;
  uint64_t* acc_full = bars + 2 * kStages;
  uint64_t* acc_empty = bars + 2 * kStages + 2;
  uint64_t* drain = bars + 2 * kStages + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? tc::cluster_ctarank() : 0u;
  const int first = kPair ? blockIdx.x >> 1 : blockIdx.x, step = kPair ? gridDim.x >> 1 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { tc::mbar_init(&full[s], 1); tc::mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], (kPair ? 2 : 1) * kEpiWarps);
    }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  griddep_launch_dependents();
  // TMEM is taken ahead of the wait below.  A kernel that holds TMEM while it waits for one that still has to take its own
  // on the same SM would stop both; the shared memory of this one leaves an SM no room for another of the library's kernels.
  static_assert(233472 - (kSmemBytes + 1024) < 2048, "a CTA has its SM's shared memory to itself");
  if (warp == 1) {
    if (kPair) {
      tc::tmem_alloc_pair(tmem_slot, kTmemCols);
      tc::tmem_relinquish_pair();
    } else {
      tc::tmem_alloc(tmem_slot, kTmemCols);
      tc::tmem_relinquish();
    }
  }
  griddep_wait();  // what earlier kernels wrote: operands, the stored gate and up
  tc::fence_before_sync();
  if (kPair) tc::cluster_sync();  // both CTAs' barriers are initialised before any copy or commit reaches them
  else __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer (both CTAs of a pair)
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    const uint32_t full0 = kPair ? tc::map_shared(tc::smem_u32(full), 0u) : tc::smem_u32(full);
    for (int u = first; u < a.units && ok; u += step) {
      const Unit t = unit_of(a, u);
      const Prob& q = a.prob[t.p];
      const int m0 = t.tm * TM + 128 * (int)rank;
      int seg = t.kb0 / q.kbs, kb = t.kb0 % q.kbs;
      for (int i = t.kb0; i < t.kb1; ++i) {
        if (!tc::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
        uint8_t* sa = smem + stage * kStageBytes;
        if (rank == 0) tc::mbar_arrive_expect_tx(&full[stage], (kPair ? 2 : 1) * kStageBytes);
        const uint32_t fb = full0 + 8u * (uint32_t)stage;
        const int k = kb * BK;
        const CUtensorMap* ma = &maps.m[q.a[seg]];
        const CUtensorMap* mb = &maps.m[q.b[seg]];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          load_box<kPair>(sa + j * kBox, ma, fb, q.a_mn ? m0 + 64 * j : k + 64 * j, q.a_mn ? k : m0, q.a_plane[seg]);
        uint8_t* sb = sa + 2 * kBox;
        if (kEpi == kFfnGlu) {
          // the first half of the tile's columns are gate rows, the second half the same up rows
          const CUtensorMap* mu = &maps.m[q.b_up[seg]];
          const int n = t.tn * kFeat;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (kPair) {
              load_box<kPair>(sb + j * kBox, rank ? mu : mb, fb, k + 64 * j, n, q.b_plane[seg]);
            } else {
              load_box<kPair>(sb + j * kBox, mb, fb, k + 64 * j, n, q.b_plane[seg]);
              load_box<kPair>(sb + j * kBox + kBox / 2, mu, fb, k + 64 * j, n, q.b_plane[seg]);
            }
          }
        } else {
          const int n = t.tn * TN + 128 * (int)rank;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            load_box<kPair>(sb + j * kBox, mb, fb, q.b_mn ? n + 64 * j : k + 64 * j, q.b_mn ? k : n, q.b_plane[seg]);
        }
        ++issued;
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
        if (++kb == q.kbs) { kb = 0; ++seg; }
      }
    }
    if (!ok) { *abort_flag = 1; atomicOr(a.st, ST_TIMEOUT); }
    // every copy this CTA issued has been consumed by an MMA (its stage was released) or is waited for here
    for (long long i = 0; i < kStages && i < issued; ++i) {
      if (--stage < 0) { stage = kStages - 1; phase ^= 1u; }
      volatile int never = 0;
      tc::mbar_wait(&empty[stage], phase, &never);
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---------------------------------------------------------------- MMA issuer (the even CTA of a pair)
    int stage = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int u = first; u < a.units && ok; u += step) {
      const Unit t = unit_of(a, u);
      const Prob& q = a.prob[t.p];
      const uint32_t idesc = tc::idesc_f16(TM, TN, a.ab_bf16 != 0, q.a_mn != 0, q.b_mn != 0);
      // a K16 step: 32 bytes inside the swizzled row (K-major; its second 64 columns in the next box) or 16 rows of
      // 128 bytes (MN-major)
      const uint32_t a_step = q.a_mn ? 2048 >> 4 : 32 >> 4, b_step = q.b_mn ? 2048 >> 4 : 32 >> 4;
      const uint32_t a_far = q.a_mn ? 4 * 2048 >> 4 : kBox >> 4, b_far = q.b_mn ? 4 * 2048 >> 4 : kBox >> 4;
      if (!tc::mbar_wait(&acc_empty[buf], acc_phase ^ 1u, abort_flag)) { ok = false; break; }
      tc::fence_after_sync();
      uint32_t dt = tmem + (uint32_t)(buf * TN);
      int begin = t.kb0;
      for (int i = t.kb0; i < t.kb1; ++i) {
        if (i - begin == kChain) {  // the chain so far goes to the epilogue, the next one starts from zero
          if (kPair) tc::mma_commit_pair(&acc_full[buf], 0x3);
          else tc::mma_commit(&acc_full[buf]);
          if (++buf == 2) { buf = 0; acc_phase ^= 1u; }
          if (!tc::mbar_wait(&acc_empty[buf], acc_phase ^ 1u, abort_flag)) { ok = false; break; }
          tc::fence_after_sync();
          dt = tmem + (uint32_t)(buf * TN);
          begin = i;
        }
        if (!tc::mbar_wait(&full[stage], phase, abort_flag)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t sa = tc::smem_u32(smem + stage * kStageBytes), sb = sa + 2 * kBox;
        const uint64_t da = q.a_mn ? tc::sdesc_mnmajor_sw128(sa, kBox) : tc::sdesc_kmajor_sw128(sa);
        const uint64_t db = q.b_mn ? tc::sdesc_mnmajor_sw128(sb, kBox) : tc::sdesc_kmajor_sw128(sb);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint32_t acc = i > begin || kk > 0;
          const uint64_t dak = da + (kk & 3) * a_step + (kk >> 2) * a_far, dbk = db + (kk & 3) * b_step + (kk >> 2) * b_far;
          if (kPair) tc::mma_f16_pair(dt, dak, dbk, idesc, acc);
          else tc::mma_f16(dt, dak, dbk, idesc, acc);
        }
        if (kPair) tc::mma_commit_pair(&empty[stage], 0x3);
        else tc::mma_commit(&empty[stage]);
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      if (kPair) tc::mma_commit_pair(&acc_full[buf], 0x3);
      else tc::mma_commit(&acc_full[buf]);
      if (++buf == 2) { buf = 0; acc_phase ^= 1u; }
    }
    if (!ok) { *abort_flag = 1; atomicOr(a.st, ST_TIMEOUT); }
    if (kPair) tc::mma_commit_pair(drain, 0x3);
    else tc::mma_commit(drain);
    volatile int never = 0;
    tc::mbar_wait(drain, 0, &never);
  } else if (warp == 1 && lane == 0) {
    // odd CTA: its TMEM and shared memory are in use until the even CTA's last MMA has completed
    volatile int never = 0;
    tc::mbar_wait(drain, 0, &never);
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int q4 = warp & 3, part = (warp - 2) >> 2;
    const uint32_t acc_empty0 = kPair ? tc::map_shared(tc::smem_u32(acc_empty), 0u) : 0u;
    uint8_t* staged = smem + kStages * kStageBytes + (warp - 2) * kBlocks * kBlock;
    int buf = 0, turn = 0;
    uint32_t acc_phase = 0;
    for (int u = first; u < a.units; u += step) {
      const Unit t = unit_of(a, u);
      const Prob& q = a.prob[t.p];
      const int mw = t.tm * TM + 128 * (int)rank + 32 * q4, m = mw + lane;
      const int n0 = t.tn * kFeat + part * kPart;
      RowOf<T> ng, nu;  // kFfnDglu: gate and up of the next block (of this one in fp32, whose registers hold no more)
      constexpr bool kAhead = sizeof(T) == 2;
      auto fetch = [&](int c) {
        const size_t at = (size_t)m * q.N + n0 + c;
        ng.load((const T*)a.in1 + at, m < q.M, q.N - n0 - c);
        nu.load((const T*)a.in2 + at, m < q.M, q.N - n0 - c);
      };
      if (kEpi == kFfnDglu && kAhead) fetch(0);
      auto wait_full = [&]() {
        if (!tc::mbar_wait(&acc_full[buf], acc_phase, abort_flag)) {
          *abort_flag = 1;
          atomicOr(a.st, ST_TIMEOUT);
          return false;
        }
        tc::fence_after_sync();
        return true;
      };
      auto free_acc = [&]() {
        tc::fence_before_sync();
        __syncwarp();
        // orders only TMEM reads (the tcgen05 fence), so a pair's arrival is relaxed
        if (lane == 0) {
          if (kPair) tc::mbar_arrive_cluster_relaxed(acc_empty0 + 8u * (uint32_t)buf);
          else tc::mbar_arrive(&acc_empty[buf]);
        }
        if (++buf == 2) { buf = 0; acc_phase ^= 1u; }
      };
      // What becomes of 32 columns at n0 + c: v the accumulators, w the up half's (kFfnGlu).
      auto finish = [&](int c, float (&v)[32], float (&w)[32]) {
        const int n = n0 + c;
        const bool some = mw < q.M && n < q.N;  // the same in the whole warp
        if (kEpi == kFfnGlu) {
          if (some) {
            if (a.out2 >= 0) store_block<T>(&maps.o[a.out2], staged, turn, lane, v, n, mw, 0);
            if (a.out3 >= 0) store_block<T>(&maps.o[a.out3], staged, turn, lane, w, n, mw, 0);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = act_value<kAct, sizeof(T) == 4>(v[i]) * w[i];
            store_block<T>(&maps.o[t.p], staged, turn, lane, v, n, mw, 0);
          }
        } else if (kEpi == kFfnDglu) {
          if (!kAhead) fetch(c);
          const RowOf<T> cg = ng, cu = nu;
          if (kAhead && c + 32 < kPart) fetch(c + 32);
          if (some) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float slope;
              const float act = act_both<kAct, sizeof(T) == 4>(cg.get(i), slope);
              w[i] = v[i] * act;
              v[i] *= cu.get(i) * slope;
            }
            store_block<T>(&maps.o[t.p], staged, turn, lane, v, n, mw, 0);
            store_block<T>(&maps.o[a.out2], staged, turn, lane, w, n, mw, 0);
          }
        } else if (some) {
          if (q.split > 1) store_block<float>(&maps.o[t.p], staged, turn, lane, v, n, mw, t.s);
          else store_block<T>(&maps.o[t.p], staged, turn, lane, v, n, mw, 0);
        }
      };
      bool ok = true;
      if constexpr (kChains) {
        float v[kPart / 32][32], w[kEpi == kFfnGlu ? kPart / 32 : 1][32];
#pragma unroll
        for (int c = 0; c < kPart / 32; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) v[c][i] = 0.f;
        if (kEpi == kFfnGlu) {
#pragma unroll
          for (int c = 0; c < kPart / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) w[c][i] = 0.f;
        }
        for (int kb = t.kb0; kb < t.kb1; kb += kChain) {
          if (!wait_full()) { ok = false; break; }
          const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(buf * TN + part * kPart);
#pragma unroll
          for (int c = 0; c < kPart / 32; ++c) {
            uint32_t r[32];
            tc::tmem_ld_32x32b_x32(taddr + 32 * c, r);
            tc::tmem_ld_wait(r);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[c][i] += __uint_as_float(r[i]);
            if (kEpi == kFfnGlu) {
              tc::tmem_ld_32x32b_x32(taddr + TN / 2 + 32 * c, r);
              tc::tmem_ld_wait(r);
#pragma unroll
              for (int i = 0; i < 32; ++i) w[c][i] += __uint_as_float(r[i]);
            }
          }
          free_acc();
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < kPart / 32; ++c) finish(32 * c, v[c], w[kEpi == kFfnGlu ? c : 0]);
      } else {
        if (!wait_full()) break;
        const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(buf * TN + part * kPart);
#pragma unroll 1
        for (int c = 0; c < kPart; c += 32) {
          uint32_t ra[32], rb[32];
          tc::tmem_ld_32x32b_x32(taddr + c, ra);
          if (kEpi == kFfnGlu) tc::tmem_ld_32x32b_x32(taddr + TN / 2 + c, rb);
          tc::tmem_ld_wait(ra);
          if (kEpi == kFfnGlu) tc::tmem_ld_wait(rb);
          float v[32], w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] = __uint_as_float(ra[i]);
            w[i] = kEpi == kFfnGlu ? __uint_as_float(rb[i]) : 0.f;
          }
          finish(c, v, w);
        }
        free_acc();
      }
    }
    if (lane == 0) tc::bulk_wait_all();
  }
  tc::fence_before_sync();
  if (kPair) tc::cluster_sync();  // no CTA leaves while the other may still signal its barriers or read its operands
  else __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    if (kPair) tc::tmem_dealloc_pair(tmem, kTmemCols);
    else tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// out = sum of the split partial sums, in order; four columns per thread.  The loads of eight splits are in flight
// together: one after the other, 16 splits of a small product took 11 us.
template <class T>
__global__ void __launch_bounds__(128)
ffn_reduce_kernel(const __grid_constant__ Args a) {
  griddep_launch_dependents();
  griddep_wait();
  for (int p = 0; p < a.nprob; ++p) {
    const Prob& q = a.prob[p];
    if (q.split < 2) continue;
    const size_t n = (size_t)q.M * q.N;
    for (size_t i = 4 * ((size_t)blockIdx.x * blockDim.x + threadIdx.x); i < n; i += 4 * (size_t)gridDim.x * blockDim.x) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int s0 = 0; s0 < q.split; s0 += 8) {
        float4 w[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s0 + s < q.split) w[s] = __ldcs(reinterpret_cast<const float4*>(q.part + (s0 + s) * n + i));
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s0 + s < q.split) { v[0] += w[s].x; v[1] += w[s].y; v[2] += w[s].z; v[3] += w[s].w; }
      }
      store_vec<T, 4>((T*)q.dst + i, v);
    }
  }
}

// Tiles, splits and units of a launch: a function of the sizes alone.
struct Plan {
  bool pair, split_any;
  size_t partial_bytes;
};
Plan make_plan(const FfnLaunch& l, Args* a) {
  Plan pl{};
  const int feat = l.epi == kFfnGlu ? 2 : 1;
  auto tiles = [&](const FfnProblem& q, int t) { return (long long)ceil_div(q.M, t) * ceil_div(q.N, t / feat); };
  long long big = 0;
  for (int p = 0; p < l.nprob; ++p) big += tiles(l.prob[p], 256);
  // Up to 36 tiles of 256 x 256, four times as many of 128 x 128 run side by side on the SMs, which is the faster way; from
  // 37 on they would take a second turn, and pairs are, though some SMs idle.  Pair against one CTA, us: gate and up at
  // 256 x 2048 x 4608 (36 tiles) 19.3, 16.0, x 5632 (44) 19.8, 24.5; 1024 x 768 x 640 (20) 11.4, 9.1, x 1280 (40) 11.8, 12.9;
  // dgate and dup at 1024 x 2048 x 2048 (32) 24.7, 17.5, 52 tiles 25.6, 27.9; the gradients at 2048 x 768 x 1024 (60) 19.0, 23.4.
  pl.pair = big >= kSms / 4;
  const int t = pl.pair ? 256 : 128, slots = pl.pair ? kSms / 2 : kSms;
  // A launch with fewer tiles than slots is split along K into units of about the same length, as long as each has two K
  // blocks.  (The gradients of 4756 x 128 x 264: 9 weight tiles of 38 K blocks beside 38 tiles of 6.)
  long long total = 0, blocks = 0;
  for (int p = 0; p < l.nprob; ++p) {
    total += tiles(l.prob[p], t);
    blocks += tiles(l.prob[p], t) * ceil_div(l.prob[p].K, BK) * l.prob[p].nseg;
  }
  const long long length = (blocks + slots - 1) / slots > 2 ? (blocks + slots - 1) / slots : 2;
  long long units = 0;
  size_t off = 0;
  for (int p = 0; p < l.nprob; ++p) {
    const FfnProblem& q = l.prob[p];
    const int kbs = ceil_div(q.K, BK), nkb = kbs * q.nseg;
    long long split = l.epi == kFfnStore && total < slots ? nkb / length : 1;
    split = split < 1 ? 1 : split > kMaxSplit ? kMaxSplit : split;
    if (a) {
      Prob& r = a->prob[p];
      r.M = q.M; r.N = q.N; r.kbs = kbs; r.nkb = nkb; r.a_mn = q.a_mn; r.b_mn = q.b_mn;
      for (int s = 0; s < 12; ++s) { r.a[s] = q.a[s]; r.b[s] = q.b[s]; r.a_plane[s] = q.a_plane[s]; r.b_plane[s] = q.b_plane[s]; r.b_up[s] = q.b_up[s]; }
      r.tiles_m = ceil_div(q.M, t); r.tiles_n = ceil_div(q.N, t / feat); r.split = (int)split; r.begin = (int)units;
      r.dst = q.out;
      r.part = (float*)off;  // an offset until the launch knows the workspace
    }
    units += tiles(q, t) * split;
    if (split > 1) {
      pl.split_any = true;
      off += align_up((size_t)split * q.M * q.N * 4, 256);
    }
  }
  if (a) { a->nprob = l.nprob; a->units = (int)units; }
  pl.partial_bytes = off;
  return pl;
}

// Boxes of 128 rows; of 64 for the weights of a one-CTA gate and up tile, which has 64 rows of each.
bool encode_planes(CUtensorMap* map, const FfnOperand& o, int dtype, bool small) {
  return encode_tmap_3d_planes(map, o.p, dtype, (uint64_t)o.cols, (uint64_t)o.rows, (uint64_t)o.planes, 64, small ? 64 : 128);
}

int device_sms() {
  int sms = kSms, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <bool kPair, int kEpi, int kAct, class T, bool kLong>
cudaError_t go(const Maps& maps, const Args& a, cudaStream_t s) {
  auto kernel = ffn_tc_kernel<kPair, kEpi, kAct, T, kLong>;
  cudaError_t e = set_max_dynamic_smem((const void*)kernel, kSmemBytes);
  if (e != cudaSuccess) return e;
  const int slots = kPair ? device_sms() / 2 : device_sms();
  const int n = a.units < slots ? a.units : slots;
  e = launch_dependent(kernel, dim3((unsigned)(kPair ? 2 * n : n)), dim3(kThreads), kSmemBytes, s, kPair ? 2 : 1, maps, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <int kEpi, int kAct, class T, bool kLong = false>
cudaError_t go_pair(bool pair, const Maps& maps, const Args& a, cudaStream_t s) {
  return pair ? go<true, kEpi, kAct, T, kLong>(maps, a, s) : go<false, kEpi, kAct, T, kLong>(maps, a, s);
}

template <int kEpi, class T>
cudaError_t go_act(int act, bool pair, const Maps& maps, const Args& a, cudaStream_t s) {
  return act == SWIMBA_SILU ? go_pair<kEpi, SWIMBA_SILU, T>(pair, maps, a, s) : go_pair<kEpi, SWIMBA_GELU, T>(pair, maps, a, s);
}

template <class T>
cudaError_t go_type(const FfnLaunch& l, const Plan& pl, const Maps& maps, const Args& a, cudaStream_t s) {
  if (l.epi == kFfnGlu) return go_act<kFfnGlu, T>(l.act, pl.pair, maps, a, s);
  if (l.epi == kFfnDglu) return go_act<kFfnDglu, T>(l.act, pl.pair, maps, a, s);
  bool is_long = false;
  for (int p = 0; p < a.nprob; ++p) is_long |= ceil_div(a.prob[p].nkb, a.prob[p].split) > longest(l.dtype == SWIMBA_BF16);
  cudaError_t e = is_long ? go_pair<kFfnStore, SWIMBA_SILU, T, sizeof(T) == 2>(pl.pair, maps, a, s)
                          : go_pair<kFfnStore, SWIMBA_SILU, T>(pl.pair, maps, a, s);
  if (e != cudaSuccess || !pl.split_any) return e;
  size_t most = 0;
  for (int p = 0; p < a.nprob; ++p)
    if (a.prob[p].split > 1 && (size_t)a.prob[p].M * a.prob[p].N > most) most = (size_t)a.prob[p].M * a.prob[p].N;
  const size_t want = (most / 4 + 127) / 128;
  e = launch_dependent(ffn_reduce_kernel<T>, dim3((unsigned)(want < 16 * kSms ? want : 16 * kSms)), dim3(128), 0, s, 1, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

size_t ffn_tc_partial_bytes(const FfnLaunch& l) { return make_plan(l, nullptr).partial_bytes; }

cudaError_t launch_ffn_tc(const FfnLaunch& l, float* partial, unsigned* st, cudaStream_t s) {
  Maps maps;
  Args a{};
  const Plan pl = make_plan(l, &a);
  for (int i = 0; i < l.nop; ++i)
    if (!encode_planes(&maps.m[i], l.op[i], l.op_dtype, l.epi == kFfnGlu && !pl.pair && i > 0)) return cudaErrorInvalidValue;
  for (int p = 0; p < a.nprob; ++p) a.prob[p].part = (float*)((char*)partial + (size_t)a.prob[p].part);
  a.ab_bf16 = l.op_dtype == SWIMBA_BF16;
  const uint32_t cols = l.dtype == SWIMBA_F32 ? 16 : 32;  // a staged block's rows are 64 bytes
  // outputs: one map per problem (of its partial sums where it is split), then the other two
  for (int p = 0; p < a.nprob; ++p) {
    const Prob& q = a.prob[p];
    const bool ok = q.split > 1 ? encode_tmap_3d_planes(&maps.o[p], q.part, SWIMBA_F32, q.N, q.M, q.split, 16, 32)
                                : encode_tmap_3d_planes(&maps.o[p], q.dst, l.dtype, q.N, q.M, 1, cols, 32);
    if (!ok) return cudaErrorInvalidValue;
  }
  void* more[2] = {l.out2, l.out3};
  int at[2] = {-1, -1};
  for (int i = 0; i < 2; ++i)
    if (more[i]) {
      at[i] = kFfnMaxProblems + i;
      if (!encode_tmap_3d_planes(&maps.o[at[i]], more[i], l.dtype, a.prob[0].N, a.prob[0].M, 1, cols, 32))
        return cudaErrorInvalidValue;
    }
  a.out2 = at[0]; a.out3 = at[1]; a.in1 = l.in1; a.in2 = l.in2;
  a.st = st;
  switch (l.dtype) {
    case SWIMBA_F32: return go_type<float>(l, pl, maps, a, s);
    case SWIMBA_BF16: return go_type<__nv_bfloat16>(l, pl, maps, a, s);
    default: return go_type<__half>(l, pl, maps, a, s);
  }
}

// x = h + m + l in three bf16 planes, each the rounding of what is left: 24 bits and more.  A value that rounds past
// bf16's largest is cut instead, and what is not finite has no rest.
namespace {
struct Splits {
  int n;
  const float* src[kFfnMaxOperands];
  __nv_bfloat16* dst[kFfnMaxOperands];
  long long count[kFfnMaxOperands];  // multiples of 8
};
__global__ void __launch_bounds__(256) ffn_split_kernel(const __grid_constant__ Splits p) {
  griddep_launch_dependents();
  griddep_wait();
  for (int k = 0; k < p.n; ++k) {
    const long long n = p.count[k];
    for (long long i = 8 * ((long long)blockIdx.x * blockDim.x + threadIdx.x); i < n; i += 8LL * gridDim.x * blockDim.x) {
      float v[8], h[8], m[8], l[8];
      load_vec<float, 8>(p.src[k] + i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[j] = to_f32(__float2bfloat16_rn(v[j]));
        if (isinf(h[j])) h[j] = __uint_as_float(__float_as_uint(v[j]) & 0xffff0000u);
        const float r = isfinite(v[j]) ? v[j] - h[j] : 0.f;
        m[j] = to_f32(__float2bfloat16_rn(r));
        l[j] = r - m[j];
      }
      store_vec<__nv_bfloat16, 8>(p.dst[k] + i, h);
      store_vec<__nv_bfloat16, 8>(p.dst[k] + n + i, m);
      store_vec<__nv_bfloat16, 8>(p.dst[k] + 2 * n + i, l);
    }
  }
}
}  // namespace

cudaError_t launch_ffn_split(int n, const float* const* src, void* const* dst, const long long* count, cudaStream_t s) {
  Splits p{};
  p.n = n;
  long long most = 0;
  for (int k = 0; k < n; ++k) {
    p.src[k] = src[k];
    p.dst[k] = (__nv_bfloat16*)dst[k];
    p.count[k] = count[k];
    if (count[k] > most) most = count[k];
  }
  const long long want = (most / 8 + 255) / 256;
  const cudaError_t e =
      launch_dependent(ffn_split_kernel, dim3((unsigned)(want < 8 * kSms ? want : 8 * kSms)), dim3(256), 0, s, 1, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}


}  // namespace swimba
