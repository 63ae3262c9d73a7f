// The products of the gated feed-forward block and of its gradients on the 5th-generation tensor cores, with the
// activation (or its gradient) in the epilogue: 16-bit operands, fp32 accumulation in TMEM.
//
// One kernel serves all of them.  Every operand is fetched in 64 x 64 boxes (128-byte swizzle): as rows of K for
// an operand stored along K, or as rows of M or N for one stored across, which the MMA then reads MN-major, so no
// operand is ever transposed in memory and one tensor map per tensor serves every role.
//   tile        256 x 256 by a CTA pair (cta_group::2, M256 N256 K16: each CTA loads 128 rows of A and 128 of B), or
//               128 x 128 by one CTA where pairs would leave SMs without work
//   warp 0      TMA producer: A 16 KB + B 16 KB per 64-wide K slice, a ring of kStages
//   warp 1      TMEM owner and MMA issuer, two accumulators in TMEM
//   warps 2..9  epilogue from TMEM: a thread holds one row, 32 columns at a time, and stores whole sectors
// Persistent over the units (problem, tile, split of K); a product with few tiles is split along K into fp32
// partial sums, added in a fixed order by a second kernel.
#include "ffn_act.cuh"
#include "ffn_tc.cuh"
#include "tc_common.cuh"

namespace swimba {

namespace {

constexpr int BK = 64, kStages = 6;
constexpr int kEpiWarps = 8, kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kBox = 64 * 128;                 // one 64 x 64 box of 16-bit values
constexpr uint32_t kStageBytes = 4 * kBox;          // two boxes of A, two of B
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + 256;
constexpr int kSms = 148;                           // what the plan fills; the launch asks the device
constexpr int kMaxSplit = 16;

struct Prob {
  int M, N, kbs, nkb, a_mn, b_mn;  // kbs: K blocks of a segment, nkb: of all
  unsigned char a[12], a_plane[12], b[12], b_plane[12], b_up;
  int tiles_m, tiles_n, split, begin;  // first unit
  void* out;
  float* part;  // [split][M][N] where split > 1
};

struct Args {
  int nprob, units, act, ab_bf16;
  void* out2;
  void* out3;
  const void* in1;
  const void* in2;
  unsigned* st;
  Prob prob[kFfnMaxProblems];
};

struct Maps {
  CUtensorMap m[kFfnMaxOperands];
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

// 32 columns of one row, those below n - c0 of them (n - c0 is a multiple of 8, of 4 in fp32).
template <class T>
__device__ __forceinline__ void store_row(T* p, const float (&v)[32], int left) {
  constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < 32 / V; ++i)
    if (i * V < left) {
      float w[V];
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = v[i * V + j];
      store_vec<T, V>(p + i * V, w);
    }
}

template <bool kPair, int kEpi, class T>
__global__ void __launch_bounds__(kThreads, 1)
ffn_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  constexpr int TM = kPair ? 256 : 128, TN = kPair ? 256 : 128;
  constexpr int kFeat = kEpi == kFfnGlu ? TN / 2 : TN;  // output columns of a tile
  constexpr uint32_t kTmemCols = 2 * TN;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
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
        for (int j = 0; j < 2; ++j) {
          const int m = m0 + 64 * j;
          load_box<kPair>(sa + j * kBox, ma, fb, q.a_mn ? m : k, q.a_mn ? k : m, q.a_plane[seg]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          int n;
          const CUtensorMap* mj = mb;
          if (kEpi == kFfnGlu) {  // the first half of the tile's columns are gate rows, the second the same up rows
            const bool up = kPair ? rank == 1 : j == 1;
            n = t.tn * kFeat + (kPair ? 64 * j : 0);
            if (up) mj = &maps.m[q.b[seg] - q.b[0] + q.b_up];
          } else {
            n = t.tn * TN + 128 * (int)rank + 64 * j;
          }
          load_box<kPair>(sa + (2 + j) * kBox, mj, fb, q.b_mn ? n : k, q.b_mn ? k : n, q.b_plane[seg]);
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
      // a K16 step: 32 bytes inside the swizzled row (K-major) or 16 rows of 128 bytes (MN-major)
      const uint32_t a_step = q.a_mn ? 2048 >> 4 : 32 >> 4, b_step = q.b_mn ? 2048 >> 4 : 32 >> 4;
      if (!tc::mbar_wait(&acc_empty[buf], acc_phase ^ 1u, abort_flag)) { ok = false; break; }
      tc::fence_after_sync();
      const uint32_t dt = tmem + (uint32_t)(buf * TN);
      for (int i = t.kb0; i < t.kb1; ++i) {
        if (!tc::mbar_wait(&full[stage], phase, abort_flag)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t sa = tc::smem_u32(smem + stage * kStageBytes), sb = sa + 2 * kBox;
        const uint64_t da = q.a_mn ? tc::sdesc_mnmajor_sw128(sa, kBox) : tc::sdesc_kmajor_sw128(sa);
        const uint64_t db = q.b_mn ? tc::sdesc_mnmajor_sw128(sb, kBox) : tc::sdesc_kmajor_sw128(sb);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint32_t acc = i > t.kb0 || kk > 0;
          if (kPair) tc::mma_f16_pair(dt, da + kk * a_step, db + kk * b_step, idesc, acc);
          else tc::mma_f16(dt, da + kk * a_step, db + kk * b_step, idesc, acc);
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
    const int q4 = warp & 3, half = (warp - 2) >> 2;
    const uint32_t acc_empty0 = kPair ? tc::map_shared(tc::smem_u32(acc_empty), 0u) : 0u;
    int buf = 0;
    uint32_t acc_phase = 0;
    for (int u = first; u < a.units; u += step) {
      const Unit t = unit_of(a, u);
      const Prob& q = a.prob[t.p];
      const int m = t.tm * TM + 128 * (int)rank + 32 * q4 + lane;
      const int n0 = t.tn * kFeat + half * (kFeat / 2);
      if (!tc::mbar_wait(&acc_full[buf], acc_phase, abort_flag)) {
        *abort_flag = 1;
        atomicOr(a.st, ST_TIMEOUT);
        break;
      }
      tc::fence_after_sync();
      const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(buf * TN + half * (kFeat / 2));
#pragma unroll 1
      for (int c = 0; c < kFeat / 2; c += 32) {
        uint32_t ra[32], rb[32];
        tc::tmem_ld_32x32b_x32(taddr + c, ra);
        if (kEpi == kFfnGlu) tc::tmem_ld_32x32b_x32(taddr + TN / 2 + c, rb);
        tc::tmem_ld_wait(ra);
        if (kEpi == kFfnGlu) tc::tmem_ld_wait(rb);
        const int n = n0 + c, left = q.N - n;
        if (m < q.M && left > 0) {
          const size_t at = (size_t)m * q.N + n;
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(ra[i]);
          if (kEpi == kFfnGlu) {
            float w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __uint_as_float(rb[i]);
            if (a.out2) store_row<T>((T*)a.out2 + at, v, left);
            if (a.out3) store_row<T>((T*)a.out3 + at, w, left);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = act_value(v[i], a.act) * w[i];
            store_row<T>((T*)q.out + at, v, left);
          } else if (kEpi == kFfnDglu) {
            constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
            for (int i = 0; i < 32 / V; ++i)
              if (i * V < left) {
                float g[V], w[V], dg[V], du[V];
                load_vec<T, V>((const T*)a.in1 + at + i * V, g);
                load_vec<T, V>((const T*)a.in2 + at + i * V, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                  float slope;
                  const float act = act_both(g[j], a.act, slope);
                  dg[j] = v[i * V + j] * w[j] * slope;
                  du[j] = v[i * V + j] * act;
                }
                store_vec<T, V>((T*)q.out + at + i * V, dg);
                store_vec<T, V>((T*)a.out2 + at + i * V, du);
              }
          } else if (q.split > 1) {
            store_row<float>(q.part + (size_t)t.s * q.M * q.N + at, v, left);
          } else {
            store_row<T>((T*)q.out + at, v, left);
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      // orders only TMEM reads (the tcgen05 fence), so a pair's arrival is relaxed
      if (lane == 0) {
        if (kPair) tc::mbar_arrive_cluster_relaxed(acc_empty0 + 8u * (uint32_t)buf);
        else tc::mbar_arrive(&acc_empty[buf]);
      }
      if (++buf == 2) { buf = 0; acc_phase ^= 1u; }
    }
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

// out = sum of the split partial sums, in order; four columns per thread.
template <class T>
__global__ void __launch_bounds__(256)
ffn_reduce_kernel(const __grid_constant__ Args a) {
  griddep_launch_dependents();
  griddep_wait();
  for (int p = 0; p < a.nprob; ++p) {
    const Prob& q = a.prob[p];
    if (q.split < 2) continue;
    const size_t n = (size_t)q.M * q.N;
    for (size_t i = 4 * ((size_t)blockIdx.x * blockDim.x + threadIdx.x); i < n; i += 4 * (size_t)gridDim.x * blockDim.x) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int s = 0; s < q.split; ++s) {
        const float4 w = __ldcs(reinterpret_cast<const float4*>(q.part + s * n + i));
        v[0] += w.x; v[1] += w.y; v[2] += w.z; v[3] += w.w;
      }
      store_vec<T, 4>((T*)q.out + i, v);
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
  pl.pair = big >= kSms / 4;
  const int t = pl.pair ? 256 : 128, slots = pl.pair ? kSms / 2 : kSms;
  long long total = 0;
  for (int p = 0; p < l.nprob; ++p) total += tiles(l.prob[p], t);
  long long units = 0;
  size_t off = 0;
  for (int p = 0; p < l.nprob; ++p) {
    const FfnProblem& q = l.prob[p];
    const int kbs = ceil_div(q.K, BK), nkb = kbs * q.nseg;
    long long split = l.epi == kFfnStore && total < slots ? slots / total : 1;
    if (split > nkb / 4) split = nkb / 4;
    split = split < 1 ? 1 : split > kMaxSplit ? kMaxSplit : split;
    if (a) {
      Prob& r = a->prob[p];
      r.M = q.M; r.N = q.N; r.kbs = kbs; r.nkb = nkb; r.a_mn = q.a_mn; r.b_mn = q.b_mn;
      for (int s = 0; s < 12; ++s) { r.a[s] = q.a[s]; r.b[s] = q.b[s]; r.a_plane[s] = q.a_plane[s]; r.b_plane[s] = q.b_plane[s]; }
      r.b_up = q.b_up;
      r.tiles_m = ceil_div(q.M, t); r.tiles_n = ceil_div(q.N, t / feat); r.split = (int)split; r.begin = (int)units;
      r.out = q.out;
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

bool encode_planes(CUtensorMap* map, const FfnOperand& o, int dtype) {
  return encode_tmap_3d_planes(map, o.p, dtype, (uint64_t)o.cols, (uint64_t)o.rows, (uint64_t)o.planes, 64, 64);
}

int device_sms() {
  int sms = kSms, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <bool kPair, int kEpi, class T>
cudaError_t go(const Maps& maps, const Args& a, cudaStream_t s) {
  auto kernel = ffn_tc_kernel<kPair, kEpi, T>;
  cudaError_t e = set_max_dynamic_smem((const void*)kernel, kSmemBytes);
  if (e != cudaSuccess) return e;
  const int slots = kPair ? device_sms() / 2 : device_sms();
  const int n = a.units < slots ? a.units : slots;
  e = launch_dependent(kernel, dim3((unsigned)(kPair ? 2 * n : n)), dim3(kThreads), kSmemBytes, s, kPair ? 2 : 1, maps, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <int kEpi, class T>
cudaError_t go_pair(bool pair, const Maps& maps, const Args& a, cudaStream_t s) {
  return pair ? go<true, kEpi, T>(maps, a, s) : go<false, kEpi, T>(maps, a, s);
}

template <class T>
cudaError_t go_type(const FfnLaunch& l, const Plan& pl, const Maps& maps, const Args& a, cudaStream_t s) {
  if (l.epi == kFfnGlu) return go_pair<kFfnGlu, T>(pl.pair, maps, a, s);
  if (l.epi == kFfnDglu) return go_pair<kFfnDglu, T>(pl.pair, maps, a, s);
  cudaError_t e = go_pair<kFfnStore, T>(pl.pair, maps, a, s);
  if (e != cudaSuccess || !pl.split_any) return e;
  size_t most = 0;
  for (int p = 0; p < a.nprob; ++p)
    if (a.prob[p].split > 1 && (size_t)a.prob[p].M * a.prob[p].N > most) most = (size_t)a.prob[p].M * a.prob[p].N;
  const size_t want = (most / 4 + 255) / 256;
  e = launch_dependent(ffn_reduce_kernel<T>, dim3((unsigned)(want < 8 * kSms ? want : 8 * kSms)), dim3(256), 0, s, 1, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

size_t ffn_tc_partial_bytes(const FfnLaunch& l) { return make_plan(l, nullptr).partial_bytes; }

cudaError_t launch_ffn_tc(const FfnLaunch& l, float* partial, unsigned* st, cudaStream_t s) {
  Maps maps;
  for (int i = 0; i < l.nop; ++i)
    if (!encode_planes(&maps.m[i], l.op[i], l.op_dtype)) return cudaErrorInvalidValue;
  Args a{};
  const Plan pl = make_plan(l, &a);
  for (int p = 0; p < a.nprob; ++p) a.prob[p].part = (float*)((char*)partial + (size_t)a.prob[p].part);
  a.act = l.act;
  a.ab_bf16 = l.op_dtype == SWIMBA_BF16;
  a.out2 = l.out2; a.out3 = l.out3; a.in1 = l.in1; a.in2 = l.in2;
  a.st = st;
  return l.dtype == SWIMBA_BF16 ? go_type<__nv_bfloat16>(l, pl, maps, a, s) : go_type<__half>(l, pl, maps, a, s);
}

}  // namespace swimba
