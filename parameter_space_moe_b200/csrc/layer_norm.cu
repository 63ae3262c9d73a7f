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
// the stored r, so that no caller has to keep them.
//
// Bounds.  Times are of captured passes over sets of inputs in turn, larger than L2 together; in brackets a user's calls on
// inputs written in between, whose lines then leave L2 beside the pass.  Forward: HBM (32768 x 2048 bf16 with the residual
// sum, 537 MB: 90 us, 0.91 of a copy's rate; [100 us, 0.82]).  Gradients: instructions and the latency of a row's four sums
// at 128 registers a thread, two blocks an SM (8192 x 768 bf16 / f32, 88 MB: 22.7 us with the partial sums' launch, 0.59 of
// a copy's rate; [24.6 us]).  Few rows: one launch's latency (256 x 2048: 3.5 us; [8 us, the host's call]).
#include "block_common.cuh"

namespace swimba {

namespace {

// A row belongs to a team of whole warps, thread i of which holds the vectors i, i + team, ... of VEC columns; a block is
// as many teams as its threads allow.  Sums over a warp and addresses cost the same for few columns a thread as for many;
// more threads hide more latency.  Columns of a thread, at most (M x D, dtype / gradients' dtype; both sides of a choice
// measured on the same inputs again and again, the ones taken within 3 % of that over sets in turn):
//   forward            16   32768 x 2048 bf16 with the residual sum: 88 us; 24 columns 102 us
//     of odd widths     8   20000 x 1001 bf16 with the residual sum: 62 us; 16 columns (spills) 94 us
//   16-bit gradients   16   8192 x 768 bf16 / f32 (12 columns): 25 us before gamma was kept; 8 columns 32 us.  20000 x 2048
//                           bf16 (16 columns, one block of 384 threads an SM, whose registers do not spill): 94 us; two
//                           of 256 96 us
//   f32 gradients       8   5000 x 1500: 35 us with the rows ahead in shared memory; 16 in registers 45 us
//     of odd widths     8   4099 x 1001 f32: 18 us with two blocks an SM; 4 columns 22 us, 8 with three (spills) 38 us
// 8 where there are few rows, and 16, 24 or, in blocks of 512 threads, 32 where a block would not hold the row otherwise.
constexpr int kMaxThreads = 512;
constexpr int threads_of(bool wide) { return wide ? kMaxThreads : 256; }
constexpr int kFwdBlocks = 3;  // of 256 threads, on an SM
constexpr int bwd_blocks(int cols, bool async) { return async ? (cols <= 8 ? 4 : cols <= 16 ? 3 : 2) : cols <= 12 ? 2 : 1; }
constexpr int bwd_threads(int cols, bool async, bool wide) { return wide ? kMaxThreads : !async && cols > 12 ? 384 : 256; }
constexpr int bwd_cols(int vec, bool async) { return vec == 1 ? 8 : async ? 8 : 16; }

// Sums go through shared memory where a team has several warps: `red` holds two copies, used in turn, so that one barrier
// of the team per sum is enough.
struct Team {
  int team, group, lane, first_warp, warps;
  float2 (*red)[kMaxThreads / 32];
  int which;
  __device__ __forceinline__ Team(int team_, float2 (*red_)[kMaxThreads / 32])
      : team(team_), group(threadIdx.x / team_), lane(threadIdx.x - group * team_), first_warp(group * (team_ / 32)),
        warps(team_ / 32), red(red_), which(0) {}
  __device__ __forceinline__ float2 sum(float a, float b) {
    // one exchange sorts a into the lower half-warp and b into the upper, four more sum both at once
    const bool up = threadIdx.x & 16;
    float x = up ? b : a;
    x += __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (warps == 1) return make_float2(__shfl_sync(0xffffffffu, x, 0), __shfl_sync(0xffffffffu, x, 16));
    if ((threadIdx.x & 15) == 0) reinterpret_cast<float*>(&red[which][threadIdx.x >> 5])[up] = x;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(team) : "memory");
    float2 s = make_float2(0.f, 0.f);
    for (int w = 0; w < warps; ++w) {
      const float2 t = red[which][first_warp + w];
      s.x += t.x;
      s.y += t.y;
    }
    which ^= 1;
    return s;
  }
  __device__ __forceinline__ float sum(float a) {
    a = warp_sum(a);
    if (warps == 1) return a;
    if ((threadIdx.x & 31) == 0) red[which][threadIdx.x >> 5].x = a;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(team) : "memory");
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += red[which][first_warp + w].x;
    which ^= 1;
    return s;
  }
};

// VEC values as they lie in memory, for a load that is issued one row ahead of its use.
template <class T, int VEC>
struct Raw {
  static constexpr int kWords = VEC * (int)sizeof(T) >= 4 ? VEC * (int)sizeof(T) / 4 : 1;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int b = 0; b < kWords / 4; ++b) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[b];
        w[4 * b] = u.x; w[4 * b + 1] = u.y; w[4 * b + 2] = u.z; w[4 * b + 3] = u.w;
      }
    } else if constexpr (kWords == 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x; w[1] = u.y;
    } else if constexpr (sizeof(T) == 4) {
      static_assert(VEC == 1, "vectors of 8 or 16 bytes");
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      static_assert(VEC == 1, "vectors of 8 or 16 bytes");
      w[0] = *reinterpret_cast<const unsigned short*>(p);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int b = 0; b < kWords; ++b) w[b] = 0u;
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[j]);
    } else {
      const unsigned short u = (unsigned short)(w[j / 2] >> (16 * (j % 2)));
      T t;
      memcpy(&t, &u, 2);
      return to_f32(t);
    }
  }
};

template <class T, int VEC, int NV>
struct Row {
  Raw<T, VEC> v[NV];
  // This thread's vectors of the row, at p, p + gap, ...; the first `live` of them hold columns, the others are 0.
  __device__ __forceinline__ void load(const T* p, int gap, int live) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i < live) v[i].load(p + i * gap);
      else v[i].zero();
    }
  }
};

template <class T, int VEC, int NV, bool kWide>
__global__ void __launch_bounds__(threads_of(kWide), kWide ? 1 : kFwdBlocks)
layer_norm_kernel(int M, int D, int team, long long xs, float eps, const T* __restrict__ x, const T* residual,
                  const float* __restrict__ gamma, const float* __restrict__ beta, T* y, T* r_out) {
  __shared__ float2 red[2][kMaxThreads / 32];
  Team k(team, red);
  const int groups = blockDim.x / team, step = gridDim.x * groups;
  const int c0 = k.lane * VEC, gap = team * VEC;                   // this thread's columns: c0, c0 + gap, ...
  const int live = c0 < D ? ((D - c0) / VEC + team - 1) / team : 0;  // vectors of them
  const float inv = 1.f / D;
  Row<T, VEC, NV> rx, rr;
  int m = blockIdx.x * groups + k.group;
  x += m * xs + c0;
  residual += residual ? (size_t)m * D + c0 : 0;
  const size_t at0 = (size_t)m * D + c0;
  y += at0;
  if (r_out) r_out += at0;
  const long long xstep = step * xs, dstep = (long long)step * D;
  auto fetch = [&](bool in) {
    rx.load(x, gap, in ? live : 0);
    rr.load(residual, gap, in && residual ? live : 0);
    x += xstep;
    if (residual) residual += dstep;
  };
  constexpr bool kAhead = !kWide;  // the next row's loads are issued before this row's sums
  if (kAhead) fetch(m < M);
  for (; m < M; m += step) {
    if (!kAhead) fetch(true);
    float v[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] = rx.v[i].get(j);
        if (residual) v[i][j] += rr.v[i].get(j);
        s += v[i][j];
      }
      if (r_out && i < live) store_vec<T, VEC>(r_out + i * gap, v[i]);
    }
    if (kAhead) fetch(m + step < M);
    const float mu = k.sum(s) * inv;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i < live) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] -= mu;
          sq += v[i][j] * v[i][j];
        }
      }
    const float rstd = rsqrtf(k.sum(sq) * inv + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i < live) {
        float g[VEC], b[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) { g[j] = 1.f; b[j] = 0.f; }
        if (gamma) load_vec<float, VEC>(gamma + c0 + i * gap, g);
        if (beta) load_vec<float, VEC>(beta + c0 + i * gap, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = v[i][j] * rstd * g[j] + b[j];
        store_vec<T, VEC>(y + i * gap, v[i]);
      }
    }
    y += dstep;
    if (r_out) r_out += dstep;
  }
}

// A thread's vectors of one row of T, one row ahead of their use: copied asynchronously to shared memory that this thread
// alone reads, or loaded to registers.
template <class T, int VEC, int NV, bool kAsync>
struct Ahead {
  static constexpr int kBytes = VEC * (int)sizeof(T);  // 16 in shared memory
  Row<T, VEC, kAsync ? 1 : NV> reg;
  uint8_t* mem;
  int stride;
  // mem_: the block's room for this row, `team` vectors of each turn together
  __device__ __forceinline__ void init(uint8_t* mem_, const Team& k) {
    mem = mem_ + k.lane * kBytes;
    stride = k.team * kBytes;
  }
  // The first `live` of this thread's vectors, at p, p + gap, ...
  __device__ __forceinline__ void fetch(const T* p, int gap, int live) {
    if constexpr (kAsync) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < live) {
          const uint32_t to = (uint32_t)__cvta_generic_to_shared(mem + i * stride);
          static_assert(kBytes == 16, "one copy per vector");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p + i * gap) : "memory");
        }
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
      reg.load(p, gap, live);
    }
  }
  __device__ __forceinline__ void get(int i, float (&v)[VEC]) const {
    if constexpr (kAsync) {
      load_vec<T, VEC>(reinterpret_cast<const T*>(mem + i * stride), v);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = reg.v[i].get(j);
    }
  }
};

// Gradients of the block's rows.  A thread keeps its columns' sums of dy xhat and dy over all of them; the teams' sums
// meet in shared memory and go to part[blockIdx.x][2][D] when `part` is given.  kAll: gamma is given, and every vector of every
// thread holds columns, of single columns every one but a thread's last, so that nothing is tested or set to 0 or 1 on the
// way.  16 columns in vectors (20000 x 2048 bf16: 101 -> 92 us) and 8 single ones (20000 x 1001 bf16: 74 -> 64 us); with
// others the compiler spills what it no longer tests (8192 x 768 f32: 25.8 -> 30.8 us).
template <class T, class G, int VEC, int NV, bool kWide, bool kAsync, bool kAll>
__global__ void __launch_bounds__(bwd_threads(NV* VEC, kAsync, kWide), kWide ? 1 : bwd_blocks(NV* VEC, kAsync))
layer_norm_bwd_kernel(int M, int D, int team, float eps, const T* __restrict__ r, const float* __restrict__ gamma,
                      const G* dy, const G* dr, G* dx, float* __restrict__ part) {
  __shared__ float2 red[2][kMaxThreads / 32];
  extern __shared__ __align__(16) uint8_t room[];  // the teams' rows ahead, then [teams][2 D] sums
  griddep_launch_dependents();
  Team k(team, red);
  const int groups = blockDim.x / team, step = gridDim.x * groups;
  const int c0 = k.lane * VEC, gap = team * VEC;                   // this thread's columns: c0, c0 + gap, ...
  constexpr int kSure = kAll ? (VEC == 1 ? NV - 1 : NV) : 0;
  const int live = kSure == NV ? NV : c0 < D ? ((D - c0) / VEC + team - 1) / team : 0;  // vectors of them
  const float inv = 1.f / D;
  Ahead<T, VEC, NV, kAsync> ar;
  Ahead<G, VEC, NV, kAsync> ad, as;
  const int slots = NV * gap;  // columns of a team's row
  uint8_t* mine = room + (size_t)k.group * slots * (sizeof(T) + 2 * sizeof(G));
  ar.init(mine, k);
  ad.init(mine + (size_t)slots * sizeof(T), k);
  as.init(mine + (size_t)slots * (sizeof(T) + sizeof(G)), k);
  float ag[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) ag[i][j] = ab[i][j] = 0.f;
  // gamma stays in registers where a thread has few columns (8192 x 768 bf16 / f32, 12 columns: 26 -> 22.7 us)
  constexpr bool kKeep = NV * VEC <= (kAsync ? 8 : 12);
  float kept[kKeep ? NV : 1][VEC];
  auto load_gamma = [&](int i, float (&g)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[j] = 1.f;
    if ((kAll || gamma) && (i < kSure || i < live)) load_vec<float, VEC>(gamma + c0 + i * gap, g);
  };
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) load_gamma(i, kept[i]);
  }
  auto get_gamma = [&](int i, float (&g)[VEC]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) g[j] = kept[i][j];
    } else {
      load_gamma(i, g);
    }
  };
  int m = blockIdx.x * groups + k.group;
  const size_t at0 = (size_t)m * D + c0;
  const long long dstep = (long long)step * D;
  r += at0;
  dy += at0;
  if (dr) dr += at0;
  dx += at0;
  auto fetch_in = [&](bool in) {
    ar.fetch(r, gap, in ? live : 0);
    ad.fetch(dy, gap, in ? live : 0);
    r += dstep;
    dy += dstep;
  };
  auto fetch_dr = [&](bool in) {
    as.fetch(dr, gap, in && dr ? live : 0);
    if (dr) dr += dstep;
  };
  const bool with_dr = dr != nullptr;
  fetch_in(m < M);
  fetch_dr(m < M);
  for (; m < M; m += step) {
    if (kAsync) asm volatile("cp.async.wait_group 1;" ::: "memory");  // r and dy are here, dr perhaps
    float v[NV][VEC], d[NV][VEC];
    float s = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float gm[VEC];
      get_gamma(i, gm);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = d[i][j] = 0.f;
      if (i < kSure || i < live) {
        ar.get(i, v[i]);
        ad.get(i, d[i]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s += v[i][j];
        sg += d[i][j] * gm[j];
      }
    }
    const float2 t1 = k.sum(s, sg);
    fetch_in(m + step < M);  // behind the sum, which has read all that this overwrites
    const float mu = t1.x * inv, mg = t1.y * inv;
    float sq = 0.f, sgc = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i < kSure || i < live) {
        float gm[VEC];
        get_gamma(i, gm);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] -= mu;
          sq += v[i][j] * v[i][j];
          sgc += d[i][j] * gm[j] * v[i][j];
        }
      }
    }
    const float2 t2 = k.sum(sq, sgc);
    const float rstd = rsqrtf(t2.x * inv + eps), mgx = t2.y * inv * rstd;
    if (kAsync) asm volatile("cp.async.wait_group 2;" ::: "memory");  // dr too
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i < kSure || i < live) {
        float gm[VEC], o[VEC];
        get_gamma(i, gm);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = 0.f;
        if (with_dr) as.get(i, o);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = v[i][j] * rstd;
          o[j] += rstd * (d[i][j] * gm[j] - mg - xh * mgx);
          ag[i][j] += d[i][j] * xh;
          ab[i][j] += d[i][j];
        }
        store_vec<G, VEC>(dx + i * gap, o);
      }
    }
    dx += dstep;
    fetch_dr(m + step < M);  // behind the stores, which have read what this overwrites
  }
  if (!part) return;
  if (kAsync) asm volatile("cp.async.wait_all;" ::: "memory");
  float* to = part + (size_t)blockIdx.x * 2 * D;
  float* sums = reinterpret_cast<float*>(room);
  if (groups > 1) {
    __syncthreads();  // every team is done with its rows' room
    to = sums + (size_t)k.group * 2 * D;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * gap;
    if (i < kSure || i < live) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) { to[c + j] = ag[i][j]; to[D + c + j] = ab[i][j]; }
    }
  }
  if (groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) {
      float t = 0.f;
      for (int g = 0; g < groups; ++g) t += sums[(size_t)g * 2 * D + c];
      part[(size_t)blockIdx.x * 2 * D + c] = t;
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
  griddep_wait();  // the partial sums
  if (c < 2 * D) {
#pragma unroll 8
    for (int p = threadIdx.y; p < P; p += 32) s += part[(size_t)p * 2 * D + c];
  }
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

// Vectors per thread, threads per row (a team), teams per block and blocks.
struct Shape {
  int nv, team, groups, blocks;
  bool wide;
};
constexpr int kCounts[] = {1, 2, 3, 4, 6, 8, 16, 24};  // the vector counts that are compiled
// most: columns of a thread.
Shape shape_of(int M, int D, int vec, int most, bool bwd, bool async) {
  const int n = ceil_div(D, vec);
  if (M < 4 * 148 && D <= 8 * 256) most = 8;  // few rows
  Shape s{0, 0, 1, 0, true};
  int best = 0;  // the share of a team's vectors that hold columns, in 1/64
  for (int warps = 1; warps <= 8 && best < 55; ++warps)
    for (int c : kCounts)
      if (c * vec <= most && c * 32 * warps >= n) {
        const int share = 64 * n / (c * 32 * warps);
        if (share > best) { best = share; s.nv = c; s.team = 32 * warps; s.wide = false; }
        break;
      }
  if (s.wide && most < 24) return shape_of(M, D, vec, most < 8 ? 8 : most < 16 ? 16 : 24, bwd, async);
  if (s.wide) {
    s.nv = kMaxThreads * (16 / vec) >= n ? 16 / vec : 32 / vec;
    s.team = 32 * ceil_div(n, 32 * s.nv);
  }
  // as many teams as a block takes, as long as every SM has rows for them
  const int threads = bwd ? bwd_threads(s.nv * vec, async, s.wide) : threads_of(s.wide);
  while ((s.groups + 1) * s.team <= threads && (long long)(s.groups + 1) * 148 <= M) ++s.groups;
  const int want = ceil_div(M, s.groups), cap = 148 * (s.wide ? 1 : bwd ? bwd_blocks(s.nv * vec, async) : kFwdBlocks);
  s.blocks = want < cap ? want : cap;
  return s;
}

// f(integral constants nv, wide) for what shape_of can choose: at most 24 columns a thread, 32 in wide rows.
template <int VEC, int NV, class F>
void with_wide(const Shape& s, F f) {
  if constexpr (NV * VEC <= 24) {
    if (!s.wide) return f(std::integral_constant<int, NV>{}, std::false_type{});
  }
  if constexpr (NV * VEC == 16 || NV * VEC == 32) {
    if (s.wide) f(std::integral_constant<int, NV>{}, std::true_type{});
  }
}
template <int VEC, class F>
void with_shape(const Shape& s, F f) {
  switch (s.nv) {
    case 1: return with_wide<VEC, 1>(s, f);
    case 2: return with_wide<VEC, 2>(s, f);
    case 3: return with_wide<VEC, 3>(s, f);
    case 4: return with_wide<VEC, 4>(s, f);
    case 6: return with_wide<VEC, 6>(s, f);
    case 8: return with_wide<VEC, 8>(s, f);
    case 16: return with_wide<VEC, 16>(s, f);
    case 24: return with_wide<VEC, 24>(s, f);
    case 32: return with_wide<VEC, 32>(s, f);
  }
}

// Row vectors are 16 bytes of the widest type that is read in them: D must keep every row aligned.
template <class T>
constexpr int full_vec() { return 16 / (int)sizeof(T); }
int bwd_vec(const NormDims& d) {
  const int v = d.dtype == SWIMBA_F32 || d.grad_dtype == SWIMBA_F32 ? 4 : 8;
  return d.D % v == 0 ? v : 1;
}
bool bwd_async(const NormDims& d) { return d.dtype == SWIMBA_F32 && bwd_vec(d) > 1; }
Shape bwd_shape(const NormDims& d) {
  const int vec = bwd_vec(d);
  return shape_of(d.M, d.D, vec, bwd_cols(vec, bwd_async(d)), true, bwd_async(d));
}

template <class T, int VEC>
cudaError_t fwd_t(const NormDims& d, const void* x, const void* residual, const float* gamma, const float* beta, void* y,
                  void* r_out, cudaStream_t s) {
  const Shape sh = shape_of(d.M, d.D, VEC, VEC == 1 ? 8 : 16, false, false);
  with_shape<VEC>(sh, [&](auto nv, auto wide) {
    layer_norm_kernel<T, VEC, decltype(nv)::value, decltype(wide)::value><<<sh.blocks, sh.groups * sh.team, 0, s>>>(
        d.M, d.D, sh.team, d.x_stride, d.eps, (const T*)x, (const T*)residual, gamma, beta, (T*)y, (T*)r_out);
  });
  count_launches(1);
  return cudaGetLastError();
}

template <class T, class G, int VEC>
cudaError_t bwd_t(const NormDims& d, const void* r, const float* gamma, const void* dy, const void* dr, void* dx,
                  float* dgamma, float* dbeta, float* part, cudaStream_t s) {
  const Shape sh = bwd_shape(d);
  if (!dgamma && !dbeta) part = nullptr;
  constexpr bool kAsync = sizeof(T) == 4 && VEC > 1;
  cudaError_t e = cudaSuccess;
  with_shape<VEC>(sh, [&](auto nv, auto wide) {
    constexpr int kNv = decltype(nv)::value;
    constexpr bool kWide = decltype(wide)::value;
    auto kernel = layer_norm_bwd_kernel<T, G, VEC, kNv, kWide, kAsync, false>;
    if constexpr (!kWide && !kAsync && kNv * VEC == (VEC == 1 ? 8 : 16)) {
      const int sure = VEC == 1 ? kNv - 1 : kNv;
      if (gamma && sure * VEC * sh.team <= d.D) kernel = layer_norm_bwd_kernel<T, G, VEC, kNv, kWide, kAsync, true>;
    }
    const size_t rows = kAsync ? (size_t)sh.groups * sh.nv * sh.team * VEC * (sizeof(T) + 2 * sizeof(G)) : 0;
    const size_t sums = sh.groups > 1 ? (size_t)sh.groups * 2 * d.D * 4 : 0, smem = rows > sums ? rows : sums;
    if (smem > 40 * 1024) e = set_max_dynamic_smem((const void*)kernel, smem);
    if (e != cudaSuccess) return;
    kernel<<<sh.blocks, sh.groups * sh.team, smem, s>>>(d.M, d.D, sh.team, d.eps, (const T*)r, gamma, (const G*)dy,
                                                        (const G*)dr, (G*)dx, part);
  });
  if (e != cudaSuccess) return e;
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (part) {
    e = launch_dependent(layer_norm_params_kernel, dim3(ceil_div(2 * d.D, 32)), dim3(32, 32), 0, s, 1, sh.blocks, d.D,
                         (const float*)part, dgamma, dbeta);
    if (e == cudaSuccess) count_launches(1);
  }
  return e;
}

template <class T, class G>
cudaError_t bwd_v(const NormDims& d, const void* r, const float* gamma, const void* dy, const void* dr, void* dx,
                  float* dgamma, float* dbeta, float* part, cudaStream_t s) {
  constexpr int V = sizeof(T) == 4 || sizeof(G) == 4 ? 4 : 8;
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

size_t layer_norm_bwd_ws(const NormDims& d) { return align_up((size_t)bwd_shape(d).blocks * 2 * d.D * 4, 256); }

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
