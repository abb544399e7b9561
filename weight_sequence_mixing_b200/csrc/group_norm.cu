// Group norm with an activation (ttt_ops.h, ttt_norm_*).
//
// Statistics of a group run over the N tokens and the C / groups channels of one batch
// entry.  sum x^2 - n mean^2 would lose the digits of a group whose mean is large, and the
// sum of squares about the mean takes a second pass over the data.  So runs of at most 32
// tokens are summed about their own first value, which a run's spread is never far
// below, and parts (count n_k, mean_k, S_k the sum of squares about it) are
// joined by
//   mean = sum n_k mean_k / n,   S = sum S_k + n_k (mean_k - mean)^2
// (two at a time: Chan, Golub, LeVeque 1979), in an order that is fixed by the sizes alone.
//
// Two forms.  A small group (16384 values at most, of a small tensor) is one block's, in
// shared memory.  Else a first kernel forms the statistics of (token range, channel) blocks
// and a second, launched behind it, joins them and normalises: x is read twice where L2
// does not keep it (the second kernel walks backwards, from what was read last).
//
// Measured, SiLU, bf16: 2 x 1048576 tokens x 128 channels in 32 groups, statistics 83 us (98%
// of the copy bandwidth), application 190 us (86%; a reciprocal shared by two values or an
// exponential from the FMA pipe gained 2%), backward sums 183 us (90%) and dx 264 us (93%).
// 8 x 6084 tokens of 6 heads of 64 (in L2): 10 and 19 us.
#include <cmath>
#include <algorithm>
#include <new>

#include "op_checks.h"
#include "per_device.h"
#include "tc_gemm.cuh"
#include "ttt_plan.cuh"
#include "vec.cuh"

namespace ttt {
namespace {

constexpr int kThreads = 256;
constexpr int kSmallThreads = 512;  // of a block that has a group to itself
constexpr int kRun = 32;  // tokens summed about one value; a multiple of the loads under way

struct NormArgs {
  const void *x, *dy;
  void *y, *dx;
  const float *weight, *bias;
  float *stats, *dweight, *dbias;        // stats [B][G][2]
  float2* parts;         // of each block and group: forward (mean, S), backward (sum q, sum q xhat)
  float2* channel_sums;  // backward: [B][ranges][C] (sum dz, sum dz xhat)
  int64_t xs[3], ys[3], dys[3], dxs[3];  // batch, group, token
  int64_t N;
  int32_t B, C, G, n;                    // n channels a group
  float eps;
  int32_t lanes, rows;                   // a block's vectors of channels, and tokens at a time
  int32_t col_blocks, row_blocks;        // blocks of channels; ranges of tokens
  int32_t range;                         // tokens of a range
  int32_t slots;                         // groups of a block of channels at most
};

// Group k's (mean, 1 / sqrt(var + eps)), each on its own: the caller's buffer is aligned to its elements only
__device__ __forceinline__ float2 load_stats(const float* stats, int64_t k) { return make_float2(stats[2 * k], stats[2 * k + 1]); }
__device__ __forceinline__ void store_stats(float* stats, int64_t k, float2 m) { stats[2 * k] = m.x, stats[2 * k + 1] = m.y; }

struct Part {  // of n values: their mean, and S the sum of squares about it
  float n, mean, S;
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m; m /= 2) v += __shfl_xor_sync(~0u, v, m);
  return v;
}
// Joins `all` parts, the warp's lanes taking them in turn: first the mean (about the first
// part's, so that it keeps its digits), then S about it.  get(e, part) loads part e; its n may
// be 0 but for the first.  Up to 256 parts are loaded once, all loads before the first sum;
// more are loaded again for the second.
template <class F>
__device__ __forceinline__ Part join_parts(int all, F&& get) {
  constexpr int kHeld = 8;
  const int lane = threadIdx.x % 32;
  Part first, v[kHeld];
  get(0, first);
  auto pass = [&](auto&& add, bool again) {
    for (int e0 = lane; e0 < all; e0 += kHeld * 32) {
      if (again) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
          if (e0 + 32 * k < all) get(e0 + 32 * k, v[k]);
      }
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (e0 + 32 * k < all) add(v[k]);
    }
  };
  float n = 0.f, s = 0.f;
  pass([&](const Part& v) { n += v.n, s = fmaf(v.n, v.mean - first.mean, s); }, true);
  n = warp_sum(n);
  const float mean = first.mean + warp_sum(s) / n;
  float S = 0.f;
  pass([&](const Part& v) { S += fmaf(v.n * (v.mean - mean), v.mean - mean, v.S); }, all > kHeld * 32);
  return {n, mean, warp_sum(S)};
}
__device__ __forceinline__ float2 finish(const Part& v, float eps) {  // mean, 1 / sqrt(var + eps)
  return make_float2(v.mean, 1.f / sqrtf(v.S / v.n + eps));
}

// sigma(z).  bf16 outputs take the hardware's exponential (2^-22 off, and 2^-24 of the
// exponent's size), fp32 ones the library's; the reciprocal is the hardware's, 2^-23 off.
template <class T, class P>
__device__ __forceinline__ P sigmoid(P z) {
  P e;
  if constexpr (sizeof(T) == 4)
    e = each(z, [](float v) { return expf(-v); });
  else
    e = each(mul_(z, P::all(-1.4426950408889634f)), [](float v) { return exp2_fast(v); });
  return each(add_(e, P::all(1.f)), [](float v) { return rcp_fast(v); });
}
// z Phi(z) and its slope Phi(z) + z phi(z).  fp32 outputs take the library's erfc.  bf16 ones:
// Phi(-t) e^(t^2 / 2) falls slowly from 1/2 to 0.03 at t = 14, below which all is 0 in fp32; a
// polynomial of degree 7 in k = 1 / (1 + 0.35 t), fitted to it for the least relative error (by
// reweighted least squares on that interval, against 64 bits), is 3.1e-7 off, 7e-7 in fp32.  The
// error is relative in the tail too: z Phi(z) is 2^-15 off at z = -13, where the exponent's rounding
// is most of it, well below bf16's half step of 2^-9 everywhere.  (Formulas with an absolute bound,
// as the layer's MLP uses among larger terms, are 12% off at -5.5.)
constexpr float kInvSqrt2 = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kHalfLog2e = 0.72134752044448170f;
// Phi and e^(-z^2 / 2)
template <class P>
__device__ __forceinline__ P normal_cdf(P z, P& e) {
  const P t = each(z, [](float v) { return fabsf(v); });
  e = each(mul_(mul_(z, z), P::all(-kHalfLog2e)), [](float v) { return exp2_fast(v); });
  const P k = each(fma_(t, P::all(0.35f), P::all(1.f)), [](float v) { return rcp_fast(v); });
  P q = P::all(0.0489424331f);
  q = fma_(q, k, P::all(-0.202119248f));
  q = fma_(q, k, P::all(0.240640777f));
  q = fma_(q, k, P::all(-0.0170234009f));
  q = fma_(q, k, P::all(0.155961469f));
  q = fma_(q, k, P::all(0.133355098f));
  q = fma_(q, k, P::all(0.140270341f));
  q = fma_(q, k, P::all(-2.73155079e-5f));
  q = mul_(q, e);  // Phi(-t)
  const P rest = sub_(P::all(1.f), q);
  float v[P::N];
#pragma unroll
  for (int i = 0; i < P::N; ++i) v[i] = z[i] < 0.f ? q[i] : rest[i];
  return P::of(v);
}
template <class T, class P>
__device__ __forceinline__ P gelu(P z) {
  if constexpr (sizeof(T) == 4) return each(z, [](float v) { return v * 0.5f * erfcf(v * -kInvSqrt2); });
  P e;
  return mul_(z, normal_cdf(z, e));
}
template <class T, class P>
__device__ __forceinline__ P gelu_slope(P z) {
  if constexpr (sizeof(T) == 4)
    return each(z, [](float v) { return fmaf(v * kInvSqrt2Pi, expf(-0.5f * v * v), 0.5f * erfcf(v * -kInvSqrt2)); });
  P e;
  const P cdf = normal_cdf(z, e);
  return fma_(mul_(z, P::all(kInvSqrt2Pi)), e, cdf);
}
template <class T, int ACT, class P>
__device__ __forceinline__ P act(P z) {
  if constexpr (ACT == TTT_ACT_SILU) return mul_(z, sigmoid<T>(z));
  if constexpr (ACT == TTT_ACT_GELU) return gelu<T>(z);
  return z;
}
// the activation's slope at z, times dy
template <class T, int ACT, class P>
__device__ __forceinline__ P act_grad(P z, P dy) {
  if constexpr (ACT == TTT_ACT_SILU) {
    const P s = sigmoid<T>(z);
    return mul_(dy, fma_(mul_(z, s), sub_(P::all(1.f), s), s));
  }
  if constexpr (ACT == TTT_ACT_GELU) return mul_(dy, gelu_slope<T>(z));
  return dy;
}

// Where a thread's vector of channels lies
struct Column {
  bool here;
  int c;            // its first channel
  int64_t group, i; // that channel's group, and place in it
  __device__ __forceinline__ int64_t at(const int64_t (&s)[3], int b) const { return b * s[0] + group * s[1] + i; }
};
__device__ __forceinline__ Column column(const NormArgs& p, int col_block, int V) {
  const int v = col_block * p.lanes + threadIdx.x % p.lanes;
  Column k;
  k.c = v * V;
  k.here = threadIdx.x / p.lanes < p.rows && k.c < p.C;
  k.group = k.c / p.n;
  k.i = k.c % p.n;
  return k;
}
__device__ __forceinline__ int block_end(const NormArgs& p, int col_block, int V) {  // the channel behind a block's
  return min(p.C, (col_block + 1) * p.lanes * V);
}

// Statistics of one range of tokens and block of channels: a thread walks down its channels,
// Q of them (all of one group) to a sum; a warp then joins the threads' parts of each group.
template <class T, int BYTES, int Q>
__global__ void __launch_bounds__(kThreads, 3) norm_parts_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  using P = typename X::P;
  constexpr int V = X::N, K = V / Q, kPacks = X::kPacks, kSums = Q > 1 ? K : kPacks, kAtOnce = 8;
  extern __shared__ float2 threads[];  // [row][sum of the block]
  cudaTriggerProgrammaticLaunchCompletion();  // the next kernel's blocks may take the places that fall free
  const int cb = blockIdx.x, rb = blockIdx.y, b = blockIdx.z;
  const Column k = column(p, cb, V);
  const int row = threadIdx.x / p.lanes;
  const int64_t t0 = int64_t(rb) * p.range;
  const int tokens = int(min(int64_t(p.range), p.N - t0));
  const int width = p.lanes * V;
  if (k.here) {
    const T* x = static_cast<const T*>(p.x) + k.at(p.xs, b) + (t0 + row) * p.xs[2];
    const int64_t hop = p.rows * p.xs[2];
    float count = 0.f, mean[K] = {}, S[K] = {};
    int left = tokens > row ? (tokens - row + p.rows - 1) / p.rows : 0;
    X v[kAtOnce];  // each place takes the vector kAtOnce rows on as soon as it is free
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      if (e < left) v[e].load(x);
      x += e < left ? hop : 0;
    }
    while (left > 0) {
      const int run = min(left, kRun);
      P off[kPacks], s[kSums], q[kSums];  // off: less the run's first value; a pack's sums side by side
      {
        float f[V];
        v[0].open(f);
#pragma unroll
        for (int i = V - 1; i >= 0; --i) f[i] = -f[Q > 1 ? i / Q * Q : i];  // a sum's first is the last to change
#pragma unroll
        for (int i = 0; i < kPacks; ++i) off[i] = P::of(f + i * P::N);
#pragma unroll
        for (int i = 0; i < kSums; ++i) s[i] = P::all(0.f), q[i] = P::all(0.f);
      }
      for (int j = 0; j < run; j += kAtOnce) {
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
          if (j + e < run) {
            P f[kPacks];
            v[e].open(f);
            if (j + e + kAtOnce < left) {
              v[e].load(x);
              x += hop;
            }
#pragma unroll
            for (int i = 0; i < kPacks; ++i) {
              const P d = add_(f[i], off[i]);
              constexpr int kEach = kPacks / kSums;  // packs to a sum
              s[i / kEach] = add_(s[i / kEach], d);
              q[i / kEach] = fma_(d, d, q[i / kEach]);
            }
          }
      }
      const float n = float(run * Q), inv = 1.f / n, all = count + n, f = n / all;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        // Q > 1: both halves of a pack are of one sum
        const int w = Q > 1 ? i : i / P::N;
        const float sum = Q > 1 && P::N == 2 ? s[w][0] + s[w][P::N - 1] : s[w][i % P::N];
        const float squares = Q > 1 && P::N == 2 ? q[w][0] + q[w][P::N - 1] : q[w][i % P::N];
        const float first = -off[i * Q / P::N][i * Q % P::N];
        const float m = sum * inv, Si = fmaxf(fmaf(-sum, m, squares), 0.f);
        const float d = first + m - mean[i];
        if (count == 0.f) {
          mean[i] = first + m;
          S[i] = Si;
        } else {
          mean[i] = fmaf(d, f, mean[i]);
          S[i] += Si + d * d * count * f;
        }
      }
      count = all;
      left -= run;
    }
#pragma unroll
    for (int i = 0; i < K; ++i)
      threads[(row * p.lanes + threadIdx.x % p.lanes) * K + i] = make_float2(mean[i], S[i]);
  }
  __syncthreads();
  const int c0 = cb * width, c1 = block_end(p, cb, V), g0 = c0 / p.n;
  const int lane = threadIdx.x % 32, each = tokens / p.rows, more = tokens - each * p.rows;  // tokens of a thread
  for (int g = g0 + threadIdx.x / 32; g <= (c1 - 1) / p.n; g += kThreads / 32) {
    const int from = (max(g * p.n, c0) - c0) / Q, wide = (min((g + 1) * p.n, c1) - c0) / Q - from;
    const Part v = join_parts(p.rows * wide, [&](int e, Part& v) {
      const int r = e / wide;
      const float2 m = threads[r * (p.lanes * K) + from + e - r * wide];
      v = {float((each + (r < more ? 1 : 0)) * Q), m.x, m.y};
    });
    if (lane == 0)
      p.parts[((int64_t(b) * p.col_blocks + cb) * p.slots + g - g0) * p.row_blocks + rb] = make_float2(v.mean, v.S);
  }
}

// Where the blocks' parts of group g are, and how many values each is of.  Where all lie in
// one block of channels (the usual case) they follow one another and are of `each` values,
// the last of `end`.  A group's parts lie together: a block that joins them reads whole lines
// (1048576 x 128 bf16 in 32 groups: 444 parts a group, forward 187 us with a block's parts
// together instead, 156 so).
struct PartsOf {
  const NormArgs& p;
  const float2* parts;
  int g, width, first, blocks, all;
  float each, end;
  __device__ __forceinline__ PartsOf(const NormArgs& p, int b, int g, int V) : p(p), g(g), width(p.lanes * V) {
    first = g * p.n / width, blocks = ((g + 1) * p.n - 1) / width - first + 1;
    all = p.row_blocks * blocks;
    each = float(p.range), end = float(p.N - int64_t(p.row_blocks - 1) * p.range);
    parts = p.parts + int64_t(b) * p.col_blocks * p.slots * p.row_blocks;
    if (blocks == 1) {
      each *= float(p.n), end *= float(p.n);
      parts += int64_t(first * p.slots + g - first * width / p.n) * p.row_blocks;
    }
  }
  __device__ __forceinline__ float2 at(int e, float* values) const {
    if (blocks == 1) {
      *values = e == all - 1 ? end : each;
      return parts[e];
    }
    const int rb = e / blocks, cb = first + e - rb * blocks, c0 = cb * width;
    const float n = float(min((g + 1) * p.n, min(p.C, c0 + width)) - max(g * p.n, c0));
    *values = (rb == p.row_blocks - 1 ? end : each) * n;
    return parts[int64_t(cb * p.slots + g - c0 / p.n) * p.row_blocks + rb];
  }
};

// Joins the parts of its groups and normalises one range of tokens and block of channels.
template <class T, int BYTES, int Q, int ACT>
__global__ void __launch_bounds__(kThreads, 3) norm_apply_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  using P = typename X::P;
  // a pack's mean is shared by the packs of kStep channels
  constexpr int V = X::N, K = V / Q, kPacks = X::kPacks, kStep = Q > P::N ? Q : P::N, kMeans = V / kStep, kAtOnce = 6;
  extern __shared__ float2 known[];  // (mean, 1 / std) of the block's groups
  const int cb = gridDim.x - 1 - blockIdx.x, rb = gridDim.y - 1 - blockIdx.y, b = gridDim.z - 1 - blockIdx.z;
  const Column k = column(p, cb, V);
  const int row = threadIdx.x / p.lanes;
  const int c0 = cb * p.lanes * V, c1 = block_end(p, cb, V), g0 = c0 / p.n;
  cudaGridDependencySynchronize();  // the parts are there
  for (int g = g0 + threadIdx.x / 32; g <= (c1 - 1) / p.n; g += kThreads / 32) {
    const PartsOf of(p, b, g, V);
    const float2 m = finish(join_parts(of.all,
                                       [&](int e, Part& v) {
                                         const float2 m = of.at(e, &v.n);
                                         v.mean = m.x, v.S = m.y;
                                       }),
                            p.eps);
    if (threadIdx.x % 32 == 0) {
      known[g - g0] = m;
      if (p.stats && rb == 0 && g * p.n >= c0) store_stats(p.stats, int64_t(b) * p.G + g, m);
    }
  }
  __syncthreads();
  if (!k.here) return;
  float2 m[K];
#pragma unroll
  for (int j = 0; j < K; ++j) m[j] = known[(k.c + j * Q) / p.n - g0];
  P mean[kMeans], scale[kPacks], shift[kPacks];  // mean: negative
#pragma unroll
  for (int i = 0; i < V; i += P::N) {
    float a[P::N], s[P::N], o[P::N];
#pragma unroll
    for (int e = 0; e < P::N; ++e) {
      a[e] = -m[(i + e) / Q].x;
      s[e] = m[(i + e) / Q].y * (p.weight ? p.weight[k.c + i + e] : 1.f);
      o[e] = p.bias ? p.bias[k.c + i + e] : 0.f;
    }
    mean[i / kStep] = P::of(a);
    scale[i / P::N] = P::of(s);
    shift[i / P::N] = P::of(o);
  }
  const int64_t t0 = int64_t(rb) * p.range;
  const int tokens = int(min(int64_t(p.range), p.N - t0));
  const T* x = static_cast<const T*>(p.x) + k.at(p.xs, b) + (t0 + row) * p.xs[2];
  T* y = static_cast<T*>(p.y) + k.at(p.ys, b) + (t0 + row) * p.ys[2];
  const int mine = tokens > row ? (tokens - row + p.rows - 1) / p.rows : 0;
  const int64_t hop = p.rows * p.xs[2], yhop = p.rows * p.ys[2];
  x += (mine - 1) * hop;
  y += (mine - 1) * yhop;
  X v[kAtOnce];  // last row to first, the loads kAtOnce rows ahead
#pragma unroll
  for (int e = 0; e < kAtOnce; ++e) {
    if (e < mine) v[e].load(x);
    x -= e < mine ? hop : 0;
  }
  for (int left = mine; left > 0; left -= kAtOnce) {
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      if (e >= left) break;
      P f[kPacks];
      v[e].open(f);
      if (e + kAtOnce < left) {
        v[e].load(x);
        x -= hop;
      }
#pragma unroll
      for (int i = 0; i < kPacks; ++i)
        f[i] = act<T, ACT>(fma_(add_(f[i], mean[i * P::N / kStep]), scale[i], shift[i]));
      X o;
      o.close(f);
      o.store(y);
      y -= yhop;
    }
  }
}

// What the backward kernels know of a thread's channels: mean (negative) and 1 / std, one of
// each for the packs of kStep channels, weight and bias
template <class P, int PACKS, int MEANS>
struct Known {
  P mean[MEANS], rstd[MEANS], weight[PACKS], bias[PACKS];
  template <int STEP>
  __device__ __forceinline__ void load(const NormArgs& p, int b, int c) {
#pragma unroll
    for (int i = 0; i < PACKS; ++i) {
      float m[P::N], r[P::N], w[P::N], o[P::N];
#pragma unroll
      for (int e = 0; e < P::N; ++e) {
        const int k = c + i * P::N + e;
        const float2 s = load_stats(p.stats, int64_t(b) * p.G + k / p.n);
        m[e] = -s.x;
        r[e] = s.y;
        w[e] = p.weight ? p.weight[k] : 1.f;
        o[e] = p.bias ? p.bias[k] : 0.f;
      }
      mean[i * P::N / STEP] = P::of(m);
      rstd[i * P::N / STEP] = P::of(r);
      weight[i] = P::of(w);
      bias[i] = P::of(o);
    }
  }
};

template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t a = uint32_t(__cvta_generic_to_shared(to));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(a), "l"(from), "n"(BYTES) : "memory");
}
// Backward, of one range of tokens and block of channels: each channel's sums of dz and dz xhat.
// A thread's vectors of x and dy come through places of its own in shared memory, kAhead rows
// ahead: the slope's arithmetic needs the registers that as many rows would take (2 x 1048576 x
// 128, SiLU, bf16: backward 444 us, 494 with four rows at a time in registers).  Eight rows ahead
// take 437 us there, but 277 instead of 219 in fp32 without an activation (2 x 262144 x 128).
constexpr int kAhead = 4;
template <int BYTES>
constexpr int kRingBytes = BYTES >= 4 ? kAhead * 2 * kThreads * BYTES : 0;  // no asynchronous copy of 2 bytes
template <class T, int BYTES, int Q, int ACT>
__global__ void __launch_bounds__(kThreads, 2) norm_sums_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  using P = typename X::P;
  constexpr int V = X::N, kPacks = X::kPacks, kStep = Q > P::N ? Q : P::N, kMeans = V / kStep;
  extern __shared__ float2 threads[];
  cudaTriggerProgrammaticLaunchCompletion();
  const int cb = blockIdx.x, rb = blockIdx.y, b = blockIdx.z;
  const Column k = column(p, cb, V);
  const int row = threadIdx.x / p.lanes;
  const int64_t t0 = int64_t(rb) * p.range;
  const int tokens = int(min(int64_t(p.range), p.N - t0));
  const int width = p.lanes * V;
  if (k.here) {
    Known<P, kPacks, kMeans> q;
    q.template load<kStep>(p, b, k.c);
    P total0[kPacks], total1[kPacks];
#pragma unroll
    for (int i = 0; i < kPacks; ++i) total0[i] = total1[i] = P::all(0.f);
    const T* x = static_cast<const T*>(p.x) + k.at(p.xs, b) + (t0 + row) * p.xs[2];
    const T* dy = static_cast<const T*>(p.dy) + k.at(p.dys, b) + (t0 + row) * p.dys[2];
    const int64_t hop = p.rows * p.xs[2], dhop = p.rows * p.dys[2];
    const int mine = tokens > row ? (tokens - row + p.rows - 1) / p.rows : 0;
    // row j's place is filled again a step after it was read
    unsigned char* const ring = reinterpret_cast<unsigned char*>(threads + p.rows * width) + threadIdx.x * BYTES;
    int next = 0;
    auto fetch = [&] {
      if constexpr (BYTES >= 4) {
        if (next < mine) {
          unsigned char* const to = ring + (next % kAhead) * (2 * kThreads * BYTES);
          copy_async<BYTES>(to, x);
          copy_async<BYTES>(to + kThreads * BYTES, dy);
          x += hop;
          dy += dhop;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++next;
      }
    };
    for (int e = 0; e < kAhead - 1; ++e) fetch();
    for (int j0 = 0; j0 < mine; j0 += kRun) {  // sums of runs, so that no long sum swallows its terms
      P s0[kPacks], s1[kPacks];
#pragma unroll
      for (int i = 0; i < kPacks; ++i) s0[i] = s1[i] = P::all(0.f);
      const int end = min(j0 + kRun, mine);
#pragma unroll (BYTES >= 4 ? 1 : 4)
      for (int j = j0; j < end; ++j) {
        X v, d;
        if constexpr (BYTES >= 4) {
          fetch();
          asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
          const unsigned char* const from = ring + (j % kAhead) * (2 * kThreads * BYTES);
          v.load(reinterpret_cast<const T*>(from));
          d.load(reinterpret_cast<const T*>(from + kThreads * BYTES));
        } else {
          v.load(x);
          d.load(dy);
          x += hop;
          dy += dhop;
        }
        P f[kPacks], g[kPacks];
        v.open(f);
        d.open(g);
#pragma unroll
        for (int i = 0; i < kPacks; ++i) {
          const P xhat = mul_(add_(f[i], q.mean[i * P::N / kStep]), q.rstd[i * P::N / kStep]);
          const P dz = act_grad<T, ACT>(fma_(xhat, q.weight[i], q.bias[i]), g[i]);
          s0[i] = add_(s0[i], dz);
          s1[i] = fma_(dz, xhat, s1[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kPacks; ++i) total0[i] = add_(total0[i], s0[i]), total1[i] = add_(total1[i], s1[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      threads[row * width + (threadIdx.x % p.lanes) * V + i] =
          make_float2(total0[i / P::N][i % P::N], total1[i / P::N][i % P::N]);
  }
  __syncthreads();
  const int c0 = cb * width, c1 = block_end(p, cb, V), g0 = c0 / p.n;
  for (int c = threadIdx.x; c < c1 - c0; c += kThreads) {
    float2 s = threads[c];
    for (int r = 1; r < p.rows; ++r) {
      s.x += threads[r * width + c].x;
      s.y += threads[r * width + c].y;
    }
    p.channel_sums[(int64_t(b) * p.row_blocks + rb) * p.C + c0 + c] = s;
    threads[c] = s;
  }
  __syncthreads();
  // of each group the sums of q = dz weight and q xhat over this block
  for (int g = g0 + threadIdx.x / 32; g <= (c1 - 1) / p.n; g += kThreads / 32) {
    float q0 = 0.f, q1 = 0.f;
    for (int c = max(g * p.n, c0) + threadIdx.x % 32; c < min((g + 1) * p.n, c1); c += 32) {
      const float w = p.weight ? p.weight[c] : 1.f;
      q0 = fmaf(threads[c - c0].x, w, q0);
      q1 = fmaf(threads[c - c0].y, w, q1);
    }
#pragma unroll
    for (int m = 16; m; m /= 2) q0 += __shfl_xor_sync(~0u, q0, m), q1 += __shfl_xor_sync(~0u, q1, m);
    if (threadIdx.x % 32 == 0)
      p.parts[((int64_t(b) * p.col_blocks + cb) * p.slots + g - g0) * p.row_blocks + rb] = make_float2(q0, q1);
  }
}

// dweight and dbias: the channel sums of all ranges and batch entries, 32 channels a block
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float2 rows[32][32];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, r = threadIdx.x / 32;
  const int64_t all = int64_t(p.B) * p.row_blocks;
  cudaGridDependencySynchronize();
  float2 s = make_float2(0.f, 0.f);
  if (c < p.C)
    for (int64_t q = r; q < all; q += 32) {
      const float2 v = p.channel_sums[q * p.C + c];
      s.x += v.x;
      s.y += v.y;
    }
  rows[r][threadIdx.x % 32] = s;
  __syncthreads();
  if (r == 0 && c < p.C) {
#pragma unroll
    for (int q = 1; q < 32; ++q) s.x += rows[q][threadIdx.x].x, s.y += rows[q][threadIdx.x].y;
    if (p.dbias) p.dbias[c] = s.x;
    if (p.dweight) p.dweight[c] = s.y;
  }
}

// dx of one range of tokens and block of channels, walked backwards
template <class T, int BYTES, int Q, int ACT>
__global__ void __launch_bounds__(kThreads, 2) norm_dx_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  using P = typename X::P;
  constexpr int V = X::N, kPacks = X::kPacks, kStep = Q > P::N ? Q : P::N, kMeans = V / kStep, kAtOnce = 4;
  extern __shared__ float2 known[];  // (mean q, mean q xhat) of the block's groups
  const int cb = gridDim.x - 1 - blockIdx.x, rb = gridDim.y - 1 - blockIdx.y, b = gridDim.z - 1 - blockIdx.z;
  const Column k = column(p, cb, V);
  const int row = threadIdx.x / p.lanes;
  const int c0 = cb * p.lanes * V, c1 = block_end(p, cb, V), g0 = c0 / p.n;
  const float inv = 1.f / (float(p.N) * float(p.n));
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();  // the sums are there
  for (int g = g0 + threadIdx.x / 32; g <= (c1 - 1) / p.n; g += kThreads / 32) {
    float q0 = 0.f, q1 = 0.f;
    const PartsOf of(p, b, g, V);
    for (int e0 = threadIdx.x % 32; e0 < of.all; e0 += 8 * 32) {
      float2 s[8];
      float n;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (e0 + 32 * k < of.all) s[k] = of.at(e0 + 32 * k, &n);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (e0 + 32 * k < of.all) q0 += s[k].x, q1 += s[k].y;
    }
#pragma unroll
    for (int m = 16; m; m /= 2) q0 += __shfl_xor_sync(~0u, q0, m), q1 += __shfl_xor_sync(~0u, q1, m);
    if (threadIdx.x % 32 == 0) known[g - g0] = make_float2(q0 * inv, q1 * inv);
  }
  __syncthreads();
  if (!k.here) return;
  Known<P, kPacks, kMeans> q;
  q.template load<kStep>(p, b, k.c);
  P m0[kMeans], m1[kMeans];  // negative
#pragma unroll
  for (int i = 0; i < V; i += P::N) {
    float a[P::N], d[P::N];
#pragma unroll
    for (int e = 0; e < P::N; ++e) {
      const float2 m = known[(k.c + i + e) / p.n - g0];
      a[e] = -m.x;
      d[e] = -m.y;
    }
    m0[i / kStep] = P::of(a);
    m1[i / kStep] = P::of(d);
  }
  const int64_t t0 = int64_t(rb) * p.range;
  const int tokens = int(min(int64_t(p.range), p.N - t0));
  const T* x = static_cast<const T*>(p.x) + k.at(p.xs, b) + (t0 + row) * p.xs[2];
  const T* dy = static_cast<const T*>(p.dy) + k.at(p.dys, b) + (t0 + row) * p.dys[2];
  T* dx = static_cast<T*>(p.dx) + k.at(p.dxs, b) + (t0 + row) * p.dxs[2];
  const int mine = tokens > row ? (tokens - row + p.rows - 1) / p.rows : 0;
  const int64_t hop = p.rows * p.xs[2], dyhop = p.rows * p.dys[2], dxhop = p.rows * p.dxs[2];
  x += (mine - 1) * hop;
  dy += (mine - 1) * dyhop;
  dx += (mine - 1) * dxhop;
  for (int left = mine; left > 0; left -= kAtOnce) {
    X v[kAtOnce], d[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      if (e < left) {
        v[e].load(x);
        d[e].load(dy);
      }
      x -= e < left ? hop : 0;
      dy -= e < left ? dyhop : 0;
    }
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      if (e < left) {
        P f[kPacks], g[kPacks];
        v[e].open(f);
        d[e].open(g);
#pragma unroll
        for (int i = 0; i < kPacks; ++i) {
          const int s = i * P::N / kStep;
          const P xhat = mul_(add_(f[i], q.mean[s]), q.rstd[s]);
          const P dz = act_grad<T, ACT>(fma_(xhat, q.weight[i], q.bias[i]), g[i]);
          f[i] = mul_(q.rstd[s], fma_(xhat, m1[s], fma_(dz, q.weight[i], m0[s])));
        }
        v[e].close(f);
        v[e].store(dx);
      }
      dx -= dxhop;
    }
  }
}

// ---- a group of a batch entry by one block: its values in shared memory as fp32, each
// read and written by one thread; mean and variance in two passes there
__device__ __forceinline__ float2 block_sum(float2 v, float2* part) {
#pragma unroll
  for (int m = 16; m; m /= 2) v.x += __shfl_xor_sync(~0u, v.x, m), v.y += __shfl_xor_sync(~0u, v.y, m);
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < kSmallThreads / 32; ++i) v.x += part[i].x, v.y += part[i].y;
  return v;
}

// lanes and rows: of the group's own channels
template <class T, int BYTES, int ACT>
__global__ void __launch_bounds__(kSmallThreads) norm_small_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  constexpr int V = X::N, kAtOnce = 8;
  extern __shared__ float values[];
  __shared__ float2 part[kSmallThreads / 32];
  const int g = blockIdx.x, b = blockIdx.y;
  const int row = threadIdx.x / p.lanes, lane = threadIdx.x % p.lanes;
  const int N = row < p.rows ? int(p.N) : 0;
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + g * p.xs[1];
  T* y = static_cast<T*>(p.y) + b * p.ys[0] + g * p.ys[1];
  const float count = float(p.N) * float(p.n);
  float2 s = make_float2(0.f, 0.f);
  for (int i = lane * V; i < p.n; i += p.lanes * V)
    for (int t = row; t < N; t += kAtOnce * p.rows) {
      X v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (t + k * p.rows < N) v[k].load(x + (t + k * p.rows) * p.xs[2] + i);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (t + k * p.rows < N) {
          float f[V];
          v[k].open(f);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            values[(t + k * p.rows) * p.n + i + e] = f[e];
            s.x += f[e];
          }
        }
    }
  const float mean = block_sum(s, part).x / count;
  s = make_float2(0.f, 0.f);
  for (int i = lane * V; i < p.n; i += p.lanes * V)
#pragma unroll 4
    for (int t = row; t < N; t += p.rows)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = values[t * p.n + i + e] - mean;
        s.x = fmaf(d, d, s.x);
        s.y += d;
      }
  s = block_sum(s, part);
  // what the mean's rounding left over, taken off the variance and added to the mean
  const float off = s.y / count, centre = mean + off;
  const float rstd = 1.f / sqrtf(fmaxf(s.x / count - off * off, 0.f) + p.eps);
  if (p.stats && threadIdx.x == 0) store_stats(p.stats, int64_t(b) * p.G + g, make_float2(centre, rstd));
  for (int i = lane * V; i < p.n; i += p.lanes * V) {
    float scale[V], shift[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      scale[e] = rstd * (p.weight ? p.weight[g * p.n + i + e] : 1.f);
      shift[e] = p.bias ? p.bias[g * p.n + i + e] : 0.f;
    }
#pragma unroll 4
    for (int t = row; t < N; t += p.rows) {
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e)
        f[e] = act<T, ACT>(One{fmaf(values[t * p.n + i + e] - centre, scale[e], shift[e])}).v;
      X v;
      v.close(f);
      v.store(y + t * p.ys[2] + i);
    }
  }
}

// Backward of the same: xhat and dz in shared memory; a channel's sums by threads of its own
template <class T, int BYTES, int ACT>
__global__ void __launch_bounds__(kSmallThreads) norm_small_grad_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  constexpr int V = X::N, kAtOnce = 4;
  extern __shared__ float values[];  // xhat, dz [N][n]; then [row][n] sums
  __shared__ float2 part[kSmallThreads / 32];
  const int g = blockIdx.x, b = blockIdx.y;
  const int row = threadIdx.x / p.lanes, lane = threadIdx.x % p.lanes;
  const bool here = row < p.rows;
  const int N = here ? int(p.N) : 0;
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + g * p.xs[1];
  const T* dy = static_cast<const T*>(p.dy) + b * p.dys[0] + g * p.dys[1];
  T* dx = static_cast<T*>(p.dx) + b * p.dxs[0] + g * p.dxs[1];
  float* const dzs = values + int(p.N) * p.n;
  float2* const sums = reinterpret_cast<float2*>(dzs + int(p.N) * p.n);
  const float2 m = load_stats(p.stats, int64_t(b) * p.G + g);
  float2 q = make_float2(0.f, 0.f);
  if (here)
    for (int i = lane * V; i < p.n; i += p.lanes * V) {
      float w[V], o[V], s0[V] = {}, s1[V] = {};
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[e] = p.weight ? p.weight[g * p.n + i + e] : 1.f;
        o[e] = p.bias ? p.bias[g * p.n + i + e] : 0.f;
      }
      for (int t = row; t < N; t += kAtOnce * p.rows) {
        X v[kAtOnce], d[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (t + k * p.rows < N) {
            v[k].load(x + (t + k * p.rows) * p.xs[2] + i);
            d[k].load(dy + (t + k * p.rows) * p.dys[2] + i);
          }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (t + k * p.rows < N) {
            float f[V], h[V];
            v[k].open(f);
            d[k].open(h);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float xhat = (f[e] - m.x) * m.y;
              const float dz = act_grad<T, ACT>(One{fmaf(xhat, w[e], o[e])}, One{h[e]}).v;
              values[(t + k * p.rows) * p.n + i + e] = xhat;
              dzs[(t + k * p.rows) * p.n + i + e] = dz;
              s0[e] += dz;
              s1[e] = fmaf(dz, xhat, s1[e]);
            }
          }
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        sums[row * p.n + i + e] = make_float2(s0[e], s1[e]);
        q.x = fmaf(s0[e], w[e], q.x);
        q.y = fmaf(s1[e], w[e], q.y);
      }
    }
  q = block_sum(q, part);
  for (int c = threadIdx.x / 32; c < p.n; c += kSmallThreads / 32) {  // a warp a channel
    float2 s = make_float2(0.f, 0.f);
    for (int r = threadIdx.x % 32; r < p.rows; r += 32) s.x += sums[r * p.n + c].x, s.y += sums[r * p.n + c].y;
    s = make_float2(warp_sum(s.x), warp_sum(s.y));
    if (threadIdx.x % 32 == 0) p.channel_sums[int64_t(b) * p.C + g * p.n + c] = s;
  }
  const float count = float(p.N) * float(p.n), m0 = q.x / count, m1 = q.y / count;
  for (int i = lane * V; i < p.n; i += p.lanes * V) {
    float w[V];
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = p.weight ? p.weight[g * p.n + i + e] : 1.f;
#pragma unroll 4
    for (int t = row; t < N; t += p.rows) {
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e)
        f[e] = m.y * (dzs[t * p.n + i + e] * w[e] - m0 - values[t * p.n + i + e] * m1);
      X v;
      v.close(f);
      v.store(dx + t * p.dxs[2] + i);
    }
  }
}

// How a call is cut up: by the sizes and the number of bytes that its vectors take.
struct Cut {
  bool small;
  int lanes, rows, col_blocks, row_blocks, slots, smem;
  int32_t range;
};
constexpr int kSmallBytes = 96 * 1024;        // of shared memory that a group may take
constexpr int kSmallValues = 16 * 1024;       // of a group, above which one block takes longer than two kernels
constexpr int64_t kSmallTotal = 1 << 21;      // values in all, above which SMs are full either way
// a block's threads over a row's vectors
void share(Cut& k, int vectors, int threads) {
  k.lanes = std::min(vectors, threads);
  k.rows = std::max(1, threads / k.lanes);
}
// one block a group; V divides the group's channels
Cut cut_small(int64_t N, int n, int V, bool backward) {
  Cut k{};
  share(k, n / V, kSmallThreads);
  k.rows = int(std::min<int64_t>(k.rows, N));
  k.small = true;
  k.smem = int(N * n * (backward ? 8 : 4) + (backward ? int64_t(k.rows) * n * 8 : 0));
  k.row_blocks = k.col_blocks = 1;
  return k;
}
bool fits_small(int32_t B, int64_t N, int C, int n, bool backward) {
  // the sums of the backward pass: rows of n channels, rows * n at most a thread's vector of 8 each (or one row)
  const int64_t bytes = N * n * (backward ? 8 : 4) + (backward ? int64_t(std::max(n, 8 * kSmallThreads)) * 8 : 0);
  return B * N * C <= kSmallTotal && N * n <= kSmallValues && bytes <= kSmallBytes;
}
Cut cut_blocks(int32_t B, int64_t N, int C, int G, int V, bool backward) {
  Cut k{};
  const int vectors = C / V;
  k.col_blocks = (vectors + kThreads - 1) / kThreads;
  share(k, (vectors + k.col_blocks - 1) / k.col_blocks, kThreads);
  k.slots = std::min(G, k.lanes * V / (C / G) + 2);
  // as many blocks as run at once (three an SM forward, two backward), of 8 tokens a thread or more
  const int64_t most = std::max<int64_t>(1, (backward ? 2 : 3) * 148 / (int64_t(B) * k.col_blocks));
  const int64_t blocks = std::min<int64_t>(most, (N + k.rows * 8 - 1) / (k.rows * 8));
  k.range = int32_t((N + blocks - 1) / blocks);
  k.row_blocks = int((N + k.range - 1) / k.range);
  k.smem = k.rows * k.lanes * V * 8;
  return k;
}
size_t workspace_of(const Cut& k, int32_t B, int C, bool backward) {
  return (k.small ? 0 : size_t(B) * k.row_blocks * k.col_blocks * k.slots * 8) +
         (backward ? size_t(B) * k.row_blocks * C * 8 : 0);
}

void put_cut(NormArgs& a, const Cut& k) {
  a.lanes = k.lanes, a.rows = k.rows, a.col_blocks = k.col_blocks, a.row_blocks = k.row_blocks;
  a.range = k.range, a.slots = k.slots;
}

template <class F>
bool allow_smem(F* kernel, OncePerDevice& once) {
  return once.run(current_device(), [&] {
           return int(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallBytes));
         }) == 0;
}

// A launch whose blocks may start while the kernel before it ends; the kernel itself waits
// for that one's results (cudaGridDependencySynchronize).
template <class F>
void launch_behind(F* kernel, dim3 grid, int threads, int smem, const NormArgs& a, cudaStream_t st) {
  cudaLaunchAttribute behind;
  behind.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  behind.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &behind;
  c.numAttrs = 1;
  cudaLaunchKernelEx(&c, kernel, a);
}

template <class T, int BYTES, int ACT>
int launch_small(bool backward, NormArgs& a, const Cut& k, cudaStream_t st) {
  static OncePerDevice once[2];
  const auto f = backward ? norm_small_grad_kernel<T, BYTES, ACT> : norm_small_kernel<T, BYTES, ACT>;
  if (!allow_smem(f, once[backward])) return TTT_ERR_CUDA;
  f<<<dim3(a.G, a.B), kSmallThreads, k.smem, st>>>(a);
  if (backward && (a.dweight || a.dbias)) launch_behind(norm_dweight_kernel, dim3((a.C + 31) / 32), 1024, 0, a, st);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}
template <class T, int BYTES, int Q, int ACT>
int launch_blocks(bool backward, NormArgs& a, const Cut& k, cudaStream_t st) {
  const dim3 grid(k.col_blocks, k.row_blocks, a.B);
  if (backward) {
    static OncePerDevice once;
    const auto sums = norm_sums_kernel<T, BYTES, Q, ACT>;
    if (once.run(current_device(), [&] {
          return int(cudaFuncSetAttribute(sums, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          kRingBytes<BYTES> + kThreads * 8 * BYTES / int(sizeof(T))));
        }) != 0)
      return TTT_ERR_CUDA;
    sums<<<grid, kThreads, k.smem + kRingBytes<BYTES>, st>>>(a);
    launch_behind(norm_dx_kernel<T, BYTES, Q, ACT>, grid, kThreads, k.slots * 8, a, st);
    if (a.dweight || a.dbias) launch_behind(norm_dweight_kernel, dim3((a.C + 31) / 32), 1024, 0, a, st);
  } else {
    norm_parts_kernel<T, BYTES, Q><<<grid, kThreads, k.smem, st>>>(a);
    launch_behind(norm_apply_kernel<T, BYTES, Q, ACT>, grid, kThreads, k.slots * 8, a, st);
  }
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}
// Q: channels of a vector that are of one group for certain
template <class T, int BYTES, int ACT>
int launch_act(bool backward, NormArgs& a, const Cut& k, cudaStream_t st) {
  constexpr int V = BYTES / int(sizeof(T));
  if (k.small) return launch_small<T, BYTES, ACT>(backward, a, k, st);
  if constexpr (V >= 4) {
    if (a.n % V == 0) return launch_blocks<T, BYTES, V, ACT>(backward, a, k, st);
    if constexpr (V == 8)
      if (a.n % 4 == 0) return launch_blocks<T, BYTES, 4, ACT>(backward, a, k, st);
  }
  return launch_blocks<T, BYTES, 1, ACT>(backward, a, k, st);
}
template <class T, int BYTES>
int launch(bool backward, int act, NormArgs& a, const Cut& k, cudaStream_t st) {
  switch (act) {
    case TTT_ACT_SILU: return launch_act<T, BYTES, TTT_ACT_SILU>(backward, a, k, st);
    case TTT_ACT_GELU: return launch_act<T, BYTES, TTT_ACT_GELU>(backward, a, k, st);
    default: return launch_act<T, BYTES, TTT_ACT_NONE>(backward, a, k, st);
  }
}

// Vectors of 16, 8 or 4 bytes or of one channel: the widest that all rows start on and that
// groups (where they lie apart, or each has a block of its own) or rows are whole numbers of.
int vector_bytes(const RowTensor* t, int nt, const ttt_strides* const* s, int C, int n, int elem, bool each) {
  int wide = 16;
  for (int i = 0; i < nt; ++i) {
    const bool together = s[i]->head == n || n == C;  // a row's groups follow one another
    while (wide > elem && (C * elem % wide || ((!together || each) && n * elem % wide))) wide /= 2;
    // channels last: rows are aligned by their first group
    RowTensor rows = t[i];
    if (together) rows.n[1] = 1;
    while (wide > elem && !rows_aligned(rows, wide)) wide /= 2;
  }
  return wide;
}

}  // namespace
}  // namespace ttt

using namespace ttt;

struct ttt_norm {
  ttt_norm_config cfg;
};

namespace {

bool norm_sizes_ok(const ttt_norm* h, int32_t B, int64_t N) { return h && B >= 1 && N >= 1; }
bool norm_supported(int32_t B, int64_t N) { return B <= 65535 && N <= (int64_t(1) << 30); }

// [B, groups, N] rows of a group's channels
RowTensor grouped(const ttt_norm* h, int32_t B, int64_t N, const void* p, const ttt_strides* s) {
  const ttt_norm_config& c = h->cfg;
  return RowTensor(p, c.dtype == TTT_BF16 ? 2 : 4, c.C / c.groups, B, s->batch, c.groups, s->head, N, s->token);
}
RowTensor floats(const float* p, int64_t n) { return RowTensor(p, 4, p ? n : 0, 1, 0, 1, 0); }

// every output is writable and shares nothing with the others or with an input,
// but for out[0], which may be in[0] itself
bool apart(const RowTensor* in, int nin, const RowTensor* out, int nout) {
  for (int i = 0; i < nin; ++i)
    if (!in[i].readable()) return false;
  for (int i = 0; i < nout; ++i) {
    if (!out[i].writable()) return false;
    for (int j = 0; j < nin; ++j)
      if (!(i == 0 && j == 0 && same_tensor(in[0], out[0])) && may_share(out[i], in[j])) return false;
    for (int j = 0; j < i; ++j)
      if (may_share(out[i], out[j])) return false;
  }
  return true;
}

void put_strides(int64_t (&to)[3], const ttt_strides* s) { to[0] = s->batch, to[1] = s->head, to[2] = s->token; }

// of 16-byte vectors down to single channels: the workspace of any alignment is the largest
size_t space_needed(const ttt_norm* h, int32_t B, int64_t N, bool backward) {
  const ttt_norm_config& c = h->cfg;
  const int elem = c.dtype == TTT_BF16 ? 2 : 4;
  if (fits_small(B, N, c.C, c.C / c.groups, backward)) return workspace_of(cut_small(N, 1, 1, backward), B, c.C, backward);
  size_t most = 0;
  for (int wide = 16; wide >= elem; wide /= 2)
    if (c.C * elem % wide == 0)
      most = std::max(most, workspace_of(cut_blocks(B, N, c.C, c.groups, wide / elem, backward), B, c.C, backward));
  return most;
}

// cuts the call up, carves the workspace and launches
int run(const ttt_norm* h, bool backward, NormArgs& a, const RowTensor* t, const ttt_strides* const* s, int nt,
        void* workspace, cudaStream_t st) {
  const ttt_norm_config& c = h->cfg;
  a.C = c.C, a.G = c.groups, a.n = c.C / c.groups, a.eps = c.eps;
  const int elem = c.dtype == TTT_BF16 ? 2 : 4;
  const bool small = fits_small(a.B, a.N, c.C, a.n, backward);
  const int wide = vector_bytes(t, nt, s, c.C, a.n, elem, small);
  const Cut k = small ? cut_small(a.N, a.n, wide / elem, backward) : cut_blocks(a.B, a.N, c.C, c.groups, wide / elem, backward);
  put_cut(a, k);
  a.channel_sums = static_cast<float2*>(workspace);
  a.parts = a.channel_sums + (backward ? size_t(a.B) * k.row_blocks * c.C : 0);
  if (elem == 2)
    return wide == 16  ? launch<__nv_bfloat16, 16>(backward, c.act, a, k, st)
           : wide == 8 ? launch<__nv_bfloat16, 8>(backward, c.act, a, k, st)
           : wide == 4 ? launch<__nv_bfloat16, 4>(backward, c.act, a, k, st)
                       : launch<__nv_bfloat16, 2>(backward, c.act, a, k, st);
  return wide == 16  ? launch<float, 16>(backward, c.act, a, k, st)
         : wide == 8 ? launch<float, 8>(backward, c.act, a, k, st)
                     : launch<float, 4>(backward, c.act, a, k, st);
}

}  // namespace

extern "C" int ttt_norm_create(const ttt_norm_config* c, ttt_norm** out) {
  if (!out) return TTT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c || c->C < 1 || c->groups < 1 || c->C % c->groups) return TTT_ERR_INVALID_ARG;
  if (c->act < TTT_ACT_NONE || c->act > TTT_ACT_GELU) return TTT_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f) || !std::isfinite(c->eps)) return TTT_ERR_INVALID_ARG;
  if (c->dtype != TTT_F32 && c->dtype != TTT_BF16) return TTT_ERR_INVALID_ARG;
  if (c->C > 65536) return TTT_ERR_UNSUPPORTED;
  ttt_norm* h = new (std::nothrow) ttt_norm();
  if (!h) return TTT_ERR_INVALID_ARG;
  h->cfg = *c;
  *out = h;
  return TTT_OK;
}

extern "C" void ttt_norm_destroy(ttt_norm* h) { delete h; }

extern "C" size_t ttt_norm_workspace_size(const ttt_norm* h, int32_t B, int64_t N, int32_t backward) {
  if (!norm_sizes_ok(h, B, N) || !norm_supported(B, N)) return 0;
  return space_needed(h, B, N, backward != 0);
}

extern "C" int ttt_norm_forward(const ttt_norm* h, int32_t B, int64_t N, const void* x, const ttt_strides* xs,
                                const float* weight, const float* bias, void* y, const ttt_strides* ys, float* stats,
                                void* workspace, size_t workspace_bytes, unsigned* status, void* stream) {
  if (!norm_sizes_ok(h, B, N) || !xs || !ys) return TTT_ERR_INVALID_ARG;
  if (!norm_supported(B, N)) return TTT_ERR_UNSUPPORTED;
  if (!is_aligned(workspace, 16) || !is_aligned(status, 4)) return TTT_ERR_INVALID_ARG;
  const ttt_norm_config& c = h->cfg;
  const RowTensor in[] = {grouped(h, B, N, x, xs), floats(weight, c.C), floats(bias, c.C)};
  const RowTensor out[] = {grouped(h, B, N, y, ys), floats(stats, int64_t(B) * c.groups * 2)};
  if (!apart(in, 3, out, 2)) return TTT_ERR_INVALID_ARG;
  const size_t need = ttt_norm_workspace_size(h, B, N, 0);
  if (need && (!workspace || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  NormArgs a{};
  a.x = x, a.y = y, a.weight = weight, a.bias = bias, a.stats = stats;
  put_strides(a.xs, xs), put_strides(a.ys, ys);
  a.N = N, a.B = B;
  const ttt_strides* const s[] = {xs, ys};
  const RowTensor t[] = {in[0], out[0]};
  return run(h, false, a, t, s, 2, workspace, static_cast<cudaStream_t>(stream));
}

extern "C" int ttt_norm_backward(const ttt_norm* h, int32_t B, int64_t N, const void* dy, const ttt_strides* dys,
                                 const void* x, const ttt_strides* xs, const float* weight, const float* bias,
                                 const float* stats, void* dx, const ttt_strides* dxs, float* dweight, float* dbias,
                                 void* workspace, size_t workspace_bytes, unsigned* status, void* stream) {
  if (!norm_sizes_ok(h, B, N) || !dys || !xs || !dxs || !stats) return TTT_ERR_INVALID_ARG;
  if (!norm_supported(B, N)) return TTT_ERR_UNSUPPORTED;
  if (!is_aligned(workspace, 16) || !is_aligned(status, 4)) return TTT_ERR_INVALID_ARG;
  const ttt_norm_config& c = h->cfg;
  const RowTensor in[] = {grouped(h, B, N, dy, dys), grouped(h, B, N, x, xs), floats(weight, c.C), floats(bias, c.C),
                          floats(stats, int64_t(B) * c.groups * 2)};
  const RowTensor out[] = {grouped(h, B, N, dx, dxs), floats(dweight, c.C), floats(dbias, c.C)};
  if (!apart(in, 5, out, 3)) return TTT_ERR_INVALID_ARG;
  const size_t need = ttt_norm_workspace_size(h, B, N, 1);
  if (need && (!workspace || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  NormArgs a{};
  a.dy = dy, a.x = x, a.weight = weight, a.bias = bias, a.stats = const_cast<float*>(stats);
  a.dx = dx, a.dweight = dweight, a.dbias = dbias;
  put_strides(a.dys, dys), put_strides(a.xs, xs), put_strides(a.dxs, dxs);
  a.N = N, a.B = B;
  const ttt_strides* const s[] = {dys, xs, dxs};
  const RowTensor t[] = {in[0], in[1], out[0]};
  return run(h, true, a, t, s, 3, workspace, static_cast<cudaStream_t>(stream));
}
