// Group norm with an activation (ttt_ops.h, ttt_norm_*).
//
// Statistics of a group run over the N tokens and the C / groups channels of one batch
// entry.  sum x^2 - n mean^2 would lose the digits of a group whose mean is large, and the
// sum of squares about the mean takes a second pass over the data.  So runs of at most 32
// tokens are summed about their own first value, which a run's spread is never far
// below, and the (count, mean, sum of squares about it) of two parts are joined by
//   mean = (n1 mean1 + n2 mean2) / n,   S = S1 + S2 + (mean2 - mean1)^2 n1 n2 / n
// (Chan, Golub, LeVeque 1979), in an order that is fixed by the sizes alone.
//
// Two forms.  Where a group of a batch entry fits in shared memory, one block does all of
// it.  Else a first kernel forms the statistics of (token range, channel) blocks and a
// second joins them and normalises; both are bound by HBM, with x read twice where L2
// does not keep it (the second kernel walks backwards, from what was read last).
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
constexpr int kRun = 32;  // tokens summed about one value

struct NormArgs {
  const void *x, *dy;
  void *y, *dx;
  const float *weight, *bias;
  float *stats, *dweight, *dbias;        // stats [B][G][2]
  float2* parts;                         // forward: (mean, S) of each block's part of a group
  float *part_sums, *sums;               // backward: [B][blocks][C][2]; [B][C][2]
  int64_t xs[3], ys[3], dys[3], dxs[3];  // batch, group, token
  int64_t N;
  int32_t B, C, G, n;                    // n channels a group
  float eps;
  int32_t lanes, rows;                   // a block's vectors of channels, and tokens at a time
  int32_t col_blocks, row_blocks;        // blocks of channels; ranges of tokens
  int64_t range;                         // tokens of a range
  int32_t slots;                         // groups of a block of channels at most
};

struct Part {  // of n values: their mean, and S the sum of squares about it
  float n, mean, S;
};
__device__ __forceinline__ Part join(const Part& a, const Part& b) {
  const float n = a.n + b.n;
  if (b.n == 0.f) return a;
  if (a.n == 0.f) return b;
  const float d = b.mean - a.mean, f = b.n / n;
  return {n, fmaf(d, f, a.mean), a.S + b.S + d * d * a.n * f};
}
// over a warp, lane 0 first; every lane has the result
__device__ __forceinline__ Part join_warp(Part v) {
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const Part o = {__shfl_down_sync(~0u, v.n, m), __shfl_down_sync(~0u, v.mean, m), __shfl_down_sync(~0u, v.S, m)};
    v = join(v, o);
  }
  return {__shfl_sync(~0u, v.n, 0), __shfl_sync(~0u, v.mean, 0), __shfl_sync(~0u, v.S, 0)};
}
__device__ __forceinline__ float2 finish(const Part& v, float eps) {  // mean, 1 / sqrt(var + eps)
  return make_float2(v.mean, 1.f / sqrtf(v.S / v.n + eps));
}

// sigma(z).  bf16 outputs take the hardware's exponential (2^-22 off, and 2^-24 of the
// exponent's size), fp32 ones the library's; the reciprocal is the hardware's, 2^-23 off.
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
template <class T>
__device__ __forceinline__ float sigmoid(float z) {
  if (sizeof(T) == 4) return rcp_fast(1.f + expf(-z));
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  return rcp_fast(1.f + e);
}
constexpr float kInvSqrt2 = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;
template <class T, int ACT>
__device__ __forceinline__ float act(float z) {
  if (ACT == TTT_ACT_SILU) return z * sigmoid<T>(z);
  if (ACT == TTT_ACT_GELU) return 0.5f * z * erfcf(-z * kInvSqrt2);
  return z;
}
template <class T, int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if (ACT == TTT_ACT_SILU) {
    const float s = sigmoid<T>(z);
    return fmaf(z * s, 1.f - s, s);
  }
  if (ACT == TTT_ACT_GELU) return fmaf(z * kInvSqrt2Pi, expf(-0.5f * z * z), 0.5f * erfcf(-z * kInvSqrt2));
  return 1.f;
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
  constexpr int V = X::N, K = V / Q, kAtOnce = 8;
  extern __shared__ float2 threads[];  // [row][sum of the block]
  const int cb = blockIdx.x, rb = blockIdx.y, b = blockIdx.z;
  const Column k = column(p, cb, V);
  const int row = threadIdx.x / p.lanes;
  const int64_t t0 = rb * p.range, tokens = min(p.range, p.N - t0);
  const int width = p.lanes * V;
  if (k.here) {
    const T* x = static_cast<const T*>(p.x) + k.at(p.xs, b) + (t0 + row) * p.xs[2];
    const int64_t hop = p.rows * p.xs[2];
    float count = 0.f, mean[K] = {}, S[K] = {};
    for (int64_t left = tokens > row ? (tokens - row + p.rows - 1) / p.rows : 0; left > 0;) {
      const int run = left < kRun ? int(left) : kRun;
      float first[K], s[K], q[K];
      for (int j = 0; j < run; j += kAtOnce) {
        X v[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
          if (j + e < run) v[e].load(x);
          x += j + e < run ? hop : 0;
        }
        if (j == 0) {
          float f[V];
          v[0].open(f);
#pragma unroll
          for (int i = 0; i < K; ++i) first[i] = f[i * Q], s[i] = 0.f, q[i] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
          if (j + e < run) {
            float f[V];
            v[e].open(f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float d = f[i] - first[i / Q];
              s[i / Q] += d;
              q[i / Q] = fmaf(d, d, q[i / Q]);
            }
          }
      }
      const float n = float(run * Q), inv = 1.f / n, all = count + n, f = n / all;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float m = s[i] * inv, Si = fmaxf(fmaf(-s[i], m, q[i]), 0.f);
        const float d = first[i] + m - mean[i];
        if (count == 0.f) {
          mean[i] = first[i] + m;
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
  const int lane = threadIdx.x % 32;
  for (int g = g0 + threadIdx.x / 32; g <= (c1 - 1) / p.n; g += kThreads / 32) {
    const int from = (max(g * p.n, c0) - c0) / Q, wide = (min((g + 1) * p.n, c1) - c0) / Q - from;
    Part v = {0.f, 0.f, 0.f};
    for (int e = lane; e < p.rows * wide; e += 32) {
      const int r = e / wide;
      const float n = tokens > r ? float((tokens - r + p.rows - 1) / p.rows * Q) : 0.f;
      const float2 m = threads[r * (p.lanes * K) + from + e % wide];
      v = join(v, {n, m.x, m.y});
    }
    v = join_warp(v);
    if (lane == 0)
      p.parts[((int64_t(b) * p.row_blocks + rb) * p.col_blocks + cb) * p.slots + g - g0] = make_float2(v.mean, v.S);
  }
}

// The statistics of a group from its blocks' parts, by one warp
__device__ __forceinline__ float2 join_parts(const NormArgs& p, int b, int g, int V) {
  const int width = p.lanes * V, lane = threadIdx.x % 32;
  const int first = g * p.n / width, blocks = ((g + 1) * p.n - 1) / width - first + 1;
  Part v = {0.f, 0.f, 0.f};
  for (int e = lane; e < p.row_blocks * blocks; e += 32) {
    const int rb = e / blocks, cb = first + e % blocks;
    const int c0 = cb * width, c1 = min(p.C, c0 + width);
    const int64_t tokens = min(p.range, p.N - rb * p.range);
    const float n = float(tokens) * float(min((g + 1) * p.n, c1) - max(g * p.n, c0));
    const float2 m = p.parts[((int64_t(b) * p.row_blocks + rb) * p.col_blocks + cb) * p.slots + g - c0 / p.n];
    v = join(v, {n, m.x, m.y});
  }
  return finish(join_warp(v), p.eps);
}

// Joins the parts of its groups and normalises one range of tokens and block of channels.
template <class T, int BYTES, int Q, int ACT>
__global__ void __launch_bounds__(kThreads, 3) norm_apply_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  constexpr int V = X::N, K = V / Q, kAtOnce = 8;
  extern __shared__ float2 known[];  // (mean, 1 / std) of the block's groups
  const int cb = gridDim.x - 1 - blockIdx.x, rb = gridDim.y - 1 - blockIdx.y, b = gridDim.z - 1 - blockIdx.z;
  const Column k = column(p, cb, V);
  const int row = threadIdx.x / p.lanes;
  const int c0 = cb * p.lanes * V, c1 = block_end(p, cb, V), g0 = c0 / p.n;
  for (int g = g0 + threadIdx.x / 32; g <= (c1 - 1) / p.n; g += kThreads / 32) {
    const float2 m = join_parts(p, b, g, V);
    if (threadIdx.x % 32 == 0) {
      known[g - g0] = m;
      if (p.stats && rb == 0 && g * p.n >= c0)
        reinterpret_cast<float2*>(p.stats)[int64_t(b) * p.G + g] = m;
    }
  }
  __syncthreads();
  if (!k.here) return;
  float mean[K], scale[V], shift[V];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const float2 m = known[(k.c + j * Q) / p.n - g0];
    mean[j] = m.x;
#pragma unroll
    for (int i = j * Q; i < (j + 1) * Q; ++i) {
      scale[i] = m.y * (p.weight ? p.weight[k.c + i] : 1.f);
      shift[i] = p.bias ? p.bias[k.c + i] : 0.f;
    }
  }
  const int64_t t0 = rb * p.range, tokens = min(p.range, p.N - t0);
  const T* x = static_cast<const T*>(p.x) + k.at(p.xs, b) + (t0 + row) * p.xs[2];
  T* y = static_cast<T*>(p.y) + k.at(p.ys, b) + (t0 + row) * p.ys[2];
  const int64_t mine = tokens > row ? (tokens - row + p.rows - 1) / p.rows : 0;
  for (int64_t j = (mine + kAtOnce - 1) / kAtOnce * kAtOnce - kAtOnce; j >= 0; j -= kAtOnce) {
    X v[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (j + e < mine) v[e].load(x + (j + e) * p.rows * p.xs[2]);
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (j + e < mine) {
        float f[V];
        v[e].open(f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = act<T, ACT>(fmaf(f[i] - mean[i / Q], scale[i], shift[i]));
        v[e].close(f);
        v[e].store(y + (j + e) * p.rows * p.ys[2]);
      }
  }
}

// Backward, of one range of tokens and block of channels: each channel's sums of dz and dz xhat
template <class T, int BYTES, int Q, int ACT>
__global__ void __launch_bounds__(kThreads, 2) norm_sums_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  constexpr int V = X::N, K = V / Q, kAtOnce = 4;
  extern __shared__ float2 threads[];
  const int cb = blockIdx.x, rb = blockIdx.y, b = blockIdx.z;
  const Column k = column(p, cb, V);
  const int row = threadIdx.x / p.lanes;
  const int64_t t0 = rb * p.range, tokens = min(p.range, p.N - t0);
  const int width = p.lanes * V;
  if (k.here) {
    float mean[K], rstd[K], w[V], o[V], total0[V] = {}, total1[V] = {};
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float2 m = reinterpret_cast<const float2*>(p.stats)[int64_t(b) * p.G + (k.c + i * Q) / p.n];
      mean[i] = m.x;
      rstd[i] = m.y;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[i] = p.weight ? p.weight[k.c + i] : 1.f;
      o[i] = p.bias ? p.bias[k.c + i] : 0.f;
    }
    const T* x = static_cast<const T*>(p.x) + k.at(p.xs, b) + (t0 + row) * p.xs[2];
    const T* dy = static_cast<const T*>(p.dy) + k.at(p.dys, b) + (t0 + row) * p.dys[2];
    const int64_t hop = p.rows * p.xs[2], dhop = p.rows * p.dys[2];
    for (int64_t left = tokens > row ? (tokens - row + p.rows - 1) / p.rows : 0; left > 0;) {
      const int run = left < kRun ? int(left) : kRun;  // sums of runs, so that no long sum swallows its terms
      float s0[V] = {}, s1[V] = {};
      for (int j = 0; j < run; j += kAtOnce) {
        X v[kAtOnce], d[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
          if (j + e < run) {
            v[e].load(x);
            d[e].load(dy);
          }
          x += j + e < run ? hop : 0;
          dy += j + e < run ? dhop : 0;
        }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
          if (j + e < run) {
            float f[V], g[V];
            v[e].open(f);
            d[e].open(g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float xhat = (f[i] - mean[i / Q]) * rstd[i / Q];
              const float dz = g[i] * act_grad<T, ACT>(fmaf(xhat, w[i], o[i]));
              s0[i] += dz;
              s1[i] = fmaf(dz, xhat, s1[i]);
            }
          }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) total0[i] += s0[i], total1[i] += s1[i];
      left -= run;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      threads[row * width + (threadIdx.x % p.lanes) * V + i] = make_float2(total0[i], total1[i]);
  }
  __syncthreads();
  const int c0 = cb * width, c1 = block_end(p, cb, V);
  for (int c = threadIdx.x; c < c1 - c0; c += kThreads) {
    float2 s = threads[c];
    for (int r = 1; r < p.rows; ++r) {
      s.x += threads[r * width + c].x;
      s.y += threads[r * width + c].y;
    }
    reinterpret_cast<float2*>(p.part_sums)[(int64_t(b) * p.row_blocks + rb) * p.C + c0 + c] = s;
  }
}

// Joins the ranges' sums, 32 channels a block: sums [B][C], and over the batch dweight and dbias
__global__ void __launch_bounds__(1024) norm_join_sums_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float2 rows[32][32];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, r = threadIdx.x / 32;
  const float2* from = reinterpret_cast<const float2*>(p.part_sums);
  float2 all = make_float2(0.f, 0.f);
  for (int b = 0; b < p.B; ++b) {
    float2 s = make_float2(0.f, 0.f);
    if (c < p.C)
      for (int rb = r; rb < p.row_blocks; rb += 32) {
        const float2 v = from[(int64_t(b) * p.row_blocks + rb) * p.C + c];
        s.x += v.x;
        s.y += v.y;
      }
    rows[r][threadIdx.x % 32] = s;
    __syncthreads();
    if (r == 0 && c < p.C) {
      for (int q = 1; q < min(32, p.row_blocks); ++q) {
        s.x += rows[q][threadIdx.x].x;
        s.y += rows[q][threadIdx.x].y;
      }
      reinterpret_cast<float2*>(p.sums)[int64_t(b) * p.C + c] = s;
      all.x += s.x;
      all.y += s.y;
    }
    __syncthreads();
  }
  if (r == 0 && c < p.C) {
    if (p.dbias) p.dbias[c] = all.x;
    if (p.dweight) p.dweight[c] = all.y;
  }
}

// dx of one range of tokens and block of channels, walked backwards
template <class T, int BYTES, int Q, int ACT>
__global__ void __launch_bounds__(kThreads, 2) norm_dx_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  constexpr int V = X::N, K = V / Q, kAtOnce = 4;
  extern __shared__ float2 known[];  // (mean q, mean q xhat) of the block's groups
  const int cb = gridDim.x - 1 - blockIdx.x, rb = gridDim.y - 1 - blockIdx.y, b = gridDim.z - 1 - blockIdx.z;
  const Column k = column(p, cb, V);
  const int row = threadIdx.x / p.lanes;
  const int c0 = cb * p.lanes * V, c1 = block_end(p, cb, V), g0 = c0 / p.n;
  const float inv = 1.f / (float(p.N) * float(p.n));
  for (int g = g0 + threadIdx.x / 32; g <= (c1 - 1) / p.n; g += kThreads / 32) {
    float q0 = 0.f, q1 = 0.f;
    for (int c = g * p.n + threadIdx.x % 32; c < (g + 1) * p.n; c += 32) {
      const float w = p.weight ? p.weight[c] : 1.f;
      const float2 s = reinterpret_cast<const float2*>(p.sums)[int64_t(b) * p.C + c];
      q0 = fmaf(s.x, w, q0);
      q1 = fmaf(s.y, w, q1);
    }
#pragma unroll
    for (int m = 16; m; m /= 2) q0 += __shfl_xor_sync(~0u, q0, m), q1 += __shfl_xor_sync(~0u, q1, m);
    if (threadIdx.x % 32 == 0) known[g - g0] = make_float2(q0 * inv, q1 * inv);
  }
  __syncthreads();
  if (!k.here) return;
  float mean[K], rstd[K], m0[K], m1[K], w[V], o[V];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int g = (k.c + i * Q) / p.n;
    const float2 m = reinterpret_cast<const float2*>(p.stats)[int64_t(b) * p.G + g];
    mean[i] = m.x;
    rstd[i] = m.y;
    m0[i] = known[g - g0].x;
    m1[i] = known[g - g0].y;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i] = p.weight ? p.weight[k.c + i] : 1.f;
    o[i] = p.bias ? p.bias[k.c + i] : 0.f;
  }
  const int64_t t0 = rb * p.range, tokens = min(p.range, p.N - t0);
  const T* x = static_cast<const T*>(p.x) + k.at(p.xs, b) + (t0 + row) * p.xs[2];
  const T* dy = static_cast<const T*>(p.dy) + k.at(p.dys, b) + (t0 + row) * p.dys[2];
  T* dx = static_cast<T*>(p.dx) + k.at(p.dxs, b) + (t0 + row) * p.dxs[2];
  const int64_t mine = tokens > row ? (tokens - row + p.rows - 1) / p.rows : 0;
  for (int64_t j = (mine + kAtOnce - 1) / kAtOnce * kAtOnce - kAtOnce; j >= 0; j -= kAtOnce) {
    X v[kAtOnce], d[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (j + e < mine) {
        v[e].load(x + (j + e) * p.rows * p.xs[2]);
        d[e].load(dy + (j + e) * p.rows * p.dys[2]);
      }
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (j + e < mine) {
        float f[V], g[V];
        v[e].open(f);
        d[e].open(g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xhat = (f[i] - mean[i / Q]) * rstd[i / Q];
          const float q = g[i] * act_grad<T, ACT>(fmaf(xhat, w[i], o[i])) * w[i];
          f[i] = rstd[i / Q] * (q - m0[i / Q] - xhat * m1[i / Q]);
        }
        v[e].close(f);
        v[e].store(dx + (j + e) * p.rows * p.dxs[2]);
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
  for (int i = 1; i < kThreads / 32; ++i) v.x += part[i].x, v.y += part[i].y;
  return v;
}

// lanes and rows: of the group's own channels
template <class T, int BYTES, int ACT>
__global__ void __launch_bounds__(kThreads) norm_small_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  constexpr int V = X::N;
  extern __shared__ float values[];
  __shared__ float2 part[kThreads / 32];
  const int g = blockIdx.x, b = blockIdx.y;
  const int row = threadIdx.x / p.lanes, lane = threadIdx.x % p.lanes;
  const bool here = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + g * p.xs[1];
  T* y = static_cast<T*>(p.y) + b * p.ys[0] + g * p.ys[1];
  const int N = int(p.N);
  const float count = float(N) * float(p.n);
  float2 s = make_float2(0.f, 0.f);
  if (here)
    for (int t = row; t < N; t += p.rows)
      for (int i = lane * V; i < p.n; i += p.lanes * V) {
        X v;
        v.load(x + t * p.xs[2] + i);
        float f[V];
        v.open(f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          values[t * p.n + i + e] = f[e];
          s.x += f[e];
        }
      }
  const float mean = block_sum(s, part).x / count;
  s = make_float2(0.f, 0.f);
  if (here)
    for (int t = row; t < N; t += p.rows)
      for (int i = lane * V; i < p.n; i += p.lanes * V)
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
  if (p.stats && threadIdx.x == 0) reinterpret_cast<float2*>(p.stats)[int64_t(b) * p.G + g] = make_float2(centre, rstd);
  if (!here) return;
  for (int i = lane * V; i < p.n; i += p.lanes * V) {
    float scale[V], shift[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      scale[e] = rstd * (p.weight ? p.weight[g * p.n + i + e] : 1.f);
      shift[e] = p.bias ? p.bias[g * p.n + i + e] : 0.f;
    }
    for (int t = row; t < N; t += p.rows) {
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = act<T, ACT>(fmaf(values[t * p.n + i + e] - centre, scale[e], shift[e]));
      X v;
      v.close(f);
      v.store(y + t * p.ys[2] + i);
    }
  }
}

// Backward of the same: xhat and dz in shared memory; a channel's sums by threads of its own
template <class T, int BYTES, int ACT>
__global__ void __launch_bounds__(kThreads) norm_small_grad_kernel(const __grid_constant__ NormArgs p) {
  using X = Vec<T, BYTES>;
  constexpr int V = X::N;
  extern __shared__ float values[];  // xhat, dz [N][n]; then [row][n] sums
  __shared__ float2 part[kThreads / 32];
  const int g = blockIdx.x, b = blockIdx.y;
  const int row = threadIdx.x / p.lanes, lane = threadIdx.x % p.lanes;
  const bool here = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + g * p.xs[1];
  const T* dy = static_cast<const T*>(p.dy) + b * p.dys[0] + g * p.dys[1];
  T* dx = static_cast<T*>(p.dx) + b * p.dxs[0] + g * p.dxs[1];
  const int N = int(p.N);
  float* const dzs = values + N * p.n;
  float2* const sums = reinterpret_cast<float2*>(dzs + N * p.n);
  const float2 m = reinterpret_cast<const float2*>(p.stats)[int64_t(b) * p.G + g];
  float2 q = make_float2(0.f, 0.f);
  if (here)
    for (int i = lane * V; i < p.n; i += p.lanes * V) {
      float w[V], o[V], s0[V] = {}, s1[V] = {};
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[e] = p.weight ? p.weight[g * p.n + i + e] : 1.f;
        o[e] = p.bias ? p.bias[g * p.n + i + e] : 0.f;
      }
      for (int t = row; t < N; t += p.rows) {
        X v, d;
        v.load(x + t * p.xs[2] + i);
        d.load(dy + t * p.dys[2] + i);
        float f[V], h[V];
        v.open(f);
        d.open(h);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xhat = (f[e] - m.x) * m.y;
          const float dz = h[e] * act_grad<T, ACT>(fmaf(xhat, w[e], o[e]));
          values[t * p.n + i + e] = xhat;
          dzs[t * p.n + i + e] = dz;
          s0[e] += dz;
          s1[e] = fmaf(dz, xhat, s1[e]);
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
  for (int c = threadIdx.x; c < p.n; c += kThreads) {
    float2 s = sums[c];
    for (int r = 1; r < p.rows; ++r) s.x += sums[r * p.n + c].x, s.y += sums[r * p.n + c].y;
    reinterpret_cast<float2*>(p.part_sums)[int64_t(b) * p.C + g * p.n + c] = s;
  }
  const float count = float(N) * float(p.n), m0 = q.x / count, m1 = q.y / count;
  if (here)
    for (int i = lane * V; i < p.n; i += p.lanes * V) {
      float w[V];
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = p.weight ? p.weight[g * p.n + i + e] : 1.f;
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
  int64_t range;
};
constexpr int kSmallBytes = 96 * 1024;        // of a group in shared memory, as fp32
constexpr int64_t kSmallTotal = 1 << 21;      // values in all, above which SMs are full either way
// of 256 threads over a row's vectors
void share(Cut& k, int vectors) {
  k.lanes = std::min(vectors, kThreads);
  k.rows = std::max(1, kThreads / k.lanes);
}
// one block a group; V divides the group's channels
Cut cut_small(int64_t N, int n, int V, bool backward) {
  Cut k{};
  share(k, n / V);
  k.rows = int(std::min<int64_t>(k.rows, N));
  k.small = true;
  k.smem = int(N * n * (backward ? 8 : 4) + (backward ? int64_t(k.rows) * n * 8 : 0));
  k.row_blocks = k.col_blocks = 1;
  return k;
}
bool fits_small(int32_t B, int64_t N, int C, int n, bool backward) {
  // with a row of sums a thread at most, 2 kThreads floats a channel vector of one
  const int64_t bytes = N * n * (backward ? 8 : 4) + (backward ? int64_t(std::max(n, kThreads)) * 8 * 8 : 0);
  return B * N * C <= kSmallTotal && bytes <= kSmallBytes;
}
Cut cut_blocks(int32_t B, int64_t N, int C, int G, int V) {
  Cut k{};
  const int vectors = C / V;
  k.col_blocks = (vectors + kThreads - 1) / kThreads;
  share(k, (vectors + k.col_blocks - 1) / k.col_blocks);
  k.slots = std::min(G, k.lanes * V / (C / G) + 2);
  // four blocks an SM in all, of at least 32 tokens a thread
  const int64_t most = std::max<int64_t>(1, 4 * 148 / (int64_t(B) * k.col_blocks));
  const int64_t blocks = std::min<int64_t>(most, (N + k.rows * kRun - 1) / (k.rows * kRun));
  k.range = (N + blocks - 1) / blocks;
  k.row_blocks = int((N + k.range - 1) / k.range);
  k.smem = k.rows * k.lanes * V * 8;
  return k;
}
size_t workspace_of(const Cut& k, int32_t B, int C, bool backward) {
  if (!backward) return k.small ? 0 : size_t(B) * k.row_blocks * k.col_blocks * k.slots * 8;
  return size_t(B) * k.row_blocks * C * 8 + size_t(B) * C * 8;
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

template <class T, int BYTES, int ACT>
int launch_small(bool backward, NormArgs& a, const Cut& k, cudaStream_t st) {
  static OncePerDevice once[2];
  const auto f = backward ? norm_small_grad_kernel<T, BYTES, ACT> : norm_small_kernel<T, BYTES, ACT>;
  if (!allow_smem(f, once[backward])) return TTT_ERR_CUDA;
  f<<<dim3(a.G, a.B), kThreads, k.smem, st>>>(a);
  if (backward && (a.dweight || a.dbias)) norm_join_sums_kernel<<<(a.C + 31) / 32, 1024, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}
template <class T, int BYTES, int Q, int ACT>
int launch_blocks(bool backward, NormArgs& a, const Cut& k, cudaStream_t st) {
  const dim3 grid(k.col_blocks, k.row_blocks, a.B);
  if (backward) {
    norm_sums_kernel<T, BYTES, Q, ACT><<<grid, kThreads, k.smem, st>>>(a);
    norm_join_sums_kernel<<<(a.C + 31) / 32, 1024, 0, st>>>(a);
    norm_dx_kernel<T, BYTES, Q, ACT><<<grid, kThreads, k.slots * 8, st>>>(a);
  } else {
    norm_parts_kernel<T, BYTES, Q><<<grid, kThreads, k.smem, st>>>(a);
    norm_apply_kernel<T, BYTES, Q, ACT><<<grid, kThreads, k.slots * 8, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}
// Q: channels of a vector that are of one group for certain
template <class T, int BYTES, int ACT>
int launch_act(bool backward, NormArgs& a, const Cut& k, cudaStream_t st) {
  constexpr int V = BYTES / int(sizeof(T));
  if (k.small) return launch_small<T, BYTES, ACT>(backward, a, k, st);
  if constexpr (BYTES == 16) {
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

// Vectors of 16 or 4 bytes or of one channel: the widest that all rows start on and that
// groups (where they lie apart, or each has a block of its own) or rows are whole numbers of.
int vector_bytes(const RowTensor* t, int nt, const ttt_strides* const* s, int C, int n, int elem, bool each) {
  int wide = 16;
  const auto narrower = [&] { wide = wide == 16 ? 4 : elem; };
  for (int i = 0; i < nt; ++i) {
    const bool together = s[i]->head == n || n == C;  // a row's groups follow one another
    while (wide > elem && (C * elem % wide || ((!together || each) && n * elem % wide))) narrower();
    // channels last: rows are aligned by their first group
    RowTensor rows = t[i];
    if (together) rows.n[1] = 1;
    while (wide > elem && !rows_aligned(rows, wide)) narrower();
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
  for (int wide : {16, 4, elem})
    if (c.C * elem % wide == 0)
      most = std::max(most, workspace_of(cut_blocks(B, N, c.C, c.groups, wide / elem), B, c.C, backward));
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
  const Cut k = small ? cut_small(a.N, a.n, wide / elem, backward) : cut_blocks(a.B, a.N, c.C, c.groups, wide / elem);
  put_cut(a, k);
  if (backward) {
    a.part_sums = static_cast<float*>(workspace);
    a.sums = a.part_sums + size_t(a.B) * k.row_blocks * c.C * 2;
  } else {
    a.parts = static_cast<float2*>(workspace);
  }
  if (elem == 2)
    return wide == 16  ? launch<__nv_bfloat16, 16>(backward, c.act, a, k, st)
           : wide == 4 ? launch<__nv_bfloat16, 4>(backward, c.act, a, k, st)
                       : launch<__nv_bfloat16, 2>(backward, c.act, a, k, st);
  return wide == 16 ? launch<float, 16>(backward, c.act, a, k, st) : launch<float, 4>(backward, c.act, a, k, st);
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
