// Group norm with an activation (ttt_ops.h, ttt_norm_*).
//
// Statistics of a group run over the N tokens and the C / groups channels of one
// batch entry.  The variance is taken about the mean in a second pass over the
// data: sum x^2 - n mean^2 would lose the digits of a group whose mean is large.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#include "op_checks.h"

namespace ttt {
namespace {

struct NormArgs {
  const void *x, *dy;
  void *y, *dx;
  const float *weight, *bias;
  float *stats, *sums, *dweight, *dbias;  // stats [B][G][2]; sums [B][C][2]
  int64_t xs[3], ys[3], dys[3], dxs[3];   // batch, group, token
  int64_t N;
  int32_t B, C, G, n;  // n channels a group
  float eps;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int ACT>
__device__ __forceinline__ float act(float z) {
  if (ACT == TTT_ACT_SILU) return z / (1.f + expf(-z));
  if (ACT == TTT_ACT_GELU) return 0.5f * z * erfcf(z * -0.70710678118654752f);
  return z;
}
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if (ACT == TTT_ACT_SILU) {
    const float s = 1.f / (1.f + expf(-z));
    return s * (1.f + z * (1.f - s));
  }
  if (ACT == TTT_ACT_GELU)
    return 0.5f * erfcf(z * -0.70710678118654752f) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
  return 1.f;
}

__device__ float block_sum(float v) {
  __shared__ float part[32];
  __syncthreads();
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(~0u, v, m);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < int(blockDim.x / 32); ++i) s += part[i];
  return s;
}

// One block per (group, batch entry).
template <class T, int ACT>
__global__ void norm_forward_kernel(const __grid_constant__ NormArgs p) {
  const int k = blockIdx.x, b = blockIdx.y;
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + k * p.xs[1];
  T* y = static_cast<T*>(p.y) + b * p.ys[0] + k * p.ys[1];
  const int64_t total = p.N * p.n;
  float s = 0.f;
  for (int64_t e = threadIdx.x; e < total; e += blockDim.x) s += to_f(x[e / p.n * p.xs[2] + e % p.n]);
  const float mean = block_sum(s) / float(total);
  s = 0.f;
  for (int64_t e = threadIdx.x; e < total; e += blockDim.x) {
    const float d = to_f(x[e / p.n * p.xs[2] + e % p.n]) - mean;
    s += d * d;
  }
  const float rstd = 1.f / sqrtf(block_sum(s) / float(total) + p.eps);
  for (int64_t e = threadIdx.x; e < total; e += blockDim.x) {
    const int64_t t = e / p.n;
    const int i = int(e % p.n), c = k * p.n + i;
    const float z = (to_f(x[t * p.xs[2] + i]) - mean) * rstd * (p.weight ? p.weight[c] : 1.f) +
                    (p.bias ? p.bias[c] : 0.f);
    put(y + t * p.ys[2] + i, act<ACT>(z));
  }
  if (p.stats && threadIdx.x == 0) {
    p.stats[(int64_t(b) * p.G + k) * 2] = mean;
    p.stats[(int64_t(b) * p.G + k) * 2 + 1] = rstd;
  }
}

// Per (channel, batch entry): the sums of dz and dz xhat over the tokens.
template <class T, int ACT>
__global__ void norm_sums_kernel(const __grid_constant__ NormArgs p) {
  const int c = blockIdx.x, b = blockIdx.y, k = c / p.n, i = c % p.n;
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + k * p.xs[1] + i;
  const T* dy = static_cast<const T*>(p.dy) + b * p.dys[0] + k * p.dys[1] + i;
  const float mean = p.stats[(int64_t(b) * p.G + k) * 2], rstd = p.stats[(int64_t(b) * p.G + k) * 2 + 1];
  const float w = p.weight ? p.weight[c] : 1.f, o = p.bias ? p.bias[c] : 0.f;
  float s0 = 0.f, s1 = 0.f;
  for (int64_t t = threadIdx.x; t < p.N; t += blockDim.x) {
    const float xhat = (to_f(x[t * p.xs[2]]) - mean) * rstd;
    const float dz = to_f(dy[t * p.dys[2]]) * act_grad<ACT>(xhat * w + o);
    s0 += dz;
    s1 += dz * xhat;
  }
  s0 = block_sum(s0);
  s1 = block_sum(s1);
  if (threadIdx.x == 0) {
    p.sums[(int64_t(b) * p.C + c) * 2] = s0;
    p.sums[(int64_t(b) * p.C + c) * 2 + 1] = s1;
  }
}

// Per channel: the gradients of weight and bias, summed over the batch entries.
__global__ void norm_dweight_kernel(const __grid_constant__ NormArgs p) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.C) return;
  float s0 = 0.f, s1 = 0.f;
  for (int b = 0; b < p.B; ++b) {
    s0 += p.sums[(int64_t(b) * p.C + c) * 2];
    s1 += p.sums[(int64_t(b) * p.C + c) * 2 + 1];
  }
  if (p.dbias) p.dbias[c] = s0;
  if (p.dweight) p.dweight[c] = s1;
}

template <class T, int ACT>
__global__ void norm_dx_kernel(const __grid_constant__ NormArgs p) {
  const int k = blockIdx.x, b = blockIdx.y;
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + k * p.xs[1];
  const T* dy = static_cast<const T*>(p.dy) + b * p.dys[0] + k * p.dys[1];
  T* dx = static_cast<T*>(p.dx) + b * p.dxs[0] + k * p.dxs[1];
  const float mean = p.stats[(int64_t(b) * p.G + k) * 2], rstd = p.stats[(int64_t(b) * p.G + k) * 2 + 1];
  float s0 = 0.f, s1 = 0.f;
  for (int i = threadIdx.x; i < p.n; i += blockDim.x) {
    const int c = k * p.n + i;
    const float w = p.weight ? p.weight[c] : 1.f;
    s0 += p.sums[(int64_t(b) * p.C + c) * 2] * w;
    s1 += p.sums[(int64_t(b) * p.C + c) * 2 + 1] * w;
  }
  const int64_t total = p.N * p.n;
  const float m0 = block_sum(s0) / float(total), m1 = block_sum(s1) / float(total);
  for (int64_t e = int64_t(blockIdx.z) * blockDim.x + threadIdx.x; e < total; e += int64_t(gridDim.z) * blockDim.x) {
    const int64_t t = e / p.n;
    const int i = int(e % p.n), c = k * p.n + i;
    const float w = p.weight ? p.weight[c] : 1.f, o = p.bias ? p.bias[c] : 0.f;
    const float xhat = (to_f(x[t * p.xs[2] + i]) - mean) * rstd;
    const float q = to_f(dy[t * p.dys[2] + i]) * act_grad<ACT>(xhat * w + o) * w;
    put(dx + t * p.dxs[2] + i, rstd * (q - m0 - xhat * m1));
  }
}

template <class T, int ACT>
void launch_forward(const NormArgs& a, cudaStream_t st) {
  norm_forward_kernel<T, ACT><<<dim3(a.G, a.B), 512, 0, st>>>(a);
}
template <class T, int ACT>
void launch_backward(const NormArgs& a, cudaStream_t st) {
  norm_sums_kernel<T, ACT><<<dim3(a.C, a.B), 256, 0, st>>>(a);
  norm_dweight_kernel<<<(a.C + 127) / 128, 128, 0, st>>>(a);
  const int64_t blocks = (a.N * a.n + 1023) / 1024;
  norm_dx_kernel<T, ACT><<<dim3(a.G, a.B, unsigned(blocks < 64 ? blocks : 64)), 256, 0, st>>>(a);
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

template <class T>
void launch(bool backward, int act, const NormArgs& a, cudaStream_t st) {
  if (act == TTT_ACT_SILU)
    backward ? launch_backward<T, TTT_ACT_SILU>(a, st) : launch_forward<T, TTT_ACT_SILU>(a, st);
  else if (act == TTT_ACT_GELU)
    backward ? launch_backward<T, TTT_ACT_GELU>(a, st) : launch_forward<T, TTT_ACT_GELU>(a, st);
  else
    backward ? launch_backward<T, TTT_ACT_NONE>(a, st) : launch_forward<T, TTT_ACT_NONE>(a, st);
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
  return backward ? size_t(B) * h->cfg.C * 2 * 4 : 0;
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
  a.N = N, a.B = B, a.C = c.C, a.G = c.groups, a.n = c.C / c.groups, a.eps = c.eps;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  c.dtype == TTT_BF16 ? launch<__nv_bfloat16>(false, c.act, a, st) : launch<float>(false, c.act, a, st);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
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
  a.dx = dx, a.dweight = dweight, a.dbias = dbias, a.sums = static_cast<float*>(workspace);
  put_strides(a.dys, dys), put_strides(a.xs, xs), put_strides(a.dxs, dxs);
  a.N = N, a.B = B, a.C = c.C, a.G = c.groups, a.n = c.C / c.groups, a.eps = c.eps;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  c.dtype == TTT_BF16 ? launch<__nv_bfloat16>(true, c.act, a, st) : launch<float>(true, c.act, a, st);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}
