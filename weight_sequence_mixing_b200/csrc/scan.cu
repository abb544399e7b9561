// Gated linear recurrence (ttt_ops.h, ttt_scan_*):
//   h_t = a_t h_{t-1} + u_t,   a = g | sigma(g) | exp(g),   u = x | (1 - a) x.
// Backward: lam_t = dh_t + mu_t with mu_t = a_{t+1} lam_{t+1}, the gradient that
// reaches h_t from the later tokens (mu_len = dh_last).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <new>

#include "op_checks.h"

namespace ttt {
namespace {

struct ScanArgs {
  const void *g, *x, *dh;
  const float *h0, *dh_last;
  const int* lengths;
  void *h, *dg, *dx;
  float *h_last, *dh0, *saved;
  int64_t gs[2], xs[2], hs[2], dhs[2], dgs[2], dxs[2];  // batch, token
  int64_t L;
  int32_t B, D;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// a and 1 - a; the complement is formed on its own, so that it keeps its digits
// where a is close to 1
template <int GATE>
__device__ __forceinline__ void gate(float g, float& a, float& rest) {
  if (GATE == TTT_GATE_VALUE) {
    a = g;
    rest = 1.f - g;
  } else if (GATE == TTT_GATE_SIGMOID) {
    a = 1.f / (1.f + expf(-g));
    rest = 1.f / (1.f + expf(g));
  } else {
    a = expf(g);
    rest = -expm1f(g);
  }
}
// d gate / d g times `v`
template <int GATE>
__device__ __forceinline__ float gate_grad(float a, float rest, float v) {
  return GATE == TTT_GATE_VALUE ? v : GATE == TTT_GATE_EXP ? v * a : v * a * rest;
}

__device__ __forceinline__ int64_t length_of(const ScanArgs& p, int b) {
  if (!p.lengths) return p.L;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

// One thread per (batch entry, channel), token after token.  saved: h_{t-1} of every
// token, fp32.
template <class T, int GATE, int INPUT>
__global__ void scan_forward_kernel(const __grid_constant__ ScanArgs p) {
  const int64_t k = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (k >= int64_t(p.B) * p.D) return;
  const int b = int(k / p.D), c = int(k % p.D);
  const int64_t len = length_of(p, b);
  const T* g = static_cast<const T*>(p.g) + b * p.gs[0] + c;
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + c;
  T* h = static_cast<T*>(p.h) + b * p.hs[0] + c;
  float s = p.h0 ? p.h0[k] : 0.f;
  for (int64_t t = 0; t < len; ++t) {
    float a, rest;
    gate<GATE>(to_f(g[t * p.gs[1]]), a, rest);
    const float v = to_f(x[t * p.xs[1]]);
    if (p.saved) p.saved[(int64_t(b) * p.L + t) * p.D + c] = s;
    s = a * s + (INPUT == TTT_SCAN_COMPLEMENT ? rest * v : v);
    put(h + t * p.hs[1], s);
  }
  if (p.h_last) p.h_last[k] = s;
}

template <class T, int GATE, int INPUT>
__global__ void scan_backward_kernel(const __grid_constant__ ScanArgs p) {
  const int64_t k = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (k >= int64_t(p.B) * p.D) return;
  const int b = int(k / p.D), c = int(k % p.D);
  const int64_t len = length_of(p, b);
  const T* g = static_cast<const T*>(p.g) + b * p.gs[0] + c;
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + c;
  const T* dh = static_cast<const T*>(p.dh) + b * p.dhs[0] + c;
  T* dg = static_cast<T*>(p.dg) + b * p.dgs[0] + c;
  T* dx = static_cast<T*>(p.dx) + b * p.dxs[0] + c;
  float mu = p.dh_last ? p.dh_last[k] : 0.f;
  for (int64_t t = len - 1; t >= 0; --t) {
    float a, rest;
    gate<GATE>(to_f(g[t * p.gs[1]]), a, rest);
    const float lam = to_f(dh[t * p.dhs[1]]) + mu;
    float d = p.saved[(int64_t(b) * p.L + t) * p.D + c];
    if (INPUT == TTT_SCAN_COMPLEMENT) d -= to_f(x[t * p.xs[1]]);
    put(dx + t * p.dxs[1], INPUT == TTT_SCAN_COMPLEMENT ? rest * lam : lam);
    put(dg + t * p.dgs[1], gate_grad<GATE>(a, rest, lam * d));
    mu = a * lam;
  }
  if (p.dh0) p.dh0[k] = mu;
}

using ScanKernel = void (*)(const ScanArgs);
template <class T>
ScanKernel pick(bool backward, int gate, int input) {
#define TTT_SCAN_PICK(G, I) \
  if (gate == G && input == I) return backward ? scan_backward_kernel<T, G, I> : scan_forward_kernel<T, G, I>;
  TTT_SCAN_PICK(TTT_GATE_VALUE, TTT_SCAN_PLAIN)
  TTT_SCAN_PICK(TTT_GATE_VALUE, TTT_SCAN_COMPLEMENT)
  TTT_SCAN_PICK(TTT_GATE_SIGMOID, TTT_SCAN_PLAIN)
  TTT_SCAN_PICK(TTT_GATE_SIGMOID, TTT_SCAN_COMPLEMENT)
  TTT_SCAN_PICK(TTT_GATE_EXP, TTT_SCAN_PLAIN)
  TTT_SCAN_PICK(TTT_GATE_EXP, TTT_SCAN_COMPLEMENT)
#undef TTT_SCAN_PICK
  return nullptr;
}

}  // namespace
}  // namespace ttt

using namespace ttt;

struct ttt_scan {
  ttt_scan_config cfg;
};

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;

bool scan_sizes_ok(const ttt_scan* h, int32_t B, int64_t L) { return h && B >= 1 && L >= 0; }

RowTensor rows(const ttt_scan* h, int32_t B, int64_t L, const void* p, const ttt_strides* s) {
  return RowTensor(p, h->cfg.dtype == TTT_BF16 ? 2 : 4, h->cfg.D, B, s->batch, L, s->token);
}
RowTensor state(const ttt_scan* h, int32_t B, const float* p) {
  return RowTensor(p, 4, p ? h->cfg.D : 0, B, h->cfg.D, 1, 0);
}
RowTensor bytes(const void* p, size_t n) { return RowTensor(p, 1, p ? int64_t(n) : 0, 1, 0, 1, 0); }

// every output is writable, shares nothing with an input and nothing with another output
bool apart(const RowTensor* in, int nin, const RowTensor* out, int nout) {
  for (int i = 0; i < nin; ++i)
    if (!in[i].readable()) return false;
  for (int i = 0; i < nout; ++i) {
    if (!out[i].writable()) return false;
    for (int j = 0; j < nin; ++j)
      if (may_share(out[i], in[j])) return false;
    for (int j = 0; j < i; ++j)
      if (may_share(out[i], out[j])) return false;
  }
  return true;
}

void put_strides(int64_t (&to)[2], const ttt_strides* s) { to[0] = s->batch, to[1] = s->token; }

}  // namespace

extern "C" int ttt_scan_create(const ttt_scan_config* c, ttt_scan** out) {
  if (!out) return TTT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c || c->D < 1 || c->gate < TTT_GATE_VALUE || c->gate > TTT_GATE_EXP) return TTT_ERR_INVALID_ARG;
  if (c->input != TTT_SCAN_PLAIN && c->input != TTT_SCAN_COMPLEMENT) return TTT_ERR_INVALID_ARG;
  if (c->dtype != TTT_F32 && c->dtype != TTT_BF16) return TTT_ERR_INVALID_ARG;
  ttt_scan* h = new (std::nothrow) ttt_scan();
  if (!h) return TTT_ERR_INVALID_ARG;
  h->cfg = *c;
  *out = h;
  return TTT_OK;
}

extern "C" void ttt_scan_destroy(ttt_scan* h) { delete h; }

extern "C" size_t ttt_scan_workspace_size(const ttt_scan* h, int32_t B, int64_t L) {
  (void)h, (void)B, (void)L;
  return 0;
}

extern "C" size_t ttt_scan_saved_size(const ttt_scan* h, int32_t B, int64_t L) {
  if (!scan_sizes_ok(h, B, L) || L > kMaxTokens) return 0;
  return size_t(B) * size_t(L) * size_t(h->cfg.D) * 4;
}

extern "C" int ttt_scan_forward(const ttt_scan* h, int32_t B, int64_t L, const void* g, const ttt_strides* gs,
                                const void* x, const ttt_strides* xs, const float* h0, const int32_t* lengths, void* ho,
                                const ttt_strides* hs, float* h_last, void* saved, void* workspace,
                                size_t workspace_bytes, unsigned* status, void* stream) {
  if (!scan_sizes_ok(h, B, L) || !gs || !xs || !hs) return TTT_ERR_INVALID_ARG;
  if (L > kMaxTokens) return TTT_ERR_UNSUPPORTED;
  if (!is_aligned(saved, 16) || !is_aligned(workspace, 16) || !is_aligned(status, 4)) return TTT_ERR_INVALID_ARG;
  const RowTensor in[] = {rows(h, B, L, g, gs), rows(h, B, L, x, xs), bytes(lengths, size_t(B) * 4)};
  const RowTensor out[] = {rows(h, B, L, ho, hs), state(h, B, h_last), bytes(saved, ttt_scan_saved_size(h, B, L))};
  if (!is_aligned(lengths, 4) || !apart(in, 3, out, 3)) return TTT_ERR_INVALID_ARG;
  const RowTensor H0 = state(h, B, h0);
  if (!H0.readable() || may_share(H0, out[0]) || may_share(H0, out[2])) return TTT_ERR_INVALID_ARG;
  if (h0 != h_last && may_share(H0, out[1])) return TTT_ERR_INVALID_ARG;
  if (workspace_bytes < ttt_scan_workspace_size(h, B, L)) return TTT_ERR_WORKSPACE;
  (void)status;
  ScanArgs a{};
  a.g = g, a.x = x, a.h0 = h0, a.lengths = lengths, a.h = ho, a.h_last = h_last;
  a.saved = static_cast<float*>(saved);
  put_strides(a.gs, gs), put_strides(a.xs, xs), put_strides(a.hs, hs);
  a.L = L, a.B = B, a.D = h->cfg.D;
  const int64_t n = int64_t(B) * a.D;
  const ScanKernel f = h->cfg.dtype == TTT_BF16 ? pick<__nv_bfloat16>(false, h->cfg.gate, h->cfg.input)
                                                : pick<float>(false, h->cfg.gate, h->cfg.input);
  const int64_t grid = (n + 127) / 128;
  if (grid > 0x7fffffff) return TTT_ERR_UNSUPPORTED;
  f<<<unsigned(grid), 128, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

extern "C" int ttt_scan_backward(const ttt_scan* h, int32_t B, int64_t L, const void* dh, const ttt_strides* dhs,
                                 const float* dh_last, const void* g, const ttt_strides* gs, const void* x,
                                 const ttt_strides* xs, const int32_t* lengths, const void* saved, void* dg,
                                 const ttt_strides* dgs, void* dx, const ttt_strides* dxs, float* dh0, void* workspace,
                                 size_t workspace_bytes, unsigned* status, void* stream) {
  if (!scan_sizes_ok(h, B, L) || !dhs || !gs || !xs || !dgs || !dxs) return TTT_ERR_INVALID_ARG;
  if (L > kMaxTokens) return TTT_ERR_UNSUPPORTED;
  if (!is_aligned(saved, 16) || !is_aligned(workspace, 16) || !is_aligned(status, 4)) return TTT_ERR_INVALID_ARG;
  const size_t nsaved = ttt_scan_saved_size(h, B, L);
  if (nsaved && !saved) return TTT_ERR_INVALID_ARG;
  const RowTensor in[] = {rows(h, B, L, dh, dhs), rows(h, B, L, g, gs),        rows(h, B, L, x, xs),
                          state(h, B, dh_last),   bytes(lengths, size_t(B) * 4), bytes(saved, nsaved)};
  const RowTensor out[] = {rows(h, B, L, dg, dgs), rows(h, B, L, dx, dxs), state(h, B, dh0)};
  if (!is_aligned(lengths, 4) || !apart(in, 6, out, 3)) return TTT_ERR_INVALID_ARG;
  if (workspace_bytes < ttt_scan_workspace_size(h, B, L)) return TTT_ERR_WORKSPACE;
  (void)status;
  ScanArgs a{};
  a.dh = dh, a.g = g, a.x = x, a.dh_last = dh_last, a.lengths = lengths, a.dg = dg, a.dx = dx, a.dh0 = dh0;
  a.saved = static_cast<float*>(const_cast<void*>(saved));
  put_strides(a.dhs, dhs), put_strides(a.gs, gs), put_strides(a.xs, xs), put_strides(a.dgs, dgs),
      put_strides(a.dxs, dxs);
  a.L = L, a.B = B, a.D = h->cfg.D;
  const int64_t n = int64_t(B) * a.D;
  const ScanKernel f = h->cfg.dtype == TTT_BF16 ? pick<__nv_bfloat16>(true, h->cfg.gate, h->cfg.input)
                                                : pick<float>(true, h->cfg.gate, h->cfg.input);
  const int64_t grid = (n + 127) / 128;
  if (grid > 0x7fffffff) return TTT_ERR_UNSUPPORTED;
  f<<<unsigned(grid), 128, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}
