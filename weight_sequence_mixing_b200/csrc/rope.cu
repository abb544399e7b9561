// Rotary positions with several axes (ttt_ops.h, ttt_rope_*).
//
// Pair i of a head belongs to one axis and turns by phi = p_axis * theta_i.  In
// turns, phi / 2 pi = p * (theta_i / 2 pi): the product is formed in 64 bits and its
// whole turns are taken off there, since in 32 bits it is off by p 2^-24 turns (a
// position of 10^6 would lose three digits of the angle).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#include "op_checks.h"

namespace ttt {
namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

struct RopeTable {
  double turns[TTT_ROPE_MAX_PAIRS];  // theta_i / 2 pi
  unsigned char axis[TTT_ROPE_MAX_PAIRS];
};

struct RopeArgs {
  const void* x;
  void* y;
  const void* pos;
  int64_t xs[3], ys[3], pos_batch;  // batch, head, token
  int64_t N;
  int32_t B, H, d, axes, pairs;
  int32_t pos_f32, interleaved;
  float sign;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// One thread per pair, and per channel that is only copied.
template <class T>
__global__ void rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTable tab) {
  const int items = a.d - a.pairs;
  const int64_t total = int64_t(a.B) * a.H * a.N * items;
  for (int64_t k = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; k < total; k += int64_t(gridDim.x) * blockDim.x) {
    const int i = int(k % items);
    const int64_t r = k / items;
    const int64_t n = r % a.N;
    const int64_t bh = r / a.N;
    const int h = int(bh % a.H), b = int(bh / a.H);
    const T* x = static_cast<const T*>(a.x) + b * a.xs[0] + h * a.xs[1] + n * a.xs[2];
    T* y = static_cast<T*>(a.y) + b * a.ys[0] + h * a.ys[1] + n * a.ys[2];
    if (i >= a.pairs) {
      y[a.pairs + i] = x[a.pairs + i];
      continue;
    }
    const int64_t at = b * a.pos_batch + n * a.axes + tab.axis[i];
    const double p = a.pos_f32 ? double(static_cast<const float*>(a.pos)[at])
                               : double(static_cast<const int*>(a.pos)[at]);
    const double turns = p * tab.turns[i];
    float sn, cs;
    sincospif(2.f * float(turns - rint(turns)), &sn, &cs);
    sn *= a.sign;
    const int ip = a.interleaved ? 2 * i : i, iq = a.interleaved ? 2 * i + 1 : i + a.pairs;
    const float u = to_f(x[ip]), v = to_f(x[iq]);
    put(y + ip, u * cs - v * sn);
    put(y + iq, v * cs + u * sn);
  }
}

}  // namespace
}  // namespace ttt

using namespace ttt;

struct ttt_rope {
  ttt_rope_config cfg;
  int32_t pairs;
  RopeTable tab;
};

extern "C" int ttt_rope_create(const ttt_rope_config* c, ttt_rope** out) {
  if (!out) return TTT_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c || c->axes < 1 || c->axes > TTT_ROPE_MAX_AXES || c->d < 1) return TTT_ERR_INVALID_ARG;
  if (c->pairing != TTT_ROPE_HALVES && c->pairing != TTT_ROPE_INTERLEAVED) return TTT_ERR_INVALID_ARG;
  if (c->dtype != TTT_F32 && c->dtype != TTT_BF16) return TTT_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int a = 0; a < c->axes; ++a) {
    if (c->pairs[a] < 1 || !(c->base[a] > 0.0) || !std::isfinite(c->base[a])) return TTT_ERR_INVALID_ARG;
    total += c->pairs[a];
  }
  if (2 * total > c->d) return TTT_ERR_INVALID_ARG;
  if (total > TTT_ROPE_MAX_PAIRS || c->d > 4096) return TTT_ERR_UNSUPPORTED;
  ttt_rope* h = new (std::nothrow) ttt_rope();
  if (!h) return TTT_ERR_INVALID_ARG;
  h->cfg = *c;
  h->pairs = int32_t(total);
  int at = 0;
  for (int a = 0; a < c->axes; ++a)
    for (int j = 0; j < c->pairs[a]; ++j, ++at) {
      h->tab.turns[at] = std::pow(c->base[a], -double(j) / c->pairs[a]) / kTwoPi;
      h->tab.axis[at] = static_cast<unsigned char>(a);
    }
  *out = h;
  return TTT_OK;
}

extern "C" void ttt_rope_destroy(ttt_rope* h) { delete h; }

extern "C" int ttt_rope_apply(const ttt_rope* h, int32_t B, int32_t H, int64_t N, const void* x, const ttt_strides* xs,
                              const void* pos, int32_t pos_dtype, int64_t pos_batch, void* y, const ttt_strides* ys,
                              int32_t inverse, void* stream) {
  if (!h || !xs || !ys || B < 1 || H < 1 || N < 0 || pos_batch < 0) return TTT_ERR_INVALID_ARG;
  if (pos_dtype != TTT_POS_I32 && pos_dtype != TTT_POS_F32) return TTT_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return TTT_ERR_INVALID_ARG;
  if (N == 0) return TTT_OK;
  if (N > (int64_t(1) << 40)) return TTT_ERR_UNSUPPORTED;
  const ttt_rope_config& c = h->cfg;
  const int e = c.dtype == TTT_BF16 ? 2 : 4;
  const RowTensor X(x, e, c.d, B, xs->batch, H, xs->head, N, xs->token);
  const RowTensor Y(y, e, c.d, B, ys->batch, H, ys->head, N, ys->token);
  const RowTensor P(pos, 4, int64_t(c.axes), B, pos_batch, N, c.axes);
  if (!X.readable() || !P.readable() || !Y.writable()) return TTT_ERR_INVALID_ARG;
  if (!same_tensor(X, Y) && may_share(X, Y)) return TTT_ERR_INVALID_ARG;
  if (may_share(P, Y)) return TTT_ERR_INVALID_ARG;
  RopeArgs a{};
  a.x = x;
  a.y = y;
  a.pos = pos;
  a.xs[0] = xs->batch, a.xs[1] = xs->head, a.xs[2] = xs->token;
  a.ys[0] = ys->batch, a.ys[1] = ys->head, a.ys[2] = ys->token;
  a.pos_batch = pos_batch;
  a.N = N;
  a.B = B, a.H = H, a.d = c.d, a.axes = c.axes, a.pairs = h->pairs;
  a.pos_f32 = pos_dtype == TTT_POS_F32;
  a.interleaved = c.pairing == TTT_ROPE_INTERLEAVED;
  a.sign = inverse ? -1.f : 1.f;
  const __int128 items = __int128(B) * H * N * (c.d - h->pairs);
  if (items > (__int128(1) << 60)) return TTT_ERR_UNSUPPORTED;
  const int64_t blocks = (int64_t(items) + 255) / 256;
  const int grid = int(blocks < (1 << 20) ? blocks : (1 << 20));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (e == 2)
    rope_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a, h->tab);
  else
    rope_kernel<float><<<grid, 256, 0, st>>>(a, h->tab);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}
