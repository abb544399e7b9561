// Rotary positions with several axes (ttt_ops.h, ttt_rope_*).
//
// Pair i of a head belongs to one axis and turns by phi = p_axis * theta_i.  In
// turns, phi / 2 pi = p * (theta_i / 2 pi): the product is formed in 64 bits and its
// whole turns are taken off there, since in 32 bits it is off by p 2^-24 turns (a
// position of 10^6 would lose three digits of the angle).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "op_checks.h"
#include "ttt_plan.cuh"

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
  int32_t units, items;       // vectors of pairs of a token; with those that are only copied
  int32_t lanes, rows;        // a block's items and tokens
  int32_t item_blocks, head_groups, heads;  // heads of a thread
};

template <class T>
__device__ __forceinline__ void open_word(uint32_t w, float (&v)[4 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(w);
  } else {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  }
}
template <class T>
__device__ __forceinline__ uint32_t close_word(const float (&v)[4 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(v[0]);
  } else {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
}

// BYTES of consecutive channels
template <class T, int BYTES>
struct Vec {
  static constexpr int N = BYTES / sizeof(T);
  static constexpr int kWords = (BYTES + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (BYTES == 16) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else if constexpr (BYTES == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x, w[1] = q.y;
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES == 16)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (BYTES == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (BYTES == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint16_t*>(p) = uint16_t(w[0]);
  }
  __device__ __forceinline__ void open(float (&v)[N]) const {
    if constexpr (BYTES == 2) {
      v[0] = __uint_as_float(w[0] << 16);
    } else {
      constexpr int K = 4 / sizeof(T);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        float u[K];
        open_word<T>(w[i], u);
#pragma unroll
        for (int k = 0; k < K; ++k) v[i * K + k] = u[k];
      }
    }
  }
  __device__ __forceinline__ void close(const float (&v)[N]) {
    if constexpr (BYTES == 2) {
      w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else {
      constexpr int K = 4 / sizeof(T);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        float u[K];
#pragma unroll
        for (int k = 0; k < K; ++k) u[k] = v[i * K + k];
        w[i] = close_word<T>(u);
      }
    }
  }
};

// A thread owns the same few pairs of every head (or channels that are only copied) and
// walks over tokens, so its frequencies stay in registers and each angle is formed once
// for all heads.  Bound by HBM: x is read and y written once, in vectors of BYTES.
//   ONE: the two channels of a pair lie in one vector (interleaved); else in two.
// bf16 takes the hardware's sine and cosine (2^-21.2 off on [-pi, pi], far below the
// output's 2^-9), fp32 sincospif.
constexpr int kHeadsAtOnce = 4;
template <class T, int BYTES, bool ONE>
__global__ void __launch_bounds__(256)
    rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTable tab) {
  using X = Vec<T, BYTES>;
  constexpr int P = ONE ? X::N / 2 : X::N;  // pairs of a thread
  const int item = blockIdx.x % a.item_blocks * a.lanes + threadIdx.x % a.lanes;
  const int row = threadIdx.x / a.lanes;
  if (row >= a.rows || item >= a.items) return;
  const int b = blockIdx.y / a.head_groups, h0 = blockIdx.y % a.head_groups * a.heads;
  const int heads = min(a.heads, a.H - h0);
  const T* const x = static_cast<const T*>(a.x) + b * a.xs[0] + h0 * a.xs[1];
  T* const y = static_cast<T*>(a.y) + b * a.ys[0] + h0 * a.ys[1];
  const int64_t n0 = int64_t(blockIdx.x / a.item_blocks) * a.rows + row;
  const int64_t hop = int64_t(gridDim.x / a.item_blocks) * a.rows;

  if (item >= a.units) {  // channels behind the pairs
    const int c = 2 * a.pairs + (item - a.units) * X::N;
    for (int64_t n = n0; n < a.N; n += hop)
      for (int h = 0; h < heads; ++h) {
        X v;
        v.load(x + h * a.xs[1] + n * a.xs[2] + c);
        v.store(y + h * a.ys[1] + n * a.ys[2] + c);
      }
    return;
  }
  const int i0 = item * P;
  const int cp = a.interleaved ? 2 * i0 : i0, cq = a.interleaved ? 2 * i0 + 1 : i0 + a.pairs;
  double turns[P];
  int axis[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    turns[k] = tab.turns[i0 + k];
    axis[k] = tab.axis[i0 + k];
  }
  for (int64_t n = n0; n < a.N; n += hop) {
    float sn[P], cs[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int64_t at = b * a.pos_batch + n * a.axes + axis[k];
      const double pos = a.pos_f32 ? double(__ldg(static_cast<const float*>(a.pos) + at))
                                   : double(__ldg(static_cast<const int*>(a.pos) + at));
      const double t = pos * turns[k];
      const float f = float(t - rint(t));
      if constexpr (sizeof(T) == 2) {
        const float r = f * 6.2831853071795865f;
        sn[k] = __sinf(r);
        cs[k] = __cosf(r);
      } else {
        sincospif(2.f * f, &sn[k], &cs[k]);
      }
      sn[k] *= a.sign;
    }
    for (int h = 0; h < heads; h += kHeadsAtOnce) {
      X p[kHeadsAtOnce], q[kHeadsAtOnce];
#pragma unroll
      for (int e = 0; e < kHeadsAtOnce; ++e)
        if (h + e < heads) {
          const T* from = x + (h + e) * a.xs[1] + n * a.xs[2];
          p[e].load(from + cp);
          if (!ONE) q[e].load(from + cq);
        }
#pragma unroll
      for (int e = 0; e < kHeadsAtOnce; ++e)
        if (h + e < heads) {
          T* to = y + (h + e) * a.ys[1] + n * a.ys[2];
          float u[X::N], v[X::N];
          p[e].open(u);
          if constexpr (ONE) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
              v[2 * k] = u[2 * k] * cs[k] - u[2 * k + 1] * sn[k];
              v[2 * k + 1] = u[2 * k + 1] * cs[k] + u[2 * k] * sn[k];
            }
            p[e].close(v);
            p[e].store(to + cp);
          } else {
            q[e].open(v);
            float yp[X::N], yq[X::N];
#pragma unroll
            for (int k = 0; k < P; ++k) {
              yp[k] = u[k] * cs[k] - v[k] * sn[k];
              yq[k] = v[k] * cs[k] + u[k] * sn[k];
            }
            p[e].close(yp);
            q[e].close(yq);
            p[e].store(to + cp);
            q[e].store(to + cq);
          }
        }
    }
  }
}

template <class T, int BYTES, bool ONE>
int launch(RopeArgs& a, const RopeTable& tab, bool copy, cudaStream_t st) {
  constexpr int V = BYTES / int(sizeof(T)), P = ONE ? V / 2 : V;
  a.units = a.pairs / P;
  a.items = a.units + (copy ? (a.d - 2 * a.pairs) / V : 0);
  a.item_blocks = (a.items + 127) / 128;
  a.lanes = (a.items + a.item_blocks - 1) / a.item_blocks;
  a.rows = 256 / a.lanes;
  // all heads in one thread share its angles; fewer where that would leave SMs idle
  const int64_t row_blocks = (a.N + a.rows - 1) / a.rows;
  const int64_t enough = int64_t(sm_count()) * 4;
  a.heads = a.H;
  auto blocks = [&] { return row_blocks * a.item_blocks * a.B * ((a.H + a.heads - 1) / a.heads); };
  while (a.heads > 1 && blocks() < enough) a.heads = (a.heads + 1) / 2;
  a.head_groups = (a.H + a.heads - 1) / a.heads;
  const int64_t gy = int64_t(a.B) * a.head_groups;
  if (gy > 65535) return TTT_ERR_UNSUPPORTED;
  const int64_t most = std::max<int64_t>(1, int64_t(sm_count()) * 16 / (a.item_blocks * gy));
  const int64_t gx = std::min(row_blocks, most) * a.item_blocks;
  rope_kernel<T, BYTES, ONE><<<dim3(unsigned(gx), unsigned(gy)), 256, 0, st>>>(a, tab);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
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
  // the widest vectors that rows, pairs and the channels behind them are whole numbers of
  const bool copy = x != y && c.d > 2 * h->pairs;
  const int part = a.interleaved ? 2 * h->pairs : h->pairs, behind = copy ? c.d - 2 * h->pairs : 0;
  int wide = 16;
  while (wide > e && (part * e % wide || behind * e % wide || !rows_aligned(X, wide) || !rows_aligned(Y, wide))) wide /= 2;
  const bool one = a.interleaved && wide > e;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (e == 2) {
    using T = __nv_bfloat16;
    if (one)
      return wide == 16 ? launch<T, 16, true>(a, h->tab, copy, st)
             : wide == 8 ? launch<T, 8, true>(a, h->tab, copy, st)
                         : launch<T, 4, true>(a, h->tab, copy, st);
    return wide == 16 ? launch<T, 16, false>(a, h->tab, copy, st)
           : wide == 8 ? launch<T, 8, false>(a, h->tab, copy, st)
           : wide == 4 ? launch<T, 4, false>(a, h->tab, copy, st)
                       : launch<T, 2, false>(a, h->tab, copy, st);
  }
  if (one) return wide == 16 ? launch<float, 16, true>(a, h->tab, copy, st) : launch<float, 8, true>(a, h->tab, copy, st);
  return wide == 16 ? launch<float, 16, false>(a, h->tab, copy, st)
         : wide == 8 ? launch<float, 8, false>(a, h->tab, copy, st)
                     : launch<float, 4, false>(a, h->tab, copy, st);
}
