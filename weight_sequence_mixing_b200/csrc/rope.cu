// Rotary positions with several axes (ttt_ops.h, ttt_rope_*).
//
// Pair i of a head belongs to one axis and turns by phi = p_axis * theta_i.  The angle is
// formed in whole turns, phi / 2 pi = p * (theta_i / 2 pi), of which only the fraction
// counts.  For an integer p that is exact arithmetic modulo 2^64: with theta_i / 2 pi as a
// 64-bit fraction, the low 64 bits of the product are the turn.  For an fp32 p the product
// and its reduction are in fp64.  (In 32 bits the product is off by p 2^-24 turns: a
// position of 10^6 would lose three digits of the angle.)
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "op_checks.h"
#include "ttt_plan.cuh"
#include "vec.cuh"

namespace ttt {
namespace {

constexpr long double kTwoPi = 6.283185307179586476925286766559L;

struct RopeTable {
  uint64_t turns[TTT_ROPE_MAX_PAIRS];  // theta_i / 2 pi: its fraction in units of 2^-64, or (fp32 positions) an fp64's bits
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
  int32_t units, items;         // vectors of pairs of a token; with those that are only copied
  int32_t lanes, rows;          // a block's items, and its tokens at a time
  int32_t item_blocks, head_groups;
  int64_t tiles;                // of tokens, times head groups and batch entries
  int64_t row_tiles;            // of tokens
};

// Sine and cosine of 2 pi (quarter / 4 + u), |u| <= 1/8: polynomials in u^2, fitted for the least
// error against 64 bits (the sine's 3e-9 relative, the cosine's 5e-11).  The sine's leading
// coefficient is in two parts, so that only the last sum rounds.
__device__ __forceinline__ void sincos_turn(float u, uint32_t quarter, float* sn, float* cs) {
  constexpr double kLead = 6.283185287;
  const float w = u * u;
  float s = fmaf(w, -75.39356282f, 81.59235357f);
  s = fmaf(s, w, -41.34166146f);
  s = fmaf(s, w, float(kLead - double(float(kLead))));
  s = fmaf(u, float(kLead), s * u);
  float c = fmaf(w, 59.24596302f, -85.4437417f);
  c = fmaf(c, w, 64.93932647f);
  c = fmaf(c, w, -19.73920869f);
  c = fmaf(c, w, 1.f);
  const uint32_t p = __float_as_uint(quarter & 1 ? c : s), q = __float_as_uint(quarter & 1 ? s : c);
  *sn = __uint_as_float(p ^ ((quarter << 30) & 0x80000000u));
  *cs = __uint_as_float(q ^ ((quarter + 1) << 30 & 0x80000000u));
}

// tokens of a thread: eight or four steps in all, of which a head takes one
constexpr int tokens_of(int bytes, bool one, int heads) { return std::max(1, (one || bytes < 16 ? 8 : 4) / heads); }

// A thread owns a vector of pairs (or of channels that are only copied) of every token: its
// frequencies stay in registers while it walks over tiles of (token, head) steps.  Of a
// tile it first issues all loads, then forms each token's angles once for its HEADS heads,
// turns and stores.  Bound by HBM (x read, y written once); what that takes is bytes in
// flight, here 64 to 128 a thread and 768 threads an SM.
//   ONE: the two channels of a pair lie in one vector (interleaved); else in two.
// bf16 takes the hardware's sine and cosine, 2^-21.2 off on [-pi, pi]: an output is off by
// 2^-20 (|x_p| + |x_q|) at most before its rounding, which only shows where the pair's two
// products cancel to less than 2^-11 of their size (fp32's forms would leave 2^-23 there, and took
// the views below from 145 to 155 us, which the angles' instructions then bound).  fp32 takes the
// quarter turns off in integers first, so that an eighth of a turn at most is rounded to 24 bits,
// and then polynomials.
// Measured: 196608 tokens x 2 heads x 512 bf16 139 us (88% of the copy bandwidth).  Angles in
// fp64, one (token, heads) step ahead, took 200 us; a tile's angles shared in shared memory 211.
template <class T, int BYTES, bool ONE, int HEADS, bool POS_F32>
__global__ void __launch_bounds__(256, ONE ? 3 : 2)
    rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTable tab) {
  using X = Vec<T, BYTES>;
  constexpr int P = ONE ? X::N / 2 : X::N;  // pairs of a thread
  constexpr int kTokens = tokens_of(BYTES, ONE, HEADS);
  const int item = blockIdx.x % a.item_blocks * a.lanes + threadIdx.x % a.lanes;
  const int row = threadIdx.x / a.lanes;
  if (row >= a.rows || item >= a.items) return;
  // copied channels take the same walk as pairs, so that the lanes of a warp stay together
  const bool rotates = item < a.units;
  const int i0 = rotates ? item * P : 0;
  const int cp = !rotates ? 2 * a.pairs + (item - a.units) * X::N : a.interleaved ? 2 * i0 : i0;
  const int cq = a.interleaved ? 2 * i0 + 1 : i0 + a.pairs;
  uint64_t freq[P];  // turns a position, as a 64-bit fraction or (fp32 positions) an fp64
  int axis[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    freq[k] = tab.turns[i0 + k];
    axis[k] = tab.axis[i0 + k];
    // held in registers: read again at each use, the lanes' different places in constant
    // memory come one after another (575 us for the views below)
    asm volatile("" : "+l"(freq[k]), "+r"(axis[k]));
  }
  const bool one_axis = axis[0] == axis[P - 1];
  const int hop = gridDim.x / a.item_blocks;
  for (int64_t tile = blockIdx.x / a.item_blocks; tile < a.tiles; tile += hop) {
    const int64_t bh = tile / a.row_tiles;
    const int b = int(bh / a.head_groups), h0 = int(bh % a.head_groups) * HEADS;
    const int64_t n0 = (tile - bh * a.row_tiles) * (kTokens * a.rows) + row;
    X p[kTokens][HEADS], q[kTokens][HEADS];
    int word[kTokens];  // the positions of the first pair, as they are stored
    {
      const int* pos = static_cast<const int*>(a.pos) + b * a.pos_batch + n0 * a.axes;
      const T* x = static_cast<const T*>(a.x) + b * a.xs[0] + h0 * a.xs[1] + n0 * a.xs[2];
#pragma unroll
      for (int g = 0; g < kTokens; ++g) {
        if (n0 + g * a.rows < a.N) {
#pragma unroll
          for (int h = 0; h < HEADS; ++h)
            if (h0 + h < a.H) {
              p[g][h].load(x + h * a.xs[1] + cp);
              if (!ONE && rotates) q[g][h].load(x + h * a.xs[1] + cq);
            }
          word[g] = __ldg(pos + axis[0]);
        }
        x += a.rows * a.xs[2];
        pos += a.rows * a.axes;
      }
    }
    const int* pos = static_cast<const int*>(a.pos) + b * a.pos_batch + n0 * a.axes;
    T* y = static_cast<T*>(a.y) + b * a.ys[0] + h0 * a.ys[1] + n0 * a.ys[2];
#pragma unroll
    for (int g = 0; g < kTokens; ++g, y += a.rows * a.ys[2], pos += a.rows * a.axes) {
      if (n0 + g * a.rows >= a.N) break;
      float cs[P], sn[P];
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int w = k == 0 || one_axis ? word[g] : __ldg(pos + axis[k]);
        // the turn: its fraction in [-1/2, 1/2], or in units of 2^-64
        double turn = 0.;
        uint64_t part = 0;
        if (POS_F32) {
          turn = double(__int_as_float(w)) * __longlong_as_double(int64_t(freq[k]));
          turn -= rint(turn);
        } else {
          part = uint64_t(int64_t(w)) * freq[k];
        }
        if constexpr (sizeof(T) == 2) {
          const float r = (POS_F32 ? float(turn) : float(int(part >> 32)) * 0x1p-32f) * 6.2831853071795865f;
          sn[k] = __sinf(r);
          cs[k] = __cosf(r);
        } else if constexpr (POS_F32) {
          const double quarters = rint(4. * turn);
          sincos_turn(float(fma(-0.25, quarters, turn)), uint32_t(int(quarters)), &sn[k], &cs[k]);
        } else {
          sincos_turn(float(int64_t(part << 2)) * 0x1p-66f, uint32_t((part + (uint64_t(1) << 61)) >> 62), &sn[k], &cs[k]);
        }
        sn[k] *= a.sign;
      }
#pragma unroll
      for (int h = 0; h < HEADS; ++h) {
        if (h0 + h >= a.H) break;
        T* const to = y + h * a.ys[1];
        if (!rotates) {
          p[g][h].store(to + cp);
          continue;
        }
        float u[X::N], v[X::N];
        p[g][h].open(u);
        if constexpr (ONE) {
#pragma unroll
          for (int k = 0; k < P; ++k) {
            v[2 * k] = u[2 * k] * cs[k] - u[2 * k + 1] * sn[k];
            v[2 * k + 1] = u[2 * k + 1] * cs[k] + u[2 * k] * sn[k];
          }
          p[g][h].close(v);
          p[g][h].store(to + cp);
        } else {
          q[g][h].open(v);
          float yp[X::N], yq[X::N];
#pragma unroll
          for (int k = 0; k < P; ++k) {
            yp[k] = u[k] * cs[k] - v[k] * sn[k];
            yq[k] = v[k] * cs[k] + u[k] * sn[k];
          }
          p[g][h].close(yp);
          q[g][h].close(yq);
          p[g][h].store(to + cp);
          q[g][h].store(to + cq);
        }
      }
    }
  }
}

template <class T, int BYTES, bool ONE, int HEADS>
int launch(RopeArgs& a, const RopeTable& tab, bool copy, cudaStream_t st) {
  constexpr int V = BYTES / int(sizeof(T)), P = ONE ? V / 2 : V;
  constexpr int kTokens = tokens_of(BYTES, ONE, HEADS);
  a.units = a.pairs / P;
  a.items = a.units + (copy ? (a.d - 2 * a.pairs) / V : 0);
  a.item_blocks = (a.items + 255) / 256;
  a.lanes = (a.items + a.item_blocks - 1) / a.item_blocks;
  a.rows = 256 / a.lanes;
  a.head_groups = (a.H + HEADS - 1) / HEADS;
  a.row_tiles = (a.N + kTokens * a.rows - 1) / (kTokens * a.rows);
  a.tiles = a.row_tiles * a.head_groups * a.B;
  const int64_t grid = std::min(a.tiles, std::max<int64_t>(1, int64_t(sm_count()) * (ONE ? 3 : 2) / a.item_blocks)) * a.item_blocks;
  if (a.pos_f32)
    rope_kernel<T, BYTES, ONE, HEADS, true><<<unsigned(grid), 256, 0, st>>>(a, tab);
  else
    rope_kernel<T, BYTES, ONE, HEADS, false><<<unsigned(grid), 256, 0, st>>>(a, tab);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

// Heads of a thread: those that share its angles.  Six where six divides the heads (in halves,
// whose pair takes two vectors), four where that leaves one place empty at most, else two (48672
// tokens x 6 heads x 64 in halves: 14.1 us with six heads a thread, 15.7 with three, 16.0 with
// two).  Narrow vectors have one form.
template <class T, int BYTES, bool ONE>
int launch_heads(RopeArgs& a, const RopeTable& tab, bool copy, cudaStream_t st) {
  if constexpr (BYTES < 16) {
    return launch<T, BYTES, ONE, 2>(a, tab, copy, st);
  } else {
    if (a.H == 1) return launch<T, BYTES, ONE, 1>(a, tab, copy, st);
    if constexpr (!ONE)
      if (a.H % 6 == 0) return launch<T, BYTES, ONE, 6>(a, tab, copy, st);
    if (a.H % 4 == 0 || a.H % 4 == 3) return launch<T, BYTES, ONE, 4>(a, tab, copy, st);
    return launch<T, BYTES, ONE, 2>(a, tab, copy, st);
  }
}

}  // namespace
}  // namespace ttt

using namespace ttt;

struct ttt_rope {
  ttt_rope_config cfg;
  int32_t pairs;
  RopeTable tab[2];  // for int32 and for fp32 positions
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
      const long double turns = powl(c->base[a], -static_cast<long double>(j) / c->pairs[a]) / kTwoPi;
      const double rounded = double(turns);
      h->tab[0].turns[at] = static_cast<uint64_t>(ldexpl(turns - floorl(turns), 64));
      std::memcpy(&h->tab[1].turns[at], &rounded, sizeof(rounded));
      h->tab[0].axis[at] = h->tab[1].axis[at] = static_cast<unsigned char>(a);
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
  if (__int128(B) * H * N > (__int128(1) << 60)) return TTT_ERR_UNSUPPORTED;
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
      return wide == 16 ? launch_heads<T, 16, true>(a, h->tab[a.pos_f32], copy, st)
             : wide == 8 ? launch_heads<T, 8, true>(a, h->tab[a.pos_f32], copy, st)
                         : launch_heads<T, 4, true>(a, h->tab[a.pos_f32], copy, st);
    return wide == 16 ? launch_heads<T, 16, false>(a, h->tab[a.pos_f32], copy, st)
           : wide == 8 ? launch_heads<T, 8, false>(a, h->tab[a.pos_f32], copy, st)
           : wide == 4 ? launch_heads<T, 4, false>(a, h->tab[a.pos_f32], copy, st)
                       : launch_heads<T, 2, false>(a, h->tab[a.pos_f32], copy, st);
  }
  if (one) return wide == 16 ? launch_heads<float, 16, true>(a, h->tab[a.pos_f32], copy, st) : launch_heads<float, 8, true>(a, h->tab[a.pos_f32], copy, st);
  return wide == 16 ? launch_heads<float, 16, false>(a, h->tab[a.pos_f32], copy, st)
         : wide == 8 ? launch_heads<float, 8, false>(a, h->tab[a.pos_f32], copy, st)
                     : launch_heads<float, 4, false>(a, h->tab[a.pos_f32], copy, st);
}
