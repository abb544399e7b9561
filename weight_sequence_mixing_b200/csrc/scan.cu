// Gated linear recurrence (ttt_ops.h, ttt_scan_*):
//   h_t = a_t h_{t-1} + u_t,   a = g | sigma(g) | exp(g),   u = x | (1 - a) x.
// Backward: lam_t = dh_t + mu_t with mu_t = a_{t+1} lam_{t+1}, the gradient that
// reaches h_t from the later tokens (mu_len = dh_last).
//
// A step is an affine map of the state, and maps compose: a run of tokens takes a
// state s to A s + H with A the product of its gates and H its result from zero.  So
// the tokens are cut into tiles.  A tile's (A, H) needs only its own rows; the state that
// enters it comes from the tiles before: each tile publishes its (A, H), finds the nearest
// earlier tile whose outgoing state is known, applies the maps in between in token order,
// and publishes its own outgoing state.  Every input is read once and every output
// written once: the bound is HBM.
//   - A block's warps have three trades.  One hands out tiles and fetches their rows into a
//     ring of stages by TMA.  Sixteen sweep a tile's rows twice: first for the maps, and one
//     tile later, when the states that enter are there, for the states themselves.  Two
//     follow the chain of states from tile to tile, the block's tiles in turn.  So a tile's
//     state is waited for while the next tile's maps are formed, and loads run on
//     throughout.  (Rows that TMA cannot address, on strides that are no multiple of 16
//     bytes, are fetched by the sweeping warps in 4-byte asynchronous copies.  A row that
//     starts on an odd multiple of 2 bytes is copied from the 2 bytes before it on, and
//     shifted where it is read.)
//   - The gates are formed in both sweeps.  Keeping them (8 bytes a value in registers) was
//     measured: it holds too few tokens in flight for the chain's latency (5.98 ms).
//   - A published map or state is a word that shows by itself whether it is there.  Flags
//     behind fences took 7.0 ms in the same form.
//   - A warp takes the same channels of a few consecutive tokens; a lane one 4-byte word
//     of channels of each.
//   - Tiles are handed out by a counter, tokens first to last, so a tile only waits for
//     tiles of blocks that already run: the order of the hardware's blocks does not matter,
//     nor what else runs on the GPU.
//   - The state that enters a tile is always a known state with the maps applied one by
//     one, so a result has the same bits whichever tile's state was found first.
// The backward pass is the same over the tokens last to first; the states h_{t-1} that the
// gates' gradient needs are formed again in fp32 from states that the forward pass kept
// (one in 128 tokens, a backward tile), not read back rounded.
//
// Measured, bf16, 1024 channels: forward over 1029120 tokens 1.22 to 1.30 ms, box by box (79 to
// 74% of the copy bandwidth; exponential gate), over 64 sequences of 2048 142 us (87%; plain gate), 187 us
// with a sigmoid and its complement, where the exponentials and reciprocals keep their unit
// 68% busy; backward 273 and 317 us (75 and 65%), bound by issue.  A single long chain adds
// its latency: 131072 tokens take 168 us forward and 338 back.  Tiles half as long, two
// blocks an SM, took 1.74 ms for the million tokens; one chain warp 2.30 (at that length).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <new>

#include "../../include/ttt_diag.h"
#include "op_checks.h"
#include "per_device.h"
#include "ptx.cuh"
#include "tc_gemm.cuh"
#include "ttt_plan.cuh"
#include "vec.cuh"

namespace ttt {
namespace {

constexpr int kWarps = 16;             // warps that sweep a tile's rows
constexpr int kChainWarp = kWarps;     // two warps that follow the chain of states, tile about
constexpr int kFeedWarp = kWarps + 2;  // the warp that hands out tiles and fetches their rows
constexpr int kThreads = 32 * (kWarps + 3);
constexpr int kRowBytes = 128;     // a tile's channels: 32 lanes of 4 bytes
constexpr int kSave = 128;         // tokens from one kept state to the next: a backward tile
constexpr int kShort = 16;         // longest sequence of the short form
constexpr int kWindow = 64;        // earlier tiles looked at
enum : int { kLoadTma = 0, kLoad4 = 1, kLoad2 = 2 };

struct ScanArgs {
  const void *g, *x, *dh;
  const float *h0, *dh_last;
  const int* lengths;
  void *h, *dg, *dx;
  float *h_last, *dh0, *saved;
  int64_t gs[2], xs[2], hs[2], dhs[2], dgs[2], dxs[2];  // batch, token
  int64_t L;
  int32_t B, D;
  // tiles
  unsigned* counter;  // next tile to hand out; null: by block index, one tile a sequence
  uint64_t* maps;     // [tile][channel of the tile] (A, H)
  uint32_t* states;   // [tile][channel of the tile]
  unsigned* status;
  int32_t cols, per_col;  // columns of channels; tiles of a sequence
  int32_t total;          // tiles in all
  int32_t load;           // kLoadTma, kLoad4, kLoad2
  int32_t wide;           // outputs take 4-byte stores
  int32_t kept;           // kept states of a sequence
  unsigned long long wait_ns;  // the longest wait
};

// The values of a lane's 4 bytes: one fp32 or two bf16.
template <class T>
struct Word;
template <>
struct Word<float> {
  static constexpr int N = 1;
  using V = One;
  static __device__ __forceinline__ V all(float v) { return {v}; }
  static __device__ __forceinline__ V make(const float (&v)[1]) { return {v[0]}; }
  static __device__ __forceinline__ V open(uint32_t w) { return {__uint_as_float(w)}; }
  static __device__ __forceinline__ uint32_t close(V v) { return __float_as_uint(v.v); }
};
template <>
struct Word<__nv_bfloat16> {
  static constexpr int N = 2;
  using V = Two;
  static __device__ __forceinline__ V all(float v) { return two(v, v); }
  static __device__ __forceinline__ V make(const float (&v)[2]) { return two(v[0], v[1]); }
  static __device__ __forceinline__ V open(uint32_t w) {
    return two(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t close(V v) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
};

// a and 1 - a of a lane's values; the complement is formed on its own, so that it keeps
// its digits where a is close to 1.  bf16 inputs take the hardware's exponential (2^-22
// off, and 2^-24 of the exponent's size), fp32 ones the library's; the reciprocal is the
// hardware's, 2^-23 off at most.
template <class T, int GATE>
__device__ __forceinline__ void gate(typename Word<T>::V g, typename Word<T>::V& a, typename Word<T>::V& rest) {
  using W = Word<T>;
  if constexpr (GATE == TTT_GATE_VALUE) {
    a = g;
    rest = sub_(W::all(1.f), g);
  } else if constexpr (sizeof(T) == 2) {
    const Two y = mul_(g, W::all(GATE == TTT_GATE_SIGMOID ? -1.4426950408889634f : 1.4426950408889634f));
    const Two e = two(exp2_fast(y[0]), exp2_fast(y[1]));
    if constexpr (GATE == TTT_GATE_SIGMOID) {
      const Two s = add_(e, W::all(1.f));
      a = two(rcp_fast(s[0]), rcp_fast(s[1]));
      // from 2^60 on the complement is one: e a would meet a reciprocal below the normal range (zero
      // from 2^126 on), or an infinite e
      const Two q = mul_(e, a);  // NaN where the gate is
      rest = two(e[0] > 0x1p60f ? 1.f : q[0], e[1] > 0x1p60f ? 1.f : q[1]);
    } else {
      a = e;
      // 1 - e^g: below 1/2 in size by the series of (1 - e^g) / -g, 2^-26 off at most, which
      // keeps the digits that the difference loses
      Two s = W::all(1.f / 362880.f);
      s = fma_(s, g, W::all(1.f / 40320.f));
      s = fma_(s, g, W::all(1.f / 5040.f));
      s = fma_(s, g, W::all(1.f / 720.f));
      s = fma_(s, g, W::all(1.f / 120.f));
      s = fma_(s, g, W::all(1.f / 24.f));
      s = fma_(s, g, W::all(1.f / 6.f));
      s = fma_(s, g, W::all(0.5f));
      s = fma_(s, g, W::all(1.f));
      s = mul_(s, g);
      const Two f = sub_(W::all(1.f), e);
      rest = two(fabsf(g[0]) < 0.5f ? -s[0] : f[0], fabsf(g[1]) < 0.5f ? -s[1] : f[1]);
    }
  } else if constexpr (GATE == TTT_GATE_SIGMOID) {  // of e^-|g| in (0, 1]: nothing overflows
    const float e = expf(-fabsf(g.v));
    const float p = rcp_fast(1.f + e), q = e * p;
    a.v = g.v < 0.f ? q : p;
    rest.v = g.v < 0.f ? p : q;
  } else {
    a.v = expf(g.v);
    rest.v = -expm1f(g.v);
  }
}
// d gate / d g times `v`
template <int GATE, class V>
__device__ __forceinline__ V gate_grad(V a, V rest, V v) {
  if constexpr (GATE == TTT_GATE_VALUE) return v;
  else if constexpr (GATE == TTT_GATE_EXP) return mul_(v, a);
  else return mul_(mul_(v, a), rest);
}

// A s + H.  A state of zero gives H even where the product of the gates overflowed.
__device__ __forceinline__ float apply(float A, float H, float s) { return s == 0.f ? H : fmaf(A, s, H); }

__device__ __forceinline__ int64_t length_of(const ScanArgs& p, int b) {
  if (!p.lengths) return p.L;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

struct Place {
  int b, col, i;  // batch entry, column of channels, tile of the sequence in token order
};
struct alignas(16) Job {
  int t;    // the tile's number as handed out, or -1: no more
  int len;  // tokens of its sequence
  int col, i, b;
  int64_t out[2];  // the tile's first element in the outputs: h; or dx and dg
};
template <bool BACKWARD>
__device__ __forceinline__ Place place_of(const ScanArgs& p, int t) {
  const int columns = p.B * p.cols;  // fits: one tile a column at least
  const int k = t / columns, r = t - k * columns;
  return {r / p.cols, r % p.cols, BACKWARD ? p.per_col - 1 - k : k};
}

// Published maps and states carry their own readiness: the memory starts as all ones (a
// NaN that no value is stored as), and a map is one 8-byte word, so a reader needs no
// flag and a writer no fence.
constexpr uint32_t kAbsent = 0xffffffffu;
__device__ __forceinline__ uint32_t present(float v) {
  const uint32_t w = __float_as_uint(v);
  return w == kAbsent ? 0x7fffffffu : w;
}
template <int N>
__device__ __forceinline__ void publish_map(const ScanArgs& p, int t, const float (&A)[N], const float (&H)[N]) {
  uint64_t w[N];
#pragma unroll
  for (int v = 0; v < N; ++v) w[v] = uint64_t(present(H[v])) << 32 | present(A[v]);
  uint64_t* to = p.maps + (int64_t(t) * 32 + threadIdx.x % 32) * N;
  if constexpr (N == 2)
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(to), "l"(w[0]), "l"(w[N - 1]) : "memory");
  else
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(to), "l"(w[0]) : "memory");
}
template <int N>
__device__ __forceinline__ void publish_state(const ScanArgs& p, int t, const float (&s)[N]) {
  uint32_t* to = p.states + (int64_t(t) * 32 + threadIdx.x % 32) * N;
  if constexpr (N == 2)
    asm volatile("st.relaxed.gpu.global.v2.u32 [%0], {%1, %2};" ::"l"(to), "r"(present(s[0])), "r"(present(s[N - 1]))
                 : "memory");
  else
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(to), "r"(present(s[0])) : "memory");
}
// This lane's words of a tile, and whether a word is there
template <int N>
__device__ __forceinline__ void load_map(const ScanArgs& p, int t, uint64_t (&w)[N]) {
  const uint64_t* from = p.maps + (int64_t(t) * 32 + threadIdx.x % 32) * N;
  if constexpr (N == 2)
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(w[0]), "=l"(w[N - 1]) : "l"(from));
  else
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w[0]) : "l"(from));
}
template <int N>
__device__ __forceinline__ void load_state(const ScanArgs& p, int t, uint32_t (&w)[N]) {
  const uint32_t* from = p.states + (int64_t(t) * 32 + threadIdx.x % 32) * N;
  if constexpr (N == 2)
    asm volatile("ld.relaxed.gpu.global.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[N - 1]) : "l"(from));
  else
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(w[0]) : "l"(from));
}
__device__ __forceinline__ float apply_word(uint64_t w, float s) {
  return apply(__uint_as_float(uint32_t(w)), __uint_as_float(uint32_t(w >> 32)), s);
}

// The state that enters tile `t` (the chain warp; `before` earlier tiles of its
// column, `step` tiles apart): see the top of the file.  Looks at kNear tiles at a time, nearest first, and
// farther as long as all nearer maps are there.  A wait that runs out gives NaN.
constexpr int kNear = 8;
template <int N>
__device__ __forceinline__ void look_back(const ScanArgs& p, int t, int before, int step, float (&s)[N]) {
  unsigned long long since = 0;
  for (int spin = 0;; ++spin) {
    for (int d = 0; d < kWindow && d < before; d += kNear) {  // tiles d + 1 .. d + kNear back
      uint64_t map[kNear][N];
      uint32_t st[kNear][N];
      // all loads first, so that one trip to L2 brings the window (past the first tile: the first again)
#pragma unroll
      for (int e = 0; e < kNear; ++e) {
        const int q = t - min(d + e + 1, before) * step;
        load_state<N>(p, q, st[e]);
        load_map<N>(p, q, map[e]);
      }
      unsigned maps = 0, states = 0;
#pragma unroll
      for (int e = 0; e < kNear; ++e) {
        const bool in = d + e < before;
        maps |= unsigned(in && uint32_t(map[e][0]) != kAbsent && uint32_t(map[e][N - 1]) != kAbsent) << e;
        states |= unsigned(in && st[e][0] != kAbsent && st[e][N - 1] != kAbsent) << e;
      }
      maps = __reduce_and_sync(~0u, maps);
      states = __reduce_and_sync(~0u, states);
      if (states) {
        const int j = __ffs(states) - 1;
        if ((~maps & ((1u << j) - 1)) == 0) {
#pragma unroll
          for (int e = kNear - 1; e >= 0; --e) {
#pragma unroll
            for (int v = 0; v < N; ++v) {
              if (e == j) s[v] = __uint_as_float(st[e][v]);
              if (e < j) s[v] = apply_word(map[e][v], s[v]);
            }
          }
          for (int q = d; q > 0; q -= kNear) {  // the windows before this one are all there
#pragma unroll
            for (int e = 0; e < kNear; ++e) load_map<N>(p, t - (q - e) * step, map[e]);
#pragma unroll
            for (int e = 0; e < kNear; ++e)
#pragma unroll
              for (int v = 0; v < N; ++v) s[v] = apply_word(map[e][v], s[v]);
          }
          return;
        }
        break;
      }
      if (maps != (1u << kNear) - 1) break;
    }
    if (spin % 64 == 63) {
      const unsigned long long now = __shfl_sync(~0u, global_ns(), 0);
      if (!since) since = now;
      if (now - since > p.wait_ns) break;
    }
  }
  if (threadIdx.x % 32 == 0 && p.status) atomicOr(p.status, kStatusTimeout);
#pragma unroll
  for (int v = 0; v < N; ++v) s[v] = __int_as_float(0x7fc00000);
}

// A row's word of one output
template <class T>
__device__ __forceinline__ void put_word(const ScanArgs& p, T* to, int c, typename Word<T>::V v) {
  const uint32_t w = Word<T>::close(v);
  if (Word<T>::N == 1 || p.wide) {
    *reinterpret_cast<uint32_t*>(to) = w;
  } else {
    uint16_t* h = reinterpret_cast<uint16_t*>(to);
    h[0] = uint16_t(w);
    if (c + 1 < p.D) h[1] = uint16_t(w >> 16);
  }
}

// A row of one output by a warp, a lane's word at channel c.  Where the row starts on an odd
// multiple of 2 bytes, the words of memory are those one channel earlier: the second half of
// the lane before and the first of one's own.
template <class T>
__device__ __forceinline__ void put_row(const ScanArgs& p, T* to, int c, typename Word<T>::V v) {
  const uint32_t w = Word<T>::close(v);
  if (Word<T>::N == 1 || p.wide) {
    if (c < p.D) *reinterpret_cast<uint32_t*>(to) = w;
    return;
  }
  uint16_t* const h = reinterpret_cast<uint16_t*>(to);
  if ((reinterpret_cast<uintptr_t>(to) & 2) == 0) {
    if (c + 1 < p.D)
      *reinterpret_cast<uint32_t*>(to) = w;
    else if (c < p.D)
      h[0] = uint16_t(w);
    return;
  }
  const int lane = threadIdx.x % 32;
  const uint32_t before = __shfl_up_sync(~0u, w, 1);
  if (lane == 0) {
    if (c < p.D) h[0] = uint16_t(w);
  } else if (c < p.D) {
    *reinterpret_cast<uint32_t*>(h - 1) = before >> 16 | w << 16;
  } else if (c == p.D) {
    h[-1] = uint16_t(before >> 16);
  }
  if (lane == 31 && c + 1 < p.D) h[1] = uint16_t(w >> 16);
}

// Tiles of 256 tokens forward and 128 backward (one tensor more), three and four stages:
// 192 KB, one block an SM.
template <class T, bool BACKWARD>
struct Shape {
  static constexpr int N = Word<T>::N;
  static constexpr int kRows = BACKWARD ? 8 : 16;  // tokens of a warp
  static constexpr int kTile = kWarps * kRows;
  static_assert(BACKWARD ? kTile == kSave : kTile % kSave == 0, "each backward tile starts from a kept state, and no other is kept");
  static constexpr int kBox = kTile * kRowBytes;  // bytes of one tensor's tile
  static constexpr int kTensors = BACKWARD ? 3 : 2;
  static constexpr int kStages = BACKWARD ? 4 : 3;
  static constexpr int kStageBytes = kTensors * kBox;
  static constexpr int kMostJobs = kStages + 2;
  struct Scratch {  // behind the stages; two of each by parity of the block's tiles
    using V = typename Word<T>::V;
    V A[2][kWarps][32];  // each warp's map: A,
    V H[2][kWarps][32];  // and H, then in its place the state that enters the warp's rows
    V R[BACKWARD ? 2 : 1][BACKWARD ? kWarps : 1][32];  // backward: the map A mu + R, then the mu that enters
    uint64_t full[kMostJobs], empty[kMostJobs];  // a tile is known, and by TMA its rows are there; is done with
    uint64_t mapped[2], entered[2];          // a tile's maps are there; its states
    Job job[kMostJobs];
    uint32_t extra[N == 2 ? kStages : 1][kTensors][kTile];  // see fetch
    int abort;
  };
  static constexpr int kSmem = 1024 + kStages * kStageBytes + int(sizeof(Scratch));
};

// A warp's rows of one tensor's tile, from token t0 on, into shared memory at the swizzle TMA
// uses.  Only the bytes of live channels are read, the rest of a word is filled with zero.
// Rows on odd multiples of 2 bytes (kLoad2): a lane's word starts one channel early, and the
// channel that this leaves out of the last lane's goes to `extra`, one word a row.
template <class T, int ROWS>
__device__ __forceinline__ void fetch(const ScanArgs& p, const void* base, const int64_t (&s)[2], int b, int c0, int64_t t0,
                                      int64_t len, uint8_t* dst, uint32_t* extra) {
  const int lane = threadIdx.x % 32, c = c0 + lane * Word<T>::N;
  const int rows = int(len - t0 >= ROWS ? ROWS : len > t0 ? len - t0 : 0);
  const T* from = static_cast<const T*>(base) + (rows ? b * s[0] + t0 * s[1] : 0);
  const uint32_t to = smem_u32(dst);
  if (p.load == kLoad4) {
    from += c < p.D ? c : 0;
#pragma unroll 16
    for (int r = 0; r < ROWS; ++r) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + r * kRowBytes + ((lane * 4) ^ ((r & 7) << 4))),
                   "l"(from), "r"(r < rows && c < p.D ? 4 : 0)
                   : "memory");
      if (r + 1 < rows) from += s[1];
    }
    return;
  }
  // bytes of the word that starts at channel f: of two channels, one or none
  auto live = [&](int f) { return f >= p.D ? 0 : f + 1 >= p.D ? 2 : 4; };
#pragma unroll 4
  for (int r = 0; r < rows; ++r, from += s[1]) {
    const int late = int(reinterpret_cast<uintptr_t>(from) >> 1 & 1);
    const int f = c - late, n = live(f);
    const uint32_t word = to + r * kRowBytes + ((lane * 4) ^ ((r & 7) << 4));
    if (f < 0 && from == static_cast<const T*>(base)) {  // nothing lies before a tensor's first element
      *reinterpret_cast<uint32_t*>(dst + r * kRowBytes + ((lane * 4) ^ ((r & 7) << 4))) =
          uint32_t(*reinterpret_cast<const uint16_t*>(from)) << 16;
    } else {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(word),
                   "l"(reinterpret_cast<uintptr_t>(n ? from + f : from) & ~uintptr_t(3)), "r"(n)
                   : "memory");
    }
    if (late && lane == 31) {
      const int e = c0 + 63, m = live(e);
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(extra + r)),
                   "l"(reinterpret_cast<uintptr_t>(m ? from + e : from) & ~uintptr_t(3)), "r"(m)
                   : "memory");
    }
  }
}

template <class T, int GATE, int INPUT, bool BACKWARD, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
    scan_tile_kernel(const __grid_constant__ ScanArgs p, const __grid_constant__ CUtensorMap mg,
                     const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap md) {
  using S = Shape<T, BACKWARD>;
  using W = Word<T>;
  using V = typename W::V;
  constexpr int N = S::N, kStages = S::kStages, kTile = S::kTile, kRows = S::kRows;
  // tiles handed to the block at a time; without TMA two more than stages, so that a warp whose own
  // places are free need not wait for the others
  constexpr int kJobs = TMA ? kStages : S::kMostJobs;
  extern __shared__ uint8_t raw[];
  uint8_t* const stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  typename S::Scratch& sc = *reinterpret_cast<typename S::Scratch*>(stages + kStages * S::kStageBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int step = p.B * p.cols;  // tiles from one of a column to its next

  if (threadIdx.x == 0) {
    for (int s = 0; s < kJobs; ++s) {
      mbar_init(&sc.full[s], 1);
      mbar_init(&sc.empty[s], kWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sc.mapped[s], kWarps);
      mbar_init(&sc.entered[s], 1);
    }
    fence_mbar_init();
    sc.abort = 0;
  }
  __syncthreads();

  // Every wait is bounded; one that runs out ends the block's work with the status set.
  auto wait = [&](uint64_t* bar, int turn) {
    const bool ok = mbar_wait(bar, turn & 1, &sc.abort, p.wait_ns);
    if (!ok && p.status && lane == 0) atomicOr(p.status, kStatusTimeout);
    return __all_sync(~0u, ok) != 0;
  };
  // the same in a warp that fetches rows itself: its copies in flight end before it does
  auto wait_or_end = [&](uint64_t* bar, int turn) {
    const bool ok = wait(bar, turn);
    if (!TMA && !ok) asm volatile("cp.async.wait_all;" ::: "memory");
    return ok;
  };

  if (warp == kFeedWarp) {
    auto hand_out = [&](int turn) {
      int t = 0;
      if (lane == 0) t = p.counter ? int(atomicAdd(p.counter, 1u) + 1u) : int(blockIdx.x) + turn * int(gridDim.x);
      return t;
    };
    int k = 0;
    bool more = true;
    int upcoming = hand_out(0);
    for (int turn = 1, ends = 0; ends < 2; ++turn) {  // an end for each chain warp
      const int t = __shfl_sync(~0u, upcoming, 0);
      more = more && t < p.total;
      ends += !more;
      Place at{};
      int64_t len = 0, t0 = 0;
      if (more) {
        upcoming = hand_out(turn);  // its answer comes while this tile is fetched
        at = place_of<BACKWARD>(p, t);
        len = length_of(p, at.b);
        t0 = int64_t(at.i) * kTile;
        if (t0 >= len) {
          if (len == 0 && at.i == 0)  // an empty sequence hands its state through
            for (int v = 0; v < N; ++v) {
              const int c = (at.col * 32 + lane) * N + v;
              if (c >= p.D) continue;
              const int64_t e = int64_t(at.b) * p.D + c;
              const float* from = BACKWARD ? p.dh_last : p.h0;
              float* to = BACKWARD ? p.dh0 : p.h_last;
              if (to) to[e] = from ? from[e] : 0.f;
            }
          continue;
        }
      }
      const int s = k % kStages, q = k % kJobs;
      if (k >= kJobs && !wait(&sc.empty[q], k / kJobs - 1)) break;
      Job job{more ? t : -1, int(len), at.col, at.i, at.b, {0, 0}};
      if (more) {
        const int64_t c = at.col * 32 * N;
        if (BACKWARD) {
          job.out[0] = at.b * p.dxs[0] + t0 * p.dxs[1] + c;
          job.out[1] = at.b * p.dgs[0] + t0 * p.dgs[1] + c;
        } else {
          job.out[0] = at.b * p.hs[0] + t0 * p.hs[1] + c;
        }
      }
      if (lane == 0) sc.job[q] = job;
      __syncwarp();
      if (lane == 0) {
        if (TMA && more) {
          uint8_t* const to = stages + s * S::kStageBytes;
          const int c0 = at.col * 32 * N;
          mbar_arrive_expect_tx(&sc.full[q], S::kStageBytes);
          tma_load_3d(to, &mg, &sc.full[q], c0, int(t0), at.b);
          tma_load_3d(to + S::kBox, &mx, &sc.full[q], c0, int(t0), at.b);
          if (BACKWARD) tma_load_3d(to + 2 * S::kBox, &md, &sc.full[q], c0, int(t0), at.b);
        } else {
          mbar_arrive(&sc.full[q]);
        }
      }
      ++k;
    }
    // copies in flight end before the block does: where a wait runs out, nobody else waits for them
    int given_up = 0;
    for (int m = k > kJobs ? k - kJobs : 0; m < k; ++m) mbar_wait(&sc.full[m % kJobs], m / kJobs & 1, &given_up, p.wait_ns);
    return;
  }

  if (warp >= kChainWarp) {
    for (int k = warp - kChainWarp;; k += 2) {
      const int par = k & 1;
      if (!wait(&sc.full[k % kJobs], k / kJobs)) return;
      const Job job = sc.job[k % kJobs];
      const int t = job.t;
      if (t < 0) return;
      const Place at{job.b, job.col, job.i};
      const int64_t len = job.len;
      const int last = int((len - 1) / kTile);
      const int before = BACKWARD ? last - at.i : at.i;
      const bool wanted = BACKWARD ? at.i > 0 : at.i < last;  // another tile needs this one's state
      const int c = (at.col * 32 + lane) * N;
      const int64_t e = int64_t(at.b) * p.D + c;
      float A[N], H[N], st[N];
#pragma unroll
      for (int v = 0; v < N; ++v) {
        const float* from = BACKWARD ? p.dh_last : p.h0;
        st[v] = before == 0 && from && c + v < p.D ? from[e + v] : 0.f;
      }
      if (BACKWARD) {
        // the states h that enter the warps' rows, from the kept one that entered the tile
        float h[N];
#pragma unroll
        for (int v = 0; v < N; ++v)
          h[v] = c + v < p.D ? __ldg(p.saved + (int64_t(at.b) * p.kept + at.i * (kTile / kSave)) * p.D + c + v) : 0.f;
        if (!wait(&sc.mapped[par], k / 2)) return;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const V a = sc.A[par][w][lane], b = sc.H[par][w][lane];
          sc.H[par][w][lane] = V::of(h);
#pragma unroll
          for (int v = 0; v < N; ++v) h[v] = apply(a[v], b[v], h[v]);
        }
      } else if (!wait(&sc.mapped[par], k / 2)) {
        return;
      }
      // the tile's map: the warps' maps in the order of the chain
      const V(*const mapA)[32] = sc.A[par];
      V(*const mapH)[32] = BACKWARD ? sc.R[BACKWARD ? par : 0] : sc.H[par];
#pragma unroll
      for (int v = 0; v < N; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        const int w = BACKWARD ? kWarps - 1 - j : j;
        const V a = mapA[w][lane], b = mapH[w][lane];
#pragma unroll
        for (int v = 0; v < N; ++v) {
          H[v] = apply(a[v], b[v], H[v]);
          A[v] *= a[v];
        }
      }
      if (before > 0) {
        if (wanted) publish_map<N>(p, t, A, H);
        look_back<N>(p, t, before, step, st);
      }
      float out[N];
#pragma unroll
      for (int v = 0; v < N; ++v) out[v] = apply(A[v], H[v], st[v]);
      if (wanted) publish_state<N>(p, t, out);
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        const int w = BACKWARD ? kWarps - 1 - j : j;
        const V a = mapA[w][lane], b = mapH[w][lane];
        mapH[w][lane] = V::of(st);
#pragma unroll
        for (int v = 0; v < N; ++v) {
          if (!BACKWARD && w * kRows % kSave == 0 && p.saved && c + v < p.D &&
              int64_t(at.i) * kTile + w * kRows < len)
            p.saved[(int64_t(at.b) * p.kept + at.i * (kTile / kSave) + w * kRows / kSave) * p.D + c + v] = st[v];
          st[v] = apply(a[v], b[v], st[v]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc.entered[par]);
#pragma unroll
      for (int v = 0; v < N; ++v)
        if (c + v < p.D) {
          if (BACKWARD) {
            if (at.i == 0 && p.dh0) p.dh0[e + v] = out[v];
          } else if (at.i == last && p.h_last) {
            p.h_last[e + v] = out[v];
          }
        }
    }
  }

  // the sweeping warps: the maps of tile k + 1, then the states of tile k
  int swizzle[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) swizzle[r] = warp * kRows * kRowBytes + ((lane * 4) ^ (r << 4));
  // Without TMA a warp fetches its own rows, kStages - 1 tiles ahead (the places of the tile
  // that it has just done with); false if the wait for the tile ran out.
  int fetched = 0;
  bool more = true;
  auto fetch_own = [&] {
    if (more) {
      const int s = fetched % kStages;
      if (!wait_or_end(&sc.full[fetched % kJobs], fetched / kJobs)) return false;
      const Job job = sc.job[fetched % kJobs];
      more = job.t >= 0;
      if (more) {
        const int c0 = job.col * 32 * N, first = warp * kRows;
        const int64_t t0 = int64_t(job.i) * kTile + first;
        uint8_t* const to = stages + s * S::kStageBytes + first * kRowBytes;
        auto& extra = sc.extra[N == 2 ? s : 0];
        fetch<T, kRows>(p, p.g, p.gs, job.b, c0, t0, job.len, to, extra[0] + first);
        fetch<T, kRows>(p, p.x, p.xs, job.b, c0, t0, job.len, to + S::kBox, extra[1] + first);
        if constexpr (BACKWARD) fetch<T, kRows>(p, p.dh, p.dhs, job.b, c0, t0, job.len, to + 2 * S::kBox, extra[2] + first);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++fetched;
    return true;
  };
  if (!TMA)
    for (int s = 0; s < kStages - 2; ++s)
      if (!fetch_own()) return;
  // the lane's word of row r (of this warp's) of a tile's tensor
  struct Rows {
    const uint8_t* stage;
    const uint32_t* extra;   // rows on odd multiples of 2 bytes (kLoad2): see fetch
    unsigned late, alternate;  // by tensor: whether row 0 starts so, and whether rows take turns
  };
  auto rows_of = [&](int stage, const Job& job) {
    Rows rows{stages + stage * S::kStageBytes, nullptr, 0u, 0u};
    if (!TMA && N == 2 && p.load == kLoad2) {
      rows.extra = sc.extra[N == 2 ? stage : 0][0] + warp * kRows;
      const int t0 = job.i * kTile + warp * kRows;
      auto parity = [&](const void* base, const int64_t(&s)[2]) {
        return unsigned(reinterpret_cast<uintptr_t>(base) >> 1) + unsigned(job.b) * unsigned(s[0]) + unsigned(t0) * unsigned(s[1]);
      };
      rows.late = (parity(p.g, p.gs) & 1) | (parity(p.x, p.xs) & 1) << 1 | (BACKWARD ? (parity(p.dh, p.dhs) & 1) << 2 : 0);
      rows.alternate = unsigned(p.gs[1] & 1) | unsigned(p.xs[1] & 1) << 1 | (BACKWARD ? unsigned(p.dhs[1] & 1) << 2 : 0);
    }
    return rows;
  };
  auto word_of = [&](const Rows& rows, int tensor, int r) {
    const uint8_t* const row = rows.stage + tensor * S::kBox + r * kRowBytes;
    uint32_t w = *reinterpret_cast<const uint32_t*>(row + swizzle[r & 7]);
    if (!TMA && N == 2 && rows.extra) {
      if ((rows.late ^ (r & 1 ? rows.alternate : 0u)) >> tensor & 1) {
        const uint8_t* const next = row + warp * kRows * kRowBytes + (((lane + 1) * 4) ^ ((r & 7) << 4));
        const uint32_t v = lane == 31 ? rows.extra[tensor * kTile + r] : *reinterpret_cast<const uint32_t*>(next);
        w = __byte_perm(w, v, 0x5432);
      }
    }
    return W::open(w);
  };
  // this warp's and lane's place in the outputs' tiles
  const int64_t mine0 = BACKWARD ? (warp * kRows + kRows - 1) * p.dxs[1] + lane * N : warp * kRows * p.hs[1] + lane * N;
  const int64_t mine1 = BACKWARD ? (warp * kRows + kRows - 1) * p.dgs[1] + lane * N : 0;
  struct Turn {  // a tile's stage and place in the ring of jobs, and the ring's round
    int stage = 0, job = 0, round = 0;
    __device__ __forceinline__ void next() {
      stage = stage + 1 == kStages ? 0 : stage + 1;
      if (++job == kJobs) job = 0, ++round;
    }
  } ahead, here;
  Job cur{};
  cur.t = -1;
  for (int k = -1;; ++k) {
    Job next{};
    next.t = -1;
    if (k < 0 || cur.t >= 0) {
      const int par = (k + 1) & 1;
      if (!TMA && !fetch_own()) return;  // tile k + kStages - 1
      if (!wait_or_end(&sc.full[ahead.job], ahead.round)) return;
      if (!TMA) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");  // tile k + 1 is there
        __syncwarp();
      }
      next = sc.job[ahead.job];
      if (next.t >= 0) {
        const int left = next.len - (next.i * kTile + warp * kRows);
        const Rows rows = rows_of(ahead.stage, next);
        auto word = [&](int tensor, int r) { return word_of(rows, tensor, r); };
        V A = W::all(1.f), H = W::all(0.f), R = W::all(0.f);
        auto token = [&](int r) {
          const V g = word(0, r), x = word(1, r);
          V a, rest;
          gate<T, GATE>(g, a, rest);
          H = fma_(a, H, INPUT == TTT_SCAN_COMPLEMENT ? mul_(rest, x) : x);
          A = mul_(A, a);
          if (BACKWARD) R = fma_(A, word(2, r), R);
        };
        if (left >= kRows) {
#pragma unroll
          for (int r = 0; r < kRows; ++r) token(r);
        } else {  // rows behind the end hold anything
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (r < left) token(r);
        }
        sc.A[par][warp][lane] = A;
        sc.H[par][warp][lane] = H;
        if constexpr (BACKWARD) sc.R[par][warp][lane] = R;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc.mapped[par]);
      }
    }
    if (k >= 0) {
      if (cur.t < 0) return;
      const int par = k & 1;
      const int left = cur.len - (cur.i * kTile + warp * kRows);
      const int c = (cur.col * 32 + lane) * N;
      // every row and channel of this warp's part is there, and takes 4-byte stores
      const bool whole = left >= kRows && (cur.col + 1) * 32 * N <= p.D && (N == 1 || p.wide);
      const Rows rows = rows_of(here.stage, cur);
      auto word = [&](int tensor, int r) { return word_of(rows, tensor, r); };
      if (!wait_or_end(&sc.entered[par], k >> 1)) return;
      V st = sc.H[par][warp][lane];
      if constexpr (!BACKWARD) {
        T* to = static_cast<T*>(p.h) + cur.out[0] + mine0;
        auto token = [&](int r) {
          const V g = word(0, r), x = word(1, r);
          V a, rest;
          gate<T, GATE>(g, a, rest);
          st = fma_(a, st, INPUT == TTT_SCAN_COMPLEMENT ? mul_(rest, x) : x);
        };
        if (whole) {
#pragma unroll
          for (int r = 0; r < kRows; ++r, to += p.hs[1]) {
            token(r);
            *reinterpret_cast<uint32_t*>(to) = W::close(st);
          }
        } else {
#pragma unroll
          for (int r = 0; r < kRows; ++r, to += p.hs[1]) {
            token(r);
            if (r < left) put_row<T>(p, to, c, st);
          }
        }
      } else {
        // h_{t-1} (less x_t) of the rows first to last, then the gradients last to first
        V a[kRows], rest[kRows], d[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const V g = word(0, r), x = word(1, r);
          gate<T, GATE>(g, a[r], rest[r]);
          d[r] = INPUT == TTT_SCAN_COMPLEMENT ? sub_(st, x) : st;
          st = fma_(a[r], st, INPUT == TTT_SCAN_COMPLEMENT ? mul_(rest[r], x) : x);
        }
        V mu = sc.R[par][warp][lane];
        T* dx = static_cast<T*>(p.dx) + cur.out[0] + mine0;  // the last row
        T* dg = static_cast<T*>(p.dg) + cur.out[1] + mine1;
        if (whole) {
#pragma unroll
          for (int r = kRows - 1; r >= 0; --r, dx -= p.dxs[1], dg -= p.dgs[1]) {
            const V lam = add_(word(2, r), mu);
            mu = mul_(a[r], lam);
            *reinterpret_cast<uint32_t*>(dx) = W::close(INPUT == TTT_SCAN_COMPLEMENT ? mul_(rest[r], lam) : lam);
            *reinterpret_cast<uint32_t*>(dg) = W::close(gate_grad<GATE>(a[r], rest[r], mul_(lam, d[r])));
          }
        } else {
#pragma unroll
          for (int r = kRows - 1; r >= 0; --r, dx -= p.dxs[1], dg -= p.dgs[1])
            if (r < left) {
              const V lam = add_(word(2, r), mu);
              mu = mul_(a[r], lam);
              put_row<T>(p, dx, c, INPUT == TTT_SCAN_COMPLEMENT ? mul_(rest[r], lam) : lam);
              put_row<T>(p, dg, c, gate_grad<GATE>(a[r], rest[r], mul_(lam, d[r])));
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc.empty[here.job]);
    }
    here = ahead;
    ahead.next();
    cur = next;
  }
}

// Sequences of at most kShort tokens (new tokens of a stream): one thread per word of
// channels, no shared memory and nothing to wait for.
template <class T, int GATE, int INPUT, bool BACKWARD>
__global__ void __launch_bounds__(128) scan_short_kernel(const __grid_constant__ ScanArgs p) {
  using W = Word<T>;
  using V = typename W::V;
  constexpr int N = W::N;
  const int words = (p.D + N - 1) / N;
  const int64_t k = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (k >= int64_t(p.B) * words) return;
  const int b = int(k / words), c = int(k % words) * N;
  const int64_t e = int64_t(b) * p.D + c;
  const int n = int(length_of(p, b));
  auto load = [&](const void* base, const int64_t(&s)[2], int t) {
    const T* from = static_cast<const T*>(base) + b * s[0] + t * s[1] + c;
    if (p.load != kLoad2) return W::open(*reinterpret_cast<const uint32_t*>(from));
    const uint16_t* h = reinterpret_cast<const uint16_t*>(from);
    return W::open(N == 2 && c + 1 < p.D ? h[0] | uint32_t(h[1]) << 16 : h[0]);
  };
  auto state = [&](const float* from) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = from && c + i < p.D ? from[e + i] : 0.f;
    return W::make(v);
  };
  auto keep = [&](float* to, V v) {
    if (to)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < p.D) to[e + i] = v[i];
  };
  V st = state(BACKWARD ? p.saved : p.h0);
  if (!BACKWARD && p.L) keep(p.saved, st);
  V a[kShort], rest[kShort], d[kShort];
#pragma unroll
  for (int r = 0; r < kShort; ++r) {
    if (r >= n) break;
    const V g = load(p.g, p.gs, r), x = load(p.x, p.xs, r);
    gate<T, GATE>(g, a[r], rest[r]);
    d[r] = INPUT == TTT_SCAN_COMPLEMENT ? sub_(st, x) : st;
    st = fma_(a[r], st, INPUT == TTT_SCAN_COMPLEMENT ? mul_(rest[r], x) : x);
    if constexpr (!BACKWARD) put_word<T>(p, static_cast<T*>(p.h) + b * p.hs[0] + r * p.hs[1] + c, c, st);
  }
  if constexpr (!BACKWARD) {
    keep(p.h_last, st);
  } else {
    V mu = state(p.dh_last);
#pragma unroll
    for (int r = kShort - 1; r >= 0; --r) {
      if (r >= n) continue;
      const V lam = add_(load(p.dh, p.dhs, r), mu);
      mu = mul_(a[r], lam);
      put_word<T>(p, static_cast<T*>(p.dx) + b * p.dxs[0] + r * p.dxs[1] + c, c,
                  INPUT == TTT_SCAN_COMPLEMENT ? mul_(rest[r], lam) : lam);
      put_word<T>(p, static_cast<T*>(p.dg) + b * p.dgs[0] + r * p.dgs[1] + c, c,
                  gate_grad<GATE>(a[r], rest[r], mul_(lam, d[r])));
    }
    keep(p.dh0, mu);
  }
}

// Zeroes the rows behind the sequences' ends: a warp a row, the rows of a block one after the other
template <class T>
__global__ void __launch_bounds__(256) scan_clear_kernel(const int* lengths, T* y, int64_t sb, int64_t st, int64_t L, int B, int D) {
  const int per = gridDim.x / B, lane = threadIdx.x % 32;  // blocks of a sequence; fewer than one: sequences of a block
  // 64 bits: the last step of up to 2^31 - 1 sequences goes beyond them
  for (int64_t b = per ? blockIdx.x / per : blockIdx.x; b < B; b += per ? B : gridDim.x) {
    const int first = per ? blockIdx.x % per : 0, hop = per ? per : 1;
    if (first >= hop) break;
    for (int64_t t = max(lengths[b], 0) + int64_t(first) * 8 + threadIdx.x / 32; t < L; t += int64_t(hop) * 8)
      for (int c = lane; c < D; c += 32) y[b * sb + t * st + c] = T(0.f);
  }
}

// Bytes of a call's workspace: the counter, then every tile's map and state.
struct Space {
  size_t maps, states, total;
};
Space space_of(int64_t tiles, int per_word) {
  Space s;
  s.maps = 16;
  s.states = s.maps + size_t(tiles) * 32 * per_word * 8;
  s.total = s.states + size_t(tiles) * 32 * per_word * 4;
  return s;
}

// `stuck`: the first tile is never handed out, so that all that waits for its state waits in vain
template <class T, int GATE, int INPUT, bool BACKWARD>
int launch(ScanArgs& a, const int64_t (*strides)[2], bool stuck, cudaStream_t st) {
  using S = Shape<T, BACKWARD>;
  if (a.L <= kShort) {
    const int64_t n = int64_t(a.B) * ((a.D + S::N - 1) / S::N), grid = (n + 127) / 128;
    if (grid > 0x7fffffff) return TTT_ERR_UNSUPPORTED;
    scan_short_kernel<T, GATE, INPUT, BACKWARD><<<unsigned(grid), 128, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
  }
  CUtensorMap m[3] = {};
  if (a.load == kLoadTma) {
    const void* base[3] = {a.g, a.x, a.dh};
    for (int k = 0; k < S::kTensors; ++k)
      if (!make_tmap(&m[k], base[k], int(sizeof(T)), a.D, a.L, a.B, strides[k][1], a.B > 1 ? strides[k][0] : 16, S::kTile))
        a.load = kLoad4;  // rows that TMA takes are on 4 bytes too
  }
  const bool tma = a.load == kLoadTma;
  const auto kernel = tma ? scan_tile_kernel<T, GATE, INPUT, BACKWARD, true> : scan_tile_kernel<T, GATE, INPUT, BACKWARD, false>;
  static OncePerDevice once[2];
  const int dev = current_device();
  if (once[tma].run(dev, [&] {
        return int(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem));
      }) != 0)
    return TTT_ERR_CUDA;
  const int grid = std::min(sm_count(), a.total);
  // all ones: nothing published, and a counter whose first answer is -1
  if (a.counter && cudaMemsetAsync(a.counter, 0xff, space_of(a.total, S::N).total, st) != cudaSuccess)
    return TTT_ERR_CUDA;
  if (stuck && cudaMemsetAsync(a.counter, 0, sizeof(unsigned), st) != cudaSuccess) return TTT_ERR_CUDA;
  kernel<<<grid, kThreads, S::kSmem, st>>>(a, m[0], m[1], m[2]);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

using Launch = int (*)(ScanArgs&, const int64_t (*)[2], bool, cudaStream_t);
template <class T, bool BACKWARD>
Launch pick(int gate, int input) {
  constexpr int P = TTT_SCAN_PLAIN, C = TTT_SCAN_COMPLEMENT;
  const bool plain = input == TTT_SCAN_PLAIN;
  if (gate == TTT_GATE_VALUE) return plain ? launch<T, TTT_GATE_VALUE, P, BACKWARD> : launch<T, TTT_GATE_VALUE, C, BACKWARD>;
  if (gate == TTT_GATE_SIGMOID)
    return plain ? launch<T, TTT_GATE_SIGMOID, P, BACKWARD> : launch<T, TTT_GATE_SIGMOID, C, BACKWARD>;
  return plain ? launch<T, TTT_GATE_EXP, P, BACKWARD> : launch<T, TTT_GATE_EXP, C, BACKWARD>;
}

}  // namespace
}  // namespace ttt

using namespace ttt;

struct ttt_scan {
  ttt_scan_config cfg;
};

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;

int words_of(const ttt_scan* h) { return h->cfg.dtype == TTT_BF16 ? 2 : 1; }
int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }
int tile_tokens(bool backward) {
  return backward ? Shape<float, true>::kTile : Shape<float, false>::kTile;
}
// tiles of a call, or -1 for more than the counter takes
int64_t tiles_of(const ttt_scan* h, int32_t B, int64_t L, bool backward) {
  const __int128 n = __int128(B) * up(h->cfg.D, 32 * words_of(h)) * std::max<int64_t>(up(L, tile_tokens(backward)), 1);
  return n > (int64_t(1) << 30) ? -1 : int64_t(n);
}
// bytes of one direction's workspace: none for sequences of one tile
size_t space_needed(const ttt_scan* h, int32_t B, int64_t L, bool backward) {
  if (L <= tile_tokens(backward) || L <= kShort) return 0;
  const int64_t n = tiles_of(h, B, L, backward);
  return n < 0 ? 0 : space_of(n, words_of(h)).total;
}

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
  if (!scan_sizes_ok(h, B, L) || L > kMaxTokens) return 0;
  return std::max(space_needed(h, B, L, false), space_needed(h, B, L, true));
}

extern "C" size_t ttt_scan_saved_size(const ttt_scan* h, int32_t B, int64_t L) {
  if (!scan_sizes_ok(h, B, L) || L > kMaxTokens) return 0;
  return size_t(B) * size_t(up(L, kSave)) * size_t(h->cfg.D) * 4;
}

namespace {

// the parts of the arguments that both directions share; a status
int prepare(const ttt_scan* h, bool backward, int32_t B, int64_t L, const RowTensor* in, int nin, const RowTensor* out, int nout,
            void* workspace, size_t workspace_bytes, unsigned* status, ScanArgs* a) {
  const bool bf16 = h->cfg.dtype == TTT_BF16;
  const int64_t tiles = tiles_of(h, B, L, backward);
  if (L > kShort && tiles < 0) return TTT_ERR_UNSUPPORTED;
  const size_t need = ttt_scan_workspace_size(h, B, L);
  if (need && (!workspace || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  a->L = L, a->B = B, a->D = h->cfg.D;
  a->wait_ns = kWaitLimitNs;
  a->status = status;
  a->per_col = int32_t(up(L, tile_tokens(backward)));
  a->kept = int32_t(up(L, kSave));
  a->cols = int32_t(up(a->D, 32 * words_of(h)));
  a->total = int32_t(tiles);
  if (space_needed(h, B, L, backward)) {
    const Space s = space_of(tiles, words_of(h));
    char* w = static_cast<char*>(workspace);
    a->counter = reinterpret_cast<unsigned*>(w);
    a->maps = reinterpret_cast<uint64_t*>(w + s.maps);
    a->states = reinterpret_cast<uint32_t*>(w + s.states);
  }
  // TMA takes rows on 16 bytes whose dimensions have a stride; 4-byte words take rows on
  // 4 bytes and whole words (bf16: an even number of channels)
  const bool whole = !bf16 || a->D % 2 == 0;
  a->load = whole ? kLoadTma : kLoad2;
  for (int i = 0; i < nin; ++i) {
    if (!rows_aligned(in[i], 16) || in[i].stride[1] == 0 || (B > 1 && in[i].stride[0] == 0))
      a->load = a->load == kLoadTma ? kLoad4 : a->load;
    if (!rows_aligned(in[i], 4)) a->load = kLoad2;
  }
  a->wide = whole;
  for (int i = 0; i < nout; ++i)
    if (!rows_aligned(out[i], 4)) a->wide = 0;
  return TTT_OK;
}

}  // namespace

namespace {

// ttt_scan_forward; with `stuck_ns`, its first tile is left out and waits are that long at most
int forward(const ttt_scan* h, int32_t B, int64_t L, const void* g, const ttt_strides* gs, const void* x, const ttt_strides* xs,
            const float* h0, const int32_t* lengths, void* ho, const ttt_strides* hs, float* h_last, void* saved,
            void* workspace, size_t workspace_bytes, unsigned* status, unsigned long long stuck_ns, void* stream) {
  if (!scan_sizes_ok(h, B, L) || !gs || !xs || !hs) return TTT_ERR_INVALID_ARG;
  if (L > kMaxTokens) return TTT_ERR_UNSUPPORTED;
  if (!is_aligned(saved, 16) || !is_aligned(workspace, 16) || !is_aligned(status, 4)) return TTT_ERR_INVALID_ARG;
  const RowTensor in[] = {rows(h, B, L, g, gs), rows(h, B, L, x, xs), bytes(lengths, size_t(B) * 4)};
  const RowTensor out[] = {rows(h, B, L, ho, hs), state(h, B, h_last), bytes(saved, ttt_scan_saved_size(h, B, L))};
  if (!is_aligned(lengths, 4) || !apart(in, 3, out, 3)) return TTT_ERR_INVALID_ARG;
  const RowTensor H0 = state(h, B, h0);
  if (!H0.readable() || may_share(H0, out[0]) || may_share(H0, out[2])) return TTT_ERR_INVALID_ARG;
  if (h0 != h_last && may_share(H0, out[1])) return TTT_ERR_INVALID_ARG;
  ScanArgs a{};
  const int r = prepare(h, false, B, L, in, 2, out, 1, workspace, workspace_bytes, status, &a);
  if (r != TTT_OK) return r;
  a.g = g, a.x = x, a.h0 = h0, a.lengths = lengths, a.h = ho, a.h_last = h_last;
  a.saved = static_cast<float*>(saved);
  put_strides(a.gs, gs), put_strides(a.xs, xs), put_strides(a.hs, hs);
  if (stuck_ns) {
    if (!a.counter) return TTT_ERR_UNSUPPORTED;  // sequences of one tile wait for nothing
    a.wait_ns = stuck_ns;
  }
  const int64_t strides[2][2] = {{gs->batch, gs->token}, {xs->batch, xs->token}};
  const Launch f = h->cfg.dtype == TTT_BF16 ? pick<__nv_bfloat16, false>(h->cfg.gate, h->cfg.input)
                                            : pick<float, false>(h->cfg.gate, h->cfg.input);
  return f(a, strides, stuck_ns != 0, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" int ttt_scan_forward(const ttt_scan* h, int32_t B, int64_t L, const void* g, const ttt_strides* gs,
                                const void* x, const ttt_strides* xs, const float* h0, const int32_t* lengths, void* ho,
                                const ttt_strides* hs, float* h_last, void* saved, void* workspace,
                                size_t workspace_bytes, unsigned* status, void* stream) {
  return forward(h, B, L, g, gs, x, xs, h0, lengths, ho, hs, h_last, saved, workspace, workspace_bytes, status, 0, stream);
}

extern "C" int ttt_selftest_scan_timeout(const ttt_scan* h, int32_t B, int64_t L, const void* g, const ttt_strides* gs,
                                         const void* x, const ttt_strides* xs, void* ho, const ttt_strides* hs,
                                         void* workspace, size_t workspace_bytes, unsigned* status, int32_t wait_ms,
                                         void* stream) {
  if (!status || wait_ms < 1 || wait_ms > 2000) return TTT_ERR_INVALID_ARG;
  return forward(h, B, L, g, gs, x, xs, nullptr, nullptr, ho, hs, nullptr, nullptr, workspace, workspace_bytes, status,
                 wait_ms * 1000000ull, stream);
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
  ScanArgs a{};
  const RowTensor tiles[] = {in[1], in[2], in[0]};
  const int r = prepare(h, true, B, L, tiles, 3, out, 2, workspace, workspace_bytes, status, &a);
  if (r != TTT_OK) return r;
  a.dh = dh, a.g = g, a.x = x, a.dh_last = dh_last, a.lengths = lengths, a.dg = dg, a.dx = dx, a.dh0 = dh0;
  a.saved = nsaved ? static_cast<float*>(const_cast<void*>(saved)) : nullptr;  // no tokens: none kept, whatever is given
  put_strides(a.dhs, dhs), put_strides(a.gs, gs), put_strides(a.xs, xs), put_strides(a.dgs, dgs),
      put_strides(a.dxs, dxs);
  const int64_t strides[3][2] = {{gs->batch, gs->token}, {xs->batch, xs->token}, {dhs->batch, dhs->token}};
  const Launch f = h->cfg.dtype == TTT_BF16 ? pick<__nv_bfloat16, true>(h->cfg.gate, h->cfg.input)
                                            : pick<float, true>(h->cfg.gate, h->cfg.input);
  return f(a, strides, false, static_cast<cudaStream_t>(stream));
}

extern "C" int ttt_scan_clear(const ttt_scan* h, int32_t B, int64_t L, const int32_t* lengths, void* y,
                              const ttt_strides* ys, void* stream) {
  if (!scan_sizes_ok(h, B, L) || !ys || !lengths || !is_aligned(lengths, 4)) return TTT_ERR_INVALID_ARG;
  if (L > kMaxTokens) return TTT_ERR_UNSUPPORTED;
  const RowTensor in[] = {bytes(lengths, size_t(B) * 4)}, out[] = {rows(h, B, L, y, ys)};
  if (!apart(in, 1, out, 1)) return TTT_ERR_INVALID_ARG;
  if (L == 0) return TTT_OK;
  constexpr int64_t kBlocks = 8 * 148;
  const unsigned grid = unsigned(B >= kBlocks ? kBlocks : B * std::min(up(L, 8), std::max<int64_t>(1, kBlocks / B)));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (h->cfg.dtype == TTT_BF16)
    scan_clear_kernel<<<grid, 256, 0, st>>>(lengths, static_cast<__nv_bfloat16*>(y), ys->batch, ys->token, L, B, h->cfg.D);
  else
    scan_clear_kernel<<<grid, 256, 0, st>>>(lengths, static_cast<float*>(y), ys->batch, ys->token, L, B, h->cfg.D);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}
