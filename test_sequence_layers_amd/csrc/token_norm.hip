// Norm of the d features of every token with gate, scale and residual, forward and backward:
//
//   y = res + scale act(gate) n,  n = xh weight + bias,  xh = (x - m) r,
//   layer: m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps);
//   rms:   m = 0, r = 1 / sqrt(mean(x^2) + eps);   l2: m = 0, r = 1 / sqrt(sum(x^2) + eps).
//
// Backward, with A = act(gate) (1 without a gate), s = scale (1 without):
//   dgate = dy s n act'(gate),  dscale = sum dy A n,  t = dy s A,  dbias = sum t,
//   dweight = sum t xh,  u = t weight,  dx = r (u - mean(u) - xh mean(u xh))
// (rms: without mean(u); l2: the sum of u xh in place of its mean), sums over the batch and
// the tokens.
//
// Both are bound by HBM: each tensor passes once (8 x 12 x 2048 rows of 64 bf16 with gate and
// residual: forward 19 us, 5.3 TB/s; backward 28 us, 4.4 TB/s, where the vector units are 80 %
// busy).  Without gate and scale the backward pass is a kernel of its own (kPlain), which needs
// 40 % fewer registers: 8191 rows of 768 bf16 take 17.3 us and not 22, 8192 of 2048 29.6 and not 44.
// A row lives in the registers of LPR lanes (part of a wave, a wave, or a workgroup), NV vectors of
// W elements a lane, so its statistics need no second read; everything between load and store is
// float32.
//
// A vector is 16 bytes.  Where rows or tensors are not aligned to that (`A` false) its loads and
// stores are not either, and the last vector of a row begins early, at d - W: its first `dup`
// elements belong to the lane before and count as absent.  (One element a load took 82 us on 2604
// rows of 4751 bf16 with gate and residual, this takes 35.)
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "gated_linear.hpp"

namespace ttt {
namespace {

enum { kLayer = 0, kRms = 1, kL2 = 2 };
enum { kActNone = 0, kSilu = 1, kGelu = 2, kSigmoid = 3 };

// W consecutive elements as they are loaded
template <typename IO, int W, bool A>
struct Vec {
  typedef IO type __attribute__((ext_vector_type(W)));
  type v;
  __device__ __forceinline__ void load(const IO* p) {
    if constexpr (W == 1) v[0] = p[0];
    else if constexpr (A) v = *reinterpret_cast<const type*>(p);
    else __builtin_memcpy(&v, p, sizeof(v));
  }
  __device__ __forceinline__ void widen(float* x, bool have, int dup) const {
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = have && (A || i >= dup) ? to_f32(static_cast<IO>(v[i])) : 0.0f;
  }
};
template <typename IO, int W, bool A>
__device__ __forceinline__ void store_vec(IO* p, const float* x, int dup) {
  if constexpr (W == 1) {
    p[0] = from_f32<IO>(x[0]);
  } else {
    typename Vec<IO, W, A>::type y;
#pragma unroll
    for (int i = 0; i < W; ++i) y[i] = from_f32<IO>(x[i]);
    if constexpr (A) {
      *reinterpret_cast<typename Vec<IO, W, A>::type*>(p) = y;
    } else if (dup == 0) {
      __builtin_memcpy(p, &y, sizeof(y));
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i >= dup) p[i] = y[i];
    }
  }
}
// where a lane's vector v begins in its row
template <int W, int LPR, bool A>
struct Place {
  int col, dup;
  bool have;
  __device__ __forceinline__ Place(int v, int in_row, int d) {
    const int at = (v * LPR + in_row) * W;
    have = at < d;
    col = !have ? 0 : A ? at : min(at, d - W);
    dup = have ? at - col : 0;
  }
};
template <int W, int LPR, int NV, bool A>
struct Places {
  Place<W, LPR, A> p[NV];
  __device__ __forceinline__ Places(int in_row, int d) : Places(in_row, d, std::make_integer_sequence<int, NV>()) {}
  template <int... V>
  __device__ __forceinline__ Places(int in_row, int d, std::integer_sequence<int, V...>)
      : p{Place<W, LPR, A>(V, in_row, d)...} {}
};
// float32 parameters of the same W columns (16 bytes at a time when W > 1)
template <int W, bool A>
__device__ __forceinline__ void load_par(const float* p, float* x) {
  if constexpr (W == 1) {
    x[0] = p[0];
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      gl_f4 y;
      if constexpr (A) y = *reinterpret_cast<const gl_f4*>(p + i);
      else __builtin_memcpy(&y, p + i, sizeof(y));
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i + j] = y[j];
    }
  }
}

__device__ __forceinline__ float act_(int act, float g) {
  return act == kSilu ? silu_(g) : act == kGelu ? gelu_(g) : act == kSigmoid ? sigmoidf_(g) : g;
}
__device__ __forceinline__ void act_grad(int act, float g, float* a, float* da) {
  if (act == kSilu || act == kSigmoid) {
    const float s = sigmoidf_(g);
    *a = act == kSilu ? g * s : s;
    *da = act == kSilu ? s * (1.0f + g * (1.0f - s)) : s * (1.0f - s);
  } else {
    *a = act == kGelu ? gelu_(g) : g;
    *da = act == kGelu ? dgelu_(g) : 1.0f;
  }
}

// Sum over the lanes of a row; for rows of a whole workgroup through LDS (`red`, one slot per
// wave, used alternately so that one barrier a sum is enough).
template <int LPR>
__device__ __forceinline__ float row_sum(float x, float (*red)[16], int* turn) {
  x = gl_lane_sum<(LPR < 64 ? LPR : 64)>(x);
  if constexpr (LPR > 64) {
    float* slot = red[*turn & 1];
    ++*turn;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < LPR / 64; ++i) x += slot[i];
  }
  return x;
}

// The row in registers: x becomes xh; returns r.
template <int W, int LPR, int NV, bool A>
__device__ __forceinline__ float normalise(float* x, const bool* live, const Place<W, LPR, A>* at, int kind,
                                           int d, float eps, float (*red)[16], int* turn) {
  constexpr int N = NV * W;
  const float inv = kind == kL2 ? 1.0f : 1.0f / d;
  if (kind == kLayer) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += x[i];
    const float m = row_sum<LPR>(sum, red, turn) * inv;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = live[i / W] && (A || i % W >= at[i / W].dup) ? x[i] - m : 0.0f;
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) ss += x[i] * x[i];
  const float r = 1.0f / sqrtf(row_sum<LPR>(ss, red, turn) * inv + eps);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] *= r;
  return r;
}

template <int LPR> struct Block {
  static constexpr int kThreads = LPR > 64 ? LPR : 256;
  static constexpr int kRows = kThreads / LPR;  // rows a workgroup holds at once
};

// A workgroup takes `passes` x kRows consecutive rows.
template <typename IO, int W, int LPR, int NV, bool A>
__global__ __launch_bounds__(Block<LPR>::kThreads) void norm_fwd_kernel(NormArgs a, int rows, int passes) {
  __shared__ float red[2][16];
  int turn = 0;
  constexpr int RB = Block<LPR>::kRows;
  const int in_row = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const IO* xp = static_cast<const IO*>(a.x);
  const IO* gp = static_cast<const IO*>(a.gate);
  const IO* rp = static_cast<const IO*>(a.res);
  IO* yp = static_cast<IO*>(a.y);
  const Places<W, LPR, NV, A> places(in_row, a.d);
  const Place<W, LPR, A>* at = places.p;
  for (int p = 0; p < passes; ++p) {
    const long long first = (static_cast<long long>(blockIdx.x) * passes + p) * RB;
    if (first >= rows) return;  // the same for every thread
    const int row = static_cast<int>(first) + group;
    const bool live = row < rows;
    const size_t base = static_cast<size_t>(live ? row : 0) * a.d;
    const size_t hb = static_cast<size_t>((live ? row : 0) / a.T % a.H) * a.d;
    float x[NV * W], gt[NV * W], rs[NV * W];
    bool have[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = at[v].col;
      have[v] = live && at[v].have;
      Vec<IO, W, A> lx, lg, lr;
      lx.load(xp + base + col);
      if (gp) lg.load(gp + base + col);
      if (rp) lr.load(rp + base + col);
      lx.widen(x + v * W, have[v], at[v].dup);
#pragma unroll
      for (int i = 0; i < W; ++i) gt[v * W + i] = rs[v * W + i] = 0.0f;
      if (gp) lg.widen(gt + v * W, true, 0);
      if (rp) lr.widen(rs + v * W, true, 0);
    }
    normalise<W, LPR, NV, A>(x, have, at, a.kind, a.d, a.eps, red, &turn);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!have[v]) continue;
      const int col = at[v].col;
      float par[W], y[W];
#pragma unroll
      for (int i = 0; i < W; ++i) y[i] = x[v * W + i];
      if (a.weight) {
        load_par<W, A>(a.weight + hb + col, par);
#pragma unroll
        for (int i = 0; i < W; ++i) y[i] *= par[i];
      }
      if (a.bias) {
        load_par<W, A>(a.bias + hb + col, par);
#pragma unroll
        for (int i = 0; i < W; ++i) y[i] += par[i];
      }
      if (gp) {
#pragma unroll
        for (int i = 0; i < W; ++i) y[i] *= act_(a.act, gt[v * W + i]);
      }
      if (a.scale) {
        load_par<W, A>(a.scale + hb + col, par);
#pragma unroll
        for (int i = 0; i < W; ++i) y[i] *= par[i];
      }
#pragma unroll
      for (int i = 0; i < W; ++i) y[i] += rs[v * W + i];
      store_vec<IO, W, A>(yp + base + col, y, at[v].dup);
    }
  }
}

// Workgroup (part, head) takes a share of the head's B T rows, and leaves its sums of the
// parameters' gradients in part[head][part][wanted sums][d].
template <typename IO, int W, int LPR, int NV, bool A, bool kPlain>
__global__ __launch_bounds__(Block<LPR>::kThreads) void norm_bwd_kernel(NormArgs a, float* part, int share) {
  if constexpr (kPlain) {
    a.gate = a.dgate = nullptr;
    a.scale = a.dscale = nullptr;
  }
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [2][wanted sums][d] (rows of a wave or less)
  __shared__ float red[2][16];
  int turn = 0;
  constexpr int RB = Block<LPR>::kRows, N = NV * W;
  const int in_row = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int head = blockIdx.y;
  const long long all = static_cast<long long>(a.B) * a.T;  // at most 2^30
  const int from = static_cast<int>(blockIdx.x) * share;  // below all
  const int to = static_cast<int>(all - from < share ? all : from + share);
  const IO* xp = static_cast<const IO*>(a.x);
  const IO* gp = static_cast<const IO*>(a.gate);
  const IO* dyp = static_cast<const IO*>(a.dy);
  IO* dxp = static_cast<IO*>(a.dx);
  IO* dgp = static_cast<IO*>(a.dgate);
  const size_t hb = static_cast<size_t>(head) * a.d;
  float sw[N], sb[N], ss[N];
#pragma unroll
  for (int i = 0; i < N; ++i) sw[i] = sb[i] = ss[i] = 0.0f;
  const Places<W, LPR, NV, A> places(in_row, a.d);
  const Place<W, LPR, A>* at = places.p;
  // a row as it is loaded; that of the next turn is on its way while one is worked on
  struct Row {
    Vec<IO, W, A> x[NV], dy[NV], gt[NV];
    size_t base;
    bool live;
  } next;
  auto fetch = [&](int first) {
    next.live = first + group < to;
    const unsigned bt = next.live ? first + group : 0;  // a valid row in any case
    const unsigned b = bt / static_cast<unsigned>(a.T), t = bt - b * static_cast<unsigned>(a.T);
    next.base = (static_cast<size_t>(b * static_cast<unsigned>(a.H) + head) * a.T + t) * a.d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = at[v].col;
      next.x[v].load(xp + next.base + col);
      next.dy[v].load(dyp + next.base + col);
      if (gp) next.gt[v].load(gp + next.base + col);
    }
  };
  constexpr bool kNext = LPR < 1024;  // 1024 threads leave a lane 128 registers: no room for a second row
  if (kNext && from < to) fetch(from);
  // the head's parameters, kept in registers while they are few
  constexpr bool kKeep = N <= 24 && kNext;
  float wt_[kKeep ? N : W], bs_[kKeep ? N : W], sc_[kKeep ? N : W];
  auto parameters = [&](int col, float* wt, float* bs, float* sc) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      wt[i] = sc[i] = 1.0f;
      bs[i] = 0.0f;
    }
    if (a.weight) load_par<W, A>(a.weight + hb + col, wt);
    if (a.bias) load_par<W, A>(a.bias + hb + col, bs);
    if (a.scale) load_par<W, A>(a.scale + hb + col, sc);
  };
  if constexpr (kKeep) {
#pragma unroll
    for (int v = 0; v < NV; ++v) parameters(at[v].col, wt_ + v * W, bs_ + v * W, sc_ + v * W);
  }
  for (int first = from; first < to; first += RB) {
    if (!kNext) fetch(first);
    const size_t base = next.base;
    float x[N], dy[N];
    Vec<IO, W, A> gv[NV];
    bool have[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      have[v] = next.live && at[v].have;
      next.x[v].widen(x + v * W, have[v], at[v].dup);
      next.dy[v].widen(dy + v * W, have[v], at[v].dup);
      if (gp) gv[v] = next.gt[v];
    }
    if (kNext && first + RB < to) fetch(first + RB);
    const float r = normalise<W, LPR, NV, A>(x, have, at, a.kind, a.d, a.eps, red, &turn);
    float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!have[v]) continue;
      const int col = at[v].col;
      float* wt = wt_ + (kKeep ? v * W : 0);
      float* bs = bs_ + (kKeep ? v * W : 0);
      float* sc = sc_ + (kKeep ? v * W : 0);
      float dg[W], gt[W];
      if (gp) gv[v].widen(gt, true, at[v].dup);
      if constexpr (!kKeep) parameters(col, wt, bs, sc);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int j = v * W + i;
        const float n = x[j] * wt[i] + bs[i];
        float act = 1.0f, dact = 0.0f;
        if (gp) act_grad(a.act, gt[i], &act, &dact);
        ss[j] += dy[j] * act * n;
        const float t0 = dy[j] * sc[i], t = t0 * act;
        dg[i] = t0 * n * dact;
        sb[j] += t;
        sw[j] += t * x[j];
        dy[j] = t * wt[i];
        m1 += dy[j];
        m2 += dy[j] * x[j];
      }
      if (dgp) store_vec<IO, W, A>(dgp + base + col, dg, at[v].dup);
    }
    const float inv = 1.0f / a.d;
    m2 = row_sum<LPR>(m2, red, &turn) * (a.kind == kL2 ? 1.0f : inv);
    m1 = a.kind == kLayer ? row_sum<LPR>(m1, red, &turn) * inv : 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!have[v]) continue;
      float dx[W];
#pragma unroll
      for (int i = 0; i < W; ++i) dx[i] = r * (dy[v * W + i] - m1 - x[v * W + i] * m2);
      store_vec<IO, W, A>(dxp + base + at[v].col, dx, at[v].dup);
    }
  }
  if (!part) return;
  // over the lanes that hold the same columns, then over the waves in a tree through LDS
  if constexpr (LPR < 64) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      sw[i] = gl_stride_sum<LPR>(sw[i]);
      sb[i] = gl_stride_sum<LPR>(sb[i]);
      ss[i] = gl_stride_sum<LPR>(ss[i]);
    }
  }
  // [wanted sums][d], those of weight, bias and scale in order
  const int nw = a.dweight ? 1 : 0, nb = a.dbias ? 1 : 0, ns = a.dscale ? 1 : 0, all_sums = (nw + nb + ns) * a.d;
  constexpr int P = W < 4 || !A ? 1 : 4;  // floats at a time
  typedef float piece __attribute__((ext_vector_type(P)));
  auto pieces = [&](int first, float* x, int dup, auto f) {
#pragma unroll
    for (int i = 0; i < W; i += P) {
      if (!A && i < dup) continue;
      piece y;
#pragma unroll
      for (int j = 0; j < P; ++j) y[j] = x[i + j];
      f(first + i, y);
#pragma unroll
      for (int j = 0; j < P; ++j) x[i + j] = y[j];
    }
  };
  auto columns = [&](auto f) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!at[v].have) continue;
      const int col = at[v].col, dup = at[v].dup;
      if (nw) pieces(col, sw + v * W, dup, f);
      if (nb) pieces(nw * a.d + col, sb + v * W, dup, f);
      if (ns) pieces((nw + nb) * a.d + col, ss + v * W, dup, f);
    }
  };
  const int wave = threadIdx.x >> 6;
  const bool mine = LPR >= 64 || static_cast<int>(threadIdx.x & 63) < LPR;
  if constexpr (LPR <= 64) {
#pragma unroll
    for (int half = Block<LPR>::kThreads / 128; half > 0; half >>= 1) {
      float* slot = sums + (wave % half) * all_sums;
      if (mine && wave >= half && wave < 2 * half)
        columns([&](int i, piece& x) { *reinterpret_cast<piece*>(slot + i) = x; });
      __syncthreads();
      if (mine && wave < half) columns([&](int i, piece& x) { x += *reinterpret_cast<const piece*>(slot + i); });
      __syncthreads();
    }
  }
  if (LPR > 64 || (mine && wave == 0)) {
    float* out = part + (static_cast<size_t>(head) * gridDim.x + blockIdx.x) * all_sums;
    columns([&](int i, piece& x) { *reinterpret_cast<piece*>(out + i) = x; });
  }
}

// out[head][col] = sum over the parts (64 bits): a workgroup takes 32 columns, 32 groups of threads
// a share of the parts each, joined through LDS in order.  Few long columns (H = 1) are bound by the
// loads' latency, so the shares are short.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormArgs a, const float* part, int parts) {
  __shared__ double share[32][33];
  const int c = threadIdx.x & 31, q = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  const int head = blockIdx.y, which = blockIdx.z;
  float* out = which == 0 ? a.dweight : which == 1 ? a.dbias : a.dscale;
  if (!out) return;
  double s = 0.0;
  if (col < a.d) {
    const int before[3] = {0, a.dweight ? 1 : 0, (a.dweight ? 1 : 0) + (a.dbias ? 1 : 0)};
    const size_t pitch = static_cast<size_t>(before[2] + (a.dscale ? 1 : 0)) * a.d;
    const float* p = part + static_cast<size_t>(head) * parts * pitch;
    p += static_cast<size_t>(before[which]) * a.d + col;
#pragma unroll 8
    for (int i = q; i < parts; i += 32) s += p[i * pitch];
  }
  share[q][c] = s;
  __syncthreads();
  if (q == 0 && col < a.d) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += share[i][c];
    out[static_cast<size_t>(head) * a.d + col] = static_cast<float>(s);
  }
}

// 16-byte vectors need whole vectors in a row and aligned tensors and parameters
bool aligned16(std::initializer_list<const void*> ps) {
  uintptr_t bits = 0;
  for (const void* p : ps) bits |= reinterpret_cast<uintptr_t>(p);
  return (bits & 15) == 0;
}
bool vectors(const NormArgs& a, int es) {
  return a.d % (16 / es) == 0 &&
         aligned16({a.x, a.weight, a.bias, a.gate, a.scale, a.res, a.y, a.dy, a.dx, a.dgate});
}

// f(W, LPR, NV) for the first layout that holds a row of d elements
template <int N> using Int = std::integral_constant<int, N>;
#define TTT_TRY(lpr, nv) \
  if (n <= lpr * nv) return f(Int<W>(), Int<lpr>(), Int<nv>())
template <int W, typename F>
hipError_t fwd_layout(int d, F f) {
  const int n = (d + W - 1) / W;
  TTT_TRY(2, 1);
  TTT_TRY(4, 1);
  TTT_TRY(8, 1);
  if constexpr (W > 1) {
    TTT_TRY(16, 1);
    TTT_TRY(32, 1);
    TTT_TRY(64, 1);
    TTT_TRY(32, 3);
    TTT_TRY(64, 2);
    TTT_TRY(64, 3);
    TTT_TRY(64, 4);
    TTT_TRY(256, 2);
    TTT_TRY(256, 3);
    TTT_TRY(256, 4);
    if constexpr (W == 4) TTT_TRY(256, 8);
    if constexpr (W == 8) TTT_TRY(1024, 2);
    if constexpr (W == 4) TTT_TRY(1024, 4);
  }
  return hipErrorInvalidValue;
}
// The backward pass holds three more rows (the parameters' sums) and the next one: no more than 16
// elements a lane, so that two waves share a SIMD's registers.  With a gate, us: 8191 rows of
// 768 bf16 as 64 x 2 vectors 23.3, as 32 x 3 32.4; 8192 of 2048 as 256 x 1 47.7, as 64 x 4 70.8; 8192 of
// 4096 as 256 x 2 77.6, as 512 x 1 91.3.  Rows of 8193 to 12288 bf16 are 512 x 3: 56.7 us for 2048
// of 12000, as 1024 x 2 71.8 (with a gate 276 and 282: the registers spill in both).
template <int W, typename F>
hipError_t bwd_layout(int d, F f) {
  const int n = (d + W - 1) / W;
  TTT_TRY(2, 1);
  TTT_TRY(4, 1);
  TTT_TRY(8, 1);
  if constexpr (W > 1) {
    TTT_TRY(16, 1);
    TTT_TRY(32, 1);
    TTT_TRY(64, 1);
    TTT_TRY(64, 2);
    TTT_TRY(256, 1);
    TTT_TRY(256, 2);
    TTT_TRY(512, 2);
    if constexpr (W == 8) TTT_TRY(512, 3);
    if constexpr (W == 8) TTT_TRY(1024, 2);
    if constexpr (W == 4) TTT_TRY(512, 4);
    if constexpr (W == 4) TTT_TRY(1024, 4);
  }
  return hipErrorInvalidValue;
}
#undef TTT_TRY
// whole rows of aligned vectors, else vectors at any element, else (rows shorter than one) elements
template <typename IO, bool kBwd, typename F>
hipError_t choose(const NormArgs& a, F f) {
  constexpr int W = 16 / static_cast<int>(sizeof(IO));
  const auto layout = [&](auto w, auto al) {
    const auto g = [&](auto w, auto lpr, auto nv) { return f(w, lpr, nv, al); };
    if constexpr (kBwd) return bwd_layout<w.value>(a.d, g);
    else return fwd_layout<w.value>(a.d, g);
  };
  if (vectors(a, sizeof(IO))) return layout(Int<W>(), std::true_type());
  if (a.d >= W) return layout(Int<W>(), std::false_type());
  return layout(Int<1>(), std::true_type());
}

template <typename IO, int W, int LPR, int NV, bool A>
hipError_t run_fwd(const NormArgs& a, hipStream_t s) {
  constexpr int RB = Block<LPR>::kRows;
  const long long rows = static_cast<long long>(a.B) * a.H * a.T;
  const long long groups = (rows + RB - 1) / RB;
  // several passes share a workgroup's start once there are workgroups enough
  // (and a grid holds less than 2^32 threads: at most 2^21 workgroups of 1024)
  const int passes = groups >= 8192 ? static_cast<int>(groups >> 21) + 4 : groups >= 4096 ? 2 : 1;
  const dim3 grid(static_cast<unsigned>((groups + passes - 1) / passes)), block(Block<LPR>::kThreads);
  norm_fwd_kernel<IO, W, LPR, NV, A><<<grid, block, 0, s>>>(a, static_cast<int>(rows), passes);
  return hipGetLastError();
}

// The backward pass's workgroups: at most 768 (three of 256 threads a CU, so that all start at
// once and end together), each with 16 rows of a head at least so that its sums stay small next to
// its rows, or 4 while there are less than 256, one a CU.  On 8 x 12 x 2048 rows of 64 bf16 with a
// gate: 512 workgroups 33.7 us, 768 28.8, 1024 34.7; on 8192 of 2048 without: 512 of them (16 rows)
// 27.3, 768 33.6; on 2048 of 8192: 128 (16 rows) 38.8, 256 27.8; on 1024 of 16384 float32: 64 (16
// rows) 101, 128 66, 256 54.
long long most_parts(int B, int H, int T) {
  const long long rows = static_cast<long long>(B) * T;
  const long long of16 = (rows + 15) / 16, of4 = (rows + 3) / 4, one_a_cu = 256 / H;
  const long long parts = of16 > one_a_cu ? of16 : of4 < one_a_cu ? of4 : one_a_cu;
  const long long most = 768 / H < parts ? 768 / H : parts;
  return most < 1 ? 1 : most;
}
// rows of a part: whole passes of `at_once` rows
int rows_of_part(int B, int H, int T, int at_once) {
  const long long rows = static_cast<long long>(B) * T, parts = most_parts(B, H, T);
  const long long share = (rows + parts - 1) / parts;
  return static_cast<int>(share < 1 ? at_once : (share + at_once - 1) / at_once * at_once);
}
int bwd_parts(int B, int H, int T, int share) {
  const long long rows = static_cast<long long>(B) * T, parts = (rows + share - 1) / share;
  return static_cast<int>(parts < 1 ? 1 : parts);
}

template <typename IO, int W, int LPR, int NV, bool A, bool kPlain>
hipError_t run_bwd(const NormArgs& a, void* ws, hipStream_t s) {
  const int share = rows_of_part(a.B, a.H, a.T, Block<LPR>::kRows), parts = bwd_parts(a.B, a.H, a.T, share);
  const bool sums = a.dweight || a.dbias || a.dscale;
  const int lds = sums && LPR <= 64 ? 2 * 3 * a.d * static_cast<int>(sizeof(float)) : 0;  // 24 KB at most
  float* part = sums ? static_cast<float*>(ws) : nullptr;
  const dim3 grid(parts, a.H), block(Block<LPR>::kThreads);
  norm_bwd_kernel<IO, W, LPR, NV, A, kPlain><<<grid, block, lds, s>>>(a, part, share);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !sums) return e;
  norm_sum_kernel<<<dim3((a.d + 31) / 32, a.H, 3), dim3(1024), 0, s>>>(a, part, parts);
  return hipGetLastError();
}

template <typename IO>
hipError_t bwd_io(const NormArgs& a, void* ws, hipStream_t s) {
  return choose<IO, true>(a, [&](auto w, auto lpr, auto nv, auto al) {
    if (a.gate || a.scale) return run_bwd<IO, w.value, lpr.value, nv.value, al.value, false>(a, ws, s);
    return run_bwd<IO, w.value, lpr.value, nv.value, al.value, true>(a, ws, s);
  });
}

template <typename IO>
hipError_t fwd_io(const NormArgs& a, hipStream_t s) {
  return choose<IO, false>(a, [&](auto w, auto lpr, auto nv, auto al) {
    return run_fwd<IO, w.value, lpr.value, nv.value, al.value>(a, s);
  });
}

}  // namespace

size_t token_norm_bwd_workspace_bytes(int B, int H, int T, int d) {
  return static_cast<size_t>(most_parts(B, H, T)) * H * 3 * d * sizeof(float);
}

hipError_t launch_token_norm_fwd(const NormArgs& a, bool bf16_io, hipStream_t s) {
  return bf16_io ? fwd_io<bf16>(a, s) : fwd_io<float>(a, s);
}

hipError_t launch_token_norm_bwd(const NormArgs& a, bool bf16_io, void* ws, hipStream_t s) {
  return bf16_io ? bwd_io<bf16>(a, ws, s) : bwd_io<float>(a, ws, s);
}

}  // namespace ttt
