// Gated linear recurrence, forward and backward, on the float32 matrix cores: d in {16, 32, 64},
// fp32 or bf16 I/O (formulas in gated_linear.hpp; backward below).  One workgroup of d / 16 waves
// per (batch, head) sequence walks its chunks; the d x d state stays in registers, 16 columns a
// wave, in the MFMA C layout, which serves as an operand of the next chunk's products as it is.
//
// Every product is a sum of 16 x 16 tiles C = A B by v_mfma_f32_16x16x4_f32.  Lane (g, r) holds
// row r of A and column r of B for k = 4 g + e (e = 0..3) of each block of 16 k, and rows
// 4 g + e of column r of C: a C tile is an operand whose k runs along its rows, with no exchange.
#include "gated_linear.hpp"

namespace ttt {
namespace {

constexpr int kC = kGlChunk;
constexpr int kPC = kGlPitch;

__device__ __forceinline__ void mma(gl_f4& c, const gl_f4& a, const gl_f4& b) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
}
// operand with k along the rows of a row-major LDS matrix: row r0 + r, k = k0 + 4 g + e
__device__ __forceinline__ gl_f4 along(const float* m, int ld, int r0, int k0, int g, int r) {
  return *reinterpret_cast<const gl_f4*>(m + (r0 + r) * ld + k0 + 4 * g);
}
// operand with k down the rows: k = k0 + 4 g + e, column c0 + r
__device__ __forceinline__ gl_f4 down(const float* m, int ld, int k0, int c0, int g, int r) {
  const float* p = m + (k0 + 4 * g) * ld + c0 + r;
  return gl_f4{p[0], p[ld], p[2 * ld], p[3 * ld]};
}
__device__ __forceinline__ gl_f4 keep4(float f, const gl_f4& x) {
  return gl_f4{gl_keep(f, x[0]), gl_keep(f, x[1]), gl_keep(f, x[2]), gl_keep(f, x[3])};
}
__device__ __forceinline__ gl_f4 at4(const float* p, int i) { return *reinterpret_cast<const gl_f4*>(p + i); }

// A token tile (kC x D) on its way from HBM to LDS as float32: each thread holds 16 elements.
template <typename IO, int D>
struct Tile {
  static constexpr int kThreads = 4 * D;
  static constexpr int kVec = static_cast<int>(sizeof(IO));       // 16-byte vectors per thread
  static constexpr int kPerVec = 16 / static_cast<int>(sizeof(IO));
  gl_u4 x[kVec];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t src, int tid) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      x[i] = __builtin_amdgcn_raw_buffer_load_b128(src, (tid + i * kThreads) * 16, 0, 0);
  }
  __device__ __forceinline__ void put(float* m, int tid) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int at = (tid + i * kThreads) * kPerVec;
      float* p = m + (at / D) * (D + 4) + at % D;
      if constexpr (sizeof(IO) == 4) {
        *reinterpret_cast<gl_u4*>(p) = x[i];
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          gl_f4 y;
          y[0] = __builtin_bit_cast(float, x[i][2 * j] << 16);
          y[1] = __builtin_bit_cast(float, x[i][2 * j] & 0xFFFF0000u);
          y[2] = __builtin_bit_cast(float, x[i][2 * j + 1] << 16);
          y[3] = __builtin_bit_cast(float, x[i][2 * j + 1] & 0xFFFF0000u);
          *reinterpret_cast<gl_f4*>(p + 4 * j) = y;
        }
      }
    }
  }
};

// four consecutive features of a token, rounded once to the I/O type
template <typename IO>
__device__ __forceinline__ void store4(const gl_f4& x, __amdgpu_buffer_rsrc_t dst, int elem) {
  if constexpr (sizeof(IO) == 4) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(gl_u4, x), dst, elem * 4, 0, 0);
  } else {
    typedef bf16 bf4 __attribute__((ext_vector_type(4)));
    const bf4 y = {from_f32<bf16>(x[0]), from_f32<bf16>(x[1]), from_f32<bf16>(x[2]), from_f32<bf16>(x[3])};
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(gl_u2, y), dst, elem * 2, 0, 0);
  }
}

// One sequence's view of the arguments.
template <typename IO>
struct Seq {
  size_t tok0;       // first element of its tokens
  size_t row0;       // first token
  int len;           // tokens that count
  const float* gate;
  const float* rate;
};
template <typename IO>
__device__ __forceinline__ Seq<IO> sequence(const GatedArgs& a, int chain, int D) {
  Seq<IO> s;
  s.row0 = static_cast<size_t>(chain) * a.T;
  s.tok0 = s.row0 * D;
  s.len = gl_length(a.lengths, chain / a.H, a.T);
  s.gate = a.gate ? a.gate + s.row0 : nullptr;
  s.rate = a.eta_tok ? a.eta_tok + s.row0 : nullptr;
  return s;
}

// the token's log decay and rate (0, 0 past the sequence)
struct GateRate {
  float g, e;
};
template <typename IO>
__device__ __forceinline__ GateRate gate_rate(const Seq<IO>& s, float eta, int t) {
  const bool in = t < s.len;
  GateRate x;
  x.g = in && s.gate ? s.gate[t] : 0.0f;
  x.e = in ? (s.rate ? eta * s.rate[t] : eta) : 0.0f;
  return x;
}

template <int D>
struct FwdLds {
  float q[kC * (D + 4)], k[kC * (D + 4)], v[kC * (D + 4)];
  float p[kC * kPC];
  GlDecays dec;
};

template <typename IO, int D>
__global__ __launch_bounds__(4 * D) void gl_fwd_kernel(GatedArgs a) {
  constexpr int NW = D / 16, PD = D + 4;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  FwdLds<D>& L = *reinterpret_cast<FwdLds<D>*>(lds_raw);
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int chain = blockIdx.x, T = a.T;
  const Seq<IO> s = sequence<IO>(a, chain, D);
  const IO* q = static_cast<const IO*>(a.q) + s.tok0;
  const IO* k = static_cast<const IO*>(a.k) + s.tok0;
  const IO* v = static_cast<const IO*>(a.v) + s.tok0;
  IO* z = static_cast<IO*>(a.z) + s.tok0;
  const int nchunks = (T + kC - 1) / kC;

  // W^T, columns j of the wave: tile ib holds W[16 wv + r][16 ib + 4 g + e]
  gl_f4 w[NW];
  const float* w0 = a.w0 + (chain / a.H) * a.w0_batch_stride + static_cast<size_t>(chain % a.H) * D * D;
  const size_t at_w = static_cast<size_t>(16 * wv + r) * D + 4 * g;
#pragma unroll
  for (int ib = 0; ib < NW; ++ib) w[ib] = *reinterpret_cast<const gl_f4*>(w0 + at_w + 16 * ib);

  Tile<IO, D> tq, tk, tv;
  GateRate gr;
  auto prefetch = [&](int c) {
    const int c0 = c * kC, bytes = min(kC, s.len - c0) * D * static_cast<int>(sizeof(IO));
    const size_t off = static_cast<size_t>(c0) * D;
    tq.load(gl_span(q + off, bytes), tid);
    tk.load(gl_span(k + off, bytes), tid);
    tv.load(gl_span(v + off, bytes), tid);
    if (wv == 0) gr = gate_rate(s, a.eta, c0 + lane);
  };
  if (nchunks > 0) prefetch(0);
  for (int c = 0; c < nchunks; ++c) {
    const int c0 = c * kC;
    gl_barrier();  // the previous chunk's tiles have been read
    tq.put(L.q, tid);
    tk.put(L.k, tid);
    tv.put(L.v, tid);
    if (wv == 0) gl_decays(gr.g, gr.e, &L.dec, lane);
    gl_barrier();
    if (c + 1 < nchunks) prefetch(c + 1);

    // P[u][s] = exp(b_u - b_s) e_s (q_u . k_s) for s <= u, the wave's blocks of 16 tokens u
#pragma unroll
    for (int it = 0; it < 4 / NW; ++it) {
      const int ut = wv + it * NW, u = 16 * ut + r;
      const float uh = L.dec.bh[u], ul = L.dec.bl[u];
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        if (st > ut) break;
        gl_f4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < NW; ++kb) mma(p, along(L.k, PD, 16 * st, 16 * kb, g, r), along(L.q, PD, 16 * ut, 16 * kb, g, r));
        const int s4 = 16 * st + 4 * g;
        const gl_f4 sh = at4(L.dec.bh, s4), sl = at4(L.dec.bl, s4), e = at4(L.dec.e, s4);
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] = s4 + x <= u ? p[x] * (gl_between(uh, ul, sh[x], sl[x]) * e[x]) : 0.0f;
        *reinterpret_cast<gl_f4*>(&L.p[u * kPC + s4]) = p;
      }
    }
    gl_barrier();

    gl_f4 vf[4];  // V, k down the tokens, the wave's features
#pragma unroll
    for (int st = 0; st < 4; ++st) vf[st] = down(L.v, PD, 16 * st, 16 * wv, g, r);
    const int rows = min(kC, T - c0);
    const __amdgpu_buffer_rsrc_t dst = gl_span(z + static_cast<size_t>(c0) * D, rows * D * static_cast<int>(sizeof(IO)));
#pragma unroll
    for (int ut = 0; ut < 4; ++ut) {  // Z^T: rows j, columns u
      gl_f4 zi = {0.0f, 0.0f, 0.0f, 0.0f}, zp = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ib = 0; ib < NW; ++ib) mma(zi, w[ib], along(L.q, PD, 16 * ut, 16 * ib, g, r));
#pragma unroll
      for (int st = 0; st <= ut; ++st) mma(zp, vf[st], along(L.p, kPC, 16 * ut, 16 * st, g, r));
      const int u = 16 * ut + r;
      const float f = L.dec.from[u];
      store4<IO>(zp + keep4(f, zi), dst, u * D + 16 * wv + 4 * g);
    }
    const float whole = L.dec.whole[0];
#pragma unroll
    for (int st = 0; st < 4; ++st) vf[st] *= at4(L.dec.to, 16 * st + 4 * g) * at4(L.dec.e, 16 * st + 4 * g);
#pragma unroll
    for (int ib = 0; ib < NW; ++ib) {
      w[ib] = keep4(whole, w[ib]);
#pragma unroll
      for (int st = 0; st < 4; ++st) mma(w[ib], down(L.k, PD, 16 * st, 16 * ib, g, r), vf[st]);
    }
  }
  if (a.w_out) {
    float* wo = a.w_out + static_cast<size_t>(chain) * D * D + at_w;
#pragma unroll
    for (int ib = 0; ib < NW; ++ib) *reinterpret_cast<gl_f4*>(wo + 16 * ib) = w[ib];
  }
}

// ---------------------------------------------------------------- backward
//
// With G_t = dL/dW_t (before the decay into t - 1), G_t = a_{t+1} G_{t+1} + dz_t q_t^T:
//   dq_u = sum_{s <= u} exp(b_u - b_s) e_s (dz_u . v_s) k_s + exp(b_u) W^T dz_u,
//   dv_s = e_s x_s,  x_s = sum_{u >= s} exp(b_u - b_s) (q_u . k_s) dz_u + exp(b_C - b_s) G k_s,
//   dk_s = e_s (sum_{u >= s} exp(b_u - b_s) (dz_u . v_s) q_u + exp(b_C - b_s) G^T v_s),
//   de_s = v_s . x_s,
// W the state before the chunk, G the gradient at its end.  Two roles share no data: one
// workgroup walks a sequence forward with W for dq, another walks it backward with G for dk and
// dv.  So no state is stored on the way.
//
// dg_t = a_t <G_t, W_{t-1}> is the sum over the pairs (s, u), s < t <= u, of what token s
// contributes to output u.  With m_us = exp(b_u - b_s) e_s (q_u . k_s)(dz_u . v_s), per chunk:
//   dg_t = sum_{u >= t} (row_u - col_u) + sum_{u >= t} in_u + sum_{s < t} out_s + past,
//   row_u = sum_{s < u} m_us, col_s = sum_{u > s} m_us (pairs inside the chunk),
//   in_u = exp(b_u) dz_u . W q_u,  out_s = exp(b_C - b_s) e_s v_s . G k_s,  past = exp(b_C) <G, W>.
// Only the row - col sums cancel, over one chunk; nothing grows with the sequence.  `past` follows
// from <G, W> at the sequence's end: past_c = <G, W>_end(c) - sum out, <G, W>_start(c) = past_c +
// sum in.  The two roles store row, in, col, out per token, and gl_dgate_kernel adds them.
template <int D>
struct BwdLds {
  float q[kC * (D + 4)], k[kC * (D + 4)], v[kC * (D + 4)], z[kC * (D + 4)];
  float p[kC * kPC], r[kC * kPC];
  float part[D / 16][kC];
  GlDecays dec;
};

template <typename IO, int D>
__global__ __launch_bounds__(4 * D) void gl_bwd_kernel(GatedArgs a) {
  constexpr int NW = D / 16, PD = D + 4;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  BwdLds<D>& L = *reinterpret_cast<BwdLds<D>*>(lds_raw);
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int chain = blockIdx.x >> 1, role = blockIdx.x & 1, T = a.T;
  const Seq<IO> s = sequence<IO>(a, chain, D);
  const IO* q = static_cast<const IO*>(a.q) + s.tok0;
  const IO* k = static_cast<const IO*>(a.k) + s.tok0;
  const IO* v = static_cast<const IO*>(a.v) + s.tok0;
  const IO* dz = static_cast<const IO*>(a.dz) + s.tok0;
  const int nchunks = (T + kC - 1) / kC;
  const size_t rows_all = static_cast<size_t>(a.B) * a.H * T;
  float* row_o = a.ws_tok ? a.ws_tok + s.row0 : nullptr;
  float* in_o = a.ws_tok ? row_o + rows_all : nullptr;
  float* col_o = a.ws_tok ? in_o + rows_all : nullptr;
  float* out_o = a.ws_tok ? col_o + rows_all : nullptr;

  Tile<IO, D> tq, tk, tv, tz;
  GateRate gr;
  auto prefetch = [&](int c) {
    const int c0 = c * kC, bytes = min(kC, s.len - c0) * D * static_cast<int>(sizeof(IO));
    const size_t off = static_cast<size_t>(c0) * D;
    tq.load(gl_span(q + off, bytes), tid);
    tk.load(gl_span(k + off, bytes), tid);
    tv.load(gl_span(v + off, bytes), tid);
    tz.load(gl_span(dz + off, bytes), tid);
    if (wv == 0) gr = gate_rate(s, a.eta, c0 + lane);
  };
  auto stage = [&]() {
    tq.put(L.q, tid);
    tk.put(L.k, tid);
    tv.put(L.v, tid);
    tz.put(L.z, tid);
    if (wv == 0) gl_decays(gr.g, gr.e, &L.dec, lane);
  };
  // over the four lanes (g) that share a token r
  auto over_g = [](float x) {
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
  };

  if (role == 0) {
    // W, columns i of the wave: tile jb holds W[16 jb + 4 g + e][16 wv + r]
    gl_f4 w[NW];
    const float* w0 = a.w0 + (chain / a.H) * a.w0_batch_stride + static_cast<size_t>(chain % a.H) * D * D;
#pragma unroll
    for (int jb = 0; jb < NW; ++jb)
#pragma unroll
      for (int e = 0; e < 4; ++e) w[jb][e] = w0[(16 * jb + 4 * g + e) * D + 16 * wv + r];
    IO* dq = static_cast<IO*>(a.dq) + s.tok0;
    if (nchunks > 0) prefetch(0);
    for (int c = 0; c < nchunks; ++c) {
      const int c0 = c * kC;
      gl_barrier();
      stage();
      gl_barrier();
      if (c + 1 < nchunks) prefetch(c + 1);
#pragma unroll
      for (int it = 0; it < 4 / NW; ++it) {
        const int ut = wv + it * NW, u = 16 * ut + r;
        const float uh = L.dec.bh[u], ul = L.dec.bl[u];
        float row = 0.0f;
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          if (st > ut) break;
          gl_f4 rd = {0.0f, 0.0f, 0.0f, 0.0f}, p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int kb = 0; kb < NW; ++kb) mma(rd, along(L.v, PD, 16 * st, 16 * kb, g, r), along(L.z, PD, 16 * ut, 16 * kb, g, r));
          const int s4 = 16 * st + 4 * g;
          const gl_f4 sh = at4(L.dec.bh, s4), sl = at4(L.dec.bl, s4), e = at4(L.dec.e, s4);
#pragma unroll
          for (int x = 0; x < 4; ++x) rd[x] = s4 + x <= u ? rd[x] * (gl_between(uh, ul, sh[x], sl[x]) * e[x]) : 0.0f;
          *reinterpret_cast<gl_f4*>(&L.r[u * kPC + s4]) = rd;
          if (row_o) {
#pragma unroll
            for (int kb = 0; kb < NW; ++kb) mma(p, along(L.k, PD, 16 * st, 16 * kb, g, r), along(L.q, PD, 16 * ut, 16 * kb, g, r));
#pragma unroll
            for (int x = 0; x < 4; ++x) row += s4 + x < u ? p[x] * rd[x] : 0.0f;
          }
        }
        if (row_o) {
          row = over_g(row);
          if (g == 0 && c0 + u < T) row_o[c0 + u] = row;
        }
      }
      gl_barrier();
      gl_f4 kf[4];
#pragma unroll
      for (int st = 0; st < 4; ++st) kf[st] = down(L.k, PD, 16 * st, 16 * wv, g, r);
      const __amdgpu_buffer_rsrc_t dst = gl_span(dq + static_cast<size_t>(c0) * D, min(kC, T - c0) * D * static_cast<int>(sizeof(IO)));
#pragma unroll
      for (int ut = 0; ut < 4; ++ut) {
        gl_f4 xi = {0.0f, 0.0f, 0.0f, 0.0f}, xp = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int jb = 0; jb < NW; ++jb) mma(xi, w[jb], along(L.z, PD, 16 * ut, 16 * jb, g, r));
#pragma unroll
        for (int st = 0; st <= ut; ++st) mma(xp, kf[st], along(L.r, kPC, 16 * ut, 16 * st, g, r));
        const int u = 16 * ut + r;
        const float f = L.dec.from[u];
        xi = keep4(f, xi);
        if (row_o) {
          const gl_f4 qu = along(L.q, PD, 16 * ut, 16 * wv, g, r);
          float in = over_g(qu[0] * xi[0] + qu[1] * xi[1] + qu[2] * xi[2] + qu[3] * xi[3]);
          if (g == 0) L.part[wv][u] = in;
        }
        store4<IO>(xi + xp, dst, u * D + 16 * wv + 4 * g);
      }
      const float whole = L.dec.whole[0];
#pragma unroll
      for (int st = 0; st < 4; ++st) kf[st] *= at4(L.dec.to, 16 * st + 4 * g) * at4(L.dec.e, 16 * st + 4 * g);
#pragma unroll
      for (int jb = 0; jb < NW; ++jb) {
        w[jb] = keep4(whole, w[jb]);
#pragma unroll
        for (int st = 0; st < 4; ++st) mma(w[jb], down(L.v, PD, 16 * st, 16 * jb, g, r), kf[st]);
      }
      if (row_o) {
        gl_barrier();
        if (wv == 0 && c0 + lane < T) {
          float in = 0.0f;
#pragma unroll
          for (int x = 0; x < NW; ++x) in += L.part[x][lane];
          in_o[c0 + lane] = in;
        }
      }
    }
    if (row_o) {  // <dL/dW, W> at the sequence's end
      double x = 0.0;
      if (a.dw_out) {
        const float* dw = a.dw_out + static_cast<size_t>(chain) * D * D;
#pragma unroll
        for (int jb = 0; jb < NW; ++jb)
#pragma unroll
          for (int e = 0; e < 4; ++e) x += static_cast<double>(w[jb][e]) * dw[(16 * jb + 4 * g + e) * D + 16 * wv + r];
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o, 64);
      if (lane == 0) a.ws_end[static_cast<size_t>(chain) * NW + wv] = x;
    }
  } else {
    // G twice: gt holds G[16 wv + r][16 ib + 4 g + e] (k along i), gn holds G[16 jb + 4 g + e][16 wv + r]
    gl_f4 gt[NW], gn[NW];
    const float* dw = a.dw_out ? a.dw_out + static_cast<size_t>(chain) * D * D : nullptr;
    const size_t at_w = static_cast<size_t>(16 * wv + r) * D + 4 * g;
#pragma unroll
    for (int ib = 0; ib < NW; ++ib)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        gt[ib][e] = dw ? dw[at_w + 16 * ib + e] : 0.0f;
        gn[ib][e] = dw ? dw[(16 * ib + 4 * g + e) * D + 16 * wv + r] : 0.0f;
      }
    IO* dk = static_cast<IO*>(a.dk) + s.tok0;
    IO* dv = static_cast<IO*>(a.dv) + s.tok0;
    float* de_o = a.deta_tok ? a.deta_tok + s.row0 : nullptr;
    if (nchunks > 0) prefetch(nchunks - 1);
    for (int c = nchunks - 1; c >= 0; --c) {
      const int c0 = c * kC;
      gl_barrier();
      stage();
      gl_barrier();
      if (c > 0) prefetch(c - 1);
      // the wave's blocks of 16 tokens s: rows of P^T and R^T (decayed, without e_s)
      float diag[4 / NW], col[4 / NW];
#pragma unroll
      for (int it = 0; it < 4 / NW; ++it) {
        const int st = wv + it * NW, ss = 16 * st + r;
        const float sh = L.dec.bh[ss], sl = L.dec.bl[ss];
        float cs = 0.0f, dg = 0.0f;
#pragma unroll
        for (int ut = 0; ut < 4; ++ut) {
          if (ut < st) continue;
          gl_f4 p = {0.0f, 0.0f, 0.0f, 0.0f}, rd = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int kb = 0; kb < NW; ++kb) {
            mma(p, along(L.q, PD, 16 * ut, 16 * kb, g, r), along(L.k, PD, 16 * st, 16 * kb, g, r));
            mma(rd, along(L.z, PD, 16 * ut, 16 * kb, g, r), along(L.v, PD, 16 * st, 16 * kb, g, r));
          }
          const int u4 = 16 * ut + 4 * g;
          const gl_f4 uh = at4(L.dec.bh, u4), ul = at4(L.dec.bl, u4);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float dec = u4 + x >= ss ? gl_between(uh[x], ul[x], sh, sl) : 0.0f;
            const float m = u4 + x >= ss ? p[x] * rd[x] * dec : 0.0f;
            p[x] = u4 + x >= ss ? p[x] * dec : 0.0f;
            rd[x] = u4 + x >= ss ? rd[x] * dec : 0.0f;
            cs += u4 + x > ss ? m : 0.0f;
            dg += u4 + x == ss ? m : 0.0f;
          }
          *reinterpret_cast<gl_f4*>(&L.p[ss * kPC + u4]) = p;
          *reinterpret_cast<gl_f4*>(&L.r[ss * kPC + u4]) = rd;
        }
        col[it] = over_g(cs);
        diag[it] = over_g(dg);
      }
      gl_barrier();
      gl_f4 zf[4], qf[4];  // dZ and Q, k down the tokens u, the wave's features
#pragma unroll
      for (int ut = 0; ut < 4; ++ut) {
        zf[ut] = down(L.z, PD, 16 * ut, 16 * wv, g, r);
        qf[ut] = down(L.q, PD, 16 * ut, 16 * wv, g, r);
      }
      const int bytes = min(kC, T - c0) * D * static_cast<int>(sizeof(IO));
      const __amdgpu_buffer_rsrc_t dstv = gl_span(dv + static_cast<size_t>(c0) * D, bytes);
      const __amdgpu_buffer_rsrc_t dstk = gl_span(dk + static_cast<size_t>(c0) * D, bytes);
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        gl_f4 vi = {0.0f, 0.0f, 0.0f, 0.0f}, vp = vi, ki = vi, kp = vi;
#pragma unroll
        for (int ib = 0; ib < NW; ++ib) {
          mma(vi, gt[ib], along(L.k, PD, 16 * st, 16 * ib, g, r));
          mma(ki, gn[ib], along(L.v, PD, 16 * st, 16 * ib, g, r));
        }
#pragma unroll
        for (int ut = st; ut < 4; ++ut) {
          mma(vp, zf[ut], along(L.p, kPC, 16 * st, 16 * ut, g, r));
          mma(kp, qf[ut], along(L.r, kPC, 16 * st, 16 * ut, g, r));
        }
        const int ss = 16 * st + r;
        const float f = L.dec.to[ss], e = L.dec.e[ss];
        vi = keep4(f, vi);
        const gl_f4 vs = along(L.v, PD, 16 * st, 16 * wv, g, r);
        const float out = over_g(vs[0] * vi[0] + vs[1] * vi[1] + vs[2] * vi[2] + vs[3] * vi[3]);
        if (g == 0) L.part[wv][ss] = out;
        store4<IO>(e * (vi + vp), dstv, ss * D + 16 * wv + 4 * g);
        store4<IO>(e * (keep4(f, ki) + kp), dstk, ss * D + 16 * wv + 4 * g);
      }
      const float whole = L.dec.whole[0];
#pragma unroll
      for (int ib = 0; ib < NW; ++ib) {
        gt[ib] = keep4(whole, gt[ib]);
        gn[ib] = keep4(whole, gn[ib]);
#pragma unroll
        for (int ut = 0; ut < 4; ++ut) {
          const gl_f4 f = at4(L.dec.from, 16 * ut + 4 * g);
          mma(gt[ib], down(L.q, PD, 16 * ut, 16 * ib, g, r), zf[ut] * f);
          mma(gn[ib], down(L.z, PD, 16 * ut, 16 * ib, g, r), qf[ut] * f);
        }
      }
      gl_barrier();
#pragma unroll
      for (int it = 0; it < 4 / NW; ++it) {
        const int ss = 16 * (wv + it * NW) + r, t = c0 + ss;
        float out = 0.0f;
#pragma unroll
        for (int x = 0; x < NW; ++x) out += L.part[x][ss];
        const float e = L.dec.e[ss];
        if (g == 0 && t < T) {
          if (de_o) de_o[t] = t < s.len ? a.eta * (col[it] + diag[it] + out) : 0.0f;
          if (col_o) {
            col_o[t] = e * col[it];
            out_o[t] = e * out;
          }
        }
      }
    }
    float* dw0 = a.dw0 + static_cast<size_t>(chain) * D * D + at_w;
#pragma unroll
    for (int ib = 0; ib < NW; ++ib) *reinterpret_cast<gl_f4*>(dw0 + 16 * ib) = gt[ib];
  }
}

// dlog_gate from the per-token sums (see above): one wave per chunk, lane = token.  Each wave
// first walks the sums of the later chunks of its sequence.
__global__ __launch_bounds__(256) void gl_dgate_kernel(GatedArgs a, int nend) {
  const int lane = threadIdx.x & 63;
  const int nchunks = (a.T + kC - 1) / kC;
  const long long item = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (item >= static_cast<long long>(a.B) * a.H * nchunks) return;
  const int chain = static_cast<int>(item / nchunks), c = static_cast<int>(item % nchunks);
  const size_t all = static_cast<size_t>(a.B) * a.H * a.T, row0 = static_cast<size_t>(chain) * a.T;
  const float* row = a.ws_tok + row0;
  const float* in = row + all;
  const float* col = in + all;
  const float* out = col + all;
  const int len = gl_length(a.lengths, chain / a.H, a.T);
  double later = 0.0;  // over the tokens of later chunks
  for (int t = (c + 1) * kC + lane; t < a.T; t += 64) later += static_cast<double>(in[t]) - out[t];
  for (int x = lane; x < nend; x += 64) later += a.ws_end[static_cast<size_t>(chain) * nend + x];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) later += __shfl_xor(later, o, 64);
  const int t = c * kC + lane;
  const bool have = t < a.T;
  double suf = have ? static_cast<double>(row[t]) - col[t] + in[t] : 0.0;  // over u >= t
  const double o_t = have ? static_cast<double>(out[t]) : 0.0;
  double pre = o_t;  // over s <= t
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double x = __shfl_down(suf, o, 64), y = __shfl_up(pre, o, 64);
    if (lane + o < 64) suf += x;
    if (lane >= o) pre += y;
  }
  const double past = later - __shfl(pre, 63, 64);
  if (!have) return;
  // a token that forgets everything (decay 0) takes no gradient
  const bool live = t < len && !(static_cast<double>(a.gate[row0 + t]) * 1.4426950408889634 <= kGlNever);
  a.dgate[row0 + t] = live ? static_cast<float>(suf + (pre - o_t) + past) : 0.0f;
}

template <typename IO, int D>
hipError_t fwd(const GatedArgs& a, hipStream_t s) {
  const auto fn = gl_fwd_kernel<IO, D>;
  constexpr int bytes = sizeof(FwdLds<D>);
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  fn<<<dim3(a.B * a.H), dim3(4 * D), bytes, s>>>(a);
  return hipGetLastError();
}

template <typename IO, int D>
hipError_t bwd(const GatedArgs& a, hipStream_t s) {
  const auto fn = gl_bwd_kernel<IO, D>;
  constexpr int bytes = sizeof(BwdLds<D>);
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  fn<<<dim3(2 * a.B * a.H), dim3(4 * D), bytes, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || !a.dgate || a.T == 0) return e;
  const long long items = static_cast<long long>(a.B) * a.H * ((a.T + kC - 1) / kC);
  gl_dgate_kernel<<<dim3(static_cast<unsigned>((items + 3) / 4)), dim3(256), 0, s>>>(a, D / 16);
  return hipGetLastError();
}

}  // namespace

size_t gated_fwd_workspace_bytes(int, int, int, int, bool) { return 0; }

size_t gated_bwd_workspace_bytes(int B, int H, int T, int d, bool gated, bool) {
  if (!gated) return 0;
  const size_t chains = static_cast<size_t>(B) * H;
  return chains * (d / 16) * sizeof(double) + chains * T * 4 * sizeof(float);
}

hipError_t launch_gated_fwd(GatedArgs a, int d, bool bf16_io, void*, hipStream_t s) {
  if (bf16_io) return d == 16 ? fwd<bf16, 16>(a, s) : d == 32 ? fwd<bf16, 32>(a, s) : fwd<bf16, 64>(a, s);
  return d == 16 ? fwd<float, 16>(a, s) : d == 32 ? fwd<float, 32>(a, s) : fwd<float, 64>(a, s);
}

hipError_t launch_gated_bwd(GatedArgs a, int d, bool bf16_io, void* ws, hipStream_t s) {
  if (a.dgate) {
    a.ws_end = static_cast<double*>(ws);
    a.ws_tok = reinterpret_cast<float*>(a.ws_end + static_cast<size_t>(a.B) * a.H * (d / 16));
  }
  if (bf16_io) return d == 16 ? bwd<bf16, 16>(a, s) : d == 32 ? bwd<bf16, 32>(a, s) : bwd<bf16, 64>(a, s);
  return d == 16 ? bwd<float, 16>(a, s) : d == 32 ? bwd<float, 32>(a, s) : bwd<float, 64>(a, s);
}

}  // namespace ttt
