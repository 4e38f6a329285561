// Gated linear recurrence, forward and backward (formulas in gated_linear.hpp; backward below):
// d in {16, 32, 64}, fp32 or bf16 I/O, any T.
//
// A sequence is cut into segments of whole chunks, one workgroup of d / 16 waves each.  When a
// sequence has several, gl_sums_kernel forms what each adds to the state, gl_scan_kernel turns
// that into the state at each segment's start, and the main kernel walks the segments' chunks.
// The d x d state stays in registers, 16 columns a wave, in the MFMA C layout.
//
// Why segments: a chunk of 64 tokens takes one workgroup 2.6 us (d = 64, bf16) however many run, so
// 96 sequences of 2048 tokens, one workgroup each, took 190 us with the chip two thirds idle;
// reading K and V once more for the segments' sums (15 us) and the scan (6 us) let the rest take
// 27 us (3.8 TB/s).  Chunks of 64: the products inside a chunk grow with it, the state's splits
// and its 24 products a wave are paid once for it.
//
// Every product is a sum of 16 x 16 tiles C = A B.  Lane (g, r) of a wave holds row r of A and
// column r of B at eight k of each block of 32, the same ones for both, and rows 4 g + e (e =
// 0..3) of column r of C.  So two C tiles are an operand whose k runs along their rows, with no
// exchange between lanes: the state feeds the next chunk's products as it is.
//
//   float32 I/O:  v_mfma_f32_16x16x4_f32.
//   bf16 I/O:     v_mfma_f32_16x16x32_bf16.  Products of inputs are exact.  Factors that are not
//     inputs are split into bf16 parts, x = hi + mid + lo: two parts (2^-16 of a term) where the
//     result is rounded to bf16, three (2^-24) where it is a float32 output or the state itself
//     (with two, final states were off by 2.4e-6 and gate gradients by 3.8e-6; with three by
//     7e-8 and 1.8e-7).
#include <type_traits>

#include "gated_linear.hpp"

namespace ttt {
namespace {

constexpr int kC = kGlChunk;

typedef bf16 gl_b4 __attribute__((ext_vector_type(4)));
typedef bf16 gl_b8 __attribute__((ext_vector_type(8)));
typedef short gl_s4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ gl_f4 at4(const float* p, int i) { return *reinterpret_cast<const gl_f4*>(p + i); }
__device__ __forceinline__ gl_f4 keep4(float f, const gl_f4& x) {
  return gl_f4{gl_keep(f, x[0]), gl_keep(f, x[1]), gl_keep(f, x[2]), gl_keep(f, x[3])};
}
__device__ __forceinline__ float dot4(const gl_f4& a, const gl_f4& b) {
  return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}
// over the four lanes (g) that share r, and over the sixteen that share g
__device__ __forceinline__ float over_g(float x) { return gl_swap16(gl_swap32(x)); }
__device__ __forceinline__ float over_r(float x) { return gl_lane_sum<16>(x); }

// Matrices in LDS hold a token (or a row of token pairs) per row.  Math<IO>: their element and
// layout, and operands over 32 k (`Half`: over 16, when d = 16).
template <typename IO> struct Math;

template <>
struct Math<float> {
  typedef float Elem;
  template <int D> static constexpr int pitch() { return D + 4; }
  struct Op { gl_f4 a, b; };
  template <int N> struct Parts { Op x; };
  template <bool Half> static __device__ __forceinline__ Op along(const float* row, int p, int g) {
    const float* m = row + 32 * p + 4 * g;
    return Op{at4(m, 0), Half ? gl_f4{0.0f, 0.0f, 0.0f, 0.0f} : at4(m, Half ? 0 : 16)};
  }
  static __device__ __forceinline__ gl_f4 down16(const float* m, int ld, int k0, int cb, int g, int r) {
    const float* q = m + (k0 + 4 * g) * ld + 16 * cb + r;
    return gl_f4{q[0], q[ld], q[2 * ld], q[3 * ld]};
  }
  template <int D> static __device__ __forceinline__ Op down(const float* m, int ld, int p, int cb, int g, int r) {
    return Op{down16(m, ld, 32 * p, cb, g, r), down16(m, ld, 32 * p + 16, cb, g, r)};
  }
  template <bool Half> static __device__ __forceinline__ gl_f4 mma(const Op& a, const Op& b, gl_f4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[e], b.a[e], c, 0, 0, 0);
    if constexpr (!Half) {
#pragma unroll
      for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[e], b.b[e], c, 0, 0, 0);
    }
    return c;
  }
  template <int N> static __device__ __forceinline__ Parts<N> split(const gl_f4& a, const gl_f4& b) {
    return Parts<N>{Op{a, b}};
  }
  // the parts as rows (A), as columns (B)
  template <int N, bool Half>
  static __device__ __forceinline__ gl_f4 mma_rows(const Parts<N>& a, const Op& b, gl_f4 c) {
    return mma<Half>(a.x, b, c);
  }
  template <int N, bool Half>
  static __device__ __forceinline__ gl_f4 mma_cols(const Op& a, const Parts<N>& b, gl_f4 c) {
    return mma<Half>(a, b.x, c);
  }
  static __device__ __forceinline__ void widen(const Op& x, gl_f4* a, gl_f4* b) {
    *a = x.a;
    *b = x.b;
  }
  // A factor of token pairs: columns 16 cb + 4 g .. + 3 of a row, and its product over block cb.
  // `Block`: the other operand over 16 tokens.
  typedef gl_f4 Block;
  static constexpr int kBlock = 16, kBlockPad = 4;  // elements of a block in a row, of a row's padding
  static __device__ __forceinline__ void put(float* row, int cb, int g, const gl_f4& x) {
    *reinterpret_cast<gl_f4*>(row + 16 * cb + 4 * g) = x;
  }
  static __device__ __forceinline__ Block block(const Op& x, int half) { return half ? x.b : x.a; }
  static __device__ __forceinline__ gl_f4 mma_factor(const Block& a, const float* row, int cb, int g, gl_f4 c) {
    const gl_f4 b = at4(row, 16 * cb + 4 * g);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  // feature of row 4 g of tile b of a state
  template <int D> static __device__ __forceinline__ int state_row(int b, int g) { return 16 * b + 4 * g; }
  // the same features of a token tile as rows of an operand, k down the tokens
  template <int D>
  static __device__ __forceinline__ Op down_state(const float* m, int ld, int p, int b, int g, int r) {
    return down<D>(m, ld, p, b, g, r);
  }
  template <int D> static __device__ __forceinline__ gl_f4 row4(const float* row, int cb, int g) {
    return at4(row, 16 * cb + 4 * g);
  }
  typedef gl_f4 Four;  // four features of a token, from element `elem` of the source
  static __device__ __forceinline__ Four load4(__amdgpu_buffer_rsrc_t src, int elem) {
    return __builtin_bit_cast(gl_f4, __builtin_amdgcn_raw_buffer_load_b128(src, elem * 4, 0, 0));
  }
  static __device__ __forceinline__ gl_f4 widen4(const Four& x) { return x; }
  static __device__ __forceinline__ void store4(const gl_f4& x, __amdgpu_buffer_rsrc_t dst, int elem) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(gl_u4, x), dst, elem * 4, 0, 0);
  }
  template <int D> static __device__ __forceinline__ void put_vec(float* m, int vec, const gl_u4& x) {
    const int at = vec * 4;
    *reinterpret_cast<gl_u4*>(m + (at / D) * pitch<D>() + at % D) = x;
  }
};

template <>
struct Math<bf16> {
  typedef bf16 Elem;
  // Rows of 160 bytes (96 at d = 32): with 64 banks of 4 bytes, 16-byte reads of 16 rows and
  // transposing reads both run without conflicts (4 and 2 cycles a wave, measured).  Rows of 144
  // bytes: 8 and 4; two 8-byte reads of a lane, which the compiler joins, take 16.
  template <int D> static constexpr int pitch() { return D == 16 ? 24 : D + 16; }
  typedef gl_b8 Op;
  template <int N> struct Parts { Op x[N]; };
  // eight k of a block: columns 32 p + 8 g .. + 7 (d = 16: 4 g .. + 3)
  template <bool Half> static __device__ __forceinline__ Op along(const bf16* row, int p, int g) {
    if constexpr (Half) {
      const gl_b4 x = *reinterpret_cast<const gl_b4*>(row + 4 * g);
      return __builtin_shufflevector(x, x, 0, 1, 2, 3, 0, 1, 2, 3);
    }
    return *reinterpret_cast<const gl_b8*>(row + 32 * p + 8 * g);
  }
  // Transposing LDS read: the 16 lanes of a group give the addresses of four rows' 16 columns
  // (lane 4 i + j: row i, columns 4 j .. + 3) and receive one column of four rows each.
  static __device__ __forceinline__ gl_s4 down16(const bf16* m, int ld, int k0, int column, int g, int r) {
    const bf16* q = m + (k0 + 4 * g + (r >> 2)) * ld + column;
    typedef __attribute__((address_space(3))) gl_s4 lds_s4;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)q);
  }
  // k = 32 p + 4 g + e and 32 p + 16 + 4 g + e down the rows, columns 16 cb + r
  template <int D> static __device__ __forceinline__ Op down(const bf16* m, int ld, int p, int cb, int g, int r) {
    return down_at(m, ld, p, 16 * cb + 4 * (r & 3), g, r);
  }
  static __device__ __forceinline__ Op down_at(const bf16* m, int ld, int p, int column, int g, int r) {
    const gl_s4 a = down16(m, ld, 32 * p, column, g, r), b = down16(m, ld, 32 * p + 16, column, g, r);
    return __builtin_bit_cast(gl_b8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  // A state's rows follow `along`: rows 4 g + e of tiles 2 p and 2 p + 1 are features 32 p + 8 g + e
  // and 32 p + 8 g + 4 + e.
  template <int D> static __device__ __forceinline__ int state_row(int b, int g) {
    return D == 16 ? 4 * g : 32 * (b >> 1) + 8 * g + 4 * (b & 1);
  }
  template <int D>
  static __device__ __forceinline__ Op down_state(const bf16* m, int ld, int p, int b, int g, int r) {
    return down_at(m, ld, p, state_row<D>(b, r & 3), g, r);
  }
  template <bool Half> static __device__ __forceinline__ gl_f4 mma(const Op& a, const Op& b, gl_f4 c) {
    if constexpr (Half) {
      const gl_b4 x = __builtin_shufflevector(a, a, 0, 1, 2, 3), y = __builtin_shufflevector(b, b, 0, 1, 2, 3);
      return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(gl_s4, x), __builtin_bit_cast(gl_s4, y),
                                                       c, 0, 0, 0);
    }
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  template <int N> static __device__ __forceinline__ Parts<N> split(const gl_f4& a, const gl_f4& b) {
    Parts<N> y;
    float rest[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      gl_u4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = gl_pack(rest[2 * i], rest[2 * i + 1]);
        if (n + 1 < N) {
          rest[2 * i] -= gl_lo(x);
          rest[2 * i + 1] -= gl_hi(x);
        }
        w[i] = x;
      }
      y.x[n] = __builtin_bit_cast(gl_b8, w);
    }
    return y;
  }
  // the parts as rows (A), as columns (B), small ones first
  template <int N, bool Half>
  static __device__ __forceinline__ gl_f4 mma_rows(const Parts<N>& a, const Op& b, gl_f4 c) {
#pragma unroll
    for (int n = N - 1; n >= 0; --n) c = mma<Half>(a.x[n], b, c);
    return c;
  }
  template <int N, bool Half>
  static __device__ __forceinline__ gl_f4 mma_cols(const Op& a, const Parts<N>& b, gl_f4 c) {
#pragma unroll
    for (int n = N - 1; n >= 0; --n) c = mma<Half>(a, b.x[n], c);
    return c;
  }
  static __device__ __forceinline__ void widen(const Op& x, gl_f4* a, gl_f4* b) {
    const gl_u4 w = __builtin_bit_cast(gl_u4, x);
    *a = gl_f4{gl_lo(w[0]), gl_hi(w[0]), gl_lo(w[1]), gl_hi(w[1])};
    *b = gl_f4{gl_lo(w[2]), gl_hi(w[2]), gl_lo(w[3]), gl_hi(w[3])};
  }
  // A factor of token pairs keeps its two parts side by side, four columns of hi and the same of
  // lo, so that a lane writes and reads 16 bytes: one product over 32 k is 16 tokens' hi and lo
  // against the other operand twice.  Rows of 96, 160, 224 and 288 bytes (no conflicts, as above).
  typedef gl_b8 Block;
  static constexpr int kBlock = 32, kBlockPad = 16;
  static __device__ __forceinline__ void put(bf16* row, int cb, int g, const gl_f4& x) {
    const uint32_t a = gl_pack(x[0], x[1]), b = gl_pack(x[2], x[3]);
    *reinterpret_cast<gl_u4*>(row + 32 * cb + 8 * g) =
        gl_u4{a, b, gl_pack(x[0] - gl_lo(a), x[1] - gl_hi(a)), gl_pack(x[2] - gl_lo(b), x[3] - gl_hi(b))};
  }
  static __device__ __forceinline__ Block block(const Op& x, int half) {
    return half ? __builtin_shufflevector(x, x, 4, 5, 6, 7, 4, 5, 6, 7)
                : __builtin_shufflevector(x, x, 0, 1, 2, 3, 0, 1, 2, 3);
  }
  static __device__ __forceinline__ gl_f4 mma_factor(const Block& a, const bf16* row, int cb, int g, gl_f4 c) {
    const gl_b8 b = *reinterpret_cast<const gl_b8*>(row + 32 * cb + 8 * g);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // columns 16 cb + 4 g .. + 3 of a row, from a 16-byte read that two g share
  template <int D> static __device__ __forceinline__ gl_f4 row4(const bf16* row, int cb, int g) {
    const gl_u4 w = *reinterpret_cast<const gl_u4*>(row + 16 * cb + 8 * (g >> 1));
    return widen4(g & 1 ? gl_u2{w[2], w[3]} : gl_u2{w[0], w[1]});
  }
  typedef gl_u2 Four;
  static __device__ __forceinline__ Four load4(__amdgpu_buffer_rsrc_t src, int elem) {
    return __builtin_amdgcn_raw_buffer_load_b64(src, elem * 2, 0, 0);
  }
  static __device__ __forceinline__ gl_f4 widen4(const Four& w) {
    return gl_f4{gl_lo(w[0]), gl_hi(w[0]), gl_lo(w[1]), gl_hi(w[1])};
  }
  static __device__ __forceinline__ void store4(const gl_f4& x, __amdgpu_buffer_rsrc_t dst, int elem) {
    const gl_u2 y = {gl_pack(x[0], x[1]), gl_pack(x[2], x[3])};
    __builtin_amdgcn_raw_buffer_store_b64(y, dst, elem * 2, 0, 0);
  }
  template <int D> static __device__ __forceinline__ void put_vec(bf16* m, int vec, const gl_u4& x) {
    const int at = vec * 8;
    *reinterpret_cast<gl_u4*>(m + (at / D) * pitch<D>() + at % D) = x;
  }
};
// Blocks (ut, st), st <= ut, of 16 tokens each in a chunk's triangle of token pairs, in order.
constexpr int kBlocks = 10;
__device__ __forceinline__ int block_row(int t) { return t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0; }
// The blocks wv, wv + NW, ... of a wave, two at a time where there are two, so that one's LDS reads
// and products run under the other's: f(n, first), n blocks first, first + NW.
template <int NW, typename F>
__device__ __forceinline__ void wave_blocks(int wv, F f) {
  constexpr int kAll = kBlocks / NW;  // of every wave
#pragma unroll
  for (int i = 0; i + 2 <= kAll; i += 2) f(std::integral_constant<int, 2>(), wv + i * NW);
  if constexpr (kAll % 2) f(std::integral_constant<int, 1>(), wv + (kAll - 1) * NW);
  if constexpr (kBlocks % NW) {
    if (wv < kBlocks % NW) f(std::integral_constant<int, 1>(), wv + kAll * NW);
  }
}

template <typename IO, int D>
struct Shape {
  typedef typename Math<IO>::Elem Elem;
  static constexpr int kNW = D / 16;                           // waves
  static constexpr int kNP = D / 32 > 0 ? D / 32 : 1;          // blocks of 32 features
  static constexpr bool kHalf = D == 16;
  static constexpr int kLd = Math<IO>::template pitch<D>();    // row pitch of a token tile
  static constexpr int kTile = kC * kLd;
  static constexpr int kFactor = 16 * (kBlocks * Math<IO>::kBlock + 4 * Math<IO>::kBlockPad);
};

// Row 16 t + r of a triangular factor: t + 1 blocks of 16 columns.
template <typename IO>
__device__ __forceinline__ typename Math<IO>::Elem* factor_row(typename Math<IO>::Elem* m, int t, int r) {
  constexpr int B = Math<IO>::kBlock, P = Math<IO>::kBlockPad;
  return m + 16 * (B * (t * (t + 1) / 2) + P * t) + r * (B * (t + 1) + P);
}

// tokens c0 .. of a tensor of D features, `rows` of them (none if negative)
template <int D, typename IO>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t token_span(const IO* base, long long c0, int rows) {
  return gl_span(base + c0 * D, max(0, min(kC, rows)) * D * static_cast<int>(sizeof(IO)));
}

// Loads.  A tile's registers are filled by buffer loads whose range ends at the last valid token
// (0 bytes for a chunk outside the segment), so every wave issues the same ones on every path.
// Loads and stores complete in order: a wait for a load issued before some stores need not wait for
// them, as long as their number is known.  So the stores of a chunk are the same on every path
// too (lanes or waves with nothing to store have an empty range), and `no_store` stands in for those
// of the chunk before the first.
template <typename IO, int D, int kThreads = 4 * D>
struct Tile {
  static constexpr int kVec = 4 * D * static_cast<int>(sizeof(IO)) / kThreads;  // 16-byte vectors a thread
  gl_u4 x[kVec];
  // tokens c0 .. of base, `rows` of them valid (may be negative)
  __device__ __forceinline__ void load(const IO* base, long long c0, int rows, int tid) {
    const __amdgpu_buffer_rsrc_t src = token_span<D>(base, c0, rows);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      x[i] = __builtin_amdgcn_raw_buffer_load_b128(src, (tid + i * kThreads) * 16, 0, 0);
  }
  __device__ __forceinline__ void put(typename Math<IO>::Elem* m, int tid) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) Math<IO>::template put_vec<D>(m, tid + i * kThreads, x[i]);
  }
};
__device__ __forceinline__ void store1(float x, __amdgpu_buffer_rsrc_t dst, int i) {
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), dst, i * 4, 0, 0);
}
template <int N>
__device__ __forceinline__ void no_store() {
#pragma unroll
  for (int i = 0; i < N; ++i) store1(0.0f, gl_span(nullptr, 0), 0);
}

// One sequence's view of the arguments.
struct Seq {
  int chain;
  size_t row0;  // first token
  int len;      // tokens that count
  const float* gate;
  const float* rate;
};
__device__ __forceinline__ Seq sequence(const GatedArgs& a, int chain) {
  Seq s;
  s.chain = chain;
  s.row0 = static_cast<size_t>(chain) * a.T;
  s.len = gl_length(a.lengths, chain / a.H, a.T);
  s.gate = a.gate ? a.gate + s.row0 : nullptr;
  s.rate = a.eta_tok ? a.eta_tok + s.row0 : nullptr;
  return s;
}
// log decays and rates of a chunk's tokens, lane = token (0, 0 past the sequence)
struct GateRate {
  float g, rate;
  __device__ __forceinline__ void load(const Seq& s, long long c0, int lane) {
    const int bytes = c0 < 0 || c0 >= s.len ? 0 : min(kC, static_cast<int>(s.len - c0)) * 4;
    g = load1(gl_span(s.gate + c0, s.gate ? bytes : 0), lane);
    rate = load1(gl_span(s.rate + c0, s.rate ? bytes : 0), lane);
  }
  __device__ __forceinline__ void decays(const Seq& s, float eta, long long c0, GlDecays* d, int lane) const {
    gl_decays(g, s.rate ? eta * rate : eta, c0 >= 0 && c0 + lane < s.len, d, lane);
  }
  static __device__ __forceinline__ float load1(__amdgpu_buffer_rsrc_t src, int i) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b32(src, i * 4, 0, 0)));
  }
};
__device__ __forceinline__ const float* initial_state(const GatedArgs& a, int chain, int dd) {
  return a.w0 + (chain / a.H) * a.w0_batch_stride + static_cast<size_t>(chain % a.H) * dd;
}

// A state in registers: row 4 g + e of tile b and column r of wave wv are the elements (f + e,
// 16 wv + r), f = state_row(b, g), of W, or of W^T (kTransposed).
template <typename IO, int D, bool kTransposed>
__device__ __forceinline__ void load_state(gl_f4* x, const float* w, int wv, int g, int r) {
#pragma unroll
  for (int b = 0; b < D / 16; ++b) {
    const int f = Math<IO>::template state_row<D>(b, g);
    if constexpr (kTransposed) {
      x[b] = w ? at4(w, (16 * wv + r) * D + f) : gl_f4{0.0f, 0.0f, 0.0f, 0.0f};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[b][e] = w ? w[(f + e) * D + 16 * wv + r] : 0.0f;
    }
  }
}
template <typename IO, int D>
__device__ __forceinline__ void store_state_transposed(const gl_f4* x, float* w, int wv, int g, int r) {
#pragma unroll
  for (int b = 0; b < D / 16; ++b)
    *reinterpret_cast<gl_f4*>(w + (16 * wv + r) * D + Math<IO>::template state_row<D>(b, g)) = x[b];
}

// x <- whole x + sum over the chunk's tokens s of a_s c_s b_s^T, a the rows of the tile A, b the
// wave's 16 columns (k down the tokens).
template <typename IO, int D, int N>
__device__ __forceinline__ void update_state(gl_f4* x, float whole, const typename Math<IO>::Elem* A,
                                             const typename Math<IO>::Op* b, const float* c, int g, int r) {
  typedef Math<IO> M;
  whole = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, whole)));
  if (whole == 0.0f) {
#pragma unroll
    for (int ab = 0; ab < D / 16; ++ab) x[ab] = gl_f4{0.0f, 0.0f, 0.0f, 0.0f};
  } else {
#pragma unroll
    for (int ab = 0; ab < D / 16; ++ab) x[ab] *= whole;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    gl_f4 lo, hi;
    M::widen(b[p], &lo, &hi);
    lo *= at4(c, 32 * p + 4 * g);
    hi *= at4(c, 32 * p + 16 + 4 * g);
    const typename M::template Parts<N> f = M::template split<N>(lo, hi);
#pragma unroll
    for (int ab = 0; ab < D / 16; ++ab)
      x[ab] = M::template mma_cols<N, false>(M::template down_state<D>(A, Shape<IO, D>::kLd, p, ab, g, r), f, x[ab]);
  }
}
// the state as an operand: parts over blocks of 32 rows
template <typename IO, int D, int N>
__device__ __forceinline__ void split_state(typename Math<IO>::template Parts<N>* y, const gl_f4* x) {
#pragma unroll
  for (int p = 0; p < Shape<IO, D>::kNP; ++p)
    y[p] = Math<IO>::template split<N>(
        x[2 * p], Shape<IO, D>::kHalf ? gl_f4{0.0f, 0.0f, 0.0f, 0.0f} : x[Shape<IO, D>::kHalf ? 0 : 2 * p + 1]);
}
// rows of the state times a token's row: C[16 rows][16 tokens]
template <typename IO, int D, int N>
__device__ __forceinline__ gl_f4 state_times(const typename Math<IO>::template Parts<N>* w,
                                             const typename Math<IO>::Elem* row, int g) {
  typedef Shape<IO, D> S;
  gl_f4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int p = 0; p < S::kNP; ++p)
    c = Math<IO>::template mma_rows<N, S::kHalf>(w[p], Math<IO>::template along<S::kHalf>(row, p, g), c);
  return c;
}
// C[16 tokens of a][16 tokens of b]: products of rows
template <typename IO, int D>
__device__ __forceinline__ gl_f4 row_products(const typename Math<IO>::Elem* a, const typename Math<IO>::Elem* b,
                                              int g) {
  typedef Math<IO> M;
  typedef Shape<IO, D> S;
  gl_f4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int p = 0; p < S::kNP; ++p)
    c = M::template mma<S::kHalf>(M::template along<S::kHalf>(a, p, g), M::template along<S::kHalf>(b, p, g), c);
  return c;
}

// ---------------------------------------------------------------- segments
//
// What a segment adds to the state from zero.  Side 0: sum over its tokens s of (decay to the
// segment's end) e_s v_s k_s^T, for the states.  Side 1 (backward): sum over its tokens u of
// (decay from the segment's start) dz_u q_u^T, for the states' gradients.
// Bound by the loads' latency: 768 workgroups of 4 chunks read K and V of 8 x 12 x 2048 tokens (d = 64,
// bf16) in 15 us, 2.9 TB/s of them.
template <typename IO, int D>
struct SumsLds {
  typename Math<IO>::Elem a[Shape<IO, D>::kTile], b[Shape<IO, D>::kTile];
  GlDecays dec[2];  // of this chunk and the next
};

template <typename IO, int D>
__global__ __launch_bounds__(4 * D) void gl_sums_kernel(GatedArgs a) {
  typedef Math<IO> M;
  typedef Shape<IO, D> S;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  SumsLds<IO, D>& L = *reinterpret_cast<SumsLds<IO, D>*>(lds_raw);
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int chain = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg, side = blockIdx.y;
  // the last segment adds to no other's start, the first to no other's end
  if (seg == (side == 0 ? a.nseg - 1 : 0)) return;
  const Seq s = sequence(a, chain);
  const IO* rows = static_cast<const IO*>(side == 0 ? a.k : a.q) + s.row0 * D;
  const IO* cols = static_cast<const IO*>(side == 0 ? a.v : a.dz) + s.row0 * D;
  const int nchunks = (a.T + kC - 1) / kC, first = seg * a.spc, n = min(a.spc, nchunks - first);
  gl_f4 x[S::kNW];
#pragma unroll
  for (int i = 0; i < S::kNW; ++i) x[i] = gl_f4{0.0f, 0.0f, 0.0f, 0.0f};
  // what a chunk's step needs in registers: its tiles, and the gates of the chunk after it
  struct Set {
    Tile<IO, D> a, b;
    GateRate gr;
  } y;
  float all = 1.0f;
  auto chunk = [&](int i) { return side == 0 ? first + i : first + n - 1 - i; };
  auto fetch = [&](int i) {
    const long long c0 = static_cast<long long>(chunk(i)) * kC;
    y.gr.load(s, static_cast<long long>(chunk(i + 1)) * kC, lane);
    const int valid = i < n ? s.len - static_cast<int>(c0) : 0;
    y.a.load(rows, c0, valid, tid);
    y.b.load(cols, c0, valid, tid);
  };
  const bool decayer = wv == S::kNW - 1;  // the wave that forms the next chunk's decays
  {
    GateRate gr;
    gr.load(s, static_cast<long long>(chunk(0)) * kC, lane);
    fetch(0);
    if (decayer) gr.decays(s, a.eta, static_cast<long long>(chunk(0)) * kC, &L.dec[0], lane);
  }
  for (int i = 0; i < n; ++i) {
    gl_barrier();  // the previous chunk's tiles have been read
    y.a.put(L.a, tid);
    y.b.put(L.b, tid);
    const GateRate gr = y.gr;
    gl_barrier();
    fetch(i + 1);
    const GlDecays& dec = L.dec[i & 1];
    if (decayer && i + 1 < n)
      gr.decays(s, a.eta, static_cast<long long>(chunk(i + 1)) * kC, &L.dec[(i + 1) & 1], lane);
    typename M::Op b[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) b[p] = M::template down<D>(L.b, S::kLd, p, wv, g, r);
    const float whole = dec.whole[0];
    all *= whole;
    update_state<IO, D, 3>(x, whole, L.a, b, side == 0 ? dec.to_e : dec.from, g, r);
  }
  float* out = (side == 0 ? a.seg_w : a.seg_g) + static_cast<size_t>(blockIdx.x) * D * D;
  store_state_transposed<IO, D>(x, out, wv, g, r);
  if (tid == 0) a.seg_decay[static_cast<size_t>(side) * a.B * a.H * a.nseg + blockIdx.x] = all;
}

// The sums become the states at the segments' starts (side 0, first to last from w0) and the
// gradients at their ends (side 1, last to first from dw_out), in place.
// VEC elements a thread; the sums of kAhead segments are loaded before the first is used (one
// after another took 22 us on 16 sequences of 43 segments, eight at a time 9 us).
template <int D, int VEC>
__global__ __launch_bounds__(256) void gl_scan_kernel(GatedArgs a) {
  typedef float vec __attribute__((ext_vector_type(VEC)));
  constexpr int kAhead = 8, kPer = D * D / VEC;  // threads per sequence
  const int item = blockIdx.x * 256 + threadIdx.x;
  const int chain = item / kPer, at = item % kPer * VEC, side = blockIdx.y;
  if (chain >= a.B * a.H) return;
  const size_t seg0 = static_cast<size_t>(chain) * a.nseg;
  float* x = (side == 0 ? a.seg_w : a.seg_g) + seg0 * D * D + at;
  const float* decay = a.seg_decay + static_cast<size_t>(side) * a.B * a.H * a.nseg + seg0;
  const float* start = side == 0  ? initial_state(a, chain, D * D)
                       : a.dw_out ? a.dw_out + static_cast<size_t>(chain) * D * D
                                  : nullptr;
  vec state = 0.0f;
  if (start) state = *reinterpret_cast<const vec*>(start + at);
  for (int i0 = 0; i0 < a.nseg; i0 += kAhead) {
    vec sum[kAhead];
    float dec[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j, m = side == 0 ? i : a.nseg - 1 - i;
      sum[j] = 0.0f;
      dec[j] = 0.0f;
      if (i + 1 < a.nseg) {  // nothing follows the last
        sum[j] = *reinterpret_cast<const vec*>(x + static_cast<size_t>(m) * D * D);
        dec[j] = decay[m];
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j, m = side == 0 ? i : a.nseg - 1 - i;
      if (i < a.nseg) *reinterpret_cast<vec*>(x + static_cast<size_t>(m) * D * D) = state;
#pragma unroll
      for (int e = 0; e < VEC; ++e) state[e] = gl_keep(dec[j], state[e]) + sum[j][e];
    }
  }
}

// The state at the segment's start (side 0) or its gradient at the segment's end (side 1).
template <int D>
__device__ __forceinline__ const float* segment_state(const GatedArgs& a, int side, int chain, int seg) {
  if (a.nseg > 1) return (side == 0 ? a.seg_w : a.seg_g) + (static_cast<size_t>(chain) * a.nseg + seg) * (D * D);
  if (side == 0) return initial_state(a, chain, D * D);
  return a.dw_out ? a.dw_out + static_cast<size_t>(chain) * (D * D) : nullptr;
}

// ---------------------------------------------------------------- forward
//
// Three barriers a chunk: tiles free, tiles staged (the next ones' loads start here), P ready.  The
// next chunk's decays are formed by one wave while the others form P.  P's ten blocks of 16 x 16
// pairs are dealt to the waves, the rest splits by output features: V, the state and its update
// need no exchange.  Bound by HBM while three workgroups share a CU: 61 us on 16 sequences of 32749
// tokens (d = 64, bf16), 4.4 TB/s of q, k, v and z.
template <typename IO, int D>
struct FwdLds {
  typename Math<IO>::Elem q[Shape<IO, D>::kTile], k[Shape<IO, D>::kTile], v[Shape<IO, D>::kTile];
  typename Math<IO>::Elem p[Shape<IO, D>::kFactor];
  GlDecays dec[2];  // of this chunk and the next
};

template <typename IO, int D>
__global__ __launch_bounds__(4 * D) void gl_fwd_kernel(GatedArgs a) {
  typedef Math<IO> M;
  typedef Shape<IO, D> S;
  constexpr int NW = S::kNW, LD = S::kLd;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  FwdLds<IO, D>& L = *reinterpret_cast<FwdLds<IO, D>*>(lds_raw);
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int chain = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg, T = a.T;
  const Seq s = sequence(a, chain);
  const IO* q = static_cast<const IO*>(a.q) + s.row0 * D;
  const IO* k = static_cast<const IO*>(a.k) + s.row0 * D;
  const IO* v = static_cast<const IO*>(a.v) + s.row0 * D;
  IO* z = static_cast<IO*>(a.z) + s.row0 * D;
  const int nchunks = (T + kC - 1) / kC, first = seg * a.spc, end = min(nchunks, first + a.spc);

  gl_f4 w[NW];  // W^T: W's rows 16 wv + r
  load_state<IO, D, true>(w, segment_state<D>(a, 0, chain, seg), wv, g, r);
  // what a chunk's step needs in registers: its tiles, and the gates of the chunk after it
  struct Set {
    Tile<IO, D> q, k, v;
    GateRate gr;
  } y;
  auto fetch = [&](int c) {
    const long long c0 = static_cast<long long>(c) * kC;
    y.gr.load(s, c0 + kC, lane);
    const int valid = c < end ? s.len - static_cast<int>(c0) : 0;
    y.q.load(q, c0, valid, tid);
    y.k.load(k, c0, valid, tid);
    y.v.load(v, c0, valid, tid);
  };
  const bool decayer = wv == NW - 1;  // the wave that forms the next chunk's decays
  {
    GateRate gr;
    gr.load(s, static_cast<long long>(first) * kC, lane);
    fetch(first);
    no_store<4>();
    if (decayer) gr.decays(s, a.eta, static_cast<long long>(first) * kC, &L.dec[0], lane);
  }
  for (int c = first; c < end; ++c) {
    const int c0 = c * kC;
    const GlDecays& dec = L.dec[(c - first) & 1];
    gl_barrier();  // the previous chunk's tiles have been read
    y.q.put(L.q, tid);
    y.k.put(L.k, tid);
    y.v.put(L.v, tid);
    const GateRate gr = y.gr;
    gl_barrier();
    fetch(c + 1);
    if (decayer && c + 1 < end)
      gr.decays(s, a.eta, static_cast<long long>(c + 1) * kC, &L.dec[(c + 1 - first) & 1], lane);

    // P[u][s] = exp(b_u - b_s) e_s (q_u . k_s) for s <= u
    wave_blocks<NW>(wv, [&](auto n, int first_block) {
      constexpr int N = n.value;
      gl_f4 p[N];
      int ut[N], st[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        ut[i] = block_row(first_block + i * NW);
        st[i] = first_block + i * NW - ut[i] * (ut[i] + 1) / 2;
        p[i] = row_products<IO, D>(L.k + (16 * st[i] + r) * LD, L.q + (16 * ut[i] + r) * LD, g);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = 16 * ut[i] + r, s4 = 16 * st[i] + 4 * g;
        const float uh = dec.bh[u], ul = dec.bl[u];
        const gl_f4 sh = at4(dec.bh, s4), sl = at4(dec.bl, s4), e = at4(dec.e, s4);
#pragma unroll
        for (int x = 0; x < 4; ++x) p[i][x] *= gl_between(uh, ul, sh[x], sl[x]) * e[x];
        if (ut[i] == st[i]) {  // the diagonal: pairs s <= u only
#pragma unroll
          for (int x = 0; x < 4; ++x) p[i][x] = s4 + x <= u ? p[i][x] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) M::put(factor_row<IO>(L.p, ut[i], r), st[i], g, p[i]);
    });
    gl_barrier();

    typename M::Op vf[2];  // V, k down the tokens, the wave's features
#pragma unroll
    for (int p = 0; p < 2; ++p) vf[p] = M::template down<D>(L.v, LD, p, wv, g, r);
    typename M::template Parts<2> wp[S::kNP];
    split_state<IO, D, 2>(wp, w);
    const __amdgpu_buffer_rsrc_t dst = token_span<D>(z, c0, T - c0);
#pragma unroll
    for (int ut = 0; ut < 4; ++ut) {  // Z^T: rows j, columns u
      const int u = 16 * ut + r;
      const gl_f4 zi = state_times<IO, D, 2>(wp, L.q + u * LD, g);
      gl_f4 zp = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st <= ut; ++st)
        zp = M::mma_factor(M::block(vf[st / 2], st % 2), factor_row<IO>(L.p, ut, r), st, g, zp);
      M::store4(zp + keep4(dec.from[u], zi), dst, u * D + 16 * wv + 4 * g);
    }
    update_state<IO, D, 3>(w, dec.whole[0], L.k, vf, dec.to_e, g, r);
  }
  if (a.w_out && seg == a.nseg - 1)
    store_state_transposed<IO, D>(w, a.w_out + static_cast<size_t>(chain) * D * D, wv, g, r);
}

// ---------------------------------------------------------------- backward
//
// With G_t = dL/dW_t (before the decay into t - 1), G_t = a_{t+1} G_{t+1} + dz_t q_t^T:
//   dq_u = sum_{s <= u} exp(b_u - b_s) e_s (dz_u . v_s) k_s + exp(b_u) W^T dz_u,
//   dv_s = e_s x_s,  x_s = sum_{u >= s} exp(b_u - b_s) (q_u . k_s) dz_u + exp(b_C - b_s) G k_s,
//   dk_s = e_s (sum_{u >= s} exp(b_u - b_s) (dz_u . v_s) q_u + exp(b_C - b_s) G^T v_s),
//   de_s = v_s . x_s,
// W the state before the chunk, G the gradient at its end.  gl_dq_kernel walks a segment forward
// with W for dq, gl_dkv_kernel walks it backward with G for dk and dv.  So no state is stored on
// the way.
//
// dg_t = a_t <G_t, W_{t-1}> is the sum over the pairs (s, u), s < t <= u, of what token s
// contributes to output u.  With m_us = exp(b_u - b_s) e_s (q_u . k_s)(dz_u . v_s), per chunk:
//   dg_t = sum_{u >= t} (row_u - col_u) + sum_{u >= t} in_u + sum_{s < t} out_s + past,
//   row_u = sum_{s < u} m_us, col_s = sum_{u > s} m_us (pairs inside the chunk),
//   in_u = exp(b_u) dz_u . W q_u,  out_s = exp(b_C - b_s) e_s v_s . G k_s,  past = exp(b_C) <G, W>.
// Only the row - col sums cancel, over one chunk; nothing grows with the sequence.  `past` follows
// from <G, W> at the segment's end: past_c = <G, W>_end(c) - sum out, <G, W>_start(c) = past_c +
// sum in.  gl_dq_kernel leaves in_u and <G, W> at the segments' ends in the workspace, and
// gl_dkv_kernel, which comes after it, adds the rest as it walks the chunks backward.
//
// Two kernels rather than one with two kinds of workgroups: dk and dv want eight waves (each
// half keeps one orientation of G: as four waves with both, 114 us for all gradients of 8 x 12 x
// 2048 tokens, d = 64, bf16; as two kernels 42 + 56).  dq then needs no Q in LDS and three of its
// workgroups fit a CU.  42 us is 3.0 TB/s of its five tensors; the factors' parts and the products of
// two parts more than the forward pass, on three waves a SIMD, keep it from HBM's rate.
template <typename IO, int D>
struct DqLds {
  typedef Shape<IO, D> S;
  typename S::Elem k[S::kTile], v[S::kTile], z[S::kTile];
  typename S::Elem r[S::kFactor];
  float part[S::kNW][kC];  // in_u, the waves' shares
  GlDecays dec[2];         // of this chunk and the next
};

template <typename IO, int D>
__global__ __launch_bounds__(4 * D) void gl_dq_kernel(GatedArgs a) {
  typedef Math<IO> M;
  typedef Shape<IO, D> S;
  constexpr int NW = S::kNW, LD = S::kLd;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  DqLds<IO, D>& L = *reinterpret_cast<DqLds<IO, D>*>(lds_raw);
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int chain = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg, T = a.T;
  const Seq s = sequence(a, chain);
  const IO* q = static_cast<const IO*>(a.q) + s.row0 * D;
  const IO* k = static_cast<const IO*>(a.k) + s.row0 * D;
  const IO* v = static_cast<const IO*>(a.v) + s.row0 * D;
  const IO* dz = static_cast<const IO*>(a.dz) + s.row0 * D;
  IO* dq = static_cast<IO*>(a.dq) + s.row0 * D;
  const int nchunks = (T + kC - 1) / kC, first = seg * a.spc, end = min(nchunks, first + a.spc);
  float* in_o = a.ws_tok ? a.ws_tok + s.row0 : nullptr;

  // what a chunk's step needs in registers: its tiles, and the gates of the chunk after it
  struct Set {
    Tile<IO, D> k, v, z;
    GateRate gr;
  } y;
  auto fetch = [&](int c) {
    const long long c0 = static_cast<long long>(c) * kC;
    y.gr.load(s, c0 + kC, lane);
    const int valid = c < end ? s.len - static_cast<int>(c0) : 0;
    y.k.load(k, c0, valid, tid);
    y.v.load(v, c0, valid, tid);
    y.z.load(dz, c0, valid, tid);
  };
  const bool decayer = wv == NW - 1;  // the wave that forms the next chunk's decays
  // in_u of a chunk whose shares are in LDS, stored by wave 0 (c < first: nothing)
  auto flush = [&](int c) {
    float in = 0.0f;
    if (wv == 0) {
#pragma unroll
      for (int x = 0; x < NW; ++x) in += L.part[x][lane];
    }
    store1(in, gl_span(in_o + c * kC, in_o && wv == 0 && c >= first ? min(kC, T - c * kC) * 4 : 0), lane);
  };

  gl_f4 w[NW];  // W's columns 16 wv + r
  {
    GateRate gr;
    gr.load(s, static_cast<long long>(first) * kC, lane);
    fetch(first);
    no_store<5>();
    if (decayer) gr.decays(s, a.eta, static_cast<long long>(first) * kC, &L.dec[0], lane);
  }
  load_state<IO, D, false>(w, segment_state<D>(a, 0, chain, seg), wv, g, r);
  for (int c = first; c < end; ++c) {
    const int c0 = c * kC, turn = (c - first) & 1;
    const GlDecays& dec = L.dec[turn];
    gl_barrier();  // the previous chunk's tiles have been read, its sums are whole
    flush(c - 1);
    y.k.put(L.k, tid);
    y.v.put(L.v, tid);
    y.z.put(L.z, tid);
    const GateRate gr = y.gr;
    // the wave's features of Q, for in_u
    typename M::Four qu[4];
    const __amdgpu_buffer_rsrc_t qsrc = token_span<D>(q, c0, in_o ? s.len - c0 : 0);
#pragma unroll
    for (int ut = 0; ut < 4; ++ut) qu[ut] = M::load4(qsrc, (16 * ut + r) * D + 16 * wv + 4 * g);
    gl_barrier();
    fetch(c + 1);
    if (decayer && c + 1 < end) gr.decays(s, a.eta, static_cast<long long>(c + 1) * kC, &L.dec[turn ^ 1], lane);
    wave_blocks<NW>(wv, [&](auto n, int first_block) {
      constexpr int N = n.value;
      gl_f4 rd[N];
      int ut[N], st[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        ut[i] = block_row(first_block + i * NW);
        st[i] = first_block + i * NW - ut[i] * (ut[i] + 1) / 2;
        rd[i] = row_products<IO, D>(L.v + (16 * st[i] + r) * LD, L.z + (16 * ut[i] + r) * LD, g);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = 16 * ut[i] + r, s4 = 16 * st[i] + 4 * g;
        const float uh = dec.bh[u], ul = dec.bl[u];
        const gl_f4 sh = at4(dec.bh, s4), sl = at4(dec.bl, s4), e = at4(dec.e, s4);
#pragma unroll
        for (int x = 0; x < 4; ++x) rd[i][x] *= gl_between(uh, ul, sh[x], sl[x]) * e[x];
        if (ut[i] == st[i]) {  // the diagonal: pairs s <= u only
#pragma unroll
          for (int x = 0; x < 4; ++x) rd[i][x] = s4 + x <= u ? rd[i][x] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) M::put(factor_row<IO>(L.r, ut[i], r), st[i], g, rd[i]);
    });
    gl_barrier();
    typename M::Op kf[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) kf[p] = M::template down<D>(L.k, LD, p, wv, g, r);
    typename M::template Parts<3> wp[S::kNP];
    split_state<IO, D, 3>(wp, w);
    const __amdgpu_buffer_rsrc_t dst = token_span<D>(dq, c0, T - c0);
#pragma unroll
    for (int ut = 0; ut < 4; ++ut) {
      const int u = 16 * ut + r;
      const gl_f4 xi = keep4(dec.from[u], state_times<IO, D, 3>(wp, L.z + u * LD, g));
      gl_f4 xp = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st <= ut; ++st)
        xp = M::mma_factor(M::block(kf[st / 2], st % 2), factor_row<IO>(L.r, ut, r), st, g, xp);
      const float in = over_g(dot4(M::widen4(qu[ut]), xi));
      if (g == 0) L.part[wv][u] = in;
      M::store4(xi + xp, dst, u * D + 16 * wv + 4 * g);
    }
    update_state<IO, D, 3>(w, dec.whole[0], L.v, kf, dec.to_e, g, r);
  }
  gl_barrier();
  flush(end - 1);
  if (in_o) {  // <G, W> at the segment's end
    gl_f4 ge[NW];
    load_state<IO, D, false>(ge, segment_state<D>(a, 1, chain, seg), wv, g, r);
    double x = 0.0;
#pragma unroll
    for (int b = 0; b < NW; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) x += static_cast<double>(w[b][e]) * ge[b][e];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o, 64);
    if (lane == 0) a.ws_end[static_cast<size_t>(blockIdx.x) * NW + wv] = x;
  }
}

// Two waves for each 16 columns: one group has G^T's columns for dv, the other G's for dk.  Bound by
// the vector units (60 % of its time: splits, decays, the pairs' sums): 56 us at the size above, 2.7
// TB/s of its six tensors.
template <typename IO, int D>
struct DkvLds {
  typedef Shape<IO, D> S;
  typename S::Elem q[S::kTile], k[S::kTile], v[S::kTile], z[S::kTile];
  typename S::Elem p[S::kFactor], r[S::kFactor];  // P^T and R^T, the tiles of rows in reverse order
  float part[S::kNW][kC];  // v_s . G k_s to the chunk's end, the waves' shares
  float pairs[4][kC];      // col_s / e_s, the blocks' shares
  float rows[4][kC];       // row_u, the blocks' shares
  float diag[kC];          // m_ss / e_s
  GlDecays dec[2];         // of this chunk and the next
};

template <typename IO, int D>
__global__ __launch_bounds__(8 * D, 4) void gl_dkv_kernel(GatedArgs a) {
  typedef Math<IO> M;
  typedef Shape<IO, D> S;
  constexpr int NW = S::kNW, LD = S::kLd;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  DkvLds<IO, D>& L = *reinterpret_cast<DkvLds<IO, D>*>(lds_raw);
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wv = wave % NW;
  const bool dk_group = wave >= NW;
  const int chain = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg, T = a.T;
  const Seq s = sequence(a, chain);
  const IO* q = static_cast<const IO*>(a.q) + s.row0 * D;
  const IO* k = static_cast<const IO*>(a.k) + s.row0 * D;
  const IO* v = static_cast<const IO*>(a.v) + s.row0 * D;
  const IO* dz = static_cast<const IO*>(a.dz) + s.row0 * D;
  IO* out = static_cast<IO*>(dk_group ? a.dk : a.dv) + s.row0 * D;
  float* de_o = a.deta_tok ? a.deta_tok + s.row0 : nullptr;
  const int nchunks = (T + kC - 1) / kC, first = seg * a.spc, end = min(nchunks, first + a.spc);
  float* dg_o = a.dgate ? a.dgate + s.row0 : nullptr;
  const float* in_i = a.dgate ? a.ws_tok + s.row0 : nullptr;

  // what a chunk's step needs in registers: its tiles, and the gates of the chunk before it
  struct Set {
    Tile<IO, D, 8 * D> q, k, v, z;
    GateRate gr;
  } y;
  // what the per-token results of the chunk after it need: its in_u and gate
  float in_u, gate_u;
  auto fetch = [&](int c, int tid) {
    const int lane = tid & 63;
    const long long c0 = static_cast<long long>(c) * kC;
    y.gr.load(s, c0 - kC, lane);
    const int tokens = c >= first && dg_o ? min(kC, T - static_cast<int>(c0)) * 4 : 0;
    in_u = GateRate::load1(gl_span(in_i + c0, tokens), lane);
    gate_u = GateRate::load1(gl_span(s.gate + c0, tokens), lane);
    const int valid = c >= first ? s.len - static_cast<int>(c0) : 0;
    y.q.load(q, c0, valid, tid);
    y.k.load(k, c0, valid, tid);
    y.v.load(v, c0, valid, tid);
    y.z.load(dz, c0, valid, tid);
  };
  const bool decayer = wave == 2 * NW - 1;  // the wave that forms the next chunk's decays
  // The per-token results of a chunk, formed by one wave while the others work on the next chunk:
  // the shares are read from LDS before that chunk's may overwrite them.
  const bool teller = wave == (NW > 1 ? 2 * NW - 2 : 0);
  struct Told {
    float col, row, out, de, in, gate;
  };
  auto shares = [&](const float* es, float in, float gate, int lane) {
    Told t = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (!teller) return t;
    float o = 0.0f, col = 0.0f, row = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) o += L.part[i][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      row += i <= lane >> 4 ? L.rows[i][lane] : 0.0f;
      col += i >= lane >> 4 ? L.pairs[i][lane] : 0.0f;
    }
    const float e = es[lane];
    t.de = a.eta * (col + L.diag[lane] + o);
    t.col = e * col;
    t.out = e * o;
    t.row = row;
    t.in = in;
    t.gate = gate;
    return t;
  };
  double later = 0.0;  // <G, W> at the end of the chunk that is next to be told
  if (dg_o && teller) {
    const double* ends = a.ws_end + static_cast<size_t>(blockIdx.x) * NW;
#pragma unroll
    for (int i = 0; i < NW; ++i) later += ends[i];
  }
  auto tell = [&](const Told& t, int c, int lane) {  // c >= end: nothing
    const int c0 = c * kC, bytes = teller && c < end ? min(kC, T - c0) * 4 : 0;
    float dg = 0.0f;
    if (dg_o && teller && c < end) {
      const double suf = gl_prefix(static_cast<double>(t.row) - t.col + t.in);
      const double pre = gl_prefix(static_cast<double>(t.out));
      const double in = gl_prefix(static_cast<double>(t.in));
      const double past = later - __shfl(pre, 63, 64);
      const double from_here = __shfl(suf, 63, 64) - suf + (static_cast<double>(t.row) - t.col + t.in);
      later = past + __shfl(in, 63, 64);
      // a token that forgets everything (decay 0) takes no gradient
      const bool live = c0 + lane < s.len && __builtin_amdgcn_exp2f(t.gate * 1.44269504f) != 0.0f;
      dg = live ? static_cast<float>(from_here + (pre - t.out) + past) : 0.0f;
    }
    store1(c0 + lane < s.len ? t.de : 0.0f, gl_span(de_o + c0, de_o ? bytes : 0), lane);
    store1(dg, gl_span(dg_o + c0, dg_o ? bytes : 0), lane);
  };

  gl_f4 x[NW];  // G's rows 16 wv + r (dv) or its columns (dk)
  float last_in = 0.0f, last_gate = 0.0f;
  if (first < end) {
    GateRate gr;
    gr.load(s, static_cast<long long>(end - 1) * kC, lane);
    fetch(end - 1, tid);
    no_store<6>();
    if (decayer) gr.decays(s, a.eta, static_cast<long long>(end - 1) * kC, &L.dec[0], lane);
  }
  if (dk_group) load_state<IO, D, false>(x, segment_state<D>(a, 1, chain, seg), wv, g, r);
  else load_state<IO, D, true>(x, segment_state<D>(a, 1, chain, seg), wv, g, r);
  for (int c = end - 1; c >= first; --c) {
    // The lane's addresses are formed anew for every chunk: kept across the loop they would not
    // fit in the 128 registers that let two workgroups share a CU (and a spilled one's reload
    // waits for the tiles on their way).
    int here = threadIdx.x;
    __asm__ __volatile__("" : "+v"(here));
    const int tid = here, lane = tid & 63, g = lane >> 4, r = lane & 15;
    const int c0 = c * kC, turn = (end - 1 - c) & 1;
    const GlDecays& dec = L.dec[turn];
    gl_barrier();  // the previous chunk's tiles have been read, its sums are whole
    const Told told = shares(L.dec[turn ^ 1].e, last_in, last_gate, lane);
    last_in = in_u;
    last_gate = gate_u;
    y.q.put(L.q, tid);
    y.k.put(L.k, tid);
    y.v.put(L.v, tid);
    y.z.put(L.z, tid);
    const GateRate gr = y.gr;
    gl_barrier();
    tell(told, c + 1, lane);
    fetch(c - 1, tid);
    if (decayer && c > first) gr.decays(s, a.eta, static_cast<long long>(c - 1) * kC, &L.dec[turn ^ 1], lane);
    // rows s of P^T and R^T (decayed, without e_s)
    wave_blocks<2 * NW>(wave, [&](auto n, int first_block) {
      constexpr int N = n.value;
      gl_f4 p[N], rd[N];
      int ut[N], st[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        ut[i] = block_row(first_block + i * 2 * NW);
        st[i] = first_block + i * 2 * NW - ut[i] * (ut[i] + 1) / 2;
        p[i] = row_products<IO, D>(L.q + (16 * ut[i] + r) * LD, L.k + (16 * st[i] + r) * LD, g);
        rd[i] = row_products<IO, D>(L.z + (16 * ut[i] + r) * LD, L.v + (16 * st[i] + r) * LD, g);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int ss = 16 * st[i] + r, u4 = 16 * ut[i] + 4 * g;
        const float sh = dec.bh[ss], sl = dec.bl[ss], es = dec.e[ss];
        const gl_f4 uh = at4(dec.bh, u4), ul = at4(dec.bl, u4);
        float cs = 0.0f, dg = 0.0f;
        gl_f4 rows;
        if (ut[i] != st[i]) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float f = gl_between(uh[j], ul[j], sh, sl);
            p[i][j] *= f;
            const float m = p[i][j] * rd[i][j];
            rd[i][j] *= f;
            cs += m;
            rows[j] = m * es;
          }
        } else {  // the diagonal: pairs u >= s only
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float f = gl_between(uh[j], ul[j], sh, sl);
            const float m = p[i][j] * rd[i][j] * f, below = u4 + j > ss ? m : 0.0f;
            p[i][j] = u4 + j >= ss ? p[i][j] * f : 0.0f;
            rd[i][j] = u4 + j >= ss ? rd[i][j] * f : 0.0f;
            cs += below;
            dg += u4 + j == ss ? m : 0.0f;
            rows[j] = below * es;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) rows[j] = over_r(rows[j]);
        if (r == 0) *reinterpret_cast<gl_f4*>(&L.rows[st[i]][u4]) = rows;
        cs = over_g(cs);
        if (g == 0) L.pairs[ut[i]][ss] = cs;
        if (ut[i] == st[i]) {
          dg = over_g(dg);
          if (g == 0) L.diag[ss] = dg;
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        M::put(factor_row<IO>(L.p, 3 - st[i], r), ut[i] - st[i], g, p[i]);
        M::put(factor_row<IO>(L.r, 3 - st[i], r), ut[i] - st[i], g, rd[i]);
      }
    });
    gl_barrier();
    const __amdgpu_buffer_rsrc_t dst = token_span<D>(out, c0, T - c0);
    // rows: the tile that the state multiplies; near, far: the tiles of the state's update;
    // f: the chunk's factor; N: the state's parts
    auto rest = [&](auto n, const typename S::Elem* rows, const typename S::Elem* near, const typename S::Elem* far,
                    typename S::Elem* f) {
      constexpr int N = n.value;
      typename M::Op b[2];  // k down the tokens u, the wave's features
#pragma unroll
      for (int p = 0; p < 2; ++p) b[p] = M::template down<D>(near, LD, p, wv, g, r);
      typename M::template Parts<N> xp[S::kNP];
      split_state<IO, D, N>(xp, x);
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        const int ss = 16 * st + r;
        const gl_f4 xi = keep4(dec.to[ss], state_times<IO, D, N>(xp, rows + ss * LD, g));
        gl_f4 xc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ut = st; ut < 4; ++ut)
          xc = M::mma_factor(M::block(b[ut / 2], ut % 2), factor_row<IO>(f, 3 - st, r), ut - st, g, xc);
        if constexpr (N == 3) {  // dv
          const float o = over_g(dot4(M::template row4<D>(L.v + ss * LD, wv, g), xi));
          if (g == 0) L.part[wv][ss] = o;
        }
        M::store4(dec.e[ss] * (xi + xc), dst, ss * D + 16 * wv + 4 * g);
      }
      update_state<IO, D, N>(x, dec.whole[0], far, b, dec.from, g, r);
    };
    if (dk_group) rest(std::integral_constant<int, 2>(), L.v, L.q, L.z, L.r);
    else rest(std::integral_constant<int, 3>(), L.k, L.z, L.q, L.p);
  }
  if (first < end) {
    gl_barrier();
    tell(shares(L.dec[(end - 1 - first) & 1].e, last_in, last_gate, lane), first, lane);
  }
  if (seg == 0 && !dk_group) store_state_transposed<IO, D>(x, a.dw0 + static_cast<size_t>(chain) * D * D, wv, g, r);
}

// ---------------------------------------------------------------- host

// Chunks per segment: the number of segments that takes the fewest rounds of chunks, where `slots`
// workgroups run at once (forward three a CU, backward two) and each spends about kStart chunks'
// time before its first.  All kernels of a call, d = 64, bf16, at 256, 512, 768, 1024 and 1536 slots:
//   forward, 96 sequences of 32 chunks: 65, 49, 47, 48, 56 us; 16 of 512: 126, 105, 107, 113, 123;
//   backward, 96 of 32: 151, 130, 133, 133, 156; 64 of 128: 318, 299, 312, 313, 346.
// `launches`: what the two further launches cost, in chunks: 12 sequences of 256 tokens take 15 us
// in one segment and 22 us in four, of 512 tokens the same 22 us.
void plan(GatedArgs* a, bool bwd) {
  constexpr int kStart = 2;
  const int launches = bwd ? 1 : 3;  // chunks' time that the two more launches take
  const int slots = bwd ? 512 : 768;
  const long long nchunks = (a->T + kC - 1) / kC, chains = static_cast<long long>(a->B) * a->H;
  long long best = -1;
  a->spc = 1;
  a->nseg = 1;
  for (long long n = 1; n <= nchunks && n <= 512; ++n) {
    const long long spc = (nchunks + n - 1) / n, nseg = (nchunks + spc - 1) / spc;
    if (nseg < n) continue;  // as many segments come from a smaller n
    const long long cost = (chains * nseg + slots - 1) / slots * (spc + kStart) + (nseg > 1 ? launches : 0);
    if (best < 0 || cost < best) {
      best = cost;
      a->spc = static_cast<int>(spc);
      a->nseg = static_cast<int>(nseg);
    }
    if (chains * nseg > 4 * slots) break;
  }
}

template <typename F>
hipError_t allow_lds(F fn, int bytes) {
  if (bytes <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename IO, int D>
hipError_t segment_states(const GatedArgs& a, int sides, hipStream_t s) {
  if (a.nseg == 1) return hipSuccess;
  const int chains = a.B * a.H;
  constexpr int bytes = sizeof(SumsLds<IO, D>);
  const auto fn = gl_sums_kernel<IO, D>;
  hipError_t e = allow_lds(fn, bytes);
  if (e != hipSuccess) return e;
  fn<<<dim3(chains * a.nseg, sides), dim3(4 * D), bytes, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  // four elements a thread once that still fills the chip (256 CUs of 2048 threads)
  const long long quads = static_cast<long long>(chains) * (D * D / 4) * sides;
  const unsigned groups = static_cast<unsigned>((quads / sides + 255) / 256);
  if (quads >= 256 * 512) gl_scan_kernel<D, 4><<<dim3(groups, sides), dim3(256), 0, s>>>(a);
  else gl_scan_kernel<D, 1><<<dim3(chains * (D * D / 256), sides), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <typename IO, int D>
hipError_t fwd(const GatedArgs& a, hipStream_t s) {
  const auto fn = gl_fwd_kernel<IO, D>;
  constexpr int bytes = sizeof(FwdLds<IO, D>);
  hipError_t e = allow_lds(fn, bytes);
  if (e == hipSuccess) e = segment_states<IO, D>(a, 1, s);
  if (e != hipSuccess) return e;
  fn<<<dim3(a.B * a.H * a.nseg), dim3(4 * D), bytes, s>>>(a);
  return hipGetLastError();
}

template <typename IO, int D>
hipError_t bwd(const GatedArgs& a, hipStream_t s) {
  const auto dq = gl_dq_kernel<IO, D>;
  const auto dkv = gl_dkv_kernel<IO, D>;
  constexpr int dq_bytes = sizeof(DqLds<IO, D>), dkv_bytes = sizeof(DkvLds<IO, D>);
  hipError_t e = allow_lds(dq, dq_bytes);
  if (e == hipSuccess) e = allow_lds(dkv, dkv_bytes);
  if (e == hipSuccess) e = segment_states<IO, D>(a, 2, s);
  if (e != hipSuccess) return e;
  const int groups = a.B * a.H * a.nseg;
  if (a.T > 0) dq<<<dim3(groups), dim3(4 * D), dq_bytes, s>>>(a);
  dkv<<<dim3(groups), dim3(8 * D), dkv_bytes, s>>>(a);
  e = hipGetLastError();
  return e;
}

// The workspace: [ends, doubles][state sums][gradient sums][decays][in_u per token], each part
// only where the call needs it; every part but the last is a multiple of 16 bytes.
size_t carve(GatedArgs* a, int d, bool bwd, bool gated, void* ws) {
  plan(a, bwd);
  const size_t segs = static_cast<size_t>(a->B) * a->H * a->nseg, dd = static_cast<size_t>(d) * d;
  unsigned char* p = static_cast<unsigned char*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    unsigned char* q = p ? p + at : nullptr;
    at += (bytes + 15) / 16 * 16;
    return q;
  };
  if (gated) a->ws_end = reinterpret_cast<double*>(take(segs * (d / 16) * sizeof(double)));
  if (a->nseg > 1) {
    a->seg_w = reinterpret_cast<float*>(take(segs * dd * sizeof(float)));
    if (bwd) a->seg_g = reinterpret_cast<float*>(take(segs * dd * sizeof(float)));
    a->seg_decay = reinterpret_cast<float*>(take(2 * segs * sizeof(float)));
  }
  if (gated) a->ws_tok = reinterpret_cast<float*>(take(static_cast<size_t>(a->B) * a->H * a->T * sizeof(float)));
  return at;
}

}  // namespace

size_t gated_fwd_workspace_bytes(int B, int H, int T, int d, bool) {
  GatedArgs a{};
  a.B = B;
  a.H = H;
  a.T = T;
  return carve(&a, d, false, false, nullptr);
}

size_t gated_bwd_workspace_bytes(int B, int H, int T, int d, bool gated, bool) {
  GatedArgs a{};
  a.B = B;
  a.H = H;
  a.T = T;
  return carve(&a, d, true, gated, nullptr);
}

hipError_t launch_gated_fwd(GatedArgs a, int d, bool bf16_io, void* ws, hipStream_t s) {
  carve(&a, d, false, false, ws);
  if (bf16_io) return d == 16 ? fwd<bf16, 16>(a, s) : d == 32 ? fwd<bf16, 32>(a, s) : fwd<bf16, 64>(a, s);
  return d == 16 ? fwd<float, 16>(a, s) : d == 32 ? fwd<float, 32>(a, s) : fwd<float, 64>(a, s);
}

hipError_t launch_gated_bwd(GatedArgs a, int d, bool bf16_io, void* ws, hipStream_t s) {
  carve(&a, d, true, a.dgate != nullptr, ws);
  if (bf16_io) return d == 16 ? bwd<bf16, 16>(a, s) : d == 32 ? bwd<bf16, 32>(a, s) : bwd<bf16, 64>(a, s);
  return d == 16 ? bwd<float, 16>(a, s) : d == 32 ? bwd<float, 32>(a, s) : bwd<float, 64>(a, s);
}

}  // namespace ttt
