// Shared pieces of the gated linear recurrence's kernels (gated_linear*.hip):
//
//   W_t = a_t W_{t-1} + e_t v_t k_t^T,  z_t = W_t q_t,  a_t = exp(g_t),  e_t = eta eta_tok[t],
//
// taken kGlChunk tokens at a time.  With b_u = sum of g from the chunk's start through token u,
// W the state before the chunk and C its last token:
//   z_u   = sum_{s <= u} exp(b_u - b_s) e_s (q_u . k_s) v_s + exp(b_u) W q_u,
//   W_end = exp(b_C) W + sum_s exp(b_C - b_s) e_s v_s k_s^T.
#pragma once

#include "common.hpp"

namespace ttt {

constexpr int kGlChunk = 64;             // tokens per chunk
constexpr int kGlPitch = kGlChunk + 4;   // row pitch (floats) of matrices with a column per token

// The decays of one chunk in LDS, one entry per token.
struct GlDecays {
  float bh[kGlChunk], bl[kGlChunk];  // b_u / ln 2 as the sum of two floats
  float e[kGlChunk];                 // e_s (0 past the sequence)
  float from[kGlChunk];              // exp(b_u): from the chunk's start (0 past the sequence)
  float to[kGlChunk];                // exp(b_C - b_s): to the chunk's end (0 past the sequence)
  float to_e[kGlChunk];              // the same times e_s
  float whole[4];                    // exp(b_C) (first entry)
};

// Base-2 logarithms below kGlLeast, whose decays float32 flushes to 0, count as kGlNever: whatever
// growth (g > 0) follows in the chunk does not bring back what they drop, and sums over a
// chunk stay below 2^18, so that two floats hold them to 2^-29 and tokens after a forgotten one (g =
// -inf, or the type's lowest value) keep exact differences.
constexpr double kGlLeast = -126.0, kGlNever = -4096.0;

// two floats rounded to bf16 in one word, and the floats that a word holds
__device__ __forceinline__ uint32_t gl_pack(float lo, float hi) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{lo, hi}, b2));
}
__device__ __forceinline__ float gl_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float gl_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

// x of the lane `kCtrl` names (row_shr within 16 lanes, or the broadcast of a row's last lane to
// the rows of the mask), 0 where there is none
template <int kCtrl, int kRows>
__device__ __forceinline__ double gl_dpp(double x) {
  typedef int pair __attribute__((ext_vector_type(2)));
  pair y = __builtin_bit_cast(pair, x);
  const int lo = __builtin_amdgcn_update_dpp(0, y[0], kCtrl, kRows, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, y[1], kCtrl, kRows, 0xF, false);
  return __builtin_bit_cast(double, pair{lo, hi});
}

// sum over the lanes up to and with this one
__device__ __forceinline__ double gl_prefix(double x) {
  x += gl_dpp<0x111, 0xF>(x);  // row_shr 1, 2, 4, 8: sums of 16 lanes
  x += gl_dpp<0x112, 0xF>(x);
  x += gl_dpp<0x114, 0xF>(x);
  x += gl_dpp<0x118, 0xF>(x);
  x += gl_dpp<0x142, 0xA>(x);  // row_bcast 15 into rows 1 and 3, row_bcast 31 into rows 2 and 3
  x += gl_dpp<0x143, 0xC>(x);
  return x;
}

// One wave, lane = token: g is the token's log decay (0 past the sequence), `live` whether it is
// one of the sequence's: no state reaches the others, whatever it holds.  The prefix sum runs in 64
// bits: b_u - b_s is a small difference of sums that may be large.
__device__ __forceinline__ void gl_decays(float g, float e, bool live, GlDecays* d, int lane) {
  double x = static_cast<double>(g) * 1.4426950408889634;
  if (x < kGlLeast) x = kGlNever;  // a NaN stays one
  x = gl_prefix(x);
  const double last = __shfl(x, kGlChunk - 1, 64);
  const float h = static_cast<float>(x), to = live ? __builtin_amdgcn_exp2f(static_cast<float>(last - x)) : 0.0f;
  e = live ? e : 0.0f;
  d->bh[lane] = h;
  d->bl[lane] = static_cast<float>(x - h);
  d->e[lane] = e;
  d->from[lane] = live ? __builtin_amdgcn_exp2f(h) : 0.0f;
  d->to[lane] = to;
  d->to_e[lane] = to * e;
  if (lane == 0) d->whole[0] = __builtin_amdgcn_exp2f(static_cast<float>(last));
}

// exp(b_u - b_s)
__device__ __forceinline__ float gl_between(float uh, float ul, float sh, float sl) {
  return __builtin_amdgcn_exp2f((uh - sh) + (ul - sl));
}

// f x, with what a decay of 0 drops left out whatever it is (a state that is not finite too)
__device__ __forceinline__ float gl_keep(float f, float x) { return f == 0.0f ? 0.0f : f * x; }

typedef float gl_f4 __attribute__((ext_vector_type(4)));
typedef uint32_t gl_u2 __attribute__((ext_vector_type(2)));
typedef uint32_t gl_u4 __attribute__((ext_vector_type(4)));

// x plus the other half's (the neighbouring row's) x: v_permlane32_swap and v_permlane16_swap of x
// with itself leave the two values side by side in two registers
__device__ __forceinline__ float gl_swap32(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto y = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a = y[0], b = y[1];
  return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}
__device__ __forceinline__ float gl_swap16(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto y = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t a = y[0], b = y[1];
  return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}
template <int kCtrl>
__device__ __forceinline__ float gl_lane(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kCtrl, 0xF, 0xF, false));
}
// Sum over aligned groups of W lanes (a power of two), in every lane, without LDS: neighbours by
// quad_perm, then the mirrored half row and row (their lanes hold equal sums), then swaps.
template <int W>
__device__ __forceinline__ float gl_lane_sum(float x) {
  if constexpr (W >= 2) x += gl_lane<0xB1>(x);
  if constexpr (W >= 4) x += gl_lane<0x4E>(x);
  if constexpr (W >= 8) x += gl_lane<0x141>(x);
  if constexpr (W >= 16) x += gl_lane<0x140>(x);
  if constexpr (W >= 32) x = gl_swap16(x);
  if constexpr (W >= 64) x = gl_swap32(x);
  return x;
}

// Sum over the lanes of a wave that are equal modulo W, in every lane: rotations within the row of
// 16, then swaps.
template <int W>
__device__ __forceinline__ float gl_stride_sum(float x) {
  if constexpr (W <= 2) x += gl_lane<0x122>(x);
  if constexpr (W <= 4) x += gl_lane<0x124>(x);
  if constexpr (W <= 8) x += gl_lane<0x128>(x);
  if constexpr (W <= 16) x = gl_swap16(x);
  if constexpr (W <= 32) x = gl_swap32(x);
  return x;
}

// Loads and stores through buffer resources whose range ends at the last valid token: rows
// past it read as zero and their stores are dropped.  The range is the same in every lane; said
// so, it stays in scalar registers (else each access is wrapped in a loop over the lanes' values).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t gl_span(const void* base, int bytes) {
  bytes = __builtin_amdgcn_readfirstlane(bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes > 0 ? bytes : 0, 0x00020000);
}

// Workgroup barrier for LDS traffic: this wave's LDS accesses are complete, then all waves
// meet.  Global loads and stores stay in flight (waves exchange data through LDS only).
__device__ __forceinline__ void gl_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0), vmcnt/expcnt unconstrained
  __asm__ __volatile__("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  __asm__ __volatile__("" ::: "memory");
}

// tokens of a sequence: lengths[b] held to [0, T], or T
__device__ __forceinline__ int gl_length(const int* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace ttt
