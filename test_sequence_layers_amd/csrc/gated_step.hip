// One token of the gated linear recurrence for every sequence, the states updated in place:
//   W <- a W + e v k^T,  z = W q,  a = exp(g),  e = eta eta_tok.
// Each state is read once and written once (2 d^2 floats a head); everything else is small, so
// the kernel is bound by that traffic: 512 x 12 states of 64 x 64 in 38.5 us, 5.3 TB/s.  A thread holds
// four consecutive columns of its rows and a row is spread over d / 4 neighbouring lanes, so that a
// wave's loads and stores are 1 KB in a row and z's sum over the columns stays within a row of lanes.
#include "gated_linear.hpp"

namespace ttt {
namespace {

template <typename IO> __device__ __forceinline__ gl_f4 load4(const IO* p);
template <> __device__ __forceinline__ gl_f4 load4<float>(const float* p) { return *reinterpret_cast<const gl_f4*>(p); }
template <> __device__ __forceinline__ gl_f4 load4<bf16>(const bf16* p) {
  const gl_u2 x = *reinterpret_cast<const gl_u2*>(p);
  return gl_f4{__builtin_bit_cast(float, x[0] << 16), __builtin_bit_cast(float, x[0] & 0xFFFF0000u),
               __builtin_bit_cast(float, x[1] << 16), __builtin_bit_cast(float, x[1] & 0xFFFF0000u)};
}

template <typename IO, int D>
__global__ __launch_bounds__(256) void gl_step_kernel(GatedArgs a, float* w) {
  constexpr int kPer = D * D / 4 < 256 ? D * D / 4 : 256;  // threads per state
  constexpr int kRows = kPer / (D / 4);                    // rows they hold at once
  const int chain = blockIdx.x * (256 / kPer) + threadIdx.x / kPer;
  if (chain >= a.B * a.H) return;  // whole groups of D / 4 lanes
  const int tid = threadIdx.x % kPer, col = 4 * (tid % (D / 4)), row = tid / (D / 4);
  const size_t tok = static_cast<size_t>(chain) * D;
  float* wc = w + static_cast<size_t>(chain) * D * D + row * D + col;
  gl_f4 x[D / kRows];
#pragma unroll
  for (int i = 0; i < D / kRows; ++i) x[i] = *reinterpret_cast<const gl_f4*>(wc + i * kRows * D);
  const gl_f4 q = load4(static_cast<const IO*>(a.q) + tok + col), k = load4(static_cast<const IO*>(a.k) + tok + col);
  float decay = 1.0f;
  if (a.gate) {
    double g = static_cast<double>(a.gate[chain]) * 1.4426950408889634;
    if (g < kGlLeast) g = kGlNever;
    decay = __builtin_amdgcn_exp2f(static_cast<float>(g));
  }
  const float e = a.eta_tok ? a.eta * a.eta_tok[chain] : a.eta;
  const IO* v = static_cast<const IO*>(a.v) + tok + row;
  IO* z = static_cast<IO*>(a.z) + tok + row;
#pragma unroll
  for (int i = 0; i < D / kRows; ++i) {
    const float ev = e * to_f32(v[i * kRows]);
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[i][c] = gl_keep(decay, x[i][c]) + ev * k[c];
      sum += x[i][c] * q[c];
    }
    *reinterpret_cast<gl_f4*>(wc + i * kRows * D) = x[i];
    sum = gl_lane_sum<D / 4>(sum);
    if (col == 0) z[i * kRows] = from_f32<IO>(sum);
  }
}

template <typename IO, int D>
hipError_t step(const GatedArgs& a, float* w, hipStream_t s) {
  constexpr int per_block = D * D / 4 < 256 ? 256 / (D * D / 4) : 1;
  gl_step_kernel<IO, D><<<dim3((a.B * a.H + per_block - 1) / per_block), dim3(256), 0, s>>>(a, w);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_step(const GatedArgs& a, float* w, int d, bool bf16_io, hipStream_t s) {
  if (bf16_io) return d == 16 ? step<bf16, 16>(a, w, s) : d == 32 ? step<bf16, 32>(a, w, s) : step<bf16, 64>(a, w, s);
  return d == 16 ? step<float, 16>(a, w, s) : d == 32 ? step<float, 32>(a, w, s) : step<float, 64>(a, w, s);
}

}  // namespace ttt
