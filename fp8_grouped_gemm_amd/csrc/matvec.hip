// Products of a few rows with 4-bit weights and group scales, and the combine of the
// experts' outputs.  Codes and packing are moe.h's MOE_INT4 (block-wise 4-bit weights with
// max-abs scales, DeepSeek-V4 lecture, tqpw.cn sec. 3.1), one scale per 32, 64 or 128
// weights of a row.
//
// One wave per (slot, output column): lanes stride over the row's words of 8 codes, each
// word's integer products are summed in fp32 and scaled once.
#include "common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

__device__ __forceinline__ void store_out(void* y, size_t i, float v, bool bf16) {
  if (bf16)
    static_cast<__bf16*>(y)[i] = (__bf16)v;              // round to nearest even, NaN kept
  else
    static_cast<float*>(y)[i] = v;
}

struct MatvecArgs {
  const void* x;
  int x_div;
  const uint8_t* q;
  const float* s7;
  int group;
  const int32_t* idx;
  int G, N, K;
  void* y;
  bool y_bf16;
};

// code word w times x[0..8)
template <bool XBF16>
__device__ __forceinline__ float dot8(uint32_t w, const void* x, size_t at) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t nib = w >> (8 * (i & 3) + 4 * (i >> 2));
    const float m = (float)(nib & 7u);
    const float v = XBF16 ? bf16_to_f32(static_cast<const uint16_t*>(x)[at + i])
                          : static_cast<const float*>(x)[at + i];
    s = fmaf((nib & 8u) ? -m : m, v, s);
  }
  return s;
}

}  // namespace

template <bool XBF16, bool SWIGLU>
__global__ __launch_bounds__(256) void matvec_int4_kernel(MatvecArgs a) {
  const int lane = threadIdx.x & 63;
  const int n = blockIdx.x * 4 + (threadIdx.x >> 6), s = blockIdx.y;
  if (n >= a.N) return;
  const int e = a.idx ? a.idx[s] : 0;
  if (e < 0 || e >= a.G) {
    if (lane == 0) store_out(a.y, (size_t)s * a.N + n, 0.f, a.y_bf16);
    return;
  }
  const int words = a.K / 8, KG = a.K / a.group, wpg = a.group / 8;
  const size_t rows = SWIGLU ? 2 * (size_t)a.N : a.N;
  const size_t x0 = (size_t)(s / a.x_div) * a.K;
  float v[2] = {0.f, 0.f};
#pragma unroll
  for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
    const size_t row = e * rows + (size_t)h * a.N + n;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) + row * words;
    const float* s7 = a.s7 + row * KG;
    for (int p = lane; p < words; p += 64)
      v[h] = fmaf(s7[p / wpg], dot8<XBF16>(q[p], a.x, x0 + (size_t)p * 8), v[h]);
    v[h] = group_sum<64>(v[h]);
  }
  if (lane == 0)
    store_out(a.y, (size_t)s * a.N + n, SWIGLU ? silu(v[0]) * v[1] : v[0], a.y_bf16);
}

__global__ __launch_bounds__(256) void few_combine_kernel(const float* __restrict__ o,
                                                          const int32_t* __restrict__ idx,
                                                          const float* __restrict__ w, int k,
                                                          int E, int d, void* __restrict__ y,
                                                          bool y_bf16) {
  const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  if (n >= d) return;
  float acc = 0.f;
  for (int j = 0; j < k; ++j) {
    const int s = t * k + j, e = idx[s];
    if (e >= 0 && e < E) acc = fmaf(w[s], o[(size_t)s * d + n], acc);
  }
  store_out(y, (size_t)t * d + n, acc, y_bf16);
}

hipError_t launch_matvec_int4(const void* x, bool x_bf16, int x_div, const uint8_t* q,
                              const float* s7, int group, const int32_t* idx, int S, int G, int N,
                              int K, bool swiglu, void* y, bool y_bf16, hipStream_t s) {
  const MatvecArgs a{x, x_div, q, s7, group, idx, G, N, K, y, y_bf16};
  const dim3 grid((unsigned)(((long)N + 3) / 4), (unsigned)S), block(256);
  if (x_bf16 && swiglu)
    hipLaunchKernelGGL((matvec_int4_kernel<true, true>), grid, block, 0, s, a);
  else if (x_bf16)
    hipLaunchKernelGGL((matvec_int4_kernel<true, false>), grid, block, 0, s, a);
  else if (swiglu)
    hipLaunchKernelGGL((matvec_int4_kernel<false, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((matvec_int4_kernel<false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_few_combine(const float* o, const int32_t* idx, const float* w, int T, int k,
                              int E, int d, void* y, bool y_bf16, hipStream_t s) {
  hipLaunchKernelGGL(few_combine_kernel, dim3((unsigned)((d + 255) / 256), (unsigned)T), dim3(256),
                     0, s, o, idx, w, k, E, d, y, y_bf16);
  return hipGetLastError();
}

}  // namespace moe
