// The training side of the router: load-balance loss with per-expert counts, and the
// gradient of the gate weights and of that loss with respect to the logits.
//
// p[t] = softmax(logits[t] + bias) (the router's biased softmax, MegaMoE walkthrough,
// discosf.com sec. 2.2, in fp32).  Per segment of n counting tokens, P_e = mean_t p[t, e]
// and f_e = counts_e / (k n); the loss is E sum f_e P_e or sum (P_e - 1/E)^2, so with
// g_e = dL/dp[t, e] every token's gradient is the softmax's, p_e (g_e - sum_i p_i g_i).
//
// One wave holds one token's E keys, KPL = ceil(E / 64) per lane.  Sums over tokens are
// taken per part of a segment in a fixed order and joined in fp64, without float atomics:
// the result does not depend on scheduling.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

constexpr int kMaxE = 1024;

// p of the row held as key[] (fp32 softmax; a row of -inf gives zeros, NaN stays NaN)
template <int KPL>
__device__ __forceinline__ void row_softmax(float (&p)[KPL]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < KPL; ++i) m = fmaxf(m, p[i]);
  m = group_max<64>(m);
  if (m == -INFINITY) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    p[i] = expf(p[i] - m);
    s += p[i];
  }
  s = group_sum<64>(s);
  const float inv = s == 0.f ? 0.f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < KPL; ++i) p[i] *= inv;
}

// keys of token t, -inf past E
template <int KPL>
__device__ __forceinline__ void load_keys(float (&key)[KPL], const float* logits,
                                          const float* bias, size_t t, int E, int lane) {
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < E ? logits[t * E + e] + (bias ? bias[e] : 0.f) : -INFINITY;
  }
}

// tokens [lo, hi) of segment b, held within [0, T] whatever the offsets are
__device__ __forceinline__ void segment(const int32_t* offsets, int b, int T, int& lo, int& hi) {
  lo = 0;
  hi = T;
  if (offsets) {
    lo = min(max(offsets[b], 0), T);
    hi = min(max(offsets[b + 1], lo), T);
  }
}

struct BalanceWs {
  float* psum;      // [B][parts][E] sums of p over a part's tokens
  int32_t* cnt;     // [B][parts][E] slots per expert
  int32_t* n;       // [B][parts] counting tokens
  double* lossb;    // [B] losses of the segments
};

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

BalanceWs balance_ws(void* ws, int T, int E, int B, size_t* total) {
  const size_t np = (size_t)B * balance_parts(T, B);
  uint8_t* p = static_cast<uint8_t*>(ws);
  BalanceWs w;
  size_t at = 0;
  w.psum = reinterpret_cast<float*>(p + at);
  at = up256(at + np * E * 4);
  w.cnt = reinterpret_cast<int32_t*>(p + at);
  at = up256(at + np * E * 4);
  w.n = reinterpret_cast<int32_t*>(p + at);
  at = up256(at + np * 4);
  w.lossb = reinterpret_cast<double*>(p + at);
  at = up256(at + (size_t)B * 8);
  *total = at;
  return w;
}

}  // namespace

template <int KPL>
__global__ __launch_bounds__(256) void balance_part_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ offsets, int T, int E, int k, BalanceWs ws) {
  __shared__ float red[4][64 * KPL];
  __shared__ int cnt[64 * KPL], nw[4];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int parts = gridDim.x, c = blockIdx.x, b = blockIdx.y;
  int lo, hi;
  segment(offsets, b, T, lo, hi);
  const int per = (int)(((long)hi - lo + parts - 1) / parts);
  const int t0 = (int)min((long)lo + (long)c * per, (long)hi), t1 = t0 + min(per, hi - t0);
  for (int e = tid; e < 64 * KPL; e += 256) cnt[e] = 0;
  __syncthreads();
  float acc[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) acc[i] = 0.f;
  int n = 0;
  for (int t = t0 + w; t < t1; t += 4) {
    if (mask && mask[t] == 0) continue;
    float p[KPL];
    load_keys(p, logits, bias, t, E, lane);
    row_softmax(p);
#pragma unroll
    for (int i = 0; i < KPL; ++i) acc[i] += p[i];
    if (lane < k) {
      const int e = idx[(size_t)t * k + lane];
      if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
    ++n;
  }
#pragma unroll
  for (int i = 0; i < KPL; ++i) red[w][lane + 64 * i] = acc[i];
  if (lane == 0) nw[w] = n;
  __syncthreads();
  const size_t part = (size_t)b * parts + c;
  for (int e = tid; e < E; e += 256) {
    ws.psum[part * E + e] = ((red[0][e] + red[1][e]) + red[2][e]) + red[3][e];
    ws.cnt[part * E + e] = cnt[e];
  }
  if (tid == 0) ws.n[part] = nw[0] + nw[1] + nw[2] + nw[3];
}

// sum over the 256 threads in a fixed order
template <typename V>
__device__ V block_sum(V v, V* red) {
  const int tid = threadIdx.x;
  red[tid] = v;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) red[tid] += red[tid + o];
    __syncthreads();
  }
  const V r = red[0];
  __syncthreads();
  return r;
}

__global__ __launch_bounds__(256) void balance_join_kernel(BalanceWs ws, int parts, int E, int k,
                                                           int B, bool square, float coef,
                                                           int32_t* __restrict__ counts,
                                                           float* __restrict__ probs,
                                                           float* __restrict__ grad,
                                                           float* __restrict__ loss) {
  __shared__ double red[256];
  __shared__ int redi[256];
  const int tid = threadIdx.x, b = blockIdx.x;
  // segments with counting tokens, and this one's
  int live = 0;
  for (int i = tid; i < B; i += 256) {
    int n = 0;
    for (int c = 0; c < parts; ++c) n |= ws.n[(size_t)i * parts + c];
    live += n != 0;
  }
  live = block_sum(live, redi);
  int n = 0;
  for (int c = tid; c < parts; c += 256) n += ws.n[(size_t)b * parts + c];
  n = block_sum(n, redi);
  double sum = 0., slots = 0.;
  for (int e = tid; e < E; e += 256) {
    double P = 0.;
    int m = 0;
    for (int c = 0; c < parts; ++c) {
      const size_t at = ((size_t)b * parts + c) * E + e;
      P += ws.psum[at];
      m += ws.cnt[at];
    }
    P = n ? P / n : 0.;
    counts[(size_t)b * E + e] = m;
    probs[(size_t)b * E + e] = (float)P;
    slots += m;
    if (n) {
      const double f = m / ((double)k * n), d = P - 1.0 / E;
      sum += square ? d * d : E * f * P;
      if (square) grad[(size_t)b * E + e] = (float)(2.0 * coef * d / ((double)n * live));
    }
  }
  sum = block_sum(sum, red);
  slots = block_sum(slots, red);
  if (!square || !n)
    for (int e = tid; e < E; e += 256) {
      const size_t at = (size_t)b * E + e;
      grad[at] = n ? (float)((double)coef * E * (counts[at] - slots / E) /
                             ((double)k * n * n * live)) : 0.f;
    }
  if (tid == 0) {
    ws.lossb[b] = coef * sum;
    if (B == 1) *loss = (float)(coef * sum);
  }
}

// loss = mean over the segments that have counting tokens (B > 1)
__global__ __launch_bounds__(256) void balance_mean_kernel(BalanceWs ws, int parts, int B,
                                                           float* __restrict__ loss) {
  __shared__ double red[256];
  __shared__ int redi[256];
  double sum = 0.;
  int live = 0;
  for (int b = threadIdx.x; b < B; b += 256) {
    int n = 0;
    for (int c = 0; c < parts; ++c) n |= ws.n[(size_t)b * parts + c];
    live += n != 0;
    sum += ws.lossb[b];
  }
  sum = block_sum(sum, red);
  live = block_sum(live, redi);
  if (threadIdx.x == 0) *loss = live ? (float)(sum / live) : 0.f;
}

// One wave per token: G = gate part + loss part, dz = p (G - sum p G); with renormalised
// gates their part goes to the chosen experts directly.
template <int KPL>
__global__ __launch_bounds__(256) void route_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ idx, const float* __restrict__ dw,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ offsets,
    const float* __restrict__ grad, const float* __restrict__ dloss, int T, int E, int k, int B,
    bool renorm, float* __restrict__ dlogits, float* __restrict__ part) {
  __shared__ float red[4][64 * KPL];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const float up = dloss ? *dloss : 1.f;
  float col[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) col[i] = 0.f;
  for (int t = blockIdx.x * 4 + w; t < T; t += gridDim.x * 4) {
    // the last segment that begins at or before t
    int b = 0, lo = 0, hi = T;
    if (offsets) {
      int top = B;
      while (top - b > 1) {
        const int mid = (b + top) >> 1;
        if (offsets[mid] <= t) b = mid; else top = mid;
      }
      segment(offsets, b, T, lo, hi);
    }
    float p[KPL], g[KPL];
    if (t < lo || t >= hi || (mask && mask[t] == 0)) {
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (lane + 64 * i < E) dlogits[(size_t)t * E + lane + 64 * i] = 0.f;
      continue;
    }
    load_keys(p, logits, bias, t, E, lane);
    row_softmax(p);
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int e = lane + 64 * i;
      g[i] = grad && e < E ? up * grad[(size_t)b * E + e] : 0.f;
    }
    float direct[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) direct[i] = 0.f;
    if (dw) {
      // lane j holds slot j
      int ej = -1;
      float dj = 0.f;
      if (lane < k) {
        ej = idx[(size_t)t * k + lane];
        if (ej < 0 || ej >= E) ej = -1;
        if (ej >= 0) dj = dw[(size_t)t * k + lane];
      }
      if (renorm) {
        // p at the chosen experts
        float pj = 0.f;
        for (int j = 0; j < k; ++j) {
          const int e = __shfl(ej, j, 64);
          float mine = 0.f;
#pragma unroll
          for (int i = 0; i < KPL; ++i)
            if (lane + 64 * i == e) mine = p[i];
          const float v = __shfl(mine, e & 63, 64);
          if (lane == j && e >= 0) pj = v;
        }
        const float s = group_sum<64>(pj);
        const float wj = s == 0.f ? 0.f : pj / s;
        dj = wj * (dj - group_sum<64>(wj * dj));
      }
      for (int j = 0; j < k; ++j) {
        const int e = __shfl(ej, j, 64);
        const float v = __shfl(dj, j, 64);
#pragma unroll
        for (int i = 0; i < KPL; ++i)
          if (lane + 64 * i == e) {
            if (renorm) direct[i] += v; else g[i] += v;
          }
      }
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) m = fmaf(p[i], g[i], m);
    m = group_sum<64>(m);
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int e = lane + 64 * i;
      const float dz = fmaf(p[i], g[i] - m, direct[i]);
      if (e < E) dlogits[(size_t)t * E + e] = dz;
      col[i] += dz;
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < KPL; ++i) red[w][lane + 64 * i] = col[i];
  __syncthreads();
  for (int e = tid; e < E; e += 256)
    part[(size_t)blockIdx.x * E + e] = ((red[0][e] + red[1][e]) + red[2][e]) + red[3][e];
}

__global__ __launch_bounds__(256) void column_sum_kernel(const float* __restrict__ part, int n,
                                                         int E, float* __restrict__ out) {
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e >= E) return;
  double s = 0.;
  for (int i = 0; i < n; ++i) s += part[(size_t)i * E + e];
  out[e] = (float)s;
}

// ------------------------------------------------------------------ launchers
// about 16 tokens per part, and no more than about 1024 parts in all
int balance_parts(int T, int B) {
  const long most = std::max(1, 1024 / B);
  return (int)std::min<long>(most, std::max<long>(1, ((long)T + 16L * B - 1) / (16L * B)));
}

size_t balance_ws_bytes(int T, int E, int B) {
  size_t total = 0;
  balance_ws(nullptr, T, E, B, &total);
  return total;
}

hipError_t launch_balance_loss(const float* logits, const float* bias, const int32_t* idx,
                               const uint8_t* mask, const int32_t* offsets, int T, int E, int k,
                               int B, bool square, float coef, int32_t* counts, float* probs,
                               float* grad, float* loss, void* ws_mem, hipStream_t s) {
  size_t total = 0;
  const BalanceWs ws = balance_ws(ws_mem, T, E, B, &total);
  const int parts = balance_parts(T, B);
  const dim3 grid((unsigned)parts, (unsigned)B), block(256);
#define MOE_BALANCE(KPL) \
  hipLaunchKernelGGL(balance_part_kernel<KPL>, grid, block, 0, s, logits, bias, idx, mask, \
                     offsets, T, E, k, ws)
  if (E <= 64) MOE_BALANCE(1);
  else if (E <= 128) MOE_BALANCE(2);
  else if (E <= 256) MOE_BALANCE(4);
  else if (E <= 512) MOE_BALANCE(8);
  else MOE_BALANCE(16);
#undef MOE_BALANCE
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_join_kernel, dim3((unsigned)B), block, 0, s, ws, parts, E, k, B,
                     square, coef, counts, probs, grad, loss);
  if ((e = hipGetLastError()) != hipSuccess || B == 1) return e;
  hipLaunchKernelGGL(balance_mean_kernel, dim3(1), block, 0, s, ws, parts, B, loss);
  return hipGetLastError();
}

int route_bwd_blocks(int T) { return std::max(1, std::min((T + 3) / 4, 1024)); }

hipError_t launch_route_bwd(const float* logits, const float* bias, const int32_t* idx,
                            const float* dw, const uint8_t* mask, const int32_t* offsets,
                            const float* grad, const float* dloss, int T, int E, int k, int B,
                            bool renorm, float* dlogits, float* dbias, void* ws, hipStream_t s) {
  const int n = route_bwd_blocks(T);
  float* part = dbias ? static_cast<float*>(ws) : nullptr;
#define MOE_ROUTE_BWD(KPL) \
  hipLaunchKernelGGL(route_bwd_kernel<KPL>, dim3((unsigned)n), dim3(256), 0, s, logits, bias, \
                     idx, dw, mask, offsets, grad, dloss, T, E, k, B, renorm, dlogits, part)
  if (E <= 64) MOE_ROUTE_BWD(1);
  else if (E <= 128) MOE_ROUTE_BWD(2);
  else if (E <= 256) MOE_ROUTE_BWD(4);
  else if (E <= 512) MOE_ROUTE_BWD(8);
  else MOE_ROUTE_BWD(16);
#undef MOE_ROUTE_BWD
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dbias) return e;
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((E + 255) / 256)), dim3(256), 0, s, part,
                     n, E, dbias);
  return hipGetLastError();
}

}  // namespace moe
