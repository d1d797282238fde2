// The training side of the router: load-balance loss with per-expert counts, and the
// gradient of the gate weights and of that loss with respect to the logits.
//
// p[t] = softmax(logits[t] + bias) (the router's biased softmax, MegaMoE walkthrough,
// discosf.com sec. 2.2, in fp32).  Per segment of n counting tokens, P_e = mean_t p[t, e]
// and f_e = counts_e / (k n); the loss is E sum f_e P_e or sum (P_e - 1/E)^2, so with
// g_e = dL/dp[t, e] every token's gradient is the softmax's, p_e (g_e - sum_i p_i g_i).
//
// Both directions are one pass over the logits, bound by that traffic for large batches and
// by latency for small ones.  A group of LP = 16 lanes holds one token's keys in registers
// (64 lanes above 256 experts), V pieces of 4 consecutive experts a lane, so a wave has four
// tokens' 16-byte loads in flight and the row sums are four rotations inside the lane row.
// Sums over tokens are taken per part in a fixed order and joined in fp64, without float
// atomics: the result does not depend on scheduling.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

struct __attribute__((packed, aligned(4))) F4 {        // 16 bytes at any 4-byte address
  float v[4];
};

template <int CTRL>
__device__ __forceinline__ float row_rotate(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// maximum / sum over a group of LP (16 or 64) lanes, the same bits in each of them
template <int LP>
__device__ __forceinline__ float lanes_max(float v) {
  v = fmaxf(v, row_rotate<0x128>(v));
  v = fmaxf(v, row_rotate<0x124>(v));
  v = fmaxf(v, row_rotate<0x122>(v));
  v = fmaxf(v, row_rotate<0x121>(v));
  if (LP == 64) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int LP>
__device__ __forceinline__ float lanes_sum(float v) {
  v += row_rotate<0x128>(v);
  v += row_rotate<0x124>(v);
  v += row_rotate<0x122>(v);
  v += row_rotate<0x121>(v);
  if (LP == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}

// The pieces of a row of E floats that lane li of a group holds: experts 4 (li + LP j) + c at
// element 4 j + c; `fill` past E.
template <int LP, int V>
__device__ __forceinline__ void load_row(float (&x)[4 * V], const float* row, int E, int li,
                                         float fill) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = 4 * (li + LP * j);
    if (e + 4 <= E) {
      const F4 f = *reinterpret_cast<const F4*>(row + e);
#pragma unroll
      for (int c = 0; c < 4; ++c) x[4 * j + c] = f.v[c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[4 * j + c] = e + c < E ? row[e + c] : fill;
    }
  }
}

// e^(key - m) on the hardware's base-2 exponential: the error is that of the two roundings of
// the argument, below 2^-23 |key - m|, and one step of the exponential
__device__ __forceinline__ float exp_below(float key, float m) {
  return __builtin_amdgcn_exp2f((key - m) * 1.44269504088896340736f);
}

// keys -> probabilities (a row of -inf gives zeros; NaN and +inf give NaN); returns the
// maximum and the reciprocal of the sum
template <int LP, int N>
__device__ __forceinline__ float2 row_softmax(float (&x)[N]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, x[i]);
  m = lanes_max<LP>(m);
  if (m == -INFINITY) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = exp_below(x[i], m);
    s += x[i];
  }
  s = lanes_sum<LP>(s);
  const float inv = s == 0.f ? 0.f : __builtin_amdgcn_rcpf(s);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] *= inv;
  return make_float2(m, inv);
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

// Column sums of a group's registers over the wave's groups and the workgroup's four waves,
// in a fixed order: red [4][E] holds one row per wave, written by the group of lanes 0..LP-1.
template <int LP, int V>
__device__ __forceinline__ void wave_columns(float (&x)[4 * V], float* red, int E, int li,
                                             int lane) {
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) {
    if (LP == 16) {
      x[i] += __shfl_xor(x[i], 16, 64);
      x[i] += __shfl_xor(x[i], 32, 64);
    }
    const int e = 4 * (li + LP * (i / 4)) + i % 4;
    if (lane < LP && e < E) red[e] = x[i];
  }
}

struct BalanceWs {
  float* psum;      // [B][parts][E] sums of p over a part's tokens
  int32_t* cnt;     // [B][parts][E] slots per expert
  int32_t* n;       // [B][parts] counting tokens
  int32_t* slots;   // [B][parts] their slots with an expert
  double* lossp;    // [join workgroups] their shares of the loss
  int32_t* done;    // join workgroups that have finished
};

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

constexpr int kJoinCols = 32, kJoinRows = 128;   // columns of a join workgroup, rows of its grid

BalanceWs balance_ws(void* ws, int T, int E, int B, size_t* total) {
  const size_t np = (size_t)B * balance_parts(T, B);
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = p + at;
    at = up256(at + bytes);
    return r;
  };
  BalanceWs w;
  w.psum = reinterpret_cast<float*>(take(np * E * 4));
  w.cnt = reinterpret_cast<int32_t*>(take(np * E * 4));
  w.n = reinterpret_cast<int32_t*>(take(np * 4));
  w.slots = reinterpret_cast<int32_t*>(take(np * 4));
  w.lossp = reinterpret_cast<double*>(
      take((size_t)((E + kJoinCols - 1) / kJoinCols) * std::min(B, kJoinRows) * 8));
  w.done = reinterpret_cast<int32_t*>(take(4));
  *total = at;
  return w;
}

}  // namespace

// Part blockIdx.x of segment blockIdx.y: sums of p, slots per expert, counting tokens.
template <int LP, int V>
__global__ __launch_bounds__(256) void balance_part_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ offsets, int T, int E, int k, BalanceWs ws) {
  constexpr int N = 4 * V, TW = 64 / LP;               // tokens a wave holds at once
  __shared__ float red[4][LP * N];
  __shared__ int cnt[LP * N], nw[4][2];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int li = lane % LP;
  const int parts = gridDim.x, c = blockIdx.x, b = blockIdx.y;
  if (tid == 0 && c == 0 && b == 0) *ws.done = 0;      // for the join launch
  int lo, hi;
  segment(offsets, b, T, lo, hi);
  const int per = (int)(((long)hi - lo + parts - 1) / parts);
  const int t0 = (int)min((long)lo + (long)c * per, (long)hi), t1 = t0 + min(per, hi - t0);
  for (int e = tid; e < E; e += 256) cnt[e] = 0;
  float bv[N];
#pragma unroll
  for (int i = 0; i < N; ++i) bv[i] = 0.f;
  if (bias) load_row<LP, V>(bv, bias, E, li, 0.f);
  __syncthreads();
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  int n = 0, m = 0;
  float next[N];
  bool live = false;
  // one turn's keys are loaded while the turn before is summed
  auto load = [&](int t) {
    live = t < t1 && !(mask && mask[t] == 0);
    if (live) load_row<LP, V>(next, logits + (size_t)t * E, E, li, -INFINITY);
  };
  int t = t0 + w * TW + lane / LP;
  load(t);
  for (int base = t0; base < t1; base += 4 * TW, t += 4 * TW) {
    float p[N];
    const bool now = live;
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = now ? next[i] + bv[i] : -INFINITY;
    load(t + 4 * TW);
    if (now) {
      for (int j = li; j < k; j += LP) {
        const int e = idx[(size_t)t * k + j];
        if (e >= 0 && e < E) {
          atomicAdd(&cnt[e], 1);
          ++m;
        }
      }
      n += li == 0;
    }
    row_softmax<LP>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += p[i];
  }
  wave_columns<LP, V>(acc, red[w], E, li, lane);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    n += __shfl_xor(n, o, 64);
    m += __shfl_xor(m, o, 64);
  }
  if (lane == 0) {
    nw[w][0] = n;
    nw[w][1] = m;
  }
  __syncthreads();
  const size_t part = (size_t)b * parts + c;
  for (int e = tid; e < E; e += 256) {
    ws.psum[part * E + e] = ((red[0][e] + red[1][e]) + red[2][e]) + red[3][e];
    ws.cnt[part * E + e] = cnt[e];
  }
  if (tid == 0) {
    ws.n[part] = nw[0][0] + nw[1][0] + nw[2][0] + nw[3][0];
    ws.slots[part] = nw[0][1] + nw[1][1] + nw[2][1] + nw[3][1];
  }
}

namespace {
// sum over the 256 threads, in every thread (integers: any order)
__device__ __forceinline__ int block_sum_int(int v, int* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}
}  // namespace

// Joins the parts: workgroup (x, y) takes the columns [32 x, 32 x + 32) of the segments
// y, y + gridDim.y, ..., eight threads a column.  The last workgroup to finish adds up the
// shares of the loss in workgroup order.
__global__ __launch_bounds__(256) void balance_join_kernel(BalanceWs ws, int parts, int E, int k,
                                                           int B, bool square, float coef,
                                                           int32_t* __restrict__ counts,
                                                           float* __restrict__ probs,
                                                           float* __restrict__ grad,
                                                           float* __restrict__ loss) {
  __shared__ int redi[4];
  __shared__ double pd[8][kJoinCols];
  __shared__ int cd[8][kJoinCols];
  __shared__ double share[kJoinCols];
  __shared__ bool last;
  const int tid = threadIdx.x, col = tid & 31, sl = tid >> 5;
  const int e = blockIdx.x * kJoinCols + col;
  // segments with counting tokens
  int live = 0;
  for (int b = tid; b < B; b += 256) {
    int any = 0;
    for (int c = 0; c < parts; ++c) any |= ws.n[(size_t)b * parts + c];
    live += any != 0;
  }
  live = block_sum_int(live, redi);
  double mine = 0.;                                     // thread < 32: its column's terms
  for (int b = blockIdx.y; b < B; b += gridDim.y) {
    int n = 0, m = 0;
    for (int c = tid; c < parts; c += 256) {
      n += ws.n[(size_t)b * parts + c];
      m += ws.slots[(size_t)b * parts + c];
    }
    n = block_sum_int(n, redi);
    m = block_sum_int(m, redi);
    double P = 0.;
    int s = 0;
    if (e < E) {
#pragma unroll 8
      for (int c = sl; c < parts; c += 8) {
        const size_t at = ((size_t)b * parts + c) * E + e;
        P += ws.psum[at];
        s += ws.cnt[at];
      }
    }
    pd[sl][col] = P;
    cd[sl][col] = s;
    __syncthreads();
    if (tid < kJoinCols && e < E) {
      P = 0.;
      s = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        P += pd[i][col];
        s += cd[i][col];
      }
      P = n ? P / n : 0.;
      const size_t at = (size_t)b * E + e;
      counts[at] = s;
      probs[at] = (float)P;
      float g = 0.f;
      if (n) {
        const double d = P - 1.0 / E;
        if (square) {
          mine += d * d;
          g = (float)(2.0 * coef * d / ((double)n * live));
        } else {
          mine += E * (s / ((double)k * n)) * P;
          g = (float)((double)coef * E * (s - m / (double)E) / ((double)k * n * n * live));
        }
      }
      grad[at] = g;
    }
    __syncthreads();
  }
  if (tid < kJoinCols) share[tid] = mine;
  __syncthreads();
  const int wgs = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
  if (tid == 0) {
    double v = 0.;
    for (int i = 0; i < kJoinCols; ++i) v += share[i];
    ws.lossp[me] = v;
    // releases the share to, and acquires the others' for, the last to arrive
    last = __hip_atomic_fetch_add(ws.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
           wgs - 1;
  }
  __syncthreads();
  if (!last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  __shared__ double red[256];
  double v = 0.;
  for (int i = tid; i < wgs; i += 256) v += ws.lossp[i];
  red[tid] = v;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) red[tid] += red[tid + o];
    __syncthreads();
  }
  if (tid == 0) *loss = live ? (float)(coef * red[0] / live) : 0.f;
}

// G = gate part + loss part, dz = p (G - sum p G); with renormalised gates their part goes to
// the chosen experts directly.  A token's k slot values reach the lanes of their experts
// through a row of E floats in LDS that is zero between tokens; slots of the same expert
// are added beforehand in slot order, so that each expert's value is stored once.
template <int LP, int V>
__global__ __launch_bounds__(256) void route_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ idx, const float* __restrict__ dw,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ offsets,
    const float* __restrict__ grad, const float* __restrict__ dloss, int T, int E, int k, int B,
    bool renorm, int per, float* __restrict__ dlogits, float* __restrict__ part) {
  constexpr int N = 4 * V, TW = 64 / LP, NG = 4 * TW;   // groups of the workgroup
  constexpr int KL = 64 / LP;                          // slots a lane may hold
  __shared__ __attribute__((aligned(16))) float chosen[NG][LP * N];
  __shared__ int2 slot[NG][64];                        // (expert, value's bits) of the slots
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int li = lane % LP, grp = w * TW + lane / LP;
  float* row = chosen[grp];
  int2* sv = slot[grp];
  const float up = dloss ? *dloss : 1.f;
  if (dw)
    for (int i = 4 * li; i < LP * N; i += 4 * LP)
      *reinterpret_cast<v4f*>(row + i) = v4f{0.f, 0.f, 0.f, 0.f};
  float bv[N], col[N], g[N];
#pragma unroll
  for (int i = 0; i < N; ++i) bv[i] = col[i] = g[i] = 0.f;
  if (bias) load_row<LP, V>(bv, bias, E, li, 0.f);

  const int t0 = (int)min((long)blockIdx.x * per, (long)T), t1 = t0 + min(per, T - t0);
  int t = t0 + grp;
  // the last segment that begins at or before the group's first token; then walked along
  int b = 0, lo = 0, hi = T, have = -1, next = T;
  if (offsets) {
    int top = B;
    while (top - b > 1) {
      const int mid = (b + top) >> 1;
      if (offsets[mid] <= t) b = mid; else top = mid;
    }
    segment(offsets, b, T, lo, hi);
    next = offsets[b + 1];
  }
  for (int base = t0; base < t1; base += NG, t += NG) {
    if (t < t1 && next <= t && b + 1 < B) {
      do {
        next = offsets[++b + 1];
      } while (next <= t && b + 1 < B);
      segment(offsets, b, T, lo, hi);
    }
    const bool in = t < t1, live = in && t >= lo && t < hi && !(mask && mask[t] == 0);
    float p[N];
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = -INFINITY;
    if (live) {
      load_row<LP, V>(p, logits + (size_t)t * E, E, li, -INFINITY);
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] += bv[i];
      if (grad && b != have) {
        load_row<LP, V>(g, grad + (size_t)b * E, E, li, 0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] *= up;
        have = b;
      }
    }
    int ej[KL];
    float dj[KL], lj[KL];
#pragma unroll
    for (int q = 0; q < KL; ++q) {
      const int j = li + LP * q;
      ej[q] = -1;
      dj[q] = lj[q] = 0.f;
      if (dw && live && j < k) {
        const int e = idx[(size_t)t * k + j];
        if (e >= 0 && e < E) {
          ej[q] = e;
          dj[q] = dw[(size_t)t * k + j];
          if (renorm) lj[q] = logits[(size_t)t * E + e] + (bias ? bias[e] : 0.f);
        }
      }
    }
    const float2 ms = row_softmax<LP>(p);
    if (dw) {
      if (renorm) {
        float s = 0.f, wd = 0.f;
#pragma unroll
        for (int q = 0; q < KL; ++q) {
          lj[q] = ej[q] >= 0 ? exp_below(lj[q], ms.x) * ms.y : 0.f;
          s += lj[q];
        }
        s = lanes_sum<LP>(s);
        const float inv = s == 0.f ? 0.f : 1.0f / s;
#pragma unroll
        for (int q = 0; q < KL; ++q) {
          lj[q] *= inv;
          wd += lj[q] * dj[q];
        }
        wd = lanes_sum<LP>(wd);
#pragma unroll
        for (int q = 0; q < KL; ++q) dj[q] = lj[q] * (dj[q] - wd);
      }
      // (a wave's LDS accesses run in order)
#pragma unroll
      for (int q = 0; q < KL; ++q)
        if (li + LP * q < k) sv[li + LP * q] = make_int2(ej[q], __float_as_int(dj[q]));
      __builtin_amdgcn_wave_barrier();
      float sum[KL];
#pragma unroll
      for (int q = 0; q < KL; ++q) sum[q] = 0.f;
      for (int j = 0; j < k; ++j) {
        const int2 o = sv[j];
#pragma unroll
        for (int q = 0; q < KL; ++q) sum[q] += o.x == ej[q] ? __int_as_float(o.y) : 0.f;
      }
#pragma unroll
      for (int q = 0; q < KL; ++q)
        if (ej[q] >= 0) row[ej[q]] = sum[q];
      __builtin_amdgcn_wave_barrier();
    }
    float d[N], m = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v4f r = {0.f, 0.f, 0.f, 0.f};
      if (dw) r = *reinterpret_cast<const v4f*>(row + 4 * (li + LP * j));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = 4 * j + c;
        d[i] = renorm ? g[i] : g[i] + r[c];
        m = fmaf(p[i], d[i], m);
      }
    }
    m = lanes_sum<LP>(m);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v4f r = {0.f, 0.f, 0.f, 0.f};
      if (dw && renorm) r = *reinterpret_cast<const v4f*>(row + 4 * (li + LP * j));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = 4 * j + c;
        d[i] = live ? fmaf(p[i], d[i] - m, r[c]) : 0.f;
        col[i] += d[i];
      }
      const int e = 4 * (li + LP * j);
      if (in) {
        float* out = dlogits + (size_t)t * E + e;
        if (e + 4 <= E) {
          *reinterpret_cast<F4*>(out) = F4{{d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]}};
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (e + c < E) out[c] = d[4 * j + c];
        }
      }
    }
    if (dw) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int q = 0; q < KL; ++q)
        if (ej[q] >= 0) row[ej[q]] = 0.f;
      __builtin_amdgcn_wave_barrier();
    }
  }
  if (!part) return;
  __syncthreads();
  wave_columns<LP, V>(col, chosen[w], E, li, lane);     // rows 0..3 of the LDS block
  __syncthreads();
  for (int e = tid; e < E; e += 256)
    part[(size_t)blockIdx.x * E + e] =
        ((chosen[0][e] + chosen[1][e]) + chosen[2][e]) + chosen[3][e];
}

// out[e] = sum of n rows of part, eight threads a column, fp64 in a fixed order
__global__ __launch_bounds__(256) void column_sum_kernel(const float* __restrict__ part, int n,
                                                         int E, float* __restrict__ out) {
  __shared__ double red[32][9];
  const int tid = threadIdx.x, col = tid & 7, sl = tid >> 3, e = blockIdx.x * 8 + col;
  double s = 0.;
  if (e < E) {
#pragma unroll 8
    for (int i = sl; i < n; i += 32) s += part[(size_t)i * E + e];
  }
  red[sl][col] = s;
  __syncthreads();
  if (tid < 8 && e < E) {
    s = 0.;
    for (int i = 0; i < 32; ++i) s += red[i][col];
    out[e] = (float)s;
  }
}

// ------------------------------------------------------------------ launchers
// about 16 tokens per part (one turn of a workgroup), and no more than about 1024 parts in all
int balance_parts(int T, int B) {
  const long most = std::max(1, 1024 / B);
  return (int)std::min<long>(most, std::max<long>(1, ((long)T + 16L * B - 1) / (16L * B)));
}

size_t balance_ws_bytes(int T, int E, int B) {
  size_t total = 0;
  balance_ws(nullptr, T, E, B, &total);
  return total;
}

// f<LP, V>() for E experts
#define MOE_BY_EXPERTS(E, F) \
  if ((E) <= 64) F(16, 1);   \
  else if ((E) <= 128) F(16, 2); \
  else if ((E) <= 256) F(16, 4); \
  else if ((E) <= 512) F(64, 2); \
  else F(64, 4)

hipError_t launch_balance_loss(const float* logits, const float* bias, const int32_t* idx,
                               const uint8_t* mask, const int32_t* offsets, int T, int E, int k,
                               int B, bool square, float coef, int32_t* counts, float* probs,
                               float* grad, float* loss, void* ws_mem, hipStream_t s) {
  size_t total = 0;
  const BalanceWs ws = balance_ws(ws_mem, T, E, B, &total);
  const int parts = balance_parts(T, B);
  const dim3 grid((unsigned)parts, (unsigned)B), block(256);
#define MOE_BALANCE(LP, V) \
  hipLaunchKernelGGL((balance_part_kernel<LP, V>), grid, block, 0, s, logits, bias, idx, mask, \
                     offsets, T, E, k, ws)
  MOE_BY_EXPERTS(E, MOE_BALANCE);
#undef MOE_BALANCE
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 join((unsigned)((E + kJoinCols - 1) / kJoinCols), (unsigned)std::min(B, kJoinRows));
  hipLaunchKernelGGL(balance_join_kernel, join, block, 0, s, ws, parts, E, k, B, square, coef,
                     counts, probs, grad, loss);
  return hipGetLastError();
}

// workgroups of the backward pass: one turn of 16 tokens each up to 1024 of them
int route_bwd_blocks(int T) { return std::max(1, std::min((T + 15) / 16, 1024)); }

hipError_t launch_route_bwd(const float* logits, const float* bias, const int32_t* idx,
                            const float* dw, const uint8_t* mask, const int32_t* offsets,
                            const float* grad, const float* dloss, int T, int E, int k, int B,
                            bool renorm, float* dlogits, float* dbias, void* ws, hipStream_t s) {
  const int n = route_bwd_blocks(T), per = (T + n - 1) / n;
  float* part = dbias ? static_cast<float*>(ws) : nullptr;
#define MOE_ROUTE_BWD(LP, V) \
  hipLaunchKernelGGL((route_bwd_kernel<LP, V>), dim3((unsigned)n), dim3(256), 0, s, logits, bias, \
                     idx, dw, mask, offsets, grad, dloss, T, E, k, B, renorm, per, dlogits, part)
  MOE_BY_EXPERTS(E, MOE_ROUTE_BWD);
#undef MOE_ROUTE_BWD
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dbias) return e;
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((E + 7) / 8)), dim3(256), 0, s, part, n, E,
                     dbias);
  return hipGetLastError();
}

#undef MOE_BY_EXPERTS

}  // namespace moe
