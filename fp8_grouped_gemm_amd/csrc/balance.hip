// The training side of the router: load-balance loss with per-expert counts, and the
// gradient of the gate weights and of that loss with respect to the logits.
//
// p[t] = softmax(logits[t] + bias) (the router's biased softmax, MegaMoE walkthrough,
// discosf.com sec. 2.2, in fp32).  Per segment of n counting tokens, P_e = mean_t p[t, e]
// and f_e = counts_e / (k n); the loss is E sum f_e P_e or sum (P_e - 1/E)^2, so with
// g_e = dL/dp[t, e] every token's gradient is the softmax's, p_e (g_e - sum_i p_i g_i).
//
// Both directions are one pass over the logits, bound by that traffic for large batches and
// by latency for small ones: the loss of 65536 x 256 takes 17 us for its pass (4.0 TB/s) and 8
// to join the parts, the backward pass of 131072 x 64 with gate weights 17 us (73 MB in and
// out, 4.3 TB/s), of 65536 x 256 30 us (4.5 TB/s); a decode step's 128 x 256 takes 5 + 5.5 us.
// A group of 8 to 64 lanes holds one token's keys in registers, up to 16 a lane in pieces of 4
// consecutive experts, so a wave has one to eight tokens' 16-byte loads in flight and what is
// done once per token costs little (16 lanes for 64 experts: 25 us for 17).  The next turn's
// tokens are loaded before the present one's are used.  Sums over tokens are taken per part in
// a fixed order and joined in fp64, without float atomics: the result does not depend on
// scheduling.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

struct __attribute__((packed, aligned(4))) F4 {        // 16 bytes at any 4-byte address
  float v[4];
};

template <int CTRL>
__device__ __forceinline__ float row_move(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// v joined over a group of LP (8, 16, 32 or 64) lanes by the commutative f, the same bits in
// each of them: exchanges inside rows of 8 lanes or rotations of rows of 16, then shuffles
template <int LP, class F>
__device__ __forceinline__ float lanes_join(float v, F f) {
  if (LP == 8) {
    v = f(v, row_move<0xB1>(v));                       // lanes 1 0 3 2
    v = f(v, row_move<0x4E>(v));                       // lanes 2 3 0 1
    v = f(v, row_move<0x141>(v));                      // lanes 7 6 5 4 3 2 1 0
  } else {
    v = f(v, row_move<0x128>(v));
    v = f(v, row_move<0x124>(v));
    v = f(v, row_move<0x122>(v));
    v = f(v, row_move<0x121>(v));
  }
  if (LP >= 32) v = f(v, __shfl_xor(v, 16, 64));
  if (LP == 64) v = f(v, __shfl_xor(v, 32, 64));
  return v;
}
template <int LP>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes_join<LP>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LP>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_join<LP>(v, [](float a, float b) { return a + b; });
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

// keys -> probabilities (a row of -inf gives zeros; NaN and +inf give NaN)
template <int LP, int N>
__device__ __forceinline__ void row_softmax(float (&x)[N]) {
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
    if (LP <= 8) x[i] += __shfl_xor(x[i], 8, 64);
    if (LP <= 16) x[i] += __shfl_xor(x[i], 16, 64);
    if (LP <= 32) x[i] += __shfl_xor(x[i], 32, 64);
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

constexpr int kJoinRows = 128;                    // rows of the join's grid, at most
// Columns of a join workgroup, whose threads cut the parts into slices: 8 columns and 1024
// threads where many parts meet few workgroups, else 32 and 256.  The loss of one segment of
// 16384 x 128 (1024 parts): 19 us with 8 columns, 58 with 32; two segments of 2048 x 256 (128
// parts each): 14.0, 17.8; but four of 2048 x 1024, 512 workgroups of 8 columns: 26.2, 22.6.
int join_cols(int parts, int E, int B) {
  return parts >= 64 && (long)((E + 7) / 8) * B <= 256 ? 8 : 32;
}

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
      take((size_t)((E + 7) / 8) * std::min(B, kJoinRows) * 8));
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
  // One turn's keys, first slots and mask are loaded while the turn before is summed.  The mask
  // does not hold the keys back: a padding token's are read and dropped.
  float next[N];
  int next_e = -1, next_on = 0;
  auto load = [&](int t) {
    next_on = 0;
    if (t < t1) {
      next_on = mask ? mask[t] : 1;
      next_e = li < k ? idx[(size_t)t * k + li] : -1;
      load_row<LP, V>(next, logits + (size_t)t * E, E, li, -INFINITY);
    }
  };
  int t = t0 + w * TW + lane / LP;
  load(t);
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
  for (int base = t0; base < t1; base += 4 * TW, t += 4 * TW) {
    float p[N];
    const bool now = next_on != 0;
    const int e0 = next_e;
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = now ? next[i] + bv[i] : -INFINITY;
    load(t + 4 * TW);
    if (now) {
      for (int j = li, e = e0; j < k; j += LP) {
        if (j >= LP) e = idx[(size_t)t * k + j];
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
// sums over the workgroup's threads, in every thread (integers: any order)
template <int WAVES>
__device__ __forceinline__ int3 block_sum_int3(int a, int b, int c, int (*red)[3]) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
    c += __shfl_xor(c, o, 64);
  }
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    red[w][0] = a;
    red[w][1] = b;
    red[w][2] = c;
  }
  __syncthreads();
  int3 s = make_int3(0, 0, 0);
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    s.x += red[i][0];
    s.y += red[i][1];
    s.z += red[i][2];
  }
  return s;
}
}  // namespace

// Joins the parts: workgroup (x, y) takes COLS columns of the segments y, y + gridDim.y, ...,
// NT / COLS threads a column.  The last workgroup to finish adds up the shares of the loss in
// workgroup order.
template <int COLS, int NT>
__global__ __launch_bounds__(NT) void balance_join_kernel(BalanceWs ws, int parts, int E, int k,
                                                           int B, bool square, float coef,
                                                           int32_t* __restrict__ counts,
                                                           float* __restrict__ probs,
                                                           float* __restrict__ grad,
                                                           float* __restrict__ loss) {
  __shared__ int redi[NT / 64][3];
  __shared__ int any[512];
  constexpr int SL = NT / COLS, NW = NT / 64;           // slices, waves
  __shared__ double pd[NW][COLS];
  __shared__ int cd[NW][COLS];
  __shared__ double share[COLS];
  __shared__ bool last;
  const int tid = threadIdx.x, col = tid % COLS, sl = tid / COLS;
  const int e = blockIdx.x * COLS + col;
  // Segments with counting tokens; with more than one part each there are at most 1024 parts.
  int live = 0, some[1024 / NT];
  if (parts == 1) {
    for (int i = tid; i < B; i += NT) live += ws.n[i] != 0;
  } else {
#pragma unroll
    for (int i = 0; i < 1024 / NT; ++i)
      some[i] = i * NT + tid < B * parts ? ws.n[i * NT + tid] : 0;
    for (int i = tid; i < B; i += NT) any[i] = 0;
  }
  double mine = 0.;                                     // thread < COLS: its column's terms
  for (int b = blockIdx.y; b < B; b += gridDim.y) {
    const bool once = b == (int)blockIdx.y;
    // everything the segment needs is asked for before the first sum over threads
    int n = 0, m = 0;
    for (int c = tid; c < parts; c += NT) {
      n += ws.n[(size_t)b * parts + c];
      m += ws.slots[(size_t)b * parts + c];
    }
    double P = 0.;
    int s = 0;
    if (e < E) {
#pragma unroll 8
      for (int c = sl; c < parts; c += SL) {
        const size_t at = ((size_t)b * parts + c) * E + e;
        P += ws.psum[at];
        s += ws.cnt[at];
      }
    }
    if (once && parts > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 1024 / NT; ++i)
        if (some[i]) any[(i * NT + tid) / parts] = 1;
      __syncthreads();
      for (int i = tid; i < B; i += NT) live += any[i];
    }
    const int3 sums = block_sum_int3<NW>(n, m, once ? live : 0, redi);
    n = sums.x;
    m = sums.y;
    if (once) live = sums.z;
#pragma unroll
    for (int o = COLS; o < 64; o <<= 1) {
      P += __shfl_xor(P, o, 64);
      s += __shfl_xor(s, o, 64);
    }
    if ((tid & 63) < COLS) {
      pd[tid >> 6][col] = P;
      cd[tid >> 6][col] = s;
    }
    __syncthreads();
    if (tid < COLS && e < E) {
      P = 0.;
      s = 0;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
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
  if (tid < COLS) share[tid] = mine;
  __syncthreads();
  const int wgs = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
  if (tid == 0) {
    double v = 0.;
    for (int i = 0; i < COLS; ++i) v += share[i];
    // Only the share has to reach the last to arrive: it is stored at, and loaded from, the
    // level that all XCDs share, and waited for before the arrival is counted.  A release would
    // write back the XCD's L2 with everyone's outputs (128 workgroups: 2 us more).
    __hip_atomic_store(ws.lossp + me, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    last = __hip_atomic_fetch_add(ws.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
           wgs - 1;
    asm volatile("" ::: "memory");
  }
  __syncthreads();
  if (!last) return;
  __shared__ double red[NT];
  double v = 0.;
  for (int i = tid; i < wgs; i += NT)
    v += __hip_atomic_load(ws.lossp + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  red[tid] = v;
  __syncthreads();
  for (int o = NT / 2; o > 0; o >>= 1) {
    if (tid < o) red[tid] += red[tid + o];
    __syncthreads();
  }
  if (tid == 0) *loss = live ? (float)(coef * red[0] / live) : 0.f;
}

// G = gate part + loss part, dz = p (G - sum p G); with renormalised gates their part goes to
// the chosen experts directly.  A token's k slot values reach the lanes of their experts
// through a row of E floats in LDS that is zero between tokens; slots of the same expert
// are added beforehand in slot order, so that each expert's value is stored once.
template <int LP, int V, int KL>
__global__ __launch_bounds__(256, 4) void route_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ idx, const float* __restrict__ dw,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ offsets,
    const float* __restrict__ grad, const float* __restrict__ dloss, int T, int E, int k, int B,
    bool renorm, int per, float* __restrict__ dlogits, float* __restrict__ part) {
  constexpr int N = 4 * V, TW = 64 / LP, NG = 4 * TW;   // groups of the workgroup
  __shared__ __attribute__((aligned(16))) float chosen[NG][LP * N];
  __shared__ __attribute__((aligned(16))) float bias_mem[LP * N];
  __shared__ int2 slot[NG][64];                        // (expert, value's bits) of the slots
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int li = lane % LP, grp = w * TW + lane / LP;
  float* row = chosen[grp];
  int2* sv = slot[grp];
  const float up = dloss ? *dloss : 1.f;

  const int t0 = (int)min((long)blockIdx.x * per, (long)T), t1 = t0 + min(per, T - t0);
  int t = t0 + grp;
  // One turn's keys, first slots and mask are loaded while the turn before is computed; the
  // mask does not hold the keys back.
  float next_p[N], next_d = 0.f;
  int next_e = -1, next_on = 0;
  auto load = [&](int t) {
    next_on = 0;
    if (t < t1) {
      next_on = mask ? mask[t] : 1;
      if (dw && li < k) {
        next_e = idx[(size_t)t * k + li];
        next_d = dw[(size_t)t * k + li];
      }
      load_row<LP, V>(next_p, logits + (size_t)t * E, E, li, -INFINITY);
    }
  };
  load(t);
  if (dw)
    for (int i = 4 * li; i < LP * N; i += 4 * LP)
      *reinterpret_cast<v4f*>(row + i) = v4f{0.f, 0.f, 0.f, 0.f};
  float col[N], g[N];
#pragma unroll
  for (int i = 0; i < N; ++i) col[i] = g[i] = 0.f;
  for (int i = tid; i < LP * N; i += 256) bias_mem[i] = bias && i < E ? bias[i] : 0.f;
  __syncthreads();
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
    const bool in = t < t1, live = in && t >= lo && t < hi && next_on != 0;
    float p[N];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const v4f bv = *reinterpret_cast<const v4f*>(bias_mem + 4 * (li + LP * j));
#pragma unroll
      for (int c = 0; c < 4; ++c) p[4 * j + c] = live ? next_p[4 * j + c] + bv[c] : -INFINITY;
    }
    int ej[KL];
    float dj[KL], lj[KL];
    ej[0] = next_e;
    dj[0] = next_d;
    load(t + NG);
    if (live && grad && b != have) {
      load_row<LP, V>(g, grad + (size_t)b * E, E, li, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] *= up;
      have = b;
    }
#pragma unroll
    for (int q = 0; q < KL; ++q) {
      const int j = li + LP * q;
      const bool has = dw && live && j < k;
      if (q > 0) {
        ej[q] = -1;
        dj[q] = 0.f;
        if (has) {
          ej[q] = idx[(size_t)t * k + j];
          dj[q] = dw[(size_t)t * k + j];
        }
      }
      const bool chosen_one = has && ej[q] >= 0 && ej[q] < E;
      ej[q] = chosen_one ? ej[q] : -1;
      dj[q] = chosen_one ? dj[q] : 0.f;
      lj[q] = 0.f;
    }
    row_softmax<LP>(p);
    if (dw) {
      if (renorm) {
        // the chosen experts' probabilities through the row (a wave's accesses run in order)
#pragma unroll
        for (int j = 0; j < V; ++j)
          *reinterpret_cast<v4f*>(row + 4 * (li + LP * j)) =
              v4f{p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]};
        __builtin_amdgcn_wave_barrier();
        float s = 0.f, wd = 0.f;
#pragma unroll
        for (int q = 0; q < KL; ++q) {
          if (ej[q] >= 0) lj[q] = row[ej[q]];
          s += lj[q];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < V; ++j)
          *reinterpret_cast<v4f*>(row + 4 * (li + LP * j)) = v4f{0.f, 0.f, 0.f, 0.f};
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
        for (int q = 0; q < KL; ++q)
          sum[q] += o.x == ej[q] ? __int_as_float(o.y) : 0.f;
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
// about 16 tokens per part, and no more than about 1024 parts in all (the loss of
// 65536 x 256: 25 us, with up to 2048 parts 5 us more)
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
  if ((E) <= 64) F(8, 2);        \
  else if ((E) <= 128) F(8, 4);  \
  else if ((E) <= 256) F(16, 4); \
  else if ((E) <= 512) F(32, 4); \
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
  const int cols = join_cols(parts, E, B);
  const dim3 join((unsigned)((E + cols - 1) / cols), (unsigned)std::min(B, kJoinRows));
  if (cols == 8)
    hipLaunchKernelGGL((balance_join_kernel<8, 1024>), join, dim3(1024), 0, s, ws, parts, E, k, B,
                       square, coef, counts, probs, grad, loss);
  else
    hipLaunchKernelGGL((balance_join_kernel<32, 256>), join, block, 0, s, ws, parts, E, k, B,
                       square, coef, counts, probs, grad, loss);
  return hipGetLastError();
}

// workgroups of the backward pass: 16 tokens each up to 1024 of them
int route_bwd_blocks(int T) { return std::max(1, std::min((T + 15) / 16, 1024)); }

hipError_t launch_route_bwd(const float* logits, const float* bias, const int32_t* idx,
                            const float* dw, const uint8_t* mask, const int32_t* offsets,
                            const float* grad, const float* dloss, int T, int E, int k, int B,
                            bool renorm, float* dlogits, float* dbias, void* ws, hipStream_t s) {
  const int n = route_bwd_blocks(T), per = (T + n - 1) / n;
  float* part = dbias ? static_cast<float*>(ws) : nullptr;
  // a lane holds one slot of its token, or as many as 64 slots need (compiled apart: the loops
  // over the others would cost the usual few slots a quarter of the pass)
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(256), 0, s, logits, bias, idx, dw, mask,
                       offsets, grad, dloss, T, E, k, B, renorm, per, dlogits, part);
  };
#define MOE_ROUTE_BWD(LP, V) \
  launch(k <= LP ? route_bwd_kernel<LP, V, 1>            \
                 : route_bwd_kernel<(LP < 16 ? 16 : LP), (LP < 16 ? V / 2 : V), \
                                    64 / (LP < 16 ? 16 : LP)>)
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
