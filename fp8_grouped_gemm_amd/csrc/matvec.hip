// Products of a few rows with 4-bit weights and group scales, and the combine of the
// experts' outputs.  Codes and packing are moe.h's MOE_INT4 (block-wise 4-bit weights with
// max-abs scales, DeepSeek-V4 lecture, tqpw.cn sec. 3.1), one scale per 32, 64 or 128
// weights of a row:
//   v[s, n] = sum_g s7[n, g] * ( sum_{k in g} q[n, k] x[s, k] ).
//
// The weights are the traffic (half a byte per multiplication and row), so each is read
// once for all slots of its expert and everything else is kept off the memory's way: the
// codes go through the 16x16x32 bf16 matrix instruction with the rows of x, which leaves the
// vector ALU the expansion of the codes (10 operations per 8 codes) and one multiply-add per
// group and output.
//
// A wave takes a tile of 32 or 16 weight rows of one expert (SwiGLU: 16 gate rows and the 16 up
// rows of the same outputs) and a slice of K in 128-deep blocks, four of them in flight; the
// slices of a tile are waves of one workgroup and are joined through LDS in slice order.  In
// the matrix instruction the weights are the right operand (lane l: weight row l % 16), so a
// lane needs the scale of one row only; up to 16 rows of x are the left one.  A row of x in
// fp32 is three rows of bf16, its leading, middle and last 8 bits (x = hi + mid + lo exactly),
// whose sums are added at the end: the products stay exact.
//
// Bound by the reading of the weights.  31 of 256 experts' gate and up rows (2 x 2048 x 7168,
// 485 MB of codes and scales) take 95 us, 5.1 TB/s.  The loads alone, in this shape, take 87
// (a bare read of such rows in the same lane order 76); the vector ALU is 44% busy.  Slices
// that interleave, 8 waves a workgroup, runs of tiles with the ring going on into the next, all
// eight waves on one tile, rings of 2 or 8 blocks, 12, 20 or 24 waves a CU and x staged before
// the first weights measured 94 to 108.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

constexpr int kMaxSlots = 1024;
// LDS for staged x, per wave: with a slice of K per wave two blocks of 13 rows fit, and the
// workgroups that the registers allow (16 waves a CU) fit the CU's LDS.
constexpr int kWaveBytes = 7168;
// Row tiles of a pass where experts have many slots, and the staged x of their workgroups:
// with K in 2 slices two blocks of 48 rows.
constexpr int kManyTiles = 3, kManyBytes = 14336;
constexpr int kRing = 4;                // blocks of codes a wave has in flight (few rows)

__device__ __forceinline__ void store_out(void* y, size_t i, float v, bool bf16) {
  if (bf16)
    static_cast<__bf16*>(y)[i] = (__bf16)v;              // round to nearest even, NaN kept
  else
    static_cast<float*>(y)[i] = v;
}

struct MatvecArgs {
  const void* x;
  const uint8_t* q;
  const float* s7;
  const int32_t* idx;
  int S, G, N, K;
  void* y;
  int y_bf16;       // 1: bf16; 0: fp32; 2: fp32 as three bf16 rows (3 s + part)
  int ks_log;       // log2 of the slices of K
  int spp;          // slots of a pass
  int k;            // joined form: slots of a token and their weights
  const float* wgt;
  uint32_t inv_div; // ceil(2^20 / x_div)
};

// How x is held: bf16 rows, three bf16 rows per row (hi, mid, lo), or fp32 rows that are
// split as they are loaded.
enum XForm { kXBf16, kXParts, kXF32 };

// One word of 8 codes -> two bf16 operands whose sum is q / 1024, by the packed FP4
// conversion (two values an instruction).  A code's sign and magnitude m = 4 b + l read as
// FP4 (e2m1) are m / 2 for l alone and 2 for the bit b alone, so two masks split the word into
// parts that convert exactly: 10 operations per word, against 14 for a byte-permute lookup of
// bf16(m) and sign, and the matrix core has the time for the second product.  Byte i
// holds the codes i and 4 + i, so the values come in the order 0 4 1 5 2 6 3 7, and x is
// staged in that order.  With the power of two a group's sum stays below the largest |x| of
// the row (128 * 7 / 1024 < 1) and cannot overflow before its scale is applied; the
// outputs take the 1024 back.
constexpr float kCodeUnit = 1024.0f;
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
__device__ __forceinline__ v8bf fp4_codes(uint32_t w) {
  constexpr float unit = 2.0f / kCodeUnit;
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, unit, 0);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, unit, 1);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, unit, 2);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, unit, 3);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// p + the products of 8 codes a lane and 8 values of x
__device__ __forceinline__ v4f mul_codes(v8bf x, uint32_t w, v4f p) {
  p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, fp4_codes(w & 0xBBBBBBBBu), p, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, fp4_codes(w & 0xCCCCCCCCu), p, 0, 0, 0);
}

__device__ __forceinline__ void swap32(int& a, int& b) {
  const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)a, (uint32_t)b, false, false);
  a = (int)r[0];
  b = (int)r[1];
}
__device__ __forceinline__ void swap16(int& a, int& b) {
  const auto r = __builtin_amdgcn_permlane16_swap((uint32_t)a, (uint32_t)b, false, false);
  a = (int)r[0];
  b = (int)r[1];
}

// A lane (row l % 16, h = l / 16) loads the 4 words 4 h .. 4 h + 3 of a 128-deep block's 16
// words of 8 codes.  One matrix instruction sums over its lanes' h, so its four words must
// lie in one group: for 64- and 32-wide groups words are exchanged between the four lanes
// of a row.  Afterwards register i of lane h holds word word_of(h, i).
template <int GROUP>
__device__ __forceinline__ void regroup(v4i& w) {
  if constexpr (GROUP < 128) {
    int a = w[0], b = w[1], c = w[2], d = w[3];
    swap32(a, c);
    swap32(b, d);
    if constexpr (GROUP == 32) {
      swap16(a, b);
      swap16(c, d);
    }
    w = v4i{a, b, c, d};
  }
}
template <int GROUP>
__device__ __forceinline__ constexpr int word_of(int h, int i) {
  return GROUP == 128 ? 4 * h + i
         : GROUP == 64 ? 8 * (i >> 1) + 4 * (h & 1) + (i & 1) + 2 * (h >> 1)
                       : 4 * i + h;
}

// 8 bf16 values in the order of the expanded codes
__device__ __forceinline__ v4i code_order(v4i x) {
  return v4i{(int)__builtin_amdgcn_perm((uint32_t)x[2], (uint32_t)x[0], 0x05040100u),
             (int)__builtin_amdgcn_perm((uint32_t)x[2], (uint32_t)x[0], 0x07060302u),
             (int)__builtin_amdgcn_perm((uint32_t)x[3], (uint32_t)x[1], 0x05040100u),
             (int)__builtin_amdgcn_perm((uint32_t)x[3], (uint32_t)x[1], 0x07060302u)};
}

// The upper half words of 8 fp32 values, i.e. their leading 8 bits as bf16, in the order of
// the expanded codes; they are then taken away from the values.
__device__ __forceinline__ v4i take_part(float (&v)[8]) {
  v4i r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = (int)__builtin_amdgcn_perm(__float_as_uint(v[4 + i]), __float_as_uint(v[i]),
                                      0x07060302u);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] -= __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u);
  return r;
}

// fp32 -> its part p (0, 1, 2) as bf16 bits
__device__ __forceinline__ uint16_t part_bits(float v, int p) {
  if (p > 0) v -= __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
  if (p > 1) v -= __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
  return (uint16_t)(__float_as_uint(v) >> 16);
}

// silu with exp and a division correct to fp32 (the epilogue runs once per output)
__device__ __forceinline__ float silu_f32(float z) { return z / (1.0f + expf(-z)); }

}  // namespace

// JOIN: the outputs of a token are the sums over its k slots, times the slots' weights, and
// each slot's product is a wave's (or several waves', over K).
// MT > 1: passes of 16 MT rows, for which a code is expanded once.
template <int NW, int XF, bool SWIGLU, int R, int GROUP, bool JOIN, int MT>
__global__ __launch_bounds__(64 * NW, MT > 1 ? 2 : 4) void matvec_int4_kernel(MatvecArgs a) {
  static_assert(!SWIGLU || R == 2, "SwiGLU: one gate and one up tile");
  constexpr int NT = NW * 64;
  constexpr int RPS = XF == kXBf16 ? 1 : 3;        // left-operand rows per slot
  constexpr int GP = 128 / GROUP;                  // groups per block
  constexpr int NO = SWIGLU ? 16 : 16 * R;         // outputs per wave
  constexpr int SCH = 16 / GP, SST = 17;           // blocks of staged scales, floats per row
  constexpr int XBYTES = NW * (MT > 1 ? kManyBytes : kWaveBytes);
  static_assert(NW * R * MT * 4 * 64 * 4 <= XBYTES, "the waves' sums reuse the staging region");
  __shared__ uint16_t slots[kMaxSlots];            // slots of the expert
  // A staged row ends 16 bytes off a multiple of the banks, so that the rows of one read fall
  // into different ones.
  __shared__ __attribute__((aligned(16))) uint8_t xs_mem[XBYTES];
  __shared__ float sc_mem[NW][16 * R * SST];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 4, l16 = lane & 15;
  const int N = a.N, K = a.K, S = a.S;
  // wave ti * KS + ks: K slice ks of the workgroup's tile ti (JOIN: of the round's slot ti)
  const int KS = 1 << a.ks_log, TW = NW >> a.ks_log;
  const int ks = wid & (KS - 1), ti = wid >> a.ks_log;
  const int nb0 = blockIdx.x * (JOIN ? NO : TW * NO), n0 = nb0 + (JOIN ? 0 : ti * NO);
  const bool y3 = a.y_bf16 == 2;
  auto store = [&](int s, int n, float v) {
    if (y3) {
#pragma unroll
      for (int p = 0; p < 3; ++p)
        static_cast<uint16_t*>(a.y)[((size_t)s * 3 + p) * N + n] = part_bits(v, p);
    } else {
      store_out(a.y, (size_t)s * N + n, v, a.y_bf16 == 1);
    }
  };

  // the expert and its slots, in slot order; every wave finds them for itself, so that the
  // first weights are asked for before the waves meet
  int e = 0, cnt = S;
  if (!JOIN && a.idx) {
    // S <= G: workgroup row y stands for slot y and works if it is its expert's first slot
    const int me = blockIdx.y;
    const bool by_slot = S <= a.G;
    int es = a.idx[min(lane, S - 1)];
    e = __builtin_amdgcn_readfirstlane(by_slot ? a.idx[me] : me);
    const bool live = e >= 0 && e < a.G;
    if (!live && me != 0) return;
    cnt = 0;
    int first = S;
    for (int s0 = 0; s0 < S; s0 += 64) {
      const int s = s0 + lane;
      if (s0 > 0) es = a.idx[min(s, S - 1)];
      const unsigned long long m = __ballot(s < S && es == e);
      if (m && first == S) first = s0 + __builtin_ctzll(m);
      if (wid == 0 && s < S) {
        if (me == 0 && blockIdx.z == 0 && (es < 0 || es >= a.G))   // no expert: zeros
#pragma unroll 1
          for (int c = 0; c < min(TW * NO, N - nb0); ++c) store(s, nb0 + c, 0.f);
        if (es == e) slots[cnt + __popcll(m & ((1ull << lane) - 1ull))] = (uint16_t)s;
      }
      cnt += __popcll(m);
    }
    if (!live || cnt == 0 || (by_slot && first != me)) return;
  }

  // weight rows of the wave's tiles and their scales, bounded by their buffers: rows past N
  // (and all rows of a slot without an expert) read as zeros and are not stored
  const int KG = K / GROUP;
  __amdgpu_buffer_rsrc_t wbuf[R], sbuf[R];
  auto rows_of = [&](int expert, int limit) {
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const int n = n0 + (SWIGLU ? 0 : 16 * t);
      const int rows = __builtin_amdgcn_readfirstlane(max(min(16, limit - n), 0));
      const size_t row0 = (size_t)expert * (SWIGLU ? 2 * (size_t)N : N) +
                          (SWIGLU ? (size_t)t * N : 0) + (rows ? n : 0);
      wbuf[t] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.q + row0 * (K / 2)),
                                                  (short)0, rows * (K / 2), 0x00020000);
      sbuf[t] = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.s7 + row0 * KG), (short)0,
                                                  rows * KG * 4, 0x00020000);
    }
  };
  constexpr uint32_t kNowhere = 0xFFFFFF00u;          // a lane offset beyond every bound
  const int KB = (K + 127) / 128;
  const int b0 = (int)(((long)ks * KB) >> a.ks_log), b1 = (int)(((long)(ks + 1) * KB) >> a.ks_log);
  const int nb_max = (KB + KS - 1) >> a.ks_log;      // blocks of the longest slice
  // codes of block kb: nothing is read past the slice; past the end of the row its last
  // piece again (x is zero there)
  const uint32_t wrow = (uint32_t)l16 * (uint32_t)(K / 2);
  auto load_w = [&](v4i (&w)[R], int kb) {
    uint32_t at = wrow + min((uint32_t)kb * 64u + 16u * h, (uint32_t)(K / 2 - 16));
    at = kb < b1 ? at : kNowhere;
#pragma unroll
    for (int t = 0; t < R; ++t)
      w[t] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(wbuf[t], at, 0, 0));
  };
  // Scales of SCH blocks from kb on, 16 groups of a row: a lane takes 4 groups of row lane / 4
  // (64 contiguous bytes a row).  They wait in registers while the blocks before them are
  // computed and then move to LDS, with zeros behind the row's last group.
  float* sc = sc_mem[wid];
  auto load_s = [&](v4f (&sv)[R], int kb) {
    const int g = kb * GP + 4 * (lane & 3);
    const uint32_t at = g < b1 * GP ? (uint32_t)((lane >> 2) * KG + g) * 4u : kNowhere;
#pragma unroll
    for (int t = 0; t < R; ++t)
      sv[t] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(sbuf[t], at, 0, 0));
  };
  auto put_s = [&](const v4f (&sv)[R], int kb) {
    const int left = KG - (kb * GP + 4 * (lane & 3));
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sc[(16 * t + (lane >> 2)) * SST + 4 * (lane & 3) + i] = i < left ? sv[t][i] : 0.f;
  };

  // spp slots a pass.  JOIN: the waves' next slots of the token, one each, whose rows the wave
  // stages by itself
  const int room = JOIN ? kWaveBytes : (XBYTES >> a.ks_log) & ~15;
  const int spp = JOIN ? TW : a.spp;
  const int s_end = JOIN ? a.k : cnt, s_step = JOIN ? TW : gridDim.z * spp;
  const int stage_i = JOIN ? 0 : ti, stage_n = JOIN ? 1 : TW;
  float tot[R] = {};
  if (!JOIN) rows_of(e, N);
  for (int s0 = JOIN ? 0 : blockIdx.z * spp; s0 < s_end; s0 += s_step) {
    const int ns = JOIN ? 1 : min(spp, cnt - s0), nr = ns * RPS;
    const int own = JOIN ? (int)blockIdx.y * a.k + min(s0 + ti, a.k - 1) : 0;
    bool valid = true;
    if constexpr (JOIN) {
      e = a.idx[own];
      valid = s0 + ti < a.k && e >= 0 && e < a.G;
      rows_of(valid ? e : 0, valid ? N : 0);
    }
    auto slot_at = [&](int i) { return JOIN ? own : a.idx ? (int)slots[s0 + i] : s0 + i; };
    // slot / x_div by a multiplication: exact for slots below 1024
    auto x_row = [&](int slot) { return (size_t)(((uint32_t)slot * a.inv_div) >> 20); };
    v4f acc[R][MT];
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[t][m] = v4f{0.f, 0.f, 0.f, 0.f};

    auto run = [&](auto MRC) {
      constexpr int MR = decltype(MRC)::value;
      constexpr int U = MR == 1 ? kRing : 2;
      static_assert(4 * (U * 256 + 16) <= kWaveBytes || MR > 1, "room for a chunk of U blocks");
      static_assert(SCH % U == 0, "the ring's turns end with the staged scales");
      // blocks of a chunk, a multiple of the ring's; bytes per staged row and per slice
      const int ch = min((room / nr - 16) / 256, max(nb_max + U - 1, U)) / U * U;
      const int xst = ch * 256 + 16;
      uint8_t* xs = xs_mem + (JOIN ? wid : ks) * room;
      // left-operand row i of a tile sits at matrix row 4 (i % 4) + i / 4, so that up to four
      // rows leave each lane one sum; rows past nr repeat the last one
      const uint8_t* xlane[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        xlane[m] = xs + min(16 * m + (l16 >> 2) + 4 * (l16 & 3), nr - 1) * xst;

      // x rows of the blocks [c0, c0 + n) of this slice by the slice's waves, zeros past K
      // and in the blocks that fill up the ring's last turn; all loads of a turn are issued
      // before the first is waited for (48 rows: a slice's whole chunk by two waves)
      auto stage = [&](int c0, int n) {
        const int nb = (n + U - 1) / U * U;
        const int nu = (XF == kXF32 ? ns : nr) * nb;   // 16-lane units: a row's block
        const float inv = 1.0f / (float)nb;
        constexpr int XV = XF == kXF32 ? 2 : 1, TURN = (MT > 1 ? 12 : 4) / XV;
        for (int u0 = stage_i * 4; u0 < nu; u0 += stage_n * 4 * TURN) {
          v4i v[TURN][XV];
          int dst[TURN];
#pragma unroll
          for (int j = 0; j < TURN; ++j) {
            const int u = u0 + stage_n * 4 * j + h;
            const int i = (int)(((float)u + 0.5f) * inv), blk = u - i * nb;
            const int k = (c0 + blk) * 128 + 8 * l16;
            dst[j] = u < nu ? (XF == kXF32 ? 3 * i : i) * xst + blk * 256 + 16 * l16 : -1;
#pragma unroll
            for (int z = 0; z < XV; ++z) v[j][z] = v4i{0, 0, 0, 0};
            if (u < nu && blk < n && k < K) {
              const size_t row = x_row(slot_at(XF == kXParts ? i / 3 : i));
              if constexpr (XF == kXF32) {
                const float* p = static_cast<const float*>(a.x) + row * K + k;
                v[j][0] = *reinterpret_cast<const v4i*>(p);
                v[j][1] = *reinterpret_cast<const v4i*>(p + 4);
              } else {
                const uint16_t* p = static_cast<const uint16_t*>(a.x) +
                                    (XF == kXParts ? row * 3 + i % 3 : row) * K + k;
                v[j][0] = *reinterpret_cast<const v4i*>(p);
              }
            }
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < TURN; ++j) {
            if (dst[j] < 0) continue;
            if constexpr (XF == kXF32) {
              float f[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) f[z] = __int_as_float(v[j][z >> 2][z & 3]);
#pragma unroll
              for (int p = 0; p < 3; ++p)
                *reinterpret_cast<v4i*>(xs + dst[j] + p * xst) = take_part(f);
            } else {
              *reinterpret_cast<v4i*>(xs + dst[j]) = code_order(v[j][0]);
            }
          }
        }
      };

      // block `at` of the chunk, block `sat` of the staged scales
      auto compute = [&](v4i (&w)[R], int at, int sat) {
        if constexpr (MT > 1) {
#pragma unroll
          for (int t = 0; t < R; ++t) {
            regroup<GROUP>(w[t]);
#pragma unroll
            for (int g = 0; g < GP; ++g) {
              v4f p[MT];
#pragma unroll
              for (int m = 0; m < MT; ++m) p[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = g * (4 / GP); i < (g + 1) * (4 / GP); ++i) {
                v8bf xa[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m)
                  xa[m] = *reinterpret_cast<const v8bf*>(xlane[m] + at * 256 +
                                                         16 * word_of<GROUP>(h, i));
                const v8bf lo = fp4_codes((uint32_t)w[t][i] & 0xBBBBBBBBu);
                const v8bf hi = fp4_codes((uint32_t)w[t][i] & 0xCCCCCCCCu);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                  p[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[m], lo, p[m], 0, 0, 0);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                  p[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[m], hi, p[m], 0, 0, 0);
              }
              const float s = sc[(16 * t + l16) * SST + sat * GP + g];
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < MR; ++r) acc[t][m][r] = fmaf(s, p[m][r], acc[t][m][r]);
            }
          }
          return;
        }
        v8bf xa[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          xa[i] = *reinterpret_cast<const v8bf*>(xlane[0] + at * 256 + 16 * word_of<GROUP>(h, i));
#pragma unroll
        for (int t = 0; t < R; ++t) {
          regroup<GROUP>(w[t]);
#pragma unroll
          for (int g = 0; g < GP; ++g) {
            v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = g * (4 / GP); i < (g + 1) * (4 / GP); ++i)
              p = mul_codes(xa[i], (uint32_t)w[t][i], p);
            const float s = sc[(16 * t + l16) * SST + sat * GP + g];
#pragma unroll
            for (int r = 0; r < MR; ++r) acc[t][0][r] = fmaf(s, p[r], acc[t][0][r]);
          }
        }
      };
      // U blocks of codes and a chunk of scales in flight; a block past the slice multiplies
      // zeros (a branch around it would let the compiler move the loads into it, next to
      // their use)
      v4i ring[U][R];
      v4f sv[R];
      load_s(sv, b0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        load_w(ring[u], b0 + u);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (!JOIN && a.idx && s0 == (int)blockIdx.z * spp) __syncthreads();   // slots
      for (int c = 0; c < nb_max; c += ch) {
        const int c0 = b0 + c, nb = min(ch, b1 - c0);
        if (c > 0) __syncthreads();                    // every wave is done with the chunk
        stage(c0, max(nb, 0));
        __syncthreads();
        for (int j = 0; j < nb; j += U) {
          const int sat = (c + j) % SCH;
          if (sat == 0) {
            put_s(sv, c0 + j);
            load_s(sv, c0 + j + SCH);
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            compute(ring[u], j + u, sat + u);
            load_w(ring[u], c0 + j + u + U);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      if constexpr (JOIN) return;
      __syncthreads();
      float* red = reinterpret_cast<float*>(xs_mem) + wid * (R * MT * 4 * 64);
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < MR; ++r) red[((t * MT + m) * 4 + r) * 64 + lane] = acc[t][m][r];
    };
    if constexpr (JOIN) {
      run(std::integral_constant<int, 1>{});
#pragma unroll
      for (int t = 0; t < R; ++t) tot[t] = valid ? fmaf(a.wgt[own], acc[t][0][0], tot[t]) : tot[t];
      continue;
    } else if (MT == 1 && nr <= 4) {
      run(std::integral_constant<int, 1>{});
    } else {
      run(std::integral_constant<int, 4>{});
    }
    __syncthreads();

    // outputs: row i's sum over the slices sits in lanes 16 (i % 4) + n, register i / 4
    const float* red = reinterpret_cast<const float*>(xs_mem);
    for (int o = tid; o < ns * TW * NO; o += NT) {
      const int c = o % NO, w0 = ((o / NO) & (TW - 1)) << a.ks_log;
      const int sl = (o / NO) / TW, n = nb0 + o % (TW * NO);
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int t2 = 0; t2 < (SWIGLU ? 2 : 1); ++t2) {
        const int t = SWIGLU ? t2 : c >> 4;
#pragma unroll
        for (int p = RPS - 1; p >= 0; --p) {
          const int i = sl * RPS + p;                  // (tile i / 16, register i / 4 % 4)
          const int at = (t * MT * 4 + (i >> 2)) * 64 + 16 * (i & 3) + (c & 15);
          float z = 0.f;
          for (int w = 0; w < KS; ++w) z += red[(w0 + w) * (R * MT * 4 * 64) + at];
          v[t2] += z;
        }
        v[t2] *= kCodeUnit;
      }
      if (n < N) store(slot_at(sl), n, SWIGLU ? silu_f32(v[0]) * v[1] : v[0]);
    }
    __syncthreads();
  }
  if constexpr (JOIN) {
    // row p of the staged three is a slot's part p: lanes 16 p + n
    __syncthreads();
    float* red = reinterpret_cast<float*>(xs_mem);
#pragma unroll
    for (int t = 0; t < R; ++t) red[(wid * R + t) * 64 + lane] = tot[t];
    __syncthreads();
    if (tid < NO && nb0 + tid < N) {
      float v = 0.f;
#pragma unroll
      for (int p = RPS - 1; p >= 0; --p) {
        float z = 0.f;
        for (int w = 0; w < NW; ++w) z += red[(w * R + (tid >> 4)) * 64 + 16 * p + (tid & 15)];
        v += z;
      }
      store((int)blockIdx.y, nb0 + tid, v * kCodeUnit);
    }
  }
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

template <int XF, bool SWIGLU, int R, int GROUP>
hipError_t launch_matvec_r(MatvecArgs a, unsigned gy, hipStream_t s) {
  constexpr int NW = 4;
  const int per = (SWIGLU ? 16 : 16 * R) * (NW >> a.ks_log);
  const unsigned gx = (unsigned)((a.N + per - 1) / per);
  // A pass takes 16 rows, or what two blocks of a slice's staging region hold; with few
  // workgroups the passes over an expert's slots run beside each other, and while they fit the
  // chip at once they take up to 4 rows, whose sums are one register a tile (16 bf16 rows, 2048
  // x 7168: 12.2 us against 17.2, 1003 x 4128: 9.2, 13.8; 4 fp32 rows 11.0, 12.9; but 8 fp32
  // rows, 1024 workgroups, 16.1, 13.1).
  constexpr int RPS = XF == kXBf16 ? 1 : 3, SMALL = 4 / RPS;
  const long wgs = (long)gx * gy, small = (a.S + SMALL - 1) / SMALL;
  a.spp = wgs * small <= 512 ? SMALL : std::min(16, (NW * kWaveBytes >> a.ks_log) / 528) / RPS;
  const unsigned gz = (unsigned)std::max<long>(
      1, std::min<long>((a.S + a.spp - 1) / a.spp, 512 / wgs));
  hipLaunchKernelGGL((matvec_int4_kernel<NW, XF, SWIGLU, R, GROUP, false, 1>), dim3(gx, gy, gz),
                     dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}

// Experts with many slots: 48 rows a pass (16 fp32 rows).
template <int XF, bool SWIGLU, int GROUP>
hipError_t launch_matvec_many(MatvecArgs a, unsigned gy, hipStream_t s) {
  constexpr int NW = 4, RPS = XF == kXBf16 ? 1 : 3;
  const int per = (SWIGLU ? 16 : 32) * NW;
  a.ks_log = (long)((a.N + per - 1) / per) * gy >= 512 ? 0 : 1;
  const unsigned gx = (unsigned)((a.N + (per >> a.ks_log) - 1) / (per >> a.ks_log));
  a.spp = 16 * kManyTiles / RPS;
  const unsigned gz = (unsigned)std::max<long>(
      1, std::min<long>((a.S + a.spp - 1) / a.spp, 512 / ((long)gx * gy)));
  hipLaunchKernelGGL((matvec_int4_kernel<NW, XF, SWIGLU, 2, GROUP, false, kManyTiles>),
                     dim3(gx, gy, gz), dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}

template <int XF, int GROUP>
hipError_t launch_matvec_g(MatvecArgs a, bool swiglu, hipStream_t s) {
  const unsigned gy = a.idx ? (unsigned)(a.S <= a.G ? a.S : a.G) : 1u;
  // Where experts have more than 16 rows of x on average, 48 rows a pass save reading and
  // expanding the codes again, if the products are large enough to fill the chip with fewer
  // workgroups (by weight rows times passes: 128 bf16 rows of 4096 x 2048, 33k, 19 us against
  // 29, 64 of them, 16k, 20 against 16; 64 fp32 rows of 2048 x 7168, 25k, 43 against 52, 32 of
  // them, 12k, 43 against 27; 24 tokens' FFN with all 4 experts, 7168 x 2048, in fp32 92 against
  // 178).
  constexpr int RPS = XF == kXBf16 ? 1 : 3;
  const long mean = ((long)a.S * RPS + (a.idx ? a.G : 1) - 1) / (a.idx ? a.G : 1);
  if (mean > 16 && (mean + 15) / 16 * gy * a.N * (swiglu ? 2 : 1) >= 20000) {
    if (!swiglu) return launch_matvec_many<XF, false, GROUP>(a, gy, s);
    if constexpr (XF != kXParts) return launch_matvec_many<XF, true, GROUP>(a, gy, s);
  }
  const long tiles = ((long)a.N + (swiglu ? 15 : 31)) / (swiglu ? 16 : 32) * gy;
  // Enough waves for the chip, in slices long enough to stream: K whole for short rows of
  // which there are many (101 experts' down products, 7168 x 2048 each: 165 us, in 2 slices
  // 182), in 2 slices from 1024 wave tiles on (8 experts' gate and up products, 2 x 2048 x
  // 7168 each: 30.5 us, in 4 slices 32.5; 101 experts': 300 us, whole 317), else in 4.
  a.ks_log = tiles >= 2048 && a.K <= 2048 ? 0 : tiles >= 1024 ? 1 : 2;
  if (swiglu) {
    if constexpr (XF == kXParts)
      return hipErrorInvalidValue;                   // (no caller has such rows)
    else
      return launch_matvec_r<XF, true, 2, GROUP>(a, gy, s);
  }
  // 16-row tiles where 32-row ones would leave CUs idle
  return tiles < 256 ? launch_matvec_r<XF, false, 1, GROUP>(a, gy, s)
                     : launch_matvec_r<XF, false, 2, GROUP>(a, gy, s);
}

template <int GROUP>
hipError_t launch_join_g(MatvecArgs a, int T, hipStream_t s) {
  constexpr int NW = 8;
  a.ks_log = a.k > 4 ? 0 : a.k > 2 ? 1 : a.k > 1 ? 2 : 3;
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)T), block(64 * NW);
  hipLaunchKernelGGL((matvec_int4_kernel<NW, kXParts, false, 1, GROUP, true, 1>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int XF>
hipError_t launch_matvec_x(const MatvecArgs& a, int group, bool swiglu, hipStream_t s) {
  return group == 32   ? launch_matvec_g<XF, 32>(a, swiglu, s)
         : group == 64 ? launch_matvec_g<XF, 64>(a, swiglu, s)
                       : launch_matvec_g<XF, 128>(a, swiglu, s);
}

hipError_t launch_matvec_int4(const void* x, FewDtype x_dt, int x_div, const uint8_t* q,
                              const float* s7, int group, const int32_t* idx, int S, int G, int N,
                              int K, bool swiglu, void* y, FewDtype y_dt, hipStream_t s) {
  const MatvecArgs a{x, q, s7, idx, S, G, N, K, y,
                     y_dt == kFewBf16 ? 1 : y_dt == kFewParts ? 2 : 0, 0, 0, 0, nullptr,
                     (uint32_t)(((1u << 20) + (uint32_t)x_div - 1) / (uint32_t)x_div)};
  return x_dt == kFewBf16    ? launch_matvec_x<kXBf16>(a, group, swiglu, s)
         : x_dt == kFewParts ? launch_matvec_x<kXParts>(a, group, swiglu, s)
                             : launch_matvec_x<kXF32>(a, group, swiglu, s);
}

hipError_t launch_join_int4(const void* h, const uint8_t* q, const float* s7, int group,
                            const int32_t* idx, const float* w, int T, int k, int E, int d, int I,
                            void* y, bool y_bf16, hipStream_t s) {
  const MatvecArgs a{h, q, s7, idx, T * k, E, d, I, y, y_bf16 ? 1 : 0, 0, 0, k, w, 1u << 20};
  return group == 32   ? launch_join_g<32>(a, T, s)
         : group == 64 ? launch_join_g<64>(a, T, s)
                       : launch_join_g<128>(a, T, s);
}

hipError_t launch_few_combine(const float* o, const int32_t* idx, const float* w, int T, int k,
                              int E, int d, void* y, bool y_bf16, hipStream_t s) {
  hipLaunchKernelGGL(few_combine_kernel, dim3((unsigned)((d + 255) / 256), (unsigned)T), dim3(256),
                     0, s, o, idx, w, k, E, d, y, y_bf16);
  return hipGetLastError();
}

}  // namespace moe
