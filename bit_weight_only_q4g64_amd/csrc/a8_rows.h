// Rows in 8 bits: the quantizer and the residual RMS norm that feed the
// 8-bit products.
//
// A row of K values becomes K OCP E4M3 codes and one float32 scale per group
// of 128 columns (the last group may be half a group):
//   a = max(max |x| over the group, 448 * 2^-126),  s = a / 448,
//   q = e4m3(x * (448 / a)),  rounded to nearest, ties to even.
// 448 is the largest finite E4M3 value, so the largest member of a group maps
// to +-448 and nothing overflows (x * (448 / a) is at most 448 (1 + 2^-23),
// which rounds to 448). The floor on a keeps s a normal float32 and 448 / a
// finite: a group of zeros gets s = 2^-126 and zero codes. A group that holds
// a NaN or an infinity gets the scale NaN and NaN codes, so the rows that a
// product makes of it are NaN. The maximum is taken over the bit patterns
// without the sign, which order like the magnitudes and put NaN on top.
//
// Both kernels are bound by memory. A lane holds 8 consecutive columns, 16
// lanes (one DPP row) a group, so a group's maximum takes four lane
// rotations and no LDS.
#pragma once

#include "common.h"

namespace q4 {

constexpr int kA8Group = 128;
constexpr float kE4m3Max = 448.0f;
constexpr float kA8Floor = 448.0f * 0x1p-126f;

enum { kRowNone = 0, kRowBf16 = 1, kRowF32 = 2, kRowA8 = 3 };

// One step of a reduction over the 16 lanes of a DPP row: the value of the
// lane N places round.
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x120 + N, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t umax32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = umax32(v, row_ror<8>(v));
  v = umax32(v, row_ror<4>(v));
  v = umax32(v, row_ror<2>(v));
  return umax32(v, row_ror<1>(v));
}

// The scale and the factor of a group whose largest magnitude has these bits.
// a / 448 without a division: with y = 1 / 448 rounded, q = a y is within one
// unit of it, fma(-448, q, a) is the exact remainder, and q + y * remainder
// rounds to the quotient (checked for every significand).
__device__ __forceinline__ void a8_scale(uint32_t abits, float& s, float& r) {
  constexpr float y = 1.0f / kE4m3Max;
  const float a = __builtin_fmaxf(__uint_as_float(abits), kA8Floor);
  const float q = a * y;
  s = __builtin_fmaf(__builtin_fmaf(-kE4m3Max, q, a), y, q);
  r = kE4m3Max / a;
  if (abits >= 0x7F800000u) s = r = __uint_as_float(0x7FC00000u);
}

// 8 values -> 8 codes, in order.
__device__ __forceinline__ u32x2 a8_codes(const float (&v)[8], float r) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * r, v[1] * r, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * r, v[3] * r, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * r, v[5] * r, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * r, v[7] * r, hi, true);
  return u32x2{(uint32_t)lo, (uint32_t)hi};
}

__device__ __forceinline__ uint32_t abs_max8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = umax32(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return m;
}

// 8 consecutive values of a row as loaded: 16 bytes of bf16 or 32 of float32.
template <int TYPE>
struct Raw8 {
  u32x4 w[TYPE == kRowF32 ? 2 : 1];
};
template <int TYPE>
__device__ __forceinline__ Raw8<TYPE> load8(const void* row, int col) {
  Raw8<TYPE> r;
  if constexpr (TYPE == kRowF32) {
    const u32x4* p = (const u32x4*)((const float*)row + col);
    r.w[0] = p[0];
    r.w[1] = p[1];
  } else {
    r.w[0] = *(const u32x4*)((const uint16_t*)row + col);
  }
  return r;
}
template <int TYPE>
__device__ __forceinline__ void to_f32(const Raw8<TYPE>& r, float (&v)[8]) {
  if constexpr (TYPE == kRowF32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r.w[e >> 2][e & 3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (e & 1) ? bf16_hi(r.w[0][e >> 1]) : bf16_lo(r.w[0][e >> 1]);
  }
}
// Two float32 -> packed bf16, to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ u32x4 pack_bf16x8(const float (&v)[8]) {
  return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

struct QuantA8Args {
  const void* x;
  int64_t ldx;
  int M, K, G;
  uint8_t* q;
  int64_t ldq;
  float* s;  // [G][lds]
  int64_t lds;
};

// A 16-lane team per (row, group), 8 columns a lane. Measured: 10.7 us at 8192 x
// 2048 bf16 with inputs that rotate through memory, 4.7 TB/s, near a copy's
// rate there; the scales' scattered 4-byte stores cost nothing that gathering
// them in LDS for runs of 16 would win back (12.4 us).
template <int TYPE>
__global__ __launch_bounds__(256) void quant_a8_kernel(QuantA8Args a) {
  const int team = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const int64_t id = (int64_t)blockIdx.x * 16 + team;
  const int m = (int)(id / a.G), g = (int)(id - (int64_t)m * a.G);
  if (m >= a.M) return;
  const uint8_t* row = (const uint8_t*)a.x + (int64_t)m * a.ldx * (TYPE == kRowF32 ? 4 : 2);
  const int col = g * kA8Group + lane * 8;
  float v[8] = {};
  if (col < a.K) to_f32<TYPE>(load8<TYPE>(row, col), v);
  float s, r;
  a8_scale(row_max(abs_max8(v)), s, r);
  if (col < a.K) *(u32x2*)(a.q + (int64_t)m * a.ldq + col) = a8_codes(v, r);
  if (lane == 0) a.s[(int64_t)g * a.lds + m] = s;
}

// Residual addition and RMS norm of a row:
//   h = x + residual, rounded to the residual's type (x itself without one),
//   y = (h * r) * gamma,  r = 1 / sqrt(sum h^2 / K + eps),
// y rounded to bf16, kept in float32, or quantized as above. The rounding of
// h is the one that storing it makes, so the result equals the norm of the
// stored sum. One pass: the row stays in registers between the sum of squares
// and the output.
struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* res;
  int64_t ldr;
  void* res_out;  // may be res or x: every element is read before it is written, by the same lane
  int64_t ldro;
  const float* gamma;
  float eps;
  int M, K;
  int out;  // kRowBf16, kRowF32 or kRowA8
  void* y;
  int64_t ldy;
  float* s;  // [G][lds] (kRowA8)
  int64_t lds;
};

// TPR lanes per row (one wave, or the workgroup of 256), CH chunks of 8
// columns per lane.
template <int TPR, int CH, int XT, int RT>
__global__ __launch_bounds__(256) void rms_norm_kernel(NormArgs a) {
  constexpr int kRows = 256 / TPR;
  const int m = (int)blockIdx.x * kRows + (int)threadIdx.x / TPR;
  const int lane = (int)threadIdx.x % TPR;
  if (TPR == 64 && m >= a.M) return;  // a whole wave (TPR = 256: the grid has one workgroup per row)
  const uint8_t* xrow = (const uint8_t*)a.x + (int64_t)m * a.ldx * (XT == kRowF32 ? 4 : 2);
  Raw8<XT> xr[CH];
  Raw8<RT == kRowNone ? kRowBf16 : RT> rr[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * TPR + lane) * 8;
    if (col < a.K) xr[c] = load8<XT>(xrow, col);
  }
  if constexpr (RT != kRowNone) {
    const uint8_t* rrow = (const uint8_t*)a.res + (int64_t)m * a.ldr * (RT == kRowF32 ? 4 : 2);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * TPR + lane) * 8;
      if (col < a.K) rr[c] = load8<RT>(rrow, col);
    }
  }
  f32x4 gm[CH][2];  // asked for before the sum, so that the output does not wait for them
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * TPR + lane) * 8;
    if (col < a.K) {
      gm[c][0] = *(const f32x4*)(a.gamma + col);
      gm[c][1] = *(const f32x4*)(a.gamma + col + 4);
    }
  }
  float v[CH][8];
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * TPR + lane) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = 0.0f;
    if (col < a.K) {
      to_f32<XT>(xr[c], v[c]);
      if constexpr (RT != kRowNone) {
        float w[8];
        to_f32<RT>(rr[c], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] += w[e];
        if constexpr (RT == kRowBf16) {
          const u32x4 p = pack_bf16x8(v[c]);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[c][e] = (e & 1) ? bf16_hi(p[e >> 1]) : bf16_lo(p[e >> 1]);
          *(u32x4*)((uint16_t*)a.res_out + (int64_t)m * a.ldro + col) = p;
        } else {
          u32x4* o = (u32x4*)((float*)a.res_out + (int64_t)m * a.ldro + col);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            o[h] = u32x4{__float_as_uint(v[c][4 * h]), __float_as_uint(v[c][4 * h + 1]), __float_as_uint(v[c][4 * h + 2]),
                         __float_as_uint(v[c][4 * h + 3])};
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[c][e], v[c][e], ss);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) ss += __shfl_xor(ss, o, 64);
  if constexpr (TPR == 256) {
    __shared__ float part[4];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
    __syncthreads();
    ss = (part[0] + part[1]) + (part[2] + part[3]);
  }
  const float mean = ss / (float)a.K + a.eps;
  float rn = 1.0f / __builtin_sqrtf(mean);
  // Squares below the least float32 or past the largest: summed again in
  // float64, whose range holds them. (From 2^-90 on, underflow takes less than
  // 2^-149 from the mean.) The factor may itself leave float32: half of its
  // power of two goes to the values first, exactly. The condition is the row's,
  // so all its lanes meet here; one value at a time, for few registers.
  // (Rows in range pay for the comparison: 1 x 2048 float32 2.29 us without
  // it, 2.31 with; 8192 x 2048 bf16 22.9 both.)
  if (__builtin_expect(!(mean >= 0x1p-90f && mean < __builtin_inff()), 0)) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s = __builtin_fma((double)v[c][e], (double)v[c][e], s);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
    if constexpr (TPR == 256) {
      __shared__ double wide[4];
      if ((threadIdx.x & 63) == 0) wide[threadIdx.x >> 6] = s;
      __syncthreads();
      s = (wide[0] + wide[1]) + (wide[2] + wide[3]);
    }
    const double r = 1.0 / __builtin_sqrt(s / (double)a.K + (double)a.eps);
    const int half = ((int)(__builtin_bit_cast(uint64_t, r) >> 52 & 0x7FF) - 1023) >> 1;
    const float first = __builtin_ldexpf(1.0f, half);
    rn = (float)__builtin_ldexp(r, -half);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] *= first;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * TPR + lane) * 8;
    if (col < a.K) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = (v[c][e] * rn) * gm[c][e >> 2][e & 3];
    }
    if (a.out == kRowA8) {
      float s, r;
      a8_scale(row_max(abs_max8(v[c])), s, r);  // lanes past K hold zeros
      if (col < a.K) {
        *(u32x2*)((uint8_t*)a.y + (int64_t)m * a.ldy + col) = a8_codes(v[c], r);
        if ((lane & 15) == 0) a.s[(int64_t)(col / kA8Group) * a.lds + m] = s;
      }
    } else if (col < a.K) {
      if (a.out == kRowBf16) {
        *(u32x4*)((uint16_t*)a.y + (int64_t)m * a.ldy + col) = pack_bf16x8(v[c]);
      } else {
        float* o = (float*)a.y + (int64_t)m * a.ldy + col;
        *(f32x4*)o = f32x4{v[c][0], v[c][1], v[c][2], v[c][3]};
        *(f32x4*)(o + 4) = f32x4{v[c][4], v[c][5], v[c][6], v[c][7]};
      }
    }
  }
}

}  // namespace q4
