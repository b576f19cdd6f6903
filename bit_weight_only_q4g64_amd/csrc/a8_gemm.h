// Products of 8-bit activations with block-FP8 weights: both sides E4M3 on the
// matrix cores, a float32 scale per row and 128 columns of the activations and
// per 128 x 128 block of the weights.
//
//   y[m][n] = sum_g (sx[g][m] * sw[n / 128][g]) * P_g[m][n],
//   P_g[m][n] = sum over the 128 columns k of group g of x8[m][k] * w8[n][k]
//
// One fma per output folds a group: acc = fma(sx * sw, P_g, acc). The scales
// are float32, so they cannot ride in the matrix instruction's own
// power-of-two scale operands.
//
// P_g comes from one of two instructions:
//   * the 8-bit one, 16 x 16 x 128 in one step, twice the bf16 rate and no
//     conversion. Its products are exact, but it adds them eight at a time
//     after aligning them to the largest, and drops what lies below 2^-13 of
//     that product's power of two (measured: 2^16 + 2^3 is exact, 2^16 + 2^2
//     gives 2^16 when the two share a run of 8 consecutive k; different runs
//     and the accumulator are added in float32, in the 32 x 32 x 64 form too:
//     2^16 + 2^-7 is exact). On normal values the result is 1.4e-5 off
//     (2-norm);
//   * the bf16 one, four chained steps of 16 x 16 x 32 on the codes converted
//     to bf16, which holds every E4M3 value. Products are exact and the sums
//     are float32: 1e-7 off.
// A float32 result takes the second: the first would leave it with 16 bits. So
// does an 8-bit result, whose scales are float32 (2.4e-5 off from the first).
// A bf16 result takes the first: its own rounding (at most 2^-8 of the value,
// 1.7e-3 in the 2-norm) is a hundred times larger than what the instruction
// drops.
//
// Weights are read in the layout pack_fp8b leaves: lane L of a wave owns, of a
// 16-column tile and 128 k, the 32 bytes of column L % 16 at
// k = 64 j + 32 h + 8 (L / 16) + e, e < 8, in two pieces of 16 (j = 0, 1).
// The instruction multiplies whatever k sits in the same lane group and byte
// of both operands, so the activations only need the same order: a lane loads
// 16 consecutive bytes of its row, at 16 u with u = 4 j + 2 (q % 2) + q / 2 for
// lane group q = L / 16, and one swap of 16-lane rows exchanges the halves
// that belong to the neighbouring group. No conversion remains.
//
// The weights are operand A, the activations operand B: D then holds row m in
// lane m % 16 and four consecutive columns in the lane's registers, so a
// lane's scale is one value per group for all its outputs of a weight block.
#pragma once

#include "a8_rows.h"
#include "common.h"

namespace q4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// D = A B + C on 16 x 16 x 128 E4M3 (format code 0 on both sides, no scales).
__device__ __forceinline__ f32x4 mfma_a8(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// The same from exact bf16 values: halves h = 0..3 of 32 k each.
__device__ __forceinline__ f32x4 mfma_exact(const bf16x8 (&a)[4], const bf16x8 (&b)[4]) {
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 4; ++h) d = mfma16(a[h], b[h], d);
  return d;
}

// The k offset of the 16 bytes a lane of group q loads for half j.
__host__ __device__ constexpr int a8_chunk(int q, int j) { return 16 * (4 * j + 2 * (q & 1) + (q >> 1)); }

// The four bf16 operands of an 8-bit one.
__device__ __forceinline__ void a8_bf16(i32x8 w, bf16x8 (&o)[4]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) o[h] = fp8_to_bf16((uint32_t)w[2 * h], (uint32_t)w[2 * h + 1]);
}

// Two loaded pieces of a row -> the operand in the weights' order.
__device__ __forceinline__ i32x8 a8_operand(u32x4 p0, u32x4 p1) {
  i32x8 r;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const u32x4 p = j ? p1 : p0;
    const auto s0 = __builtin_amdgcn_permlane16_swap(p[0], p[2], false, false);
    const auto s1 = __builtin_amdgcn_permlane16_swap(p[1], p[3], false, false);
    r[4 * j] = (int)s0[0];
    r[4 * j + 1] = (int)s1[0];
    r[4 * j + 2] = (int)s0[1];
    r[4 * j + 3] = (int)s1[1];
  }
  return r;
}

struct GemmA8Args {
  const uint8_t* pa;
  const uint8_t* pb;  // the second matrix of a SwiGLU pair
  int N, K;
  const uint8_t* x;
  int64_t ldx;
  const float* sx;  // [G][ldsx]
  int64_t ldsx;
  int M;
  int out;  // kRowF32, kRowBf16 or kRowA8
  void* y;
  int64_t ldy;
  float* sy;  // [ceil(N / 128)][ldsy] (kRowA8)
  int64_t ldsy;
};

// Four consecutive outputs of row m at column n.
__device__ __forceinline__ void a8_store4(const GemmA8Args& a, int64_t m, int n, f32x4 z) {
  if (a.out == kRowF32) *(f32x4*)((float*)a.y + m * a.ldy + n) = z;
  else *(u32x2*)((uint16_t*)a.y + m * a.ldy + n) = u32x2{pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3])};
}

// ---- few rows: operands straight from memory -------------------------------
// A workgroup owns MT tiles of 16 rows and NW x NT tiles of 16 columns (SwiGLU:
// of each matrix). Its NW x KW waves split the columns NW ways and the groups
// of K KW ways, each a run of consecutive groups; the KW partial sums of an
// output meet in LDS and are added in ascending order. Every wave loads its
// own operands from memory, D groups ahead.
//
// Up to 16 rows the weights bound it, read once and past the caches: 4 x 65536
// x 2048 22.7 us, 5.9 TB/s. A small matrix is a launch (2.2 us), one trip to
// memory and the join: 1 x 2048 x 2048 3.3 us; 16 x 2048 x 8192 7.7 us, on half
// the compute units (splitting K over workgroups too would take a second
// launch, or three round trips to hand the parts over). More waves per
// workgroup or loads further ahead are slower there (8 waves, 2 groups ahead;
// 16 waves, 2 ahead; 8 waves, 4 ahead): 8.4, 8.7 and 9.5 us with weights from
// memory, 4 x 65536 x 2048 22.7, 36 and 28 us. The kernels of more rows have
// too few registers for two groups (200 x 2048 x 8192 float32 on 32 x 32 24 us,
// with two 48 us).
template <bool EXACT_, int MT_, int NT_, bool SW_, int NW_, int KW_, int D_>
struct DirectA8 {
  static constexpr int MT = MT_, NT = NT_, NW = NW_, KW = KW_, D = D_;
  static constexpr bool SW = SW_, EXACT = EXACT_;
  static constexpr int kMats = SW ? 2 : 1, NS = NT * kMats;
  static constexpr int kThreads = NW * KW * 64;
  static constexpr int kRows = MT * 16, kTiles = NW * NT;
  static constexpr int kItems = (MT * NT + KW - 1) / KW;  // output tiles a wave finishes
  static constexpr size_t kLds = KW > 1 ? (size_t)KW * NW * MT * NS * 1024 : 0;
};

template <class C>
struct DirectFrag {
  u32x4 w[C::NS][2];
  u32x4 x[C::MT][2];
  float sx[C::MT];
  float sw[C::kMats];
};

template <class C, bool A8OUT>
__global__ __launch_bounds__(C::kThreads) void a8_direct_kernel(GemmA8Args a) {
  constexpr int MT = C::MT, NT = C::NT, NS = C::NS, KW = C::KW, NW = C::NW, D = C::D, kMats = C::kMats;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = wave % NW, kw = wave / NW;
  const int c = lane & 15, q = lane >> 4;
  const int P = (int)n_pairs(a.K), ntiles = a.N / kTileN;
  const int nblk = (ntiles + C::kTiles - 1) / C::kTiles;
  const int mb = (int)(blockIdx.x / nblk), nb = (int)blockIdx.x - mb * nblk;
  const int m0 = mb * C::kRows;
  const int rows = a.M - m0 < C::kRows ? a.M - m0 : C::kRows;
  const int t0 = (nb * NW + nw) * NT;
  const int tc = t0 < ntiles ? t0 : ntiles - 1;  // a wave past the last tile reads it and stores nothing
  const int64_t cb = codes_bytes(a.N, a.K, kFmtFp8);

  rsrc_t wres[kMats];
  const uint8_t* swp[kMats];
  const int tvalid = ntiles - tc < NT ? ntiles - tc : NT;
#pragma unroll
  for (int s = 0; s < kMats; ++s) {
    const uint8_t* p = s ? a.pb : a.pa;
    wres[s] = make_rsrc(p + (int64_t)tc * P * 2048, (uint32_t)(tvalid * P * 2048));
    swp[s] = p + cb + (int64_t)tc * P * kPairSbBytes;
  }
  const rsrc_t xres = make_rsrc(a.x + (int64_t)m0 * a.ldx, (uint32_t)((rows - 1) * a.ldx + a.K));
  uint32_t xoff[MT];
  int64_t mrow[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = mt * 16 + c;
    xoff[mt] = r < rows ? (uint32_t)(r * a.ldx + a8_chunk(q, 0)) : kOffBuffer;
    mrow[mt] = m0 + (r < rows ? r : rows - 1);
  }

  auto load = [&](DirectFrag<C>& f, int p) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int nt = s % NT;
      const uint32_t wo = nt < tvalid ? (uint32_t)lane * 16u : kOffBuffer;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t so = (uint32_t)(nt * P + p) * 2048u + j * 1024u;
        // 16 rows: the weights are read once; more: again for the next rows
        f.w[s][j] = MT == 1 ? buf_load16_nt(wres[s / NT], wo, so) : buf_load16(wres[s / NT], wo, so);
      }
    }
    const uint32_t tail = p * 128 + 64 < a.K ? 0u : kOffBuffer;  // half a group: its upper 64 columns are not the row's
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      f.x[mt][0] = buf_load16(xres, xoff[mt], (uint32_t)p * 128u);
      f.x[mt][1] = buf_load16(xres, (xoff[mt] + 64u) | tail, (uint32_t)p * 128u);
      f.sx[mt] = a.sx[(int64_t)p * a.ldsx + mrow[mt]];
    }
#pragma unroll
    for (int s = 0; s < kMats; ++s) f.sw[s] = *(const float*)(swp[s] + (int64_t)p * kPairSbBytes);
  };

  f32x4 acc[MT][NS];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[mt][s] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto fold = [&](const DirectFrag<C>& f) {
    i32x8 xb[MT];
    bf16x8 xe[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      xb[mt] = a8_operand(f.x[mt][0], f.x[mt][1]);
      if constexpr (C::EXACT) a8_bf16(xb[mt], xe[mt]);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const i32x8 wa = __builtin_bit_cast(i32x8, __builtin_shufflevector(f.w[s][0], f.w[s][1], 0, 1, 2, 3, 4, 5, 6, 7));
      bf16x8 we[4];
      if constexpr (C::EXACT) a8_bf16(wa, we);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        f32x4 d;
        if constexpr (C::EXACT) d = mfma_exact(we, xe[mt]);
        else d = mfma_a8(wa, xb[mt], f32x4{0.f, 0.f, 0.f, 0.f});
        const float sc = f.sx[mt] * f.sw[s / NT];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[mt][s][v] = __builtin_fmaf(sc, d[v], acc[mt][s][v]);
      }
    }
  };

  const int per = (P + KW - 1) / KW;
  const int p0 = kw * per, p1 = p0 + per < P ? p0 + per : P;
  DirectFrag<C> f[D];
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (p0 + d < p1) load(f[d], p0 + d);
  for (int p = p0; p < p1; p += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (p + d < p1) fold(f[d]);
      if (p + d + D < p1) load(f[d], p + d + D);
    }
  }

  // ---- join the K parts: wave (nw, kw) finishes the output tiles i = kw,
  // kw + KW, ... of its columns
  f32x4 z[C::kItems];
  if constexpr (KW > 1) {
    f32x4* part = (f32x4*)smem;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int s = 0; s < NS; ++s) part[(((size_t)kw * NW + nw) * MT * NS + mt * NS + s) * 64 + lane] = acc[mt][s];
    __syncthreads();
  }
#pragma unroll
  for (int it = 0; it < C::kItems; ++it) {
    const int i = it * KW + kw;
    if (i >= MT * NT) break;
    f32x4 sum[kMats];
#pragma unroll
    for (int s = 0; s < kMats; ++s) {
      if constexpr (KW > 1) {
        const int mt = i / NT, nt = i % NT;
        const f32x4* part = (const f32x4*)smem + ((size_t)nw * MT * NS + mt * NS + s * NT + nt) * 64 + lane;
        f32x4 t = part[0];
#pragma unroll
        for (int k = 1; k < KW; ++k) t += part[(size_t)k * NW * MT * NS * 64];
        sum[s] = t;
      } else {
        sum[s] = acc[it / NT][s * NT + it % NT];
      }
    }
    if constexpr (C::SW) {
#pragma unroll
      for (int v = 0; v < 4; ++v) z[it][v] = silu_f32(sum[0][v]) * sum[kMats - 1][v];
    } else {
      z[it] = sum[0];
    }
    const int r = (i / NT) * 16 + c, t = t0 + i % NT;
    if constexpr (!A8OUT) {
      if (r < rows && t < ntiles) a8_store4(a, (int64_t)m0 + r, t * kTileN + 4 * q, z[it]);
    }
  }
  if constexpr (A8OUT) {
    // the workgroup's columns are one group of 128 of the output
    static_assert(C::kTiles * kTileN == kA8Group, "one output group per workgroup");
    uint32_t* mx = (uint32_t*)(smem + C::kLds);  // [MT][8 tiles][16 rows]
#pragma unroll
    for (int it = 0; it < C::kItems; ++it) {
      const int i = it * KW + kw;
      if (i >= MT * NT) break;
      uint32_t b = 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) b = umax32(b, __float_as_uint(z[it][v]) & 0x7FFFFFFFu);
      if (t0 + i % NT >= ntiles) b = 0;
      b = umax32(b, (uint32_t)__shfl_xor((int)b, 16, 64));
      b = umax32(b, (uint32_t)__shfl_xor((int)b, 32, 64));
      if (q == 0) mx[((i / NT) * 8 + nw * NT + i % NT) * 16 + c] = b;
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < C::kItems; ++it) {
      const int i = it * KW + kw;
      if (i >= MT * NT) break;
      const int mt = i / NT, r = mt * 16 + c, t = t0 + i % NT;
      uint32_t b = 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) b = umax32(b, mx[(mt * 8 + u) * 16 + c]);
      float s, f8;
      a8_scale(b, s, f8);
      if (r >= rows || t >= ntiles) continue;
      int w = 0;
      w = __builtin_amdgcn_cvt_pk_fp8_f32(z[it][0] * f8, z[it][1] * f8, w, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(z[it][2] * f8, z[it][3] * f8, w, true);
      *(int*)((uint8_t*)a.y + ((int64_t)m0 + r) * a.ldy + t * kTileN + 4 * q) = w;
      if (q == 0 && nw == 0 && i % NT == 0) a.sy[(int64_t)nb * a.ldsy + m0 + r] = s;
    }
  }
}

}  // namespace q4
