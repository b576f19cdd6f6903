// Products of 8-bit activations with block-FP8 weights for many rows. The
// arithmetic is that of a8_gemm.h on the larger matrix instructions: 32 x 32 x
// 64 of E4M3 (two chained steps per group of 128 k), or 32 x 32 x 16 of bf16
// (eight) where the result is float32.
//
// A workgroup of WM x WN waves owns 32 MT WM rows and WN x NS slots of 32
// weight columns (SwiGLU: half the slots of each matrix, the same columns). A
// wave owns 32 MT rows and NS slots; each product of 32 x 32 x 128 is folded
// into its accumulator.
//
// Operands. The activations of a group move from memory to LDS by
// buffer-to-LDS DMA, PD + 1 groups ahead, and from there to registers one
// row tile ahead: the workgroup's waves share them, and load them once. The
// weights belong to one wave each and go straight from memory to registers PD
// groups ahead. What comes from memory is the scarcer path: a compute unit
// gets 64 bytes a cycle from its cache and 60 from L2, and over 200 from LDS
// (measured with 8 waves, 16 bytes a lane).
//
// What bounds it. Many rows of bf16 results: 8192 x 2048 x 8192 takes 134-141
// us with inputs that rotate through memory, 124-130 with one set of inputs,
// 2.0-2.2 PFLOP/s of 8-bit products. The matrix cores are busy 53 % of the
// cycles and the VALU issues 41 %: the 128 x 256 tile has no registers to fold
// a product one late, so a wave's matrix steps and folds take turns, and the
// one other wave of its SIMD does not fill the gaps. The clock is 1.9 GHz under
// the power limit with real values, 2.4 with zeros (97 us, the same cycles).
// Exact results: the bf16 matrix steps, half of a wave's time, and the wait for
// weights that it can ask for only one group ahead, because accumulators,
// converted operands and products leave no more registers: SwiGLU to 8 bits of
// 8192 x 8192 x 2048 in 500-517 us, 1.1 PFLOP/s. (The pair with a float32
// result is two registers short: two lane indexes lie in scratch memory from
// before the loop until after it.) One row of workgroups: the weights from
// memory, 128 x 65536 x 2048 in 33 us, 4.6 TB/s.
//
// Lane order. A lane of the instruction holds 32 bytes of k for row (column)
// L % 32. Of piece j of a column (64 k) the packed weights hold, for q = 0..3,
// the 16 bytes at k = 8 q + e and 32 + 8 q + e. Lane half h = L / 32 takes q =
// 2 h and 2 h + 1, so its k are 16 h .. 16 h + 15 and 32 + 16 h .. + 15: two
// whole 16-byte chunks of an activation row. The weights' middle words change
// places to follow the activations' order; that is all the shuffling there is.
#pragma once

#include "a8_gemm.h"
#include "pgemm.h"  // the DMA, the workgroup order, the bf16 instruction

namespace q4 {

__device__ __forceinline__ f32x16 mfma_a8_32(i32x8 a, i32x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

template <bool EXACT_, bool SW_, int WM_, int WN_, int MT_, int NS_, int PD_, bool LAG_>
struct TileA8 {
  static constexpr bool EXACT = EXACT_, SW = SW_, LAG = LAG_;
  static constexpr int WM = WM_, WN = WN_, MT = MT_, NS = NS_, PD = PD_;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
  static constexpr int kWaveRows = MT * 32, kRows = WM * kWaveRows;
  static constexpr int kMats = SW ? 2 : 1, NT = NS / kMats;
  static constexpr int kTiles = WN * NT * 2;  // 16-column tiles of the output
  static constexpr int kXBytes = kRows * 128, kStage = kXBytes + kWaves * 256, kStages = PD + 2;
  static constexpr size_t kLds = kStages * (size_t)kStage;
  static constexpr int kXDma = kRows / 8 / kWaves, kScales = kRows / kWaves;  // a wave's share of the rows
  static_assert(kRows / 8 % kWaves == 0, "each wave copies whole runs of 8 rows");
  static_assert(kScales <= 64, "and their scales at once");
  // loads a wave issues per group: activations, their scales, weights, block scales
  static constexpr int kLoads = kXDma + 1 + 4 * NS + kMats;
  static_assert((PD - 1) * kLoads < 64, "the counter of loads in flight");
  static_assert(!EXACT || LAG, "the exact form folds between the next product's steps");
  // buffers of weights: the exact form's are free once converted, so the
  // group PD ahead takes the place of the current one
  static constexpr int kRing = EXACT ? PD : PD + 1;
};

// A wave's weights of one group: NS slots of 32 columns, pieces j, q % 2, and
// the block scale of each matrix.
template <class C>
struct TileWeights {
  i32x8 w[C::NS][2];
  float sw[C::kMats];
};

// ONCE: non-temporal loads of the weights.
template <class C, bool A8OUT, bool ONCE>
__global__ __launch_bounds__(C::kThreads, 2) void a8_tile_kernel(GemmA8Args a, int nblk, int mblk) {
  constexpr int MT = C::MT, NS = C::NS, NT = C::NT, kMats = C::kMats, PD = C::PD;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int c = lane & 31, h = lane >> 5;
  int mb, nb;
  pgemm_tile((int)blockIdx.x, nblk, mblk, mb, nb);
  const int P = (int)n_pairs(a.K), ntiles = a.N / kTileN;
  const int m0 = mb * C::kRows, t0 = nb * C::kTiles;
  const int rows = a.M - m0 < C::kRows ? a.M - m0 : C::kRows;
  const int tvalid = ntiles - t0 < C::kTiles ? ntiles - t0 : C::kTiles;
  const int64_t cb = codes_bytes(a.N, a.K, kFmtFp8);

  // ---- activations: memory -> LDS, 8 rows of 128 bytes a copy. Chunk u of
  // row r lies at u ^ (r % 8), so that the 32 rows of a read spread over the
  // banks.
  const int xchunk = (lane & 7) ^ (lane >> 3);
  const uint32_t xoff = (uint32_t)((lane >> 3) * a.ldx + 16 * xchunk);
  const uint32_t stage0 = lds_addr(smem);
  // part k of n of a group's copies
  auto copy_x = [&](int p, int st, int k, int n) {
    const uint32_t base = stage0 + (uint32_t)st * C::kStage;
    // half a group: its upper 64 columns are not the row's
    const uint32_t off = p * 128 + 64 < a.K || xchunk < 4 ? xoff : kOffBuffer;
#pragma unroll
    for (int i = 0; i < C::kXDma; ++i) {
      if (i * n / C::kXDma != k) continue;
      const int r = (wave * C::kXDma + i) * 8, left = rows - r;  // reads of rows past the last return zeros
      const i32x4 res = make_srsrc(a.x + (int64_t)(m0 + (left > 0 ? r : 0)) * a.ldx,
                                   left > 0 ? (uint32_t)(((left < 8 ? left : 8) - 1) * a.ldx + a.K) : 0u);
      dma_b128(res, off, (uint32_t)p * 128u, base + (uint32_t)(wave * C::kXDma + i) * 1024u);
    }
    if (k + 1 == n) {
      const i32x4 r = make_srsrc(a.sx + (int64_t)p * a.ldsx + m0, (uint32_t)rows * 4u);
      dma_b32(r, lane < C::kScales ? (uint32_t)(wave * C::kScales + lane) * 4u : kOffBuffer, 0, base + C::kXBytes + (uint32_t)wave * 256u);
    }
  };

  // ---- weights: memory -> registers. Slots past the last read the last one;
  // their results are not stored.
  const int wt = wn * NT * 2;  // this wave's first tile (of each matrix)
  rsrc_t wres[kMats], sres[kMats];
  uint32_t wsoff[NT];
  {
    const int t = t0 + (wt < tvalid ? wt : tvalid - 2), left = ntiles - t;
#pragma unroll
    for (int s = 0; s < kMats; ++s) {
      const uint8_t* b = s ? a.pb : a.pa;
      wres[s] = make_rsrc(b + (int64_t)t * P * 2048, (uint32_t)((left < 2 * NT ? left : 2 * NT) * P * 2048));
      sres[s] = make_rsrc(b + cb + (int64_t)t * P * kPairSbBytes, (uint32_t)(P * kPairSbBytes));
    }
#pragma unroll
    for (int u = 0; u < NT; ++u) wsoff[u] = (uint32_t)((2 * u < left ? 2 * u : left - 2) * P) * 2048u;
  }
  const uint32_t woff = (uint32_t)((c >> 4) * P) * 2048u + (uint32_t)(h * 512 + (c & 15) * 16);
  // load i of a group's weights: piece j, slot s, half e of 16 bytes a lane;
  // part k of n of a group's weights: piece by piece, and the block scales
  auto load_w1 = [&](TileWeights<C>& f, int p, int i) {
    const int j = i / (2 * NS), s = i / 2 % NS, e = i % 2;
    const uint32_t so = wsoff[s % NT] + (uint32_t)p * 2048u, wo = woff + j * 1024u + e * 256u;
    const u32x4 v = ONCE ? buf_load16_nt(wres[s / NT], wo, so) : buf_load16(wres[s / NT], wo, so);
#pragma unroll
    for (int u = 0; u < 4; ++u) f.w[s][j][4 * e + u] = (int)v[u];
  };
  auto load_w = [&](TileWeights<C>& f, int p, int k, int n) {
#pragma unroll
    for (int i = 0; i < 4 * NS; ++i)
      if (i * n / (4 * NS) == k) load_w1(f, p, i);
    if (k == 0) {
#pragma unroll
      for (int s = 0; s < kMats; ++s)
        f.sw[s] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sres[s], 0, (uint32_t)p * kPairSbBytes, 0));
    }
  };

  auto arrived = [&](TileWeights<C>& f) {
#pragma unroll
    for (int s = 0; s < NS; ++s) asm volatile("" : "+v"(f.w[s][0]), "+v"(f.w[s][1]));
#pragma unroll
    for (int s = 0; s < kMats; ++s) asm volatile("" : "+v"(f.sw[s]));
  };

  f32x16 acc[MT][NS];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[mt][s][v] = 0.f;

  // A row tile from LDS: chunk u = 0..3 of the lane's row and, with the last,
  // its scale. kAhead (exact, one slot): a row tile is converted during the
  // matrix steps of the one before, and read during those of the one before that.
  constexpr bool kAhead = C::EXACT && NS == 1;
  static_assert(!kAhead || MT % 2 == 0, "the two buffers change places with every tile");
  u32x4 xr[4];
  float sr;
  bf16x8 xe[kAhead ? 2 : 1][8];
  float sxe[2];
  const uint32_t xbase = (uint32_t)((wm * C::kWaveRows + c) * 128 + ((h ^ (c & 7)) << 4));
  auto read_x1 = [&](int st, int mt, int u) {
    const uint8_t* q = smem + st * C::kStage;
    xr[u] = *(const u32x4*)(q + mt * 4096 + (xbase ^ (uint32_t)(u * 32)));
    const int r = wm * C::kWaveRows + mt * 32 + c;
    if (u == 3) sr = *(const float*)(q + C::kXBytes + r / C::kScales * 256 + r % C::kScales * 4);
  };
  auto read_x = [&](int st, int mt) {
#pragma unroll
    for (int u = 0; u < 4; ++u) read_x1(st, mt, u);
  };
  auto convert_x = [&](int b, int k) { xe[b][k] = fp8_to_bf16(xr[k / 2][2 * (k % 2)], xr[k / 2][2 * (k % 2) + 1]); };

  // Group p: its weights in f, the next group's in f1; the group PD ahead is
  // loaded into fn (past the last group: the last one again, unused). A wave
  // waits for each load to be taken, some 45 cycles with all waves asking at
  // once: so they are asked for between the matrix steps, a share per row
  // tile. The exact form does all else between its matrix steps, too: every
  // step comes with the conversions that the next steps or products need, two
  // values of the last product's fold, and early in the group a load. (With
  // the conversions ahead of the steps and the loads spread over the whole
  // group, the SwiGLU of 8192 x 8192 x 2048 takes 557 us, so 513.)
  auto group = [&](TileWeights<C>& f, TileWeights<C>& f1, TileWeights<C>& fn, int p, int& st) {
    const int st1 = st + 1 == C::kStages ? 0 : st + 1, stn = st == 0 ? C::kStages - 1 : st - 1;
    const int pw = p + PD < P ? p + PD : P - 1, px = p + PD + 1 < P ? p + PD + 1 : P - 1;
    float sw[kMats];
#pragma unroll
    for (int s = 0; s < kMats; ++s) sw[s] = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(f.sw[s])));
    bf16x8 we[NS][8];  // converted: step k of slot s
    auto convert_w = [&](int s, int k) {
      const i32x8& w = f.w[s][k / 4];
      const int e = k % 4 == 0 ? 0 : k % 4 == 1 ? 4 : k % 4 == 2 ? 2 : 6;  // the weights' order
      we[s][k] = fp8_to_bf16(w[e], w[e + 1]);
    };
    // the weights into the activations' order: words 2, 3 change places with
    // 4, 5 (in place; the compiler would copy all eight)
    if constexpr (!C::EXACT) {
#pragma unroll
      for (int i = 0; i < 2 * NS; ++i) {
        i32x8& w = f.w[i / 2][i % 2];
        int w2 = w[2], w3 = w[3], w4 = w[4], w5 = w[5];
        asm("v_swap_b32 %0, %1" : "+v"(w2), "+v"(w4));
        asm("v_swap_b32 %0, %1" : "+v"(w3), "+v"(w5));
        w[2] = w2;
        w[3] = w3;
        w[4] = w4;
        w[5] = w5;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // Product i of slot i % NS and row tile i / NS. With LAG it is folded
    // while the next one is in the matrix cores: 16 more registers, which 128 x
    // 256 workgroups do not have.
    f32x16 d[C::LAG ? 2 : 1];
    float sc[C::LAG ? 2 : 1];
    auto fold = [&](int i, int v0, int v1) {
      const int b = C::LAG ? i & 1 : 0;
#pragma unroll
      for (int v = v0; v < v1; ++v) acc[i / NS][i % NS][v] = __builtin_fmaf(sc[b], d[b][v], acc[i / NS][i % NS][v]);
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      // tile mt + n, of this group or the next one, whose stage is already
      // there: all reads of this stage have arrived before the group's barrier
      auto tile_st = [&](int n) { return mt + n < MT ? st : st1; };
      auto tile_mt = [&](int n) { return mt + n < MT ? mt + n : mt + n - MT; };
      const int xb = kAhead ? mt & 1 : 0;
      const float sx = kAhead ? sxe[xb] : sr;
      auto next = [&]() {
        if (mt + 1 == MT) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        read_x(tile_st(1), tile_mt(1));
      };
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int i = mt * NS + s, b = C::LAG ? i & 1 : 0;
#pragma unroll
        for (int v = 0; v < 16; ++v) d[b][v] = 0.f;
        if constexpr (C::EXACT) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (!kAhead && s == 0) convert_x(0, k);
            if (mt == 0 && s == 0) convert_w(0, k);
            d[b] = mfma32(we[s][k], xe[xb][k], d[b]);
            if (mt == 0 && s + 1 < NS) convert_w(s + 1, k);
            if constexpr (kAhead) {
              convert_x(xb ^ 1, k);
              if (k == 7) sxe[xb ^ 1] = sr;
              if (k % 2 == 1) read_x1(tile_st(2), tile_mt(2), k / 2);
            }
            if (i > 0) fold(i - 1, 2 * k, 2 * k + 2);
            if (i == 0 && k < 4) copy_x(px, stn, k, 4);
            if (i * 8 + k >= 4) load_w(fn, pw, i * 8 + k - 4, 8);  // a piece's registers are free once converted
            __builtin_amdgcn_sched_barrier(0);
          }
          if (!kAhead && s == 0) next();
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            d[b] = mfma_a8_32(f.w[s][j], __builtin_bit_cast(i32x8, __builtin_shufflevector(xr[2 * j], xr[2 * j + 1], 0, 1, 2, 3, 4, 5, 6, 7)),
                              d[b]);
        }
        sc[b] = sx * sw[s / NT];
        __builtin_amdgcn_sched_barrier(0);
        if (s + 1 == NS) {
          if constexpr (!C::EXACT) next();
          if constexpr (!C::EXACT) {
            load_w(fn, pw, mt, MT);
            copy_x(px, stn, mt, MT);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!C::EXACT) {
          if constexpr (!C::LAG) fold(i, 0, 16);
          else if (i > 0) fold(i - 1, 0, 16);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (C::LAG) fold(MT * NS - 1, 0, 16);
    // All but the newest PD - 1 groups' loads have arrived. The compiler
    // counts its own loads only: used here, the next weights ask for no wait
    // among the next group's loads.
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"((PD - 1) * C::kLoads) : "memory");
    arrived(f1);
    asm volatile("s_barrier" ::: "memory");
    st = st1;
  };

  constexpr int R = C::kRing;
  TileWeights<C> f[R];
  copy_x(0, 0, 0, 1);
#pragma unroll
  for (int u = 0; u < PD; ++u) {
    load_w(f[u], u < P ? u : P - 1, 0, 1);
    copy_x(u + 1 < P ? u + 1 : P - 1, u + 1, 0, 1);
  }
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"((PD - 1) * C::kLoads) : "memory");
  arrived(f[0]);
  asm volatile("s_barrier" ::: "memory");
  read_x(0, 0);
  if constexpr (kAhead) {
#pragma unroll
    for (int k = 0; k < 8; ++k) convert_x(0, k);
    sxe[0] = sr;
    read_x(0, 1);
  }
  // whole turns of the ring without a branch, so that the compiler knows in
  // every group which loads came after the weights it uses; then the rest
  int st = 0, p = 0;
  for (; p + R <= P; p += R) {
#pragma unroll
    for (int u = 0; u < R; ++u) group(f[u], f[(u + 1) % R], f[(u + PD) % R], p + u, st);
  }
#pragma unroll
  for (int u = 0; u + 1 < R; ++u)
    if (p + u < P) group(f[u], f[(u + 1) % R], f[(u + PD) % R], p + u, st);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy outlives the workgroup's LDS

  // ---- results: row m of the lane; of each slot four runs of four
  // consecutive columns, 8 u + 4 h
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if constexpr (C::SW) acc[mt][t][v] = silu_f32(acc[mt][t][v]) * acc[mt][NS - NT + t][v];
  // The stages are free once every wave is here: results turn into whole rows
  // there, and leave 16 bytes a lane. (Stored straight from the matrix order,
  // 8 bytes of 32 rows at a time, 3052 x 11712 x 64 takes 33.4 us, so 19.8;
  // 8192 x 2048 x 2048 42.6, so 36.7.)
  __syncthreads();
  if constexpr (!A8OUT) {
    constexpr int kSize = C::EXACT ? 4 : 2;               // float32 or bf16
    constexpr int kRow = NT * 32 * kSize, kPad = kRow + 16;  // a wave's part of a row, and its place in LDS
    constexpr int kChunks = kRow / 16;
    static_assert(C::kWaves * 32 * kPad <= C::kLds, "the results' place");
    uint8_t* buf = smem + wave * 32 * kPad;  // the wave's own
    const int cols = (tvalid - wt) * kTileN;  // valid columns of the wave's
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const f32x16& z = acc[mt][t];
          uint8_t* q = buf + c * kPad + (32 * t + 8 * u + 4 * h) * kSize;
          if constexpr (C::EXACT) *(f32x4*)q = f32x4{z[4 * u], z[4 * u + 1], z[4 * u + 2], z[4 * u + 3]};
          else *(u32x2*)q = u32x2{pack_bf16(z[4 * u], z[4 * u + 1]), pack_bf16(z[4 * u + 2], z[4 * u + 3])};
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 32 * kChunks / 64; ++i) {
        const int r = (i * 64 + lane) / kChunks, k = (i * 64 + lane) % kChunks, m = wm * C::kWaveRows + mt * 32 + r;
        const u32x4 v = *(const u32x4*)(buf + r * kPad + 16 * k);
        if (m < rows && k * (16 / kSize) < cols)
          *(u32x4*)((uint8_t*)a.y + (((int64_t)m0 + m) * a.ldy + (t0 + wt) * kTileN) * kSize + 16 * k) = v;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    static_assert(C::kTiles * kTileN == kA8Group, "one output group per workgroup");
    uint32_t* mx = (uint32_t*)smem;  // [WN][kRows]
    constexpr int kPad = kA8Group + 16;
    uint8_t* buf = smem + C::WN * C::kRows * 4;
    static_assert(C::WN * C::kRows * 4 + C::kRows * kPad <= C::kLds, "the results' place");
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t b = 0;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (wt + 2 * t < tvalid) {
#pragma unroll
          for (int v = 0; v < 16; ++v) b = umax32(b, __float_as_uint(acc[mt][t][v]) & 0x7FFFFFFFu);
        }
      b = umax32(b, (uint32_t)__shfl_xor((int)b, 32, 64));
      if (h == 0) mx[wn * C::kRows + wm * C::kWaveRows + mt * 32 + c] = b;
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = wm * C::kWaveRows + mt * 32 + c;
      uint32_t b = 0;
#pragma unroll
      for (int u = 0; u < C::WN; ++u) b = umax32(b, mx[u * C::kRows + r]);
      float s, f;
      a8_scale(b, s, f);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const f32x16& z = acc[mt][t];
          int w = 0;
          w = __builtin_amdgcn_cvt_pk_fp8_f32(z[4 * u] * f, z[4 * u + 1] * f, w, false);
          w = __builtin_amdgcn_cvt_pk_fp8_f32(z[4 * u + 2] * f, z[4 * u + 3] * f, w, true);
          *(int*)(buf + r * kPad + (wt + 2 * t) * kTileN + 8 * u + 4 * h) = w;
        }
      if (r < rows && h == 0 && wn == 0) a.sy[(int64_t)nb * a.ldsy + m0 + r] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C::kRows * 8 / C::kThreads; ++i) {
      const int r = (i * C::kThreads + (int)threadIdx.x) / 8, k = (int)threadIdx.x % 8;
      if (r < rows && 16 * k < tvalid * kTileN)
        *(u32x4*)((uint8_t*)a.y + ((int64_t)m0 + r) * a.ldy + t0 * kTileN + 16 * k) = *(const u32x4*)(buf + r * kPad + 16 * k);
    }
  }
}

}  // namespace q4
