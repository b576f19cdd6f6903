// Host side of the 8-bit activation path: argument validation and launch
// configuration of the row quantizer, the RMS norm and the 8-bit products.
// Every entry point validates on the host first and enqueues nothing when an
// argument is rejected.
#include "../../include/q4g64.h"

#include <math.h>

#include <atomic>
#include <stdlib.h>

#include "a8_gemm.h"
#include "a8_rows.h"
#include "a8_tile.h"
#include "common.h"
#include "host.h"

namespace {

using namespace q4host;

constexpr int64_t kNormMaxK = 16384;  // 256 lanes of 8 chunks of 8 columns

int type_size(int dtype) { return dtype == Q4_F32 ? 4 : 2; }

int check_rows(const char* fn, const char* name, const char* ldname, const void* p, int64_t ld, int64_t cols, int64_t M, int es) {
  if (int rc = check_ptr(fn, name, p, 16)) return rc;
  if (ld < cols) return fail(Q4_EINVAL, "%s: %s=%lld < %lld columns", fn, ldname, (long long)ld, (long long)cols);
  if (int rc = check_ld(fn, ldname, ld)) return rc;
  if ((ld * es) % 16 != 0) return fail(Q4_EALIGN, "%s: %s=%lld elements does not keep rows 16-byte aligned", fn, ldname, (long long)ld);
  if (M > kMaxSpan / ld) return fail(Q4_EINVAL, "%s: %lld rows of stride %s=%lld span more than 2^48 elements", fn, (long long)M, ldname, (long long)ld);
  return Q4_OK;
}

// Scales [G][ld], group-major.
int check_scales(const char* fn, const char* name, const char* ldname, const void* p, int64_t ld, int64_t M) {
  if (int rc = check_ptr(fn, name, p, 4)) return rc;
  if (ld < M) return fail(Q4_EINVAL, "%s: %s=%lld < M=%lld", fn, ldname, (long long)ld, (long long)M);
  if (ld > kPgemmMaxM) return fail(Q4_EINVAL, "%s: %s=%lld exceeds %lld", fn, ldname, (long long)ld, (long long)kPgemmMaxM);
  return Q4_OK;
}

int check_mk(const char* fn, int64_t M, int64_t K) {
  if (K <= 0 || K % 64 != 0) return fail(Q4_EINVAL, "%s: K=%lld must be a positive multiple of 64", fn, (long long)K);
  if (K > kPgemmMaxK) return fail(Q4_EUNSUPPORTED, "%s: K=%lld exceeds the limit of %lld", fn, (long long)K, (long long)kPgemmMaxK);
  if (M < 1 || M > kPgemmMaxM) return fail(Q4_EINVAL, "%s: M=%lld is outside 1..%lld", fn, (long long)M, (long long)kPgemmMaxM);
  return Q4_OK;
}

int check_dtype(const char* fn, const char* name, int dtype) {
  if (dtype != Q4_BF16 && dtype != Q4_F32) return fail(Q4_EINVAL, "%s: %s %d is not Q4_BF16 or Q4_F32", fn, name, dtype);
  return Q4_OK;
}

int groups128(int64_t n) { return (int)((n + 127) / 128); }

// A launch has fewer than 2^32 lanes. The launch functions below enqueue
// nothing and return false for more.
bool fits(int64_t blocks, int threads) { return blocks * threads < int64_t(1) << 32; }

// ---- the quantizer's instances ----------------------------------------------

bool rows_launch(const q4::QuantA8Args& a, int xt, hipStream_t s) {
  const int64_t blocks = ((int64_t)a.M * a.G + 15) / 16;
  if (!fits(blocks, 256)) return false;
  const dim3 grid((unsigned)blocks);
  if (xt == q4::kRowF32) hipLaunchKernelGGL(q4::quant_a8_kernel<q4::kRowF32>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(q4::quant_a8_kernel<q4::kRowBf16>, grid, dim3(256), 0, s, a);
  return true;
}

// ---- the norm's instances --------------------------------------------------

template <int TPR, int CH, int XT>
bool norm_launch_res(const q4::NormArgs& a, int rt, hipStream_t s) {
  const int blocks = (a.M + 256 / TPR - 1) / (256 / TPR);
  if (!fits(blocks, 256)) return false;
  const dim3 grid((unsigned)blocks);
  if (rt == q4::kRowNone) hipLaunchKernelGGL((q4::rms_norm_kernel<TPR, CH, XT, q4::kRowNone>), grid, dim3(256), 0, s, a);
  else if (rt == q4::kRowBf16) hipLaunchKernelGGL((q4::rms_norm_kernel<TPR, CH, XT, q4::kRowBf16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((q4::rms_norm_kernel<TPR, CH, XT, q4::kRowF32>), grid, dim3(256), 0, s, a);
  return true;
}

template <int TPR, int CH>
bool norm_launch_x(const q4::NormArgs& a, int xt, int rt, hipStream_t s) {
  return xt == q4::kRowBf16 ? norm_launch_res<TPR, CH, q4::kRowBf16>(a, rt, s) : norm_launch_res<TPR, CH, q4::kRowF32>(a, rt, s);
}

bool norm_launch(const q4::NormArgs& a, int xt, int rt, hipStream_t s) {
  // A wave per row of up to 1024 columns, else a workgroup of 256 lanes.
  // Measured, us with a wave / a workgroup per row (bf16, 8-bit result): 8192 x
  // 512 7.7 / 10.0, 1024 x 512 2.8 / 2.9; 256 x 2048 4.4 / 3.0, 8192 x 2048
  // 26.9 / 26.0, 4096 x 4096 28.7 / 26.3.
  if (a.K <= 512) return norm_launch_x<64, 1>(a, xt, rt, s);
  if (a.K <= 1024) return norm_launch_x<64, 2>(a, xt, rt, s);
  if (a.K <= 2048) return norm_launch_x<256, 1>(a, xt, rt, s);
  if (a.K <= 4096) return norm_launch_x<256, 2>(a, xt, rt, s);
  if (a.K <= 8192) return norm_launch_x<256, 4>(a, xt, rt, s);
  return norm_launch_x<256, 8>(a, xt, rt, s);
}

int norm_impl(const char* fn, const void* x, int x_dtype, int64_t ldx, const void* res, int res_dtype, int64_t ldr, void* res_out,
              int64_t ldro, const float* gamma, float eps, int64_t M, int64_t K, int out, void* y, int64_t ldy, float* s, int64_t lds,
              hipStream_t st) {
  if (int rc = check_mk(fn, M, K)) return rc;
  if (K > kNormMaxK) return fail(Q4_EUNSUPPORTED, "%s: K=%lld exceeds the limit of %lld", fn, (long long)K, (long long)kNormMaxK);
  if (int rc = check_dtype(fn, "x_dtype", x_dtype)) return rc;
  if (int rc = check_rows(fn, "x", "ldx", x, ldx, K, M, type_size(x_dtype))) return rc;
  int rt = q4::kRowNone;
  if (res != nullptr) {
    if (int rc = check_dtype(fn, "res_dtype", res_dtype)) return rc;
    if (int rc = check_rows(fn, "res", "ldr", res, ldr, K, M, type_size(res_dtype))) return rc;
    if (int rc = check_rows(fn, "res_out", "ldro", res_out, ldro, K, M, type_size(res_dtype))) return rc;
    rt = res_dtype == Q4_F32 ? q4::kRowF32 : q4::kRowBf16;
  } else if (res_out != nullptr) {
    return fail(Q4_EINVAL, "%s: res_out without res", fn);
  }
  if (int rc = check_ptr(fn, "gamma", gamma, 16)) return rc;
  if (!(eps >= 0.f) || !isfinite(eps)) return fail(Q4_EINVAL, "%s: eps must be >= 0 and finite", fn);
  if (int rc = check_rows(fn, out == q4::kRowA8 ? "q" : "y", out == q4::kRowA8 ? "ldq" : "ldy", y, ldy, K, M,
                          out == q4::kRowA8 ? 1 : (out == q4::kRowF32 ? 4 : 2)))
    return rc;
  if (out == q4::kRowA8)
    if (int rc = check_scales(fn, "sq", "ldsq", s, lds, M)) return rc;
  const q4::NormArgs a{x, ldx, res, ldr, res_out, ldro, gamma, eps, (int)M, (int)K, out, y, ldy, s, lds};
  if (!norm_launch(a, x_dtype == Q4_F32 ? q4::kRowF32 : q4::kRowBf16, rt, st))
    return fail(Q4_EUNSUPPORTED, "%s: M=%lld needs too many workgroups", fn, (long long)M);
  return launched(fn);
}

// ---- the products' instances -----------------------------------------------

// Lets a kernel use more than 64 KiB of LDS: once per device (a bit of
// `raised` each; devices past 64 are asked every time).
void raise_lds(const void* kern, size_t bytes, std::atomic<uint64_t>& raised) {
  int dev = 64;
  if (hipGetDevice(&dev) != hipSuccess) dev = 64;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (raised.load(std::memory_order_relaxed) & bit) return;
  if (hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == hipSuccess)
    raised.fetch_or(bit, std::memory_order_relaxed);
  else
    (void)hipGetLastError();  // the launch reports it
}

template <class C, bool A8OUT>
bool direct_launch(const q4::GemmA8Args& a, hipStream_t s) {
  const int64_t nblk = (a.N / q4::kTileN + C::kTiles - 1) / C::kTiles, mblk = (a.M + C::kRows - 1) / C::kRows;
  if (!fits(nblk * mblk, C::kThreads)) return false;
  const size_t lds = C::kLds + (A8OUT ? (size_t)C::MT * 8 * 16 * 4 : 0);
  auto kern = q4::a8_direct_kernel<C, A8OUT>;
  if (lds > 64 * 1024) {
    static std::atomic<uint64_t> raised{0};
    raise_lds((const void*)kern, lds, raised);
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)(nblk * mblk)), dim3(C::kThreads), lds, s, a);
  return true;
}

template <class C, bool A8OUT, bool ONCE = false>
bool tile_launch(const q4::GemmA8Args& a, hipStream_t s) {
  const int nblk = (a.N / q4::kTileN + C::kTiles - 1) / C::kTiles, mblk = (a.M + C::kRows - 1) / C::kRows;
  if (!fits((int64_t)nblk * mblk, C::kThreads)) return false;
  auto kern = q4::a8_tile_kernel<C, A8OUT, ONCE>;
  static std::atomic<uint64_t> raised{0};
  raise_lds((const void*)kern, C::kLds, raised);
  hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)nblk * mblk)), dim3(C::kThreads), C::kLds, s, a, nblk, mblk);
  return true;
}

// Which kernel. The larger a workgroup's tile, the fewer bytes a product
// reads; but the compute units share out whole tiles, and a tile's groups
// follow one another. So the tile is taken whose estimated time
//   us + us_k K / 1024 + (rounds - 1) (more + more_k K / 1024),
//   rounds = ceil(tiles / 256 compute units),
// is least. The constants are chosen for the least distance of the chosen tile
// from the best one over 700 to 1400 sizes per table, drawn evenly on
// logarithmic scales from 17 x 64 x 64 up to 8800 rows, 20000 columns and K =
// 11000 and timed with every tile: 0.2 to 1.3 % on average, 7 to 22 % at the
// 99th percentile. Measured, bf16 result, us at M x N x K by tile:
//                       16x16 32x32 32x64 64x64 64x128 128x128 128x256
//      62 x    64 x 11520   9.8  15.4  18.7  28.4  38.1  54.1 113.7
//     379 x   640 x 10560  30.0  14.2  18.2  24.2  36.1  52.3 109.1
//    5039 x    64 x  5312  22.3  16.7  11.1  15.4  20.6  28.8  57.6
//      94 x  7616 x 10496  99.0  47.4  43.2  32.4  41.4  69.8 127.5
//    6052 x   256 x  8256 125.0  75.5  44.8  47.5  31.1  42.5  86.7
//    1963 x  3264 x  1984 145.2  71.4  73.3  41.6  26.8  21.1  26.9
//    8689 x  3584 x    64 195.3 116.1  97.1  43.6  24.2  18.9  16.0
struct Tile {
  int rows, cols;
  float us, us_k, more, more_k;
};

int64_t tile_count(const Tile& t, int64_t M, int64_t N) { return ((M + t.rows - 1) / t.rows) * ((N + t.cols - 1) / t.cols); }

float tile_us(const Tile& t, int64_t M, int64_t N, int64_t K) {
  const int64_t rounds = (tile_count(t, M, N) + 255) / 256;
  const float k = (float)K / 1024.0f;
  return t.us + t.us_k * k + (float)(rounds - 1) * (t.more + t.more_k * k);
}

template <int n>
int best_tile(const Tile (&tiles)[n], int64_t M, int64_t N, int64_t K) {
  int best = 0;
  for (int i = 1; i < n; ++i)
    if (tile_us(tiles[i], M, N, K) < tile_us(tiles[best], M, N, K)) best = i;
  return best;
}

//                                    EXACT MT NT SW    NW KW D
template <bool E> using Part16x16 = q4::DirectA8<E, 1, 1, false, 1, 8, 2>;
template <bool E> using Part32x32 = q4::DirectA8<E, 2, 2, false, 1, 16, 1>;
template <bool E> using Part32x64 = q4::DirectA8<E, 2, 4, false, 1, 8, 1>;
template <bool E> using Part64x64 = q4::DirectA8<E, 4, 4, false, 1, 4, 1>;
template <bool E> using Pair16x16 = q4::DirectA8<E, 1, 1, true, 1, 8, 2>;
template <bool E> using Pair32x16 = q4::DirectA8<E, 2, 1, true, 1, 8, 1>;
template <bool E> using Pair32x32 = q4::DirectA8<E, 2, 2, true, 1, 8, 1>;
template <bool E> using Pair64x32 = q4::DirectA8<E, 4, 2, true, 1, 4, 1>;
using Quant16x128 = q4::DirectA8<true, 1, 2, true, 4, 4, 1>;
using Quant32x128 = q4::DirectA8<true, 2, 2, true, 4, 2, 1>;
//                                 EXACT SW WM WN MT NS PD LAG
template <bool E> using Tile64x128 = q4::TileA8<E, false, 1, 4, 2, 1, 3, true>;
template <bool E> using Tile128x128 = q4::TileA8<E, false, 1, 4, 4, 1, 2, true>;
using Tile128x256 = q4::TileA8<false, false, 1, 4, 4, 2, 1, false>;
using PairTile64x64 = q4::TileA8<false, true, 2, 2, 1, 2, 3, true>;
template <bool E> using PairTile64x128 = q4::TileA8<E, true, 1, 4, 2, 2, E ? 1 : 2, true>;
using PairTile128x128 = q4::TileA8<false, true, 1, 4, 4, 2, 1, false>;

// rows, cols, us, us_k, more, more_k
constexpr Tile kProduct[] = {{16, 16, 2.9f, 0.69f, 0.27f, 0.58f}, {32, 32, 3.2f, 1.10f, 0.87f, 1.20f}, {32, 64, 3.2f, 1.51f, 1.40f, 1.83f}, {64, 64, 4.2f, 2.60f, 1.06f, 2.05f},
                             {64, 128, 3.6f, 3.47f, 1.16f, 2.54f}, {128, 128, 3.6f, 4.40f, 1.88f, 3.69f}, {128, 256, 5.5f, 8.90f, 2.81f, 5.61f}};
constexpr Tile kProductExact[] = {{16, 16, 2.9f, 0.69f, 0.30f, 0.60f}, {32, 32, 3.3f, 1.24f, 1.04f, 1.25f}, {32, 64, 4.0f, 1.54f, 1.82f, 2.04f}, {64, 64, 4.4f, 2.90f, 1.53f, 2.43f},
                                  {64, 128, 4.0f, 4.93f, 1.87f, 3.72f}, {128, 128, 5.0f, 7.26f, 2.55f, 6.36f}};
constexpr Tile kPair[] = {{16, 16, 3.0f, 0.95f, 0.48f, 0.97f}, {32, 16, 3.2f, 0.92f, 0.32f, 1.09f}, {32, 32, 3.3f, 1.41f, 0.80f, 1.53f}, {64, 32, 4.2f, 2.92f, 0.92f, 2.19f},
                          {64, 64, 4.2f, 4.63f, 1.60f, 3.41f}, {64, 128, 4.6f, 5.32f, 1.86f, 4.51f}, {128, 128, 6.7f, 10.51f, 2.64f, 6.57f}};
constexpr Tile kPairExact[] = {{16, 16, 2.9f, 0.94f, 0.52f, 0.91f}, {32, 16, 3.2f, 1.08f, 0.61f, 1.10f}, {32, 32, 4.0f, 1.52f, 1.55f, 2.44f}, {64, 32, 3.8f, 2.90f, 1.70f, 2.22f},
                               {64, 128, 5.5f, 7.87f, 2.08f, 5.38f}};
constexpr Tile kPairQuant[] = {{16, 128, 3.6f, 5.75f, 1.88f, 7.44f}, {32, 128, 4.3f, 5.15f, 2.99f, 5.75f}, {64, 128, 4.4f, 7.11f, 1.82f, 5.73f}};

// Up to 16 rows the 16-row tile serves whatever the estimate, so that a row's
// bits do not depend on M.
constexpr int64_t kFewRows = 16;
int64_t rows16(int64_t M) { return M < kFewRows ? kFewRows : M; }

// Weights that one row of workgroups reads, more of them than the caches keep
// for the next call: loaded past the caches. Measured, us with / without: bf16
// 128 x 65536 x 2048 34.3 / 37.3, 128 x 16384 x 8192 36.2 / 40.6, float32 64 x
// 65536 x 2048 30.7 / 33.3; but 64 x 16384 x 4096 20.7 / 20.9, and with two
// rows of workgroups 256 x 32768 x 2048 28.4 / 27.7.
template <class C>
bool product_tile(const q4::GemmA8Args& a, hipStream_t s) {
  return a.M <= C::kRows && (int64_t)a.N * a.K > (int64_t(1) << 26) ? tile_launch<C, false, true>(a, s) : tile_launch<C, false>(a, s);
}

template <bool E>
bool product_launch(const q4::GemmA8Args& a, hipStream_t s) {
  int i = 0;
  if (a.M > kFewRows) {
    if constexpr (E) i = best_tile(kProductExact, a.M, a.N, a.K);
    else i = best_tile(kProduct, a.M, a.N, a.K);
  }
  switch (i) {
    case 0: return direct_launch<Part16x16<E>, false>(a, s);
    case 1: return direct_launch<Part32x32<E>, false>(a, s);
    case 2: return direct_launch<Part32x64<E>, false>(a, s);
    case 3: return direct_launch<Part64x64<E>, false>(a, s);
    case 4: return product_tile<Tile64x128<E>>(a, s);
    case 5: return product_tile<Tile128x128<E>>(a, s);
  }
  if constexpr (E) return false;  // its table ends at 5
  else return tile_launch<Tile128x256, false>(a, s);
}

template <bool E>
bool pair_launch(const q4::GemmA8Args& a, hipStream_t s) {
  int i = 0;
  if (a.M > kFewRows) {
    if constexpr (E) i = best_tile(kPairExact, a.M, a.N, a.K);
    else i = best_tile(kPair, a.M, a.N, a.K);
  }
  switch (i) {
    case 0: return direct_launch<Pair16x16<E>, false>(a, s);
    case 1: return direct_launch<Pair32x16<E>, false>(a, s);
    case 2: return direct_launch<Pair32x32<E>, false>(a, s);
    case 3: return direct_launch<Pair64x32<E>, false>(a, s);
    case 4:
      if constexpr (E) return tile_launch<PairTile64x128<true>, false>(a, s);
      else return tile_launch<PairTile64x64, false>(a, s);
  }
  if constexpr (E) return false;  // its table ends at 4
  else return i == 5 ? tile_launch<PairTile64x128<false>, false>(a, s) : tile_launch<PairTile128x128, false>(a, s);
}

// The pair with 8-bit results. A group of 128 result columns needs one scale,
// so a workgroup computes 128 columns. With few rows that leaves compute units
// without work, and it is faster to compute the pair in float32 on narrower
// workgroups into `work` and quantize that by a second launch, as soon as the
// first saves more than the second costs: 1.5 us and 4 TB/s on the GPU, and a
// host that needs 9 us for the two launches (16 x 1024 x 8192: 13 us against
// 52; 4 x 8192 x 2048: 9.3 against 14; 10 x 1152 x 64: 9.6 against 6).
// Only while the one launch has at most three workgroups per compute unit:
// there the unfilled last round is worth up to 30 % (two launches / one, us:
// 5474 x 320 x 10944 of 258 workgroups 108 / 144, 1226 x 1600 x 10368 of 507
// 118 / 130, 12 x 67648 x 11008 of 529 243 / 318, 11008 x 320 x 10368 of 516
// 193 / 206). Past that one launch is up to 43 % faster, but for up to 32 rows
// of short K (1 x 131072 x 2048 83 / 97), where the estimates keep to it too;
// they cross again where K passes the fitted range (4096 x 8192 x 28672 of 4096
// 3429 / 3396, 8192 x 8192 x 20480 of 8192 4907 / 4856), and the second launch
// would move M x N float32 values. So `work` is at most 768 x 64 x 128 floats,
// and the quantizer's launch is far inside its limit whenever the pair's has
// been enqueued.
constexpr int64_t kSplitTiles = 768;
bool quant_splits(int64_t M, int64_t N, int64_t K) {
  M = rows16(M);
  const Tile& t = kPairQuant[best_tile(kPairQuant, M, N, K)];
  if (tile_count(t, M, N) > kSplitTiles) return false;
  const float whole = tile_us(t, M, N, K);
  const float parts = tile_us(kPairExact[best_tile(kPairExact, M, N, K)], M, N, K) + 1.5f + (float)(M * N) * 9.0f / 4e6f;
  return whole > (parts > 9.0f ? parts : 9.0f);
}

bool quant_launch(const q4::GemmA8Args& a, float* work, hipStream_t s) {
  if (quant_splits(a.M, a.N, a.K)) {
    q4::GemmA8Args z = a;
    z.out = q4::kRowF32;
    z.y = work;
    z.ldy = a.N;
    return pair_launch<true>(z, s) &&
           rows_launch(q4::QuantA8Args{work, a.N, a.M, a.N, groups128(a.N), (uint8_t*)a.y, a.ldy, a.sy, a.ldsy}, q4::kRowF32, s);
  }
  switch (best_tile(kPairQuant, rows16(a.M), a.N, a.K)) {
    case 0: return direct_launch<Quant16x128, true>(a, s);
    case 1: return direct_launch<Quant32x128, true>(a, s);
  }
  return tile_launch<PairTile64x128<true>, true>(a, s);
}

size_t swiglu_work_bytes(int64_t M, int64_t N, int64_t K) { return quant_splits(M, N, K) ? (size_t)(M * N * 4) : 0; }

int gemm_impl(const char* fn, const void* pa, const void* pb, int64_t N, int64_t K, const uint8_t* x, int64_t ldx, const float* sx,
              int64_t ldsx, int64_t M, int out, void* y, int64_t ldy, float* sy, int64_t ldsy, void* work, size_t work_bytes,
              hipStream_t s) {
  if (int rc = check_nk(fn, N, K)) return rc;
  if (int rc = check_mk(fn, M, K)) return rc;
  if (int rc = check_ptr(fn, "packed_a", pa, 16)) return rc;
  if (pb != nullptr && !aligned(pb, 16)) return fail(Q4_EALIGN, "%s: packed_b is not 16-byte aligned", fn);
  if (int rc = check_rows(fn, "x", "ldx", x, ldx, K, M, 1)) return rc;
  // a 256-row tile of activations is addressed with 32-bit offsets
  if (ldx >= (int64_t(1) << 31) / 256) return fail(Q4_EUNSUPPORTED, "%s: ldx=%lld is too large for a 256-row tile", fn, (long long)ldx);
  if (int rc = check_scales(fn, "sx", "ldsx", sx, ldsx, M)) return rc;
  const bool a8 = out == q4::kRowA8;
  if (int rc = check_rows(fn, a8 ? "q" : "y", a8 ? "ldq" : "ldy", y, ldy, N, M, a8 ? 1 : (out == q4::kRowF32 ? 4 : 2))) return rc;
  if (a8) {
    if (int rc = check_scales(fn, "sq", "ldsq", sy, ldsy, M)) return rc;
    if (const size_t need = swiglu_work_bytes(M, N, K)) {
      if (int rc = check_ptr(fn, "work", work, 16)) return rc;
      if (work_bytes < need) return fail(Q4_EINVAL, "%s: work_bytes=%zu, %zu needed", fn, work_bytes, need);
    }
  }
  const q4::GemmA8Args a{(const uint8_t*)pa, (const uint8_t*)pb, (int)N, (int)K, x, ldx, sx, ldsx, (int)M, out, y, ldy, sy, ldsy};
  bool ok;
  if (a8) ok = quant_launch(a, (float*)work, s);
  else if (pb != nullptr) ok = out == q4::kRowF32 ? pair_launch<true>(a, s) : pair_launch<false>(a, s);
  else ok = out == q4::kRowF32 ? product_launch<true>(a, s) : product_launch<false>(a, s);
  if (!ok) return fail(Q4_EUNSUPPORTED, "%s: N=%lld x M=%lld needs too many workgroups", fn, (long long)N, (long long)M);
  return launched(fn);
}

}  // namespace

extern "C" {

int quant_rows_a8(const void* x, int x_dtype, int64_t ldx, int64_t M, int64_t K, uint8_t* q, int64_t ldq, float* sq, int64_t ldsq,
                  void* stream) {
  const char* fn = "quant_rows_a8";
  if (int rc = check_mk(fn, M, K)) return rc;
  if (int rc = check_dtype(fn, "x_dtype", x_dtype)) return rc;
  if (int rc = check_rows(fn, "x", "ldx", x, ldx, K, M, type_size(x_dtype))) return rc;
  if (int rc = check_rows(fn, "q", "ldq", q, ldq, K, M, 1)) return rc;
  if (int rc = check_scales(fn, "sq", "ldsq", sq, ldsq, M)) return rc;
  if (!rows_launch(q4::QuantA8Args{x, ldx, (int)M, (int)K, groups128(K), q, ldq, sq, ldsq},
                   x_dtype == Q4_F32 ? q4::kRowF32 : q4::kRowBf16, (hipStream_t)stream))
    return fail(Q4_EUNSUPPORTED, "%s: M=%lld x K=%lld needs too many workgroups", fn, (long long)M, (long long)K);
  return launched(fn);
}

int rms_norm_rows(const void* x, int x_dtype, int64_t ldx, const void* res, int res_dtype, int64_t ldr, void* res_out, int64_t ldro,
                  const float* gamma, float eps, int64_t M, int64_t K, void* y, int y_dtype, int64_t ldy, void* stream) {
  if (int rc = check_dtype("rms_norm_rows", "y_dtype", y_dtype)) return rc;
  return norm_impl("rms_norm_rows", x, x_dtype, ldx, res, res_dtype, ldr, res_out, ldro, gamma, eps, M, K,
                   y_dtype == Q4_F32 ? q4::kRowF32 : q4::kRowBf16, y, ldy, nullptr, 0, (hipStream_t)stream);
}

int rms_norm_rows_a8(const void* x, int x_dtype, int64_t ldx, const void* res, int res_dtype, int64_t ldr, void* res_out, int64_t ldro,
                     const float* gamma, float eps, int64_t M, int64_t K, uint8_t* q, int64_t ldq, float* sq, int64_t ldsq,
                     void* stream) {
  return norm_impl("rms_norm_rows_a8", x, x_dtype, ldx, res, res_dtype, ldr, res_out, ldro, gamma, eps, M, K, q4::kRowA8, q, ldq, sq,
                   ldsq, (hipStream_t)stream);
}

int qmm_a8_fp8b(const void* packed_a, const void* packed_b, int64_t N, int64_t K, const uint8_t* x, int64_t ldx, const float* sx,
                int64_t ldsx, int64_t M, void* y, int y_dtype, int64_t ldy, void* stream) {
  if (int rc = check_dtype("qmm_a8_fp8b", "y_dtype", y_dtype)) return rc;
  return gemm_impl("qmm_a8_fp8b", packed_a, packed_b, N, K, x, ldx, sx, ldsx, M, y_dtype == Q4_F32 ? q4::kRowF32 : q4::kRowBf16, y, ldy,
                   nullptr, 0, nullptr, 0, (hipStream_t)stream);
}

size_t qmm_a8_swiglu_work_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || M > kPgemmMaxM || N <= 0 || N % 64 != 0 || N > kMaxDim || K <= 0 || K % 64 != 0 || K > kPgemmMaxK) return 0;
  return swiglu_work_bytes(M, N, K);
}

int qmm_a8_swiglu_a8(const void* packed_w1, const void* packed_w3, int64_t N, int64_t K, const uint8_t* x, int64_t ldx,
                     const float* sx, int64_t ldsx, int64_t M, uint8_t* q, int64_t ldq, float* sq, int64_t ldsq, void* work, size_t work_bytes,
                     void* stream) {
  if (int rc = check_ptr("qmm_a8_swiglu_a8", "packed_w3", packed_w3, 16)) return rc;
  return gemm_impl("qmm_a8_swiglu_a8", packed_w1, packed_w3, N, K, x, ldx, sx, ldsx, M, q4::kRowA8, q, ldq, sq, ldsq, work, work_bytes,
                   (hipStream_t)stream);
}

}  // extern "C"
