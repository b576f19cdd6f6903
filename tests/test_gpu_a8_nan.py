"""How far a NaN spreads in the SwiGLU pairs: its row, its column, and with
8-bit results the 128 columns that share the column's scale."""

import numpy as np
import pytest
import torch

import bit_weight_only_q4g64_amd as q4
import oracle
import synthetic
from tests.a8_tolerance import tol_codes, tol_product
from tests.gpu_helpers import DEV, host_f64, say
from tests.test_gpu_a8 import TYPES, codes_of, dev_fp8, draw_a8, scales_of
from tests.tolerance import tol_bf16_out, tol_swiglu

pytestmark = pytest.mark.gpu

# one and two launches of the 8-bit result, every kind of kernel, half groups at the ends of N and K
SHAPES = [(3, 448, 256), (4, 448, 2048), (16, 448, 8192), (40, 448, 320), (300, 448, 256), (500, 2112, 704), (1000, 2112, 448), (1100, 2112, 1088)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_nan_in_pairs(M, N, K):
    say(f"nan in pairs {M}x{N}x{K}")
    rng = np.random.default_rng(M + N)
    w1, w3 = synthetic.draw_fp8_weight(rng, "w1", N, K), synthetic.draw_fp8_weight(rng, "w3", N, K)
    codes, scales, _ = draw_a8(rng, M, K)
    a64, A1 = oracle.matmul_a8(w1.w8, w1.scales, codes, scales)
    c64, A3 = oracle.matmul_a8(w3.w8, w3.scales, codes, scales)
    z64 = oracle.swiglu(a64, c64)
    bad, w8a, w8c = codes.copy(), w1.w8.copy(), w3.w8.copy()
    bad[1, 2], w8a[5, K - 1], w8c[200, 0] = 0x7F, 0xFF, 0x7F
    sx = scales.copy()
    sx[-1, 2] = np.nan
    x = q4.Act8(torch.from_numpy(bad).to(DEV).view(torch.float8_e4m3fn), torch.from_numpy(sx).to(DEV))
    p1, p3 = dev_fp8(w8a, w1.scales), dev_fp8(w8c, w3.scales)
    row = np.zeros((M, N), dtype=bool)
    row[1:3] = True
    want = row.copy()
    want[:, [5, 200]] = True
    for out in ("f32", "bf16"):
        y = host_f64(q4.qmm_a8_fp8b(p1, p3, N, K, x, out_dtype=TYPES[out]))
        assert np.array_equal(np.isnan(y), want), out
        T = tol_swiglu(a64, c64, tol_product(A1, K, out), tol_product(A3, K, out))
        assert np.all(np.abs(y - z64)[~want] <= (tol_bf16_out(z64, T) if out == "bf16" else T)[~want]), out
    a = q4.qmm_a8_swiglu_a8(p1, p3, N, K, x)
    got, s = codes_of(a), scales_of(a)
    groups = np.zeros((-(-N // 128), M), dtype=bool)
    groups[:, 1:3] = groups[:2] = True
    assert np.array_equal(np.isnan(s), groups)
    wide = np.repeat(groups.T, 128, axis=1)[:, :N]
    assert np.all(got[wide] & 0x7F == 0x7F) and np.all(got[~wide] & 0x7F != 0x7F)
    T = tol_swiglu(a64, c64, tol_product(A1, K, "a8"), tol_product(A3, K, "a8"))
    clean = np.where(groups, np.float32(1), s)
    err = np.abs(oracle.dequantize_a8(np.where(wide, 0, got).astype(np.uint8), clean) - z64)
    assert np.all(err[~wide] <= tol_codes(got, clean, z64, T)[~wide])
