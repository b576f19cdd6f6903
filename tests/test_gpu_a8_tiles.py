"""Every kernel of the 8-bit products through its whole pipeline, against
float64: many groups of K, ends at every place of the ring of loads, ends
inside the tiles, several blocks of rows and columns."""

import numpy as np
import pytest
import torch

import bit_weight_only_q4g64_amd as q4
import oracle
import synthetic
from tests import test_gpu_a8 as a8
from tests.a8_shapes import PAIRS, PRODUCTS
from tests.a8_tolerance import tol_codes, tol_product
from tests.gpu_helpers import DEV, host_f64, say
from tests.tolerance import tol_bf16_out, tol_swiglu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,pad", PRODUCTS)
def test_product(M, N, K, pad):
    a8.test_product(M, N, K, pad)


@pytest.mark.parametrize("M,N,K,pad", PAIRS)
def test_swiglu(M, N, K, pad):
    a8.test_swiglu(M, N, K, pad)


@pytest.mark.parametrize("M,N,K", [(8192, 2048, 8192), (8000, 8192, 2048), (1000, 1984, 2112), (128, 65536, 1024)])
def test_long_runs_repeat_their_bits(M, N, K):
    """At full load every run gives the same bits, and rows from all over agree with float64."""
    say(f"repeated {M}x{N}x{K}")
    rng = np.random.default_rng(M + K)
    g = torch.Generator(device=DEV).manual_seed(K)
    x = q4.quant_a8(torch.randn((M, K), device=DEV, generator=g))
    w = [synthetic.draw_fp8_weight(rng, n, N, K) for n in ("w1", "w3")]
    p = [a8.dev_fp8(v.w8, v.scales) for v in w]
    some = np.unique(np.concatenate([rng.integers(0, M, 24), [0, M - 1]]))
    codes, scales = a8.codes_of(x)[some], a8.scales_of(x)[:, some]
    y64, A1 = oracle.matmul_a8(w[0].w8, w[0].scales, codes, scales)
    c64, A3 = oracle.matmul_a8(w[1].w8, w[1].scales, codes, scales)
    z64 = oracle.swiglu(y64, c64)
    for out in ("f32", "bf16"):
        T1, T3 = tol_product(A1, K, out), tol_product(A3, K, out)
        for pb, v64, T in ((None, y64, T1), (p[1], z64, tol_swiglu(y64, c64, T1, T3))):
            y = q4.qmm_a8_fp8b(p[0], pb, N, K, x, out_dtype=a8.TYPES[out])
            a8.worst(np.abs(host_f64(y[torch.from_numpy(some).to(DEV)]) - v64), tol_bf16_out(v64, T) if out == "bf16" else T, out)
            for _ in range(4):
                assert torch.equal(q4.qmm_a8_fp8b(p[0], pb, N, K, x, out_dtype=a8.TYPES[out]), y)
    z = q4.qmm_a8_swiglu_a8(p[0], p[1], N, K, x)
    T = tol_swiglu(y64, c64, tol_product(A1, K, "a8"), tol_product(A3, K, "a8"))
    cz, sz = a8.codes_of(z)[some], a8.scales_of(z)[:, some]
    a8.worst(np.abs(oracle.dequantize_a8(cz, sz) - z64), tol_codes(cz, sz, z64, T), "codes")
    for _ in range(4):
        assert a8.same(q4.qmm_a8_swiglu_a8(p[0], p[1], N, K, x), z)
