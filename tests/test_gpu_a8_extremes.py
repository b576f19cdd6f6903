"""The 8-bit activation path at its largest sizes, and calls on two streams at once."""

import numpy as np
import pytest
import torch

import bit_weight_only_q4g64_amd as q4
import oracle
import synthetic
from tests.a8_tolerance import tol_norm, tol_product
from tests.gpu_helpers import DEV, host_f64, say
from tests.test_gpu_a8 import TYPES, codes_of, dev_fp8, draw_a8, pair_weights, same, scales_of, worst
from tests.tolerance import tol_bf16_out, tol_swiglu

pytestmark = pytest.mark.gpu

MAX_M, MAX_K = 2**24, 2**20


def some_rows(rng, M, n=200):
    return np.unique(np.concatenate([rng.integers(0, M, n), [0, M - 1]]))


def test_quantizer_and_norm_of_the_most_rows():
    """2^24 rows: rows from all over against the oracle, and the halves alone give the same bits."""
    say("quant_a8 and rms_norm of 2^24 rows")
    rng, K = np.random.default_rng(1), 64
    x = torch.randn((MAX_M, K), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(torch.bfloat16)
    pick = some_rows(rng, MAX_M)
    xs = x[torch.from_numpy(pick).to(DEV)].float().cpu().numpy()
    a = q4.quant_a8(x)
    codes, scales = oracle.quantize_a8(xs)
    at = torch.from_numpy(pick).to(DEV)
    assert np.array_equal(a.data.view(torch.uint8)[at].cpu().numpy(), codes) and np.array_equal(a.scales[:, at].cpu().numpy(), scales)
    half = MAX_M // 2
    for lo, hi in ((0, half), (half, MAX_M)):
        b = q4.quant_a8(x[lo:hi])
        assert torch.equal(a.data[lo:hi].view(torch.uint8), b.data.view(torch.uint8)) and torch.equal(a.scales[:, lo:hi], b.scales)
    del a, b
    gamma = torch.ones(K, device=DEV)
    y = q4.rms_norm(x, gamma, 1e-5)
    y64 = oracle.rms_norm_rows(xs, np.ones(K), 1e-5)
    worst(np.abs(host_f64(y[at]) - y64), tol_bf16_out(y64, tol_norm(y64)), "norm")
    for lo, hi in ((0, half), (half, MAX_M)):
        assert torch.equal(y[lo:hi], q4.rms_norm(x[lo:hi], gamma, 1e-5))


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_product_of_many_rows(out):
    say(f"qmm_a8_fp8b of 2^22 rows {out}")
    rng, M, N, K = np.random.default_rng(2), 2**22 + 7, 64, 192
    w = synthetic.draw_fp8_weight(rng, "w", N, K)
    x = q4.quant_a8(torch.randn((M, K), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)))
    y = q4.qmm_a8_fp8b(dev_fp8(w.w8, w.scales), None, N, K, x, out_dtype=TYPES[out])
    pick = some_rows(rng, M)
    at = torch.from_numpy(pick).to(DEV)
    y64, A = oracle.matmul_a8(w.w8, w.scales, x.data.view(torch.uint8)[at].cpu().numpy(), x.scales[:, at].cpu().numpy())
    T = tol_product(A, K, out)
    worst(np.abs(host_f64(y[at]) - y64), tol_bf16_out(y64, T) if out == "bf16" else T, out)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_longest_k(M):
    """K = 2^20: products and pairs in every type of result."""
    say(f"K = 2^20, M={M}")
    rng, N, K = np.random.default_rng(3), 64, MAX_K
    w = synthetic.draw_fp8_weight(rng, "w", N, K)
    p = dev_fp8(w.w8, w.scales)
    x = q4.quant_a8(torch.randn((M, K), device=DEV, generator=torch.Generator(device=DEV).manual_seed(M)))
    pick = some_rows(rng, M, 4)
    y64, A = oracle.matmul_a8(w.w8, w.scales, codes_of(x)[pick], scales_of(x)[:, pick])
    z64 = oracle.swiglu(y64, y64)
    for out in ("f32", "bf16"):
        T = tol_product(A, K, out)
        y = host_f64(q4.qmm_a8_fp8b(p, None, N, K, x, out_dtype=TYPES[out]))[pick]
        worst(np.abs(y - y64), tol_bf16_out(y64, T) if out == "bf16" else T, out)
        z = host_f64(q4.qmm_a8_fp8b(p, p, N, K, x, out_dtype=TYPES[out]))[pick]
        Tz = tol_swiglu(y64, y64, T, T)
        worst(np.abs(z - z64), tol_bf16_out(z64, Tz) if out == "bf16" else Tz, "pair " + out)
    q = q4.qmm_a8_swiglu_a8(p, p, N, K, x)
    want = q4.quant_a8(q4.qmm_a8_fp8b(p, p, N, K, x))
    assert np.all(np.abs(oracle.dequantize_a8(codes_of(q), scales_of(q)) - oracle.dequantize_a8(codes_of(want), scales_of(want)))
                  <= 2.0**-3 * np.abs(oracle.dequantize_a8(codes_of(want), scales_of(want))) + 2.0**-9 * np.repeat(scales_of(want).T, 128, axis=1)[:, :N])


@pytest.mark.parametrize("M", [2, 40])
def test_most_columns(M):
    """N = 2^22: columns from both ends against the oracle."""
    say(f"N = 2^22, M={M}")
    rng, N, K, ends = np.random.default_rng(4), 2**22, 64, 256
    w8 = torch.randint(0, 256, (N, K), dtype=torch.uint8, device=DEV, generator=torch.Generator(device=DEV).manual_seed(4)) & 0xF7
    sc = torch.rand((N // 128, 1), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)) + 0.5
    codes, scales, x = draw_a8(rng, M, K)
    p = q4.pack_fp8b(w8, sc)
    for out in ("f32", "bf16"):
        y = q4.qmm_a8_fp8b(p, None, N, K, x, out_dtype=TYPES[out])
        for cols in (slice(0, ends), slice(N - ends, N)):
            blocks = slice(cols.start // 128, cols.stop // 128)
            y64, A = oracle.matmul_a8(w8[cols].cpu().numpy(), sc[blocks].cpu().numpy(), codes, scales)
            T = tol_product(A, K, out)
            worst(np.abs(host_f64(y[:, cols]) - y64), tol_bf16_out(y64, T) if out == "bf16" else T, out)


def test_two_streams_at_once():
    """The whole chain on two streams at the same time, without scratch memory of the caller, gives what it gives alone."""
    say("two streams")
    rng = np.random.default_rng(6)
    N, K = 2176, 1088
    p1, p3 = pair_weights(rng, N, K)
    gamma = torch.ones(K, device=DEV)
    xs = [torch.randn((M, K), device=DEV).to(torch.bfloat16) for M in (40, 45)]  # two launches and scratch memory each

    def chain(x):
        a = q4.rms_norm_a8(x, gamma, 1e-5)
        return a, q4.qmm_a8_swiglu_a8(p1, p3, N, K, a), q4.qmm_a8_fp8b(p1, p3, N, K, a, out_dtype=torch.bfloat16)

    assert all(q4.a8_swiglu_work_bytes(x.shape[0], N, K) for x in xs)
    refs = [chain(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(chain(xs[i]))
    torch.cuda.synchronize()
    for i, ref in enumerate(refs):
        for a, z, y in got[i]:
            assert same(a, ref[0]) and same(z, ref[1]) and torch.equal(y, ref[2])
