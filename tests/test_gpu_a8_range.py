"""The norm at the ends of float32: rows whose squares leave its range."""

import numpy as np
import pytest
import torch

import bit_weight_only_q4g64_amd as q4
import oracle
from tests.a8_tolerance import tol_codes, tol_norm
from tests.gpu_helpers import DEV, host_f64, say
from tests.tolerance import tol_bf16_out

pytestmark = pytest.mark.gpu

# powers of two of a row's values: squares below the least float32, around it, past the largest one
POWERS = (-149, -126, -80, -76, -74, -70, -46, -44, 0, 60, 63, 64, 100, 126)


def rows_of_powers(rng, K, sub=1.0):
    x = rng.uniform(0.5, 1.0, (len(POWERS), K)) * np.where(rng.random((len(POWERS), K)) < 0.5, -1.0, 1.0) * sub
    return (x * np.exp2(np.array(POWERS, dtype=np.float64))[:, None]).astype(np.float32)


@pytest.mark.parametrize("eps", [0.0, 1e-38, 2.0**-120, 1e-5])
@pytest.mark.parametrize("K", [64, 512, 1024, 2112, 4096, 8192, 16384])
def test_norm_of_small_and_large_rows(K, eps):
    """Every finite row has its norm. tol_norm's bound counts the steps of the float32 form; float64 rows make fewer."""
    say(f"rms_norm range K={K} eps={eps}")
    rng = np.random.default_rng(K)
    x = rows_of_powers(rng, K)
    x[0] = np.where(rng.random(K) < 0.5, 2.0**-149, -(2.0**-148))  # subnormal values
    gamma = rng.normal(1, 0.3, K).astype(np.float32)
    xd, gd = torch.from_numpy(x).to(DEV), torch.from_numpy(gamma).to(DEV)
    y64 = oracle.rms_norm_rows(x, gamma, float(np.float32(eps)))
    assert np.all(np.isfinite(y64))
    T = tol_norm(y64)
    y = host_f64(q4.rms_norm(xd, gd, eps, out_dtype=torch.float32))
    assert np.all(np.abs(y - y64) <= T), [float(np.max(np.abs(y - y64)[i] / T[i])) for i in range(len(POWERS))]
    b = host_f64(q4.rms_norm(xd, gd, eps))
    assert np.all(np.abs(b - y64) <= tol_bf16_out(y64, T))
    a = q4.rms_norm_a8(xd, gd, eps)
    codes, scales = a.data.view(torch.uint8).cpu().numpy(), a.scales.cpu().numpy()
    assert np.all(np.abs(oracle.dequantize_a8(codes, scales) - y64) <= tol_codes(codes, scales, y64, T))
    # the same as a sum: zeros plus the row
    z, h = q4.rms_norm(torch.zeros_like(xd), gd, eps, residual=xd, out_dtype=torch.float32)
    assert torch.equal(h, xd) and np.array_equal(host_f64(z), y)


@pytest.mark.parametrize("K", [512, 2112])
def test_rows_beside_one_another_keep_their_bits(K):
    """A row out of range changes no other row, and rows in range keep the float32 form's bits."""
    say(f"rms_norm mixed rows K={K}")
    rng = np.random.default_rng(5)
    x = rng.normal(0, 1, (37, K)).astype(np.float32)
    gamma = torch.ones(K, device=DEV)
    clean = q4.rms_norm(torch.from_numpy(x).to(DEV), gamma, 0.0, out_dtype=torch.float32)
    x2 = x.copy()
    x2[::3] *= np.float32(2.0**-100)
    x2[1::3] *= np.float32(2.0**90)
    y = q4.rms_norm(torch.from_numpy(x2).to(DEV), gamma, 0.0, out_dtype=torch.float32)
    assert torch.equal(y[2::3], clean[2::3])
    want = oracle.rms_norm_rows(x, np.ones(K, np.float32), 0.0)
    assert np.all(np.abs(host_f64(y) - want) <= tol_norm(want))


def test_rows_without_a_norm():
    """A row of zeros with eps = 0 and one with a NaN are NaN; an infinity is NaN at its place and zeros elsewhere."""
    say("rms_norm rows without a norm")
    for K in (64, 2112):
        x = torch.full((4, K), 2.0**-100, device=DEV)
        x[0] = 0.0
        x[1, 7], x[2, 9] = float("nan"), float("-inf")
        y = q4.rms_norm(x, torch.ones(K, device=DEV), 0.0, out_dtype=torch.float32)
        assert torch.all(torch.isnan(y[:2])) and torch.isnan(y[2, 9]) and torch.all(y[2, :9] == 0) and torch.all(y[2, 10:] == 0)
        assert torch.all((y[3] - 1).abs() <= 2.0**-22)
