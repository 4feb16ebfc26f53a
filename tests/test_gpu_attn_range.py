"""Values, keys and scales near the ends of what the types hold, in the three attention kernels."""
import numpy as np
import pytest

from gpu_common import require_gpu, say

import dequant_gemv_q4_amd as q
from attn_common import attention64, check_attention, rounded
from test_gpu_attn_precision import ROWS, TYPES, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _check(kv_type, x, K, V, rows, scale, what):
    m, nq, hd = x.shape
    n = len(K)
    got = _run(kv_type, nq, 1, hd, 16, x, K, V, rows, scale)
    ref, A, S = (np.stack(v) for v in zip(*(attention64(x[r], K, V, 1, scale, n - m + r) for r in range(m))))
    assert (np.abs(ref) < 3.4e38).all()
    say(f"{what} type={kv_type} rows={rows} largest output {np.abs(ref).max():.3g}, got {np.abs(got).max():.3g}")
    check_attention(got.reshape(m, -1), ref.reshape(m, -1), A.reshape(m, -1), S[..., 0], [n - m + r + 1 for r in range(m)],
                    hd, kv_type, what)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("n", [200, 3000])
@pytest.mark.parametrize("kv_type,top", [(q.F16, 60000.0), (q.BF16, 1e30), (q.BF16, 1e36)])
def test_large_values(kv_type, top, n, rows):
    """V near the type's end: the output is a mean of them and no more than they are."""
    hd, nq, m = 64, 4, max(rows, 1)
    rng = np.random.default_rng([71, n])
    x = (rng.standard_normal((m, nq, hd)) * 0.5).astype(np.float32)
    K = rounded(rng.standard_normal((n, 1, hd)), kv_type)
    V = rounded(rng.uniform(-1.0, 1.0, (n, 1, hd)) * top, kv_type)
    _check(kv_type, x, K, V, rows, hd ** -0.5, f"V up to {top}")


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kv_type", TYPES)
def test_values_below_the_normal_range(kv_type, rows):
    """f16 V of its least steps; bf16 V of 1e-30."""
    hd, nq, n, m = 64, 4, 300, max(rows, 1)
    rng = np.random.default_rng(72)
    x = (rng.standard_normal((m, nq, hd)) * 0.5).astype(np.float32)
    K = rounded(rng.standard_normal((n, 1, hd)), kv_type)
    V = rounded(rng.standard_normal((n, 1, hd)) * (3e-7 if kv_type == q.F16 else 1e-30), kv_type)
    _check(kv_type, x, K, V, rows, hd ** -0.5, "small V")


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("scale", [1e-37, 2e-38, 5e-39, 1e-39, -1e-39, 1e-40])
def test_scales_below_the_normal_range(scale, rows):
    """Products of q and K near 1e38 times a scale around f32's least normal value, 1.2e-38."""
    hd, nq, n, m = 64, 4, 300, max(rows, 1)
    rng = np.random.default_rng(73)
    x, K = np.zeros((m, nq, hd), np.float32), np.zeros((n, 1, hd), np.float32)
    x[..., 0] = 1e19 * rng.uniform(0.5, 1.0, (m, nq))
    K[:, 0, 0] = rng.uniform(-1.0, 1.0, n) * min(1e19, 4.0 / abs(scale) / 1e19)
    K, V = rounded(K, q.BF16), rounded(rng.standard_normal((n, 1, hd)), q.BF16)
    _check(q.BF16, x, K, V, rows, scale, f"scale {scale}")
