"""Attention over 8-bit pages where the scales of K or V span much of f32's range, on the GPU against the
definition in 64 bits (kv_common): values of V far larger than a row sees, or that grow from step to step."""
import numpy as np
import pytest

from gpu_common import require_gpu

from kv_common import BYTES
from shared_common import Batch
from test_gpu_kv8 import _draw, attend, in_16s

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def unit(v):
    """Every position's largest |value| 1, so that all scales are alike."""
    return v / np.abs(v).max(axis=-1, keepdims=True)


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("size", [1e12, 1e18, 1e22])
@pytest.mark.parametrize("rows,n,hd", [(40, 40, 64), (300, 300, 64), (130, 800, 64), (650, 650, 64), (700, 800, 64),
                                       (60, 500, 128), (500, 700, 256)])
def test_rows_before_values_far_larger(kv_type, size, rows, n, hd):
    """V up to 2^73 times larger at the last positions: the rows that do not see them keep their precision, in
    tiles of 16 columns and of 128."""
    rng = np.random.default_rng([31, hd])
    K, V = _draw(rng, [n], 1, hd, 0.0)
    V[0][n - 5:] *= np.float32(size)
    assert in_16s(rows, 1, 4, 1, hd, n + 16384) == (rows <= 300)
    attend(kv_type, 4, 1, hd, 16, [(rows, n)], 1, K=K, V=V, extra_entries=1024)


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("seqs,nkv,prompt", [([(1, 900)] * 130, 4, False), ([(1, 900 + b) for b in range(9)], 1, False),
                                             ([(40, 900)], 1, True), ([(700, 900)], 1, True)])
def test_values_that_grow_in_steps(kv_type, seqs, nkv, prompt):
    """V 2^29 and then 2^31 times larger than at first (as many sequences as workgroup slots: none is split, a wave
    meets all three), then much further."""
    rng = np.random.default_rng(32)
    K, V = _draw(rng, [b for _, b in seqs], nkv, 64, 0.0)
    V = [unit(v) for v in V]
    for v in V:
        v[256:] *= np.float32(2.0 ** 29)
        v[512:] *= np.float32(4.0)
    rows = sum(a for a, _ in seqs)
    assert not prompt or in_16s(rows, len(seqs), 4 * nkv, nkv, 64, 900 + 16384) == (rows < 200)
    kw = dict(prompt=prompt, extra_entries=1024 if prompt else 2)
    attend(kv_type, 4 * nkv, nkv, 64, 16, seqs, 1, K=K, V=V, **kw)
    for v in V:
        v[512:] *= np.float32(2.0 ** 31)
        v[-40:] *= np.float32(2.0 ** 33)
    attend(kv_type, 4 * nkv, nkv, 64, 16, seqs, 2, K=K, V=V, **kw)


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("n,nq,form", [(6, 4, "16"), (130, 64, "parted"), (520, 16, "parted")])
def test_shares_that_end_before_values_far_larger(kv_type, n, nq, form):
    """A prefix whose last positions hold values 2^60 times larger, which only some sequences share."""
    hd, long, short = 64, 150, 100
    rng = np.random.default_rng(33)
    K, V = _draw(rng, [long], 1, hd, 0.0)
    V[0][short:] *= np.float32(1e18)
    rest = _draw(rng, [7], 1, hd, 0.0)
    share = [long if b % 3 == 0 else short for b in range(n)]
    Ks, Vs = ([np.concatenate([x[0][:s], y[0]]) for s in share] for x, y in zip((K, V), rest))
    batch = Batch(kv_type, Ks, Vs, nq, 1, hd)
    assert batch.form(1) == form
    lens = [s + 7 for s in share]
    got, flag = batch.call([0, n], share, lens)
    batch.check(got, lens)
    assert flag == 0


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("k_size,q_size", [(1e30, 1.0), (1e33, 1.0), (1e36, 1e-5), (1e-36, 1e37), (1e-30, 1e30), (1e36, 1e-36)])
@pytest.mark.parametrize("rows,n,prompt,hd", [(1, 900, False, 64), (1, 700, False, 256), (40, 300, True, 128),
                                              (700, 800, True, 64), (500, 700, True, 256)])
def test_scores_of_keys_and_queries_of_any_size(kv_type, k_size, q_size, rows, n, prompt, hd):
    """Ordinary scores of K near either end of f32's range, where the products on the way are not."""
    rng = np.random.default_rng([34, hd])
    K, V = _draw(rng, [n], 1, hd, 0.0)
    K[0] *= np.float32(k_size)
    assert not prompt or in_16s(rows, 1, 4, 1, hd, n + 16384) == (rows < 300)
    attend(kv_type, 4, 1, hd, 16, [(rows, n)], 1, K=K, V=V, prompt=prompt, extra_entries=1024 if prompt else 2,
           scale=hd ** -0.5 / (k_size * q_size), qmul=q_size)


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("rows,n", [(40, 300), (700, 800)])
def test_scores_of_keys_of_all_sizes_in_one_step(kv_type, rows, n):
    """Keys from 1e-35 to 1e35 side by side, and queries from 1e-30 to 1e2: a large one's score is the row's
    maximum or its minimum, the small ones' are near zero."""
    rng = np.random.default_rng(35)
    K, V = _draw(rng, [n], 1, 64, 0.0)
    K[0] *= (10.0 ** rng.integers(-35, 36, (n, 1, 1))).astype(np.float32)
    assert in_16s(rows, 1, 4, 1, 64, n + 16384) == (rows < 300)
    for qmul in (1e-30, 1e-10, 1e2):
        attend(kv_type, 4, 1, 64, 16, [(rows, n)], 2, K=K, V=V, extra_entries=1024, scale=1e-3, qmul=qmul)


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("n,nq,form", [(6, 4, "16"), (520, 16, "parted")])
@pytest.mark.parametrize("k_size,q_size", [(1e33, 1.0), (1e-36, 1e37)])
def test_scores_behind_a_prefix_of_keys_of_any_size(kv_type, n, nq, form, k_size, q_size):
    rng = np.random.default_rng(36)
    K, V = _draw(rng, [150] * n, 1, 64, 0.0)
    for b in range(1, n):
        K[b][:130], V[b][:130] = K[0][:130], V[0][:130]
    K = [k * np.float32(k_size) for k in K]
    batch = Batch(kv_type, K, V, nq, 1, 64, q_size=q_size, scale=0.125 / (k_size * q_size))
    assert batch.form(1) == form
    got, flag = batch.call([0, n], [130] * n, [150] * n)
    batch.check(got, [150] * n)
    assert flag == 0
