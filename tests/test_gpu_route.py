"""Expert routing on the GPU against its definition in 64 bits: the ids have to be equal, the
weights are off by at most 2^-23 relative (one rounding to f32, 2^-24, and f64 work)."""
import numpy as np
import pytest

from gpu_common import dev, host, require_gpu, say, torch

import dequant_gemv_q4_amd as q
from attn_common import route64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _route(z, score, bias, groups, gtop, keep, topk, renorm, scale=1.0):
    rows, n = z.shape
    ids = torch.full((rows, topk), -1, dtype=torch.int32, device="cuda")
    w = torch.full((rows, topk), float("nan"), device="cuda")
    q.qgemv_route(dev(z), rows, n, score, None if bias is None else dev(bias), groups, gtop, keep, topk,
                  renorm, scale, ids, w)
    return host(ids), host(w)


def _check(z, score, bias, groups, gtop, keep, topk, renorm, scale=1.0):
    say(f"route {z.shape} score={score} groups={groups}/{gtop}/{keep} topk={topk} renorm={renorm}")
    gi, gw = _route(z, score, bias, groups, gtop, keep, topk, renorm, scale)
    with np.errstate(all="ignore"):
        ri, rw = route64(z, score, bias, groups, gtop, keep, topk, renorm, scale)
    assert np.array_equal(gi, ri)
    assert np.abs(gw - rw).max() <= (2.0 ** -23 * np.abs(rw) + 1e-45).max()
    assert (np.abs(gw - rw) <= 2.0 ** -23 * np.abs(rw) + 2.0 ** -149).all()


@pytest.mark.parametrize("score", [q.SCORE_SOFTMAX, q.SCORE_SIGMOID])
@pytest.mark.parametrize("n,groups,gtop,keep,topk", [
    (64, 1, 1, 1, 8), (1, 1, 1, 1, 1), (3, 1, 1, 1, 3), (63, 7, 2, 3, 5), (65, 5, 1, 2, 8), (256, 8, 2, 4, 8),
    (160, 8, 1, 3, 6), (1000, 4, 2, 1, 8), (1024, 1024, 1, 8, 8), (1024, 1, 2, 1, 7), (128, 64, 2, 2, 4),
    (512, 2, 2, 2, 1), (37, 37, 1, 5, 5)])
@pytest.mark.parametrize("bias,renorm", [(False, True), (True, True), (True, False)])
def test_route(score, n, groups, gtop, keep, topk, bias, renorm):
    rng = np.random.default_rng([91, n, groups, topk])
    z = (rng.standard_normal((19, n)) * 2).astype(np.float32)
    b = (rng.standard_normal(n) * 0.1).astype(np.float32) if bias else None
    _check(z, score, b, groups, gtop, keep, topk, renorm, 2.5 if renorm else 1.0)


@pytest.mark.parametrize("n,groups,gtop,keep,topk", [
    (1000, 8, 2, 4, 8), (1000, 125, 1, 7, 8), (1000, 20, 2, 3, 8), (999, 27, 2, 5, 6), (660, 33, 2, 8, 8), (1020, 340, 2, 9, 8),
    (96, 32, 1, 4, 4), (10, 2, 2, 1, 3), (189, 63, 1, 8, 8)])
def test_route_groups_that_are_no_run_of_lanes(n, groups, gtop, keep, topk):
    """A group's lanes are 32 down to one; equal choices within and across them go to the lower index."""
    rng = np.random.default_rng([92, n, groups])
    z = (rng.standard_normal((9, n)) * 2).astype(np.float32)
    z[3] = np.round(z[3])
    z[4] = 0.25
    z[5, ::2] = -np.inf
    b = np.round(rng.standard_normal(n) * 8).astype(np.float32) / 64
    for bias in (None, b):
        _check(z, q.SCORE_SIGMOID, bias, groups, gtop, keep, topk, True, 1.0)
        _check(z, q.SCORE_SOFTMAX, bias, groups, gtop, keep, topk, False, 2.0)


def test_route_many_rows():
    rng = np.random.default_rng(5)
    z = rng.standard_normal((4099, 64)).astype(np.float32)
    _check(z, q.SCORE_SOFTMAX, None, 1, 1, 1, 8, True)


def test_route_matches_the_expert_workload():
    """The routed-expert workload's own ids and weights (softmax over the selected logits)."""
    import workloads as wl
    z = wl.rng(4, wl.T_ROUTER).standard_normal(size=(16, 64)).astype(np.float32)
    ids, p = wl.route_top_k(z, 8)
    gi, gw = _route(z, q.SCORE_SOFTMAX, None, 1, 1, 1, 8, True)
    assert np.array_equal(gi, ids)
    assert np.abs(gw - p).max() <= 2.0 ** -22


def test_route_ties_go_to_the_lower_index():
    z = np.zeros((3, 200), np.float32)
    z[1, 150:] = 1.0
    z[2, ::7] = 2.0
    _check(z, q.SCORE_SOFTMAX, None, 1, 1, 1, 8, True)
    _check(z, q.SCORE_SIGMOID, np.zeros(200, np.float32), 10, 2, 3, 8, True)
    _check(z, q.SCORE_SIGMOID, None, 10, 1, 3, 8, False)
    gi, _ = _route(z, q.SCORE_SOFTMAX, None, 1, 1, 1, 8, True)
    assert gi[0].tolist() == list(range(8))


def test_route_near_ties_are_decided_in_64_bits():
    """Choices that differ by less than an f32 rounding of s + bias."""
    rng = np.random.default_rng(8)
    base = rng.standard_normal(64)
    z = np.repeat(base[None], 50, 0).astype(np.float32)
    s = 1.0 / (1.0 + np.exp(-z[0].astype(np.float64)))
    b = (1.0 - s).astype(np.float32)              # every choice is 1 within 2^-24 or so
    _check(z, q.SCORE_SIGMOID, b, 1, 1, 1, 8, True)
    _check(z, q.SCORE_SIGMOID, b, 8, 2, 3, 8, True)


def test_route_extreme_logits():
    """Scores that under- and overflow, -inf logits (score 0, still selectable), large ones."""
    z = np.full((4, 70), -np.inf, np.float32)
    z[0, 3] = 1.0
    z[1, :] = np.linspace(-3e38, 3e38, 70, dtype=np.float32)
    z[2, :] = np.linspace(-200, 200, 70, dtype=np.float32)
    z[3, 5:9] = [1e-30, -1e-30, 0.0, 88.0]
    _check(z, q.SCORE_SOFTMAX, None, 1, 1, 1, 8, True)
    b = np.linspace(-1, 1, 70, dtype=np.float32)
    _check(z, q.SCORE_SOFTMAX, b, 7, 2, 2, 8, False)
    _check(z[2:], q.SCORE_SIGMOID, b, 7, 2, 2, 8, False)


def test_route_nan_choices_rank_last():
    rng = np.random.default_rng(2)
    z = rng.standard_normal((2, 40)).astype(np.float32)
    z[0, 7] = np.nan
    b = np.zeros(40, np.float32)
    b[[1, 2, 3]] = np.nan
    gi, gw = _route(z, q.SCORE_SIGMOID, b, 1, 1, 1, 8, True)
    assert not {1, 2, 3} & set(gi.reshape(-1).tolist()) and 7 not in gi[0]
    assert np.isfinite(gw).all()
    gi, _ = _route(np.full((1, 5), np.nan, np.float32), q.SCORE_SOFTMAX, None, 1, 1, 1, 5, True)
    assert gi[0].tolist() == [0, 1, 2, 3, 4]      # valid ids whatever the scores
