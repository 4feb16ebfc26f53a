"""Shared prefixes with shares, lengths and groups at the ends of what the device may find, on the GPU against the
definition in 64 bits: every form of the kernels, and what the sticky flag says."""
import numpy as np
import pytest

from gpu_common import require_gpu, torch

import dequant_gemv_q4_amd as q
from kv_common import ALL, BYTES
from shared_common import Batch
from test_gpu_kv8 import _draw

pytestmark = pytest.mark.gpu

# rows, query heads, KV heads, channels, groups: forms of the kernels
FORMS = [(5, 4, 1, 64, 1, "16"), (520, 16, 1, 64, 1, "parted"), (140, 64, 1, 192, 2, "parted")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def alike(kv_type, n, nq, nkv, hd, form, prefix=150, own=20, n_group=1, seed=0, **kw):
    """n sequences of prefix + own positions; the same prefix in all of them."""
    rng = np.random.default_rng([41, seed])
    K, V = _draw(rng, [prefix + own] * n, nkv, hd)
    for b in range(1, n):
        K[b][:prefix], V[b][:prefix] = K[0][:prefix], V[0][:prefix]
    batch = Batch(kv_type, K, V, nq, nkv, hd, **kw)
    assert batch.form(n_group) == form
    return batch


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("n,nq,nkv,hd,n_group,form", FORMS)
def test_positions_that_no_row_sees_are_not_read(kv_type, n, nq, nkv, hd, n_group, form):
    """A share that is longer than every sequence of the group (a stale one of padded slots, say): entries behind the
    longest are not read, whatever they hold, and set no flag."""
    batch = alike(kv_type, n, nq, nkv, hd, form, n_group=n_group)
    starts = [0, n] if n_group == 1 else [0, n // 2, n]
    lens = [(7 * b) % 41 for b in range(n)]                  # at most 40 positions: three pages of 16
    batch.c.table[:, 3:] = -1
    got, flag = batch.call(starts, [150] * n, lens)
    batch.check(got, lens)
    assert flag == 0
    lens = [10] + [100 - b % 60 for b in range(1, n)]        # the first is short, others see what its pages hold
    batch = alike(kv_type, n, nq, nkv, hd, form, n_group=n_group, seed=1)
    batch.c.table[:, 7:] = 2 ** 30
    got, flag = batch.call(starts, [150] * n, lens)
    batch.check(got, lens)
    assert flag == 0


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("n,nq,nkv,hd,n_group,form", FORMS)
def test_flag_only_for_what_is_left_out(kv_type, n, nq, nkv, hd, n_group, form):
    """No flag for shares below zero or beyond the table where no sequence is, nor for a share larger than the
    first's of a sequence that ends before; one for positions between that are seen, which are left out."""
    batch = alike(kv_type, n, nq, nkv, hd, form, n_group=n_group)
    starts = [0, n] if n_group == 1 else [0, n // 2, n]
    lens = [160 - b % 90 for b in range(n)]
    for share in ([-7 if b in starts else -(b % 2) for b in range(n)], [2 ** 31 - 1] * n):
        batch = alike(kv_type, n, nq, nkv, hd, form, n_group=n_group, own=10 if share[0] > 0 else 20)
        if share[0] > 0:                                     # only what the first sequences hold is shared
            lens = [min(x, 150) for x in lens]
        got, flag = batch.call(starts, share, lens)
        batch.check(got, lens)
        assert flag == 0
    share = [40 if b in starts else 64 for b in range(n)]
    lens = [90 if b in starts else 40 - b % 3 for b in range(n)]
    got, flag = batch.call(starts, share, lens)
    batch.check(got, lens)
    assert flag == 0
    lens[n - 1] = 80
    got, flag = batch.call(starts, share, lens)
    batch.check(got, [np.r_[0:40, 64:80] if b == n - 1 else lens[b] for b in range(n)])
    assert flag == 1


def broken_starts(n, n_group):
    """Starts in order, then such as are not, or leave the sequences."""
    good = [i * n // n_group for i in range(n_group)] + [n]
    swapped = list(good)
    if n_group > 2:
        swapped[n_group // 2], swapped[n_group // 2 + 1] = swapped[n_group // 2 + 1], swapped[n_group // 2]
    else:
        swapped[0], swapped[1] = 3, 1
    overlap = list(good)
    overlap[n_group // 2] = n - 1
    overlap[-1] = n - 2
    return good, [swapped, good[::-1], [-1] + good[1:], good[:-1] + [n + 1], [-2 ** 31] + good[1:], overlap,
                  good[:-1] + [2 ** 31 - 1]]


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("n,nq,nkv,hd,n_group,form,extra", [
    (5, 4, 1, 64, 1, "16", 2), (9, 40, 1, 128, 4, "16", 2), (300, 4, 2, 64, 90, "16", 2), (520, 16, 1, 64, 1, "parted", 2),
    (140, 64, 1, 192, 2, "parted", 2), (60, 160, 1, 64, 20, "parted", 2), (134, 64, 16, 64, 44, "few", 70),
    (134, 64, 16, 64, 44, "whole", 2)])
def test_group_starts_out_of_order(kv_type, n, nq, nkv, hd, n_group, form, extra):
    """The flag, every sequence by itself from its own pages, and a workspace that serves the next call."""
    prefix, own = 30, 12
    batch = alike(kv_type, n, nq, nkv, hd, form, prefix=prefix, own=own, n_group=n_group, extra_entries=extra)
    good, bad = broken_starts(n, n_group)
    lens = [prefix + own - b % 25 for b in range(n)]
    share = [prefix] * n
    first, flag = batch.call(good, share, lens)
    batch.check(first, lens)
    assert flag == 0
    for starts in bad:
        got, flag = batch.call(starts, share, lens)
        batch.check(got, lens)
        assert flag == 1
        again, flag = batch.call(good, share, lens)
        assert flag == 0 and (again == first).all()
    if n <= 9:                                              # not from the first one's pages
        batch.c.table[1, 0] = -1
        got, flag = batch.call(bad[0], share, lens)
        batch.check(got, [np.r_[16:x] if b == 1 else x for b, x in enumerate(lens)])
        assert flag == 1


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("n,nq,nkv,hd,prefix,own", [(2, 12, 2, 128, 100, 9000), (5, 8, 4, 64, 37, 3000),
                                                    (3, 40, 2, 96, 500, 2500), (3, 4, 1, 256, 64, 4000)])
def test_equally_long_positions_behind_a_short_prefix(kv_type, n, nq, nkv, hd, prefix, own):
    """Fewer sequences than slots, all of them split behind the prefix; and once more on the same workspace."""
    batch = alike(kv_type, n, nq, nkv, hd, "16", prefix=prefix, own=own, n_group=1)
    lens = [prefix + own - b for b in range(n)]
    first, flag = batch.call([0, n], [prefix] * n, lens)
    batch.check(first, lens)
    again, again_flag = batch.call([0, n], [prefix] * n, lens)
    assert flag == again_flag == 0 and (again == first).all()


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("n,nq,nkv,hd,n_group,form,prefix,own,extra", [
    (3, 4, 1, 64, 1, "16", 2000, 1200, 2), (7, 40, 2, 256, 2, "16", 300, 700, 2), (512, 16, 1, 64, 1, "16", 30, 12, 2),
    (513, 16, 1, 64, 1, "parted", 30, 12, 2), (140, 64, 1, 256, 2, "parted", 150, 9, 60),
    (129, 64, 16, 64, 44, "few", 30, 12, 130), (129, 64, 16, 64, 44, "whole", 30, 12, 2)])
def test_nothing_behind_the_workspace_is_written(kv_type, n, nq, nkv, hd, n_group, form, prefix, own, extra):
    """A workspace of just the size that is asked for, with a pattern behind it, on both sides of the number of rows
    whose halves meet in one launch."""
    batch = alike(kv_type, n, nq, nkv, hd, form, prefix=prefix, own=own, n_group=n_group, extra_entries=extra)
    starts = [i * n // n_group for i in range(n_group)] + [n]
    lens = [prefix + own - b % 7 for b in range(n)]
    size = q.qgemv_attn_workspace_bytes(q.OP_ATTN_SHARED, n, nq, nkv, hd)
    guarded = torch.full((size + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    guarded[:size] = 0
    for _ in range(2):
        got, flag = batch.call(starts, [prefix] * n, lens, ws=guarded[:size])
        batch.check(got, lens)
        assert flag == 0
    assert bool((guarded[size:] == 0xA5).all())
    counters = guarded[256:256 + (2 * 512 + 8192) * 4]       # arrivals are 0 between calls
    assert not bool(counters.any())


def spoil(batch, b, page_entry, slots, kv_type, code=0x7F):
    """Positions `slots` of a sequence's page hold NaN in K and V (8-bit: NaN scales; of f8 0x7F is a NaN as well)."""
    page = int(batch.c.table[b, page_entry])
    hd, ps = batch.hd, batch.c.page
    for pool, turned in ((batch.c.k, False), (batch.c.v, True)):
        for h in range(batch.nkv):
            block = pool[page, h * batch.c.block:(h + 1) * batch.c.block]
            data = block[:ps * hd]
            data = data.view(hd, ps).T if turned else data.view(ps, hd)
            data[slots] = code if kv_type in BYTES else float("nan")
            if kv_type in BYTES:
                block[ps * hd:].view(torch.float32)[slots] = float("nan")


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("n,nq,nkv,hd,n_group,form", FORMS)
def test_a_begun_page_holds_anything_before_the_share_ends(kv_type, n, nq, nkv, hd, n_group, form):
    batch = alike(kv_type, n, nq, nkv, hd, form, prefix=150, own=20, n_group=n_group)
    starts = [0, n] if n_group == 1 else [0, n // 2, n]
    for b in set(range(n)) - set(starts):
        spoil(batch, b, 150 // 16, slice(0, 150 % 16), kv_type)
        batch.c.table[b, 150 // 16 - 1] = -1
    lens = [170 - b % 15 for b in range(n)]
    got, flag = batch.call(starts, [150] * n, lens)
    batch.check(got, lens)
    assert flag == 0


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("n,nq,nkv,hd,n_group,form", FORMS)
def test_non_finite_queries_and_positions_reach_their_rows_alone(kv_type, n, nq, nkv, hd, n_group, form):
    """A query with a NaN or an infinity, and a position of the prefix that only some sequences share (or see) and
    that is not finite: other rows and heads are as without them."""
    starts = [0, n] if n_group == 1 else [0, n // 2, n]
    batch = alike(kv_type, n, nq, nkv, hd, form, prefix=150, own=20, n_group=n_group)
    share = [150 if b in starts or b % 3 else 100 for b in range(n)]
    lens = [s + 9 - b % 7 for b, s in enumerate(share)]
    lens[3] = 90
    bad = {1: np.nan, n // 2 + 1: np.inf, n - 1: -np.inf}
    batch.q = batch.q.clone()
    for b, x in bad.items():
        batch.q[b, 5] = float(x)                             # of head 0
    clean = [b for b in range(n) if b not in bad]
    got, flag = batch.call(starts, share, lens)
    assert flag == 0
    got = got.reshape(n, nq, hd)
    for b in bad:
        finite = int(np.isfinite(got[b, 0]).sum())
        assert finite == 0
        got[b, 0] = 0.0
    finite = bool(np.isfinite(got).all())
    assert finite
    plain = alike(kv_type, n, nq, nkv, hd, form, prefix=150, own=20, n_group=n_group)
    want, _ = plain.call(starts, share, lens)
    want = want.reshape(n, nq, hd)
    far = np.abs(got[clean] - want[clean]).max()
    assert far <= 1e-6 * np.abs(want).max()
    for b in starts[:-1]:                                   # positions 112 .. 115 of the shared pages
        spoil(plain, b, 7, slice(0, 4), kv_type, code=0)     # (as the append leaves them)
    got, flag = plain.call(starts, share, lens)
    sees = np.array([min(s, x) > 112 for s, x in zip(share, lens)])
    assert flag == 0 and sees.any() and not sees.all()
    nans = int(np.isnan(got[sees]).sum())
    assert nans == got[sees].size
    far = np.abs(got.reshape(n, nq, hd)[~sees] - want[~sees]).max()
    assert far <= 1e-6 * np.abs(want).max()


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 40.0])
def test_scales_of_any_sign_and_size(kv_type, scale):
    for n, nq, nkv, hd, n_group, form in FORMS[:2]:
        batch = alike(kv_type, n, nq, nkv, hd, form, scale=scale, seed=2)
        lens = [170 - b % 90 for b in range(n)]
        got, flag = batch.call([0, n], [150] * n, lens)
        batch.check(got, lens)
        assert flag == 0


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("form,extra", [("few", 70), ("whole", 2)])
def test_stale_shares_of_many_groups(kv_type, form, extra):
    """More groups than workgroup slots: each group's rows see less than its share, some of them nothing."""
    n, n_group = 134, 44
    batch = alike(kv_type, n, 64, 16, 64, form, prefix=90, own=6, n_group=n_group, extra_entries=extra)
    starts = [i * n // n_group for i in range(n_group)] + [n]
    lens = [max(0, (11 * b) % 53 - 5) for b in range(n)]    # at most 47: three pages of 16
    batch.c.table[:, 3:] = -1
    got, flag = batch.call(starts, [2 ** 31 - 1 if b in starts else 90 for b in range(n)], lens)
    batch.check(got, lens)
    assert flag == 0
