"""The 8-bit cache on the GPU: quantising rows as they are written, the attentions that read it, and the
fused norm, rotation and append, against their definitions in 64 bits (kv_common)."""
import ctypes

import numpy as np
import pytest

from gpu_common import dev, host, require_gpu, say, torch

import dequant_gemv_q4_amd as q
from dequant_gemv_q4_amd import device as D
from kv_common import ALL, BYTES, Cache, as_bytes, check_rows, codes64, held, parts64, quantised, scales64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------------- append

def _empty(kv_type, n_pages, page, nkv, hd, gap=0):
    """A cache whose every byte is 0x3B, and its host copy."""
    c = Cache(kv_type, [], [], page, nkv, hd, np.random.default_rng(0), spare=n_pages, extra_entries=1)
    size = 1 if kv_type in BYTES else 2
    c.page_stride += gap
    raw = np.full((n_pages, c.page_stride * size), 0x3B, np.uint8)
    dt = torch.uint8 if kv_type in BYTES else {q.F16: torch.float16, q.BF16: torch.bfloat16}[kv_type]
    c.n_pages = n_pages
    c.k, c.v = (torch.from_numpy(raw.copy()).view(dt).cuda() for _ in range(2))
    return c


def _pool(t):
    h = t.cpu()
    return h.numpy() if h.dtype == torch.uint8 else h.float().numpy()


def _expect(before, c, seqs, table, K, V, nkv):
    """The pools as the definition leaves them, as bytes (8-bit) or f32 (else); K, V [rows][nkv][hd] f64 or f32."""
    k, v = before[0].copy(), before[1].copy()
    hd, page, r = c.hd, c.page, 0
    for b, (a, n) in enumerate(seqs):
        for i in range(a):
            t = n - a + i
            if t >= 0 and t // page < table.shape[1] and 0 <= table[b, t // page] < c.n_pages:
                pg, slot = table[b, t // page], t % page
                for pool, rows, turned in ((k, K, False), (v, V, True)):
                    for h in range(nkv):
                        blk = pool[pg, h * c.block:(h + 1) * c.block]
                        body = blk[:page * hd].reshape((hd, page) if turned else (page, hd))
                        body = body[:, slot] if turned else body[slot]
                        if c.kv_type in BYTES:
                            codes, d = quantised(rows[r + i, h], c.kv_type)
                            body[:] = as_bytes(codes, c.kv_type)
                            blk[page * hd + 4 * slot:page * hd + 4 * slot + 4] = np.frombuffer(d.tobytes(), np.uint8)
                        else:
                            body[:] = held(rows[r + i, h], c.kv_type)
        r += a
    return k, v


def _same(got, want, c, what):
    """Bytes of two pools: of f8 codes the zero has two signs; NaN scales may differ in their payload."""
    if c.kv_type not in BYTES:
        assert np.array_equal(got, want, equal_nan=True), what
        return
    if c.kv_type == q.F8:
        got, want = np.where(got == 0x80, 0, got), np.where(want == 0x80, 0, want)
    body, page = c.page * c.hd, c.page
    for h in range(c.nkv):
        a, b = (x[:, h * c.block:(h + 1) * c.block] for x in (got, want))
        assert np.array_equal(a[:, :body], b[:, :body]), f"{what}: {int((a[:, :body] != b[:, :body]).sum())} codes"
        da, db = (np.ascontiguousarray(x[:, body:]).view(np.float32) for x in (a, b))
        assert np.array_equal(da, db, equal_nan=True), f"{what}: scales"
    assert np.array_equal(got[:, c.nkv * c.block:], want[:, c.nkv * c.block:]), what


def _append(kv_type, nkv, hd, page, seqs, rows=None, seed=0, decode=False, bad=None, gap=0, tail=2):
    say(f"append8 type={kv_type} nkv={nkv} hd={hd} page={page} seqs={seqs[:6]} decode={decode}")
    rng = np.random.default_rng([90, seed])
    n = sum(a for a, _ in seqs)
    need = [max(0, -(-b // page)) for _, b in seqs]
    c = _empty(kv_type, sum(need) + 2, page, nkv, hd, gap)
    table = np.full((len(seqs), max(need) + 1), -1, np.int32)
    perm, at = rng.permutation(c.n_pages), 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    if bad:
        table[bad] = c.n_pages
    total = n + (0 if decode else tail)
    x = rows if rows is not None else (rng.standard_normal((total, 2, nkv, hd)) *
                                       np.exp(rng.standard_normal((total, 2, nkv, 1)))).astype(np.float32)
    stride = 2 * nkv * hd + 8
    buf = np.zeros((total, stride), np.float32)
    buf[:, :2 * nkv * hd] = x.reshape(total, -1)
    xd, td, ws = dev(buf), dev(table), D.attn_workspace(q.OP_KV_APPEND, len(seqs), nkv, nkv, hd)
    before = _pool(c.k), _pool(c.v)
    start = None if decode else ints(np.concatenate([[0], np.cumsum([a for a, _ in seqs])]))
    q.qgemv_kv_append(kv_type, c.k, c.v, c.n_pages, page, c.page_stride, nkv, hd, td, table.shape[1], start,
                      ints(b for _, b in seqs), len(seqs), xd, xd[:, nkv * hd:], stride, total, ws)
    torch.cuda.synchronize()
    want = _expect(before, c, seqs, table, x[:, 0], x[:, 1], nkv)
    _same(_pool(c.k), want[0], c, "K")
    _same(_pool(c.v), want[1], c, "V")
    over = any(b > page * table.shape[1] for _, b in seqs)
    assert q.qgemv_attn_error(ws) == (1 if bad or over else 0)


SEQS = [(1, 1), (5, 5), (0, 0), (17, 40), (33, 33), (1, 66), (40, 39), (3, 0), (2, -4), (64, 64), (16, 48), (31, 31)]


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("nkv,hd,page", [(2, 128, 16), (1, 64, 32), (3, 96, 64), (2, 192, 128), (1, 256, 256)])
def test_append8(kv_type, nkv, hd, page):
    _append(kv_type, nkv, hd, page, SEQS, seed=hd)
    _append(kv_type, nkv, hd, page, [(1, n) for n in (1, 16, 17, 32, 200, 33, 0, -1)], seed=hd + 1, decode=True)


@pytest.mark.parametrize("kv_type", BYTES)
def test_append8_bad_pages_gaps_and_many_sequences(kv_type):
    _append(kv_type, 2, 64, 16, [(20, 50), (9, 9)], seed=1, bad=(0, 2), gap=48)
    rng = np.random.default_rng(2)
    _append(kv_type, 1, 64, 16, [(int(a), int(a + c)) for a, c in zip(rng.integers(0, 4, 300), rng.integers(0, 40, 300))],
            seed=2)


@pytest.mark.parametrize("kv_type", BYTES)
def test_append8_ties_extremes_and_non_finite_rows(kv_type):
    """Rows of integers and halves (exact ties), zeros, the least and the largest values, infinities, NaN."""
    rng = np.random.default_rng(3)
    n, hd = 40, 64
    x = np.zeros((n, 2, 1, hd), np.float32)
    top = 127.0 if kv_type == q.I8 else 448.0
    for r in range(n):
        v = rng.integers(-2 * top, 2 * top + 1, (2, hd)).astype(np.float32) / 2
        v[:, r % hd] = top
        x[r, :, 0] = v * np.float32(2.0) ** rng.integers(-40, 40)
    x[1] = 0.0
    x[2] = np.float32(1e-45)
    x[3, :, 0] = rng.standard_normal((2, hd)) * 1e-38
    x[4, :, 0] = np.float32(3.4028235e38) * rng.uniform(-1, 1, (2, hd))
    x[4, :, 0, 5] = np.float32(3.4028235e38)
    x[5, :, 0, 7], x[6, :, 0, 9], x[7, 0, 0, 63], x[8, 1, 0, 0] = np.inf, np.nan, -np.inf, np.nan
    x[9, :, 0] = rng.standard_normal((2, hd)) * 2e-36
    _append(kv_type, 1, hd, 32, [(n, n)], rows=x, tail=0)
    # many values near borders: quotients within a few last places of n + 1/2
    n = 512
    x = np.zeros((n, 2, 1, hd), np.float32)
    d = np.exp(rng.uniform(-5, 5, (n, 2, 1, 1))).astype(np.float32)
    m = rng.integers(-126, 127, x.shape) + 0.5
    x[:] = np.nextafter((m * d).astype(np.float32), rng.choice([-np.inf, np.inf, 0], x.shape).astype(np.float32))
    x[..., 0] = (d * np.float32(top))[..., 0]
    _append(kv_type, 1, hd, 64, [(n, n)], rows=x, tail=0)


# --------------------------------------------------------------------- norm, rotation and append

def _turn64(x, gamma, eps, cos, sin):
    """x [heads][hd] f64, cos and sin [half]."""
    x = x.astype(np.float64)
    if gamma is not None:
        x = x * gamma.astype(np.float64) / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    h = len(cos)
    a, b = x[:, :h].copy(), x[:, h:2 * h].copy()
    x = x.copy()
    x[:, :h], x[:, h:2 * h] = a * cos - b * sin, b * cos + a * sin
    return x


def _near(x, kv_type, hd):
    """Where a value's rounding to the type is decided by less than 2^-40 of its step: f64 sums in another
    order move a value by 2^-52 (hd + 8) at most, of 2^10 codes' worth."""
    if kv_type in BYTES:
        d = scales64(x, kv_type)
        return codes64(x, d, kv_type)[1] < 2.0 ** -30
    bits = 11 if kv_type == q.F16 else 8
    m, e = np.frexp(x)
    y = np.abs(m) * 2.0 ** bits
    return np.abs(y - np.floor(y) - 0.5) < 2.0 ** -25


def _qkv(kv_type, nq, nkv, hd, page, seqs, half, norm=True, seed=0, decode=False, in_place=False, rope_rows=None,
         tail=2, top_len=None):
    say(f"qkv type={kv_type} nq={nq} nkv={nkv} hd={hd} page={page} half={half} seqs={seqs[:6]} in_place={in_place}")
    rng = np.random.default_rng([91, seed])
    n = sum(a for a, _ in seqs)
    total = n + (0 if decode else tail)
    need = [max(0, -(-b // page)) for _, b in seqs]
    c = _empty(kv_type, sum(need) + 2, page, nkv, hd)
    table = np.full((len(seqs), max(need) + 1), -1, np.int32)
    perm, at = rng.permutation(c.n_pages), 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    longest = max(b for _, b in seqs)
    rope_rows = max(longest, 1) if rope_rows is None else rope_rows
    angle = np.arange(rope_rows)[:, None] * 10000.0 ** (-np.arange(half) / max(half, 1))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    width = (nq + 2 * nkv) * hd
    stride = width + 4
    x = rng.standard_normal((total, stride)).astype(np.float32)
    qg, kg = ((1 + 0.3 * rng.standard_normal(hd)).astype(np.float32) if norm else None for _ in range(2))
    xd = dev(x)
    out = xd if in_place else torch.full((total, nq * hd), 77.0, device="cuda")
    ws = D.attn_workspace(q.OP_QKV_APPEND, len(seqs), nq, nkv, hd)
    before = _pool(c.k), _pool(c.v)
    start = None if decode else ints(np.concatenate([[0], np.cumsum([a for a, _ in seqs])]))
    q.qgemv_qkv_append(kv_type, c.k, c.v, c.n_pages, page, c.page_stride, nkv, hd, dev(table), table.shape[1], start,
                       ints(b for _, b in seqs), len(seqs), xd, stride, total, nq, half,
                       None if qg is None else dev(qg), None if kg is None else dev(kg), 1e-6,
                       dev(cos) if half else None, dev(sin) if half else None, rope_rows if half else 0, out,
                       stride if in_place else nq * hd, ws)
    got = host(out)[:, :nq * hd]
    if in_place:
        assert np.array_equal(host(out)[:, nq * hd:], x[:, nq * hd:])
    K, V = np.zeros((n, nkv, hd)), x[:n, (nq + nkv) * hd:width].reshape(n, nkv, hd)
    kept, r = [], 0
    for a, b in seqs:
        for i in range(a):
            t = b - a + i
            if t < 0 or (half and t >= rope_rows):
                want = x[r, :nq * hd] if in_place else np.full(nq * hd, 77.0)
                assert np.array_equal(got[r], want), (r, t)
                kept.append((0, 0))
            else:
                cs, sn = (cos[t], sin[t]) if half else (np.zeros(0),) * 2
                cs, sn = cs.astype(np.float64), sn.astype(np.float64)
                ref = _turn64(x[r, :nq * hd].reshape(nq, hd), qg, 1e-6, cs, sn)
                K[r] = _turn64(x[r, nq * hd:(nq + nkv) * hd].reshape(nkv, hd), kg, 1e-6, cs, sn)
                # f32: the sum of hd squares, its root and quotient, two products, the rotation's two terms
                size = np.abs(ref)
                if half:
                    big = np.hypot(ref[:, :half], ref[:, half:2 * half])
                    size[:, :half] = size[:, half:2 * half] = 1.5 * big
                err = np.abs(got[r].reshape(nq, hd) - ref)
                assert (err <= (hd / 2 + 8) * 2.0 ** -24 * size + 1e-38).all(), (r, t, float((err / size).max()))
                kept.append((1, t + 1))
            r += 1
    assert np.array_equal(got[n:], x[n:, :nq * hd] if in_place else np.full((total - n, nq * hd), 77.0))
    # each row on its own, so that rows left out are left out
    rows = [(a, b) for a, b in kept]
    seq_of = [s for s, (a, _) in enumerate(seqs) for _ in range(a)]
    want = _expect(before, c, [(1, b) if a else (1, 0) for a, b in rows], table[seq_of] if rows else table, K, V, nkv)
    near = _near(K[[i for i, (a, _) in enumerate(rows) if a]], kv_type, hd).any() if n else False
    assert not near, "the case's inputs decide nothing"
    _same(_pool(c.k), want[0], c, "K")
    _same(_pool(c.v), want[1], c, "V")
    late = half and any(b > rope_rows and a > 0 for a, b in seqs)
    assert q.qgemv_attn_error(ws) == (1 if late else 0)


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("nq,nkv,hd,page,half", [(12, 2, 128, 16, 64), (3, 1, 64, 32, 16), (6, 3, 96, 64, 48),
                                                 (4, 2, 192, 128, 7), (2, 1, 256, 256, 128), (5, 5, 64, 16, 0)])
def test_qkv_append(kv_type, nq, nkv, hd, page, half):
    _qkv(kv_type, nq, nkv, hd, page, SEQS, half, seed=hd)
    _qkv(kv_type, nq, nkv, hd, page, [(1, n) for n in (1, 16, 17, 32, 200, 33, 0, -1)], half, seed=hd, decode=True)


@pytest.mark.parametrize("kv_type", ALL)
def test_qkv_append_in_place_without_norms_and_beyond_the_tables(kv_type):
    _qkv(kv_type, 4, 2, 128, 16, SEQS, 64, seed=1, in_place=True)
    _qkv(kv_type, 4, 2, 64, 16, SEQS, 13, seed=2, in_place=True)
    _qkv(kv_type, 4, 2, 64, 32, SEQS, 32, seed=3, norm=False)
    _qkv(kv_type, 4, 2, 64, 32, SEQS, 20, seed=4, rope_rows=37)
    _qkv(kv_type, 2, 1, 64, 16, [(1, 5), (1, 9), (1, 30)], 20, seed=5, rope_rows=9, decode=True)
    rng = np.random.default_rng(6)
    _qkv(kv_type, 2, 1, 64, 16, [(int(a), int(a + c)) for a, c in zip(rng.integers(0, 4, 300), rng.integers(0, 40, 300))],
         32, seed=7)


def test_qkv_append_is_norm_rope_and_append():
    """Against the two calls that it takes the place of, f16: at most one rounding apart."""
    nq, nkv, hd, page, nb = 12, 2, 128, 16, 7
    rng = np.random.default_rng(8)
    width = (nq + 2 * nkv) * hd
    x = rng.standard_normal((nb, width)).astype(np.float32)
    lens = [1, 5, 16, 17, 40, 3, 30]
    cos, sin = (rng.uniform(-1, 1, (40, 64)).astype(np.float32) for _ in range(2))
    g1, g2 = (dev(rng.uniform(0.5, 1.5, hd).astype(np.float32)) for _ in range(2))
    table = dev(np.arange(7 * 3, dtype=np.int32).reshape(7, 3))
    pools = [D.kv_pages(q.F16, 21, page, nkv, hd) for _ in range(2)]
    for p in pools:
        for t in p:
            t.zero_()
    ws = D.attn_workspace(q.OP_QKV_APPEND, nb, nq, nkv, hd)
    stride = nkv * page * hd
    a, b = dev(x), dev(x)
    at = [n - 1 for n in lens]
    q.qgemv_qk_norm_rope(a, nb, nq, nkv, hd, 64, g1, g2, 1e-6, dev(cos[at]), dev(sin[at]))
    q.qgemv_kv_append(q.F16, *pools[0], 21, page, stride, nkv, hd, table, 3, None, ints(lens), nb, a[:, nq * hd:],
                      a[:, (nq + nkv) * hd:], width, nb, ws)
    q.qgemv_qkv_append(q.F16, *pools[1], 21, page, stride, nkv, hd, table, 3, None, ints(lens), nb, b, width, nb, nq,
                       64, g1, g2, 1e-6, dev(cos), dev(sin), 40, b, width, ws)
    ha, hb = host(a)[:, :nq * hd], host(b)[:, :nq * hd]
    assert np.abs(ha - hb).max() <= 2 * (hd / 2 + 8) * 2.0 ** -24 * 1.5 * np.sqrt(2) * np.abs(ha).max()
    assert torch.equal(pools[0][1], pools[1][1])
    k0, k1 = host(pools[0][0]).astype(np.float64), host(pools[1][0]).astype(np.float64)
    assert np.abs(k0 - k1).max() <= 2.0 ** -10 * np.abs(k0).max() and (k0 != k1).mean() < 1e-3


# ------------------------------------------------------------------------------------- attention

def _draw(rng, lens, nkv, hd, spread=1.0):
    out = []
    for _ in range(2):
        out.append([(rng.standard_normal((max(0, n), nkv, hd)) * np.exp(spread * 0.4 * rng.standard_normal(
            (max(0, n), nkv, 1)))).astype(np.float32) for n in lens])
    return out


def attend(kv_type, nq, nkv, hd, page, seqs, seed=0, prompt=True, scale=None, qmul=1.0, extra_entries=2, tail=0,
           gap=0, bad_entry=-1, spread=1.0, K=None, V=None, ws=None):
    """seqs: (new rows, cached positions with them); not prompt: one row each by qgemv_attn."""
    say(f"attend type={kv_type} nq={nq} nkv={nkv} hd={hd} page={page} prompt={prompt} seqs={seqs[:6]}")
    rng = np.random.default_rng([92, seed])
    scale = hd ** -0.5 if scale is None else scale
    lens = [max(0, b) for _, b in seqs]
    if K is None:
        K, V = _draw(rng, lens, nkv, hd, spread)
    c = Cache(kv_type, K, V, page, nkv, hd, rng, extra_entries=extra_entries, gap=gap, bad_entry=bad_entry)
    kv = ints(b for _, b in seqs)
    start = np.concatenate([[0], np.cumsum([a for a, _ in seqs])])
    rows = int(start[-1]) + tail
    width = (nq + 2 * nkv) * hd
    x = (rng.standard_normal((rows, width)) * qmul).astype(np.float32)
    o = torch.full((rows, nq * hd), 123.5, device="cuda")
    op = q.OP_ATTN_PROMPT if prompt else q.OP_ATTN
    ws = D.attn_workspace(op, len(seqs), nq, nkv, hd) if ws is None else ws
    if prompt:
        q.qgemv_attn_prompt(*c.args(), ints(start), kv, len(seqs), dev(x), width, rows, nq, scale, o, ws)
    else:
        q.qgemv_attn(*c.args(), kv, len(seqs), dev(x), width, nq, scale, o, ws)
    got = host(o)
    assert (got[start[-1]:] == 123.5).all()
    parts, seen = [], []
    for b, (a, n) in enumerate(seqs):
        hk, hv = held(K[b], kv_type), held(V[b], kv_type)
        dv = scales64(V[b], kv_type) if kv_type in BYTES and len(V[b]) else np.ones(V[b].shape[:2])
        for i in range(a):
            last = n - a + i
            parts.append(parts64(x[start[b] + i, :nq * hd].reshape(nq, hd), hk, hv, dv, nkv, scale, last, kv_type))
            seen.append(max(0, last + 1))
    if parts:
        check_rows(got[:start[-1]], parts, seen, hd, kv_type, "attention")
    assert q.qgemv_attn_error(ws) == 0


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 128, 130, 257, 255, 256]


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("nq,nkv,hd,page", [(12, 2, 128, 16), (8, 8, 64, 32), (5, 1, 96, 16), (20, 1, 64, 64),
                                            (40, 2, 128, 128), (4, 2, 256, 16), (6, 3, 192, 256)])
def test_attn8_small_lengths(kv_type, nq, nkv, hd, page):
    attend(kv_type, nq, nkv, hd, page, [(1, n) for n in LENS], hd + page, prompt=False)


@pytest.mark.parametrize("kv_type,nq,nkv,hd,page,lens", [
    (q.I8, 12, 2, 128, 16, [5000]),
    (q.F8, 12, 2, 128, 16, [4097, 1, 0, 700]),
    (q.F8, 8, 4, 64, 64, [1500] * 9),
    (q.I8, 17, 1, 96, 32, [3001, 2]),
    (q.I8, 2, 2, 256, 128, [2049, 2047]),
    (q.F8, 3, 1, 192, 256, [20001]),
    (q.F8, 40, 2, 128, 16, [9000, 100, 3000]),
])
def test_attn8_long(kv_type, nq, nkv, hd, page, lens):
    attend(kv_type, nq, nkv, hd, page, [(1, n) for n in lens], len(lens), prompt=False)


def test_attn8_many_sequences():
    rng = np.random.default_rng(3)
    attend(q.F8, 4, 2, 64, 16, [(1, int(v)) for v in rng.integers(0, 40, 1024)], 5, prompt=False)
    lens = [int(v) for v in rng.integers(0, 60, 150)]
    lens[3], lens[90], lens[149] = 9000, 1300, 700
    attend(q.I8, 4, 1, 64, 16, [(1, n) for n in lens], 6, prompt=False)
    lens = [int(n) for n in rng.integers(1, 200, 66)]
    lens[0], lens[65], lens[7] = 6000, 1500, 0
    attend(q.I8, 8, 8, 64, 16, [(1, n) for n in lens], 7, prompt=False)


PROMPTS = [(1, 1), (2, 2), (0, 0), (7, 7), (31, 31), (33, 40), (1, 66), (5, 130), (0, 9), (64, 64), (5, 2), (3, 0),
           (2, -3)]


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("nq,nkv,hd,page", [(12, 2, 128, 16), (8, 8, 64, 32), (5, 1, 96, 16), (20, 1, 64, 64),
                                            (4, 2, 256, 16), (6, 3, 192, 256)])
def test_prompt8_small(kv_type, nq, nkv, hd, page):
    attend(kv_type, nq, nkv, hd, page, PROMPTS, hd + page, tail=3)


def in_16s(n_rows, n_seq, nq, nkv, hd, positions):
    """Whether 16-column tiles take a prompt over 8-bit pages (the launcher's own choice)."""
    fn = ctypes.CDLL(q.LIB_PATH)["_ZN2qg14prompt8_in_16sEliiiil"]
    fn.restype = ctypes.c_bool
    fn.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64]
    return fn(n_rows, n_seq, nq, nkv, hd, positions)


def _wide(kv_type, nq, nkv, hd, page, seqs, seed, entries, **kw):
    """By 128-row tiles: a table of so many positions that the smaller ones do not take the call."""
    rows = sum(a for a, _ in seqs) + kw.get("tail", 0)
    positions = (max(-(-b // page) for _, b in seqs) + entries) * page
    assert not in_16s(rows, len(seqs), nq, nkv, hd, positions)
    attend(kv_type, nq, nkv, hd, page, seqs, seed, extra_entries=entries, **kw)


def test_choice_of_tiles():
    assert in_16s(32, 1, 12, 2, 128, 20000) and in_16s(128, 1, 12, 2, 128, 4160) and in_16s(128, 1, 32, 8, 128, 4160)
    assert not in_16s(203, 1, 12, 2, 128, 30240) and not in_16s(8192, 1, 32, 8, 128, 8320)
    assert not in_16s(1200, 2, 8, 8, 64, 632) and not in_16s(1 << 20, 1024, 1024, 1, 256, 1 << 24)


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("nq,nkv,hd,page", [(12, 2, 128, 16), (10, 2, 64, 32), (5, 1, 96, 16), (20, 1, 64, 256),
                                            (4, 1, 256, 16), (6, 1, 192, 64)])
def test_prompt8_wide(kv_type, nq, nkv, hd, page):
    g = nq // nkv
    seqs = [(2100 // g, 2100 // g), (1, 1), (0, 0), (0, 9), (700 // g, 700 // g + 77), (3, 130), (30, 21)]
    _wide(kv_type, nq, nkv, hd, page, seqs, hd + page, 16384 // page, tail=3)


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("nq,nkv,hd,seqs", [(8, 8, 64, [(600, 600), (600, 611), (3, 2)]), (16, 8, 128, [(600, 900)]),
                                            (8, 8, 256, [(300, 301), (300, 300)]), (12, 12, 96, [(700, 700)])])
def test_prompt8_wide_unsplit(kv_type, nq, nkv, hd, seqs):
    """More tiles than are resident at once, over short tables: none is split."""
    _wide(kv_type, nq, nkv, hd, 32, seqs, hd, 2, tail=1)


@pytest.mark.parametrize("kv_type,nq,nkv,hd,page,seqs", [
    (q.I8, 32, 1, 128, 16, [(61, 5000)]), (q.F8, 48, 2, 64, 16, [(50, 4000), (50, 64)]),
    (q.I8, 8, 1, 256, 32, [(100, 2500)]), (q.F8, 36, 1, 96, 16, [(45, 3333)]), (q.F8, 12, 1, 192, 16, [(80, 2100)]),
    (q.I8, 64, 4, 64, 32, [(40, 6000), (300, 300), (250, 250), (0, 5000), (400, 420), (9, 3000), (330, 330), (100, 100)]),
    (q.F8, 64, 4, 128, 32, [(10, 2600), (300, 300), (250, 250), (400, 420), (330, 330), (100, 100)]),
    (q.F8, 64, 4, 256, 32, [(10, 2600), (300, 300), (250, 250), (12, 5)]),
])
def test_prompt8_long(kv_type, nq, nkv, hd, page, seqs):
    """Tiles split over the cache's length, all of them or a few among many."""
    _wide(kv_type, nq, nkv, hd, page, seqs, len(seqs), 16384 // page, tail=1)


@pytest.mark.parametrize("kv_type", BYTES)
def test_prompt8_long_by_16_columns(kv_type):
    assert in_16s(120, 1, 8, 1, 128, 9032)
    attend(kv_type, 8, 1, 128, 16, [(120, 9000)], 3, tail=1)
    attend(kv_type, 24, 2, 64, 16, [(17, 5000), (2, 3000)], 4)


@pytest.mark.parametrize("kv_type", BYTES)
def test_attention8_scales_and_sharp_scores(kv_type):
    for prompt, seqs in ((False, [(1, 300), (1, 77)]), (True, [(110, 300), (100, 131)]), (True, [(310, 350), (300, 331)])):
        kw = dict(prompt=prompt, extra_entries=1024 if prompt else 2)
        assert not prompt or in_16s(sum(a for a, _ in seqs), 2, 4, 1, 64, 17000) == (seqs[0][0] < 200)
        attend(kv_type, 4, 1, 128, 16, seqs, 1, scale=1.0, qmul=2.0, **kw)
        attend(kv_type, 4, 1, 64, 16, seqs, 2, scale=-0.09, **kw)
        attend(kv_type, 4, 1, 64, 16, seqs, 3, scale=0.0, **kw)
        attend(kv_type, 4, 1, 64, 16, seqs, 4, scale=1e-6, qmul=1e6, **kw)
        attend(kv_type, 4, 1, 64, 16, seqs, 5, scale=1e6, qmul=1e-6, **kw)
        attend(kv_type, 4, 1, 64, 16, seqs, 6, gap=32, bad_entry=2 ** 30, **kw)
        attend(kv_type, 4, 1, 64, 16, seqs, 7, spread=4.0, **kw)           # scales from 1/50 to 50


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e18, 1e30, 3e38])
def test_attention8_values_near_the_range_ends(kv_type, size):
    """V of any size (the scale is an f32), with rows of zeros among it; K large and small against the scale."""
    rng = np.random.default_rng(11)
    for prompt, seqs in ((False, [(1, 300), (1, 77)]), (True, [(110, 300), (100, 131)]), (True, [(310, 350), (300, 331)])):
        K, V = _draw(rng, [b for _, b in seqs], 1, 64, 0.0)
        for v in V:
            v /= np.abs(v).max()
            v *= np.float32(size)
            v[::7] = 0.0
        kw = dict(prompt=prompt, extra_entries=1024 if prompt else 2)
        attend(kv_type, 4, 1, 64, 16, seqs, 1, K=K, V=V, **kw)
        if 1e-20 < size < 1e20:
            attend(kv_type, 4, 1, 64, 16, seqs, 1, K=[k * np.float32(size) for k in K], V=V, scale=0.1 / size, **kw)


@pytest.mark.parametrize("kv_type", BYTES)
def test_a_large_value_reaches_only_the_rows_that_see_it(kv_type):
    """V a million times larger at later positions: earlier rows of the tile keep their precision."""
    rng = np.random.default_rng(12)
    for seqs in ([(40, 40)], [(300, 300)], [(130, 800)], [(700, 800)]):
        n = seqs[0][1]
        K, V = _draw(rng, [n], 1, 64, 0.0)
        V[0][n - 5:] *= np.float32(1e9)
        attend(kv_type, 4, 1, 64, 16, seqs, 1, K=K, V=V, extra_entries=1024)


@pytest.mark.parametrize("kv_type", BYTES)
@pytest.mark.parametrize("where", ["k", "v"])
def test_non_finite_rows_reach_only_the_rows_that_see_them(kv_type, where):
    """A position quantised from a NaN or an infinity: rows and heads that see it are not finite, others exact."""
    rng = np.random.default_rng(13)
    nq, nkv, hd, page = 4, 2, 64, 16
    for seqs in ([(50, 50), (20, 90)], [(600, 600), (200, 777)]):
        K, V = _draw(rng, [b for _, b in seqs], nkv, hd)
        spoilt = (K if where == "k" else V)[0]
        at = seqs[0][1] - 20
        spoilt[at, 1, 3] = np.nan if where == "k" else np.inf
        c = Cache(kv_type, K, V, page, nkv, hd, rng, extra_entries=1024)
        start = np.concatenate([[0], np.cumsum([a for a, _ in seqs])])
        rows = int(start[-1])
        x = rng.standard_normal((rows, nq * hd)).astype(np.float32)
        o = torch.empty((rows, nq * hd), device="cuda")
        ws = D.attn_workspace(q.OP_ATTN_PROMPT, len(seqs), nq, nkv, hd)
        q.qgemv_attn_prompt(*c.args(), ints(start), c.kv_len, len(seqs), dev(x), nq * hd, rows, nq, 0.125, o, ws)
        got = host(o).reshape(rows, nq, hd)
        clean = [np.where(np.isfinite(a), a, 0) for a in (K[0], V[0])]
        for i in range(seqs[0][0]):
            last = seqs[0][1] - seqs[0][0] + i
            sees = last >= at
            assert np.isnan(got[i, 2:]).all() == sees and np.isfinite(got[i, :2]).all()
            if not sees or i % 16 == 0:
                o64, A, _, _ = parts64(x[i].reshape(nq, hd), held(clean[0], kv_type), held(clean[1], kv_type),
                                       scales64(clean[1], kv_type), nkv, 0.125, last, kv_type)
                good = slice(None) if not sees else slice(0, 2)
                assert (np.abs(got[i, good] - o64[good]) <= 1e-4 * A[good] + 1e-9).all()
        assert np.isfinite(got[start[1]:]).all()
        one = torch.empty((2, nq * hd), device="cuda")
        wa = D.attn_workspace(q.OP_ATTN, 2, nq, nkv, hd)
        q.qgemv_attn(*c.args(), c.kv_len, 2, dev(x[:2]), nq * hd, nq, 0.125, one, wa)
        g1 = host(one).reshape(2, nq, hd)
        assert np.isnan(g1[0, 2:]).all() and np.isfinite(g1[0, :2]).all() and np.isfinite(g1[1]).all()


@pytest.mark.parametrize("kv_type", BYTES)
def test_attention8_bad_pages_are_left_out(kv_type):
    hd, nkv, nq, page = 64, 2, 4, 16
    rng = np.random.default_rng(14)
    K, V = _draw(rng, [100, 50, 64], nkv, hd)
    c = Cache(kv_type, K, V, page, nkv, hd, rng, extra_entries=0, spare=0)
    c.table[0, 2] = c.n_pages
    c.table[1, 0] = -7
    lens = [100, 50, 10 ** 6]
    c.table[2, 4:] = -1
    x = rng.standard_normal((3, nq * hd)).astype(np.float32)
    keep = [np.r_[0:32, 48:100], np.r_[16:50], np.r_[0:64]]
    parts = []
    for b in range(3):
        k, v = K[b][keep[b]], V[b][keep[b]]
        parts.append(parts64(x[b].reshape(nq, hd), held(k, kv_type), held(v, kv_type), scales64(v, kv_type), nkv, 0.125,
                            len(k) - 1, kv_type))
    for prompt in (False, True):
        o = torch.full((3, nq * hd), float("nan"), device="cuda")
        ws = D.attn_workspace(q.OP_ATTN_PROMPT if prompt else q.OP_ATTN, 3, nq, nkv, hd)
        if prompt:
            q.qgemv_attn_prompt(*c.args(), ints(range(4)), ints(lens), 3, dev(x), nq * hd, 3, nq, 0.125, o, ws)
        else:
            q.qgemv_attn(*c.args(), ints(lens), 3, dev(x), nq * hd, nq, 0.125, o, ws)
        check_rows(host(o), parts, [100, 50, 64], hd, kv_type, "bad pages")
        assert q.qgemv_attn_error(ws) == 1
        assert q.qgemv_attn_error(ws) == 0


@pytest.mark.parametrize("kv_type", BYTES)
def test_pages_beyond_32_bits(kv_type):
    """Pages more than 2^32 bytes into the pool: append, both attentions."""
    hd, nkv, page, nq, n = 128, 1, 16, 4, 40
    stride = 3 << 30
    rng = np.random.default_rng(15)
    pools = [torch.zeros(2 * stride + page * (hd + 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = ints([2, 0, 1])
    rows = rng.standard_normal((n, 2 * hd)).astype(np.float32)
    rd = dev(rows)
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, 1, nq, nkv, hd)
    q.qgemv_kv_append(kv_type, *pools, 3, page, stride, nkv, hd, table, 3, ints([0, n]), ints([n]), 1, rd, rd[:, hd:],
                      2 * hd, n, ws)
    K, V = rows[:, None, :hd], rows[:, None, hd:]
    x = rng.standard_normal((1, nq * hd)).astype(np.float32)
    part = parts64(x.reshape(nq, hd), held(K, kv_type), held(V, kv_type), scales64(V, kv_type), 1, 0.1, n - 1, kv_type)
    for prompt in (False, True):
        o = torch.empty((1, nq * hd), device="cuda")
        if prompt:
            q.qgemv_attn_prompt(kv_type, *pools, 3, page, stride, nkv, hd, table, 3, ints([0, 1]), ints([n]), 1, dev(x),
                                nq * hd, 1, nq, 0.1, o, ws)
        else:
            q.qgemv_attn(kv_type, *pools, 3, page, stride, nkv, hd, table, 3, ints([n]), 1, dev(x), nq * hd, nq, 0.1, o, ws)
        check_rows(host(o), [part], [n], hd, kv_type, "far pages")
