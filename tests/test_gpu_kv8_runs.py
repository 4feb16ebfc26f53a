"""The 8-bit cache, the fused QKV append and shared prefixes as programs run them: repeated and captured calls,
several on one workspace or on streams of their own, refusals of the binding, and a layer's prefill and decode
steps through all of them."""
import numpy as np
import pytest

from gpu_common import assert_within, dev, gpu_matrix, host, require_gpu, say, tol_gemv, torch

import dequant_gemv_q4_amd as q
from dequant_gemv_q4_amd import device as D
from kv_common import ALL, BYTES, Cache, check_rows, held, parts64, scales64
from test_gpu_kv8 import _draw, _empty, _pool, _turn64, ints
import oracle
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    oracle.build(force=False)


class Job:
    """One call over a cache of its own: op 'attn', 'prompt' or 'shared' (groups: (first sequences, shares))."""

    def __init__(self, op, kv_type, nq, nkv, hd, seqs, seed, groups=None, extra=2):
        rng = np.random.default_rng([94, seed])
        lens = [b for _, b in seqs]
        K, V = _draw(rng, lens, nkv, hd)
        tables = {}
        if groups:
            for a, b in zip(groups[0], groups[0][1:]):
                for i in range(a + 1, b):
                    s = groups[1][i]
                    K[i][:s], V[i][:s] = K[a][:s], V[a][:s]
                    tables.update({(i, e): (a, e) for e in range(s // 16)})
        self.c = Cache(kv_type, K, V, 16, nkv, hd, rng, extra_entries=extra, tables=tables)
        self.op, self.nq, self.n = op, nq, len(seqs)
        self.start = ints(np.concatenate([[0], np.cumsum([a for a, _ in seqs])]))
        self.rows = sum(a for a, _ in seqs)
        self.q = dev(rng.standard_normal((self.rows, nq * hd)).astype(np.float32))
        self.groups = groups and (ints(groups[0]), ints(groups[1]), len(groups[0]) - 1)
        self.o = torch.full((self.rows, nq * hd), float("nan"), device="cuda")

    def workspace(self):
        op = {"attn": q.OP_ATTN, "prompt": q.OP_ATTN_PROMPT, "shared": q.OP_ATTN_SHARED}[self.op]
        return D.attn_workspace(op, self.n, self.nq, self.c.nkv, self.c.hd)

    def run(self, ws, stream=None):
        c, width = self.c, self.nq * self.c.hd
        if self.op == "attn":
            q.qgemv_attn(*c.args(), c.kv_len, self.n, self.q, width, self.nq, 0.09, self.o, ws, stream=stream)
        elif self.op == "prompt":
            q.qgemv_attn_prompt(*c.args(), self.start, c.kv_len, self.n, self.q, width, self.rows, self.nq, 0.09,
                                self.o, ws, stream=stream)
        else:
            q.qgemv_attn_shared(*c.args(), c.kv_len, self.n, *self.groups, self.q, width, self.nq, 0.09, self.o, ws,
                                stream=stream)

    def fresh(self, ws):
        self.o.fill_(float("nan"))
        self.run(ws)
        return host(self.o).copy()


def _jobs():
    return [
        Job("attn", q.I8, 12, 2, 128, [(1, 9000), (1, 17), (1, 2500), (1, 0)], 1),
        Job("prompt", q.F8, 12, 2, 128, [(3, 6000), (2, 900)], 2),
        Job("prompt", q.I8, 24, 2, 64, [(200, 3000), (40, 70)], 3, extra=1024),
        Job("shared", q.F16, 24, 8, 64, [(1, 700 + i) for i in range(9)], 4, ([0, 4, 9], [640] * 4 + [333] * 5)),
        Job("shared", q.F8, 12, 2, 128, [(1, 3000 + i) for i in range(20)], 5, ([0, 20], [2990] * 20)),
        Job("shared", q.BF16, 64, 1, 64, [(1, 1300 + i % 7) for i in range(130)], 6, ([0, 130], [1299] * 130)),
        Job("shared", q.I8, 64, 16, 64, [(1, 40 + i % 50) for i in range(130)], 7, (list(range(0, 131, 2)), [33] * 130)),
        Job("attn", q.F8, 8, 8, 64, [(1, 100)] * 70, 8),
    ]


def test_repeated_calls_are_bitwise_identical():
    for job in _jobs():
        ws = job.workspace()
        ref = job.fresh(ws)
        assert np.isfinite(ref).all()
        for _ in range(12):
            assert np.array_equal(job.fresh(ws), ref), job.op


def test_operations_share_a_workspace():
    """One workspace, as large as the largest needs: calls of different kinds and sizes one after the other."""
    jobs = _jobs()
    refs = [j.fresh(j.workspace()) for j in jobs]
    size = max(j.workspace().numel() for j in jobs)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for rep in range(3):
        for j, ref in zip(jobs if rep % 2 == 0 else jobs[::-1], refs if rep % 2 == 0 else refs[::-1]):
            assert np.array_equal(j.fresh(ws), ref), (rep, j.op)
        for j in jobs:                                     # without a wait between
            j.run(ws)
        for j, ref in zip(jobs, refs):
            assert np.array_equal(host(j.o), ref), (rep, j.op)
    assert q.qgemv_attn_error(ws) == 0


def test_streams_with_workspaces_of_their_own():
    jobs = _jobs()[:6]
    wss = [j.workspace() for j in jobs]
    refs = [j.fresh(w) for j, w in zip(jobs, wss)]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(6):
        for j, w, s in zip(jobs, wss, streams):
            j.run(w, stream=s)
        torch.cuda.synchronize()
        for j, ref in zip(jobs, refs):
            assert np.array_equal(host(j.o), ref)


def test_graphs_share_a_workspace_and_follow_the_lengths():
    """Each job captured once, all on one workspace; replays with other lengths, with eager work in between, give
    the eager call's bits."""
    jobs = _jobs()[:5]
    ws = torch.zeros(max(j.workspace().numel() for j in jobs), dtype=torch.uint8, device="cuda")
    graphs = []
    for j in jobs:
        j.run(ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            j.run(ws)
        graphs.append(g)
    full = [j.c.kv_len.clone() for j in jobs]
    for rep, cut in enumerate((0, 5, 1, 100, 0)):
        for j, n in zip(jobs, full):
            j.c.kv_len.copy_((n - cut).clamp(min=0))
            j.q.normal_()
            j.o.fill_(-1)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [host(j.o).copy() for j in jobs]
        for j, a in zip(jobs, got):
            assert np.isfinite(a).all() and np.array_equal(a, j.fresh(ws)), (rep, j.op)


@pytest.mark.parametrize("kv_type", ALL)
def test_a_captured_append_follows_the_lengths(kv_type):
    nq, nkv, hd, page, n = 6, 2, 64, 16, 3
    width = (nq + 2 * nkv) * hd
    c = _empty(kv_type, 12, page, nkv, hd)
    table, kv = dev(np.arange(12, dtype=np.int32).reshape(3, 4)), ints([1, 17, 40])
    x, o = torch.randn(n, width, device="cuda"), torch.empty(n, nq * hd, device="cuda")
    cos, sin, g = torch.rand(64, 32, device="cuda"), torch.rand(64, 32, device="cuda"), torch.rand(hd, device="cuda")
    ws = D.attn_workspace(q.OP_QKV_APPEND, n, nq, nkv, hd)

    def run():
        q.qgemv_qkv_append(kv_type, c.k, c.v, 12, page, c.page_stride, nkv, hd, table, 4, None, kv, n, x, width, n, nq,
                           32, g, g, 1e-6, cos, sin, 64, o, nq * hd, ws)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep, lens in enumerate(((1, 17, 40), (2, 0, 63), (64, 33, 1), (16, 16, 16))):
        kv.copy_(torch.tensor(lens, dtype=torch.int32))
        x.normal_()
        start = [c.k.clone(), c.v.clone()]
        o.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        got = [host(o).copy(), _pool(c.k).copy(), _pool(c.v).copy()]
        c.k.copy_(start[0])
        c.v.copy_(start[1])
        o.fill_(5)
        run()
        torch.cuda.synchronize()
        for a, b in zip(got, (host(o), _pool(c.k), _pool(c.v))):
            assert np.array_equal(a, b, equal_nan=True), rep


@pytest.mark.parametrize("kv_type", ALL)
def test_qkv_append_without_norm_and_rotation_is_the_append(kv_type):
    """Bit for bit, with exact ties, zeros, infinities and NaN among the rows."""
    nq, nkv, hd, page, n = 3, 3, 96, 32, 45
    rng = np.random.default_rng(95)
    x = rng.integers(-254, 255, (n, 3, nkv, hd)).astype(np.float32) / 2
    x[..., 5] = 448.0 if kv_type == q.F8 else 127.0
    x[:20] = rng.standard_normal((20, 3, nkv, hd))
    x[7], x[8, 1:, 0, 3], x[9, 1:, 1, 9] = 0.0, np.inf, np.nan
    xd = dev(x.reshape(n, -1))
    width = 3 * nkv * hd
    table = dev(np.array([[3, 1, 2]], np.int32))
    pools = []
    for fused in (False, True):
        c = _empty(kv_type, 5, page, nkv, hd)
        ws = D.attn_workspace(q.OP_QKV_APPEND, 1, nq, nkv, hd)
        cache = (kv_type, c.k, c.v, 5, page, c.page_stride, nkv, hd, table, 3)
        if fused:
            o = torch.empty((n, nq * hd), device="cuda")
            q.qgemv_qkv_append(*cache, ints([0, n]), ints([60]), 1, xd, width, n, nq, 0, None, None, 0.0, None, None, 0,
                               o, nq * hd, ws)
            assert np.array_equal(host(o), x[:, 0].reshape(n, -1))
        else:
            q.qgemv_kv_append(*cache, ints([0, n]), ints([60]), 1, xd[:, nq * hd:], xd[:, 2 * nq * hd:], width, n, ws)
        pools.append((_pool(c.k), _pool(c.v)))
    for a, b in zip(*pools):
        if kv_type in BYTES:
            same = a == b
            assert same.all(), int((~same).sum())
        else:
            assert np.array_equal(a, b, equal_nan=True)


def test_wrong_tensors_are_refused():
    job = Job("shared", q.I8, 4, 2, 64, [(1, 40), (1, 50)], 9, ([0, 2], [32, 32]))
    c, ws = job.c, job.workspace()
    good = dict(kv_type=q.I8, k=c.k, v=c.v, n_pages=c.n_pages, page=16, stride=c.page_stride, nkv=2, hd=64, table=c.table,
                max_pages=c.max_pages, kv_len=c.kv_len, n_seq=2, start=job.groups[0], shared=job.groups[1], n_group=1,
                q=job.q, q_stride=256, nq=4, scale=0.1, o=job.o, ws=ws)

    def call(**kw):
        q.qgemv_attn_shared(*dict(good, **kw).values())

    call()
    for kw in (dict(start=job.groups[0].long()), dict(shared=job.groups[1].cpu()), dict(k=c.k.view(torch.int8)),
               dict(kv_type=q.F16), dict(o=job.o.half()), dict(q=job.q.cpu())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(q.QgemvError):
        call(n_group=3)
    with pytest.raises(q.QgemvError):
        call(ws=ws[:256])
    x = torch.randn(2, 8 * 64, device="cuda")
    t = torch.ones(64, 32, device="cuda")
    args = dict(kv_type=q.I8, k=c.k, v=c.v, n_pages=c.n_pages, page=16, stride=c.page_stride, nkv=2, hd=64, table=c.table,
                max_pages=c.max_pages, q_start=None, kv_len=c.kv_len, n_seq=2, qkv=x, qkv_stride=512, n_rows=2, nq=4,
                half=32, qg=None, kg=None, eps=1e-6, cos=t, sin=t, rope_rows=64, q=job.o, q_stride=256, ws=ws)
    q.qgemv_qkv_append(*args.values())
    for kw in (dict(qkv=x.double()), dict(cos=t.cpu()), dict(sin=t.half()), dict(q=job.o.bfloat16()),
               dict(kg=torch.ones(64)), dict(cos=torch.ones(64, 64, device="cuda")[:, ::2])):
        with pytest.raises(TypeError):
            q.qgemv_qkv_append(*dict(args, **kw).values())
    with pytest.raises(q.QgemvError):
        q.qgemv_qkv_append(*dict(args, q=x).values())


@pytest.mark.parametrize("kv_type", ALL)
def test_layer_prefill_share_and_decode(kv_type):
    """A prompt is prefilled once; three sequences share its whole pages, each with its own copy of the begun one,
    and decode two steps: QKV product, fused append, shared attention, output product.  Every step is held to its
    bound on the device's own inputs, and the caches hold what the definition gives."""
    hidden, nq, nkv, hd, page, prompt = 256, 8, 2, 64, 16, 14
    width, half, scale = (nq + 2 * nkv) * hd, hd // 2, hd ** -0.5
    g = wl.rng(2200, 1)
    Wqkv, Wo = wl.matrix(q.Q4_0, g, width, hidden), wl.matrix(q.Q4_0, g, hidden, nq * hd)
    dqkv, dwo = gpu_matrix(q.Q4_0, Wqkv, width, hidden), gpu_matrix(q.Q4_0, Wo, hidden, nq * hd)
    gamma, qg, kg = wl.gamma_f32(g, hidden), wl.gamma_f32(g, hd), wl.gamma_f32(g, hd)
    angle = np.arange(64)[:, None] / 1e4 ** (2.0 * np.arange(half)[None] / hd)
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    n_pages, max_pages = 9, 4
    kp, vp = D.kv_pages(kv_type, n_pages, page, nkv, hd)
    for t in (kp, vp):
        t.view(torch.uint8).fill_(0x7F)                    # NaN or large in every place
    tables = np.array([[5, 2, -1, -1]] * 3, np.int32)
    stride = kp.stride(0)
    ws = D.attn_workspace(q.OP_ATTN_SHARED, 3, nq, nkv, hd)
    wp = D.attn_workspace(q.OP_ATTN_PROMPT, 3, nq, nkv, hd)
    K, V = [[] for _ in range(3)], [[] for _ in range(3)]

    def step(x, n, lens, table, prefill):
        rows, seqs = len(x), len(lens)
        cache = (kv_type, kp, vp, n_pages, page, stride, nkv, hd, dev(table), max_pages)
        xd, qkv = dev(x), torch.empty((rows, width), device="cuda")
        q.qgemv_nrm(q.Q4_0, dqkv, width, hidden, xd, dev(gamma), 1e-5, rows, qkv)
        yr, A = oracle.qgemv_nrm(q.Q4_0, Wqkv, width, hidden, x, gamma, 1e-5)
        assert_within(host(qkv), yr, tol_gemv(A, yr), "qkv")
        raw = host(qkv).copy()
        qn = torch.empty((rows, nq * hd), device="cuda")
        start = ints([0, rows]) if prefill else None
        q.qgemv_qkv_append(*cache, start, ints(lens), seqs, qkv, width, rows, nq, half, dev(qg), dev(kg), 1e-6, dev(cos),
                           dev(sin), 64, qn, nq * hd, ws)
        o = torch.empty((rows, nq * hd), device="cuda")
        if prefill:
            q.qgemv_attn_prompt(*cache, start, ints(lens), 1, qn, nq * hd, rows, nq, scale, o, wp)
        else:
            q.qgemv_attn_shared(*cache, ints(lens), 3, ints([0, 3]), ints([prompt] * 3), 1, qn, nq * hd, nq, scale, o, ws)
        hq, parts, seen = host(qn), [], []
        for r in range(rows):
            b = 0 if prefill else r
            pos = r if prefill else lens[b] - 1
            c64, s64 = cos[pos].astype(np.float64), sin[pos].astype(np.float64)
            ref = _turn64(raw[r, :nq * hd].reshape(nq, hd), qg, 1e-6, c64, s64)
            assert (np.abs(hq[r].reshape(nq, hd) - ref) <= 40 * 2.0 ** -24 * 1.5 * np.abs(ref).max()).all()
            K[b].append(_turn64(raw[r, nq * hd:(nq + nkv) * hd].reshape(nkv, hd), kg, 1e-6, c64, s64))
            V[b].append(raw[r, (nq + nkv) * hd:].reshape(nkv, hd))
            dv = scales64(np.stack(V[b]), kv_type) if kv_type in BYTES else np.ones((len(V[b]), nkv))
            parts.append(parts64(hq[r].reshape(nq, hd), held(np.stack(K[b]), kv_type), held(np.stack(V[b]), kv_type), dv,
                                 nkv, scale, pos, kv_type))
            seen.append(pos + 1)
        check_rows(host(o), parts, seen, hd, kv_type, "attention")
        h = torch.empty((rows, hidden), device="cuda")
        q.qgemv_res(q.Q4_0, dwo, hidden, nq * hd, o, xd, rows, h)
        yr, A = oracle.qgemv_res(q.Q4_0, Wo, hidden, nq * hd, host(o), x)
        assert_within(host(h), yr, tol_gemv(A, yr), "output product")
        assert q.qgemv_attn_error(ws) == 0 and q.qgemv_attn_error(wp) == 0

    say(f"layer: prefill type={kv_type}")
    step(wl.normal_f32(g, (prompt, hidden)), prompt, [prompt], tables[:1], True)
    # the prompt ends inside its first page: a copy of it for each sequence
    for b, (page_id, following) in ((1, (7, 4)), (2, (0, 8))):
        for t in (kp, vp):
            t[page_id] = t[5]
        tables[b] = [page_id, following, -1, -1]
        K[b], V[b] = list(K[0]), list(V[0])
    for i in range(4):
        say(f"layer: decode step {i}")
        step(wl.normal_f32(g, (3, hidden)), 3, [prompt + i + 1] * 3, tables, False)
