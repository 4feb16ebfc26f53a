"""Host-side checks of the attention-side entry points (no GPU): workspace sizes and refusals, all
made before any HIP call."""
import pytest

import dequant_gemv_q4_amd as q

K, V, T, L, S, X, O, W = (0x7f0000000000 + (i << 36) for i in range(8))   # never touched


@pytest.fixture(scope="module")
def lib():
    return q.lib()


CACHE = dict(kv_type=q.F16, k_pages=K, v_pages=V, n_pages=100, page_size=16, page_stride=2 * 16 * 128,
             nkv=2, hd=128, table=T, max_pages=40)
ATTN = dict(CACHE, kv_len=L, n_seq=3, q=X, q_stride=2048, nq=12, scale=0.1, o=O, ws=W, ws_bytes=1 << 30,
            stream=None)
PROMPT = dict(CACHE, q_start=S, kv_len=L, n_seq=3, q=X, q_stride=2048, n_rows=50, nq=12, scale=0.1, o=O,
              ws=W, ws_bytes=1 << 30, stream=None)
APPEND = dict(CACHE, q_start=S, kv_len=L, n_seq=3, k=X, v=X + 1024, kv_stride=2048, n_rows=50, ws=W,
              ws_bytes=1 << 30, stream=None)
ROUTE = dict(logits=X, n_rows=16, n_exp=64, score=0, bias=None, n_group=1, group_top=1, topk_group=1, topk=8,
             renorm=1, scale=1.0, ids=O, wts=O + 65536, stream=None)


def _calls(lib):
    return [(lib.qgemv_attn, ATTN), (lib.qgemv_attn_prompt, PROMPT), (lib.qgemv_kv_append, APPEND)]


def _st(fn, base, **kw):
    assert set(kw) <= set(base)
    return fn(*dict(base, **kw).values())


@pytest.mark.parametrize("change,status", [
    (dict(kv_type=0), 2), (dict(kv_type=q.Q8_0), 2),
    (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(table=None), 1), (dict(kv_len=None), 1),
    (dict(page_size=8), 3), (dict(page_size=24), 3), (dict(page_size=512), 3), (dict(page_size=0), 3),
    (dict(hd=80), 3), (dict(hd=32), 3), (dict(hd=0), 3), (dict(hd=512), 3),
    (dict(nkv=0), 3), (dict(nkv=-1), 3), (dict(n_seq=0), 3), (dict(n_seq=1025), 3),
    (dict(n_pages=0), 3), (dict(n_pages=1 << 29), 3), (dict(max_pages=0), 3),
    (dict(max_pages=(1 << 26) + 1), 3),
    (dict(page_stride=2 * 16 * 128 - 8), 3), (dict(page_stride=2 * 16 * 128 + 4), 3),
    (dict(page_stride=1 << 33), 3),
    (dict(k_pages=K + 8), 4), (dict(v_pages=V + 2), 4), (dict(table=T + 2), 4), (dict(kv_len=L + 1), 4),
    (dict(ws=None), 5), (dict(ws_bytes=255), 5), (dict(ws=W + 128), 4),
    (dict(ws=K), 7), (dict(ws=V), 7), (dict(ws=T), 7), (dict(ws=L), 7), (dict(ws=X), 7),
])
def test_cache_refusals(lib, change, status):
    for fn, base in _calls(lib):
        assert _st(fn, base, **change) == status, fn


def test_attention_refusals(lib):
    for fn, base in _calls(lib)[:2]:
        assert _st(fn, base, q=None) == 1 and _st(fn, base, o=None) == 1
        assert _st(fn, base, nq=0) == 3 and _st(fn, base, nq=3) == 3 and _st(fn, base, nq=8192) == 3
        assert _st(fn, base, q_stride=12 * 128 - 4) == 3
        assert _st(fn, base, scale=float("nan")) == 3 and _st(fn, base, scale=float("inf")) == 3
        assert _st(fn, base, q=X + 4) == 4 and _st(fn, base, o=O + 8) == 4 and _st(fn, base, q_stride=2050) == 4
        assert _st(fn, base, o=X) == 7 and _st(fn, base, o=K) == 7 and _st(fn, base, o=V + 4096) == 7
        assert _st(fn, base, o=W) == 7 and _st(fn, base, o=T) == 7 and _st(fn, base, o=L) == 7
    assert _st(lib.qgemv_attn_prompt, PROMPT, q_start=None) == 1
    assert _st(lib.qgemv_attn_prompt, PROMPT, q_start=S + 2) == 4
    assert _st(lib.qgemv_attn_prompt, PROMPT, o=S) == 7 and _st(lib.qgemv_attn_prompt, PROMPT, ws=S) == 7
    assert _st(lib.qgemv_attn_prompt, PROMPT, n_rows=0) == 3
    assert _st(lib.qgemv_attn_prompt, PROMPT, n_rows=(1 << 20) + 1) == 3


def test_append_refusals(lib):
    fn = lib.qgemv_kv_append
    assert _st(fn, APPEND, k=None) == 1 and _st(fn, APPEND, v=None) == 1
    assert _st(fn, APPEND, kv_stride=252) == 3 and _st(fn, APPEND, n_rows=0) == 3
    assert _st(fn, APPEND, q_start=None) == 3                 # one row per sequence: n_rows = n_seq
    assert _st(fn, APPEND, k=X + 4) == 4 and _st(fn, APPEND, v=X + 4) == 4 and _st(fn, APPEND, kv_stride=2050) == 4
    assert _st(fn, APPEND, k=K) == 7 and _st(fn, APPEND, v=V) == 7
    assert _st(fn, APPEND, v_pages=K) == 7                    # K and V in the same place
    assert _st(fn, APPEND, v_pages=K + 4096) == 7             # blocks of 8192 bytes that overlap
    assert _st(fn, APPEND, v_pages=K + 3 * 8192) == 7         # the next pages' blocks


def test_workspace_sizes():
    for op in (q.OP_KV_APPEND, q.OP_ATTN, q.OP_ATTN_PROMPT):
        assert q.qgemv_attn_workspace_bytes(op, 16, 12, 2, 128) >= 256
        assert q.qgemv_attn_workspace_bytes(op, 0, 12, 2, 128) == -1
        assert q.qgemv_attn_workspace_bytes(op, 1025, 12, 2, 128) == -1
        assert q.qgemv_attn_workspace_bytes(op, 16, 12, 5, 128) == -1
        assert q.qgemv_attn_workspace_bytes(op, 16, 12, 0, 128) == -1
        assert q.qgemv_attn_workspace_bytes(op, 16, 12, 2, 100) == -1
    assert q.qgemv_attn_workspace_bytes(q.OP_MOE, 16, 12, 2, 128) == -1


def test_error_query_refusals(lib):
    assert lib.qgemv_attn_error(None, None, None) == 1
    assert lib.qgemv_attn_error(W, None, None) == 1


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), 1), (dict(ids=None), 1), (dict(wts=None), 1),
    (dict(n_rows=0), 3), (dict(n_rows=(1 << 20) + 1), 3), (dict(n_exp=0), 3), (dict(n_exp=1025), 3),
    (dict(score=2), 3), (dict(score=-1), 3), (dict(n_group=0), 3), (dict(n_group=5), 3), (dict(n_group=128), 3),
    (dict(group_top=0), 3), (dict(group_top=3), 3), (dict(n_group=64, group_top=2), 3),
    (dict(n_group=8, topk_group=9), 3), (dict(topk_group=0), 3), (dict(topk=0), 3), (dict(topk=9), 3),
    (dict(n_group=32, topk_group=3), 3), (dict(n_exp=7), 3), (dict(scale=float("nan")), 3),
    (dict(logits=X + 2), 4), (dict(bias=X + 1), 4), (dict(ids=O + 2), 4), (dict(wts=O + 65537), 4),
    (dict(ids=X), 7), (dict(wts=X), 7), (dict(wts=O + 4), 7), (dict(bias=O), 7),
])
def test_route_refusals(lib, change, status):
    assert _st(lib.qgemv_route, ROUTE, **change) == status
