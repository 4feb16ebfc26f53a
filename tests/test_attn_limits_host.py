"""The attention side's size limits as the header states them: the largest size passes the checks of sizes and
is refused for its missing workspace only, the next one for its size (no GPU: both before any HIP call)."""
import pytest

import dequant_gemv_q4_amd as q
from test_attn_host import APPEND, ATTN, PROMPT, _st

OK, SHAPE = 5, 3


def _both(names, **kw):
    lib = q.lib()
    for fn, base in ((lib.qgemv_attn, ATTN), (lib.qgemv_attn_prompt, PROMPT), (lib.qgemv_kv_append, APPEND)):
        if fn.__name__ in names:
            yield _st(fn, dict(base, ws=None), **kw)


ALL = ("qgemv_attn", "qgemv_attn_prompt", "qgemv_kv_append")
READ = ALL[:2]


@pytest.mark.parametrize("names,last,beyond", [
    (ALL, dict(n_pages=1 << 28), dict(n_pages=(1 << 28) + 1)),
    (ALL, dict(page_stride=(1 << 32) - 8), dict(page_stride=1 << 32)),
    (ALL, dict(max_pages=1 << 20), dict(max_pages=(1 << 20) + 1)),
    (READ, dict(nkv=4096, nq=4096, page_size=256, hd=256, max_pages=8, page_stride=1 << 28, q_stride=1 << 20),
     dict(nkv=4096, nq=4096, page_size=256, hd=256, max_pages=8, page_stride=(1 << 28) - 8, q_stride=1 << 20)),
    (READ, dict(nkv=1, nq=4096, q_stride=1 << 19), dict(nkv=1, nq=4097, q_stride=1 << 20)),
    (READ, dict(q_stride=1 << 31), dict(q_stride=(1 << 31) + 4)),
    (READ, dict(q_stride=12 * 128), dict(q_stride=12 * 128 - 4)),
    (ALL[2:], dict(nkv=4096, hd=64, page_stride=1 << 22, kv_stride=1 << 18), dict(nkv=4097, hd=64, page_stride=1 << 23, kv_stride=1 << 19)),
    (ALL[2:], dict(kv_stride=1 << 31), dict(kv_stride=(1 << 31) + 4)),
    (ALL[1:2], dict(n_rows=1 << 20, nq=1024, q_stride=1 << 17, o=1 << 50), dict(n_rows=1 << 20, nq=1026, q_stride=1 << 18, o=1 << 50)),
    (ALL[1:], dict(n_rows=1 << 20), dict(n_rows=(1 << 20) + 1)),
    (ALL, dict(n_seq=1024), dict(n_seq=1025)),
])
def test_limits(names, last, beyond):
    if names == ALL and "n_seq" in last:
        assert list(_both(("qgemv_kv_append",), q_start=None, n_rows=1024, **last)) == [OK]
    assert set(_both(names, **last)) == {OK}
    assert set(_both(names, **beyond)) == {SHAPE}
