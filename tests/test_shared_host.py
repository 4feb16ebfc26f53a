"""Host-side checks of the workspace of the shared-prefix attention (no GPU)."""
import pytest

import dequant_gemv_q4_amd as q


@pytest.mark.parametrize("n_seq,nq,nkv,hd", [(1, 1, 1, 64), (16, 24, 8, 64), (64, 32, 8, 128), (512, 16, 1, 64),
                                             (513, 16, 1, 64), (1024, 4096, 1, 256), (300, 12, 2, 96), (9, 40, 2, 192)])
def test_workspace_holds_what_the_kernels_write(n_seq, nq, nkv, hd):
    """Flag and counters; exponents and sums of both halves; their means where they meet in one launch; the parts of
    what is behind the prefix by 16 columns, and of the prefix by 128."""
    rows, slots = n_seq * nq, 512 if hd <= 128 else 256
    least = 256 + 2 * 512 * 4 + 8192 * 4 + 2 * rows * 2 * 4
    if rows <= 8192:
        least += 2 * rows * hd * 4
    least += slots * min(16, nq // nkv) * (hd + 2) * 4
    least += 256 + 1024 * 32 + slots * 128 * (hd + 2) * 4
    got = q.qgemv_attn_workspace_bytes(q.OP_ATTN_SHARED, n_seq, nq, nkv, hd)
    assert least <= got <= least + 4 * 256
    others = [q.qgemv_attn_workspace_bytes(op, n_seq, nq, nkv, hd)
              for op in (q.OP_KV_APPEND, q.OP_QKV_APPEND, q.OP_ATTN, q.OP_ATTN_PROMPT)]
    assert max(others) <= got and others[0] == others[1] == 256 + 512 * 4
