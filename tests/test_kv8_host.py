"""Host-side checks of the 8-bit cache types, the fused QKV append and the shared-prefix attention (no GPU):
refusals, made before any HIP call, and the page arrays' sizes."""
import numpy as np
import pytest

import dequant_gemv_q4_amd as q
from dequant_gemv_q4_amd import device as D
from test_attn_host import APPEND, ATTN, K, L, O, PROMPT, S, T, V, W, X, _st

torch = pytest.importorskip("torch")

C, N, G, H, Y = (0x7f0000000000 + (i << 36) for i in range(8, 13))      # never touched
BLOCK8 = 16 * (128 + 4)
QKV = dict(kv_type=q.F16, k_pages=K, v_pages=V, n_pages=100, page_size=16, page_stride=2 * 16 * 128, nkv=2, hd=128,
           table=T, max_pages=40, q_start=S, kv_len=L, n_seq=3, qkv=X, qkv_stride=2048, n_rows=50, nq=12, half=64,
           q_gamma=G, k_gamma=G + 4096, eps=1e-6, cos=C, sin=N, rope_rows=700, q=Y, q_stride=1536, ws=W,
           ws_bytes=1 << 30, stream=None)
SHARED = dict(kv_type=q.F16, k_pages=K, v_pages=V, n_pages=100, page_size=16, page_stride=2 * 16 * 128, nkv=2,
              hd=128, table=T, max_pages=40, kv_len=L, n_seq=3, group_start=G, shared_len=H, n_group=2, q=X,
              q_stride=2048, nq=12, scale=0.1, o=O, ws=W, ws_bytes=1 << 30, stream=None)


@pytest.fixture(scope="module")
def lib():
    return q.lib()


@pytest.mark.parametrize("kv_type", [q.I8, q.F8])
def test_8_bit_page_strides(lib, kv_type):
    for fn, base in ((lib.qgemv_attn, ATTN), (lib.qgemv_attn_prompt, PROMPT), (lib.qgemv_kv_append, APPEND),
                     (lib.qgemv_qkv_append, QKV), (lib.qgemv_attn_shared, SHARED)):
        kw = dict(kv_type=kv_type)
        assert _st(fn, base, page_stride=2 * 16 * 128, **kw) == 3          # no room for the scales
        assert _st(fn, base, page_stride=2 * BLOCK8 - 16, **kw) == 3
        assert _st(fn, base, page_stride=2 * BLOCK8 + 8, **kw) == 3        # pages 16-byte aligned
        assert _st(fn, base, page_stride=1 << 33, **kw) == 3
        assert _st(fn, base, page_stride=2 * BLOCK8, ws=None, **kw) == 5   # accepted up to the workspace
        assert _st(fn, base, page_stride=2 * BLOCK8 + 16, ws=None, **kw) == 5
        assert _st(fn, base, page_stride=2 * BLOCK8, k_pages=K + 8, **kw) == 4
    fn, kw = lib.qgemv_kv_append, dict(kv_type=kv_type, page_stride=2 * BLOCK8)
    assert _st(fn, APPEND, v_pages=K + BLOCK8, **kw) == 7                  # blocks that overlap
    assert _st(fn, APPEND, v_pages=K + 3 * 2 * BLOCK8 - 16, **kw) == 7
    assert _st(fn, APPEND, k=K + 16, **kw) == 7


@pytest.mark.parametrize("change,status", [
    (dict(kv_type=q.Q8_0), 2), (dict(kv_type=0), 2),
    (dict(qkv=None), 1), (dict(q=None), 1), (dict(cos=None), 1), (dict(sin=None), 1), (dict(kv_len=None), 1),
    (dict(nq=0), 3), (dict(nq=3), 3), (dict(nq=8192), 3), (dict(qkv_stride=2044), 3), (dict(q_stride=1532), 3),
    (dict(qkv_stride=(1 << 31) + 4), 3), (dict(q_stride=(1 << 31) + 4), 3),
    (dict(half=-1), 3), (dict(half=65), 3), (dict(eps=-1e-6), 3), (dict(eps=float("nan")), 3),
    (dict(eps=float("inf")), 3), (dict(rope_rows=0), 3), (dict(rope_rows=(1 << 24) + 1), 3), (dict(n_rows=0), 3),
    (dict(n_rows=(1 << 20) + 1), 3), (dict(q_start=None), 3),
    (dict(qkv=X + 4), 4), (dict(q=Y + 4), 4), (dict(qkv_stride=2050), 4), (dict(q_stride=1538), 4),
    (dict(q_gamma=G + 4), 4), (dict(k_gamma=G + 8), 4), (dict(cos=C + 4), 4), (dict(sin=N + 4), 4),
    (dict(q_start=S + 2), 4), (dict(ws=None), 5), (dict(ws_bytes=64), 5), (dict(ws=W + 16), 4),
    (dict(q=X + 16), 7), (dict(q=X), 7),                    # in place, but with another stride
    (dict(q=X + 2048 * 4, q_stride=2048), 7), (dict(q=G), 7), (dict(q=C), 7), (dict(q=N), 7), (dict(q=T), 7),
    (dict(q=L), 7), (dict(q=S), 7), (dict(q=K), 7), (dict(q=V), 7), (dict(q=W), 7), (dict(ws=C), 7), (dict(ws=X), 7),
    (dict(qkv=K), 7), (dict(cos=V), 7), (dict(v_pages=K), 7), (dict(v_pages=K + 4096), 7),
])
def test_qkv_append_refusals(lib, change, status):
    assert _st(lib.qgemv_qkv_append, QKV, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(kv_type=5), 2), (dict(group_start=None), 1), (dict(shared_len=None), 1), (dict(q=None), 1),
    (dict(o=None), 1), (dict(n_group=0), 3), (dict(n_group=4), 3), (dict(nq=3), 3), (dict(scale=float("inf")), 3),
    (dict(group_start=G + 2), 4), (dict(shared_len=H + 1), 4), (dict(q=X + 8), 4), (dict(ws=None), 5),
    (dict(ws_bytes=1024), 5), (dict(ws=W + 64), 4), (dict(o=G), 7), (dict(o=H), 7), (dict(o=X), 7), (dict(o=K), 7),
    (dict(ws=G), 7), (dict(ws=H), 7),
])
def test_shared_refusals(lib, change, status):
    assert _st(lib.qgemv_attn_shared, SHARED, **change) == status


def test_workspace_sizes_of_the_new_operations():
    for op in (q.OP_QKV_APPEND, q.OP_ATTN_SHARED):
        assert q.qgemv_attn_workspace_bytes(op, 16, 12, 2, 128) >= 256
        assert q.qgemv_attn_workspace_bytes(op, 0, 12, 2, 128) == -1
        assert q.qgemv_attn_workspace_bytes(op, 1025, 12, 2, 128) == -1
        assert q.qgemv_attn_workspace_bytes(op, 16, 12, 5, 128) == -1
        assert q.qgemv_attn_workspace_bytes(op, 16, 12, 2, 100) == -1
    assert q.qgemv_attn_workspace_bytes(q.OP_ATTN_SHARED + 1, 16, 12, 2, 128) == -1


@pytest.mark.parametrize("kv_type", [q.I8, q.F8])
def test_8_bit_page_arrays(kv_type):
    k, v = D.kv_pages(kv_type, 5, 32, 3, 96, device="cpu")
    assert k.shape == v.shape == (5, 3, 32 * 100) and k.dtype == v.dtype == torch.uint8
    k.zero_(), v.zero_()
    kc, kd, vc, vd = D.kv_parts(kv_type, k, v, 32, 96)
    assert kc.shape == (5, 3, 32, 96) and vc.shape == (5, 3, 96, 32) and kd.shape == vd.shape == (5, 3, 32)
    kd[4, 2, 31] = 2.5
    vc.view(torch.uint8)[1, 0, 7, 3] = 0x38
    assert k[4, 2].view(torch.float32)[-1] == 2.5 and int(v[1, 0, 7 * 32 + 3]) == 0x38
    assert float(vc[1, 0, 7, 3]) == (1.0 if kv_type == q.F8 else 56.0)


def test_the_definition_against_torch():
    """The oracle's codes: e4m3 against torch's conversion, ties and range of both types."""
    from kv_common import as_bytes, codes64, quantised, scales64
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((400, 64)) * np.exp(rng.standard_normal((400, 1)) * 20)).astype(np.float32)
    x[0], x[1, 1:], x[2] = 0.0, 0.0, np.float32(1e-44)
    for kv_type, most in ((q.I8, 127), (q.F8, 448)):
        c, d = quantised(x, kv_type)
        assert np.abs(c).max() <= most and (d >= 2.0 ** -126).all()
        top = np.abs(c).max(axis=1)[(np.abs(x).max(axis=1) > 1e-30)]
        assert (top > (126 if kv_type == q.I8 else 223)).all()
        assert not c[0].any() and d[0] == np.float32(2.0 ** -126)
    c, d = quantised(x, q.F8)
    assert ((np.log2(d) % 1) == 0).all()
    y = torch.from_numpy(x.astype(np.float64) / d[:, None].astype(np.float64))
    assert (y.to(torch.float8_e4m3fn).double().numpy() == c).all()
    assert (torch.from_numpy(as_bytes(c, q.F8)).view(torch.float8_e4m3fn).double().numpy() == c).all()
    d = scales64(np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -3.5]]), q.I8)
    assert codes64(np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -3.5]]), d, q.I8)[0].tolist() == [[127, 0, 2, 2, 0, -4]]
    d = scales64(np.array([[448.0, 17.0, 19.0, 2.0 ** -10]]), q.F8)
    assert d[0] == 1 and codes64(np.array([[448.0, 17.0, 19.0, 2.0 ** -10]]), d, q.F8)[0].tolist() == [[448, 16, 20, 0]]
    assert scales64(np.array([[449.0]]), q.F8)[0] == 2
    c, d = quantised(np.array([[1.0, np.inf], [np.nan, 2.0], [1.0, 2.0]], np.float32), q.I8)
    assert np.isnan(d[:2]).all() and not c[:2].any() and d[2] == np.float32(2 / 127)
