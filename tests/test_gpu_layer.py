"""A run of the operators as a model uses them: one layer with routed experts over a prefill chunk of
two sequences and then two decode steps -- QKV product, QK norm + RoPE, append, attention, output
projection + residual, routing, experts.  Every step is held to its own bound on the GPU's own
inputs, and the decode steps' caches hold what prefill and the earlier steps stored."""
import numpy as np
import pytest

from gpu_common import assert_within, dev, gpu_matrix, host, require_gpu, say, tol_gemv, torch

import dequant_gemv_q4_amd as q
from dequant_gemv_q4_amd import device as D
from attn_common import attention64, check_attention, rounded, route64
import oracle
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    oracle.build(force=False)


def test_layer_prefill_then_decode():
    hidden, nq, nkv, hd, n_exp, topk, page = 512, 8, 2, 64, 16, 4, 16
    width, rh, scale = (nq + 2 * nkv) * hd, hd // 2, hd ** -0.5
    g = wl.rng(2100, 1)
    Wqkv, Wo = wl.matrix(q.Q8_0, g, width, hidden), wl.matrix(q.Q8_0, g, hidden, nq * hd)
    Wr, We = wl.matrix(q.Q8_0, g, n_exp, hidden), wl.matrix(q.Q8_0, g, n_exp * hidden, hidden)
    dW = [gpu_matrix(q.Q8_0, W, *W_shape) for W, W_shape in
          ((Wqkv, (width, hidden)), (Wo, (hidden, nq * hd)), (Wr, (n_exp, hidden)), (We, (n_exp * hidden, hidden)))]
    gamma, qg, kg = wl.gamma_f32(g, hidden), wl.gamma_f32(g, hd), wl.gamma_f32(g, hd)
    dgamma, dqg, dkg = dev(gamma), dev(qg), dev(kg)
    bias = (g.standard_normal(n_exp) * 0.02).astype(np.float32)
    dbias = dev(bias)

    seqs = [9, 5]                                      # prompt lengths
    n_pages, max_pages = 6, 3
    kp, vp = D.kv_pages(q.BF16, n_pages, page, nkv, hd)
    kp.fill_(float("nan"))
    vp.fill_(float("nan"))
    table = torch.tensor([[4, 1, -1], [0, -1, -1]], dtype=torch.int32, device="cuda")
    cache = (q.BF16, kp, vp, n_pages, page, nkv * page * hd, nkv, hd, table, max_pages)
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, 2, nq, nkv, hd)
    Kd, Vd = [[], []], [[], []]                        # what the caches must hold

    def angles(pos):
        a = np.asarray(pos)[:, None] / 1e4 ** (2.0 * np.arange(rh)[None] / hd)
        return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)

    def step(x, starts, lens, decode):
        rows = x.shape[0]
        xd = dev(x)
        qkv = torch.empty((rows, width), device="cuda")
        q.qgemv_nrm(q.Q8_0, dW[0], width, hidden, xd, dgamma, 1e-5, rows, qkv)
        yr, A = oracle.qgemv_nrm(q.Q8_0, Wqkv, width, hidden, x, gamma, 1e-5)
        assert_within(host(qkv), yr, tol_gemv(A, yr), "qkv")
        pos = np.concatenate([np.arange(n - (starts[b + 1] - starts[b]), n) for b, n in enumerate(lens)])
        cs, sn = angles(pos)
        q.qgemv_qk_norm_rope(qkv, rows, nq, nkv, hd, rh, dqg, dkg, 1e-6, dev(cs), dev(sn))
        start, kv = dev(np.array(starts, np.int32)), dev(np.array(lens, np.int32))
        q.qgemv_kv_append(*cache, None if decode else start, kv, 2, qkv[:, nq * hd:], qkv[:, (nq + nkv) * hd:],
                          width, rows, ws)
        o = torch.empty((rows, nq * hd), device="cuda")
        if decode:
            q.qgemv_attn(*cache, kv, 2, qkv, width, nq, scale, o, ws)
        else:
            q.qgemv_attn_prompt(*cache, start, kv, 2, qkv, width, rows, nq, scale, o, ws)
        hq = host(qkv)
        parts = []
        for b in range(2):
            for r in range(starts[b], starts[b + 1]):
                Kd[b].append(rounded(hq[r, nq * hd:(nq + nkv) * hd], q.BF16).reshape(nkv, hd))
                Vd[b].append(rounded(hq[r, (nq + nkv) * hd:], q.BF16).reshape(nkv, hd))
            for r in range(starts[b], starts[b + 1]):
                parts.append(attention64(hq[r, :nq * hd].reshape(nq, hd), np.stack(Kd[b]), np.stack(Vd[b]), nkv,
                                         scale, int(pos[r])))
        ref, A, S = (np.stack([p[i].reshape(-1) for p in parts]) for i in range(3))
        check_attention(host(o), ref, A, S, pos + 1, hd, q.BF16, "attention")
        h = torch.empty((rows, hidden), device="cuda")
        q.qgemv_res(q.Q8_0, dW[1], hidden, nq * hd, o, xd, rows, h)
        ho = host(o)
        yr, A = oracle.qgemv_res(q.Q8_0, Wo, hidden, nq * hd, ho, x)
        assert_within(host(h), yr, tol_gemv(A, yr), "output projection")
        z = torch.empty((rows, n_exp), device="cuda")
        q.qgemv_nrm(q.Q8_0, dW[2], n_exp, hidden, h, dgamma, 1e-5, rows, z)
        ids = torch.empty((rows, topk), dtype=torch.int32, device="cuda")
        wts = torch.empty((rows, topk), device="cuda")
        q.qgemv_route(z, rows, n_exp, q.SCORE_SIGMOID, dbias, 4, 2, 2, topk, True, 1.5, ids, wts)
        ri, rw = route64(host(z), q.SCORE_SIGMOID, bias, 4, 2, 2, topk, True, 1.5)
        assert np.array_equal(host(ids), ri)
        assert (np.abs(host(wts) - rw) <= 2.0 ** -23 * np.abs(rw)).all()
        y = torch.empty((rows, hidden), device="cuda")
        wm = D.workspace(q.OP_MOE, q.Q8_0, hidden, hidden, rows, n_exp, topk)
        q.qgemv_moe(q.Q8_0, dW[3], n_exp, hidden, hidden, h, rows, ids, wts, topk, y, wm)
        yr, A = oracle.qgemv_moe(q.Q8_0, We, n_exp, hidden, hidden, host(h), host(ids), host(wts))
        assert_within(host(y), yr, tol_gemv(A, yr), "experts")
        assert q.qgemv_moe_error(wm, n_exp, hidden, hidden, q.Q8_0) == 0
        assert q.qgemv_attn_error(ws) == 0

    say("layer: prefill")
    step(wl.normal_f32(g, (14, hidden)), [0, 9, 14], seqs, False)
    for i in range(2):
        say(f"layer: decode step {i}")
        step(wl.normal_f32(g, (2, hidden)), [0, 1, 2], [9 + i + 1, 5 + i + 1], True)
