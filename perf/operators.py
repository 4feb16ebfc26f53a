"""The operators between the matrix products of a layer: what is measured of them.

Four operators around the library's quantized products: `qgemv_kv_append` (K and V rows of a fused
QKV output into a paged cache), `qgemv_attn` (one new token per sequence over its cache),
`qgemv_attn_prompt` (packed sequences of several new tokens, causal) and `qgemv_route` (router
logits to the ids and weights that the routed experts take).

Shared layout: the QKV buffer is f32 [rows][(nq + 2 nkv) hd] as the fused QKV product writes it;
the cache is pages of `page` positions, K [page][hd] and V [hd][page] for each page and head;
`table` [n_seq][max_pages] names each sequence's pages (-1 behind its last one); `kv_len` counts
the cached positions with the new ones.  With `own` false `run` is the plain form in elementary
torch operations; with `own` true it is the library's calls.
"""
import random

import torch

own = False

GGUF_TYPE = {"f16": 1, "bf16": 30}
TORCH_TYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of one stream: 12 Q and 2 KV heads of 128, the fused QKV workload's heads
        dict(name="append_token", op="append", seqs=1, rows=1, context=180, nkv=2, nq=12, hd=128,
             page=16, type="f16"),
        # K and V of a prefill of several prompts at once, some continuing a cached prefix
        dict(name="append_prompts", op="append", seqs=11, rows=8000, context=900, nkv=8, nq=32,
             hd=128, page=32, type="bf16"),
        # the shortest decode step: one stream, a short context, where only latency counts
        dict(name="attn_one_short", op="attn", seqs=1, longest=180, ragged=False, nq=12, nkv=2,
             hd=128, page=16, type="f16"),
        # a full row batch of ordinary chats, 24 Q and 8 KV heads of 64
        dict(name="attn_16_chats", op="attn", seqs=16, longest=2100, ragged=False, nq=24, nkv=8,
             hd=64, page=16, type="bf16"),
        # one long document among short requests, and a padded slot: the split has to follow it
        dict(name="attn_ragged_long", op="attn", seqs=7, longest=60000, ragged=True, nq=32, nkv=8,
             hd=128, page=32, type="f16"),
        # a large serving batch with long contexts: the largest cache read
        dict(name="attn_64_long", op="attn", seqs=64, longest=8000, ragged=False, nq=12, nkv=2,
             hd=128, page=64, type="bf16"),
        # a few short requests, latency-bound
        dict(name="prompt_short", op="prompt", seqs=3, rows=93, context=0, nq=12, nkv=2, hd=128,
             page=16, type="f16"),
        # a packed prefill of many requests of different lengths
        dict(name="prompt_packed", op="prompt", seqs=9, rows=4500, context=0, nq=24, nkv=8, hd=64,
             page=16, type="bf16"),
        # one whole long prompt: the largest matrix work
        dict(name="prompt_8k", op="prompt", seqs=1, rows=8192, context=0, nq=32, nkv=8, hd=128,
             page=64, type="f16"),
        # the last chunk of a long document: few rows over a long cached context
        dict(name="prompt_chunk_late", op="prompt", seqs=1, rows=203, context=30000, nq=12, nkv=2,
             hd=128, page=32, type="bf16"),
        # the routed-expert workload's router: 16 rows, 64 experts, top 8, softmax renormalised
        dict(name="route_rows_16", op="route", rows=16, experts=64, score="softmax", bias=False,
             groups=1, group_top=1, keep=1, topk=8, renorm=True),
        # the router of a prefill chunk with many experts: sigmoid, balancing bias, groups
        dict(name="route_prefill", op="route", rows=8000, experts=256, score="sigmoid", bias=True,
             groups=8, group_top=2, keep=4, topk=8, renorm=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    """One more case: sizes log-uniform over the listed range, every head layout and type."""
    op = rng.choice(["append", "attn", "attn", "prompt", "prompt", "route"])
    if op == "route":
        experts = rng.choice([8, 37, 64, 128, 160, 256, 1000, 1024])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0])
        topk = rng.randint(1, 8)
        keep = rng.randint(min(groups, -(-topk * groups // experts)), groups)
        size = experts // groups
        while keep * size < topk:
            topk -= 1
        return dict(op=op, rows=_log(rng, 1, 8000), experts=experts,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    groups=groups, group_top=rng.randint(1, min(2, size)), keep=keep, topk=topk,
                    renorm=rng.random() < 0.7)
    nq, nkv = rng.choice([(12, 2), (32, 8), (8, 8), (16, 1), (24, 8), (40, 2), (14, 2)])
    case = dict(op=op, nq=nq, nkv=nkv, hd=rng.choice([64, 96, 128, 128, 256]),
                page=rng.choice([16, 32, 64, 128]), type=rng.choice(["f16", "bf16"]))
    token = nkv * case["hd"] * 4
    if op == "attn":
        seqs = _log(rng, 1, 64)
        longest = _log(rng, 1, min(60000, 260_000_000 // (seqs * token)))
        return dict(case, seqs=seqs, longest=longest, ragged=rng.random() < 0.5)
    rows = _log(rng, 1, 8000)
    seqs = _log(rng, 1, min(16, rows))
    context = rng.choice([0, _log(rng, 1, 30000)])
    if op == "prompt":
        while rows * (rows + context) * nq * case["hd"] > 3e10 and rows > 64:
            rows -= rows // 8
        context = min(context, 30_000_000_000 // (rows * nq * case["hd"]))
        seqs = min(seqs, rows)
    return dict(case, seqs=seqs, rows=rows, context=min(context, 400_000_000 // (seqs * token)))


def _lengths(case):
    """(new rows, cached positions with them) of each sequence: a function of the case alone."""
    n = case["seqs"]
    r = random.Random(n * 1000003 + case.get("longest", case.get("rows", 0)) * 7 + case["hd"])
    if case["op"] == "attn":
        top = case["longest"]
        if case["ragged"]:
            kv = [top] + [max(1, int(top * r.random() ** 4)) for _ in range(n - 1)]
            if n >= 4:
                kv[-1] = 0                       # a padded slot of the batch
        else:
            kv = [max(1, top - r.randrange(0, top // 8 + 1)) for _ in range(n)]
        return [(1, k) for k in kv]
    weights = [0.2 + r.random() for _ in range(n)]
    q = [max(1, int(case["rows"] * w / sum(weights))) for w in weights]
    while sum(q) > case["rows"]:
        q[q.index(max(q))] -= 1
    q[0] += case["rows"] - sum(q)
    ctx = [case["context"]] + [r.randrange(0, case["context"] + 1) if r.random() < 0.5 else 0
                               for _ in range(n - 1)]
    return [(a, a + c) for a, c in zip(q, ctx)]


def work(case):
    if case["op"] == "route":
        return {"bytes": case["rows"] * (case["experts"] * 4 + case["topk"] * 8), "flops": 0}
    lens = _lengths(case)
    rows = sum(a for a, _ in lens)
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    if case["op"] == "append":
        return {"bytes": rows * nkv * hd * 2 * (4 + 2), "flops": 0}
    seen = sum(a * b - a * (a - 1) // 2 for a, b in lens if b)
    return {"bytes": sum(b for _, b in lens) * nkv * hd * 4 + rows * nq * hd * 8,
            "flops": 4 * hd * nq * seen}


# ---------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = dict(device="cuda", generator=g)
    if case["op"] == "route":
        st = dict(case, z=torch.randn(case["rows"], case["experts"], **new) * 2)
        st["b"] = torch.randn(case["experts"], **new) * 0.05 if case["bias"] else None
        st["ids"] = torch.empty(case["rows"], case["topk"], dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(case["rows"], case["topk"], device="cuda")
        return st
    lens = _lengths(case)
    n, ps, hd, nq, nkv = case["seqs"], case["page"], case["hd"], case["nq"], case["nkv"]
    dt = TORCH_TYPE[case["type"]]
    need = [-(-k // ps) for _, k in lens]
    n_pages, max_pages = sum(need) + 3, max(need) + 2
    rows = sum(a for a, _ in lens)
    perm = torch.randperm(n_pages, **new).to(torch.int32)       # pages lie anywhere in the pool
    table = torch.full((n, max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = perm[at:at + k]
        at += k
    starts = [0]
    for a, _ in lens:
        starts.append(starts[-1] + a)
    qkv = torch.randn(rows, (nq + 2 * nkv) * hd, **new)
    qkv[:, :nq * hd] *= 1.5                                      # some rows look at few positions
    st = dict(case, n_pages=n_pages, max_pages=max_pages, n_rows=rows, table=table, qkv=qkv,
              k_pages=torch.randn(n_pages, nkv, ps, hd, **new).to(dt),
              v_pages=torch.randn(n_pages, nkv, hd, ps, **new).to(dt),
              kv_len=torch.tensor([k for _, k in lens], dtype=torch.int32, device="cuda"),
              q_start=torch.tensor(starts, dtype=torch.int32, device="cuda"),
              most_kv=max(k for _, k in lens), most_q=max(a for a, _ in lens),
              o=torch.empty(rows, nq * hd, device="cuda"), scale=hd ** -0.5)
    if own:                                                      # the workspace a program keeps
        import dequant_gemv_q4_amd as lib
        from dequant_gemv_q4_amd import device
        op = {"append": lib.OP_KV_APPEND, "attn": lib.OP_ATTN, "prompt": lib.OP_ATTN_PROMPT}
        st["ws"] = device.attn_workspace(op[case["op"]], n, nq, nkv, hd)
    return st


# ------------------------------------------------------------------------------------------- run

def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attn": _attention, "prompt": _attention,
            "route": _route}[state["op"]](state)


def _own(s):
    import dequant_gemv_q4_amd as lib
    if s["op"] == "route":
        lib.qgemv_route(s["z"], s["rows"], s["experts"],
                        lib.SCORE_SIGMOID if s["score"] == "sigmoid" else lib.SCORE_SOFTMAX,
                        s["b"], s["groups"], s["group_top"], s["keep"], s["topk"], s["renorm"],
                        1.0, s["ids"], s["w"])
        return {"ids": s["ids"], "weights": s["w"]}
    cache = (GGUF_TYPE[s["type"]], s["k_pages"], s["v_pages"], s["n_pages"], s["page"],
             s["nkv"] * s["page"] * s["hd"], s["nkv"], s["hd"], s["table"], s["max_pages"])
    width = (s["nq"] + 2 * s["nkv"]) * s["hd"]
    if s["op"] == "append":
        k0 = s["nq"] * s["hd"]
        v0 = k0 + s["nkv"] * s["hd"]
        lib.qgemv_kv_append(*cache, s["q_start"], s["kv_len"], s["seqs"], s["qkv"][:, k0:],
                            s["qkv"][:, v0:], width, s["n_rows"], s["ws"])
        return {"k": s["k_pages"], "v": s["v_pages"]}
    if s["op"] == "attn":
        lib.qgemv_attn(*cache, s["kv_len"], s["seqs"], s["qkv"], width, s["nq"], s["scale"],
                       s["o"], s["ws"])
    else:
        lib.qgemv_attn_prompt(*cache, s["q_start"], s["kv_len"], s["seqs"], s["qkv"], width,
                              s["n_rows"], s["nq"], s["scale"], s["o"], s["ws"])
    return {"o": s["o"]}


def _places(s):
    """Of each row: its sequence, its index in it and its position in the cache."""
    row = torch.arange(s["n_rows"], device="cuda")
    seq = torch.bucketize(row, s["q_start"][1:].long(), right=True)
    start, end = s["q_start"].long()[seq], s["q_start"].long()[seq + 1]
    return seq, row - start, s["kv_len"].long()[seq] - (end - row)


def _append(s):
    nq, nkv, hd, ps = s["nq"], s["nkv"], s["hd"], s["page"]
    seq, _, pos = _places(s)
    page, slot = s["table"].long()[seq, pos // ps], pos % ps
    k = s["qkv"][:, nq * hd:(nq + nkv) * hd].reshape(-1, nkv, hd)
    v = s["qkv"][:, (nq + nkv) * hd:].reshape(-1, nkv, hd)
    s["k_pages"][page, :, slot] = k.to(s["k_pages"].dtype)
    s["v_pages"][page, :, :, slot] = v.to(s["v_pages"].dtype)
    return {"k": s["k_pages"], "v": s["v_pages"]}


def _attention(s):
    """Both attentions: sequences padded to the longest, scores, mask, softmax, product, in f32."""
    n, nq, nkv, hd, ps = s["seqs"], s["nq"], s["nkv"], s["hd"], s["page"]
    seq, at, pos = _places(s)
    used = -(-s["most_kv"] // ps)
    pages = s["table"][:, :used].clamp(min=0).long()
    k = s["k_pages"][pages].permute(0, 2, 1, 3, 4).reshape(n, nkv, used * ps, hd).float()
    v = s["v_pages"][pages].permute(0, 2, 1, 4, 3).reshape(n, nkv, used * ps, hd).float()
    q = torch.zeros(n, s["most_q"], nq, hd, device="cuda")
    q[seq, at] = s["qkv"][:, :nq * hd].reshape(-1, nq, hd)
    last = torch.full((n, s["most_q"]), -1, dtype=torch.long, device="cuda")
    last[seq, at] = pos
    q = q.reshape(n, s["most_q"], nkv, nq // nkv, hd).permute(0, 2, 3, 1, 4)
    q = q.reshape(n, nkv, -1, hd)                                # rows: (head of the group, token)
    p = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    p = p.reshape(n, nkv, nq // nkv, s["most_q"], used * ps)
    hidden = torch.arange(used * ps, device="cuda") > last[:, None, None, :, None]
    p.masked_fill_(hidden, -float("inf"))
    p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(n, nkv, -1, used * ps), v).reshape(*total.shape[:-1], hd)
    o = o / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, s["most_q"], nq * hd)
    s["o"].copy_(o[seq, at])
    return {"o": s["o"]}


def _route(s):
    """In 64 bits: the choice among scores next to each other must not depend on rounding."""
    z = s["z"].double()
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        score = torch.exp(z - z.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    choice = score if s["b"] is None else score + s["b"].double()
    rows, experts, groups = s["rows"], s["experts"], s["groups"]
    if groups > 1:
        inner = choice.reshape(rows, groups, experts // groups)
        best = torch.sort(inner, dim=-1, descending=True).values[..., :s["group_top"]].sum(-1)
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :s["keep"]]
        out = torch.ones(rows, groups, dtype=torch.bool, device="cuda").scatter_(1, kept, False)
        choice = inner.masked_fill(out[..., None], -float("inf")).reshape(rows, experts)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :s["topk"]]
    w = score.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    s["ids"].copy_(ids)
    s["w"].copy_(w)
    return {"ids": s["ids"], "weights": s["w"]}


# ----------------------------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs from the definitions, in 64 bits, one sequence and head after the other."""
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    lens, ps, hd, nq, nkv = _lengths(case), case["page"], case["hd"], case["nq"], case["nkv"]
    rows = s["qkv"].double()
    tables = s["table"].tolist()
    if case["op"] == "append":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        r = 0
        for (a, b), table in zip(lens, tables):
            t = 0
            while t < a:                                         # the run of rows in one page
                page, slot = table[(b - a + t) // ps], (b - a + t) % ps
                m = min(ps - slot, a - t)
                part = rows[r + t:r + t + m, nq * hd:].reshape(m, 2, nkv, hd)
                k[page, :, slot:slot + m] = part[:, 0].transpose(0, 1)
                v[page, :, :, slot:slot + m] = part[:, 1].permute(1, 2, 0)
                t += m
            r += a
        return {"k": k, "v": v}
    out = torch.zeros(len(rows), nq, hd, dtype=torch.float64, device="cuda")
    r = 0
    for (a, b), table in zip(lens, tables):
        if b:
            pages = torch.tensor(table[:-(-b // ps)], device="cuda")
            seen = torch.arange(b, device="cuda")[None] <= torch.arange(b - a, b, device="cuda")[:, None]
            for h in range(nkv):
                k = s["k_pages"][pages, h].double().reshape(-1, hd)[:b]
                v = s["v_pages"][pages, h].double().transpose(1, 2).reshape(-1, hd)[:b].contiguous()
                for j in range(h * (nq // nkv), (h + 1) * (nq // nkv)):
                    x = rows[r:r + a, j * hd:(j + 1) * hd] @ k.t().contiguous() / hd ** 0.5
                    x = torch.where(seen, x, -float("inf"))
                    out[r:r + a, j] = torch.softmax(x, -1) @ v
        r += a
    return {"o": out.reshape(len(rows), nq * hd)}


def _exact_route(s):
    z = s["z"].double()
    score = torch.sigmoid(z) if s["score"] == "sigmoid" else torch.softmax(z, -1)
    pick = score + (0 if s["b"] is None else s["b"].double())
    rows, experts = z.shape
    size = experts // s["groups"]
    if s["groups"] > 1:
        best = pick.view(rows, s["groups"], size).topk(s["group_top"], -1).values.sum(-1)
        order = torch.argsort(-best, dim=1, stable=True)
        rank = torch.empty_like(order)
        rank.scatter_(1, order, torch.arange(s["groups"], device="cuda").expand_as(order).contiguous())
        pick = torch.where((rank < s["keep"]).repeat_interleave(size, 1), pick, -float("inf"))
    ids = torch.argsort(-pick, dim=1, stable=True)[:, :s["topk"]]
    w = torch.gather(score, 1, ids)
    return {"ids": ids.to(torch.int32), "weights": w / w.sum(1, keepdim=True) if s["renorm"] else w}
