"""The quantised cache, what writes and reads it, and attention for batches that share a prefix.

Five operators around the paged key-value cache: `qgemv_kv_append` into a cache of 8-bit elements,
`qgemv_attn` (one new token per sequence) and `qgemv_attn_prompt` (packed rows, causal) over it,
`qgemv_qkv_append` (norms of the Q and K heads, position rotation and the append in one pass) and
`qgemv_attn_shared` (one new token per sequence, where the sequences of a group begin with the same
positions) over any cache.

Shared layout: the QKV buffer is f32 [rows][(nq + 2 nkv) hd] as the fused QKV product writes it; the
cache is pages of `page` positions; `table` [n_seq][max_pages] names each sequence's pages (-1 behind
its last one); `kv_len` counts the cached positions with the new ones.  Types "f16" and "bf16" hold
K [page][hd] and V [hd][page] for each page and head; "i8" and "f8" (e4m3) hold the same as bytes and
behind them one f32 scale d for each position: x = d * code, with d = max(amax / 127, 2^-126) for i8
and for f8 the least power of two with amax <= 448 d (2^-126 at least), amax over the position's hd
values.  With `own` false `run` is the plain form in elementary torch operations; with `own` true it
is the library's calls.
"""
import random

import torch

own = False

DEVICE = "cuda"
LIB_TYPE = {"f16": "F16", "bf16": "BF16", "i8": "I8", "f8": "F8"}
HALF = {"f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"i8": torch.int8, "f8": torch.float8_e4m3fn}
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of a full row batch: 16 rows, one to each sequence
        dict(name="append8_tokens", op="append", seqs=16, rows=16, context=1500, nkv=8, nq=32, hd=128,
             page=16, type="i8"),
        # a prefill of several prompts at once, some continuing a cached prefix
        dict(name="append8_prompts", op="append", seqs=11, rows=8000, context=900, nkv=8, nq=32,
             hd=128, page=32, type="f8"),
        # between the QKV product and the attention of one stream's decode step: only latency counts
        dict(name="qkv_token", op="qkv", seqs=1, rows=1, context=180, nkv=2, nq=12, hd=128, page=16,
             type="f16", half=64, norm=True),
        # the same of a prefill chunk of several prompts
        dict(name="qkv_prompts", op="qkv", seqs=9, rows=8000, context=900, nkv=8, nq=32, hd=128,
             page=64, type="i8", half=64, norm=True),
        # the shortest decode step over an 8-bit cache
        dict(name="attn8_one_short", op="attn", seqs=1, longest=180, ragged=False, nq=12, nkv=2,
             hd=128, page=16, type="i8"),
        # one long document among short requests, and a padded slot: the split has to follow it
        dict(name="attn8_ragged_long", op="attn", seqs=7, longest=60000, ragged=True, nq=32, nkv=8,
             hd=128, page=32, type="f8"),
        # a large serving batch with long contexts: the largest cache read
        dict(name="attn8_64_long", op="attn", seqs=64, longest=8000, ragged=False, nq=24, nkv=8,
             hd=64, page=64, type="i8"),
        # a packed prefill of many requests of different lengths
        dict(name="prompt8_packed", op="prompt", seqs=9, rows=4500, context=0, nq=24, nkv=8, hd=64,
             page=16, type="f8"),
        # one whole long prompt: the largest matrix work
        dict(name="prompt8_8k", op="prompt", seqs=1, rows=8192, context=0, nq=32, nkv=8, hd=128,
             page=64, type="i8"),
        # the last chunk of a long document: few rows over a long cached context
        dict(name="prompt8_chunk_late", op="prompt", seqs=1, rows=203, context=30000, nq=12, nkv=2,
             hd=128, page=32, type="f8"),
        # chats behind two system prompts of ordinary length
        dict(name="shared_chats", op="shared", seqs=16, groups=2, prefix=1800, tail=400, nq=24, nkv=8,
             hd=64, page=16, type="bf16"),
        # many questions about one long document
        dict(name="shared_document", op="shared", seqs=64, groups=1, prefix=30000, tail=600, nq=32,
             nkv=8, hd=128, page=32, type="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    """One more case: sizes log-uniform over the listed range, every head layout and type."""
    op = rng.choice(["append", "qkv", "attn", "attn", "prompt", "shared", "shared"])
    nq, nkv = rng.choice([(12, 2), (32, 8), (8, 8), (16, 1), (24, 8), (40, 2), (14, 2)])
    hd = rng.choice([64, 96, 128, 128, 192, 256])
    types = ["i8", "f8"] if op in ("append", "attn", "prompt") else ["f16", "bf16", "i8", "f8"]
    case = dict(op=op, nq=nq, nkv=nkv, hd=hd, page=rng.choice([16, 32, 64, 128]), type=rng.choice(types))
    token = nkv * hd * 4
    if op == "attn":
        seqs = _log(rng, 1, 64)
        longest = _log(rng, 1, min(60000, 500_000_000 // (seqs * token)))
        return dict(case, seqs=seqs, longest=longest, ragged=rng.random() < 0.5)
    if op == "shared":
        seqs = _log(rng, 2, 64)
        return dict(case, seqs=seqs, groups=rng.randint(1, min(4, seqs)),
                    prefix=_log(rng, 16, min(30000, 2_600_000_000 // (seqs * token))), tail=_log(rng, 1, 700))
    rows = _log(rng, 1, 8000)
    seqs = _log(rng, 1, min(16, rows))
    context = rng.choice([0, _log(rng, 1, 30000)])
    if op == "prompt":
        while rows * (rows + context) * nq * hd > 3e10 and rows > 64:
            rows -= rows // 8
        context = min(context, 30_000_000_000 // (rows * nq * hd))
        seqs = min(seqs, rows)
    if op == "qkv":
        while rows * (nq + 2 * nkv) * hd > 40_000_000:
            rows -= rows // 8
        seqs = min(seqs, rows)
        case.update(half=rng.choice([hd // 2, hd // 2, hd // 4, 7, 0]), norm=rng.random() < 0.7)
    return dict(case, seqs=seqs, rows=rows, context=min(context, 400_000_000 // (seqs * token)))


def _rng(case):
    return random.Random(case["seqs"] * 1000003 + case["hd"] + 7 * (case.get("longest") or case.get("rows") or case["prefix"]))


def _lengths(case):
    """(new rows, cached positions with them) of each sequence: a function of the case alone."""
    n, r = case["seqs"], _rng(case)
    if case["op"] == "attn":
        top = case["longest"]
        if case["ragged"]:
            kv = [top] + [max(1, int(top * r.random() ** 4)) for _ in range(n - 1)]
            if n >= 4:
                kv[-1] = 0                       # a padded slot of the batch
        else:
            kv = [max(1, top - r.randrange(0, top // 8 + 1)) for _ in range(n)]
        return [(1, k) for k in kv]
    if case["op"] == "shared":
        return [(1, shared + tail) for _, shared, tails in _groups(case) for tail in tails]
    weights = [0.2 + r.random() for _ in range(n)]
    q = [max(1, int(case["rows"] * w / sum(weights))) for w in weights]
    while sum(q) > case["rows"]:
        q[q.index(max(q))] -= 1
    q[0] += case["rows"] - sum(q)
    ctx = [case["context"]] + [r.randrange(0, case["context"] + 1) if r.random() < 0.5 else 0
                               for _ in range(n - 1)]
    return [(a, a + c) for a, c in zip(q, ctx)]


def _groups(case):
    """(first sequence, shared positions, positions behind them of each sequence) of each group."""
    n, m, r = case["seqs"], case["groups"], _rng(case)
    starts = [0] + sorted(r.sample(range(1, n), m - 1)) + [n]
    return [(a, case["prefix"] if g == 0 else r.randrange(case["prefix"] // 3, case["prefix"] + 1),
             [r.randrange(case["tail"] // 4, case["tail"]) + 1 for _ in range(a, b)])
            for g, (a, b) in enumerate(zip(starts, starts[1:]))]


def work(case):
    lens = _lengths(case)
    rows = sum(a for a, _ in lens)
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    place = 2 * nkv * (2 * hd if case["type"] in HALF else hd + 4)     # bytes of a cached position
    if case["op"] == "append":
        return {"bytes": rows * (nkv * hd * 8 + place), "flops": 0}
    if case["op"] == "qkv":
        return {"bytes": rows * ((2 * nq + 2 * nkv) * hd * 4 + place + 8 * case["half"]), "flops": 0}
    seen = sum(a * b - a * (a - 1) // 2 for a, b in lens if b)
    read = sum(b for _, b in lens)
    if case["op"] == "shared":
        read = sum(shared + sum(tails) for _, shared, tails in _groups(case))
    return {"bytes": read * place + rows * nq * hd * 8, "flops": 4 * hd * nq * seen}


# ---------------------------------------------------------------------------------------- inputs

def _codes(x, kind):
    """Codes and scales of rows of values (the last axis), by the definition, in 64 bits."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    if kind == "i8":
        d = (amax / 127).float().clamp(min=2.0 ** -126)
        return torch.round(x / d.double()).to(torch.int8), d.squeeze(-1)
    m, e = torch.frexp(amax)
    d = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875)).clamp(min=-126))
    return (x / d).to(torch.float8_e4m3fn), d.float().squeeze(-1)


def _pages(values, case, transposed):
    """Values [pages][nkv][page][hd] as page arrays of the case's type."""
    if case["type"] in HALF:
        return (values.transpose(2, 3) if transposed else values).to(HALF[case["type"]]).contiguous()
    out = torch.empty(*values.shape[:2], case["page"] * (case["hd"] + 4), dtype=torch.uint8, device=DEVICE)
    codes, scales = _parts(out, case, transposed)
    for a in range(0, len(values), 512):                 # in parts: 64 bits of a long cache are large
        c, d = _codes(values[a:a + 512], case["type"])
        codes[a:a + 512].view(torch.uint8).copy_((c.transpose(2, 3) if transposed else c).view(torch.uint8))
        scales[a:a + 512].copy_(d)
    return out


def _parts(pages, case, transposed):
    """Views of an 8-bit page array: codes [pages][nkv][page][hd] (V [hd][page]), scales [pages][nkv][page]."""
    ps, hd = case["page"], case["hd"]
    codes = pages[:, :, :ps * hd].unflatten(2, (hd, ps) if transposed else (ps, hd))
    return codes.view(CODE[case["type"]]), pages[:, :, ps * hd:].view(torch.float32)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    new = dict(device=DEVICE, generator=g)
    lens = _lengths(case)
    n, ps, hd, nq, nkv = case["seqs"], case["page"], case["hd"], case["nq"], case["nkv"]
    need = [-(-k // ps) for _, k in lens]
    n_pages, max_pages = sum(need) + 3, max(need) + 2
    rows = sum(a for a, _ in lens)
    perm = torch.randperm(n_pages, **new).to(torch.int32)       # pages lie anywhere in the pool
    table = torch.full((n, max_pages), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = perm[at:at + k]
        at += k
    starts = [0]
    for a, _ in lens:
        starts.append(starts[-1] + a)
    ints = dict(dtype=torch.int32, device=DEVICE)
    st = dict(case, n_pages=n_pages, max_pages=max_pages, n_rows=rows, table=table,
              kv_len=torch.tensor([k for _, k in lens], **ints), q_start=torch.tensor(starts, **ints),
              most_kv=max(k for _, k in lens), most_q=max(a for a, _ in lens),
              qkv=torch.randn(rows, (nq + 2 * nkv) * hd, **new), scale=hd ** -0.5)
    if case["op"] in ("append", "qkv"):                          # the pages' earlier content is not read
        for name, t in (("k_pages", False), ("v_pages", True)):
            st[name] = _pages(torch.zeros(n_pages, nkv, ps, hd, device=DEVICE), case, t)
    else:                                                        # positions of different size, as in earnest
        for name, t in (("k_pages", False), ("v_pages", True)):
            size = torch.exp(0.3 * torch.randn(n_pages, nkv, ps, 1, **new))
            st[name] = _pages(torch.randn(n_pages, nkv, ps, hd, **new).mul_(size), case, t)
        st["qkv"][:, :nq * hd] *= 1.5                            # some rows look at few positions
        st["o"] = torch.empty(rows, nq * hd, device=DEVICE)
    if case["op"] == "qkv":
        half, top = case["half"], st["most_kv"] + 5
        angle = torch.arange(top, device=DEVICE).double()[:, None] * 10000.0 ** (
            -torch.arange(half, device=DEVICE).double() / max(half, 1))
        st.update(cos=torch.cos(angle).float(), sin=torch.sin(angle).float(), rope_rows=top,
                  q=torch.empty(rows, nq * hd, device=DEVICE),
                  q_gamma=1 + 0.2 * torch.randn(hd, **new) if case["norm"] else None,
                  k_gamma=1 + 0.2 * torch.randn(hd, **new) if case["norm"] else None)
    if case["op"] == "shared":
        groups = _groups(case)
        first = [a for a, _, _ in groups] + [n]
        for (a, b), (_, shared, _) in zip(zip(first, first[1:]), groups):
            table[a:b, :-(-shared // ps)] = table[a, :-(-shared // ps)].clone()
            own_part = shared % ps                               # a page begun by the prefix is each one's own
            if own_part:
                entry = shared // ps
                left = sum(need[:a]) + entry
                table[a:b, entry] = torch.stack([perm[left + sum(need[a:i])] for i in range(a, b)])
                for pages in (st["k_pages"], st["v_pages"]):     # with the prefix's positions in it
                    pages[table[a:b, entry].long()] = pages[table[a, entry].long()].clone()
        st.update(group_start=torch.tensor(first, **ints),
                  shared_len=torch.tensor([s for _, s, tails in groups for _ in tails], **ints),
                  most_shared=max(s for _, s, _ in groups), most_tail=max(max(t) for _, _, t in groups),
                  most_members=max(b - a for a, b in zip(first, first[1:])))
    if own:                                                      # the workspace a program keeps
        import dequant_gemv_q4_amd as lib
        from dequant_gemv_q4_amd import device
        op = {"append": lib.OP_KV_APPEND, "qkv": lib.OP_QKV_APPEND, "attn": lib.OP_ATTN,
              "prompt": lib.OP_ATTN_PROMPT, "shared": lib.OP_ATTN_SHARED}
        st["ws"] = device.attn_workspace(op[case["op"]], n, nq, nkv, hd)
    return st


# ------------------------------------------------------------------------------------------- run

def run(state):
    if own:
        return _own(state)
    return {"append": _append, "qkv": _append, "attn": _attention, "prompt": _attention,
            "shared": _shared}[state["op"]](state)


def _written(s):
    """The cache as outputs: codes as the numbers they are, and scales."""
    if s["type"] in HALF:
        return {"k": s["k_pages"], "v": s["v_pages"]}
    (k, kd), (v, vd) = _parts(s["k_pages"], s, False), _parts(s["v_pages"], s, True)
    return {"k": k, "k_scale": kd, "v": v, "v_scale": vd}


def _own(s):
    import dequant_gemv_q4_amd as lib
    stride = s["nkv"] * s["page"] * (s["hd"] if s["type"] in HALF else s["hd"] + 4)
    cache = (getattr(lib, LIB_TYPE[s["type"]]), s["k_pages"], s["v_pages"], s["n_pages"], s["page"],
             stride, s["nkv"], s["hd"], s["table"], s["max_pages"])
    width = (s["nq"] + 2 * s["nkv"]) * s["hd"]
    if s["op"] == "append":
        k0 = s["nq"] * s["hd"]
        v0 = k0 + s["nkv"] * s["hd"]
        lib.qgemv_kv_append(*cache, s["q_start"], s["kv_len"], s["seqs"], s["qkv"][:, k0:],
                            s["qkv"][:, v0:], width, s["n_rows"], s["ws"])
        return _written(s)
    if s["op"] == "qkv":
        lib.qgemv_qkv_append(*cache, s["q_start"], s["kv_len"], s["seqs"], s["qkv"], width, s["n_rows"],
                             s["nq"], s["half"], s["q_gamma"], s["k_gamma"], EPS, s["cos"], s["sin"],
                             s["rope_rows"], s["q"], s["nq"] * s["hd"], s["ws"])
        return dict(_written(s), q=s["q"])
    if s["op"] == "attn":
        lib.qgemv_attn(*cache, s["kv_len"], s["seqs"], s["qkv"], width, s["nq"], s["scale"],
                       s["o"], s["ws"])
    elif s["op"] == "prompt":
        lib.qgemv_attn_prompt(*cache, s["q_start"], s["kv_len"], s["seqs"], s["qkv"], width,
                              s["n_rows"], s["nq"], s["scale"], s["o"], s["ws"])
    else:
        lib.qgemv_attn_shared(*cache, s["kv_len"], s["seqs"], s["group_start"], s["shared_len"],
                              s["groups"], s["qkv"], width, s["nq"], s["scale"], s["o"], s["ws"])
    return {"o": s["o"]}


def _places(s):
    """Of each row: its sequence, its index in it and its position in the cache."""
    row = torch.arange(s["n_rows"], device=DEVICE)
    seq = torch.bucketize(row, s["q_start"][1:].long(), right=True)
    start, end = s["q_start"].long()[seq], s["q_start"].long()[seq + 1]
    return seq, row - start, s["kv_len"].long()[seq] - (end - row)


def _turned(x, gamma, cos, sin):
    """Norm and rotation of heads [rows][heads][hd]; cos and sin [rows][1][half]."""
    if gamma is not None:
        x = x * gamma / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    half = cos.shape[-1]
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], -1)


def _append(s):
    """Both appends.  K is turned in 64 bits: it is rounded to few bits next, and a value next to a
    border must not depend on the rounding before."""
    nq, nkv, hd, ps = s["nq"], s["nkv"], s["hd"], s["page"]
    seq, _, pos = _places(s)
    page, slot = s["table"].long()[seq, pos // ps], pos % ps
    q, k, v = (x.reshape(s["n_rows"], -1, hd) for x in s["qkv"].split((nq * hd, nkv * hd, nkv * hd), -1))
    if s["op"] == "qkv":
        cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
        s["q"].copy_(_turned(q, s["q_gamma"], cos, sin).reshape(s["n_rows"], -1))
        gamma = None if s["k_gamma"] is None else s["k_gamma"].double()
        k = _turned(k.double(), gamma, cos.double(), sin.double())
    if s["type"] in HALF:
        s["k_pages"][page, :, slot] = k.to(HALF[s["type"]])
        s["v_pages"][page, :, :, slot] = v.to(HALF[s["type"]])
    else:
        for values, pages, t in ((k, s["k_pages"], False), (v, s["v_pages"], True)):
            codes, scales = _codes(values, s["type"])
            at, d = _parts(pages, s, t)
            at = at.view(torch.uint8)
            if t:
                at[page, :, :, slot] = codes.view(torch.uint8)
            else:
                at[page, :, slot] = codes.view(torch.uint8)
            d[page, :, slot] = scales
    return dict(_written(s), q=s["q"]) if s["op"] == "qkv" else _written(s)


def _values(pages, s, transposed, of):
    """K or V of the pages `of` [a][b], in 32 bits: [a][nkv][b * page][hd]."""
    if s["type"] in HALF:
        x = pages[of].float()
    else:
        codes, d = _parts(pages, s, transposed)
        x = codes.view(torch.uint8)[of].view(CODE[s["type"]]).float()
        x = x * (d[of].unsqueeze(-2) if transposed else d[of].unsqueeze(-1))
    x = x.permute(0, 2, 1, 4, 3) if transposed else x.permute(0, 2, 1, 3, 4)
    return x.reshape(len(of), s["nkv"], -1, s["hd"])


def _softmax_parts(p, hidden):
    """Scores -> weights against their maximum, in place, and that maximum."""
    p.masked_fill_(hidden, -float("inf"))
    top = p.amax(-1, keepdim=True).clamp(min=-1e30)
    return p.sub_(top).exp_(), top


def _attention(s):
    """Sequences padded to the longest, scores, mask, softmax, product, in f32."""
    n, nq, nkv, hd, ps = s["seqs"], s["nq"], s["nkv"], s["hd"], s["page"]
    seq, at, pos = _places(s)
    used = -(-s["most_kv"] // ps)
    pages = s["table"][:, :used].clamp(min=0).long()
    k, v = _values(s["k_pages"], s, False, pages), _values(s["v_pages"], s, True, pages)
    q = torch.zeros(n, s["most_q"], nq, hd, device=DEVICE)
    q[seq, at] = s["qkv"][:, :nq * hd].reshape(-1, nq, hd)
    last = torch.full((n, s["most_q"]), -1, dtype=torch.long, device=DEVICE)
    last[seq, at] = pos
    q = q.reshape(n, s["most_q"], nkv, nq // nkv, hd).permute(0, 2, 3, 1, 4)
    q = q.reshape(n, nkv, -1, hd)                                # rows: (head of the group, token)
    p = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    p = p.reshape(n, nkv, nq // nkv, s["most_q"], used * ps)
    p, _ = _softmax_parts(p, torch.arange(used * ps, device=DEVICE) > last[:, None, None, :, None])
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(n, nkv, -1, used * ps), v).reshape(*total.shape[:-1], hd)
    o = o / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, s["most_q"], nq * hd)
    s["o"].copy_(o[seq, at])
    return {"o": s["o"]}


def _shared(s):
    """The prefix once for all rows of a group, what is behind it for each sequence, then their join."""
    n, nq, nkv, hd, ps, m = s["seqs"], s["nq"], s["nkv"], s["hd"], s["page"], s["groups"]
    heads = nq // nkv
    start, shared = s["group_start"].long(), s["shared_len"].long()
    row = torch.arange(n, device=DEVICE)
    group = torch.bucketize(row, start[1:], right=True)
    member = row - start[group]
    q = s["qkv"][:, :nq * hd].reshape(n, nkv, heads, hd) * s["scale"]

    used = -(-s["most_shared"] // ps)
    pages = s["table"][start[:-1], :used].clamp(min=0).long()
    k, v = _values(s["k_pages"], s, False, pages), _values(s["v_pages"], s, True, pages)
    qg = torch.zeros(m, s["most_members"], nkv, heads, hd, device=DEVICE)
    qg[group, member] = q
    p = torch.matmul(qg.transpose(1, 2).reshape(m, nkv, -1, hd), k.transpose(-1, -2))
    hidden = torch.arange(used * ps, device=DEVICE) >= shared[start[:-1], None, None, None]
    p, top = _softmax_parts(p, hidden)
    back = lambda x: x.reshape(m, nkv, -1, heads, x.shape[-1]).transpose(1, 2)[group, member]  # noqa: E731
    o0, l0, m0 = back(torch.matmul(p, v)), back(p.sum(-1, keepdim=True)), back(top)

    first = shared // ps
    used = -(-(s["most_tail"] + ps) // ps)
    entry = (first[:, None] + torch.arange(used, device=DEVICE)).clamp(max=s["max_pages"] - 1)
    pages = s["table"].long().gather(1, entry).clamp(min=0)
    k, v = _values(s["k_pages"], s, False, pages), _values(s["v_pages"], s, True, pages)
    at = first[:, None] * ps + torch.arange(used * ps, device=DEVICE)
    hidden = (at < shared[:, None]) | (at >= s["kv_len"].long()[:, None])
    p, m1 = _softmax_parts(torch.matmul(q, k.transpose(-1, -2)), hidden[:, None, None])
    o1, l1 = torch.matmul(p, v), p.sum(-1, keepdim=True)

    top = torch.maximum(m0, m1)
    f0, f1 = torch.exp(m0 - top), torch.exp(m1 - top)
    s["o"].copy_(((o0 * f0 + o1 * f1) / (l0 * f0 + l1 * f1)).reshape(n, nq * hd))
    return {"o": s["o"]}


# ----------------------------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs from the definitions, in 64 bits, one sequence and head after the other."""
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] in ("append", "qkv") else _exact_attention(case, s)


def _exact_append(case, s):
    ps, hd, nq, nkv = case["page"], case["hd"], case["nq"], case["nkv"]
    rows = s["qkv"].double().reshape(s["n_rows"], nq + 2 * nkv, hd)
    out = _written(s)
    whole = case["type"] == "i8"
    out = {name: x.clone() if whole and "scale" not in name else x.double() for name, x in out.items()}
    if case["op"] == "qkv":
        out["q"] = torch.zeros(s["n_rows"], nq * hd, dtype=torch.float64, device=DEVICE)
    r = 0
    for b, (a, length) in enumerate(_lengths(case)):
        x, at = rows[r:r + a].clone(), list(range(length - a, length))
        if case["op"] == "qkv":
            for part, gamma in ((slice(0, nq), s["q_gamma"]), (slice(nq, nq + nkv), s["k_gamma"])):
                if gamma is not None:
                    rms = ((x[:, part] ** 2).sum(-1, keepdim=True) / hd + EPS) ** 0.5
                    x[:, part] = x[:, part] / rms * gamma.double()
            h = case["half"]
            turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
            both = torch.complex(x[:, :nq + nkv, :h], x[:, :nq + nkv, h:2 * h]) * turn
            x[:, :nq + nkv, :h], x[:, :nq + nkv, h:2 * h] = both.real, both.imag
            out["q"][r:r + a] = x[:, :nq].reshape(a, -1)
        pages = s["table"][b].long()[torch.tensor([t // ps for t in at], device=DEVICE)]
        slots = torch.tensor([t % ps for t in at], device=DEVICE)
        for name, y in (("k", x[:, nq:nq + nkv]), ("v", x[:, nq + nkv:])):
            if case["type"] not in HALF:
                big = y.abs().amax(-1)
                if whole:
                    d = (big / 127).float().double().clamp(min=2.0 ** -126)
                else:
                    d = 2.0 ** torch.ceil(torch.log2(big.clamp(min=1e-300) / 448)).clamp(min=-126)
                    d = torch.where(big > 448 * d, 2 * d, torch.where((big <= 224 * d) & (d > 2.0 ** -126), d / 2, d))
                out[name + "_scale"][pages, :, slots] = d
                y = y / d[..., None]
                if whole:
                    y = y.round().to(torch.int8)
                else:                                            # steps of 2^-3 of the binade, 2^-9 at least
                    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                    y = (y / step).round() * step
            if name == "k":
                out["k"][pages, :, slots] = y
            else:
                out["v"][pages, :, :, slots] = y
        r += a
    return out


def _exact_attention(case, s):
    lens, ps, hd, nq, nkv = _lengths(case), case["page"], case["hd"], case["nq"], case["nkv"]
    rows = s["qkv"].double()
    tables = s["table"].tolist()
    if case["op"] == "shared":                                   # the prefix from the group's first sequence
        first = s["group_start"].tolist()
        shared = s["shared_len"].tolist()
        for a, b in zip(first, first[1:]):
            for i in range(a, b):
                whole = shared[i] // ps
                tables[i] = tables[a][:whole] + tables[i][whole:]

    def dense(pages, at, h, transposed):
        if case["type"] in HALF:
            x = pages[at, h].double()
        else:
            codes, d = _parts(pages, case, transposed)
            codes = codes.view(torch.uint8)[at, h].view(CODE[case["type"]])
            x = codes.double() * (d[at, h].double().unsqueeze(1) if transposed else d[at, h].double().unsqueeze(2))
        return (x.transpose(1, 2) if transposed else x).reshape(-1, hd)

    out = torch.zeros(len(rows), nq, hd, dtype=torch.float64, device=DEVICE)
    r = 0
    for (a, b), table in zip(lens, tables):
        if b:
            at = torch.tensor(table[:-(-b // ps)], device=DEVICE)
            seen = torch.arange(b, device=DEVICE)[None] <= torch.arange(b - a, b, device=DEVICE)[:, None]
            for h in range(nkv):
                k, v = dense(s["k_pages"], at, h, False)[:b], dense(s["v_pages"], at, h, True)[:b].contiguous()
                for j in range(h * (nq // nkv), (h + 1) * (nq // nkv)):
                    x = rows[r:r + a, j * hd:(j + 1) * hd] @ k.t().contiguous() / hd ** 0.5
                    out[r:r + a, j] = torch.softmax(torch.where(seen, x, -float("inf")), -1) @ v
        r += a
    return {"o": out.reshape(len(rows), nq * hd)}
