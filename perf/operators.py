"""Cases and plain forms of the operators that continue a blended request.

A blended prefill leaves a fused cache and a first token.  What follows it
needs three operators:

  append     new keys (rotated to their positions) and values go to the pages
             of a paged cache, the queries are rotated on the way; with several
             layers and no rotation it moves a finished fused cache into pages;
  attention  the new rows of every sequence attend, causally, over its pages:
             one row per sequence while tokens are generated, chunks of rows
             for a follow-up turn or a long query;
  sample     the next token of every row of logits from a given uniform
             number, with temperature, top-k, top-p and min-p.

`run` computes an operator in elementary torch operations, or, where `own` is
true, through this package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
ROPE_BASE = 10000.0


def _paged(name, op, dtype, seqs, n_new, kv_min, kv_max, page, heads, lens, ragged=False, idle=False,
           layers=1, rotate=True):
    hq, hkv, hd = heads
    case = {"op": op, "dtype": dtype, "seqs": seqs, "n_new": n_new, "kv_min": kv_min, "kv_max": kv_max,
            "page": page, "hq": hq, "hkv": hkv, "hd": hd, "lens": lens, "ragged": ragged, "idle": idle,
            "layers": layers, "rotate": rotate}
    return {"name": name, **case} if name else case


def _sample(name, dtype, rows, vocab, policy, banned):
    case = {"op": "sample", "dtype": dtype, "rows": rows, "vocab": vocab, "policy": policy, "banned": banned}
    return {"name": name, **case} if name else case


def listed():
    g4 = (32, 8, 128)     # 32 query heads over 8 key/value heads of 128
    tiny = (4, 2, 64)     # the small float model's heads
    return [
        # the first generated token after a request of 6 x 512 + 64 tokens: one row, latency counts
        _paged("append_one", "append", "bf16", 1, 1, 3137, 3137, 16, g4, 1),
        # a decode step of a batch whose contexts reach far positions
        _paged("append_batch_far", "append", "bf16", 128, 1, 500, 131072, 32, g4, 2),
        # follow-up turns of three requests on the small float model, ragged
        _paged("append_chunks_f32", "append", "f32", 3, 701, 900, 4001, 16, tiny, 3, ragged=True),
        # a blended request's fused cache (32 layers, 3136 rows, already rotated) moves into pages
        _paged("append_import", "append", "bf16", 1, 3136, 3136, 3136, 16, g4, 4, layers=32, rotate=False),
        # one generated token over that request's cache
        _paged("decode_one", "attention", "bf16", 1, 1, 3137, 3137, 16, g4, 5),
        # a decode step of 64 requests of very different lengths, some slots of the batch idle
        _paged("decode_batch", "attention", "bf16", 64, 1, 200, 16384, 32, g4, 6, idle=True),
        # generation over two very long documents
        _paged("decode_long", "attention", "bf16", 2, 1, 120001, 131072, 64, g4, 7),
        # a follow-up question of 64 tokens over one request's cache
        _paged("chunk_question", "attention", "bf16", 1, 64, 3200, 3200, 16, g4, 8),
        # long follow-up documents, prefilled in chunks over what is there: the most arithmetic
        _paged("chunk_large", "attention", "bf16", 4, 2048, 8192, 8192, 128, g4, 9),
        # the small float model: ragged chunks, an idle slot
        _paged("chunk_f32", "attention", "f32", 5, 201, 300, 1501, 16, tiny, 10, ragged=True, idle=True),
        # one row of logits as the tied output projection gives them
        _sample("sample_one", "bf16", 1, 128256, "k+p", False),
        # a batch in which every request brings its own settings, some tokens banned
        _sample("sample_batch", "f32", 96, 151936, "mixed", True),
    ]


HEADS = [(32, 8, 128), (4, 2, 64), (8, 8, 128), (28, 4, 128), (24, 8, 64), (16, 1, 128), (64, 8, 128)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "sample"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    lens = rng.randrange(1 << 30)
    if op == "sample":
        vocab = _log(rng, 1000, 200000)
        rows = _log(rng, 1, max(1, min(256, 96 * 151936 * 4 // (vocab * BYTES[dtype]))))
        return _sample(None, dtype, rows, vocab, rng.choice(["k", "k+p", "p", "min_p", "none", "mixed"]),
                       rng.random() < 0.5)
    heads = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128])
    idle = rng.random() < 0.3
    if op == "append":
        if rng.random() < 0.3:
            rows = _log(rng, 3, 3000)
            layers = _log(rng, 2, 32)
            return _paged(None, op, dtype, 1, rows, rows, rows, page, heads, lens, layers=layers, rotate=False)
        seqs, n_new = _log(rng, 1, 128), _log(rng, 1, 2048)
        while seqs * n_new > 16384:
            seqs = max(1, seqs // 2)
        return _paged(None, op, dtype, seqs, n_new, n_new, n_new + _log(rng, 1, 100000), page, heads, lens,
                      ragged=rng.random() < 0.7, idle=idle)
    if rng.random() < 0.5:
        seqs, n_new, kv_max = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 5]), _log(rng, 8, 131072)
    else:
        seqs, n_new, kv_max = _log(rng, 1, 8), _log(rng, 6, 2048), _log(rng, 64, 32768)
    kv_max = max(kv_max, n_new)
    hq, hkv, hd = heads
    flops = 9.0e11 if dtype == "bf16" else 3.0e10      # float rows run on the CUDA cores
    while (4.0 * hd * hq * seqs * n_new * kv_max > flops or seqs * kv_max * hkv * hd * BYTES[dtype] > 1.0e9
           or seqs * hq * n_new * kv_max > 2.1e9):
        if seqs > 1:
            seqs //= 2
        elif kv_max > 2 * n_new:
            kv_max //= 2
        else:
            n_new = max(1, n_new // 2)
    return _paged(None, op, dtype, seqs, n_new, max(1, kv_max // rng.choice([1, 2, 20])), kv_max, page, heads, lens,
                  ragged=rng.random() < 0.7, idle=idle)


def _lengths(case):
    """(new rows, length with them) of every sequence; an idle slot of a batch has one row and no cache."""
    rng = random.Random(case["lens"])
    out = []
    for s in range(case["seqs"]):
        n = case["n_new"] if s == 0 or not case["ragged"] else rng.randint(1, case["n_new"])
        kv = case["kv_max"] if s == 0 else _log(rng, max(1, case["kv_min"]), case["kv_max"])
        out.append((1, 0) if case["idle"] and s % 5 == 3 else (n, max(n, kv)))
    return out


def _rows(case):
    """Sequence and position of every new row (position < 0: the slot is idle)."""
    seq, pos = [], []
    for s, (n, kv) in enumerate(_lengths(case)):
        seq += [s] * n
        pos += range(kv - n, kv)
    return seq, pos


# ---------------------------------------------------------------- inputs --
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "sample":
        return _prepare_sample(case, seed, g)
    dt, lens = TORCH[case["dtype"]], _lengths(case)
    hq, hkv, hd, page, nl = case["hq"], case["hkv"], case["hd"], case["page"], case["layers"]
    kvw, rows = hkv * hd, sum(n for n, _ in lens)
    need = [max(1, -(-kv // page)) for _, kv in lens]
    if case["op"] == "append":
        # pages below the first one that is written are only named by the table, so they share one
        first = [max(0, kv - n) // page for n, kv in lens]
    else:
        first = [0] * len(lens)
    total = sum(a - b for a, b in zip(need, first)) + 1
    perm = torch.randperm(total - 1, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), total - 1, dtype=torch.int32, device="cuda")
    at = 0
    for s, (a, b) in enumerate(zip(need, first)):
        table[s, b:a] = perm[at:at + a - b]
        at += a - b

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
    st = {"case": dict(case), "table": table, "offsets": torch.from_numpy(cu).cuda(),
          "lens": torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"), "max_kv": max(kv for _, kv in lens)}
    lead = (nl,) if nl > 1 else ()
    st["k_pages"], st["v_pages"] = randn(*lead, total, page, kvw), randn(*lead, total, page, kvw)
    if case["op"] == "append":
        st["k"], st["v"] = randn(*lead, rows, kvw), randn(*lead, rows, kvw)
        if case["rotate"]:
            st["q"] = randn(rows, hq * hd)
            st["q_out"] = torch.zeros_like(st["q"])
            # (cos, sin) per position and pair, angles in double precision
            p = torch.arange(st["max_kv"] + 1, device="cuda", dtype=torch.float64)
            e = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
            a = p[:, None] * torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device="cuda"), -2.0 * e / hd)[None]
            st["rope"] = torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()
    else:
        st["q"] = randn(rows, hq * hd)
        st["out"] = torch.zeros_like(st["q"])
    return st


def _prepare_sample(case, seed, g):
    n, v = case["rows"], case["vocab"]
    # a wide bulk and a few dozen likely continuations
    x = 2.2 * torch.randn(n, v, generator=g, device="cuda")
    likely = torch.randint(0, v, (n, 48), generator=g, device="cuda")
    x.scatter_add_(1, likely, 9.0 + 4.0 * torch.rand(n, 48, generator=g, device="cuda"))
    if case["banned"]:
        x.masked_fill_(torch.rand(n, v, generator=g, device="cuda") < 0.01, -math.inf)
    r = random.Random(int(seed))
    temp = [r.uniform(0.4, 1.4) for _ in range(n)]
    ks, ps, ms = [0] * n, [1.0] * n, [0.0] * n
    for i in range(n):
        policy = case["policy"] if case["policy"] != "mixed" else r.choice(["k", "k+p", "p", "min_p", "none", "greedy"])
        if "k" in policy:
            ks[i] = r.choice([1, 5, 20, 50, 200, 1000])
        if policy in ("p", "k+p"):
            ps[i] = r.choice([0.5, 0.8, 0.9, 0.95, 0.99])
        if policy == "min_p":
            ms[i] = r.choice([0.01, 0.05, 0.1, 0.3])
        if policy == "greedy":
            temp[i] = 0.0

    def dev(a, dt):
        return torch.tensor(a, dtype=dt, device="cuda")

    return {"case": dict(case), "logits": x.to(TORCH[case["dtype"]]), "u": torch.rand(n, generator=g, device="cuda"),
            "temperature": dev(temp, torch.float32), "top_k": dev(ks, torch.int32), "top_p": dev(ps, torch.float32),
            "min_p": dev(ms, torch.float32), "tokens": torch.zeros(n, dtype=torch.int32, device="cuda")}


# ------------------------------------------------------------------ runs --
def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _own_append, "attention": _own_attention, "sample": _own_sample}[op](st)
    return {"append": _plain_append, "attention": _plain_attention, "sample": _plain_sample}[op](st)


def _own_append(st):
    import rag_kv_cache_layer_gb300 as R
    R.cb_paged_append(st["k"], st["v"], st["offsets"], st["lens"], st["table"], st["k_pages"], st["v_pages"],
                      st["case"]["hd"], rope_table=st.get("rope"), q=st.get("q"), q_out=st.get("q_out"))
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"], "q": st.get("q_out")}


def _own_attention(st):
    import rag_kv_cache_layer_gb300 as R
    c = st["case"]
    if "ws" not in st:      # the scratch that a serving loop keeps from step to step
        st["ws"] = R.cb_paged_attention_workspace(st["q"], c["seqs"], st["max_kv"], c["hq"], c["hkv"], c["hd"])
    R.cb_paged_attention(st["q"], st["offsets"], st["lens"], st["table"], st["k_pages"], st["v_pages"], c["hq"], c["hkv"],
                         c["hd"], st["out"], max_kv_len=st["max_kv"], ws=st["ws"])
    return st["out"]


def _own_sample(st):
    import rag_kv_cache_layer_gb300 as R
    R.cb_sample_tokens(st["logits"], st["u"], st["tokens"], temperature=st["temperature"], top_k=st["top_k"],
                       top_p=st["top_p"], min_p=st["min_p"])
    return st["tokens"]


def _row_place(st):
    """Sequence, index in it and position of every new row, from the device's offsets and lengths."""
    off, lens, rows = st["offsets"].long(), st["lens"].long(), (st["k"] if "k" in st else st["q"]).shape[-2]
    r = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(off, r, right=True) - 1
    at = r - off[seq]
    return seq, at, lens[seq] - (off[seq + 1] - off[seq]) + at


def _plain_append(st):
    c = st["case"]
    hd, page, kvw = c["hd"], c["page"], c["hkv"] * c["hd"]
    seq, _, pos = _row_place(st)
    live = pos >= 0
    safe = pos.clamp(min=0)

    def rotated(x):
        cs = st["rope"][safe]
        a, b = x.float().unflatten(-1, (-1, 2, hd // 2)).unbind(-2)
        cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-2).flatten(-3)

    dst = (st["table"].long()[seq, safe // page] * page + safe % page)[live]
    k = rotated(st["k"]).to(st["k"].dtype) if c["rotate"] else st["k"]
    kp, vp = (st[n].view(*st[n].shape[:-3], -1, kvw) for n in ("k_pages", "v_pages"))
    kp[..., dst, :] = k[..., live, :]
    vp[..., dst, :] = st["v"][..., live, :]
    if c["rotate"]:
        st["q_out"][live] = rotated(st["q"]).to(st["q"].dtype)[live]
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"], "q": st.get("q_out")}


def _plain_attention(st):
    c = st["case"]
    hq, hkv, hd, page, s, n, m = c["hq"], c["hkv"], c["hd"], c["page"], c["seqs"], c["n_new"], st["max_kv"]
    seq, at, pos = _row_place(st)
    j = torch.arange(m, device="cuda")
    at_row = st["table"].long()[:, j // page] * page + j % page
    there = (j[None, :] < st["lens"].long()[:, None])[:, :, None, None]

    def cache(pages):
        x = pages.view(-1, hkv, hd)[at_row.flatten()].view(s, m, hkv, hd).float()
        return torch.where(there, x, torch.zeros((), device="cuda")).transpose(1, 2)

    q = torch.zeros(s, n, hq, hd, device="cuda")
    q[seq, at] = st["q"].float().view(-1, hq, hd)
    last = torch.full((s, n), -1, device="cuda", dtype=torch.long)
    last[seq, at] = pos
    q = q.view(s, n, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4).reshape(s, hkv, -1, hd)
    x = torch.matmul(q, cache(st["k_pages"]).transpose(2, 3)).view(s, hq, n, m).mul_(1.0 / math.sqrt(hd))
    hidden = j[None, None, None, :] > last[:, None, :, None]
    x.masked_fill_(hidden, -math.inf)
    top = x.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    x.sub_(top).exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x.view(s, hkv, -1, m), cache(st["v_pages"])).view(s, hq, n, hd)
    o = torch.where(total > 0, o / total, torch.zeros((), device="cuda")).permute(0, 2, 1, 3)
    return o[seq, at].reshape(-1, hq * hd).to(st["q"].dtype)


def _plain_sample(st):
    x = st["logits"].double()
    n, v = x.shape
    x = torch.where(x.isnan(), -math.inf, x)
    idx = torch.arange(v, device="cuda")[None]
    top = x.amax(dim=1, keepdim=True)
    greedy = torch.where(x == top, idx, v).amin(dim=1)
    temp = st["temperature"].double()[:, None]
    # weights in 64 bits: neighbours of a border differ by less than 32 bits tell apart
    w = torch.exp((x - top) / torch.where(temp > 0, temp, 1.0))
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    k = st["top_k"].long()[:, None]
    ws = torch.where((k <= 0) | (idx < k), ws, 0.0)
    p = st["top_p"].double()[:, None]
    run_sum = ws.cumsum(dim=1)
    before = run_sum - ws
    ws = torch.where((p >= 1.0) | (before < p * run_sum[:, -1:]) | (idx == 0), ws, 0.0)
    ws = torch.where(ws >= st["min_p"].double()[:, None], ws, 0.0)
    kept = torch.zeros_like(ws).scatter_(1, order, ws)
    cum = kept.cumsum(dim=1)
    hit = (cum > st["u"].double()[:, None] * cum[:, -1:]) & (kept > 0)
    token = torch.where(hit, idx, v).amin(dim=1)
    return torch.where(temp[:, 0] > 0, token, greedy).to(torch.int32)


# ------------------------------------------------------------------ work --
def work(case):
    eb = BYTES[case["dtype"]]
    if case["op"] == "sample":
        n, v = case["rows"], case["vocab"]
        return {"bytes": n * v * eb + 24 * n, "flops": 4.0 * n * v}
    lens = _lengths(case)
    hq, hkv, hd, page = case["hq"], case["hkv"], case["hd"], case["page"]
    live = sum(n for n, kv in lens if kv > 0)
    meta = 8 * len(lens) + 4 * sum(-(-kv // page) for _, kv in lens)
    if case["op"] == "append":
        per_row = 4 * hkv * hd * eb * case["layers"] + ((2 * hq * hd * eb + 4 * hd) if case["rotate"] else 0)
        return {"bytes": live * per_row + 12 * len(lens),
                "flops": live * (3.0 * (hq + hkv) * hd if case["rotate"] else 0.0)}
    pairs = sum(n * (kv - n) + n * (n + 1) // 2 for n, kv in lens if kv > 0)
    rows = sum(n for n, _ in lens)
    return {"bytes": 2 * hkv * hd * eb * sum(kv for _, kv in lens) + 2 * rows * hq * hd * eb + meta,
            "flops": 4.0 * hd * hq * pairs}


# ----------------------------------------------------------------- exact --
def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](st)


def _exact_append(st):
    c = st["case"]
    hd, half, page = c["hd"], c["hd"] // 2, c["page"]
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    seq, pos = (torch.tensor(a, device="cuda") for a in _rows(c))
    live = (pos >= 0).nonzero()[:, 0]
    pg, slot = st["table"].long()[seq[live], pos[live] // page], pos[live] % page
    if not c["rotate"]:
        kp[..., pg, slot, :] = st["k"].double()[..., live, :]
        vp[..., pg, slot, :] = st["v"].double()[..., live, :]
        return {"k_pages": kp, "v_pages": vp, "q": None}
    theta = torch.tensor([ROPE_BASE ** (-2.0 * e / hd) for e in range(half)], dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[live].double()[:, None, None] * theta)

    def turned(x):
        x = x[live].double().view(len(live), -1, hd)
        z = torch.complex(x[..., :half], x[..., half:]) * turn
        return torch.cat([z.real, z.imag], dim=-1).view(len(live), -1)

    kp[pg, slot], vp[pg, slot] = turned(st["k"]), st["v"].double()[live]
    q = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    q[live] = turned(st["q"])
    return {"k_pages": kp, "v_pages": vp, "q": q}


def _exact_attention(st):
    c = st["case"]
    hq, hkv, hd, page = c["hq"], c["hkv"], c["hd"], c["page"]
    g, out, row = hq // hkv, [], 0
    for s, (n, kv) in enumerate(_lengths(c)):
        q = st["q"][row:row + n].double().view(n, hq, hd)
        row += n
        o = torch.zeros(n, hq, hd, dtype=torch.float64, device="cuda")
        if kv > 0:
            pages = st["table"][s, :-(-kv // page)].long()
            k, v = (st[a][pages].view(-1, hkv, hd)[:kv].double() for a in ("k_pages", "v_pages"))
            late = torch.arange(kv, device="cuda")[None, :] > torch.arange(kv - n, kv, device="cuda")[:, None]
            for h in range(hkv):
                x = torch.einsum("ngd,jd->gnj", q[:, h * g:(h + 1) * g], k[:, h]) / math.sqrt(hd)
                x = torch.softmax(x.masked_fill(late, -math.inf), dim=-1)
                o[:, h * g:(h + 1) * g] = torch.einsum("gnj,jd->ngd", x, v[:, h])
        out.append(o.view(n, hq * hd))
    return torch.cat(out)


def _exact_sample(st):
    logits = st["logits"].double().cpu().numpy()
    u, temp, ks, ps, ms = (st[n].cpu().numpy().tolist() for n in ("u", "temperature", "top_k", "top_p", "min_p"))
    out = []
    for i, x in enumerate(logits):
        if temp[i] <= 0:
            out.append(int(np.argmax(x)))
            continue
        w = np.exp((x - x.max()) / temp[i])
        rank = np.lexsort((np.arange(len(x)), -x))
        if ks[i] > 0:
            rank = rank[:ks[i]]
        if ps[i] < 1:
            part = np.cumsum(w[rank])
            rank = rank[:1 + int(np.searchsorted(part, ps[i] * part[-1], side="left"))]
        rank = np.sort(rank[w[rank] >= ms[i]])
        part = np.cumsum(w[rank])
        out.append(int(rank[np.searchsorted(part, u[i] * part[-1], side="right")]))
    return torch.tensor(out, dtype=torch.int32)
