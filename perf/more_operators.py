"""Cases and plain forms of the operators that keep long contexts cheap.

A generated token reads the whole cache.  Two things make it read less:

  fewer bits   a paged cache in 4 bits (keys and values as 4-bit floats, one
               8-bit float scale for 16 dimensions of a head): `store` appends
               rows to it (keys and queries rotated on the way) and reads the
               same rows back, `attention4` attends over it;
  fewer keys   `select` keeps the bounds of every page's keys, scores the pages
               of each new row by the largest dot product that they allow, and
               picks the best; `picked` attends over the picked pages alone.

`run` computes an operator in elementary torch operations, or, where `own` is
true, through this package's entry points.
"""
import math
import random

import torch

own = False

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
ROPE_BASE = 10000.0


def _case(name, op, dtype, seqs, n_new, kv_min, kv_max, page, heads, lens, ragged=False, idle=False, layers=1,
          rotate=True, picks=0):
    hq, hkv, hd = heads
    case = {"op": op, "dtype": dtype, "seqs": seqs, "n_new": n_new, "kv_min": kv_min, "kv_max": kv_max,
            "page": page, "hq": hq, "hkv": hkv, "hd": hd, "lens": lens, "ragged": ragged, "idle": idle,
            "layers": layers, "rotate": rotate, "picks": picks}
    return {"name": name, **case} if name else case


def listed():
    g4 = (32, 8, 128)     # 32 query heads over 8 key/value heads of 128
    tiny = (4, 2, 64)     # the small float model's heads
    return [
        # a decode step of a batch whose contexts reach far positions
        _case("store_batch_far", "store", "bf16", 96, 1, 500, 131072, 32, g4, 1),
        # a blended request's fused cache (32 layers, 3136 rows, already rotated) kept in 4 bits and taken back
        _case("store_import", "store", "bf16", 1, 3136, 3136, 3136, 16, g4, 2, layers=32, rotate=False),
        # one generated token over that request's cache: latency counts
        _case("attention4_one", "attention4", "bf16", 1, 1, 3137, 3137, 16, g4, 3),
        # a decode step of 64 requests of very different lengths, some slots of the batch idle
        _case("attention4_batch", "attention4", "bf16", 64, 1, 200, 16384, 32, g4, 4, idle=True),
        # generation over two very long documents
        _case("attention4_long", "attention4", "bf16", 2, 1, 120001, 131072, 64, g4, 5),
        # long follow-up documents, prefilled in chunks over what is there: the most arithmetic
        _case("attention4_chunk", "attention4", "bf16", 2, 1024, 12288, 16384, 16, g4, 6),
        # drafts on the small float model, ragged, an idle slot
        _case("attention4_f32", "attention4", "f32", 6, 5, 300, 4001, 16, tiny, 7, ragged=True, idle=True),
        # a decode step of 64 long requests: their newest pages' bounds, then 64 pages of each
        _case("select_batch", "select", "bf16", 64, 1, 2000, 65536, 32, g4, 8, picks=64),
        # two very long documents in small pages: 128 of about 8000
        _case("select_long", "select", "bf16", 2, 1, 120001, 131072, 16, g4, 9, picks=128),
        # one generated token over 128 picked pages of a very long document
        _case("picked_one", "picked", "bf16", 1, 1, 131072, 131072, 16, g4, 10, picks=128),
        # the attention of the batch above
        _case("picked_batch", "picked", "bf16", 64, 1, 2000, 65536, 32, g4, 11, picks=64),
        # drafts on the small float model over small pages, ragged, an idle slot
        _case("picked_f32", "picked", "f32", 6, 5, 300, 9001, 8, tiny, 12, ragged=True, idle=True, picks=45),
    ]


HEADS = [(32, 8, 128), (4, 2, 64), (8, 8, 128), (28, 4, 128), (24, 8, 64), (16, 1, 128), (64, 8, 128)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "attention4", "attention4", "select", "picked"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    heads, page, lens = rng.choice(HEADS), rng.choice([8, 16, 32, 64, 128]), rng.randrange(1 << 30)
    idle, ragged = rng.random() < 0.3, rng.random() < 0.7
    hq, hkv, hd = heads
    if op == "store":
        if rng.random() < 0.3:
            rows, layers = _log(rng, 3, 3000), _log(rng, 2, 32)
            return _case(None, op, dtype, 1, rows, rows, rows, page, heads, lens, layers=layers, rotate=False)
        seqs, n_new = _log(rng, 1, 128), _log(rng, 1, 2048)
        while seqs * n_new > 16384:
            seqs = max(1, seqs // 2)
        return _case(None, op, dtype, seqs, n_new, n_new, n_new + _log(rng, 1, 100000), page, heads, lens,
                     ragged=ragged, idle=idle)
    if op == "attention4" and rng.random() < 0.5:
        seqs, n_new, kv_max = _log(rng, 1, 8), _log(rng, 6, 2048), _log(rng, 64, 32768)
    else:
        seqs, n_new, kv_max = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 5]), _log(rng, 8, 131072)
    kv_max = max(kv_max, n_new)
    picks = 0 if op == "attention4" else max(4, min(_log(rng, 4, 256), 4096 // page))

    def too_much():
        keys = min(kv_max, picks * page) if op == "picked" else kv_max
        pairs = seqs * hq * n_new * keys
        values = seqs * hkv * hd * (n_new * keys if op == "picked" else kv_max if op == "attention4" else 0)
        return (4.0 * hd * pairs > (5.0e11 if dtype == "bf16" else 3.0e10) or values > 5.0e8 or pairs > 1.0e9
                or (op == "select" and seqs * kv_max / page * hkv * hd > 1.2e8)
                or (op != "attention4" and seqs * kv_max * hkv * hd > 4.0e9))
    while too_much():
        if seqs > 1:
            seqs //= 2
        elif kv_max > 2 * n_new:
            kv_max //= 2
        else:
            n_new = max(1, n_new // 2)
    return _case(None, op, dtype, seqs, n_new, max(1, kv_max // rng.choice([1, 2, 20])), kv_max, page, heads, lens,
                 ragged=ragged, idle=idle, picks=picks)


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
# The 4-bit floats by code, and the 4-bit cache's layout.  A page holds, for one
# kv head after the other: the keys' codes [slot][hd / 2], the values' codes, the
# keys' scales [slot][hd / 16] (8-bit floats, 4 exponent and 3 mantissa bits), the
# values' scales.  A byte holds the codes of an even dimension (low) and the next.
CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
FIRST, LAST = 1, 2        # pages that are always picked: the first, the newest


def _page_bytes(case):
    return case["page"] * case["hkv"] * case["hd"] * 9 // 8


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt, lens = case["op"], TORCH[case["dtype"]], _lengths(case)
    hq, hkv, hd, page, nl = case["hq"], case["hkv"], case["hd"], case["page"], case["layers"]
    kvw, rows = hkv * hd, sum(n for n, _ in lens)
    need = [max(1, -(-kv // page)) for _, kv in lens]
    # pages that a store does not write are only named by the table, so they share one
    first = [max(0, kv - n) // page if op == "store" else 0 for n, kv in lens]
    total = sum(a - b for a, b in zip(need, first)) + 1
    perm = torch.randperm(total - 1, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), total - 1, dtype=torch.int32, device="cuda")
    at = 0
    for s, (a, b) in enumerate(zip(need, first)):
        table[s, b:a] = perm[at:at + a - b]
        at += a - b

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    cu = torch.tensor([0] + [n for n, _ in lens]).cumsum(0).to(torch.int32)
    st = {"case": dict(case), "table": table, "offsets": cu.cuda(), "max_kv": max(kv for _, kv in lens),
          "lens": torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")}
    if op == "store":
        lead = (nl,) if nl > 1 else ()
        st["pages"] = torch.zeros(*lead, total, _page_bytes(case), dtype=torch.uint8, device="cuda")
        st["k"], st["v"] = randn(*lead, rows, kvw), randn(*lead, rows, kvw)
        st["k_back"], st["v_back"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
        if case["rotate"]:
            st["q"] = randn(rows, hq * hd)
            st["q_out"] = torch.zeros_like(st["q"])
            # (cos, sin) per position and pair, angles in double precision
            p = torch.arange(st["max_kv"] + 1, device="cuda", dtype=torch.float64)
            e = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
            a = p[:, None] * torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device="cuda"), -2.0 * e / hd)[None]
            st["rope"] = torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()
        return st
    st["q"] = randn(rows, hq * hd)
    if op == "attention4":
        st["pages"], st["out"] = _random_pages(case, total, g), torch.zeros_like(st["q"])
        return st
    # keys of a page resemble one another, as neighbouring tokens' keys do
    st["k_pages"] = randn(total, page, kvw).mul_(0.8).add_(0.6 * randn(total, 1, kvw))
    if op == "select":
        st["bounds"] = torch.stack([st["k_pages"].amin(1), st["k_pages"].amax(1)], dim=1)
        st["picks"] = torch.zeros(rows, hkv, case["picks"], dtype=torch.int32, device="cuda")
        return st
    st["v_pages"], st["out"] = randn(total, page, kvw), torch.zeros_like(st["q"])
    # the newest pages of every row, the first, and some between, ascending
    _, pos = _rows(case)
    pages = torch.tensor([p // page + 1 for p in pos], device="cuda")[:, None, None]
    j = torch.arange(int(pages.max()), device="cuda")
    x = torch.rand(rows, hkv, len(j), generator=g, device="cuda")
    x = torch.where((j < FIRST) | (j >= pages - LAST), x + 1.0, x).masked_fill_(j >= pages, -1.0)
    top = torch.topk(x, min(case["picks"], len(j)), dim=-1)
    got = torch.where(top.values >= 0, top.indices, 1 << 30).sort(dim=-1).values
    st["picks"] = torch.full((rows, hkv, case["picks"]), -1, dtype=torch.int32, device="cuda")
    st["picks"][:, :, :got.shape[-1]] = torch.where(got < 1 << 30, got, -1).to(torch.int32)
    return st


def _random_pages(case, total, g):
    """Pages of a 4-bit cache of normally distributed keys and values: codes and scales as such rows get them."""
    n, hkv, hd, page = 1 << 13, case["hkv"], case["hd"], case["page"]
    codes, scales = _quantised(torch.randn(n, 16, generator=g, device="cuda", dtype=torch.float64))
    two, one = _code_bytes(codes).view(-1), scales.float().to(torch.float8_e4m3fn).view(torch.uint8).view(-1)
    out = torch.empty(total, hkv, page * hd * 9 // 8, dtype=torch.uint8, device="cuda")

    def some(values, size):
        return values[torch.randint(0, len(values), (total, hkv, size), generator=g, device="cuda", dtype=torch.int32)]

    out[..., :page * hd] = some(two, page * hd)
    out[..., page * hd:] = some(one, page * hd // 8)
    return out.view(total, -1)


# ------------------------------------------------------------------ runs --
def run(st):
    op = st["case"]["op"]
    if own:
        return {"store": _own_store, "attention4": _own_attention4, "select": _own_select, "picked": _own_picked}[op](st)
    return {"store": _plain_store, "attention4": _plain_attention4, "select": _plain_select,
            "picked": _plain_picked}[op](st)


def _own_store(st):
    import rag_kv_cache_layer_gb300 as R
    c = st["case"]
    R.cb_paged4_append(st["k"], st["v"], st["offsets"], st["lens"], st["table"], st["pages"], c["page"], c["hd"],
                       rope_table=st.get("rope"), q=st.get("q"), q_out=st.get("q_out"))
    R.cb_paged4_gather(st["offsets"], st["lens"], st["table"], st["pages"], c["page"], c["hd"], st["k_back"],
                       st["v_back"])
    return {"k": st["k_back"], "v": st["v_back"], "q": st.get("q_out")}


def _own_attention4(st):
    import rag_kv_cache_layer_gb300 as R
    c = st["case"]
    if "ws" not in st:      # the scratch that a serving loop keeps from step to step
        st["ws"] = R.cb_paged4_attention_workspace(st["q"], c["seqs"], st["max_kv"], c["hq"], c["hkv"], c["hd"])
    R.cb_paged4_attention(st["q"], st["offsets"], st["lens"], st["table"], st["pages"], c["page"], c["hq"], c["hkv"],
                          c["hd"], st["out"], max_kv_len=st["max_kv"], ws=st["ws"])
    return st["out"]


def _own_select(st):
    import rag_kv_cache_layer_gb300 as R
    c = st["case"]
    if "ws" not in st:
        st["ws"] = R.cb_paged_select_workspace(st["q"], st["max_kv"], c["page"], c["hkv"])
    R.cb_paged_bounds(st["offsets"], st["lens"], st["table"], st["k_pages"], st["bounds"], st["q"].shape[0])
    R.cb_paged_select(st["q"], st["offsets"], st["lens"], st["table"], st["bounds"], c["page"], c["hq"], c["hkv"],
                      c["hd"], st["picks"], n_first=FIRST, n_last=LAST, max_kv_len=st["max_kv"], ws=st["ws"])
    return {"bounds": st["bounds"], "picks": st["picks"]}


def _own_picked(st):
    import rag_kv_cache_layer_gb300 as R
    c = st["case"]
    if "ws" not in st:
        st["ws"] = R.cb_paged_attention_picked_workspace(st["q"], c["picks"], c["page"], c["hq"], c["hkv"], c["hd"])
    R.cb_paged_attention_picked(st["q"], st["offsets"], st["lens"], st["table"], st["k_pages"], st["v_pages"],
                                st["picks"], c["hq"], c["hkv"], c["hd"], st["out"], ws=st["ws"])
    return st["out"]


def _row_place(st):
    """Sequence, index in it and position of every new row, from the device's offsets and lengths."""
    off, lens, rows = st["offsets"].long(), st["lens"].long(), (st["k"] if "k" in st else st["q"]).shape[-2]
    r = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(off, r, right=True) - 1
    at = r - off[seq]
    return seq, at, lens[seq] - (off[seq + 1] - off[seq]) + at


def _power(e):
    """2^e in 64 bits, exactly (torch's pow and ldexp need not be)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _rounded(x, lowest, bits):
    """x >= 0 to the nearest float of `bits` mantissa bits, exponents from `lowest`; ties to even (64 bits: exact)."""
    e = (torch.frexp(x).exponent - 1).clamp(min=lowest)
    step = _power(e - bits)
    return torch.round(x / step) * step


def _quantised(x):
    """Codes' values and scales of x [..., 16] (64 bits): scale a/6 as an 8-bit float, a the largest magnitude."""
    six = torch.full((1,), 6.0, dtype=x.dtype, device="cuda")      # (by a plain number torch multiplies with its inverse)
    scale = _rounded(x.abs().amax(-1, keepdim=True) / six, -6, 3).clamp(2.0 ** -9, 448.0)
    return _rounded((x / scale).abs(), 0, 1).clamp(max=6.0).copysign(x), scale


def _code_bytes(values):
    """Two codes' bytes of values [..., even]."""
    steps = torch.tensor(CODES[:8], dtype=torch.float64, device="cuda")
    code = torch.searchsorted(steps, values.abs()) + 8 * torch.signbit(values).long()
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)


def _page_places(c):
    """Of a slot's codes of keys and values, and of its scales, the places in a page."""
    page, hkv, hd = c["page"], c["hkv"], c["hd"]
    slot, h = torch.arange(page, device="cuda")[:, None, None], torch.arange(hkv, device="cuda")[None, :, None]
    base, d, e = h * (page * hd * 9 // 8), torch.arange(hd // 2, device="cuda"), torch.arange(hd // 16, device="cuda")
    kc, ks = base + slot * (hd // 2) + d, base + page * hd + slot * (hd // 16) + e
    return kc.flatten(1), kc.flatten(1) + page * hd // 2, ks.flatten(1), ks.flatten(1) + page * hd // 16


def _values(code_bytes, scale_bytes, hd):
    """The values that codes [..., heads * hd / 2] and scales [..., heads * hd / 16] stand for (32 bits hold them)."""
    table = torch.tensor(CODES, device="cuda")
    x = torch.stack([table[(code_bytes & 15).int()], table[(code_bytes >> 4).int()]], dim=-1)
    s = scale_bytes.view(torch.float8_e4m3fn).float()
    return (x.flatten(-2).unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _plain_store(st):
    c = st["case"]
    hd, page = c["hd"], c["page"]
    seq, _, pos = _row_place(st)
    live = (pos >= 0).nonzero()[:, 0]
    at = pos[live]
    pg, slot = st["table"].long()[seq[live], at // page], at % page

    def rotated(x):
        # 64 bits: a key next to a border between two codes has to fall on its own side
        cs = st["rope"][at].double()
        a, b = x[live].double().unflatten(-1, (-1, 2, hd // 2)).unbind(-2)
        cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-2).flatten(-3)
        # at once, not by way of 32 bits, to 8 significant bits
        return (_rounded(y.abs(), -126, 7).copysign(y) if x.dtype == torch.bfloat16 else y).to(x.dtype)

    lead = (slice(None),) if c["layers"] > 1 else ()
    kcp, vcp, ksp, vsp = _page_places(c)
    for x, cp, sp, back in ((rotated(st["k"]) if c["rotate"] else st["k"][lead + (live,)], kcp, ksp, st["k_back"]),
                            (st["v"][lead + (live,)], vcp, vsp, st["v_back"])):
        values, scales = _quantised(x.double().unflatten(-1, (-1, 16)))
        codes, scales = _code_bytes(values).flatten(-2), scales.flatten(-2).float().to(torch.float8_e4m3fn).view(torch.uint8)
        st["pages"][lead + (pg[:, None], cp[slot])] = codes
        st["pages"][lead + (pg[:, None], sp[slot])] = scales
        back[lead + (live,)] = _values(st["pages"][lead + (pg[:, None], cp[slot])],
                                       st["pages"][lead + (pg[:, None], sp[slot])], hd).to(x.dtype)
    if c["rotate"]:
        st["q_out"][live] = rotated(st["q"])
    return {"k": st["k_back"], "v": st["v_back"], "q": st.get("q_out")}


def _plain_attention4(st):
    c = st["case"]
    hq, hkv, hd, page, s, n, m = c["hq"], c["hkv"], c["hd"], c["page"], c["seqs"], c["n_new"], st["max_kv"]
    seq, at, pos = _row_place(st)
    j = torch.arange(m, device="cuda")
    held = -(-m // page)
    pages = st["pages"].view(-1, hkv, page * hd * 9 // 8)[st["table"].long()[:, :held]]     # [s, pages, hkv, bytes]
    there = (j[None, :] < st["lens"].long()[:, None])[:, None, :, None]

    def cache(code_at, scale_at):
        codes = pages[..., code_at:code_at + page * hd // 2].unflatten(-1, (page, -1))
        scales = pages[..., scale_at:scale_at + page * hd // 16].unflatten(-1, (page, -1)).contiguous()
        x = _values(codes, scales, hd).transpose(1, 2).reshape(s, hkv, held * page, hd)[:, :, :m]
        return torch.where(there, x, torch.zeros((), device="cuda"))

    q = torch.zeros(s, n, hq, hd, device="cuda")
    q[seq, at] = st["q"].float().view(-1, hq, hd)
    last = torch.full((s, n), -1, device="cuda", dtype=torch.long)
    last[seq, at] = pos
    q = q.view(s, n, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4).reshape(s, hkv, -1, hd)
    x = torch.matmul(q, cache(0, page * hd).transpose(2, 3)).view(s, hq, n, m).mul_(1.0 / math.sqrt(hd))
    x.masked_fill_(j[None, None, None, :] > last[:, None, :, None], -math.inf)
    x, total = _softmax_parts(x)
    o = torch.matmul(x.view(s, hkv, -1, m), cache(page * hd // 2, page * hd + page * hd // 16)).view(s, hq, n, hd)
    o = torch.where(total > 0, o / total, torch.zeros((), device="cuda")).permute(0, 2, 1, 3)
    return o[seq, at].reshape(-1, hq * hd).to(st["q"].dtype)


def _softmax_parts(x):
    """exp(x - max) in place, and its sums (0 where every x is -inf)."""
    x.sub_(x.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)).exp_()
    return x, x.sum(dim=-1, keepdim=True)


def _plain_select(st):
    c = st["case"]
    hq, hkv, hd, page, k = c["hq"], c["hkv"], c["hd"], c["page"], c["picks"]
    seq, _, pos = _row_place(st)
    lens = st["lens"].long()
    # bounds of the pages that hold new rows, over the slots up to the length
    live = (pos >= 0).nonzero()[:, 0]
    lp = pos[live] // page
    pg = st["table"].long()[seq[live], lp]
    there = (lp[:, None] * page + torch.arange(page, device="cuda") < lens[seq[live]][:, None])[..., None]
    x = st["k_pages"][pg]
    st["bounds"][pg, 0] = torch.where(there, x, math.inf).amin(1)
    st["bounds"][pg, 1] = torch.where(there, x, -math.inf).amax(1)
    # the largest dot product that a page's bounds allow, over the group's heads; 64 bits, since
    # a border lies between two neighbours of thousands
    held = -(-st["max_kv"] // page)
    b = st["bounds"][st["table"].long()[:, :held]].double().unflatten(-1, (hkv, hd))        # [s, pages, 2, hkv, hd]
    q = st["q"].double().view(-1, hkv, hq // hkv, hd)
    rows, n = len(q), c["n_new"]
    at = torch.arange(rows, device="cuda") - st["offsets"].long()[seq]
    qs = torch.zeros(c["seqs"], n, hkv, hq // hkv, hd, dtype=torch.float64, device="cuda")
    qs[seq, at] = q
    qs = qs.permute(0, 2, 1, 3, 4).flatten(2, 3)                                            # [s, hkv, n * g, hd]
    lo, hi = (b[:, :, i].permute(0, 2, 3, 1) for i in (0, 1))
    x = torch.matmul(qs.clamp(min=0), hi) + torch.matmul(qs.clamp(max=0), lo)
    x = x.unflatten(2, (n, -1)).amax(3).permute(0, 2, 1, 3)[seq, at]                        # [rows, hkv, pages]
    j = torch.arange(held, device="cuda")
    pages = torch.div(pos, page, rounding_mode="floor")[:, None, None] + 1
    x = torch.where((j < FIRST) | (j >= pages - LAST), math.inf, x)
    x = torch.where(j < pages, x, -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :k]
    got = torch.where(order < pages, order, 1 << 30).sort(dim=-1).values
    st["picks"].fill_(-1)
    st["picks"][..., :got.shape[-1]] = torch.where(got < 1 << 30, got, -1).to(torch.int32)
    return {"bounds": st["bounds"], "picks": st["picks"]}


def _plain_picked(st):
    c = st["case"]
    hq, hkv, hd, page = c["hq"], c["hkv"], c["hd"], c["page"]
    seq, _, pos = _row_place(st)
    picks = st["picks"].long()
    rows, k = len(seq), picks.shape[-1]
    key = (picks[..., None] * page + torch.arange(page, device="cuda")).flatten(2)          # [rows, hkv, keys]
    seen = (picks[..., None] >= 0).expand(-1, -1, -1, page).flatten(2) & (key <= pos[:, None, None])
    pg = st["table"].long()[seq[:, None, None], picks.clamp(min=0)]
    h = torch.arange(hkv, device="cuda")[None, :, None]

    def cache(pages):
        x = pages.view(-1, page, hkv, hd)[pg, :, h].flatten(2, 3).float()                   # [rows, hkv, keys, hd]
        return torch.where(seen[..., None], x, torch.zeros((), device="cuda"))

    q = st["q"].float().view(rows, hkv, hq // hkv, hd)
    x = torch.matmul(q, cache(st["k_pages"]).transpose(2, 3)).mul_(1.0 / math.sqrt(hd))
    x.masked_fill_(~seen[:, :, None], -math.inf)
    x, total = _softmax_parts(x)
    o = torch.matmul(x, cache(st["v_pages"]))
    return torch.where(total > 0, o / total, torch.zeros((), device="cuda")).view(rows, -1).to(st["q"].dtype)


# ------------------------------------------------------------------ work --
def work(case):
    eb, lens = BYTES[case["dtype"]], _lengths(case)
    hq, hkv, hd, page = case["hq"], case["hkv"], case["hd"], case["page"]
    kvw = hkv * hd
    live = sum(n for n, kv in lens if kv > 0)
    rows = sum(n for n, _ in lens)
    meta = 8 * len(lens) + 4 * sum(-(-kv // page) for _, kv in lens)
    if case["op"] == "store":
        # rows in, pages, rows back; the queries in and out
        per_row = (2 * kvw * (2 * eb + 9.0 / 16)) * case["layers"] + ((2 * hq * hd * eb + 4 * hd) if case["rotate"] else 0)
        return {"bytes": live * per_row + 12 * len(lens),
                "flops": live * ((3.0 * (hq + hkv) * hd if case["rotate"] else 0.0) + 4.0 * kvw * case["layers"])}
    if case["op"] == "attention4":
        pairs = sum(n * (kv - n) + n * (n + 1) // 2 for n, kv in lens if kv > 0)
        return {"bytes": 2 * kvw * 9 / 16 * sum(kv for _, kv in lens) + 2 * rows * hq * hd * eb + meta,
                "flops": 4.0 * hd * hq * pairs}
    _, pos = _rows(case)
    pages = [p // page + 1 for p in pos if p >= 0]
    if case["op"] == "select":
        held = sum(-(-kv // page) for _, kv in lens)
        fresh = sum(kv - max(0, kv - n) // page * page for n, kv in lens)     # keys of the pages with new rows
        return {"bytes": (2 * held + fresh) * kvw * eb + rows * (hq * hd * eb + 4 * hkv * case["picks"]) + meta,
                "flops": 4.0 * hd * hq * sum(pages)}
    keys = sum(min(p + 1, case["picks"] * page) for p in pos)
    whole = sum(kv for _, kv in lens)
    return {"bytes": 2 * kvw * eb * min(keys, whole) + 2 * rows * hq * hd * eb + 4 * rows * hkv * case["picks"],
            "flops": 4.0 * hd * hq * keys}


# ----------------------------------------------------------------- exact --
def exact(case, seed):
    st = prepare(case, seed)
    return {"store": _exact_store, "attention4": _exact_attention4, "select": _exact_select,
            "picked": _exact_picked}[case["op"]](st)


def _exact_scale(a):
    """The nearest of the 8-bit floats to a/6 (ties to even, never zero): between neighbours by 6 times their mean."""
    grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16)
                        for m in range(8)][:-1], dtype=torch.float64, device="cuda")
    border = 3.0 * (grid[1:] + grid[:-1])
    up, down = torch.searchsorted(border, a, right=True), torch.searchsorted(border, a, right=False)
    i = torch.where((up != down) & (up % 2 == 1), down, up)       # on a border: the even one
    return grid[i.clamp(min=1)]


def _exact_quantised(x):
    """The values that x [..., hd] (64 bits) gets in the 4-bit cache."""
    x = x.unflatten(-1, (-1, 16))
    scale = _exact_scale(x.abs().amax(-1))[..., None]
    grid = torch.tensor(CODES[:8], dtype=torch.float64, device="cuda")
    i = torch.zeros_like(x, dtype=torch.long)
    for k in range(7):
        border = scale * (0.5 * (grid[k] + grid[k + 1]))
        i += (x.abs() >= border) if k % 2 else (x.abs() > border)
    return (torch.sign(x) * grid[i] * scale).flatten(-2)


def _exact_store(st):
    c = st["case"]
    hd, half = c["hd"], c["hd"] // 2
    seq, pos = (torch.tensor(a, device="cuda") for a in _rows(c))
    live = (pos >= 0).nonzero()[:, 0]
    out = {}
    for name in ("k", "v"):
        y = torch.zeros(st[name].shape, dtype=torch.float64, device="cuda")
        x = st[name][..., live, :]
        if name == "k" and c["rotate"]:
            # as a cache of the rows' type would hold it
            mantissa, exponent = torch.frexp(_exact_turned(st, x, pos[live], half))
            bits = 256.0 if x.dtype == torch.bfloat16 else 2.0 ** 24
            x = torch.round(mantissa * bits) / bits * _power(exponent)
        for layer in range(c["layers"]):
            to, frm = (y, x) if c["layers"] == 1 else (y[layer], x[layer])
            to[live] = _exact_quantised(frm.double().unflatten(-1, (-1, hd))).flatten(-2)
        out[name] = y
    out["q"] = None
    if c["rotate"]:
        out["q"] = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        out["q"][live] = _exact_turned(st, st["q"][live], pos[live], half)
    return out


def _exact_turned(st, x, pos, half):
    turn = torch.view_as_complex(st["rope"][pos].double())[:, None]
    x = x.double().view(len(pos), -1, 2 * half)
    z = torch.complex(x[..., :half], x[..., half:]) * turn
    return torch.cat([z.real, z.imag], dim=-1).view(len(pos), -1)


def _exact_attention4(st):
    c = st["case"]
    hq, hkv, hd, page = c["hq"], c["hkv"], c["hd"], c["page"]
    g, out, row, part = hq // hkv, [], 0, page * hd // 2
    grid = torch.tensor(CODES, dtype=torch.float64, device="cuda")
    for s, (n, kv) in enumerate(_lengths(c)):
        q = st["q"][row:row + n].double().view(n, hq, hd)
        row += n
        o = torch.zeros(n, hq, hd, dtype=torch.float64, device="cuda")
        late = torch.arange(kv, device="cuda")[None, :] > torch.arange(kv - n, kv, device="cuda")[:, None]
        for h in range(hkv if kv > 0 else 0):
            one = st["pages"][st["table"][s, :-(-kv // page)].long()].view(-1, hkv, page * hd * 9 // 8)[:, h]
            kvs = []
            for i in range(2):
                b = one[:, i * part:(i + 1) * part].reshape(-1, hd // 2)[:kv].long()
                e = one[:, 2 * part + i * part // 8:2 * part + (i + 1) * part // 8].reshape(-1, hd // 16)[:kv].long()
                mant, ex = e % 8, e // 8 % 16
                scale = torch.where(ex == 0, mant * 2.0 ** -9, (8 + mant) * _power(ex - 10))
                x = grid[torch.stack([b % 16, b // 16], dim=-1).view(len(b), hd)]
                kvs.append(x * scale.double().repeat_interleave(16, dim=1))
            x = torch.einsum("ngd,jd->gnj", q[:, h * g:(h + 1) * g], kvs[0]) / math.sqrt(hd)
            x = torch.softmax(x.masked_fill(late, -math.inf), dim=-1)
            o[:, h * g:(h + 1) * g] = torch.einsum("gnj,jd->ngd", x, kvs[1])
        out.append(o.view(n, hq * hd))
    return torch.cat(out)


def _exact_select(st):
    c = st["case"]
    hq, hkv, hd, page = c["hq"], c["hkv"], c["hd"], c["page"]
    bounds, picks, row = st["bounds"].double(), torch.full_like(st["picks"], -1), 0
    for s, (n, kv) in enumerate(_lengths(c)):
        q = st["q"][row:row + n].double().view(n, hkv, hq // hkv, hd)
        row += n
        if kv == 0:
            continue
        pg = st["table"][s, :-(-kv // page)].long()
        for j in range((kv - n) // page, len(pg)):
            x = st["k_pages"][pg[j], :min(page, kv - j * page)].double()
            bounds[pg[j]] = torch.stack([x.min(0).values, x.max(0).values])
        for i in range(n):
            p = (kv - n + i) // page + 1
            b = bounds[pg[:p]].view(p, 2, hkv, 1, hd)
            x = torch.maximum(q[i] * b[:, 0], q[i] * b[:, 1]).sum(-1).amax(-1).t().contiguous()    # [hkv, p]
            x[:, :FIRST] = math.inf
            x[:, max(0, p - LAST):] = math.inf
            best = torch.argsort(-x, dim=-1, stable=True)[:, :c["picks"]]
            picks[row - n + i, :, :best.shape[1]] = best.sort(dim=-1).values.to(torch.int32)
    return {"bounds": bounds, "picks": picks}


def _exact_picked(st):
    c = st["case"]
    hq, hkv, hd, page = c["hq"], c["hkv"], c["hd"], c["page"]
    g, (seq, pos) = hq // hkv, _rows(c)
    picks = st["picks"].cpu()
    out = torch.zeros(len(seq), hq, hd, dtype=torch.float64, device="cuda")
    kp, vp = (st[a].view(-1, page, hkv, hd) for a in ("k_pages", "v_pages"))
    for r, (s, p) in enumerate(zip(seq, pos)):
        for h in range(hkv if p >= 0 else 0):
            pg = picks[r, h][(picks[r, h] >= 0)].long()
            keys = (pg[:, None] * page + torch.arange(page)).flatten()
            seen = (keys <= p).nonzero()[:, 0].cuda()
            at = st["table"][s, pg.cuda()].long()
            k, v = (x[at, :, h].double().flatten(0, 1)[seen] for x in (kp, vp))
            x = torch.softmax(st["q"][r].double().view(hq, hd)[h * g:(h + 1) * g] @ k.t() / math.sqrt(hd), dim=-1)
            out[r, h * g:(h + 1) * g] = x @ v
    return out.view(len(seq), -1)
