"""Paged append and paged attention against their float64 definition: head
layouts, lengths from one row on, odd sizes, strides, idle slots, rows without
keys, garbage in unused slots, bad tables, graphs, streams.

Tolerances (u: half a step of the type, 2^-24 or 2^-8; F = 2^-24)
  append     y = a c - b s: the table's entries are off by F/2 each, the two
             products and the sum round in fp32: <= 3 F (|a| + |b|); the
             result rounds once: + u |y|.
  attention  a score is a sum of hd products: <= hd F A / 2 in any order of
             addition with A = scale sum |q_d k_d|; tensor-core sums may
             truncate (twice that).  With the base-2 exponential's 2^-22 and
             its argument's rounding, each probability is off by at most the
             factor d = 2 hd F A + 8 F (A + 1) + 4 F relative, its share of
             the sum by as much again; sums over n keys add n F.  So
             |err| <= (2 d + 2 n F) B, B = sum_j p_j |v_j|, + u |o| for the
             last rounding, and for bf16 + u B: probabilities are rounded to
             bf16 for the tensor cores."""
import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from gpu_common import bf16_values
from oracle import paged as OP
from rag_kv_cache_layer_gb300 import _lib as L

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BASE = 10000.0


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield


def vals(rng, shape, dt, std=1.0):
    x = (rng.standard_normal(shape) * std).astype(np.float32)
    return bf16_values(x) if dt == torch.bfloat16 else x


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """Sequences [(new rows, length)] with a page table over a shuffled pool."""

    def __init__(self, rng, seqs, page, dt, hkv, hd, extra_cols=0, spare=3, tail=0):
        self.seqs, self.page, self.dt, self.kvw, self.hd = seqs, page, dt, hkv * hd, hd
        need = [-(-kv // page) for _, kv in seqs]
        self.n_pages = sum(need) + spare
        perm = rng.permutation(self.n_pages)
        # entries past the needed ones are never read: they name no page
        self.table = np.full((len(seqs), max(1, max(need, default=0)) + extra_cols), -7, np.int64)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = perm[at:at + n]
            at += n
        self.offsets = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int64)
        self.lens = np.array([kv for _, kv in seqs], np.int64)
        self.rows = int(self.offsets[-1]) + tail

    def dev(self):
        return ints(self.offsets), ints(self.lens), ints(self.table)

    def pools(self, rng, poison=True):
        """K and V pools as float64 and device tensors; slots that hold no
        position are NaN on the device."""
        k, v = (vals(rng, (self.n_pages, self.page, self.kvw), self.dt) for _ in range(2))
        used = np.zeros((self.n_pages, self.page), bool)
        for s, (_, kv) in enumerate(self.seqs):
            j = np.arange(kv)
            used[self.table[s][j // self.page], j % self.page] = True
        dk, dv = (torch.from_numpy(x).cuda().to(self.dt) for x in (k, v))
        if poison:
            gone = torch.from_numpy(~used).cuda()
            dk[gone], dv[gone] = float("nan"), float("nan")
        return k.astype(np.float64), v.astype(np.float64), dk, dv


# ---------------------------------------------------------------- append --
APPEND = [
    ((4, 2, 64), 16, [(1, 1)]),
    ((32, 8, 128), 16, [(1, 3137)]),
    ((32, 8, 128), 8, [(1, 16), (1, 17), (1, 0), (1, 5000)]),
    ((7, 1, 64), 32, [(3, 3), (0, 9), (65, 70), (5, 2), (2, 0), (33, 64)]),
    ((5, 5, 16), 64, [(130, 1000), (1, 64), (64, 64)]),
    ((2, 1, 256), 128, [(17, 140)]),
    ((8, 8, 128), 16, [(1, 40 + i) for i in range(70)]),
]


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads,page,seqs", APPEND)
def test_append(dt, heads, page, seqs):
    hq, hkv, hd = heads
    rng = np.random.default_rng(hash((heads, page)) % 1000)
    b = Batch(rng, seqs, page, dt, hkv, hd, extra_cols=2, tail=3)
    k0, v0, dk, dv = b.pools(rng, poison=False)
    k, v, q = (vals(rng, (b.rows, w), dt) for w in (b.kvw, b.kvw, hq * hd))
    table = R.cb_rope_table_init(6000, hd, BASE)
    # rows live inside wider matrices, as slices of a fused projection would
    fused = torch.from_numpy(np.concatenate([q, k, v], 1)).cuda().to(dt)
    dq, dkn, dvn = fused[:, :hq * hd], fused[:, hq * hd:hq * hd + b.kvw], fused[:, hq * hd + b.kvw:]
    qo = torch.full((b.rows, hq * hd), 3.0, device="cuda", dtype=dt)
    R.cb_paged_append(dkn, dvn, *b.dev(), dk, dv, hd, rope_table=table, q=dq, q_out=qo)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    kp, vp = OP.paged_append(k0, v0, b.table, b.offsets, b.lens, k, v, hd, BASE)
    assert np.array_equal(f64(dv), vp)
    u = HALF[dt]
    # |a| + |b| of a pair, for every element of the pool that was written
    mag = np.zeros_like(kp)
    size = lambda x: np.tile(np.abs(x.reshape(len(x), -1, 2, hd // 2)).sum(2, keepdims=True), (1, 1, 2, 1)).reshape(len(x), -1)
    place = OP.row_positions(b.offsets, b.lens)
    for r, s, p in place:
        if p >= 0:
            mag[b.table[s][p // page], p % page] = size(k[r:r + 1].astype(np.float64))[0]
    err = np.abs(f64(dk) - kp)
    assert np.all(err <= 3 * F * mag + np.where(mag > 0, u * np.abs(kp), 0)), err.max()
    want = np.full((b.rows, hq * hd), 3.0)
    lim = np.zeros_like(want)
    for r, s, p in place:
        if p >= 0:
            x = q[r:r + 1].astype(np.float64)
            want[r] = OP.rope_rotate(x, [p], hd, BASE)[0]
            lim[r] = 3 * F * size(x)[0] + u * np.abs(want[r])
    err = np.abs(f64(qo) - want)
    assert np.all(err <= lim), (err - lim).max()


@pytest.mark.parametrize("dt", list(HALF))
def test_append_in_place_and_keys_alone(dt):
    rng = np.random.default_rng(5)
    b = Batch(rng, [(3, 20), (2, 2)], 8, dt, 2, 64)
    _, _, dk, dv = b.pools(rng, poison=False)
    dk2, dv2 = dk.clone(), dv.clone()
    k, v, q = (torch.from_numpy(vals(rng, (5, w), dt)).cuda().to(dt) for w in (128, 128, 256))
    table = R.cb_rope_table_init(64, 64, BASE)
    out = torch.empty_like(q)
    R.cb_paged_append(k, v, *b.dev(), dk, dv, 64, rope_table=table, q=q, q_out=out)
    R.cb_paged_append(k, v, *b.dev(), dk2, dv2, 64, rope_table=table)
    assert torch.equal(dk, dk2) and torch.equal(dv, dv2)
    R.cb_paged_append(k, v, *b.dev(), dk2, dv2, 64, rope_table=table, q=q)      # in place
    assert torch.equal(q, out) and torch.equal(dk, dk2)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("layers,rows,page", [(1, 5, 8), (3, 131, 16), (7, 40, 64)])
def test_append_layers_without_rotation(dt, layers, rows, page):
    """A fused cache of several layers moves into pages bit for bit."""
    rng = np.random.default_rng(layers)
    b = Batch(rng, [(rows, rows + 3)], page, dt, 2, 64)
    big = torch.from_numpy(vals(rng, (layers, rows + 9, 128), dt)).cuda().to(dt)
    k, v = big[:, 4:4 + rows], big[:, 9:]                     # strided layers
    kp = torch.full((layers, b.n_pages, page, 128), 2.0, dtype=dt, device="cuda")
    vp = torch.full_like(kp, 5.0)
    if layers == 1:
        R.cb_paged_append(k[0], v[0], *b.dev(), kp[0], vp[0], 64)
    else:
        R.cb_paged_append(k, v, *b.dev(), kp, vp, 64)
    want_k, want_v = torch.full_like(kp, 2.0), torch.full_like(kp, 5.0)
    pos = torch.arange(3, rows + 3)
    pg, sl = torch.from_numpy(b.table[0])[pos // page].cuda(), (pos % page).cuda()
    want_k[:, pg, sl], want_v[:, pg, sl] = k, v
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    assert R.device_status() == 0


def test_append_reports_bad_pages_positions_and_offsets():
    rng = np.random.default_rng(9)
    dt, table = torch.bfloat16, R.cb_rope_table_init(32, 64, BASE)
    k = torch.from_numpy(vals(rng, (4, 128), dt)).cuda().to(dt)

    def run(offsets, lens, tbl, rope=table):
        kp = torch.zeros(4, 8, 128, dtype=dt, device="cuda")
        vp = torch.zeros_like(kp)
        R.cb_paged_append(k, k, ints(offsets), ints(lens), ints(tbl), kp, vp, 64, rope_table=rope)
        torch.cuda.synchronize()
        return R.device_status(), (vp != 0).any(-1).nonzero().tolist()
    assert run([0, 2, 4], [2, 3], [[1], [0]]) == (0, [[0, 1], [0, 2], [1, 0], [1, 1]])
    # a page outside the pool: its rows are skipped, the others stored
    assert run([0, 2, 4], [2, 3], [[4], [0]]) == (L.CB_ERR_DEVICE_INDEX, [[0, 1], [0, 2]])
    assert run([0, 2, 4], [2, 3], [[-1], [0]]) == (L.CB_ERR_DEVICE_INDEX, [[0, 1], [0, 2]])
    # a position past the table's pages
    assert run([0, 2, 4], [9, 3], [[1], [0]]) == (L.CB_ERR_DEVICE_INDEX, [[0, 1], [0, 2], [1, 7]])
    # a rotation past the RoPE table
    assert run([0, 4], [40], [[0, 1, 2, 3, 0]]) == (L.CB_ERR_DEVICE_INDEX, [])
    # offsets that do not ascend or leave the rows
    assert run([0, 3, 2], [3, 3], [[1], [0]])[0] == L.CB_ERR_DEVICE_INDEX
    assert run([0, 9, 9], [9, 3], [[1], [0]]) == (L.CB_ERR_DEVICE_INDEX, [])


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("offsets,kept", [
    ([0, 5, 3, 10], [0]),                       # a sequence without rows, which no row's search meets
    ([0, 5, 5, 3, 10], [0, 1]),
    ([0, 4, 12, 4, 10], [0]),                   # past the rows, then back
    ([0, 0, -1, 2, 10], [0, 3]),
    ([-2, 3, 6, 10], [1, 2]),                   # a bad first sequence, good ones behind it
    ([0, 3, 6, 11], [0, 1]),
    ([10, 0, 0, 0], []),                        # a descent in front of empty sequences alone
    ([0, 3, 3, 7, 10], [0, 1, 2, 3]),           # ascending: nothing to record
])
def test_append_records_every_bad_offset(dt, offsets, kept):
    """Offsets that do not ascend inside the rows are recorded wherever they
    stand; sequences in order keep their rows, the others' are skipped."""
    rng = np.random.default_rng(11)
    n_seq, rows, page = len(offsets) - 1, 10, 8
    k = torch.from_numpy(vals(rng, (rows, 128), dt)).cuda().to(dt)
    kp, vp = (torch.zeros(2 * n_seq, page, 128, dtype=dt, device="cuda") for _ in range(2))
    table = np.arange(2 * n_seq).reshape(n_seq, 2)
    lens = [max(0, min(b - a, 16)) for a, b in zip(offsets, offsets[1:])]
    R.cb_paged_append(k, k, ints(offsets), ints(lens), ints(table), kp, vp, 64)
    torch.cuda.synchronize()
    good = len(kept) == n_seq
    assert R.device_status() == (0 if good else L.CB_ERR_DEVICE_INDEX)
    want = torch.zeros_like(kp)
    for s in kept:
        a, b = offsets[s], offsets[s + 1]
        want[2 * s:2 * s + 2].view(-1, 128)[:b - a] = k[a:b]
    assert torch.equal(kp, want) and torch.equal(vp, want)


# ------------------------------------------------------------- attention --
def attention_case(rng, dt, heads, page, seqs, tail=0, std=1.0, **kw):
    hq, hkv, hd = heads
    b = Batch(rng, seqs, page, dt, hkv, hd, extra_cols=1, tail=tail)
    k, v, dk, dv = b.pools(rng)
    q = vals(rng, (b.rows, hq * hd), dt, std)
    out = torch.full((b.rows, hq * hd), 9.0, dtype=dt, device="cuda")
    R.cb_paged_attention(torch.from_numpy(q).cuda().to(dt), *b.dev(), dk, dv, hq, hkv, hd, out, **kw)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    scale = kw.get("scale", hd ** -0.5)
    check_attention(out, q, k, v, b, heads, scale, dt)
    return b, q, k, v, dk, dv, out


def check_attention(out, q, k, v, b, heads, scale, dt):
    hq, hkv, hd = heads
    start = np.full((b.rows, hq * hd), 9.0)
    args = (b.table, b.offsets, b.lens, hq, hkv, hd)
    want = OP.paged_attention(q, k, v, *args, scale, start)
    B = OP.paged_attention(q, k, np.abs(v), *args, scale, np.zeros_like(start))
    lim = np.zeros_like(start)
    u = HALF[dt]
    for s, (n, kv) in enumerate(b.seqs):
        j = np.arange(kv)
        K = np.abs(k[b.table[s][j // b.page], j % b.page]).reshape(kv, hkv, hd) if kv else np.zeros((0, hkv, hd))
        for i in range(n):
            r, p = b.offsets[s] + i, kv - n + i
            for h in range(hq):
                c = slice(h * hd, (h + 1) * hd)
                if p < 0:
                    continue
                A = scale * (K[:p + 1, h // (hq // hkv)] @ np.abs(q[r, c].astype(np.float64))).max()
                d = 2 * hd * F * A + 8 * F * (A + 1) + 4 * F
                lim[r, c] = (2 * d + 2 * (p + 1) * F) * B[r, c] + u * np.abs(want[r, c])
                if dt == torch.bfloat16:
                    lim[r, c] += u * B[r, c]
    err = np.abs(f64(out) - want)
    assert np.all(err <= lim), (float((err - lim).max()), np.argwhere(err > lim)[:4].tolist())


ATTN = [
    # one row per sequence
    ((32, 8, 128), 16, [(1, 1)]),
    ((32, 8, 128), 16, [(1, 700)]),
    ((4, 2, 64), 8, [(1, 33), (1, 0), (1, 64), (1, 65), (1, 200)]),
    ((7, 1, 128), 32, [(1, 129), (1, 31), (1, 32)]),
    ((3, 3, 64), 64, [(1, 100)] * 5),
    ((16, 1, 64), 16, [(1, 257)]),
    ((40, 1, 128), 128, [(1, 300), (1, 2)]),
    ((128, 1, 64), 16, [(1, 70)]),
    # a few rows
    ((8, 2, 128), 16, [(2, 2), (4, 100), (3, 65)]),
    ((28, 4, 128), 32, [(5, 90), (2, 33)]),
    # chunks
    ((8, 2, 128), 16, [(64, 200)]),
    ((8, 2, 128), 64, [(129, 129), (1, 300), (40, 400)]),
    ((4, 4, 64), 32, [(130, 260), (17, 17)]),
    ((6, 2, 128), 128, [(50, 333), (43, 43)]),
    ((12, 1, 64), 8, [(23, 71)]),
    # rows without keys: idle slots, sequences without rows, lengths below the rows
    ((8, 2, 64), 16, [(1, 0), (0, 40), (1, 0)]),
    ((8, 2, 128), 16, [(70, 50), (0, 0), (3, 1), (1, 0), (20, 90)]),
    ((4, 2, 64), 256, [(90, 0), (10, 600)]),
]


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads,page,seqs", ATTN)
def test_attention(dt, heads, page, seqs):
    rng = np.random.default_rng(len(seqs) + page + sum(heads))
    attention_case(rng, dt, heads, page, seqs, tail=2)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 2, 64)])
@pytest.mark.parametrize("n", [1, 3, 9, 33, 100])
@pytest.mark.parametrize("kv", [1100, 2049])
def test_attention_split_over_long_keys(dt, heads, n, kv):
    """Few tiles over many keys: the range is split and joined."""
    rng = np.random.default_rng(n + kv)
    attention_case(rng, dt, heads, 32, [(n, kv)], std=2.0)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads,page", [((8, 8, 128), 16), ((32, 16, 64), 64), ((32, 16, 64), 8)])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_attention_long_loops(dt, heads, page, n):
    """Enough tiles that no range is split far: every stage is used many times."""
    rng = np.random.default_rng(n)
    seqs = [(n, int(rng.integers(1500, 4500))) for _ in range(26)]
    attention_case(rng, dt, heads, page, seqs if n < 20 else seqs[:8])


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads", [(8, 2, 128), (7, 1, 64), (5, 1, 128)])
def test_attention_mixed_lengths_in_one_call(dt, heads):
    """Generated tokens, drafts, idle slots and chunks in one batch."""
    rng = np.random.default_rng(heads[0])
    seqs = [(1, 900), (150, 700), (1, 0), (9, 10), (64, 64), (1, 1), (0, 5), (33, 2000), (16, 300), (1, 65)]
    attention_case(rng, dt, heads, 16, seqs, tail=5)


@pytest.mark.parametrize("dt", list(HALF))
def test_attention_many_sequences(dt):
    rng = np.random.default_rng(77)
    seqs = [(int(rng.integers(0, 4)), int(rng.integers(0, 60))) for _ in range(300)]
    attention_case(rng, dt, (4, 2, 64), 16, seqs)


@pytest.mark.parametrize("dt", list(HALF))
def test_full_batch_of_padded_slots(dt):
    """The most sequences of a call, two thirds of them idle or without rows."""
    rng = np.random.default_rng(5)
    seqs = [[(1, int(rng.integers(1, 90))), (1, 0), (0, 0)][i % 3] for i in range(L.CB_MAX_SEQS)]
    attention_case(rng, dt, (4, 2, 64), 16, seqs, tail=3)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("n", [1, 20, 200])
def test_table_without_pages(dt, n):
    """A batch of idle slots may come with a table of no columns: zeros."""
    kp = torch.full((1, 16, 128), float("nan"), dtype=dt, device="cuda")
    q = torch.randn(2 * n, 256, device="cuda").to(dt)
    out = torch.full_like(q, 9.0)
    table = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    R.cb_paged_attention(q, ints([0, n, 2 * n]), ints([0, 0]), table, kp, kp, 4, 2, 64, out)
    assert torch.all(out == 0) and R.device_status() == 0


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("n", [1, 6, 70])
def test_attention_steep_scores(dt, n):
    """Scores far apart: the running maximum moves, most weights vanish."""
    rng = np.random.default_rng(n)
    attention_case(rng, dt, (8, 2, 128), 16, [(n, 500)], scale=3.0)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("n", [1, 40])
def test_attention_strided_pool_and_rows(dt, n):
    """K and V interleaved page by page in one pool, slots with a gap, q and
    out as columns of wider matrices, sequences that share prefix pages."""
    rng = np.random.default_rng(3)
    hq, hkv, hd, page = 8, 2, 128, 16
    b = Batch(rng, [(n, 100), (n, 101)], page, dt, hkv, hd)
    b.table[1, :6] = b.table[0, :6]
    k, v, dk, dv = b.pools(rng, poison=False)
    pool = torch.full((b.n_pages, 2, page, hkv * hd + 8), float("nan"), dtype=dt, device="cuda")
    pool[:, 0, :, :hkv * hd], pool[:, 1, :, :hkv * hd] = dk, dv
    q = vals(rng, (2 * n, hq * hd), dt)
    wide = torch.zeros(2 * n, hq * hd + 64, dtype=dt, device="cuda")
    wide[:, 32:32 + hq * hd] = torch.from_numpy(q).cuda().to(dt)
    out = torch.full((2 * n, hq * hd + 16), 9.0, dtype=dt, device="cuda")
    R.cb_paged_attention(wide[:, 32:32 + hq * hd], *b.dev(), pool[:, 0, :, :hkv * hd], pool[:, 1, :, :hkv * hd],
                         hq, hkv, hd, out[:, 8:8 + hq * hd])
    check_attention(out[:, 8:8 + hq * hd], q, k, v, b, (hq, hkv, hd), hd ** -0.5, dt)
    assert torch.all(out[:, :8] == 9) and torch.all(out[:, 8 + hq * hd:] == 9)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("n", [1, 50])
def test_attention_reports_bad_lengths_and_pages(dt, n):
    rng = np.random.default_rng(4)
    hq, hkv, hd, page = 8, 2, 64, 16
    b = Batch(rng, [(n, 60), (n, 64), (n, 61)], page, dt, hkv, hd)
    k, v, dk, dv = b.pools(rng)
    q = vals(rng, (3 * n, hq * hd), dt)
    dq = torch.from_numpy(q).cuda().to(dt)

    def run(offsets=b.offsets, lens=b.lens, table=b.table, **kw):
        out = torch.full((3 * n, hq * hd), 9.0, dtype=dt, device="cuda")
        R.cb_paged_attention(dq, ints(offsets), ints(lens), ints(table), dk, dv, hq, hkv, hd, out, **kw)
        torch.cuda.synchronize()
        return R.device_status(), out
    ok, good = run()
    assert ok == 0
    keep = lambda out: torch.equal(out[:n], good[:n]) and torch.equal(out[2 * n:], good[2 * n:])
    # longer than the table, longer than the stated bound, negative: rows stay
    for lens, kw in (([60, 65, 61], {}), ([60, 64, 61], dict(max_kv_len=62)), ([60, -3, 61], {})):
        st, out = run(lens=lens, **kw)
        assert st == L.CB_ERR_DEVICE_INDEX and torch.all(out[n:2 * n] == 9)
        if not kw:
            assert keep(out)
    # a page outside the pool: the other sequences are not touched by it
    for page_id in (b.n_pages, -1, 2 ** 31 - 1):
        t = b.table.copy()
        t[1, 1] = page_id
        st, out = run(table=t)
        assert st == L.CB_ERR_DEVICE_INDEX and keep(out)
    # offsets out of order or past the rows
    st, out = run(offsets=[0, 2 * n, n, 3 * n])
    assert st == L.CB_ERR_DEVICE_INDEX
    st, out = run(offsets=[0, n, 2 * n, 3 * n + 1])
    assert st == L.CB_ERR_DEVICE_INDEX and torch.equal(out[:2 * n], good[:2 * n]) and torch.all(out[2 * n:] == 9)


def test_attention_and_append_past_32_bits():
    """The touched pages lie behind the first 2^32 elements of each pool."""
    rng = np.random.default_rng(6)
    hq, hkv, hd, page = 16, 8, 128, 16
    kvw = hkv * hd
    n_pages = (2 ** 32 // (page * kvw)) + 40
    kp = torch.empty(n_pages, page, kvw, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = np.arange(n_pages - 30, n_pages)[None]
    for n in (1, 37):
        kv = 400
        k, v = (vals(rng, (kv, kvw), torch.bfloat16) for _ in range(2))
        up = lambda x: torch.from_numpy(x).cuda().bfloat16()
        R.cb_paged_append(up(k), up(v), ints([0, kv]), ints([kv]), ints(table), kp, vp, hd)
        q = vals(rng, (n, hq * hd), torch.bfloat16)
        out = torch.zeros(n, hq * hd, dtype=torch.bfloat16, device="cuda")
        R.cb_paged_attention(up(q), ints([0, n]), ints([kv]), ints(table), kp, vp, hq, hkv, hd, out)
        b = Batch(rng, [(n, kv)], page, torch.bfloat16, hkv, hd)
        small = np.zeros((30, page, kvw)), np.zeros((30, page, kvw))
        for dst, src in zip(small, (k, v)):
            dst.reshape(-1, kvw)[:kv] = src
        b.table = np.arange(30)[None]
        check_attention(out, q, *small, b, (hq, hkv, hd), hd ** -0.5, torch.bfloat16)
    assert R.device_status() == 0


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("n", [1, 5, 70])
def test_repeatable_streams_and_graphs(dt, n):
    """Same bits again, on another stream, and from a recorded call that is
    replayed with other lengths; two recordings with a workspace each."""
    rng = np.random.default_rng(8)
    heads = (8, 2, 128)
    hq, hkv, hd = heads
    b = Batch(rng, [(n, 900), (n, 333)], 16, dt, hkv, hd)
    k, v, dk, dv = b.pools(rng, poison=False)
    q = torch.from_numpy(vals(rng, (2 * n, hq * hd), dt)).cuda().to(dt)
    off, lens, table = b.dev()
    out = torch.zeros_like(q)
    R.cb_paged_attention(q, off, lens, table, dk, dv, hq, hkv, hd, out, max_kv_len=900)
    again = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = R.cb_paged_attention_workspace(q, 2, 900, hq, hkv, hd)
    R.cb_paged_attention(q, off, lens, table, dk, dv, hq, hkv, hd, again, max_kv_len=900, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, again)
    outs = [torch.zeros_like(q) for _ in range(2)]
    wss = [torch.empty_like(ws) for _ in range(2)]
    graphs = []
    for o, w in zip(outs, wss):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            R.cb_paged_attention(q, off, lens, table, dk, dv, hq, hkv, hd, o, max_kv_len=900, ws=w)
        graphs.append(g)
    s2 = torch.cuda.Stream()
    for g, st in zip(graphs, (s, s2)):
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)
    lens.copy_(ints([n + 5, 200]))                # shorter now: the replay reads the new lengths
    graphs[0].replay()
    torch.cuda.synchronize()
    b.lens, b.seqs = np.array([n + 5, 200]), [(n, n + 5), (n, 200)]
    check_attention(outs[0], f64(q), k, v, b, heads, hd ** -0.5, dt)
    assert R.device_status() == 0


def test_own_workspace_belongs_to_the_calls_stream(monkeypatch):
    """The scratch a call allocates itself is not handed to the current
    stream's tensors while the call runs on another stream."""
    from rag_kv_cache_layer_gb300 import api
    plain, where = api.cb_paged_attention_workspace, []

    def noted(*args):
        w = plain(*args)
        where.append(w.data_ptr())
        return w
    monkeypatch.setattr(api, "cb_paged_attention_workspace", noted)
    rng = np.random.default_rng(12)
    heads, dt = (8, 2, 128), torch.bfloat16
    hq, hkv, hd = heads
    b = Batch(rng, [(1, 2000), (1, 700)], 16, dt, hkv, hd)
    k, v, dk, dv = b.pools(rng)
    q = vals(rng, (2, hq * hd), dt)
    dq = torch.from_numpy(q).cuda().to(dt)
    off, lens, table = b.dev()
    out = torch.full_like(dq, 9.0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    R.cb_paged_attention(dq, off, lens, table, dk, dv, hq, hkv, hd, out, max_kv_len=2000, stream=s)
    need = plain(dq, 2, 2000, hq, hkv, hd).numel()
    others = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(o.data_ptr() != where[0] for o in others)
    torch.cuda.synchronize()
    check_attention(out, q, k, v, b, heads, hd ** -0.5, dt)


def test_wrappers_refuse_shapes_and_types():
    dt = torch.bfloat16
    kp = torch.zeros(4, 16, 128, dtype=dt, device="cuda")
    off, lens, table = ints([0, 1]), ints([1]), ints([[0]])
    q, out = torch.zeros(1, 256, dtype=dt, device="cuda"), torch.zeros(1, 256, dtype=dt, device="cuda")
    good = dict(q=q, row_offsets=off, kv_lens=lens, block_table=table, k_pages=kp, v_pages=kp, n_q_heads=4,
                n_kv_heads=2, head_dim=64, out=out)
    R.cb_paged_attention(**good)
    for kw in (dict(q=q.float()), dict(out=out.float()), dict(kv_lens=lens.long()), dict(row_offsets=ints([0])),
               dict(block_table=ints([[0], [0]])), dict(v_pages=kp[:3]), dict(n_kv_heads=1), dict(q=q.cpu()),
               dict(k_pages=kp.float()), dict(q=q[:, ::2]), dict(k_pages=kp[None], v_pages=kp[None])):
        with pytest.raises(ValueError):
            R.cb_paged_attention(**{**good, **kw})
    k = torch.zeros(1, 128, dtype=dt, device="cuda")
    good = dict(k_new=k, v_new=k, row_offsets=off, kv_lens=lens, block_table=table, k_pages=kp,
                v_pages=torch.zeros_like(kp), head_dim=64)
    R.cb_paged_append(**good)
    for kw in (dict(k_new=k[:, :64]), dict(v_new=k.float()), dict(head_dim=48), dict(q_out=q), dict(k_new=k[None]),
               dict(rope_table=torch.zeros(64, device="cuda", dtype=torch.float64))):
        with pytest.raises(ValueError):
            R.cb_paged_append(**{**good, **kw})
    with pytest.raises(R._lib.CBError):
        R.cb_paged_append(**{**good, "q": q})      # a query and nothing to rotate it by
