"""The variants of the paged attention that a call's sizes lead to, at sizes that
lead to each: the chunk kernel's units of 128 and 256 rows, whole and in parts,
over many key blocks, and the few-rows kernel's cut of its line of units.

cb_debug_paged_plan says which variant a call runs; every case states the one it
is here for, so that another plan shows up as a failure and not as a gap.  The
definition is evaluated in float64 on the device, at the bounds of
test_gpu_paged.py (for bf16 outputs)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from rag_kv_cache_layer_gb300 import _lib as L
from test_gpu_paged import F, HALF, Batch, attention_case, ints, vals
from test_paged_abi import _line

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield


def plan(rows, n_seq, max_kv, heads, dt):
    """few-rows tile, its heads per item, its blocks; chunk unit, key parts, units, the few-rows kernel's limit"""
    out = (C.c_int64 * 7)()
    L.check(L.lib.cb_debug_paged_plan(rows, n_seq, max_kv, *heads, L.CB_BF16 if dt == BF16 else L.CB_F32, out))
    return list(out)


def definition(q, dk, dv, b, heads, scale):
    """float64 outputs and their bounds, [rows, hq * hd], of the sequences' rows
    (elsewhere 9 and 0); dk and dv without poison."""
    hq, hkv, hd = heads
    G = hq // hkv
    want = torch.full((b.rows, hq, hd), 9.0, dtype=torch.float64, device="cuda")
    lim = torch.zeros_like(want)
    q = q.double().view(b.rows, hq, hd)
    u = HALF[BF16]
    for s, (n, kv) in enumerate(b.seqs):
        r0, lead = int(b.offsets[s]), max(0, n - kv)           # rows in front of position 0
        want[r0:r0 + lead], lim[r0:r0 + lead] = 0.0, 0.0
        if n == lead:
            continue
        j = np.arange(kv)
        pages, slots = (torch.from_numpy(x).cuda() for x in (b.table[s][j // b.page], j % b.page))
        K, V = (x[pages, slots].double().view(kv, hkv, hd) for x in (dk, dv))
        rows = slice(r0 + lead, r0 + n)
        p = torch.arange(kv - n + lead, kv, device="cuda")
        hidden = torch.arange(kv, device="cuda")[None] > p[:, None]
        for g in range(hkv):
            c = slice(g * G, (g + 1) * G)
            Q = q[rows, c].transpose(0, 1)
            w = torch.softmax((scale * (Q @ K[:, g].T)).masked_fill_(hidden, -math.inf), dim=-1)
            want[rows, c] = (w @ V[:, g]).transpose(0, 1)
            B = (w @ V[:, g].abs()).transpose(0, 1)
            A = (scale * (Q.abs() @ K[:, g].abs().T)).masked_fill_(hidden, 0.0).amax(-1).T[..., None]
            d = 2 * hd * F * A + 8 * F * (A + 1) + 4 * F
            lim[rows, c] = (2 * d + 2 * (p[:, None, None] + 1) * F) * B + u * want[rows, c].abs() + u * B
    return want.view(b.rows, -1), lim.view(b.rows, -1)


class Call:
    """A batch with its inputs, its definition and a workspace; run() checks."""

    def __init__(self, seed, heads, page, seqs, scale=None, std=1.0, tail=3):
        rng = np.random.default_rng(seed)
        hq, hkv, hd = self.heads = heads
        self.scale = hd ** -0.5 if scale is None else scale
        self.b = Batch(rng, seqs, page, BF16, hkv, hd, extra_cols=1, tail=tail)
        k, v, self.dk, self.dv = self.b.pools(rng)
        self.q = torch.from_numpy(vals(rng, (self.b.rows, hq * hd), BF16, std)).cuda().to(BF16)
        self.max_kv = max(kv for _, kv in seqs)
        clean = [torch.from_numpy(x).cuda().to(BF16) for x in (k, v)]
        self.want, self.lim = definition(self.q, *clean, self.b, heads, self.scale)
        self.ws = R.cb_paged_attention_workspace(self.q, len(seqs), self.max_kv, *heads)

    def plan(self):
        return plan(self.b.rows, len(self.b.seqs), self.max_kv, self.heads, BF16)

    def launch(self, table=None, ws=None):
        hq, hkv, hd = self.heads
        out = torch.full_like(self.q, 9.0)
        off, lens, tab = self.b.dev()
        R.cb_paged_attention(self.q, off, lens, tab if table is None else ints(table), self.dk, self.dv, hq, hkv, hd, out,
                             max_kv_len=self.max_kv, scale=self.scale, ws=self.ws if ws is None else ws)
        torch.cuda.synchronize()
        return out

    def check(self, out):
        err = (out.double() - self.want).abs()
        assert bool((err <= self.lim).all()), (float((err - self.lim).max()), (err > self.lim).nonzero()[:4].tolist())


# (heads, page, sequences): rows per unit, whether a unit's keys are in parts
CHUNKS = [
    # 256 rows, whole: last units of 96, 160, 184 and 18 rows, lengths off the 64-key blocks
    ((32, 8, 128), 16, [(984, 3001)], 256, False),
    ((32, 8, 128), 128, [(1000, 2000)], 256, False),
    ((24, 8, 64), 8, [(1000, 2047)], 256, False),
    ((24, 8, 64), 64, [(1030, 1999)], 256, False),
    ((32, 16, 64), 16, [(600, 3000)], 256, False),
    # several sequences with a start from nothing, idle slots, rows in front of position 0, drafts, single rows
    ((32, 8, 128), 16, [(1, 900), (500, 1801), (0, 5), (300, 300), (3, 0), (200, 150), (9, 1500), (1, 0)], 256, False),
    ((32, 16, 64), 32, [(1, 900), (500, 1801), (0, 5), (300, 300), (3, 0), (200, 150), (9, 1500), (1, 0)], 256, False),
    # 256 rows, in parts: last units of 176, 64, 88 and 132 rows
    ((32, 8, 128), 16, [(300, 9000)], 256, True),
    ((8, 2, 128), 64, [(2000, 4100)], 256, True),
    ((32, 16, 64), 8, [(300, 9001)], 256, True),
    ((24, 8, 64), 128, [(300, 9000)], 256, True),
    # the same with units that see fewer key blocks than there are parts
    ((32, 8, 128), 16, [(150, 9000), (150, 150)], 256, True),
    ((32, 16, 64), 16, [(300, 9000), (300, 300)], 256, True),
    # 128 rows, whole, over 20 and more key blocks
    ((32, 8, 128), 16, [(100, 1700 - 13 * i) for i in range(26)], 128, False),
    ((32, 16, 64), 32, [(100, 1700 - 13 * i) for i in range(26)], 128, False),
    ((8, 8, 128), 16, [(500, 1500), (700, 1400), (300, 1350)], 128, False),
    # 128 rows, in parts of more than eight blocks
    ((8, 2, 128), 16, [(400, 6000)], 128, True),
    ((4, 2, 64), 16, [(600, 9000)], 128, True),
]


@pytest.mark.parametrize("heads,page,seqs,unit,parts", CHUNKS)
def test_chunk_variants(heads, page, seqs, unit, parts):
    c = Call(len(seqs) + page, heads, page, seqs)
    p = c.plan()
    assert (p[3], p[4] > 1) == (unit, parts), p
    out = c.launch()
    assert R.device_status() == 0
    c.check(out)
    c.ws.fill_(255)                              # NaN in every record: nothing of it is read before it is written
    assert torch.equal(c.launch(), out)


@pytest.mark.parametrize("heads,seqs,parts", [
    ((32, 8, 128), [(1000, 2000)], False), ((32, 16, 64), [(600, 3000)], False),
    ((32, 8, 128), [(300, 9000)], True), ((32, 16, 64), [(300, 9000)], True)])
def test_chunk_variants_with_steep_scores(heads, seqs, parts):
    """The reference maximum of both tiles moves often, at different blocks."""
    c = Call(5, heads, 16, seqs, scale=1.5, std=2.0)
    p = c.plan()
    assert (p[3], p[4] > 1) == (256, parts), p
    c.check(c.launch())
    assert R.device_status() == 0


@pytest.mark.parametrize("heads", [(32, 8, 128), (32, 16, 64)])
@pytest.mark.parametrize("seqs,parts", [([(300, 1801), (260, 1700), (300, 1650)], False), ([(300, 9000), (300, 8000)], True)])
def test_chunk_variants_report_bad_pages(heads, seqs, parts):
    """A page outside the pool is recorded and not read; the other sequences keep
    their values."""
    c = Call(9, heads, 16, seqs)
    p = c.plan()
    assert (p[3], p[4] > 1) == (256, parts), p
    good = c.launch()
    assert R.device_status() == 0
    c.check(good)
    r0, r1 = int(c.b.offsets[1]), int(c.b.offsets[2])
    for bad in (c.b.n_pages, -1, 2 ** 31 - 1):
        t = c.b.table.copy()
        t[1, 37] = bad
        out = c.launch(table=t)
        assert R.device_status() == L.CB_ERR_DEVICE_INDEX
        assert torch.equal(out[:r0], good[:r0]) and torch.equal(out[r1:], good[r1:])


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("seqs", [[(1, 300)], [(3, 2), (1, 0), (2, 700)], [(150, 130)], [(90, 4000)], [(70, 70), (1, 500), (200, 260)]])
def test_a_scale_of_zero_averages_the_values(dt, heads, seqs):
    """Every visible key weighs the same, in blocks without a visible key too."""
    attention_case(np.random.default_rng(3), dt, heads, 16, seqs, scale=0.0)


# ------------------------------------------------------- the line of units --
def block_keys(dt, hd, tile):
    """Keys per block of the few-rows kernel."""
    per = 4096 // (2 if dt == BF16 else 4) // hd
    return 2 * per if dt != BF16 and tile == 64 and hd == 128 else per


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("seed", range(30))
def test_the_devices_cut_of_the_line(dt, seed):
    """The records that the few-rows kernel leaves for its join, against the
    partition that the CPU tests show to cover every unit once."""
    rng = np.random.default_rng(seed)
    hkv, G, hd = int(rng.choice([1, 2, 5, 8])), int(rng.choice([1, 2, 4, 7])), int(rng.choice([64, 128]))
    heads = hq, _, _ = (G * hkv, hkv, hd)
    seqs = []
    for _ in range([1, 3, 9, 70][seed % 4]):
        n = int(rng.choice([0, 1, 1, 2, 5, rng.integers(1, 200)])) if dt != BF16 else int(rng.choice([0, 1, 1, 1]))
        seqs.append((n, int(rng.choice([0, n, n // 2, n + rng.integers(0, 3000)]))))
    if not any(n for n, _ in seqs):
        seqs[0] = (1, 500)
    if dt == BF16 and len(seqs) > 8:                     # rows of several tiles, still one per sequence on average
        seqs[3] = (len(seqs) - sum(n for n, _ in seqs) + seqs[3][0], 400)
    b = Batch(rng, seqs, 16, dt, hkv, hd, extra_cols=1)
    max_kv = max(kv for _, kv in seqs)
    tile, hc, grid, unit, *_ = plan(b.rows, len(seqs), max_kv, heads, dt)
    assert tile and not unit                             # the few-rows kernel alone
    dk = torch.randn(b.n_pages, 16, b.kvw, device="cuda").to(dt)
    q = torch.randn(b.rows, hq * hd, device="cuda").to(dt)
    ws = R.cb_paged_attention_workspace(q, len(seqs), max_kv, *heads)
    R.cb_paged_attention(q, *b.dev(), dk, dk, *heads, torch.empty_like(q), max_kv_len=max_kv, ws=ws)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    at = 2 * grid * tile * hc * (4 * hd + 8)             # behind the partial rows and their (m, l)
    got = np.frombuffer(ws[at:at + 24 * grid].cpu().numpy().tobytes(), np.int32).reshape(grid, 6).tolist()
    _, _, joins = _line(seqs, hkv // hc, G, tile, block_keys(dt, hd, tile), grid, 4 if hc == 1 else 1)
    want = []
    for (s, k, g), slots in joins:
        c, second = divmod(slots[0], 2)
        want.append((c, [int(b.offsets[s]), k * tile, min(tile, seqs[s][0] * G - k * tile), g * hc,
                         slots[-1] // 2, second]))
    assert [(c, r) for c, r in enumerate(got) if r[2]] == sorted(want)
