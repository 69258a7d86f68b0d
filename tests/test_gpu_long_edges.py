"""Calls of the operators for long contexts that lie beside those of the other files: page
selections that take every page, errors in each of its kernels, factors at the ends of the
exponents, borders between many scores."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from gpu_common import bf16_values
from oracle import paged as OP
from oracle import paged4 as O4
from rag_kv_cache_layer_gb300 import _lib as L
from test_gpu_paged import Batch, f64, ints, vals
from test_gpu_paged4 import dev
from test_gpu_picked import picked_case, select_case

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
F = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("n", [4, 10, 16])
def test_select_records_errors_whether_or_not_pages_are_scored(dt, n):
    """Sequences of ten pages, fewer picks than those, as many and more: where every page fits,
    only the last of the selection's kernels runs."""
    bounds, q = torch.zeros(20, 2, 64, dtype=dt, device="cuda"), torch.ones(3, 64, dtype=dt, device="cuda")
    table = ints([list(range(10)), list(range(10, 20))])

    def run(offsets, lens, **kw):
        picks = torch.full((3, 1, n), -5, dtype=torch.int32, device="cuda")
        R.cb_paged_select(q, ints(offsets), ints(lens), table, bounds, 8, 1, 1, 64, picks, **kw)
        torch.cuda.synchronize()
        return R.device_status(), picks[:, 0].tolist()
    bad, old = L.CB_ERR_DEVICE_INDEX, [-5] * n
    ok = {4: [0, 1, 2, 9], 10: list(range(10)), 16: list(range(10)) + [-1] * 6}[n]
    assert run([0, 1, 2], [80, 80]) == (0, [ok, ok, old])                   # padding behind the last row
    assert run([0, 1, 2], [80, 0]) == (0, [ok, [-1] * n, old])
    assert run([0, 1, 2], [80, 81]) == (bad, [ok, old, old])                # past the table
    assert run([0, 1, 2], [80, -1]) == (bad, [ok, old, old])
    assert run([0, 1, 2], [79, 80], max_kv_len=79) == (bad, [ok, old, old])
    assert run([0, 1, 9], [80, 80]) == (bad, [ok, old, old])
    assert run([0, 2, 1], [80, 80]) == (bad, [ok, ok, old])
    assert run([-1, 1, 2], [80, 80]) == (bad, [old, ok, old])
    # a page outside the pool is looked at where pages are scored
    table[0, 1] = 20
    assert run([0, 1, 2], [80, 80]) == ((bad, [[0, 2, 3, 9], ok, old]) if n == 4 else (0, [ok, ok, old]))
    table[0, 1] = -1
    assert run([0, 1, 2], [80, 80]) == ((bad, [[0, 2, 3, 9], ok, old]) if n == 4 else (0, [ok, ok, old]))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("pages", [60, 9000])
def test_select_keeps_the_newest_pages_where_scores_are_not_finite(dt, pages):
    for what in ("q nan", "q inf", "bounds nan", "bounds inf", "overflow"):
        gen = torch.Generator(device="cuda").manual_seed(pages)
        bounds = torch.randn(pages, 1, 64, generator=gen, device="cuda").to(dt).repeat(1, 2, 1)
        q = torch.randn(1, 128, generator=gen, device="cuda").to(dt)
        if what[0] == "q":
            q[0, 5] = float(what[2:])
        elif what == "overflow":
            bounds, q = bounds * 3e38, q * 3e38
        else:
            bounds[::3, 1, 7] = float(what[7:])
        table = torch.randperm(pages, generator=gen, device="cuda").int()[None]
        picks = torch.full((1, 1, 20), -5, dtype=torch.int32, device="cuda")
        R.cb_paged_select(q, ints([0, 1]), ints([8 * pages]), table, bounds, 8, 2, 1, 64, picks, n_first=2, n_last=3)
        torch.cuda.synchronize()
        got = [j for j in picks.flatten().tolist() if j >= 0]
        assert {0, 1, *range(pages - 3, pages)} <= set(got) and len(set(got)) == len(got), (what, got)
        assert got == sorted(got) and got[-1] == pages - 1
    assert R.device_status() == 0


def check_attention(out, q, k, v, b, heads, scale, dt):
    """The bound of test_gpu_paged4.py, whose terms are relative to the weighted values B, and the
    probabilities' absolute one, which counts where a weight close to 1 meets a value of 0: in fp16
    a small probability is off by up to 2^-25 (half its least step) where the sum is 2^8 at least
    (few rows) or 2^6 (chunks of bf16), so each of p + 1 weights by 2^-33 or 2^-31."""
    hq, hkv, hd = heads
    want = OP.paged_attention(q, k, v, b.table, b.offsets, b.lens, *heads, scale, np.full((b.rows, hq * hd), 9.0))
    B = OP.paged_attention(q, k, np.abs(v), b.table, b.offsets, b.lens, *heads, scale, np.zeros(want.shape))
    lim, u = np.zeros(want.shape), HALF[dt]
    rel, low = (2.0 ** -11, 2.0 ** -31) if dt == torch.bfloat16 else (2.0 ** -22, 2.0 ** -33)
    for r, s, p in OP.row_positions(b.offsets, b.lens):
        j = np.arange(p + 1)
        at = b.table[s][j // b.page], j % b.page
        K, V = (np.abs(x[at]).reshape(p + 1, hkv, hd) for x in (k, v))
        for h in range(hq if p >= 0 else 0):
            c = slice(h * hd, (h + 1) * hd)
            A = scale * (K[:, h // (hq // hkv)] @ np.abs(q[r, c].astype(np.float64))).max()
            d = (2 * hd + 2 * hd + 4) * F * A + 8 * F * (A + 1) + 4 * F
            lim[r, c] = (2 * d + 2 * (p + 1) * F + rel) * B[r, c] + u * np.abs(want[r, c]) + \
                low * V[:, h // (hq // hkv)].sum(0)
    err = np.abs(f64(out) - want)
    assert np.all(err <= lim), (float((err - lim).max()), np.argwhere(err > lim)[:4].tolist())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("seqs", [[(1, 300), (1, 41)], [(3, 200), (1, 0)], [(70, 130)]])     # clusters and chunks
@pytest.mark.parametrize("q_std,k_std,k_exp,scale", [
    (2.0 ** -128, 1.0, 40, 2.0 ** 88),          # scale * 2^k_exp above fp32, the scores about 10
    (2.0 ** -128, 1.0, 64, 2.0 ** 65),
    (2.0 ** -100, 1.0, -64, 2.0 ** 126),
    (2.0 ** 124, 600.0, -64, 1.75 * 2.0 ** -75),    # below fp32's normal numbers
    (2.0 ** 100, 1.0, 64, 2.0 ** -126),         # scores of 2^38 and more
])
def test_attention_scales_and_exponents_beyond_fp32_together(dt, heads, seqs, q_std, k_std, k_exp, scale):
    hq, hkv, hd = heads
    rng = np.random.default_rng(hd + len(seqs))
    b = Batch(rng, seqs, 16, dt, hkv, hd, extra_cols=1)
    pool = O4.Pool(np.zeros((b.n_pages, R.cb_paged4_page_bytes(16, hkv, hd)), np.uint8), 16, hkv, hd)
    for p in range(b.n_pages):
        for slot in range(16):
            pool.put("k", p, slot, vals(rng, (b.kvw,), dt, k_std))
            pool.put("v", p, slot, vals(rng, (b.kvw,), dt))
    q = vals(rng, (b.rows, hq * hd), dt, q_std)
    out = torch.full((b.rows, hq * hd), 9.0, dtype=dt, device="cuda")
    R.cb_paged4_attention(dev(q, dt), *b.dev(), torch.from_numpy(pool.raw).cuda(), 16, hq, hkv, hd, out, scale=scale, k_exp=k_exp)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    check_attention(out, q, pool.values("k") * 2.0 ** k_exp, pool.values("v"), b, heads, scale, dt)


@pytest.mark.parametrize("dt", DTYPES)
def test_attention_over_keys_of_zero_with_any_scale(dt):
    """Scores of zero, whatever multiplies them: the values' mean."""
    heads, rng = (8, 2, 64), np.random.default_rng(3)
    b = Batch(rng, [(1, 300), (2, 41)], 16, dt, 2, 64, extra_cols=1)
    pool = O4.Pool(np.zeros((b.n_pages, R.cb_paged4_page_bytes(16, 2, 64)), np.uint8), 16, 2, 64)
    for p in range(b.n_pages):
        for slot in range(16):
            pool.put("k", p, slot, np.zeros(128))
            pool.put("v", p, slot, vals(rng, (128,), dt))
    for std, k_exp, scale in ((2.0 ** 100, 64, 2.0 ** 126), (2.0 ** -126, -64, 2.0 ** -126), (1.0, 0, 0.0)):
        q = vals(rng, (b.rows, 512), dt, std)
        out = torch.full((b.rows, 512), 9.0, dtype=dt, device="cuda")
        R.cb_paged4_attention(dev(q, dt), *b.dev(), torch.from_numpy(pool.raw).cuda(), 16, *heads, out, scale=scale, k_exp=k_exp)
        check_attention(out, q, pool.values("k"), pool.values("v"), b, heads, 0.0, dt)
    assert R.device_status() == 0


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,kv", [(1, 4000), (3, 200), (64, 300), (150, 700)])
@pytest.mark.parametrize("power", [10, 19, 21, 25, 31, 60, 118])
def test_attention_with_scores_of_any_size(dt, hd, n, kv, power):
    """Keys along one dimension, so that every score is exact: multiples of 2^power.  The largest
    has all the weight (2^-1024 and less are left), two keys that share it a half each."""
    hq, hkv, page = 4, 2, 16
    rng = np.random.default_rng(power)
    b = Batch(rng, [(n, kv), (n, kv)], page, dt, hkv, hd)
    pool = O4.Pool(np.zeros((b.n_pages, R.cb_paged4_page_bytes(page, hkv, hd)), np.uint8), page, hkv, hd)
    v = vals(rng, (b.n_pages, page, hkv * hd), dt)
    k = np.zeros(v.shape)
    k[..., 1::hd] = 6.0                 # (q is 0 there: makes the group's scale 1)
    k[..., ::hd] = np.array([0.5, 1, 1.5, 2, 3])[rng.integers(0, 5, (b.n_pages, page, 1))]
    # one or two of the keys that every row sees are the largest
    top = rng.choice(kv - n + 1, (2, 2))
    top[1, 1] = top[1, 0]
    for s in range(2):
        for j in top[s]:
            k[b.table[s][j // page], j % page, ::hd] = 6.0
    for p in range(b.n_pages):
        for slot in range(page):
            pool.put("k", p, slot, k[p, slot])
            pool.put("v", p, slot, v[p, slot])
    q = np.zeros((b.rows, hq * hd), np.float32)
    q[:, ::hd] = 1.0
    assert np.array_equal(pool.values("k"), k)
    out = torch.full((b.rows, hq * hd), 9.0, dtype=dt, device="cuda")
    R.cb_paged4_attention(dev(q, dt), *b.dev(), torch.from_numpy(pool.raw).cuda(), page, hq, hkv, hd, out,
                          scale=2.0 ** (power + 1 - 20), k_exp=20)
    torch.cuda.synchronize()
    V = pool.values("v")
    for s in range(2):
        best = [V[b.table[s][j // page], j % page].reshape(hkv, hd) for j in set(top[s].tolist())]
        want, B = (np.mean(x, 0)[None, :, None] for x in (best, np.abs(best)))
        got = f64(out)[b.offsets[s]:b.offsets[s + 1]].reshape(n, hkv, hq // hkv, hd)
        # both probabilities are the same power of two up to the rounding of their exponent, and
        # round to fp16 (in fp32: to two halves) beside a sum that does not; the sum's reciprocal
        # and two products, each twice where parts are joined; the result's rounding
        lim = ((2.0 ** -11 if dt == torch.bfloat16 else 2.0 ** -22) + 8 * F) * B + HALF[dt] * np.abs(want)
        assert np.all(np.abs(got - want) <= lim)
    assert R.device_status() == 0


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,kv", [(1, 3000), (3, 90), (40, 400)])
@pytest.mark.parametrize("first", [True, False])
def test_attention_past_keys_of_very_low_scores(dt, hd, n, kv, first):
    """Two thirds of the keys, in front of the others or behind them, have scores of -2^24 and less:
    their weights are zero, and the others' are as without them.  (A key's sums are exact up to
    roundings of its own terms, so A is the other keys'.)"""
    hq, hkv, page = 4, 2, 16
    rng = np.random.default_rng(n)
    b = Batch(rng, [(n, kv)], page, dt, hkv, hd)
    low = np.zeros((b.n_pages, page), bool)
    j = np.arange(2 * kv // 3) if first else np.arange(kv // 3 - n, kv - n)
    j = j[j < kv - n]
    low[b.table[0][j // page], j % page] = True
    k = vals(rng, (b.n_pages, page, hkv * hd), dt, 2.0 ** -8)
    k[low] = -2688.0
    v = vals(rng, k.shape, dt)
    pool = O4.Pool(np.zeros((b.n_pages, R.cb_paged4_page_bytes(page, hkv, hd)), np.uint8), page, hkv, hd)
    for p in range(b.n_pages):
        for slot in range(page):
            pool.put("k", p, slot, k[p, slot])
            pool.put("v", p, slot, v[p, slot])
    q = np.abs(vals(rng, (b.rows, hq * hd), dt)) + np.float32(0.5)
    if dt == torch.bfloat16:
        q = bf16_values(q)
    out = torch.full((b.rows, hq * hd), 9.0, dtype=dt, device="cuda")
    R.cb_paged4_attention(dev(q, dt), *b.dev(), torch.from_numpy(pool.raw).cuda(), page, hq, hkv, hd, out, scale=128.0)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    K, V = pool.values("k"), pool.values("v")
    args = (b.table, b.offsets, b.lens, hq, hkv, hd, 128.0)
    want = OP.paged_attention(q, K, V, *args, np.zeros((b.rows, hq * hd)))
    assert 128.0 * 2688 * np.abs(q.reshape(-1, hd)).sum(1).min() > 2.0 ** 24
    # the largest |score's terms| of the others, and weights and values as in check_attention
    A = 128.0 * np.abs(q.astype(np.float64)).reshape(-1, hd).sum(1).max() * np.abs(K[~low]).max()
    d = (4 * hd + 4) * F * A + 8 * F * (A + 1) + 4 * F
    rel, few = (2.0 ** -11, 2.0 ** -31) if dt == torch.bfloat16 else (2.0 ** -22, 2.0 ** -33)
    B = OP.paged_attention(q, K, np.abs(V), *args, np.zeros(want.shape))
    lim = (2 * d + 2 * kv * F + rel) * B + HALF[dt] * np.abs(want) + few * kv * np.abs(V).max()
    assert np.all(np.abs(f64(out) - want) <= lim)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("pages,n", [(1500, 600), (2040, 64), (5000, 1000), (20000, 7)])
@pytest.mark.parametrize("kind", ["zero q", "zero bounds", "same bounds", "three bounds", "outlier page", "near", "outside"])
def test_select_at_borders_among_many_scores(dt, pages, n, kind):
    """Hundreds and thousands of pages that fp32 scores do not tell apart from the border: equal
    ones (the lower pages), a page whose bounds widen every page's margin, scores that differ
    in their last bits, pages outside the pool."""
    rng = np.random.default_rng(pages)
    hq, hkv, hd, page = 6, 2, 64, 8
    b = Batch(rng, [(1, page * pages), (2, page * pages - 3)], page, dt, hkv, hd)
    x = vals(rng, (b.n_pages, 2, b.kvw), dt)
    bounds, q = np.sort(x, axis=1), vals(rng, (b.rows, hq * hd), dt)
    if kind == "zero q":
        q[0] = 0
        q[1] = -0.0
    elif kind == "zero bounds":
        bounds[:] = 0
        bounds[::3] = -0.0
    elif kind == "same bounds":
        bounds[:] = bounds[:1]
    elif kind == "three bounds":
        bounds[:] = bounds[rng.integers(0, 3, len(bounds))]
    elif kind == "outlier page":
        bounds[b.table[0][pages // 2]] *= np.float32(2.0 ** 12)
        bounds[b.table[1][pages // 3]] *= np.float32(2.0 ** 12)
    elif kind == "near":
        bounds[:] = 1
        bounds[:, :, ::hd] = 2.0 ** 20
        bounds[:, :, 1::hd] = (rng.integers(0, 200, (b.n_pages, 1, 1)) * 2.0 ** -14).astype(np.float32)
        q = np.ones_like(q)
    table = b.table.copy()
    if kind == "outside":           # more than the picks: the lowest of them beside all that are inside
        table[:, :pages] = np.where(rng.random((2, pages)) < 0.5 * n / pages, table[:, :pages], b.n_pages + 5)
    picks = torch.full((b.rows, hkv, n), -5, dtype=torch.int32, device="cuda")
    R.cb_paged_select(dev(q, dt), ints(b.offsets), ints(b.lens), ints(table), dev(bounds, dt), page, hq, hkv, hd, picks,
                      n_first=1, n_last=2)
    torch.cuda.synchronize()
    assert R.device_status() == (L.CB_ERR_DEVICE_INDEX if kind == "outside" else 0)
    if kind == "outside":
        gone = np.nextafter(np.float32(-3e38), 0) * np.ones((1, 2, b.kvw))      # the smallest score of any
        want = np.full(picks.shape, -5)
        for r, s in ((0, 0), (1, 1), (2, 1)):
            for g in range(hkv):
                there = table[s][:pages] < b.n_pages
                x = O4.page_scores(q[r], np.concatenate([bounds, gone]), np.minimum(table[s], b.n_pages), pages, hq, hkv, hd)[g]
                x[~there] = -np.inf
                x[0] = x[-2:] = np.inf
                want[r, g] = np.sort(np.lexsort((np.arange(pages), -x))[:n])
    else:
        want = O4.select(q, bounds, b.table, b.offsets, b.lens, page, hq, hkv, hd, np.full(picks.shape, -5), 1, 2)
    assert np.array_equal(picks.cpu().numpy(), want)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("heads,page,seqs,n", [
    ((8, 2, 64), 8, [(300, 2000), (1, 900), (150, 150)], 20),
    ((12, 4, 128), 32, [(400, 1500)], 9),
    ((16, 1, 64), 16, [(700, 700), (33, 5000)], 33),
])
def test_select_for_chunks_of_rows(dt, heads, page, seqs, n):
    """Hundreds of rows of a sequence, which begin before the picks are scarce and end behind."""
    select_case(np.random.default_rng(n), dt, heads, page, seqs, n, 1, 2, tail=1)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 7, 8, 9, 16, 20, 128])
@pytest.mark.parametrize("seqs,n", [([(1, 400), (2, 90)], 5), ([(1, 300 + 7 * i) for i in range(40)], 30)])
def test_picked_probabilities_keep_16_bits(hd, group, seqs, n):
    """bf16 rows: a probability meets the values as two halves of bf16, off by 2^-8 of 2^-8 of itself;
    the other terms as in test_gpu_picked.py.  Weights that are much alike: values of both signs
    nearly cancel, so that the results' own rounding does not hide the weights'."""
    dt, hkv = torch.bfloat16, 2 if group <= 20 else 1
    rng = np.random.default_rng(group)
    heads, scale = (group * hkv, hkv, hd), 0.02
    b, q, k, v, _, _, picks, out = picked_case(rng, dt, heads, 16, seqs, n, scale=scale, tail=1)
    args = (picks, b.table, b.offsets, b.lens, *heads, scale)
    want = O4.picked_attention(q, k, v, *args, np.full(out.shape, 9.0))
    B = O4.picked_attention(q, k, np.abs(v), *args, np.zeros(out.shape))
    A = scale * np.abs(q.astype(np.float64)).reshape(b.rows, -1, hd).sum(-1).repeat(hd, -1) * np.abs(k).max()
    d = 2 * hd * F * A + 8 * F * (A + 1) + 4 * F
    lim = (2 * d + 2 * n * 16 * F + 2.0 ** -16) * B + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(f64(out) - want) <= lim)


FIRST = r"""
import torch
import rag_kv_cache_layer_gb300 as R
ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
dt, hq, hkv, hd, page, kv = torch.bfloat16, 8, 2, 64, 16, 700
torch.manual_seed(0)
k, q = (torch.randn(n, w, device="cuda").to(dt) for n, w in ((kv, hkv * hd), (1, hq * hd)))
off, lens, table = ints([0, 1]), ints([kv]), torch.arange(44, device="cuda").int()[None]
pool = torch.randint(0, 127, (44, R.cb_paged4_page_bytes(page, hkv, hd)), device="cuda").to(torch.uint8) & 0x77
kp = torch.randn(44, page, hkv * hd, device="cuda").to(dt)
picks = torch.arange(40, device="cuda").int().expand(1, hkv, 40).contiguous()
ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
a, b = torch.zeros_like(q), torch.zeros_like(q)

def step(a, b):
    R.cb_paged4_attention(q, off, lens, table, pool, page, hq, hkv, hd, a, max_kv_len=kv, ws=ws)
    R.cb_paged_attention_picked(q, off, lens, table, kp, kp, picks, hq, hkv, hd, b, ws=ws)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step(a, b)
g.replay()
c, d = torch.zeros_like(q), torch.zeros_like(q)
step(c, d)
torch.cuda.synchronize()
assert torch.equal(a, c) and torch.equal(b, d) and bool(a.any()) and bool(b.any()) and R.device_status() == 0
"""


def test_the_first_calls_of_a_process_inside_a_capture():
    """What a call asks the device once may be asked while a graph is recorded."""
    import subprocess
    import sys
    from conftest import ROOT
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def nearest(x, dt):
    """The float of type dt nearest to the fraction x, ties to even."""
    bits = 24 if dt == torch.float32 else 8
    if x == 0:
        return 0.0
    _, e = np.frexp(float(x))
    step = Fraction(2) ** (int(e) - bits)
    n = x / step
    low = n.numerator // n.denominator
    up = n - low > Fraction(1, 2) or (n - low == Fraction(1, 2) and low % 2)
    return float((low + up) * step)


@pytest.mark.parametrize("dt", DTYPES)
def test_rotated_rows_are_rounded_exactly(dt):
    """Values of few bits beside values far smaller: products and sums in the middle of two
    neighbours, or beside it by less than float64 shows.  q_out against exact fractions; the keys'
    codes are those of the same values."""
    rng = np.random.default_rng(4)
    hd, heads, rows = 64, 16, 150
    shape = (rows, heads * hd)
    few = rng.integers(-48, 49, shape) * 0.125 * np.exp2(rng.integers(-6, 6, shape))
    tiny = rng.standard_normal(shape) * np.exp2(rng.integers(-50, -10, shape))
    x = np.where(rng.random(shape) < 0.5, few, tiny).astype(np.float32)
    if dt == torch.bfloat16:
        x = bf16_values(x)
    table = R.cb_rope_table_init(256, hd, 10000.0)
    cos, sin = np.moveaxis(table.cpu().numpy().reshape(-1, hd // 2, 2), -1, 0)
    b = Batch(rng, [(rows, rows + 2)], 16, dt, heads, hd)
    pool = torch.zeros(b.n_pages, R.cb_paged4_page_bytes(16, heads, hd), dtype=torch.uint8, device="cuda")
    qo = torch.zeros(shape, dtype=dt, device="cuda")
    R.cb_paged4_append(dev(x, dt), dev(x, dt), *b.dev(), pool, 16, hd, rope_table=table, q=dev(x, dt), q_out=qo)
    torch.cuda.synchronize()
    got, want = f64(qo).reshape(rows, heads, 2, -1), np.zeros((rows, heads, 2, hd // 2))
    for r in range(rows):
        for h in range(heads):
            for e in range(hd // 2):
                u, v = (Fraction(float(x[r, h * hd + i * hd // 2 + e])) for i in (0, 1))
                c, s = Fraction(float(cos[r + 2, e])), Fraction(float(sin[r + 2, e]))
                want[r, h, 0, e], want[r, h, 1, e] = nearest(u * c - v * s, dt), nearest(v * c + u * s, dt)
    assert np.array_equal(got, want)
    stored = O4.Pool(pool.cpu().numpy(), 16, heads, hd).values("k")
    for r in range(rows):
        at = b.table[0][(r + 2) // 16], (r + 2) % 16
        assert np.array_equal(stored[at], O4.values(*O4.quantise(want[r].reshape(heads, hd))).reshape(-1))
    assert R.device_status() == 0
