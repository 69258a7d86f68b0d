"""Page bounds, page selection and attention over picked pages against their
float64 definitions: bounds and picks are equal, attention is held to the bounds
of test_gpu_paged.py (a row's keys are the picked ones)."""
import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from oracle import paged as OP
from oracle import paged4 as O4
from rag_kv_cache_layer_gb300 import _lib as L
from test_gpu_paged import Batch, f64, ints, vals

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield


def dev(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt)


# ---------------------------------------------------------------- bounds --
@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads,page,seqs", [
    ((2, 64), 8, [(1, 1), (1, 8), (1, 9), (1, 0), (3, 2), (0, 40)]),
    ((8, 128), 16, [(1, 700), (40, 90), (17, 17)]),
    ((1, 64), 128, [(300, 400), (2, 129)]),
    ((3, 64), 32, [(1, 33 + i) for i in range(60)]),
    ((5, 16), 64, [(65, 130)]),
])
def test_bounds(dt, heads, page, seqs):
    hkv, hd = heads
    rng = np.random.default_rng(page)
    b = Batch(rng, seqs, page, dt, hkv, hd, extra_cols=1, tail=2)
    k, _, dk, _ = b.pools(rng)                              # NaN in the slots that hold no position
    out = torch.full((b.n_pages, 3, b.kvw), 7.0, dtype=dt, device="cuda")
    R.cb_paged_bounds(*b.dev(), dk, out[:, :2], b.rows)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    want = O4.page_bounds(np.full((b.n_pages, 2, b.kvw), 7.0), k, b.table, b.offsets, b.lens)
    assert np.array_equal(f64(out[:, :2]), want) and (out[:, 2] == 7).all()


@pytest.mark.parametrize("dt", list(HALF))
def test_bounds_of_layers(dt):
    rng = np.random.default_rng(2)
    b = Batch(rng, [(70, 70)], 16, dt, 2, 64)
    kp = torch.randn(3, b.n_pages, 16, 128, device="cuda").to(dt)
    out = torch.zeros(3, b.n_pages, 2, 128, dtype=dt, device="cuda")
    R.cb_paged_bounds(*b.dev(), kp, out, 70)
    for l in range(3):
        assert np.array_equal(f64(out[l]), O4.page_bounds(np.zeros(out[l].shape), f64(kp[l]), b.table, b.offsets, b.lens))


# ------------------------------------------------------------- selection --
def select_case(rng, dt, heads, page, seqs, n, n_first=1, n_last=1, tail=0, integers=False, **kw):
    hq, hkv, hd = heads
    b = Batch(rng, seqs, page, dt, hkv, hd, extra_cols=1, tail=tail)
    if integers:                                            # scores that are equal in many places
        lo = rng.integers(-1, 1, (b.n_pages, 1, b.kvw)).astype(np.float32)
        bounds = np.concatenate([lo, lo + rng.integers(0, 2, lo.shape)], 1).astype(np.float32)
        q = rng.integers(-1, 2, (b.rows, hq * hd)).astype(np.float32)
    else:
        x = vals(rng, (b.n_pages, 2, b.kvw), dt)
        bounds, q = np.sort(x, axis=1), vals(rng, (b.rows, hq * hd), dt)
    picks = torch.full((b.rows, hkv, n), -5, dtype=torch.int32, device="cuda")
    args = (*b.dev(), dev(bounds, dt), page, hq, hkv, hd)
    R.cb_paged_select(dev(q, dt), *args, picks, n_first=n_first, n_last=n_last, **kw)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    want = O4.select(q, bounds, b.table, b.offsets, b.lens, page, hq, hkv, hd, np.full(picks.shape, -5), n_first, n_last)
    assert np.array_equal(picks.cpu().numpy(), want)
    return b, q, bounds, picks


SELECT = [
    ((4, 2, 64), 8, [(1, 1), (1, 0), (1, 400), (1, 65), (1, 64)], 8, 1, 1),
    ((32, 8, 128), 16, [(1, 5000)], 16, 1, 2),
    ((7, 1, 128), 16, [(1, 2000), (3, 900)], 1, 0, 1),
    ((7, 1, 128), 16, [(1, 2000), (3, 900)], 1, 0, 0),
    ((16, 1, 64), 32, [(2, 2000)], 5, 2, 3),                # nothing is left to choose
    ((8, 8, 128), 8, [(1, 200 + 37 * i) for i in range(40)], 32, 4, 4),
    ((40, 1, 64), 8, [(5, 3000), (30, 20), (0, 9)], 100, 0, 1),
    ((8, 2, 64), 16, [(20, 300), (3, 1)], 7, 1, 1),
    ((4, 2, 64), 8, [(1, 20000)], 1000, 10, 10),
]


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads,page,seqs,n,n_first,n_last", SELECT)
def test_select(dt, heads, page, seqs, n, n_first, n_last):
    rng = np.random.default_rng(n + page)
    select_case(rng, dt, heads, page, seqs, n, n_first, n_last, tail=2)
    select_case(rng, dt, heads, page, seqs, n, n_first, n_last, integers=True)


def test_select_equal_and_extreme_scores():
    """All scores equal: the lowest pages.  Scores whose fp32 sums differ by less than
    their rounding are told apart."""
    dt = torch.float32
    b = Batch(np.random.default_rng(1), [(1, 1600)], 8, dt, 1, 64)
    picks = torch.zeros(1, 1, 20, dtype=torch.int32, device="cuda")
    bounds, q = np.ones((b.n_pages, 2, 64), np.float32), np.ones((1, 64), np.float32)
    R.cb_paged_select(dev(q, dt), *b.dev(), dev(bounds, dt), 8, 1, 1, 64, picks, n_first=0, n_last=1)
    assert picks.flatten().tolist() == list(range(19)) + [199]
    bounds[:, :, 0] = 2.0 ** 20
    order = np.random.default_rng(3).permutation(b.n_pages)
    bounds[:, :, 1] = (order[:, None] * 2.0 ** -12).astype(np.float32)      # far below 2^20 + 62's last bit
    R.cb_paged_select(dev(q, dt), *b.dev(), dev(bounds, dt), 8, 1, 1, 64, picks, n_first=0, n_last=0)
    want = O4.select(q, bounds, b.table, b.offsets, b.lens, 8, 1, 1, 64, picks.cpu().numpy(), 0, 0)
    assert np.array_equal(picks.cpu().numpy(), want) and R.device_status() == 0


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("kind", ["outlier", "two values", "many equal", "wide"])
def test_select_scores_of_any_distribution(dt, kind):
    """Scores that a histogram of their range does not tell apart, more pages than a
    block holds in registers, borders between equal scores."""
    rng = np.random.default_rng(31)
    b = Batch(rng, [(1, 8 * 9000), (2, 8 * 700)], 8, dt, 2, 64)
    x = vals(rng, (b.n_pages, 1, 128), dt)
    if kind == "outlier":
        x[b.table[0][5]] *= 2.0 ** 40
    elif kind == "two values":
        x[:] = np.where(rng.random((b.n_pages, 1, 1)) < 0.01, 1.0, 0.5)
    elif kind == "many equal":
        x[rng.random(b.n_pages) < 0.7] = x[0]
    else:
        x *= np.exp2(rng.integers(-30, 30, (b.n_pages, 1, 1))).astype(np.float32)
    bounds, q = np.repeat(x, 2, 1), vals(rng, (b.rows, 4 * 64), dt)
    picks = torch.zeros(b.rows, 2, 100, dtype=torch.int32, device="cuda")
    R.cb_paged_select(dev(q, dt), *b.dev(), dev(bounds, dt), 8, 4, 2, 64, picks, n_first=1, n_last=1)
    want = O4.select(q, bounds, b.table, b.offsets, b.lens, 8, 4, 2, 64, np.zeros(picks.shape), 1, 1)
    assert np.array_equal(picks.cpu().numpy(), want) and R.device_status() == 0


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("pages", [60, 9000])
def test_select_keeps_its_places_where_scores_are_not_finite(dt, pages):
    """Not promised to be sensible, but n_picks places a row are written and no others, with
    pages of the row or -1, the forced ones among them."""
    for what in ("q nan", "q inf", "bounds nan", "bounds inf", "overflow"):
        bounds = torch.randn(pages, 1, 64, device="cuda").to(dt).repeat(1, 2, 1)
        q = torch.randn(1, 128, device="cuda").to(dt)
        if what[0] == "q":
            q[0, 5] = float(what[2:])
        elif what == "overflow":
            bounds, q = bounds * 3e38, q * 3e38
        else:
            bounds[::3, 1, 7] = float(what[7:])
        table = torch.randperm(pages, device="cuda").int()[None]
        picks = torch.full((3, 1, 20), -5, dtype=torch.int32, device="cuda")
        R.cb_paged_select(q, ints([0, 1]), ints([8 * pages]), table, bounds, 8, 2, 1, 64, picks[1:2], n_first=2, n_last=3)
        torch.cuda.synchronize()
        assert (picks[0] == -5).all() and (picks[2] == -5).all()
        got = picks[1, 0].tolist()
        assert got[:2] == [0, 1] and (got[-3:] == list(range(pages - 3, pages)) or -1 in got)
        assert all(-1 <= j < pages for j in got) and len(set(got) - {-1}) == sum(j >= 0 for j in got)
    assert R.device_status() == 0


def test_select_errors_on_the_device():
    dt, page = torch.bfloat16, 8
    bounds, q = torch.zeros(20, 2, 64, dtype=dt, device="cuda"), torch.ones(3, 64, dtype=dt, device="cuda")

    def run(offsets, lens, table, **kw):
        picks = torch.full((3, 1, 4), -5, dtype=torch.int32, device="cuda")
        R.cb_paged_select(q, ints(offsets), ints(lens), ints(table), bounds, page, 1, 1, 64, picks, **kw)
        torch.cuda.synchronize()
        return R.device_status(), picks[:, 0].tolist()
    bad, ok, old = L.CB_ERR_DEVICE_INDEX, [0, 1, 2, 9], [-5] * 4
    t = [list(range(10)), list(range(10))]
    assert run([0, 1, 2], [80, 80], t) == (0, [ok, ok, old])                # padding behind the last row
    assert run([0, 1, 2], [80, 81], t) == (bad, [ok, old, old])
    assert run([0, 1, 2], [80, -1], t) == (bad, [ok, old, old])
    assert run([0, 1, 2], [80, 80], t, max_kv_len=79) == (bad, [old, old, old])
    assert run([0, 1, 9], [80, 80], t) == (bad, [ok, old, old])
    # pages outside the pool have the smallest score
    assert run([0, 1, 2], [80, 80], [[0] + [-1] * 8 + [1], t[1]]) == (bad, [[0, 1, 2, 9], ok, old])
    assert run([0, 1, 2], [80, 80], [[0, 5, 77, 77, 77, 77, 77, 77, 77, 9], t[1]], n_first=0, n_last=0) == (bad, [[0, 1, 2, 9], [0, 1, 2, 3], old])
    assert run([0, 1, 2], [80, 80], [[0, 20, 2, 3, 4, 5, 6, 7, 8, 9], t[1]]) == (bad, [[0, 2, 3, 9], ok, old])


# ------------------------------------------------------------- attention --
def picked_case(rng, dt, heads, page, seqs, n, picks=None, tail=0, std=1.0, **kw):
    hq, hkv, hd = heads
    b = Batch(rng, seqs, page, dt, hkv, hd, extra_cols=1, tail=tail)
    k, v, dk, dv = b.pools(rng)
    q = vals(rng, (b.rows, hq * hd), dt, std)
    if picks is None:
        # any pages of the sequence, unordered, some named twice, some none, some past the row
        picks = np.full((b.rows, hkv, n), -1)
        for r, s, p in OP.row_positions(b.offsets, b.lens):
            have = -(-b.lens[s] // page)
            if have:
                picks[r] = rng.integers(-1, have, (hkv, n))
    out = torch.full((b.rows, hq * hd), 9.0, dtype=dt, device="cuda")
    R.cb_paged_attention_picked(dev(q, dt), *b.dev(), dk, dv, ints(picks), hq, hkv, hd, out, **kw)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    check_picked(out, q, k, v, picks, b, heads, kw.get("scale", hd ** -0.5), dt)
    return b, q, k, v, dk, dv, picks, out


def check_picked(out, q, k, v, picks, b, heads, scale, dt):
    hq, hkv, hd = heads
    start = np.full((b.rows, hq * hd), 9.0)
    args = (picks, b.table, b.offsets, b.lens, hq, hkv, hd)
    want = O4.picked_attention(q, k, v, *args, scale, start)
    B = O4.picked_attention(q, k, np.abs(v), *args, scale, np.zeros_like(start))
    top = np.abs(k).max(initial=0.0)
    # A: no score's terms sum to more than |q|_1 times the largest key element
    A = scale * np.abs(q.astype(np.float64)).reshape(b.rows, hq, hd).sum(-1).repeat(hd, -1) * top
    d = 2 * hd * F * A + 8 * F * (A + 1) + 4 * F
    lim = (2 * d + 2 * picks.shape[2] * b.page * F + (HALF[dt] if dt == torch.bfloat16 else 0)) * B + HALF[dt] * np.abs(want)
    err = np.abs(f64(out) - want)
    assert np.all(err <= lim), (float((err - lim).max()), np.argwhere(err > lim)[:4].tolist())


PICKED = [
    ((4, 2, 64), 8, [(1, 1), (1, 0), (1, 400), (1, 65), (1, 64)], 8),
    ((32, 8, 128), 16, [(1, 5000)], 33),
    ((7, 1, 128), 32, [(1, 129), (3, 31), (1, 2000)], 1),
    ((16, 1, 64), 64, [(2, 2000)], 5),
    ((40, 1, 128), 128, [(1, 700), (2, 3)], 6),
    ((128, 1, 64), 16, [(1, 300)], 11),
    ((8, 8, 128), 8, [(1, 200 + 37 * i) for i in range(30)], 20),
    ((8, 2, 64), 16, [(20, 300), (3, 1), (0, 50)], 7),
    ((4, 2, 64), 1024, [(3, 3000)], 2),
    ((4, 2, 128), 8, [(1, 9000)], 1024),
]


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads,page,seqs,n", PICKED)
def test_picked_attention(dt, heads, page, seqs, n):
    rng = np.random.default_rng(n + page)
    picked_case(rng, dt, heads, page, seqs, n, tail=2)
    picked_case(rng, dt, heads, page, seqs, n, std=3.0, scale=0.05)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,cluster", [(3, 1), (13, 2), (25, 4), (50, 8)])
def test_items_in_clusters(dt, hd, n, cluster):
    """Every cluster size of the one-launch form, by the plan that leads to it."""
    import ctypes
    heads, page = (24, 4, hd), 8 * {(64, False): 4, (128, False): 2, (64, True): 2, (128, True): 1}[hd, dt == torch.float32]
    out = (ctypes.c_int64 * 3)()
    assert L.lib.cb_debug_picked_plan(3, n, page, *heads, R.dtype_code(dt), out) == L.CB_OK
    assert out[0] == cluster
    rng = np.random.default_rng(n)
    picked_case(rng, dt, heads, page, [(1, 40 * page + 3), (1, 0), (1, page)], n)
    picked_case(rng, dt, (20, 1, hd), page, [(2, 30 * page + 3), (0, 5), (1, 3)], n, tail=1)    # two tiles of heads


@pytest.mark.parametrize("dt", list(HALF))
def test_all_pages_are_the_whole_attention(dt):
    """Every page picked, in any order: cb_paged_attention's rows."""
    rng = np.random.default_rng(12)
    hq, hkv, hd, page = 8, 2, 128, 16
    seqs = [(1, 333), (4, 90), (1, 0), (30, 64)]
    b = Batch(rng, seqs, page, dt, hkv, hd)
    k, v, dk, dv = b.pools(rng)
    q = dev(vals(rng, (b.rows, hq * hd), dt), dt)
    picks = np.stack([rng.permutation(21) for _ in range(b.rows * hkv)]).reshape(b.rows, hkv, 21)
    for r, s, _ in OP.row_positions(b.offsets, b.lens):
        picks[r][picks[r] >= -(-b.lens[s] // page)] = -1
    one, all_ = torch.empty_like(q), torch.empty_like(q)
    R.cb_paged_attention_picked(q, *b.dev(), dk, dv, ints(picks), hq, hkv, hd, one)
    R.cb_paged_attention(q, *b.dev(), dk, dv, hq, hkv, hd, all_)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    # two results of one value: the type's rounding twice, and P's in bf16
    lim = 4 * HALF[dt] * 4 if dt == torch.bfloat16 else 2e-5
    assert float((one.float() - all_.float()).abs().max()) <= lim


@pytest.mark.parametrize("dt", list(HALF))
def test_many_items_and_pieces(dt):
    """More items than parts, and items in several parts."""
    rng = np.random.default_rng(13)
    picked_case(rng, dt, (8, 8, 64), 16, [(3, 400 + 9 * i) for i in range(50)], 12)
    picked_case(rng, dt, (24, 8, 64), 16, [(1, 4000)] * 3, 200)


def test_errors_on_the_device():
    dt = torch.bfloat16
    kp, q = torch.zeros(4, 8, 128, dtype=dt, device="cuda"), torch.ones(3, 256, dtype=dt, device="cuda")

    def run(offsets, lens, table, picks):
        out = torch.full((3, 256), 9.0, dtype=dt, device="cuda")
        p = ints(picks)[:, None].expand(3, 2, -1).contiguous()
        R.cb_paged_attention_picked(q, ints(offsets), ints(lens), ints(table), kp, kp, p, 4, 2, 64, out)
        torch.cuda.synchronize()
        return R.device_status(), [int(x) for x in (out == 9.0).all(1)]
    bad, t, p = L.CB_ERR_DEVICE_INDEX, [[0, 1], [2, 3]], [[0, 1], [0, 1], [0, 1]]
    assert run([0, 1, 2], [16, 9], t, p) == (0, [0, 0, 1])                          # padding behind the last row
    assert run([0, 1, 2], [16, 9], [[0, 1], [2, 4]], p) == (bad, [0, 0, 1])
    assert run([0, 1, 2], [16, 9], t, [[0, 2], [0, 1], [0, 1]]) == (bad, [0, 0, 1])
    assert run([0, 1, 2], [16, 9], t, [[0, -2], [0, 1], [0, 1]]) == (bad, [0, 0, 1])
    assert run([0, 1, 2], [16, 17], t, p) == (bad, [0, 1, 1])
    assert run([0, 1, 2], [-1, 9], t, p) == (bad, [1, 0, 1])
    assert run([0, 1, 5], [16, 9], t, p) == (bad, [0, 1, 1])


# --------------------------------------------------------------- together --
@pytest.mark.parametrize("dt", list(HALF))
def test_a_recorded_step_of_append_bounds_selection_and_attention(dt):
    """A decode step's four calls in one graph, replayed token by token while the
    lengths grow, against the oracle on the cache of the moment."""
    rng = np.random.default_rng(21)
    hq, hkv, hd, page, n = 8, 2, 64, 8, 6
    b = Batch(rng, [(1, 120), (1, 41), (1, 0)], page, dt, hkv, hd, spare=40)
    b.table = rng.permutation(b.n_pages)[:3 * 18].reshape(3, 18)
    kp = dev(vals(rng, (b.n_pages, page, b.kvw), dt), dt)
    vp = dev(vals(rng, (b.n_pages, page, b.kvw), dt), dt)
    bounds = torch.stack([kp.amin(1), kp.amax(1)], 1)
    off, lens, table = b.dev()
    q, k, v = (torch.zeros(3, w, dtype=dt, device="cuda") for w in (hq * hd, b.kvw, b.kvw))
    picks, out = torch.zeros(3, hkv, n, dtype=torch.int32, device="cuda"), torch.zeros_like(q)
    rope = R.cb_rope_table_init(200, hd, 10000.0)
    ws1 = R.cb_paged_select_workspace(q, 144, page, hkv)
    ws2 = R.cb_paged_attention_picked_workspace(q, n, page, hq, hkv, hd)
    g, qr = torch.cuda.CUDAGraph(), torch.zeros_like(q)

    def step():
        R.cb_paged_append(k, v, off, lens, table, kp, vp, hd, rope_table=rope, q=q, q_out=qr)
        R.cb_paged_bounds(off, lens, table, kp, bounds, 3)
        R.cb_paged_select(qr, off, lens, table, bounds, page, hq, hkv, hd, picks, n_first=1, n_last=2, max_kv_len=144, ws=ws1)
        R.cb_paged_attention_picked(qr, off, lens, table, kp, vp, picks, hq, hkv, hd, out, ws=ws2)
    with torch.cuda.graph(g):
        step()
    for t in range(20):
        for x in (q, k, v):
            x.copy_(dev(vals(rng, tuple(x.shape), dt), dt))
        if t:
            lens.add_(ints([1, 1, 1 if t > 5 else 0]))
        g.replay()
        torch.cuda.synchronize()
        b.lens = lens.cpu().numpy().astype(np.int64)
        K, B = f64(kp), f64(bounds)
        for s in range(3):                      # every page that holds a key has its bounds... of keys up to the length
            for j in range((b.lens[s] - 1) // page, -(-b.lens[s] // page)):
                x = K[b.table[s][j], :b.lens[s] - j * page]
                assert np.array_equal(B[b.table[s][j]], np.stack([x.min(0), x.max(0)]))
        want = O4.select(f64(qr), B, b.table, b.offsets, b.lens, page, hq, hkv, hd, picks.cpu().numpy(), 1, 2)
        assert np.array_equal(picks.cpu().numpy(), want)
        check_picked(out, f64(qr), K, f64(vp), want, b, (hq, hkv, hd), hd ** -0.5, dt)
    assert R.device_status() == 0
