"""The 4-bit paged cache: codes against the format's definition, bit for bit,
rows read back, and attention over it against its float64 definition.

Codes.  A key is rotated by the table's entries, rounded to the rows' type and
quantised; every step is a rounding of an exact value, so codes and scales are
equal to the oracle's (a zero's sign aside).

Attention (F = 2^-24, u half a step of the output's type; see test_gpu_paged.py
for d, A and B).  Keys and values are exact in fp16.  q in fp16, scaled by a
power of two: a bf16 q is exact but for elements below 2^-27 of the row's
largest, off by 2^-39 of it; an fp32 q in two halves is off by 2^-23 of itself:
A grows by at most 2 F hd and 4 F.  Tensor cores may truncate: twice the sums'
error.  Probabilities round to fp16, 2^-11 with the half below (their factor of
2^8 keeps them normal down to 2^-22 of the reference and exact to 2^-33 of it
below): + 2^-11 B; in fp32 two halves: 2^-22 B."""
import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from gpu_common import bf16_values
from oracle import paged as OP
from oracle import paged4 as O4
from rag_kv_cache_layer_gb300 import _lib as L
from test_gpu_paged import Batch, f64, ints, vals

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BITS = {torch.float32: 24, torch.bfloat16: 8}
BASE = 10000.0


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield


def dev(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt)


def raw_pool(rng, b, hkv, hd, extra=0):
    """Random bytes: a pool that other sequences have used."""
    size = R.cb_paged4_page_bytes(b.page, hkv, hd)
    return torch.from_numpy(rng.integers(0, 256, (b.n_pages, size + extra), dtype=np.uint8)).cuda()


def wide(rng, shape, dt):
    """Rows whose groups differ by powers of two and hold ties, zeros and extremes."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-14, 13, shape[:-1] + (1,)))
    flat = x.reshape(-1, 16)
    kind = rng.integers(0, 8, len(flat))
    flat[kind == 0] = 0.0
    grid = rng.integers(-48, 49, flat.shape) * 0.125                  # borders between codes
    flat[kind == 1] = (grid * np.exp2(rng.integers(-8, 8, (len(flat), 1))))[kind == 1]
    flat[kind == 2] *= 2.0 ** -20                                     # below the smallest scale
    flat[kind == 3, 0] = 6.0 * O4.SCALES[rng.integers(1, 126, (kind == 3).sum())]
    x = flat.reshape(shape).astype(np.float32)
    return bf16_values(x) if dt == torch.bfloat16 else x


def stored(x, dt, b, s_pos, table=None):
    """What a cache of the rows' type would hold."""
    y = O4.rotate_by_table(x, s_pos, table) if table is not None else x.astype(np.float64)
    return O4.round_to(y, BITS[dt])


APPEND = [
    ((4, 2, 64), 8, [(1, 1)]),
    ((32, 8, 128), 16, [(1, 3137)]),
    ((8, 4, 128), 8, [(1, 16), (1, 17), (1, 0), (1, 5000)]),
    ((7, 1, 64), 32, [(3, 3), (0, 9), (65, 70), (5, 2), (2, 0), (33, 64)]),
    ((5, 5, 64), 64, [(130, 1000), (1, 64), (64, 64)]),
    ((8, 8, 128), 16, [(1, 40 + i) for i in range(70)]),
]


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads,page,seqs", APPEND)
@pytest.mark.parametrize("exps", [(0, 0), (-3, 5)])
def test_append_and_gather(dt, heads, page, seqs, exps):
    hq, hkv, hd = heads
    rng = np.random.default_rng(hd + page + len(seqs))
    b = Batch(rng, seqs, page, dt, hkv, hd, extra_cols=2, tail=3)
    pool = raw_pool(rng, b, hkv, hd, extra=32)
    want = O4.Pool(pool.cpu().numpy(), page, hkv, hd)
    k, v, q = (wide(rng, (b.rows, w), dt) for w in (b.kvw, b.kvw, hq * hd))
    table = R.cb_rope_table_init(6000, hd, BASE)
    host = table.cpu().numpy().reshape(-1, hd // 2, 2)
    fused = dev(np.concatenate([q, k, v], 1), dt)
    dq, dk, dv = fused[:, :hq * hd], fused[:, hq * hd:hq * hd + b.kvw], fused[:, hq * hd + b.kvw:]
    qo = torch.full((b.rows, hq * hd), 3.0, device="cuda", dtype=dt)
    R.cb_paged4_append(dk, dv, *b.dev(), pool, page, hd, rope_table=table, q=dq, q_out=qo, k_exp=exps[0], v_exp=exps[1])
    back = torch.full((2, b.rows, b.kvw + 8), 7.0, device="cuda", dtype=dt)
    R.cb_paged4_gather(*b.dev(), pool, page, hd, back[0, :, :b.kvw], back[1, :, :b.kvw], k_exp=exps[0], v_exp=exps[1])
    torch.cuda.synchronize()
    assert R.device_status() == 0
    got = O4.Pool(pool.cpu().numpy(), page, hkv, hd)
    want_q, want_back = np.full((b.rows, hq * hd), 3.0), np.full((2, b.rows, b.kvw + 8), 7.0)
    for r, s, p in OP.row_positions(b.offsets, b.lens):
        if p < 0:
            continue
        at = b.table[s][p // page], p % page
        want_q[r] = stored(q[r:r + 1], dt, b, [p], host)[0]
        for i, (name, x) in enumerate((("k", stored(k[r:r + 1], dt, b, [p], host)[0]), ("v", stored(v[r:r + 1], dt, b, [p])[0]))):
            want.put(name, *at, x * 2.0 ** -exps[i])
            one = [want.part[name + c][at[0], :, at[1]] for c in "cs"]
            code = np.stack([one[0].astype(int) & 15, one[0].astype(int) >> 4], -1).reshape(hkv, hd)
            want_back[i, r, :b.kvw] = (O4.values(code, one[1].astype(int)) * 2.0 ** exps[i]).reshape(-1)
    for name in ("ks", "vs"):
        assert np.array_equal(got.part[name], want.part[name])
    for name in ("kc", "vc"):
        a, c = (np.stack([x.part[name] & 15, x.part[name] >> 4]) for x in (got, want))
        assert np.array_equal(np.where(a == 8, 0, a), np.where(c == 8, 0, c))
    assert np.array_equal(pool[:, -32:].cpu().numpy(), want.raw[:, -32:])          # behind the page: untouched
    assert np.array_equal(f64(qo), want_q)
    assert np.array_equal(f64(back), want_back)


def test_infinities_and_nan_are_stored_as_numbers():
    x = torch.randn(3, 64, device="cuda")
    x[0, 3], x[0, 17], x[1, 5], x[2, 40] = float("inf"), float("-inf"), float("nan"), 1e38
    for dt in HALF:
        pool = torch.zeros(1, R.cb_paged4_page_bytes(8, 1, 64), dtype=torch.uint8, device="cuda")
        out = torch.empty(2, 3, 64, dtype=dt, device="cuda")
        args = ints([0, 3]), ints([3]), ints([[0]]), pool, 8, 64
        R.cb_paged4_append(x.to(dt), x.to(dt), *args)
        R.cb_paged4_gather(*args, out[0], out[1])
        assert torch.isfinite(out.float()).all() and torch.equal(out[0], out[1])
        assert out[0, 0, 3] == 2688 and out[0, 0, 17] == -2688 and out[0, 2, 40] == 2688
        # other groups of those rows are as without them
        y = f64(x.to(dt)[:, 48:])
        c, s = O4.quantise(y)
        assert np.array_equal(f64(out[0, :, 48:]), O4.values(c, s))


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("layers,rows,page", [(1, 5, 8), (3, 131, 16), (7, 40, 64)])
def test_layers_without_rotation(dt, layers, rows, page):
    """A fused cache of several layers goes into pages and comes back: the values of its codes."""
    rng = np.random.default_rng(layers)
    b = Batch(rng, [(rows, rows + 3)], page, dt, 2, 64)
    big = dev(vals(rng, (layers, rows + 9, 128), dt), dt)
    k, v = big[:, 4:4 + rows], big[:, 9:]                     # strided layers
    pool = torch.zeros(layers, b.n_pages, R.cb_paged4_page_bytes(page, 2, 64), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, layers, rows + 1, 128, dtype=dt, device="cuda")
    ko, vo = out[0, :, :rows], out[1, :, 1:]
    if layers == 1:
        R.cb_paged4_append(k[0], v[0], *b.dev(), pool[0], page, 64)
        R.cb_paged4_gather(*b.dev(), pool[0], page, 64, ko[0], vo[0])
    else:
        R.cb_paged4_append(k, v, *b.dev(), pool, page, 64)
        R.cb_paged4_gather(*b.dev(), pool, page, 64, ko, vo)
    for x, y in ((k, ko), (v, vo)):
        assert np.array_equal(f64(y), O4.values(*O4.quantise(f64(x))))
    assert not out[0, :, rows:].any() and not out[1, :, :1].any() and R.device_status() == 0


def test_append_in_place_and_keys_alone():
    rng = np.random.default_rng(5)
    for dt in HALF:
        b = Batch(rng, [(3, 20), (2, 2)], 8, dt, 2, 64)
        p1 = raw_pool(rng, b, 2, 64)
        p2, p3 = p1.clone(), p1.clone()
        k, v, q = (dev(vals(rng, (5, w), dt), dt) for w in (128, 128, 256))
        table, out = R.cb_rope_table_init(64, 64, BASE), torch.empty_like(q)
        R.cb_paged4_append(k, v, *b.dev(), p1, 8, 64, rope_table=table, q=q, q_out=out)
        R.cb_paged4_append(k, v, *b.dev(), p2, 8, 64, rope_table=table)
        R.cb_paged4_append(k, v, *b.dev(), p3, 8, 64, rope_table=table, q=q)       # in place
        assert torch.equal(p1, p2) and torch.equal(p1, p3) and torch.equal(q, out)


def test_bad_pages_positions_and_offsets_are_recorded():
    rng = np.random.default_rng(9)
    dt, table = torch.bfloat16, R.cb_rope_table_init(32, 64, BASE)
    k = dev(vals(rng, (4, 128), dt), dt)

    def run(offsets, lens, tbl, rope=table):
        pool = torch.zeros(4, R.cb_paged4_page_bytes(8, 2, 64), dtype=torch.uint8, device="cuda")
        out = torch.zeros(2, 4, 128, dtype=dt, device="cuda")
        R.cb_paged4_append(k, k, ints(offsets), ints(lens), ints(tbl), pool, 8, 64, rope_table=rope)
        first = R.device_status()
        R.cb_paged4_gather(ints(offsets), ints(lens), ints(tbl), pool, 8, 64, out[0], out[1])
        second = R.device_status()
        assert first == second or rope is not None
        x = O4.Pool(pool.cpu().numpy(), 8, 2, 64).values("v")
        return first, [list(map(int, i)) for i in np.argwhere((x != 0).any(-1))], (out[1] != 0).any(-1).nonzero()[:, 0].tolist()
    bad = L.CB_ERR_DEVICE_INDEX
    assert run([0, 2, 4], [2, 3], [[1], [0]]) == (0, [[0, 1], [0, 2], [1, 0], [1, 1]], [0, 1, 2, 3])
    assert run([0, 2, 4], [2, 3], [[4], [0]]) == (bad, [[0, 1], [0, 2]], [2, 3])
    assert run([0, 2, 4], [2, 3], [[-1], [0]]) == (bad, [[0, 1], [0, 2]], [2, 3])
    assert run([0, 2, 4], [9, 3], [[1], [0]]) == (bad, [[0, 1], [0, 2], [1, 7]], [0, 2, 3])
    assert run([0, 4], [40], [[0, 1, 2, 3, 0]])[:2] == (bad, [])
    assert run([0, 3, 2], [3, 3], [[1], [0]])[0] == bad
    assert run([0, 9, 9], [9, 3], [[1], [0]]) == (bad, [], [])


# ------------------------------------------------------------- attention --
def attention_case(rng, dt, heads, page, seqs, tail=0, std=1.0, exps=(0, 0), extra=0, **kw):
    hq, hkv, hd = heads
    b = Batch(rng, seqs, page, dt, hkv, hd, extra_cols=1, tail=tail)
    pool = O4.Pool(np.full((b.n_pages, R.cb_paged4_page_bytes(page, hkv, hd) + extra), 0x7f, np.uint8), page, hkv, hd)
    k, v = (vals(rng, (b.n_pages, page, b.kvw), dt) for _ in range(2))
    for s, (_, kv) in enumerate(seqs):      # slots that hold no position keep scales that are NaN
        for j in range(0, kv, page):
            n, pg = min(page, kv - j), b.table[s][j // page]
            for name, x in (("k", k), ("v", v)):
                code, scale = O4.quantise(x[pg, :n].reshape(n, hkv, hd).transpose(1, 0, 2))
                pool.part[name + "c"][pg, :, :n] = code[..., 0::2] + 16 * code[..., 1::2]
                pool.part[name + "s"][pg, :, :n] = scale
    raw = torch.from_numpy(pool.raw).cuda()
    q = vals(rng, (b.rows, hq * hd), dt, std)
    out = torch.full((b.rows, hq * hd), 9.0, dtype=dt, device="cuda")
    R.cb_paged4_attention(dev(q, dt), *b.dev(), raw, page, hq, hkv, hd, out, k_exp=exps[0], v_exp=exps[1], **kw)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    K, V = pool.values("k") * 2.0 ** exps[0], pool.values("v") * 2.0 ** exps[1]
    check_attention(out, q, K, V, b, heads, kw.get("scale", hd ** -0.5), dt)
    return b, q, K, V, raw, out


def check_attention(out, q, k, v, b, heads, scale, dt):
    hq, hkv, hd = heads
    start = np.full((b.rows, hq * hd), 9.0)
    args = (b.table, b.offsets, b.lens, hq, hkv, hd)
    want = OP.paged_attention(q, k, v, *args, scale, start)
    B = OP.paged_attention(q, k, np.abs(v), *args, scale, np.zeros_like(start))
    lim, u = np.zeros_like(start), HALF[dt]
    for s, (n, kv) in enumerate(b.seqs):
        j = np.arange(kv)
        K = np.abs(k[b.table[s][j // b.page], j % b.page]).reshape(kv, hkv, hd) if kv else np.zeros((0, hkv, hd))
        for i in range(n):
            r, p = b.offsets[s] + i, kv - n + i
            for h in range(hq if p >= 0 else 0):
                c = slice(h * hd, (h + 1) * hd)
                A = scale * (K[:p + 1, h // (hq // hkv)] @ np.abs(q[r, c].astype(np.float64))).max()
                d = (2 * hd + 2 * hd + 4) * F * A + 8 * F * (A + 1) + 4 * F
                lim[r, c] = (2 * d + 2 * (p + 1) * F + (2.0 ** -11 if dt == torch.bfloat16 else 2.0 ** -22)) * B[r, c] \
                    + u * np.abs(want[r, c])
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
    ((6, 2, 128), 8, [(50, 333), (43, 43)]),
    ((12, 1, 64), 8, [(23, 71)]),
    ((16, 2, 128), 16, [(300, 900)]),
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
    attention_case(np.random.default_rng(n + kv), dt, heads, 32, [(n, kv)], std=2.0)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads,page", [((8, 8, 128), 16), ((32, 16, 64), 8)])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_attention_long_loops(dt, heads, page, n):
    """Enough tiles that no range is split far: every stage is used many times."""
    rng = np.random.default_rng(n)
    seqs = [(n, int(rng.integers(1200, 3000))) for _ in range(26 if n < 20 else 8)]
    attention_case(rng, dt, heads, page, seqs)


def plan(n_rows, seqs, max_kv, heads, dt):
    import ctypes
    out = (ctypes.c_int64 * 6)()
    assert L.lib.cb_debug_paged4_plan(n_rows, seqs, max_kv, *heads, R.dtype_code(dt), out) == L.CB_OK
    return list(out)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,group,tile", [(1, 4, 8), (3, 4, 16), (7, 4, 16), (1, 64, 32)])
@pytest.mark.parametrize("kv,cluster", [(200, 1), (500, 2), (1000, 4), (2000, 8), (4001, 16)])
def test_tiles_in_clusters(dt, hd, n, group, tile, kv, cluster):
    """Every cluster size and tile of the one-launch form, by the plan that leads to it; lengths
    that leave some of a cluster's blocks without keys."""
    heads = (8, 2, hd) if group == 4 else (group, 1, hd)
    tile = min(tile, 16 if dt == torch.float32 else 32)
    assert plan(n, 1, kv, heads, dt)[:2] == [tile, cluster]
    rng = np.random.default_rng(n + kv)
    attention_case(rng, dt, heads, 16, [(n, kv)], max_kv_len=kv)
    attention_case(rng, dt, heads, 8, [(n, 37)], max_kv_len=kv, tail=1)
    if tile == 8:       # several sequences, one without keys, one without rows
        seqs = [(1, kv), (1, 0), (0, 9), (1, 33)]
        assert plan(3, 4, kv, heads, dt)[1] > 0
        attention_case(rng, dt, heads, 32, seqs, max_kv_len=kv)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("n,group,tile", [(1, 4, 8), (3, 4, 16), (7, 4, 16), (1, 64, 32)])
def test_tiles_on_the_line(dt, n, group, tile):
    """Many tiles, with and without padding behind them, pieces in several parts."""
    rng = np.random.default_rng(n)
    for hd, count, kv in ((64, 160, 300), (128, 160, 200), (64, 3, 9000)):
        heads, seqs = (2 * group, 2, hd), [(n, int(rng.integers(max(n, kv // 3), kv))) for _ in range(count)]
        bound = 40000 if count == 3 else kv
        tile = min(tile, 16 if dt == torch.float32 else 32)
        assert plan(n * count, count, bound, heads, dt)[:2] == [tile, 0]
        attention_case(rng, dt, heads, 16, seqs, max_kv_len=bound)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("seqs,unit,split", [
    ([(64, 3200)], 128, True),                  # few tiles over many keys: joined parts
    ([(300, 900)], 128, True),
    ([(600, 700), (512, 512), (500, 2000), (900, 1500)], 0, False),
])
def test_chunks_by_plan(hd, seqs, unit, split):
    heads, rows = (16, 4, hd), sum(n for n, _ in seqs)
    p = plan(rows, len(seqs), max(kv for _, kv in seqs), heads, torch.bfloat16)
    assert p[3] == unit or (unit == 0 and p[3] in (128, 256))
    assert (p[4] > 1) or not split
    rng = np.random.default_rng(rows)
    attention_case(rng, torch.bfloat16, heads, 16, seqs, max_kv_len=max(kv for _, kv in seqs), exps=(1, -2))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("page", [8, 32, 256])
def test_chunks_of_256_rows(hd, page):
    """Units of 256 rows (two tiles share each block), whole and with one tile alone."""
    heads, seqs = (32, 8, hd), [(450, 520), (130, 200), (33, 33), (9, 300), (1, 77)]
    p = plan(4096, 4, 4096, heads, torch.bfloat16)
    assert p[3] == 256
    rng = np.random.default_rng(page)
    # the plan follows bounds: many rows in the call, few of them in sequences
    attention_case(rng, torch.bfloat16, heads, page, seqs, tail=3500, max_kv_len=4096)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("heads", [(8, 2, 128), (7, 1, 64), (5, 1, 128)])
def test_attention_mixed_lengths_in_one_call(dt, heads):
    rng = np.random.default_rng(3)
    attention_case(rng, dt, heads, 16, [(1, 900), (40, 300), (1, 0), (4, 77), (150, 700), (1, 1), (2, 64)], tail=1)


@pytest.mark.parametrize("dt", list(HALF))
def test_exponents_scales_and_loose_bounds(dt):
    rng = np.random.default_rng(8)
    attention_case(rng, dt, (8, 2, 128), 16, [(1, 300), (9, 130)], exps=(-2, 3))
    attention_case(rng, dt, (8, 2, 64), 16, [(1, 300), (3, 130)], exps=(1, -60), scale=0.03)
    attention_case(rng, dt, (8, 2, 64), 16, [(1, 40), (3, 130)], scale=0.0)
    attention_case(rng, dt, (8, 2, 128), 32, [(2, 300), (40, 200)], max_kv_len=320, extra=48)


@pytest.mark.parametrize("dt", list(HALF))
@pytest.mark.parametrize("std", [1e-30, 1e-6, 3e4])
def test_queries_of_any_magnitude(dt, std):
    """q meets the tensor cores as fp16 behind a power of two per row: values far
    outside of fp16's range count as others do."""
    rng = np.random.default_rng(4)
    attention_case(rng, dt, (8, 2, 128), 16, [(1, 300), (20, 130)], std=std, scale=0.1 / std)


@pytest.mark.parametrize("dt", list(HALF))
def test_strided_rows_another_stream_and_a_recorded_call(dt):
    rng = np.random.default_rng(6)
    b, q, K, V, raw, ref = attention_case(rng, dt, (8, 2, 64), 16, [(1, 200), (5, 90), (1, 0)])
    wide_q = torch.zeros(b.rows, 512 + 64, dtype=dt, device="cuda")
    wide_q[:, 64:] = dev(q, dt)
    wide_o = torch.full((b.rows, 1024), 5.0, dtype=dt, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (*b.dev(), raw, 16, 8, 2, 64)
    R.cb_paged4_attention(wide_q[:, 64:], *args, wide_o[:, 256:768], stream=s)
    s.synchronize()
    assert torch.equal(wide_o[:, 256:768], ref) and (wide_o[:, :256] == 5).all() and (wide_o[:, 768:] == 5).all()
    # a recorded call follows the lengths of the moment it is replayed
    out = torch.zeros(b.rows, 512, dtype=dt, device="cuda")
    ws = R.cb_paged4_attention_workspace(ref, 3, 256, 8, 2, 64)
    off, lens, table = b.dev()
    qd, gr = dev(q, dt), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        R.cb_paged4_attention(qd, off, lens, table, raw, 16, 8, 2, 64, out, max_kv_len=256, ws=ws)
    gr.replay()
    assert torch.equal(out, ref)
    lens.copy_(ints([150, 40, 0]))
    gr.replay()
    torch.cuda.synchronize()
    b.seqs, b.lens = [(1, 150), (5, 40), (1, 0)], np.array([150, 40, 0])
    check_attention(out, q, K, V, b, (8, 2, 64), 0.125, dt)
    assert R.device_status() == 0


def test_attention_errors_on_the_device():
    dt = torch.bfloat16
    pool = torch.zeros(4, R.cb_paged4_page_bytes(8, 2, 64), dtype=torch.uint8, device="cuda")
    q = torch.ones(4, 256, dtype=dt, device="cuda")

    def run(offsets, lens, tbl, **kw):
        out = torch.full((4, 256), 9.0, dtype=dt, device="cuda")
        R.cb_paged4_attention(q, ints(offsets), ints(lens), ints(tbl), pool, 8, 4, 2, 64, out, **kw)
        torch.cuda.synchronize()
        return R.device_status(), [int(x) for x in (out == 9.0).all(1)]
    bad = L.CB_ERR_DEVICE_INDEX
    assert run([0, 2, 4], [8, 9], [[0, 1], [2, 3]]) == (0, [0, 0, 0, 0])
    assert run([0, 2, 4], [8, 9], [[0, 1], [2, 4]])[0] == bad
    assert run([0, 2, 4], [8, 9], [[-1, 1], [2, 3]])[0] == bad
    assert run([0, 2, 4], [8, 17], [[0, 1], [2, 3]]) == (bad, [0, 0, 1, 1])
    assert run([0, 2, 4], [-1, 9], [[0, 1], [2, 3]]) == (bad, [1, 1, 0, 0])
    assert run([0, 2, 4], [8, 9], [[0, 1], [2, 3]], max_kv_len=8) == (bad, [0, 0, 1, 1])
    assert run([0, 2, 1], [8, 9], [[0, 1], [2, 3]])[0] == bad
    assert run([0, 2, 2], [8, 9], [[0, 1], [2, 3]]) == (0, [0, 0, 1, 1])            # padding behind the last row
