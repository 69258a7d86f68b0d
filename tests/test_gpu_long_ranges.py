"""The operators for long contexts at the ends of their ranges: rows of any width, many rows
of many layers, pages behind 2^32 bytes of a pool, as many sequences as a call takes, calls
on two streams at once.  What a call gives does not depend on where its pages lie or on what
runs beside it: those results are compared for equality."""
import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from oracle import paged as OP
from oracle import paged4 as O4
from test_gpu_paged import Batch, f64, ints, vals
from test_gpu_paged4 import attention_case
from test_gpu_picked import picked_case, select_case

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield
    torch.cuda.synchronize()
    assert R.device_status() == 0


def dev(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("heads,hd,layers,rows", [
    (1, 64, 2, 33), (5, 128, 1, 100), (3, 64, 16, 1000), (40, 128, 2, 70), (64, 128, 1, 3), (1, 64, 20, 2100), (7, 64, 30, 450)])
def test_rows_of_any_width_and_number(dt, heads, hd, layers, rows):
    """Rows of 8 to 1024 units a thread each, blocks of one row to 32, not rotated: two
    sequences, rows behind the last one."""
    rng = np.random.default_rng(rows)
    b = Batch(rng, [(rows - 1, rows + 4), (1, 9)], 16, dt, heads, hd, tail=2)
    k, v = (torch.randn(layers, rows + 2, heads * hd, device="cuda").to(dt) for _ in range(2))
    pool = torch.zeros(layers, b.n_pages, R.cb_paged4_page_bytes(16, heads, hd), dtype=torch.uint8, device="cuda")
    out = torch.full((2, layers, rows + 2, heads * hd), 7.0, dtype=dt, device="cuda")
    R.cb_paged4_append(k, v, *b.dev(), pool, 16, hd)
    R.cb_paged4_gather(*b.dev(), pool, 16, hd, out[0], out[1])
    torch.cuda.synchronize()
    assert (out[:, :, rows:] == 7).all()
    for x, y in ((k, out[0]), (v, out[1])):
        l = int(rng.integers(layers))
        assert np.array_equal(f64(y[l, :rows]), O4.values(*O4.quantise(f64(x[l, :rows]))))
        again = torch.zeros_like(pool[:1])      # one layer alone: the same codes
        R.cb_paged4_append(k[l], v[l], *b.dev(), again[0], 16, hd)
        assert torch.equal(again[0], pool[l])


def test_pages_behind_4_gigabytes():
    """The same request in the pages at a small pool's start and in those at the end of a pool of
    more than 2^32 bytes (and of more than 2^32 elements of a 16-bit one): equal results."""
    hq, hkv, hd, page, dt = 8, 2, 128, 16, torch.bfloat16
    kv, n, kvw = 600, 3, hkv * hd
    need, far = -(-kv // page), (2 ** 32 + 2 ** 26) // (page * kvw) + 1
    torch.manual_seed(0)
    k, v = (torch.randn(kv, kvw, device="cuda").to(dt) for _ in range(2))
    q = torch.randn(n, hq * hd, device="cuda").to(dt)
    off, lens, rows = ints([0, n]), ints([kv]), ints([0, kv])
    big = [torch.zeros(far, page, kvw, dtype=dt, device="cuda") for _ in range(2)]
    got = []
    for first, pools in ((0, [x[:need].clone() for x in big]), (far - need, big)):
        table = (torch.randperm(need, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).int() + first)[None]
        total = pools[0].shape[0]
        R.cb_paged_append(k, v, rows, lens, table, *pools, hd)
        bounds = torch.zeros(total, 2, kvw, dtype=dt, device="cuda")
        R.cb_paged_bounds(rows, lens, table, pools[0], bounds, kv)
        picks = torch.zeros(n, hkv, 9, dtype=torch.int32, device="cuda")
        R.cb_paged_select(q, off, lens, table, bounds, page, hq, hkv, hd, picks)
        picked = torch.zeros_like(q)
        R.cb_paged_attention_picked(q, off, lens, table, *pools, picks, hq, hkv, hd, picked)
        got.append([picks, picked, bounds[table[0].long()]])
        del bounds
    del big, pools
    size = R.cb_paged4_page_bytes(page, hkv, hd)
    far = (2 ** 32 + 2 ** 26) // size + 1
    big = torch.zeros(far, size, dtype=torch.uint8, device="cuda")
    for i, (first, pool) in enumerate(((0, big[:need].clone()), (far - need, big))):
        table = (torch.arange(need, device="cuda").int() + first)[None]
        R.cb_paged4_append(k, v, rows, lens, table, pool, page, hd)
        kb, vb, few, many = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(q).repeat(50, 1)
        R.cb_paged4_gather(rows, lens, table, pool, page, hd, kb, vb)
        R.cb_paged4_attention(q, off, lens, table, pool, page, hq, hkv, hd, few)
        R.cb_paged4_attention(q.repeat(50, 1), ints([0, 150]), lens, table, pool, page, hq, hkv, hd, many)
        got[i] += [kb, vb, few, many]
    torch.cuda.synchronize()
    for a, c in zip(*got):
        assert torch.equal(a, c) and bool(a.any())


@pytest.mark.parametrize("dt", DTYPES)
def test_as_many_sequences_as_a_call_takes(dt):
    rng = np.random.default_rng(7)
    seqs = [(int(i % 7 != 3), int(rng.integers(1, 90)) if i % 5 else 0) for i in range(1024)]
    heads = (4, 2, 64)
    attention_case(rng, dt, heads, 8, seqs, tail=3)
    picked_case(rng, dt, heads, 8, seqs, 3, tail=3)
    select_case(rng, dt, heads, 8, seqs, 4, tail=3)
    b = Batch(rng, seqs, 8, dt, 2, 64, tail=3)
    k, v = (dev(vals(rng, (b.rows, 128), dt), dt) for _ in range(2))
    pool = torch.zeros(b.n_pages, R.cb_paged4_page_bytes(8, 2, 64), dtype=torch.uint8, device="cuda")
    out = torch.full((2, b.rows, 128), 7.0, dtype=dt, device="cuda")
    R.cb_paged4_append(k, v, *b.dev(), pool, 8, 64)
    R.cb_paged4_gather(*b.dev(), pool, 8, 64, out[0], out[1])
    want = np.full((2, b.rows, 128), 7.0)
    for r, s, p in OP.row_positions(b.offsets, b.lens):
        if p >= 0:
            for i, x in enumerate((k, v)):
                want[i, r] = O4.values(*O4.quantise(f64(x[r:r + 1])))[0]
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("dt", DTYPES)
def test_the_largest_pages_groups_and_lists(dt):
    rng = np.random.default_rng(8)
    attention_case(rng, dt, (128, 1, 128), 1024, [(2, 1500), (1, 1024)], tail=1)
    attention_case(rng, dt, (128, 1, 64), 8, [(1, 40), (3, 700)])
    picked_case(rng, dt, (128, 1, 128), 1024, [(2, 3000)], 3)
    picked_case(rng, dt, (4, 2, 64), 8, [(2, 9000), (1, 3)], 1024)
    select_case(rng, dt, (128, 1, 64), 1024, [(2, 9000)], 4)
    select_case(rng, dt, (4, 2, 64), 8, [(1, 9000), (1, 8192)], 1024)


@pytest.mark.parametrize("dt", DTYPES)
def test_two_streams_at_once(dt):
    """Calls with workspaces of their own run beside each other; each gives what it gives alone."""
    rng = np.random.default_rng(9)
    sets = []
    for i in range(2):
        b, q, _, _, raw, out = attention_case(rng, dt, (8, 2, 64), 16, [(1, 3000 + 90 * j) for j in range(40 + i)])
        p, pq, _, _, dk, dv, picks, pout = picked_case(rng, dt, (8, 2, 64), 16, [(1, 2000 + 50 * j) for j in range(40 + i)], 60)
        sets.append((b.dev(), dev(q, dt), raw, out, p.dev(), dev(pq, dt), dk, dv, ints(picks), pout, torch.cuda.Stream(),
                     R.cb_paged4_attention_workspace(out, 40 + i, 8000, 8, 2, 64),
                     R.cb_paged_attention_picked_workspace(pout, 60, 16, 8, 2, 64),
                     torch.zeros(20, *out.shape, dtype=dt, device="cuda"), torch.zeros(20, *pout.shape, dtype=dt, device="cuda")))
    torch.cuda.synchronize()
    for i in range(20):
        for bd, q, raw, out, pd, pq, dk, dv, picks, pout, stream, ws4, wsp, o, po in sets:
            R.cb_paged4_attention(q, *bd, raw, 16, 8, 2, 64, o[i], max_kv_len=8000, ws=ws4, stream=stream)
            R.cb_paged_attention_picked(pq, *pd, dk, dv, picks, 8, 2, 64, po[i], ws=wsp, stream=stream)
    torch.cuda.synchronize()
    for bd, q, raw, out, pd, pq, dk, dv, picks, pout, stream, ws4, wsp, o, po in sets:
        one = torch.empty_like(out)     # (the bound of the lengths may choose another form than the case's)
        R.cb_paged4_attention(q, *bd, raw, 16, 8, 2, 64, one, max_kv_len=8000, ws=ws4)
        torch.cuda.synchronize()
        assert (o == one).all() and (po == pout).all()
