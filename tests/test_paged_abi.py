"""Host-side refusals of the generation operators (no device needed) and hand
values of their float64 oracle."""
import ctypes as C

import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from oracle import paged as OP
from rag_kv_cache_layer_gb300 import _lib as L

P = C.c_void_p
A = P(4096)          # an aligned address that validation never follows


def _kv(**kw):
    d = dict(k_pages=4096, v_pages=4096, page_stride=16 * 256, ld=256, n_pages=4, page_size=16,
             block_table=4096, ld_table=8, max_pages=8, row_offsets=4096, kv_lens=4096, n_seq=2)
    d.update(kw)
    return L.PagedKV(*[d[f] for f, _ in L.PagedKV._fields_])


def _append(kv=None, k=A, ld_k=256, ks=0, v=A, ld_v=256, vs=0, rows=3, layers=1, cs=0, heads=2, hd=128,
            rope=A, maxp=64, q=None, ld_q=0, nq=0, qo=None, ld_qo=0, dt=L.CB_BF16):
    kv = _kv() if kv is None else kv
    return L.lib.cb_paged_append(C.byref(kv) if kv else None, k, ld_k, ks, v, ld_v, vs, rows, layers, cs, heads,
                                 hd, rope, maxp, q, ld_q, nq, qo, ld_qo, dt, None)


BAD_KV = [dict(k_pages=0), dict(v_pages=4098), dict(ld=248), dict(ld=260), dict(page_stride=256),
          dict(n_pages=0), dict(n_seq=-1), dict(n_seq=1025), dict(ld_table=7), dict(max_pages=-1),
          dict(block_table=0), dict(row_offsets=0), dict(kv_lens=0), dict(kv_lens=4098)]
BAD_PAGE = [dict(page_size=0), dict(page_size=4), dict(page_size=24), dict(page_size=2048)]


@pytest.mark.parametrize("kw", BAD_KV)
def test_paged_geometry_is_refused(kw):
    assert _append(_kv(**kw)) == L.CB_ERR_INVALID_ARG
    assert _attn(_kv(**kw)) == L.CB_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_PAGE)
def test_page_size_is_refused(kw):
    kw = dict(kw, page_stride=1 << 22)
    assert _append(_kv(**kw)) == L.CB_ERR_UNSUPPORTED
    assert _attn(_kv(**kw)) == L.CB_ERR_UNSUPPORTED
    assert "page_size" in L.lib.cb_last_error_message().decode()


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k=P(4098)), dict(ld_k=255), dict(ld_v=128), dict(rows=-1),
    dict(layers=-1), dict(layers=65536), dict(layers=2, ks=4, cs=8), dict(layers=2, ks=8, cs=4), dict(heads=0),
    dict(hd=120), dict(hd=0), dict(dt=7), dict(rope=P(4100)), dict(maxp=0),
    dict(q=A, ld_q=512, nq=4), dict(qo=A, ld_qo=512, nq=4),            # only one of the two
    dict(q=A, ld_q=512, qo=A, ld_qo=512, nq=0), dict(q=A, ld_q=504, qo=A, ld_qo=512, nq=4),
    dict(q=A, ld_q=512, qo=A, ld_qo=512, nq=4, rope=None),             # nothing to rotate by
    dict(q=A, ld_q=512, qo=A, ld_qo=512, nq=4, layers=2)])
def test_append_refusals(kw):
    assert _append(**kw) == L.CB_ERR_INVALID_ARG
    assert L.lib.cb_last_error_message()


def test_empty_calls_are_done():
    assert _append(rows=0, k=None, v=None) == L.CB_OK
    assert _append(layers=0, k=None) == L.CB_OK
    assert _append(_kv(n_seq=0, row_offsets=0, kv_lens=0, block_table=0)) == L.CB_OK
    assert _attn(rows=0, q=None) == L.CB_OK
    assert _attn(_kv(n_seq=0, row_offsets=0, kv_lens=0, block_table=0)) == L.CB_OK
    assert L.lib.cb_sample_tokens(None, 8, 0, 8, 0, None, None, None, None, None, None, None) == L.CB_OK


def _attn(kv=None, q=A, ld_q=512, rows=3, max_kv=64, hq=4, hkv=2, hd=128, out=A, ld_out=512, dt=L.CB_BF16,
          ws=A, wsb=1 << 30, scale=0.1):
    kv = _kv() if kv is None else kv
    return L.lib.cb_paged_attention(C.byref(kv) if kv else None, q, ld_q, rows, max_kv, hq, hkv, hd, scale, out,
                                    ld_out, dt, ws, wsb, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(q=P(4104)), dict(ld_q=504), dict(ld_out=508), dict(rows=-1), dict(max_kv=-1),
    dict(hq=3), dict(hq=0), dict(hkv=0), dict(hq=258, hkv=2), dict(hd=96), dict(dt=2),
    dict(scale=-0.1), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_attention_refusals(kw):
    assert _attn(**kw) == L.CB_ERR_INVALID_ARG


def test_attention_workspace():
    size = L.lib.cb_paged_attention_workspace_size
    need = size(1, 1, 100000, 32, 8, 128, L.CB_BF16)
    assert need > 256                       # one row over many keys: the range is split
    kv = _kv(ld=1024, page_stride=16 * 1024, n_seq=1)
    kw = dict(kv=kv, rows=1, max_kv=100000, hq=32, hkv=8, ld_q=4096, ld_out=4096)
    assert _attn(ws=None, **kw) == L.CB_ERR_WORKSPACE
    assert _attn(wsb=need - 1, **kw) == L.CB_ERR_WORKSPACE
    assert _attn(ws=P(4100), **kw) == L.CB_ERR_WORKSPACE
    for bad in [(-1, 1, 8, 4, 2, 128, 1), (1, 1025, 8, 4, 2, 128, 1), (1, 1, 8, 3, 2, 128, 1), (1, 1, 8, 4, 2, 80, 1)]:
        assert size(*bad) == 256


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(u=None), dict(tokens=None), dict(ld=999), dict(rows=-1), dict(rows=(1 << 20) + 1),
    dict(vocab=0), dict(dt=2), dict(logits=P(4098)), dict(u=P(4097)), dict(topk=P(4098))])
def test_sample_refusals(kw):
    a = dict(logits=A, ld=1000, rows=2, vocab=1000, dt=L.CB_F32, u=A, t=None, topk=None, topp=None, minp=None,
             tokens=A)
    a.update(kw)
    assert L.lib.cb_sample_tokens(*a.values(), None) == L.CB_ERR_INVALID_ARG


def test_sample_vocab_limit():
    assert L.lib.cb_sample_tokens(A, 1 << 20, 1, (1 << 18) + 1, L.CB_F32, A, None, None, None, None, A, None) == \
        L.CB_ERR_UNSUPPORTED


def test_python_wrappers_refuse_host_tensors():
    if not torch.cuda.is_available():
        pytest.skip("needs a current device to compare with")
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        R.cb_sample_tokens(z, torch.zeros(2), torch.zeros(2, dtype=torch.int32))


# ------------------------------------------------------------------ oracle --
def test_oracle_attention_by_hand():
    # two keys, one query at position 1 and one at position 0; head_dim 2
    k = np.zeros((3, 8, 2)); v = np.zeros((3, 8, 2))
    k[2, 0], k[2, 1] = [1, 0], [0, 1]
    v[2, 0], v[2, 1] = [1, 2], [5, 6]
    q = np.array([[3.0, 0.0], [0.0, np.log(3.0)]])
    out = OP.paged_attention(q, k, v, [[2]], [0, 2], [2], 1, 1, 2, 1.0, np.zeros((2, 2)))
    np.testing.assert_allclose(out[0], [1, 2])                 # sees key 0 only
    np.testing.assert_allclose(out[1], [0.25 * 1 + 0.75 * 5, 0.25 * 2 + 0.75 * 6])


def test_oracle_append_by_hand():
    kp, vp = OP.paged_append(np.zeros((2, 8, 2)), np.zeros((2, 8, 2)), [[1, 0]], [0, 1], [9], np.array([[1.0, 0.0]]),
                             np.array([[7.0, 8.0]]), 2, base=10000.0)
    np.testing.assert_allclose(kp[0, 0], [np.cos(8), np.sin(8)])   # position 8: page 0 of the table's second entry
    np.testing.assert_allclose(vp[0, 0], [7, 8])
    assert not kp[1].any() and not vp[1].any()


def test_oracle_sampling_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    s = lambda u, **k: OP.sample_token(x, u, **k)
    assert [s(u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [s(u, top_k=2) for u in (0.0, 0.56, 0.58, 1.0)] == [1, 1, 3, 3]           # .4 / .7
    assert [s(u, top_p=0.75) for u in (0.0, 0.43, 0.45, 0.66, 0.67)] == [1, 1, 2, 2, 3]   # .4 .2 .3 of .9
    assert [s(u, min_p=0.6) for u in (0.1, 0.56, 0.58)] == [1, 1, 3]                 # 0.3 / 0.4 = 0.75 stays
    assert s(0.99, temperature=0.0) == 1 and s(0.99, top_p=0.0) == 1 and s(0.99, top_k=1) == 1
    assert OP.sample_token([-np.inf, np.nan], 0.3) == -1
    assert OP.sample_token([np.inf, 1.0, np.inf], 0.7) == 2
    assert OP.sample_token([2.0, 2.0, 2.0], 0.5, top_k=2) == 1                       # ties: lowest indices kept


# ----------------------------------------------------- the line of units --
def _line(units, blocks, grid):
    """The decode kernel's partition, restated: (part, item, first block, end
    block, slot or None) of every piece, and (item, slots) of every join.
    units: items per sequence; blocks: units per item (0: nothing)."""
    begin = np.concatenate([[0], np.cumsum([u * b for u, b in zip(units, blocks)])])
    total = int(begin[-1])
    parts = min((total + 3) // 4, grid)
    pb = lambda c: total * c // parts
    seq = lambda u: max(s for s in range(len(units)) if begin[s] <= u)
    pieces, joins = [], []
    for c in range(parts):
        u = pb(c)
        s = seq(u)
        while u < pb(c + 1):
            while blocks[s] == 0 or (s + 1 < len(units) and begin[s + 1] <= u):
                s += 1
            item, jb = divmod(int(u - begin[s]), blocks[s])
            take = min(blocks[s] - jb, pb(c + 1) - u)
            whole = jb == 0 and take == blocks[s]
            pieces.append((c, (s, item), jb, jb + take, None if whole else 2 * c + (u != pb(c))))
            u += take
    for c in range(1, parts):
        s = seq(pb(c))
        item = int(pb(c) - begin[s]) // blocks[s]
        a = int(begin[s]) + item * blocks[s]
        if pb(c) == a or pb(c - 1) > a:
            continue
        last = max(x for x in range(parts) if pb(x) <= a + blocks[s] - 1)
        joins.append(((s, item), [2 * x + (x == c - 1 and pb(x) != a) for x in range(c - 1, last + 1)]))
    return pieces, joins


@pytest.mark.parametrize("seed", range(60))
def test_every_unit_once_and_every_split_item_joined_once(seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 9))
    units = [int(rng.integers(0, 9)) for _ in range(n)]
    blocks = [int(rng.integers(1, [3, 30, 300][seed % 3])) if u else 0 for u in units]
    if not any(units):
        units[0], blocks[0] = 2, 5
    pieces, joins = _line(units, blocks, int(rng.integers(1, 40)))
    seen = {}
    for c, item, jb, je, slot in pieces:
        assert jb < je
        seen.setdefault(item, []).append((jb, je, slot))
    for s in range(n):
        for k in range(units[s]):
            got = sorted(seen.pop((s, k)))
            assert [x[0] for x in got] == [0] + [x[1] for x in got[:-1]] and got[-1][1] == blocks[s]
            slots = [x[2] for x in got]
            found = [j for i, j in joins if i == (s, k)]
            assert found == ([] if len(got) == 1 and slots == [None] else [slots])
    assert not seen
    used = [x[4] for x in pieces if x[4] is not None]
    assert len(used) == len(set(used))
