"""Host-side refusals of the generation operators (no device needed) and hand
values of their float64 oracle."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from oracle import paged as OP
from rag_kv_cache_layer_gb300 import _lib as L

A = 4096             # an aligned address that validation never follows


def _kv(**kw):
    d = dict(k_pages=4096, v_pages=4096, page_stride=16 * 256, ld=256, n_pages=4, page_size=16,
             block_table=4096, ld_table=8, max_pages=8, row_offsets=4096, kv_lens=4096, n_seq=2)
    d.update(kw)
    return L.packer(L.PagedKV)(*[d[f] for f, _ in L.PagedKV._fields_])


def _append(kv=None, dt=L.CB_BF16, **kw):
    d = dict(k=A, v=A, ld_k=256, ld_v=256, k_layer_stride=0, v_layer_stride=0, cache_layer_stride=0, n_rows=3,
             n_layers=1, n_kv_heads=2, head_dim=128, rope_table=A, q=0, q_out=0, ld_q=0, ld_q_out=0, n_q_heads=0,
             max_positions=64)
    d.update(kw)
    rows = L.packer(L.PagedRows)(*[d[f] for f, _ in L.PagedRows._fields_])
    return L.lib.cb_paged_append(_kv() if kv is None else kv, rows, dt, None)


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
    dict(k=0), dict(v=0), dict(k=4098), dict(ld_k=255), dict(ld_v=128), dict(n_rows=-1), dict(n_layers=-1),
    dict(n_layers=65536), dict(n_layers=2, k_layer_stride=4), dict(n_layers=2, v_layer_stride=4),
    dict(n_layers=2, cache_layer_stride=4), dict(n_kv_heads=0), dict(head_dim=120), dict(head_dim=0), dict(dt=7),
    dict(rope_table=4100), dict(max_positions=0),
    dict(q=A, ld_q=512, n_q_heads=4), dict(q_out=A, ld_q_out=512, n_q_heads=4),     # only one of the two
    dict(q=A, ld_q=512, q_out=A, ld_q_out=512, n_q_heads=0), dict(q=A, ld_q=504, q_out=A, ld_q_out=512, n_q_heads=4),
    dict(q=A, ld_q=512, q_out=A, ld_q_out=512, n_q_heads=4, rope_table=0),          # nothing to rotate by
    dict(q=A, ld_q=512, q_out=A, ld_q_out=512, n_q_heads=4, n_layers=2)])
def test_append_refusals(kw):
    assert _append(**kw) == L.CB_ERR_INVALID_ARG
    assert L.lib.cb_last_error_message()


def test_empty_calls_are_done():
    assert _append(n_rows=0, k=0, v=0) == L.CB_OK
    assert _append(n_layers=0, k=0) == L.CB_OK
    assert _append(_kv(n_seq=0, row_offsets=0, kv_lens=0, block_table=0)) == L.CB_OK
    assert _attn(n_rows=0, q=0) == L.CB_OK
    assert _attn(_kv(n_seq=0, row_offsets=0, kv_lens=0, block_table=0)) == L.CB_OK
    assert L.lib.cb_sample_tokens(None, 8, 0, 8, 0, None, None, None, None, None, None, None) == L.CB_OK


def test_null_structures():
    kv = _kv()
    rows, query = bytes(C.sizeof(L.PagedRows)), bytes(C.sizeof(L.PagedQuery))
    for call, arg in ((L.lib.cb_paged_append, rows), (L.lib.cb_paged_attention, query)):
        assert call(None, arg, L.CB_BF16, None) == L.CB_ERR_INVALID_ARG
        assert call(kv, None, L.CB_BF16, None) == L.CB_ERR_INVALID_ARG
        assert call(kv, arg, L.CB_BF16, None) == L.CB_ERR_INVALID_ARG          # zeros in every field


STRUCTS = {"cb_paged_kv": L.PagedKV, "cb_paged_rows": L.PagedRows, "cb_paged_query": L.PagedQuery}


def test_ctypes_mirrors_match_c_layout(tmp_path):
    """Sizes and offsets as the C compiler sees them, and as packed."""
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "cacheblend.h"', "int main(void) {"]
    for name, cls in STRUCTS.items():
        src.append(f'printf("{name} %zu\\n", sizeof({name}));')
        src += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(src + ["return 0; }"]))
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c99", "-I", inc, str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = dict(x.rsplit(" ", 1) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                                        check=True).stdout.strip().splitlines())
    for name, cls in STRUCTS.items():
        assert int(got[name]) == C.sizeof(cls)
        values = []
        for i, (f, t) in enumerate(cls._fields_):
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)
            values.append(i + 1)
        back = cls.from_buffer_copy(L.packer(cls)(*values))
        assert [getattr(back, f) for f, _ in cls._fields_] == values


def _attn(kv=None, dt=L.CB_BF16, **kw):
    d = dict(q=A, out=A, ld_q=512, ld_out=512, ws=A, ws_bytes=1 << 30, n_rows=3, max_kv_len=64, n_q_heads=4,
             n_kv_heads=2, head_dim=128, scale=0.1)
    d.update(kw)
    query = L.packer(L.PagedQuery)(*[d[f] for f, _ in L.PagedQuery._fields_])
    return L.lib.cb_paged_attention(_kv() if kv is None else kv, query, dt, None)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(out=0), dict(q=4104), dict(ld_q=504), dict(ld_out=508), dict(n_rows=-1), dict(max_kv_len=-1),
    dict(n_q_heads=3), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_q_heads=258, n_kv_heads=2), dict(head_dim=96),
    dict(dt=2), dict(scale=-0.1), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_attention_refusals(kw):
    assert _attn(**kw) == L.CB_ERR_INVALID_ARG


def test_limits_of_lengths_scales_and_layers():
    """Key indices stay below 2^31 with a block's reach to spare, the scale in
    the log2 domain is finite, and no two layers append to one place."""
    assert _attn(max_kv_len=L.CB_MAX_KV_LEN + 1) == L.CB_ERR_UNSUPPORTED
    assert _attn(max_kv_len=2 ** 31 - 1) == L.CB_ERR_UNSUPPORTED
    assert _attn(scale=3e38) == L.CB_ERR_INVALID_ARG
    assert _append(n_layers=2, cache_layer_stride=0) == L.CB_ERR_INVALID_ARG
    assert L.CB_MAX_KV_LEN == 1 << 30


def test_attention_workspace():
    size = L.lib.cb_paged_attention_workspace_size
    need = size(1, 1, 100000, 32, 8, 128, L.CB_BF16)
    assert need > 256                       # one row over many keys: the range is split
    kw = dict(kv=_kv(ld=1024, page_stride=16 * 1024, n_seq=1), n_rows=1, max_kv_len=100000, n_q_heads=32,
              n_kv_heads=8, ld_q=4096, ld_out=4096)
    assert _attn(ws=0, **kw) == L.CB_ERR_WORKSPACE
    assert _attn(ws_bytes=need - 1, **kw) == L.CB_ERR_WORKSPACE
    assert _attn(ws=4100, **kw) == L.CB_ERR_WORKSPACE
    for bad in [(-1, 1, 8, 4, 2, 128, 1), (1, 1025, 8, 4, 2, 128, 1), (1, 1, 8, 3, 2, 128, 1), (1, 1, 8, 4, 2, 80, 1)]:
        assert size(*bad) == 256


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(u=None), dict(tokens=None), dict(ld=999), dict(rows=-1), dict(rows=(1 << 20) + 1),
    dict(vocab=0), dict(dt=2), dict(logits=4098), dict(u=4097), dict(topk=4098)])
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


def test_plan_query():
    """What a call of given sizes runs, and its workspace from that."""
    def plan(*a):
        out = (C.c_int64 * 7)(*[-5] * 7)
        st = L.lib.cb_debug_paged_plan(*a, out)
        return list(out) if st == L.CB_OK else st
    size = L.lib.cb_paged_attention_workspace_size
    for a in [(1, 1, 100000, 32, 8, 128), (64, 1, 3200, 32, 8, 128), (8192, 4, 8192, 32, 8, 128), (127, 64, 16384, 32, 8, 128),
              (2000, 1, 30000, 24, 8, 64), (300, 1, 9000, 32, 16, 64), (60, 300, 60, 4, 2, 64)]:
        for dt in (L.CB_BF16, L.CB_F32):
            tile, hc, grid, unit, parts, units, limit = plan(*a, dt)
            hkv, hd = a[4], a[5]
            assert tile in (0, 16, 32, 64) and unit in (0, 128, 256) and (tile or unit) and grid > 0 and parts >= 1
            assert not (unit and dt == L.CB_F32) and hc in (1, 64 // tile if tile else 1)
            assert limit == (0 if not tile else 64 if unit else 0x7fffffff)
            few = 2 * grid * tile * hc * (4 * hd + 8) + 24 * grid if tile else 0
            chunk = units * hkv * parts * unit * (4 * hd + 8) if parts > 1 else 0
            assert size(*a, dt) == max(256, few, chunk)
    assert plan(64, 1, 3200, 32, 8, 128, L.CB_BF16)[3] == 128 and plan(1, 1, 3200, 32, 8, 128, L.CB_BF16)[:1] == [16]
    for bad in [(0, 1, 8, 4, 2, 128, 1), (1, 0, 8, 4, 2, 128, 1), (1, 1025, 8, 4, 2, 128, 1), (1, 1, -1, 4, 2, 128, 1),
                (1, 1, L.CB_MAX_KV_LEN + 1, 4, 2, 128, 1), (1, 1, 8, 3, 2, 128, 1), (1, 1, 8, 4, 2, 80, 1), (1, 1, 8, 4, 2, 128, 2)]:
        assert plan(*bad) == L.CB_ERR_INVALID_ARG
    assert L.lib.cb_debug_paged_plan(1, 1, 8, 4, 2, 128, L.CB_BF16, None) == L.CB_ERR_INVALID_ARG


def test_a_workspace_with_gaps_or_repeats_is_refused(monkeypatch):
    """Its byte count would not be that of the memory behind its address.  Host
    tensors stand for device ones: the wrapper compares device indices, and the
    library is not reached."""
    from rag_kv_cache_layer_gb300 import api
    calls = []

    class Lib:
        def cb_paged_attention(self, *args):
            calls.append(args)
            return L.CB_OK
    monkeypatch.setattr(api, "_cur_device", lambda: -1)
    monkeypatch.setattr(api, "_cur_stream", lambda dev: 0)
    monkeypatch.setattr(api, "lib", Lib())
    ints = lambda x: torch.tensor(x, dtype=torch.int32)
    kp, q = torch.zeros(4, 16, 128), torch.zeros(1, 256)
    run = lambda ws: api.cb_paged_attention(q, ints([0, 1]), ints([1]), ints([[0]]), kp, kp, 4, 2, 64,
                                            torch.zeros_like(q), ws=ws)
    run(torch.empty(1 << 16, dtype=torch.uint8))
    assert len(calls) == 1
    for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 24), torch.empty(1 << 16, dtype=torch.uint8)[::2],
               torch.empty(64, 64).t()):
        with pytest.raises(ValueError, match="contiguous"):
            run(ws)
    assert len(calls) == 1


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
def _blocks(base, row, G, BN):
    """Key blocks that row `row` (query x G + head) of a sequence sees, at least one."""
    seen = base + row // G + 1
    return (seen - 1) // BN + 1 if seen > 0 else 1


def _line(seqs, heads, G, R, BN, grid, per):
    """The few-rows kernel's partition, restated: (part, item, first block, end
    block, slot or None) of every piece, and (item, slots) of every join.  seqs:
    (new rows, length); an item is a tile for one group of heads; per: units a
    part has at least (4 where the block's groups share a head, else 1)."""
    tiles = [-(-n * G // R) for n, _ in seqs]
    pair, units = [], []
    for (n, kv), t in zip(seqs, tiles):
        b = lambda row: _blocks(kv - n, row, G, BN)
        pair.append(0 if t == 0 else b(n * G - 1) if t == 1 else b(R - 1) + b(t * R - 1) + 2)
        mid = 0 if t % 2 == 0 else pair[-1] if t == 1 else b((t // 2 + 1) * R - 1)
        units.append(heads * (t // 2 * pair[-1] + mid))
    begin = np.concatenate([[0], np.cumsum(units)])
    total = int(begin[-1])
    parts = min((total + per - 1) // per, grid)
    if len(seqs) == 1 and total // pair[0] < parts:
        parts -= parts % (total // pair[0])
    pb = lambda c: c * total // parts
    part_of = lambda u: ((u + 1) * parts - 1) // total
    seq = lambda u: max(s for s in range(len(seqs)) if begin[s] <= u)
    pieces, joins = [], []
    for c in range(parts):
        u, u1 = pb(c), pb(c + 1)
        s = seq(u)
        while u < u1:
            while pair[s] == 0 or (s + 1 < len(seqs) and begin[s + 1] <= u):
                s += 1
            n, kv = seqs[s]
            t, local, size = tiles[s], int(u - begin[s]), pair[s]
            pairs = t // 2 * heads * size
            if local >= pairs:
                k = t // 2
                size = size if t == 1 else _blocks(kv - n, (k + 1) * R - 1, G, BN)
                g, jb = divmod(local - pairs, size)
            else:
                ph, jb = divmod(local, size)
                q, g = divmod(ph, heads)
                late = _blocks(kv - n, min((t - q) * R, n * G) - 1, G, BN)
                k, size, jb = (t - 1 - q, late, jb) if jb < late else (q, size - late, jb - late)
            item = (s, k, g)
            take, first, end = min(size - jb, u1 - u), u == pb(c), u - jb + size
            u += take
            whole = jb == 0 and take == size
            pieces.append((c, item, jb, jb + take, size, None if whole else 2 * c + (not first)))
            if u == u1 and jb == 0 and end > u1:
                last = part_of(end - 1)
                assert pb(last) <= end - 1 < pb(last + 1)
                joins.append((item, [2 * c + (not first)] + [2 * x for x in range(c + 1, last + 1)]))
    return tiles, pieces, joins


@pytest.mark.parametrize("seed", range(120))
def test_every_unit_once_and_every_split_item_joined_once(seed):
    rng = np.random.default_rng(seed)
    G, R, BN, heads = (int(rng.choice(x)) for x in ([1, 2, 4, 7, 128], [16, 32, 64], [8, 16, 32], [1, 2, 5]))
    seqs = []
    for _ in range(int(rng.integers(1, 9)) if seed % 3 else 1):
        n = int(rng.choice([0, 1, 1, 2, 5, rng.integers(1, [40, 300][seed % 2])]))
        seqs.append((n, int(rng.choice([0, n, n // 2, n + rng.integers(0, 900)]))))
    if not any(n for n, _ in seqs):
        seqs[0] = (2, 40)
    tiles, pieces, joins = _line(seqs, heads, G, R, BN, int(rng.integers(1, 60)), [1, 4][seed % 2])
    seen = {}
    for c, item, jb, je, size, slot in pieces:
        assert jb < je <= size
        seen.setdefault(item, []).append((jb, je, slot, size))
    for s, (n, kv) in enumerate(seqs):
        for k in range(tiles[s]):
            need = _blocks(kv - n, min((k + 1) * R, n * G) - 1, G, BN)
            for g in range(heads):
                got = sorted(seen.pop((s, k, g)), key=lambda x: x[0])
                assert [x[0] for x in got] == [0] + [x[1] for x in got[:-1]] and got[-1][1] == got[0][3] >= need
                slots = [x[2] for x in got]
                found = [j for i, j in joins if i == (s, k, g)]
                assert found == ([] if slots == [None] else [slots])
    assert not seen
    used = [x[5] for x in pieces if x[5] is not None]
    assert len(used) == len(set(used))
    if len(seqs) == 1 and tiles[0] == 1:      # items of one length: no part has pieces of two
        owners = [p[0] for p in pieces]
        assert heads > len(set(owners)) or len(owners) == len(set(owners))
