"""Host-side refusals of the 4-bit cache's and the picked pages' entry points (no
device needed), their structures, and hand values of their float64 oracle."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from oracle import paged4 as O4
from rag_kv_cache_layer_gb300 import _lib as L

A = 4096             # an aligned address that validation never follows


def packed(cls, d, kw):
    d = dict(d, **kw)
    return L.packer(cls)(*[d[f] for f, _ in cls._fields_])


def kv4(**kw):
    return packed(L.Paged4KV, dict(pages=A, page_stride=16 * 288, n_pages=4, page_size=16, block_table=A, ld_table=8,
                                   max_pages=8, row_offsets=A, kv_lens=A, n_seq=2, k_exp=0, v_exp=0), kw)


def kv16(**kw):
    return packed(L.PagedKV, dict(k_pages=A, v_pages=A, page_stride=16 * 256, ld=256, n_pages=4, page_size=16,
                                  block_table=A, ld_table=8, max_pages=8, row_offsets=A, kv_lens=A, n_seq=2), kw)


def append(kv=None, dt=L.CB_BF16, **kw):
    rows = packed(L.PagedRows, dict(k=A, v=A, ld_k=256, ld_v=256, k_layer_stride=0, v_layer_stride=0,
                                    cache_layer_stride=0, n_rows=3, n_layers=1, n_kv_heads=2, head_dim=128,
                                    rope_table=A, q=0, q_out=0, ld_q=0, ld_q_out=0, n_q_heads=0, max_positions=64), kw)
    return L.lib.cb_paged4_append(kv4() if kv is None else kv, rows, dt, None)


def gather(kv=None, dt=L.CB_BF16, **kw):
    rows = packed(L.PagedRowsOut, dict(k=A, v=A, ld_k=256, ld_v=256, k_layer_stride=0, v_layer_stride=0,
                                       cache_layer_stride=0, n_rows=3, n_layers=1, n_kv_heads=2, head_dim=128), kw)
    return L.lib.cb_paged4_gather(kv4() if kv is None else kv, rows, dt, None)


def query(**kw):
    return packed(L.PagedQuery, dict(q=A, out=A, ld_q=512, ld_out=512, ws=A, ws_bytes=1 << 40, n_rows=3, max_kv_len=64,
                                     n_q_heads=4, n_kv_heads=2, head_dim=128, scale=0.1), kw)


def attn4(kv=None, dt=L.CB_BF16, **kw):
    return L.lib.cb_paged4_attention(kv4() if kv is None else kv, query(**kw), dt, None)


def picked(kv=None, dt=L.CB_BF16, picks=A, n=5, **kw):
    return L.lib.cb_paged_attention_picked(kv16() if kv is None else kv, query(**kw), picks, n, dt, None)


def page_bounds(**kw):
    return packed(L.PageBounds, dict(bounds=A, page_stride=512, ld=256, bounds_layer_stride=0, cache_layer_stride=0,
                                     n_rows=3, n_layers=1, n_kv_heads=2, head_dim=128), kw)


def bounds(kv=None, dt=L.CB_BF16, **kw):
    return L.lib.cb_paged_bounds(kv16() if kv is None else kv, page_bounds(**kw), dt, None)


def select(kv=None, dt=L.CB_BF16, b=None, **kw):
    a = packed(L.PageSelect, dict(q=A, ld_q=512, picks=A, ws=A, ws_bytes=1 << 40, max_kv_len=64, n_q_heads=4,
                                  n_picks=3, n_first=1, n_last=1), kw)
    return L.lib.cb_paged_select(kv16() if kv is None else kv, page_bounds(**(b or {})), a, dt, None)


INV, UNS, WS = L.CB_ERR_INVALID_ARG, L.CB_ERR_UNSUPPORTED, L.CB_ERR_WORKSPACE


@pytest.mark.parametrize("kw", [
    dict(pages=0), dict(pages=A + 8), dict(page_stride=16 * 288 - 16), dict(page_stride=16 * 288 + 8), dict(n_pages=0),
    dict(n_seq=-1), dict(n_seq=1025), dict(ld_table=7), dict(max_pages=-1), dict(block_table=0), dict(row_offsets=0),
    dict(kv_lens=0), dict(kv_lens=A + 2), dict(k_exp=65), dict(v_exp=-65)])
def test_4bit_geometry_is_refused(kw):
    for call in (append, gather, attn4):
        assert call(kv4(**kw)) == INV and L.lib.cb_last_error_message()


@pytest.mark.parametrize("size", [0, 4, 24, 2048])
def test_page_size_is_refused(size):
    for call in (append, gather, attn4):
        assert call(kv4(page_size=size, page_stride=1 << 24)) == UNS
    for call in (bounds, select, picked):
        assert call(kv16(page_size=size, page_stride=1 << 24)) == UNS
    assert L.lib.cb_paged4_page_bytes(size, 2, 128) == 0
    with pytest.raises(ValueError):
        R.cb_paged4_page_bytes(size, 2, 128)


@pytest.mark.parametrize("kw", [
    dict(k=0), dict(v=0), dict(k=A + 2), dict(ld_k=255), dict(ld_v=128), dict(n_rows=-1), dict(n_layers=-1),
    dict(n_layers=65536), dict(n_layers=2, cache_layer_stride=0), dict(n_layers=2, cache_layer_stride=8),
    dict(n_layers=2, cache_layer_stride=16, k_layer_stride=4), dict(n_kv_heads=0), dict(n_kv_heads=4097),
    dict(head_dim=96), dict(head_dim=256), dict(dt=7)])
def test_row_refusals(kw):
    assert append(**kw) == INV and gather(**kw) == INV


@pytest.mark.parametrize("kw", [
    dict(rope_table=A + 4), dict(max_positions=0), dict(q=A, ld_q=512, n_q_heads=4), dict(q_out=A, ld_q_out=512, n_q_heads=4),
    dict(q=A, ld_q=512, q_out=A, ld_q_out=512, n_q_heads=0), dict(q=A, ld_q=512, q_out=A, ld_q_out=512, n_q_heads=4, rope_table=0)])
def test_append_refusals(kw):
    assert append(**kw) == INV


def test_gathered_layers_have_rows_of_their_own():
    assert gather(n_layers=2, cache_layer_stride=1 << 20) == INV
    assert gather(n_layers=2, cache_layer_stride=1 << 20, k_layer_stride=1024) == INV


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(out=0), dict(q=A + 8), dict(ld_q=504), dict(ld_out=508), dict(n_rows=-1), dict(n_q_heads=3),
    dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_q_heads=258), dict(head_dim=96), dict(dt=2), dict(scale=-0.1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38)])
def test_attention_refusals(kw):
    assert attn4(**kw) == INV and picked(**kw) == INV


def test_more_attention_refusals():
    assert attn4(max_kv_len=-1) == INV and attn4(max_kv_len=L.CB_MAX_KV_LEN + 1) == UNS
    assert picked(picks=0) == INV and picked(picks=A + 2) == INV
    assert picked(n=0) == INV and picked(n=1025) == INV
    for kw in (dict(k_pages=0), dict(v_pages=0), dict(ld=248), dict(page_stride=256), dict(n_seq=1025)):
        assert picked(kv16(**kw)) == INV


def test_workspaces():
    long4 = lambda **kw: attn4(max_kv_len=100000, **kw)     # (short keys join in a cluster: no workspace)
    for call, need in ((long4, L.lib.cb_paged4_attention_workspace_size(3, 2, 100000, 4, 2, 128, L.CB_BF16)),
                       (select, L.lib.cb_paged_select_workspace_size(3, 64, 16, 2)),
                       (picked, L.lib.cb_paged_attention_picked_workspace_size(3, 5, 16, 4, 2, 128, L.CB_BF16))):
        assert need >= 256
        assert call(ws=0) == WS and call(ws=A + 8) == WS
        if need > 256:                 # (256 is the least that the size calls name)
            assert call(ws_bytes=need - 1) == WS
    assert L.lib.cb_paged4_attention_workspace_size(-1, 1, 8, 4, 2, 128, 1) == 256
    assert L.lib.cb_paged_attention_picked_workspace_size(1, 5, 16, 3, 2, 128, 1) == 256
    assert L.lib.cb_paged_select_workspace_size(0, 64, 16, 2) == 256


@pytest.mark.parametrize("kw", [
    dict(bounds=0), dict(bounds=A + 8), dict(ld=248), dict(ld=260), dict(page_stride=504), dict(page_stride=516),
    dict(n_rows=-1), dict(n_kv_heads=0), dict(head_dim=0)])
def test_bounds_refusals(kw):
    assert bounds(**kw) == INV and select(b=kw) == INV


def test_more_bounds_and_selection_refusals():
    assert bounds(head_dim=120) == INV and bounds(n_layers=-1) == INV and bounds(dt=2) == INV
    assert bounds(n_layers=2, bounds_layer_stride=0, cache_layer_stride=64) == INV
    assert bounds(n_layers=2, bounds_layer_stride=4, cache_layer_stride=64) == INV
    assert bounds(kv16(k_pages=0)) == INV
    for kw in (dict(q=0), dict(ld_q=504), dict(picks=0), dict(picks=A + 2), dict(max_kv_len=-1), dict(n_picks=0),
               dict(n_picks=1025), dict(n_first=-1), dict(n_last=-1), dict(n_first=2, n_last=2), dict(n_q_heads=3),
               dict(n_first=2 ** 31 - 1, n_last=2 ** 31 - 1), dict(dt=2), dict(b=dict(head_dim=96))):
        assert select(**kw) == INV, kw
    assert select(max_kv_len=L.CB_MAX_KV_LEN + 1) == UNS


def test_empty_calls_are_done():
    none = dict(n_seq=0, row_offsets=0, kv_lens=0, block_table=0)
    for call in (append, gather, attn4, bounds, picked):
        assert call(n_rows=0) == L.CB_OK
    assert select(b=dict(n_rows=0)) == L.CB_OK
    for call in (append, gather, attn4):
        assert call(kv4(**none)) == L.CB_OK
    for call in (bounds, select, picked):
        assert call(kv16(**none)) == L.CB_OK


def test_null_structures():
    kv, z = kv16(), bytes(256)
    for f in (L.lib.cb_paged4_append, L.lib.cb_paged4_gather, L.lib.cb_paged4_attention, L.lib.cb_paged_bounds):
        assert f(None, z, L.CB_BF16, None) == INV and f(z, None, L.CB_BF16, None) == INV and f(z, z, L.CB_BF16, None) == INV
    assert L.lib.cb_paged_select(kv, None, z, L.CB_BF16, None) == INV
    assert L.lib.cb_paged_select(kv, page_bounds(), None, L.CB_BF16, None) == INV
    assert L.lib.cb_paged_select(None, page_bounds(), z, L.CB_BF16, None) == INV
    assert L.lib.cb_paged_attention_picked(kv, None, A, 1, L.CB_BF16, None) == INV
    assert L.lib.cb_paged_attention_picked(None, query(), A, 1, L.CB_BF16, None) == INV


def test_plan_queries():
    """What calls of given sizes run (148 SMs are assumed here), and the workspace from that."""
    def plan(*a):
        out = (C.c_int64 * 6)(*[-5] * 6)
        st = L.lib.cb_debug_paged4_plan(*a, out)
        return list(out) if st == L.CB_OK else st

    def plan_picked(*a):
        out = (C.c_int64 * 3)(*[-5] * 3)
        st = L.lib.cb_debug_picked_plan(*a, out)
        return list(out) if st == L.CB_OK else st
    bf, f32 = L.CB_BF16, L.CB_F32
    assert plan(1, 1, 3137, 32, 8, 128, bf)[:2] == [8, 16] and plan(64, 64, 16384, 32, 8, 128, bf)[:2] == [8, 0]
    assert plan(2048, 2, 16384, 32, 8, 128, bf)[3] == 256 and plan(2048, 2, 16384, 32, 8, 128, f32)[3] == 0
    size = L.lib.cb_paged4_attention_workspace_size
    for a in [(1, 1, 100000, 32, 8, 128), (1, 1, 900, 32, 8, 128), (64, 1, 3200, 32, 8, 128), (8192, 4, 8192, 32, 8, 128),
              (127, 64, 16384, 32, 8, 128), (2000, 1, 30000, 24, 8, 64), (300, 1, 9000, 32, 16, 64)]:
        for dt in (bf, f32):
            tile, cluster, grid, unit, parts, limit = plan(*a, dt)
            assert tile in (0, 8, 16, 32) and unit in (0, 128, 256) and (tile or unit) and cluster in (0, 1, 2, 4, 8, 16)
            assert not (unit and dt == f32) and limit == (0 if not tile else 32 if unit else 0x7fffffff)
            hkv, hd = a[4], a[5]
            few = 2 * grid * tile * (4 * hd + 8) + 24 * grid if tile and not cluster else 0
            assert size(*a, dt) >= max(256, few) and (unit or size(*a, dt) == max(256, few))
    assert plan_picked(1, 128, 16, 32, 8, 128, bf) == [8, 8, 128] and plan_picked(64, 64, 32, 32, 8, 128, bf) == [0, 512, 128]
    assert plan_picked(1, 3, 8, 40, 2, 64, f32) == [1, 4, 2]
    for bad in [(0, 1, 8, 4, 2, 128, 1), (1, 1025, 8, 4, 2, 128, 1), (1, 1, -1, 4, 2, 128, 1), (1, 1, L.CB_MAX_KV_LEN + 1, 4, 2, 128, 1),
                (1, 1, 8, 3, 2, 128, 1), (1, 1, 8, 4, 2, 80, 1), (1, 1, 8, 4, 2, 128, 2)]:
        assert plan(*bad) == INV
    for bad in [(0, 1, 8, 4, 2, 128, 1), (1, 0, 8, 4, 2, 128, 1), (1, 1025, 8, 4, 2, 128, 1), (1, 1, 12, 4, 2, 128, 1), (1, 1, 8, 4, 2, 128, 7)]:
        assert plan_picked(*bad) == INV
    assert L.lib.cb_debug_paged4_plan(1, 1, 8, 4, 2, 128, bf, None) == INV
    assert L.lib.cb_debug_picked_plan(1, 1, 8, 4, 2, 128, bf, None) == INV


STRUCTS = {"cb_paged4_kv": L.Paged4KV, "cb_paged_rows_out": L.PagedRowsOut, "cb_page_bounds": L.PageBounds,
           "cb_page_select": L.PageSelect}


def test_ctypes_mirrors_match_c_layout(tmp_path):
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "cacheblend.h"', "int main(void) {"]
    for name, cls in STRUCTS.items():
        src.append(f'printf("{name} %zu\\n", sizeof({name}));')
        src += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(src + ['printf("max %d\\n", CB_MAX_PICKS); return 0; }']))
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c99", "-I", inc, str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = dict(x.rsplit(" ", 1) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                                        check=True).stdout.strip().splitlines())
    assert int(got["max"]) == 1024
    for name, cls in STRUCTS.items():
        assert int(got[name]) == C.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)
        values = list(range(1, len(cls._fields_) + 1))
        back = cls.from_buffer_copy(L.packer(cls)(*values))
        assert [getattr(back, f) for f, _ in cls._fields_] == values


# --------------------------------------------------------------- wrappers --
class _Lib:
    """The real size calls; entry points that only count."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_size") or name == "cb_paged4_page_bytes":
            return getattr(L.lib, name)
        return lambda *a: self.calls.append(name) or L.CB_OK


@pytest.fixture
def fake(monkeypatch):
    """Host tensors stand for device ones (their device index is -1)."""
    from rag_kv_cache_layer_gb300 import api
    lib = _Lib()
    monkeypatch.setattr(api, "_cur_device", lambda: -1)
    monkeypatch.setattr(api, "_cur_stream", lambda dev: 0)
    monkeypatch.setattr(api, "lib", lib)
    return lib


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def test_wrappers_refuse_wrong_tensors(fake):
    bf = torch.bfloat16
    off, lens, table = ints([0, 1]), ints([1]), ints([[0]])
    pool, x, q = torch.zeros(3, 16 * 144, dtype=torch.uint8), torch.zeros(1, 128, dtype=bf), torch.zeros(1, 256, dtype=bf)
    kp, bd, pk = torch.zeros(3, 16, 128, dtype=bf), torch.zeros(3, 2, 128, dtype=bf), torch.zeros(1, 2, 4, dtype=torch.int32)
    ws = torch.empty(1 << 24, dtype=torch.uint8)
    calls = {
        "append": lambda **k: R.cb_paged4_append(k.get("x", x), k.get("v", x), off, lens, k.get("table", table),
                                                 k.get("pool", pool), k.get("page", 16), 64),
        "gather": lambda **k: R.cb_paged4_gather(off, lens, k.get("table", table), k.get("pool", pool), k.get("page", 16),
                                                 64, k.get("x", x), k.get("v", x)),
        "attn4": lambda **k: R.cb_paged4_attention(k.get("q", q), off, lens, k.get("table", table), k.get("pool", pool),
                                                   k.get("page", 16), 4, 2, 64, k.get("out", q.clone()), ws=k.get("ws", ws)),
        "bounds": lambda **k: R.cb_paged_bounds(off, lens, k.get("table", table), k.get("kp", kp), k.get("bd", bd), 1),
        "select": lambda **k: R.cb_paged_select(k.get("q", q), off, lens, k.get("table", table), k.get("bd", bd),
                                                k.get("page", 16), 4, 2, 64, k.get("pk", pk), ws=k.get("ws", ws)),
        "picked": lambda **k: R.cb_paged_attention_picked(k.get("q", q), off, lens, k.get("table", table), k.get("kp", kp),
                                                          k.get("kp", kp), k.get("pk", pk), 4, 2, 64,
                                                          k.get("out", q.clone()), ws=k.get("ws", ws)),
    }
    for f in calls.values():
        f()
    assert len(fake.calls) == 6
    wrong = [("append", dict(pool=pool.to(torch.int8))), ("append", dict(pool=pool[:, :-16])), ("append", dict(page=32)),
             ("append", dict(x=torch.zeros(1, 100, dtype=bf))), ("append", dict(v=torch.zeros(1, 64, dtype=bf))),
             ("append", dict(v=x.float())), ("append", dict(x=torch.zeros(2, 1, 128, dtype=bf))), ("append", dict(page=12)),
             ("append", dict(pool=torch.zeros(2, 3, 16 * 144, dtype=torch.uint8))), ("append", dict(table=table.long())),
             ("gather", dict(pool=pool[:, :-16])), ("gather", dict(v=x.float())),
             ("attn4", dict(pool=pool[:, :-16])), ("attn4", dict(q=q.float())), ("attn4", dict(out=q[:, :128])),
             ("attn4", dict(pool=pool[None])), ("attn4", dict(ws=torch.empty(1, dtype=torch.uint8).expand(1 << 24))),
             ("bounds", dict(bd=bd.float())), ("bounds", dict(bd=bd[:2])), ("bounds", dict(bd=bd[None])),
             ("bounds", dict(bd=torch.zeros(3, 2, 256, dtype=bf)[:, :, ::2])),
             ("select", dict(bd=bd.float())), ("select", dict(pk=pk.long())), ("select", dict(pk=pk[:, :1])),
             ("select", dict(pk=torch.zeros(1, 2, 8, dtype=torch.int32)[:, :, ::2])), ("select", dict(ws=ws[::2])),
             ("select", dict(bd=bd[None])),
             ("picked", dict(pk=pk.long())), ("picked", dict(pk=pk[:, :1])), ("picked", dict(q=q.float())),
             ("picked", dict(kp=kp[None])), ("picked", dict(ws=ws[::2]))]
    for name, kw in wrong:
        with pytest.raises(ValueError):
            calls[name](**kw)
    assert len(fake.calls) == 6


def test_no_layers_is_nothing_to_do(fake):
    z = torch.zeros(0, 1, 128)
    pool = torch.zeros(0, 3, 16 * 144, dtype=torch.uint8)
    R.cb_paged4_append(z, z, ints([0, 1]), ints([1]), ints([[0]]), pool, 16, 64)
    R.cb_paged4_gather(ints([0, 1]), ints([1]), ints([[0]]), pool, 16, 64, z, z)
    R.cb_paged_bounds(ints([0, 1]), ints([1]), ints([[0]]), torch.zeros(0, 3, 16, 128), torch.zeros(0, 3, 2, 128), 1)
    assert not fake.calls


# ----------------------------------------------------------------- oracle --
def test_oracle_format_by_hand():
    x = np.zeros(16)
    x[:10] = [6, -6, 0.25, 0.26, 0.75, -1.25, 2.5, 3.5, 5, 5.01]           # scale 1: ties to the even code
    c, s = O4.quantise(x)
    assert O4.SCALES[s[0]] == 1.0 and len(O4.SCALES) == 127 and O4.SCALES[-1] == 448
    assert O4.values(c, s)[:10].tolist() == [6, -6, 0, 0.5, 1, -1, 2, 4, 4, 6]
    assert O4.quantise(np.zeros(16))[1][0] == 1                                # the smallest scale, 2^-9
    assert O4.SCALES[O4.quantise(np.full(16, 1e9))[1][0]] == 448
    # a / 6 halfway between 1 and 1.125 goes to 1 (an even code); a is then 6.375 steps and saturates
    y = np.zeros(16); y[0] = 6.375
    c, s = O4.quantise(y)
    assert O4.SCALES[s[0]] == 1.0 and O4.values(c, s)[0] == 6.0
    assert O4.round_to([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -0.3], 8).tolist() == [1, 1 + 2.0 ** -6, -0.30078125]


def test_oracle_pages_by_hand():
    k = np.arange(32.0).reshape(2, 8, 2) * np.array([1, -1])
    b = O4.page_bounds(np.zeros((2, 2, 2)), k, [[1, 0]], [0, 1], [3])          # page 1's first three slots
    assert b[1].tolist() == [[16, -21], [20, -17]] and not b[0].any()
    assert O4.page_scores([1.0, 1.0], b, [1, 0], 1, 1, 1, 2).tolist() == [[20 - 17]]
    assert O4.page_scores([-1.0, 0.0, 0.0, 2.0], b, [1, 0], 1, 2, 1, 2).tolist() == [[max(-16, -34)]]
    sel = O4.select(np.ones((1, 2)), np.array([[[0, 0], [i, 0]] for i in (3, 9, 9, 1, 5)], float), [[0, 1, 2, 3, 4]],
                    [0, 1], [40], 8, 1, 1, 2, np.zeros((1, 1, 3), int), 0, 1)
    assert sel.tolist() == [[[1, 2, 4]]]
