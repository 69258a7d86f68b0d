"""The operators for long contexts as a request uses them: a prefill's cache goes into
4-bit pages and back, tokens are generated over it, in recorded steps too, and the picked
pages of a 16-bit cache give the whole attention where they hold its weight."""
import numpy as np
import pytest
import torch

import workload as W
import rag_kv_cache_layer_gb300 as R
from oracle import paged as OP
from oracle import paged4 as O4
from test_gpu_generate import SHAPES, PAGE
from test_gpu_paged import f64, ints

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield
    torch.cuda.synchronize()
    assert R.device_status() == 0


def prefilled(dtype, prompts):
    s = SHAPES[dtype]
    model = R.BlendModel.from_host(s, W.make_weights(s, 3), 1024)
    reqs = [R.Req(torch.from_numpy(p).cuda(), [R.Seg(len(p))]) for p in prompts]
    out = model.cb_full_prefill(reqs)
    off = ints(np.concatenate([[0], np.cumsum([len(p) for p in prompts])]))
    return model, s, out["k_cache"], out["v_cache"], off, off[1:] - off[:-1]


@pytest.mark.parametrize("dtype", list(SHAPES))
def test_a_prefill_cache_in_4_bits(dtype):
    """All layers of a prefill's cache go into 4-bit pages; read back they are the values of
    their codes, the nearest that the format has; attention over the 4-bit pages is that over
    a 16-bit (or fp32) cache of those values.  Both kernels' errors: probabilities in bf16
    (2^-8 of B, see test_gpu_paged.py) or fp16 (2^-11), the results' own rounding twice, and
    sums' errors below those; B and the results are at most the largest value."""
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, SHAPES[dtype].vocab, n).astype(np.int32) for n in (100, 37, 64)]
    model, s, K, V, off, lens = prefilled(dtype, prompts)
    dt, L, rows, kvw = model.dtype, *K.shape
    per = -(-128 // PAGE)
    table = torch.randperm(3 * per, device="cuda").int().view(3, per)
    pool = torch.full((L, 3 * per, R.cb_paged4_page_bytes(PAGE, s.n_kv_heads, s.head_dim)), 0x7f, dtype=torch.uint8, device="cuda")
    R.cb_paged4_append(K, V, off, lens, table, pool, PAGE, s.head_dim)
    kb, vb = torch.empty_like(K), torch.empty_like(V)
    R.cb_paged4_gather(off, lens, table, pool, PAGE, s.head_dim, kb, vb)
    for x, y in ((K, kb), (V, vb)):
        assert np.array_equal(f64(y), O4.values(*O4.quantise(f64(x))))
    kp = torch.full((L, 3 * per, PAGE, kvw), float("nan"), dtype=dt, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    R.cb_paged_append(kb, vb, off, lens, table, kp, vp, s.head_dim)
    for n in (1, 5):            # a generated token and a draft of each
        q = torch.randn(3 * n, s.n_q_heads * s.head_dim, device="cuda").to(dt)
        o = ints([0, n, 2 * n, 3 * n])
        for l in range(L):
            a, b = torch.empty_like(q), torch.empty_like(q)
            R.cb_paged4_attention(q, o, lens, table, pool[l], PAGE, s.n_q_heads, s.n_kv_heads, s.head_dim, a)
            R.cb_paged_attention(q, o, lens, table, kp[l], vp[l], s.n_q_heads, s.n_kv_heads, s.head_dim, b)
            top = float(vb[l].abs().max())
            lim = top * (3 * 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) if dt == torch.bfloat16 else top * 2e-5
            assert float((a.float() - b.float()).abs().max()) <= lim


@pytest.mark.parametrize("dtype", list(SHAPES))
def test_recorded_steps_over_4_bits(dtype):
    """A decode step (rows appended and rotated, attention) of one layer in a graph, replayed
    while the lengths grow, against the oracle on the bytes of the moment."""
    rng = np.random.default_rng(2)
    model, s, K, V, off, lens0 = prefilled(dtype, [rng.integers(0, SHAPES[dtype].vocab, n).astype(np.int32) for n in (40, 9)])
    dt, hq, hkv, hd, kvw = model.dtype, s.n_q_heads, s.n_kv_heads, s.head_dim, s.n_kv_heads * s.head_dim
    per = -(-64 // PAGE)
    table = torch.randperm(2 * per, device="cuda").int().view(2, per)
    pool = torch.zeros(2 * per, R.cb_paged4_page_bytes(PAGE, hkv, hd), dtype=torch.uint8, device="cuda")
    R.cb_paged4_append(K[0], V[0], off, lens0, table, pool, PAGE, hd)
    lens, step = lens0.clone(), ints([0, 1, 2])
    q, k, v = (torch.zeros(2, w, dtype=dt, device="cuda") for w in (hq * hd, kvw, kvw))
    qr, out = torch.zeros_like(q), torch.zeros_like(q)
    ws = R.cb_paged4_attention_workspace(q, 2, 64, hq, hkv, hd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.cb_paged4_append(k, v, step, lens, table, pool, PAGE, hd, rope_table=model.rope_table, q=q, q_out=qr)
        R.cb_paged4_attention(qr, step, lens, table, pool, PAGE, hq, hkv, hd, out, max_kv_len=64, ws=ws)
    for _ in range(12):
        lens += 1
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda").to(dt))
        g.replay()
        torch.cuda.synchronize()
        P = O4.Pool(pool.cpu().numpy(), PAGE, hkv, hd)
        n, t = lens.cpu().numpy(), table.cpu().numpy()
        # the newest row is what the rotated key's codes stand for
        host = model.rope_table.cpu().numpy().reshape(-1, hd // 2, 2)
        for b in range(2):
            at, slot = t[b][(n[b] - 1) // PAGE], (n[b] - 1) % PAGE
            key = O4.round_to(O4.rotate_by_table(f64(k[b:b + 1]), [n[b] - 1], host), 8 if dt == torch.bfloat16 else 24)
            assert np.array_equal(P.values("k")[at, slot], O4.values(*O4.quantise(key))[0])
        want = OP.paged_attention(f64(qr), P.values("k"), P.values("v"), t, [0, 1, 2], n, hq, hkv, hd, hd ** -0.5, np.zeros(q.shape))
        top = np.abs(P.values("v")).max()
        lim = top * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) if dt == torch.bfloat16 else top * 1e-5
        assert np.abs(f64(out) - want).max() <= lim


@pytest.mark.parametrize("dtype", list(SHAPES))
def test_picked_pages_that_hold_the_weight(dtype):
    """Some keys answer a query far better than the others: the pages that the bounds pick
    hold them, and attention over these pages is that over all, but for the weight left out."""
    s = SHAPES[dtype]
    dt = torch.bfloat16 if s.dtype == "bf16" else torch.float32
    hq, hkv, hd, page, n = s.n_q_heads, s.n_kv_heads, s.head_dim, 16, 2000
    gen = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *a: torch.randn(*a, generator=gen, device="cuda")
    q = rnd(1, hq * hd).to(dt)
    k = 0.1 * rnd(n, hkv, hd)
    for h in range(hkv):                # eight keys along a head's query each, in pages of their own
        where = torch.randperm(n // page - 2, generator=gen, device="cuda")[:8] * page + 21
        k[where, h] = 3.0 * q.view(hkv, -1, hd)[h, 0].float() / q.view(hkv, -1, hd)[h, 0].float().norm() * hd ** 0.5
    q = q.view(hkv, -1, hd)[:, :1].expand(-1, hq // hkv, -1).reshape(1, -1).contiguous()    # one query a group
    k, v = k.view(n, -1).to(dt), rnd(n, hkv * hd).to(dt)
    per = -(-n // page)
    table = torch.randperm(per, generator=gen, device="cuda").int()[None]
    kp = torch.zeros(per, page, hkv * hd, dtype=dt, device="cuda")
    vp, bounds = torch.zeros_like(kp), torch.zeros(per, 2, hkv * hd, dtype=dt, device="cuda")
    R.cb_paged_append(k, v, ints([0, n]), ints([n]), table, kp, vp, hd)
    R.cb_paged_bounds(ints([0, n]), ints([n]), table, kp, bounds, n)
    picks = torch.zeros(1, hkv, 12, dtype=torch.int32, device="cuda")
    one, all_ = torch.empty_like(q), torch.empty_like(q)
    args = (q, ints([0, 1]), ints([n]), table)
    R.cb_paged_select(*args, bounds, page, hq, hkv, hd, picks, n_first=1, n_last=2)
    R.cb_paged_attention_picked(*args, kp, vp, picks, hq, hkv, hd, one)
    R.cb_paged_attention(*args, kp, vp, hq, hkv, hd, all_)
    # the weight left out, from the definition
    x = np.einsum("hd,nhd->hn", f64(q).reshape(hkv, -1, hd)[:, 0], f64(k).reshape(n, hkv, hd)) * hd ** -0.5
    w = np.exp(x - x.max(1, keepdims=True))
    kept = np.zeros((hkv, n), bool)
    for h in range(hkv):
        for j in picks[0, h].tolist():
            kept[h, j * page:(j + 1) * page] = True
    left = (w * ~kept).sum(1) / w.sum(1)
    assert left.max() < 1e-3
    lim = float(v.float().abs().max()) * (2 * left.max() + (4 * 2.0 ** -8 if dt == torch.bfloat16 else 2e-5))
    assert float((one.float() - all_.float()).abs().max()) <= lim
