"""The generation operators together, as a request uses them: a prefill's cache
moves into pages, then tokens run one by one (or as a chunk) through the
layers with cb_paged_append and cb_paged_attention, and cb_sample_tokens draws
from the tied output projection's logits.  The reference is the library's own
full prefill of the longer sequence, at the bounds its caches and hidden states
are held to (max-abs 1e-4 in fp32, 2e-2 RMS-relative in bf16)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import workload as W
import rag_kv_cache_layer_gb300 as R
from gpu_common import assert_close, host
from oracle import paged as OP
from rag_kv_cache_layer_gb300 import _lib as L

pytestmark = pytest.mark.gpu
SHAPES = {
    "f32": W.TINY_F32,
    "bf16": W.ModelShape("generate", 2, 512, 8, 2, 128, 1024, 4096, dtype="bf16"),
}
PAGE = 16


def rms(x, gain, eps):
    return x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps) * gain


class Generator:
    """One batch of sequences over a paged cache, layer by layer."""

    def __init__(self, dtype, n_seq, max_tokens):
        self.shape = s = SHAPES[dtype]
        self.model = R.BlendModel.from_host(s, W.make_weights(s, 3), 1024)
        self.dt, self.kvw = self.model.dtype, s.n_kv_heads * s.head_dim
        per = -(-max_tokens // PAGE)
        perm = torch.randperm(n_seq * per + 2, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        self.table = perm[:n_seq * per].view(n_seq, per).cuda()
        pool = (s.n_layers, n_seq * per + 2, PAGE, self.kvw)
        self.K, self.V = (torch.full(pool, float("nan"), dtype=self.dt, device="cuda") for _ in range(2))
        self.lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")

    def prefill(self, prompts):
        """Full prefill of every prompt, its cache moved into the pages."""
        reqs = [R.Req(torch.from_numpy(p).cuda(), [R.Seg(len(p))]) for p in prompts]
        out = self.model.cb_full_prefill(reqs)
        off = torch.tensor(np.concatenate([[0], np.cumsum([len(p) for p in prompts])]), dtype=torch.int32, device="cuda")
        self.lens.copy_(off[1:] - off[:-1])
        R.cb_paged_append(out["k_cache"], out["v_cache"], off, self.lens, self.table, self.K, self.V, self.shape.head_dim)
        return out["first_token"]

    def step(self, tokens, counts):
        """Hidden states of the new rows: tokens [rows], counts rows per sequence."""
        s, m, w = self.shape, self.model, self.model.w
        n = int(sum(counts))
        off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        self.lens += off[1:] - off[:-1]
        h = w["embed"][tokens.long()].float()
        qw = s.n_q_heads * s.head_dim
        empty = lambda c, dt=self.dt: torch.empty(n, c, dtype=dt, device="cuda")
        for l, lw in enumerate(w["layers"]):
            qkv, q, o = empty(s.qkv_rows), empty(qw), empty(qw)
            m.cb_linear(rms(h, lw["norm1"], s.norm_eps).to(self.dt), lw["w_qkv"], qkv)
            R.cb_paged_append(qkv[:, qw:qw + self.kvw], qkv[:, qw + self.kvw:], off, self.lens, self.table,
                              self.K[l], self.V[l], s.head_dim, rope_table=m.rope_table, q=qkv[:, :qw], q_out=q)
            R.cb_paged_attention(q, off, self.lens, self.table, self.K[l], self.V[l], s.n_q_heads, s.n_kv_heads,
                                 s.head_dim, o)
            m.cb_linear(o, lw["w_o"], h, L.CB_EPI_RESID)
            g = empty(s.d_ffn)
            m.cb_linear(rms(h, lw["norm2"], s.norm_eps).to(self.dt), lw["w_gate"], g, L.CB_EPI_SWIGLU, W2=lw["w_up"])
            m.cb_linear(g, lw["w_down"], h, L.CB_EPI_RESID)
        return h

    def logits(self, h):
        s, w = self.shape, self.model.w
        out = torch.empty(h.shape[0], s.vocab, dtype=self.dt, device="cuda")
        self.model.cb_linear(rms(h, w["final_norm"], s.norm_eps).to(self.dt), w["embed"], out)
        return out


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield
    torch.cuda.synchronize()
    assert R.device_status() == 0


def full_hidden(model, tokens):
    req = R.Req(torch.from_numpy(tokens).cuda(), [R.Seg(len(tokens))])
    out = model.cb_full_prefill([req])
    return host(out["hidden"]), int(out["first_token"][0])


@pytest.mark.parametrize("dtype", list(SHAPES))
@pytest.mark.parametrize("chunk", [1, 5, 40])
def test_incremental_rows_equal_the_full_prefill(dtype, chunk):
    rng = np.random.default_rng(chunk)
    lens, more = [97, 33, 160], 40
    seqs = [rng.integers(0, SHAPES[dtype].vocab, n + more).astype(np.int32) for n in lens]
    g = Generator(dtype, 3, max(lens) + more)
    g.prefill([s[:n] for s, n in zip(seqs, lens)])
    got = [[] for _ in lens]
    for a in range(0, more, chunk):
        # the second sequence sits out every other step
        counts = [chunk, 0 if chunk == 5 and (a // chunk) % 2 else chunk, chunk]
        at = [int(x) for x in g.lens.tolist()]
        toks = np.concatenate([s[p:p + c] for s, p, c in zip(seqs, at, counts)])
        h = host(g.step(torch.from_numpy(toks).cuda(), counts))
        for i, rows in enumerate(np.split(h, np.cumsum(counts)[:-1])):
            got[i].append(rows)
    for i, (s, n) in enumerate(zip(seqs, lens)):
        rows = np.concatenate(got[i])
        ref, token = full_hidden(g.model, s[:n + len(rows)])
        assert_close(rows, ref[n:], g.dt)
        if dtype == "f32":
            tok = torch.zeros(1, dtype=torch.int32, device="cuda")
            R.cb_sample_tokens(g.logits(torch.from_numpy(rows[-1:]).float().cuda()), torch.zeros(1, device="cuda"), tok,
                               temperature=torch.zeros(1, device="cuda"))
            assert int(tok[0]) == token          # the greedy draw is the prefill's own token


@pytest.mark.parametrize("dtype", list(SHAPES))
def test_sampled_generation_is_reproducible(dtype):
    """Eight sampled tokens for two requests, twice, each checked against the
    float64 definition on the same logits."""
    rng = np.random.default_rng(4)
    prompts = [rng.integers(0, SHAPES[dtype].vocab, n).astype(np.int32) for n in (50, 81)]
    u = rng.random((8, 2)).astype(np.float32)
    dev = lambda a, dt=torch.float32: torch.tensor(a, dtype=dt, device="cuda")
    t, k, p = [0.7, 1.3], [0, 40], [0.9, 1.0]
    runs = []
    for _ in range(2):
        g = Generator(dtype, 2, 100)
        tok = g.prefill(prompts)
        seen = [tok.tolist()]
        for i in range(8):
            logits = g.logits(g.step(tok, [1, 1]))
            tok = torch.empty(2, dtype=torch.int32, device="cuda")
            R.cb_sample_tokens(logits, dev(u[i]), tok, dev(t), dev(k, torch.int32), dev(p))
            x = logits.double().cpu().numpy()
            f = np.float32
            assert tok.tolist() == [OP.sample_token(x[r], float(u[i, r]), float(f(t[r])), k[r], float(f(p[r])))
                                    for r in range(2)]
            seen.append(tok.tolist())
        runs.append(seen)
    assert runs[0] == runs[1]


@pytest.mark.parametrize("dtype", list(SHAPES))
@pytest.mark.parametrize("n", [1, 7, 60])
def test_paged_attention_agrees_with_the_fused_cache(dtype, n):
    """A blended request's fused cache in pages: its last rows attend to the
    same keys as cb_sparse_query_attention reads in place."""
    s = SHAPES[dtype]
    rng = np.random.default_rng(9)
    model = R.BlendModel.from_host(s, W.make_weights(s, 3), 1024)
    chunks = {i: rng.integers(0, s.vocab, 90).astype(np.int32) for i in range(3)}
    store = R.ChunkStore(model, 270)
    store.prefill({i: torch.from_numpy(c).cuda() for i, c in chunks.items()})
    query = rng.integers(0, s.vocab, 61).astype(np.int32)
    toks = torch.from_numpy(np.concatenate([*chunks.values(), query])).cuda()
    out = model.cb_blend_prefill([R.Req(toks, [store.seg(i) for i in chunks] + [R.Seg(len(query))])], 1500)
    T, kvw = toks.numel(), s.n_kv_heads * s.head_dim
    K = torch.full((s.n_layers, 24, PAGE, kvw), float("nan"), dtype=model.dtype, device="cuda")
    V = torch.full_like(K, float("nan"))
    table = torch.randperm(24, generator=torch.Generator().manual_seed(2)).to(torch.int32)[None].cuda()
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    R.cb_paged_append(out["k_cache"], out["v_cache"], ints([0, T]), ints([T]), table, K, V, s.head_dim)
    q = torch.randn(n, s.n_q_heads * s.head_dim, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    q = q.to(model.dtype)
    pos = torch.arange(T - n, T, dtype=torch.int32, device="cuda")
    for l in range(s.n_layers):
        a, b = torch.empty_like(q), torch.empty_like(q)
        R.cb_sparse_query_attention(q, pos, [(0, n, 0, T)], out["k_cache"][l], out["v_cache"][l], s.n_q_heads,
                                    s.n_kv_heads, s.head_dim, a)
        R.cb_paged_attention(q, ints([0, n]), ints([T]), table, K[l], V[l], s.n_q_heads, s.n_kv_heads, s.head_dim, b)
        assert_close(host(b), host(a), model.dtype)


def test_recorded_generation_step():
    """append, attention and sampling of a step recorded once and replayed
    while the lengths advance on the device."""
    s = SHAPES["bf16"]
    hq, hkv, hd = s.n_q_heads, s.n_kv_heads, s.head_dim
    kvw, n = hkv * hd, 4
    gen = torch.Generator("cuda").manual_seed(3)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda").bfloat16()
    rope = R.cb_rope_table_init(256, hd, s.rope_base)
    table = torch.arange(n * 8, dtype=torch.int32, device="cuda").view(n, 8)
    off = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([3, 40, 17, 0], dtype=torch.int32, device="cuda")      # the last slot is idle
    live = (lens > 0).int()
    state = dict(K=rnd(n * 8, PAGE, kvw), V=rnd(n * 8, PAGE, kvw), lens=lens)
    k, v, q = rnd(n, kvw), rnd(n, kvw), rnd(n, hq * hd)
    qr, o, tok = torch.empty_like(q), torch.empty_like(q), torch.zeros(n, dtype=torch.int32, device="cuda")
    u = torch.rand(n, generator=gen, device="cuda")

    def step(st, qr, o, tok):
        st["lens"] += live
        R.cb_paged_append(k, v, off, st["lens"], table, st["K"], st["V"], hd, rope_table=rope, q=q, q_out=qr)
        R.cb_paged_attention(qr, off, st["lens"], table, st["K"], st["V"], hq, hkv, hd, o)
        R.cb_sample_tokens(o, u, tok)
    other = {a: b.clone() for a, b in state.items()}
    outs = [torch.empty_like(x) for x in (qr, o, tok)]
    step({a: b.clone() for a, b in state.items()}, *outs)                       # warm: attributes, status word
    graph = torch.cuda.CUDAGraph()
    kept = {a: b.clone() for a, b in state.items()}
    with torch.cuda.graph(graph):
        step(state, qr, o, tok)
    for a in state:
        state[a].copy_(kept[a])
    for _ in range(5):
        graph.replay()
        step(other, *outs)
        torch.cuda.synchronize()
        assert torch.equal(o, outs[1]) and torch.equal(tok, outs[2])
        assert all(torch.equal(state[a], other[a]) for a in state)
        assert not o[3].any()                                                   # the idle slot attends to nothing


FIRST_CALLS = """
import torch, rag_kv_cache_layer_gb300 as R
g = torch.Generator(device="cuda").manual_seed(3)
ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
kn, vn, q = (torch.randn(70, w, device="cuda", generator=g).bfloat16() for w in (256, 256, 1024))
kp, vp = torch.zeros(8, 16, 256, device="cuda").bfloat16(), torch.zeros(8, 16, 256, device="cuda").bfloat16()
off, lens, table = ints([0, 1, 70]), ints([1, 69]), ints([[7, 0, 0, 0, 0], [3, 1, 4, 0, 6]])
rope = R.cb_rope_table_init(128, 128, 10000.0)
logits, u = torch.randn(2, 5000, device="cuda", generator=g), torch.rand(2, device="cuda", generator=g)
outs = [(torch.zeros_like(q), torch.zeros_like(q), torch.zeros(2, dtype=torch.int32, device="cuda")) for _ in range(2)]
ws = R.cb_paged_attention_workspace(q, 2, 80, 8, 2, 128)
top_p = torch.full((2,), 0.9, device="cuda")
def step(qr, out, tokens):
    R.cb_paged_append(kn, vn, off, lens, table, kp, vp, 128, rope_table=rope, q=q, q_out=qr)
    R.cb_paged_attention(qr, off, lens, table, kp, vp, 8, 2, 128, out, max_kv_len=80, ws=ws)
    R.cb_sample_tokens(logits, u, tokens, top_p=top_p)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step(*outs[0])
graph.replay()
step(*outs[1])
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(*outs)) and R.device_status() == 0
assert float(outs[0][1].float().abs().sum()) > 0
print("recorded first")
"""


def test_the_first_calls_of_a_process_may_be_recorded():
    """Nothing is set up at a first call that a recording would refuse."""
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0 and "recorded first" in run.stdout, run.stderr[-2000:]
