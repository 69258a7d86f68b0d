"""Token sampling against its float64 definition.  The kernel's weights are
exact to about 2^-38, so a token may differ from the definition only where u
meets a border that closely: the random cases below must agree everywhere, and
the constructed ones meet borders exactly."""
import numpy as np
import pytest
import torch

import rag_kv_cache_layer_gb300 as R
from gpu_common import bf16_values
from oracle import paged as OP

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.synchronize()
    R.device_status()
    yield
    torch.cuda.synchronize()
    assert R.device_status() == 0


def dev(a, dt=torch.float32):
    return torch.tensor(np.asarray(a), dtype=dt, device="cuda")


def sample(x, u, dt=torch.float32, temperature=None, top_k=None, top_p=None, min_p=None, ld=None):
    x = np.atleast_2d(np.asarray(x, np.float32))
    n, v = x.shape
    logits = dev(x).to(dt)
    if ld:
        wide = torch.full((n, ld), float("inf"), dtype=dt, device="cuda")
        wide[:, ld - v:] = logits
        logits = wide[:, ld - v:]
    full = lambda a, d: None if a is None else dev(np.broadcast_to(np.asarray(a), (n,)).copy(), d)
    tokens = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    R.cb_sample_tokens(logits, full(u, torch.float32), tokens, full(temperature, torch.float32),
                       full(top_k, torch.int32), full(top_p, torch.float32), full(min_p, torch.float32))
    return tokens.cpu().numpy().tolist()


def reference(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    x = np.atleast_2d(x)
    b = lambda a, d=np.float32: np.broadcast_to(np.asarray(a, d), (len(x),))
    return [OP.sample_token(x[i], float(b(u)[i]), float(b(temperature)[i]), int(b(top_k, np.int64)[i]),
                            float(b(top_p)[i]), float(b(min_p)[i])) for i in range(len(x))]


def logits(rng, n, v, dt, spread=2.5, banned=0.01):
    x = (rng.standard_normal((n, v)) * spread).astype(np.float32)
    for r in x:
        r[rng.integers(0, v, 16)] += rng.random(16).astype(np.float32) * 6
    x[rng.random((n, v)) < banned] = -np.inf
    x[:, 0] = 0.5                                # never an empty row
    return bf16_values(x) if dt == torch.bfloat16 else x


POLICIES = [dict(), dict(top_k=1), dict(top_k=7), dict(top_k=50), dict(top_k=3000), dict(top_p=0.3), dict(top_p=0.9),
            dict(top_p=0.999), dict(min_p=0.05), dict(min_p=1e-4), dict(top_k=40, top_p=0.8),
            dict(top_k=500, top_p=0.95, min_p=0.02), dict(top_k=10, min_p=0.5), dict(top_p=0.99, min_p=0.001)]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 1000, 4097, 32001, 128256, 151936, 262144])
def test_policies(dt, vocab):
    rng = np.random.default_rng(vocab)
    n = 6 if vocab > 5000 else 24
    for i, kw in enumerate(POLICIES if vocab > 2 else POLICIES[:6]):
        x, u = logits(rng, n, vocab, dt), rng.random(n).astype(np.float32)
        t = rng.uniform(0.3, 1.8, n).astype(np.float32)
        assert sample(x, u, dt, temperature=t, **kw) == reference(x, u, t, **kw), (i, kw)


@pytest.mark.parametrize("dt", DTYPES)
def test_mixed_rows_of_a_large_batch(dt):
    rng = np.random.default_rng(1)
    n, v = 300, 5003
    x, u = logits(rng, n, v, dt), rng.random(n).astype(np.float32)
    t = np.where(rng.random(n) < 0.2, 0, rng.uniform(0.2, 3, n)).astype(np.float32)
    kw = dict(top_k=rng.choice([0, -1, 1, 2, 60, 5002, 5003, 9999], n), top_p=rng.choice([0.1, 0.7, 0.97, 1.0, 2.0], n),
              min_p=rng.choice([0.0, 0.01, 0.3, 1.0], n))
    assert sample(x, u, dt, temperature=t, ld=v + 10, **kw) == reference(x, u, t, **kw)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("v", [9, 70000])
def test_exact_borders_of_equal_weights(dt, v):
    """2^m equal logits: every border is a multiple of 2^-m, met exactly; the
    lowest index whose running weight exceeds u is the next token."""
    x = np.full((1, v), -np.inf, np.float32)
    at = np.arange(8) * (v // 9) + 1
    x[0, at] = 1.25
    for j in range(8):
        assert sample(x, j / 8, dt) == [at[j]]
        assert sample(x, np.nextafter(np.float32((j + 1) / 8), np.float32(0)), dt) == [at[j]]
    # the lowest indices of a tie are kept
    assert sample(x, 0.99, dt, top_k=3) == [at[2]]
    assert sample(x, 0.99, dt, top_p=0.25) == [at[1]]
    assert sample(x, 0.99, dt, top_p=float(np.nextafter(np.float32(0.25), np.float32(1)))) == [at[2]]
    assert sample(x, 0.99, dt, top_k=4, top_p=0.5) == [at[1]]
    assert sample(x, 0.99, dt, min_p=1.0) == [at[7]]


def test_ties_at_the_cut():
    """A tie larger than what is left of top_k or top_p, spread over the row."""
    rng = np.random.default_rng(3)
    for v in (500, 40000):
        x = np.round(rng.standard_normal((4, v)) * 2).astype(np.float32)      # a few dozen distinct values
        u = rng.random(4).astype(np.float32)
        for kw in (dict(top_k=37), dict(top_p=0.4), dict(top_k=int(v * 0.6)), dict(top_k=300, top_p=0.77)):
            for dt in DTYPES:
                assert sample(x, u, dt, **kw) == reference(x, u, **kw)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("v", [3000, 60000])
@pytest.mark.parametrize("levels", [3, 40, 5000])
def test_lists_of_any_length_and_crowding(dt, v, levels):
    """Border lists from a few tokens to more than the first block takes, with
    few equal logits and with hundreds of them."""
    rng = np.random.default_rng(v + levels)
    k = np.array([2, 31, 63, 64, 65, 127, 200, 511, 512, 513, 700, 1000, 1023, 1500, 2047, 2048, 2049, 2600])
    x = rng.standard_normal((len(k), v)).astype(np.float32)
    x = (np.round(x * levels / 8) * (8 / levels)).astype(np.float32)
    x = bf16_values(x) if dt == torch.bfloat16 else x
    u, t = rng.random(len(k)).astype(np.float32), rng.uniform(0.5, 2, len(k)).astype(np.float32)
    for kw in (dict(), dict(top_p=0.5), dict(top_p=0.95, min_p=0.1)):
        assert sample(x, u, dt, temperature=t, top_k=k, **kw) == reference(x, u, t, k, **kw), kw
    p = np.linspace(0.01, 0.999, len(k)).astype(np.float32)
    assert sample(x, u, dt, temperature=t, top_p=p) == reference(x, u, t, top_p=p)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("temperature", [0.02, 1.0])
def test_top_k_past_the_tokens_that_weigh(dt, temperature):
    """More asked for than lie within the weights' range (all others are at
    -inf, or so far below that they weigh nothing): top_k keeps them all, and
    top_p is of their whole weight."""
    rng = np.random.default_rng(9)
    x = np.full((6, 20000), -np.inf, np.float32)
    for r in x:
        r[rng.permutation(20000)[:800]] = bf16_values(rng.standard_normal(800).astype(np.float32) * 2)
    u = rng.random(6).astype(np.float32)
    for kw in (dict(top_k=5000), dict(top_k=5000, top_p=0.9), dict(top_k=801, top_p=0.5), dict(top_k=800, top_p=0.5),
               dict(top_k=19999, top_p=0.99, min_p=0.01)):
        assert sample(x, u, dt, temperature=temperature, **kw) == reference(x, u, np.float32(temperature), **kw), kw


def test_greedy_and_degenerate_settings():
    x = np.array([[1.0, 5.0, 5.0, -2.0], [-0.0, 0.0, -1.0, 0.0], [3.0, np.nan, 2.0, np.inf]], np.float32)
    top = [1, 0, 3]
    for kw in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(top_k=1),
               dict(top_p=0.0), dict(top_p=-3.0)):
        assert sample(x, 0.7, **kw) == top
    # values that switch a filter off
    for kw in (dict(top_k=0), dict(top_k=-5), dict(top_k=4), dict(top_p=1.0), dict(top_p=7.0), dict(top_p=float("nan")),
               dict(min_p=0.0), dict(min_p=-1.0), dict(min_p=float("nan"))):
        assert sample(x[:1], [0.7], **kw) == sample(x[:1], [0.7])
    # u outside [0, 1)
    assert sample(x[:1], -0.5) == sample(x[:1], 0.0) == [0]
    assert sample(x[:1], 1.0) == sample(x[:1], 7.0) == [3]
    assert sample(x[:1], float("nan")) == [0]
    # tiny and huge temperatures
    assert sample(x[:1], 0.49, temperature=1e-38) == [1] and sample(x[:1], 0.51, temperature=1e-38) == [2]
    assert [sample(x[:1], a, temperature=1e30)[0] for a in (0.2, 0.3, 0.6, 0.8)] == [0, 1, 2, 3]


@pytest.mark.parametrize("dt", DTYPES)
def test_infinities_and_nan(dt):
    inf, nan = np.inf, np.nan
    assert sample([[-inf, nan, -inf]], 0.5, dt) == [-1]
    assert sample([[-inf, nan, -inf]], 0.5, dt, temperature=0.0) == [-1]
    assert sample([[-inf, 2.0, nan]], 0.999, dt) == [1]
    assert [sample([[1.0, inf, 0.0, inf]], a, dt)[0] for a in (0.1, 0.49, 0.5, 0.9)] == [1, 1, 3, 3]
    assert sample([[1.0, inf, 0.0, inf]], 0.9, dt, top_k=1) == [1]
    big = 3e38
    assert sample([[-big, big, -big]], 0.99, dt) == [1]
    v = 20000
    x = np.full((2, v), nan, np.float32)
    x[0, 12345] = -4.0
    assert sample(x, 0.6, dt) == [12345, -1]
    assert sample(x, 0.6, dt, top_k=5, top_p=0.9, min_p=0.1) == [12345, -1]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shift", range(8))
def test_any_element_alignment(dt, shift):
    rng = np.random.default_rng(shift)
    x, u = logits(rng, 3, 9001 + shift, dt), rng.random(3).astype(np.float32)
    for kw in (dict(), dict(top_k=20, top_p=0.9)):
        assert sample(x, u, dt, ld=9001 + 2 * shift + 3, **kw) == reference(x, u, **kw)


def test_distribution():
    """100,000 draws with stratified u: each token's count is its share of
    them, off by at most its two borders."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal(40).astype(np.float32)
    n = 100000
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    got = np.bincount(sample(np.broadcast_to(x, (n, 40)).copy(), u, temperature=0.7), minlength=40)
    w = np.exp(x.astype(np.float64) / np.float32(0.7))
    assert np.all(np.abs(got - n * w / w.sum()) <= 2)


def test_recorded_call_reads_new_inputs():
    rng = np.random.default_rng(2)
    x = dev(rng.standard_normal((4, 30000)))
    u, tok = dev(rng.random(4)), torch.zeros(4, dtype=torch.int32, device="cuda")
    t, k, p, m = dev([0.5, 1.0, 0.0, 2.0]), dev([0, 9, 0, 0], torch.int32), dev([0.9, 1.0, 1.0, 1.0]), dev([0.0, 0.0, 0, 0.1])
    R.cb_sample_tokens(x, u, tok, t, k, p, m)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.cb_sample_tokens(x, u, tok, t, k, p, m)
    for seed in (3, 4):
        rng = np.random.default_rng(seed)
        x.copy_(dev(rng.standard_normal((4, 30000))))
        u.copy_(dev(rng.random(4)))
        g.replay()
        f = lambda a: a.cpu().numpy()
        assert tok.cpu().numpy().tolist() == reference(f(x), f(u), f(t), f(k), f(p), f(m))


def test_wrapper_refusals():
    x, u, tok = torch.zeros(2, 8, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in (dict(u=u.double()), dict(tokens=tok.long()), dict(top_k=u), dict(top_p=u[:1]), dict(logits=x[:, ::2]),
               dict(logits=x[0]), dict(min_p=u.cpu()), dict(logits=x.half())):
        with pytest.raises(ValueError):
            R.cb_sample_tokens(**{**dict(logits=x, u=u, tokens=tok), **kw})
