"""Plain float64 restatement of the generation operators: appending to a
paged cache, causal attention over it, and token sampling."""
import numpy as np


def rope_rotate(x, pos, head_dim, base):
    """x [rows, heads * head_dim] rotated to positions pos, rotate-half pairs."""
    half = head_dim // 2
    ang = np.multiply.outer(np.asarray(pos, np.float64), base ** (-np.arange(half) / half))
    z = np.asarray(x, np.float64).reshape(len(x), -1, 2, half)
    a, b = z[:, :, 0], z[:, :, 1]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    return np.stack([a * c - b * s, b * c + a * s], axis=2).reshape(len(x), -1)


def row_positions(offsets, lens):
    """(row, sequence, position) of every row inside the offsets."""
    out = []
    for s in range(len(lens)):
        n = offsets[s + 1] - offsets[s]
        out += [(offsets[s] + i, s, lens[s] - n + i) for i in range(n)]
    return out


def paged_append(k_pages, v_pages, table, offsets, lens, k_new, v_new, head_dim, base=None):
    """New pools with the rows appended; base None copies the keys."""
    kp, vp = np.array(k_pages, np.float64), np.array(v_pages, np.float64)
    page = kp.shape[1]
    for r, s, p in row_positions(offsets, lens):
        if p < 0:
            continue
        k = np.asarray(k_new[r:r + 1], np.float64)
        kp[table[s][p // page], p % page] = rope_rotate(k, [p], head_dim, base)[0] if base else k[0]
        vp[table[s][p // page], p % page] = v_new[r]
    return kp, vp


def paged_attention(q, k_pages, v_pages, table, offsets, lens, n_q_heads, n_kv_heads, head_dim,
                    scale, out):
    """`out` (float64 [rows, n_q_heads * head_dim]) with the sequences' rows set."""
    out = np.array(out, np.float64)
    page, G = k_pages.shape[1], n_q_heads // n_kv_heads
    for s in range(len(lens)):
        n, kv = offsets[s + 1] - offsets[s], lens[s]
        r0 = offsets[s]
        j = np.arange(kv)
        pages = np.asarray(table[s])[j // page] if kv else np.zeros(0, int)
        K = k_pages[pages, j % page].astype(np.float64).reshape(kv, n_kv_heads, head_dim)
        V = v_pages[pages, j % page].astype(np.float64).reshape(kv, n_kv_heads, head_dim)
        for i in range(n):
            p = kv - n + i
            if p < 0:
                out[r0 + i] = 0.0
                continue
            for h in range(n_q_heads):
                qh = np.asarray(q[r0 + i, h * head_dim:(h + 1) * head_dim], np.float64)
                x = scale * (K[:p + 1, h // G] @ qh)
                w = np.exp(x - x.max())
                out[r0 + i, h * head_dim:(h + 1) * head_dim] = (w / w.sum()) @ V[:p + 1, h // G]
    return out


def sample_token(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token of one row of logits for the uniform number u."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1
    if not temperature > 0 or top_p <= 0:
        return int(np.argmax(x))
    w = np.zeros(len(x))
    with np.errstate(invalid="ignore"):
        w = np.where(x == top, 1.0, np.where(x == -np.inf, 0.0, np.exp((x - top) / temperature)))
    rank = np.lexsort((np.arange(len(x)), -x))
    if 0 < top_k < len(x):
        rank = rank[:top_k]
    if top_p < 1:
        acc = np.cumsum(w[rank])
        rank = rank[:1 + int(np.searchsorted(acc, top_p * acc[-1], side="left"))]
    if min_p > 0:
        rank = rank[w[rank] >= min(min_p, 1.0)]
    rank = np.sort(rank[w[rank] > 0])
    acc = np.cumsum(w[rank])
    at = int(np.searchsorted(acc, max(u, 0.0) * acc[-1], side="right"))
    return int(rank[min(at, len(rank) - 1)])
