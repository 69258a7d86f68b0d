"""Plain float64 restatement of the 4-bit cache's format, of page bounds, page
selection and attention over picked pages."""
import numpy as np

from . import paged as OP

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the positive 8-bit floats (4 exponent, 3 mantissa bits), by code
SCALES = np.array([m * 2.0 ** -9 for m in range(8)] +
                  [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def _nearest(grid, x):
    """Index of the entry of an ascending grid nearest to x >= 0, ties to the even index."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    return np.where((lo < hi) | ((lo == hi) & ((i - 1) % 2 == 0)), i - 1, i)


def quantise(x):
    """x [..., 16 k] -> 4-bit codes (sign in bit 3) and scale codes [..., k]."""
    g = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], -1, 16)
    a = np.abs(g).max(-1)
    # a / 6 nearest to s is a nearest to 6 s: no quotient to round
    s = np.maximum(_nearest(6 * SCALES, np.minimum(a, 6 * 448.0)), 1)
    step = SCALES[s][..., None]
    code = np.zeros(g.shape, int)
    for k in range(7):          # borders between neighbours, met ones go to the even code
        border = 0.5 * (CODES[k] + CODES[k + 1]) * step
        code += (np.abs(g) >= border) if k % 2 else (np.abs(g) > border)
    code += 8 * np.signbit(g)
    return code.reshape(np.shape(x)), s


def values(code, scale):
    v = CODES[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(*v.shape[:-1], -1, 16) * SCALES[scale][..., None]).reshape(v.shape)


def round_to(x, bits):
    """float64 to `bits` significant bits, ties to even."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.round(m * 2.0 ** bits) / 2.0 ** bits, e)


def rotate_by_table(x, pos, table):
    """x [rows, heads * hd] rotated by the (cos, sin) pairs table [positions, hd / 2, 2]."""
    half = table.shape[1]
    z = np.asarray(x, np.float64).reshape(len(x), -1, 2, half)
    c, s = (table[pos][:, None, :, i].astype(np.float64) for i in (0, 1))
    a, b = z[:, :, 0], z[:, :, 1]
    return np.stack([a * c - b * s, b * c + a * s], 2).reshape(len(x), -1)


class Pool:
    """A pool of pages as bytes, and as codes and scales by slot."""

    def __init__(self, raw, page, hkv, hd):
        self.page, self.hkv, self.hd = page, hkv, hd
        self.raw = np.array(raw, np.uint8)
        h = self.raw[:, :page * hkv * hd * 9 // 8].reshape(len(raw), hkv, -1)
        n, self.part = page * hd // 2, {}
        for name, at, w in (("kc", 0, hd // 2), ("vc", n, hd // 2), ("ks", 2 * n, hd // 16),
                            ("vs", 2 * n + page * hd // 16, hd // 16)):
            # [pages, heads, slots, bytes]
            self.part[name] = h[:, :, at:at + page * w].reshape(len(raw), hkv, page, w)

    def put(self, which, pg, slot, x):
        """Row x [hkv * hd] (already divided by its power of two) to a slot."""
        code, scale = quantise(np.asarray(x).reshape(self.hkv, self.hd))
        self.part[which + "c"][pg, :, slot] = code[:, 0::2] + 16 * code[:, 1::2]
        self.part[which + "s"][pg, :, slot] = scale

    def values(self, which):
        """[pages, slots, hkv * hd]; slots whose scale is a NaN read as zeros."""
        b, s = self.part[which + "c"].astype(int), self.part[which + "s"].astype(int) & 127
        code = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], self.hd)
        v = values(code, np.minimum(s, 126))
        v = np.where(np.repeat(s == 127, 16, -1), 0.0, v)
        return v.transpose(0, 2, 1, 3).reshape(len(v), self.page, -1)


def page_bounds(bounds, k_pages, table, offsets, lens):
    """New bounds [pages, 2, row] with the pages of the new rows brought up to date."""
    out, page = np.array(bounds, np.float64), k_pages.shape[1]
    for s in range(len(lens)):
        n, kv = offsets[s + 1] - offsets[s], lens[s]
        for j in sorted({p // page for p in range(max(0, kv - n), kv)}):
            x = k_pages[table[s][j], :min(page, kv - j * page)]
            out[table[s][j], 0], out[table[s][j], 1] = x.min(0), x.max(0)
    return out


def page_scores(q, bounds, table_row, pages, n_q_heads, n_kv_heads, head_dim):
    """[n_kv_heads, pages] of one row q."""
    b = bounds[np.asarray(table_row)[:pages]].reshape(pages, 2, n_kv_heads, 1, head_dim)
    x = np.asarray(q, np.float64).reshape(1, n_kv_heads, -1, head_dim)
    return np.maximum(x * b[:, 0], x * b[:, 1]).sum(-1).max(-1).T


def select(q, bounds, table, offsets, lens, page, n_q_heads, n_kv_heads, head_dim, picks, n_first, n_last):
    """New picks [rows, n_kv_heads, n] with the sequences' rows set."""
    out, n = np.array(picks), picks.shape[2]
    for r, s, p in OP.row_positions(offsets, lens):
        out[r] = -1
        pages = p // page + 1 if p >= 0 else 0
        if pages <= n:
            out[r, :, :pages] = np.arange(pages)
            continue
        x = page_scores(q[r], bounds, table[s], pages, n_q_heads, n_kv_heads, head_dim)
        x[:, :n_first] = x[:, pages - n_last:] = np.inf
        for g in range(n_kv_heads):
            out[r, g] = np.sort(np.lexsort((np.arange(pages), -x[g]))[:n])
    return out


def picked_attention(q, k_pages, v_pages, picks, table, offsets, lens, n_q_heads, n_kv_heads, head_dim, scale, out):
    """`out` with the sequences' rows set; a page named twice counts twice."""
    out, page, G = np.array(out, np.float64), k_pages.shape[1], n_q_heads // n_kv_heads
    for r, s, p in OP.row_positions(offsets, lens):
        out[r] = 0.0
        for g in range(n_kv_heads):
            key = np.concatenate([j * page + np.arange(page) for j in picks[r, g] if j >= 0] + [np.zeros(0, int)]).astype(int)
            key = key[key <= p]
            if not len(key):
                continue
            at = np.asarray(table[s])[key // page], key % page
            c = slice(g * head_dim, (g + 1) * head_dim)
            K, V = k_pages[at][:, c].astype(np.float64), v_pages[at][:, c].astype(np.float64)
            for h in range(g * G, (g + 1) * G):
                d = slice(h * head_dim, (h + 1) * head_dim)
                x = scale * (K @ np.asarray(q[r, d], np.float64))
                w = np.exp(x - x.max())
                out[r, d] = (w / w.sum()) @ V
    return out
