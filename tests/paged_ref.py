"""The paged INT8 key/value cache and its operators in numpy and binary64,
from the definitions in include/qlin.h, without the library."""
import numpy as np

from w4a16_linear_layers_gb300 import synth

D = 128
BLOCK = 4224


def code_places():
    """[16, 128]: the byte of a block at which component d of token r stands (keys; values 2048 later)."""
    out = np.empty((16, D), np.int64)
    for r in range(16):
        for j in range(4):
            out[r, 32 * j:32 * j + 32] = 128 * r + 32 * (j ^ (r // 4)) + np.arange(32)
    return out


PLACES = code_places()


class Cache:
    """A cache's bytes as codes and scales of tokens."""

    def __init__(self, raw):
        self.raw = raw                       # uint8 [pages, kv_heads, page / 16, 4224]
        self.pages, self.kv_heads, blocks, n = raw.shape
        assert n == BLOCK
        self.page = 16 * blocks

    def _at(self, table, b, j):
        """The page of token j, or None."""
        p = int(table[b, j // self.page])
        return p if 0 <= p < self.pages else None

    def get(self, table, b, j):
        """(codes [2, kv_heads, 128] as int, scales fp32 [2, kv_heads]) of token j, None on no page."""
        p = self._at(table, b, j)
        if p is None:
            return None
        blk = self.raw[p, :, (j % self.page) // 16]
        r = j % 16
        codes = np.stack([blk[:, PLACES[r]], blk[:, 2048 + PLACES[r]]]).astype(np.int64) - 128
        s = np.stack([blk[:, 4096 + 4 * r:4100 + 4 * r], blk[:, 4160 + 4 * r:4164 + 4 * r]])
        return codes, np.ascontiguousarray(s).view(np.float32)[..., 0]

    def put(self, table, b, j, codes, scales):
        p = self._at(table, b, j)
        if p is None:
            return
        blk = self.raw[p, :, (j % self.page) // 16]
        r = j % 16
        for w in range(2):
            blk[:, 2048 * w + PLACES[r]] = (codes[w] + 128).astype(np.uint8)
            blk[:, 4096 + 64 * w + 4 * r:4100 + 64 * w + 4 * r] = \
                np.ascontiguousarray(scales[w].astype(np.float32)).view(np.uint8).reshape(-1, 4)

    def values(self, table, b, first, last):
        """K and V of tokens first .. last - 1 in binary64 [n, kv_heads, 128]
        and which of them are on a page."""
        n = max(last - first, 0)
        kv = np.zeros((2, n, self.kv_heads, D))
        ok = np.zeros(n, bool)
        for j in range(first, last):
            got = self.get(table, b, j)
            if got is not None:
                ok[j - first] = True
                kv[:, j - first] = got[0] * got[1].astype(np.float64)[..., None]
        return kv[0], kv[1], ok


def lengths(total, new, T, most):
    """(length, new tokens) of each sequence as the calls take them."""
    total = np.clip(np.asarray(total, np.int64), 0, most)
    top = np.minimum(T, total)
    return total, top if new is None else np.clip(np.asarray(new, np.int64), 0, top)


def rotate(u, c, s):
    """u [..., 128] turned by cosines and sines [..., R / 2], and the sums of the products' magnitudes."""
    half = c.shape[-1]
    y, size = u.copy(), np.abs(u)
    a, b = u[..., :half], u[..., half:2 * half]
    y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    size[..., :half] = np.abs(a * c) + np.abs(b * s)
    size[..., half:2 * half] = np.abs(b * c) + np.abs(a * s)
    return y, size


def codes_of(y):
    """Nearest integers to 127 y / max|y| [..., 128], the even one of two, and max|y|."""
    top = np.abs(y).max(-1, keepdims=True)
    return np.rint(127.0 * y / np.where(top > 0, top, 1.0)).astype(np.int64), top[..., 0]


def write(qkv, cache, table, total, q_heads, T, new=None, q_gamma=None, k_gamma=None, eps=1e-6, cos_sin=None,
          positions=None, axes=None):
    """qkv in binary64 [B T, heads * 128].  Yields (row, b, token, q [q_heads, 128],
    size of q's terms, codes [2, kv_heads, 128], scales in binary64 [2, kv_heads])
    for each row that is not padding."""
    B = table.shape[0]
    kv = cache.kv_heads
    x = qkv.reshape(B * T, q_heads + 2 * kv, D)
    total, new = lengths(total, new, T, table.shape[1] * cache.page)
    for b in range(B):
        for t in range(new[b]):
            row, pos = b * T + t, int(total[b] - new[b] + t)
            heads = {"q": x[row, :q_heads], "k": x[row, q_heads:q_heads + kv], "v": x[row, q_heads + kv:]}
            rho = {"v": np.ones((kv, 1))}
            size = {}
            for name, gamma in (("q", q_gamma), ("k", k_gamma)):
                h = heads[name]
                rho[name] = np.ones((h.shape[0], 1))
                if gamma is not None:
                    mean = (h * h).mean(-1, keepdims=True) + eps
                    rho[name] = np.where(mean > 0, 1.0 / np.sqrt(np.where(mean > 0, mean, 1.0)), 0.0)
                    h = h * gamma
                size[name] = np.abs(h)
                if cos_sin is not None:
                    P, R = cos_sin.shape
                    half = R // 2
                    if positions is None:
                        at = np.full(half, pos)
                    else:
                        A = positions.shape[0]
                        axis = np.zeros(half, int) if axes is None else np.minimum(axes.astype(int), A - 1)
                        at = positions[axis, row]
                    at = np.clip(at, 0, P - 1)
                    i = np.arange(half)
                    h, size[name] = rotate(h, cos_sin[at, i].astype(np.float64), cos_sin[at, half + i].astype(np.float64))
                heads[name] = h
            out = [codes_of(heads[name]) for name in ("k", "v")]
            scales = np.stack([out[0][1] * rho["k"][:, 0], out[1][1]]) / 127.0
            yield (row, b, pos, heads["q"] * rho["q"], size["q"] * rho["q"], np.stack([out[0][0], out[1][0]]), scales)


def attention(q, cache, table, total, T, new=None, scale=None, softcap=0.0, window=0, causal=True):
    """q in binary64 [B T, q_heads * 128].  Returns (out, A, X, N): the output,
    sum_j p_j |V_j| of it, the largest sum of a score's terms' magnitudes of each
    row's head, the largest |V|, and the rows that are not padding."""
    B = table.shape[0]
    heads = q.shape[1] // D
    G = heads // cache.kv_heads
    scale = D ** -0.5 if scale is None else scale
    total, new = lengths(total, new, T, table.shape[1] * cache.page)
    out = np.zeros((B * T, heads, D))
    A, X, big = np.zeros_like(out), np.zeros((B * T, heads, 1)), np.zeros((B * T, heads, 1))
    rows = np.zeros(B * T, bool)
    q = q.reshape(B * T, heads, D)
    for b in range(B):
        k, v, ok = cache.values(table, b, 0, int(total[b]))
        for t in range(new[b]):
            row, i = b * T + t, int(total[b] - new[b] + t)
            rows[row] = True
            j = np.arange(total[b])
            see = ok & ((j <= i) if causal else (j < total[b]))
            if window > 0:
                see &= np.abs(i - j) < window
            if not see.any():
                continue
            for h in range(heads):
                kk, vv = k[see, h // G], v[see, h // G]
                x = scale * (kk @ q[row, h])
                if softcap > 0:
                    x = softcap * np.tanh(x / softcap)
                p = np.exp(x - x.max())
                p /= p.sum()
                out[row, h], A[row, h] = p @ vv, p @ np.abs(vv)
                X[row, h], big[row, h] = abs(scale) * (np.abs(kk) @ np.abs(q[row, h])).max(), np.abs(vv).max()
    return out.reshape(B * T, -1), A.reshape(B * T, -1), np.repeat(X, D, 2).reshape(B * T, -1), \
        np.repeat(big, D, 2).reshape(B * T, -1), rows


def bf16(a):
    return synth.bf16_bits(np.asarray(a))


def bf16_to_f64(bits):
    return synth.bf16_values(bits).astype(np.float64)
