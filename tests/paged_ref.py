"""A paged KV cache in numpy, and the paged calls' results in 64 bits."""
import numpy as np


def quantise(x):
    """Q8 of x [..., head_dim] (float32): (codes int8, scales float16 [..., head_dim / 32])."""
    b = x.astype(np.float64).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        d = (np.abs(b).max(-1) / 127.0).astype(np.float16)
        bad = ~np.isfinite(b).all(-1) | ~np.isfinite(d)
        df = np.where(bad, 0, d.astype(np.float64))[..., None]
        code = np.where(df > 0, np.clip(np.rint(b / np.where(df > 0, df, 1.0)), -127, 127), 0.0)
    code = np.where(bad[..., None], 0.0, code)
    d = np.where(bad, np.float16(np.nan), d).astype(np.float16)
    return code.astype(np.int8).reshape(x.shape), d


def values(codes, d):
    """What Q8 codes stand for: f16(code * d)."""
    b = codes.astype(np.float64).reshape(*codes.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        return (b * d.astype(np.float64)[..., None]).astype(np.float16).reshape(codes.shape)


class Cache:
    """Random pages and a batch: sequence s has new[s] new tokens of total[s] positions."""

    def __init__(self, new, total, n_kv, hd, page, q8=False, seed=0, n_tokens=None, spare=2, width=None):
        rng = self.rng = np.random.default_rng(seed)
        self.new, self.total, self.n_kv, self.hd, self.page, self.q8 = list(new), list(total), n_kv, hd, page, q8
        used = [-(-t // page) for t in total]
        self.width = width or max(max(used), 1) + 1
        self.n_pages = sum(used) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(self.new), self.width), -1, np.int32)
        at = 0
        for s, n in enumerate(used):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.lens = np.asarray(self.total, np.int32)
        self.n_tokens = int(self.starts[-1]) if n_tokens is None else n_tokens
        self.pages, self.scales = {}, {}
        for name in "kv":
            x = rng.normal(size=(self.n_pages, n_kv, page, hd)).astype(np.float32)
            if q8:
                self.pages[name], self.scales[name] = quantise(x)
            else:
                self.pages[name], self.scales[name] = x.astype(np.float16), None

    def stored(self, name, s, length):
        """(values [n_kv][length][hd] float64, which positions are in a page)."""
        out = np.zeros((self.n_kv, length, self.hd))
        there = np.zeros(length, bool)
        for t in range(0, length, self.page):
            e = t // self.page
            p = self.table[s, e] if e < self.width else -1
            if not 0 <= p < self.n_pages:
                continue
            x = values(self.pages[name][p], self.scales[name][p]) if self.q8 else self.pages[name][p]
            n = min(self.page, length - t)
            out[:, t:t + n] = x.astype(np.float64)[:, :n]
            there[t:t + n] = True
        return out, there

    def position(self, s, i):
        return self.total[s] - self.new[s] + i

    def attend(self, q, n_q, window=0, sinks=0):
        """q [n_tokens][n_q * hd] -> (out, error bound), both [n_tokens][n_q * hd]; rows of no sequence are NaN.

        The bound, per element: the output's rounding to binary16 is half a
        step, 2^-11 of the value or 2^-25, and each softmax weight's is 2^-11 of it or 2^-25 (against a largest
        weight of at least one): together (2^-10 + small) sum w|v| + n 2^-25 max|v| + 2^-24.  A score's error is at
        most 2^-20 S, S = sum |q k| / sqrt(hd): queries kept to 2^-22, the sum of at most 256 exact products in
        fp32 steps of 2^-24 and the exponent's few roundings; a weight's relative error is the score's (twice: its
        own and the sum's)."""
        g, hd = n_q // self.n_kv, self.hd
        out = np.full((self.n_tokens, n_q * hd), np.nan)
        tol = np.full_like(out, np.nan)
        for s in range(len(self.new)):
            k, there = self.stored("k", s, self.total[s])
            v, _ = self.stored("v", s, self.total[s])
            for i in range(self.new[s]):
                r, p = int(self.starts[s]) + i, self.position(s, i)
                t = np.arange(self.total[s])
                sees = (t <= p) & there
                if window:
                    sees &= (t > p - window) | (t < sinks)
                if not sees.any():
                    out[r], tol[r] = 0.0, 0.0
                    continue
                ks, vs = k[:, sees], v[:, sees]
                x = q[r].astype(np.float64).reshape(self.n_kv, g, hd)
                with np.errstate(all="ignore"):
                    sc = np.einsum("kgd,ktd->kgt", x, ks) / np.sqrt(hd)
                    size = np.einsum("kgd,ktd->kgt", np.abs(x), np.abs(ks)).max(-1) / np.sqrt(hd)
                    w = np.exp(sc - sc.max(-1, keepdims=True))
                    w /= w.sum(-1, keepdims=True)
                    o = np.einsum("kgt,ktd->kgd", w, vs)
                    a = np.einsum("kgt,ktd->kgd", w, np.abs(vs))
                    most = np.abs(np.where(np.isfinite(vs), vs, 0.0)).max()
                    b = (2.0 ** -10 + 2.0 ** -19 * size)[..., None] * a + sees.sum() * 2.0 ** -25 * most + 2.0 ** -24
                out[r], tol[r] = o.reshape(-1), b.reshape(-1)
        return out, tol
