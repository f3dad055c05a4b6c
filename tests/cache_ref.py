"""Plain 64-bit forms of the paged-cache operators, and how far their kernels
may be from them.

Everything is loops over sequences and heads on the CPU in fp64, from the
operators' definitions; nothing is shared with the library.
"""
import numpy as np
import torch

CACHE = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
IN = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative to the value


def round_e4m3(y):
    """Nearest e4m3 value (half to even) of |y| <= 448, fp64: three bits behind
    the leading one, steps of 2^-9 below 2^-6."""
    _, e = np.frexp(np.abs(y))  # |y| = m 2^e, m in [0.5, 1)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.round(y / step) * step


def quantise(x, cache):
    """(stored values as numbers, scales or None) of rows x [..., D] in fp64."""
    x = np.asarray(x, np.float64)
    if cache in ("bf16", "f32"):
        return torch.from_numpy(x).to(CACHE[cache]).double().numpy(), None
    fine = np.isfinite(x).all(-1)
    top = np.abs(np.where(fine[..., None], x, 0.0)).max(-1)
    safe = np.where(top == 0, 1.0, top)
    if cache == "e4m3":
        m, e = np.frexp(safe)
        s = np.exp2(np.maximum(np.where(m <= 0.875, e - 9, e - 8), -126).astype(np.float64))
        q = round_e4m3(np.where(fine[..., None], x, 0.0) / s[..., None])
    else:
        s = (safe.astype(np.float32) / np.float32(127)).astype(np.float64)
        q = np.round(np.where(fine[..., None], x, 0.0) * 127 / safe[..., None])
    s = np.where(top == 0, 1.0, s)
    return q, np.where(fine, s, np.nan)


class Paged:
    """A cache of random rows on the CPU, a page table whose pages are out of
    order, and the values its rows stand for."""

    def __init__(self, B, Hkv, D, kv, page, cache, seed=0, garbage=True, wide=None):
        g = np.random.Generator(np.random.PCG64(seed))
        self.B, self.Hkv, self.D, self.page, self.cache = B, Hkv, D, page, cache
        self.kv = list(kv)
        need = [-(-a // page) for a in self.kv]
        self.pages = sum(need) + 2
        self.wide = wide or max(1, max(need))
        order = g.permutation(self.pages)
        self.table = np.full((B, self.wide), -1, np.int32)  # pages that no position needs: none
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.t = {}
        for x in ("k", "v"):
            rows = g.standard_normal((self.pages, Hkv, page, D)).astype(np.float32)
            q, s = quantise(rows, cache)
            self.t[x] = torch.from_numpy(q).to(CACHE[cache])
            self.t[x + "_s"] = None if s is None else torch.from_numpy(s).float()
        if garbage:  # rows of pages that no position names: NaN where the type has one
            used = torch.zeros(self.pages, page, dtype=torch.bool)
            for b in range(B):
                for p in range(self.kv[b]):
                    used[self.table[b, p // page], p % page] = True
            for x in ("k", "v"):
                if cache in ("bf16", "f32"):
                    self.t[x].masked_fill_(~used[:, None, :, None], float("nan"))
                else:
                    self.t[x + "_s"].masked_fill_(~used[:, None], float("nan"))

    def where(self, b, p):
        return self.table[b, p // self.page], p % self.page

    def values(self, x):
        y = self.t[x].double()
        s = self.t[x + "_s"]
        return (y if s is None else y * s.double()[..., None]).numpy()

    def rows(self, x, b, lo, hi):
        """Values of positions lo .. hi - 1 of sequence b, [Hkv, hi - lo, D]; a
        table entry that names no page: zeros."""
        val = self.values(x)
        out = np.zeros((self.Hkv, max(0, hi - lo), self.D))
        for i, p in enumerate(range(lo, hi)):
            pg, r = self.where(b, p)
            if 0 <= pg < self.pages:
                out[:, i] = val[pg, :, r]
        return out

    def gpu(self):
        """The calls' cache arguments on the device."""
        c = dict(k_cache=self.t["k"].cuda(), v_cache=self.t["v"].cuda(),
                 table=torch.from_numpy(self.table).cuda(),
                 kv_len=torch.tensor(self.kv, dtype=torch.int32).cuda())
        if self.t["k_s"] is not None:
            c.update(k_scale=self.t["k_s"].cuda(), v_scale=self.t["v_s"].cuda())
        return c


def attend(P, q, new, scale, causal=True, window=0, q_type="bf16"):
    """(o, lse, tol_o, tol_lse) in fp64, of q [B, Hq, n, D] (a CPU tensor); rows i >= new[b] NaN.

    tol: with A = sum_t p_t |v_t| and every fp32 sum of m terms off by at most
    m 2^-24 of the sum of their magnitudes,
      logits   d = |scale| max_t sum_e |q_e k_te| (D + 4) 2^-24 + 2^-22 |logit|
               (an int8 row's scale, the softmax scale, base 2: 4 roundings),
      weights  2 d + 2^-20 (exp2 to 2^-22, its argument's rounding is in d),
      sums     (keys + 64) 2^-24 for the numerator and for the denominator,
      bf16     2^-8 A: the weights rounded once for the tensor cores,
    and the output's own rounding, half a step of o.
    """
    B, Hq, n, D = q.shape
    G = Hq // P.Hkv
    q = q.double().numpy()
    o = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:3], np.nan)
    to, tl = np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        K, V = P.rows("k", b, 0, P.kv[b]), P.rows("v", b, 0, P.kv[b])
        for i in range(new[b]):
            pos = P.kv[b] - new[b] + i
            hi = min(P.kv[b], pos + 1) if causal else P.kv[b]
            lo = max(0, pos - window + 1) if causal and window else 0
            for h in range(Hq):
                if hi <= lo:
                    o[b, h, i], lse[b, h, i] = 0.0, -np.inf
                    continue
                k, v = K[h // G, lo:hi], V[h // G, lo:hi]
                x = scale * (k @ q[b, h, i])
                m = x.max()
                p = np.exp(x - m)
                total = p.sum()
                p /= total
                o[b, h, i] = p @ v
                lse[b, h, i] = m + np.log(total)
                u = 2.0 ** -24
                d = abs(scale) * (np.abs(k) @ np.abs(q[b, h, i])).max() * (D + 4) * u
                d += np.abs(x).max() * 2.0 ** -22
                e = 2 * d + 2.0 ** -20 + 2 * (hi - lo + 64) * u
                A = p @ np.abs(v)
                to[b, h, i] = A * (e + (HALF["bf16"] if q_type == "bf16" else 0)) * 1.01
                to[b, h, i] += HALF[q_type] * np.abs(o[b, h, i]) * 1.01 + 1e-30
                tl[b, h, i] = e + 4 * u * abs(lse[b, h, i]) + 1e-6
    return o, lse, to, tl
