"""Plain 64-bit implementations of the paged cache's operations, and batches to
run them on, shared by the tests.  The 4-bit format is written out here from
its definition: e2m1 magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6 with a sign, one
e4m3 scale per 16 elements, to nearest with ties to the even code."""
from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])  # 0 .. 448; byte 0x7F is NaN


def nearest(x: np.ndarray, levels: np.ndarray) -> np.ndarray:
    """Index of the nearest level (ascending), a tie to the even index, above the last to the last."""
    x = x.astype(np.float64)
    hi = np.clip(np.searchsorted(levels, x), 1, len(levels) - 1)
    lo = hi - 1
    down, up = x - levels[lo], levels[hi] - x
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantise(x: np.ndarray, g: float):
    """fp32 row(s) [..., d] -> (codes [..., d], scale bytes [..., d/16]), each step rounded to fp32."""
    y = (x.astype(np.float32) / np.float32(g)).reshape(*x.shape[:-1], -1, 16)
    with np.errstate(invalid="ignore"):
        bad = ~np.isfinite(y).all(-1)
        y = np.where(bad[..., None], np.float32(0), y)
        byte = nearest(np.abs(y).max(-1) / np.float32(6), E4M3)
        s = E4M3[byte].astype(np.float32)
        z = np.where(s[..., None] > 0, y / np.where(s > 0, s, np.float32(1))[..., None], np.float32(0))
    code = nearest(np.abs(z), E2M1) + np.where(z < 0, 8, 0)
    code = np.where((bad | (byte == 0))[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 0x7F, byte).astype(np.uint8)


def values(code: np.ndarray, byte: np.ndarray, g: float) -> np.ndarray:
    """The values that codes and scale bytes stand for, in 64 bits."""
    s = np.where(byte == 0x7F, np.nan, E4M3[np.minimum(byte, 126)])
    v = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    return (v.reshape(*s.shape, 16) * s[..., None]).reshape(code.shape) * float(np.float32(g))


class Batch:
    """A cache with `lens[b]` positions of each sequence, of which the last
    `new[b]` are new rows, and everything a call on it needs (on the device).
    Pages are dealt out at random; the rest of the cache holds NaN."""

    def __init__(self, fmt, d, page, Hkv, lens, new, seed=0, scales=True, spare=2, max_pages=None, poison=True,
                 amplitude=1.0):
        from exact_attention_98_gb300 import fa

        self.fmt, self.d, self.page, self.Hkv, self.lens, self.new = fmt, d, page, Hkv, list(lens), list(new)
        rng = np.random.default_rng(seed)
        self.rng = rng
        need = [-(-n // page) for n in lens]
        self.max_pages = max_pages or max(1, max(need))
        self.num_pages = max(1, sum(need) + spare)
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), self.max_pages), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.k_scale = self.v_scale = None
        if fmt == "fp4" and scales:
            self.k_scale = rng.uniform(0.5, 2.0, Hkv).astype(np.float32)
            self.v_scale = rng.uniform(0.05, 0.2, Hkv).astype(np.float32)
        # every sequence's rows, in 64 bits as the cache holds them: [2][b][len, Hkv, d]
        self.rows = [[None] * len(lens), [None] * len(lens)]
        if fmt == "bf16":
            fill = np.full((self.num_pages, Hkv, 2, page, d), np.nan if poison else 0.0, np.float32)
        else:
            half = page * (d // 2 + d // 16)
            fill = np.full((self.num_pages, Hkv, 2, half), 0x7F if poison else 0, np.uint8)
        for kv in range(2):
            for b, n in enumerate(lens):
                x = torch.from_numpy(rng.standard_normal((n, Hkv, d)).astype(np.float32) * amplitude).to(torch.bfloat16)
                x = x.float().numpy()
                held = x.astype(np.float64)
                for h in range(Hkv):
                    g = 1.0 if self.k_scale is None else float((self.k_scale, self.v_scale)[kv][h])
                    if fmt == "fp4" and n:
                        code, byte = quantise(x[:, h], g)
                        held[:, h] = values(code, byte, g)
                    for pg in range(need[b]):
                        lo, hi = pg * page, min(n, (pg + 1) * page)
                        at = self.table[b, pg]
                        if fmt == "bf16":
                            fill[at, h, kv, : hi - lo] = x[lo:hi, h]
                        else:
                            codes = fill[at, h, kv, : page * d // 2].reshape(page, d // 2)
                            codes[: hi - lo] = code[lo:hi, 0::2] | (code[lo:hi, 1::2] << 4)
                            fill[at, h, kv, page * d // 2:].reshape(page, d // 16)[: hi - lo] = byte[lo:hi]
                self.rows[kv][b] = held
        self.pages = torch.from_numpy(fill).cuda()
        if fmt == "bf16":
            self.pages = self.pages.to(torch.bfloat16)
        self.cu_list = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.cu_list[-1])
        self.cu = torch.from_numpy(self.cu_list).cuda()
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.page_table = torch.from_numpy(self.table).cuda()
        dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
        self.kw = dict(k_scale=dev(self.k_scale), v_scale=dev(self.v_scale))
        self.fa = fa

    def tables(self):
        return self.pages, self.page_table, self.seq_lens, self.cu

    def forward(self, q, **kw):
        kw = {"max_new": max(1, max(self.new)), **self.kw, **kw}
        return self.fa.paged_forward(q, self.pages, self.page_table, self.seq_lens, self.cu, **kw)


def attend(q, rows_k, rows_v, length, window, sinks, scale):
    """64-bit attention of the last rows q [n, H, d] of a sequence over its positions.
    Returns O, LSE, sum_j p_j |v_j| and the largest sum_t |q_t k_t| of each row."""
    n, H, d = q.shape
    Hkv = rows_k.shape[1]
    o, lse, mag = np.zeros((n, H, d)), np.full((n, H), -np.inf), np.zeros((n, H, d))
    dot = np.zeros((n, H))
    for i in range(n):
        p = length - n + i
        if p < 0:
            continue
        j = np.arange(p + 1)
        j = j[(p - j < window) | (j < sinks)] if window else j
        for h in range(H):
            k, v = rows_k[j, h * Hkv // H], rows_v[j, h * Hkv // H]
            s = scale * (k @ q[i, h])
            m = s.max()
            w = np.exp(s - m)
            lse[i, h] = m + math.log(w.sum())
            w /= w.sum()
            o[i, h], mag[i, h] = w @ v, w @ np.abs(v)
            dot[i, h] = scale * (np.abs(k) @ np.abs(q[i, h])).max()
    return o, lse, mag, dot
