"""Plain 64-bit implementations of the 4-bit KV cache's operators on the CPU, written from their
definitions (include/splitzip_kv4.h), and bounds on what rounding may add.

Bounds.  u(t) = finfo(t).eps / 2 is the largest relative error of one rounding to type t; sums of n
terms held in fp32 are off by at most n u(fp32) of the sum of absolute terms."""
from __future__ import annotations

import math

import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U32 = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def quantize(x: np.ndarray):
    """Codes (one a byte) and scale bytes of x [..., D], float64 values."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    codes = np.zeros(b.shape, np.uint8)
    scales = np.zeros(b.shape[:-1], np.uint8)
    for at in np.ndindex(*scales.shape):
        v = b[at]
        if not np.isfinite(v).all():
            scales[at] = 255
            continue
        top = np.abs(v).max()
        e = 2 - 127
        while e < 252 - 127 and top >= 7 * 2.0 ** e:
            e += 1
        scales[at] = e + 127
        for i, y in enumerate(np.abs(v) / 2.0 ** e):
            gap = np.abs(GRID - min(y, 6.0))
            near = np.flatnonzero(gap == gap.min())
            c = near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]
            codes[at + (i,)] = c | (8 if np.signbit(v[i]) else 0)
    return codes.reshape(x.shape), scales


def dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    sign = np.where(codes & 8, -1.0, 1.0)
    v = (sign * GRID[codes & 7]).reshape(*codes.shape[:-1], -1, 32)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(codes.shape)


class Cache:
    """A cache's buffers on the host, token by token, in 64 bits."""

    def __init__(self, cache):
        self.page = cache.page_size
        self.k = self._values(cache.k_codes, cache.k_scales)
        v = cache.v_codes.permute(0, 1, 2, 4, 3, 5).flatten(2, 3).flatten(3)      # [P, H, page, D / 2]
        self.v = self._values(v, cache.v_scales.transpose(2, 3))
        self.w = cache.weights.cpu().double()

    @staticmethod
    def _values(codes, scales):
        b = codes.cpu().numpy()
        nib = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)
        return torch.from_numpy(dequantize(nib, scales.cpu().numpy()))

    def tokens(self, row, n):
        """Keys and values [n, H, D] of a table row's first n tokens; usable [n]: on a page that exists."""
        k = torch.zeros(n, self.k.shape[1], self.k.shape[3], dtype=torch.float64)
        v, ok = torch.zeros_like(k), torch.zeros(n, dtype=torch.bool)
        for j in range(n):
            p = int(row[j // self.page])
            if 0 <= p < len(self.k):
                k[j], v[j], ok[j] = self.k[p, :, j % self.page], self.v[p, :, j % self.page], True
        return k, v, ok


def sees(m: int, n: int, window, sinks) -> torch.Tensor:
    """[m, n]: which of n tokens the last m queries see."""
    i = torch.arange(m)[:, None] + n - m
    j = torch.arange(n)[None]
    ok = j <= i
    if window is not None:
        ok &= (j > i - window) | (j < sinks)
    return ok


def scores(q, k, scale):
    """[m, n] scores of one head, and the error a sum of D products in fp32 may have."""
    d = q.shape[1]
    return q @ k.T * scale, (d + 8) * U32 * (q.abs() @ k.abs().T * abs(scale))


def attend(ref: Cache, q, rows, lens, counts, scale, window, sinks, out_dtype):
    """out, lse in 64 bits and their bounds, for q [total, Hq, D] (float64 on the CPU)."""
    total, hq, d = q.shape
    group = hq // ref.k.shape[1]
    out, out_tol = torch.zeros(total, hq, d, dtype=torch.float64), torch.zeros(total, hq, d, dtype=torch.float64)
    lse, lse_tol = torch.full((total, hq), -math.inf, dtype=torch.float64), torch.zeros(total, hq, dtype=torch.float64)
    # the probabilities of the second product: bf16, or two halves of 8 bits
    up = half_step(torch.bfloat16) if out_dtype == torch.bfloat16 else half_step(torch.bfloat16) ** 2
    uo = half_step(out_dtype)
    at = 0
    for row, n, m in zip(rows, lens, counts):
        k, v, ok = ref.tokens(row, n)
        see = sees(m, n, window, sinks) & ok
        for f in range(hq):
            h = f // group
            s, es = scores(q[at:at + m, f], k[:, h], scale)
            for i in range(m):
                j = see[i].nonzero()[:, 0]
                if len(j) == 0:
                    continue
                x, e = s[i, j], float(es[i, j].max())
                p = torch.softmax(x, 0)
                o, a = p @ v[j, h], p @ v[j, h].abs()
                big = float(x.abs().max())
                # an exponent off by e plus the roundings of its argument changes p by that factor; the
                # normalizing sum has the same; both products add up in fp32
                rel = 2 * e + 8 * U32 * (big + 8) + 2 * (len(j) + 64) * U32
                out[at + i, f] = o
                out_tol[at + i, f] = (uo * o.abs() + (up + rel) * a) * (1 + 2.0 ** -6) + 2.0 ** -25 * (out_dtype == torch.float16)
                lse[at + i, f] = torch.logsumexp(x, 0)
                lse_tol[at + i, f] = e + (len(j) + 64) * U32 + 8 * U32 * (big + 8 + math.log(len(j)))
        at += m
    return out, out_tol, lse, lse_tol


def weigh(ref: Cache, q, lse, rows, lens, counts, scale, window, sinks):
    """New weights [P, H, page] in 64 bits and their bounds."""
    total, hq, d = q.shape
    group = hq // ref.k.shape[1]
    w, tol = ref.w.clone(), torch.zeros_like(ref.w)
    at = 0
    for row, n, m in zip(rows, lens, counts):
        k, _, ok = ref.tokens(row, n)
        see = sees(m, n, window, sinks) & ok
        for f in range(hq):
            h = f // group
            s, es = scores(q[at:at + m, f], k[:, h], scale)
            L = lse[at:at + m, f, None]
            e = torch.where(see & (L != -math.inf), s - L, torch.full_like(s, -math.inf))
            p = torch.exp(e)
            rel = es + 8 * U32 * (s.abs() + torch.where(L.isfinite(), L.abs(), 0.0) + 8) + (m * hq + 8) * U32
            t = torch.where(p > 0, p * rel, 0.0).sum(0)
            for j in range(n):
                if ok[j]:
                    w[int(row[j // ref.page]), h, j % ref.page] += p[:, j].sum()
                    tol[int(row[j // ref.page]), h, j % ref.page] += t[j]
        at += m
    return w, tol + 2 * U32 * w.abs()


def choose(weights, n: int, budget: int, sinks: int, recent: int):
    """Kept tokens of one sequence and head from its n weights."""
    if n <= budget:
        return list(range(n))
    room = budget - sinks - recent
    mid = sorted(range(sinks, n - recent),
                 key=lambda j: (0 if not math.isnan(weights[j]) else 1, -weights[j] if not math.isnan(weights[j]) else 0.0, j))
    return sorted([*range(sinks), *mid[:room], *range(n - recent, n)])
