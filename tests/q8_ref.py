"""Plain reference of the paged 8-bit cache, in Python lists and float64: block
bookkeeping one block at a time, quantisation one block at a time, attention one
head at a time.  Shares nothing with the library."""
from __future__ import annotations

import math
from typing import List

import numpy as np
import torch


class Blocks:
    """Requests' block lists and a free stack."""

    def __init__(self, lens: List[int], table: List[List[int]], free: List[int], block: int, max_blocks: int):
        self.len, self.table, self.free = list(lens), [list(r) for r in table], list(free)
        self.block, self.max_blocks = block, max_blocks

    def count(self, n: int) -> int:
        return -(-n // self.block)

    def change(self, add: List[int], n_rows: int):
        """(start, slot, granted, refused) of one ckv_plan_blocks call."""
        before = list(self.len)
        back = []
        for b, a in enumerate(add):
            if a < 0:
                self.len[b] = max(0, self.len[b] + a)
                keep = self.count(self.len[b])
                back += self.table[b][keep:]
                self.table[b] = self.table[b][:keep]
        self.free += back[::-1]
        start, refused, asked = [0], False, 0
        room = len(self.free)
        slot = [-1] * n_rows
        for b, a in enumerate(add):
            first = start[-1]
            start.append(first + max(a, 0))
            if a <= 0:
                continue
            n = self.len[b]
            if n + a > self.max_blocks * self.block or start[-1] > n_rows:
                refused = True
                continue
            need = self.count(n + a) - self.count(n)
            asked += need
            if need and asked > room:
                refused = True
                continue
            for _ in range(need):
                self.table[b].append(self.free.pop())
            for i in range(a):
                pos = n + i
                slot[first + i] = self.table[b][pos // self.block] * self.block + pos % self.block
            self.len[b] = n + a
        return start, slot, [x - y for x, y in zip(self.len, before)], refused


def scale_of(amax: float, fmt: str) -> float:
    amax = max(float(amax), 2.0 ** -100)
    if fmt == "int8":
        return float(np.float32(amax) / np.float32(127))
    s = 2.0 ** math.floor(math.log2(amax / 448.0))
    while amax > 448.0 * s:
        s *= 2.0
    while amax <= 224.0 * s:
        s /= 2.0
    return s


def codes_of(x: np.ndarray, f: float, fmt: str) -> np.ndarray:
    """Nearest code to x f (x, f hold fp32 values), ties to even, as a float64 value."""
    y = x.astype(np.float64) * f
    if fmt == "int8":
        return np.clip(np.rint(y), -127, 127)
    a = np.abs(y)
    # e4m3: steps of 2^(e-3) at 2^e, 2^-9 below 2^-6
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    e = np.where(a >= 2.0 ** (e + 1), e + 1, e)
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.sign(y) * np.minimum(np.rint(a / step) * step, 448.0)


class Pool:
    """Code values and scales of one of K or V: dicts by (block, head)."""

    def __init__(self, codes: np.ndarray, scales: np.ndarray, block: int, fmt: str):
        self.codes, self.scales = codes.astype(np.float64).copy(), scales.astype(np.float64).copy()
        self.block, self.fmt = block, fmt

    def append(self, blocks: Blocks, granted: List[int], rows: List[np.ndarray]) -> None:
        """rows[b]: [granted[b], Hkv, d]; lengths already count them."""
        bs = self.block
        for b, a in enumerate(granted):
            if a <= 0:
                continue
            pos = blocks.len[b] - a
            done = 0
            while done < a:
                blk, lo = blocks.table[b][pos // bs], pos % bs
                m = min(a - done, bs - lo)
                for h in range(self.codes.shape[1]):
                    x = rows[b][done: done + m, h]
                    s = scale_of(np.abs(x).max(), self.fmt)
                    old = self.scales[blk, h]
                    if lo > 0:
                        s = max(s, old)
                    inv = float(np.float32(1) / np.float32(s))
                    if lo > 0 and s != old:
                        f = float(np.float32(old) * np.float32(inv))
                        self.codes[blk, h, :lo] = codes_of(self.codes[blk, h, :lo], f, self.fmt)
                    self.codes[blk, h, lo: lo + m] = codes_of(x, inv, self.fmt)
                    self.scales[blk, h] = s
                done += m
                pos += m

    def rows(self, blocks: Blocks, b: int, positions) -> np.ndarray:
        """Values held at positions of request b: [n, Hkv, d]."""
        bs = self.block
        out = np.zeros((len(positions), self.codes.shape[1], self.codes.shape[3]))
        for i, p in enumerate(positions):
            blk = blocks.table[b][p // bs]
            out[i] = self.codes[blk, :, p % bs] * self.scales[blk][:, None]
        return out


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray):
    """One head: q [d], k and v [n, d] in float64; (out, S) with S the largest sum of |q_i k_i| / sqrt(d)."""
    if len(k) == 0:
        return np.zeros(q.shape), 0.0
    x = k @ q / math.sqrt(q.shape[0])
    p = np.exp(x - x.max())
    return (p / p.sum()) @ v, float((np.abs(k) @ np.abs(q)).max() / math.sqrt(q.shape[0]))


def attention_tol(S: float, n: int, vmax: float) -> float:
    """Error bound of one output.  A score, in base-2 units at most S / ln 2 in
    magnitude sum: q as two fp16 terms (2^-22 relative), d/16 <= 8 products added
    in fp32 with 2^-23 each (a truncating accumulator), two more roundings for
    the scales: <= 14 * 2^-23 S/ln 2 absolute, so a weight is off by at most that
    times ln 2, plus 2^-22 (exp2), 2^-22 (weight as two fp16 terms) and 2 * 2^-24
    (scale products).  The sums add 2^-23 per tile of 16 tokens and per join
    (<= 300 of those).  Numerator and denominator both carry it; twice the whole
    since first-order terms are dropped."""
    rel = 14 * 2.0 ** -23 * S + 2 * 2.0 ** -22 + 2.0 ** -23 + 2.0 ** -23 * (n / 16 / 8 + 8 + 300)
    return 2 * 2 * rel * vmax


def code_values(t: torch.Tensor) -> np.ndarray:
    return t.float().cpu().numpy().astype(np.float64)
