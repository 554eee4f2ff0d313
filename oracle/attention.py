"""Oracle of a decode step's attention side (TEST INFRASTRUCTURE ONLY):
rotary positions, the paged key-value cache in the activation formats, and
the attention of one query row per sequence over it, in float64."""
from __future__ import annotations

import numpy as np

from . import quant
from .formats import decode_bf16


def rotary(x, positions, inv_freq, layout="half", factor=1.0, inverse=False):
    """x [T, H, D] -> float64 [T, H, D]: pair i of the first R = 2 len(inv_freq)
    elements turned by positions * inv_freq[i], the rest copied."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    r = 2 * len(inv_freq)
    ang = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = factor * np.cos(ang), factor * np.sin(ang) * (-1.0 if inverse else 1.0)
    i0 = np.arange(r // 2) if layout == "half" else np.arange(0, r, 2)
    i1 = i0 + (r // 2 if layout == "half" else 1)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i0] * s + x[..., i1] * c
    return y


def quantize_rows(bits, fmt):
    """bf16 bit patterns uint16 [N, D] -> (code bytes [N, row], scale bytes [N, scale bytes])."""
    n = bits.shape[0]
    if fmt == "bf16":
        return np.ascontiguousarray(bits).view(np.uint8).reshape(n, -1), np.zeros((n, 0), np.uint8)
    x = decode_bf16(bits)
    if fmt == "fp8_token":
        c, s = quant.quant_fp8_per_token(x.astype(np.float32))
        return c, np.ascontiguousarray(s).view(np.uint8).reshape(n, 4)
    return quant.quant_mxfp8(x) if fmt == "mxfp8" else quant.quant_mxfp4(x)


def row_values(codes, scales, fmt):
    """Code and scale bytes of rows -> float64 [N, D]."""
    n = codes.shape[0]
    if fmt == "bf16":
        return decode_bf16(np.ascontiguousarray(codes).view(np.uint16).reshape(n, -1))
    if fmt == "fp8_token":
        return quant.dequant_fp8_per_token(codes, np.ascontiguousarray(scales).view(np.float32).reshape(n))
    return (quant.dequant_mxfp8 if fmt == "mxfp8" else quant.dequant_mxfp4)(codes, scales)


def row_bytes(fmt, d):
    return {"bf16": 2 * d, "fp8_token": d, "mxfp8": d, "mxfp4": d // 2}[fmt], \
        {"bf16": 0, "fp8_token": 4, "mxfp8": d // 32, "mxfp4": d // 32}[fmt]


class Cache:
    """The cache's bytes [pages][heads][unit] in the layout hum.h documents."""

    def __init__(self, fmt, pages, page_size, heads, d, fill=0):
        self.fmt, self.ps, self.heads, self.d = fmt, page_size, heads, d
        self.row, self.scale = row_bytes(fmt, d)
        self.buf = np.full((pages, heads, 2 * page_size * (self.row + self.scale)), fill, np.uint8)

    def _where(self, which, at):
        """(code offset, offsets of the row's scale bytes) of token `at` of a page."""
        code = (which * self.ps + at) * self.row
        base = 2 * self.ps * self.row + which * self.ps * self.scale
        if which and self.fmt.startswith("mx"):
            return code, base + np.arange(self.scale) * self.ps + at
        return code, base + at * self.scale + np.arange(self.scale)

    def write(self, slots, k_bits, v_bits):
        for which, bits in ((0, k_bits), (1, v_bits)):
            t = bits.shape[0]
            codes, scales = quantize_rows(bits.reshape(t * self.heads, self.d), self.fmt)
            codes, scales = codes.reshape(t, self.heads, -1), scales.reshape(t, self.heads, -1)
            for i, s in enumerate(slots):
                if not 0 <= s < self.buf.shape[0] * self.ps:
                    continue
                off, sc = self._where(which, s % self.ps)
                self.buf[s // self.ps, :, off:off + self.row] = codes[i]
                self.buf[s // self.ps][:, sc] = scales[i]

    def rows(self, slots, which):
        """float64 [len(slots), heads, d]; zeros for a slot outside the cache."""
        out = np.zeros((len(slots), self.heads, self.d))
        for i, s in enumerate(slots):
            if 0 <= s < self.buf.shape[0] * self.ps:
                off, sc = self._where(which, s % self.ps)
                page = self.buf[s // self.ps]
                out[i] = row_values(page[:, off:off + self.row], page[:, sc], self.fmt)
        return out


def attention(cache, q, block_table, seq_lens, scale, window=0):
    """q float64 [B, Hq, D] -> (out [B, Hq, D], lse [B, Hq], bound terms):
    the terms are sum_t p_t |v_t| [B, Hq, D] and max_t scale sum_d |q_d k_td|
    [B, Hq], from which a test derives what roundings may cost."""
    b, hq, d = q.shape
    out, mag = np.zeros((b, hq, d)), np.zeros((b, hq, d))
    lse, big = np.full((b, hq), -np.inf), np.zeros((b, hq))
    for i in range(b):
        n = int(np.clip(seq_lens[i], 0, block_table.shape[1] * cache.ps))
        t = np.arange(max(0, n - window) if window else 0, n)
        page = block_table[i][t // cache.ps].astype(np.int64)
        t, page = t[(page >= 0) & (page < cache.buf.shape[0])], page[(page >= 0) & (page < cache.buf.shape[0])]
        if len(t) == 0:
            continue
        slots = page * cache.ps + t % cache.ps
        k, v = cache.rows(slots, 0), cache.rows(slots, 1)
        for h in range(hq):
            hk = h // (hq // cache.heads)
            s = scale * (k[:, hk] @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            lse[i, h] = m + np.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ v[:, hk]
            mag[i, h] = p @ np.abs(v[:, hk])
            big[i, h] = (abs(scale) * (np.abs(k[:, hk]) @ np.abs(q[i, h]))).max()
    return out, lse, mag, big


