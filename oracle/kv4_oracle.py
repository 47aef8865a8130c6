"""Oracle of the key-value cache in 4 bits and of the page pool.

Plain numpy and lists from the definitions in include/spec_tree.h, sharing no code with the CUDA path.  Vectors are
float64 arrays of values of the model's type (`bits`: 8 of a bf16's significand, 11 of an f16's).  Test
infrastructure only.
"""
from __future__ import annotations

import numpy as np


def towards_zero(x, bits: int, least: int):
    """x >= 0 rounded towards zero to `bits` significand bits, no step below 2^least."""
    x = np.asarray(x, np.float64)
    e = np.maximum(np.frexp(x)[1] - bits, least)
    return np.trunc(np.ldexp(x, -e)) * np.ldexp(1.0, e)


def quantise(x, bits: int = 8):
    """(codes [..., D] uint8, scale [...], zero [...]) of vectors [..., D]; the range and the quotients in float32."""
    x = np.asarray(x, np.float32)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        zero = x.min(-1)
        spread = x.max(-1) - zero
        fine = np.isfinite(spread)
        spread = np.where(fine, spread, np.float32(0))
        scale = towards_zero(spread / np.float32(15), bits, -133 if bits == 8 else -24).astype(np.float32)
        quotient = (x - zero[..., None]) / scale[..., None]
    codes = np.where((scale > 0)[..., None], np.minimum(np.rint(quotient), 15), 0)
    codes = np.where(fine[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(fine, scale, np.nan).astype(np.float64), np.where(fine, zero, np.nan).astype(np.float64)


def values(codes, scale, zero):
    """float64 vectors that codes stand for."""
    return np.asarray(zero)[..., None] + np.asarray(scale)[..., None] * codes


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(data):
    return np.stack([data & 15, data >> 4], -1).reshape(data.shape[:-1] + (2 * data.shape[-1],))


class Pages:
    """The page pool: rows of pages, and a stack of those that nobody holds."""

    def __init__(self, B: int, n_pages: int, page_size: int, max_pages: int, stack):
        self.rows, self.stack = [[] for _ in range(B)], list(stack)
        self.n_pages, self.page_size, self.max_pages = n_pages, page_size, max_pages

    def reserve(self, lens, count: int, n_nodes=None):
        """(slots [B][count], whether some sequence got too little)."""
        slots, empty, short = [], False, False
        for b, length in enumerate(lens):
            n = count if n_nodes is None else min(count, max(0, n_nodes[b]))
            need = -(-(length + n) // self.page_size) if length >= 0 else 0
            if need > self.max_pages:
                need, short = 0, True
            lack = max(0, need - len(self.rows[b]))
            if lack > 0 and (empty or lack > len(self.stack)):
                empty = short = True
            else:
                for _ in range(lack):
                    self.rows[b].append(self.stack.pop())
            row = []
            for i in range(count):
                t = length + i
                there = length >= 0 and i < n and t // self.page_size < len(self.rows[b])
                row.append(self.rows[b][t // self.page_size] * self.page_size + t % self.page_size if there else -1)
            slots.append(row)
        return slots, short

    def release(self, keep):
        back = []
        for b, n in enumerate(keep):
            if n >= 0:
                kept = -(-n // self.page_size)
                back += self.rows[b][kept:]
                self.rows[b] = self.rows[b][:kept]
        self.stack += back[::-1]
