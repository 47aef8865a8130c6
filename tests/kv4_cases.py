"""Inputs of the tests of the key-value cache in 4 bits: the 16-bit cases of kv_cases, quantised by the oracle."""
import numpy as np
import torch

import kv_cases
from oracle import kv4_oracle as O4

BITS = {torch.bfloat16: 8, torch.float16: 11}
FEW_ROWS = 16


def quantised(c):
    """(key codes, value codes: uint8 [layers][pages][page][Hkv][D / 2]; scale [layers][pages][Hkv][page][4]; the pools
    of float64 values that they stand for) of a case."""
    out = []
    for x in (c.k, c.v):
        codes, s, z = O4.quantise(x.double().numpy(), BITS[c.dtype])
        out.append((O4.pack(codes), s, z, O4.values(codes, s, z)))
    four = np.stack([out[0][1], out[0][2], out[1][1], out[1][2]], -1)
    scale = torch.from_numpy(np.ascontiguousarray(np.swapaxes(four, 2, 3))).to(c.dtype)
    return torch.from_numpy(out[0][0]), torch.from_numpy(out[1][0]), scale, out[0][3], out[1][3]


def steps(c, pool4, scale, which):
    """What the error bounds of attention are made of, per token and head of one layer's pool of values: the scale s and
    the middle z + 8 s of each vector, as arrays like the pool without its last dimension."""
    four = np.swapaxes(scale.double().numpy(), 2, 3)
    s, z = four[..., 2 * which], four[..., 2 * which + 1]
    return s, z + 8 * s


def attend_bound(dtype, out, k_abs, q_k, floor_k, floor_v, mean_v, steps_v, D, tokens, few):
    """|error| of an attention output over values of 4 bits; all terms are sums over what a row sees.

    few rows: codes n are exact, a score is s (q . n) + z sum q in float32 (k_abs: the largest scale * sum |q| (15 s + |z|)),
    D + 16 roundings 2^-23 of it; the weights times the values' scales are rounded to f16's 11 bits, half a step 2^-11 of
    sum p 15 s (steps_v), those 2^-29 below the largest to its least step (2^-39 of the largest each); products of up to
    sum p 15 s + |z| are summed in float32.
    more rows: keys and values are rounded to f16's 11 bits, half a step 2^-11 of |k| (q_k: the largest scale * sum |q| |k|)
    and of |v| (mean_v), and to 2^-25 of the largest element of a tile of 128 tokens (floor_k: the same sum with the largest element of
    all; floor_v: that of the values), D + 8 roundings of the products; the weights, times a power of two, to 2^-11.
    Both: an error e in the scores is a factor exp(2 e) between weights; sums over the tokens and the exponential
    cost (tokens + 16) 2^-23; then one rounding to dtype."""
    h = kv_cases.half_step(dtype)
    if few:
        delta = np.expm1(2 * (D + 16) * 2.0 ** -23 * k_abs[..., None]) + (tokens + 32) * 2.0 ** -23
        before = delta * mean_v + 2.0 ** -11 * (1 + delta) * steps_v + (tokens + 16) * 2.0 ** -23 * (steps_v + mean_v)
    else:
        delta = np.expm1(2 * (2.0 ** -11 * q_k + 2.0 ** -25 * floor_k + (D + 8) * 2.0 ** -23 * k_abs)[..., None])
        delta = delta + 2.0 ** -11 + (tokens + 16) * 2.0 ** -23
        before = delta * (1 + 2.0 ** -11) * mean_v + 2.0 ** -11 * mean_v + 2.0 ** -24 * floor_v
    return before + h * (np.abs(out) + before) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133)
