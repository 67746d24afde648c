"""Plain fp64 CPU oracle of the many-tensor operators: the AdamW step, its
8-bit moments and the global gradient norm with clipping.

TEST INFRASTRUCTURE ONLY, like dimuon_oracle: numpy float64 throughout, no
code shared with the CUDA library.  Rounding happens only where the step
stores a weight, an 8-bit moment or a clipped gradient.  The 8-bit codes are
found from the formats' definitions (a search in the table of all values of the format),
not from bit patterns of fp32 numbers.

moments_f32 alone works in float32: the library defines the new moments as
fp32 products and sums rounded one by one, and the stochastic rounding
compares their bits with its noise, so codes can be compared exactly only
from them.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np

from .dimuon_oracle import f32, store_round

BLOCK = 128


@dataclass
class AdamWParams:
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01


@dataclass
class AdamWResult:
    W: np.ndarray    # before storage rounding
    m: np.ndarray
    v: np.ndarray
    update: np.ndarray  # lr mhat / (sqrt(vhat) + eps)


def adamw_step(W, G, m, v, hp: AdamWParams, t: int, *, grad_scale=1.0, lr_mult=1.0,
               decay_mult=1.0) -> AdamWResult:
    """One step in float64 from float64 arrays; scalars pass through float32."""
    b1, b2, eps = f32(hp.beta1), f32(hp.beta2), f32(hp.eps)
    lr = f32(hp.lr) * f32(lr_mult)
    wd = f32(hp.weight_decay) * f32(decay_mult)
    g = np.asarray(G, np.float64) * f32(grad_scale)
    m1 = b1 * np.asarray(m, np.float64) + (1.0 - b1) * g
    v1 = b2 * np.asarray(v, np.float64) + (1.0 - b2) * g * g
    upd = lr * (m1 / (1.0 - b1 ** t)) / (np.sqrt(v1 / (1.0 - b2 ** t)) + eps)
    W = np.asarray(W, np.float64)
    return AdamWResult(W - lr * wd * W - upd, m1, v1, upd)


def moments_f32(G, m, v, hp: AdamWParams, grad_scale=1.0):
    """(m', v') with every product and sum rounded to float32."""
    F = np.float32
    b1, b2 = F(hp.beta1), F(hp.beta2)
    c1, c2 = F(1.0 - float(b1)), F(1.0 - float(b2))
    g = np.asarray(G, F) * F(grad_scale)
    with np.errstate(over="ignore", invalid="ignore"):
        return (np.asarray(m, F) * b1 + g * c1).astype(F), \
               (np.asarray(v, F) * b2 + (g * g) * c2).astype(F)


# ----------------------------------------------------------------------------
# 8-bit moments
# ----------------------------------------------------------------------------
def format_values(mantissa, bias, count):
    """Values of the codes 0 .. count - 1 of a float format: subnormals, then
    (1 + f / 2^mantissa) 2^(e - bias)."""
    out = []
    for c in range(count):
        e, f = c >> mantissa, c & ((1 << mantissa) - 1)
        out.append(f / 2 ** mantissa * 2.0 ** (1 - bias) if e == 0
                   else (1 + f / 2 ** mantissa) * 2.0 ** (e - bias))
    return np.array(out)


E4M3 = format_values(3, 7, 127)    # 0 .. 448
E5M2 = format_values(2, 15, 124)   # 0 .. 57344


def block_scales(x, top):
    """Smallest power of two >= 2^-110 with each block's largest |x| <= top * it."""
    pad = np.zeros(-(-len(x) // BLOCK) * BLOCK)
    pad[:len(x)] = np.abs(x)
    out = []
    for a in pad.reshape(-1, BLOCK).max(1):
        k = -110
        if a > 0:
            k = max(-110, math.frexp(a / top)[1] - 1)
            while a > top * 2.0 ** k:
                k += 1
        out.append(2.0 ** k)
    return np.array(out)


def stochastic_codes(x, scales, table, u):
    """Codes of |x| / scale: the neighbour below, or the one above where the
    remainder plus u (in [0, 1)) reaches the distance between them."""
    y = np.abs(np.asarray(x, np.float64)) / np.repeat(scales, BLOCK)[:len(x)]
    lo = np.clip(np.searchsorted(table, y, side="right") - 1, 0, len(table) - 1)
    hi = np.minimum(lo + 1, len(table) - 1)
    gap = table[hi] - table[lo]
    up = np.where(gap > 0, (y - table[lo]) / np.where(gap > 0, gap, 1.0) + u >= 1.0, False)
    return np.where(up, hi, lo)


def mix(x):
    """A bijection of 32-bit words (C. Wellons, "Prospecting for Hash Functions", 2018)."""
    x = np.asarray(x, np.uint64)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x7FEB352D)) % np.uint64(2 ** 32)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x846CA68B)) % np.uint64(2 ** 32)
    return x ^ (x >> np.uint64(16))


def noise(seed, t, tensor, n, first=0):
    """(u1, u2) in [0, 1): the two moments' 16-bit noise of elements first ..
    first + n - 1 of the call's tensor number `tensor`."""
    w = 2 ** 32
    gold = 0x9E3779B9
    i = np.arange(first, first + n, dtype=np.uint64)
    key = int(mix((int(mix((seed + gold * (t % w)) % w)) + tensor) % w))
    hi = (i >> np.uint64(4)) >> np.uint64(32)
    k = mix((np.uint64(key) + hi) % np.uint64(w))
    x = mix(k ^ ((i >> np.uint64(4)) % np.uint64(w)))
    x = (x + (i % np.uint64(16)) * np.uint64(gold)) % np.uint64(w)
    x = (x * np.uint64(0x7FEB352D)) % np.uint64(w)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x846CA68B)) % np.uint64(w)
    x = x ^ (x >> np.uint64(16))
    return (x >> np.uint64(16)).astype(np.float64) / 65536, \
           (x % np.uint64(65536)).astype(np.float64) / 65536


LARGEST = 1.75 * 2.0 ** 127  # second moment that is stored


def hold(m, v):
    """v as it is stored: up to LARGEST, also an infinite one beside a finite m
    (a finite gradient whose square overflowed)."""
    return np.where((np.asarray(v) > LARGEST) & np.isfinite(m), LARGEST, v)


def pack_moments(m, v, seed, t, tensor):
    """(codes1, scales1, codes2, scales2) of the new moments; codes1 carries
    the sign in bit 7, and a positive v never gets code 0."""
    v = hold(m, v)
    u1, u2 = noise(seed, t, tensor, len(m))
    s1, s2 = block_scales(m, 448.0), block_scales(v, 57344.0)
    c1 = stochastic_codes(m, s1, E4M3, u1) + 128 * np.signbit(m)
    c2 = stochastic_codes(v, s2, E5M2, u2)
    c2 = np.where((c2 == 0) & (np.asarray(v) > 0), 1, c2)
    return c1.astype(np.uint8), s1, c2.astype(np.uint8), s2


def unpack(codes, scales, table):
    c = np.asarray(codes, np.int64)
    x = table[c & 127] * np.where(c & 128, -1.0, 1.0)
    return x * np.repeat(scales, BLOCK)[:len(c)]


# ----------------------------------------------------------------------------
# gradient norm and clipping
# ----------------------------------------------------------------------------
def grad_clip(grads, max_norm, out_dtypes=None):
    """(norm, coefficient, clipped gradients rounded to out_dtypes)."""
    norm = math.sqrt(math.fsum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads))
    c = min(1.0, max_norm / norm) if norm > 0 else 1.0
    outs = [store_round(np.asarray(g, np.float64) * c, d) if d else None
            for g, d in zip(grads, out_dtypes or [None] * len(grads))]
    return norm, c, outs
