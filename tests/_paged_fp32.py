"""Inputs on which an fp32 output shows every part of the softmax weights, and
the bound that it has to meet there.

The queries and keys are zero but for their first elements, so that a score is
one exact product.  Token t's value row is a unit vector, element t % 128 (zero
where that is not below d), so that an element of the output is one token's
probability, or the sum of one a tile of 128.  With s the scores in base 2,
|s| <= 1:
  s          scaling by a rounded factor and the product's rounding: 2^-23;
  s - m      |s - m| <= 2, one rounding: 2^-23; so a weight's exponent is off by
             3 * 2^-23 and the weight by 2.1 * 2^-23 of itself, plus 2^-22 of
             the exponential (its documented bound): W = 2.1 * 2^-23 + 2^-22;
  weights    enter the second product in three parts of 8 bits: 2^-24;
  output     a tile adds three parts: 3 * 2^-24 a tile;
  sum        W, and 8 + tiles additions: 2^-24 each;
  joining    (rows that may be cut: of more than one unit of the split, 64
             tokens where there are few, else 128) two levels, each with an
             exponential (W) and two roundings, in the numerator and the
             denominator alike, over at most 8 + tiles states;
  quotient   2 units in the last place: 2^-22, and 2^-24 for the result.
Two parts instead of three would leave up to 2^-16 of each weight.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from tests import _paged as P


def inputs(seed, lens, hkv, G, d, page):
    c = P.random_cache(seed, lens, hkv, d, page, weights=False)
    g = torch.Generator().manual_seed(seed + 1)
    b = c["lens"].shape[0]
    q = torch.zeros(b, hkv * G, d)
    top = math.sqrt(d) / 1.4426950408889634 / 1.02      # |q k| log2(e) / sqrt(d) stays below 1
    q[:, :, 0] = top * (0.5 + 0.5 * torch.rand(b, hkv * G, generator=g))
    for x in range(b):
        for h in range(hkv):
            t = torch.arange(int(c["lens"][x, h]))
            p, r = c["table"][x, h].long()[t // page], t % page
            k, v = torch.zeros(len(t), d), torch.zeros(len(t), d)
            k[:, 0] = 2 * torch.rand(len(t), generator=g) - 1
            v[t[t % 128 < d], t[t % 128 < d] % 128] = 1
            c["k"][p, r], c["v"][p, r] = k.bfloat16(), v.bfloat16()
    return c, q.bfloat16()


def bound(n, unit):
    """Relative bound of an element of the output of a row of n tokens, split
    in units of `unit` tokens."""
    tiles = -(-n // 128)
    u = 2.0 ** -24
    W = 4.2 * u + 4 * u
    join = 2 * (2 * (W + 2 * u)) + (8 + tiles) * u if n > unit else 0
    return 2 * W + u + tiles * 3 * u + (8 + tiles) * u + join + 4 * u + u


def bf16(x):
    return torch.as_tensor(x, dtype=torch.float32).bfloat16().double().numpy()


def expected(c, q, parts=None):
    """The outputs, in 64 bits; with `parts`, their weights cut to so many parts
    of bf16 (relative to the row's largest)."""
    b, hq, d = q.shape
    G = hq // c["lens"].shape[1]
    o = np.zeros((b, hq, d))
    for x in range(b):
        for h in range(hq):
            n = int(c["lens"][x, h // G])
            t = np.arange(n)
            if not n:
                continue
            p, r = c["table"][x, h // G].numpy()[t // c["page"]], t % c["page"]
            s = P.f64(c["k"])[p, r, 0] * float(q[x, h, 0]) / math.sqrt(d)
            w = np.exp(s - s.max())
            total = w.sum()
            if parts:
                left, cut = np.float32(w).astype(np.float64), 0.0
                for _ in range(parts):
                    part = bf16(left)
                    cut, left = cut + part, left - part
                w = cut
            own = t % 128 < d
            np.add.at(o[x, h], t[own] % 128, (w / total)[own])
    return o


def check(c, q, out, unit=64):
    """The largest error of each row, over its bound; [batch, num_kv_heads]."""
    want = expected(c, q)
    G = q.shape[1] // c["lens"].shape[1]
    got = P.f64(out) if isinstance(out, torch.Tensor) else out
    over = np.zeros(tuple(c["lens"].shape))
    for x in range(over.shape[0]):
        for h in range(over.shape[1]):
            n = int(c["lens"][x, h])
            a, e = got[x, h * G:(h + 1) * G], want[x, h * G:(h + 1) * G]
            err = np.abs(a - e) / np.where(e == 0, 1, e)
            over[x, h] = err.max() / bound(max(n, 1), unit)
    return over
