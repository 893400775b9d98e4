"""Bounds in norm for the dense products on random data of one size.  Elementwise worst cases grow
with K and hide a lost column of a long row; these do not.

Rounded operands: the error of h (dg, du), at most r = eps / 2 of each value, adds up over K as the
products themselves do, so it is at most r of the output's norm, and the output's own rounding
another r; with a third for sizes too few for a norm.  A lost column of K is sqrt(1 / K).

Float outputs: the tensor core adds 32 products a step (16 bits: 16).  What a step drops is
at most 2^-22 of the sum so far and of the step's products (a step's result and the
alignment of its terms, truncated).  Sums of random terms grow with the root, so with
n = K / step steps the sums add up to 2/3 n of the output and the products to at most n * step /
sqrt(K) of it; all dropped the same way that is the bound."""
import math

import torch


def rounded(dtype):
    return 3 * torch.finfo(dtype).eps / 2


def summed(cols, step=32):
    n = cols / step
    return 2.0 ** -22 * n * (2 / 3 + step / math.sqrt(cols))


def check(got, want, limit, what=""):
    err = float((got.double() - want).norm() / want.norm())
    assert err <= limit, (what, err, limit)
    return err
