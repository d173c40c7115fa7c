"""Inputs of the attention whose right answer is known and whose wrong ones are far away, with tolerances from arithmetic.

Two slots, V = 0 and V = 1, logits 0 and l < 0: out = p / (1 + p), p = e^l, in every element.  With u = 2^-24, relative to out:
  l in units of log2: the scale's rounding and the product's, 2 u |l| ln 2 <= 5.5 u for |l| <= 4; ex2.approx 4 u (2^-22);
  p in three bf16 parts 0.5 u, their sum in the tensor core at most 2 u a part (6 u); 1 + p, the quotient: 2 u.
Together 18 u; the bound is 24 u.  In two parts p alone is off by up to 2^-18 = 64 u.

Long runs, all logits 0 (p = 1): a chunk of 16 slots holds 15 values of 1 and one of 15 * 2^-15, whose sum is exact.  Over a run
of r chunks the output is a sum of r such chunks in fp32; near r = 500 it ends in [4096, 8192), where a step is 2^-11: a
truncated addition loses 15/16 of a step there, a rounded one gains 1/16.  `drift` adds them up.  The joins: 8 parts in a CTA,
then the CTAs' parts (up to 160) over 8 or 16 threads of 20 or 10 each, the threads, and a quotient: 37 u at most.
"""
import numpy as np

U = 2.0 ** -24
TWO_SLOTS = 24 * U
JOINS = 37 * U
RUN = 500
SMALL = 15 * 2.0 ** -15
CHUNK = np.array([1.0] * 15 + [SMALL])


def drift(chunks, truncate=False):
    """Relative error of `chunks` chunk sums added one after another in fp32."""
    s = np.float32(0)
    c = np.float64(CHUNK.sum())
    for _ in range(chunks):
        exact = np.float64(s) + c
        s = np.float32(exact)
        if truncate and np.float64(s) > exact:
            s = np.nextafter(s, np.float32(0))
    return float(s) / (c * chunks) - 1


def parts(p, count):
    """p (64 bits) as the sum of `count` bf16 parts of its fp32 value."""
    import torch
    rest, total = torch.from_numpy(p.astype(np.float32)), torch.zeros(p.shape, dtype=torch.float64)
    for _ in range(count):
        h = rest.to(torch.bfloat16).float()
        rest = rest - h
        total += h.double()
    return total.numpy()
