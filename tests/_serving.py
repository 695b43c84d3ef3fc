"""Shared helpers of the serving operators' tests: error bounds and caches."""
import numpy as np
import torch

import oracle.serving as S

# A rounding to a type is off by at most half a step, relative to the value.
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().cpu().double().numpy()


def attn_bound(ref, spread, reach, scale, c, n, dt=torch.bfloat16):
    """Elementwise bound of an attention output.  Parts: the output's rounding;
    each weight's rounding to bf16 before the value product (one half step of
    the weight, so of the weighted |v|; none on the fp32 path); the logits'
    fp32 error d = scale * (c + 4) 2^-24 * max sum|q k| (c products summed in
    any order, the scale and the log2(e) factor), which moves weights by at
    most e^{2d} - 1 relative to their sum (2 d in the logit and as much in the
    normaliser); 2^-21 for the exponentials' approximation on both sides and
    2^-24 n for summing n weights and products in fp32."""
    d = 2 * abs(scale) * (c + 4) * 2.0 ** -24 * reach
    # logits beyond the running maximum: their difference is rounded as well
    rel = np.expm1(2 * d) + 2.0 ** -21 + 2 * (n + 16) * 2.0 ** -24
    if dt != torch.float32:
        rel = rel + 2.0 ** -8
    first = np.abs(ref) + rel * spread
    return HALF[dt] * first + rel * spread + 1e-30


def decode_bound(ref, spread, reach, far, under, scale, c, n):
    """As attn_bound for the 4-bit cache's attention: its weights are f16 (a
    half step of 2^-11), formed as 2^(logit + exponent - reference) in fp32
    from numbers up to |logit| + 512 (a rounding each of the sum and the
    difference), and query elements far below a head's largest keep 2^-25 of
    it.  A weight p r below 2^-14 of the largest is an f16 subnormal: it is off
    by up to half a subnormal step, 2^-25, in units of the reference, which is
    at most the largest p r; times |v| / r, summed over the rows, that is
    2^-25 under."""
    d = 2 * abs(scale) * ((c + 6) * 2.0 ** -24 * reach + 2.0 ** -25 * far)
    logit = 1.45 * abs(scale) * reach + 512
    rel = np.expm1(2 * d) + 2.0 ** -21 + 2 * (n + 16) * 2.0 ** -24 + 2.0 ** -11 + 2 * logit * 2.0 ** -24
    off = rel * spread + 2.0 ** -25 * under
    return 2.0 ** -8 * (np.abs(ref) + off) + off + 1e-30


def check(got, ref, bound, what=""):
    g = f64(got) if torch.is_tensor(got) else got
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    err = np.abs(g - ref)
    assert np.all(np.isfinite(g)), what
    bad = err > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} beyond the bound, worst " \
                          f"{(err / bound).max():.2f} of it"


def random_table(rng, lens, block_tokens, max_blocks, spare=2):
    """int32 table over a shuffled pool, and the pool's size."""
    need = [-(-int(n) // block_tokens) for n in lens]
    pool = sum(need) + spare
    perm = rng.permutation(pool)
    t = np.full((len(lens), max_blocks), -1, np.int32)
    i = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[i:i + n]
        i += n
    return t, pool


def filled_cache(rng, pool, nkv, c, block_tokens):
    """A numpy cache whose every image holds valid random rows."""
    cache = np.zeros((pool, nkv, block_tokens // 16, 18 * c + 32), np.uint8)
    cache[..., :16 * c] = rng.integers(1, 16, cache[..., :16 * c].shape)
    hi = rng.integers(1, 16, cache[..., :16 * c].shape).astype(np.uint8)
    cache[..., :16 * c] |= hi << 4
    cache[..., 16 * c:18 * c] = rng.integers(0, 110, cache[..., 16 * c:18 * c].shape)
    # scales up to 2^5, codes up to 7: exponents that bring rows near 1
    cache[..., 18 * c:] = rng.integers(117, 122, cache[..., 18 * c:].shape)
    return cache


__all__ = ["S", "HALF", "f64", "attn_bound", "decode_bound", "check", "random_table", "filled_cache", "np", "torch"]
