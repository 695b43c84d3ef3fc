"""Values that are not finite in window attention: seen they show, hidden they
change nothing, and neither costs the call more than a bounded time."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_11_b200 as csa
from _serving import S, attn_bound, check, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


def sees(t, u, W, first):
    return u <= t and (u > t - W or u < first)


@pytest.mark.parametrize("nq,nk,nh,nkv,c,W,first,bad", [
    (300, 300, 4, 1, 128, 64, 0, {17: INF, 130: -INF, 299: float("nan")}),
    (300, 300, 4, 1, 64, 64, 4, {2: INF, 5: float("nan"), 128: -INF}),      # a first token; one behind them
    (700, 700, 2, 2, 128, 37, 0, {100: INF, 101: -INF, 400: INF}),          # both infinities in one dim
    (520, 520, 16, 1, 64, 200, 131, {130: INF, 131: INF, 135: -INF, 300: float("nan")}),
    (260, 260, 3, 1, 128, 500, 0, {0: INF, 259: INF}),                      # every query sees the first
    (40, 40, 128, 1, 64, 9, 2, {20: -INF, 1: INF}),                         # a token a query tile
    (100, 640, 8, 2, 128, 256, 4, {400: INF, 500: float("nan"), 639: -INF}),
    (1, 777, 8, 2, 64, 256, 4, {500: INF, 776: -INF, 9: float("nan")}),
])
def test_shown_and_hidden(nq, nk, nh, nkv, c, W, first, bad):
    g = torch.Generator().manual_seed(nk + c)
    q, k, v = (torch.randn((1, n, h, c), generator=g).bfloat16() for n, h in ((nq, nh), (nk, nkv), (nk, nkv)))
    scale, z = c ** -0.5, torch.randn(nh, generator=g)
    dims = {u: (7 * i) % c if i < 2 else c - 1 - i for i, u in enumerate(sorted(bad))}
    if len(bad) == 3 and nq == 700:
        dims = {u: 3 for u in bad}
    v2 = v.clone()
    for u, x in bad.items():
        v2[0, u, nkv - 1, dims[u]] = x
    out = csa.csa_window_attn(q.to(DEV), k.to(DEV), v2.to(DEV), W, first, z.to(DEV), scale)
    csa.csa_check()
    got = f64(out[0])
    # every row against the clean values, except where a bad one is seen
    ref, spread, reach = S.window_attn(f64(q[0]), f64(k[0]), f64(v[0]), W, first, f64(z), scale, range(nq))
    want = ref.copy()
    for i in range(nq):
        for u, x in bad.items():
            if sees(nk - nq + i, u, W, first):
                with np.errstate(invalid="ignore"):
                    want[i, nh - nh // nkv:, dims[u]] += x
    odd = ~np.isfinite(want)
    assert odd.any() and not odd.all()
    assert np.array_equal(got[odd], want[odd], equal_nan=True)
    fine = np.where(odd, 0, got)
    check(fine, np.where(odd, 0, ref), attn_bound(ref, spread, reach, scale, c, nk), "rows that see none of them")


def test_finite_rows_keep_their_bits_where_no_tile_holds_one():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((1, 1200, h, 128), generator=g).bfloat16().to(DEV) for h in (8, 2, 2))
    clean = csa.csa_window_attn(q, k, v, 100, 0, None, 0.1)
    v[0, 900:, :, 5] = INF
    out = csa.csa_window_attn(q, k, v, 100, 0, None, 0.1)
    assert torch.equal(out[:, :768], clean[:, :768]) and torch.equal(out[..., :5], clean[..., :5])


def timed(call, reps):
    for _ in range(2):
        call()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(reps):
        call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / reps


def test_a_seen_infinity_costs_nothing_and_a_padded_batch_little():
    """One infinite value that all 16384 queries see: the same products as
    without it (recomputing its rows key by key would be 5 10^8 keys).  Padding of
    NaN behind the tokens: some 100 edge tiles, not every padded query's window."""
    g = torch.Generator(device=DEV).manual_seed(4)
    q, k, v = (torch.randn((1, 16384, h, 128), generator=g, device=DEV).bfloat16() for h in (8, 2, 2))
    call = lambda x: (lambda: csa.csa_window_attn(q, k, x, 16384, 0, None, 0.1))  # noqa: E731
    base = timed(call(v), 5)
    seen = v.clone()
    seen[0, 3, 0, 9] = INF
    assert timed(call(seen), 5) < 2 * base + 1
    out = csa.csa_window_attn(q, k, seen, 16384, 0, None, 0.1)
    assert bool(torch.isinf(out[0, 3:, :4, 9]).all()) and bool(torch.isfinite(out[0, :3]).all())
    padded = v.clone()
    padded[0, 12000:] = float("nan")
    assert timed(call(padded), 5) < 4 * base + 5
    csa.csa_check()


def test_many_first_tokens():
    """An infinite value among 12000 first tokens, seen by every later query: no
    tile of theirs hides a key, so the call takes what it takes without."""
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (torch.randn((1, 16384, h, 64), generator=g, device=DEV).bfloat16() for h in (8, 2, 2))
    call = lambda x: (lambda: csa.csa_window_attn(q, k, x, 128, 12000, None, 0.1))  # noqa: E731
    base = timed(call(v), 5)
    seen = v.clone()
    seen[0, 300, 1, 9] = INF
    assert timed(call(seen), 5) < 2 * base + 1
    out, clean = call(seen)(), call(v)()
    assert bool(torch.isinf(out[0, 300:, 4:, 9]).all()) and torch.equal(out[..., :9], clean[..., :9])
    assert torch.equal(out[0, :, :4], clean[0, :, :4]) and torch.equal(out[0, :256], clean[0, :256])
    csa.csa_check()
