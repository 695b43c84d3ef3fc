"""4-bit decode attention where rows of very different size meet in one output:
a row with a loud channel must not cost the dims in which it holds little, and
many small weights must add up beside a large one, at long contexts too."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_11_b200 as csa
from _serving import check, decode_bound, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def attend(q, cache, table, n, scale, g, loud=()):
    """The call, its 64-bit value from the rows fetched back, and its bound: each
    weight to 2^-11 of itself and to 2^-28 of the head's largest (in place of
    decode_bound's term of the weights times the rows' sizes)."""
    pos = torch.tensor([n - 1], device=DEV)
    out = csa.csa_kv4_decode_attn(q, cache, table, pos, scale)
    csa.csa_check()
    k, v = (x[0].double() for x in csa.csa_kv4_fetch(cache, table, pos - (n - 1), n, dtype=torch.float32))
    kk, vv = (x.repeat_interleave(g, 1).transpose(0, 1) for x in (k, v))
    l = torch.einsum("hd,hud->hu", q[0].double(), kk) * scale
    p = torch.softmax(l, 1)
    ref, spread = (torch.einsum("hu,hud->hd", p, x) for x in (vv, vv.abs()))
    reach = torch.einsum("hd,hud->hu", q[0].double().abs(), kk.abs()).amax(1, keepdim=True)
    far = q[0].double().abs().amax(1, keepdim=True) * kk.abs().sum(2).amax(1, keepdim=True)
    least = 2.0 ** -28 * p.amax(1, keepdim=True) * vv.abs().sum(1)
    bound = decode_bound(*[f64(x) for x in (ref, spread, reach, far)], 0.0, scale, q.shape[-1], n)
    check(out[0], f64(ref), bound + (1 + 2.0 ** -8) * f64(least), "decode")
    return p, out


def stored(k, v, P):
    n, nkv, c = k.shape[1:]
    nb = -(-n // P)
    cache = csa.csa_kv4_cache(nb, nkv, c, P)
    table = torch.randperm(nb, generator=torch.Generator().manual_seed(n)).to(torch.int32)[None].to(DEV)
    csa.csa_kv4_store(cache, table, torch.zeros(1, dtype=torch.int64, device=DEV), k, v)
    return cache, table


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("c,g,n,loud,quiet", [
    (128, 8, 1000, 1e3, 1e-2), (64, 4, 1000, 1e3, 1e-2), (128, 16, 900, 1e6, 1e-2), (64, 16, 3000, 1e6, 1.0),
    (128, 1, 1000, 1e12, 1e-3), (128, 8, 1000, 1e20, 1e-2), (64, 8, 20, 1e9, 1.0), (128, 4, 30000, 1e4, 1e-2),
    (64, 5, 300, 1e-30, 1e-37), (128, 8, 500, 1e37, 1e20),
])
def test_loud_channel(c, g, n, loud, quiet, at):
    """One row with half of the weight and one loud channel, zeros elsewhere;
    the others, of some 1 / n each, make up every other dim alone."""
    gen = torch.Generator().manual_seed(n + c)
    q = torch.randn((1, g, c), generator=gen)
    q[:, 1:] = q[:, :1] + 0.05 * q[:, 1:]          # heads that agree on the loud row
    u = {"first": 0, "middle": n // 2 + 3, "last": n - 1}[at]
    k = 0.02 * torch.randn((1, n, 1, c), generator=gen)
    k[0, u, 0] = q[0, 0] * (np.log(n) / float(q[0, 0].pow(2).sum()))
    v = quiet * (1 + torch.rand((1, n, 1, c), generator=gen))
    v[0, u] = 0
    v[0, u, 0, 21] = loud
    cache, table = stored(k.bfloat16().to(DEV), v.bfloat16().to(DEV), 32)
    p, out = attend(q.bfloat16().to(DEV), cache, table, n, 1.0, g)
    assert 0.3 < float(p[0, u]) < 0.7
    if abs(np.log10(quiet)) < 30:      # (beside it the quiet dims are what they are)
        other = f64(out[0])[:, np.arange(c) != 21]
        assert (other > 0.3 * quiet).all() and (other < 2.1 * quiet).all()


def test_rows_of_every_size_in_their_own_dims():
    """Each row holds one dim, its size 2^-40 to 2^40 times its neighbours', all
    weights alike: every dim is one row's value over n."""
    c = n = 128
    gen = torch.Generator().manual_seed(5)
    size = torch.exp2(torch.randint(-40, 41, (n,), generator=gen).float())
    v = torch.diag(size)[None, :, None]
    k = torch.zeros((1, n, 1, c))
    cache, table = stored(k.bfloat16().to(DEV), v.bfloat16().to(DEV), 16)
    q = torch.randn((1, 8, c), generator=gen).bfloat16().to(DEV)
    _, out = attend(q, cache, table, n, 0.3, 8)
    fetched = csa.csa_kv4_fetch(cache, table, torch.zeros(1, dtype=torch.int64, device=DEV), n, dtype=torch.float32)[1]
    want = fetched[0, :, 0].diagonal().double() / n
    # the output's rounding, and 2^-11 of each weight and its sum
    assert bool(((out[0].double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -10)).all())


@pytest.mark.parametrize("c,g,n", [(64, 8, 200_000), (128, 4, 120_001)])
def test_long_context_beside_a_first_token(c, g, n):
    """The first token takes half of the weight, with a value near zero; the
    others' weights, 1 / n of it, make up the output."""
    gen = torch.Generator(device=DEV).manual_seed(n)
    q = torch.randn((1, g, c), generator=gen, device=DEV)
    q[:, 1:] = q[:, :1]
    k = 0.01 * torch.randn((1, n, 1, c), generator=gen, device=DEV)
    k[0, 0, 0] = q[0, 0] * (np.log(n) / float(q[0, 0].pow(2).sum()))
    v = 1 + 0.5 * torch.randn((1, n, 1, c), generator=gen, device=DEV)
    v[0, 0] *= 1e-3
    cache, table = stored(k.bfloat16(), v.bfloat16(), 256)
    p, _ = attend(q.bfloat16(), cache, table, n, 1.0, g)
    assert float(p[0, 0]) > 0.2
