"""csa_window_attn against its 64-bit definition: separate keys and values on
the tensor cores, and shared rows."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_11_b200 as csa
import oracle as O
from _serving import S, attn_bound, check, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(B, nq, nk, nh, nkv, c, seed, packed=False):
    g = torch.Generator().manual_seed(seed)
    if packed:      # q, k and v are views of one projection's output
        qkv = torch.randn((B, nk, (nh + 2 * nkv) * c), generator=g).bfloat16()
        q, k, v = qkv.to(DEV).split([nh * c, nkv * c, nkv * c], -1)
        return q.unflatten(-1, (nh, c)), k.unflatten(-1, (nkv, c)), v.unflatten(-1, (nkv, c))
    return [torch.randn((B, n, h, c), generator=g).bfloat16().to(DEV)
            for n, h in ((nq, nh), (nk, nkv), (nk, nkv))]


def some_rows(nq, group, limit=60):
    """Queries at both ends, around the edges of query tiles, and some between."""
    tt = 128 // group
    r = {0, 1, nq - 1, nq - 2, nq // 2, nq // 3}
    for e in (tt, 2 * tt, 4 * tt):
        r |= {e - 1, e, e + 1}
    r |= set(np.random.default_rng(nq).integers(0, nq, 20).tolist())
    return sorted(x for x in r if 0 <= x < nq)[:limit]


def compare(out, q, k, v, W, first, z, scale, rows, dt=torch.bfloat16):
    for b in range(q.shape[0]):
        ref, spread, reach = S.window_attn(f64(q[b]), f64(k[b]), f64(v[b]), W, first,
                                           None if z is None else f64(z), scale, rows)
        check(out[b, rows], ref, attn_bound(ref, spread, reach, scale, q.shape[-1], k.shape[1], dt), f"b={b}")


@pytest.mark.parametrize("B,nq,nk,nh,nkv,c,W,first,sink,packed", [
    (1, 1, 1, 1, 1, 128, 1, 0, False, False),
    (2, 5, 5, 8, 2, 64, 3, 1, True, False),
    (1, 333, 333, 8, 2, 64, 100, 3, False, True),
    (2, 400, 400, 4, 4, 128, 128, 4, True, False),        # g = 1: 128 tokens a tile
    (1, 700, 700, 2, 2, 128, 37, 0, False, False),         # query tiles that skip key tiles
    (1, 300, 300, 6, 2, 128, 64, 9, True, False),          # g = 3: 126 of 128 rows
    (1, 260, 260, 40, 1, 64, 70, 20, False, True),         # g = 40: 3 tokens a tile
    (1, 50, 50, 128, 1, 64, 20, 2, False, False),          # one token a tile
    (1, 90, 90, 100, 1, 128, 33, 1, True, False),
    (1, 900, 900, 8, 1, 128, 900, 0, False, False),        # plain causal
    (1, 900, 900, 8, 1, 64, 5000, 7, False, False),
    (1, 1500, 1500, 8, 2, 128, 200, 300, True, False),     # many first tokens
    (1, 1500, 1500, 8, 2, 64, 200, 128, False, False),     # a whole tile of them
    (1, 1500, 1500, 4, 1, 128, 200, 260, False, True),     # two tiles and 8 rows more (4 of them padding)
    (1, 800, 800, 4, 1, 64, 130, 700, False, False),       # they reach past most windows
    (2, 100, 777, 8, 2, 128, 256, 4, True, False),         # a chunk at the end of a prompt
    (1, 1, 777, 8, 2, 128, 256, 4, False, False),
    (3, 129, 640, 5, 5, 64, 1, 1, False, False),           # each sees itself and the first
])
def test_matches_definition(B, nq, nk, nh, nkv, c, W, first, sink, packed):
    q, k, v = make(B, nq, nk, nh, nkv, c, nq + W, packed)
    z = torch.randn(nh, generator=torch.Generator().manual_seed(1)).to(DEV) if sink else None
    scale = c ** -0.5
    out = csa.csa_window_attn(q, k, v, W, first, z, scale)
    csa.csa_check()
    compare(out, q, k, v, W, first, z, scale, some_rows(nq, nh // nkv))


@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_scales(scale):
    q, k, v = make(1, 300, 300, 4, 1, 128, 5)
    out = csa.csa_window_attn(q, k, v, 150, 4, None, scale)
    compare(out, q, k, v, 150, 4, None, scale, some_rows(300, 4))


def test_growing_logits_rescale():
    """Keys that grow along the sequence move every row's maximum again and again."""
    q, k, v = make(1, 600, 600, 4, 1, 128, 6)
    k = (k.float() * torch.linspace(0.05, 6, 600, device=DEV)[None, :, None, None]).bfloat16()
    out = csa.csa_window_attn(q, k, v, 600, 0, None, 0.2)
    compare(out, q, k, v, 600, 0, None, 0.2, some_rows(600, 4))


def test_hidden_infinities_do_not_leak():
    """NaN and infinite keys and values where the mask hides them: behind the
    last token of a padded batch, and before the window."""
    q, k, v = make(1, 400, 400, 8, 2, 128, 7)
    clean = csa.csa_window_attn(q, k, v, 64, 4, None, 0.1)
    k2, v2 = k.clone(), v.clone()
    k2[:, 300:], v2[:, 300:] = float("nan"), float("inf")      # 300 valid tokens
    v2[:, 50, 0, 9] = float("nan")
    k2[:, 51] = -float("inf")
    out = csa.csa_window_attn(q, k2, v2, 64, 4, None, 0.1)
    ok = [t for t in range(300) if t < 50 or t >= 51 + 64]
    compare(out, q, k, v, 64, 4, None, 0.1, ok[::7])
    # rows whose tiles hold nothing but finite values keep their bits (the
    # heads of key/value head 1); the others, computed key by key, are finite
    assert np.isfinite(f64(out[:, ok])).all()
    assert torch.equal(out[:, :40, 4:], clean[:, :40, 4:])
    # where they are seen they show, and only in the dim and head that holds them
    assert np.isnan(f64(out[0, 60])).any()
    o = csa.csa_window_attn(q, k, torch.where(torch.arange(400, device=DEV)[None, :, None, None] == 50,
                                              v2, v), 64, 4, None, 0.1)
    bad = ~np.isfinite(f64(o[0]))
    assert bad[50:114, :4, 9].all() and bad.sum() == 64 * 4


def test_shared_rows_on_the_tensor_cores():
    g = torch.Generator().manual_seed(8)
    for n, W, first, sink in ((1, 128, 4, True), (300, 128, 4, True), (260, 128, 0, False), (200, 30, 150, True)):
        q = torch.randn((1, n, 64, 512), generator=g).bfloat16().to(DEV)
        kv = torch.randn((1, n, 512), generator=g).bfloat16().to(DEV)
        z = torch.randn(64, generator=g).to(DEV) if sink else None
        out = csa.csa_window_attn(q, kv, None, W, first, z, 512 ** -0.5)
        compare(out, q, kv[:, :, None], kv[:, :, None], W, first, z, 512 ** -0.5, some_rows(n, 64, 16))
    csa.csa_check()


@pytest.mark.parametrize("dt,nh,c,W,first", [(torch.float32, 3, 64, 20, 2), (torch.float32, 9, 128, 500, 0),
                                             (torch.bfloat16, 5, 96, 33, 40)])
def test_shared_rows_of_other_shapes(dt, nh, c, W, first):
    g = torch.Generator().manual_seed(9)
    q = torch.randn((2, 150, nh, c), generator=g).to(dt).to(DEV)
    kv = torch.randn((2, 150, c), generator=g).to(dt).to(DEV)
    z = torch.randn(nh, generator=g).to(DEV)
    out = csa.csa_window_attn(q, kv, None, W, first, z, 0.2)
    compare(out, q, kv[:, :, None], kv[:, :, None], W, first, z, 0.2, some_rows(150, 1), dt)


def test_shared_rows_without_first_tokens_are_hca_attn_without_entries():
    """With fewer tokens than one heavy block HCA attention is the window alone."""
    g = torch.Generator().manual_seed(10)
    q = torch.randn((1, 200, 64, 512), generator=g).bfloat16().to(DEV)
    kv = torch.randn((1, 200, 512), generator=g).bfloat16().to(DEV)
    z = torch.randn(64, generator=g).to(DEV)
    a = csa.hca_attn(q, torch.empty((1, 0, 512), dtype=torch.bfloat16, device=DEV), kv, 128, z, 0.05, 256)
    assert torch.equal(a, csa.csa_window_attn(q, kv, None, 128, 0, z, 0.05))
    ref = O.hca_attn(f64(q[0]), np.zeros((0, 512)), f64(kv[0]), 128, f64(z), 0.05, 256, rows=[0, 150])
    assert np.abs(ref - f64(a[0, [0, 150]])).max() < 2e-2


def test_chunks_equal_the_whole_prompt_and_padding_is_left_alone():
    q, k, v = make(1, 500, 500, 8, 2, 64, 11)
    whole = csa.csa_window_attn(q, k, v, 90, 5, None, 0.125)
    rows = []
    for lo, hi in ((0, 130), (130, 131), (131, 500)):
        rows.append(csa.csa_window_attn(q[:, lo:hi].contiguous(), k[:, :hi].contiguous(), v[:, :hi].contiguous(),
                                        90, 5, None, 0.125))
    got = torch.cat(rows, 1)
    # equal up to the order of the sums: other tiles
    assert (got.float() - whole.float()).abs().max() <= 2 ** -6 * whole.float().abs().max()
    # rows of `out` behind the queries stay as they were
    big = torch.full((1, 600, 8, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    csa.csa_window_attn(q, k, v, 90, 5, None, 0.125, out=big[:, :500])
    assert bool((big[:, 500:] == 7).all()) and torch.equal(big[:, :500], whole)


def test_graph_replay_streams_and_repeats():
    q, k, v = make(2, 200, 200, 8, 2, 128, 12)
    out = torch.empty_like(q)
    call = lambda: csa.csa_window_attn(q, k, v, 64, 4, None, 0.1, out=out)  # noqa: E731
    call()
    first = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    out.zero_()
    graph.replay()
    assert torch.equal(out, first)
    outs = []
    for _ in range(3):
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs.append(csa.csa_window_attn(q, k, v, 64, 4, None, 0.1))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
