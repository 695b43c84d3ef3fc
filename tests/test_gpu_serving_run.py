"""The serving operators together: a prompt through head norms, rotation and
window attention into the 4-bit cache, a fork, decode steps (also as a
captured graph), a freed sequence and a compacted pool.  Each stage is held
to its 64-bit definition on the values that it was given."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_11_b200 as csa
from _serving import S, attn_bound, check, decode_bound, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("c,P,W,first", [(64, 16, 40, 4), (128, 32, 0, 0)])
def test_prompt_fork_decode_free_compact(c, P, W, first):
    nh, nkv, rows, mb, pool = 8, 2, 4, 12, 30
    scale, g = c ** -0.5, torch.Generator().manual_seed(c)
    rnd = lambda *s: torch.randn(s, generator=g).bfloat16().to(DEV)  # noqa: E731
    qg, kg = (1 + 0.1 * torch.randn((h, c), generator=g).to(DEV) for h in (nh, nkv))
    z = torch.randn(nh, generator=g).to(DEV)
    lens = [101, 64]
    n = max(lens)
    cache = csa.csa_kv4_cache(pool, nkv, c, P)
    table = torch.full((rows, mb), -1, dtype=torch.int32, device=DEV)
    free = list(np.random.default_rng(1).permutation(pool))
    for b in range(2):
        need = -(-(lens[b] + 8) // P)
        table[b, :need] = i32([free.pop() for _ in range(need)])

    # ---- prompt (padded batch of two) ----
    qkv = rnd(2, n, (nh + 2 * nkv) * c)
    q, k, v = qkv.split([nh * c, nkv * c, nkv * c], -1)
    q, k, v = q.unflatten(-1, (nh, c)), k.unflatten(-1, (nkv, c)), v.unflatten(-1, (nkv, c))
    v[1, lens[1]:] = float("nan")                                     # padding holds anything
    raw = f64(q), f64(k)
    pos = torch.arange(n, device=DEV).repeat(2, 1)
    q, k = csa.csa_qk_norm_rope(q, k, pos, qg, kg, rope_dims=c // 2, q_out=q, k_out=k)
    for got, x, w in ((q, raw[0], qg), (k, raw[1], kg)):
        ref = S.qk_norm_rope(x.reshape(2 * n, -1, c), f64(w), f64(pos).reshape(1, -1), [c // 4], c // 2, False)
        check(got, ref.reshape(got.shape), 2.0 ** -7 * np.abs(ref).max(-1, keepdims=True).reshape(*got.shape[:-1], 1))
    out = csa.csa_window_attn(q, k, v, W or n, first, z, scale)
    for b in range(2):
        some = [0, 3, lens[b] // 2, lens[b] - 1]
        ref, spread, reach = S.window_attn(f64(q[b, :lens[b]]), f64(k[b, :lens[b]]), f64(v[b, :lens[b]]), W or n, first,
                                           f64(z), scale, some)
        check(out[b, some], ref, attn_bound(ref, spread, reach, scale, c, n), "prompt")
    start = torch.zeros(rows, dtype=torch.int64, device=DEV)
    count = i32(lens + [0, 0])
    pad = lambda x: torch.cat([x, torch.zeros_like(x)])  # noqa: E731
    csa.csa_kv4_store(cache, table, start, pad(k), pad(v), count)

    # ---- sequence 0 forks to row 2 ----
    table, cs, cd = csa.csa_blocks_fork(table, i32([0]), i32([2]), torch.tensor([lens[0]], device=DEV),
                                        i32([int(free.pop())]), P)
    csa.csa_blocks_copy([cache], cs, cd)
    spare = [int(free.pop()) for _ in range(2)]
    used = int((table[2] >= 0).sum())
    table[2, used:used + 1] = i32(spare[:1])                          # room for the fork's next tokens
    at = torch.tensor([lens[0], lens[1], lens[0], -1], device=DEV)

    # ---- decode steps, captured once and replayed ----
    x = rnd(rows, 1, (nh + 2 * nkv) * c)
    x[2] = x[0]                                                       # the fork decodes the same token first
    o = torch.empty((rows, nh, c), dtype=torch.bfloat16, device=DEV)
    qo, ko = (torch.empty((rows, 1, h, c), dtype=torch.bfloat16, device=DEV) for h in (nh, nkv))
    ws = torch.empty(csa.csa_kv4_decode_workspace(nh, nkv, c), dtype=torch.uint8, device=DEV)

    def step():
        a, b, d = x.split([nh * c, nkv * c, nkv * c], -1)
        csa.csa_qk_norm_rope(a.unflatten(-1, (nh, c)), b.unflatten(-1, (nkv, c)), at, qg, kg, rope_dims=c // 2,
                             q_out=qo, k_out=ko)
        csa.csa_kv4_store(cache, table, at, ko, d.unflatten(-1, (nkv, c)))
        csa.csa_kv4_decode_attn(qo[:, 0], cache, table, at, scale, W, first, z, ws=ws, out=o)

    def held(what):
        ref, spread, reach, far, under = S.kv4_decode(f64(qo[:, 0]), cache.cpu().numpy(), table.cpu().numpy(), at.tolist(),
                                               scale, W, first, f64(z))
        check(o, ref, decode_bound(ref, spread, reach, far, under, scale, c, n + 8), what)

    step()
    held("first step")
    assert torch.equal(o[0], o[2]) and torch.count_nonzero(o[3]) == 0
    before = cache.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph.replay()                                                    # the same tokens: the same bytes
    assert torch.equal(cache, before)
    for t in range(3):
        x.copy_(rnd(*x.shape))
        at.add_(torch.tensor([1, 1, 1, 0], device=DEV))
        graph.replay()
        held(f"step {t}")
    assert not torch.equal(o[0], o[2])

    # ---- sequence 0 ends: the fork keeps the shared blocks ----
    new, freed, nfreed = csa.csa_blocks_free(table, i32([0]), pool)
    ref = S.blocks_free(table.cpu().numpy(), [0], pool)
    assert np.array_equal(new.cpu().numpy(), ref[0]) and int(nfreed) == ref[2] > 0
    last = o.clone()
    packed, cs, cd, counts = csa.csa_blocks_compact(new, pool)
    csa.csa_blocks_copy([cache], cs, cd, counts)
    assert int(packed.max()) == int(counts[1]) - 1
    table.copy_(packed)
    at[0] = -1
    again = csa.csa_kv4_decode_attn(qo[:, 0].contiguous(), cache, table, at, scale, W, first, z)
    assert torch.equal(again[1:3], last[1:3]) and torch.count_nonzero(again[0]) == 0
    csa.csa_check()


def test_views_that_are_no_token_views_are_refused():
    x = torch.zeros((2, 6, 4, 64), dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros((2, 6), dtype=torch.int64, device=DEV)
    for bad in (x.transpose(1, 2), x[..., ::2], x[:, :3].expand(2, 3, 4, 64)[:, ::2], x[:, :5]):
        with pytest.raises(ValueError):
            csa.csa_qk_norm_rope(bad, None, pos[:, :bad.shape[1]].contiguous(), rope_dims=bad.shape[-1])
    with pytest.raises(csa.CsaError):      # a token stride of 65 elements is no whole 16-byte unit
        y = torch.zeros((6, 65), dtype=torch.bfloat16, device=DEV)[:, :64].unflatten(1, (1, 64))
        csa.csa_qk_norm_rope(y, None, pos[0])
    with pytest.raises(ValueError):
        csa.csa_qk_norm_rope(x, None, pos[:, :5].contiguous())
    with pytest.raises(ValueError):
        csa.csa_qk_norm_rope(x, None, pos.int())
    # one sequence of a batch, and every second token, are token views
    csa.csa_qk_norm_rope(x[1], None, pos[1].contiguous())
    csa.csa_qk_norm_rope(x[0, ::2], None, pos[0, ::2].contiguous())
