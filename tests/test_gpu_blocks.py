"""Copied, forked, freed and compacted blocks of paged caches against plain
loops, on bare tables and on the framework's own paged cache."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_11_b200 as csa
import csa_inputs as G
from _serving import S, random_table

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x, dt=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dt).to(DEV)


@pytest.mark.parametrize("shapes", [
    [((512,), torch.uint8)],
    [((448 * 32,), torch.uint8), ((32,), torch.float32), ((64 * 32,), torch.bfloat16)],
    [((4,), torch.uint8), ((7,), torch.uint8), ((3, 5), torch.float32), ((0,), torch.uint8)],
    [((40000,), torch.uint8), ((32769,), torch.uint8), ((65536 + 4,), torch.uint8)],
])
def test_copy(shapes):
    rng = np.random.default_rng(3)
    nb = 23
    regs = [torch.from_numpy(rng.integers(0, 100, (nb, *s))).to(dt).to(DEV) for s, dt in shapes]
    ref = [r.cpu().float().numpy() for r in regs]
    src, dst = [0, 5, -1, 9, 22, 30, 7, 4], [1, 2, 3, -1, 10, 11, 23, 4]   # -1, out of the pool, itself
    csa.csa_blocks_copy(regs, dev(src), dev(dst))
    for r, x in zip(regs, ref):
        S.blocks_copy(x, src, dst)
        assert np.array_equal(r.cpu().float().numpy(), x)


@pytest.mark.parametrize("count,n", [(0, 0), (2, 2), (-3, 0), (99, 3)])
def test_copy_takes_count_from_the_device(count, n):
    r = torch.arange(10, device=DEV).float()[:, None].repeat(1, 8).contiguous()
    x = r.cpu().numpy()
    csa.csa_blocks_copy([r], dev([1, 2, 3]), dev([5, 6, 7]), dev([count, 77]))
    S.blocks_copy(x, [1, 2, 3], [5, 6, 7], n)
    assert np.array_equal(r.cpu().numpy(), x)


def forked_table(rng, rows, mb, nb):
    t = np.full((rows, mb), -1, np.int32)
    for b in range(rows):
        n = rng.integers(0, mb + 1)
        t[b, :n] = rng.choice(nb, n, replace=False)
    return t


@pytest.mark.parametrize("seed,rows,mb", [(0, 6, 4), (1, 40, 9), (2, 1, 1), (3, 300, 33)])
def test_fork(seed, rows, mb):
    rng = np.random.default_rng(seed)
    P, nb = 16, 4000
    table = forked_table(rng, rows, mb, nb)
    n = rows + 3
    # the same destination twice, rows that are source and destination, rows and
    # blocks that are none, lengths from none to beyond the table
    src, dst = rng.integers(-2, rows + 2, n), rng.integers(-2, rows + 2, n)
    tokens, fresh = rng.integers(-5, (mb + 1) * P, n), rng.integers(-1, nb, n)
    tokens[::3] -= tokens[::3] % P
    ref = S.blocks_fork(table, src, dst, tokens, fresh, P)
    dt = dev(table)
    got = csa.csa_blocks_fork(dt, dev(src), dev(dst), dev(tokens, torch.int64), dev(fresh), P)
    for a, b in zip(got, ref):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(dt.cpu().numpy(), table)


@pytest.mark.parametrize("seed,rows,mb,nb", [(0, 6, 4, 30), (1, 40, 9, 500), (2, 1, 1, 1), (3, 300, 33, 20001),
                                             (4, 5, 700, 33), (5, 2000, 40, 300000)])
def test_free_and_compact(seed, rows, mb, nb):
    rng = np.random.default_rng(seed)
    table = forked_table(rng, rows, min(mb, nb), nb)
    table[rng.random(table.shape) < 0.1] = -1
    table[rng.random(table.shape) < 0.02] = nb + 3           # no block of the pool
    dt = dev(table)
    seqs = np.concatenate([rng.integers(0, rows, max(1, rows // 3)), [-1, rows, rows + 40]])
    got = [x.cpu().numpy() for x in csa.csa_blocks_free(dt, dev(seqs), nb)]
    ref = S.blocks_free(table, seqs, nb)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1]) and got[2][0] == ref[2]
    out, cs, cd, counts = [x.cpu().numpy() for x in csa.csa_blocks_compact(dt, nb)]
    t, src, dst, live = S.blocks_compact(table, nb)
    m = len(src)
    assert list(counts) == [m, live]
    assert np.array_equal(cs[:m], src) and np.array_equal(cd[:m], dst)
    assert (cs[m:] == -1).all() and (cd[m:] == -1).all()
    assert np.array_equal(out, t)
    assert np.array_equal(dt.cpu().numpy(), table)


def test_empty_table_and_nothing_to_do():
    t = dev(np.full((3, 2), -1))
    out, freed, n = csa.csa_blocks_free(t, dev([]), 5)
    assert torch.equal(out, t) and int(n) == 0 and bool((freed == -1).all())
    out, cs, cd, counts = csa.csa_blocks_compact(t, 5)
    assert counts.tolist() == [0, 0]
    out, cs, cd = csa.csa_blocks_fork(t, dev([]), dev([]), dev([], torch.int64), dev([]))
    assert torch.equal(out, t) and cs.numel() == 0


def test_compact_is_the_same_twice_and_in_a_graph():
    rng = np.random.default_rng(7)
    table = forked_table(rng, 20, 12, 400)
    dt, pool = dev(table), torch.randint(0, 255, (400, 4096), dtype=torch.uint8, device=DEV)
    want = [pool[v].clone() if v >= 0 else None for v in table[3]]
    out = torch.empty_like(dt)
    csa.csa_blocks_compact(dt, 400, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _, cs, cd, counts = csa.csa_blocks_compact(dt, 400, out)
        csa.csa_blocks_copy([pool], cs, cd, counts)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        graph.replay()
        for v, w in zip(out[3].tolist(), want):
            assert (v < 0) == (w is None) and (w is None or torch.equal(pool[v], w))
    assert int(out.max()) < int(counts[1])


# ------------------------------------------- the framework's own paged cache ---

def _csa_cache(is_hca, table, nb, dev_buf=None):
    w = dict(c=128, rope_dims=32, m=128 if is_hca else 4, window=8, nh=8, is_hca=is_hca)
    if not is_hca:
        w |= dict(c_i=64, nh_i=4, k=12)
    return csa.CsaCache(table.shape[0], 0, device=DEV, block_table=table, num_blocks=nb, **w), w


@pytest.mark.parametrize("is_hca", [False, True])
def test_forked_sequence_of_the_csa_cache_decodes_like_its_source(is_hca):
    """A CSA / HCA layer: sequence 0 is forked to row 1, the pool is
    compacted, and a decode step of both gives what the source alone gave."""
    rng = np.random.default_rng(12)
    nb, mb, B = 12, 4, 2
    table = np.full((B, mb), -1, np.int32)
    table[0, :3] = [7, 2, 9]
    m = 128 if is_hca else 4
    tok = 128 * 2 + 44                                         # the third block is partly filled
    E, epb = tok // m, 128 // m
    cache, w = _csa_cache(is_hca, dev(table), nb)
    cache.buffer.copy_(torch.randint(0, 64, cache.buffer.shape, dtype=torch.uint8, device=DEV))
    g = torch.Generator().manual_seed(5)
    nrm = lambda *s: torch.randn(s, generator=g).bfloat16().to(DEV)  # noqa: E731
    kv = nrm(1, E, 128).repeat(B, 1, 1).contiguous()
    ik = None if is_hca else nrm(1, E, 64).repeat(B, 1, 1).contiguous()
    cache.store_entries(0, kv, ik)
    names = ("ca", "za", "kv_win") if is_hca else ("ca", "cb", "za", "zb", "ica", "icb", "iza", "izb", "kv_win")
    dim = lambda nm: 64 if nm.startswith("i") else 128  # noqa: E731
    tail = {nm: nrm(B, 60 if not is_hca else tok, dim(nm)) for nm in names}
    cache.write_rows(tok - tail["kv_win"].shape[1], tail)
    step = {nm: nrm(1, dim(nm)).repeat(B, 1).contiguous() for nm in names}
    bias = {nm: torch.zeros((m, dim(nm)), device=DEV) for nm in (("ba",) if is_hca else ("ba", "bb", "iba", "ibb"))}
    if not is_hca:
        bias["iba"], bias["ibb"] = (torch.zeros((m, 64), device=DEV) for _ in range(2))
    q = nrm(1, 8, 128).repeat(B, 1, 1).contiguous()
    qi = None if is_hca else nrm(1, 4, 64).repeat(B, 1, 1).contiguous()
    wi = None if is_hca else torch.rand((1, 4), generator=g).to(DEV).repeat(B, 1).contiguous()
    pos = torch.tensor([tok, tok], device=DEV)
    sink = torch.zeros(8, device=DEV)

    new, cs, cd = csa.csa_blocks_fork(cache.block_table, dev([0]), dev([1]), dev([tok], torch.int64), dev([4]))
    assert cs.tolist() == [9] and cd.tolist() == [4] and new[1].tolist() == [7, 2, 4, -1]
    cache.copy_blocks(cs, cd)
    cache.copy_sequences(dev([0]), dev([1]))
    packed, cs, cd, counts = csa.csa_blocks_compact(new, nb)
    cache.copy_blocks(cs, cd, counts)
    assert sorted(set(packed[packed >= 0].tolist())) == [0, 1, 2, 3]
    cache.block_table.copy_(packed)
    out = cache.decode_step(pos, step, bias, sink, 0.1, q, qi, wi)
    assert torch.equal(out[0], out[1])
    # the source alone, in a cache of its own
    lone, _ = _csa_cache(is_hca, dev(table[:1]), nb)
    lone.store_entries(0, kv[:1].contiguous(), None if ik is None else ik[:1].contiguous())
    lone.write_rows(tok - tail["kv_win"].shape[1], {nm: t[:1].contiguous() for nm, t in tail.items()})
    one = lambda t: None if t is None else t[:1].contiguous()  # noqa: E731
    ref = lone.decode_step(pos[:1].contiguous(), {nm: one(t) for nm, t in step.items()}, bias, sink, 0.1, one(q),
                           one(qi), one(wi))
    assert torch.equal(out[0], ref[0])


def test_contiguous_cache_copies_whole_sequences():
    cache = csa.CsaCache(3, 40, 128, 32, 4, 8, 8, False, c_i=64, nh_i=4, k=12)
    cache.buffer.copy_(torch.randint(0, 255, cache.buffer.shape, dtype=torch.uint8, device=DEV))
    cache.copy_sequences(dev([2]), dev([0]))
    e = cache.entries()
    for name, x in e.items():
        assert torch.equal(x[0].view(torch.uint8), x[2].view(torch.uint8)), name
    assert torch.equal(cache.region("window", torch.uint8, (3, 8 * 128 * 2))[0],
                       cache.region("window", torch.uint8, (3, 8 * 128 * 2))[2])
    with pytest.raises(ValueError):
        cache.copy_blocks(dev([0]), dev([1]))
