"""The 4-bit key/value cache: stored bytes, values read back, and attention of
single tokens over it, against the 64-bit definitions."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_11_b200 as csa
from _serving import S, check, decode_bound, f64, filled_cache, random_table

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


@pytest.mark.parametrize("c,nkv,P,dt,pos,n,count", [
    (128, 2, 128, torch.bfloat16, [0, 0], 40, None),
    (128, 1, 16, torch.bfloat16, [5, 30, 0], 19, [19, 3, 0]),     # ragged, starts inside an image
    (64, 3, 32, torch.bfloat16, [0, 17], 33, [33, 16]),
    (64, 1, 48, torch.float32, [3], 70, None),
    (128, 2, 64, torch.float32, [15, 16, 63], 1, None),           # a decode step
    (128, 1, 16, torch.bfloat16, [-1, 3], 20, [20, -4]),          # nothing to store
])
def test_store_bytes_and_fetch(c, nkv, P, dt, pos, n, count):
    rng = np.random.default_rng(c + n)
    B, mb = len(pos), -(-(max(pos) + n) // P) + 1
    table, pool = random_table(rng, [max(0, p) + n for p in pos], P, mb)
    cache = rng.integers(0, 256, (pool, nkv, P // 16, 18 * c + 32)).astype(np.uint8)  # must survive around the rows
    g = torch.Generator().manual_seed(n)
    buf = (torch.randn((B, n, 2 * nkv + 1, c), generator=g) * torch.exp2(
        torch.randint(-20, 20, (B, n, 2 * nkv + 1, 1), generator=g).float())).to(dt)
    k, v = buf[:, :, :nkv], buf[:, :, nkv:2 * nkv]
    ref = cache.copy()
    S.kv4_store(ref, table, pos, f64(k), f64(v), count)
    dc, dtab = dev(cache), dev(table)
    dpos = torch.tensor(pos, device=DEV)
    dcnt = None if count is None else torch.tensor(count, dtype=torch.int32, device=DEV)
    db = buf.to(DEV)
    csa.csa_kv4_store(dc, dtab, dpos, db[:, :, :nkv], db[:, :, nkv:2 * nkv], dcnt)
    got = dc.cpu().numpy()
    if dt == torch.bfloat16:
        assert np.array_equal(got, ref)
    else:
        # fp32 quotients next to a tie may round across it: rare, one code apart
        assert (got != ref).mean() < 1e-4
        ref = got.copy()
    for out_dt in (torch.bfloat16, torch.float32):
        fk, fv = csa.csa_kv4_fetch(dc, dtab, dpos, n, dcnt, dtype=out_dt)
        for b in range(B):
            rows = n if count is None else max(0, count[b])
            for i in range(n):
                for h in range(nkv):
                    img = S.kv4_image(ref, table, b, h, pos[b] + i) if i < rows and pos[b] >= 0 else None
                    for x, is_v in ((fk, False), (fv, True)):
                        want = np.zeros(c) if img is None else S.read_row(img, (pos[b] + i) % 16, c, is_v)
                        assert np.array_equal(f64(x[b, i, h]), want), (b, i, h, is_v)


def test_values_are_near_what_was_stored():
    """Within a step and a half of a code: half a step for the code's own
    rounding, and the clamp at 7 when the scale rounded down by its half step
    of 2^-4: |x| / s <= 7 (1 + 2^-4), 0.44 steps beyond 7."""
    g = torch.Generator().manual_seed(9)
    k, v = torch.randn((2, 1, 64, 1, 128), generator=g).bfloat16().to(DEV)
    cache = csa.csa_kv4_cache(4, 1, 128, 16)
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    pos = torch.zeros(1, dtype=torch.int64, device=DEV)
    csa.csa_kv4_store(cache, table, pos, k, v)
    for x, y in zip((k, v), csa.csa_kv4_fetch(cache, table, pos, 64)):
        grp = x.float().unflatten(-1, (-1, 16))
        step = grp.abs().amax(-1, keepdim=True) / 7 * (1 + 2 ** -4)
        assert bool(((y.float().unflatten(-1, (-1, 16)) - grp).abs() <= 0.51 * step).all())


def test_special_rows():
    """Zeros, subnormal rows, a NaN, an infinity, and rows of the type's ends."""
    c, P = 128, 16
    x = torch.randn((1, 8, 1, c), generator=torch.Generator().manual_seed(1))
    x[0, 0] = 0
    x[0, 1] *= 2.0 ** -130
    x[0, 2, 0, 17] = float("nan")
    x[0, 3, 0, 99] = -float("inf")
    x[0, 4] = torch.finfo(torch.bfloat16).max
    x[0, 5, 0, 16:] = 0
    x[0, 6, 0, :64] *= 2.0 ** -30          # groups far below the row's largest
    x = x.bfloat16()
    cache = torch.full((1, 1, 1, 18 * c + 32), 7, dtype=torch.uint8, device=DEV)
    table = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    pos = torch.zeros(1, dtype=torch.int64, device=DEV)
    ref = cache.cpu().numpy().copy()
    S.kv4_store(ref, table.cpu().numpy(), [0], f64(x), f64(x.flip(1)))
    csa.csa_kv4_store(cache, table, pos, x.to(DEV), x.flip(1).to(DEV))
    assert np.array_equal(cache.cpu().numpy(), ref)
    k, _ = csa.csa_kv4_fetch(cache, table, pos, 8, dtype=torch.float32)
    assert torch.isnan(k[0, 2:4]).all() and torch.isfinite(k[0, [0, 1, 4, 5, 6, 7]]).all()
    assert torch.count_nonzero(k[0, 0]) == 0


def test_absent_blocks_are_not_written_and_read_as_zeros():
    cache = csa.csa_kv4_cache(3, 2, 64, 16)
    table = torch.tensor([[-1, 1, 3, 2]], dtype=torch.int32, device=DEV)   # 3 is no block of the pool
    pos = torch.zeros(1, dtype=torch.int64, device=DEV)
    k = torch.ones((1, 80, 2, 64), dtype=torch.bfloat16, device=DEV)       # 16 rows behind the table
    csa.csa_kv4_store(cache, table, pos, k, k)
    assert torch.count_nonzero(cache[0]) == 0
    y, _ = csa.csa_kv4_fetch(cache, table, pos, 80)
    there = torch.zeros(80, dtype=torch.bool)
    there[16:32] = there[48:64] = True
    assert torch.equal((y[0, :, 0, 0] != 0).cpu(), there)


def test_positions_behind_every_table():
    cache = csa.csa_kv4_cache(4, 1, 64, 16)
    table = torch.arange(4, dtype=torch.int32, device=DEV).reshape(2, 2)
    k = torch.ones((2, 5, 1, 64), dtype=torch.bfloat16, device=DEV)
    for p in (32, 2 ** 31, 2 ** 40, 2 ** 63 - 3):
        pos = torch.tensor([p, 3], dtype=torch.int64, device=DEV)
        csa.csa_kv4_store(cache, table, pos, k, k)
        assert torch.count_nonzero(cache[:2]) == 0
        for y in csa.csa_kv4_fetch(cache, table, pos, 5):
            # a row of ones: r = 2^-10, s = E4M3(1024 / 7 = 146.3) = 144 (steps of 16),
            # code = rint(1024 / 144 = 7.1) = 7: 7 * 144 / 1024
            assert torch.count_nonzero(y[0]) == 0 and (y[1] == 63 / 64).all()


# ------------------------------------------------------------------- attention ---

def decode_case(c, nkv, g, P, lens, W, first, sink, seed, scale=None):
    rng = np.random.default_rng(seed)
    mb = -(-max(max(lens), 1) // P) + 1
    table, pool = random_table(rng, lens, P, mb)
    cache = filled_cache(rng, pool, nkv, c, P)
    q = torch.from_numpy(rng.standard_normal((len(lens), nkv * g, c))).bfloat16()
    z = rng.standard_normal(nkv * g).astype(np.float32) if sink else None
    pos = [n - 1 for n in lens]
    scale = c ** -0.5 if scale is None else scale
    out = csa.csa_kv4_decode_attn(q.to(DEV), dev(cache), dev(table), torch.tensor(pos, device=DEV),
                                  scale, W, first, None if z is None else dev(z))
    ref, spread, reach, far, under = S.kv4_decode(f64(q), cache, table, pos, scale, W, first, z)
    check(out, ref, decode_bound(ref, spread, reach, far, under, scale, c, max(max(lens), 1)), "decode")
    csa.csa_check()


@pytest.mark.parametrize("c,nkv,g,P,lens,W,first,sink", [
    (128, 1, 1, 128, [1], 0, 0, False),
    (128, 2, 8, 128, [777], 0, 0, False),
    (128, 2, 4, 16, [1, 15, 16, 17, 300], 0, 0, True),
    (128, 1, 16, 64, [500, 3], 0, 0, True),
    (128, 1, 11, 32, [129, 128, 127], 0, 0, False),       # a head tile with empty rows
    (64, 3, 5, 48, [0, 250, 0, 64], 0, 0, True),           # sequences that see nothing
    (64, 1, 40, 32, [200], 0, 0, False),                   # three head tiles
    (64, 2, 16, 16, [700, 33], 0, 0, False),
    (128, 2, 4, 32, [600, 90, 41], 40, 0, False),
    (128, 2, 4, 32, [600, 90, 41, 44], 40, 4, True),
    (64, 1, 8, 16, [600, 320, 330], 100, 230, True),       # the first tokens reach into the window
    (64, 2, 2, 64, [513, 5], 1, 17, False),
    (128, 4, 8, 128, [1500, 1, 800], 256, 1, False),
])
def test_decode_matches_definition(c, nkv, g, P, lens, W, first, sink):
    decode_case(c, nkv, g, P, lens, W, first, sink, seed=sum(lens) + c)


@pytest.mark.parametrize("c,nkv,g,lens,W,first", [(128, 8, 8, [9000, 300, 12000, 5, 7777] * 4, 0, 0),
                                                  (64, 8, 16, [16000, 130, 9001] * 6, 0, 0),
                                                  (128, 8, 4, [20000, 19999, 150] * 8, 3000, 40)])
def test_decode_long_shares(c, nkv, g, lens, W, first):
    """Enough work that every CTA streams many units and several sequences."""
    P, B = 128, len(lens)
    rng = np.random.default_rng(B)
    table, pool = random_table(rng, lens, P, -(-max(lens) // P))
    cache = csa.csa_kv4_cache(pool, nkv, c, P)
    gen = torch.Generator(device=DEV).manual_seed(1)
    cache[..., :16 * c] = torch.randint(17, 256, cache[..., :16 * c].shape, generator=gen, device=DEV, dtype=torch.uint8)
    cache[..., 16 * c:18 * c] = torch.randint(30, 70, cache[..., 16 * c:18 * c].shape, generator=gen, device=DEV,
                                              dtype=torch.uint8)
    cache[..., 18 * c:] = torch.randint(122, 126, cache[..., 18 * c:].shape, generator=gen, device=DEV, dtype=torch.uint8)
    q = torch.randn((B, nkv * g, c), generator=gen, device=DEV).bfloat16()
    pos = torch.tensor(lens, device=DEV) - 1
    out = csa.csa_kv4_decode_attn(q, cache, dev(table), pos, c ** -0.5, W, first)
    csa.csa_check()
    for b in (0, 1, B - 2, B - 1):      # the rows fetched, then plain fp64 on the device
        k, v = (x[0].double() for x in csa.csa_kv4_fetch(cache, dev(table[b:b + 1]), torch.zeros(1, dtype=torch.int64,
                                                                                              device=DEV),
                                                         lens[b], dtype=torch.float32))
        u = torch.arange(lens[b], device=DEV)
        u = u[(u >= lens[b] - W) | (u < first)] if W else u
        kk, vv = (x[u].repeat_interleave(g, 1).transpose(0, 1) for x in (k, v))
        l = torch.einsum("hd,hud->hu", q[b].double(), kk) * c ** -0.5
        p = torch.softmax(l, 1)
        ref, spread = (torch.einsum("hu,hud->hd", p, x) for x in (vv, vv.abs()))
        reach = torch.einsum("hd,hud->hu", q[b].double().abs(), kk.abs()).amax(1, keepdim=True)
        far = q[b].double().abs().amax(1, keepdim=True) * kk.abs().sum(2).amax(1, keepdim=True)
        # value exponents within 2^4 of one another: r_u / r_w <= 16
        under = 16 * p.amax(1, keepdim=True) * vv.abs().sum(1)
        check(out[b], f64(ref), decode_bound(*[f64(x) for x in (ref, spread, reach, far, under)], c ** -0.5, c,
                                             len(u)), f"b={b}")


def test_decode_many_sequences_and_large_logits():
    decode_case(64, 2, 2, 16, [(37 * i) % 90 for i in range(70)], 0, 0, True, seed=3)
    decode_case(128, 1, 8, 16, [400], 0, 0, False, seed=4, scale=3.0)      # nearly one-hot weights
    decode_case(128, 1, 8, 16, [400], 0, 0, True, seed=5, scale=0.0)
    decode_case(128, 1, 8, 16, [400], 0, 0, True, seed=6, scale=-0.2)


@pytest.mark.parametrize("c", [64, 128])
def test_decode_rows_of_very_different_size(c):
    """Value rows from 2^-40 to 2^40, the largest with weights near 0, and query
    heads of every size (one of zeros): no row drowns another."""
    rng = np.random.default_rng(31)
    n, nkv, g, P = 300, 2, 4, 32
    table, pool = random_table(rng, [n], P, 10)
    cache = filled_cache(rng, pool, nkv, c, P)
    cache[..., 18 * c + 1::2] = rng.integers(87, 160, cache[..., 18 * c + 1::2].shape)   # value exponents
    for h in range(nkv):       # keys that hide the largest values' rows: the query below is positive
        for u in range(n):
            img = S.kv4_image(cache, table, 0, h, u)
            E = img[18 * c + 2 * (8 * ((u >> 1) & 1) + 2 * (u >> 2 & 3) + (u & 1)) + 1]
            if E > 127:
                S.write_row(img, u % 16, c, False, np.full(c, -7), np.full(c // 16, 56), int(127 + (E - 127) // 16))
    q = np.abs(rng.standard_normal((1, nkv * g, c))) * 2.0 ** np.array([-100, -20, 0, 3, 60, 126, -140, 0])[None, :, None]
    q[0, 7] = 0
    q = torch.from_numpy(q).bfloat16()
    for scale in (0.05, 1e-30):
        out = csa.csa_kv4_decode_attn(q.to(DEV), dev(cache), dev(table), torch.tensor([n - 1], device=DEV), scale)
        ref, spread, reach, far, under = S.kv4_decode(f64(q), cache, table, [n - 1], scale, 0, 0, None)
        fine = [h for h in range(nkv * g) if np.abs(scale * reach[0, h]) < 1e4]
        assert len(fine) >= 5
        check(out[:, fine], ref[:, fine], decode_bound(ref, spread, reach, far, under, scale, c, n)[:, fine], str(scale))


def test_decode_hidden_rows_do_not_leak():
    """NaN rows and garbage bytes outside what is seen, absent blocks inside it."""
    c, P, n = 128, 16, 200
    rng = np.random.default_rng(8)
    table, pool = random_table(rng, [n], P, 14)
    cache = filled_cache(rng, pool, 1, c, P)
    W, first = 50, 5
    for u in list(range(first, n - W)) + list(range(n, 208)):
        img = S.kv4_image(cache, table, 0, 0, u)
        S.write_row(img, u % 16, c, False, np.full(c, 7), np.full(8, 127), 255)
        S.write_row(img, u % 16, c, True, np.full(c, -7), np.full(8, 255), 255)
    table[0, 11] = -1                                       # 16 of the window's rows
    q = torch.from_numpy(rng.standard_normal((1, 4, c))).bfloat16()
    out = csa.csa_kv4_decode_attn(q.to(DEV), dev(cache), dev(table), torch.tensor([n - 1], device=DEV),
                                  0.1, W, first)
    ref, spread, reach, far, under = S.kv4_decode(f64(q), cache, table, [n - 1], 0.1, W, first, None)
    check(out, ref, decode_bound(ref, spread, reach, far, under, 0.1, c, n), "hidden")
    # one that is seen makes its heads NaN
    S.write_row(S.kv4_image(cache, table, 0, 0, n - 1), (n - 1) % 16, c, True, np.zeros(c, int), np.zeros(8, int), 255)
    out = csa.csa_kv4_decode_attn(q.to(DEV), dev(cache), dev(table), torch.tensor([n - 1], device=DEV),
                                  0.1, W, first)
    assert torch.isnan(out).all()


def test_decode_positions_beyond_the_table_and_before_the_start():
    c, P = 64, 16
    rng = np.random.default_rng(11)
    table, pool = random_table(rng, [64, 64], P, 4)
    cache = filled_cache(rng, pool, 1, c, P)
    q = torch.from_numpy(rng.standard_normal((2, 4, c))).bfloat16()
    for pos, W, first in (([100, -1], 0, 0), ([100, -7], 50, 3), ([500, 63], 20, 0)):
        out = csa.csa_kv4_decode_attn(q.to(DEV), dev(cache), dev(table), torch.tensor(pos, device=DEV), 0.125,
                                      W, first)
        ref, spread, reach, far, under = S.kv4_decode(f64(q), cache, table, pos, 0.125, W, first, None)
        check(out, ref, decode_bound(ref, spread, reach, far, under, 0.125, c, 64), str(pos))


def test_offsets_past_32_bits():
    """Blocks far beyond 4 GB into the pool."""
    nkv, c, P, B = 8, 128, 128, 2
    by = csa.csa_kv4_block_bytes(nkv, c, P)
    pool = (5 << 30) // by
    cache = torch.zeros((pool, nkv, P // 16, 18 * c + 32), dtype=torch.uint8, device=DEV)
    table = torch.tensor([[pool - 1, 3], [pool // 2 + 9, pool - 2]], dtype=torch.int32, device=DEV)
    small = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    little = csa.csa_kv4_cache(4, nkv, c, P)
    g = torch.Generator().manual_seed(2)
    k, v = torch.randn((2, B, 200, nkv, c), generator=g).bfloat16().to(DEV)
    q = torch.randn((B, 16, c), generator=g).bfloat16().to(DEV)
    pos = torch.zeros(B, dtype=torch.int64, device=DEV)
    res = []
    for ch, tb in ((cache, table), (little, small)):
        csa.csa_kv4_store(ch, tb, pos, k, v)
        res.append((csa.csa_kv4_decode_attn(q, ch, tb, pos + 199, 0.1), *csa.csa_kv4_fetch(ch, tb, pos, 200)))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    # and the copy of such blocks
    csa.csa_blocks_copy([cache], torch.tensor([pool - 1], dtype=torch.int32, device=DEV),
                        torch.tensor([pool - 7], dtype=torch.int32, device=DEV))
    assert torch.equal(cache[pool - 7], cache[pool - 1])


def test_decode_graph_streams_and_repeats():
    """A captured call replays for new positions; two calls at once with
    workspaces of their own; equal calls give equal bits."""
    rng = np.random.default_rng(21)
    lens = [300, 77]
    table, pool = random_table(rng, [400, 400], 16, 25)
    cache, tab = dev(filled_cache(rng, pool, 2, 128, 16)), dev(table)
    q = torch.from_numpy(rng.standard_normal((2, 8, 128))).bfloat16().to(DEV)
    pos = torch.tensor([n - 1 for n in lens], device=DEV)
    out = torch.empty_like(q)
    ws = torch.empty(csa.csa_kv4_decode_workspace(8, 2, 128), dtype=torch.uint8, device=DEV)
    call = lambda: csa.csa_kv4_decode_attn(q, cache, tab, pos, 0.1, ws=ws, out=out)  # noqa: E731
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
    pos += 50
    graph.replay()
    assert torch.equal(out, csa.csa_kv4_decode_attn(q, cache, tab, pos, 0.1))
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs.append(csa.csa_kv4_decode_attn(q, cache, tab, pos, 0.1))
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)
