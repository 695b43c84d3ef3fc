"""Refusals of the serving operators: each bad argument set returns a status
and a reason before anything is launched, and empty work returns without a
launch, so none of this needs a GPU."""
import ctypes

import pytest
import torch

import compressed_sparse_attention_11_b200 as csa

OK, BAD, UNSUP, WS = csa.CSA_OK, csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_UNSUPPORTED, csa.CSA_ERR_WORKSPACE
FAKE = 0x10000          # aligned, never dereferenced
ODD = 0x10002


def why():
    return csa.lib().csa_last_error().decode()


# ---------------------------------------------------------- head norms, rotation ---

def rope(**kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, tokens=4, nh=8, nkv=2, c=128, pos=FAKE, dt=1, qo=FAKE, qos=1024,
             ko=FAKE, kos=256, qg=FAKE, kg=FAKE, per_head=0, eps=1e-6, R=64, base=1e4, halves=0, axes=1,
             sec=(32, 0, 0, 0), p=True)
    a.update(kw)
    p = csa.QkRope(a["qg"], a["kg"], a["per_head"], a["eps"], a["R"], a["base"], a["halves"], a["axes"],
                   (ctypes.c_int32 * 4)(*a["sec"]))
    return csa.lib().csa_qk_norm_rope(a["q"], a["qs"], a["k"], a["ks"], a["tokens"], a["nh"], a["nkv"], a["c"],
                                      a["pos"], ctypes.byref(p) if a["p"] else None, a["dt"], a["qo"], a["qos"],
                                      a["ko"], a["kos"], None)


@pytest.mark.parametrize("kw,status,reason", [
    (dict(p=False), BAD, "p is NULL"),
    (dict(dt=9), BAD, "dt must"),
    (dict(tokens=-1), BAD, "tokens"),
    (dict(nh=0, nkv=0), BAD, "nh and nkv"),
    (dict(nh=-1), BAD, "nh and nkv"),
    (dict(c=20), BAD, "multiple of 8"),
    (dict(c=0), BAD, "multiple of 8"),
    (dict(eps=-1.0), BAD, "eps"),
    (dict(eps=float("nan")), BAD, "eps"),
    (dict(R=12), BAD, "rope_dims"),
    (dict(R=136), BAD, "rope_dims"),
    (dict(base=1.0), BAD, "rope_base"),
    (dict(base=float("inf")), BAD, "rope_base"),
    (dict(per_head=2), BAD, "per_head"),
    (dict(halves=-1), BAD, "halves"),
    (dict(axes=0), BAD, "axes"),
    (dict(axes=5), BAD, "axes"),
    (dict(sec=(31, 0, 0, 0)), BAD, "add up"),
    (dict(axes=2, sec=(40, -8, 0, 0)), BAD, "sections"),
    (dict(qs=1020), BAD, "q strides"),
    (dict(qs=512), BAD, "q strides"),
    (dict(kos=128), BAD, "k strides"),
    (dict(q=None), BAD, "q is NULL"),
    (dict(qo=None), BAD, "q_out is NULL"),
    (dict(k=ODD), BAD, "k is not 16-byte"),
    (dict(qos=2048), BAD, "in place"),
    (dict(qg=ODD), BAD, "q_gamma"),
    (dict(pos=None), BAD, "pos is NULL"),
    (dict(pos=ODD), BAD, "pos is misaligned"),
    (dict(c=520, qs=8320, qos=8320, ks=1040, kos=1040), UNSUP, "c <= 512"),
    (dict(c=264, qs=2112, qos=2112, ks=528, kos=528), UNSUP, "multiple of 16"),
    (dict(c=272, R=24, halves=1, sec=(12, 0, 0, 0), qs=2176, qos=2176, ks=544, kos=544), UNSUP, "rope_dims as well"),
    (dict(nh=70000, qs=70000 * 128, qos=70000 * 128), UNSUP, "65536"),
])
def test_qk_norm_rope_refuses(kw, status, reason):
    assert rope(**kw) == status and reason in why()


def test_qk_norm_rope_empty_and_left_out():
    assert rope(tokens=0, q=None, k=None, pos=None) == OK
    assert rope(tokens=0, nh=0, q=None, qo=None, qs=0) == OK


# ------------------------------------------------------------------ window attention ---

def window(**kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, W=16, first=0, sink=None, scale=0.1, B=1, nq=8, nk=8,
             nh=8, nkv=2, c=128, dt=1, out=FAKE)
    a.update(kw)
    return csa.lib().csa_window_attn(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["W"], a["first"],
                                     a["sink"], a["scale"], a["B"], a["nq"], a["nk"], a["nh"], a["nkv"], a["c"],
                                     a["dt"], a["out"], None)


@pytest.mark.parametrize("kw,status,reason", [
    (dict(dt=3), BAD, "dt must"),
    (dict(B=-1), BAD, "batch"),
    (dict(nk=7), BAD, "n_k >= n_q"),
    (dict(nkv=3), BAD, "multiple of nkv"),
    (dict(nkv=0), BAD, "multiple of nkv"),
    (dict(c=12), BAD, "multiple of 8"),
    (dict(W=0), BAD, "window"),
    (dict(first=-1), BAD, "first"),
    (dict(scale=float("nan")), BAD, "scale"),
    (dict(scale=float("inf")), BAD, "scale"),
    (dict(qs=1000), BAD, "strides"),
    (dict(vs=252), BAD, "strides"),
    (dict(q=None), BAD, "q is NULL"),
    (dict(k=ODD), BAD, "k is not 16-byte"),
    (dict(v=ODD), BAD, "v is not 16-byte"),
    (dict(out=None), BAD, "out is NULL"),
    (dict(sink=0x10001), BAD, "sink"),
    (dict(dt=0), UNSUP, "bf16"),
    (dict(c=96, qs=768), UNSUP, "c = 64 or 128"),
    (dict(nh=258, nkv=2, qs=258 * 128), UNSUP, "nh / nkv"),
    (dict(nk=1 << 31), UNSUP, "2^30"),
    (dict(B=1 << 20, nq=1 << 12, nk=1 << 12), UNSUP, "too many rows"),
    (dict(B=(1 << 31) - 1, nq=1 << 29, nk=1 << 29), UNSUP, "too many rows"),     # the product passes 2^60
    (dict(v=None), UNSUP, "shared"),
    (dict(v=None, nkv=1, nq=4, ks=128), UNSUP, "shared"),
    (dict(v=None, nkv=1, ks=256), UNSUP, "shared"),
    (dict(v=None, nkv=1, c=136, qs=1088, ks=136), UNSUP, "c <= 512"),
])
def test_window_attn_refuses(kw, status, reason):
    assert window(**kw) == status and reason in why()


def test_window_attn_empty():
    assert window(B=0, q=None) == OK
    assert window(nq=0, nk=5, out=None) == OK


# ---------------------------------------------------------------------- 4-bit cache ---

def desc(**kw):
    a = dict(data=FAKE, block_table=FAKE, batch=2, max_blocks=4, num_blocks=9, nkv=2, c=128, block_tokens=32)
    a.update(kw)
    return csa.Kv4Desc(*a.values())


def store(d=None, fetch=False, **kw):
    a = dict(pos=FAKE, n=3, count=None, k=FAKE, ks=256, v=FAKE, vs=256, dt=1)
    a.update(kw)
    r = None if d == "null" else ctypes.byref(d if d is not None else desc())
    if fetch:
        return csa.lib().csa_kv4_fetch(r, a["pos"], a["n"], a["count"], a["dt"], a["k"], a["v"], None)
    return csa.lib().csa_kv4_store(r, a["pos"], a["n"], a["count"], a["k"], a["ks"], a["v"], a["vs"], a["dt"], None)


def decode(d=None, **kw):
    a = dict(pos=FAKE, q=FAKE, nh=8, W=0, first=0, sink=None, scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return csa.lib().csa_kv4_decode_attn(ctypes.byref(d or desc()), a["pos"], a["q"], a["nh"], a["W"], a["first"],
                                         a["sink"], a["scale"], a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status,reason", [
    (dict(batch=-1), BAD, "batch"),
    (dict(num_blocks=0), BAD, "num_blocks"),
    (dict(max_blocks=0), BAD, "max_blocks"),
    (dict(nkv=0), BAD, "nkv"),
    (dict(c=40), BAD, "multiple of 16"),
    (dict(block_tokens=24), BAD, "block_tokens"),
    (dict(block_tokens=0), BAD, "block_tokens"),
    (dict(data=None), BAD, "data is NULL"),
    (dict(data=ODD), BAD, "data is not 16-byte"),
    (dict(block_table=None), BAD, "block_table is NULL"),
    (dict(block_table=0x10001), BAD, "misaligned"),
    (dict(c=256), UNSUP, "c = 64 or 128"),
    (dict(batch=5000), UNSUP, "4096"),
    (dict(nkv=2000), UNSUP, "1024"),
    (dict(max_blocks=1 << 28), UNSUP, "2^31 tokens"),
    (dict(block_tokens=131072), UNSUP, "65536"),
])
def test_kv4_descriptor_refused(kw, status, reason):
    stride = kw.get("nkv", 2) * kw.get("c", 128)
    for call in (lambda d: store(d, ks=max(stride, 8), vs=max(stride, 8)), lambda d: store(d, fetch=True),
                 lambda d: decode(d, nh=8 * max(1, kw.get("nkv", 2)))):
        assert call(desc(**kw)) == status and reason in why()


@pytest.mark.parametrize("kw,reason", [
    (dict(dt=5), "dt must"), (dict(n=-1), "n must"), (dict(ks=200), "strides"), (dict(vs=260), "strides"),
    (dict(pos=None), "pos is NULL"), (dict(pos=0x10004), "pos is misaligned"), (dict(k=None), "k is NULL"),
    (dict(v=ODD), "v is not 16-byte"), (dict(count=ODD), "count is misaligned"),
])
def test_kv4_store_and_fetch_refuse(kw, reason):
    assert store(**kw) == BAD and reason in why()
    if not {"ks", "vs"} & set(kw):
        assert store(fetch=True, **kw) == BAD and reason in why()


def test_kv4_null_descriptor_and_empty_work():
    assert store("null") == BAD and "cache is NULL" in why()
    assert store(n=0, k=None, v=None, pos=None) == OK
    assert store(desc(batch=0, data=None, block_table=None)) == OK
    assert decode(desc(batch=0, data=None, block_table=None), q=None, ws=None) == OK


@pytest.mark.parametrize("kw,status,reason", [
    (dict(nh=7), BAD, "multiple of nkv"), (dict(nh=0), BAD, "multiple of nkv"), (dict(W=-1), BAD, "window"),
    (dict(first=-2), BAD, "first"), (dict(scale=float("inf")), BAD, "scale"), (dict(pos=None), BAD, "pos"),
    (dict(q=ODD), BAD, "q is not 16-byte"), (dict(out=None), BAD, "out is NULL"), (dict(sink=ODD), BAD, "sink"),
    (dict(ws=None), WS, "workspace"), (dict(wsb=100), WS, "workspace"), (dict(ws=ODD), BAD, "ws is not"),
])
def test_kv4_decode_refuses(kw, status, reason):
    assert decode(**kw) == status and reason in why()


def test_kv4_sizes():
    assert csa.csa_kv4_block_bytes(8, 128, 128) == 8 * 8 * (18 * 128 + 32)
    assert csa.csa_kv4_block_bytes(1, 64, 16) == 18 * 64 + 32
    for bad in ((0, 128, 128), (1, 96, 128), (1, 128, 24), (1, 128, 0)):
        assert csa.csa_kv4_block_bytes(*bad) == 0
    assert csa.csa_kv4_decode_workspace(32, 8, 128) > 0
    for bad in ((32, 5, 128), (0, 1, 128), (8, 0, 128), (8, 2, 96)):
        assert csa.csa_kv4_decode_workspace(*bad) == 0


# --------------------------------------------------------------------------- blocks ---

def test_blocks_copy_refuses():
    L = csa.lib()
    def call(regions=((FAKE, 64),), nb=4, src=FAKE, dst=FAKE, pairs=2, count=None, n=None):
        arr = (csa.BlockRegion * max(1, len(regions)))(*[csa.BlockRegion(*r) for r in regions])
        return L.csa_blocks_copy(arr, len(regions) if n is None else n, nb, src, dst, pairs, count, None)
    assert call(n=17) == BAD and "nregions" in why()
    assert call(n=-1) == BAD
    assert call(nb=-1) == BAD and "num_blocks" in why()
    assert call(nb=1 << 31) == BAD
    assert call(pairs=-1) == BAD and "pairs" in why()
    assert call(regions=((None, 64),)) == BAD and "region 0 is NULL" in why()
    assert call(regions=((FAKE, 64), (ODD, 4))) == BAD and "region 1" in why()
    assert call(src=None) == BAD and "src" in why()
    assert call(dst=0x10001) == BAD and "dst" in why()
    assert call(count=ODD) == BAD and "count" in why()
    assert L.csa_blocks_copy(None, 1, 4, FAKE, FAKE, 1, None, None) == BAD
    assert call(regions=((FAKE, 1 << 41),)) == UNSUP
    assert call(pairs=0, src=None) == OK
    assert call(regions=((None, 0),)) == OK
    assert call(nb=0, regions=((None, 64),)) == OK


def test_block_tables_refuse():
    L = csa.lib()
    out = 0x90000000
    fork = lambda t=FAKE, r=4, m=8, s=FAKE, d=FAKE, tk=FAKE, f=FAKE, n=2, P=16, o=out, cs=FAKE, cd=FAKE: \
        L.csa_blocks_fork(t, r, m, s, d, tk, f, n, P, o, cs, cd, None)  # noqa: E731
    free = lambda t=FAKE, r=4, m=8, nb=9, s=FAKE, n=1, o=out, fr=FAKE, nf=FAKE: \
        L.csa_blocks_free(t, r, m, nb, s, n, o, fr, nf, None)  # noqa: E731
    comp = lambda t=FAKE, r=4, m=8, nb=9, o=out, cs=FAKE, cd=FAKE, c=FAKE: \
        L.csa_blocks_compact(t, r, m, nb, o, cs, cd, c, None)  # noqa: E731
    for call in (fork, free, comp):
        assert call(t=None) == BAD and "table is NULL" in why()
        assert call(o=None) == BAD and "out is NULL" in why()
        assert call(t=0x10001) == BAD and "misaligned" in why()
        assert call(o=FAKE) == BAD and "overlap" in why()
        assert call(o=FAKE + 4 * 31) == BAD and "overlap" in why()
        assert call(r=-1) == BAD and "rows" in why()
        assert call(r=1 << 21) == UNSUP
    assert fork(n=-1) == BAD and fork(P=0) == BAD and fork(s=None) == BAD and fork(tk=0x10004) == BAD
    assert fork(cs=None) == BAD and fork(cd=None) == BAD and fork(f=None) == BAD
    assert fork(r=0, n=1) == BAD and "table" in why()
    assert fork(r=0, n=0, t=None, o=None) == OK
    assert free(n=-1) == BAD and free(nb=0) == BAD and free(s=None) == BAD and free(fr=None) == BAD
    assert free(nf=ODD) == BAD and free(nb=1 << 20) == UNSUP and free(r=70000) == UNSUP
    assert comp(nb=0) == BAD and comp(cs=None) == BAD and comp(c=None) == BAD and comp(nb=1 << 20) == UNSUP


# ------------------------------------------------------------------ the Python binding ---

def test_binding_refuses_host_tensors_and_wrong_shapes():
    bf = torch.bfloat16
    q, k = torch.zeros((2, 4, 8, 128), dtype=bf), torch.zeros((2, 4, 2, 128), dtype=bf)
    i32, i64 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    tab = torch.zeros((2, 3), dtype=torch.int32)
    cache = torch.zeros((4, 2, 2, 18 * 128 + 32), dtype=torch.uint8)
    for call in (lambda: csa.csa_qk_norm_rope(q, k, i64), lambda: csa.csa_window_attn(q, k, k, 4),
                 lambda: csa.csa_kv4_store(cache, tab, i64, k, k), lambda: csa.csa_kv4_fetch(cache, tab, i64, 4),
                 lambda: csa.csa_kv4_decode_attn(q[:, 0], cache, tab, i64, 0.1),
                 lambda: csa.csa_blocks_copy([cache], i32, i32), lambda: csa.csa_blocks_free(tab, i32, 4),
                 lambda: csa.csa_blocks_fork(tab, i32, i32, i64, i32), lambda: csa.csa_blocks_compact(tab, 4)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    for call in (lambda: csa.csa_qk_norm_rope(None, None, i64), lambda: csa.csa_qk_norm_rope(q.half(), k, i64),
                 lambda: csa.csa_window_attn(q, k[:, :, :, :64], k, 4), lambda: csa.csa_window_attn(q, k, k.float(), 4),
                 lambda: csa.csa_window_attn(q[0], k, k, 4), lambda: csa.csa_kv4_cache(4, 2, 96),
                 lambda: csa.csa_kv4_fetch(cache.int(), tab, i64, 4), lambda: csa.csa_kv4_fetch(cache[0], tab, i64, 4),
                 lambda: csa.csa_blocks_free(tab.long(), i32, 4), lambda: csa.csa_blocks_fork(tab[0], i32, i32, i64, i32)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="18 c"):      # the rows of no head dim
        csa.csa_kv4_fetch(torch.zeros((4, 2, 2, 18 * 128 + 48), dtype=torch.uint8), tab, i64, 4)
    csa.csa_blocks_copy([], i32, i32)      # no regions: nothing to do

