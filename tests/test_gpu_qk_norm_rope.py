"""csa_qk_norm_rope against its 64-bit definition."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_11_b200 as csa
from _serving import HALF, S, check, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bound(ref, dt):
    """The output's rounding; in fp32 before it: the norm (a sum of up to 512
    squares, a root, a division: 2^-16 relative covers 512 2^-24 twice over),
    the angle's turn (fraction rounded to 2^-25 of a turn, sincospi: 2^-21 of
    the pair's size) -- both relative to the row's largest value."""
    top = np.abs(ref).max(-1, keepdims=True)
    return HALF[dt] * np.abs(ref) + (2.0 ** -16 * np.abs(ref) + 2.0 ** -20 * top) * 1.01 + 1e-30


def run(T, nh, nkv, c, R, halves, sections, dt, per_head, gamma, far, packed, inplace, seed=0):
    g = torch.Generator().manual_seed(seed)
    if packed:
        buf = torch.randn((T, (nh + 2 * nkv) * c), generator=g).to(dt).to(DEV)
        q, k = buf[:, :nh * c].unflatten(1, (nh, c)), buf[:, nh * c:(nh + nkv) * c].unflatten(1, (nkv, c))
    else:
        q = (3 * torch.randn((T, nh, c), generator=g)).to(dt).to(DEV)
        k = torch.randn((T, nkv, c), generator=g).to(dt).to(DEV)
    pos = torch.randint(-far if far < 100 else 0, far, (len(sections), T), generator=g)
    ga = [None, None]
    if gamma:
        ga = [(1 + 0.3 * torch.randn((h, c) if per_head else (c,), generator=g)) for h in (nh, nkv)]
    ref = [S.qk_norm_rope(f64(x), None if w is None else w.numpy(), pos.numpy(), sections, R, halves)
           for x, w in zip((q, k), ga)]
    rest = buf[:, (nh + nkv) * c:].clone() if packed else None
    out = csa.csa_qk_norm_rope(q, k, pos.to(DEV), *[None if w is None else w.to(DEV) for w in ga],
                               rope_dims=R, halves=halves, sections=sections,
                               q_out=q if inplace else None, k_out=k if inplace else None)
    for o, r, nm in zip(out, ref, "qk"):
        check(o, r, bound(r, dt), nm)
    if packed:
        assert torch.equal(buf[:, (nh + nkv) * c:], rest)


@pytest.mark.parametrize("T,nh,nkv,c,R,halves,sections,dt,per_head,packed,inplace", [
    (1, 32, 8, 128, 128, True, (64,), torch.bfloat16, False, True, False),
    (37, 32, 8, 128, 128, True, (64,), torch.bfloat16, False, True, True),
    (700, 5, 1, 128, 64, False, (32,), torch.bfloat16, True, False, False),
    (53, 16, 16, 128, 96, False, (16, 16, 16), torch.bfloat16, True, False, True),
    (53, 4, 2, 64, 64, True, (12, 10, 10), torch.bfloat16, False, False, False),
    (9, 64, 1, 512, 64, False, (32,), torch.bfloat16, False, False, False),
    (9, 3, 2, 512, 128, True, (20, 40, 4), torch.float32, True, True, True),
    (130, 3, 2, 256, 256, True, (128,), torch.float32, False, False, False),
    (21, 7, 3, 40, 16, False, (0, 8), torch.float32, True, False, False),
    (21, 7, 3, 72, 72, False, (9, 9, 9, 9), torch.bfloat16, False, True, False),
    (4, 2, 2, 8, 8, False, (4,), torch.bfloat16, False, False, False),
    (33, 2, 2, 272, 32, True, (16,), torch.bfloat16, False, False, False),
    (33, 2, 2, 64, 24, True, (5, 7), torch.bfloat16, True, False, True),
    (3, 9, 3, 400, 80, True, (40,), torch.float32, False, False, False),
    (7, 3, 2, 80, 40, False, (11, 9), torch.bfloat16, True, False, False),
    (3, 9, 3, 400, 40, False, (20,), torch.bfloat16, False, True, False),
    (2500, 40, 3, 128, 128, True, (64,), torch.bfloat16, True, False, False),
])
def test_matches_definition(T, nh, nkv, c, R, halves, sections, dt, per_head, packed, inplace):
    run(T, nh, nkv, c, R, halves, sections, dt, per_head, True, 50, packed, inplace)


def test_far_positions_keep_their_angle():
    run(64, 4, 2, 128, 128, True, (64,), torch.float32, False, True, 8_000_000, False, False)


def test_rotation_without_norm_and_norm_without_rotation():
    run(17, 4, 2, 128, 128, False, (64,), torch.float32, False, False, 50, False, False)
    run(17, 4, 2, 128, 0, False, (0,), torch.bfloat16, False, True, 50, False, False)


def test_one_tensor_alone_equals_both():
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn((2, 19, h, 128), generator=g).bfloat16().to(DEV) for h in (8, 2))
    pos = torch.arange(38, device=DEV).view(2, 19)
    w = torch.ones(128, device=DEV)
    both = csa.csa_qk_norm_rope(q, k, pos, w, w, rope_dims=64)
    assert both[0].shape == q.shape
    assert torch.equal(csa.csa_qk_norm_rope(q, None, pos, w, rope_dims=64)[0], both[0])
    assert torch.equal(csa.csa_qk_norm_rope(None, k, pos, None, w, rope_dims=64)[1], both[1])


def test_agrees_with_norm_rope_rows():
    """The layer's own window rows: one shared weight, positions t, 64 trailing dims."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn((2, 40, 4, 512), generator=g).bfloat16().to(DEV)
    w = (1 + 0.2 * torch.randn(512, generator=g)).to(DEV)
    a = csa.csa_norm_rope_rows(x, w)
    pos = torch.arange(40, device=DEV).repeat(2, 1)
    b = csa.csa_qk_norm_rope(x, None, pos, w)[0]
    # two fp32 computations of the same values, each rounded once
    ref = f64(a)
    check(b, ref, 2 * bound(ref, torch.bfloat16), "rows")


def test_no_tokens_and_zero_rows():
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    out, _ = csa.csa_qk_norm_rope(q, None, torch.zeros(0, dtype=torch.int64, device=DEV))
    assert out.shape == q.shape
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device=DEV)   # 0 / sqrt(eps) stays 0
    out, _ = csa.csa_qk_norm_rope(q, None, torch.arange(3, device=DEV), torch.ones(64, device=DEV))
    assert torch.count_nonzero(out) == 0


def test_graph_replay_and_side_stream():
    g = torch.Generator().manual_seed(5)
    q, k = (torch.randn((16, h, 128), generator=g).bfloat16().to(DEV) for h in (8, 2))
    pos, w = torch.arange(16, device=DEV), torch.ones(128, device=DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    call = lambda: csa.csa_qk_norm_rope(q, k, pos, w, w, rope_dims=128, halves=True, q_out=qo, k_out=ko)  # noqa: E731
    call()
    ref = qo.clone(), ko.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        call()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.current_stream().wait_stream(s)
    pos += 7
    graph.replay()
    again = csa.csa_qk_norm_rope(q, k, pos, w, w, rope_dims=128, halves=True)
    assert torch.equal(qo, again[0]) and torch.equal(ko, again[1])
    assert not torch.equal(qo, ref[0])
