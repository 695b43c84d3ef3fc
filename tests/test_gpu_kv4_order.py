"""4-bit decode attention between the calls around it: what follows a call in
the stream (a reader of its output, a store into the blocks it read, the next
call on the same workspace) sees it finished, also where every sequence is
short enough that one block of threads writes its output."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_11_b200 as csa
from _serving import filled_cache, random_table

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEPS = 6


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def setting(B, lens, W, nh, nkv, c, P, seed):
    rng = np.random.default_rng(seed)
    table, pool = random_table(rng, [n + STEPS for n in lens], P, -(-(max(lens) + STEPS) // P))
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).bfloat16().to(DEV)  # noqa: E731
    return dict(cache=dev(filled_cache(rng, pool, nkv, c, P)), table=dev(table), W=W,
                pos=torch.tensor(lens, dtype=torch.int64, device=DEV) - 1,
                q=[rnd(B, nh, c) for _ in range(STEPS)], k=[rnd(B, 1, nkv, c) for _ in range(STEPS)],
                v=[rnd(B, 1, nkv, c) for _ in range(STEPS)], out=torch.empty((B, nh, c), dtype=torch.bfloat16, device=DEV),
                ws=torch.empty(csa.csa_kv4_decode_workspace(nh, nkv, c), dtype=torch.uint8, device=DEV),
                got=torch.zeros((STEPS, B, nh, c), device=DEV))


def steps(s, between=lambda: None):
    """Decode, read the output, overwrite the newest row of every sequence in
    place, decode again at once with other queries into the same output."""
    for i in range(STEPS):
        for q in (s["q"][i], s["q"][-1 - i]):
            csa.csa_kv4_decode_attn(q, s["cache"], s["table"], s["pos"], 0.1, window=s["W"], ws=s["ws"], out=s["out"])
            between()
        s["got"][i].copy_(s["out"])
        between()
        csa.csa_kv4_store(s["cache"], s["table"], s["pos"], s["k"][i], s["v"][i])
        between()


CASES = [
    (200, [100] * 200, 0, 8, 2, 128, 32),                       # one unit a sequence and head
    (200, [1 + (37 * i) % 128 for i in range(200)], 0, 16, 1, 64, 16),
    (64, [1000 + 31 * i for i in range(64)], 100, 8, 2, 128, 128),   # a short window over long contexts
    (1, [64], 0, 8, 8, 128, 64),
    (3, [90, 5000, 128], 0, 8, 2, 128, 64),                     # some in one piece, one in many
]


@pytest.mark.parametrize("B,lens,W,nh,nkv,c,P", CASES)
def test_calls_behind_one_another(B, lens, W, nh, nkv, c, P):
    ref = setting(B, lens, W, nh, nkv, c, P, B)
    steps(ref, torch.cuda.synchronize)
    for _ in range(3):
        s = setting(B, lens, W, nh, nkv, c, P, B)
        torch.cuda.synchronize()
        steps(s)
        torch.cuda.synchronize()
        assert torch.equal(s["got"], ref["got"]) and torch.equal(s["cache"], ref["cache"])
    csa.csa_check()


@pytest.mark.parametrize("B,lens,W,nh,nkv,c,P", CASES)
def test_captured(B, lens, W, nh, nkv, c, P):
    ref = setting(B, lens, W, nh, nkv, c, P, B)
    steps(ref, torch.cuda.synchronize)
    s = setting(B, lens, W, nh, nkv, c, P, B)
    start = s["cache"].clone()
    steps(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        steps(s)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        s["cache"].copy_(start)
        s["got"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s["got"], ref["got"]) and torch.equal(s["cache"], ref["cache"])
    csa.csa_check()
