"""Shapes that csa_qk_norm_rope takes and refuses.  The call into the library
is intercepted, so host tensors stand for device ones and no GPU is needed."""
import pytest
import torch

import compressed_sparse_attention_11_b200 as csa

BF, I64 = torch.bfloat16, torch.int64
NH, NKV, C = 8, 2, 64
AXES = (8, 12, 12)


@pytest.fixture
def calls(monkeypatch):
    """The arguments that reach the library."""
    made = []
    monkeypatch.setattr(csa, "_device", lambda t: t.get_device())
    monkeypatch.setattr(csa, "_call", lambda fn, dev, *args: made.append(args))
    return made


def go(lead_q=(2, 3), lead_k=None, qg=None, kg=None, pos=None, sections=None, q=True, k=True):
    t = lambda shape, dt: None if shape is None else torch.zeros(shape, dtype=dt)  # noqa: E731
    return csa.csa_qk_norm_rope(t((*lead_q, NH, C), BF) if q else None,
                                t((*(lead_k or lead_q), NKV, C), BF) if k else None,
                                t(lead_q if pos is None else pos, I64), t(qg, torch.float32), t(kg, torch.float32),
                                sections=sections)


@pytest.mark.parametrize("kw", [
    dict(qg=(1, NH, C)), dict(qg=(NH, 1, C)), dict(qg=(C, NH)), dict(qg=(NH * C,)), dict(qg=(1, C)), dict(qg=(NH, C, 1)),
    dict(qg=(NKV, C)), dict(kg=(1, NKV, C)), dict(kg=(C, NKV)), dict(kg=(NH, C)), dict(kg=(1, 1, C)),
    dict(qg=(1, NH, C), k=False), dict(kg=(NKV, 1, C), q=False),
])
def test_weights_of_other_shapes_are_refused(calls, kw):
    with pytest.raises(ValueError, match=r"must be \[c\] or \[heads, c\]"):
        go(**kw)
    assert not calls


def test_one_shared_weight_and_one_per_head_are_refused(calls):
    with pytest.raises(ValueError, match="both be"):
        go(qg=(C,), kg=(NKV, C))
    with pytest.raises(ValueError, match="both be"):
        go(qg=(NH, C), kg=(C,))


@pytest.mark.parametrize("kw", [
    dict(lead_q=(6,), pos=(6, 3), sections=AXES),           # [tokens, axes]
    dict(lead_q=(2, 3), pos=(2, 3, 3), sections=AXES),
    dict(lead_q=(2, 3), pos=(18,), sections=AXES),
    dict(lead_q=(2, 3), pos=(3, 3, 2), sections=AXES),
    dict(lead_q=(2, 3), pos=(3, 2)),
    dict(lead_q=(2, 3), pos=(5,)),
    dict(lead_q=(2, 3), pos=(6, 1)),
    dict(lead_q=(2, 3), pos=(2, 2, 3)),
])
def test_positions_of_other_shapes_are_refused(calls, kw):
    with pytest.raises(ValueError, match="pos must"):
        go(**kw)
    assert not calls


@pytest.mark.parametrize("lead_q,lead_k", [((2, 3), (3, 2)), ((2, 3), (6,)), ((6,), (1, 6)), ((2, 3), (2, 4))])
def test_unequal_leading_dims_are_refused(calls, lead_q, lead_k):
    with pytest.raises(ValueError, match="leading dims"):
        go(lead_q=lead_q, lead_k=lead_k)
    assert not calls


@pytest.mark.parametrize("kw,per_head", [
    (dict(), 0), (dict(qg=(C,), kg=(C,)), 0), (dict(qg=(NH, C), kg=(NKV, C)), 1), (dict(qg=(NH, C)), 1),
    (dict(kg=(NKV, C)), 1), (dict(kg=(C,)), 0), (dict(qg=(NH, C), k=False), 1), (dict(kg=(NKV, C), q=False), 1),
    (dict(pos=(6,)), 0), (dict(pos=(1, 2, 3)), 0), (dict(pos=(1, 6), sections=(32,)), 0),
    (dict(pos=(3, 2, 3), sections=AXES), 0), (dict(pos=(3, 6), sections=AXES), 0),
    (dict(lead_q=(), pos=(3,), sections=AXES), 0), (dict(lead_q=(), pos=()), 0), (dict(lead_q=(3,), pos=(3, 3), sections=AXES), 0),
])
def test_documented_shapes_reach_the_library(calls, kw, per_head):
    go(**kw)
    (args,) = calls
    p = args[9]._obj            # (the ctypes reference to the options)
    assert p.per_head == per_head
    tokens = 1
    for n in kw.get("lead_q", (2, 3)):
        tokens *= n
    assert args[4] == tokens
