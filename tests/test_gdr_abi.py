"""Refusals of the gated delta rule and the block plan (no GPU: every call fails its
checks on the host, or is empty)."""
import ctypes

import pytest
import torch

from linear_attention_serving_prefill_b200 import binding as B
from tests import gdr_testutil as U

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BF16, F32 = 0, 1
AUTO, CORE, TC, SPLIT = 0, 1, 2, 3
P = 0x10000    # a device address that nothing reads


def prefill(**kw):
    a = dict(q=P, k=P, v=P, g=P, beta=P, cu=P, host=None, N=2, T=10, Hk=2, H=4, dk=128, dv=128,
             dt=BF16, scale=1.0, state=P, rows=4, src=P, dst=P, ctx=None, table=None, cols=0,
             block=0, o=P, ws=None, ws_bytes=0, algo=AUTO, stream=None)
    a.update(kw)
    return B._lib.kda_gdr_prefill(*a.values())


def decode(**kw):
    a = dict(q=P, k=P, v=P, g=P, beta=P, B=4, Tq=1, Hk=2, H=4, dk=128, dv=128, dt=BF16, scale=1.0,
             state=P, rows=4, src=None, dst=None, nt=None, update=1, o=P, stream=None)
    a.update(kw)
    return B._lib.kda_gdr_decode(*a.values())


def plan(**kw):
    a = dict(new=P, ctx=None, N=2, free=P, F=3, head=P, table=P, cols=4, bs=16, T=10, cu=P, pos=P,
             slots=P, src=P, dst=P, head_out=P, stream=None)
    a.update(kw)
    return B._lib.kda_block_plan(*a.values())


SIZES = [(dict(dk=96), UNSUPPORTED), (dict(dv=48), UNSUPPORTED), (dict(dk=0), INVALID),
         (dict(dv=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID),
         (dict(Hk=3), INVALID), (dict(Hk=8), INVALID), (dict(dt=5), INVALID),
         (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
         (dict(rows=-1), INVALID), (dict(q=P + 8), INVALID), (dict(v=P + 2), INVALID),
         (dict(o=P + 4), INVALID), (dict(state=P + 4), INVALID), (dict(g=P + 2), INVALID),
         (dict(src=P + 1), INVALID), (dict(dst=P + 2), INVALID), (dict(k=None), INVALID),
         (dict(g=None), INVALID), (dict(beta=None), INVALID)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(cu=None), INVALID), (dict(algo=9), INVALID),
    (dict(o=None), INVALID), (dict(algo=SPLIT), UNSUPPORTED), (dict(algo=TC, dt=F32), UNSUPPORTED),
    (dict(algo=TC, dk=64), UNSUPPORTED), (dict(block=32, table=P, cols=1), INVALID),
    (dict(block=-64, table=P, cols=1), INVALID), (dict(block=64), INVALID),
    (dict(block=64, table=P, cols=0), INVALID), (dict(block=64, table=P + 2, cols=1), INVALID),
    (dict(cols=-1), INVALID), (dict(state=None, rows=0), INVALID),
    (dict(state=None, src=None), INVALID), (dict(state=None, dst=None), INVALID),
    (dict(state=None, src=None, dst=None, block=64, table=P, cols=1), INVALID),
    (dict(ctx=P + 2), INVALID), (dict(cu=P + 2), INVALID)], ids=str)
def test_prefill_refusals(kw, code):
    assert prefill(**kw) == code


@pytest.mark.parametrize("cu", [[1, 5, 10], [0, 5, 9], [0, 7, 5], [0, 11, 10]], ids=str)
def test_prefill_host_offsets(cu):
    arr = (ctypes.c_int32 * 3)(*cu)
    assert prefill(host=ctypes.addressof(arr)) == INVALID


def test_empty_calls():
    assert prefill(N=0, T=0, cu=None) == OK
    assert decode(B=0) == OK
    assert prefill(N=0, T=0, dk=96) == UNSUPPORTED
    assert decode(B=0, H=5) == INVALID


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(B=-1), INVALID), (dict(Tq=0), INVALID), (dict(Tq=65), INVALID),
    (dict(update=2), INVALID), (dict(update=0, dst=P), INVALID), (dict(update=0, o=None), INVALID),
    (dict(state=None), INVALID), (dict(rows=3), INVALID), (dict(nt=P + 1), INVALID),
    (dict(B=1 << 26, Tq=64, src=P), INVALID)], ids=str)
def test_decode_refusals(kw, code):
    assert decode(**kw) == code


@pytest.mark.parametrize("kw", [
    dict(N=-1), dict(F=-1), dict(cols=-1), dict(cols=0), dict(bs=0), dict(bs=-16), dict(T=-1),
    dict(cu=None), dict(head=None), dict(head_out=None), dict(new=None), dict(table=None),
    dict(free=None), dict(slots=P + 4), dict(pos=P + 2), dict(new=P + 1), dict(cu=P + 2),
    dict(table=P + 2), dict(src=P + 3), dict(dst=P + 1), dict(free=P + 2), dict(head=P + 2),
    dict(head_out=P + 2), dict(ctx=P + 2), dict(N=1 << 16, cols=1 << 15)], ids=str)
def test_plan_refusals(kw):
    assert plan(**kw) == INVALID


def test_workspace_size_is_defined_for_every_call():
    assert B.kda_gdr_prefill_workspace_size(100, 2, 2, 4, 128, 128) >= 0
    assert B._lib.kda_gdr_prefill_workspace_size(100, 2, 3, 4, 128, 128, BF16, AUTO) == 0


def test_workspace_where_long_sequences_may_be_divided():
    """Few (sequence, head) pairs with many tokens need a workspace; a call without it, or with
    a smaller one, is refused before any launch."""
    need = B.kda_gdr_prefill_workspace_size(5000, 1, 1, 2, 128, 128)
    assert need > 0
    assert B.kda_gdr_prefill_workspace_size(5000, 1, 1, 148, 128, 128) == 0
    assert B.kda_gdr_prefill_workspace_size(500, 1, 1, 2, 128, 128) == 0
    assert B.kda_gdr_prefill_workspace_size(5000, 1, 1, 2, 64, 64) == 0
    assert B.kda_gdr_prefill_workspace_size(5000, 1, 1, 2, 128, 128, torch.float32) == 0
    one = dict(N=1, T=5000, Hk=1, H=2)
    assert prefill(**one) == WORKSPACE
    assert prefill(**one, ws=P, ws_bytes=need - 1) == WORKSPACE
    assert prefill(**one, ws=P + 8, ws_bytes=need) == INVALID


def test_binding_refuses_host_tensors():
    x = U.tokens((4,), 1, 2, 32, 32, torch.float32, seed=0)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        B.kda_gdr_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu)
    with pytest.raises(ValueError):
        B.kda_gdr_decode(x["q"], x["k"], x["v"], x["g"], x["beta"], torch.zeros(4, 2, 32, 32))
    one = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.kda_block_plan(one, None, one, one, torch.zeros(1, 1, dtype=torch.int32), 16, 1)


def test_reference_step_is_the_product_form():
    """The plain form used by the GPU tests against S = e^g (I - beta k k^T) S + beta k v^T."""
    x = U.tokens((6,), 1, 1, 8, 4, torch.float32, seed=3)
    state = U.pool(2, 1, 8, 4, seed=4)
    o, S = U.reference(x, [(0, 6)], 1, 0.5, state, [0], [1])
    M = state[0, 0].double()
    for t in range(6):
        k, v, q = x["k"][t, 0].double(), x["v"][t, 0].double(), x["q"][t, 0].double()
        b, a = float(x["beta"][t, 0].double()), float(torch.exp(x["g"][t, 0].double()))
        M = a * (M - b * torch.outer(k, k @ M)) + b * torch.outer(k, v)
        assert torch.allclose(o[t, 0], 0.5 * (M.T @ q), rtol=0, atol=1e-14)
    assert torch.allclose(S[1, 0], M, rtol=0, atol=1e-14)
    assert torch.equal(S[0], state[0].double())


def decode_blocks(**kw):
    a = dict(q=P, k=P, v=P, g=P, beta=P, B=4, Tq=3, Hk=2, H=4, dk=128, dv=128, dt=BF16, scale=1.0,
             state=P, rows=4, src=None, dst=None, nt=None, ctx=None, table=P, cols=2, block=64, o=P, stream=None)
    a.update(kw)
    return B._lib.kda_gdr_decode_blocks(*a.values())


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(B=-1), INVALID), (dict(Tq=0), INVALID), (dict(Tq=65), INVALID), (dict(state=None), INVALID),
    (dict(rows=3), INVALID), (dict(nt=P + 1), INVALID), (dict(ctx=P + 2), INVALID), (dict(table=P + 2), INVALID),
    (dict(table=None), INVALID), (dict(cols=0), INVALID), (dict(cols=-1), INVALID), (dict(block=0), INVALID),
    (dict(block=-64), INVALID)], ids=str)
def test_decode_blocks_refusals(kw, code):
    assert decode_blocks(**kw) == code


def test_decode_blocks_empty():
    assert decode_blocks(B=0, table=None, cols=0) == OK
    assert decode_blocks(B=0, block=0) == INVALID


def test_empty_verify():
    """A verify pass of no sequences: its empty output arrives as a null pointer."""
    assert decode(B=0, update=0, o=None) == OK
    assert decode(B=0, update=0, o=None, q=None, k=None, v=None, g=None, beta=None) == OK
    assert decode(B=0, update=0, dst=P) == INVALID and decode(B=0, update=2) == INVALID


def test_empty_prefill():
    """No sequences: nothing is read, whatever the blocks' empty table, the offsets or a
    padded token count would need otherwise."""
    assert prefill(N=0, T=0, block=64, table=None, cols=4) == OK
    assert prefill(N=0, T=0, block=64, table=None, cols=0) == OK
    assert prefill(N=0, T=5000, Hk=1, H=2) == OK
    assert B.kda_gdr_prefill_workspace_size(5000, 0, 1, 2, 128, 128) == 0
    assert prefill(N=0, T=0, block=32) == INVALID and prefill(N=0, T=0, cols=-1) == INVALID
    assert prefill(N=0, T=-1) == INVALID and prefill(N=0, rows=-1) == INVALID


def test_binding_refuses_sizes_past_32_bits():
    """The C interface counts in 32 bits; a larger number is refused, not taken modulo 2^32."""
    x = U.tokens((4,), 1, 2, 32, 32, torch.float32, seed=0)
    one, table = torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    cu, state = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(4, 2, 32, 32)
    for bad in (1 << 31, (1 << 32) + 64, -(1 << 32) + 64):
        with pytest.raises(ValueError, match="block_size"):
            B.kda_gdr_prefill(*x.values(), cu, state=state, block_table=table, block_size=bad)
        with pytest.raises(ValueError, match="block_size"):
            B.kda_gdr_decode(*x.values(), state, block_table=table, block_size=bad)
        with pytest.raises(ValueError, match="block_size"):
            B.kda_block_plan(one, None, one, one, table, bad, 1)
        with pytest.raises(ValueError, match="total_tokens"):
            B.kda_block_plan(one, None, one, one, table, 16, bad)
