"""Calls with a ``stream`` other than the current one. What a call allocates is
written on that stream, so it has to be that stream's memory: memory of the
current stream may still be in use by what is queued there."""
import numpy as np
import pytest
import torch

from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def randn(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def as_tuple(x):
    return x if isinstance(x, tuple) else (x,)


def tables_call():
    table = torch.full((40, 9), -1, dtype=torch.int32, device=DEV)
    new, old, free = i32([100] * 40), i32([0] * 40), torch.randperm(400, device=DEV).int()
    return lambda **kw: pkv.paged_build_tables(new, old, free, table, 4000, 400, **kw)


def rope_call():
    q, k = randn(1, 600, 8, 64), randn(2, 600, 2, 64)
    angle = torch.rand(600, 32, device=DEV)
    cs, pos = torch.cat([angle.cos(), angle.sin()], 1), torch.arange(600, dtype=torch.int32, device=DEV)
    return lambda **kw: pkv.paged_qk_norm_rope(q, k, pos, cs, **kw)


def prompt_call():
    q, k, v = randn(1, 600, 8, 64), randn(2, 600, 2, 64), randn(3, 600, 2, 64)
    qsl = i32([0, 250, 600])
    return lambda **kw: pkv.pkv_prompt_attention(q, k, v, qsl, 0.125, **kw)


def slots_call():
    table = torch.randperm(400, device=DEV).int().view(40, 10)
    lens, qsl = i32([150] * 40), i32([100 * r for r in range(41)])
    return lambda **kw: pkv.paged_slot_mapping(table, lens, qsl, 4000, 400, **kw)


def gather_call():
    pool, ids = randn(4, 90, 2, 2, 16, 64), torch.randperm(90, device=DEV)[:70].int()
    return lambda **kw: pkv.paged_kv_gather_blocks(pool, ids, **kw)


def attention_call():
    pool, q = randn(5, 400, 2, 2, 16, 64), randn(6, 40, 8, 64)
    table = torch.randperm(400, device=DEV).int().view(40, 10)
    lens, qsl = i32([150] * 40), i32(list(range(41)))
    return lambda **kw: pkv.paged_attention(q, pool, table, lens, qsl, 0.125, **kw)


CALLS = {"tables": tables_call, "rope": rope_call, "prompt": prompt_call, "slots": slots_call, "gather": gather_call,
         "attention": attention_call}


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_outputs_do_not_share_memory_with_work_on_the_current_stream(name, form):
    """Fills of blocks of the outputs' sizes wait on the current stream when the
    call runs on another: the outputs keep the call's values."""
    call = CALLS[name]()
    want = [x.clone() for x in as_tuple(call())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # tens of milliseconds
    waiting = [torch.empty_like(x) for x in want]
    for x in waiting:
        x.fill_(7)
    del waiting, x  # free for the current stream's next allocations, behind the fills
    got = as_tuple(call(stream=side if form == "stream" else side.cuda_stream))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_outputs_that_are_dropped_stay_the_calls_until_it_is_done(name):
    """Results that nobody keeps go back to the stream they were written on: the
    current stream's next tensors do not get their memory."""
    call = CALLS[name]()
    sizes = [torch.empty_like(x) for x in as_tuple(call())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    call(stream=side)
    mine = [torch.full_like(x, 7) for x in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in mine)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_the_default_stream_by_handle(name):
    call = CALLS[name]()
    want = [x.clone() for x in as_tuple(call())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = as_tuple(call(stream=0))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_attention_keeps_its_own_workspace_until_it_is_done():
    """The workspace that paged_attention makes for a call on another stream is
    not given to the current stream's next tensors while the call is queued."""
    call = attention_call()
    want = call().clone()
    size = pkv.paged_attention_workspace_bytes(40, 40, 8, 400, 2, 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = call(stream=side)
    mine = [torch.full((size // 8,), 7, dtype=torch.int64, device=DEV) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((x == 7).all()) for x in mine)
