"""paged_kv4_attention on batches whose chunks go through the tensor-core kernel
(kv4_chunk.cu), alone and beside decode rows, against a plain 64-bit
implementation."""
import numpy as np
import pytest
import torch

import kv4_oracle as ko
from paged_attention_kv_gb300 import binding as pkv
from test_kv4_gpu import DEV, Batch, i32, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (32, 4, 64), (8, 8, 64), (16, 2, 128), (12, 4, 128)])
@pytest.mark.parametrize("lens,new", [([160], [160]), ([128, 256, 129, 127], [128, 100, 129, 1]), ([700, 33, 20], [131, 1, 0]),
                                      ([300, 17, 500, 64], [64, 17, 90, 64])])
def test_chunks_beside_decode_rows(hq, hkv, d, lens, new):
    b = Batch(sum(lens) + hq, hq, hkv, d, lens, new)
    for longest in (max(new), 0):
        st = status()
        b.check(pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=longest, status=st))
        assert pkv.pkv_read_status(st) == 0


def test_more_items_than_the_device_runs_at_once():
    """800 items of one tile, so that items are claimed; the counter is right again afterwards."""
    b = Batch(3, 16, 16, 64, [70, 80, 90, 66] * 13, [64, 70, 65, 66] * 13)
    ws = pkv.alloc_kv4_workspace(b.pool)
    before = ws[:10].clone()
    outs = [pkv.paged_kv4_attention(*b.tensors(), b.scale, workspace=ws) for _ in range(5)]
    assert all(torch.equal(o, outs[0]) for o in outs) and torch.equal(ws[:10], before)
    b.check(outs[0])


@pytest.mark.parametrize("hq,hkv,d,lens,new", [
    (32, 8, 128, [3000], [64]), (8, 8, 64, [5000], [100]), (16, 2, 128, [9000, 700], [130, 64]), (4, 1, 64, [2000], [2000]),
    (32, 4, 64, [1200, 40, 2500], [16, 1, 9]), (128, 1, 128, [1030], [1]), (12, 4, 128, [4000, 600, 90], [50, 40, 30])])
def test_items_that_several_ctas_share(hq, hkv, d, lens, new):
    b = Batch(sum(lens) + hq, hq, hkv, d, lens, new)
    ws, st = pkv.alloc_kv4_workspace(b.pool), status()
    before = ws[:70].clone()
    call = pkv.prepare_kv4_attention(*b.tensors(), b.scale, max_query_len=max(new), workspace=ws, status=st)
    want = call().clone()
    b.check(want)
    for _ in range(10):
        call.outputs.zero_()
        assert torch.equal(call(), want)
    assert torch.equal(ws[:70], before) and pkv.pkv_read_status(st) == 0
    pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=max(new), workspace=torch.zeros_like(ws), status=st)
    assert pkv.pkv_read_status(st) & pkv.PKV_DEV_BAD_WORKSPACE


def test_values_that_are_not_finite_in_one_part_of_an_item():
    b = Batch(19, 8, 2, 128, [4000], [70])
    clean = pkv.paged_kv4_attention(*b.tensors(), b.scale)
    b.v[3950, 1, 40] = float("nan")  # position 3950: query 20 on, heads 4 to 7
    b.k[2600, 0, 3] = float("nan")   # in the middle: all of heads 0 to 3
    pkv.paged_kv4_write(b.k.to(DEV), b.v.to(DEV), i32(b.slots), b.pool)
    out = pkv.paged_kv4_attention(*b.tensors(), b.scale)
    assert torch.isnan(out[:, :4]).all() and torch.isnan(out[20:, 4:, 32:48]).all()
    rest = out.clone()
    rest[:, :4], rest[20:, 4:, 32:48] = clean[:, :4], clean[20:, 4:, 32:48]
    assert torch.equal(rest, clean)


def test_references_that_move_and_rows_of_any_size():
    b = Batch(4, 32, 8, 128, [600, 40], [150, 1])
    ramp = torch.linspace(0.01, 20, 600)[:, None, None]
    b.k[:600] = (b.k[:600].float() * ramp).to(torch.bfloat16)
    pkv.paged_kv4_write(b.k.to(DEV), b.v.to(DEV), i32(b.slots), b.pool)
    b.q[3] *= 2.0 ** 20
    b.q[4] *= 2.0 ** -100
    b.q[5, 0] = 0
    b.q[6] *= 2.0 ** -130
    b.check(pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=150))


def test_values_that_are_not_finite_reach_the_rows_that_see_them():
    for kv, d in (("k", 128), ("v", 128), ("v", 64)):
        b = Batch(9, 32, 8, d, [444, 300], [100, 300])
        clean = pkv.paged_kv4_attention(*b.tensors(), b.scale)
        x = b.k if kv == "k" else b.v
        x[444 + 130, 2, 17] = float("nan")  # request 1, position 130: its rows from 130 on, heads 8 to 11
        x[400, 5, 3] = float("nan")         # request 0, position 400: query 400 - 344 = 56 on, heads 20 to 23
        pkv.paged_kv4_write(b.k.to(DEV), b.v.to(DEV), i32(b.slots), b.pool)
        out = pkv.paged_kv4_attention(*b.tensors(), b.scale)
        rest = out.clone()
        for first, stop, heads, col in ((100 + 130, 400, slice(8, 12), slice(16, 32)), (56, 100, slice(20, 24), slice(0, 16))):
            cols = col if kv == "v" else slice(0, d)
            assert torch.isnan(out[first:stop, heads, cols]).all()
            rest[first:stop, heads, cols] = clean[first:stop, heads, cols]
        assert torch.equal(rest, clean)


def test_bad_metadata_beside_chunks():
    b = Batch(7, 32, 8, 64, [300, 200, 90], [200, 120, 2])
    exact, tol = b.want()
    q, pool, table, lens, qsl = b.tensors()

    def right(out, rows):
        return (np.abs(out[rows].double().cpu().numpy() - exact[rows]) <= tol[rows]).all()

    for bad in (-1, pool.shape[0], 2 ** 31 - 1):
        t, st = table.clone(), status()
        t[0, 5] = bad
        out = pkv.paged_kv4_attention(q, pool, t, lens, qsl, b.scale, status=st)
        assert pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_BLOCK and right(out, slice(200, 322))
    st, out = status(), torch.full_like(q, 9.0)
    pkv.paged_kv4_attention(q, pool, table, i32([300, 100, 90]), qsl, b.scale, out=out, status=st)
    assert pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_LEN
    assert right(out, slice(0, 200)) and right(out, slice(320, 322)) and (out[200:320] == 9).all()
    ws = torch.zeros_like(pkv.alloc_kv4_workspace(pool))
    pkv.paged_kv4_attention(q, pool, table, lens, qsl, b.scale, workspace=ws, status=st)
    assert pkv.pkv_read_status(st) & pkv.PKV_DEV_BAD_WORKSPACE


def test_in_a_graph_and_behind_other_kernels_that_use_tensor_memory():
    b = Batch(8, 32, 8, 128, [400, 260, 50], [256, 130, 1])
    q, pool, table, lens, qsl = b.tensors()
    call = pkv.prepare_kv4_attention(q, pool, table, lens, qsl, b.scale, max_query_len=256)
    x = torch.randn(512, 32, 128, device=DEV).to(torch.bfloat16)
    other = pkv.prepare_prompt_attention(x, x[:, :8].contiguous(), x[:, 8:16].contiguous(), i32([0, 200, 512]), 0.09)
    want = call().clone()
    b.check(want)
    other()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            other()
            call()
    call.outputs.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(call.outputs, want)
