"""Argument checks of the operators of the 4-bit pool and of shared pages:
refused on the host, before anything is enqueued (the pointers below are never
dereferenced)."""
import ctypes

import pytest
import torch

from paged_attention_kv_gb300 import binding as pkv

vp, f32 = ctypes.c_void_p, ctypes.c_float
NAN, INF = float("nan"), float("inf")


def desc(nb=64, bs=16, hkv=8, d=128):
    return pkv.CacheDesc(nb, bs, hkv, d)


POOLS = [(dict(bs=8), pkv.PKV_E_BLOCK_SIZE), (dict(d=96), pkv.PKV_E_HEAD_SIZE), (dict(d=256), pkv.PKV_E_HEAD_SIZE),
         (dict(nb=0), pkv.PKV_E_DIMS), (dict(hkv=0), pkv.PKV_E_DIMS), (dict(nb=2 ** 31 // 16), pkv.PKV_E_DIMS)]


def write(pool={}, **kw):
    a = dict(k=0x1000, ks=1024, v=0x2000, vs=1024, slots=0x3000, t=4, kv=0x4000, a=1.0, b=1.0, status=0x5000)
    a.update(kw)
    return pkv.LIB.paged_kv4_write(vp(a["k"]), a["ks"], vp(a["v"]), a["vs"], vp(a["slots"]), a["t"], vp(a["kv"]),
                                   ctypes.byref(desc(**pool)), f32(a["a"]), f32(a["b"]), vp(a["status"]), None)


def read(pool={}, **kw):
    a = dict(kv=0x4000, slots=0x3000, t=4, a=1.0, b=1.0, k=0x1000, v=0x2000, status=0x5000)
    a.update(kw)
    return pkv.LIB.paged_kv4_read(vp(a["kv"]), ctypes.byref(desc(**pool)), vp(a["slots"]), a["t"], f32(a["a"]),
                                  f32(a["b"]), vp(a["k"]), vp(a["v"]), vp(a["status"]), None)


def attend(pool={}, **kw):
    a = dict(q=0x1000, qs=4096, t=4, hq=32, kv=0x2000, bt=0x3000, r=2, m=8, sl=0x4000, qsl=0x5000, longest=0, scale=0.1,
             a=1.0, b=1.0, out=0x6000, ws=0x10000, n=1 << 40, status=0x7000)
    a.update(kw)
    return pkv.LIB.paged_kv4_attention(vp(a["q"]), a["qs"], a["t"], a["hq"], vp(a["kv"]), ctypes.byref(desc(**pool)),
                                       vp(a["bt"]), a["r"], a["m"], vp(a["sl"]), vp(a["qsl"]), a["longest"],
                                       f32(a["scale"]), f32(a["a"]), f32(a["b"]), vp(a["out"]), vp(a["ws"]), a["n"],
                                       vp(a["status"]), None)


def fork(**kw):
    a = dict(par=0x1000, r=4, bt=0x2000, m=8, sl=0x3000, nb=64, sh=0x4000, free=0x5000, nf=60, cur=0x6000, bto=0x7000,
             slo=0x8000, src=0x9000, dst=0xa000, status=0xb000)
    a.update(kw)
    return pkv.LIB.paged_fork_tables(vp(a["par"]), a["r"], vp(a["bt"]), a["m"], vp(a["sl"]), a["nb"], vp(a["sh"]),
                                     vp(a["free"]), a["nf"], vp(a["cur"]), vp(a["bto"]), vp(a["slo"]), vp(a["src"]),
                                     vp(a["dst"]), vp(a["status"]), None)


def copy(pools=(0x1000, 0x2000), **kw):
    a = dict(n=len(pools), size=4096, nb=64, src=0x3000, dst=0x4000, pairs=4, status=0x5000)
    a.update(kw)
    return pkv.LIB.paged_copy_blocks((vp * max(1, len(pools)))(*pools), a["n"], a["size"], a["nb"], vp(a["src"]),
                                     vp(a["dst"]), a["pairs"], vp(a["status"]), None)


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("pool,code", POOLS)
def test_pools(call, pool, code):
    assert call(pool) == code


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("name", ["a", "b"])
@pytest.mark.parametrize("s", [0.0, -1.0, 3.0, 1.0000001, 2.0 ** -61, 2.0 ** 61, NAN, INF])
def test_scales_are_powers_of_two(call, name, s):
    assert call(**{name: s}) == pkv.PKV_E_DIMS


@pytest.mark.parametrize("kw,code", [
    (dict(t=-1), pkv.PKV_E_DIMS), (dict(t=2 ** 31 - 1), pkv.PKV_E_DIMS), (dict(t=0), pkv.PKV_OK), (dict(k=0), pkv.PKV_E_NULL),
    (dict(v=0), pkv.PKV_E_NULL),
    (dict(slots=0), pkv.PKV_E_NULL), (dict(kv=0), pkv.PKV_E_NULL), (dict(k=0x1008), pkv.PKV_E_ALIGN),
    (dict(kv=0x4008), pkv.PKV_E_ALIGN), (dict(slots=0x3002), pkv.PKV_E_ALIGN), (dict(status=0x5001), pkv.PKV_E_ALIGN),
    (dict(ks=1020), pkv.PKV_E_DIMS), (dict(vs=1016), pkv.PKV_E_DIMS), (dict(ks=-1024), pkv.PKV_E_DIMS)])
def test_write(kw, code):
    assert write(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(t=-1), pkv.PKV_E_DIMS), (dict(t=0), pkv.PKV_OK), (dict(k=0, v=0), pkv.PKV_E_NULL),
    (dict(slots=0), pkv.PKV_E_NULL), (dict(kv=0), pkv.PKV_E_NULL), (dict(k=0x1008), pkv.PKV_E_ALIGN),
    (dict(v=0x2004), pkv.PKV_E_ALIGN), (dict(status=0x5001), pkv.PKV_E_ALIGN), (dict(t=2 ** 31 - 1), pkv.PKV_E_DIMS),
    (dict(v=0x1000), pkv.PKV_E_DIMS)])
def test_read(kw, code):
    assert read(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(t=-1), pkv.PKV_E_DIMS), (dict(r=-1), pkv.PKV_E_DIMS), (dict(m=-1), pkv.PKV_E_DIMS),
    (dict(longest=-1), pkv.PKV_E_DIMS), (dict(m=2 ** 31 // 16), pkv.PKV_E_DIMS), (dict(hq=33), pkv.PKV_E_GQA),
    (dict(hq=0), pkv.PKV_E_GQA), (dict(hq=8 * 129, qs=8 * 129 * 128), pkv.PKV_E_DIMS),
    (dict(t=2 ** 30), pkv.PKV_E_DIMS), (dict(scale=0.0), pkv.PKV_E_DIMS),
    (dict(scale=-1.0), pkv.PKV_E_DIMS), (dict(scale=NAN), pkv.PKV_E_DIMS), (dict(scale=2e30), pkv.PKV_E_DIMS),
    (dict(qs=4092), pkv.PKV_E_DIMS), (dict(qs=4088), pkv.PKV_E_DIMS), (dict(t=0), pkv.PKV_OK), (dict(r=0), pkv.PKV_OK),
    (dict(q=0), pkv.PKV_E_NULL), (dict(kv=0), pkv.PKV_E_NULL), (dict(bt=0), pkv.PKV_E_NULL), (dict(sl=0), pkv.PKV_E_NULL),
    (dict(qsl=0), pkv.PKV_E_NULL), (dict(out=0), pkv.PKV_E_NULL), (dict(ws=0), pkv.PKV_E_NULL),
    (dict(r=2 ** 31 - 1), pkv.PKV_E_DIMS), (dict(out=0x1000), pkv.PKV_E_DIMS),
    (dict(q=0x1008), pkv.PKV_E_ALIGN), (dict(kv=0x2004), pkv.PKV_E_ALIGN), (dict(out=0x6008), pkv.PKV_E_ALIGN),
    (dict(ws=0x10008), pkv.PKV_E_ALIGN), (dict(bt=0x3001), pkv.PKV_E_ALIGN), (dict(status=0x7002), pkv.PKV_E_ALIGN)])
def test_attention(kw, code):
    assert attend(**kw) == code


@pytest.mark.parametrize("pool,ws,code", [p[:1] + (0x1000,) + p[1:] for p in POOLS] +
                         [({}, 0, pkv.PKV_E_NULL), ({}, 0x1008, pkv.PKV_E_ALIGN)])
def test_workspace(pool, ws, code):
    assert pkv.LIB.paged_kv4_attention_init(ctypes.byref(desc(**pool)), vp(ws), 1 << 40, None) == code
    n = ctypes.c_size_t(0)
    if pool:
        assert pkv.LIB.paged_kv4_attention_workspace_bytes(ctypes.byref(desc(**pool)), ctypes.byref(n)) == code
    assert pkv.LIB.paged_kv4_attention_workspace_bytes(None, ctypes.byref(n)) == pkv.PKV_E_NULL
    assert pkv.LIB.paged_kv4_attention_init(None, vp(0x1000), 1 << 40, None) == pkv.PKV_E_NULL


@pytest.mark.parametrize("kw,code", [
    (dict(r=-1), pkv.PKV_E_DIMS), (dict(r=4097), pkv.PKV_E_DIMS), (dict(m=-1), pkv.PKV_E_DIMS), (dict(nb=0), pkv.PKV_E_DIMS),
    (dict(nf=-1), pkv.PKV_E_DIMS), (dict(r=4096, m=131073), pkv.PKV_E_DIMS), (dict(nb=2 ** 31 // 16), pkv.PKV_E_DIMS),
    (dict(r=0), pkv.PKV_OK), (dict(par=0), pkv.PKV_E_NULL), (dict(bt=0), pkv.PKV_E_NULL), (dict(sl=0), pkv.PKV_E_NULL),
    (dict(sh=0), pkv.PKV_E_NULL), (dict(free=0), pkv.PKV_E_NULL), (dict(cur=0), pkv.PKV_E_NULL),
    (dict(bto=0), pkv.PKV_E_NULL), (dict(slo=0), pkv.PKV_E_NULL), (dict(src=0), pkv.PKV_E_NULL),
    (dict(dst=0), pkv.PKV_E_NULL), (dict(bto=0x2000), pkv.PKV_E_DIMS), (dict(slo=0x3000), pkv.PKV_E_DIMS),
    (dict(par=0x1002), pkv.PKV_E_ALIGN), (dict(sh=0x4001), pkv.PKV_E_ALIGN), (dict(status=0xb003), pkv.PKV_E_ALIGN)])
def test_fork(kw, code):
    assert fork(**kw) == code


@pytest.mark.parametrize("pools,kw,code", [
    ((0x1000,), dict(n=-1), pkv.PKV_E_DIMS), ((0x1000,) * 129, {}, pkv.PKV_E_DIMS), ((), {}, pkv.PKV_OK),
    ((0x1000,), dict(pairs=0), pkv.PKV_OK), ((0x1000,), dict(pairs=-1), pkv.PKV_E_DIMS),
    ((0x1000,), dict(pairs=2 ** 31 - 1), pkv.PKV_E_DIMS), ((0x1000,), dict(size=0), pkv.PKV_E_DIMS),
    ((0x1000,), dict(size=1000), pkv.PKV_E_DIMS), ((0x1000,), dict(nb=0), pkv.PKV_E_DIMS),
    ((0x1000, 0), {}, pkv.PKV_E_NULL), ((0x1000, 0x2008), {}, pkv.PKV_E_ALIGN), ((0x1000,), dict(src=0), pkv.PKV_E_NULL),
    ((0x1000,), dict(dst=0), pkv.PKV_E_NULL), ((0x1000,), dict(src=0x3002), pkv.PKV_E_ALIGN)])
def test_copy(pools, kw, code):
    assert copy(pools, **kw) == code


def test_sizes():
    assert pkv.paged_kv4_cache_bytes(10, 8, 128) == 10 * 8 * 16 * (2 * 64 + 2 * 8)
    assert pkv.paged_kv4_cache_bytes(3, 4, 64) == 3 * 4 * 16 * (2 * 32 + 2 * 4)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv4_cache_bytes(10, 8, 80)


def test_binding_rejects_host_tensors_wrong_types_and_shapes():
    k = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros(5, 8, 18 * 64, dtype=torch.uint8)
    for call in (lambda: pkv.paged_kv4_write(k, k, i, pool), lambda: pkv.paged_kv4_read(pool, i),
                 lambda: pkv.paged_kv4_attention(k, pool, i.view(2, 2), i[:2], i[:3], 0.1),
                 lambda: pkv.paged_fork_tables(i[:2], i.view(2, 2), i[:2], i, i, i[:1]),
                 lambda: pkv.paged_copy_blocks([pool], i, i)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        pkv.paged_copy_blocks([], i, i)
    with pytest.raises(TypeError):
        pkv.paged_kv4_write(k, k, i, pool.float())
