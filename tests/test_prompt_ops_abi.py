"""Argument checks of paged_build_tables, paged_qk_norm_rope and
pkv_prompt_attention: refused on the host, before anything is enqueued (the
pointers below are never dereferenced)."""
import ctypes

import pytest
import torch

from paged_attention_kv_gb300 import binding as pkv

vp = ctypes.c_void_p


def tables(**kw):
    a = dict(ql=0x1000, cl=0x2000, r=4, free=0x3000, nf=9, cur=0x4000, t=8, nb=64, bt=0x5000, m=4, sl=0x6000,
             qsl=0x7000, pos=0x8000, slots=0x9000, cout=0xa000, status=0xb000)
    a.update(kw)
    return pkv.LIB.paged_build_tables(vp(a["ql"]), vp(a["cl"]), a["r"], vp(a["free"]), a["nf"], vp(a["cur"]), a["t"],
                                      a["nb"], vp(a["bt"]), a["m"], vp(a["sl"]), vp(a["qsl"]), vp(a["pos"]),
                                      vp(a["slots"]), vp(a["cout"]), vp(a["status"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(r=-1), pkv.PKV_E_DIMS), (dict(t=-1), pkv.PKV_E_DIMS), (dict(nf=-1), pkv.PKV_E_DIMS),
    (dict(m=-1), pkv.PKV_E_DIMS), (dict(nb=0), pkv.PKV_E_DIMS), (dict(nb=2 ** 31 // 16), pkv.PKV_E_DIMS),
    (dict(m=2 ** 31 // 16), pkv.PKV_E_DIMS), (dict(t=2 ** 31 - 1), pkv.PKV_E_DIMS),
    (dict(ql=0), pkv.PKV_E_NULL), (dict(cl=0), pkv.PKV_E_NULL), (dict(free=0), pkv.PKV_E_NULL),
    (dict(bt=0), pkv.PKV_E_NULL), (dict(sl=0), pkv.PKV_E_NULL), (dict(qsl=0), pkv.PKV_E_NULL),
    (dict(slots=0), pkv.PKV_E_NULL),
    (dict(ql=0x1002), pkv.PKV_E_ALIGN), (dict(pos=0x8001), pkv.PKV_E_ALIGN), (dict(status=0xb002), pkv.PKV_E_ALIGN),
])
def test_build_tables_host_validation(kw, code):
    assert tables(**kw) == code


def rope(desc=None, **kw):
    d = dict(num_q_heads=32, num_kv_heads=8, head_size=128, rotary_dim=128, interleaved=0, num_axes=1,
             num_positions=4096, eps=1e-6, q_stride=4096, k_stride=1024, v_stride=1024, q_out_stride=4096,
             k_out_stride=1024)
    pairs = kw.pop("pairs", (0, 0, 0, 0))
    d.update(desc or {})
    rd = pkv.RopeDesc(**d)
    for i, p in enumerate(pairs):
        rd.axis_pairs[i] = p
    a = dict(q=0x1000, k=0x2000, v=0x3000, t=4, qw=0x4000, kw=0x5000, pos=0x6000, cs=0x7000, qo=0x8000, ko=0x9000,
             slots=0xa000, kv=0xb000, nb=64, status=0xc000)
    a.update(kw)
    return pkv.LIB.paged_qk_norm_rope(ctypes.byref(rd), vp(a["q"]), vp(a["k"]), vp(a["v"]), a["t"], vp(a["qw"]),
                                      vp(a["kw"]), vp(a["pos"]), vp(a["cs"]), vp(a["qo"]), vp(a["ko"]),
                                      vp(a["slots"]), vp(a["kv"]), a["nb"], vp(a["status"]), None)


@pytest.mark.parametrize("desc,kw,code", [
    (dict(head_size=120), {}, pkv.PKV_E_HEAD_SIZE), (dict(head_size=272), {}, pkv.PKV_E_HEAD_SIZE),
    (dict(head_size=0), {}, pkv.PKV_E_HEAD_SIZE), (dict(rotary_dim=8), {}, pkv.PKV_E_DIMS),
    (dict(rotary_dim=24), {}, pkv.PKV_E_DIMS), (dict(rotary_dim=144), {}, pkv.PKV_E_DIMS),
    (dict(num_axes=0), {}, pkv.PKV_E_DIMS), (dict(num_axes=5), {}, pkv.PKV_E_DIMS),
    (dict(num_axes=3), dict(pairs=(16, 24, 23, 0)), pkv.PKV_E_DIMS),
    (dict(num_axes=2), dict(pairs=(80, -16, 0, 0)), pkv.PKV_E_DIMS),
    (dict(num_positions=0), {}, pkv.PKV_E_DIMS), (dict(eps=-1.0), {}, pkv.PKV_E_DIMS),
    (dict(eps=float("nan")), {}, pkv.PKV_E_DIMS), (dict(num_kv_heads=0), {}, pkv.PKV_E_DIMS),
    (dict(q_stride=4097), {}, pkv.PKV_E_DIMS), (dict(q_stride=4088), {}, pkv.PKV_E_DIMS),
    (dict(k_stride=1016), {}, pkv.PKV_E_DIMS), (dict(v_stride=8), {}, pkv.PKV_E_DIMS),
    (dict(q_out_stride=0), {}, pkv.PKV_E_DIMS), (dict(k_out_stride=1000), {}, pkv.PKV_E_DIMS),
    ({}, dict(t=-1), pkv.PKV_E_DIMS), ({}, dict(nb=0), pkv.PKV_E_DIMS), ({}, dict(t=0), pkv.PKV_OK),
    ({}, dict(q=0), pkv.PKV_E_NULL), ({}, dict(cs=0), pkv.PKV_E_NULL), ({}, dict(v=0), pkv.PKV_E_NULL),
    ({}, dict(slots=0), pkv.PKV_E_NULL), ({}, dict(ko=0, kv=0), pkv.PKV_E_NULL), ({}, dict(qo=0), pkv.PKV_E_NULL),
    ({}, dict(q=0x1008), pkv.PKV_E_ALIGN), ({}, dict(cs=0x7008), pkv.PKV_E_ALIGN),
    ({}, dict(kw=0x5002), pkv.PKV_E_ALIGN), ({}, dict(pos=0x6002), pkv.PKV_E_ALIGN),
    (dict(q_stride=6144), dict(qo=0x1000), pkv.PKV_E_DIMS), (dict(k_out_stride=6144), dict(ko=0x2000), pkv.PKV_E_DIMS),
])
def test_qk_norm_rope_host_validation(desc, kw, code):
    assert rope(desc, **kw) == code


def prompt(**kw):
    a = dict(q=0x1000, qs=4096, k=0x2000, ks=1024, v=0x3000, vs=1024, t=40, hq=32, hkv=8, d=128, qsl=0x4000, r=2,
             scale=0.09, out=0x5000, status=0x6000)
    a.update(kw)
    return pkv.LIB.pkv_prompt_attention(vp(a["q"]), a["qs"], vp(a["k"]), a["ks"], vp(a["v"]), a["vs"], a["t"], a["hq"],
                                        a["hkv"], a["d"], vp(a["qsl"]), a["r"], ctypes.c_float(a["scale"]),
                                        vp(a["out"]), vp(a["status"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), pkv.PKV_E_HEAD_SIZE), (dict(d=256), pkv.PKV_E_HEAD_SIZE), (dict(t=-1), pkv.PKV_E_DIMS),
    (dict(r=-1), pkv.PKV_E_DIMS), (dict(hkv=0), pkv.PKV_E_DIMS), (dict(hkv=5), pkv.PKV_E_GQA),
    (dict(hq=0), pkv.PKV_E_GQA), (dict(hq=129, hkv=1), pkv.PKV_E_GQA), (dict(scale=0.0), pkv.PKV_E_DIMS),
    (dict(scale=-1.0), pkv.PKV_E_DIMS), (dict(scale=float("nan")), pkv.PKV_E_DIMS),
    (dict(scale=float("inf")), pkv.PKV_E_DIMS), (dict(scale=2e30), pkv.PKV_E_DIMS), (dict(qs=4092), pkv.PKV_E_DIMS), (dict(ks=1020), pkv.PKV_E_DIMS),
    (dict(vs=1016), pkv.PKV_E_DIMS), (dict(t=0), pkv.PKV_OK), (dict(r=0), pkv.PKV_OK), (dict(q=0), pkv.PKV_E_NULL),
    (dict(qsl=0), pkv.PKV_E_NULL), (dict(out=0), pkv.PKV_E_NULL), (dict(k=0x2008), pkv.PKV_E_ALIGN),
    (dict(out=0x5004), pkv.PKV_E_ALIGN), (dict(qsl=0x4002), pkv.PKV_E_ALIGN),
])
def test_prompt_attention_host_validation(kw, code):
    assert prompt(**kw) == code


def test_binding_rejects_host_tensors_and_wrong_types():
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.pkv_prompt_attention(q, q, q, i, 0.1)
    with pytest.raises(TypeError):
        pkv.pkv_prompt_attention(q.float(), q, q, i, 0.1)
    with pytest.raises(ValueError):
        pkv.paged_qk_norm_rope(q, q, i, torch.zeros(8, 64))
    with pytest.raises(ValueError):
        pkv.paged_build_tables(i, i, i, i.view(4, 1), 4, 64)
