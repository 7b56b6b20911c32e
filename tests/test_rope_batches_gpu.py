"""paged_qk_norm_rope on batches in which a warp takes several of a token's
heads one after another, from q to k to v: every row of q, k and the pool."""
import pytest
import torch

import prompt_oracle as po
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"

# q heads, kv heads, head size, tokens. Warps of 8, 4 and 2 heads at once: 2 to
# 12 steps a token, taken by one warp, and at (4, 2, 256, 4000) by two, at (32, 8,
# 128, 2240) by three.
BATCHES = [(12, 4, 128, 7500), (12, 4, 128, 2500), (24, 8, 64, 7500), (24, 8, 64, 3000), (6, 2, 256, 7500),
           (4, 2, 256, 4000), (5, 1, 80, 7500), (32, 8, 128, 2240)]


def rows_of(seed, tokens, width):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(tokens, width, generator=g, device=DEV).to(torch.bfloat16), g


def inputs(hq, hkv, d, tokens, seed, axes=1):
    """Slices of one projection's rows, a shuffled pool, some tokens that are
    padding, some that are not written to the pool."""
    rows, g = rows_of(seed, tokens, (hq + 2 * hkv) * d)
    q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split([hq * d, hkv * d, hkv * d], 1))
    pos = torch.randint(0, 5000, (axes, tokens), generator=g, device=DEV, dtype=torch.int32)
    pos[:, 5::97] = -1
    nb = tokens // 16 + 9
    slots = torch.randperm(nb * 16, generator=g, device=DEV)[:tokens].int()
    slots[3::41] = -1
    pool = torch.randn(nb, 2, hkv, 16, d, generator=g, device=DEV).to(torch.bfloat16)
    qw, kw = (1 + 0.2 * torch.randn(2, d, generator=g, device=DEV)).to(torch.bfloat16)
    return q, k, v, pos, slots, pool, qw, kw


def table(n, rotary):
    half = rotary // 2
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([a.cos(), a.sin()], 1).float().to(DEV)


def check(got, before, x, weight, pos, cs, eps, interleaved, sections):
    used = (pos >= 0).all(0)
    assert torch.equal(got[~used], before[~used])
    want, mag = po.norm_rope(x[used], weight, pos[:, used], cs, eps, interleaved, sections)
    assert po.worst(got[used].cpu(), want, po.norm_rope_tolerance(want, mag)) <= 1.0


def check_pool(pool, before, k, v, pos, slots):
    """K as the call wrote it to k_out, V as it came, nothing else touched."""
    want = before.clone()
    put = (pos >= 0).all(0) & (slots >= 0)
    s = slots[put].long()
    want[s // 16, 0, :, s % 16] = k[put]
    want[s // 16, 1, :, s % 16] = v[put]
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("hq,hkv,d,tokens", BATCHES)
@pytest.mark.parametrize("norm,interleaved,axes", [(True, False, 1), (True, True, 3), (False, True, 1),
                                                   (False, False, 2)])
def test_every_row_of_a_large_batch(hq, hkv, d, tokens, norm, interleaved, axes):
    q, k, v, pos, slots, pool, qw, kw = inputs(hq, hkv, d, tokens, hq + d + tokens, axes)
    rotary = d // 2 // 16 * 16 if d > 64 else d
    half = rotary // 2
    sections = [half] if axes == 1 else [half - (axes - 1) * (half // 3)] + [half // 3] * (axes - 1)
    cs = table(5000, rotary)
    if not norm:
        qw = kw = None
    qo, ko = torch.full_like(q.contiguous(), 3.0), torch.full_like(k.contiguous(), 3.0)
    b_q, b_k, b_pool, status = qo.clone(), ko.clone(), pool.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.paged_qk_norm_rope(q, k, pos, cs, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=interleaved,
                           axis_sections=sections, v=v, slot_mapping=slots, kv_cache=pool, q_out=qo, k_out=ko,
                           status=status)
    assert pkv.pkv_read_status(status) == 0
    check(qo, b_q, q, qw, pos, cs, 1e-5, interleaved, sections)
    check(ko, b_k, k, kw, pos, cs, 1e-5, interleaved, sections)
    check_pool(pool, b_pool, ko, v, pos, slots)


@pytest.mark.parametrize("hq,hkv,d,tokens", BATCHES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_on_a_large_batch(hq, hkv, d, tokens, interleaved):
    """Heads are read ahead of those being written: in place gives the bits of
    separate outputs, in the rows and in the pool."""
    q, k, v, pos, slots, pool, qw, kw = inputs(hq, hkv, d, tokens, 1 + hq + d + tokens)
    cs = table(5000, d)
    kw_args = dict(q_weight=qw, k_weight=kw, interleaved=interleaved, v=v, slot_mapping=slots)
    qo, ko, other = q.contiguous(), k.contiguous(), pool.clone()  # padding: rows as they were
    pkv.paged_qk_norm_rope(q, k, pos, cs, kv_cache=pool, q_out=qo, k_out=ko, **kw_args)
    before_v = v.clone()
    pkv.paged_qk_norm_rope(q, k, pos, cs, kv_cache=other, q_out=q, k_out=k, **kw_args)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, before_v)
    assert torch.equal(pool.view(torch.int16), other.view(torch.int16))
