"""The prompt-step operators on arrays of more than 2^31 elements and pools of
more than 2^32: offsets that do not fit 32 bits."""
import pytest
import torch

import prompt_oracle as po
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"
HQ, HKV, D = 32, 2, 128
TOKENS = 2 ** 31 // (HQ * D) + 5000


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def gen_of(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    """In place of a float tensor of the whole size: piece by piece."""
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for piece in x.split(1 << 16):
        piece.copy_(torch.randn(piece.shape, generator=g, device=DEV))
    return x


def test_prompt_attention_past_2_31_elements():
    g, n = gen_of(1), 700
    lens = [n] * (TOKENS // n)
    q, k, v = randn(g, TOKENS, HQ, D), randn(g, TOKENS, HKV, D), randn(g, TOKENS, HKV, D)
    out = torch.full_like(q, 3.0)
    qsl = torch.arange(len(lens) + 1, device=DEV, dtype=torch.int32) * n
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.pkv_prompt_attention(q, k, v, qsl, D ** -0.5, out=out, status=status)
    assert pkv.pkv_read_status(status) == 0
    for r in (0, len(lens) // 2, 2 ** 31 // (HQ * D) // n, len(lens) - 1):
        at = slice(r * n, (r + 1) * n)
        want, mag = po.prompt(q[at], k[at], v[at], [n], D ** -0.5)
        assert po.worst(out[at], want, po.prompt_tolerance(want, mag)) <= 1.0
    assert bool((out[len(lens) * n:] == 3).all())


def test_norm_rope_past_2_31_elements_and_a_pool_past_2_32():
    g = gen_of(2)
    q, k, v = randn(g, TOKENS, HQ, D), randn(g, TOKENS, HKV, D), randn(g, TOKENS, HKV, D)
    nb = 2 ** 32 // (2 * HKV * 16 * D) + 600
    pool = torch.zeros(nb, 2, HKV, 16, D, dtype=torch.bfloat16, device=DEV)
    slots = (nb * 16 - 1 - torch.arange(TOKENS, device=DEV)).int()  # from the pool's end
    pos = (torch.arange(TOKENS, device=DEV) % 1000).int()
    angle = torch.rand(1000, D // 2, generator=g, device=DEV)
    cs = torch.cat([angle.cos(), angle.sin()], 1)
    w = randn(g, D)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.paged_qk_norm_rope(q, k, pos, cs, q_weight=w, k_weight=w, v=v, slot_mapping=slots, kv_cache=pool, q_out=qo,
                           k_out=ko)
    for t in (0, TOKENS // 2, 2 ** 31 // (HQ * D) - 1, 2 ** 31 // (HQ * D), TOKENS - 1):
        at = slice(t, t + 1)
        for got, x in ((qo, q), (ko, k)):
            want, mag = po.norm_rope(x[at], w, pos[at], cs)
            assert po.worst(got[at].cpu(), want, po.norm_rope_tolerance(want, mag)) <= 1.0
    s = slots.long()
    flat = pool.permute(1, 0, 3, 2, 4)
    for i, x in enumerate((ko, v)):
        for a in range(0, TOKENS, 1 << 17):
            e = slice(a, a + (1 << 17))
            assert torch.equal(flat[i][s[e] // 16, s[e] % 16], x[e])


def test_tables_past_2_31_entries():
    """Rows of a block table whose entries lie past 2^31."""
    reqs, width = 700, 2 ** 31 // 690
    table = torch.full((reqs, width), -1, dtype=torch.int32, device=DEV)
    new = torch.tensor([3 + r % 40 for r in range(reqs)], dtype=torch.int32, device=DEV)
    old = torch.tensor([(16 * width - 100) * (r % 2) for r in range(reqs)], dtype=torch.int32, device=DEV)
    table[1::2, width - 7] = torch.arange(350, dtype=torch.int32, device=DEV)
    free = torch.arange(350, 3000, dtype=torch.int32, device=DEV)
    t = int(new.sum())
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens, qsl, pos, slots, cur = pkv.paged_build_tables(new, old, free, table, t, 3000, status=status)
    assert pkv.pkv_read_status(status) == 0
    assert torch.equal(lens, old + new) and torch.equal(qsl[1:].long(), new.cumsum(0))
    taken, n, o = 350, new.tolist(), old.tolist()
    pos, slots = pos.tolist(), slots.tolist()
    for r in range(reqs):
        at, held = int(qsl[r]), -(-o[r] // 16)
        blocks = -(-(o[r] + n[r]) // 16) - held
        row = table[r, held:held + blocks].tolist()
        assert row == list(range(taken, taken + blocks))
        taken += blocks
        for i in range(n[r]):
            p = o[r] + i
            b = row[p // 16 - held] if p // 16 >= held else r // 2
            assert pos[at + i] == p and slots[at + i] == b * 16 + p % 16
    assert cur.tolist() == [taken - 350]
