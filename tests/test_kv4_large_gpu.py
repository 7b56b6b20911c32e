"""The operators of the 4-bit pool and block copies on pools past 2^32 bytes and
rows past 2^31 elements: offsets that do not fit 32 bits."""
import numpy as np
import pytest
import torch

import kv4_oracle as ko
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"
HKV, D = 8, 128
BLOCKS = 2 ** 32 // (HKV * 18 * D) + 30000  # 4.8 GB


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("lens,new", [([70, 33], [1, 1]), ([70, 300], [4, 2]), ([300, 40], [200, 40])])
def test_blocks_at_the_end_of_a_large_pool(lens, new):
    rng = np.random.default_rng(sum(lens))
    pool, st = pkv.alloc_kv4_cache(BLOCKS, HKV, D), torch.zeros(1, dtype=torch.int32, device=DEV)
    held = [-(-n // 16) for n in lens]
    ids = rng.permutation(sum(held))
    table = np.full((2, max(held)), -1)
    table[0, :held[0]], table[1, :held[1]] = BLOCKS - 1 - ids[:held[0]], BLOCKS - 1 - ids[held[0]:]
    slots = np.array([table[r, j // 16] * 16 + j % 16 for r, n in enumerate(lens) for j in range(n)])
    k, v, q = bf16(rng, len(slots), HKV, D), bf16(rng, len(slots), HKV, D), bf16(rng, sum(new), 32, D)
    pkv.paged_kv4_write(k.to(DEV), v.to(DEV), i32(slots), pool, status=st)
    small = np.zeros((sum(held), HKV, 18 * D), dtype=np.uint8)
    for i, s in enumerate(slots):
        ko.pack_token(small, (s // 16 - (BLOCKS - sum(held))) * 16 + s % 16, k[i].double().numpy(), v[i].double().numpy())
    assert np.array_equal(pool[-sum(held):].cpu().numpy(), small)
    assert not pool[:-sum(held)].any()
    vals = ko.unpack(small)
    a, b = (x.double().cpu().numpy() for x in pkv.paged_kv4_read(pool, i32(slots), status=st))
    at = slots // 16 - (BLOCKS - sum(held))
    assert np.array_equal(a, vals[at, 0, :, slots % 16]) and np.array_equal(b, vals[at, 1, :, slots % 16])
    qsl = [0, new[0], sum(new)]
    out = pkv.paged_kv4_attention(q.to(DEV), pool, i32(table), i32(lens), i32(qsl), 0.09, max_query_len=max(new), status=st)
    low = np.where(table >= 0, table - (BLOCKS - sum(held)), -1)
    want, tol = ko.attend(q.double().numpy(), vals, low, lens, qsl, 0.09)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    src, dst = i32([BLOCKS - 1, 5]), i32([3, BLOCKS - sum(held) - 1])
    pool[5] = 7
    pkv.paged_copy_blocks([pool], src, dst, status=st)
    assert torch.equal(pool[3], pool[-1]) and (pool[BLOCKS - sum(held) - 1] == 7).all()
    assert pkv.pkv_read_status(st) == 0


def test_tokens_past_2_31_elements():
    """One projection's rows of 2^31 elements and more: q, k, v, out and what is read back."""
    hq, width = 12, 12 * D + 2 * 4 * D
    tokens = 2 ** 31 // (4 * D) + 5000  # what is read back passes 2^31 too
    block = torch.randn(1 << 14, width, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).to(torch.bfloat16)
    rows = block.repeat(-(-tokens // len(block)), 1)[:tokens]
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split([hq * D, 4 * D, 4 * D], dim=1))
    n = 100
    reqs = tokens // n
    pool = pkv.alloc_kv4_cache(reqs * 7, 4, D)
    table = torch.arange(reqs * 7, dtype=torch.int32, device=DEV).view(reqs, 7)
    t = torch.arange(tokens, device=DEV)
    slots = torch.where(t < reqs * n, t // n * 112 + t % n, -1).int()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.paged_kv4_write(k, v, slots, pool, status=st)
    qsl = torch.arange(reqs + 1, dtype=torch.int32, device=DEV) * n
    out = torch.full((tokens, hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
    lens = torch.full((reqs,), n, dtype=torch.int32, device=DEV)
    back = pkv.paged_kv4_read(pool, slots, status=st)
    pkv.paged_kv4_attention(q, pool, table, lens, qsl, 0.09, out=out, status=st)
    assert pkv.pkv_read_status(st) == 0 and (out[reqs * n:] == 3).all()
    for r in (0, reqs // 2, 2 ** 31 // width // n, reqs - 1):
        mine = slice(r * n, (r + 1) * n)
        vals = ko.unpack(pool[7 * r:7 * r + 7].cpu().numpy())
        for i, (x, y) in enumerate(zip(back, (k, v))):
            want = vals[:, i].transpose(0, 2, 1, 3).reshape(112, 4, D)[:n]
            assert np.array_equal(x[mine].double().cpu().numpy(), want)
            c, s = ko.quantise(y[mine].double().cpu().numpy())
            assert np.array_equal(want, np.where(c & 8, -1, 1) * ko.CODES[c & 7] * np.repeat(ko.e4m3(s), 16, -1))
        want, tol = ko.attend(q[mine].double().cpu().numpy(), vals, [list(range(7))], [n], [0, n], 0.09)
        assert (np.abs(out[mine].double().cpu().numpy() - want) <= tol).all()
