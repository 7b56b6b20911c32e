"""paged_build_tables, paged_qk_norm_rope and pkv_prompt_attention on the GPU
against plain 64-bit implementations, alone and as one step runs them."""
import numpy as np
import pytest
import torch

import prompt_oracle as po
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)


def gen_of(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------

def make_tables(rng, reqs, max_new, max_old, zero_share=0.2):
    new = [0 if rng.random() < zero_share else int(rng.integers(1, max_new + 1)) for _ in range(reqs)]
    old = [int(rng.integers(0, max_old + 1)) for _ in range(reqs)]
    width = max(-(-(o + n) // 16) for o, n in zip(old, new)) + 1
    held = [-(-o // 16) for o in old]
    need = sum(-(-(o + n) // 16) - h for o, n, h in zip(old, new, held))
    nb = sum(held) + need + 7
    perm = [int(x) for x in rng.permutation(nb)]
    table, at = np.full((reqs, width), -1), 0
    for r, h in enumerate(held):
        table[r, :h] = perm[at:at + h]
        at += h
    return new, old, perm[at:], table, nb


def check_tables(new, old, free, table, T, nb, cursor=None, expect_status=0):
    bt, status = i32(table), torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pkv.paged_build_tables(i32(new), i32(old), i32(free) if len(free) else i32([0])[:0], bt, T, nb,
                                 cursor=None if cursor is None else i32([cursor]), status=status)
    lens, qsl, pos, slots, cur, want_table, refused = po.build_tables(new, old, free, table.tolist(), T, nb,
                                                                      cursor or 0)
    assert po.as_lists(got[0]) == lens
    assert po.as_lists(got[1]) == qsl
    assert po.as_lists(got[2]) == pos
    assert po.as_lists(got[3]) == slots
    assert po.as_lists(got[4]) == [cur]
    assert po.as_lists(bt) == want_table
    assert pkv.pkv_read_status(status) == expect_status
    return refused


@pytest.mark.parametrize("reqs,max_new,max_old,pad", [
    (1, 1, 0, 0), (1, 1, 16, 0), (1, 17, 15, 3), (7, 40, 100, 0), (64, 1, 2000, 5), (300, 64, 300, 33),
    (1023, 3, 40, 0), (1024, 1, 64, 1), (1025, 2, 20, 0), (2500, 9, 100, 11), (3, 9000, 50, 2), (20, 2000, 1, 0),
    (256, 9, 70, 4), (257, 9, 70, 4), (200, 1300, 90, 7), (2, 400000, 33, 1), (1100, 700, 5, 3)])
def test_tables_match_the_definition(reqs, max_new, max_old, pad):
    rng = np.random.default_rng(reqs * 7 + max_new)
    new, old, free, table, nb = make_tables(rng, reqs, max_new, max_old)
    check_tables(new, old, free, table, sum(new) + pad, nb)


def test_tables_only_empty_requests_and_none():
    check_tables([0, 0, 0], [0, 5, 16], [], np.full((3, 2), 1), 4, 8)
    for T in (0, 5):
        out = pkv.paged_build_tables(i32([])[:0], i32([])[:0], i32([3]), torch.zeros((0, 4), dtype=torch.int32, device=DEV),
                                     T, 8, cursor=i32([1]))
        assert po.as_lists(out[1]) == [0] and po.as_lists(out[3]) == [-1] * T and po.as_lists(out[4]) == [1]


def test_tables_cursor_starts_inside_the_free_list():
    rng = np.random.default_rng(5)
    new, old, free, table, nb = make_tables(rng, 12, 50, 60)
    check_tables(new, old, [0, 1, 2] + free, table, sum(new), nb, cursor=3)


@pytest.mark.parametrize("keep", [0, 1, 5, 9])
def test_tables_refuse_requests_that_the_free_list_does_not_cover(keep):
    rng = np.random.default_rng(6)
    new, old, free, table, nb = make_tables(rng, 12, 50, 60, zero_share=0)
    new[8], old[8] = 1, 3        # needs no block: served even behind a refused request
    table[8, 0] = 2
    refused = check_tables(new, old, free[:keep], table, sum(new), nb, expect_status=pkv.PKV_DEV_NO_BLOCKS)
    assert any(refused) and not refused[8]


@pytest.mark.parametrize("cursor", [-1, 40])
def test_tables_cursor_outside_the_free_list_hands_out_nothing(cursor):
    refused = check_tables([3, 1], [0, 5], [4, 5, 6], np.array([[-1, -1], [7, -1]]), 4, 16, cursor=cursor,
                           expect_status=pkv.PKV_DEV_NO_BLOCKS)
    assert refused == [True, False]


def test_tables_refuse_bad_lengths():
    table = np.arange(15).reshape(5, 3)
    check_tables([4, -2, 4, 45, 3], [0, 5, -1, 4, 30], [40, 41, 42, 43], table, 56, 64,
                 expect_status=pkv.PKV_DEV_BAD_QSL | pkv.PKV_DEV_BAD_LEN)


def test_tables_refuse_rows_beyond_the_step():
    table = np.full((4, 8), -1)
    check_tables([10, 30, 5, 0], [0, 0, 0, 0], list(range(20)), table, 25, 64, expect_status=pkv.PKV_DEV_BAD_QSL)


def test_tables_report_bad_ids():
    table = np.array([[99, -1], [3, -1]])
    check_tables([2, 20], [5, 10], [-7, 5], table, 22, 64, expect_status=pkv.PKV_DEV_BAD_BLOCK)


def test_tables_huge_lengths_do_not_wrap():
    table = np.full((3, 2), -1)
    big = 2 ** 31 - 1
    check_tables([big, big, big], [0, 0, 0], [1, 2], table, 40, 64,
                 expect_status=pkv.PKV_DEV_BAD_LEN | pkv.PKV_DEV_BAD_QSL)


@pytest.mark.parametrize("reqs,max_new", [(40, 5), (1500, 12), (200, 40), (30, 500), (100, 200)])
def test_tables_in_place_over_many_steps(reqs, max_new):
    """Lengths and cursor updated in place, step after step without the host."""
    rng = np.random.default_rng(reqs)
    steps = 6
    new = [int(x) for x in rng.integers(0, max_new + 1, reqs)]
    width = -(-max_new * steps // 16) + 1
    free = [int(x) for x in rng.permutation(reqs * width)]
    bt, lens, cursor = i32(np.full((reqs, width), -1)), i32([0] * reqs), i32([0])
    table, old, cur = np.full((reqs, width), -1).tolist(), [0] * reqs, 0
    call = pkv.prepare_build_tables(i32(new), lens, i32(free), bt, sum(new), len(free), cursor=cursor,
                                    cursor_out=cursor, seq_lens=lens)
    got = [[x.clone() for x in call()] for _ in range(steps)]
    for s in range(steps):
        old, qsl, pos, slots, cur, table, _ = po.build_tables(new, old, free, table, sum(new), len(free), cur)
        assert [po.as_lists(x) for x in got[s]] == [old, qsl, pos, slots, [cur]]
    assert po.as_lists(bt) == table


# ---------------------------------------------------------------------------
# norms, rotation, KV write
# ---------------------------------------------------------------------------

def rope_table(n, rotary):
    half = rotary // 2
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).to(DEV)


def check_rows(got, want, mag):
    assert po.worst(got.cpu(), want, po.norm_rope_tolerance(want, mag)) <= 1.0


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (32, 4, 64), (3, 1, 16), (5, 5, 96), (4, 2, 256), (7, 1, 80)])
@pytest.mark.parametrize("tokens", [1, 37])
@pytest.mark.parametrize("norm,interleaved,part", [(True, False, 1), (False, True, 1), (True, True, 2), (False, False, 2)])
def test_norm_rope_values_and_pool(hq, hkv, d, tokens, norm, interleaved, part):
    gen = gen_of(hq * 1000 + d + tokens)
    rotary = max(16, d // part // 16 * 16)
    rows = randn(gen, tokens, (hq + 2 * hkv) * d + 8)  # packed, with a gap between rows
    q, k, v = (x.unflatten(1, (-1, d)) for x in rows[:, :-8].split([hq * d, hkv * d, hkv * d], 1))
    qw, kw = (1 + 0.2 * randn(gen, 2, d).float()).to(torch.bfloat16) if norm else (None, None)
    cs = rope_table(1000, rotary)
    pos = torch.randint(0, 1000, (tokens,), generator=gen, device=DEV, dtype=torch.int32)
    nb = tokens // 16 + 3
    pool = randn(gen, nb, 2, hkv, 16, d)
    before = pool.clone()
    slots = torch.randperm(nb * 16, generator=gen, device=DEV)[:tokens].int()
    slots[tokens // 2] = -1
    status = i32([0])
    qo, ko = pkv.paged_qk_norm_rope(q, k, pos, cs, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=interleaved, v=v,
                                    slot_mapping=slots, kv_cache=pool, k_out=torch.empty_like(k.contiguous()),
                                    status=status)
    assert pkv.pkv_read_status(status) == 0
    check_rows(qo, *po.norm_rope(q, qw, pos, cs, 1e-5, interleaved))
    check_rows(ko, *po.norm_rope(k, kw, pos, cs, 1e-5, interleaved))
    want = before.clone()
    for t, s in enumerate(po.as_lists(slots)):
        if s >= 0:
            want[s // 16, 0, :, s % 16] = ko[t]
            want[s // 16, 1, :, s % 16] = v[t]
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("sections", [(16, 24, 24), (64, 0, 0), (0, 1, 63), (30, 33, 1), (17, 47), (10, 20, 30, 4)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_with_several_axes(sections, interleaved):
    gen = gen_of(len(sections))
    t, d = 50, 128
    q, k = randn(gen, t, 6, d), randn(gen, t, 2, d)
    cs = rope_table(4096, d)
    pos = torch.randint(0, 4096, (len(sections), t), generator=gen, device=DEV, dtype=torch.int32)
    qo, ko = pkv.paged_qk_norm_rope(q, k, pos, cs, axis_sections=sections, interleaved=interleaved)
    check_rows(qo, *po.norm_rope(q, None, pos, cs, 0, interleaved, sections))
    check_rows(ko, *po.norm_rope(k, None, pos, cs, 0, interleaved, sections))


def test_norm_of_one_side_only():
    gen = gen_of(3)
    q, k = randn(gen, 20, 4, 64), randn(gen, 20, 2, 64)
    w = randn(gen, 64)
    cs, pos = rope_table(64, 64), torch.arange(20, dtype=torch.int32, device=DEV)
    for qw, kw in ((w, None), (None, w)):
        qo, ko = pkv.paged_qk_norm_rope(q, k, pos, cs, q_weight=qw, k_weight=kw)
        check_rows(qo, *po.norm_rope(q, qw, pos, cs))
        check_rows(ko, *po.norm_rope(k, kw, pos, cs))


def test_norm_rope_in_place_gives_the_same_bits():
    gen = gen_of(4)
    rows = randn(gen, 300, 48 * 128)
    q, k, v = (x.unflatten(1, (-1, 128)) for x in rows.split([4096, 1024, 1024], 1))
    w = randn(gen, 128)
    cs, pos = rope_table(512, 128), torch.arange(300, dtype=torch.int32, device=DEV)
    qo, ko = pkv.paged_qk_norm_rope(q, k, pos, cs, q_weight=w, k_weight=w)
    before_v = v.clone()
    pkv.paged_qk_norm_rope(q, k, pos, cs, q_weight=w, k_weight=w, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, before_v)


def test_padding_and_bad_positions_leave_their_rows():
    gen = gen_of(5)
    t, d = 24, 64
    q, k, v = randn(gen, t, 4, d), randn(gen, t, 2, d), randn(gen, t, 2, d)
    cs = rope_table(100, d)
    pos = torch.arange(t, dtype=torch.int32, device=DEV).repeat(2, 1)
    pos[0, 3], pos[1, 7], pos[0, 20] = -1, -1, 100
    slots = torch.arange(t, dtype=torch.int32, device=DEV)
    slots[9] = 32           # past the pool
    pool, qo, ko = randn(gen, 2, 2, 2, 16, d), randn(gen, t, 4, d), randn(gen, t, 2, d)
    b_pool, b_qo, b_ko = pool.clone(), qo.clone(), ko.clone()
    status = i32([0])
    pkv.paged_qk_norm_rope(q, k, pos, cs, axis_sections=(20, 12), v=v, slot_mapping=slots, kv_cache=pool, q_out=qo,
                           k_out=ko, status=status)
    assert pkv.pkv_read_status(status) == pkv.PKV_DEV_BAD_POS | pkv.PKV_DEV_BAD_SLOT
    skip = [3, 7, 20]
    rows = [i for i in range(t) if i not in skip]
    want = po.norm_rope(q, None, pos.clamp(0, 99), cs, 0, False, (20, 12))
    check_rows(qo[rows], want[0][rows], want[1][rows])
    assert torch.equal(qo[skip], b_qo[skip]) and torch.equal(ko[skip], b_ko[skip])
    for s in skip + [9] + list(range(t, 32)):
        assert torch.equal(pool[s // 16, :, :, s % 16], b_pool[s // 16, :, :, s % 16]), s
    assert torch.equal(pool[0, 1, :, 4], v[4])


@pytest.mark.parametrize("tokens", [700, 1300, 2500, 9000])
def test_norm_rope_large_batches(tokens):
    gen = gen_of(tokens)
    q, k = randn(gen, tokens, 12, 128), randn(gen, tokens, 4, 128)
    w = randn(gen, 128)
    cs = rope_table(tokens, 128)
    pos = torch.arange(tokens, dtype=torch.int32, device=DEV)
    qo, ko = pkv.paged_qk_norm_rope(q, k, pos, cs, q_weight=w, k_weight=w)
    at = [0, 1, tokens // 2, tokens - 1]
    check_rows(qo[at], *po.norm_rope(q[at], w, pos[at], cs))
    check_rows(ko[at], *po.norm_rope(k[at], w, pos[at], cs))
    again, _ = pkv.paged_qk_norm_rope(q[5:], k[5:], pos[5:], cs, q_weight=w, k_weight=w)
    assert torch.equal(again, qo[5:])


# ---------------------------------------------------------------------------
# prompt attention
# ---------------------------------------------------------------------------

def run_prompt(lens, hq, hkv, d, seed, packed=False, tail=0, scale=None):
    gen = gen_of(seed)
    t = sum(lens) + tail
    if packed:
        rows = randn(gen, t, (hq + 2 * hkv) * d)
        q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split([hq * d, hkv * d, hkv * d], 1))
    else:
        q, k, v = randn(gen, t, hq, d), randn(gen, t, hkv, d), randn(gen, t, hkv, d)
    qsl = i32(np.concatenate([[0], np.cumsum(lens)]).astype(int).tolist())
    return q, k, v, qsl, scale or d ** -0.5


def crowd(qsl, extra=200):
    """The same sequences with empty ones behind them: enough for the kernel's
    form for many items, where a few items have their keys split."""
    return torch.cat([qsl, qsl[-1:].repeat(extra)])


def check_prompt(q, k, v, lens, qsl, scale, out=None):
    status = i32([0])
    got = pkv.pkv_prompt_attention(q, k, v, qsl, scale, out=out, status=status)
    assert pkv.pkv_read_status(status) == 0
    want, mag = po.prompt(q, k, v, lens, scale)
    n = sum(lens)
    assert po.worst(got[:n], want, po.prompt_tolerance(want, mag)) <= 1.0
    return got


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (8, 8, 128), (4, 1, 64), (16, 2, 64)])
@pytest.mark.parametrize("lens", [[1], [2], [17, 40], [128], [129], [255, 1, 0, 256], [0, 0, 300], [64, 65, 63],
                                  [511, 513]], ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("many", [False, True])
def test_prompt_matches_the_definition(hq, hkv, d, lens, many):
    q, k, v, qsl, scale = run_prompt(lens, hq, hkv, d, 7 + sum(lens))
    check_prompt(q, k, v, lens, crowd(qsl) if many else qsl, scale)


@pytest.mark.parametrize("hq,hkv,d", [(3, 1, 128), (10, 2, 64), (32, 4, 64), (32, 8, 128), (12, 4, 128), (128, 1, 64),
                                      (100, 1, 128), (1, 1, 64)])
def test_prompt_group_sizes(hq, hkv, d):
    lens = [5, 140, 33]
    q, k, v, qsl, scale = run_prompt(lens, hq, hkv, d, hq, packed=True)
    check_prompt(q, k, v, lens, qsl, scale)
    check_prompt(q, k, v, lens, crowd(qsl), scale)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_long_and_ragged(d):
    rng = np.random.default_rng(d)
    lens = [int(x) for x in rng.integers(1, 900, 30)] + [3000]
    q, k, v, qsl, scale = run_prompt(lens, 8, 2, d, 11, packed=True)
    got = check_prompt(q, k, v, lens, qsl, scale)
    again = pkv.pkv_prompt_attention(q, k, v, qsl, scale)
    assert torch.equal(got, again)


def test_prompt_many_sequences():
    """More sequences than the kernel keeps in shared memory."""
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 4, 4600)] + [200, 1]
    q, k, v, qsl, scale = run_prompt(lens, 2, 1, 64, 12)
    check_prompt(q, k, v, lens, qsl, scale)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_rising_scores_move_the_reference(many, d):
    """Scores that grow along the keys by far more than 2^8: the running
    reference moves and O is rescaled, in every tile."""
    lens = [1000, 300]
    q, k, v, qsl, scale = run_prompt(lens, 4, 2, d, 13)
    if many:
        qsl = crowd(qsl)
    q.copy_(q.abs())
    ramp = torch.linspace(0, 2.0, 1300, device=DEV)[:, None, None]
    k.copy_(k * 0.1 + ramp)
    got = pkv.pkv_prompt_attention(q, k, v, qsl, scale)
    want, mag = po.prompt(q, k, v, lens, scale)
    # scores up to 128 * 0.8 * 2 * scale = 18 and their 32-bit sums' errors,
    # D * 2^-24 * 18 < 2^-12, twice: 2^-11 still covers them
    assert po.worst(got, want, po.prompt_tolerance(want, mag)) <= 1.0


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [290, 200])
def test_prompt_rows_do_not_show_in_each_other(at, many, d):
    """A token whose scores move its own reference changes no bit of the others'
    outputs, in tiles with masked keys and without."""
    q, k, v, qsl, scale = run_prompt([300], 4, 1, d, 17)
    if many:
        qsl = crowd(qsl)
    k[64:] += 0.1 * k[64:].sign()
    before = pkv.pkv_prompt_attention(q, k, v, qsl, scale).clone()
    q[at] = 8.0 * k[at - 1]
    after = pkv.pkv_prompt_attention(q, k, v, qsl, scale)
    same = [i for i in range(300) if i != at]
    assert torch.equal(before[same], after[same])
    assert not torch.equal(before[at], after[at])


def test_prompt_rows_behind_the_last_sequence_are_left():
    lens = [33, 100]
    q, k, v, qsl, scale = run_prompt(lens, 8, 2, 128, 14, tail=50)
    for x in (q, k, v):
        x[133:] = float("nan")
    for bounds in (qsl, crowd(qsl)):
        out = torch.full_like(q, 7.0)
        got = check_prompt(q, k, v, lens, bounds, scale, out=out)
        assert bool((got[133:] == 7).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("many", [False, True])
def test_prompt_values_that_are_not_finite_reach_only_their_readers(d, bad, which, many):
    """A token with such a value is seen by itself and what follows in its
    sequence: earlier rows, and the neighbouring sequences, keep their values."""
    lens = [150, 200, 90]
    q, k, v, qsl, scale = run_prompt(lens, 4, 1, d, 15)
    want, mag = po.prompt(q, k, v, lens, scale)
    at = 150 + 70
    (k if which == "k" else v)[at] = bad
    got = pkv.pkv_prompt_attention(q, k, v, crowd(qsl) if many else qsl, scale)
    sees = torch.zeros(440, dtype=torch.bool, device=DEV)
    sees[at:350] = True
    tol = po.prompt_tolerance(want, mag)
    assert po.worst(got[~sees], want[~sees], tol[~sees]) <= 1.0
    after, _ = po.prompt(q, k, v, lens, scale)
    g, w = got[sees].double(), after[sees]
    if which == "v":
        assert torch.equal(torch.isnan(g), torch.isnan(w)) and torch.equal(torch.isinf(g), torch.isinf(w))
    else:  # a score of minus infinity leaves a row finite
        ok = torch.isfinite(w)
        assert torch.equal(torch.isfinite(g), ok)
        assert bool(((g - w).abs()[ok] <= (w.abs() * 2.0 ** -8 + 0.05)[ok]).all())


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_scores_of_minus_infinity(d, many):
    """Keys whose score is minus infinity for every row: a row that sees no
    other key is not a number, as in the formula; the others leave them out,
    even where they fill a row's first key tiles."""
    lens, dead = [420], 300
    q, k, v, qsl, scale = run_prompt(lens, 4, 1, d, 18)
    q.copy_(q.abs() + 0.01)
    k[:dead] = -float("inf")
    got = pkv.pkv_prompt_attention(q, k, v, crowd(qsl) if many else qsl, scale)
    assert bool(torch.isnan(got[:dead]).all())
    want, mag = po.prompt(q[dead:], k[dead:], v[dead:], [lens[0] - dead], scale)
    assert po.worst(got[dead:], want, po.prompt_tolerance(want, mag)) <= 1.0


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_nothing_finite_anywhere_ends(d):
    """Every item is done twice, the second time guarded."""
    lens = [700, 1, 333]
    q, k, v, qsl, scale = run_prompt(lens, 8, 2, d, 19)
    for x in (q, k, v):
        x.fill_(float("nan"))
    status = i32([0])
    for bounds in (qsl, crowd(qsl)):
        got = pkv.pkv_prompt_attention(q, k, v, bounds, scale, status=status)
        assert bool(torch.isnan(got).all()) and pkv.pkv_read_status(status) == 0
    q, k, _, qsl, scale = run_prompt(lens, 8, 2, d, 19)
    for bounds in (qsl, crowd(qsl)):
        got = pkv.pkv_prompt_attention(q, k, v, bounds, scale, status=status)
        assert bool(torch.isnan(got).all()) and pkv.pkv_read_status(status) == 0


def test_prompt_odd_output_address():
    """An output on a 16-byte boundary that is no 32-byte one."""
    lens = [70, 200]
    q, k, v, qsl, scale = run_prompt(lens, 4, 2, 64, 21)
    out = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device=DEV)[8:].view(q.shape)
    assert out.data_ptr() % 32 == 16
    assert torch.equal(check_prompt(q, k, v, lens, qsl, scale, out=out), pkv.pkv_prompt_attention(q, k, v, qsl, scale))


def test_prompt_bad_bounds_are_reported_and_skipped():
    lens = [40, 40, 40]
    q, k, v, qsl, scale = run_prompt(lens, 4, 2, 64, 16)
    want, mag = po.prompt(q, k, v, lens, scale)
    tol = po.prompt_tolerance(want, mag)
    for bounds, good in (([0, 40, 30, 120], range(0)), ([-5, 40, 80, 120], range(40, 120)),
                         ([0, 40, 80, 121], range(0, 80))):
        out, status = torch.full_like(q, 3.0), i32([0])
        pkv.pkv_prompt_attention(q, k, v, i32(bounds), scale, out=out, status=status)
        assert pkv.pkv_read_status(status) == pkv.PKV_DEV_BAD_QSL
        rows = list(good)
        if rows:
            assert po.worst(out[rows], want[rows], tol[rows]) <= 1.0
            rest = [i for i in range(120) if i not in good]
            assert bool((out[rest] == 3).all())


def test_prompt_overlapping_sequences_are_refused():
    q, k, v, _, scale = run_prompt([400], 4, 2, 64, 22)
    out, status = torch.full_like(q, 3.0), i32([0])
    pkv.pkv_prompt_attention(q, k, v, i32([0, 400, 0, 400, 0, 400, 0, 400, 0, 400]), scale, out=out, status=status)
    assert pkv.pkv_read_status(status) == pkv.PKV_DEV_BAD_QSL
    assert bool((out == 3).all())


def test_prompt_agrees_with_chunked_paged_attention():
    """The same prompt through the pool, in two chunks, gives the same rows."""
    lens = [500]
    q, k, v, qsl, scale = run_prompt(lens, 32, 8, 128, 17)
    want = check_prompt(q, k, v, lens, qsl, scale)
    pool = torch.zeros((40, 2, 8, 16, 128), dtype=torch.bfloat16, device=DEV)
    table = torch.randperm(40, device=DEV)[:32].int().view(1, 32).contiguous()
    for a, b in ((0, 200), (200, 500)):
        qs = i32([0, b - a])
        slots = pkv.paged_slot_mapping(table, i32([b]), qs, b - a, 40)
        pkv.paged_kv_write(k[a:b], v[a:b], slots, pool)
        out = pkv.paged_attention(q[a:b], pool, table, i32([b]), qs, scale)
        ref, mag = po.prompt(q, k, v, lens, scale)
        assert po.worst(out, ref[a:b], 2 * po.prompt_tolerance(ref[a:b], mag[a:b])) <= 1.0
        assert bool(((out.double() - want[a:b].double()).abs() <= 3 * po.prompt_tolerance(ref, mag)[a:b]).all())


# ---------------------------------------------------------------------------
# streams, graphs, a whole step
# ---------------------------------------------------------------------------

def test_calls_on_two_streams_at_once():
    lens = [700, 300]
    sets = [run_prompt(lens, 8, 2, 128, 20 + s) for s in range(2)]
    want = [pkv.pkv_prompt_attention(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(pkv.pkv_prompt_attention(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


class Layer:
    """Tables, norms with rotation and pool write, attention: what one step of
    an engine runs, on buffers of a fixed size."""

    def __init__(self, seed, rows, reqs, hq=8, hkv=2, d=128, blocks=64):
        gen = gen_of(seed)
        self.hq, self.hkv, self.d, self.scale = hq, hkv, d, d ** -0.5
        self.qkv = randn(gen, rows, (hq + 2 * hkv) * d)
        self.q, self.k, self.v = (x.unflatten(1, (-1, d)) for x in self.qkv.split([hq * d, hkv * d, hkv * d], 1))
        self.qw, self.kw = (1 + 0.2 * randn(gen, 2, d).float()).to(torch.bfloat16)
        self.cs = rope_table(4096, d)
        self.pool = randn(gen, blocks, 2, hkv, 16, d)
        self.new, self.lens, self.cursor = i32([0] * reqs), i32([0] * reqs), i32([0])
        self.free = torch.randperm(blocks, generator=gen, device=DEV).int()
        self.table = torch.full((reqs, blocks // reqs), -1, dtype=torch.int32, device=DEV)
        self.status = i32([0])
        self.tables = pkv.prepare_build_tables(self.new, self.lens, self.free, self.table, rows, blocks,
                                               cursor=self.cursor, cursor_out=self.cursor, seq_lens=self.lens,
                                               status=self.status)
        _, self.qsl, pos, slots, _ = self.tables.outputs
        self.q_out = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device=DEV)
        self.k_out = torch.zeros((rows, hkv, d), dtype=torch.bfloat16, device=DEV)
        self.rope = pkv.prepare_qk_norm_rope(self.q, self.k, pos, self.cs, q_weight=self.qw, k_weight=self.kw, v=self.v,
                                             slot_mapping=slots, kv_cache=self.pool, q_out=self.q_out,
                                             k_out=self.k_out, status=self.status)
        self.prompt = pkv.prepare_prompt_attention(self.q_out, self.k_out, self.v, self.qsl, self.scale,
                                                   status=self.status)
        self.out = self.prompt.outputs
        self.work = pkv.alloc_workspace(reqs, rows, hq, self.pool)

    def prefill(self):
        self.tables()
        self.rope()
        return self.prompt()

    def decode(self):
        self.tables()
        self.rope()
        return pkv.paged_attention(self.q_out, self.pool, self.table, self.lens, self.qsl, self.scale,
                                   workspace=self.work)


def history(layer, seed_rows, pos):
    """64-bit q and k of one token set, from the projections."""
    q, _ = po.norm_rope(seed_rows[0], layer.qw, pos, layer.cs)
    k, _ = po.norm_rope(seed_rows[1], layer.kw, pos, layer.cs)
    return q, k


def test_a_prompt_step_and_decode_steps_without_the_host():
    """Prompts through tables, norms and prompt attention, then decode steps
    through the pool: every output row against 64-bit attention over the whole
    history. q, k carry bf16 roundings (2^-8 each): a score of |q||k| scale
    (about 11 after the norms, rounded independently per column: 11 * 2^-8 *
    sqrt(2) / sqrt(128) * 4 sigma) moves by less than 0.025, a probability by
    that share, the output by twice it of sum p |v|."""
    lens, rows = [37, 5, 0, 130], 172
    a = Layer(30, rows, 4)
    a.new.copy_(i32(lens))
    out = a.prefill().clone()
    assert pkv.pkv_read_status(a.status) == 0
    hist_k, hist_v, at = [], [], 0
    for n in lens:
        pos = torch.arange(n, dtype=torch.int32)
        q, k = history(a, (a.q[at:at + n], a.k[at:at + n]), pos)
        v = a.v[at:at + n].double().cpu()
        if n:
            want, mag = po.prompt(q, k, v, [n], a.scale)
            tol = po.prompt_tolerance(want, mag) + 0.05 * mag
            assert po.worst(out[at:at + n].cpu(), want, tol) <= 1.0
        hist_k.append(k)
        hist_v.append(v)
        at += n
    b = Layer(31, 4, 4)
    for name in ("pool", "table", "lens", "cursor", "free"):
        getattr(b, name).copy_(getattr(a, name))
    b.qw.copy_(a.qw)
    b.kw.copy_(a.kw)
    b.new.copy_(i32([1, 1, 1, 1]))
    gen = gen_of(32)
    for step in range(20):
        b.qkv.copy_(randn(gen, *b.qkv.shape))
        got = b.decode().cpu()
        for r in range(4):
            pos = torch.tensor([len(hist_k[r])], dtype=torch.int32)
            q, k = history(b, (b.q[r:r + 1], b.k[r:r + 1]), pos)
            hist_k[r] = torch.cat([hist_k[r], k])
            hist_v[r] = torch.cat([hist_v[r], b.v[r:r + 1].double().cpu()])
            if step % 5 and step != 19:
                continue
            n = len(hist_k[r])
            full_q = torch.zeros((n, b.hq, b.d), dtype=torch.float64)
            full_q[-1] = q[0]
            want, mag = po.prompt(full_q, hist_k[r], hist_v[r], [n], b.scale)
            tol = po.prompt_tolerance(want[-1], mag[-1]) + 0.05 * mag[-1]
            assert po.worst(got[r], want[-1], tol) <= 1.0, (step, r)
    assert pkv.pkv_read_status(b.status) == 0 and pkv.pkv_read_status(b.work) == 0
    assert po.as_lists(b.lens) == [n + 20 for n in lens]


def test_two_captured_steps_replayed_in_turn():
    """Two captured prompt steps of different lengths, replayed in turn with
    new inputs and lengths, give the eager calls' bits."""
    layers = [Layer(40, 300, 3), Layer(41, 64, 2)]
    lens = [[[100, 30, 170], [1, 299, 0], [64, 64, 64]], [[10, 54], [64, 0], [0, 5]]]
    graphs = []
    for a, n in zip(layers, lens):
        a.new.copy_(i32(n[0]))
        a.prefill()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.prefill()
        graphs.append(g)
    for step in range(3):
        for i, a in enumerate(layers):
            a.qkv.copy_(randn(gen_of(50 + step), *a.qkv.shape))
            results = []
            for how in (graphs[i].replay, a.prefill):
                a.new.copy_(i32(lens[i][step]))
                a.lens.zero_()
                a.cursor.zero_()
                a.table.fill_(-1)
                a.out.zero_()
                a.pool.zero_()
                how()
                torch.cuda.synchronize()
                results.append([x.clone() for x in (a.out, a.pool, a.table, a.lens, a.qsl, a.q_out)])
            for x, y in zip(*results):
                assert torch.equal(x, y)


def test_tables_go_straight_to_paged_attention():
    """Tables written by the kernel right before kernels that read them ahead
    of their own waits: 200 steps back to back, against steps with a
    synchronisation behind the tables."""
    outs = []
    for sync in (True, False):
        a = Layer(60, 8, 8, blocks=256)
        a.new.copy_(i32([1] * 8))
        got = []
        for _ in range(200):
            a.tables()
            if sync:
                torch.cuda.synchronize()
            _, qsl, _, slots, _ = a.tables.outputs
            pkv.paged_kv_write(a.k.contiguous(), a.v.contiguous(), slots, a.pool)
            got.append(pkv.paged_attention(a.q.contiguous(), a.pool, a.table, a.lens, qsl, a.scale, workspace=a.work))
        torch.cuda.synchronize()
        assert pkv.pkv_read_status(a.status) == 0 and pkv.pkv_read_status(a.work) == 0
        outs.append(torch.stack(got))
    assert torch.equal(outs[0], outs[1])
