"""pkv_prompt_attention's running reference: scores of any finite size, and
outputs and sums that follow the reference when it moves."""
import numpy as np
import pytest
import torch

import prompt_oracle as po
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"
TILE = 128  # keys of a tile


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def gen_of(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)


def bounds(lens, many):
    """Query starts; ``many``: with empty sequences behind, for the kernel's
    form for many items, where a few have their keys split."""
    return i32(np.concatenate([[0], np.cumsum(lens), np.full(200 if many else 0, sum(lens))]).astype(int).tolist())


def run(q, k, v, lens, scale, many):
    status = i32([0])
    got = pkv.pkv_prompt_attention(q, k, v, bounds(lens, many), scale, status=status)
    assert pkv.pkv_read_status(status) == 0
    return got


@pytest.mark.parametrize("scale", [1e4, 3e8, 1e9, 1e20, 1e30])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_finite_scores_of_any_size(d, many, sign, scale):
    """q and k are small whole numbers, so that the products are exact and a
    row's largest score stands alone or in exact ties (the next is below it by
    at least the scale, and weighs exp(-1e4) at most): the output is the mean
    of the tied values, whatever the scale and the scores' sign."""
    gen, lens = gen_of(d + sign), [1, 2, 200, 420]
    t = sum(lens)
    q = torch.randint(1, 4, (t, 4, d), generator=gen, device=DEV).to(torch.bfloat16)
    k = (sign * torch.randint(1, 4, (t, 2, d), generator=gen, device=DEV)).to(torch.bfloat16)
    v = randn(gen, t, 2, d)
    got = run(q, k, v, lens, scale, many)
    want, mag = po.prompt(q, k, v, lens, scale)
    assert po.worst(got, want, po.prompt_tolerance(want, mag)) <= 1.0


@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-30])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("many", [False, True])
def test_scales_that_leave_no_difference(d, many, scale):
    """Every visible key weighs the same: the mean of the values seen."""
    gen, lens = gen_of(d), [3, 300]
    q, k, v = randn(gen, 303, 4, d), randn(gen, 303, 2, d), randn(gen, 303, 2, d)
    got = run(q, k, v, lens, scale, many)
    want, mag = po.prompt(q, k, v, lens, scale)
    assert po.worst(got, want, po.prompt_tolerance(want, mag)) <= 1.0


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [70, 200, 290])
@pytest.mark.parametrize("power", [36, 60])
def test_one_token_with_huge_scores(power, at, many, d):
    """A query 2^36 or 2^60 times its neighbours' takes the value of its largest
    key, and no bit of the other tokens' outputs changes."""
    gen, lens = gen_of(power + at), [300]
    q, k, v = randn(gen, 300, 4, d), randn(gen, 300, 1, d), randn(gen, 300, 1, d)
    before = run(q, k, v, lens, d ** -0.5, many).clone()
    q[at] *= 2.0 ** power
    after = run(q, k, v, lens, d ** -0.5, many)
    same = [i for i in range(300) if i != at]
    assert torch.equal(before[same], after[same])
    s = torch.einsum("hd,kd->hk", q[at].double(), k[:at + 1, 0].double())
    top = torch.topk(s, 2, dim=1).values
    # a sum of D products in 32 bits is off by D 2^-24 of their magnitudes at
    # most: the largest stands clear of that
    size = torch.einsum("hd,kd->hk", q[at].double().abs(), k[:at + 1, 0].double().abs()).amax(1)
    assert bool((top[:, 0] - top[:, 1] > 2 * d * 2.0 ** -24 * size).all())
    assert torch.equal(after[at], v[s.argmax(1), 0])


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_the_reference_moves_in_every_tile(d, many):
    """Each key tile's scores lie about 16 bits above the tile before, past the
    14 that move the reference, and its values 2^14 below: a row's output is
    made of several tiles, so that O and the sum have to follow every move, in
    tiles with masked keys and without."""
    gen, lens = gen_of(d), [5 * TILE, 300]
    t = sum(lens)
    tile = torch.cat([torch.arange(n, device=DEV) // TILE for n in lens])
    level = 11.0 * tile + 0.25 * torch.randint(0, 3, (t,), generator=gen, device=DEV)
    q = torch.ones(t, 4, d, device=DEV, dtype=torch.bfloat16)
    k = level[:, None, None].expand(t, 2, d).to(torch.bfloat16).contiguous()
    v = (randn(gen, t, 2, d).double() * 2.0 ** (-14.0 * tile)[:, None, None]).to(torch.bfloat16)
    # what makes the test one: the tiles' maxima, in bits, as the kernel sees them
    score = k[:, 0, 0].double() * np.log2(np.e)
    for n in (1, 2, 3, 4):
        assert 14.5 < float(score[n * TILE:(n + 1) * TILE].min() - score[(n - 1) * TILE:n * TILE].max())
    got = run(q, k, v, lens, 1.0 / d, many)
    want, mag = po.prompt(q, k, v, lens, 1.0 / d)
    # scores are exact, up to 45 * log2(e) = 65; their product with the scale
    # is off by 2^-24 of that, under 2^-17, as the tolerance's 2^-11 covers
    assert po.worst(got, want, po.prompt_tolerance(want, mag)) <= 1.0
    # and the old tiles show: the tile before the last weighs 2^-16 of it with
    # values 2^14 as large, a quarter of a mean of 128 normal values, 0.022 by
    # its deviation in the last tile's units, against a tolerance of about 0.005
    last = slice(5 * TILE - 8, 5 * TILE)
    s = torch.softmax(q[last, 0].double() @ k[4 * TILE:5 * TILE, 0].double().T / d, -1)
    alone = s @ v[4 * TILE:5 * TILE, 0].double()
    assert bool(((alone - want[last, 0]).abs() > 2 * po.prompt_tolerance(want, mag)[last, 0]).double().mean() > 0.5)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("base", [2 ** 22, -2 ** 22])
def test_the_reference_moves_far_from_zero(base, d, many):
    """As above, 17 bits a tile, on top of a common score of 2^22. All scores are
    whole numbers below 2^23, exact in 32 bits; scaled to base 2 a reference is
    rounded by up to 2^-2, which must be the same wherever it is used (the error
    would be a factor of 2^(1/4) between the tiles)."""
    gen, lens = gen_of(d), [5 * TILE, 300]
    t = sum(lens)
    tile = torch.cat([torch.arange(n, device=DEV) // TILE for n in lens])
    level = 12 * tile + torch.randint(0, 2, (t,), generator=gen, device=DEV)
    q, k = torch.zeros(2, t, 4, d, device=DEV, dtype=torch.bfloat16)
    k = k[:, :2].contiguous()
    q[..., 0], q[..., 1] = 2.0 ** 11, 1.0
    k[..., 0], k[..., 1] = base / 2.0 ** 11, level[:, None]
    v = (randn(gen, t, 2, d).double() * 2.0 ** (-16.0 * tile)[:, None, None]).to(torch.bfloat16)
    got = run(q, k, v, lens, 1.0, many)
    want, mag = po.prompt(q, k, v, lens, 1.0)
    assert po.worst(got, want, po.prompt_tolerance(want, mag)) <= 1.0


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [290, 200])
@pytest.mark.parametrize("bits", [15.0, 17.0])
def test_one_row_that_moves_its_reference_keeps_its_old_keys(bits, at, many, d):
    """The key before token ``at`` scores 15 or 17 bits above the rest for that
    token, in a tile with masked keys; the keys before it have values 2^12 times
    as large, so that they weigh in."""
    gen, lens = gen_of(at), [300]
    q, k, v = randn(gen, 300, 4, d) * 0.01, randn(gen, 300, 1, d) * 0.01, randn(gen, 300, 1, d)
    v[:TILE] *= 2.0 ** 12
    k[at - 1] = 1.0
    q[at] = bits * np.log(2) * d ** -0.5
    got = run(q, k, v, lens, d ** -0.5, many)
    want, mag = po.prompt(q, k, v, lens, d ** -0.5)
    s = torch.einsum("hd,kd->hk", q[at].double(), k[:at + 1, 0].double()) * d ** -0.5 * np.log2(np.e)
    moved = s[:, at - 1] - s[:, :TILE].amax(1)
    assert bool((moved > 14.2).all()) and bool((moved < 18).all())
    assert po.worst(got[at], want[at], po.prompt_tolerance(want, mag)[at]) <= 1.0


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("local", [0, 70, 140])
def test_an_infinite_column_of_k_gives_scores_of_both_infinities(local, bad, d, many):
    """One column of a key is infinite: a row that sees it has a score of plus
    or minus infinity by its own sign there, and is not a number, or leaves the
    key out."""
    lens = [150, 200, 90]
    gen, at = gen_of(15), 150 + local
    q, k, v = randn(gen, 440, 4, d), randn(gen, 440, 1, d), randn(gen, 440, 1, d)
    k[at, 0, 5] = bad
    assert bool((q[..., 5] != 0).all())
    want, mag = po.prompt(q, k, v, lens, d ** -0.5)
    got = run(q, k, v, lens, d ** -0.5, many)
    ok = torch.isfinite(want)
    sees = slice(at, 350)
    assert bool(ok[sees].any()) and not bool(ok[sees].all()) and bool(torch.isnan(want[~ok]).all())
    assert torch.equal(torch.isnan(got), ~ok)
    assert po.worst(got[ok], want[ok], po.prompt_tolerance(want, mag)[ok]) <= 1.0
