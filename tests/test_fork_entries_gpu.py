"""paged_fork_tables on tables with entries outside the pool: passed on, neither
counted nor copied, and reported, in rows that end, go on once, or several times."""
import numpy as np
import pytest
import torch

from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def fork(parents, table, lens, shares, free, cursor, nb, width):
    """By the definition, entries outside the pool allowed."""
    shares, free = list(shares), list(free)
    inside = lambda b: 0 <= b < nb  # noqa: E731
    children = [[r for r, p in enumerate(parents) if p == q] for q in range(len(lens))]
    bad = False
    for q, n in enumerate(lens):
        bad |= any(not inside(b) for b in table[q][:-(-n // 16)])
        for b in table[q][:n // 16 if children[q] else -(-n // 16)]:
            if inside(b):
                shares[b] += len(children[q]) - 1
    gone = []
    for q, n in enumerate(lens):
        for b in table[q][:-(-n // 16)] if not children[q] else ():
            if inside(b) and shares[b] == -1:
                shares[b] = 0
                gone.append(b)
    cursor -= len(gone)
    free[cursor:cursor + len(gone)] = gone
    out, out_lens, src, dst = [], [], [], []
    for r, p in enumerate(parents):
        n = lens[p] if p >= 0 else 0
        line = list(table[p][:-(-n // 16)]) if p >= 0 else []
        s = d = -1
        if n % 16 and children[p][0] != r and inside(line[-1]):
            s, d = line[-1], free[cursor]
            line[-1] = d
            cursor += 1
        out.append(line + [-1] * (width - len(line)))
        out_lens.append(n)
        src.append(s)
        dst.append(d)
    return out, out_lens, shares, free, cursor, src, dst, bad


def check(parents, table, lens, nb, free, cursor, shares=None):
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)  # noqa: E731
    shares = shares or [0] * nb
    sh, fr, cur, st = i32(shares), i32(free), i32([cursor]), i32([0])
    got = pkv.paged_fork_tables(i32(parents), i32(table), i32(lens), sh, fr, cur, status=st)
    want = fork(parents, table, lens, shares, free, cursor, nb, len(table[0]))
    for g, w in zip((got[0], got[1], sh, fr, cur, got[2], got[3]), (*want[:4], [want[4]], *want[5:7])):
        assert g.cpu().tolist() == list(w)
    assert pkv.pkv_read_status(st) == (pkv.PKV_DEV_BAD_BLOCK if want[7] else 0)
    return want


BAD = [-1, 20, -2 ** 31, 2 ** 31 - 1]


@pytest.mark.parametrize("bad", BAD)
def test_the_partly_filled_entry_of_a_row_that_goes_on_twice(bad):
    """It stays as it is in all children, no block is taken for them and none of their copies is numbered."""
    table, free = [[3, 4, -1], [5, bad, -1], [7, 8, 9]], list(range(20))
    want = check([1, 1, 2], table, [20, 30, 40], 20, free, 12)
    assert [line[1] for line in want[0][:2]] == [bad, bad] and want[5] == [-1] * 3 and want[4] == 12 - 2
    want = check([1, 1, 1], table, [20, 30, 48], 20, free, 12)
    assert want[6] == [-1] * 3
    # beside rows whose copies are made: those take the blocks that they would without it
    want = check([1, 2, 1, 2, 1, 2], table + [[-1] * 3] * 3, [20, 30, 40, 0, 0, 0], 20, free, 12)
    assert want[6] == [-1, -1, -1, 3, -1, 4]


@pytest.mark.parametrize("rows", [33, 300, 1500])
def test_bad_entries_among_many_rows(rows):
    rng = np.random.default_rng(rows)
    width = 5
    lens = [int(x) for x in rng.integers(0, 16 * width + 1, rows)]
    held = [-(-n // 16) for n in lens]
    nb = sum(held) + rows + 10
    perm = [int(x) for x in rng.permutation(nb)]
    table, at = [], 0
    for h in held:
        table.append(perm[at:at + h] + [-1] * (width - h))
        at += h
    for r in rng.choice(rows, rows // 3, replace=False):
        if held[r]:
            e = held[r] - 1 if rng.random() < 0.6 else int(rng.integers(0, held[r]))
            table[r][e] = int(rng.choice([-1, nb, -2 ** 31, 2 ** 31 - 1]))
    parents = [-1 if rng.random() < 0.2 else int(rng.integers(0, rows)) for _ in range(rows)]
    want = check(parents, table, lens, nb, perm, at)
    assert want[7] and any(d >= 0 for d in want[6])


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("lens", [[20, 32, 40], [20, 30, 40]])
@pytest.mark.parametrize("parents", [[0, 1, 2], [0, 1, 0], [2, 0, 1], [1, -1, -1]])
def test_a_row_that_goes_on_once_is_looked_at_too(bad, lens, parents):
    """Entry 1 is a whole block or the partly filled one; the row goes on unchanged."""
    want = check(parents, [[3, 4, -1], [5, bad, -1], [7, 8, 9]], lens, 20, list(range(20)), 12)
    assert want[7] and want[0][parents.index(1)] == [5, bad, -1]


@pytest.mark.parametrize("bad", BAD)
def test_a_row_that_ends(bad):
    want = check([0, -1, 2], [[3, 4, -1], [5, bad, -1], [7, 8, 9]], [20, 32, 40], 20, list(range(20)), 12)
    assert want[7] and want[4] == 11 and want[3][11] == 5


def test_entries_behind_a_rows_length_are_not_looked_at():
    want = check([1, 1, 2], [[-7, 99, -1], [5, 50, -1], [7, -1, 9]], [0, 16, 16], 20, list(range(20)), 12)
    assert not want[7]
