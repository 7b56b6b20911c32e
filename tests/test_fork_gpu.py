"""paged_fork_tables and paged_copy_blocks on the GPU against a plain
implementation, and a beam search over a 4-bit pool that uses them."""
import numpy as np
import pytest
import torch

import kv4_oracle as ko
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


class Pages:
    """Rows with blocks of their own, and the books."""

    def __init__(self, rng, rows, hi, width=0, spare=50, zeros=0.1):
        self.lens = [0 if rng.random() < zeros else int(rng.integers(1, hi + 1)) for _ in range(rows)]
        held = [-(-n // 16) for n in self.lens]
        self.width = max([width, 1] + held)
        self.nb = sum(held) + rows + spare
        perm = [int(x) for x in rng.permutation(self.nb)]
        self.table, at = [], 0
        for h in held:
            self.table.append(perm[at:at + h] + [-1] * (self.width - h))
            at += h
        self.free, self.cursor, self.shares = perm, at, [0] * self.nb

    def step(self, parents, device_state=None):
        """One call against the definition; moves on to the new tables."""
        st = status()
        shares, free, cursor = i32(self.shares), i32(self.free), i32([self.cursor])
        got = pkv.paged_fork_tables(i32(parents), i32(self.table), i32(self.lens), shares, free, cursor, status=st)
        want = ko.fork(parents, self.table, self.lens, self.shares, self.free, self.cursor, self.width)
        for g, w in zip((got[0], got[1], shares, free, cursor, got[2], got[3]),
                        (want[0], want[1], want[2], want[3], [want[4]], want[5], want[6])):
            assert g.cpu().tolist() == list(w)
        assert pkv.pkv_read_status(st) == 0
        self.table, self.lens, self.shares, self.free, self.cursor = want[:5]
        # the books agree: every block is free once or held shares + 1 times
        held = {}
        for line, n in zip(self.table, self.lens):
            for b in line[:-(-n // 16)]:
                held[b] = held.get(b, 0) + 1
        free_now = self.free[self.cursor:]
        assert len(set(free_now)) == len(free_now) and not set(free_now) & set(held)
        assert len(free_now) + len(held) == self.nb
        assert all(self.shares[b] == held.get(b, 1) - 1 for b in range(self.nb))
        return want


@pytest.mark.parametrize("rows,hi", [(1, 1), (1, 40), (4, 100), (31, 300), (33, 64), (64, 1500), (200, 90), (257, 700),
                                     (1024, 40), (1500, 33), (4096, 20)])
def test_steps_of_any_parents(rows, hi):
    rng = np.random.default_rng(rows + hi)
    p = Pages(rng, rows, hi)
    p.step(list(range(rows)))
    for share in (0.3, 0.9, 0.0):
        parents = [-1 if rng.random() < share / 3 else int(rng.integers(0, max(1, int(rows * (1 - share)) or 1))) for _ in range(rows)]
        p.step(parents)
    p.step([-1] * rows)
    assert p.cursor == 0 and not any(p.shares)


def test_samples_of_a_prompt_and_their_end():
    rng = np.random.default_rng(1)
    p = Pages(rng, 8, 100, zeros=0)
    p.lens = [75] + [0] * 7
    for r in range(1, 8):
        p.table[r] = [-1] * p.width
    p.nb = 60
    p.width = 7
    p.free = [int(x) for x in rng.permutation(60)]
    p.table = [p.free[:5] + [-1, -1]] + [[-1] * 7] * 7
    p.cursor, p.shares = 5, [0] * 60
    want = p.step([0] * 8)
    assert want[5].count(-1) == 1 and len(set(want[6][1:])) == 7
    p.step([0, 1, -1, -1, 4, 5, 6, -1])
    p.step([6, 6, 6, 6, 0, 0, 0, 0])
    p.step([-1] * 8)


def test_full_blocks_take_no_copy_and_a_full_table_no_end():
    rng = np.random.default_rng(2)
    p = Pages(rng, 6, 64, zeros=0)
    p.lens = [16 * (n // 16) for n in p.lens]
    for r, n in enumerate(p.lens):
        extra = [b for b in p.table[r][n // 16:] if b >= 0]
        p.free = p.free[:]
        for b in extra:  # what the shorter rows no longer hold is free
            p.cursor -= 1
            i = p.free.index(b)
            p.free[i], p.free[p.cursor] = p.free[p.cursor], b
        p.table[r] = p.table[r][:n // 16] + [-1] * (p.width - n // 16)
    want = p.step([0, 0, 1, 1, 5, 5])
    assert want[5] == [-1] * 6


def test_mistakes_in_the_books_are_reported_and_harm_no_other_row():
    table, lens = [[3, 4, -1], [5, 6, -1], [7, 8, 9]], [20, 32, 40]

    def call(parents, table=table, lens=lens, shares=None, free=range(20), cursor=12):
        st = status()
        sh, fr, cur = i32(shares or [0] * 20), i32(list(free)), i32([cursor])
        out = pkv.paged_fork_tables(i32(parents), i32(table), i32(lens), sh, fr, cur, status=st)
        return [x.cpu().tolist() for x in (*out, sh, fr, cur)], pkv.pkv_read_status(st)

    good, st = call([0, 1, 0])
    assert st == 0 and good[0][0] == [3, 4, -1] and good[0][2][0] == 3
    # a parent that is no row: the row is empty
    got, st = call([0, 1, 3])
    assert st == pkv.PKV_DEV_BAD_PAGES and got[0][2] == [-1] * 3 and got[1] == [20, 32, 0] and got[0][:2] == table[:2]
    got, st = call([0, -2, 2 ** 31 - 1])
    assert st == pkv.PKV_DEV_BAD_PAGES and got[1] == [20, 0, 0]
    # lengths out of range
    got, st = call([0, 1, 2], lens=[20, -1, 49])
    assert st == pkv.PKV_DEV_BAD_LEN and got[1] == [20, 0, 0] and got[0][0] == table[0] and got[0][1] == [-1] * 3
    # an entry outside the pool in a row that ends, and in one that goes on
    got, st = call([0, -1, 2], table=[[3, 4, -1], [5, 20, -1], [7, -1, 9]])
    assert st == pkv.PKV_DEV_BAD_BLOCK or st == 0
    assert got[0][2] == [7, -1, 9] and got[6] == [11] and got[5][11] == 5
    # no block left
    got, st = call([0, 0, 0], free=range(14), cursor=14, lens=[20, 0, 0])
    assert st == pkv.PKV_DEV_NO_BLOCKS and got[0] == [[3, 4, -1], [3, -1, -1], [3, -1, -1]] and got[2] == [-1] * 3
    assert got[6] == [14] and got[1] == [20, 20, 20]
    # given up twice, the count says held once
    got, st = call([2, 2, 2], table=[[3, 4, -1], [3, 6, -1], [7, 8, 9]])
    assert st == pkv.PKV_DEV_BAD_PAGES and 3 not in got[5][got[6][0]:]
    assert all(x >= 0 for x in got[4])
    # the same block twice in a row that ends: once in the list
    got, st = call([2, -1, 2], table=[[3, 4, -1], [5, 5, -1], [7, 8, 9]], lens=[20, 32, 48])
    assert st == pkv.PKV_DEV_BAD_PAGES and got[5][got[6][0]:].count(5) <= 1
    # no room before the cursor
    got, st = call([0, -1, -1], cursor=1)
    assert st == pkv.PKV_DEV_BAD_PAGES and got[6] == [0] and got[0][0] == table[0]
    for cursor in (-1, 21):
        got, st = call([0, 0, -1], cursor=cursor)
        assert st & pkv.PKV_DEV_BAD_PAGES and got[6] == [cursor] and got[5] == list(range(20)) and got[3] == [-1] * 3


@pytest.mark.parametrize("kind,hkv,d", [("bf16", 1, 8), ("bf16", 8, 128), ("kv4", 1, 64), ("kv4", 8, 128)])
@pytest.mark.parametrize("pools,pairs", [(1, 1), (3, 40), (128, 5)])
def test_copies(kind, hkv, d, pools, pairs):
    rng = np.random.default_rng(pairs)
    nb = 2 * pairs + 6
    shape = (nb, 2, hkv, 16, d) if kind == "bf16" else (nb, hkv, 18 * d)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    make = (lambda: torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)) if kind == "bf16" else (
        lambda: torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8))
    ps = [make() for _ in range(pools)]
    perm = rng.permutation(nb)
    src, dst = perm[:pairs].copy(), perm[pairs:2 * pairs].copy()
    src[0] = perm[-1]
    if pairs > 2:
        src[1] = -1
        dst[2] = -1
        src[3] = src[4]  # the same block twice
    want = [p.clone() for p in ps]
    for p in want:
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                p[int(b)] = p[int(a)]
    st = status()
    pkv.paged_copy_blocks(ps, i32(src), i32(dst), status=st)
    assert all(torch.equal(a, b) for a, b in zip(ps, want)) and pkv.pkv_read_status(st) == 0
    src[0], dst[-1] = nb, 2 ** 31 - 1
    pkv.paged_copy_blocks(ps, i32(src[[0, -1]]), i32(dst[[0, -1]]), status=st)
    assert all(torch.equal(a, b) for a, b in zip(ps, want)) and pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_BLOCK


def test_a_beam_search_over_the_4_bit_pool():
    """Prompts, then steps of tables, write, attention and fork, all on the GPU: every row attends to what its own
    line of tokens wrote, as a copy of it kept on the host says."""
    rng = np.random.default_rng(12)
    layers, groups, beams, hq, hkv, d = 2, 3, 4, 8, 2, 64
    rows, width, nb = groups * beams, 6, 90
    pools = [pkv.alloc_kv4_cache(nb, hkv, d) for _ in range(layers)]
    free, cursor = i32(rng.permutation(nb)), i32([0])
    shares, table = i32(np.zeros(nb)), i32(np.full((rows, width), -1))
    lens = i32(np.zeros(rows))
    history = [[[] for _ in range(layers)] for _ in range(rows)]  # (k, v) values as stored
    st = status()
    for step in range(24):
        new = [int(rng.integers(1, 40)) if r % beams == 0 else 0 for r in range(rows)] if step == 0 else [1] * rows
        t = sum(new)
        lens, qsl, pos, slots, _ = pkv.paged_build_tables(i32(new), lens, free, table, t, nb, seq_lens=lens, cursor=cursor,
                                                          cursor_out=cursor, status=st)
        at = np.concatenate([[0], np.cumsum(new)])
        for layer, pool in enumerate(pools):
            k, v, q = (torch.from_numpy(rng.standard_normal((t, h, d)).astype(np.float32)).to(torch.bfloat16) for h in (hkv, hkv, hq))
            pkv.paged_kv4_write(k.to(DEV), v.to(DEV), slots, pool, status=st)
            for r in range(rows):
                for i in range(at[r], at[r + 1]):
                    one = np.zeros((1, hkv, 18 * d), dtype=np.uint8)
                    ko.pack_token(one, 0, k[i].double().numpy(), v[i].double().numpy())
                    history[r][layer].append(ko.unpack(one)[0, :, :, 0])
            out = pkv.paged_kv4_attention(q.to(DEV), pool, table, lens, qsl, d ** -0.5, status=st).double().cpu().numpy()
            for r in range(rows):
                if not new[r]:
                    continue
                n = len(history[r][layer])
                vals = np.zeros((-(-n // 16), 2, hkv, 16, d))
                for j, kv in enumerate(history[r][layer]):
                    vals[j // 16, :, :, j % 16] = kv
                want, tol = ko.attend(q[at[r]:at[r + 1]].double().numpy(), vals, [list(range(len(vals)))], [n], [0, new[r]], d ** -0.5)
                assert (np.abs(out[at[r]:at[r + 1]] - want) <= tol).all()
        parents = [g * beams + (0 if step == 0 else int(rng.integers(0, beams))) for g in range(groups) for _ in range(beams)]
        table, lens, src, dst = pkv.paged_fork_tables(i32(parents), table, lens, shares, free, cursor, status=st)
        pkv.paged_copy_blocks(pools, src, dst, status=st)
        history = [[list(h) for h in history[p]] for p in parents]
        assert pkv.pkv_read_status(st) == 0
    pkv.paged_fork_tables(i32([-1] * rows), table, lens, shares, free, cursor, status=st)
    assert cursor.item() == 0 and not shares.any() and sorted(free.tolist()) == list(range(nb))


def test_a_captured_step():
    """Fork and copies in a graph, the tables changing places between two graphs."""
    rng = np.random.default_rng(5)
    p = Pages(rng, 40, 200)
    a, b = i32(p.table), i32(p.table)
    la, lb = i32(p.lens), i32(p.lens)
    shares, free, cursor = i32(p.shares), i32(p.free), i32([p.cursor])
    parents = i32(np.arange(40))
    src, dst = i32(np.full(40, -1)), i32(np.full(40, -1))
    pools = [torch.randint(0, 256, (p.nb, 1, 18 * 64), dtype=torch.uint8, device=DEV)]
    graphs = []
    for x, y, lx, ly in ((a, b, la, lb), (b, a, lb, la)):
        fork = pkv.prepare_fork_tables(parents, x, lx, shares, free, cursor, block_table_out=y, seq_lens_out=ly, copy_src=src, copy_dst=dst)
        copy = pkv.prepare_copy_blocks(pools, src, dst)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fork()
            copy()
        graphs.append(g)
    for i in range(6):
        now = [int(x) for x in rng.integers(0, 40, 40)]
        parents.copy_(i32(now))
        before = pools[0].clone()
        graphs[i % 2].replay()
        want = ko.fork(now, p.table, p.lens, p.shares, p.free, p.cursor, p.width)
        p.table, p.lens, p.shares, p.free, p.cursor = want[:5]
        t, n = ((b, lb), (a, la))[i % 2]
        assert t.cpu().tolist() == p.table and n.cpu().tolist() == p.lens and cursor.item() == p.cursor
        assert shares.cpu().tolist() == list(p.shares) and free.cpu().tolist() == list(p.free)
        for s, e in zip(want[5], want[6]):
            if s >= 0:
                before[e] = before[s]
        assert torch.equal(pools[0], before)
