"""How attention over the 4-bit pool cuts a batch into shares (kv4_plan.h): on
the host, every block of every item in exactly one share, and every cut item's
partials counted."""
import os
import random
import subprocess

import pytest

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "kv4_plan.h"
using namespace pkv;
// in: reqs group heads rows ctas warps, then (n, len) of each. Walks every share as a warp of the kernel does.
int main() {
    int R, group, heads, rows, ctas, warps;
    while (scanf("%d %d %d %d %d %d", &R, &group, &heads, &rows, &ctas, &warps) == 6) {
        std::vector<Kv4Request> q(R);
        std::vector<long long> first(R + 1, 0);
        int q0 = 0;
        for (int r = 0; r < R; ++r) {
            int n, len;
            if (scanf("%d %d", &n, &len) != 2) return 1;
            q[r] = kv4_request(q0, n, len, group, rows);
            q0 += n;
            first[r + 1] = first[r] + kv4_cost(q[r], heads, q[r].tiles);
        }
        const long long total = first[R];
        const Kv4Shares sh = kv4_shares(total, ctas, warps, kv4_least(rows), R, heads);
        if (sh.per_cta > warps || (long long)sh.per_cta * ctas < sh.count) { printf("%d shares, %d a CTA\n", sh.count, sh.per_cta); return 1; }
        // next block expected of each item, and its pieces: seen, told by the first, told by the others
        std::vector<std::vector<int>> next(R), seen(R), told(R);
        for (int r = 0; r < R; ++r) next[r].assign(q[r].tiles * heads, 0), seen[r].assign(q[r].tiles * heads, 0), told[r].assign(q[r].tiles * heads, -1);
        for (int k = 0; k < sh.count; ++k) {
            const long long from = sh.begin(k), to = sh.begin(k + 1);
            if (!(from < to)) { printf("empty share %d\n", k); return 1; }
            int r = 0;
            while (first[r + 1] <= from) ++r;
            int i, h, pieces = 0;
            bool ended = false;
            long long start;
            kv4_locate(q[r], heads, from - first[r], &i, &h, &start);
            start += first[r];
            while (true) {
                const Kv4Tiling tl = kv4_tile(q[r], i, group, rows);
                const long long cost = kv4_item_cost(q[r], i), stop = start + cost;
                if (!(start <= from || start < to) || stop <= from || tl.rows < 1 || tl.keys < 1 || tl.keys > q[r].len) { printf("bad item\n"); return 1; }
                const Kv4Piece p = kv4_piece(sh, k, start, cost, tl.blocks);
                if (p.b0 < p.b1) {
                    int &n = next[r][i * heads + h];
                    if (p.b0 != n || p.b1 > tl.blocks) { printf("blocks %d..%d, %d next\n", p.b0, p.b1, n); return 1; }
                    n = p.b1;
                    if (p.begun != (p.b0 > 0) || p.cut != (p.b1 < tl.blocks) || ended || (p.begun && pieces)) { printf("order\n"); return 1; }
                    if (p.begun || p.cut) {
                        const int held = p.last - p.first + 1;
                        int &m = told[r][i * heads + h], &at = seen[r][i * heads + h];
                        if (m < 0) m = held;
                        if (held != m || p.first + at != k || (p.cut && (tl.blocks < 4 || p.b1 - p.b0 < 2))) { printf("shares %d..%d, %d of %d seen by %d\n", p.first, p.last, at, m, k); return 1; }
                        ++at;
                    }
                    ended = p.cut;
                    ++pieces;
                } else if (p.b0 > p.b1 || (p.begun && p.cut)) { printf("empty piece\n"); return 1; }
                if (p.more != (stop < to)) { printf("more\n"); return 1; }
                if (!p.more) break;
                start = stop;
                if (++h == heads) {
                    h = 0;
                    if (++i == q[r].tiles) {
                        i = 0;
                        do ++r; while (q[r].tiles == 0);
                    }
                }
            }
        }
        for (int r = 0; r < R; ++r)
            for (int i = 0; i < q[r].tiles; ++i)
                for (int h = 0; h < heads; ++h) {
                    const int k = i * heads + h, blocks = kv4_tile(q[r], i, group, rows).blocks;
                    if (next[r][k] != blocks) { printf("r %d i %d h %d: %d of %d blocks\n", r, i, h, next[r][k], blocks); return 1; }
                    if (seen[r][k] != (told[r][k] < 0 ? 0 : told[r][k])) { printf("partials %d, told %d\n", seen[r][k], told[r][k]); return 1; }
                }
        printf("ok %d\n", sh.count);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv4_plan")
    (d / "plan.cpp").write_text(PROGRAM)
    exe = str(d / "plan")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(REPO, "paged_attention_kv_gb300", "csrc"), str(d / "plan.cpp"), "-o", exe], check=True)
    return exe


def walk(program, batches):
    text = "\n".join(" ".join(map(str, [len(reqs), *head] + [x for r in reqs for x in r])) for head, reqs in batches)
    res = subprocess.run([program], input=text, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout[-500:]
    lines = res.stdout.split("\n")[:-1]
    assert len(lines) == len(batches) and all(x.startswith("ok") for x in lines)
    return [int(x.split()[1]) for x in lines]


def test_named_batches(program):
    counts = walk(program, [
        ((8, 4, 8, 152, 12), [(1, 17), (1, 40)]),
        ((4, 8, 8, 152, 12), [(1, 1)]),
        ((4, 8, 32, 152, 8), [(0, 0), (512, 512), (0, 5), (1, 2_000_000), (300, 301), (0, 0)]),
        ((128, 1, 32, 152, 8), [(3, 90)] * 40),
        ((3, 5, 8, 152, 12), [(7, 1000)] * 9),
        ((4, 8, 8, 152, 12), [(1, 3000)] * 256),
        ((4, 8, 8, 152, 12), []), ((4, 8, 8, 152, 12), [(0, 0)] * 7)])
    assert counts[-2:] == [0, 0] and counts[5] == 1824


def test_random_batches(program):
    rng = random.Random(4)
    batches = []
    for _ in range(1500):
        rows = rng.choice((8, 16, 32))
        reqs = []
        for _ in range(rng.randint(1, 40)):
            n = rng.choice((0, 1, 1, rng.randint(1, 9), rng.randint(1, 400)))
            reqs.append((n, n + rng.choice((0, 0, rng.randint(0, 50), rng.randint(0, 5000)))))
        batches.append(((rng.choice((1, 2, 3, 4, 5, 8, 16, 33, 128)), rng.randint(1, 8), rows, *rng.choice(((1, 1), (7, 1), (3, 5), (152, 8), (152, 12)))), reqs))
    walk(program, batches)


def test_parts_of_a_chunk_item(tmp_path):
    """Every key tile in one part, four in each at least, and no more pieces than CTAs."""
    (tmp_path / "parts.cpp").write_text(r"""
#include <cstdio>
#include "kv4_plan.h"
using namespace pkv;
int main() {
    const int some[] = {1, 2, 5, 152};
    for (int sms : some)
        for (long long items = 0; items < 700; ++items) {
            const Kv4Splits sp = kv4_splits(items, sms);
            if (sp.count < 1 || sp.count > kKv4MaxSplits || (sp.count > 1 && (sp.count * items > 2 * sms || items > sms))) return 1;
            for (int tiles = 1; tiles < 600; tiles += 1 + tiles / 50) {
                const int parts = kv4_parts(tiles, sp);
                if (parts < 1 || parts > sp.count || kv4_part_begin(tiles, parts, 0) != 0 || kv4_part_begin(tiles, parts, parts) != tiles) return 2;
                for (int s = 0; parts > 1 && s < parts; ++s)
                    if (kv4_part_begin(tiles, parts, s + 1) - kv4_part_begin(tiles, parts, s) < 4) return 3;
            }
        }
    return kv4_splits(1LL << 40, 152).count == 1 && kv4_part_begin(1 << 24, 8, 8) == 1 << 24 ? 0 : 4;
}
""")
    exe = str(tmp_path / "parts")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(REPO, "paged_attention_kv_gb300", "csrc"), str(tmp_path / "parts.cpp"), "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0
