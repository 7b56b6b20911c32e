"""paged_kv4_write, paged_kv4_read and paged_kv4_attention on the GPU against
plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import kv4_oracle as ko
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bf16(rng, *shape, by=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * by).astype(np.float32)).to(torch.bfloat16)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# writing and reading back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,hkv,d", [(1, 1, 64), (1, 1, 128), (7, 4, 64), (64, 4, 64), (33, 8, 128), (50, 3, 128),
                                          (300, 2, 64), (129, 1, 128), (5, 33, 64)])
def test_write_and_read_are_the_definition(tokens, hkv, d):
    rng = np.random.default_rng(tokens * 31 + hkv)
    nb = tokens // 8 + 4
    k, v = bf16(rng, tokens, hkv, d), bf16(rng, tokens, hkv, d, by=0.01)
    # groups of zeros, of equal values, of one large value, of values on ties and near the smallest scale
    k[0, 0, :16] = 0
    v[0, 0, :16] = -0.0
    k[-1, -1, -16:] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0.])
    v[-1, 0, :16] = torch.linspace(-1, 1, 16) * 2.0 ** -9 * 0.125
    slots = rng.permutation(nb * 16)[:tokens].astype(np.int32)
    slots[tokens // 2] = -1 if tokens > 1 else slots[0]
    pool = torch.from_numpy(rng.integers(0, 256, (nb, hkv, 18 * d), dtype=np.uint8))
    want = pool.numpy().copy()
    for t, s in enumerate(slots):
        if s >= 0:
            ko.pack_token(want, s, k[t].double().numpy(), v[t].double().numpy(), 1.0, 0.125)
    got, st = pool.to(DEV), status()
    pkv.paged_kv4_write(k.to(DEV), v.to(DEV), i32(slots), got, v_scale=0.125, status=st)
    assert np.array_equal(got.cpu().numpy(), want)
    ko_, vo_ = pkv.paged_kv4_read(got, i32(slots), v_scale=0.125, status=st)
    vals = ko.unpack(want)
    for t, s in enumerate(slots):
        if s >= 0:
            assert np.array_equal(ko_[t].double().cpu().numpy(), vals[s // 16, 0, :, s % 16], equal_nan=True)
            assert np.array_equal(vo_[t].double().cpu().numpy(), vals[s // 16, 1, :, s % 16] * 0.125, equal_nan=True)
        else:
            assert not ko_[t].any() and not vo_[t].any()
    assert pkv.pkv_read_status(st) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_every_bf16_magnitude_rounds_as_defined(d):
    """All positive bf16 values against a scale set by a group's largest, both signs."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16)
    rng = np.random.default_rng(d)
    tops = torch.from_numpy(rng.choice(np.array([1.0, 6.0, 0.09, 2688.0, 3.3, 448.0, 1e-3, 5.9, 7.1], np.float32), 2200)).to(torch.bfloat16)
    rows = -(-len(x) // 15)
    g = torch.zeros(rows, 16, dtype=torch.bfloat16)
    g[:, 0] = tops[:rows]
    flat = torch.zeros(rows * 15, dtype=torch.bfloat16)
    flat[:len(x)] = x[torch.from_numpy(rng.permutation(len(x)))]
    g[:, 1:] = flat.view(rows, 15)
    g *= torch.from_numpy(rng.choice([-1.0, 1.0], (rows, 16))).to(torch.bfloat16)
    n = rows // (d // 16)
    k = g[:n * (d // 16)].reshape(n, 1, d)
    pool = torch.zeros((n // 16 + 1, 1, 18 * d), dtype=torch.uint8)
    want = pool.numpy().copy()
    for t in range(n):
        ko.pack_token(want, t, k[t].double().numpy(), k[t].double().numpy(), 1.0, 2.0 ** 30)
    got = pool.to(DEV)
    pkv.paged_kv4_write(k.to(DEV), k.to(DEV), i32(np.arange(n)), got, v_scale=2.0 ** 30)
    assert np.array_equal(got.cpu().numpy(), want)


def test_values_that_are_not_finite():
    k = torch.ones(2, 1, 64, dtype=torch.bfloat16)
    k[0, 0, 3] = float("inf")
    k[0, 0, 20] = float("-inf")
    k[1, 0, 40] = float("nan")
    pool = torch.zeros((1, 1, 18 * 64), dtype=torch.uint8, device=DEV)
    pkv.paged_kv4_write(k.to(DEV), torch.ones_like(k).to(DEV), i32([4, 9]), pool)
    a, b = pkv.paged_kv4_read(pool, i32([4, 9]))
    a, b = a.cpu(), b.cpu()
    one = 6 * 0.171875  # 1 / 6 = 0.16667 lies between the scales 0.15625 and 0.171875, nearer to the second
    assert a[0, 0, 3] == 2688 and a[0, 0, 20] == -2688 and (a[0, 0, 32:] == one).all() and torch.isfinite(a[0]).all()
    assert torch.isnan(a[1, 0, 32:48]).all() and (a[1, 0, :32] == one).all() and (a[1, 0, 48:] == one).all()
    assert (b == one).all()


def test_slices_of_a_projection_bad_slots_and_repeated_reads():
    rng = np.random.default_rng(3)
    rows = bf16(rng, 40, 4 * 128 + 2 * 2 * 128).to(DEV)
    _, k, v = rows.split([512, 256, 256], dim=1)
    k, v = k.unflatten(1, (2, 128)), v.unflatten(1, (2, 128))
    one, two, st = (torch.zeros((3, 2, 18 * 128), dtype=torch.uint8, device=DEV) for _ in range(3))
    st = status()
    pkv.paged_kv4_write(k, v, i32(np.arange(40)), one)
    pkv.paged_kv4_write(k.contiguous(), v.contiguous(), i32(np.arange(40)), two, status=st)
    assert torch.equal(one, two) and pkv.pkv_read_status(st) == 0
    slots = np.arange(40)
    slots[[5, 6]] = [48, 2 ** 31 - 1]
    pkv.paged_kv4_write(v, k, i32(slots), two, status=st)
    assert pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_SLOT
    assert np.array_equal(ko.unpack(two.cpu().numpy())[0, :, :, 5], ko.unpack(one.cpu().numpy())[0, :, :, 5])
    st.zero_()
    a, _ = pkv.paged_kv4_read(one, i32([7, 7, -5, 48, 7]), status=st)
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[4]) and not a[2].any() and not a[3].any()
    assert pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_SLOT
    only = torch.full((40, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    got = pkv.paged_kv4_read(one, i32(np.arange(40)), v_out=only)
    assert got[0] is None and got[1] is only
    assert np.array_equal(only.double().cpu().numpy(), ko.unpack(one.cpu().numpy())[:, 1].transpose(0, 2, 1, 3).reshape(48, 2, 128)[:40])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Batch:
    """A pool of normal values whose unused rows and blocks hold NaN scales and random codes."""

    def __init__(self, seed, hq, hkv, d, lens, new, width=0, spread=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.lens, self.new = hq, hkv, d, list(lens), list(new)
        held = [-(-n // 16) for n in lens]
        nb = sum(held) + 5
        perm = rng.permutation(nb)
        width = max(width, max(held + [1]))
        self.table = np.full((len(lens), width), -1, dtype=np.int64)
        at = 0
        for r, h in enumerate(held):
            self.table[r, :h] = perm[at:at + h]
            at += h
        pool = rng.integers(0, 256, (nb, hkv, 18 * d), dtype=np.uint8)
        pool[..., 16 * d:] = 0x7f
        slots = [self.table[r, j // 16] * 16 + j % 16 for r, n in enumerate(lens) for j in range(n)]
        self.slots = np.array(slots, dtype=np.int64)
        t = len(slots)
        self.k, self.v = bf16(rng, t, hkv, d, by=spread), bf16(rng, t, hkv, d)
        self.pool = torch.from_numpy(pool).to(DEV)
        pkv.paged_kv4_write(self.k.to(DEV), self.v.to(DEV), i32(self.slots) if t else i32([0])[:0], self.pool)
        self.qsl = [0] + list(np.cumsum(new))
        self.q = bf16(rng, sum(new), hq, d)
        self.scale = d ** -0.5

    def tensors(self):
        return (self.q.to(DEV), self.pool, i32(self.table), i32(self.lens) if self.lens else i32([0])[:0], i32(self.qsl))

    def want(self, **kw):
        return ko.attend(self.q.double().numpy(), ko.unpack(self.pool.cpu().numpy()), self.table, self.lens, self.qsl,
                         self.scale, **kw)

    def check(self, out, **kw):
        want, tol = self.want(**kw)
        got = out.double().cpu().numpy()
        mine = ~np.isnan(tol)
        assert np.isfinite(got[mine]).all()
        worst = (np.abs(got - want) / tol)[mine].max() if mine.any() else 0.0
        assert worst <= 1.0, f"{worst:.3g} times the bound"


SHAPES = [(32, 4, 64), (32, 8, 128), (12, 4, 128), (8, 8, 64), (16, 2, 128), (4, 4, 128)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("lens", [[17, 40], [1], [16], [15, 16, 17, 1, 32, 33, 31], [700, 3, 129, 511, 64]])
def test_decode(hq, hkv, d, lens):
    b = Batch(len(lens) * 100 + d + hq, hq, hkv, d, lens, [1] * len(lens))
    for longest in (1, 0):
        st = status()
        b.check(pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=longest, status=st))
        assert pkv.pkv_read_status(st) == 0


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (6, 2, 64), (10, 2, 128), (64, 1, 64), (33, 1, 128), (128, 1, 128), (3, 1, 64)])
@pytest.mark.parametrize("lens,new", [([9, 40], [2, 4]), ([5, 20, 100, 1], [5, 0, 3, 1]), ([90, 77], [33, 77]),
                                      ([16, 32, 48, 64], [16, 16, 1, 48])])
def test_several_tokens_a_request(hq, hkv, d, lens, new):
    b = Batch(sum(lens) + hq, hq, hkv, d, lens, new)
    outs = [pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=m) for m in (max(new), 0, 1, 10 ** 6)]
    for o in outs:
        b.check(o)


@pytest.mark.parametrize("hq,hkv,d,lens,new", [
    (32, 8, 128, [3000], [1]), (8, 8, 64, [20000], [1]), (16, 2, 128, [9000, 5], [1, 1]), (8, 2, 128, [4000, 900, 1], [3, 200, 1]),
    (4, 1, 64, [6000], [40]), (4, 1, 128, [30000], [2])])
def test_contexts_cut_into_many_shares(hq, hkv, d, lens, new):
    b = Batch(sum(lens), hq, hkv, d, lens, new)
    b.check(pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=max(new)))
    b.check(pkv.paged_kv4_attention(*b.tensors(), b.scale))


@pytest.mark.parametrize("reqs", [130, 384, 385, 900])
def test_many_requests(reqs):
    rng = np.random.default_rng(reqs)
    lens = [int(x) for x in rng.integers(1, 90, reqs)]
    new = [int(min(n, rng.choice([0, 1, 1, 1, 2, 5]))) for n in lens]
    b = Batch(reqs, 8, 2, 64, lens, new)
    b.check(pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=max(new)))
    b.check(pkv.paged_kv4_attention(*b.tensors(), b.scale))


def test_scales_and_slices_and_one_workspace():
    b = Batch(5, 8, 2, 128, [300, 40, 7], [1, 6, 2])
    q, pool, table, lens, qsl = b.tensors()
    rows = torch.full((9, 8 * 128 + 64), 3.0, dtype=torch.bfloat16, device=DEV)
    rows[:, :1024] = q.flatten(1)
    sliced = rows[:, :1024].unflatten(1, (8, 128))
    ws = pkv.alloc_kv4_workspace(pool)
    outs = []
    for fill in (0, -1, 0x7fc000007fc00000):
        ws[200:].fill_(fill)  # what partials were there before does not matter, the counters in front do
        outs.append(pkv.paged_kv4_attention(sliced, pool, table, lens, qsl, b.scale, k_scale=0.25, v_scale=8.0, workspace=ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    b.check(outs[0], k_by=0.25, v_by=8.0)


def test_a_workspace_that_was_not_prepared_is_reported():
    b = Batch(5, 8, 2, 128, [9000, 4000], [1, 2])
    q, pool, table, lens, qsl = b.tensors()
    ws = pkv.alloc_kv4_workspace(pool)
    for fill in (0, -1, 5):
        st = status()
        pkv.paged_kv4_attention(q, pool, table, lens, qsl, b.scale, workspace=torch.full_like(ws, fill), status=st)
        assert pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_WORKSPACE
    st = status()
    for _ in range(3):
        b.check(pkv.paged_kv4_attention(q, pool, table, lens, qsl, b.scale, workspace=ws, status=st))
    assert pkv.pkv_read_status(st) == 0
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv4_attention(q, pool, table, lens, qsl, b.scale, workspace=ws[:-1])


def test_rows_of_no_request_and_requests_without_queries_are_left():
    b = Batch(6, 8, 2, 64, [30, 0, 20, 50], [2, 0, 0, 1])
    q, pool, table, lens, qsl = b.tensors()
    pad = torch.cat([q, torch.ones(4, 8, 64, dtype=torch.bfloat16, device=DEV)])
    out, st = torch.full_like(pad, 5.0), status()
    pkv.paged_kv4_attention(pad, pool, table, lens, qsl, b.scale, out=out, status=st)
    assert (out[3:] == 5).all()
    assert pkv.pkv_read_status(st) == 0
    b.check(out[:3])
    none = pkv.paged_kv4_attention(q[:0], pool, table[:0], lens[:0], qsl[:1], b.scale)
    assert none.shape == (0, 8, 64)


def test_bad_metadata_skips_its_request_only():
    b = Batch(7, 8, 2, 64, [40, 50, 60, 70], [1, 2, 3, 4])
    exact, tol = b.want()

    def right(out, t):  # a skipped request moves the cuts of the others, so their sums may have another order
        return (np.abs(out[t].double().cpu().numpy() - exact[t]) <= tol[t]).all()

    for lens, bit, rows in (([0, 50, 60, 70], pkv.PKV_DEV_BAD_LEN, range(0, 1)), ([40, 1, 60, 70], pkv.PKV_DEV_BAD_LEN, range(1, 3)),
                            ([40, 50, 60, 10 ** 6], pkv.PKV_DEV_BAD_LEN, range(6, 10)),
                            ([40, 50, -5, 2 ** 31 - 1], pkv.PKV_DEV_BAD_LEN, range(3, 10))):
        q, pool, table, _, qsl = b.tensors()
        out, st = torch.full_like(q, 9.0), status()
        pkv.paged_kv4_attention(q, pool, table, i32(lens), qsl, b.scale, out=out, status=st)
        assert pkv.pkv_read_status(st) == bit
        for t in range(10):
            assert (out[t] == 9).all() if t in rows else right(out, t)
    q, pool, table, lens, _ = b.tensors()
    out, st = torch.full_like(q, 9.0), status()
    pkv.paged_kv4_attention(q, pool, table, lens, i32([0, 1, -7, 6, 10]), b.scale, out=out, status=st)
    assert pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_QSL
    assert right(out, 0) and all(right(out, t) for t in range(6, 10)) and (out[1:6] == 9).all()


@pytest.mark.parametrize("n", [4, 150])
def test_requests_that_overlap_to_more_tokens_than_there_are(n):
    b = Batch(7, 16, 2, 64, [200], [n])
    q, pool, table, _, _ = b.tensors()
    out, st = torch.full_like(q, 9.0), status()
    pkv.paged_kv4_attention(q, pool, table.repeat(5, 1), i32([200] * 5), i32([0, n, 0, n, 0, n]), b.scale, out=out, status=st)
    assert pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_QSL and (out == 9).all()
    st.zero_()
    pkv.paged_kv4_attention(q, pool, table.repeat(2, 1), i32([200] * 2), i32([n, 0, n]), b.scale, out=out, status=st)
    assert pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_QSL
    b.check(out)


@pytest.mark.parametrize("new", [1, 3, 100])
@pytest.mark.parametrize("by", [-115, -100, 100])
def test_a_scale_far_from_q(new, by):
    """Rows of very small or large q with a scale that brings their scores back."""
    b = Batch(15, 16, 2, 128, [300, 140], [new, 1])
    b.q *= 2.0 ** by
    b.scale *= 2.0 ** -max(by, -100)
    b.check(pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=new))


@pytest.mark.parametrize("new", [1, 100])
def test_scores_of_zero_beside_a_factor_past_the_largest_value(new):
    b = Batch(16, 16, 2, 128, [300, 140], [new, 1], spread=0.0)
    b.q *= 2.0 ** 120
    b.scale = 1e30
    b.check(pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=new))


def test_a_scale_near_the_smallest_value():
    """Scores times 2^-126 and less are 0: a mean over the keys that a row sees."""
    for new in (3, 100):
        b = Batch(12, 16, 2, 128, [300, 40], [new, 1])
        b.scale = 1e-38
        for k_scale in (1.0, 2.0 ** -60):
            out = pkv.paged_kv4_attention(*b.tensors(), b.scale, k_scale=k_scale)
            b.check(out, k_by=k_scale)


@pytest.mark.parametrize("new", [1, 3, 200])
def test_calls_at_the_same_time_with_a_workspace_each(new):
    b = Batch(13, 16, 4, 128, [1700, 600, 300], [new] * 3)
    q, pool, table, lens, qsl = b.tensors()
    want = pkv.paged_kv4_attention(q, pool, table, lens, qsl, b.scale, max_query_len=new)
    b.check(want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [pkv.alloc_kv4_workspace(pool, stream=s) for s in streams]
    outs = [[pkv.paged_kv4_attention(q, pool, table, lens, qsl, b.scale, max_query_len=new, workspace=w, stream=s)
             for s, w in zip(streams, spaces)] for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for os in outs for o in os)


def test_a_captured_step_of_write_attention_and_read():
    """New tokens' slots and lengths change between replays; negative slots are padding."""
    rng = np.random.default_rng(14)
    pool = pkv.alloc_kv4_cache(40, 2, 64)
    k, v, q = (bf16(rng, 4, h, 64).to(DEV) for h in (2, 2, 8))
    slots, lens, qsl, table = i32([-1] * 4), i32([0] * 4), i32(range(5)), i32(rng.permutation(40).reshape(4, 10))
    ws, out = pkv.alloc_kv4_workspace(pool), torch.zeros_like(q)
    calls = [pkv.prepare_kv4_write(k, v, slots, pool), pkv.prepare_kv4_read(pool, slots),
             pkv.prepare_kv4_attention(q, pool, table, lens, qsl, 0.125, max_query_len=1, out=out, workspace=ws)]
    qsl[1:] = 0  # no request has a token while the calls are made for the first time
    for c in calls:
        c()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c()
    qsl.copy_(i32(range(5)))
    for step in range(40):
        live = 3 if step < 20 else 4  # the fourth row is padding at first
        k.copy_(bf16(rng, 4, 2, 64)), v.copy_(bf16(rng, 4, 2, 64)), q.copy_(bf16(rng, 4, 8, 64))
        at = [step + 7 if step < 20 else step - 13, step, step + 30, step - 20]
        if step == 0:
            for r, n in enumerate(at[:3]):
                if n:
                    pkv.paged_kv4_write(bf16(rng, n, 2, 64).to(DEV), bf16(rng, n, 2, 64).to(DEV),
                                        table[r, torch.arange(n, device=DEV) // 16] * 16 + torch.arange(n, device=DEV).int() % 16, pool)
        t = table.cpu().numpy()
        slots.copy_(i32([t[r, n // 16] * 16 + n % 16 if r < live else -1 for r, n in enumerate(at)]))
        lens.copy_(i32([n + 1 if r < live else 0 for r, n in enumerate(at)]))
        qsl.copy_(i32([min(r, live) for r in range(5)]))
        before = out[live:].clone()
        g.replay()
        vals = ko.unpack(pool.cpu().numpy())
        want, tol = ko.attend(q.double().cpu().numpy(), vals, t, lens.tolist(), qsl.tolist(), 0.125)
        got = out.double().cpu().numpy()
        assert (np.abs(got - want) <= tol)[:live].all() and torch.equal(out[live:], before)
        back = calls[1].outputs[0].double().cpu().numpy()
        for r in range(live):
            s = int(slots[r])
            assert np.array_equal(back[r], vals[s // 16, 0, :, s % 16])


def test_a_block_id_outside_the_pool_touches_its_request_only():
    b = Batch(8, 8, 2, 128, [100, 200], [1, 2])
    want = pkv.paged_kv4_attention(*b.tensors(), b.scale)
    for bad in (-1, b.pool.shape[0], 2 ** 31 - 1, -2 ** 31):
        q, pool, table, lens, qsl = b.tensors()
        table[0, 3] = bad
        st = status()
        out = pkv.paged_kv4_attention(q, pool, table, lens, qsl, b.scale, status=st)
        assert pkv.pkv_read_status(st) == pkv.PKV_DEV_BAD_BLOCK
        assert torch.equal(out[1:], want[1:])


def test_a_value_that_is_not_finite_reaches_the_rows_that_see_it_and_no_other():
    for kv, hq, hkv, d in (("k", 4, 2, 64), ("v", 4, 2, 64), ("k", 8, 1, 128), ("v", 8, 1, 128), ("v", 40, 1, 128)):
        b = Batch(9, hq, hkv, d, [44, 61], [12, 30])
        clean = pkv.paged_kv4_attention(*b.tensors(), b.scale)
        x = b.k if kv == "k" else b.v
        x[44 + 40, 0, 17] = float("nan")  # request 1, position 40: rows 12 + 9 on see it
        pkv.paged_kv4_write(b.k.to(DEV), b.v.to(DEV), i32(b.slots), b.pool)
        g = hq // hkv
        for longest in (30, 1):
            out = pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=longest)
            ref = pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=30)
            first = 12 + 40 - 31
            cols = slice(16, 32) if kv == "v" else slice(0, d)
            assert torch.isnan(out[first:, :g, cols]).all()
            rest = out.clone()
            rest[first:, :g, cols] = clean[first:, :g, cols]
            assert torch.isfinite(rest).all()
            if longest == 30:
                assert torch.equal(rest[:first], clean[:first]) and torch.equal(rest[first:, g:], clean[first:, g:])
            assert ref.shape == out.shape


def test_large_and_small_scores():
    """Scores far apart, growing along the context (references move), and q rows of very different sizes."""
    b = Batch(10, 8, 2, 128, [500, 90], [3, 1])
    ramp = torch.linspace(0.01, 30, 500)[:, None, None]
    b.k[:500] = (b.k[:500].float() * ramp).to(torch.bfloat16)
    pkv.paged_kv4_write(b.k.to(DEV), b.v.to(DEV), i32(b.slots), b.pool)
    b.q[0] *= 2.0 ** 20
    b.q[1] *= 2.0 ** -100
    b.q[2, 0] = 0
    b.q[2, 1] *= 2.0 ** -130
    b.q[2, 2, :] = 3.0
    for longest in (3, 1):
        out = pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=longest)
        b.check(out[:])


def test_same_bits_every_time_and_in_a_graph():
    b = Batch(11, 32, 8, 128, [900, 1500, 40, 2600], [1, 4, 2, 1])
    call = pkv.prepare_kv4_attention(*b.tensors(), b.scale, max_query_len=4)
    want = call().clone()
    for _ in range(20):
        assert torch.equal(call(), want)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs share the workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    call.outputs.zero_()
    for g in graphs * 3:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(call.outputs, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = pkv.paged_kv4_attention(*b.tensors(), b.scale, max_query_len=4, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
