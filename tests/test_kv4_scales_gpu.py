"""paged_kv4_write with k_scale and v_scale far from 1: infinities and values past
the range keep their sign, and every other value rounds as defined."""
import numpy as np
import pytest
import torch

import kv4_oracle as ko
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"
SCALES = [2.0 ** e for e in (-60, -40, -20, -10, -9, -8, 0, 20, 60)]
INF = float("inf")
MOST = 255 * 2.0 ** 120  # the largest finite bf16 value


def write(k, v, slots, nb, k_scale, v_scale):
    """The pool as the call leaves it, and as the definition does; both start from the same random bytes."""
    n, hkv, d = k.shape
    pool = np.random.default_rng(n).integers(0, 256, (nb, hkv, 18 * d), dtype=np.uint8)
    want = pool.copy()
    for t, s in enumerate(slots):
        ko.pack_token(want, s, k[t].double().numpy(), v[t].double().numpy(), k_scale, v_scale)
    got = torch.from_numpy(pool).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.paged_kv4_write(k.to(DEV), v.to(DEV), torch.tensor(slots, dtype=torch.int32, device=DEV), got, k_scale=k_scale,
                        v_scale=v_scale, status=st)
    assert pkv.pkv_read_status(st) == 0
    return got.cpu().numpy(), want


@pytest.mark.parametrize("by", SCALES)
@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 2)])
def test_values_past_the_range_keep_their_sign(by, d, hkv):
    """Groups whose largest magnitude is infinite or past 2688 times the scale: in whole blocks and token by token."""
    large = [x for x in (INF, MOST, 1e38, 1e36, 1e30, 1e24, 1e18, 3000 * by, 2688 * by, 2500 * by) if x >= 2500 * by]
    groups = [(s * x, t * y) for x in large for s in (-1, 1) for y in (x, 2500 * by, by) for t in (-1, 1)]
    rows = -(-len(groups) // (hkv * d // 16))
    rng = np.random.default_rng(5)
    x = rng.standard_normal((rows * hkv * d // 16, 16)) * by
    for i, (a, b) in enumerate(groups):
        x[i, i % 16], x[i, (i + 5) % 16] = a, b
    k = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).view(rows, hkv, d)
    n = -(-rows // 16) * 16
    k = torch.cat([k, k[:1].repeat(n - rows, 1, 1)])
    v = k.roll(3, 0)
    nb = n // 16 + 2
    for slots in (np.arange(n) + 16, np.random.default_rng(7).permutation(nb * 16)[:n]):
        got, want = write(k, v, slots, nb, by, by)
        assert np.array_equal(got, want)
        vals = ko.unpack(got)[slots // 16, 0, :, slots % 16] * by
        x = k.double().numpy()
        past = np.abs(x) >= 2688 * by
        assert past.sum() >= len(large) and np.array_equal(vals[past], np.sign(x[past]) * 2688 * by)


@pytest.mark.parametrize("by", SCALES)
def test_every_bf16_magnitude_rounds_as_defined(by):
    """All bf16 magnitudes in both signs in random groups (many past the range), and those near the scale's range."""
    rng = np.random.default_rng(11)
    mag = torch.arange(0, 0x7f80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double().numpy()
    near = mag[(mag > by * 2.0 ** -14) & (mag < by * 2.0 ** 13)]
    n = 1280
    x = np.concatenate([rng.permutation(np.resize(mag, n * 32)), rng.permutation(np.resize(near, n * 32))]).reshape(n, 1, 64)
    order = np.sort(x[n // 2:].reshape(-1, 16 * 40), 1).reshape(-1, 40, 16)  # groups of values near to one another
    x[n // 2:] = order[rng.permutation(len(order))].reshape(n // 2, 1, 64)
    x *= rng.choice([-1.0, 1.0], x.shape)
    k = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(k.double().numpy(), x)
    got, want = write(k, k.flip(0), rng.permutation(n + 64)[:n], n // 16 + 4, by, by)
    assert np.array_equal(got, want)
