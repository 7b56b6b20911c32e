"""paged_kv4_attention with scale * k_scale below the smallest normal 32-bit value and
q so large that the scores are not."""
import numpy as np
import pytest
import torch

from paged_attention_kv_gb300 import binding as pkv
from test_kv4_gpu import Batch, DEV, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 4, 12, 100])
@pytest.mark.parametrize("by", (-86, -84, -82, -76, -70, -67, -66, -65, -60))
def test_scores_of_a_small_factor_and_large_q(new, by):
    """Keys all 2688 or half of it, values 1 or -1: two weights that tell the factor's error."""
    b = Batch(21, 8, 2, 128, [150, 260], [new, 1])
    b.k[:] = torch.where(torch.arange(410)[:, None, None] % 3 == 0, 2688.0, 1344.0)
    b.v[:] = torch.where(torch.arange(410)[:, None, None] % 3 == 0, 1.0, -1.0)
    pkv.paged_kv4_write(b.k.to(DEV), b.v.to(DEV), i32(b.slots), b.pool)
    # scores of 2.5 and 1.2: 128 columns, q, 2688 * 2^-60 and the scale (a quarter of that with 2^-86)
    b.q[:] = 2.0 ** min(126, 42 - by) * 1.875
    b.scale = 2.0 ** by
    out = pkv.paged_kv4_attention(*b.tensors(), b.scale, k_scale=2.0 ** -60, max_query_len=new)
    want, _ = b.want(k_by=2.0 ** -60)
    assert 0.01 < np.abs(want[-1]).max() < 0.99
    b.check(out, k_by=2.0 ** -60)
