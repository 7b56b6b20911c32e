"""README's example of a 4-bit pool and of shared pages, run as it stands: a
prompt step, three samples of one prompt and an ended request, and a step of those."""
import os
import re

import numpy as np
import pytest
import torch

import kv4_oracle as ko
from conftest import REPO
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def example():
    """What is made once, a step's calls, and the rows' change."""
    with open(os.path.join(REPO, "README.md"), encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    block, = [b for b in blocks if "paged_fork_tables" in b]
    once, rest = block.split("# every step")
    step, fork = rest.split("# row r goes on")
    return once, "#" + step, "#" + fork


def test_the_example():
    rng = np.random.default_rng(5)
    hq, hkv, d, nb = 8, 2, 64, 60
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    once, step, fork = example()
    free = i32(rng.permutation(nb).tolist())
    cursor, lens = i32([0]), i32([0] * 4)
    ns = dict(torch=torch, pkv=pkv, D=d, num_blocks=nb, num_kv_heads=hkv, free_blocks=free, cursor=cursor,
              block_table=torch.full((4, 12), -1, dtype=torch.int32, device=DEV))
    exec(once, ns)

    def tokens(new):
        t = sum(new)
        bf = lambda h: torch.from_numpy(rng.standard_normal((t, h, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
        ns["seq_lens"], ns["qsl"], _, ns["slots"], _ = pkv.paged_build_tables(
            i32(new), lens, free, ns["block_table"], t, nb, cursor=cursor, cursor_out=cursor)
        ns["q"], ns["k"], ns["v"] = bf(hq), bf(hkv), bf(hkv)
        exec(step, ns)
        want, tol = ko.attend(ns["q"].double().cpu().numpy(), ko.unpack(ns["kv4_cache"].cpu().numpy()),
                              ns["block_table"].cpu().numpy(), ns["seq_lens"].tolist(), ns["qsl"].tolist(), d ** -0.5)
        assert (np.abs(ns["out"].double().cpu().numpy() - want) <= tol).all()

    tokens([37, 50, 16, 0])
    before = ko.unpack(ns["kv4_cache"].cpu().numpy())
    old = ns["block_table"].cpu().numpy()
    ns["parents"] = i32([0, 0, 2, 0])  # three samples of request 0; request 1 has ended
    exec(fork, ns)
    assert ns["seq_lens"].tolist() == [37, 37, 16, 37]
    assert cursor.tolist() == [3 + 1 + 2] and int(ns["shares"].sum()) == 4
    after, table = ko.unpack(ns["kv4_cache"].cpu().numpy()), ns["block_table"].cpu().numpy()
    for r in (1, 3):
        assert (table[r, :2] == old[0, :2]).all() and table[r, 2] not in old[0]
        assert np.array_equal(after[table[r, 2], :, :, :5], before[old[0, 2], :, :, :5])
    lens = ns["seq_lens"]
    tokens([1, 1, 1, 1])
    assert len(set(ns["block_table"].cpu().numpy()[[0, 1, 3], 2].tolist())) == 3
