"""README's loop of steps and forks of the tables, its code as it stands and
nothing between: what a fork leaves behind is what the next step goes on from."""
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
    """What is made once, the step's tables, its calls on the 4-bit pool, and the rows' change."""
    with open(os.path.join(REPO, "README.md"), encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    loop, = [b for b in blocks if "paged_build_tables" in b]
    block, = [b for b in blocks if "paged_fork_tables" in b]
    once, rest = loop.split("# every step")
    tables = "#" + rest[:rest.index("q, k = ")]
    more, rest = block.split("# every step")
    step, fork = rest.split("# row r goes on")
    return once + more, tables, "#" + step, "#" + fork


def test_steps_and_forks_in_turn():
    rng = np.random.default_rng(8)
    hq, hkv, d, nb = 8, 2, 64, 40
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    once, tables, step, fork = example()
    ns = dict(torch=torch, pkv=pkv, D=d, num_blocks=nb, num_kv_heads=hkv, num_reqs=4, free_blocks=i32(rng.permutation(nb).tolist()),
              block_table=torch.full((4, 12), -1, dtype=torch.int32, device=DEV))
    exec(once, ns)
    lens = [0] * 4

    def tokens(new):
        for r, n in enumerate(new):
            lens[r] += n
        t = sum(new)
        bf = lambda h: torch.from_numpy(rng.standard_normal((t, h, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
        ns.update(query_lens=i32(new), num_tokens=t)
        exec(tables, ns)
        assert ns["seq_lens"].tolist() == lens and ns["context_lens"].tolist() == lens
        ns["q"], ns["k"], ns["v"] = bf(hq), bf(hkv), bf(hkv)
        exec(step, ns)
        table = ns["block_table"].cpu().numpy()
        held = [int(b) for r, n in enumerate(lens) for b in table[r, :-(-n // 16)]]
        assert min(held) >= 0
        partly = [int(table[r, n // 16]) for r, n in enumerate(lens) if n % 16]
        assert len(set(partly)) == len(partly) and all(held.count(b) == 1 for b in partly)
        want, tol = ko.attend(ns["q"].double().cpu().numpy(), ko.unpack(ns["kv4_cache"].cpu().numpy()), table, lens,
                              ns["qsl"].tolist(), d ** -0.5)
        assert (np.abs(ns["out"].double().cpu().numpy() - want) <= tol).all()

    def go_on(parents):
        ns["parents"] = i32(parents)
        exec(fork, ns)
        lens[:] = [lens[p] if p >= 0 else 0 for p in parents]
        assert ns["context_lens"].tolist() == lens  # what the next step's tables start from
        table = ns["block_table"].cpu().numpy()
        held = {int(b) for r, n in enumerate(lens) for b in table[r, :-(-n // 16)]}
        free = ns["free_blocks"].tolist()[int(ns["cursor"]):]
        assert len(set(free)) == len(free) and not set(free) & held and len(free) + len(held) == nb

    tokens([37, 50, 16, 0])
    go_on([0, 0, 2, 0])      # three samples of request 0; request 1 has ended
    tokens([1, 1, 1, 1])
    go_on([3, -1, 1, -1])    # two of them go on, two rows are free
    tokens([1, 0, 11, 0])
    tokens([1, 20, 1, 70])   # new requests in those rows
    go_on([1, 1, 3, 3])
    tokens([13, 12, 3, 1])
    go_on([-1] * 4)
    assert int(ns["cursor"]) == 0 and not ns["shares"].any()
