"""README's example of a step from lengths and projections, run as it stands
for a prompt step and a decode step behind it."""
import os
import re

import pytest
import torch

import prompt_oracle as po
from conftest import REPO
from paged_attention_kv_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def example():
    """(what is made once, a step) of the code block that builds the tables, and
    the block with attention for prompts alone."""
    with open(os.path.join(REPO, "README.md"), encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    block, = [b for b in blocks if "paged_build_tables" in b]
    prompt, = [b for b in blocks if "pkv_prompt_attention" in b]
    once, mark, step = block.rpartition("# every step")
    return once, mark + step, prompt


def test_the_readme_example_over_two_steps():
    hq, hkv, d, nb, lens = 8, 2, 64, 64, [37, 5, 130]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)

    angle = torch.rand(256, d // 2, generator=gen, device=DEV)
    table = torch.full((3, 16), -1, dtype=torch.int32, device=DEV)
    kv_cache = torch.zeros(nb, 2, hkv, 16, d, device=DEV, dtype=torch.bfloat16)
    ns = dict(torch=torch, pkv=pkv, D=d, num_reqs=3, num_blocks=nb, block_table=table, kv_cache=kv_cache,
              cos_sin=torch.cat([angle.cos(), angle.sin()], 1), qw=randn(d), kw=randn(d),
              free_blocks=torch.randperm(nb, generator=gen, device=DEV).int(),
              context_lens=torch.zeros(3, dtype=torch.int32, device=DEV))
    once, step, prompt = example()
    exec(once, ns)
    history = [[], [], []]
    for new, codes in ((lens, (step, prompt)), ([1, 1, 1], (step,))):
        t = sum(new)
        v = randn(t, hkv, d)
        ns.update(query_lens=torch.tensor(new, dtype=torch.int32, device=DEV), num_tokens=t, v=v, q=randn(t, hq, d),
                  k=randn(t, hkv, d))
        outs = []
        for code in codes:  # the second is in the first's place, on its q, k and v
            exec(code, ns)
            outs.append(ns["out"])
        at = 0
        for r, n in enumerate(new):
            history[r].append((ns["k"][at:at + n].clone(), v[at:at + n]))
            k, vv = (torch.cat(x) for x in zip(*history[r]))
            q = torch.zeros(len(k), hq, d, device=DEV, dtype=torch.bfloat16)
            q[-n:] = ns["q"][at:at + n]
            want, mag = po.prompt(q, k, vv, [len(k)], d ** -0.5)
            for out in outs:
                # paged_attention rounds as prompt attention does, and joins parts in 32 bits
                assert po.worst(out[at:at + n], want[-n:], 2 * po.prompt_tolerance(want, mag)[-n:]) <= 1.0
            at += n
        ns["context_lens"] = ns["seq_lens"]
        held = [int(b) for r, row in enumerate(table.tolist()) for b in row[:-(-int(ns["seq_lens"][r]) // 16)]]
        assert len(set(held)) == len(held) and min(held) >= 0
