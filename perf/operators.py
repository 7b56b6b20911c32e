"""Timed cases of the operators around a prompt step, in plain form and as this library's kernels.

Three operators of one engine step over a ragged batch (``query_start_loc``):

``tables``  block tables, sequence lengths, positions and slot mapping from
            the requests' lengths (``paged_build_tables``);
``rope``    per-head norms of q and k, the position rotation (one axis or
            several) and the KV write, in one pass (``paged_qk_norm_rope``);
``prompt``  causal attention of whole prompts, packed, with grouped heads
            (``pkv_prompt_attention``).

``own`` chooses between the plain form (elementary torch operations in 32
bits, rounded once at the end) and the library's calls. A case names its
lengths by ``seqs``, ``lo``, ``hi`` and ``pick``: ``seqs`` lengths,
log-uniform in [lo, hi], from a generator seeded with ``pick``.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
SHAPES = {"32-4-64": (32, 4, 64), "32-8-128": (32, 8, 128), "12-4-128": (12, 4, 128), "8-8-64": (8, 8, 64),
          "16-2-128": (16, 2, 128)}


def _ceil(a, b):
    return -(-a // b)


def lengths(seqs, lo, hi, pick):
    r = random.Random(pick)
    return [min(hi, max(lo, int(round(math.exp(r.uniform(math.log(lo), math.log(hi + 1)) - 1e-9) - 0.5))))
            for _ in range(seqs)]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _tables(name, decode, prompts, lo, hi, pick, pad=0):
    """``decode`` requests with one new token and a context in [512, 4096],
    ``prompts`` with [lo, hi] new tokens (every other one after a prior
    chunk), shuffled; ``pad`` unused token rows at the end."""
    return {"name": name, "op": "tables", "decode": decode, "prompts": prompts, "lo": lo, "hi": hi, "pick": pick,
            "pad": pad}


def _rope(name, shape, tokens, norm, axes, interleaved, rotary, packed, cache, k_out, positions):
    """q and k of ``tokens`` tokens; ``packed``: q, k and v are slices of one
    projection's rows; ``cache``: k and v also go to the paged pool."""
    return {"name": name, "op": "rope", "shape": shape, "tokens": tokens, "norm": norm, "axes": axes,
            "interleaved": interleaved, "rotary": rotary, "packed": packed, "cache": cache, "k_out": k_out,
            "positions": positions}


def _prompt(name, shape, seqs, lo, hi, pick, packed):
    return {"name": name, "op": "prompt", "shape": shape, "seqs": seqs, "lo": lo, "hi": hi, "pick": pick,
            "packed": packed}


def listed():
    return [
        # a decode step's tables, the batch of the Llama-3-8B workload: latency
        _tables("tables-decode256", 256, 0, 1, 1, 3),
        # 4 chunks of 512 tokens among 192 decode requests, rows padded to a captured size
        _tables("tables-mixed", 192, 4, 512, 512, 4, pad=64),
        # a large prefill step: hundreds of ragged prompts
        _tables("tables-prefill", 0, 700, 1, 1500, 5),
        # one step of the 64-request TinyLlama decode batch: rotation and KV write, no norms
        _rope("rope-decode64", "32-4-64", 64, False, 1, False, 64, True, True, False, 4096),
        # the Llama-shaped decode batch with per-head norms
        _rope("rope-norm-decode256", "32-8-128", 256, True, 1, False, 128, True, True, False, 8192),
        # a mixed step's tokens; adjacent-pair rotation of half the head, no pool
        _rope("rope-pairs-2240", "32-8-128", 2240, True, 1, True, 64, False, False, True, 8192),
        # image and video prompts: three axes, norms, pool and contiguous k, larger than L2
        _rope("rope-axes-32768", "32-8-128", 32768, True, 3, False, 128, True, True, True, 32768),
        # two short prompts (17 to 40 tokens): latency
        _prompt("prompt-tiny", "32-4-64", 2, 17, 40, 1, False),
        # ragged chat prompts of a serving step, slices of one projection
        _prompt("prompt-ragged", "32-8-128", 24, 16, 2048, 6, True),
        # head 64, longer documents
        _prompt("prompt-d64", "32-4-64", 6, 700, 4096, 7, True),
        # a batch of long prompts
        _prompt("prompt-4x4096", "32-8-128", 4, 4096, 4096, 8, False),
        # one very long prompt
        _prompt("prompt-16384", "32-8-128", 1, 16384, 16384, 9, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tables", "rope", "prompt"))
    pick = rng.randrange(1 << 30)
    if op == "tables":
        prompts = rng.choice((0, _log(rng, 1, 700)))
        decode = _log(rng, 1, 700) if prompts == 0 or rng.random() < 0.6 else 0
        hi = _log(rng, 2, max(2, min(4096, 131072 // max(1, prompts))))
        c = _tables("", decode, prompts, rng.randint(1, hi), hi, pick, rng.choice((0, rng.randint(1, 300))))
    elif op == "rope":
        shape = rng.choice(sorted(SHAPES))
        d = SHAPES[shape][2]
        cache = rng.random() < 0.7
        c = _rope("", shape, _log(rng, 1, 32768), rng.random() < 0.6, rng.choice((1, 1, 2, 3)), rng.random() < 0.4,
                  rng.choice((d, d, d // 2)), rng.random() < 0.5, cache, not cache or rng.random() < 0.4,
                  rng.choice((4096, 32768, 131072)))
    else:
        shape = rng.choice(sorted(SHAPES))
        hi = _log(rng, 2, 12000)
        seqs = _log(rng, 1, max(1, min(64, (12000 // hi) ** 2 + 32000 // hi // 4)))
        c = _prompt("", shape, seqs, max(1, hi // rng.choice((1, 2, 16, 200))), hi, pick, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _table_lengths(case):
    r = random.Random(case["pick"])
    new = lengths(case["prompts"], case["lo"], case["hi"], case["pick"])
    old = [0 if i % 2 else r.randint(0, 1024) for i in range(len(new))]
    new += [1] * case["decode"]
    old += [r.randint(511, 4095) for _ in range(case["decode"])]
    order = list(range(len(new)))
    r.shuffle(order)
    return [old[i] for i in order], [new[i] for i in order]


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _qkv(gen, tokens, shape, packed):
    hq, hkv, d = shape
    if packed:
        rows = _randn(gen, tokens, (hq + 2 * hkv) * d)
        q, k, v = rows.split([hq * d, hkv * d, hkv * d], dim=1)
        return q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
    return _randn(gen, tokens, hq, d), _randn(gen, tokens, hkv, d), _randn(gen, tokens, hkv, d)


def _sections(half, axes):
    """Frequencies of each axis: the first (time) takes what the others leave."""
    rest = [half * 3 // 8 if axes == 3 else half // 2] * (axes - 1)
    return [half - sum(rest)] + rest


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).to("cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": case}
    if case["op"] == "tables":
        old, new = _table_lengths(case)
        shift = seed % 16  # inputs of another seed: other contexts
        old = [x + shift if x else 0 for x in old]
        r = len(old)
        width = max(_ceil(o + n + 16, BLOCK) for o, n in zip(old, new))
        held = [_ceil(o, BLOCK) for o in old]
        need = sum(_ceil(o + n, BLOCK) - h for o, n, h in zip(old, new, held))
        nb = int(1.25 * (sum(held) + need)) + 8
        perm = rng.permutation(nb).astype(np.int32)
        table = np.full((r, width), -1, dtype=np.int32)
        at = 0
        for i, h in enumerate(held):
            table[i, :h] = perm[at:at + h]
            at += h
        s.update(context_lens=_i32(old), query_lens=_i32(new), block_table=torch.from_numpy(table).to("cuda"),
                 free_blocks=torch.from_numpy(perm[at:].copy()).to("cuda"), num_blocks=nb,
                 num_tokens=sum(new) + case["pad"])
        t = s["num_tokens"]
        s.update(cursor=_i32([0]), cursor_out=_i32([0]), seq_lens=_i32(old), query_start_loc=_i32([0] * (r + 1)),
                 positions=torch.zeros(t, dtype=torch.int32, device="cuda"),
                 slot_mapping=torch.zeros(t, dtype=torch.int32, device="cuda"))
    elif case["op"] == "rope":
        hq, hkv, d = SHAPES[case["shape"]]
        t, half = case["tokens"], case["rotary"] // 2
        q, k, v = _qkv(gen, t, (hq, hkv, d), case["packed"])
        angle = (np.arange(case["positions"], dtype=np.float64)[:, None]
                 * 10000.0 ** (-np.arange(half, dtype=np.float64) / half)[None])
        cos_sin = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).to("cuda")
        start = int(rng.integers(0, max(1, case["positions"] - t)))
        if case["axes"] == 1:
            pos = (start + np.arange(t)) % case["positions"] if t > 256 else rng.integers(0, case["positions"], t)
        else:  # frames of 16 x 24 patches
            n = np.arange(t)
            pos = np.stack([start + n // 384, start + n // 24 % 16, start + n % 24][:case["axes"]]) % case["positions"]
        s.update(q=q, k=k, v=v, cos_sin=cos_sin, positions=torch.from_numpy(pos.astype(np.int32)).to("cuda"),
                 sections=_sections(half, case["axes"]) if case["axes"] > 1 else None, q_weight=None, k_weight=None,
                 slot_mapping=None, kv_cache=None, q_out=torch.zeros((t, hq, d), dtype=torch.bfloat16, device="cuda"),
                 k_out=torch.zeros((t, hkv, d), dtype=torch.bfloat16, device="cuda") if case["k_out"] else None)
        if case["norm"]:
            s["q_weight"] = (1 + 0.1 * _randn(gen, d).float()).to(torch.bfloat16)
            s["k_weight"] = (1 + 0.1 * _randn(gen, d).float()).to(torch.bfloat16)
        if case["cache"]:
            nb = _ceil(t, BLOCK) * 5 // 4 + 2
            s["kv_cache"] = _randn(gen, nb, 2, hkv, BLOCK, d)
            if t > 256:  # prompts: whole blocks, in the order of a shuffled pool
                ids = rng.permutation(nb)[:_ceil(t, BLOCK)]
                slots = (ids[:, None] * BLOCK + np.arange(BLOCK)).reshape(-1)[:t]
            else:        # decode: one slot in each of many blocks
                slots = rng.permutation(nb * BLOCK)[:t]
            s["slot_mapping"] = torch.from_numpy(slots.astype(np.int32)).to("cuda")
    else:
        shape = SHAPES[case["shape"]]
        lens = lengths(case["seqs"], case["lo"], case["hi"], case["pick"])
        q, k, v = _qkv(gen, sum(lens), shape, case["packed"])
        s.update(q=q, k=k, v=v, lens=lens, query_start_loc=_i32([0] + list(np.cumsum(lens))),
                 scale=shape[2] ** -0.5, out=torch.zeros(tuple(q.shape), dtype=torch.bfloat16, device="cuda"))
    if own:
        s["call"] = _call(s)
    return s


def _call(s):
    """The library's prepared call on this state's buffers."""
    from paged_attention_kv_gb300 import binding as pkv
    op = s["case"]["op"]
    if op == "tables":
        return pkv.prepare_build_tables(s["query_lens"], s["context_lens"], s["free_blocks"], s["block_table"],
                                        s["num_tokens"], s["num_blocks"], cursor=s["cursor"],
                                        cursor_out=s["cursor_out"], seq_lens=s["seq_lens"],
                                        query_start_loc=s["query_start_loc"], positions=s["positions"],
                                        slot_mapping=s["slot_mapping"])
    if op == "rope":
        return pkv.prepare_qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], q_weight=s["q_weight"],
                                        k_weight=s["k_weight"], eps=1e-6, interleaved=s["case"]["interleaved"],
                                        axis_sections=s["sections"], v=s["v"] if s["case"]["cache"] else None,
                                        slot_mapping=s["slot_mapping"], kv_cache=s["kv_cache"], q_out=s["q_out"],
                                        k_out=s["k_out"])
    return pkv.prepare_prompt_attention(s["q"], s["k"], s["v"], s["query_start_loc"], s["scale"], out=s["out"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    if own:
        if "call" not in state:
            state["call"] = _call(state)
        state["call"]()
    else:
        PLAIN[state["case"]["op"]](state)
    return _outputs(state)


def _outputs(s):
    op = s["case"]["op"]
    if op == "tables":
        return {k: s[k] for k in ("block_table", "seq_lens", "query_start_loc", "positions", "slot_mapping",
                                  "cursor_out")}
    if op == "rope":
        return {k: s[k] for k in ("q_out", "k_out", "kv_cache") if s[k] is not None}
    return {"out": s["out"]}


def plain_tables(s):
    old, new = s["context_lens"].long(), s["query_lens"].long()
    ends = torch.cumsum(new, 0)
    held = (old + BLOCK - 1) // BLOCK
    need = (old + new + BLOCK - 1) // BLOCK - held
    first = s["cursor"] + torch.cumsum(need, 0) - need
    t = torch.arange(s["num_tokens"], device="cuda")
    used = t < ends[-1]
    t = torch.minimum(t, ends[-1] - 1)  # padding rows repeat the last token
    r = torch.searchsorted(ends, t, right=True)
    pos = old[r] + t - (ends - new)[r]
    blk = pos // BLOCK
    fresh = blk - held[r]
    ids = torch.where(fresh >= 0, s["free_blocks"][torch.clamp(first[r] + fresh, 0, len(s["free_blocks"]) - 1)],
                      s["block_table"][r, blk])
    s["block_table"][r, blk] = ids  # tokens of one block write the same id
    s["seq_lens"].copy_(old + new)
    s["query_start_loc"][1:] = ends
    s["positions"].copy_(torch.where(used, pos, -1))
    s["slot_mapping"].copy_(torch.where(used, ids * BLOCK + pos % BLOCK, -1))
    s["cursor_out"].copy_(s["cursor"] + need.sum())


def _axis_of(sections):
    return torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to("cuda")


def plain_norm_rope(x, weight, cos, sin, rotary, interleaved):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    a, b = (x[..., 0:rotary:2], x[..., 1:rotary:2]) if interleaved else (x[..., :rotary // 2], x[..., rotary // 2:rotary])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rotary:]], -1).to(torch.bfloat16)


def plain_rope(s):
    c = s["case"]
    half = c["rotary"] // 2
    if c["axes"] == 1:
        cs = s["cos_sin"][s["positions"].long()]
        cos, sin = cs[:, None, :half], cs[:, None, half:]
    else:
        pos = s["positions"].long()[_axis_of(s["sections"])].t()  # [T][half]
        col = torch.arange(half, device="cuda")
        cos, sin = s["cos_sin"][pos, col][:, None], s["cos_sin"][pos, col + half][:, None]
    s["q_out"].copy_(plain_norm_rope(s["q"], s["q_weight"], cos, sin, c["rotary"], c["interleaved"]))
    k = plain_norm_rope(s["k"], s["k_weight"], cos, sin, c["rotary"], c["interleaved"])
    if c["k_out"]:
        s["k_out"].copy_(k)
    if c["cache"]:
        slot = s["slot_mapping"].long()
        s["kv_cache"][slot // BLOCK, 0, :, slot % BLOCK] = k
        s["kv_cache"][slot // BLOCK, 1, :, slot % BLOCK] = s["v"]


def plain_prompt(s):
    hq, hkv, d = SHAPES[s["case"]["shape"]]
    g, at = hq // hkv, 0
    for n in s["lens"]:
        q = s["q"][at:at + n].float().view(n, hkv, g, d).permute(1, 2, 0, 3)  # [Hkv][g][n][D]
        k = s["k"][at:at + n].float().permute(1, 2, 0)                        # [Hkv][D][n]
        v = s["v"][at:at + n].float().permute(1, 0, 2)
        step = max(16, min(n, (1 << 28) // (hq * n)))  # rows at a time: 1 GiB of scores
        for i in range(0, n, step):
            m, seen = min(step, n - i), min(n, i + step)
            x = torch.matmul(q[:, :, i:i + m].reshape(hkv, g * m, d), k[:, :, :seen]) * s["scale"]
            x = x.view(hkv, g, m, seen)
            x.masked_fill_(torch.arange(seen, device="cuda")[None] > torch.arange(i, i + m, device="cuda")[:, None],
                           -math.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.matmul(x.view(hkv, g * m, seen), v[:, :seen]).view(hkv, g, m, d) / x.sum(-1, keepdim=True)
            s["out"][at + i:at + i + m] = o.permute(2, 0, 1, 3).reshape(m, hq, d).to(torch.bfloat16)
        at += n


PLAIN = {"tables": plain_tables, "rope": plain_rope, "prompt": plain_prompt}


# ---------------------------------------------------------------------------
# work and exact answers
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "tables":
        old, new = _table_lengths(case)
        t = sum(new) + case["pad"]
        ids = sum(_ceil(o + n, BLOCK) - _ceil(o, BLOCK) for o, n in zip(old, new))
        # lengths read; positions, slots, new table entries and lengths written; free ids read
        return {"bytes": 4 * (2 * len(new) + 2 * t + 2 * ids + 2 * len(new) + 3), "flops": 8 * t}
    hq, hkv, d = SHAPES[case["shape"]]
    if case["op"] == "rope":
        t = case["tokens"]
        rows = hq + hkv                        # read and written: q, k
        moved = 2 * rows + hkv * (2 if case["cache"] else 0) + (hkv if case["cache"] and case["k_out"] else 0)
        table = 4 * case["rotary"] * min(t, case["positions"])
        return {"bytes": t * (moved * d * 2 + 4 * case["axes"] + (4 if case["cache"] else 0)) + table,
                "flops": t * rows * (3 * case["rotary"] + (4 * d if case["norm"] else 0))}
    lens = lengths(case["seqs"], case["lo"], case["hi"], case["pick"])
    pairs = sum(n * (n + 1) // 2 for n in lens)
    return {"bytes": 2 * sum(lens) * d * (2 * hq + 2 * hkv), "flops": 4 * d * hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        old, new = s["context_lens"].tolist(), s["query_lens"].tolist()
        free, table = s["free_blocks"].tolist(), s["block_table"].cpu().numpy()
        qsl, lens, pos, slots = [0], [], [], []
        taken = 0
        for r, (o, n) in enumerate(zip(old, new)):
            for b in range(_ceil(o, BLOCK), _ceil(o + n, BLOCK)):
                table[r, b] = free[taken]
                taken += 1
            p = np.arange(o, o + n)
            pos.append(p)
            slots.append(table[r, p // BLOCK].astype(np.int64) * BLOCK + p % BLOCK)
            lens.append(o + n)
            qsl.append(qsl[-1] + n)
        tail = [np.full(s["num_tokens"] - qsl[-1], -1)]
        return {"block_table": torch.from_numpy(table).cuda(), "seq_lens": _i32(lens), "query_start_loc": _i32(qsl),
                "positions": _i32(np.concatenate(pos + tail).tolist()),
                "slot_mapping": _i32(np.concatenate(slots + tail).tolist()), "cursor_out": _i32([taken])}
    if case["op"] == "rope":
        half = case["rotary"] // 2
        table = s["cos_sin"].double()
        pos = s["positions"].reshape(case["axes"], -1).long()
        axis = [a for a, n in enumerate(s["sections"] or [half]) for _ in range(n)]

        def turn(x, w):
            y = x.double().clone()
            if w is not None:
                y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + 1e-6) * w.double()
            z = y.clone()
            for f in range(half):
                i, j = (2 * f, 2 * f + 1) if case["interleaved"] else (f, f + half)
                c = table[pos[axis[f]], f][:, None]
                sn = table[pos[axis[f]], f + half][:, None]
                z[..., i] = y[..., i] * c - y[..., j] * sn
                z[..., j] = y[..., j] * c + y[..., i] * sn
            return z

        out = {"q_out": turn(s["q"], s["q_weight"])}
        k = turn(s["k"], s["k_weight"])
        if case["k_out"]:
            out["k_out"] = k
        if case["cache"]:
            pool = s["kv_cache"].double()
            flat = s["slot_mapping"].long()
            pool[:, 0].transpose(1, 2)[flat // BLOCK, flat % BLOCK] = k
            pool[:, 1].transpose(1, 2)[flat // BLOCK, flat % BLOCK] = s["v"].double()
            out["kv_cache"] = pool
        return out
    hq, hkv, d = SHAPES[case["shape"]]
    if work(case)["flops"] > 1.5e12:
        return None
    out = torch.empty((sum(s["lens"]), hq, d), dtype=torch.float64, device="cuda")
    at = 0
    for n in s["lens"]:
        for h in range(hq):
            kk, vv = s["k"][at:at + n, h // (hq // hkv)].double(), s["v"][at:at + n, h // (hq // hkv)].double()
            for i in range(0, n, 2048):
                e = min(n, i + 2048)
                z = (s["q"][at + i:at + e, h].double() * s["scale"]) @ kk[:e].T
                z = z + torch.triu(torch.full((e - i, e), -math.inf, dtype=torch.float64, device="cuda"), diagonal=i + 1)
                out[at + i:at + e, h] = torch.softmax(z, dim=-1) @ vv[:e]
        at += n
    return {"out": out}
