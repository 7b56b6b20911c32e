"""Plain 64-bit implementations of the prompt-step operators, by their
formulas, with the magnitudes that the tests' tolerances are made of."""
import numpy as np
import torch


def build_tables(query_lens, context_lens, free, table, num_tokens, num_blocks, cursor=0):
    """Request by request. Returns (seq_lens, qsl, positions, slots, cursor, table, refused)."""
    table = [list(row) for row in table]
    width = len(table[0]) if table else 0
    T = num_tokens
    pos, slots = [-1] * T, [-1] * T
    qsl, lens, refused = [0], [], []
    tok, short = 0, False
    avail = len(free) - cursor if 0 <= cursor <= len(free) else 0
    taken = 0
    for r, (n, old) in enumerate(zip(query_lens, context_lens)):
        n = max(n, 0)
        start, tok = tok, tok + n
        bad_len = old < 0 or old + n > 16 * width
        need = 0 if bad_len else -(-(old + n) // 16) - -(-old // 16)
        bad = bad_len or (n > 0 and tok > T)
        if need:
            short = short or taken + need > avail
            bad = bad or short
        qsl.append(min(tok, T))
        refused.append(bad)
        lens.append(old if bad else old + n)
        if bad:
            continue
        for b in range(-(-old // 16), -(-(old + n) // 16)):
            i = free[cursor + taken]
            table[r][b] = i if 0 <= i < num_blocks else -1
            taken += 1
        for i in range(n):
            p = old + i
            pos[start + i] = p
            i_b = table[r][p // 16]
            slots[start + i] = i_b * 16 + p % 16 if 0 <= i_b < num_blocks else -1
    return lens, qsl, pos, slots, cursor + taken, table, refused


def norm_rope(x, weight, positions, cos_sin, eps=1e-6, interleaved=False, sections=None):
    """x [T][H][D]; positions [axes][T]. Returns (y, |a c| + |b s| per element)."""
    x = x.double().cpu()
    table = cos_sin.double().cpu()
    half = table.shape[1] // 2
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    sections = sections or [half]
    positions = positions.cpu().long().reshape(len(sections), x.shape[0])
    y, mag = x.clone(), x.abs()
    f = 0
    for axis, n in enumerate(sections):
        for _ in range(n):
            i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
            c, s = table[positions[axis], f][:, None], table[positions[axis], half + f][:, None]
            a, b = x[..., i], x[..., j]
            y[..., i], y[..., j] = a * c - b * s, b * c + a * s
            mag[..., i], mag[..., j] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
            f += 1
    return y, mag


def norm_rope_tolerance(y, mag):
    """One rounding to bf16 (2^-8 of the value), and the 32-bit steps before
    it: the mean of squares (a sum of D <= 256 terms in a tree of depth 16 +
    4), the root (2 ulp), three products and one sum: under 32 roundings of
    2^-24 of the magnitudes, 2^-19."""
    return y.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + mag * 2.0 ** -19 + 1e-30


def prompt(q, k, v, lens, scale):
    """Returns (out, sum_j p_j |v_j| / sum_j p_j), both [sum(lens)][Hq][D] in 64 bits."""
    q, k, v = (x.double() for x in (q, k, v))
    g = q.shape[1] // k.shape[1]
    out, mag = torch.empty_like(q[:sum(lens)]), torch.empty_like(q[:sum(lens)])
    at = 0
    for n in lens:
        for h in range(q.shape[1]):
            kk, vv = k[at:at + n, h // g], v[at:at + n, h // g]
            for i in range(0, n, 1024):
                e = min(n, i + 1024)
                s = (q[at + i:at + e, h] @ kk[:e].T) * scale
                s = s.masked_fill(torch.ones(e - i, e, dtype=torch.bool, device=s.device).triu(i + 1), -float("inf"))
                p = torch.softmax(s, -1)
                out[at + i:at + e, h] = p @ vv[:e]
                mag[at + i:at + e, h] = p @ vv[:e].abs()
        at += n
    return out, mag


def prompt_tolerance(out, mag):
    """The output's rounding to bf16, 2^-8 of the value; each probability's
    rounding to bf16 before the product with V, 2^-8 of its term; and the
    scores: 32-bit sums of D <= 128 products of normal values (D * 2^-24 *
    sum |q k| * scale, under 2^-13) and the exponential's 2^-22, twice (value
    and sum): 2^-11 of the terms covers them."""
    return out.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -11) * (1 + 2.0 ** -8) + 1e-30


def worst(got, want, tol):
    """Largest error over its tolerance."""
    got = got.double().to(want.device)
    assert bool(torch.isfinite(got).all())
    return float(((got - want).abs() / tol).max()) if got.numel() else 0.0


def as_lists(t):
    return np.asarray(t.cpu()).tolist()
