"""Plain 64-bit forms of the paged-cache operators, written out for the tests,
and how far a kernel may be from them.

Rounding: a value rounded to a type is off by at most half a step, eps / 2
relative to it (bf16 2^-8, fp16 2^-11, fp32 2^-24), or half the spacing of the
type's subnormals. What the kernels compute before that rounding is fp32; each
bound below counts its operations.
"""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def plan(lens, want, table, free, count, page, capacity):
    """Request by request. Returns a dict of int lists; table and free as after the call."""
    table = [list(r) for r in table]
    free = list(free)
    P, width = len(free), len(table[0]) if table else 0
    top = min(max(count, 0), P)
    stack = free[:top]
    ceil = lambda n: -(-n // page)  # noqa: E731
    fine = lambda n: 0 <= n <= width * page  # noqa: E731
    returned = 0
    for n, (a, b) in enumerate(zip(lens, want)):
        if fine(a) and fine(b) and b < a:
            for j in range(ceil(b), ceil(a)):
                if len(stack) < P:
                    stack.append(table[n][j])
                    returned += 1
    new_lens, cu, slots, pos = [], [0], [], []
    taken = refused = 0
    closed = False
    for n, (a, b) in enumerate(zip(lens, want)):
        if fine(a) and fine(b) and b > a:
            need = ceil(b) - ceil(a)
            closed = closed or need > len(stack) or len(slots) + b - a > capacity
            if not closed:
                for j in range(ceil(a), ceil(b)):
                    table[n][j] = stack.pop()
                taken += need
                for t in range(a, b):
                    p = table[n][t // page]
                    slots.append(p * page + t % page if 0 <= p < P else -1)
                    pos.append(t)
                a = b
        elif fine(a) and fine(b):
            a = b
        refused += a != b
        new_lens.append(a)
        cu.append(len(slots))
    free[top:len(stack)] = stack[top:]
    info = [len(slots), taken, returned, refused]
    slots += [-1] * (capacity - len(slots))
    pos += [0] * (capacity - len(pos))
    return dict(new_lens=new_lens, cu_new=cu, slot_map=slots, positions=pos,
                new_count=[len(stack)], info=info, table=table, free=free)


def norm_rope(x, w, positions, inv_freq, interleaved, scale, eps=1e-6):
    """x [T, H, D] fp64; w [D] or None; positions [axes, T]; inv_freq [R / 2].
    Returns the rows and, per element, the size of what was added up for it."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt(np.mean(y ** 2, axis=-1, keepdims=True) + eps) * w
    size = np.abs(y)
    h = 0 if inv_freq is None else len(inv_freq)
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        theta = positions[i % len(positions)].astype(np.float64) * inv_freq[i]
        c, s = np.cos(theta)[:, None] * scale, np.sin(theta)[:, None] * scale
        u, v = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
        size[..., a] = size[..., b] = (np.abs(u) + np.abs(v)) * abs(scale)
    return y, size


def norm_rope_bound(ref, size, D, dtype):
    """The sum of D squares, root, quotient and weight are each within
    (D / 2 + 8) 2^-24 relative; cos and sin within 2^-22 (angle 2^-31 half
    turns, two last places); products and sum 2^-23."""
    return HALF[dtype] * np.abs(ref) + TINY[dtype] + ((D / 2 + 8) * 2.0 ** -24 + 2.0 ** -21) * size


def decode(q, k_rows, v_rows, scale, gate=None):
    """One sequence: q [H_q, D]; k_rows, v_rows [L, H_kv, D] fp64. Returns o, lse
    and, per output element, the bound on an fp32 evaluation's error:
      scores: D products and sums of 2^-23 relative to sum |q k|, twice in a weight;
      weights in two 16-bit parts: 2^-16; exponential and its argument: 2^-21;
      sums over L tokens by 4 warps of 16 rows: L / 8 + 64 steps of 2^-24."""
    H_q, D = q.shape
    L, H_kv, _ = k_rows.shape
    G = H_q // H_kv
    o, lse, err = np.zeros((H_q, D)), np.full(H_q, -np.inf), np.zeros((H_q, D))
    lse_err = np.zeros(H_q)
    if L:
        for h in range(H_q):
            k, v = k_rows[:, h // G], v_rows[:, h // G]
            x = k @ q[h] * scale
            m = x.max()
            p = np.exp(x - m)
            lse[h] = m + math.log(p.sum())
            p /= p.sum()
            o[h] = p @ v
            size = (np.abs(k) @ np.abs(q[h]) * scale).max()
            rel = 2 * D * 2.0 ** -23 * size + 2.0 ** -16 + 2.0 ** -21 + (L / 8 + 64) * 2.0 ** -24
            err[h] = rel * (p @ np.abs(v))
            lse_err[h] = rel + 2.0 ** -22 * (abs(m) + math.log(L) + 1)
    if gate is not None:
        g = 1 / (1 + np.exp(-gate))
        o, err = o * g, err * g + np.abs(o * g) * 2.0 ** -20
    return o, lse, err, lse_err
