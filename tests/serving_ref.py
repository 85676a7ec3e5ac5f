"""Plain 64-bit forms of the serving-step calls, and the tolerances of their results.

Everything here runs on CPU tensors, row by row from the definitions in the
header; it shares no code with the library.
"""
import math

import torch

# half a step of a type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


def plan(seqlens, new_lens, table, free, n_free, L, page):
    """(table, slots, lens, n_free, status) from lists; a request without room asks for nothing, one that
    the pages do not reach for still counts for those after it."""
    table = [list(r) for r in table]
    asked, given, slots, lens, status = 0, 0, [], [], []
    for b, (s, n) in enumerate(zip(seqlens, new_lens)):
        used, total = -(-s // page), -(-(s + n) // page)
        fits = total <= len(table[b])
        need = total - used if fits else 0
        served = fits and (need == 0 or asked + need <= n_free)
        if served:
            for k in range(need):
                table[b][used + k] = free[n_free - 1 - asked - k]
            given += need
        asked += need
        rows = range(s, s + n) if served else []
        slots.append([table[b][r // page] * page + r % page for r in rows] + [-1] * (L - len(rows)))
        lens.append(s + n if served else s)
        status.append(0 if served else 1)
    return table, slots, lens, n_free - given, status


def release(seqlens, keep, table, free, n_free, page):
    free = list(free)
    for b, (s, k) in enumerate(zip(seqlens, keep)):
        for c in range(-(-k // page), -(-s // page)):
            free[n_free] = table[b][c]
            n_free += 1
    return free, n_free


def axis_of(i, n_axes, sections, cycle):
    if cycle:
        a = i % n_axes
        return a if a > 0 and i // n_axes < sections[a] else 0
    a = 0
    while i >= sections[a]:
        i -= sections[a]
        a += 1
    return a


def rope(x, positions, inv_freq, sections, cycle, adjacent):
    """x [B,L,H,D] turned in 64 bits, and per element the sum |a| + |b| of its pair (for the tolerance)."""
    n = inv_freq.shape[0]
    axis = [axis_of(i, positions.shape[0], sections, cycle) for i in range(n)]
    t = torch.stack([positions[a].double() * inv_freq[i].double() for i, a in enumerate(axis)], -1) if n else \
        torch.zeros(*x.shape[:2], 0, dtype=torch.float64)
    c, s = t.cos()[:, :, None], t.sin()[:, :, None]
    x = x.double()
    lo = 2 * torch.arange(n) if adjacent else torch.arange(n)
    hi = lo + 1 if adjacent else lo + n
    y, size = x.clone(), x.abs()
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    size[..., lo] = size[..., hi] = a.abs() + b.abs()
    return y, size


def tree_sees(n, size, T, mask):
    """[T, n] bool: which of a sequence's n rows each node sees; mask [T, T] bool."""
    see = torch.zeros(T, n, dtype=torch.bool)
    for i in range(size):
        for r in range(n):
            j = r - (n - size)
            see[i, r] = j < 0 or bool(mask[i, j])
    return see


def tree(q, k_rows, v_rows, sees, scale):
    """One sequence: q [Hq,T,D], k_rows / v_rows [Hkv,n,D], sees [T,n] -> out [Hq,T,D], lse [Hq,T] in 64 bits and
    the tolerance of out.

    Error of out: the weights are rounded to bf16 (relative 2^-8 each, and they are normalised by the sum of the
    rounded weights, so an error e_r moves out by w_r e_r (V_r - out): at most 2^-8 (A + |out|), A = sum p_r |V_r|),
    the result is rounded to bf16 (2^-8 |out|), and scores in fp32 (below) move weights by less than 2e-4 relative
    (4e-4 (A + |out|) for weight and norm)."""
    Hq, T, D = q.shape
    Hkv, n = k_rows.shape[0], k_rows.shape[1]
    out = torch.zeros(Hq, T, D, dtype=torch.float64)
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        for i in range(T):
            rows = sees[i].nonzero().flatten()
            if rows.numel() == 0:
                continue
            s = (k_rows[g, rows].double() @ q[h, i].double()) * scale
            lse[h, i] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[h, i])
            v = v_rows[g, rows].double()
            out[h, i] = p @ v
            tol[h, i] = 2 ** -8 * (p @ v.abs() + 2 * out[h, i].abs()) + 4e-4 * (p @ v.abs() + out[h, i].abs()) + 1e-30
    return out, lse, tol


# LSE: a score's fp32 error is at most (D + 2) 2^-24 sum|q k| scale, about 258 * 6e-8 * 13 = 2e-4 for unit normals at
# D = 256 (sum|q k| scale = 256 * 0.64 / 16 = 10, 13 with its spread); the sum of exponentials adds ex2's and the
# additions' few 2^-22 and log2's; 4e-4 in all.
LSE_TOL = 4e-4


def check_tree(out, lse, ref, what=""):
    o, l, tol = ref
    out, lse = out.double().cpu(), lse.double().cpu()
    seen = l > -math.inf
    assert torch.equal(lse > -math.inf, seen), f"{what}: rows that see nothing differ"
    assert (out[~seen] == 0).all(), f"{what}: rows that see nothing must be 0"
    bad = (out - o).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((out - o).abs() - tol).max():.3e}"
    assert seen.sum() == 0 or (lse - l)[seen].abs().max() <= LSE_TOL, f"{what}: lse {(lse - l)[seen].abs().max():.3e}"
