"""fp64 oracle of the gated linear recurrence over a forest: row by row along every segment from
its parent's last row, and the reverse sweep.  Row indices come from the caller's layout
(seg_offset); nothing of the library is used."""
import numpy as np


def _roots(parent):
    out, n = {}, 0
    for v, p in enumerate(parent):
        if p < 0:
            out[v] = n
            n += 1
    return out


def scan_forest(parent, seg_len, seg_offset, x, g, mix, h0=None):
    """(h [C, D], state before every row [C, D])."""
    h, prev = np.empty_like(x), np.empty_like(x)
    roots = _roots(parent)
    for v, p in enumerate(parent):
        if p >= 0:
            s = h[seg_offset[p] + seg_len[p] - 1]
        else:
            s = np.zeros(x.shape[1]) if h0 is None else h0[roots[v]]
        for r in range(seg_offset[v], seg_offset[v] + seg_len[v]):
            prev[r] = s
            s = np.exp(g[r]) * s + (-np.expm1(g[r]) * x[r] if mix else x[r])
            h[r] = s
    return h, prev


def scan_forest_bwd(parent, seg_len, seg_offset, x, g, mix, prev, d_h, h0=None, d_end=None):
    """prev: state before every row.  d_end: {row: gradient of the state behind it}.
    Returns (dx, dg, dh0, lam)."""
    n, D = len(parent), x.shape[1]
    lam, dx, dg = np.empty_like(x), np.empty_like(x), np.empty_like(x)
    roots = _roots(parent)
    dh0 = np.zeros((len(roots), D))
    carry = np.zeros((n, D))                    # from a segment's children
    for v in range(n - 1, -1, -1):
        c = carry[v]
        for r in range(seg_offset[v] + seg_len[v] - 1, seg_offset[v] - 1, -1):
            lam[r] = d_h[r] + c + (0.0 if d_end is None or r not in d_end else d_end[r])
            a = np.exp(g[r])
            c = a * lam[r]
            dx[r] = -np.expm1(g[r]) * lam[r] if mix else lam[r]
            dg[r] = c * (prev[r] - x[r] if mix else prev[r])
        if parent[v] >= 0:
            carry[parent[v]] += c
        else:
            dh0[roots[v]] = c
    return dx, dg, dh0, lam
