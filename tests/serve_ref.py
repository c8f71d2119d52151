"""Plain fp64 forms of the norm, cache and tree operators, on CPU tensors, for
the tests: written from the definitions, one row or sequence at a time."""
from __future__ import annotations

import math

import torch


def pairs(rot, interleaved):
    j = torch.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def angles(cos, sin, positions, sections):
    """cos, sin [T, 1, rot/2] in fp64 of every token."""
    positions = positions.reshape(-1, positions.shape[-1]).long()
    cols, start = [], 0
    for axis, n in enumerate(sections):
        cols.append((axis, slice(start, start + n)))
        start += n
    c = torch.cat([cos.double()[positions[a]][:, s] for a, s in cols], -1)
    s_ = torch.cat([sin.double()[positions[a]][:, s] for a, s in cols], -1)
    return c[:, None], s_[:, None]


def norm_rope(x, w, c, s, rot, interleaved, eps):
    """fp64 output, and the sum of magnitudes that each output channel is made of."""
    x, w = x.double(), w.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    out, mag = y.clone(), y.abs()
    if rot:
        a, b = pairs(rot, interleaved)
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        both = y[..., a].abs() + y[..., b].abs()
        mag[..., a] = both
        mag[..., b] = both
    return out, mag


def norm_rope_backward(x, w, g, c, s, rot, interleaved, eps):
    """fp64 dx, dw, a magnitude for each dx, and sum |terms| of each dw."""
    x, w, g = x.double(), w.double(), g.double()
    gr, mag = g.clone(), g.abs()
    if rot:
        a, b = pairs(rot, interleaved)
        gr[..., a] = g[..., a] * c + g[..., b] * s
        gr[..., b] = g[..., b] * c - g[..., a] * s
        both = g[..., a].abs() + g[..., b].abs()
        mag[..., a] = both
        mag[..., b] = both
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    dn = gr * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dx_mag = r * (mag * w.abs() + n.abs() * (mag * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, (gr * n).sum((0, 1)), dx_mag, (mag * n.abs()).sum((0, 1))


def e4m3(y):
    """fp64 values to the nearest e4m3 value, ties to the even code, at most 448."""
    _, e = torch.frexp(y)
    step = torch.exp2((e.double() - 1).clamp_min(-6.0) - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def quantise(x):
    """(code values, scales) of bf16 rows [..., d] by the cache's fp32 formula, held in fp64 after."""
    x = x.float()
    scale = (x.abs().amax(-1) / 448.0).clamp_min(2.0 ** -64)
    return e4m3((x * (1.0 / scale)[..., None]).double()), scale


def row_index(table, page, b, pos):
    return table[b].long()[pos // page] * page + pos % page


def tree(q, k_rows, v_rows, table, page, lens, cu, mask, scale):
    """fp64 O [total, Hq, d], LSE [total, Hq], A = sum_j p_j |v_j| and S = the
    largest scale * sum |q k| of a row, from cache rows [rows, H, d] in fp64.
    Hidden keys are left out, whatever they hold."""
    total, Hq, d = q.shape
    H = k_rows.shape[1]
    G = Hq // H
    o = torch.full((total, Hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((total, Hq), math.nan, dtype=torch.float64)
    A, S = torch.zeros_like(o), torch.zeros_like(lse)
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        at = row_index(table, page, b, torch.arange(L))
        for i in range(n):
            t = cu[b] + i
            seen = list(range(L - n))
            for j in range(n):
                if (j <= i) if mask is None else (int(mask[t]) >> j) & 1:
                    seen.append(L - n + j)
            if not seen:
                o[t], lse[t] = 0.0, -math.inf
                continue
            rows = at[torch.tensor(seen)]
            kk = k_rows[rows].double().repeat_interleave(G, 1)  # [keys, Hq, d]
            vv = v_rows[rows].double().repeat_interleave(G, 1)
            qk = q[t].double()[None] * kk
            x = scale * qk.sum(-1)  # [keys, Hq]
            lse[t] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[t])
            o[t] = (p[..., None] * vv).sum(0)
            A[t] = (p[..., None] * vv.abs()).sum(0)
            S[t] = scale * qk.abs().sum(-1).amax(0)
    return o, lse, A, S
