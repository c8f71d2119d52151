"""Plain forms of draft verification and of the next batch's page table, on CPU
values, for the tests: written from the definitions, one sequence or page at a time."""
from __future__ import annotations

import torch


def verify(tokens, probs, cu, u, u_next, draft, mask):
    """(path, accepted, next tokens, distance of the nearest test or draw to its border) by
    the definition in fp64; probs and draft [total, V] already between 0 and 1."""
    path, kept, nxt, near = [], [], [], 1.0
    for b in range(len(cu) - 1):
        lo, n = cu[b], cu[b + 1] - cu[b]
        if n == 0:
            kept.append(0)
            nxt.append(-1)
            continue
        parent = []
        for i in range(n):
            seen = [j for j in range(i) if (mask is None and j == i - 1) or (mask is not None and int(mask[lo + i]) >> j & 1)]
            parent.append(seen[-1] if seen else -1)
        cur, walk, s, z, out = 0, [0], 0.0, 1.0, set()
        p = probs[lo].double()
        for i in range(1, n):
            if parent[i] != cur:
                continue
            x = int(tokens[lo + i])
            w = (p - s * draft[lo + cur].double()).clamp_min(0) if draft is not None else p.clone()
            if draft is None and out:
                w[list(out)] = 0
            ok = 0 <= x < len(p)
            left = float(w[x]) if ok else 0.0
            test = float(u[lo + i]) * z * (float(draft[lo + cur, x]) if draft is not None and ok else 1.0)
            if ok:
                near = min(near, abs(test - left))
            if ok and test < left:
                walk.append(i)
                cur, s, z, out = i, 0.0, 1.0, set()
                p = probs[lo + i].double()
            elif draft is not None:
                s += z
                z = float((p - s * draft[lo + cur].double()).clamp_min(0).sum())
            else:
                z -= left
                if ok:
                    out.add(x)
        w = (p - s * draft[lo + cur].double()).clamp_min(0) if draft is not None else p.clone()
        if draft is None and out:
            w[list(out)] = 0
        if float(w.sum()) <= 0:
            w = p
        total = float(w.sum())
        if total <= 0:
            nxt.append(-1)
        else:
            c = w.cumsum(0)
            over = (c > float(u_next[b]) * float(c[-1])).nonzero()
            last = int(w.nonzero()[-1])
            nxt.append(min(int(over[0]), last) if len(over) else last)
            near = min(near, float((c[w > 0] - float(u_next[b]) * float(c[-1])).abs().min()) / total)
        path += walk + [-1] * (n - len(walk))
        kept.append(len(walk))
    return path, kept, nxt, near


def fork(table, lens, parents, new, refs, page):
    """(table, refs, copy_src, copy_dst) of the next batch, as lists."""
    pages = lambda n: -(-n // page)
    width = len(table[0]) if table else 0
    free = [p for p, n in enumerate(refs) if n == 0]
    now, out, src, dst = list(refs), [], [], []
    for b, n in enumerate(lens):
        for j in range(pages(n)):
            now[table[b][j]] -= 1
    for i, r in enumerate(parents):
        old = lens[r] if r >= 0 else 0
        mine = table[r][:min(pages(old), pages(new[i]))] if r >= 0 else []
        a = b = -1
        if new[i] > old and old % page:
            others = [k for k, q in enumerate(parents) if q == r and pages(new[k]) >= pages(old)]
            alone = refs[mine[-1]] == 1 and all(new[k] > old for k in others) and others[0] == i
            if not alone:
                a, b = mine[-1], free.pop(0)
                mine = mine[:-1] + [b]
        while len(mine) < pages(new[i]):
            mine = mine + [free.pop(0)]
        for p in mine:
            now[p] += 1
        out.append(mine)
        src.append(a)
        dst.append(b)
    return [m + [-1] * (width - len(m)) for m in out], now, src, dst
