"""Sampling several continuations of one prompt, and drafts that are verified, as measured work.

Five operators around the paged cache: attention of new tokens for sequences
that share a prefix, read once for all of them (`attend`); verification of
drafted tokens, a chain or a tree, against the target's probabilities from given
random numbers (`verify`); the next batch's page table, with forked, dropped,
grown and trimmed sequences (`fork`); copying pages (`copy`) and moving the rows
of accepted drafts together (`compact`).  `run` computes them in plain torch
when `own` is false and through the framework's calls when it is true; `exact`
is a separate restatement in fp64.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # four answers to one short question, one token each: latency
        dict(name="attend few", op="attend", B=4, groups=1, T=1, P=1000, S=60, Hq=32, Hk=8, d=128, kv="bf16", page=16, spread=0.4, chain=True),
        # 64 samples of one long prompt, a token each: the prefix is arithmetic, the samples' own keys are reading
        dict(name="attend samples", op="attend", B=64, groups=1, T=1, P=16384, S=1024, Hq=32, Hk=8, d=128, kv="bf16", page=64, spread=0.6, chain=True),
        # eight prompts with 16 samples each over an 8-bit cache, prompts and samples ragged
        dict(name="attend prompts e4m3", op="attend", B=128, groups=8, T=1, P=8192, S=512, Hq=64, Hk=8, d=128, kv="e4m3", page=16, spread=0.5, chain=True),
        # trees of 16 drafts for 32 samples of one long document: the most arithmetic
        dict(name="attend drafts", op="attend", B=32, groups=1, T=16, P=32768, S=777, Hq=32, Hk=8, d=128, kv="bf16", page=128, spread=0.3, chain=False),
        # four drafts in a row for a few sequences, the draft's tokens taken as certain, an odd vocabulary
        dict(name="verify chains", op="verify", B=8, T=5, V=50021, kind="bf16", draft=False, spread=0.0, chain=True),
        # trees of up to 16 drafts for 64 sequences, with the draft's probabilities
        dict(name="verify trees", op="verify", B=64, T=16, V=131072, kind="fp32", draft=True, spread=0.5, chain=False),
        # a decoding step: every sequence goes on by a few tokens, some share the page that they write to
        dict(name="fork step", op="fork", B=64, N=64, W=256, page=16, L=2000, T=5, spare=4096, turnover=0.0, spread=0.7),
        # sampling starts: a third of the rows goes, the others fork into their places and into more
        dict(name="fork samples", op="fork", B=256, N=512, W=512, page=16, L=6000, T=64, spare=65536, turnover=0.4, spread=0.8),
        # a few half-filled pages that forked sequences write to
        dict(name="copy few", op="copy", n=24, hit=0.6, pages=600, Hk=8, d=128, kv="bf16", page=16),
        # a batch's pages moved together
        dict(name="copy batch", op="copy", n=2000, hit=1.0, pages=4100, Hk=8, d=128, kv="e4m3", page=64),
        # accepted drafts of a few chains over a small cache
        dict(name="compact few", op="compact", B=4, T=6, L=900, Hk=4, d=64, kv="bf16", page=16, spread=0.3),
        # accepted drafts of many large trees over an 8-bit cache
        dict(name="compact trees", op="compact", B=256, T=64, L=700, Hk=8, d=128, kv="e4m3", page=32, spread=0.4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "verify", "verify", "fork", "copy", "compact"])
    spread = round(rng.random() * 0.9, 3)
    if op == "verify":
        return dict(op=op, B=_log_int(rng, 1, 64), T=_log_int(rng, 1, 16), V=_log_int(rng, 1000, 131072), kind=rng.choice(["fp32", "bf16"]),
                    draft=rng.random() < 0.6, spread=spread, chain=rng.random() < 0.4)
    if op == "fork":
        page, L, B = rng.choice([16, 32, 64, 128, 256]), _log_int(rng, 1, 6000), _log_int(rng, 1, 256)
        T = _log_int(rng, 1, 64)
        return dict(op=op, B=B, N=_log_int(rng, 1, 2 * B + 1), W=(L + T) // page + rng.randrange(1, 40), page=page, L=L, T=T,
                    spare=_log_int(rng, 100, 65536), turnover=round(rng.random(), 3), spread=spread)
    kv, page, d, Hk = rng.choice(["bf16", "e4m3"]), rng.choice([16, 32, 64, 128, 256]), rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    if op == "copy":
        n = _log_int(rng, 1, max(1, 128000 // page))
        return dict(op=op, n=n, hit=rng.choice([1.0, 0.5]), pages=2 * n + rng.randrange(1, 50), Hk=Hk, d=d, kv=kv, page=page)
    if op == "compact":
        T = _log_int(rng, 1, 64)
        return dict(op=op, B=_log_int(rng, 1, 256), T=T, L=_log_int(rng, T, 700), Hk=Hk, d=d, kv=kv, page=page, spread=spread)
    T = rng.choice([1, 1, _log_int(rng, 2, 16)])
    B = _log_int(rng, 2, 128 // T if T > 1 else 128)
    return dict(op=op, B=B, groups=min(B, rng.choice([1, 1, 2, 5, 8])), T=T, P=_log_int(rng, 100, 32768), S=_log_int(rng, T, 1024),
                Hq=Hk * rng.choice([1, 2, 3, 4]), Hk=Hk, d=d, kv=kv, page=page, spread=spread, chain=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs --
def _spread(n, top, spread, least=1):
    """n lengths up to `top`, spread evenly over the last `spread` of it; the first is `top`."""
    return [max(least, top - int(spread * top * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]


def _new_lens(c):
    return _spread(c["B"], c["T"], c["spread"])


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _cache(c, g, pages):
    """A paged cache filled with plausible keys and values."""
    s = {}
    for n in ("k", "v"):
        x = _normal(g, pages, c["page"], c["Hk"], c["d"])
        s[n + "_cache"], s[n + "_scale"] = x, None
        if c["kv"] == "e4m3":  # one scale for each row
            x = x.float()
            scale = (x.abs().amax(-1) / 448.0).clamp_min(2.0 ** -64)
            s[n + "_cache"] = (x * (1.0 / scale)[..., None]).clamp(-448.0, 448.0).to(FP8)
            s[n + "_scale"] = scale.permute(0, 2, 1).contiguous()  # [pages, Hk, page]
    return s


def _shuffled(g, pages):
    return torch.randperm(pages, generator=g, device="cuda").to(torch.int32)


def _tree_mask(lens, seed):
    """Random trees: each drafted token sees itself and its ancestors. One 64-bit word for each token."""
    import random
    rng, words = random.Random(seed), []
    for n in lens:
        mine = []
        for i in range(n):
            up = mine[rng.randrange(max(0, i - 6), i)] if i else 0
            mine.append(up | (1 << i))
        words += mine
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")


def _members(c):
    """Offsets of the groups in the batch: about as many sequences each."""
    return [i * c["B"] // c["groups"] for i in range(c["groups"] + 1)]


def _plan(c):
    """(groups' offsets, their prefixes, sequences' lengths, their new tokens) of an attend case."""
    at, new = _members(c), _new_lens(c)
    prefix = _spread(c["groups"], c["P"], c["spread"])
    mine = [prefix[g] for g in range(c["groups"]) for _ in range(at[g], at[g + 1])]
    lens = [p + max(n, s) for p, n, s in zip(mine, new, _spread(c["B"], c["S"], c["spread"]))]
    return at, prefix, lens, new


def _prepare_attend(c, g, seed):
    at, prefix, lens, new = _plan(c)
    page = c["page"]
    per = [-(-n // page) for n in lens]
    shared = [p // page for p in prefix]  # whole pages
    pages = sum(shared) + sum(per[b] - shared[k] for k in range(c["groups"]) for b in range(at[k], at[k + 1])) + 3
    s = _cache(c, g, pages)
    order = _shuffled(g, pages)
    table = torch.zeros((c["B"], max(per)), dtype=torch.int32, device="cuda")
    used = 0
    for k in range(c["groups"]):
        common = order[used:used + shared[k]]
        used += shared[k]
        for b in range(at[k], at[k + 1]):
            table[b, :shared[k]] = common
            table[b, shared[k]:per[b]] = order[used:used + per[b] - shared[k]]
            used += per[b] - shared[k]
    cu = _offsets(new)
    s.update(page_table=table, seqlens=_int(lens), cu=_int(cu), total=cu[-1], max_new=max(new), max_len=max(lens),
             cu_groups=_int(at), prefix_lens=_int(prefix), max_prefix=max(prefix),
             max_group=max(cu[at[k + 1]] - cu[at[k]] for k in range(c["groups"])),
             longest_tail=max(lens[b] - shared[k] * page for k in range(c["groups"]) for b in range(at[k], at[k + 1])))
    s["q"] = _normal(g, cu[-1], c["Hq"], c["d"], std=1.5)
    s["mask"] = None if c["chain"] else _tree_mask(new, seed)
    return s


def _prepare_verify(c, g, seed):
    new = _new_lens(c)
    cu = _offsets(new)
    total, V = cu[-1], c["V"]
    kind = torch.float32 if c["kind"] == "fp32" else torch.bfloat16
    target = torch.randn(total, V, generator=g, device="cuda") * 3.0
    draft = target + 0.8 * torch.randn(total, V, generator=g, device="cuda")
    s = {"probs": target.softmax(-1).to(kind), "cu": _int(cu), "max_new": max(new)}
    del target
    draft = draft.softmax(-1).to(kind)
    s["mask"] = None if c["chain"] else _tree_mask(new, seed)
    # node i's token is drawn from the draft's distribution at its parent
    b, i = _owner(s["cu"], total)
    up = s["cu"].long()[b] + _parents(s["mask"], i).clamp_min(0)
    noise = torch.empty(total, V, device="cuda").exponential_(generator=g)
    s["tokens"] = (draft[up].float() / noise).argmax(-1).to(torch.int32)
    s["draft_probs"] = draft if c["draft"] else None
    s["u"] = torch.rand(total, generator=g, device="cuda")
    s["u_next"] = torch.rand(c["B"], generator=g, device="cuda")
    s["seqlens"] = _int([700 + 13 * k + n for k, n in enumerate(new)])
    return s


def _fork_plan(c, seed):
    """(old lengths, parents, new lengths)."""
    import random
    rng = random.Random(seed)
    lens = _spread(c["B"], c["L"], c["spread"])
    lens = [lens[b - 1] if b % 6 == 2 else n for b, n in enumerate(lens)]
    room = c["W"] * c["page"]
    fresh = c["turnover"]
    parents = []
    for i in range(c["N"]):
        x = rng.random()
        parents.append(i if i < c["B"] and x >= fresh else -1 if x < 0.1 * fresh else rng.randrange(c["B"]))
    new = []
    for p in parents:
        old = lens[p] if p >= 0 else 0
        new.append(max(0, min(room, old + rng.randrange(-(c["T"] // 3), c["T"] + 1) if fresh else old + rng.randrange(1, c["T"] + 1))))
    return lens, parents, new


def _fork_pages(c, lens):
    """A pool with room for all rows, old and new."""
    return sum(-(-n // c["page"]) for n in lens) + c["N"] * (-(-(c["L"] + c["T"]) // c["page"]) + 1) + c["spare"]


def _prepare_fork(c, g, seed):
    lens, parents, new = _fork_plan(c, seed)
    page = c["page"]
    per = [-(-n // page) for n in lens]
    pages = _fork_pages(c, lens)
    order = _shuffled(g, pages)
    table = torch.full((c["B"], c["W"]), -1, dtype=torch.int32, device="cuda")
    used = 0
    for b, n in enumerate(per):
        # some rows were forked from the one before them: all its pages, or whole ones of a common beginning
        take = n if b % 6 == 2 else min(lens[b - 1], lens[b]) // (2 * page) if b % 6 == 5 else 0
        if take:
            table[b, :take] = table[b - 1, :take]
        table[b, take:n] = order[used:used + n - take]
        used += n - take
    held = table[table >= 0].long()
    refs = torch.bincount(held, minlength=pages).to(torch.int32)
    return {"page_table": table, "seqlens": _int(lens), "parents": _int(parents), "new_seqlens": _int(new), "refs": refs}


def _prepare_copy(c, g, seed):
    s = _cache(c, g, c["pages"])
    order = _shuffled(g, c["pages"] - 1)  # the last page stays free
    hit = torch.rand(c["n"], generator=g, device="cuda") < c["hit"]
    hit[0] = True
    s["src"] = torch.where(hit, order[:c["n"]], -1)
    s["dst"] = torch.where(hit, order[c["n"]:2 * c["n"]], -1)
    return s


def _prepare_compact(c, g, seed):
    import random
    rng = random.Random(seed)
    new = _new_lens(c)
    lens = [max(a, b) for a, b in zip(new, _spread(c["B"], c["L"], c["spread"]))]
    per = [-(-n // c["page"]) for n in lens]
    pages = sum(per) + 3
    s = _cache(c, g, pages)
    order = _shuffled(g, pages)
    table = torch.zeros((c["B"], max(per)), dtype=torch.int32, device="cuda")
    at = _offsets(per)
    for b, n in enumerate(per):
        table[b, :n] = order[at[b]:at[b + 1]]
    path, kept = [], []
    for n in new:  # the root, then an increasing walk through the drafts
        keep, i = [0], 0
        while rng.random() < 0.8:
            i += rng.randrange(1, 4)
            if i >= n:
                break
            keep.append(i)
        path += keep + [-1] * (n - len(keep))
        kept.append(len(keep))
    s.update(page_table=table, seqlens=_int(lens), cu=_int(_offsets(new)), total=sum(new), path=_int(path), accepted=_int(kept))
    return s


def prepare(case, seed):
    make = {"attend": _prepare_attend, "verify": _prepare_verify, "fork": _prepare_fork, "copy": _prepare_copy, "compact": _prepare_compact}
    s = make[case["op"]](case, _gen(seed), seed)
    s["case"] = case
    return s


# --------------------------------------------------------------- plain form --
def _owner(cu, total):
    """Sequence of each packed token, and its place there."""
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(cu.long(), t, right=True) - 1
    return b, t - cu.long()[b]


def _parents(mask, i):
    """Each token's parent in its tree: the highest token below it that it sees; -1 without one."""
    if mask is None:
        return i - 1
    j = torch.arange(64, device="cuda")
    seen = ((mask[:, None] >> j) & 1).bool() & (j < i[:, None])
    return torch.where(seen, j, -1).amax(-1)


def _take(cache, scale, page, at):
    """fp32 rows of a cache."""
    if scale is None:
        return cache[page, at].float()
    codes = cache.view(torch.uint8)[page, at].view(FP8).float()
    return codes * scale.permute(0, 2, 1)[page, at][..., None]


def _part(q, k, v, seen):
    """(sum of weighted values, sum of weights, largest score) of rows q [n, Hk, r, d] over keys [n, l, Hk, d]; seen [n, 1, r, l]."""
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(q.shape[-1] ** -0.5).masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp_min(-1e30)
    p = scores.sub_(top).exp_()
    return torch.matmul(p, v.permute(0, 2, 1, 3)), p.sum(-1, keepdim=True), top


def _attend(s):
    c = s["case"]
    B, T, Hk, d, page, G, R = c["B"], s["max_new"], c["Hk"], c["d"], c["page"], c["Hq"] // c["Hk"], s["max_group"]
    b, i = _owner(s["cu"], s["total"])
    new, lens, cu = (s["cu"][1:] - s["cu"][:-1]).long(), s["seqlens"].long(), s["cu"].long()
    group = torch.searchsorted(s["cu_groups"].long(), torch.arange(B, device="cuda"), right=True) - 1
    shared = s["prefix_lens"].long() // page * page  # whole pages are shared
    rows = s["q"].float().view(-1, Hk, G, d)

    def keys(table, pos, last):
        pos = torch.minimum(pos, last)
        at = torch.gather(table.long(), 1, pos // page)
        return [_take(s[n + "_cache"], s[n + "_scale"], at, pos % page) for n in ("k", "v")]

    # every group's rows over its prefix
    n = c["groups"]
    q = torch.zeros((n, R, Hk, G, d), device="cuda")
    slot = torch.arange(s["total"], device="cuda") - cu[s["cu_groups"].long()[group[b]]]
    q[group[b], slot] = rows
    pos = torch.arange(max(1, s["max_prefix"] // page * page), device="cuda")[None].expand(n, -1)
    k, v = keys(s["page_table"][s["cu_groups"][:-1].long()], pos, (shared[:, None] - 1).clamp_min(0))
    o1, l1, m1 = _part(q.permute(0, 2, 1, 3, 4).reshape(n, Hk, R * G, d), k, v, (pos < shared[:, None])[:, None, None])
    o1, l1, m1 = (x.view(n, Hk, R, G, -1).permute(0, 2, 1, 3, 4)[group[b], slot] for x in (o1, l1, m1))
    # every sequence's over what is its own
    q = torch.zeros((B, T, Hk, G, d), device="cuda")
    q[b, i] = rows
    pos = shared[group][:, None] + torch.arange(s["longest_tail"], device="cuda")
    k, v = keys(s["page_table"], pos, lens[:, None] - 1)
    draft = pos - (lens - new)[:, None]  # < 0: context
    word = torch.zeros((B, T), dtype=torch.int64, device="cuda")
    word[b, i] = s["mask"] if s["mask"] is not None else -1
    bit = (word[:, :, None] >> draft.clamp(0, 63)[:, None]) & 1
    seen = (draft < 0)[:, None] | (bit.bool() & (pos < lens[:, None])[:, None])
    if s["mask"] is None:
        seen = seen & (draft[:, None] <= torch.arange(T, device="cuda")[None, :, None])
    seen = seen[:, :, None].expand(-1, -1, G, -1).reshape(B, 1, T * G, -1)
    o2, l2, m2 = _part(q.permute(0, 2, 1, 3, 4).reshape(B, Hk, T * G, d), k, v, seen)
    o2, l2, m2 = (x.view(B, Hk, T, G, -1).permute(0, 2, 1, 3, 4)[b, i] for x in (o2, l2, m2))
    top = torch.maximum(m1, m2)
    w1, w2 = (m1 - top).exp(), (m2 - top).exp()
    l = l1 * w1 + l2 * w2
    o = (o1 * w1 + o2 * w2) / l.clamp_min(1e-30)
    return o.reshape(-1, c["Hq"], d).to(torch.bfloat16), (top + l.log()).reshape(-1, c["Hq"])


def _verify(s):
    """The walk through each tree, in 64 bits: a test and the residual of a rejection lie next to borders."""
    cu, tokens, q = s["cu"].long(), s["tokens"].long(), s["draft_probs"]
    start, n = cu[:-1], cu[1:] - cu[:-1]
    total, B = tokens.numel(), n.numel()
    _, i = _owner(s["cu"], total)
    parent = _parents(s["mask"], i)
    path = torch.full((total + 1,), -1, dtype=torch.int32, device="cuda")  # the last takes what has no place
    path[torch.where(n > 0, start, total)] = 0
    cur = torch.zeros(B, dtype=torch.int64, device="cuda")
    kept = (n > 0).long()
    s_, z = torch.zeros(B, dtype=torch.float64, device="cuda"), torch.ones(B, dtype=torch.float64, device="cuda")
    out = torch.zeros((B, s["probs"].shape[1]), dtype=torch.bool, device="cuda")  # tokens rejected at the node, without q
    seq = torch.arange(B, device="cuda")

    def row(x):
        return x[(start + cur).clamp_max(total - 1)].double()

    def left():
        """What is left of the node's distribution."""
        if q is None:
            return row(s["probs"]).masked_fill(out, 0.0)
        return (row(s["probs"]) - s_[:, None] * row(q)).clamp_min(0.0)

    for at in range(1, s["max_new"]):
        node = (start + at).clamp_max(total - 1)
        here = (at < n) & (parent[node] == cur)
        tok = tokens[node]
        w = left()
        mine = w[seq, tok]
        test = s["u"][node].double() * z
        test = test if q is None else test * q[(start + cur).clamp_max(total - 1), tok].double()
        yes = here & (test < mine)
        no = here & ~yes
        if q is None:
            z = torch.where(no, z - mine, z)
            out[seq, tok] |= no
        else:
            s_ = torch.where(no, s_ + z, s_)
            z = torch.where(no, left().sum(-1), z)
        path[torch.where(yes, start + kept, total)] = at
        cur, kept = torch.where(yes, at, cur), kept + yes
        s_, z = s_.masked_fill(yes, 0.0), z.masked_fill(yes, 1.0)
        out &= ~yes[:, None]
    w = left()
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, row(s["probs"]))
    cdf = w.cumsum(-1)
    nxt = (cdf <= s["u_next"].double()[:, None] * cdf[:, -1:]).sum(-1)
    last = torch.where(w > 0, torch.arange(w.shape[1], device="cuda"), -1).amax(-1)
    nxt = torch.where(n > 0, torch.minimum(nxt, last), -1)
    return path[:total], kept.to(torch.int32), nxt.to(torch.int32), (s["seqlens"] - n + kept).to(torch.int32)


def _fork(s):
    page, table, lens, new, refs = s["case"]["page"], s["page_table"].long(), s["seqlens"].long(), s["new_seqlens"].long(), s["refs"]
    B, W = table.shape
    N, pages = new.numel(), refs.numel()
    up = s["parents"].long().clamp_min(0)
    old = torch.where(s["parents"] >= 0, lens[up], 0)
    had, needs = (old + page - 1) // page, (new + page - 1) // page
    keep = torch.minimum(had, needs)
    held = table[up]
    last = held.gather(1, (had - 1).clamp_min(0)[:, None])[:, 0].clamp_min(0)
    grows = (new > old) & (old % page != 0)  # into a page that holds something
    # one writer may keep that page: the first, where no other sequence reads it
    stays = (s["parents"] >= 0) & (keep == had) & ~grows
    read = torch.zeros(B, dtype=torch.int64, device="cuda").scatter_reduce(0, up, stays.long(), "amax")
    i = torch.arange(N, device="cuda")
    first = torch.full((B,), N, device="cuda").scatter_reduce(0, up, torch.where(grows, i, N), "amin")
    copies = grows & ~((refs[last] == 1) & (read[up] == 0) & (first[up] == i))
    asks = copies.long() + needs - keep
    at = (asks.cumsum(0) - asks)[:, None]
    # free pages in order
    free = refs == 0
    order = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    order[torch.where(free, free.long().cumsum(0) - 1, pages)] = torch.arange(pages, device="cuda")
    j = torch.arange(W, device="cuda")[None]
    fresh = order[(at + copies[:, None] + j - keep[:, None]).clamp(0, pages)]
    out = torch.where(j < keep[:, None], held, torch.where(j < needs[:, None], fresh, -1))
    moved = order[at.clamp_max(pages)]
    out = torch.where(copies[:, None] & (j == had[:, None] - 1), moved, out)
    now = torch.cat([refs, refs.new_zeros(1)])  # the last counts what is no page
    had_all = (lens[:, None] + page - 1) // page
    now.index_add_(0, torch.where(j < had_all, table, pages).flatten(), torch.full((B * W,), -1, dtype=torch.int32, device="cuda"))
    now.index_add_(0, torch.where(j < needs[:, None], out, pages).flatten(), torch.ones(N * W, dtype=torch.int32, device="cuda"))
    return (out.to(torch.int32), now[:pages], torch.where(copies, last, -1).to(torch.int32), torch.where(copies, moved[:, 0], -1).to(torch.int32))


def _buffers(s):
    return [(s[n], n.endswith("scale")) for n in ("k_cache", "v_cache", "k_scale", "v_scale") if s[n] is not None]


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == FP8 else x  # indexing moves bytes


def _copy(s):
    spare = s["case"]["pages"] - 1
    src, dst = torch.where(s["src"] >= 0, s["src"], spare).long(), torch.where(s["src"] >= 0, s["dst"], spare).long()
    for x, _ in _buffers(s):
        _bytes(x)[dst] = _bytes(x)[src]
    return tuple(x for x, _ in _buffers(s))


def _compact(s):
    page = s["case"]["page"]
    b, i = _owner(s["cu"], s["total"])
    base = (s["seqlens"] - (s["cu"][1:] - s["cu"][:-1])).long()[b]
    to, come = base + i, base + torch.where(i < s["accepted"][b], s["path"].long(), i)  # other rows stay
    at = [(s["page_table"][b, p // page].long(), p % page) for p in (to, come)]
    for x, scale in _buffers(s):
        x = _bytes(x.permute(0, 2, 1) if scale else x)
        x[at[0]] = x[at[1]]
    return tuple(x for x, _ in _buffers(s))


def _plain(s):
    return {"attend": _attend, "verify": _verify, "fork": _fork, "copy": _copy, "compact": _compact}[s["case"]["op"]](s)


def _own(s):
    import io_aware_exact_06_gb300 as fa
    op = s["case"]["op"]
    if op == "attend":
        return fa.prefix_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seqlens"], s["cu"], s["max_new"], s["max_len"],
                                s["cu_groups"], s["prefix_lens"], s["max_group"], s["max_prefix"], mask=s["mask"],
                                k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "verify":
        return fa.verify_drafts(s["tokens"], s["probs"], s["cu"], s["u"], s["u_next"], draft_probs=s["draft_probs"], mask=s["mask"],
                                seqlens=s["seqlens"])
    if op == "fork":
        return fa.cache_fork(s["page_table"], s["seqlens"], s["parents"], s["new_seqlens"], s["refs"], s["case"]["page"])
    if op == "copy":
        fa.cache_copy(s["k_cache"], s["v_cache"], s["src"], s["dst"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        fa.cache_compact(s["k_cache"], s["v_cache"], s["page_table"], s["seqlens"], s["cu"], s["path"], s["accepted"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"])
    return tuple(x for x, _ in _buffers(s))


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work --
def work(case):
    c = case
    if c["op"] == "verify":  # a row of the target's, and of the draft's, for the last node of each sequence
        size = 4 if c["kind"] == "fp32" else 2
        rows = c["B"] * (2 if c["draft"] else 1)
        return {"bytes": rows * c["V"] * size + 16 * sum(_new_lens(c)), "flops": 3 * c["B"] * c["V"]}
    if c["op"] == "fork":
        lens, _, _ = _fork_plan(c, 0)
        held, pages = sum(-(-n // c["page"]) for n in lens), _fork_pages(c, lens)
        return {"bytes": 4 * (held + c["N"] * c["W"] + 2 * pages), "flops": pages + held + c["N"] * c["W"]}
    size, scale = (1, 4) if c["kv"] == "e4m3" else (2, 0)
    row = c["Hk"] * (c["d"] * size + scale)  # a token's keys (or values) in the cache
    if c["op"] == "copy":
        rows = c["page"] * max(1, int(c["n"] * c["hit"]))
        return {"bytes": 4 * rows * row, "flops": 0}
    if c["op"] == "compact":  # a walk keeps four drafts or so
        rows = sum(min(4, n) for n in _new_lens(c))
        return {"bytes": 4 * rows * row, "flops": 0}
    at, prefix, lens, new = _plan(c)
    whole = [p // c["page"] * c["page"] for p in prefix]
    keys = sum(whole) + sum(lens[b] - whole[k] for k in range(c["groups"]) for b in range(at[k], at[k + 1]))
    return {"bytes": 2 * keys * row + sum(new) * c["Hq"] * (4 * c["d"] + 4) + (0 if c["chain"] else 8 * sum(new)),
            "flops": sum(4 * t * n * c["Hq"] * c["d"] for t, n in zip(new, lens))}


# ------------------------------------------------------------------- exact --
def _exact_attend(s, c):
    """One sequence after the other, over its own page table alone."""
    starts, lens, table, G = s["cu"].tolist(), s["seqlens"].tolist(), s["page_table"].long(), c["Hq"] // c["Hk"]
    outs, lses = [], []
    for b, L in enumerate(lens):
        T = starts[b + 1] - starts[b]
        p = torch.arange(L, device="cuda")
        where = table[b][p // c["page"]], p % c["page"]
        kv = []
        for n in ("k", "v"):
            if s[n + "_scale"] is None:
                kv.append(s[n + "_cache"][where].double())
            else:
                kv.append(s[n + "_cache"].view(torch.uint8)[where].view(FP8).double() * s[n + "_scale"].transpose(1, 2)[where].double()[..., None])
        q = s["q"][starts[b]:starts[b + 1]].double().unflatten(1, (c["Hk"], G))
        see = torch.ones((T, L), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            see[:, L - T:] = torch.ones((T, T), device="cuda").tril().bool()
        else:
            words = s["mask"][starts[b]:starts[b + 1]]
            see[:, L - T:] = (words[:, None] >> torch.arange(T, device="cuda")) % 2 == 1
        x = torch.einsum("thgd,lhd->htgl", q, kv[0]) / math.sqrt(c["d"])
        x = torch.where(see[None, :, None], x, -math.inf)
        lse = torch.logsumexp(x, -1)
        o = torch.einsum("htgl,lhd->thgd", (x - lse[..., None]).exp(), kv[1])
        outs.append(o.flatten(1, 2))
        lses.append(lse.transpose(0, 1).flatten(1, 2))
    return torch.cat(outs), torch.cat(lses)


def _exact_verify(s, c):
    """One sequence after the other: draw from the normed residual, subtract, norm again."""
    cu, tokens, u = s["cu"].tolist(), s["tokens"].tolist(), s["u"].tolist()
    words = None if s["mask"] is None else s["mask"].tolist()
    path, kept, nxt = [], [], []
    for b in range(c["B"]):
        lo, n = cu[b], cu[b + 1] - cu[b]
        walk, node = [0], 0
        dist = s["probs"][lo].double()
        for i in range(1, n):
            below = [j for j in range(i) if words is None or words[lo + i] >> j & 1]
            if not below or below[-1] != node:
                continue
            x = tokens[lo + i]
            other = torch.zeros_like(dist).index_fill_(0, torch.tensor([x], device="cuda"), 1.0) if s["draft_probs"] is None \
                else s["draft_probs"][lo + node].double()
            if u[lo + i] * float(other[x]) < float(dist[x]):
                walk.append(i)
                node, dist = i, s["probs"][lo + i].double()
            else:
                rest = (dist - other).clamp_min(0.0)
                # without the draft's probabilities the target's are taken to add up to one
                size = float(rest.sum()) if s["draft_probs"] is not None else 1.0 - float(dist[x])
                dist = rest / size if size > 0 else rest
        if float(dist.sum()) <= 0:
            dist = s["probs"][lo + node].double()
        cdf = dist.cumsum(0)
        at = int(torch.searchsorted(cdf, cdf[-1:] * float(s["u_next"][b]), right=True))
        nxt.append(min(at, int(dist.nonzero()[-1])))
        path += walk + [-1] * (n - len(walk))
        kept.append(len(walk))
    lens = [L - (cu[b + 1] - cu[b]) + kept[b] for b, L in enumerate(s["seqlens"].tolist())]
    return _int(path), _int(kept), _int(nxt), _int(lens)


def _exact_fork(s, c):
    """Page after page, on the host."""
    page, refs = c["page"], s["refs"].tolist()
    table, lens, new, parents = (s[n].tolist() for n in ("page_table", "seqlens", "new_seqlens", "parents"))
    pages_of = lambda n: -(-n // page)  # noqa: E731
    free = iter([p for p, n in enumerate(refs) if n == 0])
    now = list(refs)
    for b, n in enumerate(lens):
        for j in range(pages_of(n)):
            now[table[b][j]] -= 1
    children = {}
    for i, r in enumerate(parents):
        children.setdefault(r, []).append(i)
    out, src, dst = [], [], []
    for i, r in enumerate(parents):
        old = lens[r] if r >= 0 else 0
        mine = list(table[r][:min(pages_of(old), pages_of(new[i]))]) if r >= 0 else []
        a = b = -1
        if new[i] > old and old % page:
            holders = [k for k in children[r] if pages_of(new[k]) >= pages_of(old)]
            if not (refs[mine[-1]] == 1 and i == holders[0] and all(new[k] > old for k in holders)):
                a, b = mine[-1], next(free)
                mine[-1] = b
        while len(mine) < pages_of(new[i]):
            mine.append(next(free))
        for p in mine:
            now[p] += 1
        src.append(a)
        dst.append(b)
        out.append(mine + [-1] * (c["W"] - len(mine)))
    return _int(out), _int(now), _int(src), _int(dst)


def _exact_move(s, c):
    """Rows (or whole pages) moved one by one in a copy of the cache, on the host's list of them."""
    moves = []
    if c["op"] == "copy":
        moves = [(a * c["page"], b * c["page"], c["page"]) for a, b in zip(s["src"].tolist(), s["dst"].tolist()) if a >= 0]
    else:
        table, lens, cu, path, kept = (s[n].tolist() for n in ("page_table", "seqlens", "cu", "path", "accepted"))
        for b, L in enumerate(lens):
            base = L - (cu[b + 1] - cu[b])
            spot = lambda p: table[b][p // c["page"]] * c["page"] + p % c["page"]  # noqa: E731
            moves += [(spot(base + path[cu[b] + j]), spot(base + j), 1) for j in range(kept[b])]
    outs = []
    for x, scale in _buffers(s):
        x = x.double()
        flat = (x.transpose(1, 2) if scale else x).flatten(0, 1).clone()
        was = flat.clone()
        for length in sorted({m[2] for m in moves}):
            step = torch.arange(length, device="cuda")
            come, to = (torch.tensor([m[e] for m in moves], device="cuda")[:, None] + step for e in (0, 1))
            flat[to.flatten()] = was[come.flatten()]
        flat = flat.unflatten(0, (-1, c["page"]))
        outs.append(flat.transpose(1, 2) if scale else flat)
    return tuple(outs)


def exact(case, seed):
    s = prepare(case, seed)
    make = {"attend": _exact_attend, "verify": _exact_verify, "fork": _exact_fork, "copy": _exact_move, "compact": _exact_move}
    return make[case["op"]](s, case)
