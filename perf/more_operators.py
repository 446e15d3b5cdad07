"""The pages of a 4-bit cache and attention over pages that sessions share: what is timed, the plain
forms and the 64-bit definitions.

Four passes, on the slots of a page pool (slot b's row of the page table holds held[b] pages, refs[p]
counts the rows that hold page p, 0 = free) and on the ragged layout of a verify batch:

* ``branch``: sessions are forked (rows copied, pages shared), pages are reserved for the next round
  (a shared page that the round writes is replaced), and the replaced pages' tokens are copied;
* ``release``: pages past a length are given back;
* ``compact``: live pages move to the front of the pool, tables and bytes with them;
* ``attend``: attention of a round's rows over the paged 4-bit cache in groups of sessions that have
  their first pages in common.

The three passes over pages change the pool, so each begins by setting its tables back (one copy of a
few hundred kilobytes at most, on both sides).  Pages are bytes to them: they come back as the bytes
they are, equal bit for bit.

Cache layout: page p, head h holds a key block and a value block (pages[p, h, 0 / 1]).  A block of P
tokens of D channels is [D/32][P][16] bytes of codes, then [P][D/32] scale bytes.  The 16 bytes of a
group of 32 channels are four little-endian words of 8 channels each; channel e of a word is in bits
4 (e / 2 + 4 (e mod 2)) upwards, as n + 8 with n in -7..7.  A scale byte 8 e + m (8..167) stands for
(1 + m / 8) 2^(e - 15); the value is n times the scale.
"""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
GROUP = 32


# ---- cases --------------------------------------------------------------------------

def listed():
    return [
        # a few sessions that try two continuations each: only the latency of the calls counts
        dict(name="branch_small", op="branch", parents=3, kids_lo=1, kids_hi=2, ctx_lo=10, ctx_hi=300, rows_lo=1, rows_hi=5, page=16,
             kv_heads=2, head_dim=64),
        # a full verify batch, three candidate continuations a session
        dict(name="branch_verify", op="branch", parents=64, kids_lo=3, kids_hi=3, ctx_lo=500, ctx_hi=8200, rows_lo=9, rows_hi=9, page=64,
             kv_heads=8, head_dim=128),
        # a search over many sessions with a ragged number of branches, large pages
        dict(name="branch_large", op="branch", parents=300, kids_lo=0, kids_hi=7, ctx_lo=100, ctx_hi=4000, rows_lo=1, rows_hi=17, page=128,
             kv_heads=8, head_dim=128),
        # the end of a round: most sessions give back what a rejection left over, some end
        dict(name="release_round", op="release", slots=512, family=4, common=1000, ctx_lo=10, ctx_hi=6000, back=17, ended=0.1, page=16),
        # long contexts that end together, all but one, their common prompt among their pages
        dict(name="release_long", op="release", slots=64, family=16, common=90001, ctx_lo=10000, ctx_hi=30000, back=1, ended=1.0, page=16),
        # a small pool
        dict(name="compact_small", op="compact", n_pages=130, slots=7, live=0.5, page=16, kv_heads=4, head_dim=64),
        # a pool after hours of sessions that come and go
        dict(name="compact_large", op="compact", n_pages=12000, slots=200, live=0.55, page=64, kv_heads=8, head_dim=128),
        # four continuations of one prompt, a token each: latency
        dict(name="attend_single", op="attend", groups=1, size_lo=4, size_hi=4, m_lo=0, m_hi=0, q_heads=32, kv_heads=8, head_dim=128, page=16,
             prefix_lo=2001, prefix_hi=2001, own_lo=1, own_hi=40),
        # verify batches of eight sessions a prompt: 9 rows a session, 8 query heads on a cached head
        dict(name="attend_verify", op="attend", groups=8, size_lo=8, size_hi=8, m_lo=8, m_hi=8, q_heads=64, kv_heads=8, head_dim=128, page=64,
             prefix_lo=4000, prefix_hi=8200, own_lo=100, own_hi=1000),
        # many ragged groups, sessions alone among them, small heads
        dict(name="attend_ragged", op="attend", groups=40, size_lo=1, size_hi=8, m_lo=1, m_hi=16, q_heads=28, kv_heads=4, head_dim=64, page=32,
             prefix_lo=10, prefix_hi=6000, own_lo=0, own_hi=500),
        # one long document, sixteen sessions that ask about it
        dict(name="attend_long", op="attend", groups=1, size_lo=16, size_hi=16, m_lo=4, m_hi=4, q_heads=32, kv_heads=8, head_dim=128, page=64,
             prefix_lo=100001, prefix_hi=100001, own_lo=20, own_hi=600),
        # one system prompt for a whole verify batch
        dict(name="attend_wide", op="attend", groups=1, size_lo=64, size_hi=64, m_lo=8, m_hi=8, q_heads=64, kv_heads=8, head_dim=128, page=64,
             prefix_lo=6000, prefix_hi=6000, own_lo=1, own_hi=600),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n))


def draw(rng):
    """One more case: sizes over the whole range, with the work bounded by the largest listed ones."""
    while True:
        case = _drawn(rng)
        if case is not None:
            return case


def _drawn(rng):
    op = rng.choice(["branch", "branch", "release", "compact", "attend", "attend", "attend"])
    dim, page, kv_heads = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8])
    page_bytes = page * kv_heads * 2 * (dim // 2 + dim // GROUP)
    if op == "release":
        slots, hi = _log(rng, 2, 512), _log(rng, 10, 60000)
        case = dict(op=op, slots=slots, family=_log(rng, 1, 16), common=rng.choice([0, _log(rng, 1, 90000)]), ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    back=_log(rng, 1, 200), ended=rng.choice([0.0, 0.1, 1.0]), page=page)
        return case if slots * (case["common"] + hi) // page <= 500000 else None
    if op == "compact":
        n = _log(rng, 10, 30000)
        return dict(op=op, n_pages=n, slots=_log(rng, 1, 300), live=rng.choice([0.05, 0.3, 0.55, 0.9, 1.0]), page=page, kv_heads=kv_heads,
                    head_dim=dim) if n * page_bytes <= 830e6 else None
    if op == "branch":
        parents, kids, hi = _log(rng, 1, 300), _log(rng, 1, 8), _log(rng, 1, 16000)
        rows = _log(rng, 1, 65)
        case = dict(op=op, parents=parents, kids_lo=rng.randint(0, kids), kids_hi=kids, ctx_lo=rng.randint(0, hi), ctx_hi=hi, rows_lo=rng.randint(1, rows),
                    rows_hi=rows, page=page, kv_heads=kv_heads, head_dim=dim)
        most = parents * (hi // page + 2 + (kids + 1) * (rows // page + 2))
        return case if most * page_bytes <= 1.2e9 else None
    groups, size = _log(rng, 1, 64), _log(rng, 1, 64)
    m_hi = rng.choice([0, _log(rng, 1, 64), _log(rng, 1, 16)])
    share = rng.choice([1, 2, 4, 5, 7, 8])
    prefix, tail = _log(rng, 1, 100000), _log(rng, 1, 2000)
    case = dict(op=op, groups=groups, size_lo=rng.randint(1, size), size_hi=size, m_lo=rng.randint(0, m_hi), m_hi=m_hi, q_heads=kv_heads * share,
                kv_heads=kv_heads, head_dim=dim, page=page, prefix_lo=rng.randint(0, prefix), prefix_hi=prefix, own_lo=rng.randint(0, tail), own_hi=tail)
    sessions, tokens = groups * size, prefix + tail + m_hi + 1
    small = sessions <= 512 and sessions * tokens * kv_heads * dim <= 1.7e9 and sessions * tokens * (m_hi + 1) * case["q_heads"] <= 3e8
    return case if small else None


def _shape(case):
    """The ragged sizes of a case, fixed by the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    many = lambda lo, hi, n: [rng.randint(lo, hi) for _ in range(n)]  # noqa: E731
    if case["op"] == "branch":
        kids = many(case["kids_lo"], case["kids_hi"], case["parents"])
        n = case["parents"] + sum(kids)
        return dict(kids=kids, n=n, ctx=many(case["ctx_lo"], case["ctx_hi"], case["parents"]), rows=many(case["rows_lo"], case["rows_hi"], n),
                    spare=many(0, 1, case["parents"]))
    if case["op"] == "release":
        n = case["slots"]
        return dict(n=n, own=many(case["ctx_lo"], case["ctx_hi"], n), back=many(0, case["back"], n),
                    what=[rng.random() for _ in range(n)])
    if case["op"] == "compact":
        cuts = sorted(many(0, int(case["n_pages"] * case["live"]), case["slots"] - 1))
        ends = [0] + cuts + [int(case["n_pages"] * case["live"])]
        return dict(n=case["slots"], pages=[b - a for a, b in zip(ends, ends[1:])], common=[rng.random() < 0.3 for _ in range(case["slots"])])
    sizes = many(case["size_lo"], case["size_hi"], case["groups"])
    n = sum(sizes)
    prefix = many(case["prefix_lo"], case["prefix_hi"], case["groups"])
    group = [g for g, k in enumerate(sizes) for _ in range(k)]
    tail = many(case["own_lo"], case["own_hi"], n)
    return dict(n=n, sizes=sizes, prefix=prefix, group=group, m=many(case["m_lo"], case["m_hi"], n), ctx=[prefix[g] + t for g, t in zip(group, tail)])


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    sh = _shape(case)
    page = case["page"]
    if case["op"] == "attend":
        token = case["kv_heads"] * 2 * (case["head_dim"] // 2 + case["head_dim"] // GROUP)  # bytes of a cached token
        rows = sum(sh["m"]) + sh["n"]
        own_part = sum(c + m + 1 - sh["prefix"][g] // page * page for c, m, g in zip(sh["ctx"], sh["m"], sh["group"]))
        seen = own_part + sum(p // page * page for p in sh["prefix"])
        pairs = sum((c + 1) * (m + 1) + m * (m + 1) // 2 for c, m in zip(sh["ctx"], sh["m"]))
        return {"bytes": seen * token + rows * 2 * case["q_heads"] * case["head_dim"] * 2, "flops": 4.0 * pairs * case["q_heads"] * case["head_dim"]}
    if case["op"] == "release":
        held, _, keep = _release_sizes(case, sh)
        gone = sum(h - min(h, _pages(k, page)) for h, k in zip(held, keep) if k >= 0)
        return {"bytes": 16 * gone + 8 * sh["n"], "flops": 2 * gone}  # an entry read and cleared, a count read and lowered
    token = case["kv_heads"] * 2 * (case["head_dim"] // 2 + case["head_dim"] // GROUP)
    if case["op"] == "compact":
        live = sum(sh["pages"])
        moved = live * (case["n_pages"] - live) / case["n_pages"]  # of shuffled pages
        return {"bytes": 2 * moved * page * token + 4 * case["n_pages"] + 8 * live, "flops": case["n_pages"] + live}
    forked = sum(k * _pages(c, page) for k, c in zip(sh["kids"], sh["ctx"]))
    copied = sum((k + 1) * (c % page) for k, c in zip(sh["kids"], sh["ctx"]) if k)
    return {"bytes": 2 * copied * token + 16 * forked + 12 * sh["n"], "flops": 2 * forked}


# ---- inputs -------------------------------------------------------------------------

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _offsets(counts):
    return _ints([0] + np.cumsum(counts).tolist())


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    s = dict(case=case, **_shape(case))
    {"branch": _prepare_branch, "release": _prepare_release, "compact": _prepare_compact, "attend": _prepare_attend}[case["op"]](s, case, gen)
    if own:  # the objects that a serving program makes once: the descriptions of pool and cache, scratch
        from speculative_decoding_verification_sdcp_gb300 import sdcp
        if case["op"] != "attend":
            s["pool"] = sdcp.KvPool(s["n_pages"], case["page"], page_table=s["page_table"], held=s["held"], refs=s["refs"])
            s["scratch"] = sdcp.alloc_pool_workspace(s["pool"])
        if "pages" in s:
            s["cache"] = sdcp.KvCache(s["n_pages"], case["page"], case["kv_heads"], case["head_dim"], DEVICE, pages=s["pages"])
        if case["op"] == "attend":
            s["scratch"] = sdcp.alloc_attend_shared_workspace(s["n"], s["total"], case["groups"], case["q_heads"], case["kv_heads"], case["head_dim"], DEVICE)
    return s


def _pool(s, table, held, n_pages):
    """The pool's state: page_table, held and refs as parts of one array, and a copy of it to set it back."""
    refs = np.zeros(n_pages, dtype=np.int32)
    inside = np.arange(table.shape[1])[None, :] < np.asarray(held)[:, None]
    np.add.at(refs, table[inside], 1)
    flat = np.concatenate([table.reshape(-1), np.asarray(held, dtype=np.int32), refs]).astype(np.int32)
    s["state"] = torch.from_numpy(flat).to(DEVICE)
    s["begin"] = s["state"].clone()
    n = table.size
    s["page_table"], s["held"], s["refs"] = s["state"][:n].view(table.shape), s["state"][n:n + len(held)], s["state"][n + len(held):]
    s["n_pages"] = n_pages


def _bytes_of_pages(s, case, gen):
    block = case["page"] * (case["head_dim"] // 2 + case["head_dim"] // GROUP)
    words = torch.randint(-2**31, 2**31, (s["n_pages"], case["kv_heads"], 2, block // 4), generator=gen, device=DEVICE, dtype=torch.int64)
    s["pages"] = words.to(torch.int32).view(torch.uint8)


def _copies(s, most):
    s["copies"] = torch.full((most, 4), -1, dtype=torch.int32, device=DEVICE)
    s["n_copies"] = torch.zeros(1, dtype=torch.int32, device=DEVICE)
    s["copied"] = torch.zeros(1, dtype=torch.int32, device=DEVICE)


def _prepare_branch(s, case, gen):
    page, parents, n = case["page"], case["parents"], s["n"] + 2  # two slots are idle
    ctx, kids = s["ctx"], s["kids"]
    held = [_pages(c, page) + x for c, x in zip(ctx, s["spare"])] + [0] * (n - parents)
    parent = [-1] * parents + [a for a, k in enumerate(kids) for _ in range(k)] + [-1, -1]
    length = [0] * parents + [c for c, k in zip(ctx, kids) for _ in range(k)] + [0, 0]
    kv_len = ctx + length[parents:]
    upto = [c + r for c, r in zip(kv_len, s["rows"])] + [0, 0]
    wide = max(max(_pages(u, page) for u in upto), max(held)) + 1
    used = sum(held)
    n_pages = used + sum(r // page + 2 for r in s["rows"])
    order = torch.randperm(n_pages, generator=gen, device=DEVICE).cpu().numpy()
    table, at = np.full((n, wide), -1, dtype=np.int32), 0
    for b in range(parents):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    _pool(s, table, held, n_pages)
    _bytes_of_pages(s, case, gen)
    _copies(s, n)
    s["parent"], s["length"], s["kv_len"], s["upto"] = _ints(parent), _ints(length), _ints(kv_len), _ints(upto)
    s["forked"], s["reserved"] = torch.empty(n, dtype=torch.int32, device=DEVICE), torch.empty(n, dtype=torch.int32, device=DEVICE)


def _release_sizes(case, sh):
    """Pages each slot holds, how many of them are its family's first slot's, and the tokens it keeps (-1: all)."""
    page, common = case["page"], case["common"] // case["page"]
    held = [common + _pages(c, page) for c in sh["own"]]
    shared = [0 if b % case["family"] == 0 else common for b in range(sh["n"])]
    keep = [0 if w < case["ended"] else -1 if w > 0.95 else max(0, h * page - x) for w, h, x in zip(sh["what"], held, sh["back"])]
    return held, shared, [-1] + keep[1:]  # the first session goes on


def _prepare_release(s, case, gen):
    held, shared, keep = _release_sizes(case, s)
    n_pages = sum(h - c for h, c in zip(held, shared)) + 5
    order = torch.randperm(n_pages, generator=gen, device=DEVICE).cpu().numpy()
    table, at = np.full((s["n"], max(held) + 1), -1, dtype=np.int32), 0
    for b in range(s["n"]):
        table[b, :shared[b]] = table[b - b % case["family"], :shared[b]]
        table[b, shared[b]:held[b]] = order[at:at + held[b] - shared[b]]
        at += held[b] - shared[b]
    _pool(s, table, held, n_pages)
    s["keep"] = _ints(keep)
    s["released"] = torch.empty(s["n"], dtype=torch.int32, device=DEVICE)


def _prepare_compact(s, case, gen):
    n_pages = case["n_pages"]
    order = torch.randperm(n_pages, generator=gen, device=DEVICE).cpu().numpy()
    extra = [s["pages"][b - 1] // 2 if b and c else 0 for b, c in enumerate(s["common"])]  # of the slot before
    held = [p + x for p, x in zip(s["pages"], extra)]
    table, at = np.full((s["n"], max(held) + 1), -1, dtype=np.int32), 0
    for b, (p, x) in enumerate(zip(s["pages"], extra)):
        table[b, :x] = table[b - 1, :x]
        table[b, x:x + p] = order[at:at + p]
        at += p
    _pool(s, table, held, n_pages)
    _bytes_of_pages(s, case, gen)
    _copies(s, n_pages // 2 + 1)
    s["n_live"] = torch.zeros(1, dtype=torch.int32, device=DEVICE)


def _prepare_attend(s, case, gen):
    page, dim, n = case["page"], case["head_dim"], s["n"]
    common = [p // page for p in s["prefix"]]
    need = [_pages(c + m + 1, page) for c, m in zip(s["ctx"], s["m"])]
    s["n_pages"] = sum(common) + sum(k - common[g] for k, g in zip(need, s["group"]))
    order = torch.randperm(s["n_pages"], generator=gen, device=DEVICE).cpu().numpy()
    first = np.concatenate([[0], np.cumsum(common)])
    table, at = np.full((n, max(need)), -1, dtype=np.int32), int(first[-1])
    for b, g in enumerate(s["group"]):
        table[b, :common[g]] = order[first[g]:first[g + 1]]
        table[b, common[g]:need[b]] = order[at:at + need[b] - common[g]]
        at += need[b] - common[g]
    s["page_table"] = torch.from_numpy(table).to(DEVICE)
    # keys with a few large channels, plain values
    shape = (s["n_pages"], case["kv_heads"], page, dim)
    s["pages"] = torch.empty((s["n_pages"], case["kv_heads"], 2, page * (dim // 2 + dim // GROUP)), dtype=torch.uint8, device=DEVICE)
    for which in (0, 1):
        x = torch.randn(shape, generator=gen, device=DEVICE)
        if which == 0:
            x[..., ::16] *= 3
        s["pages"][:, :, which] = _block(*_quantise(x))
    s["total"], s["m_offsets"], s["kv_len"], s["group_offsets"] = sum(s["m"]), _offsets(s["m"]), _ints(s["ctx"]), _offsets(s["sizes"])
    # scores with a spread of about two: a few tokens carry most of the weight
    s["q"] = torch.randn((s["total"] + n, case["q_heads"], dim), generator=gen, device=DEVICE).mul_(1.5).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["status"] = torch.empty(n, dtype=torch.int32, device=DEVICE)
    s["scale"] = dim ** -0.5


# ---- one pass -----------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op != "attend":
        s["state"].copy_(s["begin"])
    if own:
        return {"branch": _own_branch, "release": _own_release, "compact": _own_compact, "attend": _own_attend}[op](s)
    return {"branch": _plain_branch, "release": _plain_release, "compact": _plain_compact, "attend": _plain_attend}[op](s)


def _own_branch(s):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    sdcp.sdcp_fork_kv(s["pool"], s["parent"], s["length"], s["forked"])
    sdcp.sdcp_reserve_kv(s["pool"], s["kv_len"], s["upto"], s["copies"], s["n_copies"], s["reserved"], s["scratch"])
    sdcp.sdcp_copy_pages(s["cache"], s["copies"], s["n_copies"], s["copied"])
    return s["state"], s["copies"], s["n_copies"], s["pages"], s["forked"], s["reserved"], s["copied"]


def _own_release(s):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    sdcp.sdcp_release_kv(s["pool"], s["keep"], s["released"])
    return s["state"], s["released"]


def _own_compact(s):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    sdcp.sdcp_compact_kv(s["pool"], s["copies"], s["n_copies"], s["n_live"], s["scratch"])
    sdcp.sdcp_copy_pages(s["cache"], s["copies"], s["n_copies"], s["copied"])
    return s["state"], s["copies"], s["n_copies"], s["n_live"], s["pages"], s["copied"]


def _own_attend(s):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    sdcp.sdcp_attend_shared_kv(s["cache"], s["page_table"], s["m_offsets"], s["total"], s["kv_len"], s["group_offsets"], s["q"], s["out"], s["status"],
                               s["scratch"], scale=s["scale"])
    return s["out"], s["status"]


# ---- plain forms --------------------------------------------------------------------

def _plain_fork(s):
    page, table = s["case"]["page"], s["page_table"]
    child = s["parent"] >= 0
    n = torch.where(child, (s["length"] + page - 1) // page, 0)
    takes = torch.arange(table.shape[1], device=DEVICE)[None, :] < n[:, None]
    rows = table[s["parent"].clamp(min=0).long()]
    table.copy_(torch.where(takes, rows, table))
    s["refs"].index_add_(0, rows.clamp(min=0).long().flatten(), takes.int().flatten())
    s["held"].copy_(torch.where(child, n, s["held"]))
    s["forked"].zero_()


def _plain_reserve(s):
    page, table, refs, held = s["case"]["page"], s["page_table"], s["refs"], s["held"]
    kv_len, upto = s["kv_len"], s["upto"]
    at = torch.arange(table.shape[1], device=DEVICE)[None, :]
    active = upto > kv_len
    first, need = kv_len // page, (upto + page - 1) // page
    here = active[:, None] & (at >= first[:, None]) & (at < need[:, None])
    old = table.clamp(min=0).long()
    shared = here & (at < held[:, None]) & (refs[old] > 1)
    want = shared | (here & (at >= held[:, None]))
    count = want.sum(dim=1)
    free = refs == 0
    fits = (count == 0) | (count.cumsum(0) <= free.sum())
    want &= fits[:, None]
    shared &= fits[:, None]
    # the free pages in order, then one for each entry wanted, in the order of slots and entries
    none = refs.shape[0]
    ranks = torch.where(free, free.cumsum(0) - 1, none)
    in_order = torch.zeros(none + 1, dtype=torch.int32, device=DEVICE).scatter_(0, ranks, torch.arange(none, dtype=torch.int32, device=DEVICE))
    rank = (want.flatten().cumsum(0) - 1).clamp(min=0).view(want.shape)
    new = in_order[rank.clamp(max=none)]
    copy = (shared & (at == first[:, None])).any(dim=1) & (kv_len % page > 0)
    entry = first.clamp(max=table.shape[1] - 1).long()[:, None]
    record = torch.cat([table.gather(1, entry), new.gather(1, entry), (kv_len % page)[:, None], torch.zeros_like(entry, dtype=torch.int32)], dim=1)
    place = torch.where(copy, copy.cumsum(0) - 1, table.shape[0])
    padded = torch.cat([s["copies"], s["copies"][:1]])
    s["copies"].copy_(padded.index_copy(0, place, torch.where(copy[:, None], record, padded[-1:]))[:-1])
    s["n_copies"].copy_(copy.sum()[None])
    refs.index_add_(0, old.flatten(), -shared.int().flatten())
    refs.index_add_(0, torch.where(want, new, 0).long().flatten(), want.int().flatten())
    table.copy_(torch.where(want, new, table))
    held.copy_(torch.where(active & fits, torch.maximum(held, need), held))
    s["reserved"].copy_(torch.where(fits, 0, 2))


def _plain_copy_pages(s):
    case, pages = s["case"], s["pages"]
    page, dim = case["page"], case["head_dim"]
    c = s["copies"][:int(s["n_copies"])].long()
    byte = torch.arange(pages.shape[-1], device=DEVICE)
    token = torch.where(byte < page * dim // 2, byte // 16 % page, (byte - page * dim // 2) // (dim // GROUP))
    pages[c[:, 1]] = torch.where(token[None, None, None, :] < c[:, 2, None, None, None], pages[c[:, 0]], pages[c[:, 1]])
    s["copied"].zero_()


def _plain_branch(s):
    _plain_fork(s)
    _plain_reserve(s)
    _plain_copy_pages(s)
    return s["state"], s["copies"], s["n_copies"], s["pages"], s["forked"], s["reserved"], s["copied"]


def _plain_release(s):
    table, held, keep = s["page_table"], s["held"], s["keep"]
    left = torch.where(keep >= 0, torch.minimum((keep + s["case"]["page"] - 1) // s["case"]["page"], held), held)
    at = torch.arange(table.shape[1], device=DEVICE)[None, :]
    gone = (at >= left[:, None]) & (at < held[:, None])
    s["refs"].index_add_(0, table.clamp(min=0).long().flatten(), -gone.int().flatten())
    table.copy_(torch.where(gone, -1, table))
    held.copy_(left)
    s["released"].zero_()
    return s["state"], s["released"]


def _plain_compact(s):
    table, refs = s["page_table"], s["refs"]
    n = refs.shape[0]
    at = torch.arange(n, device=DEVICE)
    live = refs > 0
    n_live = live.sum()
    high, hole = live & (at >= n_live), ~live & (at < n_live)
    from_top = torch.where(high, high.flip(0).cumsum(0).flip(0) - 1, n)
    from_bottom = torch.where(hole, hole.cumsum(0) - 1, n)
    most = s["copies"].shape[0]
    src = torch.full((n + 1,), -1, device=DEVICE).scatter_(0, from_top, at)[:most]
    dst = torch.full((n + 1,), -1, device=DEVICE).scatter_(0, from_bottom, at)[:most]
    moves = torch.arange(most, device=DEVICE) < high.sum()
    record = torch.stack([src, dst, torch.full_like(src, s["case"]["page"]), torch.zeros_like(src)], dim=1).int()
    s["copies"].copy_(torch.where(moves[:, None], record, s["copies"]))
    s["n_copies"].copy_(moves.sum()[None])
    to = torch.arange(n + 1, device=DEVICE).scatter_(0, torch.where(moves, src, n), dst)[:n]
    inside = torch.arange(table.shape[1], device=DEVICE)[None, :] < s["held"][:, None]
    table.copy_(torch.where(inside, to[table.clamp(min=0).long()].int(), table))
    refs.copy_(torch.zeros_like(refs).index_add_(0, to, refs))
    s["n_live"].copy_(n_live[None])
    _plain_copy_pages(s)
    return s["state"], s["copies"], s["n_copies"], s["n_live"], s["pages"], s["copied"]


def _quantise(x):
    """Codes -7..7 (float) and scale bytes of float32 groups of 32 channels."""
    g = x.unflatten(-1, (-1, GROUP))
    most = g.abs().amax(dim=-1)
    t = most / torch.full_like(most, 7)
    byte = (((t.view(torch.int32) + 0xFFFFF) >> 20) - (112 << 3)).clamp_(8, 167)
    scale = ((byte + (112 << 3)) << 20).view(torch.float32)
    return (g / scale[..., None]).round().clamp(-7, 7), byte


def _block(code, byte):
    """Codes [..., P, D/32, 32] and scale bytes [..., P, D/32] as the bytes of blocks."""
    n = (code + 8).to(torch.uint8).unflatten(-1, (4, 4, 2))       # word, pair, which of the pair
    n = n.transpose(-1, -2).flatten(-2)                            # nibbles of a word, low ones first
    packed = (n[..., 0::2] | (n[..., 1::2] << 4)).flatten(-2)      # 16 bytes of a group
    packed = packed.transpose(-2, -3)                              # [..., D/32, P, 16]
    return torch.cat([packed.flatten(-3), byte.to(torch.uint8).flatten(-2)], dim=-1)


def _values(pages, page, dim):
    """What blocks of bytes [..., bytes] stand for: float32 [..., P, D]."""
    groups = dim // GROUP
    packed = pages[..., :page * dim // 2].unflatten(-1, (groups, page, 4, 4))
    n = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2)  # [..., groups, P, word, nibble]
    n = n.unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-3)        # channels of a group
    byte = pages[..., page * dim // 2:].unflatten(-1, (page, groups)).int()
    scale = ((byte + (112 << 3)) << 20).view(torch.float32)
    return ((n.transpose(-2, -3).float() - 8) * scale[..., None]).flatten(-2)


def _plain_attend(s):
    case, n = s["case"], s["n"]
    heads, share, dim = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["head_dim"]
    first = s["m_offsets"].long() + torch.arange(n + 1, device=DEVICE)
    row = torch.arange(s["q"].shape[0], device=DEVICE)
    session = torch.searchsorted(first, row, right=True) - 1
    i = row - first[session]
    wide = max(s["m"]) + 1
    q = torch.zeros((n, wide, case["q_heads"], dim), device=DEVICE)
    q[session, i] = s["q"].float()
    q = q.unflatten(2, (heads, share)).permute(0, 2, 1, 3, 4).flatten(2, 3)            # [n, heads, rows x share, D]
    values = _values(s["pages"], case["page"], dim)                                     # [pages, heads, 2, P, D]
    kv = values[s["page_table"].long().clamp(min=0)].permute(0, 2, 3, 1, 4, 5).flatten(3, 4)  # [n, heads, 2, tokens, D]
    del values
    score = torch.matmul(q, kv[:, :, 0].transpose(-1, -2)) * s["scale"]
    at = torch.arange(kv.shape[3], device=DEVICE)[None, None, :]
    last = (s["kv_len"].long()[:, None] + torch.arange(wide, device=DEVICE)[None, :])[:, :, None]
    score = torch.where((at <= last).repeat_interleave(share, dim=1)[:, None], score, -math.inf)
    p = torch.exp(score - score.amax(dim=-1, keepdim=True))
    del score
    o = torch.matmul(p, kv[:, :, 1]) / p.sum(dim=-1, keepdim=True)
    o = o.unflatten(2, (wide, share)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o[session, i].to(torch.bfloat16), torch.zeros(n, dtype=torch.int32, device=DEVICE)


# ---- the definition in 64 bits --------------------------------------------------------

def exact(case, seed):
    """The attention's output; the passes over pages give whole numbers alone."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    size, dim, heads = case["page"], case["head_dim"], case["kv_heads"]
    share = case["q_heads"] // heads
    t, d = torch.arange(size, device=DEVICE)[:, None], torch.arange(dim, device=DEVICE)[None, :]
    g, word, e = d // 32, (d % 32) // 8, d % 8
    bit = 4 * (e // 2 + 4 * (e % 2))
    code, shift, scale = (g * size + t) * 16 + word * 4 + bit // 8, bit % 8, size * dim // 2 + t * (dim // 32) + g
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
    row = 0
    for b, (c, m) in enumerate(zip(s["ctx"], s["m"])):
        raw = s["pages"][s["page_table"][b, :_pages(c + m + 1, size)].long()]
        n, byte = (raw[..., code] >> shift) & 15, raw[..., scale].short()
        v = (n.short() - 8).double() * (1 + (byte % 8).double() / 8) * torch.exp2((byte // 8 - 15).double())
        k, v = v.permute(2, 0, 3, 1, 4).flatten(1, 2)[:, :c + m + 1]
        q = s["q"][row:row + m + 1].double().reshape(m + 1, heads, share, dim)
        score = torch.einsum("ihgd,thd->hgit", q, k) * s["scale"]
        score.masked_fill_(torch.arange(c + m + 1, device=DEVICE)[None, :] > c + torch.arange(m + 1, device=DEVICE)[:, None], -math.inf)
        out[row:row + m + 1] = torch.einsum("hgit,thd->ihgd", torch.softmax(score, dim=-1), v).reshape(m + 1, case["q_heads"], dim)
        row += m + 1
    return out, None
