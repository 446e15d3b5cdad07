"""The serving operators around a verify batch: what is timed, their plain forms and their
64-bit definitions.

Four operators, on the ragged layout of a verify batch (B sessions, session b with m_b drafts
and m_b + 1 scored rows):

* ``adjust``: penalties for repeated tokens, biases and grammar masks on the target or draft rows;
* ``append``: the round's keys and values into a paged cache of 4-bit codes, with the position
  rotation of queries and keys on the way (the rows just written are read back as values);
* ``read``: stretches of cached tokens as values;
* ``attend``: attention of the round's rows over the paged 4-bit cache.

Cache layout: page p, head h holds a key block and a value block (pages[p, h, 0 / 1]).  A block of P
tokens of D channels is [D/32][P][16] bytes of codes, then [P][D/32] scale bytes.  The 16 bytes of a
group of 32 channels are four little-endian words of 8 channels each; channel e of a word is in bits
4 (e / 2 + 4 (e mod 2)) upwards, as n + 8 with n in -7..7.  A scale byte 8 e + m (8..167) stands for
(1 + m / 8) 2^(e - 15); the value is n times the scale.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
GROUP = 32


# ---- cases --------------------------------------------------------------------------

def listed():
    return [
        # a test-sized verify batch: only the latency of the call counts
        dict(name="adjust_tiny", op="adjust", rows="target", sessions=4, m_lo=4, m_hi=4, vocab=1000, dtype="f32",
             history=40, biases=3, masked=0.5),
        # draft rows of a ragged batch, an odd vocabulary (rows start at any element), long prompts
        dict(name="adjust_draft_odd", op="adjust", rows="draft", sessions=96, m_lo=1, m_hi=16, vocab=50257, dtype="bf16",
             history=16384, biases=0, masked=1.0),
        # the target rows of the largest batch: bandwidth
        dict(name="adjust_large", op="adjust", rows="target", sessions=1024, m_lo=4, m_hi=4, vocab=152064, dtype="bf16",
             history=1024, biases=16, masked=0.25),
        # plain decoding: one token a session
        dict(name="append_single", op="append", sessions=16, m_lo=0, m_hi=0, q_heads=32, kv_heads=8, head_dim=128, page=16,
             dtype="bf16", ctx=4000, rot=128, layout="half"),
        # a round of ragged proposals, part of the head rotated in pairs of neighbours
        dict(name="append_ragged", op="append", sessions=256, m_lo=1, m_hi=16, q_heads=64, kv_heads=8, head_dim=128, page=64,
             dtype="bf16", ctx=8000, rot=64, layout="interleaved"),
        # prompts of two sessions in one call, 32-bit activations, small heads
        dict(name="append_prompt", op="append", sessions=2, m_lo=7001, m_hi=9001, q_heads=28, kv_heads=4, head_dim=64, page=32,
             dtype="f32", ctx=0, rot=64, layout="half"),
        # the last tokens of a few sessions
        dict(name="read_tail", op="read", sessions=7, ctx_lo=1, ctx_hi=129, kv_heads=4, head_dim=64, page=16),
        # whole sessions that move to another machine
        dict(name="read_export", op="read", sessions=12, ctx_lo=8000, ctx_hi=24000, kv_heads=8, head_dim=128, page=64),
        # one session decoding alone: latency
        dict(name="attend_single", op="attend", sessions=1, m_lo=0, m_hi=0, q_heads=32, kv_heads=8, head_dim=128, page=16,
             ctx_lo=2001, ctx_hi=2001, window=0),
        # a full verify batch: 9 rows a session, 8 query heads on a cached head
        dict(name="attend_verify", op="attend", sessions=64, m_lo=8, m_hi=8, q_heads=64, kv_heads=8, head_dim=128, page=64,
             ctx_lo=500, ctx_hi=8200, window=0),
        # a few long contexts
        dict(name="attend_long", op="attend", sessions=4, m_lo=4, m_hi=4, q_heads=32, kv_heads=8, head_dim=128, page=64,
             ctx_lo=90001, ctx_hi=120001, window=0),
        # ragged proposals over a sliding window, small heads
        dict(name="attend_window", op="attend", sessions=192, m_lo=1, m_hi=16, q_heads=28, kv_heads=4, head_dim=64, page=32,
             ctx_lo=10, ctx_hi=6000, window=1000),
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
    op = rng.choice(["adjust", "adjust", "append", "append", "read", "attend", "attend", "attend"])
    sessions = _log(rng, 1, 512)
    m_hi = rng.choice([0, _log(rng, 1, 64), _log(rng, 1, 16)])
    m_lo = rng.randint(0, m_hi)
    if op == "adjust":
        case = dict(op=op, rows=rng.choice(["target", "draft"]), sessions=sessions, m_lo=m_lo, m_hi=m_hi, vocab=_log(rng, 500, 262144),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), history=_log(rng, 1, 32768), biases=rng.choice([0, _log(rng, 1, 300)]),
                    masked=rng.choice([0.0, 0.3, 1.0]))
        if case["rows"] == "draft" and m_lo == 0:
            case["m_lo"], case["m_hi"] = 1, max(1, m_hi)
        small = sessions * (case["m_hi"] + 1) * case["vocab"] <= 6e8
        return case if small and 3072 not in (case["vocab"], case["history"]) else None
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    share = rng.choice([1, 2, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    q_heads = kv_heads * share
    if op == "append":
        if rng.random() < 0.25:  # prompts
            sessions, m_hi = rng.randint(1, 4), _log(rng, 100, 9000)
            m_lo = m_hi // 2
        rot = rng.choice([dim, dim // 2, 16, 0])
        case = dict(op=op, sessions=sessions, m_lo=m_lo, m_hi=m_hi, q_heads=q_heads, kv_heads=kv_heads, head_dim=dim, page=page,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), ctx=_log(rng, 1, 16000), rot=rot, layout=rng.choice(["half", "interleaved"]))
        cost = sessions * (m_hi + 1) * (q_heads + 2 * kv_heads) * dim
        return case if cost <= 4e7 and (q_heads + 2 * kv_heads) * dim != 3072 and sessions * case["ctx"] <= 1e6 else None
    hi = _log(rng, 1, 120000)
    lo = rng.randint(0, hi)
    cost = sessions * hi * kv_heads * dim
    if op == "read":
        return dict(op=op, sessions=sessions, ctx_lo=lo, ctx_hi=hi, kv_heads=kv_heads, head_dim=dim, page=page) if cost <= 2.5e8 else None
    case = dict(op=op, sessions=sessions, m_lo=m_lo, m_hi=m_hi, q_heads=q_heads, kv_heads=kv_heads, head_dim=dim, page=page,
                ctx_lo=lo, ctx_hi=hi, window=rng.choice([0, 0, _log(rng, 1, 8000)]))
    small = cost <= 4e8 and cost * (m_hi + 1) * share <= 1.5e10 and sessions * hi * (m_hi + 1) * q_heads <= 2e9
    return case if small and q_heads * dim != 3072 else None


def _shape(case):
    """The ragged sizes of a case: drafts and cached tokens of each session, fixed by the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["sessions"]
    m = [rng.randint(case.get("m_lo", 0), case.get("m_hi", 0)) for _ in range(n)]
    if "ctx_lo" in case:
        ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    else:
        ctx = [rng.randint(0, case.get("ctx", 0)) for _ in range(n)]
    hist = [rng.randint(0, case.get("history", 0)) for _ in range(n)]
    return m, ctx, hist


def work(case):
    m, ctx, hist = _shape(case)
    if case["op"] == "adjust":
        rows = sum(m) + (case["sessions"] if case["rows"] == "target" else 0)
        e = SIZE[case["dtype"]]
        nbytes = rows * case["vocab"] * 2 * e + int(rows * case["masked"]) * case["vocab"] / 8 + 4 * sum(hist) + 8 * case["biases"] * case["sessions"]
        return {"bytes": nbytes, "flops": rows * case["vocab"]}
    token = case["kv_heads"] * 2 * (case["head_dim"] // 2 + case["head_dim"] // GROUP)  # bytes of a cached token
    value = case["kv_heads"] * 2 * case["head_dim"] * 2                                # and of its values read back
    if case["op"] == "append":
        rows = sum(m) + case["sessions"]
        e = SIZE[case["dtype"]]
        acts = (2 * case["q_heads"] + 2 * case["kv_heads"]) * case["head_dim"] * e
        return {"bytes": rows * (acts + 4 * case["rot"] + 2 * token + value), "flops": rows * (case["q_heads"] + 4 * case["kv_heads"]) * case["head_dim"] * 3}
    if case["op"] == "read":
        return {"bytes": sum(ctx) * (token + value), "flops": sum(ctx) * value / 2}
    seen = pairs = rows = 0
    for mb, c in zip(m, ctx):
        w = case["window"] or c + mb + 1
        seen += c + mb + 1 - max(0, c + 1 - w)
        pairs += sum(min(w, c + i + 1) for i in range(mb + 1))
        rows += mb + 1
    return {"bytes": seen * token + rows * 2 * case["q_heads"] * case["head_dim"] * 2, "flops": 4.0 * pairs * case["q_heads"] * case["head_dim"]}


# ---- inputs -------------------------------------------------------------------------

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _offsets(counts):
    total, out = 0, [0]
    for c in counts:
        total += c
        out.append(total)
    return _ints(out)


def _paged(case, tokens, gen):
    """A page table for sessions of `tokens` tokens, in a shuffled order, -1 where a session has no page."""
    need = [-(-t // case["page"]) for t in tokens]
    total = max(1, sum(need))
    order = torch.randperm(total, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32, device=DEVICE)
    at = torch.arange(table.shape[1], device=DEVICE)[None, :] < _ints(need)[:, None]
    table[at] = order[:int(sum(need))]
    return table, total


def _tokens_like_text(shape, vocab, gen):
    return (torch.rand(shape, generator=gen, device=DEVICE).pow(3) * vocab).to(torch.int32).clamp_(max=vocab - 1)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    m, ctx, hist = _shape(case)
    s = dict(case=case, m=m, ctx=ctx, m_offsets=_offsets(m), total=sum(m), status=torch.empty(len(m), dtype=torch.int32, device=DEVICE))
    {"adjust": _prepare_adjust, "append": _prepare_append, "read": _prepare_read, "attend": _prepare_attend}[case["op"]](s, case, m, ctx, hist, gen)
    if own:  # the objects that a serving program makes once: the cache's description, the call's scratch
        from speculative_decoding_verification_sdcp_gb300 import sdcp
        if "pages" in s:
            s["cache"] = sdcp.KvCache(s["n_pages"], case["page"], case["kv_heads"], case["head_dim"], DEVICE, pages=s["pages"])
        if case["op"] == "append" and case["rot"]:
            s["rotary"] = sdcp.Rotary(s["table"], sdcp.ROTARY_HALF if case["layout"] == "half" else sdcp.ROTARY_INTERLEAVED)
        if case["op"] == "attend":
            s["scratch"] = sdcp.alloc_attend_workspace(len(m), s["total"], case["q_heads"], case["kv_heads"], case["head_dim"], DEVICE)
    return s


def _prepare_adjust(s, case, m, ctx, hist, gen):
    n, vocab = len(m), case["vocab"]
    s["rows"] = sum(m) + (n if case["rows"] == "target" else 0)
    s["logits"] = torch.randn((s["rows"], vocab), generator=gen, device=DEVICE, dtype=TYPES[case["dtype"]]).mul_(3)
    s["out"] = torch.empty_like(s["logits"])
    s["draft_tokens"] = _tokens_like_text((sum(m),), vocab, gen)
    s["history"] = _tokens_like_text((n, max(1, case["history"])), vocab, gen)
    rng = random.Random(int(gen.initial_seed()))
    s["prompt"] = [rng.randint(0, h) for h in hist]
    s["hist"] = hist
    s["penalties"] = [(rng.choice([1.0, 1.1, 1.3]), rng.choice([0.0, 0.2, 0.7]), rng.choice([0.0, 0.5, -0.25])) for _ in m]
    import numpy as np
    rec = np.zeros(n, dtype=[("repetition", "<f4"), ("frequency", "<f4"), ("presence", "<f4"), ("history_len", "<u4"), ("prompt_len", "<u4"),
                             ("bias_offset", "<u4"), ("bias_count", "<u4"), ("reserved", "<u4")])
    rec["repetition"], rec["frequency"], rec["presence"] = zip(*s["penalties"])
    rec["history_len"], rec["prompt_len"] = hist, s["prompt"]
    k = min(case["biases"], vocab)
    rec["bias_count"], rec["bias_offset"] = k, np.arange(n, dtype=np.uint32) * k
    s["controls"] = torch.from_numpy(rec.view(np.uint8).copy()).to(DEVICE)
    s["bias_tokens"] = s["bias_values"] = s["masks"] = s["mask_rows"] = None
    if k:  # ids rising within a session
        s["bias_tokens"] = torch.rand((n, vocab), generator=gen, device=DEVICE).topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32).reshape(-1)
        s["bias_values"] = torch.randn((n * k,), generator=gen, device=DEVICE).mul_(5)
    masked = int(s["rows"] * case["masked"])
    if masked:  # a mask for each of them, some that leave most tokens and some that leave few
        words = (vocab + 31) // 32
        bits = torch.randint(-2**31, 2**31, (6, masked, words), generator=gen, device=DEVICE, dtype=torch.int64).to(torch.int32)
        few = bits[0] & bits[1] & bits[2] & bits[3] & bits[4] & bits[5]
        most = bits[0] | bits[1] | bits[2] | bits[3]
        s["masks"] = torch.where((torch.arange(masked, device=DEVICE) % 2 == 0)[:, None], few, most).contiguous()
        s["mask_rows"] = torch.full((s["rows"],), -1, dtype=torch.int32, device=DEVICE)
        s["mask_rows"][torch.randperm(s["rows"], generator=gen, device=DEVICE)[:masked]] = torch.arange(masked, dtype=torch.int32, device=DEVICE)


def _prepare_append(s, case, m, ctx, hist, gen):
    n, rows, d = len(m), sum(m) + len(m), case["head_dim"]
    s["page_table"], s["n_pages"] = _paged(case, [c + k + 1 for c, k in zip(ctx, m)], gen)
    s["pages"] = torch.zeros((s["n_pages"], case["kv_heads"], 2, case["page"] * (d // 2 + d // GROUP)), dtype=torch.uint8, device=DEVICE)
    s["kv_len"] = _ints(ctx)
    heads = case["q_heads"] + 2 * case["kv_heads"]
    fused = torch.randn((rows, heads, d), generator=gen, device=DEVICE)  # the projection's output: q, k and v of a row side by side
    fused[:, case["q_heads"]:case["q_heads"] + case["kv_heads"], ::16] *= 6  # keys have a few large channels
    fused = fused.to(TYPES[case["dtype"]])
    s["q"], s["k"], s["v"] = fused.split([case["q_heads"], case["kv_heads"], case["kv_heads"]], dim=1)
    s["q_out"] = torch.empty((rows, case["q_heads"], d), dtype=TYPES[case["dtype"]], device=DEVICE)
    s["k_out"] = torch.empty((rows, case["kv_heads"], d), dtype=torch.bfloat16, device=DEVICE)
    s["v_out"] = torch.empty_like(s["k_out"])
    s["row_offsets"] = _offsets([k + 1 for k in m])
    if case["rot"]:
        at = torch.arange(max(c + k + 1 for c, k in zip(ctx, m)), device=DEVICE, dtype=torch.float64)
        angle = at[:, None] * (10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEVICE, dtype=torch.float64) / case["rot"]))[None, :]
        s["table"] = torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32)


def _filled(s, case, tokens, gen):
    """Pages that hold `tokens` tokens a session, of keys with a few large channels and plain values."""
    d = case["head_dim"]
    s["page_table"], s["n_pages"] = _paged(case, tokens, gen)
    shape = (s["n_pages"], case["kv_heads"], case["page"], d)
    s["pages"] = torch.empty((s["n_pages"], case["kv_heads"], 2, case["page"] * (d // 2 + d // GROUP)), dtype=torch.uint8, device=DEVICE)
    for which in (0, 1):
        x = torch.randn(shape, generator=gen, device=DEVICE)
        if which == 0:
            x[..., ::16] *= 3
        code, byte, _ = _quantise(x)
        s["pages"][:, :, which] = _block(code, byte)


def _prepare_read(s, case, m, ctx, hist, gen):
    rng = random.Random(int(gen.initial_seed()))
    start = [rng.randint(0, 40) for _ in ctx]  # the stretch begins anywhere
    _filled(s, case, [a + c for a, c in zip(start, ctx)], gen)
    s["start"], s["row_offsets"], s["tokens"], s["starts"] = _ints(start), _offsets(ctx), sum(ctx), start
    s["k_out"] = torch.empty((sum(ctx), case["kv_heads"], case["head_dim"]), dtype=torch.bfloat16, device=DEVICE)
    s["v_out"] = torch.empty_like(s["k_out"])


def _prepare_attend(s, case, m, ctx, hist, gen):
    _filled(s, case, [c + k + 1 for c, k in zip(ctx, m)], gen)
    s["kv_len"] = _ints(ctx)
    # scores with a spread of about two: a few tokens carry most of the weight
    s["q"] = torch.randn((sum(m) + len(m), case["q_heads"], case["head_dim"]), generator=gen, device=DEVICE).mul_(1.5).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = case["head_dim"] ** -0.5


# ---- one pass -----------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"adjust": _own_adjust, "append": _own_append, "read": _own_read, "attend": _own_attend}[op](s)
    return {"adjust": _plain_adjust, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[op](s)


def _own_adjust(s):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    sdcp.sdcp_adjust_logits(s["logits"], s["out"], s["m_offsets"], s["total"], s["draft_tokens"], s["controls"], s["history"], s["status"],
                            rows=sdcp.ROWS_TARGET if s["case"]["rows"] == "target" else sdcp.ROWS_DRAFT, bias_tokens=s["bias_tokens"],
                            bias_values=s["bias_values"], masks=s["masks"], mask_rows=s["mask_rows"])
    return s["out"], s["status"]


def _own_append(s):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    rows = s["q"].shape[0]
    sdcp.sdcp_append_kv(s["cache"], s["page_table"], s["m_offsets"], s["total"], s["kv_len"], s["k"], s["v"], s["status"],
                        rotary=s.get("rotary"), q=s["q"], q_out=s["q_out"])
    sdcp.sdcp_read_kv(s["cache"], s["page_table"], s["row_offsets"], rows, s["kv_len"], s["k_out"], s["v_out"], s["status"])
    return s["q_out"], s["k_out"], s["v_out"], s["status"]


def _own_read(s):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    sdcp.sdcp_read_kv(s["cache"], s["page_table"], s["row_offsets"], s["tokens"], s["start"], s["k_out"], s["v_out"], s["status"])
    return s["k_out"], s["v_out"], s["status"]


def _own_attend(s):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    sdcp.sdcp_attend_kv(s["cache"], s["page_table"], s["m_offsets"], s["total"], s["kv_len"], s["q"], s["out"], s["status"], s["scratch"],
                        scale=s["scale"], window=s["case"]["window"])
    return s["out"], s["status"]


# ---- plain forms --------------------------------------------------------------------

def _plain_adjust(s):
    case, n, vocab, rows = s["case"], len(s["m"]), s["case"]["vocab"], s["rows"]
    first = s["m_offsets"].long() + (torch.arange(n + 1, device=DEVICE) if case["rows"] == "target" else 0)
    row = torch.arange(rows, device=DEVICE)
    session = torch.searchsorted(first, row, right=True) - 1
    i = row - first[session]
    rec = s["controls"].view(n, 32)
    real, whole = rec[:, :12].contiguous().view(torch.float32), rec[:, 12:].contiguous().view(torch.int32).long()
    at = torch.arange(s["history"].shape[1], device=DEVICE)[None, :]
    in_prompt, in_output = at < whole[:, 1:2], (at >= whole[:, 1:2]) & (at < whole[:, :1])
    ids = s["history"].long()
    prompt = torch.zeros((n, vocab), device=DEVICE).scatter_add_(1, ids, in_prompt.float())
    count = torch.zeros((n, vocab), device=DEVICE).scatter_add_(1, ids, in_output.float())
    del in_prompt, in_output, ids
    c = count[session]
    if s["total"]:  # the drafts before a row's own position
        j = torch.arange(max(s["m"]), device=DEVICE)[None, :]
        where = (s["m_offsets"].long()[session][:, None] + j).clamp_(max=s["total"] - 1)
        c.scatter_add_(1, s["draft_tokens"].long()[where], (j < i[:, None]).float())
    z = s["logits"].float()
    r = real[session, 0:1]
    z = torch.where((prompt[session] > 0) | (c > 0), torch.where(z > 0, z / r, z * r), z)
    z = z - real[session, 1:2] * c
    z = z - real[session, 2:3] * (c > 0)
    del c
    if s["bias_tokens"] is not None:
        bias = torch.zeros((n, vocab), device=DEVICE).scatter_(1, s["bias_tokens"].long().view(n, -1), s["bias_values"].view(n, -1))
        z = z + bias[session]
    if s["masks"] is not None:
        bit = torch.arange(32, device=DEVICE, dtype=torch.int32)
        left = (((s["masks"][:, :, None] >> bit) & 1) > 0).flatten(1)[:, :vocab]
        which = s["mask_rows"].long()
        z = torch.where(left[which.clamp(min=0)] | (which < 0)[:, None], z, -math.inf)
    return z.to(s["logits"].dtype), torch.zeros(n, dtype=torch.int32, device=DEVICE)


def _quantise(x):
    """Codes -7..7 (float), scale bytes and scales of float32 groups of 32 channels."""
    g = x.unflatten(-1, (-1, GROUP))
    most = g.abs().amax(dim=-1)
    t = most / torch.full_like(most, 7)
    byte = (((t.view(torch.int32) + 0xFFFFF) >> 20) - (112 << 3)).clamp_(8, 167)
    scale = ((byte + (112 << 3)) << 20).view(torch.float32)
    code = (g / scale[..., None]).round().clamp(-7, 7)
    return code, byte, scale


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


def _rotate(x, table, at, layout):
    """float32 rows x [rows, heads, D] turned by their positions `at`."""
    rot = table.shape[1]
    cos, sin = table[at][:, None, :rot // 2], table[at][:, None, rot // 2:]
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _positions(offsets, start, rows):
    """Session and position of each row of a ragged list."""
    row = torch.arange(rows, device=DEVICE)
    session = torch.searchsorted(offsets.long(), row, right=True) - 1
    return session, start.long()[session] + row - offsets.long()[session]


def _read(s, session, at):
    case = s["case"]
    page, dim = case["page"], case["head_dim"]
    where, slot = s["page_table"].long()[session, at // page], at % page
    groups = dim // GROUP
    codes = s["pages"][..., :page * dim // 2].unflatten(-1, (groups, page, 16))
    bytes_ = s["pages"][..., page * dim // 2:].unflatten(-1, (page, groups))
    one = torch.cat([codes[where, :, :, :, slot].flatten(-2), bytes_[where, :, :, slot]], dim=-1)  # [rows, heads, 2, bytes of a token]
    return _values(one, 1, dim)[..., 0, :]


def _plain_append(s):
    case = s["case"]
    page, dim = case["page"], case["head_dim"]
    session, at = _positions(s["row_offsets"], s["kv_len"], s["q"].shape[0])
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if case["rot"]:
        q, k = _rotate(q, s["table"], at, case["layout"]), _rotate(k, s["table"], at, case["layout"])
    where, slot = s["page_table"].long()[session, at // page], at % page
    groups = dim // GROUP
    codes = s["pages"][..., :page * dim // 2].unflatten(-1, (groups, page, 16))
    bytes_ = s["pages"][..., page * dim // 2:].unflatten(-1, (page, groups))
    code, byte, _ = _quantise(torch.stack([k, v], dim=2))
    packed = _block(code[..., None, :, :], byte[..., None, :])  # a token by itself
    codes[where, :, :, :, slot] = packed[..., :dim // 2].unflatten(-1, (groups, 16))
    bytes_[where, :, :, slot] = packed[..., dim // 2:]
    got = _read(s, session, at)
    return q.to(s["q"].dtype), got[:, :, 0].to(torch.bfloat16), got[:, :, 1].to(torch.bfloat16), torch.zeros(len(s["m"]), dtype=torch.int32, device=DEVICE)


def _plain_read(s):
    session, at = _positions(s["row_offsets"], s["start"], s["tokens"])
    got = _read(s, session, at)
    return got[:, :, 0].to(torch.bfloat16), got[:, :, 1].to(torch.bfloat16), torch.zeros(len(s["m"]), dtype=torch.int32, device=DEVICE)


def _plain_attend(s):
    case, n = s["case"], len(s["m"])
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
    seen = at <= last
    if case["window"]:
        seen &= at > last - case["window"]
    score = torch.where(seen.repeat_interleave(share, dim=1)[:, None], score, -math.inf)
    p = torch.exp(score - score.amax(dim=-1, keepdim=True))
    del score
    o = torch.matmul(p, kv[:, :, 1]) / p.sum(dim=-1, keepdim=True)
    o = o.unflatten(2, (wide, share)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o[session, i].to(torch.bfloat16), torch.zeros(n, dtype=torch.int32, device=DEVICE)


# ---- the definitions in 64 bits -------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"adjust": _exact_adjust, "append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _exact_adjust(s):
    case, vocab = s["case"], s["case"]["vocab"]
    extra = 1 if case["rows"] == "target" else 0
    out = torch.empty(s["logits"].shape, dtype=torch.float64, device=DEVICE)
    row = at = 0
    for b, m in enumerate(s["m"]):
        r, f, p = (float(torch.tensor(x, dtype=torch.float32)) for x in s["penalties"][b])
        ids = s["history"][b].long()
        prompt = torch.bincount(ids[:s["prompt"][b]], minlength=vocab) > 0
        count = torch.bincount(ids[s["prompt"][b]:s["hist"][b]], minlength=vocab).double()
        for i in range(m + extra):
            if i:
                count[s["draft_tokens"][at + i - 1].long()] += 1
            z = s["logits"][row].double()
            seen = prompt | (count > 0)
            z = torch.where(seen & (z > 0), z / r, torch.where(seen, z * r, z)) - f * count - p * (count > 0).double()
            if s["bias_tokens"] is not None:
                k = min(case["biases"], vocab)
                z[s["bias_tokens"][b * k:(b + 1) * k].long()] += s["bias_values"][b * k:(b + 1) * k].double()
            out[row] = z
            row += 1
        at += m
    if s["mask_rows"] is not None:
        which = s["mask_rows"].tolist()
        t = torch.arange(vocab, device=DEVICE)
        for row, w in enumerate(which):
            if w >= 0:
                out[row][(s["masks"][w].long()[t // 32] >> (t % 32)) & 1 == 0] = -math.inf
    return out, None


def _exact_session(s, b, tokens, cache):
    """float64 keys and values [tokens, heads, D] of a session."""
    if not cache:
        case = s["case"]
        size, dim = case["page"], case["head_dim"]
        t, d = torch.arange(size, device=DEVICE)[:, None], torch.arange(dim, device=DEVICE)[None, :]
        g, word, e = d // 32, (d % 32) // 8, d % 8
        bit = 4 * (e // 2 + 4 * (e % 2))
        cache.update(code=(g * size + t) * 16 + word * 4 + bit // 8, shift=bit % 8, byte=size * dim // 2 + t * (dim // 32) + g)
    need = -(-tokens // s["case"]["page"])
    raw = s["pages"][s["page_table"][b, :need].long()]
    n = (raw[..., cache["code"]] >> cache["shift"]) & 15
    byte = raw[..., cache["byte"]].short()
    v = (n.short() - 8).double() * (1 + (byte % 8).double() / 8) * torch.exp2((byte // 8 - 15).double())  # [pages, heads, 2, P, D]
    v = v.permute(2, 0, 3, 1, 4).flatten(1, 2)[:, :tokens]
    return v[0], v[1]


def _exact_append(s):
    case = s["case"]
    rot = case["rot"]
    at = torch.cat([torch.arange(c, c + m + 1, device=DEVICE) for c, m in zip(s["ctx"], s["m"])])

    def turn(x):
        x = x.double().clone()
        if rot:
            cos, sin = s["table"][at].double()[:, :rot // 2, None], s["table"][at].double()[:, rot // 2:, None]
            first = torch.arange(rot // 2, device=DEVICE) * (1 if case["layout"] == "half" else 2)
            second = first + (rot // 2 if case["layout"] == "half" else 1)
            a, b = x[:, :, first].transpose(1, 2), x[:, :, second].transpose(1, 2)
            x[:, :, first], x[:, :, second] = (a * cos - b * sin).transpose(1, 2), (a * sin + b * cos).transpose(1, 2)
        return x

    def held(x):
        x = x.double()
        g = x.reshape(*x.shape[:-1], -1, 32)
        most = g.abs().max(dim=-1, keepdim=True).values / 7
        e = torch.floor(torch.log2(most.clamp(min=2.0**-14)))
        scale = torch.ceil(most / torch.exp2(e) * 8).clamp(min=8) / 8 * torch.exp2(e)
        scale = scale.clamp(2.0**-14, 60.0)
        return ((g / scale).round().clamp(-7, 7) * scale).reshape(x.shape)

    return turn(s["q"]), held(turn(s["k"])), held(s["v"]), None


def _exact_read(s):
    ks, vs, cache = [], [], {}
    for b, (a, c) in enumerate(zip(s["starts"], s["ctx"])):
        if c:
            k, v = _exact_session(s, b, a + c, cache)
            ks.append(k[a:])
            vs.append(v[a:])
    if not ks:
        return None
    return torch.cat(ks), torch.cat(vs), None


def _exact_attend(s):
    case = s["case"]
    share = case["q_heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
    row, cache = 0, {}
    for b, (c, m) in enumerate(zip(s["ctx"], s["m"])):
        k, v = _exact_session(s, b, c + m + 1, cache)
        q = s["q"][row:row + m + 1].double().reshape(m + 1, case["kv_heads"], share, -1)
        score = torch.einsum("ihgd,thd->hgit", q, k) * s["scale"]
        last = c + torch.arange(m + 1, device=DEVICE)[:, None]
        t = torch.arange(c + m + 1, device=DEVICE)[None, :]
        hidden = t > last
        if case["window"]:
            hidden |= t <= last - case["window"]
        score.masked_fill_(hidden, -math.inf)
        p = torch.softmax(score, dim=-1)
        out[row:row + m + 1] = torch.einsum("hgit,thd->ihgd", p, v).reshape(m + 1, case["q_heads"], -1)
        row += m + 1
    return out, None
