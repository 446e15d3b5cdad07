"""Offsets out of order, in every call that takes them: two sessions' rows may then overlap, and each
would be written by both.  Every session of such a batch is refused; offsets in order that leave rows out
at the ends are taken.  The scores' tolerance is that of tests/test_gpu_attend.py."""
import numpy as np
import pytest
import torch

import serving_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P, D = 16, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _shuffled(B, seed):
    r = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(r.integers(0, 4, B))])
    total = int(off[-1])
    at = r.integers(0, B + 1, max(2, B // 20))
    off[at] = np.clip(off[at] + r.integers(-9, 10, at.size), 0, total)
    return off.tolist(), total


OFFSETS = [([0, 5, 3, 6], 6), ([0, 3, 6, 2, 8], 8), ([4, 0, 4], 4), ([0, 0, 2, 1, 1, 3], 3), ([1, 3, 3, 4], 6)] + [_shuffled(B, B) for B in (9, 60, 140, 300)]
MANY = [_shuffled(5000, 5000), (list(range(700)), 699)]  # more than a block looks over by itself


def _own_rows(off, total, status, extra):
    """Rows of the sessions that are SDCP_S_OK; none is shared."""
    assert set(status) == ({3} if min(np.diff(off)) < 0 else {0})
    rows = {}
    for b, st in enumerate(status):
        for r in range(off[b] + b * extra, off[b + 1] + (b + 1) * extra if st == 0 else 0):
            assert r not in rows
            rows[r] = b
    return rows


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("off,total", OFFSETS + MANY)
def test_adjust(off, total, kind):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    B, V, extra = len(off) - 1, 700, 1 - kind
    n = total + B * extra
    logits = np.random.default_rng(1).integers(-9, 9, (n, V)).astype(np.float32)
    ctl = np.zeros(B, dtype=sdcp.CONTROLS_DTYPE)
    ctl["repetition"], ctl["frequency"], ctl["history_len"] = 1.0, 2.0, 1
    out, st = torch.full((n, V), 7.5, device=DEV), torch.full((B,), -9, dtype=torch.int32, device=DEV)
    sdcp.sdcp_adjust_logits(dev(logits), out, dev(np.array(off, dtype=np.int32)), total, dev(np.full(total, -1, dtype=np.int32)),
                            sdcp.controls_tensor(ctl, DEV), dev((np.arange(B) % V).astype(np.int32)[:, None]), st, rows=kind)
    want = np.full((n, V), 7.5, dtype=np.float32)
    for r, b in _own_rows(off, total, st.tolist(), extra).items():
        want[r] = logits[r]
        want[r, b % V] -= 2.0
    assert np.array_equal(out.cpu().numpy(), want)


def test_a_session_refused_among_many():
    """Refused for its own controls: all its rows become NaN, whichever of its blocks comes first."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    B, V = 700, 9000
    logits = torch.ones((B, V), device=DEV)
    ctl = np.zeros(B, dtype=sdcp.CONTROLS_DTYPE)
    ctl["repetition"] = 1.0
    ctl["repetition"][::3] = 0.0
    st = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    sdcp.sdcp_adjust_logits(logits, logits, dev(np.zeros(B + 1, dtype=np.int32)), 0, None, sdcp.controls_tensor(ctl, DEV), None, st)
    got = logits.cpu().numpy()
    assert np.isnan(got[::3]).all() and (got[1::3] == 1).all() and (got[2::3] == 1).all()
    assert st.tolist() == [sdcp.S_BAD_PARAMS if b % 3 == 0 else 0 for b in range(B)]


def test_an_offset_out_of_range_among_many():
    """In order, but the last session's end is past the rows: it alone is refused, in every call."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    B = 700
    off = np.minimum(np.arange(B + 1), B - 1)
    off[B] = B + 5
    want = [0] * (B - 1) + [sdcp.S_BAD_PARAMS]
    offs, total = dev(off.astype(np.int32)), B
    st = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    ctl = np.zeros(B, dtype=sdcp.CONTROLS_DTYPE)
    ctl["repetition"] = 1.0
    logits = torch.ones((total + B, 5000), device=DEV)
    sdcp.sdcp_adjust_logits(logits, logits, offs, total, dev(np.zeros(total, dtype=np.int32)), sdcp.controls_tensor(ctl, DEV), None, st)
    assert st.tolist() == want and float(logits.min()) == float(logits.max()) == 1.0
    cache, _, table = _cache(sdcp, B, 2, 8)
    lens = dev(np.zeros(B, dtype=np.int32))
    x = torch.ones((total + B, 1, D), device=DEV)
    sdcp.sdcp_append_kv(cache, dev(table), offs, total, lens, x, x, st.fill_(-9))
    assert st.tolist() == want
    sdcp.sdcp_read_kv(cache, dev(table), offs, total, lens, x, x.clone(), st.fill_(-9))
    assert st.tolist() == want
    q = x.to(torch.bfloat16)
    sdcp.sdcp_attend_kv(cache, dev(table), offs, total, lens, q, torch.empty_like(q), st.fill_(-9),
                        sdcp.alloc_attend_workspace(B, total, 1, 1, D, DEV))
    assert st.tolist() == want


def _cache(sdcp, B, per, seed):
    r = np.random.default_rng(seed)
    pages = r.integers(0, 256, size=(B * per, 1, 2, P * (D // 2 + D // 32)), dtype=np.uint8)
    pages[..., :P * D // 2] |= 0x11
    pages[..., P * D // 2:] = r.integers(100, 120, size=pages[..., P * D // 2:].shape)
    table = r.permutation(B * per).astype(np.int32).reshape(B, per)
    return sdcp.KvCache(B * per, P, 1, D, DEV, pages=dev(pages)), pages, table


@pytest.mark.parametrize("off,total", OFFSETS + MANY[1:])
def test_append(off, total):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    B = len(off) - 1
    per = (max(np.diff(off)) + 4) // P + 2
    cache, pages, table = _cache(sdcp, B, per, 2)
    x = np.random.default_rng(3).normal(0, 1, size=(total + B, 2, D)).astype(np.float32)
    st = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    t = dev(x)
    sdcp.sdcp_append_kv(cache, dev(table), dev(np.array(off, dtype=np.int32)), total, dev(np.full(B, 3, dtype=np.int32)), t[:, :1], t[:, 1:], st)
    for r, b in _own_rows(off, total, st.tolist(), 1).items():
        pos = 3 + r - off[b] - b
        for which in (0, 1):
            ref.write_token(pages[table[b, pos // P], 0, which], pos % P, P, D, *ref.quantise_row(x[r, which]))
    assert np.array_equal(cache.pages.cpu().numpy(), pages)


@pytest.mark.parametrize("off,total", OFFSETS + MANY)
def test_read(off, total):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    B = len(off) - 1
    cache, pages, table = _cache(sdcp, B, (max(np.diff(off)) + 5) // P + 2, 4)
    k = torch.full((total, 1, D), 9.0, device=DEV)
    v, st = torch.full_like(k, 9.0), torch.full((B,), -9, dtype=torch.int32, device=DEV)
    sdcp.sdcp_read_kv(cache, dev(table), dev(np.array(off, dtype=np.int32)), total, dev(np.full(B, 5, dtype=np.int32)), k, v, st)
    want = np.zeros((2, total, D))
    for r, b in _own_rows(off, total, st.tolist(), 0).items():
        pos = 5 + r - off[b]
        for which in (0, 1):
            want[which, r] = ref.token_values(pages[table[b, pos // P], 0, which], pos % P, P, D)
    assert np.array_equal(torch.stack([k, v])[:, :, 0].cpu().numpy(), want)


@pytest.mark.parametrize("off,total", OFFSETS + MANY[1:])
def test_attend(off, total):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    B, share = len(off) - 1, 2
    per = (max(np.diff(off)) + 150) // P + 2
    cache, pages, table = _cache(sdcp, B, per, 6)
    values = ref.block_values(pages[table], P, D).transpose(0, 3, 2, 1, 4, 5).reshape(B, 2, per * P, D)
    q = ref.bf16(np.random.default_rng(7).normal(0, 1, size=(total + B, share, D)))
    lens = np.arange(B) % 150
    out = torch.full((total + B, share, D), 5.0, dtype=torch.bfloat16, device=DEV)
    st = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    ws = sdcp.alloc_attend_workspace(B, total, share, 1, D, DEV)
    sdcp.sdcp_attend_kv(cache, dev(table), dev(np.array(off, dtype=np.int32)), total, dev(lens.astype(np.int32)),
                        dev(q).to(torch.bfloat16), out, st, ws)
    got = out.double().cpu().numpy()
    own = _own_rows(off, total, st.tolist(), 1)
    claimed = {r for b in range(B) for r in range(max(0, off[b]) + b, min(max(off[b], off[b + 1]), total) + b + 1)}
    for r in range(total + B):
        if r not in own:
            assert (got[r] == (0 if r in claimed else 5)).all()
            continue
        b = own[r]
        last = int(lens[b]) + r - off[b] - b
        for h in range(share):
            k, v = values[b]
            want, mass, a = ref.attend_row(q[r, h].astype(np.float64), k, v, np.float64(np.float32(D ** -0.5)), 0, last)
            tol = 2.0**-8 * np.abs(want) + (2.0**-10 + 2.0**-18 * a) * mass + 2.0**-31 * np.abs(v[:last + 1]).sum(axis=0)
            assert (np.abs(got[r, h] - want) <= tol).all()
