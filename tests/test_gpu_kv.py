"""sdcp_append_kv and sdcp_read_kv against the plain implementation (tests/serving_reference.py).

The definition fixes every rounding, so the cache's bytes are equal bit for bit to the plain
implementation's with binary32 steps, and q_out is its rotated row rounded once.  Against 64 bits: a
cached value is within half a scale of the rotated key (plus the rotation's three binary32 roundings,
3 * 2^-24 of the pair's magnitudes), and no smaller scale would have held the group."""
import numpy as np
import pytest
import torch

import serving_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


class Round:
    def __init__(self, ms, lens, P, Hkv, Hq, D, dtype, rot, layout, seed, spread=4):
        r = np.random.default_rng(seed)
        self.ms, self.lens, self.P, self.Hkv, self.Hq, self.D = ms, lens, P, Hkv, Hq, D
        self.rot, self.layout, self.dtype = rot, layout, dtype
        B = len(ms)
        self.off = np.concatenate([[0], np.cumsum(ms)]).astype(np.int32)
        self.total = int(self.off[-1])
        self.rows = self.total + B
        need = [-(-(c + m + 1) // P) for c, m in zip(lens, ms)]
        self.n_pages = sum(need) + 2
        order = r.permutation(self.n_pages)
        self.table = np.full((B, max(need) + 1), -1, dtype=np.int32)
        k = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[k:k + n]
            k += n
        self.pages = r.integers(0, 256, size=(self.n_pages, Hkv, 2, P * (D // 2 + D // 32)), dtype=np.uint8)
        x = r.normal(0, 1, size=(self.rows, Hq + 2 * Hkv, D)) * np.exp2(r.integers(-spread, spread + 1, size=(self.rows, Hq + 2 * Hkv, 1)))
        self.x = ref.bf16(x) if dtype == torch.bfloat16 else x.astype(np.float32)
        self.rope = None
        if rot:
            a = np.arange(max(c + m + 1 for c, m in zip(lens, ms)))[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)[None, :]
            self.rope = np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)

    def run(self, with_q=True, gap=0, stream=None):
        from speculative_decoding_verification_sdcp_gb300 import sdcp
        self.cache = sdcp.KvCache(self.n_pages, self.P, self.Hkv, self.D, DEV, pages=dev(self.pages))
        wide = torch.full((self.rows, (self.Hq + 2 * self.Hkv) * self.D + gap), float("nan"), dtype=self.dtype, device=DEV)
        wide[:, :wide.shape[1] - gap] = dev(self.x).to(self.dtype).flatten(1)
        heads = wide[:, :wide.shape[1] - gap].unflatten(1, (-1, self.D))
        q, k, v = heads[:, :self.Hq], heads[:, self.Hq:self.Hq + self.Hkv], heads[:, self.Hq + self.Hkv:]
        q_out = torch.full((self.rows, self.Hq, self.D), float("nan"), dtype=self.dtype, device=DEV)
        status = torch.full((len(self.ms),), -9, dtype=torch.int32, device=DEV)
        rotary = None if self.rope is None else sdcp.Rotary(dev(self.rope), self.layout)
        args = (self.cache, dev(self.table), dev(self.off), self.total, dev(np.array(self.lens, dtype=np.int32)), k, v, status)
        torch.cuda.synchronize()
        sdcp.sdcp_append_kv(*args, rotary=rotary, q=q if with_q else None, q_out=q_out if with_q else None,
                            stream=None if stream is None else stream.cuda_stream)
        torch.cuda.synchronize()
        return q_out.float().cpu().numpy(), self.cache.pages.cpu().numpy(), status.cpu().numpy()

    def check(self, q_out, pages, status, bad=(), with_q=True):
        want = self.pages.copy()
        row = 0
        for b, (m, c) in enumerate(zip(self.ms, self.lens)):
            for i in range(m + 1):
                if b not in bad:
                    pos = c + i
                    t = None if self.rope is None else self.rope[pos]
                    page, slot = self.table[b, pos // self.P], pos % self.P
                    for h in range(self.Hq + 2 * self.Hkv):
                        x = self.x[row, h]
                        if h < self.Hq:
                            if with_q:
                                y = ref.rotate_row(x, t, self.layout, np.float32)
                                assert np.array_equal(q_out[row, h], ref.bf16(y) if self.dtype == torch.bfloat16 else y, equal_nan=True)
                            continue
                        kh, which = (h - self.Hq, 0) if h < self.Hq + self.Hkv else (h - self.Hq - self.Hkv, 1)
                        t2 = t if which == 0 else None
                        y = ref.rotate_row(x, t2, self.layout, np.float32)
                        n, sbs = ref.quantise_row(y)
                        ref.write_token(want[page, kh, which], slot, self.P, self.D, n, sbs)
                        if np.isfinite(x).all() and np.abs(x).max() < 290:
                            y64 = ref.rotate_row(x, t2, self.layout, np.float64)
                            s = np.repeat([ref.scale_of(int(z)) for z in sbs], 32)
                            err = 3 * 2.0**-24 * 2 * np.abs(x).max()
                            assert (np.abs(n * s - y64) <= s / 2 + err).all()
                            for g, sb in enumerate(sbs):
                                if sb > 8:
                                    assert np.abs(y64[g * 32:g * 32 + 32]).max() + err > 7 * ref.scale_of(int(sb) - 1)
                row += 1
        assert np.array_equal(pages, want)
        for b in range(len(self.ms)):
            assert (status[b] == 0) == (b not in bad)


CASES = [dict(ms=[0], lens=[0], P=16, Hkv=1, Hq=1, D=64, rot=64, layout=0),
         dict(ms=[0, 3, 16], lens=[15, 14, 100], P=16, Hkv=2, Hq=6, D=128, rot=128, layout=0),
         dict(ms=[4, 0], lens=[31, 1], P=32, Hkv=3, Hq=5, D=64, rot=32, layout=1),
         dict(ms=[40], lens=[0], P=16, Hkv=1, Hq=0, D=128, rot=16, layout=0),
         dict(ms=[2, 2], lens=[63, 64], P=64, Hkv=8, Hq=8, D=128, rot=6, layout=0),
         dict(ms=[2, 1], lens=[127, 5], P=128, Hkv=1, Hq=7, D=64, rot=2, layout=1),
         dict(ms=[1, 5, 0, 9], lens=[1023, 1020, 0, 7], P=1024, Hkv=2, Hq=2, D=64, rot=0, layout=0),
         dict(ms=[1], lens=[3], P=16, Hkv=2, Hq=20, D=128, rot=100, layout=0),
         dict(ms=[1], lens=[3], P=16, Hkv=2, Hq=3, D=128, rot=126, layout=1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_append_against_plain(ci, dtype):
    c = dict(CASES[ci])
    with_q = c["Hq"] > 0
    r = Round(dtype=dtype, seed=40 + ci, **c)
    r.check(*r.run(with_q=with_q, gap=8 * (ci % 3)), with_q=with_q)


def test_many_sessions_and_a_long_round():
    """Sessions found among many, and a prompt over several pages."""
    r = Round(ms=[i % 3 for i in range(70)] + [150], lens=[i % 37 for i in range(71)], P=16, Hkv=1, Hq=1, D=64,
              dtype=torch.bfloat16, rot=16, layout=1, seed=2)
    r.check(*r.run())


def test_values_at_the_ends_of_the_range():
    r = Round(ms=[8], lens=[0], P=16, Hkv=1, Hq=1, D=64, dtype=torch.float32, rot=0, layout=0, seed=3)
    r.x[0] = 0.0
    r.x[1] = 1e-30
    r.x[2, :, ::2] = 1e6
    r.x[3, :, 5] = np.inf
    r.x[4, :, 6] = np.nan
    r.x[5] = np.nan
    r.x[6, :, 7] = -np.inf
    r.x[7] = 7 * 1.125      # a largest magnitude that is seven scales exactly
    r.x[8] = np.where(np.arange(64) % 2, 7.0, 2.5)  # ties between codes
    r.check(*r.run())


def test_sessions_that_are_refused_write_nothing():
    from speculative_decoding_verification_sdcp_gb300 import sdcp

    def case(change, bad, want):
        r = Round(ms=[2, 3, 1], lens=[5, 30, 0], P=16, Hkv=2, Hq=2, D=64, dtype=torch.bfloat16, rot=16, layout=0, seed=9)
        change(r)
        q, pages, st = r.run()
        r.check(q, pages, st, bad)
        assert all(st[b] == want for b in bad)

    case(lambda r: r.lens.__setitem__(0, -1), (0,), sdcp.S_BAD_PARAMS)
    case(lambda r: r.table.__setitem__((1, 2), -1), (1,), sdcp.S_BAD_PARAMS)
    case(lambda r: r.table.__setitem__((1, 2), r.n_pages), (1,), sdcp.S_BAD_PARAMS)
    case(lambda r: r.lens.__setitem__(2, 16 * r.table.shape[1] - 1), (2,), sdcp.S_LIMIT)
    case(lambda r: r.lens.__setitem__(2, 2**31 - 1), (2,), sdcp.S_LIMIT)
    case(lambda r: setattr(r, "rope", r.rope[:33]), (1,), sdcp.S_LIMIT)


def test_offsets_out_of_order():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    r = Round(ms=[2, 2], lens=[0, 0], P=16, Hkv=1, Hq=1, D=64, dtype=torch.bfloat16, rot=0, layout=0, seed=1)
    r.off = np.array([0, 9, 4], dtype=np.int32)
    _, pages, st = r.run()
    assert st.tolist() == [sdcp.S_BAD_PARAMS] * 2 and np.array_equal(pages, r.pages)


@pytest.mark.parametrize("D,P,dtype", [(64, 16, torch.bfloat16), (128, 64, torch.float32), (128, 16, torch.bfloat16)])
def test_read_against_plain(D, P, dtype):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    r = np.random.default_rng(D + P)
    ns, starts, Hkv = [0, 1, 33, 0, 70, 8], [3, 15, 0, 9, 17, 40], 3
    need = [-(-(s + n) // P) for s, n in zip(starts, ns)]
    n_pages = sum(need) + 1
    table = np.full((len(ns), max(need)), -1, dtype=np.int32)
    order, k = r.permutation(n_pages), 0
    for b, n in enumerate(need):
        table[b, :n] = order[k:k + n]
        k += n
    pages = r.integers(0, 256, size=(n_pages, Hkv, 2, P * (D // 2 + D // 32)), dtype=np.uint8)
    pages[..., P * D // 2:] = r.integers(8, 168, size=pages[..., P * D // 2:].shape)
    off = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    cache = sdcp.KvCache(n_pages, P, Hkv, D, DEV, pages=dev(pages))
    ko = torch.full((sum(ns), Hkv, D), 9.0, dtype=dtype, device=DEV)
    vo = torch.full_like(ko, 9.0)
    st = torch.full((len(ns),), -9, dtype=torch.int32, device=DEV)
    table[2, 1 if need[2] > 1 else 0] = n_pages  # session 2 is refused
    sdcp.sdcp_read_kv(cache, dev(table), dev(off), sum(ns), dev(np.array(starts, dtype=np.int32)), ko, vo, st)
    only = torch.full_like(ko, 9.0)
    sdcp.sdcp_read_kv(cache, dev(table), dev(off), sum(ns), dev(np.array(starts, dtype=np.int32)), None, only, st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0, sdcp.S_BAD_PARAMS, 0, 0, 0]
    assert torch.equal(only, vo)
    for b, (n, s) in enumerate(zip(ns, starts)):
        for i in range(n):
            for h in range(Hkv):
                for which, t in ((0, ko), (1, vo)):
                    got = t[off[b] + i, h].double().cpu().numpy()
                    pos = s + i
                    want = np.zeros(D) if b == 2 else ref.token_values(pages[table[b, pos // P], h, which], pos % P, P, D)
                    assert np.array_equal(got, want)  # n s is exact in both types


def test_pages_past_2_32_bytes_and_another_stream():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    r = Round(ms=[3], lens=[61], P=64, Hkv=8, Hq=2, D=128, dtype=torch.bfloat16, rot=64, layout=0, seed=21)
    q, pages, st = r.run(stream=torch.cuda.Stream())
    r.check(q, pages, st)
    n = (5 << 30) // int(sdcp.lib.sdcp_kv_page_bytes(64, 8, 128))
    big = sdcp.KvCache(n, 64, 8, 128, DEV, pages=torch.empty((n, 8, 2, 64 * 68), dtype=torch.uint8, device=DEV))
    table = np.array([[n - 1, n - 2, -1]], dtype=np.int32)
    x = dev(r.x).to(torch.bfloat16)
    status = torch.empty(1, dtype=torch.int32, device=DEV)
    ko = torch.empty((4, 8, 128), dtype=torch.bfloat16, device=DEV)
    vo, k2, v2 = torch.empty_like(ko), torch.empty_like(ko), torch.empty_like(ko)
    lens, off, four = dev(np.array([61], dtype=np.int32)), dev(r.off), dev(np.array([0, 4], dtype=np.int32))
    rope = sdcp.Rotary(dev(r.rope), 0)
    sdcp.sdcp_append_kv(big, dev(table), off, r.total, lens, x[:, 2:10], x[:, 10:], status, rotary=rope)
    sdcp.sdcp_read_kv(big, dev(table), four, 4, lens, ko, vo, status)
    sdcp.sdcp_read_kv(r.cache, dev(r.table), four, 4, lens, k2, v2, status)
    torch.cuda.synchronize()
    assert status.tolist() == [0] and torch.equal(ko, k2) and torch.equal(vo, v2)
