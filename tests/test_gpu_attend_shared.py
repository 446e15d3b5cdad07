"""sdcp_attend_shared_kv against the plain 64-bit implementation (tests/serving_reference.py).

The tolerance is the one of tests/test_gpu_attend.py, and holds for the same reasons: the result is rounded
to bfloat16 (2^-8 of it at most), weights to 11 bits (2^-11 of sum p |v|; the rest of 2^-10 of it is for the
sums, the exponentials and the division in binary32), a score of magnitude sum A rounds by at most 2^-19 A,
and weights below 2^-31 of a reference that is at most the largest may be lost."""
import numpy as np
import pytest
import torch

from test_gpu_attend import DEV, Case, dev
import serving_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()


class Shared(Case):
    """Groups of `sizes` sessions, group g's rows alike in their first common[g] pages."""

    def __init__(self, sizes, common, ms, lens, P, Hkv, share, D, seed, **kw):
        super().__init__(ms, lens, P, Hkv, share, D, seed, **kw)
        self.group_offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        for g, n in enumerate(common):
            b0, b1 = self.group_offsets[g], self.group_offsets[g + 1]
            assert all(lens[b] >= n * P for b in range(b0, b1))
            if b0 < b1:
                self.table[b0:b1, :n] = self.table[b0, :n]

    def tensors(self, gap=0, pages=None, groups=True, workspace_fill=255):
        from speculative_decoding_verification_sdcp_gb300 import sdcp
        B = len(self.ms)
        cache = sdcp.KvCache(self.n_pages, self.P, self.Hkv, self.D, DEV, pages=dev(self.pages) if pages is None else pages)
        wide = torch.full((self.total + B, self.Hq * self.D + gap), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, :self.Hq * self.D] = dev(self.q).flatten(1).to(torch.bfloat16)
        q = wide[:, :self.Hq * self.D].unflatten(1, (self.Hq, self.D))
        out = torch.full((self.total + B, self.Hq, self.D), 5.0, dtype=torch.bfloat16, device=DEV)
        st = torch.full((B,), -9, dtype=torch.int32, device=DEV)
        n = len(self.group_offsets) - 1 if groups else 0
        ws = sdcp.alloc_attend_shared_workspace(B, self.total, n, self.Hq, self.Hkv, self.D, DEV).fill_(workspace_fill)
        return [cache, dev(self.table), dev(self.off), self.total, dev(np.array(self.lens, dtype=np.int32)),
                dev(self.group_offsets) if groups else None, q, out, st, ws]

    def run(self, stream=None, **kw):
        from speculative_decoding_verification_sdcp_gb300 import sdcp
        t = self.tensors(**kw)
        torch.cuda.synchronize()
        sdcp.sdcp_attend_shared_kv(*t, scale=self.scale, stream=None if stream is None else stream.cuda_stream)
        torch.cuda.synchronize()
        return t[7], t[8].cpu().numpy()


def ragged(seed, n, m_hi, common, P, tail):
    """Sizes of n sessions in one group with `common` pages."""
    r = np.random.default_rng(seed)
    return dict(ms=r.integers(0, m_hi + 1, n).tolist(), lens=(common * P + r.integers(0, tail + 1, n)).tolist(), sizes=[n], common=[common], P=P)


CASES = [dict(sizes=[1], common=[0], ms=[0], lens=[0], P=16, Hkv=1, share=1, D=64),
         dict(sizes=[2], common=[8], ms=[0, 0], lens=[128, 128], P=16, Hkv=2, share=4, D=128),           # no tail but the row itself
         dict(sizes=[2], common=[7], ms=[0, 1], lens=[112, 130], P=16, Hkv=1, share=8, D=128),           # too little to share
         dict(sizes=[3, 1, 2], common=[9, 0, 20], ms=[0, 4, 8, 2, 0, 16], lens=[144, 160, 300, 77, 350, 320], P=16, Hkv=2, share=7, D=64),
         dict(sizes=[4], common=[3], ms=[3, 0, 1, 7], lens=[200, 192, 500, 333], P=64, Hkv=2, share=4, D=128),
         dict(**ragged(1, 9, 6, 10, 32, 200), Hkv=1, share=8, D=128),                                    # two blocks and a rest
         dict(**ragged(2, 20, 9, 2, 128, 300), Hkv=2, share=8, D=64),                                    # several items of 256 pairs
         dict(sizes=[2], common=[1], ms=[70, 130], lens=[1024, 1500], P=1024, Hkv=1, share=3, D=128),    # long rounds
         dict(sizes=[1], common=[0], ms=[300], lens=[0], P=16, Hkv=1, share=2, D=64),                    # a prompt by itself
         dict(sizes=[0, 5, 0, 0, 1, 0], common=[0, 30, 0, 0, 0, 0], ms=[0] * 6, lens=[480, 481, 495, 600, 512, 9], P=16, Hkv=4, share=1, D=128),
         dict(sizes=[40], common=[16], ms=[0] * 40, lens=[256 + 7 * i for i in range(40)], P=16, Hkv=1, share=20, D=64),
         dict(sizes=[2], common=[300], ms=[1, 0], lens=[4800, 4823], P=16, Hkv=1, share=1, D=64)]        # one item over many blocks


def stretched(case, k):
    """The case with pages and contexts k times as long: short stretches are attended session by session."""
    return {**case, "P": case["P"] * k, "lens": [n * k for n in case["lens"]]}


@pytest.mark.parametrize("k", [1, 8])
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_against_plain(ci, k):
    if CASES[ci]["P"] * k > 1024:
        k = 1024 // CASES[ci]["P"]
    c = Shared(seed=170 + ci, **stretched(CASES[ci], k))
    c.check(*c.run(gap=8 * (ci % 3)))
    if len(c.group_offsets) == 2:
        x, st = c.run(groups=False, workspace_fill=0)
        c.check(x, st)


@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("n,groups", [(300, 40), (300, 290), (60, 1)])
def test_many_sessions_and_groups(n, groups, P):
    """More sessions, and more groups, than a block looks over by itself."""
    r = np.random.default_rng(n + groups)
    cuts = np.sort(r.integers(0, n + 1, groups - 1)).tolist()
    sizes = np.diff([0] + cuts + [n]).tolist()
    common = [int(r.integers(0, 14)) for _ in sizes]
    lens = [common[g] * P + int(r.integers(0, 150)) for g, k in enumerate(sizes) for _ in range(k)]
    c = Shared(sizes, common, r.integers(0, 4, n).tolist(), lens, P=P, Hkv=1, share=4, D=64, seed=n)
    c.check(*c.run())


@pytest.mark.parametrize("q_scale,scale", [(0.0, None), (1.0, 0.0), (6.0, 0.5), (3.0, -0.3), (40.0, 1.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_flat_sharp_and_negative_scores(D, q_scale, scale):
    c = Shared([3], [20], [3, 0, 1], [700, 640, 641], P=32, Hkv=2, share=4, D=D, seed=5, q_scale=q_scale, scale=scale)
    c.check(*c.run())


@pytest.mark.parametrize("scale_bytes", [(8, 9), (8, 168), (160, 168)])
def test_scales_over_the_whole_range(scale_bytes):
    c = Shared([2], [16], [3, 1], [260, 264], P=16, Hkv=1, share=8, D=128, seed=6, scale_bytes=scale_bytes, scale=1e-3)
    c.check(*c.run())


@pytest.mark.parametrize("members", [2, 60])
def test_rising_scores_move_the_reference(members):
    """Later tokens score far above the earlier ones, tile after tile, in one block of pairs and in two."""
    c = Shared([members], [90], [2] * members, [1440 + i for i in range(members)], P=16, Hkv=1, share=4, D=64, seed=7, q_scale=0.01)
    for t in range(1440):
        blk = c.pages[c.table[0, t // 16], 0, 0]
        blk[16 * 32 + (t % 16) * 2:16 * 32 + (t % 16) * 2 + 2] = min(167, 90 + t // 22)
        for g in range(2):
            blk[(g * 16 + t % 16) * 16:(g * 16 + t % 16) * 16 + 16] = 0xFF  # n = 7 everywhere
    c.q[:] = ref.bf16(np.abs(c.q))
    c.check(*c.run())


@pytest.mark.parametrize("k", [1, 8])
def test_a_row_with_nan_or_infinities_keeps_to_itself(k):
    c = Shared([2, 1], [10, 0], [3, 2, 1], [200 * k, 177 * k, 20], P=16 * k, Hkv=2, share=4, D=128, seed=8)
    c.q[1, 2, 5] = np.nan
    c.q[5, 7, 0] = np.inf
    c.q[5, 7, 1] = -np.inf
    c.q[5, 7, 2:] = np.nan
    c.q[8, 0, 3] = np.nan
    c.check(*c.run(), nan_rows={(1, 2), (5, 7), (8, 0)})


@pytest.mark.parametrize("k", [1, 8])
def test_sessions_that_are_refused_are_zero_and_leave_their_group(k):
    from speculative_decoding_verification_sdcp_gb300 import sdcp

    def case(change, bad, want):
        c = Shared([4], [10], [2, 3, 1, 0], [165 * k, 160 * k, 180 * k, 300 * k], P=16 * k, Hkv=2, share=2, D=64, seed=9)
        change(c)
        out, st = c.run()
        c.check(out, st, bad)
        assert all(st[b] == want for b in bad)

    case(lambda c: c.lens.__setitem__(0, -1), (0,), sdcp.S_BAD_PARAMS)
    case(lambda c: c.lens.__setitem__(1, -5), (1,), sdcp.S_BAD_PARAMS)
    case(lambda c: c.table.__setitem__((0, 2), -1), (0,), sdcp.S_BAD_PARAMS)
    case(lambda c: c.table.__setitem__((2, 10), c.n_pages), (2,), sdcp.S_BAD_PARAMS)
    case(lambda c: c.table.__setitem__((slice(0, 4), 1), -7), (0, 1, 2, 3), sdcp.S_BAD_PARAMS)
    case(lambda c: c.lens.__setitem__(3, 2**31 - 1), (3,), sdcp.S_LIMIT)


def test_offsets_out_of_order():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    for groups in ([0, 3, 2, 4], [1, 4], [0, 3], [0, 5], [-1, 4]):
        c = Shared([4], [10], [2, 3, 1, 0], [165, 160, 180, 300], P=16, Hkv=1, share=2, D=64, seed=1)
        c.group_offsets = np.array(groups, dtype=np.int32)
        out, st = c.run()
        assert st.tolist() == [sdcp.S_BAD_PARAMS] * 4 and (out == 0).all()
    c = Shared([2], [10], [2, 2], [165, 160], P=16, Hkv=1, share=2, D=64, seed=1)
    c.off = np.array([0, 9, 4], dtype=np.int32)
    out, st = c.run()
    assert st.tolist() == [sdcp.S_BAD_PARAMS] * 2 and (out == 0).all()


@pytest.mark.parametrize("k", [1, 8])
def test_last_offsets_past_the_batch(k):
    """The last session's own pair is out of range: it is refused, the others' rows are theirs alone."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    c = Shared([3], [10], [2, 3, 1], [165 * k, 160 * k, 180 * k], P=16 * k, Hkv=1, share=4, D=64, seed=2)
    c.off = c.off.copy()
    c.off[3] += 1000
    out, st = c.run()
    assert st.tolist() == [0, 0, sdcp.S_BAD_PARAMS]
    c.check(out, st, (2,))


def test_another_stream_and_repeats_are_bit_equal():
    c = Shared([2, 3], [40, 9], [4, 0, 7, 1, 2], [1500, 3000, 400, 288, 301], P=32, Hkv=2, share=8, D=128, seed=10)
    x, _ = c.run()
    y, st = c.run(stream=torch.cuda.Stream(), workspace_fill=0)
    assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    c.check(y, st)


def test_captured_and_replayed_with_new_contents():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    a = Shared([2, 2], [90, 9], [1, 2, 0, 3], [1600, 1560, 150, 160], P=16, Hkv=2, share=4, D=64, seed=11)
    b = Shared([2, 2], [9, 80], [1, 2, 0, 3], [150, 170, 1330, 1321], P=16, Hkv=2, share=4, D=64, seed=12)
    wide = max(a.table.shape[1], b.table.shape[1])
    n = max(a.n_pages, b.n_pages)
    for c in (a, b):
        c.table = np.pad(c.table, ((0, 0), (0, wide - c.table.shape[1])), constant_values=-1)
        c.pages = np.pad(c.pages, ((0, n - c.n_pages), (0, 0), (0, 0), (0, 0)))
        c.n_pages = n
    t = a.tensors()
    sdcp.sdcp_attend_shared_kv(*t, scale=a.scale)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdcp.sdcp_attend_shared_kv(*t, scale=a.scale)
    for c in (b, a):
        new = c.tensors()
        t[0].pages.copy_(new[0].pages)
        for k in (1, 2, 4, 5):
            t[k].copy_(new[k])
        t[6].copy_(new[6])
        t[7].fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check(t[7], t[8].cpu().numpy())


def test_pages_past_2_32_bytes():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    c = Shared([2], [23], [2, 0], [1500, 1530], P=64, Hkv=8, share=1, D=128, seed=12)
    x, _ = c.run()
    n = (5 << 30) // int(sdcp.lib.sdcp_kv_page_bytes(64, 8, 128))
    big = torch.empty((n, 8, 2, 64 * 68), dtype=torch.uint8, device=DEV)
    big[n - c.n_pages:] = dev(c.pages)
    c.table[c.table >= 0] += n - c.n_pages
    c.n_pages = n
    y, st = c.run(pages=big)
    assert st.tolist() == [0, 0] and torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,members,prefix", [(0, 4, 20000), (8, 30, 3000), (3, 64, 640)])
def test_large_batches_against_the_attention_of_sessions(m, members, prefix, D):
    """Sizes that the plain implementation is slow at: every output within two tolerances of sdcp_attend_kv's."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    P, heads, share = 64, 2, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(m)
    common, r = prefix // P, np.random.default_rng(m)
    lens = [common * P + int(r.integers(0, 500)) for _ in range(members)]
    per = [-(-(n + m + 1) // P) - common for n in lens]
    cache = sdcp.KvCache(common + sum(per), P, heads, D, DEV)
    for which in (0, 1):
        cache.pages[:, :, which, :P * D // 2].random_(0, 256, generator=g)
        cache.pages[:, :, which, P * D // 2:].random_(96, 112, generator=g)
    cache.pages[..., :P * D // 2] |= 0x11  # codes of -7 at least
    table, at = torch.full((members, common + max(per)), -1, dtype=torch.int32, device=DEV), common
    for b, k in enumerate(per):
        table[b, :common] = torch.arange(common, dtype=torch.int32)
        table[b, common:common + k] = torch.arange(at, at + k, dtype=torch.int32)
        at += k
    off, kv_len = torch.arange(members + 1, dtype=torch.int32, device=DEV) * m, torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.randn((members * (m + 1), heads * share, D), generator=g, device=DEV).to(torch.bfloat16)
    x, y, st = torch.empty_like(q), torch.empty_like(q), torch.empty(members, dtype=torch.int32, device=DEV)
    sdcp.sdcp_attend_kv(cache, table, off, members * m, kv_len, q, x, st, sdcp.alloc_attend_workspace(members, members * m, heads * share, heads, D, DEV))
    sdcp.sdcp_attend_shared_kv(cache, table, off, members * m, kv_len, None, q, y, st,
                               sdcp.alloc_attend_shared_workspace(members, members * m, 0, heads * share, heads, D, DEV))
    assert st.tolist() == [0] * members
    # |v| <= 7 * the largest scale of the pages; scores as small as these leave A below 2^7
    most = 7 * ref.scale_of(111)
    assert bool(((x.double() - y.double()).abs() <= 2 * (2.0**-8 * x.double().abs() + (2.0**-10 + 2.0**-11) * most)).all())


@pytest.mark.parametrize("share", [130, 300])
def test_more_heads_on_a_cached_one_than_a_block_has_pairs(share):
    c = Shared([2], [13], [1, 0], [1700, 1664], P=128, Hkv=1, share=share, D=64, seed=31)
    c.check(*c.run())


def test_two_calls_at_once():
    """Two streams, a workspace each: what each gives by itself."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    cases = [Shared([4], [40], [3, 0, 8, 1], [1290, 1400, 1281, 1300], P=32, Hkv=2, share=8, D=D, seed=32 + D) for D in (64, 128)]
    alone = [c.run()[0] for c in cases]
    streams, tensors = [torch.cuda.Stream() for _ in cases], [c.tensors() for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, t in zip(cases, streams, tensors):
            sdcp.sdcp_attend_shared_kv(*t, scale=c.scale, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for c, t, want in zip(cases, tensors, alone):
        assert torch.equal(t[7].view(torch.int16), want.view(torch.int16)) and t[8].tolist() == [0] * 4


def test_rows_behind_the_batch_stay():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    c = Shared([3], [13], [1, 0, 2], [1700, 1664, 1669], P=128, Hkv=1, share=4, D=128, seed=33)
    t = c.tensors()
    more = lambda x, v: torch.cat([x, torch.full_like(x[:2], v)])  # noqa: E731
    t[6], t[7] = more(t[6], float("nan")), more(t[7], 7.0)
    sdcp.sdcp_attend_shared_kv(*t, scale=c.scale)
    assert bool((t[7][-2:] == 7.0).all())
    c.check(t[7][:-2], t[8].cpu().numpy())


def test_a_wide_range_of_magnitudes():
    """Queries of 2^-120 .. 2^100.  Where the largest score leads by more than scores round, its token has all the weight."""
    c = Shared([2], [13], [3, 3], [1700, 1669], P=128, Hkv=1, share=4, D=64, seed=34, scale=1.0)
    for r in range(8):
        c.q[r] = ref.bf16(c.q[r] * np.float32(2.0) ** [-120, -60, -20, -5, 0, 8, 20, 100][r])
    out, st = c.run()
    assert st.tolist() == [0, 0]
    c.check(out, st)
    got, alone = out.double().cpu().numpy(), 0
    v = ref.block_values(c.pages[c.table[1, :14]], c.P, c.D).transpose(2, 1, 0, 3, 4).reshape(2, -1, c.D)
    for r in (6, 7):
        for h in range(4):
            q = c.q[r, h].astype(np.float64)
            seen = v[0, :1669 + r - 3]
            s, a = seen @ q, (np.abs(seen) @ np.abs(q)).max()
            top = np.sort(s)[-2:]
            if top[1] - top[0] > 2.0**-17 * a + 100:
                want, alone = v[1, s.argmax()], alone + 1
                assert (np.abs(got[r, h] - want) <= 2.0**-8 * np.abs(want)).all()
    assert alone >= 4
