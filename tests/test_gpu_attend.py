"""sdcp_attend_kv against the plain 64-bit implementation (tests/serving_reference.py).

Tolerance, from the arithmetic: the result is rounded to bfloat16 (2^-9 of it); a weight may be
rounded to 16 bits with 11 significant ones on the way (2^-12 of it, at most 2^-10 of sum p |v| with
the sums' own roundings); a score of magnitude sum A rounds by at most 2^-19 A, which scales a weight by
that much (twice, with the normaliser).  Weights are held as numbers of a finite range: one that is
below 2^-31 of the largest may be lost, sum |v| 2^-31 at most over the tokens.  So
|got - want| <= 2^-8 |want| + (2^-10 + 2^-18 A) sum p |v| + 2^-31 sum |v|."""
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


class Case:
    def __init__(self, ms, lens, P, Hkv, share, D, seed, window=0, q_scale=1.0, scale=None, scale_bytes=(104, 124)):
        r = np.random.default_rng(seed)
        self.ms, self.lens, self.P, self.Hkv, self.Hq, self.D = ms, lens, P, Hkv, Hkv * share, D
        self.share, self.window, self.scale = share, window, D ** -0.5 if scale is None else scale
        B = len(ms)
        self.off = np.concatenate([[0], np.cumsum(ms)]).astype(np.int32)
        self.total = int(self.off[-1])
        need = [-(-(c + m + 1) // P) for c, m in zip(lens, ms)]
        self.n_pages = sum(need) + 3
        order, k = r.permutation(self.n_pages), 0
        self.table = np.full((B, max(need) + 1), -1, dtype=np.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = order[k:k + n]
            k += n
        # every byte is garbage (scale bytes of any value) but for the cached tokens
        size = P * (D // 2 + D // 32)
        self.pages = r.integers(0, 256, size=(self.n_pages, Hkv, 2, size), dtype=np.uint8)
        for b in range(B):
            for p in range(need[b]):
                used = min(P, lens[b] + ms[b] + 1 - p * P)
                at = P * D // 2 + np.arange(used * (D // 32))
                self.pages[self.table[b, p], :, :, P * D // 2:P * D // 2 + at.size] = r.integers(*scale_bytes, size=(Hkv, 2, at.size))
                codes = self.pages[self.table[b, p]]
                for g in range(D // 32):  # codes -7..7
                    sl = codes[:, :, g * P * 16:(g * P + used) * 16]
                    lo, hi = sl & 15, sl >> 4
                    sl[:] = np.maximum(lo, 1) | (np.maximum(hi, 1) << 4)
        self.q = ref.bf16(r.normal(0, q_scale, size=(self.total + B, self.Hq, D)))

    def run(self, gap=0, stream=None, pages=None, workspace_fill=None):
        from speculative_decoding_verification_sdcp_gb300 import sdcp
        B = len(self.ms)
        cache = sdcp.KvCache(self.n_pages, self.P, self.Hkv, self.D, DEV, pages=dev(self.pages) if pages is None else pages)
        wide = torch.full((self.total + B, self.Hq * self.D + gap), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, :self.Hq * self.D] = dev(self.q).flatten(1).to(torch.bfloat16)
        q = wide[:, :self.Hq * self.D].unflatten(1, (self.Hq, self.D))
        out = torch.full((self.total + B, self.Hq, self.D), 5.0, dtype=torch.bfloat16, device=DEV)
        st = torch.full((B,), -9, dtype=torch.int32, device=DEV)
        ws = sdcp.alloc_attend_workspace(B, self.total, self.Hq, self.Hkv, self.D, DEV)
        ws.fill_(255 if workspace_fill is None else workspace_fill)
        args = (cache, dev(self.table), dev(self.off), self.total, dev(np.array(self.lens, dtype=np.int32)), q, out, st, ws)
        torch.cuda.synchronize()
        sdcp.sdcp_attend_kv(*args, scale=self.scale, window=self.window, stream=None if stream is None else stream.cuda_stream)
        torch.cuda.synchronize()
        return out, st.cpu().numpy()

    def check(self, out, status, bad=(), nan_rows=()):
        got = out.double().cpu().numpy()
        row = 0
        for b, (m, c) in enumerate(zip(self.ms, self.lens)):
            if b in bad:
                assert status[b] != 0 and (got[row:row + m + 1] == 0).all()
                row += m + 1
                continue
            assert status[b] == 0
            need = -(-(c + m + 1) // self.P)
            v = ref.block_values(self.pages[np.clip(self.table[b, :need], 0, self.n_pages - 1)], self.P, self.D)
            v = v.transpose(2, 1, 0, 3, 4).reshape(2, self.Hkv, -1, self.D)
            for i in range(m + 1):
                last = c + i
                first = max(0, last - self.window + 1) if self.window else 0
                for h in range(self.Hq):
                    if (row, h) in nan_rows:
                        assert np.isnan(got[row, h]).all()
                        continue
                    k = h // self.share
                    want, mass, a = ref.attend_row(self.q[row, h].astype(np.float64), v[0, k], v[1, k], np.float64(np.float32(self.scale)), first, last)
                    tol = 2.0**-8 * np.abs(want) + (2.0**-10 + 2.0**-18 * a) * mass + 2.0**-31 * np.abs(v[1, k][first:last + 1]).sum(axis=0)
                    assert (np.abs(got[row, h] - want) <= tol).all(), (b, i, h, np.abs(got[row, h] - want).max(), tol.min())
                row += 1


CASES = [dict(ms=[0], lens=[0], P=16, Hkv=1, share=1, D=64),
         dict(ms=[0, 0, 0], lens=[1, 127, 128], P=16, Hkv=2, share=4, D=128),
         dict(ms=[4, 0, 8], lens=[0, 300, 126], P=32, Hkv=2, share=8, D=128),
         dict(ms=[1, 16, 3], lens=[999, 15, 16], P=64, Hkv=1, share=7, D=64),
         dict(ms=[64], lens=[200], P=16, Hkv=1, share=5, D=128),
         dict(ms=[200, 0], lens=[0, 40], P=128, Hkv=1, share=2, D=64),
         dict(ms=[2], lens=[2500], P=1024, Hkv=3, share=1, D=128),
         dict(ms=[0], lens=[5000], P=64, Hkv=2, share=20, D=128),
         dict(ms=[i % 5 for i in range(40)], lens=[(i * 37) % 400 for i in range(40)], P=16, Hkv=2, share=4, D=64),
         dict(ms=[130], lens=[130], P=16, Hkv=1, share=1, D=128)]


@pytest.mark.parametrize("window", [0, 1, 5, 128, 200])
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_against_plain(ci, window):
    c = Case(seed=70 + ci, window=window, **CASES[ci])
    c.check(*c.run(gap=8 * (ci % 3)))


@pytest.mark.parametrize("q_scale,scale", [(0.0, None), (1.0, 0.0), (6.0, 0.5), (3.0, -0.3), (40.0, 1.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_flat_sharp_and_negative_scores(D, q_scale, scale):
    c = Case(ms=[3, 0], lens=[700, 64], P=32, Hkv=2, share=4, D=D, seed=5, q_scale=q_scale, scale=scale)
    c.check(*c.run())


@pytest.mark.parametrize("scale_bytes", [(8, 9), (8, 168), (160, 168)])
def test_scales_over_the_whole_range(scale_bytes):
    c = Case(ms=[3, 1], lens=[260, 64], P=16, Hkv=1, share=8, D=128, seed=6, scale_bytes=scale_bytes, scale=1e-3)
    c.check(*c.run())


def test_rising_scores_move_the_reference():
    """Later tokens score far above the earlier ones, tile after tile."""
    c = Case(ms=[2], lens=[1500], P=16, Hkv=1, share=4, D=64, seed=7, q_scale=0.01)
    per = 64 // 32
    for t in range(1503):
        blk = c.pages[c.table[0, t // 16], 0, 0]
        blk[16 * 32 + (t % 16) * per:16 * 32 + (t % 16) * per + per] = min(167, 90 + t // 22)
        for g in range(2):
            blk[(g * 16 + t % 16) * 16:(g * 16 + t % 16) * 16 + 16] = 0xFF  # n = 7 everywhere
    c.q[:] = ref.bf16(np.abs(c.q))
    c.check(*c.run())


def test_a_row_with_nan_or_infinities_keeps_to_itself():
    c = Case(ms=[3, 2], lens=[200, 77], P=16, Hkv=2, share=4, D=128, seed=8)
    c.q[1, 2, 5] = np.nan
    c.q[5, 7, 0] = np.inf
    c.q[5, 7, 1] = -np.inf
    c.q[5, 7, 2:] = np.nan
    c.check(*c.run(), nan_rows={(1, 2), (5, 7)})


def test_sessions_that_are_refused_are_zero():
    from speculative_decoding_verification_sdcp_gb300 import sdcp

    def case(change, bad, want, window=0):
        c = Case(ms=[2, 3, 1], lens=[5, 60, 0], P=16, Hkv=2, share=2, D=64, seed=9, window=window)
        change(c)
        out, st = c.run()
        c.check(out, st, bad)
        assert all(st[b] == want for b in bad)

    case(lambda c: c.lens.__setitem__(0, -1), (0,), sdcp.S_BAD_PARAMS)
    case(lambda c: c.table.__setitem__((1, 0), -1), (1,), sdcp.S_BAD_PARAMS)
    case(lambda c: c.table.__setitem__((1, 3), c.n_pages), (1,), sdcp.S_BAD_PARAMS)
    case(lambda c: c.lens.__setitem__(2, 16 * c.table.shape[1] - 1), (2,), sdcp.S_LIMIT)
    case(lambda c: c.lens.__setitem__(2, 2**31 - 1), (2,), sdcp.S_LIMIT)
    # a page that no row's window reaches may be gone
    case(lambda c: c.table.__setitem__((1, 0), -1), (), 0, window=20)


def test_offsets_out_of_order():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    c = Case(ms=[2, 2], lens=[40, 40], P=16, Hkv=1, share=2, D=64, seed=1)
    c.off = np.array([0, 9, 4], dtype=np.int32)
    out, st = c.run()
    assert st.tolist() == [sdcp.S_BAD_PARAMS] * 2 and (out == 0).all()


def test_another_stream_and_repeats_are_bit_equal():
    c = Case(ms=[4, 0, 7], lens=[900, 3000, 31], P=32, Hkv=2, share=4, D=128, seed=10)
    x, _ = c.run()
    y, st = c.run(stream=torch.cuda.Stream(), workspace_fill=0)
    assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    c.check(y, st)


def test_pages_past_2_32_bytes():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    c = Case(ms=[2], lens=[150], P=64, Hkv=8, share=1, D=128, seed=12)
    x, _ = c.run()
    n = (5 << 30) // int(sdcp.lib.sdcp_kv_page_bytes(64, 8, 128))
    big = torch.empty((n, 8, 2, 64 * 68), dtype=torch.uint8, device=DEV)
    big[n - c.n_pages:] = dev(c.pages)
    c.table[c.table >= 0] += n - c.n_pages
    c.n_pages = n
    y, st = c.run(pages=big)
    assert st.tolist() == [0] and torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ms,lens", [([23, 23], [300, 5]), ([23, 0, 22, 1, 11, 0, 40], [130, 900, 0, 257, 64, 1, 700])])
def test_items_of_unlike_widths_on_a_short_line(ms, lens, D):
    """Fewer tiles than there are thread blocks, some dearer than a block's share: blocks without any."""
    c = Case(ms=ms, lens=lens, P=16, Hkv=2, share=4, D=D, seed=21)
    c.check(*c.run())
