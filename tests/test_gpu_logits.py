"""sdcp_adjust_logits against the plain 64-bit implementation (tests/serving_reference.py).

Tolerance, from the arithmetic: each of the at most five binary32 steps of an entry rounds by 2^-24
of the largest magnitude it goes through, and the result is rounded once more to the row's type
(2^-9 of it for bfloat16, nothing for binary32).  What nothing applies to is equal bit for bit."""
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


class Batch:
    def __init__(self, V, ms, dtype, kind, seed, history=40, biases=0, masks=True, offset=0):
        from speculative_decoding_verification_sdcp_gb300 import sdcp
        r = np.random.default_rng(seed)
        self.V, self.ms, self.kind, self.dtype = V, ms, kind, dtype
        B = len(ms)
        self.off = np.concatenate([[0], np.cumsum(ms)]).astype(np.int32)
        self.total = int(self.off[-1])
        self.extra = 1 if kind == sdcp.ROWS_TARGET else 0
        self.n_rows = self.total + B * self.extra
        l = r.normal(0, 3, size=(self.n_rows, V)).astype(np.float32)
        if V > 8 and self.n_rows:
            l[0, :5] = [0.0, -0.0, np.inf, -np.inf, np.nan]
        self.logits = ref.bf16(l) if dtype == torch.bfloat16 else l
        self.draft = r.integers(0, max(1, min(V, 9)), self.total).astype(np.int32)
        self.history = r.integers(0, max(1, min(V, 30)), size=(B, max(1, history))).astype(np.int32)
        self.ctl = np.zeros(B, dtype=sdcp.CONTROLS_DTYPE)
        self.ctl["repetition"] = r.choice([1.0, 1.1, 1.7, 0.5], B)
        self.ctl["frequency"] = r.choice([0.0, 0.2, -0.6], B)
        self.ctl["presence"] = r.choice([0.0, 0.5, -0.25], B)
        self.ctl["history_len"] = r.integers(0, history + 1, B)
        self.ctl["prompt_len"] = [r.integers(0, h + 1) for h in self.ctl["history_len"]]
        toks, vals = [], []
        for b in range(B):
            k = int(r.integers(0, min(biases, V) + 1)) if biases else 0
            self.ctl["bias_offset"][b], self.ctl["bias_count"][b] = len(toks), k
            toks += sorted(r.choice(V, size=k, replace=False).tolist())
            vals += r.normal(0, 4, size=k).tolist()
        self.bias_tokens, self.bias_values = np.array(toks, dtype=np.int32), np.array(vals, dtype=np.float32)
        self.masks = self.mask_rows = None
        if masks and self.n_rows:
            self.masks = r.integers(0, 2**32, size=(3, (V + 31) // 32 + 1), dtype=np.uint32)
            self.masks[1] = 0  # leaves nothing
            self.mask_rows = r.integers(-1, 3, self.n_rows).astype(np.int32)
        self.offset = offset

    def device_logits(self):
        """The rows, at an address `offset` elements past an aligned one."""
        flat = torch.zeros(self.n_rows * self.V + self.offset, dtype=self.dtype, device=DEV)
        t = flat[self.offset:].view(self.n_rows, self.V)
        t.copy_(torch.from_numpy(self.logits).to(DEV))
        return t

    def run(self, in_place=False, out_offset=None, stream=None):
        from speculative_decoding_verification_sdcp_gb300 import sdcp
        dev = lambda x: None if x is None else torch.from_numpy(x).to(DEV)  # noqa: E731
        l = self.device_logits()
        out = l
        if not in_place:
            o = self.offset if out_offset is None else out_offset
            out = torch.full((self.n_rows * self.V + o,), 7.0, dtype=self.dtype, device=DEV)[o:].view(self.n_rows, self.V)
        status = torch.full((len(self.ms),), -9, dtype=torch.int32, device=DEV)
        masks = None if self.masks is None else dev(self.masks.view(np.int32))
        args = (dev(self.off), self.total, dev(self.draft), sdcp.controls_tensor(self.ctl, DEV), dev(self.history), status)
        kw = dict(rows=self.kind, bias_tokens=dev(self.bias_tokens) if self.bias_tokens.size else None,
                  bias_values=dev(self.bias_values) if self.bias_tokens.size else None, masks=masks, mask_rows=dev(self.mask_rows))
        torch.cuda.synchronize()
        sdcp.sdcp_adjust_logits(l, out, *args, stream=None if stream is None else stream.cuda_stream, **kw)
        torch.cuda.synchronize()
        return out, status.cpu().numpy()

    def check(self, out, status, bad=()):
        got = out.float().cpu().numpy()
        raw = self.logits
        row = 0
        for b, m in enumerate(self.ms):
            c = self.ctl[b]
            h = self.history[b]
            for i in range(m + self.extra):
                if b in bad:
                    assert np.isnan(got[row]).all()
                else:
                    k0, k1 = int(c["bias_offset"]), int(c["bias_offset"] + c["bias_count"])
                    mr = -1 if self.mask_rows is None else int(self.mask_rows[row])
                    want, most, applied = ref.adjust_row(
                        raw[row], h[:c["prompt_len"]], h[c["prompt_len"]:c["history_len"]], self.draft[self.off[b]:self.off[b] + i],
                        (c["repetition"], c["frequency"], c["presence"]), zip(self.bias_tokens[k0:k1], self.bias_values[k0:k1]),
                        None if mr < 0 else self.masks[mr])
                    assert np.array_equal(got[row][~applied], raw[row][~applied], equal_nan=True)
                    assert np.array_equal(np.isnan(got[row]), np.isnan(want))
                    fine = np.isfinite(want)
                    assert np.array_equal(got[row][~fine], want[~fine].astype(np.float32), equal_nan=True)
                    tol = 5 * 2.0**-24 * most[fine] + (2.0**-8 if self.dtype == torch.bfloat16 else 2.0**-24) * np.abs(want[fine]) + 1e-38
                    assert (np.abs(got[row][fine] - want[fine]) <= tol).all()
                row += 1
        for b in range(len(self.ms)):
            assert (status[b] == 0) == (b not in bad)


CASES = [dict(V=1, ms=[0, 2], masks=True), dict(V=3, ms=[1, 0, 4]), dict(V=31, ms=[3]), dict(V=1000, ms=[4, 4, 4, 4], biases=5),
         dict(V=1001, ms=[2, 0, 7], biases=300, history=200), dict(V=4096, ms=[1, 3], biases=1), dict(V=4097, ms=[64], history=3),
         dict(V=9001, ms=[1, 16, 2], masks=False), dict(V=50257, ms=[2], history=700), dict(V=257, ms=[0, 0, 0], history=0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_against_plain(ci, kind, dtype):
    b = Batch(dtype=dtype, kind=kind, seed=100 + ci, **CASES[ci])
    b.check(*b.run())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset,out_offset", [(1, 1), (3, 3), (1, 0), (0, 2)])
def test_addresses_off_a_boundary(offset, out_offset, dtype):
    b = Batch(V=777, ms=[3, 5], dtype=dtype, kind=0, seed=5, biases=4, offset=offset)
    b.check(*b.run(out_offset=out_offset))


@pytest.mark.parametrize("V", [64, 1001, 8192])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place_equals_out_of_place(V, dtype):
    b = Batch(V=V, ms=[3, 0, 6], dtype=dtype, kind=0, seed=V, biases=3)
    x, _ = b.run()
    y, st = b.run(in_place=True)
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    assert torch.equal(x.view(bits), y.view(bits))
    b.check(y, st)


def test_ids_out_of_the_vocabulary_count_for_nothing():
    b = Batch(V=100, ms=[3, 3], dtype=torch.float32, kind=0, seed=8)
    b.history[:, ::3] = -1
    b.history[:, 1::3] = 100
    b.history[0, 2] = 2**31 - 1
    b.history[1, 2] = -2**31
    b.draft[1] = -7
    b.draft[4] = 5000
    b.check(*b.run())


def test_sessions_that_are_refused():
    from speculative_decoding_verification_sdcp_gb300 import sdcp

    def case(change, bad, want):
        b = Batch(V=300, ms=[2, 3, 1], dtype=torch.bfloat16, kind=0, seed=3, biases=6)
        b.ctl["bias_count"] = 2
        b.ctl["bias_offset"] = [0, 2, 4]
        b.bias_tokens = np.array([1, 7, 3, 299, 0, 5], dtype=np.int32)
        b.bias_values = np.arange(6, dtype=np.float32)
        change(b)
        out, st = b.run()
        b.check(out, st, bad)
        assert all(st[k] == want for k in bad)

    P = sdcp.S_BAD_PARAMS
    for v in (0.0, -1.0, np.inf, np.nan):
        case(lambda b: b.ctl["repetition"].__setitem__(1, v), (1,), P)
    case(lambda b: b.ctl["frequency"].__setitem__(0, np.nan), (0,), P)
    case(lambda b: b.ctl["presence"].__setitem__(2, np.inf), (2,), P)
    case(lambda b: b.ctl["history_len"].__setitem__(1, 41), (1,), P)
    case(lambda b: b.ctl["prompt_len"].__setitem__(1, b.ctl["history_len"][1] + 1), (1,), P)
    case(lambda b: b.ctl["bias_offset"].__setitem__(2, 5), (2,), P)
    case(lambda b: b.ctl["bias_offset"].__setitem__(2, 2**32 - 1), (2,), P)
    case(lambda b: b.bias_tokens.__setitem__(slice(0, 2), [7, 7]), (0,), P)
    case(lambda b: b.bias_tokens.__setitem__(3, 300), (1,), P)
    case(lambda b: b.bias_tokens.__setitem__(4, -1), (2,), P)
    case(lambda b: b.mask_rows.__setitem__(4, 3), (1,), P)
    case(lambda b: b.mask_rows.__setitem__(0, -2), (0,), P)


def test_too_many_drafts():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    b = Batch(V=50, ms=[2, 65, 64], dtype=torch.float32, kind=0, seed=4)
    out, st = b.run()
    b.check(out, st, (1,))
    assert st[1] == sdcp.S_LIMIT


def test_a_refused_session_commits_nothing_and_a_masked_row_is_seen():
    """The adjusted rows go into a verify call: NaN rows and rows without a token are BAD_PARAMS."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    b = Batch(V=300, ms=[2, 2, 2], dtype=torch.float32, kind=0, seed=6)
    b.logits[0, :5] = 0.5
    b.mask_rows[:] = -1
    b.mask_rows[4] = 1           # session 1, leaves nothing
    b.ctl["repetition"][2] = 0.0  # refused
    out, st = b.run()
    ver = sdcp.Verifier(300, 3, b.total, DEV)
    prm = np.zeros(3, dtype=sdcp.PARAMS_DTYPE)
    prm["rule_id"], prm["temperature_milli"], prm["top_p_milli"] = 1, 1000, 1000
    got = ver(out, None, torch.from_numpy(b.off).to(DEV), torch.from_numpy(b.draft).to(DEV), sdcp.params_tensor(prm, DEV))
    assert got[3].cpu().tolist() == [0, sdcp.S_BAD_PARAMS, sdcp.S_BAD_PARAMS]


def test_offsets_out_of_order_write_nothing():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    b = Batch(V=64, ms=[2, 2], dtype=torch.float32, kind=0, seed=6, masks=False)
    b.off = np.array([0, 9, 4], dtype=np.int32)
    out, st = b.run()
    assert st.tolist() == [sdcp.S_BAD_PARAMS] * 2
    assert (out == 7.0).all()


def test_another_stream_and_repeats_are_bit_equal():
    b = Batch(V=5000, ms=[8] * 6, dtype=torch.bfloat16, kind=0, seed=11, biases=20, history=900)
    x, _ = b.run()
    y, st = b.run(stream=torch.cuda.Stream())
    assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    b.check(y, st)


def test_rows_past_2_31_elements():
    """A batch whose last rows start beyond 2^31 elements."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    V, B = 1 << 22, 520
    logits = torch.zeros((B, V), dtype=torch.bfloat16, device=DEV)
    ctl = np.zeros(B, dtype=sdcp.CONTROLS_DTYPE)
    ctl["repetition"], ctl["frequency"], ctl["history_len"] = 1.0, 2.0, 2
    history = torch.tensor([[V - 1, V - 1]] * B, dtype=torch.int32, device=DEV)
    status = torch.empty(B, dtype=torch.int32, device=DEV)
    off = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    sdcp.sdcp_adjust_logits(logits, logits, off, 0, None, sdcp.controls_tensor(ctl, DEV), history, status)
    torch.cuda.synchronize()
    assert (status == 0).all()
    assert (logits[:, V - 1] == -4).all() and float(logits[:, :V - 1].abs().amax()) == 0.0
