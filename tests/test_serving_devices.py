"""The serving calls' binding refuses tensors that are not on the call's CUDA device, before the library
sees their addresses (no GPU work: the library's functions are stood in for)."""
import pytest
import torch


@pytest.fixture()
def sdcp(monkeypatch):
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()
    from speculative_decoding_verification_sdcp_gb300 import sdcp as m

    def reached(*a):
        raise AssertionError("the library was called")

    for name in ("sdcp_adjust_logits", "sdcp_append_kv", "sdcp_read_kv", "sdcp_attend_kv"):
        monkeypatch.setattr(m.lib, name, reached)
    monkeypatch.setattr(m, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return m


class On(torch.Tensor):
    """A tensor in host memory that says it is on a CUDA device."""
    index = 0
    is_cuda = property(lambda s: True)
    device = property(lambda s: torch.device("cuda", s.index))

    def get_device(self):
        return self.index


def on(t, index=0):
    t = t.as_subclass(On)
    t.index = index
    return t


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def make(m, call):
    """(function, positional tensors by name, keywords) of a call that is right but for its devices."""
    page, vec = torch.zeros((2, 1, 2, 16 * 34), dtype=torch.uint8), torch.zeros((3, 1, 64))
    t = dict(table=ints(2, 1), off=ints(3), lens=ints(2), status=ints(2), pages=page)
    if call == "adjust":
        t = dict(off=ints(3), status=ints(2), logits=torch.zeros((3, 64)), out=torch.zeros((3, 64)), draft=ints(1), history=ints(2, 4),
                 controls=torch.zeros(64, dtype=torch.uint8), bias_tokens=ints(2), bias_values=torch.zeros(2), masks=ints(1, 2), mask_rows=ints(3))
        return t, lambda t: m.sdcp_adjust_logits(t["logits"], t["out"], t["off"], 1, t["draft"], t["controls"], t["history"], t["status"],
                                                 bias_tokens=t["bias_tokens"], bias_values=t["bias_values"], masks=t["masks"], mask_rows=t["mask_rows"])
    cache = lambda t: m.KvCache(2, 16, 1, 64, None, pages=t["pages"])  # noqa: E731
    if call == "append":
        t.update(k=vec.clone(), v=vec.clone(), q=vec.clone(), q_out=vec.clone(), rope=torch.zeros((16, 64)))
        return t, lambda t: m.sdcp_append_kv(cache(t), t["table"], t["off"], 1, t["lens"], t["k"], t["v"], t["status"],
                                             rotary=m.Rotary(t["rope"]), q=t["q"], q_out=t["q_out"])
    if call == "read":
        t.update(k=vec.clone(), v=vec.clone())
        return t, lambda t: m.sdcp_read_kv(cache(t), t["table"], t["off"], 3, t["lens"], t["k"], t["v"], t["status"])
    t.update(q=vec.bfloat16(), out=vec.bfloat16(), ws=torch.zeros(1 << 10, dtype=torch.uint8))
    return t, lambda t: m.sdcp_attend_kv(cache(t), t["table"], t["off"], 1, t["lens"], t["q"], t["out"], t["status"], t["ws"])


@pytest.mark.parametrize("call", ["adjust", "append", "read", "attend"])
def test_every_tensor_is_looked_at(sdcp, call):
    t, run = make(sdcp, call)
    good = {k: on(v) for k, v in t.items()}
    with pytest.raises(AssertionError, match="library was called"):
        run(good)
    for k in t:
        for other in (t[k], on(t[k], 1)):
            with pytest.raises(ValueError, match="device"):
                run({**good, k: other})
    with pytest.raises(ValueError, match="device"):
        run(t)
