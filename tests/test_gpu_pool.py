"""The calls on a cache's pages against tests/pool_reference.py: whole numbers and bytes, equal."""
import numpy as np
import pytest
import torch

import pool_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Both:
    """A pool on the GPU and its plain twin; each call is made on both and everything is compared."""

    def __init__(self, n_pages, P, slots, max_pages, stream=None):
        from speculative_decoding_verification_sdcp_gb300 import sdcp
        self.m, self.stream = sdcp, stream
        self.plain = ref.Pool(n_pages, P, slots, max_pages)
        self.pool = sdcp.KvPool(n_pages, P, slots, max_pages, DEV)
        self.ws = sdcp.alloc_pool_workspace(self.pool).fill_(255)
        self.slots = slots

    def load(self):
        """The plain twin's state into the GPU's."""
        self.pool.page_table.copy_(ints(self.plain.table).view(self.pool.page_table.shape))
        self.pool.held.copy_(ints(self.plain.held))
        self.pool.refs.copy_(ints(self.plain.refs))

    def same(self, status, want):
        torch.cuda.synchronize()
        assert status.tolist() == want
        assert self.pool.held.tolist() == self.plain.held
        assert self.pool.refs.tolist() == self.plain.refs
        assert self.pool.page_table.tolist() == self.plain.table

    def _handle(self):
        torch.cuda.synchronize()
        return None if self.stream is None else self.stream.cuda_stream

    def fork(self, parent, length):
        st = ints([-9] * self.slots)
        self.m.sdcp_fork_kv(self.pool, ints(parent), ints(length), st, stream=self._handle())
        want = self.plain.fork(parent, length)
        self.same(st, want)
        return want

    def _list(self, most):
        return torch.full((most, 4), -7, dtype=torch.int32, device=DEV), ints([-9])

    def reserve(self, kv_len, upto):
        st, (copies, n) = ints([-9] * self.slots), self._list(self.slots)
        self.m.sdcp_reserve_kv(self.pool, ints(kv_len), ints(upto), copies, n, st, self.ws, stream=self._handle())
        want, listed = self.plain.reserve(kv_len, upto)
        self.same(st, want)
        assert n.tolist() == [len(listed)]
        assert copies.tolist() == [list(c) for c in listed] + [[-7] * 4] * (self.slots - len(listed))
        return want, copies, n

    def release(self, keep):
        st = ints([-9] * self.slots)
        self.m.sdcp_release_kv(self.pool, ints(keep), st, stream=self._handle())
        want = self.plain.release(keep)
        self.same(st, want)
        return want

    def compact(self, most):
        (copies, n), live = self._list(most), ints([-9])
        self.m.sdcp_compact_kv(self.pool, copies, n, live, self.ws, stream=self._handle())
        want, listed = self.plain.compact(most)
        self.same(ints([]), [])
        assert live.tolist() == [want] and n.tolist() == [len(listed)]
        assert copies.tolist() == [list(c) for c in listed] + [[-7] * 4] * (most - len(listed))
        return want, copies, n


# slots below, at and past a block's and a cluster's threads; rows longer than a thread's and a block's step
SIZES = [(40, 16, 3, 12), (300, 32, 40, 20), (5000, 16, 9, 2100), (20000, 64, 1500, 30), (1, 16, 1, 1), (70000, 16, 9000, 12)]


@pytest.mark.parametrize("n_pages,P,slots,max_pages", SIZES)
def test_a_life_of_a_pool(n_pages, P, slots, max_pages):
    r = np.random.default_rng(n_pages)
    x = Both(n_pages, P, slots, max_pages, stream=torch.cuda.Stream() if slots == 40 else None)
    lens = [0] * slots
    seen = set()
    most = max_pages * P
    for step in range(8):
        # rounds of any length on some slots, prompts among them
        grow = [0 if r.random() < 0.4 else int(r.integers(1, max(2, most // (2 if r.random() < 0.15 else 12)))) for _ in range(slots)]
        upto = [min(n + g, most + 1) for n, g in zip(lens, grow)]
        st, _, _ = x.reserve(lens, upto)
        seen |= set(st)
        lens = [u if s == 0 and u > n else n for n, u, s in zip(lens, upto, st)]
        # forks of some into empty ones, at any length (of too long a one and of a child too)
        empty = [b for b in range(slots) if x.plain.held[b] == 0]
        full = [b for b in range(slots) if x.plain.held[b]]
        parent, length = [-1] * slots, [0] * slots
        for b in empty:
            if full and r.random() < 0.7:
                parent[b] = int(r.choice(full if r.random() < 0.95 else range(slots)))
                length[b] = int(r.integers(0, lens[parent[b]] + 1)) if r.random() < 0.95 else most + 5
        st = x.fork(parent, length)
        lens = [length[b] if parent[b] >= 0 and s == 0 else lens[b] for b, s in enumerate(st)]
        # the verdicts: some keep all, some a part, some end
        keep = [-1 if r.random() < 0.4 else 0 if r.random() < 0.3 else int(r.integers(0, lens[b] + 1)) for b in range(slots)]
        x.release(keep)
        lens = [n if k < 0 else min(n, k) for n, k in zip(lens, keep)]
        if step % 3 == 2:
            x.compact(int(r.integers(0, n_pages // 2 + 1)) if step == 2 else n_pages // 2 + 1)
    assert n_pages < 300 or seen >= {0}


def test_free_pages_run_out_in_the_order_of_the_slots():
    x = Both(10, 16, 6, 8)
    st, _, _ = x.reserve([0] * 6, [3 * 16, 4 * 16, 0, 4 * 16, 16, 16])  # 3 + 4 of 10, the next is counted too
    assert st == [0, 0, 0, 2, 2, 2]
    st, _, _ = x.reserve([48, 64, 0, 0, 0, 0], [48, 64, 48, 0, 0, 0])
    assert st == [0] * 6 and sorted(x.plain.refs) == [1] * 10


def test_shared_pages_are_replaced_and_their_tokens_listed():
    x = Both(64, 16, 8, 8)
    x.reserve([0] * 8, [50] + [0] * 7)                 # pages of 50 tokens
    x.fork([-1, 0, 0, 0] + [-1] * 4, [0, 50, 48, 20] + [0] * 4)
    st, copies, n = x.reserve([50, 50, 48, 20, 0, 0, 0, 0], [55, 70, 49, 60, 0, 0, 0, 0])
    # slots 0 and 1 share the fourth page (2 tokens of it), slot 3 the second (4 tokens); slot 2 is at a page's start
    assert [c[2] for c in copies.tolist()[:n.item()]] == [2, 2, 4]
    # a rollback into shared pages: those at and past it are replaced, the ones before stay shared
    st, copies, n = x.reserve([17, -1, 0, 0, 0, 0, 0, 0], [64, -1, 0, 0, 0, 0, 0, 0])
    assert n.tolist() == [1] and copies[0, 2].item() == 1


def test_long_rows_in_shared_pages():
    """More shared entries than a thread does alone, and than a block does at once."""
    x = Both(9000, 16, 5, 3000)
    x.reserve([0] * 5, [2500 * 16, 9, 300 * 16, 0, 0])
    x.fork([-1, -1, -1, 0, 2], [0, 0, 0, 2400 * 16 + 3, 299 * 16])
    x.reserve([35, 0, 100 * 16, 2400 * 16, 0], [2600 * 16, 0, 301 * 16, 2999 * 16, 17])
    x.release([0, 0, -1, 1, 0])


def test_what_is_refused_is_left_as_it_was():
    x = Both(30, 16, 6, 4)
    x.reserve([0] * 6, [40, 16, 0, 0, 0, 0])
    big = 2**31 - 1
    assert x.fork([-1, -1, 9, 2, -2, 3], [0, 0, 5, 5, 5, 5]) == [0, 0, 3, 3, 3, 3]
    assert x.fork([-1, 0, 0, 0, 1, 5], [0, 3, 49, -1, 17, 1]) == [0, 3, 2, 3, 3, 3]  # (4: its parent is named to be forked too)
    assert x.reserve([49, -1, 1, big, 0, 0], [50, 5, 9, big, 65, big])[0] == [3, 3, 3, 0, 2, 2]
    # rows that are not in order
    x.plain.held[1], x.plain.held[3] = -3, 5
    x.plain.table[0][1] = 30
    x.load()
    assert x.fork([-1, -1, 0, -1, 1, 3], [0, 0, 32, 0, 1, 1]) == [0, 0, 3, 0, 3, 3]
    assert x.fork([-1, -1, 0, -1, -1, -1], [0, 0, 16, 0, 0, 0]) == [0] * 6
    assert x.release([0, 0, -1, 0, big, 0]) == [3, 3, 0, 3, 0, 0]
    assert x.reserve([16, 0, 0, 0, 0, 0], [48, 5, 0, 5, 0, 0])[0] == [3, 3, 0, 3, 0, 0]
    x.plain.table[0][1] = -1
    x.load()
    assert x.release([16, -1, -1, -1, -1, -1])[0] == 3


def test_reserve_without_slots_or_needs():
    x = Both(30, 16, 4, 4)
    x.reserve([0] * 4, [0, -5, 0, 0])
    x = Both(30, 16, 0, 4)
    x.reserve([], [])
    x.compact(3)


@pytest.mark.parametrize("D,P,heads", [(128, 64, 8), (64, 16, 1), (64, 128, 3), (128, 16, 2), (128, 1024, 1)])
def test_copies(D, P, heads):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    r = np.random.default_rng(P + D)
    n = 40
    cache = sdcp.KvCache(n, P, heads, D, DEV, pages=torch.from_numpy(r.integers(0, 256, size=(n, heads, 2, P * (D // 2 + D // 32)), dtype=np.uint8)).to(DEV))
    order = r.permutation(n).tolist()
    copies = [(order[i], order[20 + i], int(t), 77) for i, t in enumerate([P, 0, 1, P - 1, P // 2, 3, 7, 8, 9, 15] + r.integers(0, P + 1, 8).tolist())]
    want = cache.pages.cpu().numpy().copy()
    listed, count, st = torch.full((25, 4), 3, dtype=torch.int32, device=DEV), ints([len(copies)]), ints([-9])
    listed[:len(copies)] = ints(copies)
    sdcp.sdcp_copy_pages(cache, listed, count, st)
    assert ref.copy_pages(want, copies, P, D)
    assert st.tolist() == [0] and np.array_equal(cache.pages.cpu().numpy(), want)
    # records that are not usable are left out, the others are done
    bad = [(-1, 2, 3, 0), (0, n, 3, 0), (n, 0, 3, 0), (5, 5, 1, 0), (2, 3, P + 1, 0), (2, 3, -1, 0), (order[0], order[21], P, 0)]
    listed[:len(bad)] = ints(bad)
    count.fill_(len(bad))
    sdcp.sdcp_copy_pages(cache, listed, count, st)
    assert not ref.copy_pages(want, bad, P, D)
    assert st.tolist() == [3] and np.array_equal(cache.pages.cpu().numpy(), want)
    for wrong in (-1, 26):
        count.fill_(wrong)
        sdcp.sdcp_copy_pages(cache, listed, count, st)
        assert st.tolist() == [3] and np.array_equal(cache.pages.cpu().numpy(), want)
    count.fill_(0)
    sdcp.sdcp_copy_pages(cache, listed, count, st)
    assert st.tolist() == [0] and np.array_equal(cache.pages.cpu().numpy(), want)


def test_copies_past_2_32_bytes():
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    n = (5 << 30) // int(sdcp.lib.sdcp_kv_page_bytes(64, 8, 128))
    cache = sdcp.KvCache(n, 64, 8, 128, DEV, pages=torch.zeros((n, 8, 2, 64 * 68), dtype=torch.uint8, device=DEV))
    cache.pages[n - 1].random_(0, 256)
    cache.pages[2].random_(0, 256)
    st = ints([-9])
    sdcp.sdcp_copy_pages(cache, ints([(n - 1, 5, 64, 0), (2, n - 2, 64, 0)]), ints([2]), st)
    assert st.tolist() == [0] and torch.equal(cache.pages[5], cache.pages[n - 1]) and torch.equal(cache.pages[n - 2], cache.pages[2])


def test_a_captured_branch_and_release():
    """Fork, reserve, copy and release in one graph: replayed, it finds the state that it left."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    x = Both(200, 16, 12, 10)
    x.reserve([0] * 12, [70, 33, 120] + [0] * 9)
    cache = sdcp.KvCache(200, 16, 2, 64, DEV)
    cache.pages.random_(0, 256)
    parent, length = ints([-1] * 3 + [0, 0, 1, 2, 2, 2, -1, -1, -1]), ints([0] * 3 + [70, 60, 33, 120, 96, 1, 0, 0, 0])
    upto = length + ints([0] * 3 + [9] * 6 + [0] * 3)
    keep = ints([-1] * 3 + [0] * 9)
    copies, n, sts = torch.full((12, 4), -1, dtype=torch.int32, device=DEV), ints([0]), [ints([-9] * 12) for _ in range(3)] + [ints([-9])]

    def calls():
        sdcp.sdcp_fork_kv(x.pool, parent, length, sts[0])
        sdcp.sdcp_reserve_kv(x.pool, length, upto, copies, n, sts[1], x.ws)
        sdcp.sdcp_copy_pages(cache, copies, n, sts[3])
        sdcp.sdcp_release_kv(x.pool, keep, sts[2])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    x.plain.fork(parent.tolist(), length.tolist())
    x.plain.reserve(length.tolist(), upto.tolist())
    x.plain.release(keep.tolist())
    x.same(sts[2], [0] * 12)
    first = copies.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        graph.replay()
    x.same(sts[2], [0] * 12)
    assert torch.equal(copies, first) and n.item() == 5 and all(set(s.tolist()) == {0} for s in sts)


def test_a_captured_compaction():
    """Compact and copy in one graph, replayed on two fillings of the pool and on a compact one."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    x = Both(200, 16, 12, 10)
    cache = sdcp.KvCache(200, 16, 2, 64, DEV)
    (copies, n), live, st = x._list(101), ints([-9]), ints([-9])

    def calls():
        sdcp.sdcp_compact_kv(x.pool, copies, n, live, x.ws)
        sdcp.sdcp_copy_pages(cache, copies, n, st)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    r = np.random.default_rng(4)
    for _ in range(2):
        x.reserve([0] * 12, r.integers(0, 160, 12).tolist())
        x.release([int(k) for k in r.integers(-40, 60, 12)])
        x.reserve([16 * h for h in x.plain.held], [16 * h + int(k) for h, k in zip(x.plain.held, r.integers(0, 50, 12))])
        cache.pages.random_(0, 256)
        for again in range(2):
            rows = [[cache.pages[p].clone() for p in x.plain.table[b][:x.plain.held[b]]] for b in range(12)]
            want, listed = x.plain.compact(101)
            graph.replay()
            x.same(ints([]), [])
            assert live.tolist() == [want] and n.tolist() == [len(listed)] and st.tolist() == [0] and (len(listed) == 0 or not again)
            for b in range(12):  # every row still finds its bytes
                assert all(torch.equal(cache.pages[p], y) for p, y in zip(x.plain.table[b], rows[b]))
        x.release([0] * 12)
