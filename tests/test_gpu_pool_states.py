"""The calls on pages where a pool was filled by hand, where a row is very long, and where pages run out."""
import numpy as np
import numpy as np
import pytest
import torch

from test_gpu_pool import DEV, SIZES, Both, _built, ints  # noqa: F401  (_built: a fixture, the library is built)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entries", [2**24, 2**24 + 1])
def test_a_long_row_without_a_usable_entry_is_refused(entries):
    """However many entries are outside the pool, the slot is left as it was; another gets its page."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    pool = sdcp.KvPool(10, 16, 2, entries, DEV)
    pool.held[0] = entries
    copies, n, st = torch.full((2, 4), -7, dtype=torch.int32, device=DEV), ints([-9]), ints([-9, -9])
    sdcp.sdcp_reserve_kv(pool, ints([0, 0]), ints([entries * 16, 16]), copies, n, st, sdcp.alloc_pool_workspace(pool).fill_(255))
    assert st.tolist() == [sdcp.S_BAD_PARAMS, sdcp.S_OK] and n.tolist() == [0]
    assert pool.held.tolist() == [entries, 1] and pool.refs.tolist() == [1] + [0] * 9
    assert bool((pool.page_table[0] == -1).all()) and pool.page_table[1, 0].item() == 0 and bool((pool.page_table[1, 1:] == -1).all())


@pytest.mark.parametrize("n_pages", [40, 9000])
def test_an_entry_that_names_a_free_page_stays(n_pages):
    """Compaction renumbers pages that it moves, and no other entry."""
    x = Both(n_pages, 16, 4, 12)
    x.reserve([0] * 4, [16 * 12, 16 * 8, 16 * 12, 16])
    x.release([16, -1, 0, -1])  # holes before the second slot's pages
    x.plain.held[2] = 4
    x.plain.table[2][:4] = [n_pages - 1, 30, 2, n_pages + 5]  # free ones past the live pages and before, one outside the pool
    x.load()
    assert x.compact(20)[0] == 10
    assert x.plain.table[2][:4] == [n_pages - 1, 30, 2, n_pages + 5]


@pytest.mark.parametrize("n_pages,P,slots,max_pages", [s for s in SIZES if s[2] * s[3] > s[0]])
def test_pages_run_out_at_every_size(n_pages, P, slots, max_pages):
    """Slots grow until too few pages are free, forks among them; what is given back is taken again."""
    r = np.random.default_rng(slots)
    x, most, lens = Both(n_pages, P, slots, max_pages), max_pages * P, [0] * slots
    out = 0
    for _ in range(12):
        upto = [min(n + int(r.integers(0, most // 2 + 1)), most) for n in lens]
        st = x.reserve(lens, upto)[0]
        assert set(st) <= {0, 2}  # (every row has an entry for upto: a refusal is for want of pages)
        out += 2 in st
        lens = [u if s == 0 else n for n, u, s in zip(lens, upto, st)]
        if out:
            break
    assert out and 0 in st
    ended = [b % 3 == 0 for b in range(slots)]
    x.release([0 if e else -1 for e in ended])
    parent = [-1 if not e else b + 1 if b + 1 < slots and lens[b + 1] else -1 for b, e in enumerate(ended)]
    assert set(x.fork(parent, [lens[p] if p >= 0 else 0 for p in parent])) == {0}
    lens = [(lens[p] if p >= 0 else 0) if e else n for n, p, e in zip(lens, parent, ended)]
    st = x.reserve(lens, [min(n + int(r.integers(0, 3 * P)), most) for n in lens])[0]
    assert 0 in st
