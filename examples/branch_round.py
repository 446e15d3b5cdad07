"""Sessions that try several continuations: pages shared by forks, attended once, given back by the losers.

    python examples/branch_round.py [--sessions 4] [--branches 3] [--rounds 6] [--drafts 4]

The toy model of examples/verify_round.py.  Each session has a prompt, and `branches` continuations of it run
side by side, each with its own drafts and its own random values:

  1. sdcp_fork_kv gives each continuation the pages of its session's prompt; no byte is copied;
  2. each round, sdcp_reserve_kv takes pages for the positions that the round writes, in the place of shared
     ones too, and sdcp_copy_pages moves the tokens that these hold already; a continuation that gets none is
     kept out of the round;
  3. sdcp_append_kv writes the round, and sdcp_attend_shared_kv attends it, a session's continuations as one
     group: the prompt's pages are read once for them;
  4. after the verdict, sdcp_release_kv takes back what a rejection left over;
  5. at the end a continuation is chosen, sdcp_release_kv frees the others, and sdcp_compact_kv with
     sdcp_copy_pages moves what is left to the front of the pool.
"""
from __future__ import annotations

import argparse

import numpy as np
import torch

import verify_round
from verify_round import Model, rotary_table, sdcp


class Branches(verify_round.Rounds):
    """The continuations of a batch of prompts; slot s * branches + k is continuation k of prompt s."""

    def __init__(self, model: Model, prompts, branches, pool_pages, max_tokens=512, page_tokens=16):
        dev = self.device = model.device
        self.branches, slots = branches, len(prompts) * branches
        super().__init__(model, [p[:1] for p in prompts for _ in range(branches)], max_tokens=page_tokens, page_tokens=page_tokens)
        self.history, self.prompt_len = [list(p) for p in prompts for _ in range(branches)], [len(p) for p in prompts for _ in range(branches)]
        self.cparams = self.cparams.clone()
        self.cparams.view(self.B, 48)[:, :4] = torch.tensor([max_tokens], dtype=torch.int32).view(torch.uint8).to(dev)  # max_new
        self.rotary = sdcp.Rotary(rotary_table(max_tokens, model.head_dim, dev))
        self.cache = sdcp.KvCache(pool_pages, page_tokens, model.kv_heads, model.head_dim, dev)
        self.pool = sdcp.KvPool(pool_pages, page_tokens, slots, -(-max_tokens // page_tokens), dev)
        self.scratch = sdcp.alloc_pool_workspace(self.pool)
        self.copies = torch.empty((max(slots, pool_pages // 2 + 1), 4), dtype=torch.int32, device=dev)
        self.n_copies, self.copied, self.n_live = self._int([0]), self._int([0]), self._int([0])
        self.groups = self._int(list(range(0, slots + 1, branches)))
        # the prompts but their last tokens, by each session's first slot; the others fork it
        self.kv_len = [0] * slots
        rows = [p[:-1] if s % branches == 0 else [] for s, p in enumerate(self.history)]
        if any(rows):  # (nothing, of prompts of one token)
            status = self.score(rows, grouped=False)[3]
            self._checked(status, "the prompts")
        self.kv_len = [len(p) - 1 for p in self.history]
        forked = self._int([0] * slots)
        sdcp.sdcp_fork_kv(self.pool, self._int([-1 if s % branches == 0 else s - s % branches for s in range(slots)]), self._int(self.kv_len), forked)
        self._checked(forked, "the forks")

    def _checked(self, status, what):
        bad = {s: st for s, st in enumerate(status.tolist()) if st}
        if bad:
            raise ValueError("%s were refused: %s" % (what, bad))

    def score(self, rows, sessions=None, grouped=True):
        """As Rounds.score, with pages taken from the pool on the way; slots without rows are left out."""
        m, dev = self.model, self.device
        slots = [s for s, r in enumerate(rows) if r]
        reserved = self._int([0] * len(rows))
        sdcp.sdcp_reserve_kv(self.pool, self._int(self.kv_len), self._int([n + len(r) for n, r in zip(self.kv_len, rows)]), self.copies, self.n_copies,
                             reserved, self.scratch)
        sdcp.sdcp_copy_pages(self.cache, self.copies, self.n_copies, self.copied)  # (of each layer's cache)
        rows = [rows[s] for s in slots]
        n, off, total = len(rows), self._int(np.concatenate([[0], np.cumsum([len(r) - 1 for r in rows])]).tolist()), sum(len(r) - 1 for r in rows)
        # a slot that got no pages may hold shared ones where it would write: -1 keeps it out of the calls below
        table, reserved = self.pool.page_table[slots], reserved[slots]
        kv_len = torch.where(reserved == sdcp.S_OK, self._int([self.kv_len[s] for s in slots]), -1)
        x = m.embed[torch.tensor([t for r in rows for t in r], device=dev)]
        q, k, v = m.qkv(x)
        turned, out = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(q, memory_format=torch.contiguous_format)
        appended, attended = self._int([0] * n), self._int([0] * n)
        sdcp.sdcp_append_kv(self.cache, table, off, total, kv_len, k, v, appended, rotary=self.rotary, q=q, q_out=turned)
        groups = self.groups if grouped else self._int(list(range(n + 1)))
        scratch = sdcp.alloc_attend_shared_workspace(n, total, groups.numel() - 1, m.q_heads, m.kv_heads, m.head_dim, dev)
        sdcp.sdcp_attend_shared_kv(self.cache, table, off, total, kv_len, groups, turned, out, attended, scratch)
        return m.logits(x, out), off, total, torch.stack([reserved, appended, attended, self.copied.expand(n)]).amax(0)

    def release(self, keep):
        """Slots keep the pages of their first keep[s] tokens (-1: all)."""
        status = self._int([0] * self.B)
        sdcp.sdcp_release_kv(self.pool, self._int(keep), status)
        self._checked(status, "releases")

    def round(self, drafts, number):
        emitted = super().round(drafts, number)
        self.release(self.kv_len)
        return emitted

    def keep(self, chosen):
        """One continuation of each session stays; the pool is compacted.  The number of live pages."""
        self.release([-1 if s % self.branches == chosen[s // self.branches] else 0 for s in range(self.B)])
        sdcp.sdcp_compact_kv(self.pool, self.copies, self.n_copies, self.n_live, self.scratch)
        sdcp.sdcp_copy_pages(self.cache, self.copies, self.n_copies, self.copied)
        self._checked(self.copied, "copies")
        return int(self.n_live)

    def cached(self, slot):
        """The keys and values of a slot's cached tokens."""
        n = self.kv_len[slot]
        k = torch.empty((n, self.model.kv_heads, self.model.head_dim), dtype=torch.bfloat16, device=self.device)
        v, status = torch.empty_like(k), self._int([0])
        sdcp.sdcp_read_kv(self.cache, self.pool.page_table[slot:slot + 1].contiguous(), self._int([0, n]), n, self._int([0]), k, v, status)
        self._checked(status, "reads")
        return k, v


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--sessions", type=int, default=4)
    ap.add_argument("--branches", type=int, default=3)
    ap.add_argument("--rounds", type=int, default=6)
    ap.add_argument("--drafts", type=int, default=4)
    a = ap.parse_args()
    rng = np.random.default_rng(0)
    model = Model()
    prompts = [rng.integers(0, model.vocab, 200 + 19 * s).tolist() for s in range(a.sessions)]
    run = Branches(model, prompts, a.branches, pool_pages=64 * a.sessions)
    print("%d pages hold %d continuations" % (int((run.pool.refs > 0).sum()), run.B))
    for r in range(1, a.rounds + 1):
        run.round([rng.integers(0, model.vocab, int(rng.integers(1, a.drafts + 1))).tolist() for _ in range(run.B)], r)
        print("round %d: lengths %s, %d pages live" % (r, run.kv_len, int((run.pool.refs > 0).sum())))
    live = run.keep([int(rng.integers(0, a.branches)) for _ in range(a.sessions)])
    print("one continuation of each kept: %d pages, the first of the pool" % live)


if __name__ == "__main__":
    main()
