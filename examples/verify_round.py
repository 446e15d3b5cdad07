"""A verifier's rounds from scoring to commit, with the serving operators around the verify call.

    python examples/verify_round.py [--sessions 8] [--rounds 6] [--drafts 4]

A model of one attention layer with random weights stands in for the target model (the point is the
order of the calls, not the text).  Each round, for a ragged batch of proposals:

  1. the M_b + 1 rows of every session are projected, and sdcp_append_kv turns their queries and
     keys by position and puts keys and values into the session's pages, in 4 bits;
  2. sdcp_attend_kv attends them over the cached context, causally among themselves;
  3. sdcp_adjust_logits applies the session's penalties, biases and grammar mask to the rows, row i
     in the context of the drafts before it;
  4. sdcp_verify_batch accepts a prefix of the drafts and emits one more token, and
     sdcp_commit_batch truncates and updates the session's state;
  5. the host adds n_out[b] to kv_len[b] and to the history: what was rejected is overwritten by
     the next round's append.

Each call has a status of its own for every session, and they refuse different things (a position past
the rotation's table is the append's to see, the attention then reads what was in the cache before).  So
the statuses are joined, and a session that any call refused commits nothing.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_verification_sdcp_gb300 import sdcp  # noqa: E402


class Model:
    """One attention layer: embedding, fused q/k/v projection, output projection, head."""

    def __init__(self, vocab=1000, q_heads=8, kv_heads=2, head_dim=64, device="cuda:0", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.vocab, self.q_heads, self.kv_heads, self.head_dim, self.device = vocab, q_heads, kv_heads, head_dim, device
        width = q_heads * head_dim
        rand = lambda *s, k: torch.randn(s, generator=g, device=device).mul_(k).to(torch.bfloat16)  # noqa: E731
        self.embed = rand(vocab, width, k=1.0)
        self.w_qkv = rand(width, (q_heads + 2 * kv_heads) * head_dim, k=width ** -0.5)
        self.w_out = rand(width, width, k=width ** -0.5)
        self.head = rand(width, vocab, k=3.0 * width ** -0.5)

    def qkv(self, x):
        y = (x @ self.w_qkv).unflatten(1, (-1, self.head_dim))
        return y.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)

    def logits(self, x, attended):
        return ((x + attended.flatten(1) @ self.w_out) @ self.head).contiguous()


def rotary_table(n_positions, rot_dim, device, base=10000.0, stretch=1.0):
    """Cosines and sines of each position (positions divided by `stretch` for longer contexts)."""
    at = torch.arange(n_positions, device=device, dtype=torch.float64)[:, None] / stretch
    angle = at * base ** (-torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64) / rot_dim)
    return torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32)


class Rounds:
    """The sessions of one batch: their pages, histories and states."""

    def __init__(self, model: Model, prompts, max_tokens=512, page_tokens=32, repetition=1.2, banned=()):
        self.model, self.device, self.B = model, model.device, len(prompts)
        dev = self.device
        self.history = [list(p) for p in prompts]
        self.prompt_len = [len(p) for p in prompts]
        per = -(-max_tokens // page_tokens)
        self.cache = sdcp.KvCache(self.B * per, page_tokens, model.kv_heads, model.head_dim, dev)
        self.page_table = torch.arange(self.B * per, dtype=torch.int32, device=dev).view(self.B, per)
        self.rotary = sdcp.Rotary(rotary_table(max_tokens, model.head_dim, dev))
        self.repetition = repetition
        words = np.full((1, (model.vocab + 31) // 32), 0xFFFFFFFF, dtype=np.uint32)
        for t in banned:
            words[0, t // 32] &= np.uint32(0xFFFFFFFF ^ (1 << (t % 32)))
        self.masks = torch.from_numpy(words.view(np.int32)).to(dev)
        self.state = torch.zeros(self.B * 64, dtype=torch.uint8, device=dev)
        cp = np.zeros(self.B, dtype=sdcp.COMMIT_PARAMS_DTYPE)
        cp["max_new"], cp["m_max"], cp["low_rounds"], cp["self_load"] = max_tokens, sdcp.MAX_M, 4, sdcp.NO_SELF_LOAD
        cp["fallback_len"], cp["fallback"][:, 0] = 1, sdcp.ACTION_REDUCE
        self.cparams = torch.from_numpy(cp.view(np.uint8).copy()).to(dev)
        self.refused = {}  # status of the sessions that the last round refused
        # all of a prompt but its last token, which is the first row of the first round, is one long round
        # of the sessions that have more
        if not all(prompts):
            raise ValueError("a prompt has at least one token")
        self.kv_len = [0] * self.B
        longer = [b for b, p in enumerate(prompts) if len(p) > 1]
        if longer:
            status = self.score([prompts[b][:-1] for b in longer], longer)[3].tolist()
            if any(status):
                raise ValueError("prompts refused: %s" % {b: st for b, st in zip(longer, status) if st})
            self.kv_len = [len(p) - 1 for p in prompts]

    def _int(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def score(self, rows, sessions=None):
        """Logits of new rows (lists of tokens) of the sessions (default: all), which are appended to the
        cache; offsets, number of drafts, and the sessions' status."""
        m = self.model
        kv_len, table = self.kv_len, self.page_table
        if sessions is not None:
            kv_len, table = [kv_len[b] for b in sessions], table[sessions]
        off = self._int(np.concatenate([[0], np.cumsum([len(r) - 1 for r in rows])]).tolist())
        total = sum(len(r) - 1 for r in rows)
        x = m.embed[torch.tensor([t for r in rows for t in r], device=self.device)]
        q, k, v = m.qkv(x)
        turned, out = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(q, memory_format=torch.contiguous_format)
        n = len(rows)
        kv_len, appended, attended = self._int(kv_len), self._int([0] * n), self._int([0] * n)
        sdcp.sdcp_append_kv(self.cache, table, off, total, kv_len, k, v, appended, rotary=self.rotary, q=q, q_out=turned)
        scratch = sdcp.alloc_attend_workspace(n, total, m.q_heads, m.kv_heads, m.head_dim, self.device)
        sdcp.sdcp_attend_kv(self.cache, table, off, total, kv_len, turned, out, attended, scratch)
        return m.logits(x, out), off, total, torch.maximum(appended, attended)

    def controls(self):
        c = np.zeros(self.B, dtype=sdcp.CONTROLS_DTYPE)
        c["repetition"], c["frequency"], c["presence"] = self.repetition, 0.1, 0.1
        c["history_len"], c["prompt_len"] = [len(h) for h in self.history], self.prompt_len
        return sdcp.controls_tensor(c, self.device)

    def round(self, drafts, number):
        """One round with the sessions' drafts (lists of 1 .. 64 tokens): the tokens it emitted, none for
        the sessions that it refused."""
        logits, off, total, scored = self.score([[h[-1]] + list(d) for h, d in zip(self.history, drafts)])
        tokens = self._int([t for d in drafts for t in d])
        longest = max(len(h) for h in self.history)
        history = self._int([h + [-1] * (longest - len(h)) for h in self.history])
        adjusted = self._int([0] * self.B)
        sdcp.sdcp_adjust_logits(logits, logits, off, total, tokens, self.controls(), history, adjusted, masks=self.masks,
                                mask_rows=self._int([0] * logits.shape[0]))
        params = np.zeros(self.B, dtype=sdcp.PARAMS_DTYPE)
        params["rule_id"], params["temperature_milli"], params["top_p_milli"] = sdcp.SDCP_RULE_GREEDY, 1000, 1000
        params["seed"], params["round"], params["session_tag"] = 1, number, np.arange(self.B)
        ver = sdcp.Verifier(self.model.vocab, self.B, total, self.device)
        accepted, n_out, out, st = ver(logits, None, off, tokens, sdcp.params_tensor(params, self.device))
        status, action = torch.maximum(torch.maximum(scored, adjusted), st), self._int([0] * self.B)
        sdcp.sdcp_commit_batch(off, accepted, n_out, out, status, self.cparams, None, self.state, 0, action)
        self.refused = {b: s for b, s in enumerate(status.tolist()) if s != sdcp.S_OK}
        emitted, first = [], off.tolist()
        for b, n in enumerate(n_out.tolist()):
            n = 0 if b in self.refused else n
            got = out[first[b] + b:first[b] + b + n].tolist()
            self.history[b] += got
            self.kv_len[b] += n
            emitted.append(got)
        return emitted


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--sessions", type=int, default=8)
    ap.add_argument("--rounds", type=int, default=6)
    ap.add_argument("--drafts", type=int, default=4)
    a = ap.parse_args()
    rng = np.random.default_rng(0)
    model = Model()
    sessions = Rounds(model, [rng.integers(0, model.vocab, 5 + 9 * b).tolist() for b in range(a.sessions)])
    for r in range(1, a.rounds + 1):
        got = sessions.round([rng.integers(0, model.vocab, int(rng.integers(1, a.drafts + 1))).tolist() for _ in range(a.sessions)], r)
        print("round %d emitted %s%s" % (r, got, " refused %s" % sessions.refused if sessions.refused else ""))


if __name__ == "__main__":
    main()
