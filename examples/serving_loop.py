"""A speculative serving loop on the paged 8-bit cache, with a toy model of random weights.

Every round, for a batch of sequences of different lengths:

1. the draft proposes K tokens one after the other (``ssd_sample`` under temperature and
   top-k, which also writes the filtered logits: the draft's q);
2. ``ssd_kv_plan`` commits what the last round accepted, gives pages beyond it back and gives
   the K+1 tokens to be fed their pages and slots, all on the GPU;
3. the target layer's keys and values of those tokens go into the cache (``ssd_kv_append``) and
   its queries attend over it (``ssd_kv_attend``);
4. the target's logits are truncated the same way (top-p), and ``ssd_round`` accepts, draws the
   bonus token and builds the next speculation cache.

The target is one attention layer, the draft a table of next-token logits; both share one
vocabulary.  Nothing in a round waits for the GPU but the copy of the round's outcome that
the loop prints.

    python examples/serving_loop.py --batch 16 --rounds 20
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import speculative_decoding_verification_ssd_gb300 as ssd  # noqa: E402


class Target:
    """One layer: embeddings with positions, grouped-query attention, logits."""

    def __init__(self, V, width, Hq, Hkv, D, gen):
        dev = "cuda"
        rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
        self.V, self.Hq, self.Hkv, self.D = V, Hq, Hkv, D
        self.emb, self.head = rnd(V, width).to(torch.bfloat16), rnd(V, width).to(torch.bfloat16)
        self.sharp = 3 / width ** 0.5
        self.qkv = (rnd(width, (Hq + 2 * Hkv) * D) / width ** 0.5).to(torch.bfloat16)
        self.out = (rnd(Hq * D, width) / (Hq * D) ** 0.5).to(torch.bfloat16)
        self.freq = torch.exp(torch.linspace(0, -9, width // 2, device=dev))

    def hidden(self, tokens, positions):
        a = positions.to(torch.float32)[:, None] * self.freq
        return self.emb[tokens] + 0.5 * torch.cat([a.sin(), a.cos()], dim=1).to(torch.bfloat16)

    def split(self, h):
        x = (h @ self.qkv).view(h.shape[0], self.Hq + 2 * self.Hkv, self.D)
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]

    def logits(self, h, attended):
        y = h + attended.reshape(h.shape[0], -1) @ self.out
        return (y @ self.head.T).float() * self.sharp


class Loop:
    def __init__(self, B=8, K=4, V=4096, width=256, Hq=8, Hkv=2, D=64, page=32, pages=512, max_blocks=48, tau=0.9, top_p=0.95,
                 top_k=64, budget=16, seed=0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.K, self.V, self.page = B, K, V, page
        self.target = Target(V, width, Hq, Hkv, D, self.gen)
        # a draft that knows the target's logits without its attention, and some noise
        t = self.target
        self.draft = t.emb.float() @ t.head.float().T * t.sharp + 0.5 * torch.randn((V, V), generator=self.gen, device="cuda")
        self.state = ssd.kv_state(B, max_blocks, pages)
        shape = (pages, Hkv, page, D)
        self.k, self.v = (torch.zeros(shape, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.zeros((pages, Hkv), device="cuda") for _ in range(2))
        self.workspace = ssd.kv_workspace()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        f = lambda n, x: torch.full((n,), x, device="cuda")  # noqa: E731
        self.tau, self.rows_tau = f(B, tau), f(B * (K + 1), tau)
        self.top_p, self.top_k = f(B * (K + 1), top_p), torch.full((B,), top_k, dtype=torch.int32, device="cuda")
        self.F, _ = ssd.ssd_fanout(K, budget, 0.6, 1.0, V)
        self.budget = budget
        self.accept = None          # of the last round
        self.last = None            # [B] the token that each sequence feeds first
        self.sm_scale = D ** -0.5

    def _uniform(self, *shape):
        return torch.rand(shape, generator=self.gen, device="cuda")

    def _forward(self, tokens, new, cap, max_new):
        """The target over `cap` packed tokens, `new` of each sequence: their logits."""
        st = self.state
        plan = ssd.ssd_kv_plan(st["seq_len"], new, st["held"], st["block_table"], st["ring"], st["ring_state"], self.page, cap,
                               accept_len=self.accept, dev_status=self.status)
        h = self.target.hidden(tokens, plan["positions"])
        q, k, v = self.target.split(h)
        ssd.ssd_kv_append(k, v, plan["slots"], self.k, self.v, self.ks, self.vs, dev_status=self.status)
        o = ssd.ssd_kv_attend(q, self.k, self.v, self.ks, self.vs, st["block_table"], plan["cu_new"], plan["kv_len"], max_new,
                              self.sm_scale, workspace=self.workspace, dev_status=self.status)
        return self.target.logits(h, o)

    def prompt(self, prompts):
        """Feeds all but the last token of each prompt (lists of token ids)."""
        new = [len(p) - 1 for p in prompts]
        self.last = torch.tensor([p[-1] for p in prompts], device="cuda")
        n = torch.tensor(new, dtype=torch.int32, device="cuda")
        if sum(new):
            tokens = torch.tensor([t for p in prompts for t in p[:-1]], device="cuda")
            self._forward(tokens, n, sum(new), max(new))
        self.accept = n - 1         # everything fed stays

    def round(self):
        """One round: returns (accept_len [B], bonus [B], draft tokens [B, K]) on the GPU."""
        B, K, V = self.B, self.K, self.V
        token, drafts, q = self.last, [], []
        for _ in range(K):
            d = ssd.ssd_sample(self.draft[token], self.tau, self._uniform(B), top_k=self.top_k, filtered=True, dev_status=self.status)
            token = d["tokens"].long()
            drafts.append(d["tokens"])
            q.append(d["filtered"])
        drafts = torch.stack(drafts, dim=1)
        fed = torch.cat([self.last[:, None], drafts.long()], dim=1)
        new = torch.full((B,), K + 1, dtype=torch.int32, device="cuda")
        logits = self._forward(fed.reshape(-1), new, B * (K + 1), K + 1)
        p = ssd.ssd_sample(logits, self.rows_tau, self._uniform(B * (K + 1)), top_p=self.top_p, filtered=True,
                           dev_status=self.status)["filtered"]
        out = ssd.ssd_round(p.view(B, K + 1, V), torch.stack(q, dim=1), drafts, self._uniform(B, K + 1), self.tau, self.F,
                            self.budget, dev_status=self.status)
        self.accept, self.last = out["accept_len"], out["bonus"].long()
        return out["accept_len"], out["bonus"], drafts


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--rounds", type=int, default=20)
    ap.add_argument("--draft-tokens", type=int, default=4)
    a = ap.parse_args()
    loop = Loop(B=a.batch, K=a.draft_tokens, pages=64 * a.batch)
    g = torch.Generator().manual_seed(1)
    loop.prompt([torch.randint(0, loop.V, (int(n),), generator=g).tolist() for n in torch.randint(1, 200, (a.batch,), generator=g)])
    total = 0
    for i in range(a.rounds):
        accept, _, _ = loop.round()
        total += int(accept.sum()) + a.batch
    print(f"{a.rounds} rounds of {a.batch} sequences: {total} tokens, {total / a.rounds / a.batch:.2f} a sequence and round, "
          f"status {int(loop.status)}, {int(loop.state['ring_state'][1])} pages free")


if __name__ == "__main__":
    main()
