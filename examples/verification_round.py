"""Speculative rounds with a toy target: what the library's calls look like next to each other.

One attention layer with random weights stands for the target model.  A round takes the last committed token and gamma
drafted ones, attends over the 8-bit cache and the round's own rows, turns the result into logits, applies penalties to
the target's rows and the draft's alike, verifies, and commits the keys and values of the accepted rows alone.  The draft
model is the target's logits with noise.

    python examples/verification_round.py [--rounds 4] [--tree]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_verification_spec_gb300 as sv  # noqa: E402


class Toy:
    """Embedding, one attention layer over the cache, output projection; bf16 on the GPU."""

    def __init__(self, V=5003, hq=16, hkv=4, D=128, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[0] ** 0.5).bfloat16()
        self.V, self.hq, self.hkv, self.D = V, hq, hkv, D
        self.embed, self.head = w(V, hq * D) * V ** 0.5, w(hq * D, V)
        self.wq, self.wk, self.wv = w(hq * D, hq * D), w(hq * D, hkv * D), w(hq * D, hkv * D)

    def qkv(self, tokens):
        x = self.embed[tokens.long()]
        cut = lambda y, h: y.unflatten(-1, (h, self.D))
        return x, cut(x @ self.wq, self.hq), cut(x @ self.wk, self.hkv), cut(x @ self.wv, self.hkv)

    def logits(self, x, attended):
        return ((x + attended.flatten(-2)) @ self.head).contiguous()


def run(rounds=4, B=3, prompt=150, gamma=5, page=64, tree=False, seed=0, temperature=0.8):
    """Returns the history [B, H], its lengths, and the accepted length of every round."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    toy = Toy(seed=seed)
    V, room = toy.V, prompt + rounds * (gamma + 1) + gamma + 2
    per = -(-room // page)
    cache = sv.kv_cache(B * per, toy.hkv, page, toy.D)
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    i32 = dict(dtype=torch.int32, device="cuda")
    history = torch.zeros(B, room, **i32)
    history[:, :prompt] = torch.randint(0, V, (B, prompt), generator=g, device="cuda").to(torch.int32)
    hist_len = torch.full((B,), prompt, **i32)
    prompt_len = hist_len.clone()
    f32 = lambda x: torch.full((B,), x, device="cuda")
    penalties = dict(repetition=f32(1.15), presence=f32(0.1), frequency=f32(0.05))

    # the prompt, but for its last token, which the first round starts from
    _, _, k, v = toy.qkv(history[:, :prompt - 1])
    lens = sv.kv_cache_write(k, v, cache, table, torch.zeros(B, **i32))["lens"]
    accepted = []
    for _ in range(rounds):
        last = history.gather(1, hist_len.long()[:, None] - 1)
        # a draft: tokens from the target's logits after `last`, blurred; in the tree every other node hangs off the frontier
        drafts = torch.randint(0, V, (B, gamma), generator=g, device="cuda").to(torch.int32)
        parents = None
        if tree:
            parents = (torch.arange(gamma, device="cuda") // 2 - 1).to(torch.int32).expand(B, gamma).contiguous()
        x, q, k, v = toy.qkv(torch.cat([last, drafts], 1))
        out = sv.verify_attention(q, cache, table, lens, k=k, v=v, parents=parents)["out"]
        raw = toy.logits(x, out)
        blurred = (raw.float() + torch.randn(raw.shape, generator=g, device="cuda")).bfloat16()
        path = dict(tokens=drafts, parents=parents, history=history, prompt_len=prompt_len, history_len=hist_len)
        p = sv.process_logits(raw, **path, **penalties)["logits"]
        if tree:
            # let the tree hold what the target would say, so that something is accepted
            drafts[:, 0] = p[:, 0].argmax(-1).to(torch.int32)
            x, q, k, v = toy.qkv(torch.cat([last, drafts], 1))
            out = sv.verify_attention(q, cache, table, lens, k=k, v=v, parents=parents)["out"]
            p = sv.process_logits(toy.logits(x, out), **path, **penalties)["logits"]
            r = sv.tree_verify_greedy(p, parents, drafts)
            nodes = r["out_nodes"]
        else:
            d = sv.process_logits(blurred[:, :gamma], **path, **penalties)["logits"]
            u = torch.rand(B, gamma + 2, generator=g, device="cuda")
            r = sv.spec_verify(p, d, drafts, u, temperature)
            nodes = None
        # only the accepted rows' keys and values enter the cache
        lens = sv.kv_cache_write(k, v, cache, table, lens, accepted_len=r["accepted_len"], out_nodes=nodes)["lens"]
        a = r["accepted_len"]
        at = torch.arange(r["out_tokens"].shape[1], device="cuda")[None]
        live = at <= a[:, None]
        where = torch.where(live, hist_len[:, None] + at, torch.full_like(hist_len[:, None] + at, room - 1)).long()
        history.scatter_(1, where, torch.where(live, r["out_tokens"], history[:, -1:]))
        hist_len = torch.where(a >= 0, hist_len + a + 1, hist_len).to(torch.int32)
        accepted.append(a)
    back = sv.kv_cache_read(cache, table, lens, max_len=room, dtype=torch.float32)
    return dict(history=history, hist_len=hist_len, lens=lens, accepted=torch.stack(accepted), cache_k=back["k"], toy=toy)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=4)
    ap.add_argument("--tree", action="store_true")
    a = ap.parse_args()
    r = run(rounds=a.rounds, tree=a.tree)
    print("accepted per round and request:", r["accepted"].tolist())
    print("tokens:", r["hist_len"].tolist(), " in the cache:", r["lens"].tolist())
