"""A small striped stack served with a paged 8-bit cache.

Runs the library's operators together the way a server of a StripedHyena 2 model
uses them (random weights, one mixer per block), every projection in 8 bits:

    page_map                     once per step: tables, slots and positions of the new tokens
    per block:
      add_rmsnorm_fp8            residual addition, norm, 8-bit input of in_proj
      linear_fp8                 in_proj
      h: chunk_fwd_tokmajor      the modal Hyena mixer, its state carried per request
      a: qk_norm_rope            norms of the query and key heads, rotary positions, in place
         kv_append_fp8 + attn_paged_fp8   attention over the cache
      quantize_fp8 + linear_fp8  out_proj
      add_rmsnorm_fp8            residual addition, norm, 8-bit input of the MLP
      gated_linear_fp8           both projections, gelu and product, 8-bit output
      linear_fp8                 the MLP's last projection
    add_rmsnorm                  final norm, then the unembedding (torch)

Prompts of different lengths are prefilled in chunks, then all requests decode
together; a request that ends gives its pages back and another takes its place.
`python examples/striped_serving.py` prints the time of a decode step and
compares the served hidden states with a single prefill of the whole sequences.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import genomic_lm_amd as G  # noqa: E402
from genomic_lm_amd import serving  # noqa: E402

BF = torch.bfloat16


class StripedServer:
    """Weights, caches and states of a stack of `pattern` mixers (h: Hyena, a: attention)."""

    def __init__(self, pattern="hah", dim=256, heads=4, modes=8, vocab=512, requests=4, max_len=1024,
                 page=64, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale).to(device)  # noqa: E731
        self.pattern, self.dim, self.heads, self.page, self.device = pattern, dim, heads, page, device
        self.embed = rand(vocab, dim).to(BF)
        self.norms = [1 + rand(dim, scale=0.1) for _ in range(2 * len(pattern) + 1)]
        inner = -(-11 * dim // 64) * 16                 # 2.75 dim, in whole 16 columns
        # weights in 8 bits with their scales, quantised once
        weight = lambda *s: G.quantize_weight_fp8(rand(*s, scale=s[1] ** -0.5))  # noqa: E731
        self.w_in = [weight(3 * dim, dim) for _ in pattern]
        self.w_out = [weight(dim, dim) for _ in pattern]
        self.w_gate, self.w_up = ([weight(inner, dim) for _ in pattern] for _ in range(2))
        self.w_down = [weight(dim, inner) for _ in pattern]
        self.head_norms = [[1 + rand(dim // heads, scale=0.1) for _ in "qk"] for _ in pattern]
        self.inv_freq = G.rotary_inv_freq(dim // heads, device=device)
        # poles with memories of one to a thousand tokens
        self.log_poles = [-torch.exp(torch.rand((dim, modes), generator=g) * -6.9).to(device) for _ in pattern]
        self.residues = [rand(dim, modes, scale=modes ** -0.5) for _ in pattern]
        self.skip = [rand(dim) for _ in pattern]

        per = -(-max_len // page)
        self.pages = requests * per
        self.free = torch.randperm(self.pages, generator=g).to(torch.int32).to(device)
        self.head = torch.zeros(1, dtype=torch.int32, device=device)
        self.table = torch.full((requests, per), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.unplaced = torch.zeros(1, dtype=torch.int32, device=device)
        self.caches = {i: serving.new_cache(self.pages, heads, page, dim // heads, device)
                       for i, kind in enumerate(pattern) if kind == "a"}
        self.states = {i: torch.zeros((requests, dim, modes), device=device)
                       for i, kind in enumerate(pattern) if kind == "h"}

    def _hyena(self, i, proj, new):
        """The modal mixer over each request's tokens: (T, 3 dim) -> (T, dim)."""
        par = (self.log_poles[i], self.residues[i], self.skip[i])
        state = self.states[i]
        if all(n == 1 for n in new):
            y, _ = G.chunk_fwd_tokmajor(proj[:, None], *par, state_in=state, state_out=state)
            return y[:, 0]
        out, at = torch.empty((proj.shape[0], self.dim), dtype=BF, device=self.device), 0
        for r, n in enumerate(new):
            if n:
                G.chunk_fwd_tokmajor(proj[None, at:at + n], *par, state_in=state[r:r + 1],
                                     state_out=state[r:r + 1], out=out[None, at:at + n])
            at += n
        return out

    def _attention(self, i, proj, cu, lens, positions, slots, most):
        q, k, v = proj.view(-1, 3, self.heads, self.dim // self.heads).unbind(1)
        G.qk_norm_rope(q, k, positions, self.inv_freq, *self.head_norms[i], eps=1e-6, q_out=q, k_out=k)
        G.kv_append_fp8(k, v, slots, *self.caches[i])
        o = G.attn_paged_fp8(q, *self.caches[i], self.table, lens, cu, most)
        return o.view(-1, self.dim)

    def step(self, ids, new):
        """New tokens of each request (new: how many, on the host; ids: all of them in a row).
        Returns the normed hidden state of every new token and the logits of each last one."""
        tokens = sum(new)
        brings = torch.tensor(new, dtype=torch.int32).to(self.device)
        cu, lens, positions, slots, status = G.page_map(self.lens, brings, self.table, self.free, self.head,
                                                        self.page, tokens)
        x, res = self.embed[ids], None
        for i, kind in enumerate(self.pattern):
            q, scale, summed = G.add_rmsnorm_fp8(x, self.norms[2 * i], res, group=128)
            res = x if summed is None else summed
            proj = G.linear_fp8(q, scale, *self.w_in[i])
            y = (self._hyena(i, proj, new) if kind == "h"
                 else self._attention(i, proj, cu, lens, positions, slots, max(new)))
            x = G.linear_fp8(*G.quantize_fp8(y, group=128), *self.w_out[i])
            q, scale, res = G.add_rmsnorm_fp8(x, self.norms[2 * i + 1], res, group=128)
            q, scale = G.gated_linear_fp8(q, scale, *self.w_gate[i], *self.w_up[i], act="gelu",
                                          dtype=torch.float8_e4m3fn)
            x = G.linear_fp8(q, scale, *self.w_down[i])
        hidden, _ = G.add_rmsnorm(x, self.norms[-1], res)
        self.lens, self.head = lens, status[:1].clone()
        self.unplaced += status[1:]           # tokens without a page: looked at when the host next waits
        return hidden, hidden[(cu[1:] - 1).clamp(min=0).long()] @ self.embed.t()

    def finish(self, r):
        """Request r ends: its pages go back to the free list, its states are cleared."""
        n = -(-int(self.lens[r]) // self.page)
        head = int(self.head)
        self.free[head - n:head] = self.table[r, :n]
        self.head -= n
        self.table[r] = -1
        self.lens[r] = 0
        for s in self.states.values():
            s[r] = 0


def serve(server, prompts, steps, chunk):
    """Prefills the prompts in chunks of at most `chunk` tokens, then decodes `steps` tokens
    greedily.  Returns per request its tokens and its hidden states."""
    R, device = len(prompts), server.device
    done, seqs, hidden = [0] * R, [list(p) for p in prompts], [[] for _ in range(R)]
    last = [None] * R

    def run(pieces):
        new = [len(p) for p in pieces]
        ids = torch.tensor([t for p in pieces for t in p], device=device)
        h, logits = server.step(ids, new)
        at = 0
        pick = logits.argmax(-1).tolist()
        for r, n in enumerate(new):
            if n:
                hidden[r].append(h[at:at + n])
                last[r] = pick[r]
            at += n

    while any(done[r] < len(prompts[r]) for r in range(R)):
        pieces = [prompts[r][done[r]:done[r] + chunk] for r in range(R)]
        run(pieces)
        done = [d + len(p) for d, p in zip(done, pieces)]
    for _ in range(steps):
        for r in range(R):
            seqs[r].append(last[r])
        run([[s[-1]] for s in seqs])
    return seqs, [torch.cat(h) for h in hidden]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=48)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 33, 128, 1])
    ap.add_argument("--chunk", type=int, default=256)
    ap.add_argument("--page", type=int, default=64)
    a = ap.parse_args(argv)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(4, 512, (n,), generator=g).tolist() for n in a.prompts]
    rounds = 20
    most = max(max(a.prompts) + a.steps + 1, a.page + 3) + rounds
    build = lambda: StripedServer(dim=a.dim, heads=a.heads, requests=len(prompts), max_len=most, page=a.page)  # noqa: E731
    server = build()
    seqs, hidden = serve(server, prompts, a.steps, a.chunk)

    # the same sequences, each in one prefill on a fresh server
    whole = build()
    _, want = serve(whole, seqs, 0, most)
    far = [float((h.float() - w.float()).norm() / w.float().norm()) for h, w in zip(hidden, want)]

    # a request ends, another takes its place and pages
    server.finish(1)
    again = torch.randint(4, 512, (a.page + 3,), generator=g).tolist()
    new = [1] * len(prompts)
    new[1] = len(again)
    ids = torch.tensor([t for r in range(len(prompts)) for t in (again if r == 1 else [seqs[r][-1]])],
                       device=server.device)
    h, _ = server.step(ids, new)

    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(rounds):
        server.step(ids[:len(prompts)], [1] * len(prompts))
    torch.cuda.synchronize()
    ms = (time.perf_counter() - began) / rounds * 1e3
    if int(server.unplaced) or int(whole.unplaced):
        raise RuntimeError("tokens without a page: the pool is too small")
    print(f"{len(prompts)} requests, {len(server.pattern)} blocks of {a.dim}: {ms:.3f} ms per decode step")
    print("served against one prefill, relative difference per request:",
          " ".join(f"{x:.3f}" for x in far))
    return far, torch.isfinite(h.float()).all().item()


if __name__ == "__main__":
    main()
