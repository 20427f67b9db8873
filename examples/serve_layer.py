"""A decoder stack served with gated maps: prompts in chunks, then one token a step.

    python examples/serve_layer.py [--width 4096 --heads 16 --layers 2 --prompts 700 1300 --steps 16]

Every layer runs its four projections as gated maps (`linear`), and between
them the serving operators: the step's pages and slots (`paged_plan`, once for
all layers), the split of the qkv rows into queries and cached keys and values
(`cache_append`), attention of the new tokens over the pages
(`paged_attention`), and the norm after a block, its gate, the residual and the
norm before the next block in one pass (`norm_residual`).  Weights and tokens
are random; with --check the hidden states are compared with a plain float64
model of the same layers.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_rank_subspace_gb300 as gsi  # noqa: E402


class Layer:
    def __init__(self, width, heads, kv_heads, hidden, rank, gen):
        head_dim = width // heads
        self.heads = heads

        def weight(d_out, d):
            return (torch.randn(d_out, d, device="cuda", generator=gen) * d ** -0.5).bfloat16()

        def basis(d):
            return torch.linalg.qr(torch.randn(d, rank, device="cuda", generator=gen))[0].bfloat16().contiguous()

        def gated(d_out, d):
            return gsi.make_map(weight(d_out, d), basis(d))

        def norm(kind):
            w = 1 + 0.1 * torch.randn(width, device="cuda", generator=gen)
            return gsi.Norm(kind, w, 0.1 * torch.randn(width, device="cuda", generator=gen) if kind == "layer" else None)

        self.qkv = gated((heads + 2 * kv_heads) * head_dim, width)
        self.out = gated(width, width)
        self.up = gated(hidden, width)
        self.down = gated(width, hidden)
        self.before, self.after_attention, self.before_mlp = norm("layer"), norm("rms"), norm("layer")
        self.gate = 0.5 + 0.1 * torch.randn(width, device="cuda", generator=gen)  # on the attention block


class Server:
    """The layers, their caches and the page tables of a batch of requests."""

    def __init__(self, layers, requests, max_tokens, pages, page_size=64, eps=0.05):
        self.layers, self.eps, self.page_size = layers, eps, page_size
        qkv = layers[0].qkv
        self.width, self.heads = qkv.d, layers[0].heads
        self.head_dim = self.width // self.heads
        kv_heads = (qkv.d_out // self.head_dim - self.heads) // 2
        self.caches = [gsi.PagedCache.empty(pages, kv_heads, page_size, self.head_dim) for _ in layers]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((requests, pages), -1, **i32)
        self.free = torch.arange(pages, **i32)
        self.n_free = torch.tensor([pages], **i32)
        self.cached = torch.zeros(requests, **i32)
        maps = [m for layer in layers for m in (layer.qkv, layer.out, layer.up, layer.down)]
        self.map_workspace = gsi.new_workspace(max(gsi.workspace_size(m, t) for m in maps for t in {1, 2, 16, max_tokens}))
        self.workspace = gsi.new_workspace(gsi.paged_attention_workspace_size(self.caches[0], self.heads))

    def linear(self, m, x):
        return gsi.linear(m, x, self.eps, workspace=self.map_workspace, want_rho=False)[0]

    def step(self, tokens, fresh):
        """tokens: the new tokens' embeddings (sum of `fresh`, width) float32; fresh: how many of each request.
        Returns the hidden states."""
        T = tokens.shape[0]
        plan = gsi.paged_plan(self.cached, torch.tensor(fresh, dtype=torch.int32).cuda(), self.table, self.free, self.n_free,
                              self.page_size, T)
        h, x = gsi.norm_residual(tokens, pre=self.layers[0].before)
        for i, (layer, cache) in enumerate(zip(self.layers, self.caches)):
            q = gsi.cache_append(cache, self.linear(layer.qkv, x), plan.slots, self.heads)
            o = gsi.paged_attention(cache, q, plan.q_start, plan.kv_len, self.table, max_q=max(fresh), workspace=self.workspace)
            y = self.linear(layer.out, o.view(T, self.width))
            h, x = gsi.norm_residual(h, y, post=layer.after_attention, gate=layer.gate, pre=layer.before_mlp, h_out=h)
            u = torch.nn.functional.gelu(self.linear(layer.up, x)).bfloat16()
            following = self.layers[i + 1].before if i + 1 < len(self.layers) else None
            h, x = gsi.norm_residual(h, self.linear(layer.down, u), pre=following, h_out=h)
        # the next step goes on from this one's lengths and free pages
        self.cached, self.n_free, self.status = plan.kv_len, plan.n_free, plan.status
        return h

    def finish(self, request):
        """Gives a finished request's pages back."""
        pages = self.table[request][self.table[request] >= 0]
        n = int(self.n_free)
        self.free[n:n + len(pages)] = pages
        self.n_free = self.n_free + len(pages)
        self.table[request] = -1
        self.cached = self.cached.clone()
        self.cached[request] = 0


def plain(layers, tokens):
    """The same layers over one whole sequence in float64, every token on the exact path."""
    def norm(n, v):
        if n.kind == "layer":
            v = v - v.mean(-1, keepdim=True)
        v = v * (v.square().mean(-1, keepdim=True) + n.eps).rsqrt() * n.weight.double()
        return v if n.bias is None else v + n.bias.double()

    h = tokens.double()
    T = h.shape[0]
    hidden = torch.ones(T, T, device="cuda", dtype=torch.bool).triu(1)
    for layer in layers:
        D = h.shape[1] // layer.heads
        qkv = (norm(layer.before, h) @ layer.qkv.W.double().T).view(T, -1, D).transpose(0, 1)
        kv_heads = (qkv.shape[0] - layer.heads) // 2
        q, k, v = qkv.split([layer.heads, kv_heads, kv_heads])
        k, v = (t.repeat_interleave(layer.heads // kv_heads, 0) for t in (k, v))
        p = torch.softmax((q @ k.transpose(1, 2) * D ** -0.5).masked_fill(hidden, -float("inf")), -1)
        o = (p @ v).transpose(0, 1).reshape(T, -1)
        h = h + layer.gate.double() * norm(layer.after_attention, o @ layer.out.W.double().T)
        u = torch.nn.functional.gelu(norm(layer.before_mlp, h) @ layer.up.W.double().T)
        h = h + u @ layer.down.W.double().T
    return h


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=None)
    ap.add_argument("--hidden", type=int, default=None)
    ap.add_argument("--rank", type=int, default=256)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 1300])
    ap.add_argument("--chunk", type=int, default=512, help="a prompt's tokens of one step, at most")
    ap.add_argument("--steps", type=int, default=16, help="tokens added to every prompt")
    ap.add_argument("--eps", type=float, default=0.05)
    ap.add_argument("--check", action="store_true", help="compare with float64 (use --eps 0: the exact path)")
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    layers = [Layer(a.width, a.heads, a.kv_heads or a.heads, a.hidden or 4 * a.width, a.rank, gen) for _ in range(a.layers)]
    total = [p + a.steps for p in a.prompts]
    tokens = [torch.randn(n, a.width, device="cuda", generator=gen) for n in total]
    page = 64
    server = Server(layers, len(total), a.chunk * len(total), sum(-(-n // page) for n in total) + 1, page, a.eps)
    done, states, steps = [0] * len(total), [[] for _ in total], []
    while any(d < n for d, n in zip(done, total)):
        # whoever still has prompt brings a chunk of it, the others one token
        fresh = [min(a.chunk, p - d) if d < p else min(1, n - d) for d, p, n in zip(done, a.prompts, total)]
        new = torch.cat([t[d:d + f] for t, d, f in zip(tokens, done, fresh)])
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        h = server.step(new, fresh)
        torch.cuda.synchronize()
        steps.append((sum(fresh), time.perf_counter() - t0))
        for s, part in zip(states, h.split(fresh)):
            s.append(part)
        done = [d + f for d, f in zip(done, fresh)]
    assert int(server.status) == 0 and gsi.workspace_status(server.workspace) == 0
    for n, s in steps[:4] + steps[-2:]:
        print(f"{n} tokens: {s * 1e3:.3f} ms")
    worst = 0.0
    if a.check:
        for t, s in zip(tokens, states):
            want = plain(layers, t)
            worst = max(worst, float((torch.cat(s).double() - want).norm() / want.norm()))
        print(f"relative error against float64: {worst:.2e}")
    free = int(server.n_free)
    for r in range(len(total)):
        server.finish(r)
    assert int(server.n_free) == free + sum(-(-n // page) for n in total)
    return worst


if __name__ == "__main__":
    main()
