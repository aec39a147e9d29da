"""One attention layer serving several requests from a paged CQ cache, with
trees of drafted tokens verified in one step.

    python -m examples.verify_drafts [--requests 16] [--context 512] [--steps 8]

Weights, prompts and the draft model are random (nothing is trained here): what
the example shows is how the calls of a step go together, and that a tree's
verified path gives what the same tokens give one at a time.

A step of `Layer.step`:
  cq_kv_plan          blocks and slots of the step's tokens, from the lengths
  cq_gemm_grouped     query, key and value projections of CQ weights (int8 activations)
  cq_qk_norm_rope     per-head norms and rotation; queries to fp16
  cq_kv_write_slots   keys and values into the cache
  cq_kv_tree_attend   each token over its context and its ancestors
  cq_gemm             output projection
"""
from __future__ import annotations

import argparse
import time

import numpy as np
import torch

import hadamard_rotated_codebook_gb300 as cq

BLOCK = 16


class Layer:
    """8 query heads of 64 over 4 key/value heads, width 512; CQ4 weights and cache."""

    def __init__(self, requests: int, blocks: int, max_tokens: int, seed: int = 0, device: str = "cuda"):
        self.hq, self.hkv, self.d, self.width, self.bits = 8, 4, 64, 512, 4
        g = torch.Generator().manual_seed(seed)
        self.cb = cq.cq_codebook_init(self.bits, 128)

        def weight(out, n_in):
            return cq.cq_encode((torch.randn(out, n_in, generator=g) * n_in ** -0.5).to(device), self.bits, self.cb)

        self.wq, self.wo = weight(self.hq * self.d, self.width), weight(self.width, self.hq * self.d)
        self.wk, self.wv = weight(self.hkv * self.d, self.width), weight(self.hkv * self.d, self.width)
        self.q_norm, self.k_norm = (torch.zeros(self.d, device=device) for _ in range(2))  # zero-centred
        self.rates = cq.cq_rope_init(self.d)
        self.geom = cq.cq_kv_geometry(self.hq, self.hkv, self.d, self.d, self.bits, self.bits, self.cb, self.cb, self.d ** -0.5)
        self.cap = blocks * BLOCK
        size = cq.cq_packed_bytes(self.cap, self.hkv * self.d, 128, self.bits)
        self.k_cache, self.v_cache = (torch.zeros(size, dtype=torch.uint8, device=device) for _ in range(2))
        i32 = dict(dtype=torch.int32, device=device)
        self.lens = torch.zeros(requests, **i32)
        self.held = torch.zeros(requests, **i32)
        self.table = torch.full((requests, blocks), -1, **i32)
        self.free = torch.arange(blocks, **i32)
        self.n_free = torch.full((1,), blocks, **i32)
        self.room = max_tokens

    def step(self, x: torch.Tensor, new: torch.Tensor, mask=None, depth=None, max_nodes: int = 0) -> torch.Tensor:
        """x fp32 [tokens, width], the requests' new[s] tokens in order. With a
        tree, `mask` holds each token's ancestors and itself and `depth` its
        distance from the context; without, the tokens follow each other.
        The cache holds the tokens afterwards, but lens does not count them
        yet: accept() does."""
        n = x.shape[0]
        plan = cq.cq_kv_plan(self.lens, new, self.held, self.table, self.free, self.n_free, BLOCK, self.room)
        self.held, self.n_free = plan["held_out"], plan["n_free_out"]
        positions = plan["positions"][:n]
        if depth is not None:
            positions = self.lens[plan["token_seq"][:n].long()] + depth
        xq, s = cq.cq_act_quant_int8(x)
        q, k, v = cq.cq_gemm_grouped([{"blob": w, "out": out, "in": self.width, "bits": self.bits, "codebook": self.cb, "Xq": xq,
                                       "x_scale": s} for w, out in ((self.wq, self.hq * self.d), (self.wk, self.hkv * self.d),
                                                                    (self.wv, self.hkv * self.d))])
        q, k = cq.cq_qk_norm_rope(q.view(n, self.hq, self.d), k.view(n, self.hkv, self.d), positions.contiguous(), self.rates,
                                  self.q_norm, self.k_norm, weight_offset=1.0, q_dtype=torch.float16)
        cq.cq_kv_write_slots(self.geom, self.k_cache, self.v_cache, self.cap, k, v, plan["slots"][:n])
        o = cq.cq_kv_tree_attend(self.geom, q, self.k_cache, self.v_cache, self.cap, self.table, BLOCK, self.lens, plan["cu_new"],
                                 mask, max_nodes or n)
        self.last = k, v, plan
        oq, s = cq.cq_act_quant_int8(o.float().view(n, -1))
        return cq.cq_gemm(self.wo, self.width, self.hq * self.d, self.bits, self.cb, oq, s)

    def accept(self, chosen: torch.Tensor, counts: torch.Tensor) -> None:
        """Keeps counts[s] tokens of each request's last step: `chosen` holds
        their places in the step, request after request, each request's in the
        order of its path. A path's tokens need not have lain side by side: they are
        written again at the positions that follow the context. What else was
        drafted is overwritten by the next step."""
        k, v, plan = self.last
        cu = plan["cu_new"][:-1].long()
        first = torch.cumsum(counts, 0) - counts
        seq = torch.repeat_interleave(torch.arange(counts.numel(), device=counts.device), counts)
        place = cu[seq] + torch.arange(chosen.numel(), device=chosen.device) - first[seq]
        cq.cq_kv_write_slots(self.geom, self.k_cache, self.v_cache, self.cap, k[chosen].contiguous(), v[chosen].contiguous(),
                             plan["slots"][place].contiguous())
        self.lens = self.lens + counts.to(torch.int32)


def random_tree(nodes: int, rng: np.random.RandomState):
    """Parents, depths, and the mask words of a random tree."""
    parent = np.array([rng.randint(-1, i) if i else -1 for i in range(nodes)])
    bits, depth = np.zeros((nodes, 32 * ((nodes + 31) // 32)), dtype=bool), np.zeros(nodes, dtype=np.int32)
    for i in range(nodes):
        if parent[i] >= 0:
            bits[i], depth[i] = bits[parent[i]], depth[parent[i]] + 1
        bits[i, i] = True
    return parent, depth, np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def path_to(node: int, parent) -> list:
    out = []
    while node >= 0:
        out.append(node)
        node = parent[node]
    return out[::-1]


def run(requests: int = 16, context: int = 512, nodes: int = 16, steps: int = 8, seed: int = 0, check: bool = True):
    """Prefills `requests` prompts and verifies `steps` trees of `nodes` drafted
    tokens each, accepting a random path. With `check`, a second layer with
    the same weights gets the accepted tokens one after another; returns the
    largest relative difference of an output, the tokens accepted and the seconds the
    steps took."""
    rng = np.random.RandomState(seed)
    blocks = requests * ((context + steps * nodes + nodes) // BLOCK + 3)
    tree_layer = Layer(requests, blocks, max(requests * 256, requests * nodes), seed)
    line = Layer(requests, blocks, max(requests * 256, requests * nodes), seed) if check else None
    embed = torch.randn(4096, tree_layer.width, generator=torch.Generator().manual_seed(seed + 1)).cuda()
    worst, accepted, spent = 0.0, 0, 0.0
    for at in range(0, context, 256):  # prompts, a chunk at a time
        n = min(256, context - at)
        x = embed[torch.from_numpy(rng.randint(0, 4096, requests * n)).cuda()]
        new = torch.full((requests,), n, dtype=torch.int32, device="cuda")
        every = torch.arange(requests * n, device="cuda")
        for layer in filter(None, (tree_layer, line)):
            layer.step(x, new, max_nodes=n)
            layer.accept(every, new.long())
    for _ in range(steps):
        trees = [random_tree(nodes, rng) for _ in range(requests)]
        tokens = torch.from_numpy(rng.randint(0, 4096, requests * nodes)).cuda()
        mask = torch.from_numpy(np.concatenate([t[2] for t in trees])).cuda()
        depth = torch.from_numpy(np.concatenate([t[1] for t in trees])).cuda()
        new = torch.full((requests,), nodes, dtype=torch.int32, device="cuda")
        paths = [path_to(int(rng.randint(nodes)), t[0]) for t in trees]
        chosen = torch.from_numpy(np.concatenate([np.array(p) + i * nodes for i, p in enumerate(paths)])).cuda()
        counts = torch.tensor([len(p) for p in paths], device="cuda")
        torch.cuda.synchronize()
        began = time.perf_counter()
        y = tree_layer.step(embed[tokens], new, mask, depth, nodes)
        tree_layer.accept(chosen, counts)
        torch.cuda.synchronize()
        spent += time.perf_counter() - began
        accepted += int(counts.sum())
        if line is not None:
            longest = int(counts.max())
            for j in range(longest):  # the j-th token of every path that is that long
                live = [i for i, p in enumerate(paths) if len(p) > j]
                where = torch.tensor([paths[i][j] + i * nodes for i in live], device="cuda")
                one = torch.zeros(requests, dtype=torch.int32, device="cuda")
                one[live] = 1
                z = line.step(embed[tokens[where]], one, max_nodes=1)
                line.accept(torch.arange(len(live), device="cuda"), one.long())
                worst = max(worst, float(((z - y[where]).norm(dim=1) / y[where].norm(dim=1)).max()))
    cq.cq_device_status()
    return worst, accepted, spent


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--context", type=int, default=512)
    ap.add_argument("--nodes", type=int, default=16)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    worst, accepted, spent = run(a.requests, a.context, a.nodes, a.steps)
    print(f"{a.steps} steps of {a.requests} trees of {a.nodes}: {accepted} tokens accepted in {spent * 1e3:.1f} ms; "
          f"against one token at a time an output is off by {worst:.2e} at most")


if __name__ == "__main__":
    main()
