"""Softmax-attention layers beside the GDN layers: the step executor of their paged
8-bit cache, and greedy generation through a hybrid synthetic stack.

An engine step of the attention layers (``PagedAttentionLayers``):

* once per step, ``begin_step``: the block tables, positions and page pieces of the
  step's tokens and the row tiles of its attention, built on the device from the
  sequences' lengths and reused by every layer;
* per layer, ``layer``: rotary positions on q and k with the append of k and v to the
  layer's cache (one launch), then causal attention over it.

``HybridServingStack`` is the synthetic stack of ``serving`` with every fourth layer an
attention layer. Its q, k and v are, like the GDN layers' inputs, slices of the
normalised stream x = (q | k | v | rest); its output takes the place of the delta
rule's in the residual.

    python -m gated_deltanet_linear_build_gb300.hybrid [--sequences N] [--decode STEPS]
"""
from __future__ import annotations

import argparse
import time

import torch

from . import gdn
from .serving import SyntheticServingStack


def _blocks(tokens: int, block_tokens: int) -> int:
    return -(-tokens // block_tokens)


class PagedAttentionLayers:
    """Caches of ``layers`` attention layers for ``n_seqs`` sequences.

    A sequence's tokens lie in blocks of ``block_tokens`` that all layers number alike:
    ``num_blocks`` of them are handed out as sequences grow (lowest free numbers first)
    and come back with ``release``. The host keeps the lengths and the free list; the
    block tables themselves are built on the device.
    """

    def __init__(self, layers: int, n_seqs: int, *, num_blocks: int, max_seq_tokens: int,
                 hq: int = 16, hk: int = 2, d: int = 256, rot_dim: int = 64, base: float = 1.0e7,
                 block_tokens: int = 64, max_step_tokens: int = 2048, device="cuda"):
        dev = torch.device(device)
        self.device, self.layers, self.n_seqs = dev, layers, n_seqs
        self.hq, self.hk, self.d, self.block_tokens = hq, hk, d, block_tokens
        self.scale = d ** -0.5
        self.max_step_tokens = max_step_tokens
        self.width = _blocks(max_seq_tokens, block_tokens)
        cache = (layers, num_blocks, hk, block_tokens, d)
        self.k_cache = torch.zeros(cache, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        self.v_cache = torch.zeros(cache, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        self.k_scale = torch.zeros((layers, num_blocks, hk), device=dev)
        self.v_scale = torch.zeros((layers, num_blocks, hk), device=dev)
        self.phases = gdn.rotary_phases(rot_dim, base, device=dev)

        def ints(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device=dev)
        self.table = ints(n_seqs, self.width)
        self.kv_lens, self.counts = ints(n_seqs), ints(2)
        self.positions = ints(max_step_tokens)
        self.slots = ints(max_step_tokens, dtype=torch.int64)
        self.pieces = ints(max_step_tokens // block_tokens + 2 * n_seqs, 4)
        self.q_rot = torch.empty((max_step_tokens, hq, d), dtype=torch.bfloat16, device=dev)
        ws = gdn.paged_attention_workspace_size(max_step_tokens, n_seqs, hq, hk, d)
        self.workspace = torch.empty((ws,), dtype=torch.uint8, device=dev)
        self.context = [0] * n_seqs
        self.blocks = [[] for _ in range(n_seqs)]
        self.free = list(range(num_blocks))
        self.tokens = self.longest = 0
        self.cu = None

    def begin_step(self, new):
        """Open a step of new[n] tokens for each sequence n, packed in that order."""
        new = [int(l) for l in new]
        if len(new) != self.n_seqs or min(new) < 0 or sum(new) > self.max_step_tokens:
            raise ValueError(f"a step takes {self.n_seqs} lengths of {self.max_step_tokens} tokens in all")
        after = [c + l for c, l in zip(self.context, new)]
        need = [_blocks(a, self.block_tokens) - len(b) for a, b in zip(after, self.blocks)]
        if max(_blocks(a, self.block_tokens) for a in after) > self.width:
            raise ValueError(f"a sequence holds {self.width * self.block_tokens} tokens at most")
        if sum(need) > len(self.free):
            raise RuntimeError(f"the step takes {sum(need)} blocks, {len(self.free)} are free")
        self.tokens, self.longest = sum(new), max(new)
        cu = [0]
        for l in new:
            cu.append(cu[-1] + l)
        taken = self.free[:sum(need)]
        # One copy for all lengths: cu_seqlens, context lengths, the blocks to take.
        lens = torch.tensor(cu + self.context + taken, dtype=torch.int32).to(self.device)
        N, T = self.n_seqs, self.tokens
        self.cu = lens[:N + 1]
        gdn.build_block_tables(self.cu, lens[N + 1:2 * N + 1], lens[2 * N + 1:], self.table, self.kv_lens,
                               self.positions[:T], self.slots[:T], self.pieces, self.counts,
                               block_tokens=self.block_tokens)
        gdn.paged_attention_plan(self.cu, self.kv_lens, self.workspace, T=T, Hq=self.hq, Hk=self.hk, d=self.d,
                                 block_tokens=self.block_tokens, max_blocks=self.width,
                                 max_new_tokens=self.longest)
        for n, m in enumerate(need):
            self.blocks[n] += taken[:m]
            taken = taken[m:]
        self.free = self.free[sum(need):]
        self.context = after

    def layer(self, l: int, q, k, v, out):
        """Layer l of the open step: q [T, hq, d], k and v [T, hk, d] BF16 (rows may be
        views of a wider row) into out [T, hq, d]."""
        T = self.tokens
        q_rot = self.q_rot[:T]
        gdn.rotary_kv_append(q, k, v, self.positions[:T], self.phases, self.pieces, self.counts, q_rot,
                             self.k_cache[l], self.v_cache[l], self.k_scale[l], self.v_scale[l])
        gdn.paged_attention(q_rot, self.k_cache[l], self.v_cache[l], self.k_scale[l], self.v_scale[l],
                            self.table, self.cu, self.kv_lens, out, self.workspace,
                            softmax_scale=self.scale, max_new_tokens=self.longest, planned=True)

    def release(self, seq: int):
        """Give the sequence's blocks back; its slot begins an empty sequence."""
        self.free = sorted(self.free + self.blocks[seq])
        self.blocks[seq] = []
        self.context[seq] = 0


class HybridServingStack(SyntheticServingStack):
    """The synthetic stack with attention at layers every - 1, 2 every - 1, ...

    ``hq`` heads of width ``d_attn`` make up the same output width as the GDN layers'
    hv heads of width d."""

    def __init__(self, weights, device="cuda", budget: int = 2048, *, every: int = 4, hq: int = 16, hk: int = 2,
                 d_attn: int = 256, rot_dim: int = 64, block_tokens: int = 64):
        super().__init__(weights, device, budget)
        if hq * d_attn != self.hv * self.d or (hq + 2 * hk) * d_attn > self.C:
            raise ValueError("the attention heads do not fit the stream")
        self.every = every
        self.attn_sizes = dict(hq=hq, hk=hk, d=d_attn, rot_dim=rot_dim, block_tokens=block_tokens)
        self.attn = None

    def _is_attention(self, l):
        return (l + 1) % self.every == 0

    def _begin_run(self, n_decode):
        B = self.attn_sizes["block_tokens"]
        most = [len(p) + n_decode for p in self.prompts]
        self.attn = PagedAttentionLayers(self.layers // self.every, self.n_seqs,
                                         num_blocks=sum(_blocks(m, B) for m in most), max_seq_tokens=max(most),
                                         max_step_tokens=max(self.budget, self.n_seqs), device=self.device,
                                         **self.attn_sizes)

    def _begin_step(self, new):
        self.attn.begin_step(new)

    def _attention(self, l, x, o):
        T, hq, hk, d = x.shape[0], self.attn.hq, self.attn.hk, self.attn.d
        q, k, v = (t.unflatten(1, (-1, d)) for t in x[:, :(hq + 2 * hk) * d].split([hq * d, hk * d, hk * d], 1))
        self.attn.layer(l // self.every, q, k, v, o.view(T, hq, d))

    def _prefill_mix(self, stack, l, cu_d, has_d, first, n, x, y, o):
        if self._is_attention(l):
            self._attention(l, x, o)
        else:
            super()._prefill_mix(stack, l, cu_d, has_d, first, n, x, y, o)

    def _decode_mix(self, stack, l, x, y, o):
        if self._is_attention(l):
            self._attention(l, x, o)
        else:
            super()._decode_mix(stack, l, x, y, o)


def main(argv=None):
    from . import synth
    ap = argparse.ArgumentParser(description="greedy generation through the hybrid synthetic stack")
    ap.add_argument("--sequences", type=int, default=32)
    ap.add_argument("--decode", type=int, default=64)
    args = ap.parse_args(argv)
    stack = HybridServingStack(synth.serving_stack(4, n_seqs=args.sequences))
    stack.generate(2)                                            # warm-up
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    ids, _ = stack.generate(args.decode)
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    tokens = sum(len(p) for p in stack.prompts) + args.decode * args.sequences
    print(f"{stack.layers} layers, {stack.attn.layers} of them attention; {args.sequences} sequences, "
          f"{tokens} tokens in {dt:.2f} s; first ids {ids[0, :8].tolist()}")


if __name__ == "__main__":
    main()
