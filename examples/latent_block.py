"""One transformer block on an MI355X: latent attention over a paged cache, then the routed-expert MoE layer.

A prompt goes through the expanded form (append, expand, prefill), the tokens after it through the absorbed form
(append, project, decode, project), each followed by the same MoE layer.  The block's last token is then computed a
second time as part of a longer prompt, and both results are compared: one cache, two ways to read it.

    python examples/latent_block.py [--prompt 200] [--steps 8] [--fp8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_expert_ffn_amd as moe  # noqa: E402
import synth  # noqa: E402
from synth.device import upload_layer  # noqa: E402

HEADS, RANK, NOPE, V, ROPE, PAGE = 8, 256, 128, 128, moe.COLI_MLA_ROPE, 16


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Block:
    """Weights, cache and workspaces of one block for one sequence of up to `limit` tokens."""

    def __init__(self, limit: int, fp8: bool, dtype=torch.bfloat16, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, fan):
            return (torch.randn(shape, generator=g, device="cuda") / fan ** 0.5).to(dtype)
        self.spec, self.dtype, hidden = synth.TINY, dtype, synth.TINY.hidden
        self.w_q = weight(HEADS * (NOPE + ROPE), hidden, fan=hidden)
        self.w_kv_a = weight(RANK + ROPE, hidden, fan=hidden)
        self.w_kv_b = weight(HEADS, NOPE + V, RANK, fan=RANK)
        self.w_o = weight(hidden, HEADS * V, fan=HEADS * V)
        # the absorbed form's halves of w_kv_b, laid out once
        self.w_k_t, self.w_v = self.w_kv_b[:, :NOPE].transpose(1, 2).contiguous(), self.w_kv_b[:, NOPE:].contiguous()
        self.gain = torch.ones(RANK, dtype=dtype, device="cuda")
        self.inv_freq = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
        self.dims = moe.make_mla_dims(HEADS, RANK, NOPE, V, PAGE, dtype, moe.COLI_KV_E4M3 if fp8 else moe.COLI_KV_PLAIN)
        n_pages = -(-limit // PAGE) + 1
        row = moe.coli_mla_row_bytes(self.dims)
        self.pages = (torch.zeros(n_pages, PAGE, row, dtype=torch.uint8, device="cuda") if fp8
                      else torch.zeros(n_pages, PAGE, row // 2, dtype=dtype, device="cuda"))
        self.kv_scale = torch.zeros(n_pages * PAGE, device="cuda") if fp8 else None
        self.table = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
        self.limit, self.length = limit, 0
        self.ws = torch.zeros(moe.coli_mla_workspace_bytes(self.dims, 1, 1, limit), dtype=torch.uint8, device="cuda")
        layer = synth.tiny_layer(seed=seed, S=1)
        self.layer = upload_layer(layer, device="cuda")
        self.moe_dims = moe.make_dims(self.spec)
        self.moe_ws = torch.zeros(moe.coli_moe_workspace_bytes(self.moe_dims, limit), dtype=torch.uint8, device="cuda")

    def _empty(self, *shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device="cuda")

    def _append(self, x, apart: bool):
        """Queries of x's tokens and their rotated part, in place or apart; their latents and keys go into the cache."""
        n = x.shape[0]
        h = norm(x).to(self.dtype)
        q = (h @ self.w_q.t()).view(n, HEADS, NOPE + ROPE)
        at = torch.arange(self.length, self.length + n, device="cuda")
        slots = self.table[0].long()[at // PAGE] * PAGE + at % PAGE
        q_pe = self._empty(n, HEADS, ROPE) if apart else q[..., NOPE:]
        moe.coli_mla_append(self.dims, h @ self.w_kv_a.t(), self.gain, at.to(torch.int32), slots, self.inv_freq,
                            q[..., NOPE:], q_pe, self.pages, self.kv_scale, self.ws)
        self.length += n
        return q, q_pe

    def _finish(self, x, attended):
        """Output projection and residual, then the MoE layer and its residual."""
        n = x.shape[0]
        x = x + (attended.view(n, HEADS * V) @ self.w_o.t()).float()
        h = norm(x).contiguous()
        idx, w = self._empty(n, self.spec.top_k, dtype=torch.int32), self._empty(n, self.spec.top_k, dtype=torch.float32)
        out = torch.empty_like(h)
        moe.coli_moe_layer(self.moe_dims, h, self.layer["router_w"], self.layer["bias"], self.layer["table"],
                           self.layer["shared"], idx, w, out, self.moe_ws)
        return x + out

    def prompt(self, x):
        n = x.shape[0]
        q, _ = self._append(x, apart=False)   # prefill takes whole queries
        kv, k_pe = self._empty(self.length, HEADS, NOPE + V), self._empty(self.length, ROPE)
        cu_q = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        cu_k = torch.tensor([0, self.length], dtype=torch.int32, device="cuda")
        out = self._empty(n, HEADS, V)
        moe.coli_mla_expand(self.dims, self.pages, self.kv_scale, self.table, cu_k, self.w_kv_b, kv, k_pe, self.ws)
        moe.coli_mla_prefill(self.dims, q, kv[..., :NOPE], k_pe, kv[..., NOPE:], cu_q, cu_k, n, True, out, None, self.ws)
        return self._finish(x, out)

    def step(self, x):
        """One token."""
        q, q_pe = self._append(x, apart=True)   # decode takes the parts
        q_lat, o_lat, out = self._empty(1, HEADS, RANK), self._empty(1, HEADS, RANK), self._empty(1, HEADS, V)
        lens = torch.tensor([self.length], dtype=torch.int32, device="cuda")
        moe.coli_mla_project(q[..., :NOPE], self.w_k_t, q_lat)
        moe.coli_mla_decode(self.dims, q_lat, q_pe, self.pages, self.kv_scale, self.table, lens, self.limit, o_lat, None,
                            self.ws)
        moe.coli_mla_project(o_lat, self.w_v, out)
        return self._finish(x, out)

    def check(self):
        for ws in (self.ws, self.moe_ws):
            if moe.coli_moe_status(ws):
                raise RuntimeError(moe.coli_moe_last_error())


def main(argv=None) -> float:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--prompt", type=int, default=200)
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--fp8", action="store_true", help="E4M3 latents in the cache")
    a = p.parse_args(argv)
    n = a.prompt + a.steps
    x = torch.randn(n, synth.TINY.hidden, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    block = Block(n, a.fp8)
    block.prompt(x[:a.prompt])
    for i in range(a.prompt, n):
        stepped = block.step(x[i:i + 1])
    block.check()
    whole = Block(n, a.fp8)
    prompted = whole.prompt(x)[-1:]
    whole.check()
    off = float((stepped - prompted).norm() / prompted.norm())
    print(f"{a.prompt} tokens of prompt, {a.steps} steps: the last token differs by {off:.2e} (relative L2) from the same "
          "token of one longer prompt")
    return off


if __name__ == "__main__":
    sys.exit(0 if main() < 2e-2 else 1)
