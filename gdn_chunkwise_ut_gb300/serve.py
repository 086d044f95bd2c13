"""A Gated DeltaNet layer served from a pool of states: prompts, samples forked from one, decode steps.

    python -m gdn_chunkwise_ut_gb300.serve

``GdnLayer`` runs the operators together as a server does.  A prompt goes through the norm, the
projection, ``gdn_prep_fwd``, the chunked delta rule and the gated norm, and leaves its states in its
slot; a decode step takes the same way with ``gdn_recurrent_fwd`` in the chunked rule's place, and is
the same kernels at fixed addresses each time, so that it can be captured into a CUDA graph.  The
projections are one plain matrix product, whose parts the operators read in place; random weights.
"""
from __future__ import annotations

import argparse
import time

import torch

from .api import chunk_gated_delta_rule
from .layer import add_rms_norm_fwd, gated_rms_norm_fwd, gdn_prep_fwd, gdn_recurrent_fwd, gdn_state_copy
from .pool import StatePool


class GdnLayer:
    """One layer of ``dim`` channels with Hk key heads and Hv value heads of 128, random weights."""

    def __init__(self, dim: int = 2048, Hk: int = 16, Hv: int = 32, *, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.dim, self.Hk, self.Hv, self.d, self.taps = dim, Hk, Hv, 128, 4
        D = (2 * Hk + Hv) * self.d

        def randn(*shape, scale=1.0, dtype=torch.bfloat16):
            return (scale * torch.randn(shape, generator=gen, device=device, dtype=torch.float32)).to(dtype)

        self.norm = 1.0 + randn(dim, scale=0.1)
        # one product for all projections, cut into the convolution's channels, the gates' inputs and z
        # (padded so that z, and the next token's channels, begin on 16 bytes)
        self.parts = [D, Hv, Hv, -2 * Hv % 8, Hv * self.d]
        self.proj = randn(dim, sum(self.parts), scale=dim ** -0.5)
        self.conv = randn(D, self.taps, scale=0.5)
        self.A_log = torch.log(1.0 + 15.0 * torch.rand(Hv, generator=gen, device=device))
        self.dt_bias = randn(Hv, dtype=torch.float32) - 4.0
        self.out_norm = 1.0 + randn(self.d, scale=0.1)
        self.out = randn(Hv * self.d, dim, scale=(Hv * self.d) ** -0.5)

    def pool(self, num_slots: int) -> StatePool:
        return StatePool(num_slots, 1, self.Hk, self.Hv, self.d, self.d, taps=self.taps, device=self.proj.device)

    def _inputs(self, x, residual, pool, slots, cu_seqlens, expand):
        h, _, residual = add_rms_norm_fwd(x, self.norm, residual)
        qkv, a, b, _, z = (h @ self.proj).split(self.parts, dim=-1)
        q, k, v, g, beta = gdn_prep_fwd(qkv, self.conv, a, b, self.A_log, self.dt_bias, pool.convs[0], Hk=self.Hk,
                                        Hv=self.Hv, dk=self.d, dv=self.d, slots=slots, cu_seqlens=cu_seqlens,
                                        expand=expand)
        return z.unflatten(-1, (self.Hv, self.d)), residual, q, k, v, g, beta

    def _outputs(self, o, z):
        y, _ = gated_rms_norm_fwd(o, z, self.out_norm)
        return y.flatten(-2) @ self.out

    def prefill(self, x, residual, pool: StatePool, slots, cu_seqlens):
        """Packed prompts x, residual [1, T, dim]: returns (output, new residual); the slots take the
        prompts' states on from the ones that they hold."""
        z, residual, q, k, v, g, beta = self._inputs(x, residual, pool, slots, cu_seqlens, True)
        n = slots.shape[0]
        first = torch.arange(n, dtype=torch.int32, device=x.device)
        state = torch.empty((n, self.Hv, self.d, self.d), dtype=torch.float32, device=x.device)
        gdn_state_copy(state, first, pool.states[0], slots)
        o, final = chunk_gated_delta_rule(q, k, v, g, beta, initial_state=state, output_final_state=True,
                                          cu_seqlens=cu_seqlens)
        gdn_state_copy(pool.states[0], slots, final, first)
        return self._outputs(o, z), residual

    def decode(self, x, residual, pool: StatePool, slots):
        """One token a sequence, x, residual [N, 1, dim]: returns (output, new residual)."""
        z, residual, q, k, v, g, beta = self._inputs(x, residual, pool, slots, None, False)
        o = gdn_recurrent_fwd(q, k, v, beta, pool.states[0], g=g, slots=slots)
        return self._outputs(o, z), residual


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", type=int, default=16)
    ap.add_argument("--samples", type=int, default=4, help="samples forked from each prompt")
    ap.add_argument("--tokens", type=int, default=512, help="tokens of a prompt")
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args()
    layer = GdnLayer()
    n = args.prompts * args.samples
    pool = layer.pool(n)
    prompts = pool.alloc(args.prompts)
    x = torch.randn((1, args.prompts * args.tokens, layer.dim), device="cuda").to(torch.bfloat16)
    cu = torch.arange(args.prompts + 1, device="cuda", dtype=torch.int32) * args.tokens
    layer.prefill(x, x, pool, pool.index(prompts), cu)
    slots = pool.index([s for p in prompts for s in [p] + pool.fork(p, args.samples - 1)])

    x = torch.randn((n, 1, layer.dim), device="cuda").to(torch.bfloat16)
    residual = torch.zeros_like(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.decode(x, residual, pool, slots)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            layer.decode(x, residual, pool, slots)
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(args.steps):
        graph.replay()
    torch.cuda.synchronize()
    us = (time.perf_counter() - began) / max(1, args.steps) * 1e6
    print(f"{args.prompts} prompts of {args.tokens} tokens, {n} sequences: {us:.1f} us a decode step")


if __name__ == "__main__":
    main()
