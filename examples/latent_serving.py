"""A serving loop over one KDA layer and one latent-attention layer.

Prompts of different lengths are taken in packed: block tables and slot maps are
planned on the GPU, the KDA layer runs its chunked form and keeps its states,
the latent layer writes its rows into the paged cache and attends in the
expanded form.  Then tokens are decoded one a request and step: the KDA layer
updates its states in place, the latent layer appends a row a request and
attends in the absorbed form over the cache.  Weights and tokens are random.
With several samples a prompt, each prompt is forked: its samples share the
prompt's pages, and decoding reads a prompt once for all of them.

    python examples/latent_serving.py [--requests 8] [--longest 700] [--steps 16] [--heads 8] [--samples 1]

At the end the last step's latent attention is computed once more for whole
sequences in the expanded form and compared: both forms state the same function.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kimi_delta_attention_05_gb300 import (get_status, kda_fwd, kda_fwd_recurrent, latent_append,  # noqa: E402
                                           latent_decode, latent_decode_shared, latent_fork, latent_plan,
                                           latent_prefill, latent_release)

PAGE = 64


class Layers:
    """Random weights of the two mixers (no feed-forward part, no norms between)."""

    def __init__(self, width, heads, device, gen):
        def w(*shape):
            return (torch.randn(shape, generator=gen, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.heads = heads
        self.kda_in = w(4 * heads * 128 + heads, width)      # q, k, v, g, beta
        self.kda_out = w(width, heads * 128)
        self.a_log = torch.rand(heads, generator=gen, device=device)
        self.dt_bias = torch.randn((heads, 128), generator=gen, device=device) * 0.1
        self.q = w(heads * 192, width)
        self.latent = w(576, width)                          # latents and shared key part
        self.norm = torch.ones(512, device=device)
        self.up = w(heads, 256, 512)                         # keys (128) and values (128) of a head from the latent
        self.out = w(width, heads * 128)

    def kda(self, x, states, cu=None):
        """x [B, T, width] (packed with cu); states [N, H, 128, 128] updated in place."""
        B, T, _ = x.shape
        H = self.heads
        y = x @ self.kda_in.T
        q, k, v, g = (y[..., i * H * 128:(i + 1) * H * 128].reshape(B, T, H, 128).contiguous() for i in range(4))
        beta = y[..., 4 * H * 128:].contiguous()
        # one token updates the states in place; the chunked form reads its initial states from a buffer of their own
        call, initial = (kda_fwd_recurrent, states) if T == 1 else (kda_fwd, states.clone())
        out = call(q, k, v, g, beta, 128 ** -0.5, A_log=self.a_log, dt_bias=self.dt_bias, lower_bound=-5.0,
                   initial_state=initial, final_state=states, cu_seqlens=cu, qk_l2norm=True)
        return x + out.reshape(B, T, -1) @ self.kda_out.T

    def queries(self, x):
        return (x @ self.q.T).reshape(*x.shape[:-1], self.heads, 192)

    def store(self, x, slot_map, cache):
        rows = x.reshape(-1, x.shape[-1]) @ self.latent.T
        latent_append(rows[:, :512], rows[:, 512:], slot_map, cache, self.norm)

    def expanded(self, x, rows, cu):
        """Latent attention of packed prompts from their cache rows [T, 576]."""
        kv = torch.einsum("tc,hdc->thd", rows[:, :512], self.up)
        o = latent_prefill(self.queries(x), kv[None, :, :, :128], rows[None, :, 512:], kv[None, :, :, 128:], 192 ** -0.5,
                           cu_seqlens=cu)
        return o.reshape(*x.shape[:2], -1) @ self.out.T

    def absorbed(self, x, cache, table, lens, groups=None):
        """Latent attention of the newest token of every request, x [B, 1, width]; groups: offsets of the requests that
        share a prompt, and the prompts' lengths."""
        q = self.queries(x)
        q = torch.cat([torch.einsum("brhd,hdc->brhc", q[..., :128], self.up[:, :128]), q[..., 128:]], -1).contiguous()
        if groups is None:
            o = latent_decode(q, cache, table, lens, 192 ** -0.5)
        else:
            o = latent_decode_shared(q, cache, table, lens, *groups, 192 ** -0.5)
        o = torch.einsum("brhc,hdc->brhd", o, self.up[:, 128:])
        return o.reshape(*x.shape[:2], -1) @ self.out.T


def serve(requests=8, longest=700, steps=16, heads=8, width=512, seed=0, samples=1):
    """Runs the loop; returns the last step's latent-attention output [requests * samples, width] and
    what the expanded form gives for the same tokens."""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    layers = Layers(width, heads, dev, gen)
    lens = torch.randint(1, longest + 1, (requests,), generator=gen, device=dev, dtype=torch.int32)
    tokens, n = int(lens.sum()), requests * samples  # prompt p is row p * samples, its other samples the rows behind
    pages = samples * sum(-(-(x + steps) // PAGE) for x in lens.tolist())
    cache = torch.empty((pages, PAGE, 576), dtype=torch.bfloat16, device=dev)
    free = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    shares = torch.zeros(pages, dtype=torch.int32, device=dev)
    table = torch.zeros((n, -(-(longest + steps) // PAGE)), dtype=torch.int32, device=dev)
    states = torch.zeros((requests, heads, 128, 128), device=dev)

    def sample(n):
        return torch.randn((1, n, width), generator=gen, device=dev).to(torch.bfloat16)

    # ---- prompts, packed ----
    plan = latent_plan(torch.zeros_like(lens), lens, table[::samples], free, PAGE, tokens)
    x = layers.kda(sample(tokens), states, plan["cu_seqlens"])
    layers.store(x, plan["slot_map"], cache)
    rows = cache.view(-1, 576)[plan["slot_map"]]
    x + layers.expanded(x, rows, plan["cu_seqlens"])  # what the next layer would get
    inputs = [p for p in torch.split(x[0], lens.tolist()) for _ in range(samples)]
    free = free[int(plan["pages_taken"]):]

    # ---- samples of a prompt go on from it: pages shared, the last one copied, and the KDA layer's states ----
    groups, cached = None, plan["seq_lens"]
    if samples > 1:
        row = torch.arange(n, dtype=torch.int32, device=dev)
        children = row[row % samples != 0]
        cached = torch.zeros(n, dtype=torch.int32, device=dev)
        cached[::samples] = lens
        fork = latent_fork(children // samples * samples, children, cached, table, free, shares, cache)
        cached, free = fork["seq_lens"], free[int(fork["pages_taken"]):]
        states = states.repeat_interleave(samples, 0)
        groups = torch.arange(0, n + 1, samples, device=dev), lens

    # ---- decoding ----
    one = torch.ones(n, dtype=torch.int32, device=dev)
    for _ in range(steps):
        plan = latent_plan(cached, one, table, free, PAGE, n, shares=shares)
        cached = plan["seq_lens"]
        x = layers.kda(sample(n).view(n, 1, width), states)
        layers.store(x, plan["slot_map"], cache)
        y = layers.absorbed(x, cache, table, cached, groups)
        free = free[int(plan["pages_taken"]):]
        inputs = [torch.cat([a, b]) for a, b in zip(inputs, x)]

    # ---- the last step once more, expanded over whole sequences ----
    total = plan["seq_lens"].long()
    cu = torch.cat([total.new_zeros(1), total.cumsum(0)])
    packed = torch.cat(inputs)[None]
    at = torch.arange(int(total.max()), device=dev)
    slots = table[:, at // PAGE].long() * PAGE + at % PAGE
    rows = cache.view(-1, 576)[slots[at[None, :] < total[:, None]]]
    again = layers.expanded(packed, rows, cu)[0, cu[1:] - 1]

    # ---- all requests end: every page is free again ----
    gone = latent_release(torch.arange(n, dtype=torch.int32, device=dev), cached, table, shares, PAGE)
    assert int(gone["count"]) + free.numel() == pages and get_status() == 0
    return y[:, 0], again


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("requests", 8), ("longest", 700), ("steps", 16), ("heads", 8), ("samples", 1)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    y, again = serve(a.requests, a.longest, a.steps, a.heads, samples=a.samples)
    off = (y.double() - again.double()).norm() / again.double().norm()
    print(f"{a.requests} requests, {a.steps} steps: absorbed against expanded, relative RMS {off:.2e}")


if __name__ == "__main__":
    main()
