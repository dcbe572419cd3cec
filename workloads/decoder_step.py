"""The attention half of a text decoder, one token per request and step, as a
server runs it: int4 q, k and v products, the step's block tables and slot
maps, the append to a paged cache, attention over the cache, the int4 o
product; and the same against an encoder's states (q product, cross attention,
o product). Synthetic weights and states, no norms and no MLP.

    python -m workloads.decoder_step [--batch 8] [--steps 16]

prints the time of a step and how many blocks its requests hold. Sizes
are Whisper-small's decoder (width 768, 12 heads of 64, 12 layers, block 64;
"sherpa-onnx STT int4", section "whisper-small") over the 1500 frames of its
encoder.
"""

import argparse

import torch

from block_wise_int4_amd import mnb

WIDTH, HEADS, DIM, LAYERS, BLOCK, FRAMES = 768, 12, 64, 12, 64, 1500


def packed(n, k, gen, device):
    w = torch.randn((n, k), generator=gen, device=device) * 0.02
    q, s, z = mnb.mnb_quantize_rtn(w, BLOCK, torch.float16)
    return mnb.mnb_pack(q, s, z, n, k, BLOCK)


class Layer:
    def __init__(self, gen, device, blocks, page):
        self.q, self.k, self.v, self.o, self.cross_q, self.cross_k, self.cross_v, self.cross_o = (
            packed(WIDTH, WIDTH, gen, device) for _ in range(8))
        self.cache = mnb.KvCache.new(blocks, HEADS, page, DIM, torch.float16, device)
        self.states = None      # the encoder's keys and values, projected once

    def encode(self, states):
        B, T, _ = states.shape
        rows = states.reshape(B * T, WIDTH)
        self.states = [mnb.mnb_gemm(rows, w).view(B, T, HEADS, DIM) for w in (self.cross_k, self.cross_v)]

    def append(self, x, slots):
        mnb.mnb_kv_append(mnb.mnb_gemm(x, self.k).view(-1, HEADS, DIM), mnb.mnb_gemm(x, self.v).view(-1, HEADS, DIM),
                          slots, self.cache)


class Decoder:
    """Requests that share a paged cache. `tokens` bounds a request's length."""

    def __init__(self, batch, tokens, page=16, layers=LAYERS, seed=0, device="cuda"):
        self.batch, self.page, self.device = batch, page, device
        gen = torch.Generator(device).manual_seed(seed)
        width = -(-tokens // page)
        self.max_len = width * page
        self.layers = [Layer(gen, device, batch * width, page) for _ in range(layers)]
        i32 = dict(dtype=torch.int32, device=device)
        self.free = torch.randperm(batch * width, generator=gen, device=device).to(torch.int32)
        self.table = torch.full((batch, width), -1, **i32)
        self.lens = torch.zeros(batch, **i32)
        self.host_lens = [0] * batch
        q = torch.empty((batch, HEADS, DIM), dtype=torch.float16, device=device)
        self.work = mnb.paged_attn_workspace(q, self.layers[0].cache, self.max_len)
        self.cross_work = None

    def encode(self, states, lens):
        """An encoder's states [batch, frames, width], lens [batch] valid each."""
        for layer in self.layers:
            layer.encode(states)
        self.frames = lens
        q = torch.empty((self.batch, 1, HEADS, DIM), dtype=torch.float16, device=self.device)
        self.cross_work = mnb.cross_attn_workspace(q, self.layers[0].states[0])

    def place(self, added):
        """Room for added[b] new tokens of each request: the tables' new
        entries, the lengths, and the slot of each token. The host follows the
        lengths, so that it knows what was taken without waiting for it."""
        if any(held + n > self.max_len for held, n in zip(self.host_lens, added)):
            raise ValueError(f"a request holds at most {self.max_len} tokens")
        slots = torch.empty(sum(added), dtype=torch.int64, device=self.device)
        lens, *_ = mnb.mnb_kv_tables(self.lens, torch.tensor(added, dtype=torch.int32, device=self.device), self.free,
                                     self.table, self.page, slots)
        taken = 0
        for b, n in enumerate(added):
            taken += -(-(self.host_lens[b] + n) // self.page) - -(-self.host_lens[b] // self.page)
            self.host_lens[b] += n
        self.free, self.lens = self.free[taken:], lens
        return slots

    def prompt(self, x, added):
        """Keys and values of prompts, x [sum(added), width]. Attention among a
        prompt's rows is not among the operators over this cache (it is over the
        one in 8 bits, mnb_paged_attn_i8): every layer is given the embeddings x,
        where a model would give it the layer before's output."""
        slots = self.place(added)
        for layer in self.layers:
            layer.append(x, slots)

    def step(self, x):
        """One new token of each request, x [batch, width]."""
        slots = self.place([1] * self.batch)
        for layer in self.layers:
            layer.append(x, slots)
            q = mnb.mnb_gemm(x, layer.q).view(self.batch, HEADS, DIM)
            a = mnb.mnb_paged_attn(q, layer.cache, self.table, self.lens, self.max_len,
                                   workspace=self.work)
            x = x + mnb.mnb_gemm(a.view(self.batch, WIDTH), layer.o)
            q = mnb.mnb_gemm(x, layer.cross_q).view(self.batch, 1, HEADS, DIM)
            a = mnb.mnb_cross_attn(q, *layer.states, self.frames, workspace=self.cross_work)
            x = x + mnb.mnb_gemm(a.view(self.batch, WIDTH), layer.cross_o)
        return x


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--steps", type=int, default=16)
    args = ap.parse_args()
    gen = torch.Generator("cuda").manual_seed(1)
    half = dict(dtype=torch.float16, device="cuda", generator=gen)
    prompts = [4 + 7 * b % 60 for b in range(args.batch)]
    d = Decoder(args.batch, max(prompts) + args.steps + 4)
    d.encode(torch.randn((args.batch, FRAMES, WIDTH), **half),
             torch.tensor([FRAMES - 150 * (b % 8) for b in range(args.batch)], dtype=torch.int32, device="cuda"))
    d.prompt(torch.randn((sum(prompts), WIDTH), **half), prompts)
    xs = [torch.randn((args.batch, WIDTH), **half) for _ in range(args.steps)]   # the new tokens' embeddings
    for x in xs[:4]:
        d.step(x)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for x in xs:
        x = d.step(x)
    b.record()
    torch.cuda.synchronize()
    ms = a.elapsed_time(b) / args.steps
    print(f"{args.batch} requests, {LAYERS} layers: {ms:.3f} ms per step, {1e3 * args.batch / ms:.0f} tokens/s, "
          f"lengths {min(d.host_lens)}..{max(d.host_lens)}, {int((d.table >= 0).sum())} blocks, "
          f"finite {bool(torch.isfinite(x).all())}")


if __name__ == "__main__":
    main()
