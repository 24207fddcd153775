"""Decode steps of one transformer layer on 4-bit records: the projections are
weight-only products with NVFP4 records, the keys and values go to a paged cache (NVFP4 or
bf16), every sequence's new token attends over its pages, and the MLP's weights are MXFP4
records.  The step's launches are captured once and replayed for every token.

    python examples/decode_step.py --cache nvfp4 --batch 16 --prompt 1000 --steps 64
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp4_block_quantization_amd import fos


def random_bf16(rows, cols, scale, gen, device):
    return (scale * torch.randn(rows, cols, generator=gen)).to(device, torch.bfloat16)


def normed(x):
    return torch.nn.functional.rms_norm(x, x.shape[-1:], eps=1e-6)


class Layer:
    """Random weights as records: the fused q, k, v projection and the output projection in
    NVFP4, the two matrices of the MLP in MXFP4."""

    def __init__(self, width, q_heads, kv_heads, head_dim, hidden, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        self.width, self.q_heads, self.kv_heads, self.head_dim = width, q_heads, kv_heads, head_dim
        qkv = (q_heads + 2 * kv_heads) * head_dim
        weight = lambda n, k: random_bf16(n, k, k ** -0.5, gen, device)
        self.w_qkv = fos.quantize(weight(qkv, width))
        self.w_out = fos.quantize(weight(width, q_heads * head_dim))
        self.w_up = fos.mx_quantize(weight(hidden, width))
        self.w_down = fos.mx_quantize(weight(width, hidden))
        self.b_qkv = random_bf16(1, qkv, 0.1, gen, device)[0]

    def project(self, x):
        """q, k, v of x: views of one product, no copies."""
        qkv = fos.wlinear_fwd(normed(x), self.w_qkv, bias=self.b_qkv)
        sizes = [self.q_heads, self.kv_heads, self.kv_heads]
        return [t.unflatten(1, (-1, self.head_dim))
                for t in qkv.split([n * self.head_dim for n in sizes], dim=1)]

    def step(self, x, cache, slots, table, lens, ws):
        """One new token of every sequence.  Returns the layer's output and, by name, what
        was computed on the way."""
        q, k, v = self.project(x)
        fos.kv_append(cache, k, v, slots)
        a = fos.paged_decode(q, cache, table, lens, ws=ws)
        h = x + fos.wlinear_fwd(a.flatten(1), self.w_out)
        u = torch.nn.functional.silu(fos.mx_wlinear_fwd(normed(h), self.w_up))
        y = h + fos.mx_wlinear_fwd(u, self.w_down)
        return y, dict(q=q, k=k, v=v, attention=a, h=h, u=u)


class Pages:
    """Which pages of the cache each sequence holds, on the host, and what the device reads
    of it: block table, lengths and the new tokens' slots (tensors that keep their place,
    so that a captured step sees each new token)."""

    def __init__(self, batch, pages_per_seq, page_size, num_pages, seed=0, device="cuda"):
        self.page_size = page_size
        self.free = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.held = [[] for _ in range(batch)]
        self.count = [0] * batch
        self.table = torch.full((batch, pages_per_seq), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.slots = torch.full((batch,), -1, dtype=torch.int64, device=device)

    def advance(self):
        """Room for one more token of every sequence."""
        slots = []
        for b, held in enumerate(self.held):
            at = self.count[b] % self.page_size
            if at == 0:
                held.append(self.free.pop())
                self.table[b, len(held) - 1] = held[-1]
            slots.append(held[-1] * self.page_size + at)
            self.count[b] += 1
        self.slots.copy_(torch.tensor(slots))
        self.lens.copy_(torch.tensor(self.count, dtype=torch.int32))
        return self.slots


def make_cache(layer, fmt, num_pages, page_size, x):
    """A cache whose tensor scales leave twice the range of the keys and values of x."""
    scales = {}
    if fmt == "nvfp4":
        _, k, v = layer.project(x)
        scales = {name: 2 * fos.tensor_scale(t.flatten(1).contiguous())
                  for name, t in (("k_tensor_scale", k), ("v_tensor_scale", v))}
    return fos.kv_cache(num_pages, page_size, layer.kv_heads, layer.head_dim, fmt, device=x.device,
                        **scales)


class Decoder:
    """A layer, its cache and its pages; ``step(x)`` runs one token, from a graph after the
    first call."""

    def __init__(self, layer, fmt, batch, max_tokens, page_size=64, seed=0, graph=True):
        dev = layer.b_qkv.device
        per_seq = -(-max_tokens // page_size)
        gen = torch.Generator().manual_seed(seed + 1)
        self.layer, self.use_graph = layer, graph
        self.x = torch.zeros(batch, layer.width, dtype=torch.bfloat16, device=dev)
        self.cache = make_cache(layer, fmt, batch * per_seq, page_size,
                                random_bf16(max(batch, 64), layer.width, 1.0, gen, dev))
        self.pages = Pages(batch, per_seq, page_size, batch * per_seq, seed, dev)
        # the graph keeps the workspace, so it is no other call's
        self.ws = fos.paged_decode_workspace(batch, layer.q_heads, layer.kv_heads, layer.head_dim, dev)
        self.graph = self.out = None

    def run(self):
        p = self.pages
        return self.layer.step(self.x, self.cache, p.slots, p.table, p.lens, self.ws)

    def prefill(self, xs):
        """Keys and values of earlier tokens (xs: [tokens, batch, width]), appended for all
        sequences at once, without their attention."""
        slots = torch.stack([self.pages.advance().clone() for _ in range(xs.shape[0])])
        _, k, v = self.layer.project(xs.flatten(0, 1))
        fos.kv_append(self.cache, k, v, slots.flatten())

    def step(self, x):
        self.x.copy_(x)
        self.pages.advance()
        if not self.use_graph:
            return self.run()
        if self.graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.run()                      # what is allocated once, before the capture
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = self.run()
        self.graph.replay()
        return self.out


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--cache", choices=("nvfp4", "bf16"), default="nvfp4")
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=12288)
    ap.add_argument("--q-heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--eager", action="store_true", help="launch every step instead of replaying a graph")
    args = ap.parse_args()
    layer = Layer(args.width, args.q_heads, args.kv_heads, args.head_dim, args.hidden)
    gen = torch.Generator(device="cuda").manual_seed(7)
    d = Decoder(layer, args.cache, args.batch, args.prompt + args.steps + 1, graph=not args.eager)
    tokens = lambda *shape: torch.randn(*shape, args.width, generator=gen, device="cuda").bfloat16()
    for at in range(0, args.prompt, 128):
        d.prefill(tokens(min(128, args.prompt - at), args.batch))
    x = tokens(args.batch)
    x, _ = d.step(x)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(args.steps):
        x, parts = d.step(x)
    end.record()
    torch.cuda.synchronize()
    assert x.isfinite().all()
    print(f"{args.cache} cache, {args.batch} sequences of {d.pages.count[0]} tokens: "
          f"{1e3 * start.elapsed_time(end) / args.steps:.1f} us per step of the layer, "
          f"host work included")


if __name__ == "__main__":
    main()
