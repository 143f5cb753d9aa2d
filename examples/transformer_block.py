"""One transformer block on an MI355X, every linear in low precision:

    h, codes = norm(x)                svdq_add_rmsnorm, INT8 codes and row scales
    q, k, v  = codes W_qkv + b        svdq_gemm_act_residual
    q, k     = turn(norm(q)), ...     svdq_rope_axes, three axes (time, height, width)
    x        = attn(q, k, v) W_o + b + x      svdq_gemm_act_residual in fp16, residual in the epilogue
    h        = norm(x) / lambda_1     svdq_add_rmsnorm, 16-bit output, the smoothing folded into its weight
    y        = fc2(gelu(fc1(h)))      svdq_linear_folded and svdq_linear, W4A4 with their low-rank branches
    x        = x + y                  the next block's svdq_add_rmsnorm

The attention between is torch's, of all tokens to all.  With a paged cache of keys and values the block
takes a step's tokens of several sequences instead, each seeing what came before it:

    q        = turn(norm(q)); k, v to the cache          svdq_rope_append
    a        = attn(q, the sequence's cache)             svdq_tree_attention, a chain or a tree of drafted tokens
    the tokens kept of a draft, moved together           svdq_cache_keep, once for all blocks' caches

Weights are random.

    python examples/transformer_block.py            # sizes of a 3072-wide block, 4608 tokens
    python examples/transformer_block.py --cached   # prompts, a drafted tree and its accepted path
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_w4a4_quantized_amd import binding, prepare  # noqa: E402


class Block:
    def __init__(self, dim, heads, ffn, axis_pairs, seed=0, rank=32, w4="int4_e2m3", w8="int8"):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.dim, self.heads, self.axis_pairs, self.w4, self.w8 = dim, heads, axis_pairs, w4, w8
        d = dim // heads
        self.raw = {"n1": 1 + 0.1 * rand(dim), "n2": 1 + 0.1 * rand(dim), "qn": 1 + 0.1 * rand(d), "kn": 1 + 0.1 * rand(d),
                    "wqkv": rand(3 * dim, dim) / dim ** 0.5, "bqkv": 0.1 * rand(3 * dim),
                    "wo": rand(dim, dim) / dim ** 0.5, "bo": 0.1 * rand(dim),
                    "w1": rand(dim, ffn) / dim ** 0.5, "b1": 0.1 * rand(ffn), "w2": rand(ffn, dim) / ffn ** 0.5,
                    "b2": 0.1 * rand(dim)}
        r = self.raw
        self.n1, self.qn, self.kn = r["n1"].cuda(), r["qn"].cuda(), r["kn"].cuda()
        codes, scales = prepare.quantize_rows(r["wqkv"], w8)
        self.wqkv, self.wqkv_s = codes.cuda(), scales.cuda()
        self.bqkv, self.wo, self.bo = (r[n].half().cuda() for n in ("bqkv", "wo", "bo"))
        self.freq = prepare.rope_frequencies(axis_pairs).cuda()
        # the W4A4 pair, calibrated on normed activations and on what fc1 makes of them
        cal = rand(256, dim) * r["n2"]
        mid = torch.nn.functional.gelu(cal @ r["w1"] + r["b1"], approximate="tanh")
        layer = lambda c, w, b: prepare.prepare_host(c.numpy(), w.numpy(), b.numpy().astype(np.float16), rank)  # noqa: E731
        self.h1, self.h2 = layer(cal, r["w1"], r["b1"]), layer(mid, r["w2"], r["b2"])
        self.fc1, self.fc2 = prepare.to_device(self.h1, w4), prepare.to_device(self.h2, w4)
        # fc1's smoothing divides its input's channels: folded into the norm's weight
        self.n2 = (r["n2"] / torch.from_numpy(self.h1.lam)).cuda()

    def __call__(self, x, y, positions, cache=None, batch=None, tree=None):
        """x fp16 [T, dim], the stream; y the previous block's MLP output (or None); returns (x, y).  With cache
        and batch the tokens are a step's, appended to their sequences."""
        T, D, H = x.shape[0], self.dim, self.heads
        codes, scales, stream = binding.svdq_add_rmsnorm(x if y is None else y, self.n1, residual=None if y is None else x,
                                                         out_format=self.w8)
        x = x if stream is None else stream
        qkv = binding.svdq_gemm_act_residual(codes, self.wqkv, scales, self.wqkv_s, self.bqkv)
        heads = lambda i: qkv[:, i * D:(i + 1) * D].unflatten(-1, (H, D // H))  # noqa: E731
        if cache is not None:
            q = binding.svdq_rope_append(cache, batch, heads(0), heads(1), heads(2), positions, self.freq, self.axis_pairs,
                                         q_weight=self.qn, k_weight=self.kn)
            a = binding.svdq_tree_attention(cache, batch, q, tree=tree).view(T, D)
        else:
            q, k = binding.svdq_rope_axes(heads(0), heads(1), positions, self.freq, self.axis_pairs, q_weight=self.qn,
                                          k_weight=self.kn, heads_first=True)
            a = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], heads(2).transpose(0, 1)[None])
            a = a[0].transpose(0, 1).reshape(T, D)
        x = binding.svdq_gemm_act_residual(a, self.wo, bias=self.bo, residual=x)
        h, _, _ = binding.svdq_add_rmsnorm(x, self.n2, out_format="same")
        f1, f2 = self.fc1, self.fc2
        h = binding.svdq_linear_folded(h, None, f1.l1t, f1.wq, f1.ws, f1.l2, f1.bias, f2.lam, self.w4)
        return x, binding.svdq_linear(h, f2.l1t, f2.wq, f2.ws, f2.l2, f2.bias, self.w4)

    def plain(self, x, y, positions):
        """The same block from the unquantized weights in fp32, on the CPU."""
        r, D, H = self.raw, self.dim, self.heads
        norm = lambda v, w: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
        x = x.cpu().float() + (0 if y is None else y.cpu().float())
        q, k, v = (norm(x, r["n1"]) @ r["wqkv"].T + r["bqkv"]).unflatten(-1, (3, H, D // H)).unbind(-3)
        axis = sum(([i] * n for i, n in enumerate(self.axis_pairs)), [])
        angle = positions.cpu().float()[:, axis] * self.freq.cpu()
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        turned = lambda u, w: torch.view_as_real(  # noqa: E731
            torch.view_as_complex(norm(u, w).unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        q, k = turned(q, r["qn"]).transpose(0, 1), turned(k, r["kn"]).transpose(0, 1)
        a = torch.softmax(q @ k.transpose(-1, -2) / (D // H) ** 0.5, -1) @ v.transpose(0, 1)
        x = x + a.transpose(0, 1).flatten(1) @ r["wo"].T + r["bo"]
        h = torch.nn.functional.gelu(norm(x, r["n2"]) @ r["w1"] + r["b1"], approximate="tanh")
        return x, h @ r["w2"] + r["b2"]


def image_positions(text, height, width):
    """int32 [text + height * width, 3]: text at the origin, then the image's rows and columns."""
    i = torch.arange(height * width)
    image = torch.stack([torch.zeros_like(i), i // width, i % width], -1)
    return torch.cat([torch.zeros(text, 3, dtype=image.dtype), image]).to(torch.int32).cuda()


def main(dim=3072, heads=24, ffn=12288, axis_pairs=(8, 28, 28), text=512, side=64, blocks=2, check=False):
    torch.manual_seed(0)
    pos = image_positions(text, side, side)
    net = Block(dim, heads, ffn, axis_pairs)
    x0 = torch.randn(pos.shape[0], dim).half().cuda()
    x, y = x0, None
    for _ in range(blocks):
        x, y = net(x, y, pos)
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        net(x0, y, pos)
    end.record()
    torch.cuda.synchronize()
    print(f"block {dim} x {heads} heads, {pos.shape[0]} tokens: {start.elapsed_time(end) / 10 * 1e3:.0f} us")
    if not check:
        return None
    px, py = x0, None
    for _ in range(blocks):
        px, py = net.plain(px, py, pos)
    rel = lambda a, b: float((a.cpu().float() - b).norm() / b.norm())  # noqa: E731
    return rel(x, px), rel(y, py)


class Serving:
    """A stack of blocks over paged caches, one a block, with a page table shared by all."""

    def __init__(self, blocks, sequences, longest, page=64, kind=torch.float8_e4m3fn):
        self.blocks, self.page = blocks, page
        width = -(-longest // page)
        self.caches = [binding.PagedCache.empty(sequences * width, page, b.heads, b.dim // b.heads, kind) for b in blocks]
        # any page may serve any sequence
        self.table = torch.randperm(sequences * width).view(sequences, width).to(torch.int32).cuda()
        self.length = torch.zeros(sequences, dtype=torch.int32, device="cuda")

    def step(self, x, counts, depth=None, tree=None):
        """x fp16 [tokens, dim]: counts[b] tokens of each sequence b, one behind the other; the blocks' (x, y) and the
        batch, for keep.  depth [tokens]: how far behind its sequence's context a token of a tree is (a chain: its
        number)."""
        starts = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
        batch = binding.PagedBatch(self.table, starts, self.length.clone())
        of = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).cuda()
        at = torch.arange(len(x), device="cuda") - starts[of] if depth is None else depth
        axes = len(self.blocks[0].axis_pairs)
        positions = (self.length[of] + at).to(torch.int32)[:, None].expand(-1, axes).contiguous()
        y = None
        for block, cache in zip(self.blocks, self.caches):
            x, y = block(x, y, positions, cache, batch, tree)
        self.length += torch.tensor(counts, dtype=torch.int32).cuda()
        return x, y, batch

    def keep(self, batch, path):
        """Of the last step's tokens only a path's stay: int32 [sequences, width], negative behind a path's end."""
        path = path.cuda()
        for cache in self.caches:
            binding.svdq_cache_keep(cache, batch, path)
        self.length.copy_(batch.context + (path >= 0).sum(1).to(torch.int32))


def cached(dim=2048, heads=16, ffn=8192, axis_pairs=(64,), prompts=(700, 64, 1300), blocks=2):
    """Prompts, a tree of drafted tokens for each sequence, an accepted path of it and one more token; the last
    token's output."""
    torch.manual_seed(0)
    net = Block(dim, heads, ffn, axis_pairs)
    serving = Serving([net] * blocks, len(prompts), max(prompts) + 16)
    rand = lambda n: torch.randn(n, dim).half().cuda()  # noqa: E731
    serving.step(rand(sum(prompts)), list(prompts))
    parent = [-1, 0, 0, 1, 1, 2, 4]
    sees, depth = torch.eye(len(parent), dtype=torch.bool), [0] * len(parent)
    for i, up in enumerate(parent):
        if up >= 0:
            sees[i] |= sees[up]
            depth[i] = depth[up] + 1
    n = len(prompts)
    _, _, batch = serving.step(rand(n * len(parent)), [len(parent)] * n, torch.tensor(depth).cuda().repeat(n),
                               sees.repeat(n, 1).cuda())
    accepted = torch.tensor([[0, 1, 4, 6], [0, 2, -1, -1], [0, 2, 5, -1]])[torch.arange(n) % 3].to(torch.int32)
    serving.keep(batch, accepted)
    x, y, _ = serving.step(rand(n), [1] * n)
    torch.cuda.synchronize()
    print(f"lengths {serving.length.tolist()}, last outputs finite: {bool(torch.isfinite(x + y).all())}")
    return x + y


if __name__ == "__main__":
    cached() if "--cached" in sys.argv[1:] else main()
