"""examples/transformer_block.py over paged caches, its outputs: prompts, a drafted tree, its accepted path and one more
token, against a plain fp32 block over the accepted tokens alone, and against the same steps without a tree.

Bounds: to the plain block those of the uncached example (test_gpu_block_example.py: 0.15 of the stream, 0.3 of the MLP's
output; an E4M3 cache adds 2^-4 of a value at most, 0.03 on average, to the attention's part).  To the steps without a tree
only roundings differ, 2^-11 of a value here and there: they move about one code in a thousand of a 4-bit layer's operands
by one step, a third of the values' size: 0.011 a layer, below 0.05 through both blocks."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

PARENT = [-1, 0, 0, 1, 1, 2, 4]
PATHS = [[0, 1, 4, 6], [0, 2], [0, 2, 5]]
PROMPTS = [6, 1, 13]


@pytest.fixture(scope="module")
def net():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_block
    return transformer_block.Block(512, 4, 2048, (64,))


def plain(net, x, y):
    """A block over one sequence's tokens, each seeing those up to itself, from the unquantized weights in fp32."""
    r, D, H = net.raw, net.dim, net.heads
    norm = lambda v, w: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    x = x if y is None else x + y
    q, k, v = (norm(x, r["n1"]) @ r["wqkv"].T + r["bqkv"]).unflatten(-1, (3, H, D // H)).unbind(-3)
    angle = torch.arange(len(x)).float()[:, None] * net.freq.cpu()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    turned = lambda u, w: torch.view_as_real(  # noqa: E731
        torch.view_as_complex(norm(u, w).unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
    q, k = turned(q, r["qn"]).transpose(0, 1), turned(k, r["kn"]).transpose(0, 1)
    z = (q @ k.transpose(-1, -2) / (D // H) ** 0.5).masked_fill(~torch.ones(len(x), len(x)).tril().bool(), -torch.inf)
    x = x + (torch.softmax(z, -1) @ v.transpose(0, 1)).transpose(0, 1).flatten(1) @ r["wo"].T + r["bo"]
    h = torch.nn.functional.gelu(norm(x, r["n2"]) @ r["w1"] + r["b1"], approximate="tanh")
    return x, h @ r["w2"] + r["b2"]


def last_of_plain(net, tokens):
    """(x, y) of each sequence's last token after two blocks."""
    out = []
    for x in tokens:
        x, y = x.float(), None
        for _ in range(2):
            x, y = plain(net, x, y)
        out.append((x[-1], y[-1]))
    return [torch.stack(t) for t in zip(*out)]


def off(got, want):
    return float((got.float().cpu() - want.float().cpu()).norm() / want.float().cpu().norm())


def test_cached_block_values(net):
    import transformer_block
    g = torch.Generator().manual_seed(191)
    rand = lambda n: torch.randn(n, 512, generator=g).half()  # noqa: E731
    B, N = len(PROMPTS), len(PARENT)
    prompts, drafts, last = [rand(n) for n in PROMPTS], [rand(N) for _ in range(B)], rand(B)
    sees, depth = torch.eye(N, dtype=torch.bool), [0] * N
    for i, up in enumerate(PARENT):
        if up >= 0:
            sees[i] |= sees[up]
            depth[i] = depth[up] + 1
    path = torch.tensor([p + [-1] * (4 - len(p)) for p in PATHS], dtype=torch.int32)

    tree = transformer_block.Serving([net] * 2, B, max(PROMPTS) + 16, page=8)
    tree.step(torch.cat(prompts).cuda(), PROMPTS)
    _, _, batch = tree.step(torch.cat(drafts).cuda(), [N] * B, torch.tensor(depth).cuda().repeat(B), sees.repeat(B, 1).cuda())
    tree.keep(batch, path)
    x, y, _ = tree.step(last.cuda(), [1] * B)
    assert tree.length.tolist() == [n + len(p) + 1 for n, p in zip(PROMPTS, PATHS)]

    chain = transformer_block.Serving([net] * 2, B, max(PROMPTS) + 16, page=8)
    chain.step(torch.cat(prompts).cuda(), PROMPTS)
    chain.step(torch.cat([d[p] for d, p in zip(drafts, PATHS)]).cuda(), [len(p) for p in PATHS])
    cx, cy, _ = chain.step(last.cuda(), [1] * B)

    tokens = lambda paths: [torch.cat([a, d[p], e[None]]) for a, d, p, e in zip(prompts, drafts, paths, last)]  # noqa: E731
    px, py = last_of_plain(net, tokens(PATHS))
    # the bounds tell the path from another one, and from none
    for wrong in ([[0, 1, 3, 5], [0, 1], [0, 1, 4]], [[], [], []]):
        wx, wy = last_of_plain(net, tokens(wrong))
        assert off(wx, px) > 0.05 and off(wy, py) > 0.05
    print(f"plain: stream off by {off(x, px):.3g}, MLP output by {off(y, py):.3g}; chain: {off(x, cx):.3g}, {off(y, cy):.3g}")
    assert off(x, px) < 0.15 and off(y, py) < 0.3
    assert off(x, cx) < 0.05 and off(y, cy) < 0.05
