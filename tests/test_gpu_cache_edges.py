"""svdq_tree_attention and its neighbours where the parts of their work meet: tiles cut behind whole rounds of tiles,
every kernel with less workspace than it asks for, pages shorter than one load's rows, trees of any width, padded
batches, graphs and streams that run at once.  Tolerances are those of test_gpu_cache.py."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402
from test_gpu_block import BF16, E4M3, F16, U, check, gen, randn  # noqa: E402
from test_gpu_cache import (I8, KINDS, QMAX, Pages, _gpu, append_case, attend, attention64, attention_case, random_tree,  # noqa: E402, F401
                            raw)


def need(p, q):
    return binding.tree_attention_workspace_bytes(len(p.counts), q.shape[0], q.shape[1], p.heads, p.dim, p.width, p.page)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_whole_tiles_and_cut_ones(dtype, cache):
    """576 tiles of 128 rows, 512 at once: the last 64 are cut along the keys; with less workspace into fewer parts,
    with none not at all."""
    g = gen(61)
    p = Pages(g, [1100], [400], 64, 16, cache, 64)
    q = (2 * randn(g, 1100, 64, 16)).to(dtype)
    room = need(p, q)
    assert room >= 2 * 64 * 128 * 18 * 4
    want, tol = attention64(p, q, None, 0.25, U[F16] if cache in QMAX else U[dtype])
    for share in (room, room // 2, 0):
        ws = torch.full((share + 64,), 99, dtype=torch.uint8, device="cuda")
        check(attend(p, q, None, workspace=ws[:share]), want, tol, f"workspace of {share}")
        assert bool((ws[share:] == 99).all())


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("rows,dim", [(1, 64), (1, 128), (1, 256), (20, 64), (20, 128), (20, 256), (60, 64), (60, 128), (60, 256)])
def test_parts(rows, dim, dtype, cache):
    """Each kernel's parts at each type, a sequence that has fewer keys than there are parts beside a long one; as
    chain and tree, with all the workspace and with some."""
    g = gen(rows + dim)
    p = Pages(g, [rows, rows], [1900, 5], 1, dim, cache, 32)
    q = (2 * randn(g, 2 * rows, 1, dim)).to(dtype)
    room = need(p, q)
    assert room
    for tree in (None, random_tree(g, p.counts)):
        want, tol = attention64(p, q, tree, dim ** -0.5, U[F16] if cache in QMAX else U[dtype])
        for share in (room, 2 * room // 3):
            ws = torch.empty(share, dtype=torch.uint8, device="cuda")
            check(attend(p, q, tree, workspace=ws), want, tol, f"{rows} rows, workspace of {share}")


@pytest.mark.parametrize("dtype,cache", [KINDS[0], KINDS[3], KINDS[4]])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32])
def test_short_pages(page, dtype, cache):
    for dim in (64, 128, 256):
        attention_case([130], [150], 1, 1, dim, dtype, cache, page, dim == 64)
        attention_case([18], [150], 1, 1, dim, dtype, cache, page, dim == 128)


@pytest.mark.parametrize("rows", [6, 25, 140])
@pytest.mark.parametrize("width", [0, 1, 2, 3, 4, 5, 7, 24, 200])
def test_tree_widths(rows, width):
    """Trees narrower and wider than the step, at odd addresses, rows apart, marks of any value; a context that ends
    anywhere in a tile."""
    g = gen(rows + width)
    p = Pages(g, [rows, 3], [37 + width % 5, 0], 1, 64, F16, 16)
    q = randn(g, rows + 3, 2, 64).to(F16)
    marks = torch.randint(0, 4, (rows + 3, width), generator=g, dtype=torch.uint8)
    tree = torch.where(marks == 3, torch.tensor([1, 2, 16, 64, 128, 255], dtype=torch.uint8)[
        torch.randint(0, 6, marks.shape, generator=g)], torch.zeros_like(marks))
    wide = torch.full((rows + 3, width + 11), 255, dtype=torch.uint8)
    for off in (0, 1, 3):
        wide[:, off:off + width] = tree
        got = binding.svdq_tree_attention(p.cache, p.batch, q.cuda(), tree=wide.cuda()[:, off:off + width])
        want, tol = attention64(p, q, tree, 0.125, U[F16])
        check(got.cpu(), want, tol, f"width {width} at {off}")


def test_odd_queries():
    """Queries at odd addresses and strides, in a packed projection."""
    g = gen(63)
    for n, dtype, cache in ((2, F16, F16), (30, BF16, I8), (140, F16, E4M3)):
        p = Pages(g, [n], [50], 2, 72 if cache is F16 else 80, cache, 16)
        packed = torch.zeros(n, 4 * (p.dim + 1) + 3, dtype=dtype)
        x = packed[:, 1:1 + 4 * (p.dim + 1)].unflatten(-1, (4, p.dim + 1))[..., :p.dim]
        x.copy_(randn(g, n, 4, p.dim))
        dev = packed.cuda()
        xd = dev[:, 1:1 + 4 * (p.dim + 1)].unflatten(-1, (4, p.dim + 1))[..., :p.dim]
        want, tol = attention64(p, x, None, p.dim ** -0.5, U[F16] if cache in QMAX else U[dtype])
        check(binding.svdq_tree_attention(p.cache, p.batch, xd).cpu(), want, tol, "odd queries")
        out = binding.svdq_tree_attention(p.cache, p.batch, xd, out=xd)
        check(out.cpu(), want, tol, "odd queries in place")
        packed[:, 1:1 + 4 * (p.dim + 1)].unflatten(-1, (4, p.dim + 1))[..., :p.dim] = out.cpu()
        assert torch.equal(dev.cpu(), packed)


@pytest.mark.parametrize("n", [1, 5, 70])
def test_padded_batch(n):
    """A batch of room for more sequences and tokens than a step has: empty ones without pages at its end, tokens
    behind the last; the same as without them."""
    g = gen(64 + n)
    p = Pages(g, [n, n], [200, 31], 2, 64, F16, 16)
    q, k, v = (randn(g, 2 * n, h, 64).to(F16) for h in (4, 2, 2))
    pos, freq = torch.arange(2 * n, dtype=torch.int32)[:, None].contiguous(), torch.full((32,), 0.05)
    room, more = 9, 2 * n + 33
    table = torch.full((room, p.width + 3), -1, dtype=torch.int32)
    table[:2, :p.width] = p.table
    starts = torch.tensor(p.starts + [2 * n] * (room - 2), dtype=torch.int32)
    context = torch.tensor(p.contexts + [0] * (room - 2), dtype=torch.int32)
    padded = binding.PagedBatch(table.cuda(), starts.cuda(), context.cuda())
    results = []
    for batch, size in ((p.batch, 2 * n), (padded, more)):
        p2 = Pages(gen(64 + n), [n, n], [200, 31], 2, 64, F16, 16)
        assert torch.equal(p2.table, p.table)
        fill = lambda t: torch.cat([t, torch.ones(size - 2 * n, *t.shape[1:], dtype=t.dtype)]).cuda()  # noqa: E731
        turned = binding.svdq_rope_append(p2.cache, batch, fill(q), fill(k), fill(v), fill(pos), freq.cuda(), (32,))
        out = torch.full((size, 4, 64), 9.0, dtype=F16, device="cuda")
        binding.svdq_tree_attention(p2.cache, batch, turned, out=out)
        p.host["k"], p.host["v"] = p2.dev["k"].cpu(), p2.dev["v"].cpu()
        want, tol = attention64(p, turned[:2 * n].cpu(), None, 0.125, U[F16])
        check(out[:2 * n].cpu(), want, tol, "padded" if size == more else "as it is")
        assert bool((out[2 * n:] == 9).all())
        path = torch.full((batch.sequences, 2), -1, dtype=torch.int32)
        path[0, 0] = n - 1
        binding.svdq_cache_keep(p2.cache, batch, path.cuda())
        results.append((turned[:2 * n], p2.dev["k"], p2.dev["v"]))
    assert all(torch.equal(a, b) for a, b in zip(*results))


def graph_of(f):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    return graph, out


def test_two_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn with other work between them."""
    g = gen(65)
    ps = [Pages(g, [1, 1], [900, 700], 2, 64, F16, 16), Pages(g, [40], [1500], 1, 128, E4M3, 32)]
    qs = [randn(g, 2, 4, 64).to(F16).cuda(), randn(g, 40, 2, 128).to(F16).cuda()]
    ws = torch.zeros(max(need(p, q) for p, q in zip(ps, qs)), dtype=torch.uint8, device="cuda")
    assert all(need(p, q) for p, q in zip(ps, qs))
    graphs = [graph_of(lambda p=p, q=q: binding.svdq_tree_attention(p.cache, p.batch, q, workspace=ws))
              for p, q in zip(ps, qs)]
    for i in range(4):
        for q in qs:
            q.copy_(randn(g, *q.shape))
        for (graph, out), p, q in list(zip(graphs, ps, qs))[::1 if i % 2 else -1]:
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            ws.fill_(255)                    # NaN: nothing is taken from the call before
            assert torch.equal(got, binding.svdq_tree_attention(p.cache, p.batch, q, workspace=ws))


def test_two_calls_at_once():
    """Two streams, a workspace each, many calls in flight."""
    g = gen(66)
    p = Pages(g, [2, 30], [1200, 600], 2, 128, BF16, 16)
    qs = [randn(g, 32, 8, 128).to(BF16).cuda() for _ in range(2)]
    want = [binding.svdq_tree_attention(p.cache, p.batch, q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(binding.svdq_tree_attention(p.cache, p.batch, qs[i], stream=s.cuda_stream))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("cache", [F16, I8])
def test_batches_that_hold_anything(cache):
    """Starts that fall and leave the step, contexts out of range, entries that are no pages: nothing outside the
    outputs' rows is written, and a batch that is in order then gives what it gave."""
    g = gen(67)
    p = Pages(g, [3, 40, 2], [30, 20, 9], 1, 64, cache, 8)
    q, k, v = (randn(g, 45, h, 64).to(F16).cuda() for h in (2, 1, 1))
    before = attend(p, q.cpu(), None)
    pos, freq = torch.arange(45, dtype=torch.int32, device="cuda")[:, None].contiguous(), torch.full((32,), 0.05, device="cuda")
    anything = torch.tensor([0, -1, 2 ** 31 - 1, -2 ** 31, 7, 40, 45, 46, 2 ** 30, 2 ** 30 + 1], dtype=torch.int32)
    tree = torch.ones(45, 45, dtype=torch.bool, device="cuda")
    for i in range(30):
        pick = lambda *s: anything[torch.randint(0, len(anything), s, generator=g)].cuda()  # noqa: E731
        batch = binding.PagedBatch(torch.where(pick(3, p.width) == 7, -1, p.pages).to(torch.int32), pick(4), pick(3))
        buf = torch.full((47, 2, 64), 4.0, dtype=F16, device="cuda")
        binding.svdq_rope_append(p.cache, batch, q, k, v, pos, freq, (32,), q_out=buf[1:46])
        buf.fill_(4.0)
        binding.svdq_tree_attention(p.cache, batch, q, tree=tree if i % 2 else None, out=buf[1:46])
        binding.svdq_cache_keep(p.cache, batch, pick(3, 5))
        assert bool((buf[0] == 4).all()) and bool((buf[46] == 4).all())
        assert bool(((buf == 4) | (buf == 0)).all())         # no page: rows that see nothing, or of no sequence
    for name, t in p.host.items():
        if t is not None:
            assert torch.equal(raw(p.dev[name]).cpu(), raw(t))
    assert torch.equal(attend(p, q.cpu(), None), before)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("dim,pairs", [(64, 16), (64, 24), (80, 8), (80, 32), (96, 40), (128, 32), (128, 8), (256, 64), (256, 120),
                                       (208, 56), (32, 8)])
def test_append_halves_of_a_part(dim, pairs, dtype, cache):
    """Pairs half of the turned part apart, the rest of the head as it is."""
    append_case([1, 5, 0, 3], [40, 7, 9, 0], 5, 3, dim, dtype, cache, 8, (pairs // 2, pairs - pairs // 2), "halves", dim != 64)


@pytest.mark.parametrize("dim,pairs", [(72, 8), (72, 24), (88, 40), (136, 8), (24, 8)])
def test_append_halves_of_a_part_odd(dim, pairs):
    append_case([2, 7], [5, 1], 3, 2, dim, BF16, BF16, 16, (pairs,), "halves", True)
    append_case([2, 7], [5, 1], 3, 2, dim, F16, F16, 16, (pairs,), "halves", False)


def test_append_halves_of_a_part_several_tokens_a_wave():
    counts = [1 + (b * 7) % 5 for b in range(1500)]
    append_case(counts, [b % 3 for b in range(1500)], 2, 1, 64, F16, E4M3, 4, (16,), "halves", True, behind=5)


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_append_keeps_what_lies_behind_the_pairs(pairs):
    """Infinities, NaN and minus zero behind the turned part stay where they are."""
    g = gen(68)
    p = Pages(g, [3], [2], 1, 64, F16, 8)
    q, k, v = (randn(g, 3, h, 64).to(F16) for h in (2, 1, 1))
    for t in (q, k):
        t[..., 32:] = torch.tensor([float("inf"), float("nan"), -0.0, 7.0] * 8).to(F16)
    pos, freq = torch.arange(3, dtype=torch.int32, device="cuda")[:, None].contiguous(), torch.full((16,), 0.3, device="cuda")
    got = binding.svdq_rope_append(p.cache, p.batch, q.cuda(), k.cuda(), v.cuda(), pos, freq, (16,), pairs).cpu()
    assert torch.equal(got[..., 32:].view(torch.int16), q[..., 32:].view(torch.int16)) and bool(torch.isfinite(got[..., :32]).all())
    for t in range(3):
        at = p.dev["k"][int(p.table[0, (2 + t) // 8]), (2 + t) % 8].cpu()
        assert torch.equal(at[..., 32:].view(torch.int16), k[t, :, 32:].view(torch.int16))
        assert bool(torch.isfinite(at[..., :32]).all())


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64])
def test_absent_pages(page, dtype, cache):
    """Absent pages anywhere in the tiles of every kernel, small ones that only some of a workgroup's waves load."""
    for rows, dim in ((140, 64), (140, 128), (140, 256), (24, 128), (3, 64)):
        g = gen(page + rows + dim)
        p = Pages(g, [rows], [230], 1, dim, cache, page)
        gone = torch.rand(p.table.shape, generator=g) < 0.15
        gone[0, 0] = True
        p.table[gone] = torch.where(torch.rand(p.table.shape, generator=g) < 0.5, -1, p.pages).to(torch.int32)[gone]
        p.upload()
        q = (2 * randn(g, rows, 1, dim)).to(dtype)
        want, tol = attention64(p, q, None, dim ** -0.5, U[F16] if cache in QMAX else U[dtype])
        check(attend(p, q, None), want, tol, f"absent pages of {page}, {rows} rows of {dim}")


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("page", [4, 8, 16, 64])
def test_one_absent_page(page, dtype, cache):
    """A single absent page, in each place of a tile in turn."""
    for col in range(64 // page if page < 64 else 3):
        g = gen(page + col)
        p = Pages(g, [70], [200], 2, 128, cache, page)
        p.table[0, 64 // page + col if page < 64 else col] = -1
        p.upload()
        q = (2 * randn(g, 70, 4, 128)).to(dtype)
        want, tol = attention64(p, q, None, 128 ** -0.5, U[F16] if cache in QMAX else U[dtype])
        check(attend(p, q, None), want, tol, f"absent page {col} of {page}")
