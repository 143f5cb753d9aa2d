"""Refusals of the operators around a paged cache (svdq_rope_append, svdq_tree_attention, svdq_cache_keep), on the
CPU: the C ABI's status codes, returned before any HIP call, the binding's argument checks, raised before the
library is called, and the lookups of slots and pages with tables and starts that hold anything."""
import ctypes
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_amd import binding  # noqa: E402
from bit_w4a4_quantized_amd.binding import BatchStruct, CacheStruct, RopeOperand  # noqa: E402
from test_block_checks import Dev, rec  # noqa: E402, F401

OK, NULL, SHAPE, ALIGN, FORMAT = 0, -1, -2, -3, -4
P, ODD, EIGHT = 4096, 4097, 4104          # fake pointers, never dereferenced on these paths
T16, TB, T32, I8, E4 = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")
CACHE = dict(k=P, v=P, k_scales=P, v_scales=P, type=I8, pages=9, page_size=16, heads=2, dim=64, page_stride=2048,
             token_stride=128, head_stride=64, scale_page_stride=32, scale_token_stride=2, scale_head_stride=1)
BATCH = dict(page_table=P, table_stride=4, table_width=4, starts=P, context=P, sequences=3)


def structs(kw):
    c = CacheStruct(**{n: kw.pop("c_" + n, v) for n, v in CACHE.items()})
    b = BatchStruct(**{n: kw.pop("b_" + n, v) for n, v in BATCH.items()})
    return c, b


# what all three refuse
SHARED = [
    (dict(c_type=T32), FORMAT), (dict(c_type=77), FORMAT), (dict(c_pages=-1), SHAPE), (dict(c_pages=1 << 31), SHAPE),
    (dict(c_page_size=0), SHAPE), (dict(c_page_size=24), SHAPE), (dict(c_page_size=1 << 17), SHAPE), (dict(c_page_size=-16), SHAPE),
    (dict(c_heads=0), SHAPE), (dict(c_dim=0), SHAPE), (dict(c_dim=72), SHAPE), (dict(c_dim=272), SHAPE),
    (dict(c_token_stride=136), SHAPE), (dict(c_page_stride=-2048), SHAPE), (dict(c_head_stride=1 << 41), SHAPE),
    (dict(c_scale_page_stride=-1), SHAPE), (dict(b_sequences=-1), SHAPE), (dict(b_table_width=-1), SHAPE),
    (dict(b_table_width=(1 << 26) + 1), SHAPE), (dict(b_table_stride=-4), SHAPE),
    (dict(b_starts=None), NULL), (dict(b_context=None), NULL), (dict(b_page_table=None), NULL), (dict(c_k=None), NULL),
    (dict(c_v_scales=None), NULL), (dict(b_starts=4098), ALIGN), (dict(b_page_table=4098), ALIGN), (dict(c_v=EIGHT), ALIGN),
    (dict(c_k_scales=4098), ALIGN), (dict(cache=None), NULL), (dict(batch=None), NULL),
]


def append(tokens=5, t=T16, pos=P, pf=0, f=P, axes=(8, 24), halves=0, eps=1e-6, v=P, vt=128, vh=64, q=True, k=True, n_axes=None,
           cache=True, batch=True, q_heads=4, **kw):
    c, b = structs(kw)
    one = dict(inp=P, out=P, weight=None, heads=2, in_batch=0, in_token=256, in_head=64, out_batch=0, out_token=256, out_head=64)
    qo, ko = RopeOperand(**{**one, "heads": q_heads, **kw}), RopeOperand(**{**one, **{n: x for n, x in kw.items() if n != "out"}})
    ax = (ctypes.c_int * 8)(*axes) if axes is not None else None
    n = (len(axes) if axes is not None else 1) if n_axes is None else n_axes
    ref = lambda s, on: ctypes.addressof(s) if on else None  # noqa: E731
    return binding.lib().svdq_rope_append(ref(c, cache), ref(b, batch), ref(qo, q), ref(ko, k), v, vt, vh, tokens, t, pos, pf, f,
                                          n, ax, halves, eps, None)


@pytest.mark.parametrize("bad,status", SHARED + [
    (dict(t=T32), FORMAT), (dict(t=I8), FORMAT), (dict(c_type=TB), FORMAT), (dict(k=False), NULL), (dict(axes=None), NULL),
    (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 24) + 1), SHAPE), (dict(n_axes=0), SHAPE), (dict(n_axes=5), SHAPE),
    (dict(axes=(8, 25)), SHAPE), (dict(axes=(0, 0)), SHAPE), (dict(axes=(-1, 8)), SHAPE), (dict(heads=3), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(q_heads=1 << 20), SHAPE), (dict(in_token=-1), SHAPE), (dict(out_head=1 << 41), SHAPE),
    (dict(vt=-1), SHAPE), (dict(vh=1 << 41), SHAPE), (dict(weight=P, eps=0.0), SHAPE), (dict(weight=P, eps=NAN), SHAPE),
    (dict(tokens=1 << 24, q_heads=1 << 10), SHAPE), (dict(pos=None), NULL), (dict(f=None), NULL), (dict(inp=None), NULL),
    (dict(out=None), NULL), (dict(v=None), NULL), (dict(pos=4098), ALIGN), (dict(f=4098), ALIGN), (dict(inp=ODD), ALIGN),
    (dict(out=ODD), ALIGN), (dict(v=ODD), ALIGN), (dict(weight=4098), ALIGN),
    (dict(tokens=0, pos=None, f=None, inp=None, v=None, b_starts=None, c_k=None), OK),
])
def test_append_statuses(bad, status):
    assert append(**bad) == status


def attention(q=P, qt=256, qh=64, heads=4, tokens=5, t=T16, scale=0.125, tree=P, ts=8, tw=8, out=P, ot=256, oh=64, ws=P, wb=0,
              cache=True, batch=True, **kw):
    c, b = structs(kw)
    ref = lambda s, on: ctypes.addressof(s) if on else None  # noqa: E731
    return binding.lib().svdq_tree_attention(ref(c, cache), ref(b, batch), q, qt, qh, heads, tokens, t, scale, tree, ts, tw, out, ot,
                                             oh, ws, wb, None)


@pytest.mark.parametrize("bad,status", SHARED + [
    (dict(t=T32), FORMAT), (dict(t=E4), FORMAT), (dict(c_type=TB), FORMAT), (dict(tokens=-1), SHAPE), (dict(heads=3), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=1 << 17), SHAPE), (dict(tokens=1 << 24, heads=1 << 10), SHAPE),
    (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=NAN), SHAPE), (dict(scale=INF), SHAPE),
    (dict(qt=-1), SHAPE), (dict(oh=1 << 41), SHAPE), (dict(ts=-1), SHAPE), (dict(tw=-1), SHAPE), (dict(q=None), NULL),
    (dict(out=None), NULL), (dict(q=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(ws=EIGHT), ALIGN),
    (dict(tokens=0, q=None, out=None, b_starts=None), OK), (dict(b_sequences=0, b_starts=None, q=None), OK),
])
def test_attention_statuses(bad, status):
    assert attention(**bad) == status


def keep(path=P, ps=8, pw=8, cache=True, batch=True, **kw):
    c, b = structs(kw)
    ref = lambda s, on: ctypes.addressof(s) if on else None  # noqa: E731
    return binding.lib().svdq_cache_keep(ref(c, cache), ref(b, batch), path, ps, pw, None)


@pytest.mark.parametrize("bad,status", SHARED + [
    (dict(pw=-1), SHAPE), (dict(pw=(1 << 16) + 1), SHAPE), (dict(ps=-1), SHAPE), (dict(path=None), NULL), (dict(path=4098), ALIGN),
    (dict(pw=0, path=None), OK), (dict(b_sequences=0, path=None, c_k=None), OK),
])
def test_keep_statuses(bad, status):
    assert keep(**bad) == status


def test_workspace_bytes():
    f = binding.lib().svdq_tree_attention_workspace_bytes
    assert f(1, 1, 32, 8, 128, 1024, 64) > 0 and f(1, 1, 32, 8, 128, 0, 64) == 0
    for bad in ((0, 1, 32, 8, 128, 64, 64), (1, 0, 32, 8, 128, 64, 64), (1, 1, 0, 8, 128, 64, 64), (1, 1, 33, 8, 128, 64, 64),
                (1, 1, 32, 0, 128, 64, 64), (1, 1, 32, 8, 0, 64, 64), (1, 1, 32, 8, 257, 64, 64), (1, 1, 32, 8, 128, -1, 64),
                (1, 1, 32, 8, 128, 64, 0), (-1, 1, 32, 8, 128, 64, 64)):
        assert f(*bad) == 0


def test_lookups_and_statuses_under_address_and_undefined_behaviour_sanitizers():
    if not (os.path.exists("/opt/rocm/bin/hipcc") or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    from bit_w4a4_quantized_amd.build import BUILD_DIR, build_host_check
    exe = build_host_check(check="abi_check_cache.cpp", exe=os.path.join(BUILD_DIR, "svdq_abi_check_cache"))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "OK: 0 failure(s)" in r.stdout, r.stdout


# ------------------------------------------------------------------ the binding
F16, BF16, F32, I8T, I32, E4T = torch.float16, torch.bfloat16, torch.float32, torch.int8, torch.int32, torch.float8_e4m3fn


def cache(dtype=I8T, shape=(9, 16, 2, 64), **kw):
    scale = None if dtype in (F16, BF16) else Dev(shape[:3], F32)
    a = dict(k=Dev(shape, dtype), v=Dev(shape, dtype), k_scales=scale, v_scales=scale)
    return binding.PagedCache(**{**a, **kw})


def batch(**kw):
    a = dict(page_table=Dev((3, 4), I32, (6, 1)), starts=Dev((4,), I32), context=Dev((3,), I32))
    return binding.PagedBatch(**{**a, **kw})


class Moved(Dev):
    def data_ptr(self):
        return EIGHT


def test_cache_handle(rec):  # noqa: F811
    c = cache(F16, k=Dev((9, 16, 2, 64), F16, (2048, 64, 1024, 1)), v=Dev((9, 16, 2, 64), F16, (2048, 64, 1024, 1)))
    s = c._struct
    assert (s.page_stride, s.token_stride, s.head_stride, s.pages, s.page_size, s.heads, s.dim, s.type) == (2048, 64, 1024, 9, 16, 2, 64, 0)
    assert cache(E4T)._struct.scale_page_stride == 32
    one = Dev((1, 16, 2, 64), F16, (5, 128, 64, 1))       # the stride of a single page means nothing
    assert cache(F16, k=one, v=one)._struct.page_stride == 0
    bad = Dev((9, 16, 2, 64), I8T)
    for kw in (dict(k=None), dict(v=None), dict(k=Dev((9, 16, 2, 64), I8T, cuda=False)), dict(dtype=F32), dict(shape=(9, 24, 2, 64)),
               dict(shape=(9, 16, 2, 72)), dict(shape=(9, 16, 2, 512)), dict(shape=(9, 16, 0, 64)), dict(shape=(9, 16, 128)),
               dict(shape=(9, 0, 2, 64)), dict(v=Dev((9, 16, 2, 64), E4T)), dict(v=Dev((9, 16, 1, 64), I8T)),
               dict(k=Dev((9, 16, 2, 64), I8T, (2048, 128, 1, 2))), dict(k=Dev((9, 16, 2, 64), I8T, (4096, 128, 64, 1))),
               dict(k=Dev((9, 16, 2, 64), I8T, (2048, 0, 64, 1)), v=Dev((9, 16, 2, 64), I8T, (2048, 0, 64, 1))),
               dict(k=Dev((9, 16, 2, 64), I8T, (2200, 136, 64, 1)), v=Dev((9, 16, 2, 64), I8T, (2200, 136, 64, 1))),
               dict(k=Moved((9, 16, 2, 64), I8T)), dict(k_scales=None), dict(v_scales=Dev((9, 16, 2), F16)),
               dict(v_scales=Dev((9, 16, 1), F32)), dict(k_scales=Dev((9, 16, 2), F32, (64, 4, 1))),
               dict(k_scales=Dev((9, 16, 2), F32, (0, 2, 1)), v_scales=Dev((9, 16, 2), F32, (0, 2, 1))),
               dict(dtype=F16, k_scales=Dev((9, 16, 2), F32)), dict(v=Dev((9, 16, 2, 64), I8T, device="cuda:1"))):
        with pytest.raises(ValueError):
            cache(**kw)
    assert bad is not None


def test_batch_handle(rec):  # noqa: F811
    s = batch()._struct
    assert (s.table_stride, s.table_width, s.sequences) == (6, 4, 3)
    for kw in (dict(page_table=None), dict(page_table=Dev((3, 4), torch.int64)), dict(page_table=Dev((3, 4), I32, (1, 3))),
               dict(page_table=Dev((12,), I32)), dict(page_table=Dev((3, 4), I32, cuda=False)), dict(starts=None), dict(starts=Dev((3,), I32)),
               dict(starts=Dev((4,), torch.int64)), dict(context=Dev((4,), I32)), dict(context=Dev((3,), F32)),
               dict(context=Dev((3,), I32, device="cuda:1"))):
        with pytest.raises(ValueError):
            batch(**kw)


def append_args(**kw):
    a = dict(cache=cache(), batch=batch(), q=Dev((5, 4, 64), F16, (512, 64, 1)), k=Dev((5, 2, 64), F16, (512, 64, 1)),
             v=Dev((5, 2, 64), F16, (512, 64, 1)), positions=Dev((5, 2), I32), inv_freq=Dev((32,), F32), axis_pairs=(8, 24),
             q_weight=Dev((64,), F32), k_weight=Dev((64,), F32), q_out=Dev((5, 4, 64), F16))
    return {**a, **kw}


def test_append_binding(rec):  # noqa: F811
    binding.svdq_rope_append(**append_args())
    binding.svdq_rope_append(**append_args(q=None, q_weight=None, q_out=None, positions=Dev((5, 2), F32), pairs="halves"))
    assert [c[0] for c in rec.calls] == ["svdq_rope_append"] * 2
    assert rec.calls[0][1][4:12] == (P, 512, 64, 5, 0, P, 0, P) and rec.calls[1][1][2] is None
    assert rec.calls[1][1][10] == 1 and rec.calls[1][1][14] == 1
    for bad in (dict(cache=None), dict(batch=None), dict(batch=cache()), dict(k=None), dict(v=None), dict(k=Dev((5, 2, 64), F32)),
                dict(k=Dev((5, 2, 64), BF16)), dict(q=Dev((5, 4, 64), BF16)), dict(q=Dev((4, 4, 64), F16)), dict(q=Dev((5, 4, 32), F16)),
                dict(q=Dev((5, 0, 64), F16)), dict(q=Dev((5, 4, 64), F16, (256, 1, 4))), dict(k=Dev((5, 3, 64), F16)),
                dict(k=Dev((5, 128), F16)), dict(v=Dev((6, 2, 64), F16)), dict(v=Dev((5, 2, 64), F16, cuda=False)),
                dict(q=None), dict(cache=cache(BF16)), dict(pairs="both"), dict(positions=None), dict(positions=Dev((5, 3), I32)),
                dict(positions=Dev((4, 2), I32)), dict(positions=Dev((5, 2), torch.int64)), dict(positions=Dev((5, 2), I32, (1, 5))),
                dict(inv_freq=Dev((31,), F32)), dict(inv_freq=None), dict(q_weight=Dev((32,), F32)), dict(k_weight=Dev((64,), F16)),
                dict(q_out=Dev((5, 4, 64), F16, (0, 64, 1))), dict(q_out=Dev((5, 2, 64), F16)), dict(q_out=Dev((5, 4, 64), BF16)),
                dict(k=Dev((5, 2, 64), F16, (512, 64, 1), device="cuda:1"))):
        with pytest.raises(ValueError):
            binding.svdq_rope_append(**append_args(**bad))
    assert len(rec.calls) == 2


def attention_args(**kw):
    a = dict(cache=cache(), batch=batch(), q=Dev((5, 4, 64), F16, (512, 64, 1)), tree=Dev((5, 8), torch.bool, (16, 1)),
             out=Dev((5, 4, 64), F16, (512, 128, 1)))
    return {**a, **kw}


def test_attention_binding(rec):  # noqa: F811
    binding.tree_attention_workspace_bytes.cache_clear()
    binding.svdq_tree_attention(**attention_args())
    binding.svdq_tree_attention(**attention_args(tree=None, scale=0.5, cache=cache(F16)))
    binding.svdq_tree_attention(**attention_args(tree=Dev((5, 0), torch.uint8)))
    assert rec.calls[0][1][2:] == (P, 512, 64, 4, 5, 0, 0.125, P, 16, 8, P, 512, 128, None, 0, 7)
    assert rec.calls[1][1][8:12] == (0.5, None, 0, 0) and rec.calls[2][1][9] and rec.calls[2][1][11] == 0
    for bad in (dict(cache=None), dict(batch=None), dict(q=None), dict(q=Dev((5, 4, 64), F32)), dict(q=Dev((5, 4, 64), F16, cuda=False)),
                dict(q=Dev((5, 4, 32), F16)), dict(q=Dev((5, 256), F16)), dict(q=Dev((5, 3, 64), F16)), dict(q=Dev((5, 0, 64), F16)),
                dict(q=Dev((5, 4, 64), F16, (256, 1, 4))), dict(cache=cache(BF16)), dict(tree=Dev((4, 8), torch.bool)),
                dict(tree=Dev((5, 8), F16)), dict(tree=Dev((5, 8), torch.bool, (1, 5))), dict(out=Dev((5, 4, 64), BF16)),
                dict(out=Dev((5, 2, 64), F16)), dict(out=Dev((5, 4, 64), F16, (0, 64, 1))), dict(out=Dev((5, 4, 64), F16, (256, 1, 4))),
                dict(tree=Dev((5, 8), torch.bool, device="cuda:1"))):
        with pytest.raises(ValueError):
            binding.svdq_tree_attention(**attention_args(**bad))
    assert len(rec.calls) == 3
    binding.tree_attention_workspace_bytes.cache_clear()


def test_keep_binding(rec):  # noqa: F811
    binding.svdq_cache_keep(cache(), batch(), Dev((3, 5), I32, (9, 1)))
    assert rec.calls[0][1][2:] == (P, 9, 5, 7)
    for bad in (None, Dev((3, 5), torch.int64), Dev((4, 5), I32), Dev((3, 5), I32, (1, 3)), Dev((15,), I32),
                Dev((3, 5), I32, device="cuda:1")):
        with pytest.raises(ValueError):
            binding.svdq_cache_keep(cache(), batch(), bad)
    with pytest.raises(ValueError):
        binding.svdq_cache_keep(None, batch(), Dev((3, 5), I32))
    assert len(rec.calls) == 1
