"""Paged 4-bit cache without a GPU: the oracle's pins, the library's argument
validation (before any launch) and the binding's tensor checks."""
import ctypes
import subprocess
import sys

import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import qcache as Q

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def K():
    __graft_entry__.build()
    from long_context_anchor_gb300 import kascade
    return kascade


# ------------------------------------------------------------------ oracle pins --

def test_e4m3_table_is_torchs():
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(Q.E4M3, bits)


def test_nearest_even_against_torch_rounding():
    rng = np.random.default_rng(0)
    x = np.concatenate([np.exp(rng.uniform(-9, 6.1, 4000)), (Q.E4M3[1:] + Q.E4M3[:-1]) / 2, Q.E4M3])
    x = x[x <= 448]
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    exact = x.astype(np.float32).astype(np.float64)     # torch rounds the fp32 value
    assert np.array_equal(Q.E4M3[Q.nearest_even(exact, Q.E4M3)], want)


@pytest.mark.parametrize("x,want", [(0.25, 0.0), (0.2500001, 0.5), (0.75, 1.0), (1.25, 1.0),
                                    (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0), (5.01, 6.0),
                                    (7.0, 6.0)])
def test_e2m1_ties_by_hand(x, want):
    assert Q.E2M1[Q.nearest_even(x, Q.E2M1)] == want


def test_stored_rows_by_hand():
    row = np.zeros(64)
    row[:16] = np.arange(16) - 8.0          # amax 8: scale 8/6 -> 1.375
    row[16:32] = 6.0                        # scale 1, exact
    row[32:48] = 1e-5                       # amax/6 < 2^-10: stored as zeros
    row[48] = np.nan
    got = Q.stored(row)
    assert np.array_equal(got[16:32], row[16:32]) and not got[32:48].any()
    assert np.isnan(got[48:]).all()
    assert got[0] == -8.25 and got[8] == 0.0 and got[9] == 1.375 * 0.5 and got[15] == 1.375 * 6
    # saturation, and a power-of-two scale that undoes it
    big = np.full(64, 1e6)
    assert (Q.stored(big) == 2688.0).all()
    assert np.allclose(Q.stored(big, 2.0 ** 10), 1e6, rtol=1 / 16)


def test_stored_error_bound():
    """|stored - x| <= s * half the widest e2m1 step (1) once the scale covers amax."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 128))
    b = x.reshape(200, 8, 16)
    amax = np.abs(b).max(-1, keepdims=True)
    # scale within 1/16 of amax/6, so codes above 6 exceed it by at most 6/16
    err = np.abs(Q.stored(x).reshape(b.shape) - b)
    assert (err <= amax / 6 * (17 / 16)).all()


def test_plan_by_hand():
    table = np.array([[5, 7, -1], [1, 2, 3], [-1, -1, -1]])
    free = np.array([0, 4, 6, -1, -1, -1, -1, -1])
    # 0: 30 -> 33 takes one; 1: 40 -> 16 gives two (2, 3); 2: 0 -> 1 takes one
    slots, cu, lens, count, t, f = Q.plan([30, 40, 0], [3, -24, 1], table, free, 3, 16, 6)
    assert list(f[:5]) == [0, 4, 6, 2, 3] and count == 3
    assert t[0, 2] == 3 and t[2, 0] == 2            # popped from the top: 3, then 2
    assert list(lens) == [33, 16, 1] and list(cu) == [0, 3, 3, 4]
    assert list(slots) == [7 * 16 + 14, 7 * 16 + 15, 3 * 16, 2 * 16, -1, -1]
    assert Q.plan([30, 40, 0], [3, 0, 40], table, free, 3, 16, 99) is None    # 4 blocks of 3
    assert Q.plan([30, 40, 0], [3, 0, 1], table, free, 3, 16, 3) is None      # 4 tokens, 3 slots


def test_attention_oracle_is_softmax():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal(64), rng.standard_normal((9, 64)), rng.standard_normal((9, 64))
    want = torch.nn.functional.scaled_dot_product_attention(
        *[torch.from_numpy(x).view(1, 1, -1, 64) for x in (q, k, v)]).numpy().reshape(64)
    assert np.allclose(Q.attention(q, k, v, 0.125)[0], want, atol=1e-12)
    assert not Q.attention(q, k, v, 0.125, [])[0].any()


# ------------------------------------------------------------------- refusals --

def test_validation_before_launch(K):
    L = K._lib
    ref = ctypes.byref
    p = ctypes.c_void_p(1 << 20)            # aligned, never dereferenced on these paths
    odd = ctypes.c_void_p((1 << 20) + 8)
    desc = K.make_desc(2, 8, 2, 128, 1000, K.BF16)
    geo = K.QCache(64, 40, 16, 0.0, 0.0)
    size = L.kascade_qcache_workspace_size
    n0, n1 = size(ref(desc), ref(geo), 0), size(ref(desc), ref(geo), 32)
    assert 0 < n0 < n1
    assert L.kascade_qcache_bytes(ref(geo), 2, 128) == 40 * 2 * 4 * 2304
    for bad in [(48, 40, 16, 0, 0), (8, 40, 16, 0, 0), (512, 40, 16, 0, 0), (64, 0, 16, 0, 0),
                (64, 40, 0, 0, 0), (64, 40, 15, 0, 0), (64, 40, 16, 3.0, 0), (64, 40, 16, 0, -1.0),
                (64, 40, 16, float("inf"), 0), (64, 40, 16, 0, float("nan")),
                (256, 1 << 23, 16, 0, 0)]:
        assert size(ref(desc), ref(K.QCache(*bad)), 0) == 0, bad
    for ok in [(16, 40, 64, 0, 0), (256, 40, 4, 0.125, 4.0)]:
        assert size(ref(desc), ref(K.QCache(*ok)), 0) > 0, ok
    dense, anchor, reuse = (L.kascade_qcache_dense_decode, L.kascade_qcache_anchor_decode,
                            L.kascade_qcache_reuse_decode)
    d, g = ref(desc), ref(geo)
    assert dense(d, g, odd, p, p, p, p, None, p, n0, None) == K.INVALID_ARG
    assert dense(d, g, p, odd, p, p, p, None, p, n0, None) == K.INVALID_ARG
    assert dense(d, g, p, p, None, p, p, None, p, n0, None) == K.INVALID_ARG
    assert dense(d, g, p, p, p, None, p, None, p, n0, None) == K.INVALID_ARG
    assert dense(d, g, p, p, p, p, p, odd, p, n0, None) == K.INVALID_ARG
    assert dense(d, g, p, p, p, p, p, None, p, n0 - 1, None) == K.WORKSPACE
    assert dense(d, g, p, p, p, p, p, None, odd, n0, None) == K.WORKSPACE
    assert dense(d, None, p, p, p, p, p, None, p, n0, None) == K.INVALID_ARG
    for k in (0, 1001):
        assert anchor(d, g, p, p, p, p, k, p, p, None, p, 1 << 40, None) == K.INVALID_ARG
        assert reuse(d, g, p, p, p, p, k, p, p, p, 1 << 40, None) == K.INVALID_ARG
    assert anchor(d, g, p, p, p, p, 32, p, p, None, p, n0, None) == K.WORKSPACE
    # per-head sets beyond 262144 keys
    far = K.make_desc(1, 8, 2, 128, 262145, K.BF16)
    wide = K.QCache(256, 40, 1025, 0.0, 0.0)
    assert reuse(ref(far), ref(wide), p, p, p, p, 32, p, p, p, 1 << 50, None) == K.UNSUPPORTED
    st = (ctypes.c_int64 * 4)(256, 128, 256, 128)
    app, read = L.kascade_qcache_append, L.kascade_qcache_read
    assert app(g, 2, 128, K.BF16, p, p, st, p, 4, p, p, 255, None) == K.WORKSPACE
    assert app(g, 2, 96, K.BF16, p, p, st, p, 4, p, p, 256, None) == K.UNSUPPORTED
    assert app(g, 0, 128, K.BF16, p, p, st, p, 4, p, p, 256, None) == K.INVALID_ARG
    assert app(g, 2, 128, 7, p, p, st, p, 4, p, p, 256, None) == K.INVALID_ARG
    assert app(g, 2, 128, K.BF16, p, odd, st, p, 4, p, p, 256, None) == K.INVALID_ARG
    assert app(g, 2, 128, K.BF16, p, p, st, p, -1, p, p, 256, None) == K.INVALID_ARG
    bad = (ctypes.c_int64 * 4)(256, 128, 256, 124)
    assert app(g, 2, 128, K.BF16, p, p, bad, p, 4, p, p, 256, None) == K.INVALID_ARG
    assert read(g, 2, 128, K.BF16, p, p, 4, p, p, bad, p, 256, None) == K.INVALID_ARG
    assert read(g, 2, 128, K.BF16, p, p, 4, None, p, st, p, 256, None) == K.INVALID_ARG
    plan = L.kascade_qcache_plan
    assert plan(g, 0, p, p, p, p, p, p, p, p, p, 4, p, 256, None) == K.INVALID_ARG
    assert plan(g, 16385, p, p, p, p, p, p, p, p, p, 4, p, 256, None) == K.UNSUPPORTED
    assert plan(g, 2, p, p, p, None, p, p, p, p, p, 4, p, 256, None) == K.INVALID_ARG
    assert plan(g, 2, p, p, p, p, p, p, p, p, None, 4, p, 256, None) == K.INVALID_ARG
    assert plan(g, 2, p, p, p, p, p, p, p, p, p, -1, p, 256, None) == K.INVALID_ARG
    assert plan(g, 2, p, p, p, p, p, p, p, p, p, 4, p, 255, None) == K.WORKSPACE
    # stack: every layer's pointers, the anchors and the plan's state before any launch
    a = 1 << 20
    arr = lambda xs: (ctypes.c_void_p * 2)(*xs)
    good, last = arr([a, a]), arr([a, a + 8])
    an = (ctypes.c_int32 * 2)(0, 1)
    run = L.kascade_qcache_run_stack

    def step(**kw):
        vals = dict(block_table=a, kv_lens=a, new_lens=a, free_blocks=a, free_count=a, cu_new=a,
                    slot_map=a, max_new=2)
        vals.update(kw)
        return K.QCacheStep(*[vals[f] for f, _ in K.QCacheStep._fields_])

    def call(s=None, q=good, kn=good, vn=good, pg=good, k=32, m=1, anchors=an, nb=n1, out=good):
        return run(d, g, ref(s or step()), 2, q, kn, vn, pg, k, anchors, m, out, p, p, nb, None)

    assert call(q=last) == K.INVALID_ARG and call(kn=last) == K.INVALID_ARG
    assert call(pg=last) == K.INVALID_ARG and call(out=last) == K.INVALID_ARG
    assert call(vn=None) == K.INVALID_ARG
    assert call(step(free_count=None)) == K.INVALID_ARG
    assert call(step(slot_map=None)) == K.INVALID_ARG
    assert call(anchors=(ctypes.c_int32 * 2)(1, 0), m=2) == K.INVALID_ARG
    assert call(k=0) == K.INVALID_ARG and call(nb=n1 - 1) == K.WORKSPACE


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append(name)
            if name.endswith("workspace_size") or name.endswith("_bytes"):
                return 4096
            return b"fake" if name == "kascade_status_string" else 0
        return fn


@pytest.fixture
def fake(K, monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(K, "_lib", rec)
    monkeypatch.setattr(K, "_stream", lambda stream=None: None)
    monkeypatch.setattr(K, "_DEVICE_TYPE", "cpu")
    K._qdesc.cache_clear()
    yield rec
    K._qdesc.cache_clear()      # its sizes came from the stand-in


def _state(B=3, Hq=8, Hkv=2, d=128, bs=32, nb=20, width=5, dtype=BF):
    return dict(q=torch.zeros(B, Hq, d, dtype=dtype),
                pages=torch.zeros(nb, Hkv, bs // 16, 18 * d, dtype=torch.uint8),
                table=torch.zeros(B, width, dtype=I32), lens=torch.zeros(B, dtype=I32))


def test_refused_sizes(K):
    """Sizes whose numbering would leave 32 bits (pieces of new rows, groups of the cache)."""
    L, ref, p = K._lib, ctypes.byref, ctypes.c_void_p(1 << 20)
    g = ref(K.QCache(64, 40, 16, 0.0, 0.0))
    st = (ctypes.c_int64 * 4)(0, 0, 0, 0)
    for n in (1 << 28, (1 << 31) - 1):
        assert L.kascade_qcache_append(g, 2, 128, K.BF16, p, p, st, p, n, p, p, 256,
                                       None) == K.UNSUPPORTED
        assert L.kascade_qcache_read(g, 2, 64, K.F32, p, p, n, p, p, st, p, 256,
                                     None) == K.UNSUPPORTED
        assert L.kascade_qcache_plan(g, 2, p, p, p, p, p, p, p, p, p, n, p, 256,
                                     None) == K.UNSUPPORTED
    desc = K.make_desc(1, 64, 64, 128, 1000, K.BF16)
    most = ((1 << 28) - 2) // 64
    size = L.kascade_qcache_workspace_size
    assert size(ref(desc), ref(K.QCache(16, most, 63, 0.0, 0.0)), 0) > 0
    assert size(ref(desc), ref(K.QCache(16, most + 1, 63, 0.0, 0.0)), 0) == 0



def test_documented_calls_pass(K, fake):
    ws = K.Workspace("cpu")
    s = _state()
    a = (s["q"], s["pages"], s["table"], s["lens"])
    assert K.qcache_dense_decode(*a, ws=ws).shape == (3, 8, 128)
    out, sc = K.qcache_dense_decode(*a, kv_len=100, return_scores=True, ws=ws)
    assert sc.shape == (3, 8, 100) and sc.dtype == torch.float32
    out, idx, sc = K.qcache_anchor_decode(*a, 16, return_scores=True, pooled=True, ws=ws)
    assert idx.shape == (3, 2, 16) and sc.shape == (3, 2, 160)
    K.qcache_reuse_decode(*a, torch.zeros(3, 8, 16, dtype=I32), ws=ws)
    K.qcache_reuse_decode(*a, torch.zeros(3, 2, 16, dtype=I32), pooled=True, ws=ws)
    i = lambda n: torch.zeros(n, dtype=I32)
    slots, cu, lens, count = K.qcache_plan(s["lens"], i(3), s["table"], i(20), i(1), 32, 7, ws=ws)
    assert slots.shape == (7,) and cu.shape == (4,) and lens.shape == (3,) and count.shape == (1,)
    k = torch.zeros(2, 7, 128, dtype=BF).transpose(0, 1)        # a prefill layer's layout
    assert K.qcache_append(k, k, slots, s["pages"], ws=ws) is s["pages"]
    rk, rv = K.qcache_read(s["pages"], slots, dtype=torch.float32, ws=ws)
    assert rk.shape == (7, 2, 128) and rk.dtype == torch.float32
    K.qcache_read(s["pages"], slots, k=k, v=k.clone(), ws=ws)
    pool = K.qcache_alloc(20, 2, 128, 32, device="cpu")
    assert pool.shape == s["pages"].shape
    rows = [torch.zeros(3, 2, 128, dtype=BF) for _ in range(2)]
    outs, ib = K.qcache_run_stack([s["q"]] * 2, [s["pages"]] * 2, s["table"], s["lens"], 16, [0],
                                  new_ks=rows, new_vs=rows, new_lens=i(3), free_blocks=i(20),
                                  free_count=i(1), ws=ws)
    assert len(outs) == 2 and ib.shape == (3, 8, 16)
    assert {"kascade_qcache_plan", "kascade_qcache_append", "kascade_qcache_read",
            "kascade_qcache_dense_decode", "kascade_qcache_anchor_decode",
            "kascade_qcache_reuse_decode", "kascade_qcache_run_stack"} <= set(fake.calls)


def test_wrong_tensors_raise_before_the_library(K, fake):
    ws = K.Workspace("cpu")
    s = _state()
    i = lambda *n: torch.zeros(*n, dtype=I32)
    q, pages, table, lens = s["q"], s["pages"], s["table"], s["lens"]
    dense = lambda **kw: K.qcache_dense_decode(
        **{**dict(q=q, pages=pages, block_table=table, kv_lens=lens, ws=ws), **kw})
    bad = [dict(q=q[:, :, ::2]), dict(q=q[..., :64].contiguous()), dict(q=q.half()),
           dict(pages=pages[..., :100]), dict(pages=pages.to(torch.int8)),
           dict(pages=pages[:, :, :, ::2]), dict(pages=pages[0]), dict(block_table=table.long()),
           dict(block_table=table[:2]), dict(block_table=table[:, ::2]), dict(kv_lens=lens[:2]),
           dict(kv_lens=lens.long()), dict(out=q[:2]), dict(out=q.float())]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            dense(**kw)
    a = (q, pages, table, lens)
    for idx in (i(3, 8), i(3, 2, 16), i(3, 8, 16).long(), i(3, 8, 32)[..., ::2]):
        with pytest.raises((ValueError, TypeError)):
            K.qcache_reuse_decode(*a, idx, ws=ws)
    with pytest.raises(ValueError):
        K.qcache_anchor_decode(*a, 16, idx=i(3, 2, 16), ws=ws)
    rows = torch.zeros(4, 2, 128, dtype=BF)
    for k, v, m in ((rows, rows, i(3)), (rows, rows.float(), i(4)), (rows, rows, i(4).long()),
                    (rows[:, :1], rows[:, :1], i(4)), (rows.transpose(1, 2), rows, i(4)),
                    (torch.zeros(4, 2, 132, dtype=BF)[..., 4:], rows, i(4)),
                    (torch.zeros(4, 2, 129, dtype=BF)[..., :128], rows, i(4))):
        with pytest.raises((ValueError, TypeError)):
            K.qcache_append(k, v, m, pages, ws=ws)
    one = torch.zeros(1, 2, 128, dtype=BF).expand(4, 2, 128)    # rows on top of one another
    with pytest.raises(ValueError):
        K.qcache_read(pages, i(4), k=one, v=one, ws=ws)
    with pytest.raises(ValueError):
        K.qcache_read(pages, i(4), k=rows, ws=ws)
    plan = lambda **kw: K.qcache_plan(**{**dict(
        kv_lens=lens, new_lens=i(3), block_table=table, free_blocks=i(20), free_count=i(1),
        block_size=32, max_new=4, ws=ws), **kw})
    for kw in (dict(kv_lens=i(2)), dict(new_lens=i(3).long()), dict(free_count=i(2)),
               dict(block_table=i(4, 5)), dict(free_blocks=i(4, 5)), dict(kv_lens_out=i(2)),
               dict(free_count_out=i(3))):
        with pytest.raises((ValueError, TypeError)):
            plan(**kw)
    stack = lambda **kw: K.qcache_run_stack(**{**dict(
        qs=[q] * 2, pages=[pages] * 2, block_table=table, kv_lens=lens, topk=16, anchors=[0],
        ws=ws), **kw})
    r2 = [torch.zeros(3, 2, 128, dtype=BF)] * 2
    for kw in (dict(pages=[pages]), dict(new_ks=r2), dict(new_ks=r2, new_vs=r2),
               dict(new_lens=i(3)), dict(new_ks=r2, new_vs=r2[:1], slot_map=i(3)),
               dict(new_ks=r2, new_vs=r2, slot_map=i(4)),
               dict(new_lens=i(3), free_blocks=i(19), free_count=i(1)),
               dict(qs=[q, q[:2]]), dict(idx_buf=i(3, 8, 8)), dict(outs=[q])):
        with pytest.raises((ValueError, TypeError)):
            stack(**kw)
    assert not [c for c in fake.calls if c.startswith("kascade_qcache") and
                not c.endswith(("_size", "_bytes"))]


def test_captured_workspace_does_not_grow(K, fake):
    ws = K.Workspace("cpu")
    ws.get(4096)
    ws.captured = True
    assert ws.get(1024) is ws.buf
    with pytest.raises(RuntimeError, match="captured"):
        ws.get(8192)


def test_plan_refuses_a_bad_block_that_new_tokens_go_to():
    """The partly filled block of a growing sequence is neither given back nor taken."""
    free = np.array([1, 2, 3, 0])
    for bad in (-1, 4, 2 ** 31 - 1):
        table = np.array([[0, bad, -1]])
        assert Q.plan([20], [5], table, free, 3, 16, 8) is None
        assert Q.plan([20], [0], table, free, 3, 16, 8) is not None     # nothing goes there
        assert Q.plan([32], [5], table, free, 3, 16, 8) is not None     # full: not touched


_WITHOUT_PRIVATE_NAMES = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream", "_cuda_isCurrentStreamCapturing"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from long_context_anchor_gb300 import kascade as K
assert K._current_device is torch.cuda.current_device
assert K._capturing is torch.cuda.is_current_stream_capturing
class Stream:
    cuda_stream = 77
torch.cuda.current_stream = lambda index: Stream() if index == 3 else None
assert K._current_raw_stream(3) == 77
"""


def test_binding_without_torchs_private_functions(K):
    """The functions behind torch.cuda's public ones are a shortcut, not a need."""
    r = subprocess.run([sys.executable, "-c", _WITHOUT_PRIVATE_NAMES], cwd=__graft_entry__.ROOT,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("pooled", [False, True])
def test_reuse_workspace_holds_no_logits(K, pooled):
    """A reuse layer's workspace: below an anchor layer's by the logits and what ranks them, and
    refused one byte short of it."""
    B, Hq, Hkv, N = 64, 32, 8, 131072
    desc = K.make_desc(B, Hq, Hkv, 128, N, K.BF16, pooled=pooled)
    geo = K.QCache(64, 4096, N // 64, 0.0, 0.0)
    L, ref, p = K._lib, ctypes.byref, ctypes.c_void_p(1 << 20)
    dense = K.qcache_workspace_size(desc, geo, 0)
    anchor = K.qcache_workspace_size(desc, geo, 4096)
    reuse = K.qcache_workspace_size(desc, geo, 4096, reuse=True)
    logits = B * Hq * N * 4
    assert dense <= reuse <= anchor - logits
    if pooled:
        assert reuse == dense and anchor - reuse >= logits + B * Hkv * N * 4
    else:
        assert reuse == anchor - logits
    assert L.kascade_qcache_reuse_decode(ref(desc), ref(geo), p, p, p, p, 4096, p, p, p, reuse - 1,
                                         None) == K.WORKSPACE
    assert L.kascade_qcache_anchor_decode(ref(desc), ref(geo), p, p, p, p, 4096, p, p, None, p,
                                          reuse, None) == K.WORKSPACE
    size = L.kascade_qcache_reuse_workspace_size
    assert size(ref(desc), ref(geo), 0) == 0 and size(ref(desc), None, 1) == 0


def test_growing_workspace_keeps_the_error_word(K, fake):
    ws = K.Workspace("cpu")
    ws.get(256)[:8] = torch.tensor([16, 0, 0, 0, 1, 5, 0, 0], dtype=torch.uint8)
    assert ws.get(4096).numel() == 4096
    assert ws.buf[:8].tolist() == [16, 0, 0, 0, 1, 5, 0, 0]
