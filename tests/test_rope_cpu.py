"""Rotation without a GPU: the oracle's pins, the library's argument validation (before any
launch) and the binding's tensor checks."""
import ctypes
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import rope as R

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def K():
    __graft_entry__.build()
    from long_context_anchor_gb300 import kascade
    return kascade


def test_oracle_turns_by_hand():
    tab = R.table([np.pi / 2, np.pi], 3)
    c, s = R.turn_of(tab, np.array([1, 7]))
    x = np.array([[1.0, 2.0, 3.0, 4.0, 5.0]] * 2)
    half, mag = R.turned(x, c, s, False)          # pairs (0, 2) by 90 degrees, (1, 3) by 180
    assert np.allclose(half[0], [-3, -2, 1, -4, 5]) and np.array_equal(half[1], x[1])
    assert np.allclose(mag[0], [3, 2, 1, 4, 5])
    inter, _ = R.turned(x, c, s, True)            # pairs (0, 1) and (2, 3)
    assert np.allclose(inter[0], [-2, 1, -3, -4, 5])
    c, s = R.turn_of(tab, np.array([[1], [2]]), [1, 0])
    assert np.allclose(R.turned(x[:1], c, s, False)[0], [-1, -2, -3, -4, 5])


def test_oracle_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 64))
    tab = R.table(100.0 ** (-np.arange(32) / 32), 50)
    def at(x, p):
        c, s = R.turn_of(tab, np.array(p))
        return R.turned(x, c, s, True)[0]
    assert np.isclose(np.linalg.norm(at(q, 33)), np.linalg.norm(q))
    assert np.isclose(at(q, 41) @ at(k, 30), at(q, 12) @ at(k, 1))


def test_oracle_norm():
    x = np.array([[3.0, 4.0]])
    assert np.allclose(R.normalised(x, np.array([1.0, 2.0]), 0.0), [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]])


def test_table_on_the_cpu(K):
    tab = K.rope_table([1.0, 0.5], 4, scale=2.0, device="cpu")
    want = 2.0 * R.table([1.0, 0.5], 4)
    assert tab.dtype == torch.float32 and np.abs(tab.numpy() - want).max() < 2.0 ** -23
    with pytest.raises(ValueError):
        K.rope_table([[1.0]], 4, device="cpu")


FAKE = 1 << 20      # an aligned address that these paths never read


def row_call(K, rope=True, B=1, N=4, Hq=4, Hkv=2, d=64, dtype=None, pairs=32, q=FAKE, k=FAKE, wq=0,
             wk=0, eps=1e-6, pos=FAKE, qo=FAKE, ko=FAKE, strides=None, ws=FAKE, nws=256, axes=None,
             n_axes=1, n_pos=10, table=FAKE):
    arr = None if axes is None else (ctypes.c_int32 * len(axes))(*axes)
    r = K.Rope(table, n_pos, pairs, 0, n_axes, arr)
    st = strides or [0, 64 * Hq, 64] * 4
    return K._lib.kascade_qk_norm_rope(ctypes.byref(r) if rope else None, B, N, Hq, Hkv, d,
                                       K.BF16 if dtype is None else dtype, q, k, wq, wk, eps, pos,
                                       qo, ko, (ctypes.c_int64 * 12)(*st), ws, nws, None)


def test_rows_are_validated_before_the_launch(K):
    bad = K.INVALID_ARG
    assert row_call(K, N=0) == K.OK and row_call(K, B=0) == K.OK
    assert row_call(K, d=96) == K.UNSUPPORTED
    assert row_call(K, pairs=24) == K.UNSUPPORTED
    assert row_call(K, pairs=48) == bad                 # 2 * 48 > 64
    assert row_call(K, pairs=0) == bad and row_call(K, n_pos=0) == bad
    assert row_call(K, table=FAKE + 4) == bad and row_call(K, table=None) == bad
    assert row_call(K, n_axes=5) == bad and row_call(K, n_axes=0) == bad
    assert row_call(K, axes=[0] * 31 + [1]) == bad and row_call(K, axes=[0] * 31 + [-1]) == bad
    assert row_call(K, dtype=7) == bad
    assert row_call(K, eps=-1.0) == bad and row_call(K, eps=float("nan")) == bad
    assert row_call(K, eps=float("inf")) == bad
    assert row_call(K, Hq=257) == bad and row_call(K, Hq=0, Hkv=0) == bad and row_call(K, N=-1) == bad
    assert row_call(K, B=1 << 14, N=1 << 14) == K.UNSUPPORTED
    for name in ("q", "k", "qo", "ko"):
        assert row_call(K, **{name: FAKE + 8}) == bad
        assert row_call(K, **{name: None}) == bad
    assert row_call(K, wq=FAKE + 2) == bad
    assert row_call(K, pos=None) == bad and row_call(K, pos=FAKE + 2) == bad
    for i in range(12):
        st = [0, 256, 64] * 4
        st[i] = 4                                        # 8 bytes
        assert row_call(K, strides=st) == bad
        st[i] = -64
        assert row_call(K, strides=st) == bad
    assert row_call(K, ws=FAKE + 16) == K.WORKSPACE and row_call(K, nws=255) == K.WORKSPACE


def append_call(K, rope=True, Hq=4, Hkv=2, d=64, k=FAKE, q=FAKE, qo=FAKE, wk=0, wq=0, eps=1e-6,
                slots=FAKE, T=4, pos=FAKE, cu=0, lens=0, n=0, pages=FAKE, ws=FAKE, nws=256,
                strides=None, bs=16, pairs=32):
    r = K.Rope(FAKE, 10, pairs, 0, 1, None)
    geo = K.QCache(bs, 4, 1, 0.0, 0.0)
    st = strides or [64 * Hkv, 64] * 2 + [64 * Hq, 64] * 2
    return K._lib.kascade_qcache_append_rope(ctypes.byref(geo), ctypes.byref(r) if rope else None,
                                             Hq, Hkv, d, K.BF16, k, FAKE, q,
                                             (ctypes.c_int64 * 8)(*st), wk, wq, eps, slots, T, pos,
                                             cu, lens, n, pages, qo, ws, nws, None)


def test_appends_are_validated_before_the_launch(K):
    bad = K.INVALID_ARG
    assert append_call(K, T=0) == K.OK
    assert append_call(K, bs=48) == K.UNSUPPORTED and append_call(K, pairs=8) == K.UNSUPPORTED
    assert append_call(K, k=FAKE + 8) == bad and append_call(K, q=FAKE + 8) == bad
    assert append_call(K, qo=None) == bad and append_call(K, Hq=0) == bad
    assert append_call(K, slots=None) == bad and append_call(K, pages=FAKE + 4) == bad
    assert append_call(K, wk=FAKE + 2) == bad and append_call(K, wq=FAKE + 2) == bad
    assert append_call(K, eps=-1.0) == bad
    assert append_call(K, pos=None) == bad                              # no positions at all
    assert append_call(K, cu=FAKE, lens=FAKE, n=2) == bad               # both ways
    assert append_call(K, pos=None, cu=FAKE, n=2) == bad
    assert append_call(K, pos=None, lens=FAKE, n=2) == bad
    assert append_call(K, pos=None, cu=FAKE, lens=FAKE, n=0) == bad
    assert append_call(K, pos=None, cu=FAKE, lens=FAKE, n=16385) == K.UNSUPPORTED
    for i in range(8):
        st = [128, 64] * 2 + [256, 64] * 2
        st[i] += 4
        assert append_call(K, strides=st) == bad
    assert append_call(K, nws=0) == K.WORKSPACE and append_call(K, ws=None) == K.WORKSPACE


@pytest.mark.parametrize("call", ["Hq=0, q=None, qo=None", "Hq=0, q=None, qo=None, T=5000",
                                  "Hq=0, q=None, qo=None, pos=None, cu=FAKE, lens=FAKE, n=2",
                                  "pos=None, cu=FAKE, lens=FAKE, n=2, T=0"])
def test_appends_of_keys_or_queries_alone_reach_the_launch(K, call):
    """What the library reckons in front of a launch, in a process that sees no GPU: the
    launch fails with a status, and the process lives to report it."""
    code = ("import os, sys; os.environ['CUDA_VISIBLE_DEVICES'] = ''; sys.path[:0] = %r\n"
            "from test_rope_cpu import FAKE, append_call\n"
            "from long_context_anchor_gb300 import kascade as K\n"
            "sys.exit(0 if append_call(K, %s) == K.CUDA else 3)\n"
            % ([str(Path(__file__).parent), str(Path(__file__).parent.parent)], call))
    assert subprocess.run([sys.executable, "-c", code], timeout=300).returncode == 0


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def fake(K, monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(K, "_lib", rec)
    monkeypatch.setattr(K, "_stream", lambda stream=None: None)
    monkeypatch.setattr(K, "_DEVICE_TYPE", "cpu")
    return rec


def last(fake, name):
    return [a for n, a in fake.calls if n == name][-1]


def test_binding_takes_the_documented_layouts(K, fake):
    ws = K.Workspace("cpu")
    proj = torch.zeros(2, 9, 8, 64, dtype=BF)
    q, k = proj[:, :, :4].transpose(1, 2), proj[:, :, 4:6].transpose(1, 2)
    tab, pos = torch.zeros(20, 2, 32), torch.zeros(2, 9, dtype=I32)
    gq, gk = K.qk_norm_rope(q, k, pos, tab, ws=ws)
    assert gq.shape == (2, 4, 9, 64) and gk.shape == (2, 2, 9, 64) and gq.is_contiguous()
    args = last(fake, "kascade_qk_norm_rope")
    assert list(args[15]) == [9 * 512, 512, 64, 9 * 512, 512, 64, 4 * 9 * 64, 64, 9 * 64,
                              2 * 9 * 64, 64, 9 * 64]
    assert args[1:7] == (2, 9, 4, 2, 64, K.BF16)
    # rows, one axis of length 1 whose stride does not matter; q alone; in place
    row = torch.zeros(1, 4, 64, dtype=BF)
    assert K.qk_norm_rope(row, None, pos[0, :1], tab, q_out=row, ws=ws)[0] is row
    # several axes, one more than the pairs name
    K.qk_norm_rope(q, k, torch.zeros(3, 2, 9, dtype=I32), tab, axes=[i % 2 for i in range(32)], ws=ws)
    K.qk_norm_rope(q, k, q_weight=torch.zeros(64, dtype=BF), ws=ws)       # a norm alone
    pages, slots = torch.zeros(4, 2, 1, 1152, dtype=torch.uint8), torch.zeros(9, dtype=I32)
    rows = proj[0]
    got = K.qcache_append_rope(rows[:, 4:6], rows[:, 6:], slots, pages, tab, positions=pos[0],
                               q=rows[:, :4], ws=ws)
    assert got.shape == (9, 4, 64)
    cu, lens = torch.zeros(4, dtype=I32), torch.zeros(3, dtype=I32)
    got = K.qcache_append_rope(rows[:, 4:6], rows[:, 6:], slots, pages, tab, q=rows[:3, :4],
                               cu_new=cu, kv_lens=lens, ws=ws)
    assert got.shape == (3, 4, 64)
    assert K.qcache_append_rope(rows[:, 4:6], rows[:, 6:], slots, pages, tab, positions=pos[0],
                                ws=ws) is None


def test_binding_refuses(K, fake):
    ws = K.Workspace("cpu")
    q, k = torch.zeros(9, 4, 64, dtype=BF), torch.zeros(9, 2, 64, dtype=BF)
    tab, pos = torch.zeros(20, 2, 32), torch.zeros(9, dtype=I32)
    call = lambda **kw: K.qk_norm_rope(**dict(dict(q=q, k=k, positions=pos, rope=tab, ws=ws), **kw))
    call()
    n = len(fake.calls)
    wide = torch.zeros(9, 4, 65, dtype=BF)
    wrong = [dict(q=None), dict(q=q[0]), dict(q=q.half()), dict(q=wide[..., :64]),
             dict(q=wide[..., 1:]), dict(k=k[:8]), dict(k=k.float()), dict(k=k[..., :32]),
             dict(k=k.unsqueeze(0)), dict(positions=None), dict(positions=pos[:8]),
             dict(positions=pos.long()), dict(positions=pos.expand(2, 9)), dict(rope=None),
             dict(rope=tab.double()), dict(rope=tab[:, 0]), dict(rope=tab.transpose(0, 2)),
             dict(axes=[0] * 31), dict(axes=[0] * 32), dict(q_weight=torch.zeros(64)),
             dict(k_weight=torch.zeros(32, dtype=BF)), dict(q_out=torch.zeros(9, 4, 64)),
             dict(q_out=torch.zeros(1, 4, 64, dtype=BF).expand(9, 4, 64)),
             dict(q_out=torch.zeros(9, 3, 64, dtype=BF)), dict(k=None, k_out=k),
             dict(k=None, k_weight=torch.zeros(64, dtype=BF)), dict(k_out=torch.zeros(9, 4, 64, dtype=BF))]
    for kw in wrong:
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    square = torch.zeros(4, 4, 64, dtype=BF)
    with pytest.raises(ValueError):                 # the input's memory, other order
        K.qk_norm_rope(square, None, pos[:4], tab, q_out=square.transpose(0, 1), ws=ws)
    pages, slots = torch.zeros(4, 2, 1, 1152, dtype=torch.uint8), torch.zeros(9, dtype=I32)
    cu, lens = torch.zeros(4, dtype=I32), torch.zeros(3, dtype=I32)
    call = lambda **kw: K.qcache_append_rope(**dict(dict(k=k, v=k, slot_map=slots, pages=pages,
                                                         rope=tab, positions=pos, ws=ws), **kw))
    call()
    for kw in [dict(positions=None), dict(cu_new=cu, kv_lens=lens), dict(positions=None, cu_new=cu),
               dict(positions=None, kv_lens=lens), dict(rope=None), dict(q=q[:8]), dict(q=q.float()),
               dict(q=q[0]), dict(positions=None, cu_new=cu, kv_lens=lens, q=q),
               dict(positions=None, cu_new=cu[:3], kv_lens=lens), dict(q_out=q),
               dict(q_weight=torch.zeros(64, dtype=BF)), dict(v=k[:8]), dict(k=k.half()),
               dict(axes=[0] * 32), dict(slot_map=slots.long()), dict(pages=pages.float())]:
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    assert len([c for c in fake.calls[n:] if "rope" in c[0]]) == 1


def test_binding_refuses_outputs_whose_rows_meet(K, fake):
    ws, base = K.Workspace("cpu"), torch.zeros(1 << 14, dtype=BF)
    tab, pos = torch.zeros(20, 2, 32), torch.zeros(9, dtype=I32)
    q = torch.zeros(9, 4, 64, dtype=BF)
    slots, pages = torch.zeros(9, dtype=I32), torch.zeros(4, 4, 1, 1152, dtype=torch.uint8)

    def both(strides, shape=q.shape):
        out = base.as_strided(shape, strides)
        K.qk_norm_rope(q[:shape[0], :shape[1]], None, pos[:shape[0]], tab, q_out=out, ws=ws)
        n = shape[0]
        K.qcache_append_rope(q[:n], q[:n], slots[:n], pages, tab, positions=pos[:n],
                             q=q[:n, :shape[1]], q_out=out, ws=ws)

    for strides in [(256, 64, 1), (64, 576, 1), (320, 72, 1), (1024, 64, 1)]:
        both(strides)
    both((8, 64, 1), (1, 4, 64))                    # one token: its stride is not used
    both((64, 8, 1), (9, 1, 64))
    n = len(fake.calls)
    for strides in [(64, 64, 1), (256, 32, 1), (248, 64, 1), (64, 568, 1), (56, 576, 1), (0, 64, 1),
                    (256, 0, 1)]:
        with pytest.raises(ValueError):
            both(strides)
    # sequences that reach into each other
    four, pos2 = torch.zeros(2, 4, 3, 64, dtype=BF), torch.zeros(2, 3, dtype=I32)
    for first in (64 * 11, 0, 8):
        with pytest.raises(ValueError):
            K.qk_norm_rope(four, None, pos2, tab, ws=ws,
                           q_out=base.as_strided(four.shape, (first, 64, 256, 1)))
    assert len(fake.calls) == n
    K.qk_norm_rope(four, None, pos2, tab, ws=ws, q_out=base.as_strided(four.shape, (64 * 12, 64, 256, 1)))


def test_binding_takes_one_row_in_place_whatever_its_strides(K, fake):
    """Strides of axes of length 1 say nothing about the order."""
    ws, proj = K.Workspace("cpu"), torch.zeros(1, 8, 64, dtype=BF)
    tab, pos = torch.zeros(20, 2, 32), torch.zeros(1, dtype=I32)
    q, k, v = proj[:, :4], proj[:, 4:6], proj[:, 6:]
    flat = proj.view(-1)[:256].view(1, 4, 64), proj.view(-1)[256:384].view(1, 2, 64)
    assert flat[0].data_ptr() == q.data_ptr() and flat[0].stride() != q.stride()
    out = K.qk_norm_rope(q, k, pos, tab, q_out=flat[0], k_out=flat[1], ws=ws)
    assert out[0] is flat[0] and out[1] is flat[1]
    slots, pages = torch.zeros(1, dtype=I32), torch.zeros(4, 2, 1, 1152, dtype=torch.uint8)
    assert K.qcache_append_rope(k, v, slots, pages, tab, positions=pos, q=q, q_out=flat[0],
                                ws=ws) is flat[0]
    one = torch.zeros(4, 1, 64, dtype=BF)           # one head
    K.qk_norm_rope(one, None, pos.expand(4).contiguous(), tab,
                   q_out=one.as_strided((4, 1, 64), (64, 256, 1)), ws=ws)
    square = torch.zeros(4, 4, 64, dtype=BF)
    for call in (lambda t: K.qk_norm_rope(square, None, pos.expand(4).contiguous(), tab, q_out=t, ws=ws),
                 lambda t: K.qcache_append_rope(square[:, :2], square[:, :2], slots.expand(4).contiguous(),
                                                pages, tab, positions=pos.expand(4).contiguous(),
                                                q=square, q_out=t, ws=ws)):
        call(square)
        with pytest.raises(ValueError):
            call(square.transpose(0, 1))


@pytest.mark.parametrize("bad", [4, -1, 1 << 32, -(1 << 32), (1 << 32) + 1])
def test_binding_refuses_axes_that_are_none(K, fake, bad):
    """Nothing is cut to 32 bits on its way into the library."""
    ws, q, cu = K.Workspace("cpu"), torch.zeros(3, 4, 64, dtype=BF), torch.zeros(4, dtype=I32)
    tab, slots = torch.zeros(20, 2, 32), torch.zeros(3, dtype=I32)
    pages = torch.zeros(4, 4, 1, 1152, dtype=torch.uint8)
    call = lambda axes: K.qcache_append_rope(q, q, slots, pages, tab, cu_new=cu, kv_lens=slots, q=q,
                                             axes=axes, ws=ws)
    call([0] * 31 + [3])
    n = len(fake.calls)
    with pytest.raises(ValueError):
        call([0] * 31 + [bad])
    with pytest.raises(ValueError):
        call([bad] * 32)
    assert len(fake.calls) == n
