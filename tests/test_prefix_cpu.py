"""Decode over a shared prefix without a GPU: the library's argument validation (before any
launch), its workspace sizes and the binding's tensor checks."""
import ctypes

import pytest
import torch

import __graft_entry__

BF, I32 = torch.bfloat16, torch.int32
P = ctypes.c_void_p(1 << 20)            # aligned, never read on these paths
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def K():
    __graft_entry__.build()
    from long_context_anchor_gb300 import kascade
    return kascade


def call(K, desc, geo, prefix, nws, q=P, pages=P, table=P, lens=P, out=P, ws=P, always=0):
    return K._lib.kascade_qcache_prefix_decode(
        None if desc is None else ctypes.byref(desc), None if geo is None else ctypes.byref(geo), q,
        pages, table, lens, prefix, always, out, ws, nws, None)


def test_validation_before_launch(K):
    desc, geo = K.make_desc(2, 8, 2, 128, 1000, K.BF16), K.QCache(64, 40, 16, 0.0, 0.0)
    n = K.qcache_prefix_workspace_size(desc, geo, 512)
    assert n > 0
    for prefix in (-64, -1, 1, 500, 1024, (1 << 31) - 64):     # whole blocks within kv_len
        assert K._lib.kascade_qcache_prefix_workspace_size(ctypes.byref(desc), ctypes.byref(geo),
                                                           prefix) == 0
        assert call(K, desc, geo, prefix, 1 << 40) == K.INVALID_ARG
    assert call(K, desc, geo, 960, 0) == K.WORKSPACE
    for name in ("q", "pages", "out"):
        assert call(K, desc, geo, 512, n, **{name: ODD}) == K.INVALID_ARG
        assert call(K, desc, geo, 512, n, **{name: None}) == K.INVALID_ARG
    for name in ("table", "lens"):
        assert call(K, desc, geo, 512, n, **{name: None}) == K.INVALID_ARG
    assert call(K, desc, geo, 512, n - 1) == K.WORKSPACE
    assert call(K, desc, geo, 512, n, ws=ODD) == K.WORKSPACE
    assert call(K, desc, geo, 512, n, ws=None) == K.WORKSPACE
    for always in (-1, 2):
        assert call(K, desc, geo, 512, n, always=always) == K.INVALID_ARG
    assert call(K, desc, geo, 512, n - 1, always=1) == K.WORKSPACE
    assert call(K, None, geo, 512, n) == K.INVALID_ARG
    assert call(K, desc, None, 512, n) == K.INVALID_ARG
    assert call(K, desc, K.QCache(64, 40, 15, 0.0, 0.0), 512, n) == K.INVALID_ARG  # 960 < kv_len
    assert call(K, desc, K.QCache(48, 40, 32, 0.0, 0.0), 480, n) != K.OK
    assert call(K, K.make_desc(2, 8, 2, 96, 1000, K.BF16), geo, 512, n) == K.UNSUPPORTED


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 1, 1), (3, 16, 2), (128, 64, 8), (512, 32, 8)])
def test_workspace_sizes(K, B, Hq, Hkv, d):
    """The dense call's workspace, and behind it the states of the rows' own parts and two or
    more pieces of each tile of 128 queries."""
    for dtype in (K.BF16, K.F32):
        desc = K.make_desc(B, Hq, Hkv, d, 1 << 17, dtype)
        geo = K.QCache(64, 4096, 2048, 0.0, 0.0)
        dense = K.qcache_workspace_size(desc, geo, 0)
        assert K.qcache_prefix_workspace_size(desc, geo, 0) == dense
        tiles = Hkv * -(-B * (Hq // Hkv) // 128)
        for prefix in (64, 1 << 12, 1 << 17):
            n = K.qcache_prefix_workspace_size(desc, geo, prefix)
            assert n >= dense + B * Hq * (d + 2) * 4 + 2 * tiles * 128 * (d + 2) * 4
            # far below what one product per sequence and run would take
            assert n <= dense + B * Hq * (d + 2) * 4 + 4 * (tiles + 256) * 128 * (d + 8) * 4


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            if name.endswith("workspace_size"):
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


def tensors(B=3, Hq=8, Hkv=2, d=128, bs=32, nb=20, width=5, dtype=BF):
    return dict(q=torch.zeros(B, Hq, d, dtype=dtype),
                pages=torch.zeros(nb, Hkv, bs // 16, 18 * d, dtype=torch.uint8),
                block_table=torch.zeros(B, width, dtype=I32), kv_lens=torch.zeros(B, dtype=I32))


def test_binding_takes_the_documented_call(K, fake):
    ws, t = K.Workspace("cpu"), tensors()
    out = K.qcache_prefix_decode(**t, prefix_len=64, kv_len=100, ws=ws)
    assert out.shape == (3, 8, 128) and out.dtype == BF
    into = torch.empty_like(t["q"])
    assert K.qcache_prefix_decode(**t, prefix_len=0, out=into, scale=0.5, k_scale=2.0, ws=ws,
                                  group_map=[0, 1] * 4) is into
    name, args = fake.calls[-1]
    assert name == "kascade_qcache_prefix_decode" and args[6:8] == (0, 0) and args[8] == into.data_ptr()
    K.qcache_prefix_decode(**t, prefix_len=32, always=True, ws=ws)
    assert [a[6:8] for n, a in fake.calls if n == name] == [(64, 0), (0, 0), (32, 1)]
    sizes = [a for n, a in fake.calls if n == "kascade_qcache_prefix_workspace_size"]
    assert [a[2] for a in sizes] == [64, 0, 32]


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros(3, 8, 64, dtype=BF)), dict(q=torch.zeros(3, 8, 128, dtype=torch.float16)),
    dict(q=torch.zeros(8, 3, 128, dtype=BF).transpose(0, 1)),
    dict(q=torch.zeros(3, 8, 1, 128, dtype=BF)), dict(q=None),
    dict(block_table=torch.zeros(2, 5, dtype=I32)), dict(block_table=torch.zeros(3, 5)),
    dict(block_table=torch.zeros(3, 10, dtype=I32)[:, ::2]),
    dict(kv_lens=torch.zeros(4, dtype=I32)), dict(kv_lens=torch.zeros(3, dtype=torch.int64)),
    dict(pages=torch.zeros(20, 2, 2, 100, dtype=torch.uint8)),
    dict(out=torch.zeros(3, 8, 128)), dict(out=torch.zeros(2, 8, 128, dtype=BF))])
def test_binding_refuses(K, fake, change):
    args = dict(tensors(), prefix_len=64, ws=K.Workspace("cpu"))
    args.update(change)
    with pytest.raises((ValueError, TypeError)):
        K.qcache_prefix_decode(**args)
    assert not any(n.endswith("decode") for n, _ in fake.calls)


def test_binding_raises_what_the_library_refuses(K):
    desc, geo = K.make_desc(2, 8, 2, 128, 1000, K.BF16), K.QCache(64, 40, 16, 0.0, 0.0)
    for prefix in (-64, 100, 1024):
        with pytest.raises(K.KascadeError):
            K.qcache_prefix_workspace_size(desc, geo, prefix)


@pytest.mark.parametrize("prefix", [1 << 32, (1 << 32) + 64, -(1 << 32) + 64, 1 << 31])
def test_binding_refuses_a_prefix_beyond_32_bits(K, fake, prefix):
    """It is not cut to a length that the library takes."""
    with pytest.raises(K.KascadeError):
        K.qcache_prefix_decode(**tensors(), prefix_len=prefix, ws=K.Workspace("cpu"))
    assert not any(n.endswith("decode") for n, _ in fake.calls)
