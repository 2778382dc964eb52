"""Norm and rotation of queries and keys on the GPU, through the binding, against the
float64 oracle (oracle/rope.py).

Tolerance of an element y = a c - b s (or b c + a s), M = |a c| + |b s| with the oracle's
normalised a, b: two products and a sum in fp32, each off by at most 2^-24 of its value:
2^-23 M. A norm's sum of d squares is off by at most d 2^-24 of itself (all terms are
positive), its mean and eps by 2 2^-24, rsqrt by 2^-22 (two units), the factors r and w by
2 2^-24: half of the first two, 2^-22 and the last, at most (d / 2 + 8) 2^-24 of a and b.
Then half a step of the output's type."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
from gpu_helpers import f64
from oracle import qcache as Q
from oracle import rope as R

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPS = 1e-6
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def K():
    __graft_entry__.build()
    from long_context_anchor_gb300 import kascade
    return kascade


def ints(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=I32).cuda()


def make_table(K, pairs, n):
    tab = K.rope_table(10000.0 ** (-np.arange(pairs) / pairs), n)
    assert tab.shape == (n, 2, pairs) and tab.dtype == F32
    return tab


def axes_of(kind, pairs):
    if kind is None:
        return None
    return [i % 3 for i in range(pairs)] if kind == "cyclic" else \
        [0 if i < pairs // 4 else 1 if i < pairs // 2 else 2 for i in range(pairs)]


def expected(x, tab, pos, axes, weight, interleaved, dtype):
    """(reference, tolerance) of rows x [..., H, d] with positions [...] ([axes, ...])."""
    y = f64(x)
    d = y.shape[-1]
    rel = 2.0 ** -23
    if weight is not None:
        y = R.normalised(y, f64(weight), EPS)
        rel += (d / 2 + 8) * 2.0 ** -24
    mag = np.abs(y)
    if tab is not None:
        cos, sin = R.turn_of(f64(tab), pos, axes)
        y, mag = R.turned(y, cos[..., None, :], sin[..., None, :], interleaved)
    tol = rel * mag
    return y, tol + HALF[dtype] * (np.abs(y) + tol)


def check(got, want):
    err = np.abs(f64(got) - want[0])
    assert (err <= want[1]).all(), float((err / np.maximum(want[1], 1e-300)).max())


def test_table(K):
    n, freq = 300000, 500000.0 ** (-np.arange(32) / 32)
    tab = f64(K.rope_table(freq, n))
    pick = np.r_[0, 1, 77, n - 2, n - 1]
    angle = pick[:, None] * freq
    want = np.stack([np.cos(angle), np.sin(angle)], 1)
    # 64-bit angles are off by half a step of themselves, at most 2^-53 * 3e5
    assert (np.abs(tab[pick] - want) <= 2.0 ** -25 + 2.0 ** -34).all()


@pytest.mark.parametrize("T,Hq,Hkv,d,pairs,dtype,inter,axes,norm", [
    (1, 32, 8, 128, 64, BF, False, None, "qk"),
    (8, 4, 2, 64, 32, F32, False, None, "qk"),
    (7, 5, 3, 128, 16, BF, True, None, ""),
    (33, 1, 1, 64, 16, F32, True, "cyclic", "q"),
    (129, 9, 1, 128, 48, F32, False, "sections", "k"),
    (1000, 32, 8, 128, 64, BF, True, "sections", "qk"),
    (4001, 64, 8, 64, 32, BF, False, None, ""),
    (3000, 6, 0, 128, 32, F32, False, "cyclic", "q"),
    (5, 256, 256, 64, 32, BF, False, None, "qk"),
    (77, 3, 2, 64, 0, BF, False, None, "qk")])
def test_rows(K, T, Hq, Hkv, d, pairs, dtype, inter, axes, norm):
    """Rows of a projection's output, taken where they lie."""
    rng = np.random.default_rng(T + d)
    proj = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, d)) * 3).to(dtype).cuda()
    before = proj.clone()
    q, k = proj[:, :Hq], proj[:, Hq:Hq + Hkv] if Hkv else None
    tab = make_table(K, pairs, 700) if pairs else None
    ax = axes_of(axes, pairs)
    pos = rng.integers(0, 700, (T,) if ax is None else (3, T))
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).to(dtype).cuda() for _ in range(2)]
    wq, wk = w[0] if "q" in norm else None, w[1] if "k" in norm and Hkv else None
    gq, gk = K.qk_norm_rope(q, k, ints(pos) if pairs else None, tab, q_weight=wq, k_weight=wk,
                            eps=EPS, interleaved=inter, axes=ax)
    assert torch.equal(proj, before) and gq.is_contiguous() and gq.shape == q.shape
    check(gq, expected(q, tab, pos, ax, wq, inter, dtype))
    if Hkv:
        check(gk, expected(k, tab, pos, ax, wk, inter, dtype))
    else:
        assert gk is None
    assert K.default_workspace("cuda").device_error() == K.OK


@pytest.mark.parametrize("B,N,Hq,Hkv,d,dtype", [(1, 300, 8, 2, 128, BF), (3, 65, 4, 4, 64, F32),
                                                (2, 2500, 16, 8, 128, BF)])
def test_prefill_layout(K, B, N, Hq, Hkv, d, dtype):
    """From the projection's [B,N,heads,d] to the prefill calls' [B,heads,N,d]."""
    rng = np.random.default_rng(N)
    proj = torch.from_numpy(rng.standard_normal((B, N, Hq + Hkv, d))).to(dtype).cuda()
    q, k = proj[:, :, :Hq].transpose(1, 2), proj[:, :, Hq:].transpose(1, 2)
    tab = make_table(K, d // 2, N + 9)
    pos = np.stack([np.arange(N) + b for b in range(B)])
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal((2, d))).to(dtype).cuda()
    gq, gk = K.qk_norm_rope(q, k, ints(pos), tab, q_weight=w[0], k_weight=w[1], eps=EPS)
    assert gq.shape == (B, Hq, N, d) and gq.is_contiguous() and gk.is_contiguous()
    rows = lambda t: t.transpose(1, 2)
    check(rows(gq), expected(rows(q), tab, pos, None, w[0], False, dtype))
    check(rows(gk), expected(rows(k), tab, pos, None, w[1], False, dtype))
    # the same in place, bit for bit
    iq, ik = K.qk_norm_rope(q, k, ints(pos), tab, q_weight=w[0], k_weight=w[1], eps=EPS, q_out=q,
                            k_out=k)
    assert iq is q and torch.equal(iq, gq) and torch.equal(ik, gk)


def test_positions_outside_the_table(K):
    rng = np.random.default_rng(5)
    q = torch.from_numpy(rng.standard_normal((6, 4, 64))).to(F32).cuda()
    tab = make_table(K, 32, 10)
    pos = np.array([0, 9, 10, -1, 2 ** 31 - 1, 3])
    ws = K.Workspace("cuda")
    got, _ = K.qk_norm_rope(q, None, ints(pos), tab, ws=ws)
    assert ws.device_error() == K.BAD_INPUT and ws.device_error() == K.OK
    check(got, expected(q, tab, pos, None, None, False, F32))
    assert torch.equal(got[2:5], q[2:5])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kind", ["cyclic", "sections"])
def test_one_axis_outside_the_table(K, kind, inter):
    """Its pairs alone keep their values, in rows and in cached keys."""
    rng = np.random.default_rng(15)
    q, v = (torch.from_numpy(rng.standard_normal((6, 4, 64))).to(F32).cuda() for _ in range(2))
    tab, ax = make_table(K, 32, 10), axes_of(kind, 32)
    pos = rng.integers(1, 10, (3, 6))
    pos[0, 1], pos[1, 2], pos[2, 3], pos[:, 4] = 10, -1, 2 ** 31 - 1, 99
    ws = K.Workspace("cuda")
    got, _ = K.qk_norm_rope(q, None, ints(pos), tab, axes=ax, interleaved=inter, ws=ws)
    assert ws.device_error() == K.BAD_INPUT
    check(got, expected(q, tab, pos, ax, None, inter, F32))
    for t, axis in ((1, 0), (2, 1), (3, 2)):
        pairs = np.array([i for i in range(32) if ax[i] == axis])
        kept = np.r_[2 * pairs, 2 * pairs + 1] if inter else np.r_[pairs, pairs + 32]
        assert np.array_equal(f64(got[t])[:, kept], f64(q[t])[:, kept])
    assert torch.equal(got[4], q[4])
    pages, slots = K.qcache_alloc(1, 4, 64, 16), ints(np.arange(6))
    K.qcache_append_rope(q, v, slots, pages, tab, positions=ints(pos), axes=ax, interleaved=inter, ws=ws)
    assert ws.device_error() == K.BAD_INPUT
    ck, _ = K.qcache_read(pages, slots, dtype=F32)
    assert np.array_equal(f64(ck), Q.stored(f32_turned(q, tab, pos, ax, inter)))


@pytest.mark.parametrize("ax", [[0, 2] * 16, [2] * 32, [0] * 16 + [2] * 16])
def test_axes_that_no_pair_follows(K, ax):
    """Positions there may be anything."""
    rng = np.random.default_rng(16)
    q, k = (torch.from_numpy(rng.standard_normal((6, h, 64))).to(BF).cuda() for h in (4, 2))
    tab, pos = make_table(K, 32, 10), rng.integers(0, 10, (4, 6))
    pos[1], pos[3] = -5, 2 ** 31 - 1
    ws = K.Workspace("cuda")
    got = K.qk_norm_rope(q, k, ints(pos), tab, axes=ax, ws=ws)
    assert ws.device_error() == K.OK
    check(got[0], expected(q, tab, pos, ax, None, False, BF))
    check(got[1], expected(k, tab, pos, ax, None, False, BF))
    pages, slots = K.qcache_alloc(1, 2, 64, 16), ints(np.arange(6))
    to = K.qcache_append_rope(k, k, slots, pages, tab, positions=ints(pos), q=q, axes=ax, ws=ws)
    assert ws.device_error() == K.OK and torch.equal(to, got[0])
    ck, _ = K.qcache_read(pages, slots, dtype=F32)
    assert np.array_equal(f64(ck), Q.stored(f32_turned(k, tab, pos, ax, False)))


def test_special_values_stay_in_their_pair(K):
    q = torch.ones(2, 1, 64, dtype=F32, device="cuda")
    q[0, 0, 3], q[1, 0, 60] = float("nan"), float("inf")
    tab = make_table(K, 16, 4)                       # elements 32 .. 63 are not turned
    got, _ = K.qk_norm_rope(q, None, ints([1, 2]), tab)
    bad = ~torch.isfinite(got)
    assert bad[0, 0].nonzero().flatten().tolist() == [3, 19]
    assert bad[1, 0].nonzero().flatten().tolist() == [60] and got[1, 0, 60] == float("inf")


def test_graph_stream_and_empty(K):
    rng = np.random.default_rng(6)
    q = torch.from_numpy(rng.standard_normal((40, 8, 128))).to(BF).cuda()
    k = torch.from_numpy(rng.standard_normal((40, 2, 128))).to(BF).cuda()
    tab, pos = make_table(K, 64, 64), ints(np.arange(40))
    want = K.qk_norm_rope(q, k, pos, tab)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = K.qk_norm_rope(q, k, pos, tab, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ws = K.Workspace("cuda")
    out = torch.empty_like(q), torch.empty_like(k)
    K.qk_norm_rope(q, k, pos, tab, q_out=out[0], k_out=out[1], ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.qk_norm_rope(q, k, pos, tab, q_out=out[0], k_out=out[1], ws=ws)
    q.mul_(2)
    pos.add_(3)
    g.replay()
    want = K.qk_norm_rope(q, k, pos, tab)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    none = K.qk_norm_rope(q[:0], k[:0], pos[:0], tab)
    assert none[0].shape == (0, 8, 128) and none[1].shape == (0, 2, 128)


# ---------------------------------------------------------------- into the cache --

def f32_turned(x, tab, pos, axes, inter):
    """Turned rows as the cache takes them: every product and sum rounded to fp32."""
    cos, sin = R.turn_of(tab.cpu().numpy(), pos, axes)
    return R.turned(x.float().cpu().numpy(), cos[:, None], sin[:, None], inter)[0]


@pytest.mark.parametrize("T,Hq,Hkv,d,pairs,bs,dtype,inter,axes,scales", [
    (1, 4, 1, 128, 64, 64, BF, False, None, (1.0, 1.0)),
    (70, 32, 8, 128, 64, 64, BF, False, None, (1.0, 1.0)),
    (33, 6, 3, 64, 32, 16, BF, True, "cyclic", (0.25, 8.0)),
    (129, 0, 5, 64, 16, 256, F32, False, None, (1.0, 2.0)),
    (300, 8, 8, 128, 48, 32, F32, True, "sections", (1.0, 1.0)),
    (5000, 16, 4, 64, 32, 128, BF, False, "sections", (1.0, 1.0))])
def test_append(K, T, Hq, Hkv, d, pairs, bs, dtype, inter, axes, scales):
    rng = np.random.default_rng(T)
    nb = (T + bs - 1) // bs + 2
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    skip = rng.random(T) < 0.1
    slots[skip] = -1 - rng.integers(0, 5, skip.sum())
    proj = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, d)) * 2).to(dtype).cuda()
    q = proj[:, :Hq] if Hq else None
    k, v = proj[:, Hq:Hq + Hkv], proj[:, Hq + Hkv:]
    tab, ax = make_table(K, pairs, 900), axes_of(axes, pairs)
    pos = rng.integers(0, 900, (T,) if ax is None else (3, T))
    pages = torch.full((nb, Hkv, bs // 16, 18 * d), 255, dtype=torch.uint8, device="cuda")
    same = pages.clone()
    ws = K.Workspace("cuda")
    got = K.qcache_append_rope(k, v, ints(slots), pages, tab, positions=ints(pos), q=q,
                               interleaved=inter, axes=ax, k_scale=scales[0], v_scale=scales[1],
                               ws=ws)
    assert ws.device_error() == K.OK
    if Hq:
        alone, _ = K.qk_norm_rope(q, None, ints(pos), tab, interleaved=inter, axes=ax)
        assert torch.equal(got, alone)
        check(got, expected(q, tab, pos, ax, None, inter, dtype))
    else:
        assert got is None
    ck, cv = K.qcache_read(pages, ints(slots), dtype=F32, k_scale=scales[0], v_scale=scales[1])
    live = slots >= 0
    assert np.array_equal(f64(ck)[live], Q.stored(f32_turned(k, tab, pos, ax, inter), scales[0])[live])
    assert np.array_equal(f64(cv)[live], Q.stored(f64(v), scales[1])[live])
    assert not f64(ck)[~live].any()
    # nothing else is written: the rows' bytes equal those that qcache_append writes
    # of the turned rows
    turned = torch.from_numpy(f32_turned(k, tab, pos, ax, inter)).cuda()
    K.qcache_append(turned, v.float().contiguous(), ints(slots), same, k_scale=scales[0],
                    v_scale=scales[1])
    assert torch.equal(pages, same)


@pytest.mark.parametrize("dtype,d,inter", [(BF, 128, False), (F32, 64, True)])
def test_append_with_norm(K, dtype, d, inter):
    """A normalised key is what qk_norm_rope gives in fp32, then quantised."""
    rng = np.random.default_rng(d)
    T, Hq, Hkv, bs = 50, 12, 3, 16
    q, k, v = (torch.from_numpy(rng.standard_normal((T, h, d))).to(dtype).cuda()
               for h in (Hq, Hkv, Hkv))
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal((2, d))).to(dtype).cuda()
    tab, pos = make_table(K, d // 2, 64), rng.integers(0, 64, T)
    slots = rng.permutation(64)[:T]
    pages = K.qcache_alloc(4, Hkv, d, bs)
    got = K.qcache_append_rope(k, v, ints(slots), pages, tab, positions=ints(pos), q=q,
                               q_weight=w[0], k_weight=w[1], eps=EPS, interleaved=inter)
    check(got, expected(q, tab, pos, None, w[0], inter, dtype))
    _, k32 = K.qk_norm_rope(q.float(), k.float(), ints(pos), tab, q_weight=w[0].float(),
                            k_weight=w[1].float(), eps=EPS, interleaved=inter)
    ck, cv = K.qcache_read(pages, ints(slots), dtype=F32)
    assert np.array_equal(f64(ck), Q.stored(f64(k32)))
    assert np.array_equal(f64(cv), Q.stored(f64(v)))


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("dtype,d,norm", [(BF, 128, True), (F32, 64, True), (BF, 64, False)])
def test_append_without_a_rotation(K, dtype, d, norm, planned):
    """The C call without a rotation, and so without positions (the binding wants one): a norm
    alone, or what qcache_append does."""
    rng = np.random.default_rng(d + planned)
    T, Hq, Hkv, bs, B = 50, 12, 3, 16, 4
    q = torch.from_numpy(rng.standard_normal((B if planned else T, Hq, d))).to(dtype).cuda()
    k, v = (torch.from_numpy(rng.standard_normal((T, Hkv, d))).to(dtype).cuda() for _ in range(2))
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal((2, d))).to(dtype).cuda()
    slots = ints(rng.permutation(64)[:T])
    cu, lens = ints([0, 20, 20, 21, T]), ints([20, 7, 9, T])
    pages, out, ws = K.qcache_alloc(4, Hkv, d, bs), torch.empty_like(q), K.Workspace("cuda")
    geo, buf = K.QCache(bs, 4, 1, 0.0, 0.0), ws.get(256)
    strides = [Hkv * d, d] * 2 + [Hq * d, d] * 2
    at = lambda t, used=True: t.data_ptr() if used else None
    status = K._lib.kascade_qcache_append_rope(
        ctypes.byref(geo), None, Hq, Hkv, d, K.F32 if dtype is F32 else K.BF16, at(k), at(v), at(q),
        (ctypes.c_int64 * 8)(*strides), at(w[1], norm), at(w[0], norm), EPS, at(slots), T, None,
        at(cu, planned), at(lens, planned), B if planned else 0, at(pages), at(out), at(buf),
        buf.numel(), torch.cuda.current_stream().cuda_stream)
    assert status == K.OK and ws.device_error() == K.OK
    wq, wk = (w[0], w[1].float()) if norm else (None, None)
    assert torch.equal(out, K.qk_norm_rope(q, None, q_weight=wq, eps=EPS)[0])
    k32 = K.qk_norm_rope(k.float(), None, q_weight=wk, eps=EPS)[0]
    ck, cv = K.qcache_read(pages, slots, dtype=F32)
    assert np.array_equal(f64(ck), Q.stored(f64(k32)))
    assert np.array_equal(f64(cv), Q.stored(f64(v)))


@pytest.mark.parametrize("B", [1, 3, 33, 1100])
def test_append_from_a_plan(K, B):
    """Positions from the plan's own outputs: sequences that start, grow by several
    tokens, stay, shrink and end; rows behind the last new token are padding."""
    rng = np.random.default_rng(B)
    bs, Hq, Hkv, d = 16, 4, 2, 64
    lens = rng.integers(0, 60, B)
    new = rng.choice([-7, 0, 1, 1, 1, 5, 19], B)
    new[rng.random(B) < 0.1] = -1000
    if B == 1:
        new[0] = 3
    width = 6
    have = [(n + bs - 1) // bs for n in lens]
    nb = sum(have) + 3 * B
    ids = rng.permutation(nb)
    table, at = np.full((B, width), -1), 0
    for b, m in enumerate(have):
        table[b, :m] = ids[at:at + m]
        at += m
    free = np.concatenate([ids[at:], np.full(at, -1)])
    total = int(np.maximum(0, np.where(lens + new > lens, new, 0)).sum())
    tbl = ints(table)
    slots, cu, now, _ = K.qcache_plan(ints(lens), ints(new), tbl, ints(free), ints([nb - at]), bs,
                                      total + 9)
    T = total + 9
    k, v = (torch.from_numpy(rng.standard_normal((T, Hkv, d))).to(BF).cuda() for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((B, Hq, d))).to(BF).cuda()
    tab = make_table(K, d // 2, width * bs)
    pages = K.qcache_alloc(nb, Hkv, d, bs)
    ws = K.Workspace("cuda")
    got = K.qcache_append_rope(k, v, slots, pages, tab, q=q, cu_new=cu, kv_lens=now, ws=ws)
    assert ws.device_error() == K.OK
    to = np.maximum(0, lens + new)
    assert np.array_equal(now.cpu().numpy(), to)
    pos = np.concatenate([np.arange(a, b) for a, b in zip(lens, to)] + [np.zeros(9)]).astype(int)
    assert len(pos) == T
    check(got, expected(q, tab, np.maximum(0, to - 1), None, None, False, BF))
    ck, _ = K.qcache_read(pages, slots, dtype=F32)
    want = Q.stored(f32_turned(k, tab, pos, None, False))
    want[total:] = 0
    assert np.array_equal(f64(ck), want)


def test_append_bad_positions_and_slots(K):
    rng = np.random.default_rng(9)
    k, v = (torch.from_numpy(rng.standard_normal((4, 2, 64))).to(F32).cuda() for _ in range(2))
    tab, pages = make_table(K, 32, 8), K.qcache_alloc(2, 2, 64, 16)
    ws = K.Workspace("cuda")
    pos = np.array([1, 8, 2, 3])
    K.qcache_append_rope(k, v, ints([0, 1, 5, 32]), pages, tab, positions=ints(pos), ws=ws)
    assert ws.device_error() == K.BAD_INPUT
    ck, cv = K.qcache_read(pages, ints([0, 1, 5]), dtype=F32)
    assert np.array_equal(f64(ck), Q.stored(f32_turned(k, tab, pos, None, False))[:3])
    assert np.array_equal(f64(cv), Q.stored(f64(v))[:3])


@pytest.mark.parametrize("axis", [0, 1, 2])
def test_rows_that_lie_beyond_32_bits(K, axis):
    """Strides of 2^31 elements and more between sequences, heads or tokens, in and out."""
    rng = np.random.default_rng(20 + axis)
    shape = (2, 2, 2, 64)
    strides = [256, 128, 64, 1]
    strides[axis] = (1 << 31) + 64
    base = torch.empty((1 << 31) + 1024, dtype=BF, device="cuda")
    q = base.as_strided(shape, strides)
    rows = torch.from_numpy(rng.standard_normal(shape)).to(BF).cuda()
    q.copy_(rows)
    pos = torch.tensor([[3, 0], [7, 5]], dtype=I32, device="cuda")
    tab = K.rope_table(100.0 ** (-np.arange(32) / 32), 8)
    want, _ = K.qk_norm_rope(rows, None, pos, tab)
    got, _ = K.qk_norm_rope(q, None, pos, tab)
    assert torch.equal(got, want)
    K.qk_norm_rope(rows, None, pos, tab, q_out=q)
    assert torch.equal(q, want)
