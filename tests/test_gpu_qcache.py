"""Paged 4-bit key/value cache on the GPU, through the binding, against the
float64 oracle (oracle/qcache.py).

Tolerances of attention outputs, per element, with A = sum_j p_j |v_j| the mean
magnitude the row averages over and e_s the error of a logit:
  e_s   the fp32 sum of d products: d * 2^-23 * sigma sum |q_i k_i| (an fp32 q as
        two fp16 terms adds 2^-21 max|q| per element: sigma 2^-21 max|q| sum |k_i|);
  bf16  2^-8 |out| (the output's half step) + (2^-11 + 2 e_s) A (weights held in
        fp16, half a step 2^-11; a logit error moves numerator and sum);
  fp32  2^-24 |out| + (2^-21 + n 2^-23 + 2 e_s) A (weights as two fp16 terms, fp32
        sums over n keys).
  Weights are held as multiples of 2^-24 of 2^14 p: half a step adds 2^-39 p_max sum_j |v_j|,
        which these bounds leave out. It matters where every heavy key's V is zero
        (test_dense_weights_below_the_smallest_step has it).
Everything the cache stores or plans is compared exactly."""
import numpy as np
import pytest
import torch

import __graft_entry__
from gpu_helpers import f64
from oracle import qcache as Q
from oracle.topk import topk_indices

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def K():
    __graft_entry__.build()
    from long_context_anchor_gb300 import kascade
    return kascade


def ints(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=I32).cuda()


def table_of(rng, lens, bs, nb, width):
    """Random distinct blocks for every sequence; -1 where it has none."""
    ids = rng.permutation(nb)
    table = np.full((len(lens), width), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(lens):
        m = (n + bs - 1) // bs
        table[b, :m] = ids[at:at + m]
        at += m
    return table


def filled(K, rng, lens, Hkv, d, bs, dtype=BF, k_scale=1.0, v_scale=1.0, spare=2, width=None):
    """Pages whose unused bytes are all 0xff (NaN scales), the sequences' rows
    appended on the GPU; (pages, table, per-sequence stored K, V from the
    oracle's reading of the pages' bytes)."""
    need = sum((n + bs - 1) // bs for n in lens)
    width = width or max(1, max((n + bs - 1) // bs for n in lens))
    nb = need + spare
    table = table_of(rng, lens, bs, nb, width)
    pages = torch.full((nb, Hkv, bs // 16, 18 * d), 255, dtype=torch.uint8, device="cuda")
    slots = np.concatenate([table[b, np.arange(n) // bs] * bs + np.arange(n) % bs
                            for b, n in enumerate(lens)] + [np.zeros(0, dtype=np.int64)])
    k = torch.from_numpy(rng.standard_normal((len(slots), Hkv, d)) * k_scale).to(dtype).cuda()
    v = torch.from_numpy(rng.standard_normal((len(slots), Hkv, d)) * v_scale).to(dtype).cuda()
    K.qcache_append(k, v, ints(slots), pages, k_scale=k_scale, v_scale=v_scale)
    return pages, table


def bounds(q, k, v, p, sel, out, scale, f32):
    """The tolerance above for one head's output."""
    qa, ka = np.abs(q), np.abs(k[sel])
    d = len(q)
    es = d * 2.0 ** -23 * scale * (ka @ qa).max()
    if f32:
        es += scale * 2.0 ** -21 * qa.max() * ka.sum(-1).max()
    avg = p @ np.abs(v[sel])
    if f32:
        return 2.0 ** -24 * np.abs(out) + (2.0 ** -21 + len(sel) * 2.0 ** -23 + 2 * es) * avg
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2 * es) * avg


def check_attention(q, got, pages, table, lens, Hkv, d, heads_kv, sets=None, pooled=False,
                    k_scale=1.0, v_scale=1.0, scores=None, scale=None, max_units=40):
    """Every (sequence, head), or a sample of max_units sequences' heads, against the oracle."""
    f32 = q.dtype == F32
    qn, on, pg = f64(q), f64(got), pages.cpu().numpy()
    scale = d ** -0.5 if scale is None else scale
    B, Hq = qn.shape[:2]
    units = [(b, g) for b in range(B) for g in range(Hkv)]
    if len(units) > max_units:
        pick = np.random.default_rng(7).choice(len(units), max_units, replace=False)
        units = [units[i] for i in pick]
    for b, g in units:
        n = lens[b]
        k, v = Q.rows_of(pg, table[b], n, g, d, k_scale, v_scale)
        for h in [h for h in range(Hq) if heads_kv[h] == g]:
            sel = np.arange(n) if sets is None else sets[b][g if pooled else h]
            ref, logits, p = Q.attention(qn[b, h], k, v, scale, sel)
            if len(sel) == 0:
                assert not on[b, h].any(), (b, h)
                continue
            tol = bounds(qn[b, h], k, v, p, sel, ref, scale, f32)
            err = np.abs(on[b, h] - ref)
            assert (err <= tol).all(), (b, h, float((err / tol).max()))
            if scores is not None:
                row = f64(scores[b, h])
                assert (row[n:] == -np.inf).all()
                es = (d * 2.0 ** -23 + 2.0 ** -24) * scale * (np.abs(k) @ np.abs(qn[b, h]))
                es += 2.0 ** -21 * scale * np.abs(qn[b, h]).max() * np.abs(k).sum(-1)
                assert (np.abs(row[:n] - logits) <= es + 1e-30).all(), (b, h)


# ---------------------------------------------------------------- rows --

def special_rows(rng, T, Hkv, d):
    """Rows where rounding matters: ties of the codes and of the scale, tiny and
    huge blocks, zeros, infinities, a NaN."""
    x = rng.standard_normal((T, Hkv, d)) * np.exp(rng.uniform(-8, 4, (T, Hkv, 1)))
    b = x.reshape(T, Hkv, d // 16, 16)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for t in range(T):
        kind = t % 6
        s = 2.0 ** rng.integers(-6, 5) * rng.integers(8, 16) / 8
        if kind == 0:      # every code tie of a representable scale
            b[t, :, :, :8] = ties * s
            b[t, :, :, 8:] = -ties * s
        elif kind == 1:    # amax / 6 halfway between two scales
            b[t, 0, 0] *= 0.01 * s / np.abs(b[t, 0, 0]).max()
            b[t, 0, 0, 3] = 6.0 * s * (1 + 1 / 16)
        elif kind == 2 and t % 4 == 0:
            b[t, 0, 0] = 0.0
            b[t, 0, 1] = 6.0 * 2.0 ** -10 * (1 + rng.integers(-1, 2) / 64)
            b[t, -1, -1, 5] = 1e5
    return x


@pytest.mark.parametrize("d,bs,dtype,Hkv,T", [
    (128, 64, BF, 8, 70), (64, 16, BF, 3, 33), (128, 16, F32, 2, 40), (64, 256, F32, 1, 1),
    (64, 32, BF, 5, 129), (128, 128, BF, 1, 300)])
@pytest.mark.parametrize("ks,vs", [(1.0, 1.0), (0.125, 4.0)])
def test_append_read_exact(K, d, bs, dtype, Hkv, T, ks, vs):
    rng = np.random.default_rng(T * d + bs)
    nb = (T + bs - 1) // bs + 2
    k = torch.from_numpy(special_rows(rng, T, Hkv, d) * ks).to(dtype)
    v = torch.from_numpy(special_rows(rng, T, Hkv, d) * vs).to(dtype)
    slots = rng.permutation(nb * bs)[:T]
    pad = rng.random(T) < 0.1
    slots[pad] = -1
    pages = torch.full((nb, Hkv, bs // 16, 18 * d), 255, dtype=torch.uint8, device="cuda")
    ws = K.Workspace()
    K.qcache_append(k.cuda(), v.cuda(), ints(slots), pages, ks, vs, ws=ws)
    gk, gv = K.qcache_read(pages, ints(slots), dtype=F32, k_scale=ks, v_scale=vs, ws=ws)
    bk, bv = K.qcache_read(pages, ints(slots), dtype=BF, k_scale=ks, v_scale=vs, ws=ws)
    assert ws.device_error() == K.OK
    for x, got, b16, scale in ((k, gk, bk, ks), (v, gv, bv, vs)):
        want = Q.stored(f64(x), scale)
        want[pad] = 0.0
        assert np.array_equal(f64(got), want)
        assert torch.equal(b16.float(), got)        # exact in bf16
    # rows of other slots are as they were
    pg = pages.cpu().numpy()
    used = np.zeros(nb * bs, dtype=bool)
    used[slots[~pad]] = True
    for f in Q.group_fields(pg, d):                  # [nb, Hkv, groups, 16, bytes]
        rest = f.transpose(0, 2, 3, 1, 4).reshape(nb * bs, -1)[~used]
        assert (rest == 255).all()


def test_append_takes_prefill_layout_and_strides(K):
    rng = np.random.default_rng(3)
    Hkv, N, d, bs = 4, 77, 128, 32
    nb = (N + bs - 1) // bs
    kv = torch.from_numpy(rng.standard_normal((2, Hkv, N, d))).to(BF).cuda()
    slots = ints(rng.permutation(nb * bs)[:N])
    a = K.qcache_alloc(nb, Hkv, d, bs)
    b = K.qcache_alloc(nb, Hkv, d, bs)
    K.qcache_append(kv[0].transpose(0, 1), kv[1].transpose(0, 1), slots, a)
    wide = torch.zeros(N, Hkv + 1, d + 8, dtype=BF, device="cuda")
    wide[:, 1:, 8:] = kv[0].transpose(0, 1)
    K.qcache_append(wide[:, 1:, 8:], kv[1].transpose(0, 1).contiguous(), slots, b)
    assert torch.equal(a, b)
    out = torch.full((2, Hkv, N, d), 7.0, dtype=BF, device="cuda")
    K.qcache_read(a, slots, k=out[0].transpose(0, 1), v=out[1].transpose(0, 1))
    ref = K.qcache_read(a, slots)
    assert torch.equal(out[0].transpose(0, 1), ref[0]) and torch.equal(out[1].transpose(0, 1), ref[1])


def test_append_nan_and_infinity(K):
    x = torch.randn(3, 1, 64, device="cuda").to(BF)
    x[0, 0, 5] = float("nan")
    x[1, 0, 20], x[1, 0, 40] = float("inf"), float("-inf")
    pages = K.qcache_alloc(1, 1, 64, 16)
    slots = ints([0, 1, 2])
    K.qcache_append(x, x, slots, pages)
    got = f64(K.qcache_read(pages, slots, dtype=F32)[0])
    assert np.isnan(got[0, 0, :16]).all() and np.isfinite(got[0, 0, 16:]).all()
    assert got[1, 0, 20] == 2688.0 and got[1, 0, 40] == -2688.0
    assert np.array_equal(got[2], Q.stored(f64(x))[2])


def test_rows_out_of_range_are_reported_and_skipped(K):
    pages = K.qcache_alloc(2, 1, 64, 16)
    before = pages.clone()
    x = torch.randn(2, 1, 64, device="cuda").to(BF)
    ws = K.Workspace()
    K.qcache_append(x, x, ints([32, -5]), pages, ws=ws)
    assert ws.device_error() == K.BAD_INPUT and torch.equal(pages, before)
    k, _ = K.qcache_read(pages, ints([2 ** 31 - 1, -1]), ws=ws)
    assert ws.device_error() == K.BAD_INPUT and not k.any()
    K.qcache_append(x[:0], x[:0], ints([]), pages, ws=ws)
    assert K.qcache_read(pages, ints([]), ws=ws)[0].shape == (0, 1, 64)
    assert ws.device_error() == K.OK


# ------------------------------------------------------------------- plan --

def random_step(rng, lens, width, bs):
    new = []
    for n in lens:
        r = rng.random()
        if r < 0.1:
            new.append(-n - int(rng.integers(0, 3)))         # ends
        elif r < 0.25:
            new.append(-int(rng.integers(0, n + 1)))         # rolls back
        elif r < 0.35:
            new.append(int(rng.integers(0, width * bs - n + 1)))
        elif r < 0.45:
            new.append(0)
        else:
            new.append(1 if n < width * bs else 0)
    return new


@pytest.mark.parametrize("B,bs,width", [(1, 16, 1), (7, 16, 9), (64, 64, 5), (1025, 32, 3),
                                        (2100, 16, 4), (3, 256, 40)])
def test_plan_against_oracle(K, B, bs, width):
    rng = np.random.default_rng(B + bs)
    nb = B * width + 3
    lens = [int(x) for x in rng.integers(0, width * bs + 1, B)]
    table = table_of(rng, lens, bs, nb, width)
    held = set(table[table >= 0].tolist())
    free = np.full(nb, -1, dtype=np.int64)
    rest = [x for x in rng.permutation(nb).tolist() if x not in held]
    free[:len(rest)] = rest
    count = len(rest)
    dl, dt, df, dc = ints(lens), ints(table), ints(free), ints([count])
    ws = K.Workspace()
    for it in range(6):
        new = random_step(rng, lens, width, bs)
        max_new = sum(max(0, x) for x in new) + int(rng.integers(0, 5))
        slots, cu, l2, count, table, free = Q.plan(lens, new, table, free, count, bs, max_new)
        inplace = it % 2 == 0
        got = K.qcache_plan(dl, ints(new), dt, df, dc, bs, max_new, ws=ws,
                            kv_lens_out=dl if inplace else None,
                            free_count_out=dc if inplace else None)
        if not inplace:
            dl, dc = got[2], got[3]
        assert np.array_equal(got[0].cpu().numpy(), slots)
        assert np.array_equal(got[1].cpu().numpy(), cu)
        assert np.array_equal(dl.cpu().numpy(), l2) and int(dc) == count
        assert np.array_equal(dt.cpu().numpy(), table)
        assert np.array_equal(df.cpu().numpy()[:count], free[:count])
        lens = [int(x) for x in l2]
        live = [table[b, j] for b in range(B) for j in range((lens[b] + bs - 1) // bs)]
        assert len(set(live) | set(free[:count].tolist())) == len(live) + count == nb
    assert ws.device_error() == K.OK


@pytest.mark.parametrize("what", ["blocks", "slots", "width", "length", "given", "free", "count",
                                  "big", "full"])
@pytest.mark.parametrize("nb", [12, 3012])      # one launch, two launches
def test_plan_refusals_change_nothing(K, what, nb):
    bs, width = 16, 4
    lens, new = [20, 33, 64], [5, 30, -40]
    table = np.array([[0, 1, -1, -1], [2, 3, 4, -1], [5, 6, 7, 8]])
    free = np.array([9, 10, 11] + [-1] * (nb - 3))
    count, max_new = 3, 99
    assert Q.plan(lens, new, table, free, count, bs, max_new) is not None
    if what == "blocks":
        new, count = [40, 1, 0], 1
    if what == "slots":
        max_new = 34
    if what == "length":
        lens = [-1, 33, 64]
    if what == "given":
        table[2, 3] = nb
    if what == "free":
        free[1] = nb + 87
        new = [40, 1, 0]
    if what == "count":
        count = nb + 1
    if what == "big":
        new = [2 ** 31 - 1, 0, 0]
    if what == "full":
        count = nb - 1                   # with the 2 given back: more than the cache has
    if what == "width":
        new = [50, 1, 0]
    assert Q.plan(lens, new, table, free, count, bs, max_new) is None
    d = [ints(x) for x in (lens, new, table, free, [count])]
    ws = K.Workspace()
    slots, cu, l2, c2 = K.qcache_plan(d[0], d[1], d[2], d[3], d[4], bs, max_new, ws=ws)
    assert ws.device_error() == K.BAD_INPUT
    assert (slots == -1).all() and not cu.any()
    assert torch.equal(l2, ints(lens)) and int(c2) == count
    assert torch.equal(d[2], ints(table)) and torch.equal(d[3], ints(free))
    # and the next step is served
    good = Q.plan([20, 33, 64], [5, 30, -40], np.array([[0, 1, -1, -1], [2, 3, 4, -1], [5, 6, 7, 8]]),
                  np.array([9, 10, 11] + [-1] * (nb - 3)), 3, bs, 99)
    got = K.qcache_plan(ints([20, 33, 64]), ints([5, 30, -40]),
                        ints([[0, 1, -1, -1], [2, 3, 4, -1], [5, 6, 7, 8]]),
                        ints([9, 10, 11] + [-1] * (nb - 3)), ints([3]), bs, 99, ws=ws)
    assert np.array_equal(got[0].cpu().numpy(), good[0]) and int(got[3]) == good[3]
    assert ws.device_error() == K.OK


# ------------------------------------------------------------------ dense --

DENSE = [   # lens, Hq, Hkv, d, bs, dtype, scores, width (blocks per table row)
    ([1], 1, 1, 64, 16, BF, True, None),
    ([512], 4, 2, 64, 16, F32, True, None),
    ([0, 1, 15, 16, 17, 31, 33, 100], 8, 2, 128, 16, BF, True, None),
    ([0, 5, 300], 8, 1, 128, 64, F32, True, 9),
    ([129, 1000, 64], 16, 4, 128, 256, BF, False, None),
    ([700, 0, 0, 3], 10, 5, 64, 32, BF, True, 40),
    ([2049, 4097], 32, 8, 128, 64, BF, False, None),
    ([5000, 3, 777], 16, 2, 64, 128, F32, False, None),
    ([33] * 70 + [0] * 3 + [1] * 60, 8, 8, 64, 16, BF, False, None),
    ([40000], 8, 1, 128, 64, BF, False, None),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,bs,dtype,scores,width", DENSE)
def test_dense(K, lens, Hq, Hkv, d, bs, dtype, scores, width):
    rng = np.random.default_rng(len(lens) * 1000 + d + bs)
    pages, table = filled(K, rng, lens, Hkv, d, bs, width=width)
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, d))).to(dtype).cuda()
    ws = K.Workspace()
    kv_len = None if width else max(1, max(lens))
    got = K.qcache_dense_decode(q, pages, ints(table), ints(lens), kv_len=kv_len,
                                return_scores=scores, ws=ws)
    out, sc = got if scores else (got, None)
    assert ws.device_error() == K.OK
    kv = [h // (Hq // Hkv) for h in range(Hq)]
    check_attention(q, out, pages, table, lens, Hkv, d, kv, scores=sc)
    again = K.qcache_dense_decode(q, pages, ints(table), ints(lens), kv_len=kv_len, ws=ws)
    assert torch.equal(again, out)


def test_dense_group_map_scale_and_cache_scales(K):
    rng = np.random.default_rng(11)
    lens, Hkv, d, bs = [200, 77], 2, 64, 32
    gm = [1, 0, 0, 1]
    for dtype in (BF, F32):
        pages, table = filled(K, rng, lens, Hkv, d, bs, k_scale=0.25, v_scale=8.0)
        q = torch.from_numpy(rng.standard_normal((2, 4, d)) * 3).to(dtype).cuda()
        out, sc = K.qcache_dense_decode(q, pages, ints(table), ints(lens), group_map=gm, scale=0.3,
                                        k_scale=0.25, v_scale=8.0, return_scores=True)
        sc = sc[:, :, :200]
        check_attention(q, out, pages, table, lens, Hkv, d, gm, k_scale=0.25, v_scale=8.0,
                        scale=0.3, scores=sc)


def test_dense_wide_range_of_q(K):
    """Queries whose heads differ by 60 orders of magnitude, and a head of zeros (uniform
    weights): the per-head power-of-two scaling neither overflows nor loses them."""
    rng = np.random.default_rng(12)
    lens, d = [300], 128
    pages, table = filled(K, rng, lens, 1, d, 64)
    for dtype in (BF, F32):
        q = torch.from_numpy(rng.standard_normal((1, 8, d))).float()
        q *= torch.tensor([1e-30, 1e-10, 1e-3, 1.0, 4.0, 0.0, 1e-38, 2.0 ** -130]).view(1, 8, 1)
        q = q.to(dtype).cuda()
        out, sc = K.qcache_dense_decode(q, pages, ints(table), ints(lens), kv_len=300,
                                        return_scores=True)
        check_attention(q, out, pages, table, lens, 1, d, [0] * 8)
        assert not sc[0, 5].any()
        big = q * 1e30                      # logits of 1e30: one key takes all
        out, sc = K.qcache_dense_decode(big[:, 3:4].contiguous(), pages, ints(table), ints(lens),
                                        return_scores=True)
        _, v = Q.rows_of(pages.cpu().numpy(), table[0], 300, 0, d)
        assert np.abs(f64(out[0, 0]) - v[int(sc[0, 0, :300].argmax())]).max() <= 2.0 ** -8 * 24


def test_dense_extreme_logits_and_many_small_weights(K):
    """One dominant key among many keys 2^-20 below it: their sum still counts."""
    n, d, bs = 20000, 64, 64
    rng = np.random.default_rng(5)
    nb = (n + bs - 1) // bs
    table = rng.permutation(nb).reshape(1, nb)
    k = torch.zeros(n, 1, d)
    k[:, 0, 0] = 1.0
    k[777, 0, 0] = 4.0
    v = torch.ones(n, 1, d)
    v[777] = -1.0
    pages = K.qcache_alloc(nb, 1, d, bs)
    slots = table[0, np.arange(n) // bs] * bs + np.arange(n) % bs
    K.qcache_append(k.cuda(), v.cuda(), ints(slots), pages)
    q = torch.zeros(1, 1, d)
    q[0, 0, 0] = 20 * np.log(2) / 3        # logits 20 ln 2 apart
    for dtype in (BF, F32):
        qd = q.to(dtype).cuda()
        out = K.qcache_dense_decode(qd, pages, ints(table), ints([n]), kv_len=n, scale=1.0)
        check_attention(qd, out, pages, table, [n], 1, d, [0], scale=1.0)


def test_dense_nan_row_reaches_its_sequence_only(K):
    rng = np.random.default_rng(6)
    lens, d, bs = [100, 50], 128, 16
    pages, table = filled(K, rng, lens, 2, d, bs)
    x = torch.full((1, 2, d), float("nan"), device="cuda", dtype=BF)
    K.qcache_append(x, x, ints([table[0, 2] * bs + 3]), pages)
    q = torch.randn(2, 4, d, device="cuda").to(BF)
    out = K.qcache_dense_decode(q, pages, ints(table), ints(lens), kv_len=100)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    inf = q.clone()
    inf[0, 0, 0] = float("inf")
    out = K.qcache_dense_decode(inf, pages, ints(table), ints([0, 50]), kv_len=100)
    assert not out[0].any() and torch.isfinite(out[1]).all()


def test_bad_lengths_and_tables_are_reported(K):
    rng = np.random.default_rng(8)
    lens, d, bs = [100, 50], 64, 16
    pages, table = filled(K, rng, lens, 1, d, bs, width=8)
    q = torch.randn(2, 2, d, device="cuda").to(BF)
    ws = K.Workspace()
    good = K.qcache_dense_decode(q, pages, ints(table), ints(lens), ws=ws)
    for bad_lens in ([-1, 50], [129, 50], [2 ** 31 - 1, 50]):
        out = K.qcache_dense_decode(q, pages, ints(table), ints(bad_lens), ws=ws)
        assert ws.device_error() == K.BAD_INPUT
        # where a sequence is split depends on the batch's lengths, so its sums
        # may be taken in another order: equal within the tolerance, not to the bit
        check_attention(q[1:], out[1:], pages, table[1:], [50], 1, d, [0, 0])
    for entry in (-1, pages.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.copy()
        t[0, 2] = entry
        out = K.qcache_dense_decode(q, pages, ints(t), ints(lens), ws=ws)
        assert ws.device_error() == K.BAD_INPUT
        assert torch.equal(out[1], good[1])
        # the block's keys count as masked
        keep = [j for j in range(100) if j // bs != 2]
        kv = [0, 0]
        check_attention(q[:1], out[:1], pages, table, [100], 1, d, kv, sets=[[keep, keep]])
    assert torch.equal(K.qcache_dense_decode(q, pages, ints(table), ints(lens), ws=ws), good)
    assert ws.device_error() == K.OK


# --------------------------------------------------------- anchor and reuse --

ANCHOR = [([700, 33, 0, 129], 8, 2, 128, 64, 40, BF), ([512, 40], 4, 2, 64, 16, 32, F32),
          ([3000, 1, 100], 16, 2, 64, 256, 300, BF), ([5000], 8, 8, 128, 32, 5000, BF)]


@pytest.mark.parametrize("pooled", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,d,bs,k,dtype", ANCHOR)
def test_anchor(K, lens, Hq, Hkv, d, bs, k, dtype, pooled):
    rng = np.random.default_rng(k)
    pages, table = filled(K, rng, lens, Hkv, d, bs)
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, d))).to(dtype).cuda()
    ws = K.Workspace()
    N = max(lens)
    args = (q, pages, ints(table), ints(lens))
    out, idx, sc = K.qcache_anchor_decode(*args, k, kv_len=N, return_scores=True, pooled=pooled,
                                          ws=ws)
    out2, idx2 = K.qcache_anchor_decode(*args, k, kv_len=N, pooled=pooled, ws=ws)
    dense, logits = K.qcache_dense_decode(*args, kv_len=N, return_scores=True, ws=ws)
    assert ws.device_error() == K.OK
    assert torch.equal(out, dense) and torch.equal(out2, out) and torch.equal(idx, idx2)
    G = Hq // Hkv
    sn, ln, got = f64(sc), f64(logits), idx.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(Hkv if pooled else Hq):
            assert (sn[b, h, n:] == -np.inf).all()
            if pooled and n:
                s = ln[b, h * G:(h + 1) * G, :n]
                w = np.exp(s - s.max(-1, keepdims=True))
                w = (w / w.sum(-1, keepdims=True)).sum(0)
                # fp32 weights of logits that are equal to the last bit
                assert (np.abs(sn[b, h, :n] - w) <= 1e-4 * w + 1e-30).all()
            elif n:
                assert np.array_equal(sn[b, h, :n], ln[b, h, :n])
            m = min(k, n)
            want = topk_indices(sn[b, h, :n], m) if m else np.zeros(0, dtype=np.int64)
            assert np.array_equal(got[b, h, :m], want) and (got[b, h, m:] == -1).all()


def random_sets(rng, lens, H, k, empty=False):
    sets = [[np.sort(rng.choice(n, min(n, k), replace=False)) for _ in range(H)] for n in lens]
    if empty:
        sets[-1][0] = sets[-1][0][:0]
        sets[-1][-1] = sets[-1][-1][:1]
    idx = np.full((len(lens), H, k), -1, dtype=np.int64)
    for b in range(len(lens)):
        for h in range(H):
            idx[b, h, :len(sets[b][h])] = sets[b][h]
    return sets, idx


REUSE = [([700, 33, 0, 129], 8, 2, 128, 64, 40, BF), ([512, 40], 4, 2, 64, 16, 32, F32),
         ([1], 1, 1, 64, 16, 1, BF), ([3000, 1, 100], 16, 2, 64, 256, 300, BF),
         ([6000, 2500], 8, 1, 128, 32, 2000, BF), ([777, 3, 388], 8, 4, 128, 32, 96, F32),
         ([300] * 40, 32, 8, 64, 16, 17, BF), ([2100], 5, 5, 128, 128, 2100, BF)]


@pytest.mark.parametrize("pooled", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,d,bs,k,dtype", REUSE)
def test_reuse(K, lens, Hq, Hkv, d, bs, k, dtype, pooled):
    rng = np.random.default_rng(k + d)
    pages, table = filled(K, rng, lens, Hkv, d, bs)
    sets, idx = random_sets(rng, lens, Hkv if pooled else Hq, k, empty=True)
    # rows that no head of the group selects are poisoned
    clean = pages.clone()
    pg = pages.cpu().numpy().copy()
    parts = Q.group_fields(pg, d)
    for b, n in enumerate(lens):
        for g in range(Hkv):
            hs = [g] if pooled else range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
            unused = np.setdiff1d(np.arange(n), np.concatenate([sets[b][h] for h in hs]))
            at = (table[b, unused // bs], g, unused % bs // 16, unused % 16)
            for f in parts:
                f[at] = 255
    size = 18 * d
    flat = np.concatenate([f.reshape(f.shape[:3] + (-1,)) for f in parts], -1)
    assert flat.shape[-1] == size
    poisoned = torch.from_numpy(flat).cuda()
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, d))).to(dtype).cuda()
    ws = K.Workspace()
    kw = dict(kv_len=max(lens), pooled=pooled, ws=ws)
    out = K.qcache_reuse_decode(q, poisoned, ints(table), ints(lens), ints(idx), **kw)
    ref = K.qcache_reuse_decode(q, clean, ints(table), ints(lens), ints(idx), **kw)
    assert ws.device_error() == K.OK and torch.equal(out, ref)
    kv = [h // (Hq // Hkv) for h in range(Hq)]
    check_attention(q, out, clean, table, lens, Hkv, d, kv, sets=sets, pooled=pooled)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_reuse_nan_row_reaches_the_heads_that_select_it(K, d, dtype):
    rng = np.random.default_rng(d)
    lens, Hq, bs, k = [400], 8, 32, 50
    pages, table = filled(K, rng, lens, 1, d, bs)
    sets, idx = random_sets(rng, lens, Hq, k)
    q = torch.from_numpy(rng.standard_normal((1, Hq, d))).to(dtype).cuda()
    args = (ints(table), ints(lens), ints(idx))
    good = K.qcache_reuse_decode(q, pages, *args)
    row = torch.full((1, 1, d), float("nan"), device="cuda", dtype=BF)
    val = torch.zeros(1, 1, d, device="cuda", dtype=BF)
    for head, at in ((3, 7), (0, 0), (7, 49), (5, 20), (2, 33)):
        key = int(sets[0][head][at])
        holders = [h for h in range(Hq) if key in sets[0][h]]
        for kk, vv in ((row, val), (val, row)):
            bad = pages.clone()
            K.qcache_append(kk, vv, ints([table[0, key // bs] * bs + key % bs]), bad)
            out = K.qcache_reuse_decode(q, bad, *args)
            for h in range(Hq):
                if h in holders:
                    assert torch.isnan(out[0, h]).all()
                else:
                    assert torch.equal(out[0, h], good[0, h])


@pytest.mark.parametrize("pooled", [False, True])
def test_reuse_bad_sets_are_reported_and_not_read(K, pooled):
    rng = np.random.default_rng(9)
    lens, Hq, Hkv, d, bs, k = [100, 60], 4, 2, 64, 16, 8
    pages, table = filled(K, rng, lens, Hkv, d, bs)
    H = Hkv if pooled else Hq
    _, idx = random_sets(rng, lens, H, k)
    idx[0, 0] = [3, 9, 20, 41, 50, 77, 90, 99]
    q = torch.randn(2, Hq, d, device="cuda").to(BF)
    ws = K.Workspace()
    run = lambda i: K.qcache_reuse_decode(q, pages, ints(table), ints(lens), ints(i), pooled=pooled,
                                          kv_len=100, ws=ws)
    good = run(idx)
    assert ws.device_error() == K.OK
    for pos, val in ((7, 100), (7, 2 ** 31 - 1), (0, -2), (3, 20), (2, -1), (4, 2 ** 24)):
        bad = idx.copy()
        bad[0, 0, pos] = val
        out = run(bad)
        assert ws.device_error() == K.BAD_INPUT, (pos, val)
        assert torch.equal(out[1], good[1])
    assert torch.equal(run(idx), good) and ws.device_error() == K.OK


def test_reuse_of_every_key_is_dense(K):
    rng = np.random.default_rng(10)
    lens, Hq, Hkv, d = [500, 77], 8, 2, 128
    pages, table = filled(K, rng, lens, Hkv, d, 64)
    q = torch.randn(2, Hq, d, device="cuda").to(BF)
    out, idx = K.qcache_anchor_decode(q, pages, ints(table), ints(lens), 500, kv_len=500)
    again = K.qcache_reuse_decode(q, pages, ints(table), ints(lens), idx, kv_len=500)
    kv = [h // 4 for h in range(Hq)]
    check_attention(q, again, pages, table, lens, Hkv, d, kv)


# ------------------------------------------------------------------- together --

@pytest.mark.parametrize("pooled", [False, True])
@pytest.mark.parametrize("dtype,d,bs", [(BF, 128, 64), (F32, 64, 16)])
def test_decode_steps_through_the_stack(K, dtype, d, bs, pooled):
    """Several steps of a small server: prompts written, then decode steps of the
    stack (plan, append, anchor / reuse / dense layers) with requests that end
    and begin, each against the same calls made one by one."""
    rng = np.random.default_rng(21)
    B, Hq, Hkv, L, k, width, nb = 5, 8, 2, 4, 24, 6, 40
    N = width * bs
    anchors = [1, 3]
    pages = [K.qcache_alloc(nb, Hkv, d, bs) for _ in range(L)]
    table = torch.full((B, width), -1, dtype=I32, device="cuda")
    lens = torch.zeros(B, dtype=I32, device="cuda")
    free, count = ints(rng.permutation(nb)), ints([nb])
    ws = K.Workspace()
    prompts = [90, 1, 33, 0, 64]
    slots, cu, lens, count = K.qcache_plan(lens, ints(prompts), table, free, count, bs,
                                           sum(prompts), ws=ws)
    for l in range(L):
        kv = torch.randn(2, sum(prompts), Hkv, d, device="cuda").to(dtype)
        K.qcache_append(kv[0], kv[1], slots, pages[l], ws=ws)
    for new in ([1, 1, 1, 1, 1], [1, -2, 1, 1, -65], [1, 0, 1, 1, 1], [2, 0, 0, 1, 0]):
        T = 6
        qs = [torch.randn(B, Hq, d, device="cuda").to(dtype) for _ in range(L)]
        nk = [torch.randn(T, Hkv, d, device="cuda").to(dtype) for _ in range(L)]
        nv = [torch.randn(T, Hkv, d, device="cuda").to(dtype) for _ in range(L)]
        # one by one, on copies
        t2, f2, p2 = table.clone(), free.clone(), [p.clone() for p in pages]
        s2, _, l2, c2 = K.qcache_plan(lens, ints(new), t2, f2, count, bs, T, ws=ws)
        want, idx = [], None
        for l in range(L):
            K.qcache_append(nk[l], nv[l], s2, p2[l], ws=ws)
            a = (qs[l], p2[l], t2, l2)
            if l in anchors:
                o, idx = K.qcache_anchor_decode(*a, k, pooled=pooled, ws=ws)
            elif idx is not None:
                o = K.qcache_reuse_decode(*a, idx, pooled=pooled, ws=ws)
            else:
                o = K.qcache_dense_decode(*a, ws=ws)
            want.append(o)
        outs, ib = K.qcache_run_stack(qs, pages, table, lens, k, anchors, new_ks=nk, new_vs=nv,
                                      new_lens=ints(new), free_blocks=free, free_count=count,
                                      pooled=pooled, ws=ws)
        assert ws.device_error() == K.OK
        assert torch.equal(table, t2) and torch.equal(lens, l2) and torch.equal(count, c2)
        assert torch.equal(ib, idx) and all(torch.equal(x, y) for x, y in zip(outs, want))
        assert all(torch.equal(x, y) for x, y in zip(pages, p2))
        n = lens.cpu().tolist()
        kv_of = [h // 4 for h in range(Hq)]
        check_attention(qs[0], outs[0], pages[0], table.cpu().numpy(), n, Hkv, d, kv_of)
        # the rows just written are the last of their sequences
        cuh = np.concatenate([[0], np.cumsum(np.maximum(new, 0))])
        for b in range(B):
            if new[b] > 0:
                rows = Q.rows_of(pages[2].cpu().numpy(), table[b].cpu().numpy(), n[b], 0, d)[0]
                assert np.array_equal(rows[-new[b]:], Q.stored(f64(nk[2][cuh[b]:cuh[b + 1], 0])))


def test_prefill_then_decode_on_the_cache(K):
    """A prompt's keys and values from the prefill layer go into the cache; the
    read-back rows give the dense prefill of the stored prompt, whose last row
    is what decoding the last query over the cache gives."""
    Hq, Hkv, N, d, bs = 8, 2, 300, 128, 64
    torch.manual_seed(0)
    q = torch.randn(1, Hq, N, d, device="cuda").to(BF)
    k = torch.randn(1, Hkv, N, d, device="cuda").to(BF)
    v = torch.randn(1, Hkv, N, d, device="cuda").to(BF)
    pages = K.qcache_alloc(6, Hkv, d, bs)
    table, free, count = ints([[-1] * 6]), ints([4, 2, 0, 1, 3, 5]), ints([6])
    slots, _, lens, count = K.qcache_plan(ints([0]), ints([N]), table, free, count, bs, N)
    K.qcache_append(k[0].transpose(0, 1), v[0].transpose(0, 1), slots, pages)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    K.qcache_read(pages, slots, k=k2[0].transpose(0, 1), v=v2[0].transpose(0, 1))
    full = K.dense_prefill(q, k2, v2)
    one = K.qcache_dense_decode(q[:, :, -1].contiguous(), pages, table, lens)
    # both round their output to bf16 (2^-8) and their weights to 8 (2^-8) or 11 bits
    err = np.abs(f64(full[:, :, -1]) - f64(one))
    assert err.max() <= 2.0 ** -6


def test_graph_replay_and_workspaces(K):
    rng = np.random.default_rng(14)
    lens, Hq, Hkv, d, bs, k = [300, 40], 8, 2, 128, 32, 64
    pages, table = filled(K, rng, lens, Hkv, d, bs, spare=8, width=12)
    T, dl, q = ints(table), ints(lens), torch.randn(2, Hq, d, device="cuda").to(BF)
    _, idx = random_sets(rng, lens, Hq, k)
    di = ints(idx)
    ws, big = K.Workspace(), K.Workspace()
    out, o2 = torch.empty_like(q), torch.empty_like(q)

    def step(w):
        K.qcache_dense_decode(q, pages, T, dl, out=out, ws=w)
        K.qcache_reuse_decode(q, pages, T, dl, di, out=o2, ws=w)

    g = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError, match="workspace|captured"):
        with torch.cuda.graph(g):
            step(None)
    with pytest.raises(ValueError, match="workspace|captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            step(K.Workspace())
    step(ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(ws)
    with pytest.raises(RuntimeError, match="captured"):
        ws.get(ws.buf.numel() + 1)
    for n in ([300, 40], [250, 0], [0, 17]):
        dl.copy_(ints(n))
        q.copy_(torch.randn(2, Hq, d, device="cuda").to(BF))
        _, idx = random_sets(rng, n, Hq, k)
        di.copy_(ints(idx))
        out.fill_(9.0)
        o2.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, K.qcache_dense_decode(q, pages, T, dl, ws=big))
        assert torch.equal(o2, K.qcache_reuse_decode(q, pages, T, dl, di, ws=big))
    assert ws.device_error() == K.OK


def test_other_streams(K):
    rng = np.random.default_rng(15)
    lens, Hq, Hkv, d, bs = [3000, 1000], 8, 2, 128, 64
    pages, table = filled(K, rng, lens, Hkv, d, bs)
    q = torch.randn(2, Hq, d, device="cuda").to(BF)
    want = K.qcache_dense_decode(q, pages, ints(table), ints(lens))
    T, dl = ints(table), ints(lens)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    w1, w2 = K.Workspace(), K.Workspace()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):                      # two calls at once, a workspace each
        got.append(K.qcache_dense_decode(q, pages, T, dl, ws=w1, stream=s1))
        with torch.cuda.stream(s2):
            got.append(K.qcache_dense_decode(q, pages, T, dl, ws=w2))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


def test_streams_do_not_share_the_default_workspace(K):
    rng = np.random.default_rng(25)
    lens, d, bs = [6000, 100], 64, 32
    pages, table = filled(K, rng, lens, 2, d, bs)
    T, dl = ints(table), ints(lens)
    qs = [torch.randn(2, 8, d, device="cuda").to(BF) for _ in range(3)]
    want = [K.qcache_dense_decode(q, pages, T, dl) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [(i, K.qcache_dense_decode(qs[i], pages, T, dl, stream=streams[i]))
           for _ in range(10) for i in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i, x in got)
    bufs = {K.default_workspace("cuda", s).buf.data_ptr() for s in streams + [None]}
    assert len(bufs) == 4
    assert K.default_workspace("cuda", streams[0]).device_error(streams[0]) == K.OK


@pytest.mark.parametrize("d,Hq", [(128, 8), (64, 2)])
def test_largest_batch(K, d, Hq):
    """16384 sequences, most of a few tokens, one long: the line's places fill
    the shared memory beside the rings."""
    B, bs = 16384, 16
    rng = np.random.default_rng(d)
    lens = rng.integers(0, 4, B)
    lens[rng.choice(B, 40, replace=False)] = rng.integers(0, 300, 40)
    lens[77] = 5000
    pages, table = filled(K, rng, lens.tolist(), 1, d, bs)
    q = torch.from_numpy(rng.standard_normal((B, Hq, d))).to(BF).cuda()
    out = K.qcache_dense_decode(q, pages, ints(table), ints(lens), kv_len=5000)
    assert not out[torch.from_numpy(lens == 0).cuda()].any()
    pick = np.concatenate([np.nonzero(lens > 3)[0], rng.choice(B, 200, replace=False)])
    check_attention(q[pick], out[pick], pages, table[pick], lens[pick].tolist(), 1, d, [0] * Hq,
                    max_units=400)


def test_captured_steps_of_the_stack(K):
    """A step with its plan captured once: every replay takes the state the one
    before left, as eager steps on a copy do."""
    rng = np.random.default_rng(31)
    B, Hq, Hkv, d, bs, width, nb, L, k = 4, 8, 2, 128, 16, 8, 36, 3, 12
    pages = [K.qcache_alloc(nb, Hkv, d, bs) for _ in range(L)]
    state = dict(block_table=torch.full((B, width), -1, dtype=I32, device="cuda"),
                 kv_lens=torch.zeros(B, dtype=I32, device="cuda"),
                 free_blocks=ints(rng.permutation(nb)), free_count=ints([nb]))
    copy = {n: t.clone() for n, t in state.items()}
    pages2 = [p.clone() for p in pages]
    new = ints([1] * B)
    qs = [torch.randn(B, Hq, d, device="cuda").to(BF) for _ in range(L)]
    nk = [torch.randn(B, Hkv, d, device="cuda").to(BF) for _ in range(L)]
    nv = [torch.randn(B, Hkv, d, device="cuda").to(BF) for _ in range(L)]
    outs, idx = [torch.empty_like(q) for q in qs], torch.empty(B, Hq, k, dtype=I32, device="cuda")
    slots, cu = torch.empty(B, dtype=I32, device="cuda"), torch.empty(B + 1, dtype=I32, device="cuda")
    ws, eager = K.Workspace(), K.Workspace()

    def step(st, pg, w, **kw):
        return K.qcache_run_stack(qs, pg, st["block_table"], st["kv_lens"], k, [1], new_ks=nk,
                                  new_vs=nv, new_lens=new, free_blocks=st["free_blocks"],
                                  free_count=st["free_count"], ws=w, **kw)

    step({n: t.clone() for n, t in state.items()}, [p.clone() for p in pages], ws)   # sizes ws
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(state, pages, ws, outs=outs, idx_buf=idx, slot_map=slots, cu_new=cu)
    grow = [[1, 1, 1, 1]] * 20 + [[40, 0, 1, 3], [-9, 1, -99, 1], [1, 1, 1, 0]]
    for n in grow:
        new.copy_(ints(n))
        for t in qs + nk + nv:
            t.copy_(torch.randn_like(t.float()).to(BF))
        if sum(max(0, x) for x in n) > B:       # more rows than the step has: refused
            before = state["kv_lens"].clone()
            g.replay()
            torch.cuda.synchronize()
            assert ws.device_error() == K.BAD_INPUT and torch.equal(state["kv_lens"], before)
            continue
        g.replay()
        want, wi = step(copy, pages2, eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and torch.equal(idx, wi)
        assert all(torch.equal(state[x], copy[x]) for x in state)
        assert all(torch.equal(a, b) for a, b in zip(pages, pages2))
    assert ws.device_error() == K.OK and eager.device_error() == K.OK


def test_workspace_shared_with_other_calls(K):
    """One workspace, calls of many shapes and of the other entry points in turn."""
    rng = np.random.default_rng(16)
    ws = K.Workspace()
    ws.get(64 << 20)
    ref = []
    shapes = [([5000], 8, 1, 128, 64), ([40] * 30, 16, 8, 64, 16), ([9000, 1], 8, 2, 64, 256)]
    cases = []
    for lens, Hq, Hkv, d, bs in shapes:
        pages, table = filled(K, rng, lens, Hkv, d, bs)
        q = torch.randn(len(lens), Hq, d, device="cuda").to(BF)
        cases.append((q, pages, ints(table), ints(lens), max(lens)))
    kd = torch.randn(2, 2, 3000 - 1, 128, device="cuda").to(BF)
    qd = torch.randn(2, 8, 128, device="cuda").to(BF)
    for i in range(3):
        got = [K.qcache_dense_decode(*c[:4], kv_len=c[4], ws=ws) for c in cases]
        got += list(K.anchor_decode(qd, kd, kd, 50, ws=ws))
        got += [K.qcache_anchor_decode(*c[:4], 20, kv_len=c[4], ws=ws)[1] for c in cases]
        if i == 0:
            ref = got
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
    assert ws.device_error() == K.OK


def test_offsets_beyond_32_bits(K):
    """A 5.2 GB cache: rows at its far end are written, read and attended to."""
    Hkv, d, bs = 8, 128, 256
    nb = 17500                                # 294912 bytes each
    pages = torch.empty(nb, Hkv, bs // 16, 18 * d, dtype=torch.uint8, device="cuda")
    ids = [nb - 1, 0, nb - 2, 8000]
    n = 4 * bs - 3
    slots = ints([ids[p // bs] * bs + p % bs for p in range(n)])
    x = torch.randn(2, n, Hkv, d, device="cuda").to(BF)
    K.qcache_append(x[0], x[1], slots, pages)
    k, v = K.qcache_read(pages, slots, dtype=F32)
    assert np.array_equal(f64(k), Q.stored(f64(x[0])))
    small = torch.zeros(4, Hkv, bs // 16, 18 * d, dtype=torch.uint8, device="cuda")
    for i, b in enumerate(ids):
        small[i] = pages[b]
    q = torch.randn(1, 32, d, device="cuda").to(BF)
    idx = ints(np.sort(np.random.default_rng(0).choice(n, 200, replace=False)).reshape(1, 1, 200))
    idx = idx.expand(1, 32, 200).contiguous()
    far, near = ints([ids]), ints([[0, 1, 2, 3]])
    for fn in (lambda p, t: K.qcache_dense_decode(q, p, t, ints([n]), kv_len=n),
               lambda p, t: K.qcache_reuse_decode(q, p, t, ints([n]), idx, kv_len=n)):
        assert torch.equal(fn(pages, far), fn(small, near))
    out = K.qcache_dense_decode(q, small, near, ints([n]), kv_len=n)
    check_attention(q, out, small, [[0, 1, 2, 3]], [n], Hkv, d, [h // 4 for h in range(32)])


@pytest.mark.parametrize("kind", ["plan", "append", "read", "dense", "anchor", "reuse"])
def test_profiling_command(kind, monkeypatch, capsys):
    from long_context_anchor_gb300 import runcase
    argv = ["runcase", "qcache_" + kind, "--kv-len", "333", "--topk", "40", "--reps", "1",
            "--block-size", "32"]
    monkeypatch.setattr("sys.argv", argv)
    runcase.main()
    assert capsys.readouterr().out == "ok qcache_%s\n" % kind


def test_sequences_that_share_blocks(K):
    """A common prefix held once: every sequence attends over it as over its own copy."""
    rng = np.random.default_rng(11)
    Hkv, d, bs, n = 2, 128, 32, 150
    own, table = filled(K, rng, [n], Hkv, d, bs, spare=20)
    first = table[0, :5]
    used = set(first.tolist())
    spare = [x for x in range(own.shape[0]) if x not in used]
    copy = own.clone()
    shared = np.stack([first, first, np.concatenate([first[:3], spare[:2]])])
    apart = np.stack([first, spare[5:10], np.concatenate([spare[10:13], spare[:2]])])
    for row in apart[1:]:
        for j, b in enumerate(row):
            if b not in spare[:2]:
                copy[int(b)] = own[int(first[j])]
    lens = [n, 77, 96]
    q = torch.from_numpy(rng.standard_normal((3, 8, d))).to(BF).cuda()
    ws = K.Workspace()
    for fn in (lambda p, t: (K.qcache_dense_decode(q, p, ints(t), ints(lens), ws=ws),),
               lambda p, t: K.qcache_anchor_decode(q, p, ints(t), ints(lens), 20, ws=ws)):
        for x, y in zip(fn(own, shared), fn(copy, apart)):
            assert torch.equal(x, y)
    assert ws.device_error() == K.OK


@pytest.mark.parametrize("pooled", [False, True])
def test_repeated_calls_give_the_same_bits(K, pooled):
    rng = np.random.default_rng(12)
    Hkv, d, bs = 4, 64, 16
    lens = [9000, 0, 1, 2500, 700, 31]
    pages, table = filled(K, rng, lens, Hkv, d, bs)
    q = torch.from_numpy(rng.standard_normal((len(lens), 16, d))).to(BF).cuda()
    t, l, ws = ints(table), ints(lens), K.Workspace()
    out, idx = K.qcache_anchor_decode(q, pages, t, l, 600, ws=ws, pooled=pooled)
    reuse = K.qcache_reuse_decode(q, pages, t, l, idx, ws=ws, pooled=pooled)
    for _ in range(30):
        o, i = K.qcache_anchor_decode(q, pages, t, l, 600, ws=ws, pooled=pooled)
        assert torch.equal(o, out) and torch.equal(i, idx)
        assert torch.equal(K.qcache_reuse_decode(q, pages, t, l, idx, ws=ws, pooled=pooled), reuse)
    assert ws.device_error() == K.OK


def test_step_without_new_tokens(K):
    """max_new = 0: sequences that end or roll back only; nothing to append."""
    pages, table = filled(K, np.random.default_rng(13), [40, 20], 1, 64, 16)
    free = ints([-1] * pages.shape[0])
    slots, cu, lens, count = K.qcache_plan(ints([40, 20]), ints([-40, -5]), ints(table), free,
                                           ints([0]), 16, 0)
    assert slots.shape == (0,) and not cu.any()
    assert lens.tolist() == [0, 15] and int(count) == 4
    assert free[:4].tolist() == list(table[0, :3]) + [table[1, 1]]
    with pytest.raises(K.KascadeError):
        K.qcache_plan(lens, lens, ints(table), free, count, 16, -1)
    x = torch.empty(0, 1, 64, dtype=BF, device="cuda")
    before = pages.clone()
    K.qcache_append(x, x, slots, pages)
    assert torch.equal(pages, before)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_into_strided_rows(K, dtype):
    """Only the rows asked for are written, at their strides; one token and one head too."""
    for T, Hkv in ((5, 3), (1, 3), (5, 1), (1, 1)):
        pages = K.qcache_alloc(2, Hkv, 64, 16)
        x = torch.randn(2, T, Hkv, 64, device="cuda").to(dtype)
        slots = ints([3, 17, 31, 0, 8][:T])
        K.qcache_append(x[0], x[1], slots, pages)
        want = K.qcache_read(pages, slots, dtype=dtype)
        out = torch.full((2, Hkv + 2, T + 1, 80), 7.0, dtype=dtype, device="cuda")
        k, v = (out[i, 1:Hkv + 1, :T, 8:72].transpose(0, 1) for i in range(2))
        K.qcache_read(pages, slots, k=k, v=v)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])
        k.fill_(7.0)
        v.fill_(7.0)
        assert (out == 7.0).all()


def rows_beside_ties(d):
    """fp32 rows [T, 1, d] of blocks whose codes, or whose scales, lie on a tie or one or two
    last places beside it: every significand of the scale, every tie of both formats."""
    def near(x):
        x = np.float32(x)
        return [(x.view(np.int32) + np.int32(i)).view(np.float32) for i in range(-2, 3)]

    blocks = []
    for s in [m / 8 * 2.0 ** e for e in (-6, -1, 0, 7) for m in range(8, 16)]:
        x = [y for a, b in zip(Q.E2M1, Q.E2M1[1:]) for y in near((a + b) / 2 * s)]
        x = [-y if i % 2 else y for i, y in enumerate(x)]
        x += [0.0] * (-len(x) % 15)
        blocks += [[6 * s] + x[i:i + 15] for i in range(0, len(x), 15)]   # 6 s: the scale is s
    for a, b in zip(Q.E4M3, Q.E4M3[1:]):
        blocks += [[y] + [y * np.float32(f) for f in np.linspace(-0.99, 0.99, 15)]
                   for y in near((a + b) / 2 * 6)]
    blocks += [[0.0] * 16] * (-len(blocks) % (d // 16))
    return np.array(blocks, dtype=np.float32).reshape(-1, 1, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -7, 2.0 ** 20])
def test_append_rounds_fp32_beside_ties_once(K, d, scale):
    x = torch.from_numpy(rows_beside_ties(d) * np.float32(scale))
    T = len(x)
    pages = K.qcache_alloc((T + 15) // 16, 1, d, 16)
    slots = ints(range(T))
    K.qcache_append(x.cuda(), x.cuda(), slots, pages, scale, scale)
    want = Q.stored(f64(x), scale)
    for got in K.qcache_read(pages, slots, dtype=F32, k_scale=scale, v_scale=scale):
        assert np.array_equal(f64(got), want)


@pytest.mark.parametrize("nb", [12, 3012])      # one launch, two launches
@pytest.mark.parametrize("bad", [-1, "nb", 2 ** 31 - 1, -2 ** 31])
def test_plan_refuses_a_bad_block_that_new_tokens_go_to(K, nb, bad):
    """Sequence 1's partly filled block is out of range: the other sequences' changes do not
    happen either. A sequence that does not grow, or whose last block is full, may hold such
    an entry."""
    bs, bad = 16, nb if bad == "nb" else bad
    table = np.array([[0, 1, -1, -1], [2, 3, bad, -1], [5, 6, 7, 8]])
    free = np.array([9, 10, 11] + [-1] * (nb - 3))
    ws = K.Workspace()
    for lens, new, ok in (([20, 33, 64], [15, 5, -40], False), ([20, 47, 64], [15, 1, -40], False),
                          ([20, 33, 64], [15, 0, -40], True), ([20, 48, 64], [15, 1, -40], True)):
        want = Q.plan(lens, new, table, free, 3, bs, 30)
        assert (want is not None) == ok
        d = [ints(x) for x in (lens, new, table, free, [3])]
        slots, cu, l2, c2 = K.qcache_plan(*d, bs, 30, ws=ws)
        assert ws.device_error() == (K.OK if ok else K.BAD_INPUT)
        if ok:
            assert np.array_equal(slots.cpu().numpy(), want[0])
            assert np.array_equal(d[2].cpu().numpy(), want[4]) and int(c2) == want[3]
            continue
        assert (slots == -1).all() and not cu.any()
        assert torch.equal(l2, d[0]) and int(c2) == 3
        assert torch.equal(d[2], ints(table)) and torch.equal(d[3], ints(free))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pooled", [False, True])
def test_reuse_stays_within_its_workspace(K, pooled, dtype):
    """A workspace of exactly a reuse layer's size, with guard bytes behind it."""
    rng = np.random.default_rng(41)
    lens, Hq, Hkv, d, bs, k = [5000, 0, 300], 16, 4, 64, 32, 700
    pages, table = filled(K, rng, lens, Hkv, d, bs)
    H = Hkv if pooled else Hq
    _, idx = random_sets(rng, lens, H, k)
    q = torch.from_numpy(rng.standard_normal((3, Hq, d))).to(dtype).cuda()
    args = (q, pages, ints(table), ints(lens), ints(idx))
    big = K.Workspace()
    want = K.qcache_reuse_decode(*args, pooled=pooled, ws=big)
    width = table.shape[1]
    desc = K.make_desc(3, Hq, Hkv, d, width * bs, K.BF16 if dtype is BF else K.F32, pooled=pooled)
    n = K.qcache_workspace_size(desc, K.QCache(bs, pages.shape[0], width, 0.0, 0.0), k, reuse=True)
    assert n < K.qcache_workspace_size(desc, K.QCache(bs, pages.shape[0], width, 0.0, 0.0), k)
    assert big.buf.numel() == n
    buf = torch.zeros(n + (1 << 20), dtype=torch.uint8, device="cuda")
    buf[n:] = 171
    ws = K.Workspace()
    ws.buf = buf[:n]
    assert torch.equal(K.qcache_reuse_decode(*args, pooled=pooled, ws=ws), want)
    assert ws.device_error() == K.OK and bool((buf[n:] == 171).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dense_weights_below_the_smallest_step(K, dtype):
    """One key takes nearly all the weight and its V is zero in half of the row, where keys of
    2^-36 to 2^-44 of its weight decide: within the head's bounds and half a step per key."""
    rng = np.random.default_rng(51)
    n, d, bs = 3000, 64, 32
    nb = (n + bs - 1) // bs
    table = rng.permutation(nb).reshape(1, nb)
    k = np.zeros((n, 1, d))
    k[:, 0, 0] = -6.0
    k[:, 0, 16] = rng.choice([-6.0, -3.0, -0.5, 0.0, 1.0, 4.0, 6.0], n)
    k[:, 0, 1:16] = k[:, 0, 17:32] = 6.0      # these blocks' scale is 1
    k[1234, 0, [0, 16]] = 0.0
    v = rng.standard_normal((n, 1, d))
    v[1234, 0, :32] = 0.0
    pages = K.qcache_alloc(nb, 1, d, bs)
    slots = table[0, np.arange(n) // bs] * bs + np.arange(n) % bs
    rows = [torch.from_numpy(x).float().cuda() for x in (k, v)]
    K.qcache_append(rows[0], rows[1], ints(slots), pages)
    q = torch.zeros(1, 1, d)
    q[0, 0, 0], q[0, 0, 16] = 40 * np.log(2) / 6, 4 * np.log(2) / 6
    q = q.to(dtype).cuda()
    out = K.qcache_dense_decode(q, pages, ints(table), ints([n]), kv_len=n, scale=1.0)
    kk, vv = Q.rows_of(pages.cpu().numpy(), table[0], n, 0, d)
    ref, _, p = Q.attention(f64(q)[0, 0], kk, vv, 1.0)
    tol = bounds(f64(q)[0, 0], kk, vv, p, np.arange(n), ref, 1.0, dtype is F32)
    tol += 2.0 ** -39 * p.max() * np.abs(vv).sum(0)
    assert (np.abs(f64(out)[0, 0] - ref) <= tol).all()
    assert np.abs(ref[:32]).max() < 1e-7 and np.abs(ref[32:]).max() > 0.1


def test_every_call_on_another_stream(K):
    """stream=: each entry point on a stream that is not the current one, its results those of
    the current one."""
    rng = np.random.default_rng(61)
    B, Hq, Hkv, d, bs, width, nb, k = 3, 8, 2, 128, 16, 8, 30, 20
    side = torch.cuda.Stream()
    new = ints([70, 1, 33])
    rows = torch.randn(2, 104, Hkv, d, device="cuda").to(BF)
    more = [torch.randn(3, Hkv, d, device="cuda").to(BF) for _ in range(4)]
    qs = [torch.randn(B, Hq, d, device="cuda").to(BF) for _ in range(2)]
    order, one = ints(rng.permutation(nb)), ints([1, 1, 1])
    ws = [K.Workspace(), K.Workspace()]
    got = []
    for w, kw in ((ws[0], {}), (ws[1], dict(stream=side))):
        table, free, count = ints(np.full((B, width), -1)), order.clone(), ints([nb])
        lens = ints([0] * B)
        pages = [K.qcache_alloc(nb, Hkv, d, bs) for _ in range(2)]
        torch.cuda.synchronize()
        kw = dict(ws=w, **kw)
        slots, cu, lens, count = K.qcache_plan(lens, new, table, free, count, bs, 104, **kw)
        K.qcache_append(rows[0], rows[1], slots, pages[0], **kw)
        K.qcache_append(rows[1], rows[0], slots, pages[1], **kw)
        res = list(K.qcache_read(pages[0], slots, **kw))
        res += list(K.qcache_dense_decode(qs[0], pages[0], table, lens, return_scores=True, **kw))
        for pooled in (False, True):
            res += list(K.qcache_anchor_decode(qs[0], pages[0], table, lens, k, pooled=pooled,
                                               return_scores=True, **kw))
            res.append(K.qcache_reuse_decode(qs[1], pages[1], table, lens, res[-2], pooled=pooled,
                                             **kw))
        outs, idx = K.qcache_run_stack(qs, pages, table, lens, k, [0], new_ks=more[:2],
                                       new_vs=more[2:], new_lens=one, free_blocks=free,
                                       free_count=count, **kw)
        torch.cuda.synchronize()
        assert w.device_error() == K.OK
        got.append(res + list(outs) + [idx, slots, cu, lens, count, table, free] + pages)
    assert len(got[0]) == len(got[1]) and all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("pooled", [False, True])
@pytest.mark.parametrize("dtype,anchors", [(BF, [1]), (F32, [0, 2]), (BF, [])])
def test_stack_without_a_plan(K, dtype, anchors, pooled):
    """Rows go to the caller's slots (some of them padding) and the lengths count them already;
    group map, scale, cache scales and kv_len reach every layer."""
    rng = np.random.default_rng(62)
    lens, Hq, Hkv, d, bs, k, L = [90, 0, 41], 4, 2, 64, 16, 12, 4
    gm = [1, 0, 0, 1]
    cs = dict(k_scale=0.5, v_scale=4.0)
    pages, table = filled(K, rng, lens, Hkv, d, bs, width=9, **cs)
    pages = [pages.clone() for _ in range(L)]
    T, dl = ints(table), ints(lens)
    slots = ints([table[0, 5] * bs + 9, -1, table[2, 2] * bs + 8])     # the last tokens of 0 and 2
    rows = lambda x: [torch.randn(3, Hkv, d, device="cuda").to(dtype) * x for _ in range(L)]
    nk, nv = rows(0.5), rows(4.0)
    qs = [torch.randn(3, Hq, d, device="cuda").to(dtype) for _ in range(L)]
    kw = dict(kv_len=100, group_map=gm, scale=0.2, ws=K.Workspace(), **cs)
    ref, want, idx = [p.clone() for p in pages], [], None
    for l in range(L):
        K.qcache_append(nk[l], nv[l], slots, ref[l], ws=kw["ws"], **cs)
        a = (qs[l], ref[l], T, dl)
        if l in anchors:
            o, idx = K.qcache_anchor_decode(*a, k, pooled=pooled, **kw)
        elif idx is not None:
            o = K.qcache_reuse_decode(*a, idx, pooled=pooled, **kw)
        else:
            o = K.qcache_dense_decode(*a, **kw)
        want.append(o)
    outs, ib = K.qcache_run_stack(qs, pages, T, dl, k, anchors, new_ks=nk, new_vs=nv,
                                  slot_map=slots, pooled=pooled, **kw)
    assert kw["ws"].device_error() == K.OK
    assert all(torch.equal(x, y) for x, y in zip(outs, want))
    assert all(torch.equal(x, y) for x, y in zip(pages, ref))
    assert idx is None or torch.equal(ib, idx)
    assert torch.equal(dl, ints(lens)) and torch.equal(T, ints(table))
    if 0 not in anchors:
        check_attention(qs[0], outs[0], pages[0], table, lens, Hkv, d, gm, scale=0.2, **cs)


def test_largest_plan(K):
    """16384 sequences that start, grow, roll back and end in one step."""
    rng = np.random.default_rng(63)
    B, bs, width = 16384, 16, 3
    nb = B * width
    lens = rng.integers(0, width * bs + 1, B).tolist()
    table = table_of(rng, lens, bs, nb, width)
    held = set(table[table >= 0].tolist())
    rest = [x for x in rng.permutation(nb).tolist() if x not in held]
    free = np.full(nb, -1, dtype=np.int64)
    free[:len(rest)] = rest
    new = random_step(rng, lens, width, bs)
    max_new = sum(max(0, x) for x in new)
    want = Q.plan(lens, new, table, free, len(rest), bs, max_new)
    d = [ints(x) for x in (lens, new, table, free, [len(rest)])]
    ws = K.Workspace()
    got = K.qcache_plan(*d, bs, max_new, ws=ws)
    assert ws.device_error() == K.OK
    for x, y in zip(got[:3], want[:3]):
        assert np.array_equal(x.cpu().numpy(), y)
    assert int(got[3]) == want[3] and np.array_equal(d[2].cpu().numpy(), want[4])
    assert np.array_equal(d[3].cpu().numpy()[:want[3]], want[5][:want[3]])


@pytest.mark.parametrize("pooled", [False, True])
def test_longest_sets_per_query_head(K, pooled):
    """kv_len 262144, the most that sets per query head take: one full sequence beside short
    and empty ones, the anchor's sets exact on its own scores, the reuse layer on them."""
    rng = np.random.default_rng(64)
    lens, Hq, Hkv, d, bs, k = [262144, 3, 0, 5000], 4, 2, 64, 256, 1500
    pages, table = filled(K, rng, lens, Hkv, d, bs)
    q = torch.from_numpy(rng.standard_normal((4, Hq, d))).to(BF).cuda()
    ws = K.Workspace()
    kw = dict(kv_len=262144, pooled=pooled, ws=ws)
    args = (q, pages, ints(table), ints(lens))
    out, idx, sc = K.qcache_anchor_decode(*args, k, return_scores=True, **kw)
    again = K.qcache_reuse_decode(*args, idx, **kw)
    assert ws.device_error() == K.OK
    sn, got = f64(sc), idx.cpu().numpy()
    sets = [[] for _ in lens]
    for b, n in enumerate(lens):
        for h in range(Hkv if pooled else Hq):
            m = min(k, n)
            want = topk_indices(sn[b, h, :n], m) if m else np.zeros(0, dtype=np.int64)
            assert np.array_equal(got[b, h, :m], want) and (got[b, h, m:] == -1).all()
            assert (sn[b, h, n:] == -np.inf).all()
            sets[b].append(want)
    kv = [h // (Hq // Hkv) for h in range(Hq)]
    check_attention(q, out, pages, table, lens, Hkv, d, kv)
    check_attention(q, again, pages, table, lens, Hkv, d, kv, sets=sets, pooled=pooled)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_and_infinite_queries_stay_in_their_head(K, d, dtype):
    """Over every key and over sets: the head's own output is NaN, the others within bounds."""
    rng = np.random.default_rng(65)
    lens, Hq, bs, k = [300, 70], 8, 32, 40
    pages, table = filled(K, rng, lens, 1, d, bs)
    q = torch.from_numpy(rng.standard_normal((2, Hq, d))).to(dtype).cuda()
    sets, idx = random_sets(rng, lens, Hq, k)
    args = (pages, ints(table), ints(lens))
    bad = q.clone()
    bad[0, 2, 5], bad[1, 7, 0], bad[1, 0, d - 1] = float("nan"), float("inf"), -float("inf")
    hit = np.zeros((2, Hq), dtype=bool)
    hit[0, 2] = hit[1, 7] = hit[1, 0] = True
    for run, s in ((lambda x: K.qcache_dense_decode(x, *args), None),
                   (lambda x: K.qcache_reuse_decode(x, *args, ints(idx)), sets)):
        out = run(bad)
        nan = torch.isnan(out).cpu().numpy()
        assert (nan.all(-1) == hit).all() and (nan.any(-1) == hit).all()
        fixed = torch.where(torch.from_numpy(hit).cuda()[..., None], run(q), out)
        check_attention(q, fixed, pages, table, lens, 1, d, [0] * Hq, sets=s)


def test_dropped_inputs_of_another_stream_are_not_given_out_again(K):
    """Tensors that the caller drops while the stream has yet to read them keep their memory.
    The stream waits behind a bounded delay, so the call has not run when they are dropped."""
    rng = np.random.default_rng(66)
    B, Hq, Hkv, d, bs, width, nb, k = 2, 8, 2, 128, 16, 8, 20, 10
    side, ws = torch.cuda.Stream(), K.Workspace()
    lens = [100, 37]
    pages, table = filled(K, rng, lens, Hkv, d, bs, width=width, spare=nb)
    _, idx = random_sets(rng, lens, Hq, k)
    nblk = pages.shape[0]
    fresh = dict(
        q=lambda: torch.randn(B, Hq, d, device="cuda").to(BF), pages=lambda: pages.clone(),
        block_table=lambda: ints(table), kv_lens=lambda: ints(lens), idx=lambda: ints(idx),
        rows=lambda: torch.randn(2, Hkv, d, device="cuda").to(BF), slot_map=lambda: ints([-1, -1]),
        new_lens=lambda: ints([0, 0]), free_blocks=lambda: ints([-1] * nblk),
        free_count=lambda: ints([0]))
    attn = ("q", "pages", "block_table", "kv_lens")
    step = ("block_table", "kv_lens", "new_lens", "free_blocks", "free_count")
    calls = [
        (lambda t: K.qcache_dense_decode(*[t[x] for x in attn], ws=ws, stream=side), attn),
        (lambda t: K.qcache_anchor_decode(*[t[x] for x in attn], k, ws=ws, stream=side), attn),
        (lambda t: K.qcache_reuse_decode(*[t[x] for x in attn], t["idx"], ws=ws, stream=side),
         attn + ("idx",)),
        (lambda t: K.qcache_append(t["rows"], t["rows"], t["slot_map"], t["pages"], ws=ws,
                                   stream=side), ("rows", "slot_map", "pages")),
        (lambda t: K.qcache_read(t["pages"], t["slot_map"], ws=ws, stream=side),
         ("slot_map", "pages")),
        (lambda t: K.qcache_plan(t["kv_lens"], t["new_lens"], *[t[x] for x in (
            "block_table", "free_blocks", "free_count")], bs, 4, ws=ws, stream=side), step),
        (lambda t: K.qcache_run_stack([t["q"]], [t["pages"]], t["block_table"], t["kv_lens"], k, [0],
                                      new_ks=[t["rows"]], new_vs=[t["rows"]],
                                      new_lens=t["new_lens"], free_blocks=t["free_blocks"],
                                      free_count=t["free_count"], ws=ws, stream=side),
         ("q", "pages", "rows") + step)]
    for call, names in calls:
        first, t = ({n: fresh[n]() for n in names} for _ in range(2))
        old = {n: (x.data_ptr(), x.shape, x.dtype) for n, x in t.items()}
        torch.cuda.synchronize()
        call(first)                                      # sizes the workspace
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)               # about 50 ms
        kept = call(t)
        t.clear()
        new = [torch.empty(s, dtype=ty, device="cuda") for _, s, ty in old.values()]
        assert not side.query()                          # it has not come to the call yet
        assert not {x.data_ptr() for x in new} & {p for p, _, _ in old.values()}, names
        torch.cuda.synchronize()
        del kept, new
    assert ws.device_error() == K.OK


def test_growing_workspace_keeps_the_error(K):
    """A refused plan in a workspace of 256 bytes is still reported after a call that grows it."""
    rng = np.random.default_rng(67)
    lens, d, bs = [100, 50], 64, 16
    pages, table = filled(K, rng, lens, 1, d, bs, width=8)
    ws = K.Workspace()
    K.qcache_plan(ints([-1, 50]), ints([1, 1]), ints(table), ints([-1] * pages.shape[0]), ints([0]),
                  bs, 2, ws=ws)
    small = ws.buf.numel()
    q = torch.randn(2, 2, d, device="cuda").to(BF)
    out = K.qcache_dense_decode(q, pages, ints(table), ints(lens), ws=ws)
    assert ws.buf.numel() > small
    assert ws.device_error() == K.BAD_INPUT and ws.device_error() == K.OK
    assert torch.equal(out, K.qcache_dense_decode(q, pages, ints(table), ints(lens)))


def test_growing_workspace_keeps_the_old_memory_for_its_stream(K):
    """The buffer that a growing workspace drops, last used on another stream than its own, is
    not given out again before that stream has come past its calls."""
    rng = np.random.default_rng(68)
    lens, d, bs = [100, 50], 64, 16
    pages, table = filled(K, rng, lens, 1, d, bs, width=8)
    T, dl, slots = ints(table), ints(lens), ints([-1])
    x = torch.zeros(1, 1, d, device="cuda").to(BF)
    q = torch.randn(2, 2, d, device="cuda").to(BF)
    side, ws = torch.cuda.Stream(), K.Workspace()
    ws.get(3 << 20)                                      # on the current stream
    old = ws.buf.data_ptr()
    n = K.Workspace()
    K.qcache_anchor_decode(q, pages, T, dl, 10, ws=n)
    want = n.buf.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                   # about 50 ms
    K.qcache_append(x, x, slots, pages, ws=ws, stream=side)
    with torch.cuda.stream(side):
        ws.get(max(want, 4 << 20))
    new = torch.empty(3 << 20, dtype=torch.uint8, device="cuda")
    assert not side.query() and new.data_ptr() != old and ws.buf.data_ptr() != old
    K.qcache_anchor_decode(q, pages, T, dl, 10, ws=ws, stream=side)
    torch.cuda.synchronize()
    assert ws.device_error() == K.OK
