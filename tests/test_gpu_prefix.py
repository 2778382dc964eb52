"""Decode over a prefix that a batch shares, on the GPU, through the binding, against the
float64 oracle (oracle/qcache.py): every sequence on its own over all of its tokens. The
tolerances are those of tests/test_gpu_qcache.py: the same operands, roundings of the
weights (2^-11 and 2^-21) and fp32 sums."""
import numpy as np
import pytest
import torch

import __graft_entry__
from gpu_helpers import f64
from oracle import qcache as Q
from oracle import rope as R
from test_gpu_qcache import check_attention, ints

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def K():
    __graft_entry__.build()
    from long_context_anchor_gb300 import kascade
    return kascade


def shared_decode(K, *args, **kw):
    """With the prefix shared, however small the batch is."""
    return K.qcache_prefix_decode(*args, always=True, **kw)


def shared_batch(K, rng, lens, P, Hkv, d, bs, dtype, scales=(1.0, 1.0), garbage=255, extra=0):
    """Pages (unused bytes all 0xff: NaN scales) and tables: sequences of at least P tokens
    share their first blocks, shorter ones have blocks of their own."""
    front = P // bs
    width = max(1, front, max((n + bs - 1) // bs for n in lens)) + extra
    own = [((n + bs - 1) // bs) - (front if n >= P else 0) for n in lens]
    nb = front + sum(own) + 2
    ids = rng.permutation(nb)
    table, at = np.full((len(lens), width), -1, dtype=np.int64), front
    for b, n in enumerate(lens):
        lo = front if n >= P else 0
        if n >= P:
            table[b, :front] = ids[:front]
        table[b, lo:lo + own[b]] = ids[at:at + own[b]]
        at += own[b]
    pages = torch.full((nb, Hkv, bs // 16, 18 * d), garbage, dtype=torch.uint8, device="cuda")
    slots = [table[b, np.arange(lo, n) // bs] * bs + np.arange(lo, n) % bs
             for b, n in enumerate(lens) for lo in [P if n >= P else 0]]
    slots = np.concatenate(slots + [(ids[:front, None] * bs + np.arange(bs)).reshape(-1)
                                    if any(n >= P for n in lens) else np.zeros(0, np.int64)])
    k = torch.from_numpy(rng.standard_normal((len(slots), Hkv, d)) * scales[0]).to(dtype).cuda()
    v = torch.from_numpy(rng.standard_normal((len(slots), Hkv, d)) * scales[1]).to(dtype).cuda()
    K.qcache_append(k, v, ints(slots), pages, k_scale=scales[0], v_scale=scales[1])
    return pages, table


def queries(rng, B, Hq, d, dtype):
    return torch.from_numpy(rng.standard_normal((B, Hq, d)) * 1.5).to(dtype).cuda()


def straight(Hq, Hkv):
    return [h // (Hq // Hkv) for h in range(Hq)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,G,Hkv,d,bs,P", [
    (1, 1, 1, 128, 16, 16), (1, 4, 2, 64, 64, 64), (3, 2, 2, 64, 16, 48), (5, 8, 1, 128, 32, 224),
    (16, 8, 2, 64, 64, 1024), (32, 4, 2, 128, 16, 1040), (33, 4, 1, 128, 64, 640),
    (40, 8, 1, 64, 128, 2048), (64, 4, 1, 128, 256, 768), (65, 4, 1, 64, 16, 80),
    (9, 1, 3, 128, 16, 4112), (130, 2, 1, 128, 32, 96), (2, 8, 8, 128, 64, 8192)])
def test_ragged_batches(K, B, G, Hkv, d, bs, P, dtype):
    """One row up to several tiles of rows, prefixes that end inside a tile of keys, own
    parts of zero, one and more tokens, and (from five sequences on) shorter ones."""
    rng = np.random.default_rng(B * 1000 + P)
    lens = [P + int(x) for x in rng.integers(0, 150, B)]
    lens[0] = P
    if B >= 3:
        lens[1] = P + 1
    if B >= 5:
        lens[2], lens[3], lens[4] = 0, 1, P - 1
        lens = [lens[i] for i in rng.permutation(B)]
    pages, table = shared_batch(K, rng, lens, P, Hkv, d, bs, dtype)
    q = queries(rng, B, G * Hkv, d, dtype)
    ws = K.Workspace("cuda")
    args = (q, pages, ints(table), ints(lens))
    got = shared_decode(K, *args, P, ws=ws)
    assert ws.device_error() == K.OK
    check_attention(q, got, pages, table, lens, Hkv, d, straight(G * Hkv, Hkv))
    assert torch.equal(got, shared_decode(K, *args, P, ws=ws))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_head_map_scales_and_wide_tables(K, dtype, d):
    rng = np.random.default_rng(3)
    B, P, bs, Hkv = 12, 320, 32, 2
    heads = [1, 0, 0, 1, 1, 0, 1, 0]
    scales = (0.125, 4.0)
    lens = [P + 7 * b for b in range(B)]
    pages, table = shared_batch(K, rng, lens, P, Hkv, d, bs, dtype, scales, extra=3)
    q = queries(rng, B, 8, d, dtype) * 8
    got = shared_decode(K, q, pages, ints(table), ints(lens), P, kv_len=max(lens),
                        group_map=heads, scale=0.07, k_scale=scales[0], v_scale=scales[1])
    check_attention(q, got, pages, table, lens, Hkv, d, heads, k_scale=scales[0],
                    v_scale=scales[1], scale=0.07)


def test_no_sequence_has_the_prefix_and_no_prefix(K):
    rng = np.random.default_rng(4)
    lens, P, bs = [0, 30, 47, 5], 48, 16
    pages, table = shared_batch(K, rng, lens, P, 2, 64, bs, BF)
    q = queries(rng, 4, 8, 64, BF)
    for p in (P, 0):
        ws = K.Workspace("cuda")
        got = shared_decode(K, q, pages, ints(table), ints(lens), p, kv_len=48, ws=ws)
        assert ws.device_error() == K.OK
        check_attention(q, got, pages, table, lens, 2, 64, straight(8, 2))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_row_tiles_and_a_long_prefix(K, dtype):
    rng = np.random.default_rng(5)
    P, bs = 16384, 64
    lens = [P + int(x) for x in rng.integers(0, 40, 150)]
    lens[17], lens[149] = 0, P
    pages, table = shared_batch(K, rng, lens, P, 2, 64, bs, dtype)
    q = queries(rng, 150, 8, 64, dtype)
    got = shared_decode(K, q, pages, ints(table), ints(lens), P)
    check_attention(q, got, pages, table, lens, 2, 64, straight(8, 2))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rising_scores(K, dtype):
    """Keys whose scores rise along the prefix by far more than a reference's slack, and
    fall again: sums and outputs are rescaled at every tile."""
    rng = np.random.default_rng(6)
    P, bs, d = 1024, 32, 128
    lens = [P + 20] * 9
    pages, table = shared_batch(K, rng, lens, P, 1, d, bs, dtype)
    pos = np.arange(P)
    ramp = np.where(pos < 700, pos, 1400 - pos) / 8.0
    k = np.zeros((P, 1, d))
    k[:, 0, :16] = ramp[:, None]                       # one block of 16 equal elements
    v = rng.standard_normal((P, 1, d))
    slots = table[0, pos // bs] * bs + pos % bs
    K.qcache_append(torch.from_numpy(k).to(dtype).cuda(), torch.from_numpy(v).to(dtype).cuda(),
                    ints(slots), pages)
    q = torch.zeros(9, 4, d, dtype=dtype, device="cuda")
    q[..., :16] = torch.from_numpy(rng.choice([-1.0, 1.0, 2.0], (9, 4, 1))).to(dtype).cuda()
    got = shared_decode(K, q, pages, ints(table), ints(lens), P)
    check_attention(q, got, pages, table, lens, 1, d, straight(4, 1))


def test_nan_values_reach_only_their_readers(K):
    """A NaN block of V in the prefix: dims of that block of the sequences that read it. A
    shorter sequence, and what lies behind a prefix that ends inside a tile, stay clean."""
    rng = np.random.default_rng(7)
    P, bs, d = 80, 16, 64
    lens = [P + 3, P, 40, 0, P + 30]
    pages, table = shared_batch(K, rng, lens, P, 2, d, bs, BF)
    q = queries(rng, 5, 4, d, BF)
    clean = shared_decode(K, q, pages, ints(table), ints(lens), P)
    assert torch.isfinite(clean).all()
    block = int(table[0, 2])
    pages[block, 1, 0, 17 * d + 5 * (d // 16) + 1] = 0x7f       # key 37's V, dims 16 .. 31
    got = shared_decode(K, q, pages, ints(table), ints(lens), P)
    bad = torch.isnan(got)
    for b, n in enumerate(lens):
        for h in range(4):
            want = torch.zeros(d, dtype=torch.bool)
            if n >= P and h >= 2:
                want[16:32] = True
            assert torch.equal(bad[b, h].cpu(), want), (b, h)
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_huge_and_infinite_queries(K, dtype):
    rng = np.random.default_rng(8)
    P, bs, d = 192, 64, 64
    lens = [P + 5] * 6
    pages, table = shared_batch(K, rng, lens, P, 1, d, bs, dtype)
    q = queries(rng, 6, 2, d, dtype)
    q[1] *= 2.0 ** 60
    q[2] *= 2.0 ** -60
    q[3] = 0.0
    q[4, 0, 3] = float("inf")
    q[5, 1, 7] = float("nan")
    got = shared_decode(K, q, pages, ints(table), ints(lens), P)
    fine = [b for b in range(6) if b != 1]
    for b in fine:
        for h in range(2):
            k, v = Q.rows_of(pages.cpu().numpy(), table[b], lens[b], 0, d, 1.0, 1.0)
            if (b, h) in ((4, 0), (5, 1)):
                assert torch.isnan(got[b, h]).all()
                continue
            want = Q.attention(f64(q[b, h]), k, v, d ** -0.5)[0]
            assert np.abs(f64(got[b, h]) - want).max() <= 2.0 ** -6 * np.abs(v).max()
    # a huge query: the weight is all on one key
    for h in range(2):
        k, v = Q.rows_of(pages.cpu().numpy(), table[1], lens[1], 0, d, 1.0, 1.0)
        want = v[np.argmax(k @ f64(q[1, h]))]
        assert np.abs(f64(got[1, h]) - want).max() <= 2.0 ** -8 * np.abs(want).max()


def test_device_errors(K):
    rng = np.random.default_rng(9)
    P, bs, d = 128, 16, 64
    lens = [P + 4] * 4
    pages, table = shared_batch(K, rng, lens, P, 1, d, bs, BF)
    q = queries(rng, 4, 4, d, BF)
    ws = K.Workspace("cuda")
    run = lambda t, n: shared_decode(K, q, pages, ints(t), ints(n), P, ws=ws)
    run(table, lens)
    assert ws.device_error() == K.OK
    other = table.copy()
    other[2, 3] = table[0, 4]                       # another block than the other sequences'
    run(other, lens)
    assert ws.device_error() == K.BAD_INPUT
    bad = table.copy()
    bad[:, 5] = pages.shape[0]                      # outside the cache: its keys are masked
    got = run(bad, lens)
    assert ws.device_error() == K.BAD_INPUT
    pg = pages.cpu().numpy()
    for b in range(4):
        k, v = Q.rows_of(pg, table[b], lens[b], 0, d, 1.0, 1.0)
        sel = np.r_[0:80, 96:lens[b]]
        for h in range(4):
            want = Q.attention(f64(q[b, h]), k, v, d ** -0.5, sel)[0]
            assert np.abs(f64(got[b, h]) - want).max() < 2e-2
    run(table, [P + 4, -1, P + 4, 10 ** 6])         # lengths out of range
    assert ws.device_error() == K.BAD_INPUT
    run(table, lens)
    assert ws.device_error() == K.OK


def test_graph_stream_and_one_workspace_for_many_shapes(K):
    rng = np.random.default_rng(10)
    P, bs = 256, 32
    ws = K.Workspace("cuda")
    for B, G, Hkv, d, dtype in ((20, 4, 2, 128, BF), (3, 8, 1, 64, F32), (70, 2, 1, 64, BF)):
        lens = [P + 5 * (b % 9) for b in range(B)]
        pages, table = shared_batch(K, rng, lens, P, Hkv, d, bs, dtype)
        q, t, n = queries(rng, B, G * Hkv, d, dtype), ints(table), ints(lens)
        want = shared_decode(K, q, pages, t, n, P, ws=ws)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = shared_decode(K, q, pages, t, n, P, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got, want)
        own, out = K.Workspace("cuda"), torch.empty_like(q)
        shared_decode(K, q, pages, t, n, P, ws=own, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            shared_decode(K, q, pages, t, n, P, ws=own, out=out)
        q.mul_(-0.5)
        n.sub_(3)                     # those of exactly P tokens no longer take part
        g.replay()
        assert torch.equal(out, shared_decode(K, q, pages, t, n, P, ws=ws))
        assert own.device_error() == K.OK and ws.device_error() == K.OK
        dense = K.qcache_dense_decode(q, pages, t, n)
        step = 2.0 ** -7 if dtype == BF else 2.0 ** -18
        assert (out.float() - dense.float()).abs().max() <= step * dense.abs().max()


def test_pages_beyond_32_bits(K):
    """Blocks whose bytes lie behind 2^32."""
    rng = np.random.default_rng(11)
    bs, d, Hkv, P = 256, 128, 8, 512
    nb = (5 << 30) // (Hkv * (bs // 16) * 18 * d)
    pages = torch.empty(nb, Hkv, bs // 16, 18 * d, dtype=torch.uint8, device="cuda")
    lens = [P + 9, P, P + 300]
    table = np.array([[nb - 1, nb - 3, nb - 5, -1], [nb - 1, nb - 3, -1, -1],
                      [nb - 1, nb - 3, nb - 2, nb - 7]])
    slots = np.concatenate([table[2, np.arange(P + 300) // bs] * bs + np.arange(P + 300) % bs,
                            (nb - 5) * bs + np.arange(9)])
    k, v = (torch.from_numpy(rng.standard_normal((len(slots), Hkv, d))).to(BF).cuda()
            for _ in range(2))
    K.qcache_append(k, v, ints(slots), pages)
    q = queries(rng, 3, 16, d, BF)
    got = shared_decode(K, q, pages, ints(table), ints(lens), P)
    used = sorted({int(x) for x in table.reshape(-1) if x >= 0})
    small = pages[torch.tensor(used, device="cuda")]
    at = {x: i for i, x in enumerate(used)}
    back = np.array([[at.get(int(x), -1) for x in row] for row in table])
    check_attention(q, got, small, back, lens, Hkv, d, straight(16, Hkv))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B", [1, 2, 70])
def test_batches_that_sharing_does_not_help(K, B, dtype):
    """Unless told otherwise a small batch gets the dense call's results, bit for bit, and the
    check of its tables."""
    rng = np.random.default_rng(13)
    P, bs = 64, 16
    lens = [P + 3 * (b % 7) for b in range(B)]
    pages, table = shared_batch(K, rng, lens, P, 2, 64, bs, dtype)
    q, t, n = queries(rng, B, 8, 64, dtype), ints(table), ints(lens)
    ws, out = K.Workspace("cuda"), torch.empty_like(q)
    assert torch.equal(K.qcache_prefix_decode(q, pages, t, n, P, ws=ws, out=out),
                       K.qcache_dense_decode(q, pages, t, n))
    assert ws.device_error() == K.OK
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.qcache_prefix_decode(q, pages, t, n, P, ws=ws, out=out)
    t[B - 1, 2] = (t[B - 1, 2] + 1) % pages.shape[0]
    q.mul_(-1)
    g.replay()
    assert ws.device_error() == (K.BAD_INPUT if B > 1 else K.OK)
    if B > 1:
        n[B - 1] = P - 1              # then its blocks are its own
        g.replay()
        assert ws.device_error() == K.OK
        assert torch.equal(out, K.qcache_dense_decode(q, pages, t, n))


@pytest.mark.parametrize("B,G,Hkv,d,P,own", [(520, 4, 8, 128, 1024, 40), (2048, 8, 4, 64, 512, 20)])
def test_more_rows_than_sms(K, B, G, Hkv, d, P, own):
    """Several CTAs after one another on an SM, beside the own parts: against the dense call."""
    rng = np.random.default_rng(14)
    bs = 16
    lens = [P + int(x) for x in rng.integers(0, own, B)]
    lens[5] = 7
    pages, table = shared_batch(K, rng, lens, P, Hkv, d, bs, BF)
    q, t, n = queries(rng, B, G * Hkv, d, BF), ints(table), ints(lens)
    ws = K.Workspace("cuda")
    got = shared_decode(K, q, pages, t, n, P, kv_len=P + own, ws=ws)
    assert ws.device_error() == K.OK
    dense = K.qcache_dense_decode(q, pages, t, n)
    # either is off by its weights' 2^-11 and an output's 2^-8 of the values it averages
    assert (got.float() - dense.float()).abs().max() <= 2.0 ** -7 * dense.abs().max()
    some = rng.choice(B, 6, replace=False)
    check_attention(q[some], got[some], pages, table[some], [lens[b] for b in some], Hkv, d,
                    straight(G * Hkv, Hkv))


def test_two_streams_at_once(K):
    """Calls of two streams that share the GPU, each with its workspace: the results of calls
    one after the other."""
    rng = np.random.default_rng(15)
    sets = []
    for B, G, Hkv, d, P, dtype in ((40, 4, 2, 128, 2048, BF), (24, 8, 4, 64, 4096, F32)):
        lens = [P + 11 * (b % 13) for b in range(B)]
        pages, table = shared_batch(K, rng, lens, P, Hkv, d, 32, dtype)
        args = (queries(rng, B, G * Hkv, d, dtype), pages, ints(table), ints(lens), P)
        sets.append((args, shared_decode(K, *args), torch.cuda.Stream(), K.Workspace("cuda")))
    torch.cuda.synchronize()
    outs = [[] for _ in sets]
    for _ in range(25):
        for (args, _, s, ws), got in zip(sets, outs):
            got.append(shared_decode(K, *args, ws=ws, stream=s))
    torch.cuda.synchronize()
    for (_, want, _, ws), got in zip(sets, outs):
        assert ws.device_error() == K.OK
        assert all(torch.equal(x, want) for x in got)


def test_a_server_over_one_prefix(K):
    """Plan, turned appends and decode together: a prompt that is cached once, requests
    that start behind it, grow, end and start again; the oracle follows every token."""
    rng = np.random.default_rng(12)
    bs, Hkv, G, d, B, P = 16, 2, 4, 64, 6, 96
    Hq, width, nb = Hkv * G, 14, 60
    table, lens = torch.full((B, width), -1, dtype=I32, device="cuda"), ints([0] * B)
    free, count = ints(rng.permutation(nb)), ints([nb])
    pages = K.qcache_alloc(nb, Hkv, d, bs)
    tab = K.rope_table(10000.0 ** (-np.arange(d // 2) / (d // 2)), width * bs)
    ws = K.Workspace("cuda")

    def rows(n, heads):
        return torch.from_numpy(rng.standard_normal((n, heads, d))).to(BF).cuda()

    # the prompt, cached by sequence 0
    start = [P] + [0] * (B - 1)
    slots, cu, lens, count = K.qcache_plan(lens, ints(start), table, free, count, bs, P, ws=ws)
    k, v = rows(P, Hkv), rows(P, Hkv)
    K.qcache_append_rope(k, v, slots, pages, tab, cu_new=cu, kv_lens=lens, ws=ws)
    table[1:, :P // bs] = table[0, :P // bs]
    lens.fill_(P)
    truth = [[(P, k, v)] for _ in range(B)]         # (length, new keys, new values)
    total = [P] * B
    for step in range(14):
        new = rng.choice([0, 1, 1, 1, 7], B)
        for b in range(B):
            if total[b] > P + 60 or (step in (5, 9) and b % 2):
                new[b] = P - total[b]                # the request ends, its own blocks go back
        grow = int(np.maximum(new, 0).sum())
        T = grow + 2
        slots, cu, lens, count = K.qcache_plan(lens, ints(new), table, free, count, bs, T, ws=ws)
        k, v, q = rows(T, Hkv), rows(T, Hkv), rows(B, Hq)
        turned = K.qcache_append_rope(k, v, slots, pages, tab, q=q, cu_new=cu, kv_lens=lens, ws=ws)
        out = K.qcache_prefix_decode(turned, pages, table, lens, P, ws=ws)
        assert ws.device_error() == K.OK
        at = 0
        for b in range(B):
            if new[b] < 0:
                truth[b] = truth[b][:1]
            elif new[b] > 0:
                truth[b].append((int(new[b]), k[at:at + new[b]], v[at:at + new[b]]))
                at += int(new[b])
            total[b] += int(new[b])
        assert lens.tolist() == total
        freq = 10000.0 ** (-np.arange(d // 2) / (d // 2))
        for b in (step % B, (step + 3) % B):
            n = total[b]
            ks = torch.cat([x[1] for x in truth[b]]).float().cpu().numpy()
            vs = torch.cat([x[2] for x in truth[b]]).double().cpu().numpy()
            c, s = R.turn_of(tab.cpu().numpy(), np.arange(n))
            ks = Q.stored(R.turned(ks, c[:, None], s[:, None], False)[0])
            vs = Q.stored(vs)
            for h in range(Hq):
                c, s = R.turn_of(R.table(freq, n), np.array(n - 1))
                qt = f64(turned[b, h])
                want_q = R.turned(f64(q[b, h]), c, s, False)[0]
                assert (np.abs(qt - want_q) <= 2.0 ** -7 * np.abs(f64(q[b, h])).max()).all()
                want, _, p = Q.attention(qt, ks[:, h // G], vs[:, h // G], d ** -0.5)
                avg = p @ np.abs(vs[:, h // G])
                err = np.abs(f64(out[b, h]) - want)
                assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * avg).all(), (step, b, h)
    assert count.item() == nb - P // bs - sum((n + bs - 1) // bs - P // bs for n in total)
