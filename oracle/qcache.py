"""Paged 4-bit key/value cache in plain numpy: the number format, the block
planner and decode attention over the cache, in float64. Test infrastructure;
shares no code with the CUDA path."""
import numpy as np

GROUP = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 finite non-negative e4m3 numbers: 3 fraction bits, bias 7, subnormals
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                 for e in range(16) for m in range(8)][:127])


def nearest_even(x, grid):
    """Index of the grid number nearest to each x >= 0; the even index at a tie;
    the last one above the grid."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    left, right = x - grid[lo], grid[hi] - x
    return np.where((right < left) | ((right == left) & (hi % 2 == 0)), hi, lo)


def stored(x, scale=1.0):
    """The values that rows x [..., d] have once they are in the cache."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16)) / scale
    nan = np.isnan(b).any(-1, keepdims=True)
    b = np.clip(np.where(np.isnan(b), 0.0, b), -1e30, 1e30)
    s = E4M3[nearest_even(np.abs(b).max(-1) / 6.0, E4M3)][..., None]
    y = E2M1[nearest_even(np.abs(b) / np.where(s > 0, s, 1.0), E2M1)] * (s > 0)
    out = np.where(nan, np.nan, np.sign(b) * y * s) * scale
    return out.reshape(x.shape)


def group_fields(pages, d):
    """pages uint8 [nb, Hkv, groups, 18 d] -> K codes, K scales, V codes, V scales,
    each [nb, Hkv, groups, 16, bytes]."""
    pages = np.asarray(pages)
    sizes = [8 * d, d, 8 * d, d]
    at = np.cumsum([0] + sizes)
    return [pages[..., at[i]:at[i + 1]].reshape(pages.shape[:3] + (GROUP, -1)) for i in range(4)]


def decode_rows(codes, scales, scale=1.0):
    """Codes [..., d/2] and scales [..., d/16] bytes -> values [..., d]."""
    lo, hi = codes & 15, codes >> 4
    code = np.stack([lo, hi], -1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    val = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    e4 = np.append(E4M3, np.nan)
    s = np.where(scales >= 128, -1.0, 1.0) * e4[scales & 127]
    blocks = val.reshape(val.shape[:-1] + (scales.shape[-1], 16))
    return (blocks * s[..., None]).reshape(val.shape) * scale


def rows_of(pages, table_row, n, head, d, k_scale=1.0, v_scale=1.0):
    """The n cached rows (K [n, d], V [n, d]) of one sequence and KV head."""
    bs = pages.shape[2] * GROUP
    pos = np.arange(n)
    block = np.asarray(table_row)[pos // bs]
    kc, ks, vc, vs = group_fields(pages, d)
    at = (block, head, (pos % bs) // GROUP, pos % GROUP)
    return decode_rows(kc[at], ks[at], k_scale), decode_rows(vc[at], vs[at], v_scale)


def plan(kv_lens, new_lens, table, free, count, bs, max_new):
    """One step: (slot_map, cu_new, lens, count, table, free), or None if it cannot be served.
    Inputs are not changed."""
    table, free = np.array(table), np.array(free)
    nb, width = len(free), table.shape[1]
    cap = width * bs
    to = [max(0, int(l) + int(n)) for l, n in zip(kv_lens, new_lens)]
    if any(not 0 <= l <= cap for l in kv_lens) or any(t > cap for t in to):
        return None
    blocks = lambda t: (int(t) + bs - 1) // bs
    given = [int(table[b, j]) for b in range(len(to)) for j in range(blocks(to[b]), blocks(kv_lens[b]))]
    taken = [(b, j) for b in range(len(to)) for j in range(blocks(kv_lens[b]), blocks(to[b]))]
    if not 0 <= count <= nb or count + len(given) > nb or len(taken) > count + len(given):
        return None
    new = [max(0, t - int(l)) for t, l in zip(to, kv_lens)]
    if sum(new) > max_new:
        return None
    stack = [int(x) for x in free[:count]] + given
    used = [stack[len(stack) - 1 - i] for i in range(len(taken))]
    # the partly filled block that a growing sequence's first new tokens go to
    tail = [int(table[b, int(l) // bs]) for b, l in enumerate(kv_lens) if to[b] > l and l % bs]
    if any(not 0 <= x < nb for x in given + used + tail):
        return None
    free[count:count + len(given)] = given
    for (b, j), x in zip(taken, used):
        table[b, j] = x
    slots = [int(table[b, p // bs]) * bs + p % bs
             for b in range(len(to)) for p in range(int(kv_lens[b]), to[b])]
    slots += [-1] * (max_new - len(slots))
    return (np.array(slots, dtype=np.int64), np.concatenate([[0], np.cumsum(new)]), np.array(to),
            count + len(given) - len(taken), table, free)


def attention(q, k, v, scale, keys=None):
    """One query head over the rows `keys` (all by default): (out [d], logits over all
    rows, weights over the chosen rows). No row: zeros."""
    logits = scale * (k @ q)
    sel = np.arange(len(k)) if keys is None else np.asarray(keys, dtype=np.int64)
    if len(sel) == 0:
        return np.zeros(v.shape[-1]), logits, np.zeros(0)
    s = logits[sel]
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v[sel], logits, p
