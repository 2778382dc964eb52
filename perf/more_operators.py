"""Rotary positions on the way into attention, and a prefix that a batch shares: what is measured.

Three operators that serve next to the paged 4-bit key/value cache:

* rotate: queries and keys divided by their root mean square per head (where a weight is
  given) and turned by their positions, in one pass; positions of one axis or several.
* append: new keys turned by their positions and quantised into the cache with their
  values, and the queries turned in the same call.
* prefix: decode attention for a batch whose sequences begin with the same blocks.

The rotation table is float32 [positions, 2, pairs]: cosines, then sines. Pair i of a head is
elements (i, i + pairs), or (2 i, 2 i + 1) where interleaved; elements behind 2 * pairs
stay as they are. A stored key is quantised from its turned elements in 32 bits, the two
products of an element rounded apart.

The cache is uint8 [num_blocks, Hkv, block_size / 16, 18 d]: groups of 16 tokens, each
group its 16 rows of key codes (d / 2 bytes, two 4-bit e2m1 values per byte, the even
element in the low half), of key scales (d / 16 bytes, one e4m3 number per 16 elements),
of value codes and of value scales. A stored element is code * scale.
"""
import math

import torch

own = False      # True: the framework's calls; False: elementary torch operations

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------- cases --

def listed():
    return [
        # queries and keys of one decode step of eight requests, the 8B shape
        {"name": "rotate_step", "op": "rotate", "B": 1, "N": 8, "Hq": 32, "Hkv": 8, "d": 128,
         "rot": 128, "dtype": "bf16", "norm": True, "interleaved": False, "axes": "",
         "layout": "rows"},
        # two images' or clips' tokens behind text, positions of three axes, in 32 bits
        {"name": "rotate_video", "op": "rotate", "B": 2, "N": 5003, "Hq": 16, "Hkv": 4, "d": 64,
         "rot": 64, "dtype": "f32", "norm": True, "interleaved": True, "axes": "sections",
         "layout": "heads"},
        # a 16384-token prompt of the 8B shape, from the projection's rows to the prefill layout
        {"name": "rotate_prompt", "op": "rotate", "B": 1, "N": 16384, "Hq": 32, "Hkv": 8,
         "d": 128, "rot": 128, "dtype": "bf16", "norm": True, "interleaved": False, "axes": "",
         "layout": "heads"},
        # the 64-head long shape's whole context, half of each head turned, no norm
        {"name": "rotate_long", "op": "rotate", "B": 1, "N": 131072, "Hq": 64, "Hkv": 8, "d": 64,
         "rot": 32, "dtype": "bf16", "norm": False, "interleaved": False, "axes": "",
         "layout": "heads"},
        # one decode step of eight requests: a new token each, one layer of the 8B shape
        {"name": "append_step", "op": "append", "form": "plan", "B": 8, "most": 1, "N": 32768,
         "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "bs": 64, "dtype": "bf16",
         "interleaved": False, "axes": "", "pad": 0},
        # a busy server's step: 500 requests, most with one token, some with none or a piece
        # of their prompt
        {"name": "append_busy", "op": "append", "form": "plan", "B": 500, "most": 64, "N": 16384,
         "Hq": 64, "Hkv": 8, "d": 64, "rot": 64, "bs": 16, "dtype": "bf16",
         "interleaved": False, "axes": "", "pad": 100},
        # a piece of a prompt in 32 bits, odd sizes, part of each head turned
        {"name": "append_piece", "op": "append", "form": "rows", "T": 1531, "N": 40000, "Hq": 6,
         "Hkv": 3, "d": 128, "rot": 96, "bs": 32, "dtype": "f32", "interleaved": True,
         "axes": "", "pad": 29},
        # a whole 16384-token prompt of the 8B shape
        {"name": "append_prompt", "op": "append", "form": "rows", "T": 16384, "N": 16384,
         "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "bs": 64, "dtype": "bf16",
         "interleaved": False, "axes": "", "pad": 0},
        # the bring-up shape in 32 bits: three short requests over one instruction text
        {"name": "prefix_tiny", "op": "prefix", "B": 3, "Hq": 4, "Hkv": 2, "d": 64, "P": 512,
         "more": 100, "bs": 16, "dtype": "f32", "empty": 1},
        # 32 requests over one long instruction text, each with a conversation of its own
        {"name": "prefix_chat", "op": "prefix", "B": 32, "Hq": 32, "Hkv": 8, "d": 128, "P": 8192,
         "more": 2047, "bs": 64, "dtype": "bf16", "empty": 0},
        # sixteen questions about one document of the 64-head long shape's length
        {"name": "prefix_document", "op": "prefix", "B": 16, "Hq": 64, "Hkv": 8, "d": 64,
         "P": 131072, "more": 300, "bs": 64, "dtype": "bf16", "empty": 0},
        # 128 answers sampled from one 32768-token prompt of the 8B shape
        {"name": "prefix_samples", "op": "prefix", "B": 128, "Hq": 32, "Hkv": 8, "d": 128,
         "P": 32768, "more": 1000, "bs": 64, "dtype": "bf16", "empty": 3},
    ]


def draw(rng):
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotate", "append", "prefix", "prefix"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "f32"])
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 8])
    case = {"op": op, "Hq": Hkv * G, "Hkv": Hkv, "d": d, "dtype": dtype}
    size = 2 if dtype == "bf16" else 4
    if op in ("rotate", "append"):
        case["rot"] = rng.choice([32, 64, d, d])
        case["interleaved"] = rng.random() < 0.4
        case["axes"] = rng.choice(["", "", "sections", "cyclic"])
    if op == "rotate":
        # rows in and out cost no more than the largest listed case's
        most = (131072 * 72 * 64 * 2) // ((Hkv * G + Hkv) * d * size)
        N = span(1, min(131072, most))
        case.update(B=span(1, max(1, min(16, most // N))), N=N, norm=rng.random() < 0.6,
                    layout=rng.choice(["rows", "heads"]))
        return case
    case["bs"] = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        most = min(16384, (16384 * 48 * 128 * 2) // ((Hkv * G + 2 * Hkv) * d * size))
        case.update(form=rng.choice(["rows", "plan"]), N=span(256, 131072),
                    pad=rng.choice([0, 0, rng.randint(1, 64)]))
        if case["form"] == "rows":
            case["T"] = span(1, most)
        else:
            case.update(B=span(1, min(512, most)), most=1)
            case["most"] = span(1, max(1, min(256, case["N"], most * 4 // case["B"])))
        return case
    P = case["bs"] * max(1, span(16, 131072) // case["bs"])
    most = (128 * 32 * 33000 * 128) // (Hkv * G * (P + 256) * d)
    B = span(1, max(1, min(128, most if dtype == "bf16" else most // 2)))
    case.update(B=B, P=P, more=span(1, max(1, min(4096, 128 * 1000 * 8 // (B * Hkv)))),
                empty=rng.choice([0, 0, rng.randint(0, B // 4)]))
    return case


def blocks_of(tokens, bs):
    return (tokens + bs - 1) // bs


def table_len(case):
    """Positions that the rotation table holds."""
    return case["N"] if case["op"] == "append" else max(64, case["N"])


def pair_axes(case):
    """The axis that turns each pair, or None where there is one axis."""
    n = case["rot"] // 2
    if case["axes"] == "sections":       # a quarter for time, the rest for height and width
        return [0 if i < n // 4 else 1 if i < n // 4 + 3 * n // 8 else 2 for i in range(n)]
    return [i % 3 for i in range(n)] if case["axes"] == "cyclic" else None


def new_tokens(case):
    """New tokens per sequence of an append in the plan's form, before shuffling."""
    B, most = case["B"], case["most"]
    return [most if most > 1 and i % 61 == 7 else 0 if most > 1 and i % 13 == 5 else 1
            for i in range(B)]


def tokens_of(case):
    return case["T"] if case["form"] == "rows" else sum(new_tokens(case))


def lengths(case):
    """Cached tokens per sequence of a prefix case, before shuffling: some rows of a padded
    batch have none, or end within the prefix."""
    B, P, more = case["B"], case["P"], case["more"]
    out = [P + int(more * ((i + 1) / B) ** 2) for i in range(B)]
    for i in range(case["empty"]):
        out[i] = 0 if i % 3 == 0 else P // 2 + i if i % 3 == 1 else P
    return out


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "rotate":
        T = case["B"] * case["N"]
        axes = 3 if case["axes"] else 1
        # rows in and out, the table's rows that positions name, positions, weights
        return {"bytes": 2 * T * (Hq + Hkv) * d * size + min(T, table_len(case)) * case["rot"] * 4
                + 4 * axes * T + 8 * d * case["norm"],
                "flops": T * (Hq + Hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "append":
        T = tokens_of(case)
        queries = case["B"] if case["form"] == "plan" else T + case["pad"]
        # queries in and out; keys and values in, into the cache, read back from it, out
        return {"bytes": 2 * queries * Hq * d * size + T * Hkv * d * (4 * size) + T * Hkv * d * 9 // 4
                + T * (case["rot"] * 4 + 8),
                "flops": (queries * Hq + T * Hkv) * 3 * case["rot"] + T * Hkv * d * 8}
    lens = lengths(case)
    own_tokens = sum(max(0, n - case["P"]) for n in lens)
    read = min(case["P"], max(lens)) + own_tokens
    return {"bytes": read * Hkv * (d * 9 // 8) + 2 * case["B"] * Hq * d * size
            + 4 * read // case["bs"],
            "flops": 4 * d * Hq * sum(lens)}


# ------------------------------------------------------------------------ inputs --

def to_e4m3(x):
    """Nearest e4m3 number (ties to even) of non-negative 64-bit numbers, in 64 bits."""
    e = torch.frexp(x)[1] - 1
    q = torch.exp2((e.clamp(min=-6) - 3).double())
    return (torch.round(x / q) * q).clamp(max=448.0)


def quantise(x):
    """Rows [..., d] -> (codes uint8 [..., d / 2], scales uint8 [..., d / 16]), in 64 bits:
    the scale is the block's largest magnitude / 6, each code the nearest e2m1 number."""
    x = x.double().unflatten(-1, (-1, 16))
    scale = to_e4m3(x.abs().amax(-1) / 6.0)
    y = x.abs() / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)
    step = torch.where(y < 2.0, 0.5, torch.where(y < 4.0, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6.0)
    y = torch.where(scale.unsqueeze(-1) > 0, y, torch.zeros_like(y))
    code = torch.where(y < 2.0, 2.0 * y, torch.where(y < 4.0, y + 2.0, 0.5 * y + 4.0))
    code = code.to(torch.uint8) | ((x < 0) & (y > 0)).to(torch.uint8) * 8
    code = code.flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4),
            scale.float().to(torch.float8_e4m3fn).view(torch.uint8))


def fields(cache, d):
    """The cache's key codes, key scales, value codes and value scales, [nb, Hkv, groups, 16, .]."""
    a, b = 8 * d, d
    at = [0, a, a + b, 2 * a + b, 2 * a + 2 * b]
    return [cache[..., at[i]:at[i + 1]].unflatten(-1, (16, -1)) for i in range(4)]


def rotation_table(case, dev):
    """Cosines and sines of every position, from 64-bit angles."""
    n = case["rot"] // 2
    freq = 500000.0 ** (-torch.arange(n, dtype=torch.float64, device=dev) / n)
    angle = torch.arange(table_len(case), dtype=torch.float64, device=dev).unsqueeze(1) * freq
    return torch.stack((torch.cos(angle), torch.sin(angle)), 1).float()


def grid_positions(n, limit, dev):
    """Positions [3, n] of text, then frames of 16 x 16 tokens (time, height, width)."""
    i = torch.arange(n, device=dev)
    text = min(n, 64)
    j = (i - text).clamp(min=0)
    base = torch.where(i < text, i, text)
    live = (i >= text).long()
    pos = torch.stack((base + j // 256, base + live * (j // 16 % 16), base + live * (j % 16)))
    return pos.clamp(max=limit - 1).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    dtype = DTYPES[case["dtype"]]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "prefix":
        return prefix_state(case, normal, g, dev)
    state = {"case": case, "rope": rotation_table(case, dev), "axes": pair_axes(case)}
    if case["op"] == "rotate":
        B, N = case["B"], case["N"]
        # a projection's rows [B, N, heads of queries, keys and values]; keys with a few
        # strong channels
        rows = torch.empty(B, N, Hq + 2 * Hkv, d, dtype=dtype, device=dev)
        gain = torch.exp(0.5 * normal(Hq + 2 * Hkv, d))
        for b in range(B):
            for lo in range(0, N, 16384):
                n = min(16384, N - lo)
                rows[b, lo:lo + n] = (normal(n, Hq + 2 * Hkv, d) * gain).to(dtype)
        if case["layout"] == "rows":
            q, k = rows[:, :, :Hq].flatten(0, 1), rows[:, :, Hq:Hq + Hkv].flatten(0, 1)
        else:
            q, k = rows[:, :, :Hq].transpose(1, 2), rows[:, :, Hq:Hq + Hkv].transpose(1, 2)
        if case["axes"]:
            pos = grid_positions(N, table_len(case), dev).unsqueeze(1).repeat(1, B, 1)
        else:
            pos = torch.arange(N, device=dev, dtype=torch.int32).repeat(B, 1)
        if case["layout"] == "rows":
            pos = pos.flatten(-2)
        w = (1.0 + 0.2 * normal(2, d)).to(dtype) if case["norm"] else (None, None)
        state.update(q=q, k=k, pos=pos.contiguous(), wq=w[0], wk=w[1])
        return state
    T, bs, N = tokens_of(case), case["bs"], case["N"]
    rows = T + case["pad"]
    gain = torch.exp(0.5 * normal(Hkv, d))
    proj = normal(rows, Hq + 2 * Hkv, d)
    proj[:, Hq:Hq + Hkv] *= gain
    proj = proj.to(dtype)
    nb = blocks_of(T, bs) + 3
    at = torch.arange(rows, device=dev)
    ids = torch.randperm(nb, generator=g, device=dev)
    slots = torch.where(at < T, ids[(at // bs).clamp(max=nb - 1)] * bs + at % bs, -1).int()
    cache = torch.zeros(nb, Hkv, bs // 16, 18 * d, dtype=torch.uint8, device=dev)
    state.update(k=proj[:, Hq:Hq + Hkv], v=proj[:, Hq + Hkv:], slots=slots, cache=cache)
    if case["form"] == "rows":
        start = int(torch.randint(0, max(1, N - rows), (1,), generator=g, device=dev))
        pos = (start + at).clamp(max=N - 1).int()
        if case["axes"]:
            pos = torch.stack((pos, grid_positions(rows, N, dev)[1], grid_positions(rows, N, dev)[2]))
        state.update(q=proj[:, :Hq], pos=pos.contiguous())
        return state
    new = torch.tensor(new_tokens(case), dtype=torch.int32, device=dev)
    new = new[torch.randperm(case["B"], generator=g, device=dev)]
    lens = torch.randint(0, N, (case["B"],), generator=g, device=dev)
    lens = torch.minimum((lens + new).clamp(max=N), torch.full_like(lens, N)).int()
    lens = torch.maximum(lens, new)
    state.update(q=normal(case["B"], Hq, d).to(dtype), lens=lens,
                 cu=torch.cat((new.new_zeros(1), new.cumsum(0))).int())
    return state


def prefix_state(case, normal, g, dev):
    """Blocks of the prefix once, blocks of their own behind it, for every sequence."""
    B, Hq, Hkv, d, bs, P = (case[x] for x in ("B", "Hq", "Hkv", "d", "bs", "P"))
    lens = torch.tensor(lengths(case), dtype=torch.int32, device=dev)
    lens = lens[torch.randperm(B, generator=g, device=dev)]
    front = P // bs
    width = blocks_of(P + case["more"], bs)
    have = (lens + bs - 1) // bs
    col = torch.arange(width, device=dev)
    used = (col < have.unsqueeze(1)) & (col >= front)
    nb = front + sum(max(0, blocks_of(n, bs) - front) for n in lengths(case)) + 2
    ids = torch.randperm(nb, generator=g, device=dev).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    table[:, :front] = ids[:front]
    table[used] = ids[front:nb - 2]
    table[col >= have.unsqueeze(1)] = -1
    cache = torch.empty(nb, Hkv, bs // 16, 18 * d, dtype=torch.uint8, device=dev)
    parts = fields(cache, d)
    gain = torch.exp(0.5 * normal(Hkv, 1, 1, d))
    step = max(1, (1 << 27) // (Hkv * bs * d))
    for lo in range(0, nb, step):
        for i in (0, 2):
            x = normal(min(step, nb - lo), Hkv, bs // 16, 16, d)
            c, s = quantise((x * gain if i == 0 else x).bfloat16())
            parts[i][lo:lo + step], parts[i + 1][lo:lo + step] = c, s
    return {"case": case, "q": normal(B, Hq, d).to(DTYPES[case["dtype"]]), "cache": cache,
            "table": table, "lens": lens}


# ------------------------------------------------------------------- plain forms --

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def values(codes, scales):
    """Stored rows as 32-bit numbers."""
    lut = torch.tensor(E2M1, device=codes.device)
    x = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def angles(rope, pos, axes):
    """Cosines and sines [..., pairs] of positions pos [...], or [axes, ...]."""
    if axes is None:
        return rope[pos.long(), 0], rope[pos.long(), 1]
    at = pos.long()[torch.tensor(axes, device=pos.device)].movedim(0, -1)
    pair = torch.arange(len(axes), device=pos.device)
    return rope[at, 0, pair], rope[at, 1, pair]


def turned(x, cos, sin, weight, interleaved):
    """Rows x [..., d] in 32 bits: normalised where there is a weight, then turned."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    n = cos.shape[-1]
    head, rest = x[..., :2 * n], x[..., 2 * n:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
    else:
        a, b = head[..., :n], head[..., n:]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((head, rest), -1)


def rotate_plain(st):
    cos, sin = angles(st["rope"], st["pos"], st["axes"])
    cos, sin = (x.unsqueeze(-2 if st["q"].dim() == 3 else -3) for x in (cos, sin))
    flag = st["case"]["interleaved"]
    return {"q": turned(st["q"], cos, sin, st["wq"], flag).to(st["q"].dtype),
            "k": turned(st["k"], cos, sin, st["wk"], flag).to(st["k"].dtype)}


def append_plain(st):
    case, cache, k, v = st["case"], st["cache"], st["k"], st["v"]
    T, Hkv, d = k.shape
    bs = case["bs"]
    at = torch.arange(T, device=k.device)
    if case["form"] == "rows":
        kpos = qpos = st["pos"]
    else:
        lens, cu = st["lens"].long(), st["cu"].long()
        who = torch.searchsorted(cu, at, right=True).clamp(max=case["B"]) - 1
        kpos = lens[who] - cu[who + 1] + at
        kpos = torch.where(at < cu[-1], kpos, 0)     # behind the last token
        qpos = (lens - 1).clamp(min=0)
        if case["axes"]:                             # one position for all axes
            kpos, qpos = kpos.expand(3, -1), qpos.expand(3, -1)
    cos, sin = angles(st["rope"], kpos, st["axes"])
    k = turned(k, cos.unsqueeze(1), sin.unsqueeze(1), None, case["interleaved"])
    cos, sin = angles(st["rope"], qpos, st["axes"])
    q = turned(st["q"], cos.unsqueeze(1), sin.unsqueeze(1), None, case["interleaved"])
    parts = fields(cache, d)
    live = st["slots"] >= 0
    slot = st["slots"][live].long()
    block, row = slot // bs, slot % bs
    to = (block.view(-1, 1), torch.arange(Hkv, device=k.device), (row // 16).view(-1, 1),
          (row % 16).view(-1, 1))
    parts[0][to], parts[1][to] = quantise(k[live])
    parts[2][to], parts[3][to] = quantise(v[live])
    out_k, out_v = torch.zeros_like(v), torch.zeros_like(v)
    out_k[live] = values(parts[0][to], parts[1][to]).to(v.dtype)
    out_v[live] = values(parts[2][to], parts[3][to]).to(v.dtype)
    return {"q": q.to(st["q"].dtype), "k": out_k, "v": out_v}


def prefix_plain(st):
    """Scores against the prefix's rows, read once for all sequences, then each sequence's own."""
    case, q, table, lens = st["case"], st["q"], st["table"], st["lens"]
    B, Hq, d = q.shape
    Hkv, P, front = case["Hkv"], case["P"], case["P"] // case["bs"]
    G = Hq // Hkv
    shared = lens.clamp(max=P)
    ids = table.index_select(0, shared.argmax().view(1))[0, :front].clamp(min=0).long()
    kc, ks, vc, vs = (x[ids].transpose(0, 1).flatten(1, 3) for x in fields(st["cache"], d))
    qs = q.float().view(B, Hkv, G, d) * (1.0 / math.sqrt(d))
    s = torch.matmul(qs.transpose(0, 1).reshape(Hkv, B * G, d), values(kc, ks).transpose(1, 2))
    s = s.view(Hkv, B, G, P).transpose(0, 1)                       # [B, Hkv, G, P]
    live = torch.arange(P, device=q.device) < shared.view(B, 1, 1, 1)
    s = torch.where(live, s, -math.inf)
    # what lies behind the longest sequence's last token is not read
    v = torch.where(torch.arange(P, device=q.device).view(P, 1) < shared.max(), values(vc, vs), 0.0)
    rest = table[:, front:].clamp(min=0).long()
    own_rows = [x[rest].transpose(1, 2).flatten(2, 4) for x in fields(st["cache"], d)]
    t = torch.matmul(qs, values(own_rows[0], own_rows[1]).transpose(-1, -2))
    live = (torch.arange(t.shape[-1], device=q.device) + P) < lens.view(B, 1, 1, 1)
    t = torch.where(live, t, -math.inf)
    w = torch.where(live.transpose(-1, -2), values(own_rows[2], own_rows[3]), 0.0)
    m = torch.maximum(s.amax(-1, keepdim=True), t.amax(-1, keepdim=True))
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    s, t = torch.exp(s - m), torch.exp(t - m)
    total = s.sum(-1, keepdim=True) + t.sum(-1, keepdim=True)
    o = torch.matmul(s.transpose(0, 1).reshape(Hkv, B * G, P), v)
    o = o.view(Hkv, B, G, d).transpose(0, 1) + torch.matmul(t, w)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": o.reshape(B, Hq, d).to(q.dtype)}


# --------------------------------------------------------------------- one pass --

def run(state):
    case = state["case"]
    if not own:
        plain = {"rotate": rotate_plain, "append": append_plain, "prefix": prefix_plain}
        return plain[case["op"]](state)
    from long_context_anchor_gb300 import kascade as K
    if case["op"] == "rotate":
        q, k = K.qk_norm_rope(state["q"], state["k"], state["pos"], state["rope"],
                              q_weight=state["wq"], k_weight=state["wk"], eps=EPS,
                              interleaved=case["interleaved"], axes=state["axes"])
        return {"q": q, "k": k}
    if case["op"] == "append":
        at = ({"positions": state["pos"]} if case["form"] == "rows" else
              {"cu_new": state["cu"], "kv_lens": state["lens"]})
        q = K.qcache_append_rope(state["k"], state["v"], state["slots"], state["cache"],
                                 state["rope"], q=state["q"], interleaved=case["interleaved"],
                                 axes=state["axes"], **at)
        k, v = K.qcache_read(state["cache"], state["slots"], dtype=state["k"].dtype)
        return {"q": q, "k": k, "v": v}
    return {"out": K.qcache_prefix_decode(state["q"], state["cache"], state["table"],
                                          state["lens"], case["P"])}


# ------------------------------------------------------------------ definition --

def nearest(x, grid):
    """The nearest number of an ascending grid to each x >= 0 (its even-numbered one at a tie)."""
    hi = torch.searchsorted(grid, x).clamp(1, grid.numel() - 1)
    lo = hi - 1
    left, right = x - grid[lo], grid[hi] - x
    up = (right < left) | ((right == left) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def tables(dev):
    e2m1 = torch.tensor(E2M1[:8], dtype=torch.float64, device=dev)
    e4m3 = torch.tensor([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64,
                        device=dev)
    return e2m1, e4m3


def stored_exact(x):
    """What a row holds after it went into the cache: by search in the tables of e4m3 and e2m1."""
    e2m1, e4m3 = tables(x.device)
    x = x.double().reshape(*x.shape[:-1], -1, 16)
    s = e4m3[nearest((x.abs().max(-1).values / 6.0).contiguous(), e4m3)].unsqueeze(-1)
    y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    return (torch.sign(x) * e2m1[nearest(y, e2m1)] * s).flatten(-2)


def row_exact(cache, block, head, row, d):
    """Keys and values [n, d] of one KV head at (block, row) pairs, in 64 bits."""
    e2m1, e4m3 = tables(cache.device)
    e2m1, e4m3 = torch.cat((e2m1, -e2m1)), torch.cat((e4m3, e4m3.new_full((1,), math.nan)))
    rec = cache[block, head, row // 16]
    out = []
    for base in (0, 9 * d):
        byte = base + (row % 16 * (d // 2)).unsqueeze(1) + torch.arange(d, device=row.device) // 2
        code = rec.gather(1, byte) >> (torch.arange(d, device=row.device) % 2 * 4).to(torch.uint8)
        byte = base + 8 * d + (row % 16 * (d // 16)).unsqueeze(1)
        byte = byte + torch.arange(d, device=row.device) // 16
        out.append(e2m1[(code & 15).long()] * e4m3[(rec.gather(1, byte) & 127).long()])
    return out


def turned_exact(x, table, pos, axes, weight, interleaved):
    """Rows x [T, H, d] at positions pos [T] or [axes, T]: pairs as complex numbers times e^(i angle)."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    n = table.shape[2]
    turn = torch.complex(table[:, 0].double(), table[:, 1].double())          # [positions, pairs]
    if axes is None:
        turn = turn[pos.long()]
    else:
        turn = torch.stack([turn[pos[a].long(), i] for i, a in enumerate(axes)], -1)
    out = x.clone()
    i = torch.arange(n, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    z = torch.complex(x[..., a], x[..., b]) * turn.unsqueeze(1)
    out[..., a], out[..., b] = z.real, z.imag
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotate":
        pos, out = st["pos"], {}
        for name, weight in (("q", st["wq"]), ("k", st["wk"])):
            x = st[name]
            if x.dim() == 3:
                out[name] = turned_exact(x, st["rope"], pos, st["axes"], weight, case["interleaved"])
                continue
            out[name] = torch.stack([
                turned_exact(x[b].transpose(0, 1), st["rope"], pos[..., b, :], st["axes"], weight,
                             case["interleaved"]).transpose(0, 1) for b in range(x.shape[0])])
        return out
    if case["op"] == "append":
        T, axes = st["k"].shape[0], st["axes"]
        if case["form"] == "rows":
            kpos = qpos = st["pos"]
        else:
            lens, cu = st["lens"].tolist(), st["cu"].tolist()
            kpos = [lens[b] - cu[b + 1] + t for b in range(case["B"]) for t in range(cu[b], cu[b + 1])]
            kpos = torch.tensor(kpos + [0] * (T - len(kpos)), device=st["k"].device)
            qpos = torch.tensor([max(0, n - 1) for n in lens], device=st["k"].device)
            if axes is not None:
                kpos, qpos = kpos.expand(3, -1), qpos.expand(3, -1)
        live = (st["slots"] >= 0).view(-1, 1, 1)
        flag = case["interleaved"]
        return {"q": turned_exact(st["q"], st["rope"], qpos, axes, None, flag),
                "k": torch.where(live, stored_exact(turned_exact(st["k"], st["rope"], kpos, axes,
                                                                 None, flag)), 0.0),
                "v": torch.where(live, stored_exact(st["v"]), 0.0)}
    q, table, bs, d = st["q"].double(), st["table"].long(), case["bs"], case["d"]
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros_like(q)
    for b, n in enumerate(st["lens"].tolist()):
        pos = torch.arange(n, device=q.device)
        if n == 0:
            continue
        for g in range(case["Hkv"]):
            k, v = row_exact(st["cache"], table[b, pos // bs], g, pos % bs, d)
            s = q[b, g * G:(g + 1) * G] @ k.T / math.sqrt(d)
            out[b, g * G:(g + 1) * G] = torch.softmax(s, -1) @ v
    return {"out": out}
