"""Attention over long and shared caches as a serving program calls it: a pool
of 4-bit values (append with position rotation, gather, attention) and
attention of a batch whose sequences share prefixes, each as one pass (`run`),
in a plain form of elementary torch operations in 32 bits and, with `own`,
through the library's entry points.

4-bit rows. A row holds H heads' codes, two elements a byte (the even one in
the low half), and then one scale byte for every 16 elements. A code is a
sign, two bits of exponent and one of mantissa (0, .5, 1, 1.5, 2, 3, 4, 6); a
scale byte is the upper half, sign apart, of a 16-bit float: five bits of
exponent and three of mantissa.

Lengths follow from the case alone; everything else from the seed.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- the cases

def _case(name, op, cache, **more):
    base = dict(name=name, op=op, cache=cache, type="bf16", heads=8, q_heads=32, dim=128, page=16, layers=2, layer=1,
                seqs=1, len_lo=1, len_hi=1, new_lo=1, new_hi=1, axes=1, interleaved=False, rotary=128, lse=False,
                groups=0, prefix_lo=0, prefix_hi=0)
    base.update(more)
    return base


def listed():
    return [
        # one decode step of 256 conversations, a token each, into a 4-bit cache; the step's values are read out again
        _case("append decode 4-bit", "append", "4", seqs=256, len_lo=40, len_hi=128),
        # prompts of image and video tokens (time, height, width): 16 x 2048 rows into a 4-bit cache
        _case("append prompts 4-bit", "append", "4", type="fp16", page=64, seqs=16, len_lo=2048, len_hi=2048,
              new_lo=2048, new_hi=2048, axes=3),
        # the last 128 tokens of every conversation in 16 bits (for another device or a draft model)
        _case("gather windows 4-bit", "gather", "4", dim=64, page=32, seqs=512, len_lo=129, len_hi=999, new_lo=128,
              new_hi=128),
        # whole prefixes read out in 16 bits
        _case("gather prefixes 4-bit", "gather", "4", seqs=64, len_lo=1001, len_hi=8191, new_lo=1001, new_hi=8191),
        # the smallest attention call: one conversation, one token, a short context
        _case("attend one short 4-bit", "attend", "4", seqs=1, len_lo=203, len_hi=203),
        # decode of 256 conversations of 4096 tokens
        _case("attend decode 4-bit", "attend", "4", seqs=256, len_lo=4096, len_hi=4096),
        # drafted tokens checked over contexts from a few tokens to a long document
        _case("attend drafts 4-bit", "attend", "4", type="fp16", seqs=40, len_lo=9, len_hi=40961, new_lo=1, new_hi=4,
              lse=True),
        # prompt chunks over long contexts
        _case("attend chunks 4-bit", "attend", "4", page=32, seqs=4, len_lo=6001, len_hi=8190, new_lo=901,
              new_hi=1023),
        # four answers sampled from one short prompt
        _case("shared one prompt", "shared", "16", seqs=4, groups=1, prefix_lo=608, prefix_hi=608, len_lo=5,
              len_hi=61),
        # decode of 256 conversations behind one long system prompt
        _case("shared decode bf16", "shared", "16", seqs=256, groups=1, prefix_lo=8192, prefix_hi=8192, len_lo=1,
              len_hi=512),
        # questions about 24 documents, one to nine readers each, with drafted tokens, 8-bit cache
        _case("shared documents e4m3", "shared", "e4m3", type="fp16", page=32, seqs=150, groups=24, prefix_lo=1001,
              prefix_hi=16001, len_lo=4, len_hi=700, new_lo=1, new_hi=4, lse=True),
        # four system prompts of 128 conversations in a 4-bit cache
        _case("shared decode 4-bit", "shared", "4", seqs=128, groups=4, prefix_lo=2048, prefix_hi=6144, len_lo=9,
              len_hi=900),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(("append", "append", "gather", "attend", "attend", "shared", "shared", "shared"))
    cache = rng.choice(("16", "e4m3", "4")) if op == "shared" else "4"
    heads = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 128))
    c = dict(op=op, cache=cache, type=rng.choice(("bf16", "fp16")), heads=heads,
             q_heads=heads * rng.choice((1, 2, 3, 4, 5, 8)), dim=dim, page=rng.choice((4, 16, 32, 64)), layers=2,
             layer=rng.randrange(2), axes=1, interleaved=rng.random() < 0.4, rotary=dim, lse=False, groups=0,
             prefix_lo=0, prefix_hi=0)
    if op == "append":
        c["rotary"] = rng.choice((dim // 2, dim))
        c["axes"] = rng.choice((1, 1, 2, 3))
        if rng.random() < 0.5:
            c.update(seqs=_log(rng, 1, 512), new_lo=1, new_hi=rng.choice((1, 5)))
        else:
            c.update(seqs=rng.randint(1, 12), new_lo=_log(rng, 65, 300), new_hi=_log(rng, 301, 2048))
        c.update(len_lo=c["new_hi"], len_hi=c["new_hi"] + _log(rng, 1, 300))
    elif op == "gather":
        c.update(seqs=_log(rng, 1, 128), new_lo=1, new_hi=_log(rng, 2, 4000))
        c.update(len_lo=c["new_hi"], len_hi=c["new_hi"] + _log(rng, 1, 1000))
    elif op == "attend":
        if rng.random() < 0.65:  # single tokens and drafts
            seqs = _log(rng, 1, 256)
            c.update(seqs=seqs, new_lo=1, new_hi=rng.choice((1, 1, 4, 7)))
            c.update(len_lo=c["new_hi"], len_hi=c["new_hi"] + _log(rng, 8, min(60000, 500000 // seqs)))
        else:  # prompts and chunks
            c.update(seqs=rng.randint(1, 6), new_lo=_log(rng, 30, 300), new_hi=_log(rng, 301, 1500))
            c.update(len_lo=c["new_hi"], len_hi=c["new_hi"] + _log(rng, 1, 4000))
        c["lse"] = rng.random() < 0.3
    else:
        seqs = _log(rng, 2, 256)
        most = min(16000, 1200000 // seqs)
        c.update(seqs=seqs, groups=_log(rng, 1, min(32, seqs)), new_lo=1, new_hi=rng.choice((1, 1, 4, 9)))
        c.update(prefix_lo=_log(rng, 40, most // 2), prefix_hi=_log(rng, most // 2, most))
        c.update(len_lo=c["new_hi"], len_hi=c["new_hi"] + _log(rng, 1, min(2000, most)))
        c["lse"] = rng.random() < 0.3
    while c["seqs"] > 1 and _cost(c) > LIMIT:
        c["seqs"] = (c["seqs"] + 1) // 2
        c["groups"] = min(c["groups"], c["seqs"])
    return c


LIMIT = 2e9  # bytes, or operations / 50, of a drawn case: below the largest listed one


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _spread(n, lo, hi, salt):
    """n whole numbers over [lo, hi], the ends among them when n > 1."""
    if n == 1:
        return [hi]
    v = [lo + (s * 2654435761 + salt * 40503) % (1 << 32) * (hi - lo + 1) // (1 << 32) for s in range(n)]
    v[0], v[-1] = lo, hi
    return v


def _groups(c):
    """First sequence of each group and its prefix in tokens (whole pages), and each sequence's prefix."""
    S, n = c["seqs"], c["groups"]
    if not n:
        return [], [], [0] * S
    cuts = sorted(set(_spread(n, 0, S - 1, 3)) | {0})
    pre = [max(1, p // c["page"]) * c["page"] for p in _spread(len(cuts), c["prefix_lo"], c["prefix_hi"], 4)]
    return cuts, pre, [pre[sum(x <= s for x in cuts) - 1] for s in range(S)]


def _lengths(c):
    """(tokens, new tokens) of each sequence, prefixes included."""
    n = _spread(c["seqs"], c["len_lo"], c["len_hi"], 1)
    new = _spread(c["seqs"], c["new_lo"], c["new_hi"], 2)
    new = [min(a, b) for a, b in zip(n, new)]
    return [a + p for a, p in zip(n, _groups(c)[2])], new


def _row_bytes(c):
    """Bytes of a token's K (or V) of one layer, and of them those of one head."""
    D = c["dim"]
    head = D * 2 if c["cache"] == "16" else D if c["cache"] == "e4m3" else D // 2 + D // 16
    return -(-c["heads"] * head // 16) * 16, head


def work(case):
    c = case
    n, new = _lengths(c)
    rows, D, H, Q = sum(new), c["dim"], c["heads"], c["q_heads"]
    head = _row_bytes(c)[1]
    if c["op"] == "append":  # rows in, codes and queries out, and the codes read out as 16-bit values
        return {"bytes": rows * (2 * H * (D * 2 + head) + 2 * Q * D * 2 + 2 * H * (head + D * 2)) + rows * 8 * c["axes"],
                "flops": 3 * rows * D * (H + Q)}
    if c["op"] == "gather":
        return {"bytes": rows * 2 * H * (head + 2 * D), "flops": rows * D * 2 * H}
    cuts, pre, each = _groups(c)
    keys = sum(pre) + sum(a - p for a, p in zip(n, each))
    pairs = sum(b * (a - b) + b * (b + 1) // 2 for a, b in zip(n, new))
    return {"bytes": keys * 2 * H * head + rows * D * Q * 4, "flops": 4 * D * Q * pairs}


# ------------------------------------------------------------- what is in hand

def _rows(state):
    """Sequence and token index of every row."""
    r = torch.arange(state["n_rows"], device="cuda")
    s = torch.searchsorted(state["cu"][1:].contiguous(), r, right=True)
    return s, state["start"][s].long() + r - state["cu"][s]


def _scale_bytes(amax):
    """The scale byte of blocks whose largest magnitude is amax: a sixth of it in 16 bits, then its upper 8 bits."""
    h = (amax * torch.tensor(1 / 6, dtype=torch.float32, device=amax.device)).clamp(max=8192.0).half()
    b = h.view(torch.int16).int()
    return (b + 63 + (b >> 7 & 1)) >> 7


def _scale_of(byte):
    return (byte.int() << 7).short().view(torch.float16).float()


def _encode(x):
    """x [..., D] in 32 bits -> code bytes [..., D / 2] and scale bytes [..., D / 16]."""
    b = x.unflatten(-1, (-1, 16))
    s = _scale_bytes(b.abs().amax(-1))
    S = _scale_of(s)
    inv = torch.where(S > 0, 1.0 / S, 0.0)
    y = b * inv[..., None]
    m = y.abs()
    # a value next to a border goes to the code whose last bit is 0
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int()
            + (m >= 3.5).int() + (m > 5.0).int())
    code = (code | torch.signbit(y).int() << 3).flatten(-2)
    return (code[..., 0::2] | code[..., 1::2] << 4).byte(), s.byte()


def _decode(codes, scales):
    """Code bytes [..., D / 2] and scale bytes [..., D / 16] -> values in 32 bits."""
    table = torch.tensor(CODES + tuple(-v for v in CODES), device=codes.device)
    x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return (table[x].unflatten(-1, (-1, 16)) * _scale_of(scales)[..., None]).flatten(-2)


def _split(c, raw):
    """Bytes of the pool -> code bytes [..., H, D / 2] and scale bytes [..., H, D / 16] of every row."""
    H, D = c["heads"], c["dim"]
    rows = raw.view(-1, _row_bytes(c)[0])
    return rows[:, :H * D // 2].unflatten(-1, (H, D // 2)), \
        rows[:, H * D // 2:H * D // 2 + H * D // 16].unflatten(-1, (H, D // 16))


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    n, new = _lengths(c)
    D, H, Q, ps, L = c["dim"], c["heads"], c["q_heads"], c["page"], c["layers"]
    t = TYPES[c["type"]]
    cuts, pre, each = _groups(c)
    tails = [-(-a // ps) - p // ps for a, p in zip(n, each)]  # a sequence's own pages
    heads = [p // ps for p in pre]
    P = sum(tails) + sum(heads) + 1  # page 0 is the sink
    order = (torch.randperm(P - 1, generator=g, device="cuda") + 1).cpu().int()
    table = torch.full((c["seqs"], max(-(-a // ps) for a in n)), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(heads):
        end = cuts[i + 1] if i + 1 < len(cuts) else c["seqs"]
        table[cuts[i]:end, :k] = order[at:at + k]
        at += k
    for s in range(c["seqs"]):
        table[s, each[s] // ps:each[s] // ps + tails[s]] = order[at:at + tails[s]]
        at += tails[s]
    row = _row_bytes(c)[0]
    rows = (P + 1) * 2 * L * ps  # the last page's worth is the tail pad
    st = {"case": c, "n_rows": sum(new), "table": table.cuda(),
          "len": torch.tensor(n, dtype=torch.int32, device="cuda"),
          "start": torch.tensor([a - b for a, b in zip(n, new)], dtype=torch.int32, device="cuda"),
          "cu": torch.tensor([0] + new, device="cuda").cumsum(0), "max_len": max(n), "max_new": max(new)}
    if c["cache"] == "16":
        st["raw"] = normal(rows * H * D, dtype=t).view(torch.uint8)
    elif c["cache"] == "e4m3":
        raw = torch.empty(rows * H * D, dtype=torch.float8_e4m3fn, device="cuda")
        raw.copy_(normal(rows * H * D, dtype=torch.float16).mul_(100).clamp_(-448, 448))
        st["raw"] = raw.view(torch.uint8)
        # powers of two, as an append leaves them
        e = torch.randint(-8, -5, (P, L, 2, H), generator=g, device="cuda")
        st["scales"] = ((e + 127) << 23).int().view(torch.float32)
    else:
        st["raw"] = torch.zeros(rows * row, dtype=torch.uint8, device="cuda")
        codes, scales = _split(c, st["raw"])
        for a in range(0, rows, 1 << 17):  # normal values as an append leaves them
            b = min(rows, a + (1 << 17))
            codes[a:b], scales[a:b] = _encode(normal(b - a, H, D))
    if c["op"] == "append":
        st["k"], st["v"] = normal(st["n_rows"], H, D, dtype=t), normal(st["n_rows"], H, D, dtype=t)
        st["q"] = normal(st["n_rows"], Q, D, dtype=t)
        rd = c["rotary"]
        s, j = _rows(st)
        if c["axes"] == 1:
            pos = j[None]
        else:  # frames of 24 x 36 patches
            pos = torch.stack([j // 864, j // 36 % 24, j % 36][: c["axes"]])
        st["pos"] = pos.int().contiguous()
        freq = 10000.0 ** (-torch.arange(rd // 2, dtype=torch.float64, device="cuda") * 2 / rd)
        ang = torch.arange(max(n), dtype=torch.float64, device="cuda")[:, None] * freq
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["axis_pairs"] = _axis_pairs(c)
    elif c["op"] != "gather":
        st["q"] = normal(st["n_rows"], Q, D, dtype=t)
        st["scale"] = D ** -0.5
    if c["op"] == "shared":
        st["group"] = torch.tensor(cuts + [c["seqs"]], dtype=torch.int32, device="cuda")
        st["prefix"] = torch.tensor(pre, dtype=torch.int32, device="cuda")
    if own:
        _prepare_own(st)
    return st


def _axis_pairs(c):
    half, a = c["rotary"] // 2, c["axes"]
    first = half - (a - 1) * (3 * half // 8)  # as image models split it: 16, 24, 24 of 64
    return [first] + [3 * half // 8] * (a - 1)


def _prepare_own(st):
    """The pool's handle, the batch's descriptors and the buffers that calls write to."""
    import gather_translate_kv_gb300 as gt

    c = st["case"]
    H, D, Q, n = c["heads"], c["dim"], c["q_heads"], st["n_rows"]
    P = st["raw"].numel() // (2 * c["layers"] * c["page"] * _row_bytes(c)[0]) - 1  # the last is the tail pad
    more = {"format": gt.KV_FORMAT_E2M1} if c["cache"] == "4" else {}
    desc = gt.make_desc(c["layers"], H, D, 2 if c["cache"] == "16" else 1, c["page"], P, **more)
    st["pool"] = gt.kv_pool_create(desc, st["raw"])
    st["batch"] = gt.kv_batch(st["table"], st["len"], st["cu"], n, seq_start=st["start"])
    if c["op"] == "append":
        st["rot"] = gt.kv_rotary(st["cos_sin"], positions=st["pos"], axis_pairs=st["axis_pairs"],
                                 interleaved=c["interleaved"])
        st["q_out"] = torch.empty_like(st["q"])
    if c["op"] in ("append", "gather"):
        st["out_k"] = torch.empty(n, H, D, dtype=TYPES[c["type"]], device="cuda")
        st["out_v"] = torch.empty_like(st["out_k"])
        return
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(n, Q, device="cuda") if c["lse"] else None
    if c["op"] == "shared":
        st["groups"] = gt.kv_prefix_groups(st["group"], st["prefix"])
        size = gt.kv_attend_shared_workspace_bytes(st["pool"], Q, c["seqs"], n)
    else:
        size = gt.kv_attend_workspace_bytes(st["pool"], Q, c["seqs"], n)
    st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")


# -------------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import gather_translate_kv_gb300 as gt

    c = st["case"]
    if c["op"] == "append":
        gt.kv_append_layer(st["pool"], c["layer"], st["batch"], st["k"], st["v"], rotary=st["rot"], q=st["q"],
                           q_out=st["q_out"])
    if c["op"] in ("append", "gather"):
        gt.kv_gather_layer_scaled(st["pool"], c["layer"], st["batch"], None, st["out_k"], st["out_v"])
        out = {"k": st["out_k"], "v": st["out_v"]}
        return {"q": st["q_out"], **out} if c["op"] == "append" else out
    if c["op"] == "shared":
        gt.kv_attend_shared_layer(st["pool"], c["layer"], st["batch"], st["groups"], st["q"], st["out"], st["scale"],
                                  st["workspace"], scales=st.get("scales"), lse=st["lse"])
    else:
        gt.kv_attend_layer(st["pool"], c["layer"], st["batch"], st["q"], st["out"], st["scale"], st["workspace"],
                           lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]} if c["lse"] else {"out": st["out"]}


def _cached(st, which, page, off):
    """K (0) or V (1) of the layer at (page, offset), [..., heads, dim] in 32 bits."""
    c = st["case"]
    row = (page * 2 * c["layers"] + 2 * c["layer"] + which) * c["page"] + off
    if c["cache"] == "4":
        codes, scales = _split(c, st["raw"])
        return _decode(codes[row], scales[row])
    if c["cache"] == "16":
        return st["raw"].view(TYPES[c["type"]]).view(-1, c["heads"], c["dim"])[row].float()
    x = st["raw"].view(-1, c["heads"], c["dim"])[row].view(torch.float8_e4m3fn).float()
    return x.mul_(st["scales"][page, c["layer"], which][..., None])


def _rotate(x, st):
    """x [rows, heads, dim] in 32 bits, turned pair by pair."""
    c = st["case"]
    rd = c["rotary"]
    axis = torch.repeat_interleave(torch.arange(c["axes"], device="cuda"),
                                   torch.tensor(st["axis_pairs"], device="cuda"), output_size=rd // 2)
    p = st["pos"].long()[axis].T  # [rows, pairs]
    f = torch.arange(rd // 2, device="cuda")
    cos, sin = st["cos_sin"][p, f][:, None], st["cos_sin"][p, f + rd // 2][:, None]
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rd // 2], x[..., rd // 2: rd]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rd:]], -1)


def _run_plain(st):
    c = st["case"]
    if c["op"] in ("attend", "shared"):
        return _attend_plain(st)
    s, j = _rows(st)
    page, off = st["table"][s, j // c["page"]].long(), j % c["page"]
    out = {}
    if c["op"] == "append":
        codes, scales = _split(c, st["raw"])
        for which, x in ((0, _rotate(st["k"], st)), (1, st["v"].float())):
            row = (page * 2 * c["layers"] + 2 * c["layer"] + which) * c["page"] + off
            codes[row], scales[row] = _encode(x)
        out["q"] = _rotate(st["q"], st).to(st["q"].dtype)
    out["k"], out["v"] = (_cached(st, w, page, off).to(TYPES[c["type"]]) for w in (0, 1))
    return out


def _attend_plain(st):
    c = st["case"]
    S, n, m, H, D = c["seqs"], st["max_len"], st["max_new"], c["heads"], c["dim"]
    j = torch.arange(n, device="cuda")
    s, i = _rows(st)
    t = i - st["start"][s]
    q = torch.zeros(S, m, H, c["q_heads"] // H, D, device="cuda")
    q[s, t] = st["q"].float().view(-1, H, c["q_heads"] // H, D)
    q = q.permute(0, 2, 3, 1, 4).reshape(S, H, -1, D)
    y = torch.empty(S, H, q.shape[2], D, device="cuda")
    e = torch.empty(S, H, q.shape[2], device="cuda")
    step = max(1, int(4e8 // (n * H * D)))  # sequences at once
    for a in range(0, S, step):
        b = min(S, a + step)
        page = st["table"][a:b, j // c["page"]].clamp(min=0).long()
        off = (j % c["page"]).expand(b - a, n)
        x = torch.matmul(q[a:b], _cached(st, 0, page, off).permute(0, 2, 3, 1)).view(b - a, H, -1, m, n)
        x *= st["scale"]
        at = st["start"][a:b].long()[:, None] + torch.arange(m, device="cuda")
        seen = (j <= at[..., None]) & (j < st["len"][a:b, None, None])
        x.masked_fill_(~seen[:, None, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        x -= top
        x.exp_()
        total = x.sum(-1, keepdim=True)
        V = _cached(st, 1, page, off)
        V *= (j < st["len"][a:b, None])[..., None, None]
        y[a:b] = torch.matmul(x.view(b - a, H, -1, n), V.permute(0, 2, 1, 3)) / total.view(b - a, H, -1, 1)
        e[a:b] = (top + total.log()).view(b - a, H, -1)
    y = y.view(S, H, -1, m, D).permute(0, 3, 1, 2, 4)[s, t]
    out = {"out": y.reshape(-1, c["q_heads"], D).to(st["q"].dtype)}
    if c["lse"]:
        out["lse"] = e.view(S, H, -1, m).permute(0, 3, 1, 2)[s, t].reshape(-1, c["q_heads"])
    return out


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c = case
    st = prepare(c, seed)
    n, new = _lengths(c)
    L, l, ps, H, D, Q = c["layers"], c["layer"], c["page"], c["heads"], c["dim"], c["q_heads"]
    table = st["table"].cpu()
    row = _row_bytes(c)[0]
    if c["cache"] == "4":
        pool = st["raw"].view(-1, 2 * L, ps, row)
        steps = torch.tensor(CODES, dtype=torch.float64, device="cuda")
    else:
        kind = TYPES[c["type"]] if c["cache"] == "16" else torch.uint8
        pool = st["raw"].view(kind).view(-1, 2 * L, ps, H, D)

    def power(e):
        """2^e, exactly."""
        return (e.long() + 1023 << 52).view(torch.float64)

    def held(s, a, b, which):
        """Tokens [a, b) of sequence s in the cache, K (0) or V (1), as [b - a, H, D]."""
        p = table[s, a // ps: -(-b // ps)].long().cuda()
        x = pool[p, 2 * l + which].flatten(0, 1)[a - a // ps * ps:][: b - a]
        if c["cache"] == "16":
            return x.double()
        if c["cache"] == "e4m3":
            f = st["scales"][p, l, which].double().repeat_interleave(ps, 0)[a - a // ps * ps:][: b - a]
            return x.view(torch.float8_e4m3fn).double() * f[..., None]
        byte = x[:, :H * D // 2].long()
        y = torch.empty(len(x), H * D, dtype=torch.float64, device="cuda")
        for half in (0, 1):
            code = byte >> 4 * half & 15
            y[:, half::2] = steps[code & 7] * (1 - 2 * (code >> 3))
        f = x[:, H * D // 2: H * D // 2 + H * D // 16].long()
        e, frac = f >> 3, (f & 7).double() / 8
        f = torch.where(e > 0, (1 + frac) * power(e - 15), frac * 2.0 ** -14)
        return (y.view(len(x), -1, 16) * f[..., None]).view(-1, H, D)

    def turned(x):
        half = c["rotary"] // 2
        y = x.double().clone()
        f = 0
        for a, count in enumerate(st["axis_pairs"]):
            for _ in range(count):
                cs_sn = st["cos_sin"].double()[st["pos"][a].long()]
                cs, sn = cs_sn[:, f, None], cs_sn[:, half + f, None]
                i1, i2 = (2 * f, 2 * f + 1) if c["interleaved"] else (f, f + half)
                u, w = x[..., i1].double(), x[..., i2].double()
                y[..., i1], y[..., i2] = u * cs - w * sn, w * cs + u * sn
                f += 1
        return y

    if c["op"] == "gather":
        return {name: torch.cat([held(s, n[s] - new[s], n[s], w) for s in range(c["seqs"])]) for w, name in
                ((0, "k"), (1, "v"))}
    if c["op"] == "append":  # (keys: a rotation's last bit decides between two codes)
        x = st["v"].view(-1, H, D // 16, 16).double()
        sixth = float(torch.tensor(1 / 6, dtype=torch.float32))
        h = (x.abs().amax(-1) * sixth).float().clamp(max=8192.0).half().double()
        ulp = power(torch.frexp(h.clamp(min=2.0 ** -14)).exponent - 4)
        S = (h / ulp).round() * ulp
        y = (x * torch.where(S > 0, 1 / S, 0.0).float().double()[..., None]).float().double()
        step = power(torch.frexp(y.abs().clamp(min=1.0)).exponent - 2)  # 1/2, from 2 on 1, from 4 on 2
        y = ((y / step).round() * step).clamp(-6, 6) * S[..., None]
        return {"q": turned(st["q"]), "k": None, "v": y.view(-1, H, D)}
    outs, lses, at = [], [], 0
    for s in range(c["seqs"]):
        q = st["q"][at: at + new[s]].double().view(new[s], H, Q // H, D)
        at += new[s]
        K, V = held(s, 0, n[s], 0), held(s, 0, n[s], 1)
        i = torch.arange(n[s] - new[s], n[s], device="cuda")[:, None]
        seen = torch.arange(n[s], device="cuda")[None] <= i
        y = torch.empty(new[s], H, Q // H, D, dtype=torch.float64, device="cuda")
        e = torch.empty(new[s], H, Q // H, dtype=torch.float64, device="cuda")
        for h in range(H):
            x = torch.einsum("tgd,nd->tgn", q[:, h], K[:, h]) * st["scale"]
            x = x.masked_fill(~seen[:, None], -math.inf)
            y[:, h] = torch.einsum("tgn,nd->tgd", torch.softmax(x, -1), V[:, h])
            e[:, h] = torch.logsumexp(x, -1)
        outs.append(y.view(new[s], Q, D))
        lses.append(e.view(new[s], Q))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)} if c["lse"] else {"out": torch.cat(outs)}
