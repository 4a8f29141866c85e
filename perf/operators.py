"""The cache operators as a serving program calls them: append with position
rotation, attention over the pages, and the scaled gather, each as one pass
(`run`), in a plain form of elementary torch operations in 32 bits and, with
`own`, through the library's entry points.

A batch is a set of sequences over one page-major pool: sequence s holds
`len` tokens through its block table, the last `new` of them are this pass's
rows. Lengths follow from the case alone; everything else from the seed.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- the cases

def _case(name, op, cache, **more):
    base = dict(name=name, op=op, cache=cache, type="bf16", heads=8, q_heads=32, dim=128, page=16, layers=2, layer=1,
                seqs=1, len_lo=1, len_hi=1, new_lo=1, new_hi=1, window=0, sinks=0, axes=1, interleaved=False,
                rotary=128, lse=False)
    base.update(more)
    return base


def listed():
    return [
        # one decode step of 256 conversations: a token each, rotated and appended with its queries
        _case("append decode bf16", "append", "16", seqs=256, len_lo=40, len_hi=128),
        # prompts of image and video tokens: positions in time, height and width, 16 x 2048 rows
        _case("append prompts 3 axes", "append", "16", page=64, seqs=16, len_lo=2048, len_hi=2048, new_lo=2048,
              new_hi=2048, axes=3),
        # a decode step of a sliding-window model with an 8-bit cache
        _case("append decode e4m3", "append", "e4m3", dim=64, rotary=64, page=32, seqs=512, len_lo=33, len_hi=255),
        # chunks of prompts appended to an 8-bit cache from the middle of a page on
        _case("append chunks e4m3", "append", "e4m3", type="fp16", interleaved=True, seqs=12, len_lo=1203,
              len_hi=3301, new_lo=1001, new_hi=1201),
        # the smallest call: one conversation, one token, a short context
        _case("attend one short", "attend", "16", seqs=1, len_lo=203, len_hi=203),
        # decode of 256 conversations of 4096 tokens
        _case("attend decode bf16", "attend", "16", seqs=256, len_lo=4096, len_hi=4096),
        # drafted tokens checked over contexts from a few tokens to a long document, 8-bit cache
        _case("attend drafts e4m3", "attend", "e4m3", seqs=40, len_lo=9, len_hi=40961, new_lo=1, new_hi=4, lse=True),
        # decode of a sliding-window model: 128 tokens and the first 4 stay visible
        _case("attend window e4m3", "attend", "e4m3", type="fp16", dim=64, page=32, seqs=512, len_lo=57, len_hi=1999,
              window=128, sinks=4),
        # whole prompts: 16 x 2048 tokens
        _case("attend prompts bf16", "attend", "16", page=64, seqs=16, len_lo=2048, len_hi=2048, new_lo=2048,
              new_hi=2048),
        # prompt chunks over long contexts, 8-bit cache
        _case("attend chunks e4m3", "attend", "e4m3", page=32, seqs=4, len_lo=6001, len_hi=8190, new_lo=901,
              new_hi=1023),
        # the visible window of every conversation in 16 bits (another device's or a draft model's copy)
        _case("gather windows e4m3", "gather", "e4m3", dim=64, page=32, seqs=512, len_lo=129, len_hi=999, new_lo=128,
              new_hi=128),
        # whole prefixes read out in 16 bits
        _case("gather prefixes e4m3", "gather", "e4m3", seqs=64, len_lo=1001, len_hi=8191, new_lo=1001, new_hi=8191),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(("append", "append", "attend", "attend", "attend", "gather"))
    cache = "e4m3" if op == "gather" else rng.choice(("16", "e4m3"))
    heads = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 128))
    c = dict(op=op, cache=cache, type=rng.choice(("bf16", "fp16")), heads=heads,
             q_heads=heads * rng.choice((1, 2, 3, 4, 5, 8)), dim=dim, page=rng.choice((4, 16, 32, 64)), layers=2,
             layer=rng.randrange(2), window=0, sinks=0, axes=1, interleaved=rng.random() < 0.4, rotary=dim, lse=False)
    if op == "append":
        c["rotary"] = rng.choice((dim // 2, dim))
        c["axes"] = rng.choice((1, 1, 2, 3))
        if rng.random() < 0.5:
            c.update(seqs=_log(rng, 1, 512), new_lo=1, new_hi=rng.choice((1, 5)))
        else:
            c.update(seqs=rng.randint(1, 12), new_lo=_log(rng, 65, 300), new_hi=_log(rng, 301, 2048))
        c.update(len_lo=c["new_hi"], len_hi=c["new_hi"] + _log(rng, 1, 300))
    elif op == "attend":
        if rng.random() < 0.65:  # single tokens and drafts
            seqs = _log(rng, 1, 256)
            c.update(seqs=seqs, new_lo=1, new_hi=rng.choice((1, 1, 4, 7)))
            c.update(len_lo=c["new_hi"], len_hi=c["new_hi"] + _log(rng, 8, min(60000, 500000 // seqs)))
        else:  # prompts and chunks
            c.update(seqs=rng.randint(1, 6), new_lo=_log(rng, 30, 300), new_hi=_log(rng, 301, 1500))
            c.update(len_lo=c["new_hi"], len_hi=c["new_hi"] + _log(rng, 1, 4000))
        if rng.random() < 0.4:
            c.update(window=_log(rng, 5, 2000), sinks=rng.choice((0, 1, 4, 19, 70)))
        c["lse"] = rng.random() < 0.3
    else:
        c.update(seqs=_log(rng, 1, 128), new_lo=1, new_hi=_log(rng, 2, 4000))
        c.update(len_lo=c["new_hi"], len_hi=c["new_hi"] + _log(rng, 1, 1000))
    while c["seqs"] > 1 and _cost(c) > LIMIT:
        c["seqs"] = (c["seqs"] + 1) // 2
    return c


LIMIT = 9e9  # bytes, or operations / 50, of a drawn case: below the largest listed one


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


def _lengths(c):
    """(tokens, new tokens) of each sequence."""
    n = _spread(c["seqs"], c["len_lo"], c["len_hi"], 1)
    new = _spread(c["seqs"], c["new_lo"], c["new_hi"], 2)
    return n, [min(a, b) for a, b in zip(n, new)]


def work(case):
    c = case
    n, new = _lengths(c)
    rows, D, H, Q, ps = sum(new), c["dim"], c["heads"], c["q_heads"], c["page"]
    it = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "append":
        nbytes = rows * D * (2 * H * (2 + it) + 2 * Q * 2) + rows * 8 * c["axes"]
        if it == 1:  # the touched pages are read out again: codes in, 16-bit values out
            back = sum(a - (a - b) // ps * ps for a, b in zip(n, new))
            nbytes += back * D * 2 * H * (1 + 2)
        return {"bytes": nbytes, "flops": 3 * rows * D * (H + Q)}
    if c["op"] == "gather":
        return {"bytes": rows * D * 2 * H * (it + 2), "flops": rows * D * 2 * H}
    keys = pairs = 0
    for a, b in zip(n, new):
        W = c["window"] or a
        lo = max(0, a - b - W + 1)  # first token of the first row's window
        keys += a - lo + min(c["sinks"], lo)
        for i in range(a - b, a):
            w = max(0, i - W + 1)
            pairs += i - w + 1 + min(c["sinks"], w)
    return {"bytes": keys * D * 2 * H * it + rows * D * Q * 4, "flops": 4 * D * Q * pairs}


# ------------------------------------------------------------- what is in hand

def _rows(state):
    """Sequence and token index of every row."""
    r = torch.arange(state["n_rows"], device="cuda")
    s = torch.searchsorted(state["cu"][1:].contiguous(), r, right=True)
    return s, state["start"][s].long() + r - state["cu"][s]


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    n, new = _lengths(c)
    D, H, Q, ps, L = c["dim"], c["heads"], c["q_heads"], c["page"], c["layers"]
    t = TYPES[c["type"]]
    pages = [-(-a // ps) for a in n]
    P = sum(pages) + 1  # page 0 is the sink
    order = torch.randperm(P - 1, generator=g, device="cuda") + 1
    table = torch.full((c["seqs"], max(pages)), -1, dtype=torch.int32)
    at = torch.tensor([0] + pages).cumsum(0)
    order = order.cpu()
    for s in range(c["seqs"]):
        table[s, :pages[s]] = order[at[s]:at[s + 1]].int()
    it = 1 if c["cache"] == "e4m3" else 2
    total = P * 2 * L * ps * H * D
    pad = 2 * L * ps * H * D
    st = {"case": c, "n_rows": sum(new), "table": table.cuda(),
          "len": torch.tensor(n, dtype=torch.int32, device="cuda"),
          "start": torch.tensor([a - b for a, b in zip(n, new)], dtype=torch.int32, device="cuda"),
          "cu": torch.tensor([0] + new, device="cuda").cumsum(0), "max_len": max(n), "max_new": max(new)}
    if it == 2:
        raw = normal(total + pad, dtype=t)
        st["values"] = raw
        st["raw"] = raw.view(torch.uint8)
    else:
        raw = torch.empty(total + pad, dtype=torch.float8_e4m3fn, device="cuda")
        raw.copy_(normal(total + pad, dtype=torch.float16).mul_(100).clamp_(-448, 448))
        st["raw"] = raw.view(torch.uint8)
        # powers of two, as an append leaves them
        e = torch.randint(-8, -5, (P, L, 2, H), generator=g, device="cuda")
        st["scales"] = ((e + 127) << 23).int().view(torch.float32)
    if c["op"] == "append":
        st["k"], st["v"] = normal(st["n_rows"], H, D, dtype=t), normal(st["n_rows"], H, D, dtype=t)
        st["q"] = normal(st["n_rows"], Q, D, dtype=t)
        rd = c["rotary"]
        if c["axes"] == 1:
            s, j = _rows(st)
            pos = j[None]
        else:  # frames of 24 x 36 patches
            s, j = _rows(st)
            pos = torch.stack([j // 864, j // 36 % 24, j % 36][: c["axes"]])
        st["pos"] = pos.int().contiguous()
        freq = 10000.0 ** (-torch.arange(rd // 2, dtype=torch.float64, device="cuda") * 2 / rd)
        ang = torch.arange(max(n), dtype=torch.float64, device="cuda")[:, None] * freq
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["axis_pairs"] = _axis_pairs(c)
        if it == 1:  # the read-out starts with the first touched page
            st["read_start"] = (st["start"] // ps * ps).int()
            st["read_cu"] = torch.cat([st["cu"][:1], (st["len"] - st["read_start"]).long().cumsum(0)])
            st["read_rows"] = int(st["read_cu"][-1])
    elif c["op"] == "attend":
        st["q"] = normal(st["n_rows"], Q, D, dtype=t)
        st["scale"] = D ** -0.5
    if own:
        _prepare_own(st)
    return st


def _axis_pairs(c):
    half, a = c["rotary"] // 2, c["axes"]
    first = half - (a - 1) * (3 * half // 8)  # as image models split it: 16, 24, 24 of 64
    return [first] + [3 * half // 8] * (a - 1)


def _prepare_own(st):
    """The pool's handle, the batch's and rotation's descriptors and the buffers that calls write to."""
    import gather_translate_kv_gb300 as gt

    c = st["case"]
    it = 1 if c["cache"] == "e4m3" else 2
    P = st["raw"].numel() // (2 * c["layers"] * c["page"] * c["heads"] * c["dim"] * it) - 1  # the last is the tail pad
    st["pool"] = gt.kv_pool_create(gt.make_desc(c["layers"], c["heads"], c["dim"], it, c["page"], P), st["raw"])
    st["batch"] = gt.kv_batch(st["table"], st["len"], st["cu"], st["n_rows"], seq_start=st["start"])
    H, D = c["heads"], c["dim"]
    if c["op"] == "append":
        st["rot"] = gt.kv_rotary(st["cos_sin"], positions=st["pos"], axis_pairs=st["axis_pairs"],
                                 interleaved=c["interleaved"])
        st["q_out"] = torch.empty_like(st["q"])
        if c["cache"] == "e4m3":
            st["read"] = gt.kv_batch(st["table"], st["len"], st["read_cu"], st["read_rows"],
                                     seq_start=st["read_start"])
            st["out_k"] = torch.empty(st["read_rows"], H, D, dtype=torch.bfloat16, device="cuda")
            st["out_v"] = torch.empty_like(st["out_k"])
    elif c["op"] == "attend":
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(st["n_rows"], c["q_heads"], device="cuda") if c["lse"] else None
        st["workspace"] = torch.empty(gt.kv_attend_workspace_bytes(st["pool"], c["q_heads"], c["seqs"], st["n_rows"]),
                                      dtype=torch.uint8, device="cuda")
    else:
        st["out_k"] = torch.empty(st["n_rows"], H, D, dtype=torch.bfloat16, device="cuda")
        st["out_v"] = torch.empty_like(st["out_k"])


# -------------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import gather_translate_kv_gb300 as gt

    c = st["case"]
    scales = st.get("scales")
    if c["op"] == "append":
        gt.kv_append_layer(st["pool"], c["layer"], st["batch"], st["k"], st["v"], rotary=st["rot"], q=st["q"],
                           q_out=st["q_out"], scales=scales)
        if c["cache"] != "e4m3":
            return {"q": st["q_out"], "cache": st["values"]}
        gt.kv_gather_layer_scaled(st["pool"], c["layer"], st["read"], scales, st["out_k"], st["out_v"])
        return {"q": st["q_out"], "k": st["out_k"], "v": st["out_v"]}
    if c["op"] == "attend":
        gt.kv_attend_layer(st["pool"], c["layer"], st["batch"], st["q"], st["out"], st["scale"], window=c["window"],
                           sinks=c["sinks"], scales=scales, lse=st["lse"], workspace=st["workspace"])
        return {"out": st["out"], "lse": st["lse"]} if c["lse"] else {"out": st["out"]}
    gt.kv_gather_layer_scaled(st["pool"], c["layer"], st["batch"], scales, st["out_k"], st["out_v"])
    return {"k": st["out_k"], "v": st["out_v"]}


def _views(st):
    """K and V of the layer as [pages, page, heads, dim], and their scales as [pages, heads]."""
    c = st["case"]
    L, l, dt = c["layers"], c["layer"], torch.float8_e4m3fn if c["cache"] == "e4m3" else TYPES[c["type"]]
    v = st["raw"].view(dt).view(-1, 2 * L, c["page"], c["heads"], c["dim"])[:-1]
    if c["cache"] != "e4m3":
        return v[:, 2 * l], v[:, 2 * l + 1], None, None
    return v[:, 2 * l], v[:, 2 * l + 1], st["scales"][:, l, 0], st["scales"][:, l, 1]


def _at(x, *where):
    """x[where] as 32-bit values, codes taken as bytes first."""
    if x.dtype == torch.float8_e4m3fn:
        return x.view(torch.uint8)[where].view(x.dtype).float()
    return x[where].float()


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


def _power_of_two(amax):
    """The least power of two 2^e, e >= -60, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -60)).clamp_(min=-60)
    return ((e + 127) << 23).int().view(torch.float32)


def _append_scaled(cache, scales, x, page, off, st):
    """New values x (32 bits) into a cache of codes with a scale for each page and head."""
    ps = st["case"]["page"]
    first = st["table"].gather(1, (st["start"] // ps).long()[:, None])[:, 0].long()  # first touched pages
    held = (st["start"] % ps).long()  # their tokens from before
    amax = torch.zeros_like(scales).scatter_reduce_(0, page[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    base = torch.zeros_like(scales)
    base[first] = torch.where(held[:, None] > 0, scales[first], 0.0)
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda")
    touched[page] = True
    fresh = torch.where(touched[:, None], torch.maximum(base, _power_of_two(amax)), scales)
    codes = cache.view(torch.uint8)
    old = codes[first]
    again = (old.view(cache.dtype).float() * (base / fresh)[first][:, None, :, None]).to(cache.dtype)
    keep = (torch.arange(ps, device="cuda") < held[:, None])[..., None, None]
    codes[first] = torch.where(keep, again.view(torch.uint8), old)
    codes[page, off] = (x / fresh[page][..., None]).to(cache.dtype).view(torch.uint8)
    scales.copy_(fresh)


def _read(st, start, cu, rows):
    c = st["case"]
    k, v, sk, sv = _views(st)
    r = torch.arange(rows, device="cuda")
    s = torch.searchsorted(cu[1:].contiguous(), r, right=True)
    j = start[s].long() + r - cu[s]
    page, off = st["table"][s, j // c["page"]].long(), j % c["page"]
    return {n: (_at(x, page, off) * z[page][..., None]).to(torch.bfloat16) for n, x, z in
            (("k", k, sk), ("v", v, sv))}


def _run_plain(st):
    c = st["case"]
    if c["op"] == "gather":
        return _read(st, st["start"], st["cu"], st["n_rows"])
    if c["op"] == "attend":
        return _attend_plain(st)
    k, v, sk, sv = _views(st)
    s, j = _rows(st)
    page, off = st["table"][s, j // c["page"]].long(), j % c["page"]
    q = _rotate(st["q"], st).to(st["q"].dtype)
    if c["cache"] == "e4m3":
        _append_scaled(k, sk, _rotate(st["k"], st), page, off, st)
        _append_scaled(v, sv, st["v"].float(), page, off, st)
        return {"q": q, **_read(st, st["read_start"], st["read_cu"], st["read_rows"])}
    k[page, off] = _rotate(st["k"], st).to(k.dtype)
    v[page, off] = st["v"]
    return {"q": q, "cache": st["values"]}


def _attend_plain(st):
    c = st["case"]
    k, v, sk, sv = _views(st)
    S, n, m, H, D = c["seqs"], st["max_len"], st["max_new"], c["heads"], c["dim"]
    j = torch.arange(n, device="cuda")
    page = st["table"][:, j // c["page"]].clamp(min=0).long()  # [S, n]
    off = (j % c["page"]).expand(S, n)
    K, V = _at(k, page, off), _at(v, page, off)
    if sk is not None:
        K *= sk[page][..., None]
        V *= sv[page][..., None]
    s, i = _rows(st)
    t = i - st["start"][s]
    q = torch.zeros(S, m, H, c["q_heads"] // H, D, device="cuda")
    q[s, t] = st["q"].float().view(-1, H, c["q_heads"] // H, D)
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(S, H, -1, D), K.permute(0, 2, 3, 1)).view(S, H, -1, m, n)
    del K
    x *= st["scale"]
    at = st["start"].long()[:, None] + torch.arange(m, device="cuda")  # [S, m]
    seen = j <= at[..., None]
    if c["window"]:
        seen &= (at[..., None] - j < c["window"]) | (j < c["sinks"])
    seen &= (j < st["len"][:, None])[:, None]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    x -= top
    x.exp_()
    total = x.sum(-1, keepdim=True)
    V *= (j < st["len"][:, None])[..., None, None]
    y = torch.matmul(x.view(S, H, -1, n), V.permute(0, 2, 1, 3)).view(S, H, -1, m, D)
    y = torch.where(total > 0, y / total, 0.0).permute(0, 3, 1, 2, 4)[s, t]
    out = {"out": y.reshape(-1, c["q_heads"], D).to(st["q"].dtype)}
    if c["lse"]:
        out["lse"] = (top + total.log())[..., 0].permute(0, 3, 1, 2)[s, t].reshape(-1, c["q_heads"])
    return out


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c = case
    st = prepare(c, seed)
    n, new = _lengths(c)
    L, l, ps, H, D, Q = c["layers"], c["layer"], c["page"], c["heads"], c["dim"], c["q_heads"]
    bits = c["cache"] == "e4m3"
    pool = st["raw"].view(torch.float8_e4m3fn if bits else TYPES[c["type"]]).view(-1, 2 * L, ps, H, D)
    table = st["table"].cpu()

    def held(s, a, b, which):
        """Tokens [a, b) of sequence s in the cache, K (0) or V (1), as [b - a, H, D]."""
        p = table[s, a // ps: -(-b // ps)].long().cuda()
        x = _at(pool, p, 2 * l + which).double()
        if bits:
            x = x * st["scales"][p, l, which].double()[:, None, :, None]
        x = x.reshape(-1, H, D)
        return x[a - a // ps * ps:][: b - a]

    def turned(x):
        rd, half = c["rotary"], c["rotary"] // 2
        y = x.double().clone()
        f = 0
        for a, count in enumerate(st["axis_pairs"]):
            for _ in range(count):
                row = st["cos_sin"].double()[st["pos"][a].long()]
                cs, sn = row[:, f, None], row[:, half + f, None]
                i1, i2 = (2 * f, 2 * f + 1) if c["interleaved"] else (f, f + half)
                u, w = x[..., i1].double(), x[..., i2].double()
                y[..., i1], y[..., i2] = u * cs - w * sn, w * cs + u * sn
                f += 1
        return y

    if c["op"] == "gather":
        return {name: torch.cat([held(s, n[s] - new[s], n[s], w) for s in range(c["seqs"])]) for w, name in
                ((0, "k"), (1, "v"))}
    if c["op"] == "append":
        q, k, v = turned(st["q"]), turned(st["k"]), st["v"].double()
        at = [0]
        for b in new:
            at.append(at[-1] + b)
        if bits:  # what the 8 bits stand for: the values themselves
            out = {"q": q}
            for w, name, x in ((0, "k", k), (1, "v", v)):
                parts = []
                for s in range(c["seqs"]):
                    a = n[s] - new[s]
                    parts += [held(s, a // ps * ps, a, w), x[at[s]:at[s + 1]]] if a % ps else [x[at[s]:at[s + 1]]]
                out[name] = torch.cat(parts)
            return out
        cache = pool.double()
        for s in range(c["seqs"]):
            for i in range(0, new[s], 1 if new[s] < 8 else ps):
                a = n[s] - new[s] + i
                b = min(n[s], a + 1 if new[s] < 8 else a + ps)
                j = torch.arange(a, b)
                p = table[s, j // ps].long().cuda()
                cache[p, 2 * l, (j % ps).cuda()] = k[at[s] + i: at[s] + i + b - a]
                cache[p, 2 * l + 1, (j % ps).cuda()] = v[at[s] + i: at[s] + i + b - a]
        return {"q": q, "cache": cache.view(-1)}
    outs, lses, at = [], [], 0
    for s in range(c["seqs"]):
        q = st["q"][at: at + new[s]].double().view(new[s], H, Q // H, D)
        at += new[s]
        K, V = held(s, 0, n[s], 0), held(s, 0, n[s], 1)
        i = torch.arange(n[s] - new[s], n[s], device="cuda")[:, None]
        j = torch.arange(n[s], device="cuda")[None]
        seen = j <= i
        if c["window"]:
            seen = seen & ((i - j < c["window"]) | (j < c["sinks"]))
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
