"""Plain 64-bit forms of the operators of kv_attention.h, token by token on
the CPU, and random batches for their tests. Shares no code with the library:
pages are kept as arrays [page][layer][K or V][offset][head][element]."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn
CACHE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": E4M3}


@dataclass
class World:
    """One layer's view of a pool and a batch over it, all on the CPU."""

    L: int
    H: int
    D: int
    ps: int
    P: int
    cache: str
    raw: torch.Tensor            # uint8, total + tail pad
    scales: torch.Tensor | None  # float32 [P, L, 2, H]
    lens: list
    news: list
    gap: list                    # unused rows after each sequence's
    table: np.ndarray            # int32 [S, max_pages], physical

    @property
    def S(self):
        return len(self.lens)

    @property
    def cu(self):
        return np.concatenate([[0], np.cumsum([n + g for n, g in zip(self.news, self.gap)])]).astype(np.int64)

    @property
    def n_rows(self):
        return int(self.cu[-1])

    def rows(self):
        """(row, sequence, token index) of every row that is a token."""
        for s in range(self.S):
            for t in range(self.news[s]):
                yield int(self.cu[s]) + t, s, self.lens[s] - self.news[s] + t

    def view(self, raw=None):
        """[P, L, 2, ps, H, D] elements."""
        raw = self.raw if raw is None else raw
        n = self.P * self.L * 2 * self.ps * self.H * self.D
        t = CACHE[self.cache]
        return raw[: n * t.itemsize].view(t).view(self.P, self.L, 2, self.ps, self.H, self.D)

    def values(self, raw=None, scales=None):
        v = self.view(raw).double()
        if self.cache == "e4m3":
            s = self.scales if scales is None else scales
            v = v * s.double()[:, :, :, None, :, None]
        return v


def world(seed, lens, news, *, L=2, H=2, D=64, ps=16, cache="bf16", tombs=0, spare=3, gap=False, odd_scales=False,
          extra_pages=0):
    rng = np.random.default_rng(seed)
    pages = [-(-n // ps) for n in lens]
    mp = max(max(pages), 1) + extra_pages
    P = sum(pages) + 1 + spare
    order = rng.permutation(np.arange(1, P))
    table = np.full((len(lens), mp), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n]
        table[s, n:] = 0x7ffffff0  # entries past a sequence are never read
        at += n
    for _ in range(tombs):
        s = int(rng.integers(len(lens)))
        if pages[s]:
            table[s, rng.integers(pages[s])] = rng.choice([0, -1, -7])
    g = torch.Generator().manual_seed(seed)
    n = (P + 1) * L * 2 * ps * H * D
    t = CACHE[cache]
    if cache == "e4m3":
        raw = (torch.randn(n, generator=g) * 90).clamp(-448, 448).to(t).view(torch.uint8)
        e = torch.randint(-8, -4, (P, L, 2, H), generator=g).float()
        scales = torch.exp2(e)
        if odd_scales:
            scales = scales * (1 + torch.rand(P, L, 2, H, generator=g))
    else:
        raw, scales = torch.randn(n, generator=g).to(t).view(torch.uint8), None
    gaps = [int(rng.integers(0, 3)) if gap else 0 for _ in lens]
    return World(L, H, D, ps, P, cache, raw, scales, list(lens), list(news), gaps, table)


def page_of(w: World, s: int, j: int) -> int:
    """Physical page of a token, 0 for a tombstone."""
    return max(int(w.table[s, j // w.ps]), 0)


# ------------------------------------------------------------------- attention

def attend(w: World, layer, q, scale, window=0, sinks=0):
    """q [n_rows, Q, D] (any float type) -> out, lse, and the weighted mean of
    |v| that error bounds are made of; rows that are no token stay NaN."""
    Q = q.shape[1]
    G = Q // w.H
    val = w.values()
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    size = out.clone()
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float64)
    for r, s, i in w.rows():
        js = [j for j in range(i + 1) if (window == 0 or i - j < window or j < sinks) and page_of(w, s, j)]
        if not js:
            out[r], size[r], lse[r] = 0.0, 0.0, -float("inf")
            continue
        pg = torch.tensor([page_of(w, s, j) for j in js])
        off = torch.tensor([j % w.ps for j in js])
        K, V = val[pg, layer, 0, off], val[pg, layer, 1, off]  # [n, H, D]
        x = torch.einsum("hgd,nhd->hgn", q[r].double().view(w.H, G, -1), K) * scale
        p = torch.softmax(x, -1)
        out[r] = torch.einsum("hgn,nhd->hgd", p, V).reshape(Q, -1)
        size[r] = torch.einsum("hgn,nhd->hgd", p, V.abs()).reshape(Q, -1)
        lse[r] = torch.logsumexp(x, -1).reshape(Q)
    return out, lse, size


# ---------------------------------------------------------------------- append

@dataclass
class Rotation:
    table: torch.Tensor          # float32 [n_positions, rd]
    axis_pairs: list
    interleaved: bool
    positions: torch.Tensor | None  # int32 [axes, n_rows]


def rotation(seed, rd, n_pos, n_rows, axes=1, interleaved=False, given=False):
    half = rd // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * f
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(0, half + 1, size=axes - 1))
    pairs = np.diff(np.concatenate([[0], cuts, [half]])).tolist()
    pos = torch.from_numpy(rng.integers(0, n_pos, size=(axes, n_rows)).astype(np.int32)) if given or axes > 1 else None
    return Rotation(torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(), pairs, interleaved, pos)


def rotate(rot: Rotation | None, x, r, j, dtype):
    """Row r's heads x [heads, D], token index j, in the given precision (products and sums apart)."""
    y = x.to(dtype).clone()
    if rot is None:
        return y
    half = rot.table.shape[1] // 2
    f = torch.arange(half)
    if rot.positions is None:
        p = torch.full((half,), j)
    else:
        p = rot.positions[torch.repeat_interleave(torch.arange(len(rot.axis_pairs)), torch.tensor(rot.axis_pairs)), r].long()
    c, s = rot.table[p, f].to(dtype), rot.table[p, f + half].to(dtype)
    a, b = (2 * f, 2 * f + 1) if rot.interleaved else (f, f + half)
    x1, x2 = x[:, a].to(dtype), x[:, b].to(dtype)
    y[:, a], y[:, b] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


def power_of_two(amax: float) -> float:
    e = -60
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(w: World, layer, k, v, rot):
    """The pool's raw bytes and scales after an append, with 32-bit rotation
    (bit-exact for every cache type)."""
    raw = w.raw.clone()
    pool = w.view(raw)
    scales = None if w.scales is None else w.scales.clone()
    runs: dict = {}
    for r, s, j in w.rows():
        pg = page_of(w, s, j)
        if pg:
            runs.setdefault((s, pg), []).append((r, j))
    for (s, pg), toks in runs.items():
        offs = [j % w.ps for _, j in toks]
        for which, x in ((0, k), (1, v)):
            new = torch.stack([rotate(rot if which == 0 else None, x[r], r, j, torch.float32) for r, j in toks])
            if w.cache != "e4m3":
                for o, y in zip(offs, new):
                    pool[pg, layer, which, o] = y.to(pool.dtype)
                continue
            for h in range(w.H):
                y = new[:, h]
                fin = y.isfinite()
                amax = float(torch.where(fin, y.abs(), torch.zeros(())).max())
                base = float(scales[pg, layer, which, h]) if offs[0] > 0 else 0.0
                if not (base > 0 and np.isfinite(base)):
                    base = 0.0
                S = max(base, power_of_two(amax))
                if offs[0] > 0 and S != base:
                    old = pool[pg, layer, which, : offs[0], h].float() * (torch.tensor(base) / torch.tensor(S))
                    pool[pg, layer, which, : offs[0], h] = old.to(E4M3)
                codes = torch.where(fin, y, torch.full((), float("nan"))) * (torch.tensor(1.0) / torch.tensor(S))
                for o, c in zip(offs, codes):
                    pool[pg, layer, which, o, h] = c.to(E4M3)
                scales[pg, layer, which, h] = S
    return raw, scales
