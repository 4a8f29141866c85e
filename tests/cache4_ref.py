"""Plain forms for pools of 4-bit values (KV_FORMAT_E2M1): rows of codes and
scale bytes, a World over such a pool, and its append, on the CPU. Shares no
code with the library."""
from __future__ import annotations

import numpy as np
import torch

import attention_ref as ref

STEPS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def row_bytes(H, D):
    return -(-(H * D // 2 + H * D // 16) // 16) * 16


def scale_value(byte):
    """Bytes (any integer array) -> scales in 64 bits; above 0xE0 NaN."""
    b = np.asarray(byte).astype(np.int64)
    e, m = b >> 3, b & 7
    s = np.where(e > 0, (1 + m / 8) * np.exp2(e - 15.0), m / 8 * 2.0 ** -14)
    return np.where(b > 0xE0, np.nan, s)


def decode(rows, H, D):
    """[..., R] bytes -> [..., H, D] in 64 bits."""
    x = np.asarray(rows)
    lead = x.shape[:-1]
    codes = x[..., :H * D // 2].reshape(*lead, H, D // 2)
    scales = x[..., H * D // 2:H * D // 2 + H * D // 16].reshape(*lead, H, D // 16)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*lead, H, D)
    v = np.where(c & 8, -1.0, 1.0) * STEPS[c & 7]
    return torch.from_numpy(v * np.repeat(scale_value(scales), 16, -1))


def nearest(y):
    """Codes of values in 32 bits: the nearest step, of two the one with an even code, at most 6."""
    m = np.minimum(np.abs(y), 8).astype(np.float64)
    d = np.abs(m[..., None] - STEPS)
    best = d.min(-1, keepdims=True)
    tie = (d == best) * np.array([2, 1] * 4)  # even codes first
    return (tie.argmax(-1) | np.where(np.signbit(y), 8, 0)).astype(np.uint8)


def encode(x):
    """[H, D] in 32 bits -> (codes [H, D / 2], scales [H, D / 16]), and which blocks are not finite."""
    b = np.asarray(x, dtype=np.float32).reshape(x.shape[0], -1, 16)
    bad = ~np.isfinite(b).all(-1)
    amax = np.abs(np.where(bad[..., None], 0, b)).max(-1).astype(np.float32)
    sixth = np.minimum(amax * (np.float32(1) / np.float32(6)), np.float32(8192))
    h = sixth.astype(np.float16).astype(np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(h, 2.0 ** -14))) - 3)
    S = np.rint(h / step) * step
    byte = (S.astype(np.float16).view(np.uint16) >> 7).astype(np.uint8)
    assert (scale_value(byte) == S).all()
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.where(S > 0, np.float32(1) / S.astype(np.float32), np.float32(0)).astype(np.float32)
        y = b * inv[..., None]
    c = nearest(np.where(bad[..., None], 0, y)).reshape(x.shape[0], -1)
    byte = np.where(bad, 0xFF, byte).astype(np.uint8)
    return c[:, 0::2] | c[:, 1::2] << 4, byte, bad


class World4(ref.World):
    @property
    def R(self):
        return row_bytes(self.H, self.D)

    def rows_view(self, raw=None):
        """[P, L, 2, ps, R] bytes."""
        raw = self.raw if raw is None else raw
        return raw[: self.P * self.L * 2 * self.ps * self.R].view(self.P, self.L, 2, self.ps, self.R)

    def scale_bytes(self, raw=None):
        """[P, L, 2, ps, H, D / 16] bytes, a view."""
        a = self.H * self.D // 2
        return self.rows_view(raw)[..., a:a + self.H * self.D // 16].unflatten(-1, (self.H, self.D // 16))

    def values(self, raw=None, scales=None):
        return decode(self.rows_view(raw).numpy(), self.H, self.D)


def world(seed, lens, news, *, H=2, D=64, L=2, ps=16, lo=0x58, hi=0x78, **kw):
    """A World over random codes, scale bytes in [lo, hi]."""
    w = ref.world(seed, lens, news, H=1, D=16, L=L, ps=ps, cache="bf16", **kw)
    n = (w.P + 1) * L * 2 * ps
    g = torch.Generator().manual_seed(seed)
    rows = torch.randint(0, 256, (n, row_bytes(H, D)), generator=g, dtype=torch.uint8)
    a = H * D // 2
    rows[:, a:a + H * D // 16] = torch.randint(lo, hi + 1, (n, H * D // 16), generator=g, dtype=torch.uint8)
    return World4(L, H, D, ps, w.P, "e2m1", rows.flatten(), None, w.lens, w.news, w.gap, w.table)


def append(w: World4, layer, k, v, rot):
    """The pool's bytes after an append, and a mask of the code bytes that are
    not specified (those of blocks that are not finite)."""
    raw = w.raw.clone()
    free = torch.zeros_like(raw)
    pool, mask = w.rows_view(raw), w.rows_view(free)
    a, nb = w.H * w.D // 2, w.H * w.D // 16
    for r, s, j in w.rows():
        pg = ref.page_of(w, s, j)
        if not pg:
            continue
        for which, x in ((0, k), (1, v)):
            y = ref.rotate(rot if which == 0 else None, x[r], r, j, torch.float32).numpy()
            codes, scales, bad = encode(y)
            at = pool[pg, layer, which, j % w.ps]
            at[:a] = torch.from_numpy(codes.reshape(-1))
            at[a:a + nb] = torch.from_numpy(scales.reshape(-1))
            mask[pg, layer, which, j % w.ps, :a] = torch.from_numpy(np.repeat(bad.reshape(-1), 8).astype(np.uint8))
    return raw, free.bool()
