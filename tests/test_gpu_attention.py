"""Append with rotation, attention over the pages and the scaled gather on the
GPU, against the plain 64-bit forms of attention_ref.py.

Bounds. u is the unit roundoff of the 16-bit output type (2^-8 for bf16, 2^-11
for fp16). An output is rounded once (u |out|); softmax weights may meet the
values rounded to the same 16 bits (u * A, A the weighted mean of |v|); scores
are 32-bit sums of at most 256 products of magnitudes that add up to about
100 here, scaled by D^-0.5, so a weight's relative error stays below 2^-12
(2^-12 * A); fp16's subnormal step is 2^-24. The log-sum-exp carries the
scores' error alone: 2^-12.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as ref
import gather_translate_kv_gb300 as gt

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gather_translate_kv_gb300 import build

    build.build()


class Dev:
    """A World's pool, batch and scales on the device."""

    def __init__(self, w: ref.World, kernel_facing=False):
        self.w = w
        self.raw = w.raw.cuda()
        it = ref.CACHE[w.cache].itemsize
        self.pool = gt.kv_pool_create(gt.make_desc(w.L, w.H, w.D, it, w.ps, w.P), self.raw)
        self.scales = None if w.scales is None else w.scales.cuda()
        if self.scales is not None:
            assert gt.kv_scale_bytes(self.pool) == self.scales.numel() * 4
        table = w.table.copy()
        if kernel_facing:
            live = (table > 0) & (table < w.P)
            table[live] *= 2 * w.L
        self.batch = gt.kv_batch(torch.from_numpy(table).cuda(), torch.tensor(w.lens, dtype=torch.int32).cuda(),
                                 torch.from_numpy(w.cu).cuda(), w.n_rows,
                                 seq_start=torch.tensor([a - b for a, b in zip(w.lens, w.news)],
                                                        dtype=torch.int32).cuda(), kernel_facing=kernel_facing)

    def error(self):
        return gt.kv_pool_last_error(self.pool)

    def attend(self, layer, q, scale, out=None, lse=None, stream=None, **kw):
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
        ws = torch.full((gt.kv_attend_workspace_bytes(self.pool, q.shape[1], self.w.S, self.w.n_rows),), 0xA5,
                        dtype=torch.uint8, device="cuda")
        gt.kv_attend_layer(self.pool, layer, self.batch, q, out, scale, ws, scales=self.scales, lse=lse, stream=stream,
                           **kw)
        return out


def check_attend(w, Q, dtype, *, layer=1, window=0, sinks=0, seed=0, kernel_facing=False, scale=None, qmul=1.0):
    d = Dev(w, kernel_facing)
    q = (torch.randn(w.n_rows, Q, w.D, generator=torch.Generator().manual_seed(seed + 77)) * qmul).to(T[dtype])
    scale = w.D ** -0.5 if scale is None else scale
    lse = torch.full((w.n_rows, Q), 7.0, device="cuda")
    out = d.attend(layer, q.cuda(), scale, lse=lse, window=window, sinks=sinks)
    assert d.error() == 0
    want, wlse, size = ref.attend(w, layer, q, scale, window, sinks)
    rows = [r for r, _, _ in w.rows()]
    rest = sorted(set(range(w.n_rows)) - set(rows))
    got = out.cpu().double()
    assert (got[rest] == 7.0).all() and (lse.cpu()[rest] == 7.0).all(), "rows of no token were written"
    u = U[T[dtype]]
    tol = u * want.abs() + (u + 2.0 ** -12) * size + (2.0 ** -24 if dtype == "fp16" else 0.0)
    bad = ~((got - want).abs() <= tol)[rows]
    assert not bad.any(), (int(bad.sum()), bad.numel(), np.argwhere(bad.numpy())[:3].tolist(),
                           float(((got - want).abs() / tol)[rows].nan_to_num(1e9).max()))
    e = lse.cpu().double()[rows]
    wl = wlse[rows]
    assert torch.equal(e.isinf(), wl.isinf())
    fin = ~wl.isinf()
    assert ((e - wl).abs()[fin] <= 2.0 ** -12 * wl.abs().clamp(min=1)[fin]).all()
    return out


CACHES = [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")]

# lens, news: one token, many, ragged, empty sequences
LENGTHS = {
    "one": ([1], [1]),
    "decode": ([1, 17, 64, 65, 200, 33, 128], [1] * 7),
    "long": ([1500, 3], [1, 1]),
    "drafts": ([5, 90, 301, 16], [5, 3, 4, 1]),
    "prompt": ([70], [70]),
    "chunks": ([150, 40, 333], [60, 40, 97]),
    "mixed": ([300, 0, 129, 7, 260, 12], [1, 0, 129, 0, 34, 2]),
}


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("D", [64, 128])
def test_attend(cache, dtype, lengths, D):
    w = ref.world(len(lengths) * 7 + D, *LENGTHS[lengths], D=D, cache=cache, gap=lengths == "mixed")
    check_attend(w, 8, dtype)


@pytest.mark.parametrize("cache,dtype", CACHES[1:3])
@pytest.mark.parametrize("ps", [1, 4, 7, 16, 24, 64, 256])
@pytest.mark.parametrize("lengths", ["decode", "drafts", "chunks"])
def test_attend_page_sizes(cache, dtype, ps, lengths):
    w = ref.world(ps, *LENGTHS[lengths], ps=ps, cache=cache, odd_scales=True)
    check_attend(w, 6, dtype, kernel_facing=ps % 2 == 0)


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("H,G", [(1, 1), (1, 71), (2, 1), (3, 5), (4, 2), (8, 8), (5, 16), (2, 17)])
def test_attend_head_layouts(cache, dtype, H, G):
    w = ref.world(H * 100 + G, [40, 130, 9], [1, 3, 9], H=H, cache=cache)
    check_attend(w, H * G, dtype)


@pytest.mark.parametrize("cache,dtype", CACHES[:3])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (33, 4), (64, 70), (100, 16), (1000, 3), (5, 1000)])
@pytest.mark.parametrize("lengths", ["decode", "chunks", "drafts"])
def test_attend_window_and_sinks(cache, dtype, window, sinks, lengths):
    w = ref.world(window + sinks, *LENGTHS[lengths], cache=cache)
    check_attend(w, 4, dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("cache,dtype", CACHES[:3])
@pytest.mark.parametrize("lengths", ["decode", "chunks", "drafts"])
@pytest.mark.parametrize("ps", [4, 16, 32])
def test_attend_tombstones_and_empty_rows(cache, dtype, lengths, ps):
    """Cleared pages are not visible; rows that see nothing give 0 and -inf."""
    w = ref.world(5, *LENGTHS[lengths], ps=ps, cache=cache, tombs=12)
    w.table[0, :] = -1  # a sequence with nothing left
    check_attend(w, 4, dtype)
    check_attend(w, 4, dtype, window=9, sinks=2)


@pytest.mark.parametrize("D,H", [(8, 2), (16, 1), (48, 2), (80, 2), (96, 1), (112, 2), (192, 1), (256, 1)])
@pytest.mark.parametrize("cache,dtype", CACHES[:3])
def test_attend_other_head_sizes(D, H, cache, dtype):
    w = ref.world(D, [1, 37, 90], [1, 2, 20], D=D, H=H, cache=cache)
    check_attend(w, 2 * H, dtype)


@pytest.mark.parametrize("cache,dtype", CACHES)
def test_attend_large_scores(cache, dtype):
    """Scores of several hundred: one key takes nearly all the weight, and the running maximum moves far."""
    w = ref.world(3, [300, 64, 200], [1, 40, 3], cache=cache)
    d = Dev(w)
    q = (torch.randn(w.n_rows, 4, w.D, generator=torch.Generator().manual_seed(1)) * 40).to(T[dtype])
    out = d.attend(1, q.cuda(), 0.3).cpu().double()
    want, _, size = ref.attend(w, 1, q, 0.3)
    # scores of magnitude up to 64 * 40 * 4 * 0.3 ~ 3000, summed in 32 bits: 2^-24 * 3000 * 8 in the exponent
    u = U[T[dtype]]
    tol = u * want.abs() + (u + 2.0 ** -9) * size + 2.0 ** -24
    assert ((out - want).abs() <= tol).all(), float(((out - want).abs() / tol).max())


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("mul", [2.0 ** -20, 2.0 ** 12])
def test_attend_scales_far_from_one(cache, dtype, mul):
    """Values (8-bit: their scales) far from 1 keep the result's relative precision."""
    if cache == "fp16":
        pytest.skip("outside fp16's range")
    if dtype == "fp16":
        mul = 2.0 ** -8 if mul < 1 else 2.0 ** 6
    w = ref.world(8, [100, 50, 200], [1, 30, 2], cache=cache)
    if cache == "e4m3":
        w.scales[:, :, 1] *= mul
        w.scales[1::3, :, 1] *= 2.0 ** -6
    else:
        w.view()[:, :, 1] *= mul
    check_attend(w, 4, dtype)


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("lengths", ["decode", "chunks", "drafts"])
@pytest.mark.parametrize("fill", ["nan", "inf"])
def test_what_is_not_seen_changes_nothing(cache, dtype, lengths, fill):
    """NaN and infinities past a sequence's end, before its window, in the sink page and in cleared pages."""
    w = ref.world(11, *LENGTHS[lengths], cache=cache, tombs=2)
    kw = dict(window=40, sinks=3)
    clean = check_attend(w, 4, dtype, **kw)
    seen = torch.zeros(w.P, w.ps, dtype=torch.bool)
    for r, s, i in w.rows():
        for j in range(i + 1):
            if i - j < 40 or j < 3:
                seen[ref.page_of(w, s, j), j % w.ps] = True
    seen[0] = False
    v = w.view()
    poison = 0x7F if cache == "e4m3" else None
    if cache == "e4m3":
        b = v.view(torch.uint8)
        b.copy_(torch.where(seen[:, None, None, :, None, None], b, torch.full_like(b, poison)))
        if fill == "inf":
            w.scales[0] = float("inf")
    else:
        v.copy_(torch.where(seen[:, None, None, :, None, None], v, torch.full_like(v, float(fill))))
    again = check_attend(w, 4, dtype, **kw)
    rows = [r for r, _, _ in w.rows()]
    assert torch.equal(again[rows], clean[rows])


@pytest.mark.parametrize("cache,dtype", CACHES[:3])
@pytest.mark.parametrize("news", [5, 60, 300, 700])
@pytest.mark.parametrize("window", [0, 90])
def test_a_value_that_is_not_finite_reaches_every_row_that_sees_it(cache, dtype, news, window):
    """One element of one value: NaN in that element of the rows that see it, and nowhere else."""
    n, group = news + 20, 1
    w = ref.world(13, [n], [news], cache=cache)
    q = torch.randn(w.n_rows, group * w.H, w.D, generator=torch.Generator().manual_seed(3)).to(T[dtype])
    clean = Dev(w).attend(1, q.cuda(), 0.125, window=window)
    for at in (n - 1, n - news, n - news // 2, 7):
        bad = ref.World(**{**w.__dict__, "raw": w.raw.clone()})
        pg, off = ref.page_of(w, 0, at), at % w.ps
        if cache == "e4m3":
            bad.view().view(torch.uint8)[pg, 1, 1, off, 0, 9] = 0x7F
        else:
            bad.view()[pg, 1, 1, off, 0, 9] = float("nan")
        out = Dev(bad).attend(1, q.cuda(), 0.125, window=window)
        pos = torch.arange(news) + n - news
        sees = (pos >= at) & ((window == 0) | (pos - at < window))
        want = torch.zeros(out.shape, dtype=torch.bool)
        want[:news, 0, 9] = sees
        assert torch.equal(out.isnan().cpu(), want)
        assert torch.equal(out[:news][~sees], clean[:news][~sees])


@pytest.mark.parametrize("cache,dtype", CACHES[:3])
@pytest.mark.parametrize("news", [3, 40, 150])
def test_a_later_token_does_not_change_an_earlier_row(cache, dtype, news):
    """A NaN or infinite key or value of one of the new tokens reaches only the rows that see it."""
    n = 200
    w = ref.world(12, [n], [news], cache=cache)
    d = Dev(w)
    q = torch.randn(w.n_rows, 4, w.D, generator=torch.Generator().manual_seed(2)).to(T[dtype])
    clean = d.attend(1, q.cuda(), 0.125)
    at = n - news // 2 - 1
    pg, off = ref.page_of(w, 0, at), at % w.ps
    for which in (0, 1):
        bad = ref.World(**{**w.__dict__, "raw": w.raw.clone()})
        v = bad.view()
        if cache == "e4m3":
            v.view(torch.uint8)[pg, 1, which, off] = 0x7F
        else:
            v[pg, 1, which, off] = float("nan") if which == 0 else float("inf")
        out = Dev(bad).attend(1, q.cuda(), 0.125)
        before = at - (n - news)
        assert torch.equal(out[:before], clean[:before])
        assert not out[before:].isfinite().all(-1).any()


def test_attend_offsets_past_32_bits():
    """A pool of 6 GiB: rows past 2^32 bytes on both sides of the K and V blocks."""
    w = ref.world(4, [100, 70], [1, 40], D=128, H=8, L=2, ps=16, cache="bf16", spare=0)
    d0 = Dev(w)
    q = torch.randn(w.n_rows, 16, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    want = d0.attend(1, q, 0.1)
    P = 6 * 2 ** 30 // (4 * 16 * 2048)
    raw = torch.zeros((P + 1) * 4 * 16 * 2048, dtype=torch.uint8, device="cuda")
    pool = gt.kv_pool_create(gt.make_desc(2, 8, 128, 2, 16, P), raw)
    page = 4 * 16 * 2048
    table = w.table.copy()
    for s in range(w.S):
        for k in range(-(-w.lens[s] // 16)):
            far = P - 1 - int(w.table[s, k])
            raw[far * page:(far + 1) * page] = d0.raw[w.table[s, k] * page:(int(w.table[s, k]) + 1) * page]
            table[s, k] = far
    b = gt.kv_batch(torch.from_numpy(table).cuda(), d0.batch.tensors[1], d0.batch.tensors[2], w.n_rows,
                    seq_start=d0.batch.tensors[3])
    out = torch.empty_like(q)
    ws = torch.empty(gt.kv_attend_workspace_bytes(pool, 16, w.S, w.n_rows), dtype=torch.uint8, device="cuda")
    gt.kv_attend_layer(pool, 1, b, q, out, 0.1, ws)
    assert torch.equal(out, want)
    k = torch.randn(w.n_rows, 8, 128, device="cuda").to(torch.bfloat16)
    gt.kv_append_layer(pool, 1, b, k, k)
    assert gt.kv_pool_last_error(pool) == 0
    for r, s, j in list(w.rows())[::7]:
        at = int(table[s, j // 16]) * page + 3 * 16 * 2048 + (j % 16) * 2048
        assert torch.equal(raw[at:at + 2048].view(torch.bfloat16), k[r].flatten())


@pytest.mark.parametrize("cache,dtype", CACHES[:3])
def test_attend_many_splits_and_repeatability(cache, dtype):
    """A single long sequence is cut over the whole GPU; the result is the same every time, on any stream."""
    w = ref.world(21, [5003], [1], H=1, D=128, L=1, cache=cache)
    out = check_attend(w, 4, dtype, layer=0)
    d = Dev(w)
    q = torch.randn(w.n_rows, 4, 128, generator=torch.Generator().manual_seed(77)).to(T[dtype]).cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for i in range(5):
        again = d.attend(0, q, 128 ** -0.5, stream=st if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(again, out)


@pytest.mark.parametrize("lengths", ["drafts", "chunks"])
def test_attend_strided_queries_and_graph(lengths):
    w = ref.world(31, *LENGTHS[lengths], D=128)
    d = Dev(w)
    wide = torch.randn(w.n_rows, 4 * 128 + 40, device="cuda").to(torch.bfloat16)
    odd = torch.randn(w.n_rows, 4 * 128 + 41, device="cuda").to(torch.bfloat16)
    for x in (wide[:, 8:520], wide[:, 3:515], odd[:, 1:513]):
        q = x.unflatten(1, (4, 128))
        assert torch.equal(d.attend(1, q, 0.1), d.attend(1, q.contiguous(), 0.1))
    q = wide[:, :512].unflatten(1, (4, 128)).contiguous()
    want = d.attend(1, q, 0.1)
    out = torch.zeros_like(q)
    ws = torch.empty(gt.kv_attend_workspace_bytes(d.pool, 4, w.S, w.n_rows), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gt.kv_attend_layer(d.pool, 1, d.batch, q, out, 0.1, ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_attend_device_errors_are_reported_and_harmless():
    w = ref.world(41, [40, 50, 60], [2, 3, 20], D=64)
    good, _, _ = ref.attend(w, 1, torch.zeros(w.n_rows, 2, 64), 1.0)
    q = torch.zeros(w.n_rows, 2, 64, dtype=torch.bfloat16, device="cuda")
    # a page past the pool: its tokens drop out like a tombstone's
    bad = ref.World(**{**w.__dict__, "table": w.table.copy()})
    bad.table[0, 0] = w.P + 5
    d = Dev(bad)
    out = d.attend(1, q, 1.0)
    assert d.error() == gt.KV_DEV_ERR_ROW
    bad.table[0, 0] = 0
    want, _, _ = ref.attend(bad, 1, torch.zeros(w.n_rows, 2, 64), 1.0)
    assert (out.cpu().double() - want).abs().max() < 0.02
    # off the kernel-facing grid
    d = Dev(w, kernel_facing=True)
    d.batch.tensors[0][1, 1] += 1
    d.attend(1, q, 1.0)
    assert d.error() == gt.KV_DEV_ERR_FORM
    # inconsistent metadata: the sequence takes no part, the others are answered
    for which, value in ((1, 10 ** 6), (3, -4)):
        d = Dev(w)
        d.batch.tensors[which][1] = value
        out = d.attend(1, q, 1.0).cpu().double()
        assert d.error() == gt.KV_DEV_ERR_TABLE
        assert (out[2:5] == 7.0).all()
        assert (out[[0, 1] + list(range(5, 25))] - good[[0, 1] + list(range(5, 25))]).abs().max() < 0.02
    d = Dev(w)
    d.batch.tensors[2][3] = 10 ** 9
    d.attend(1, q, 1.0)
    assert d.error() == gt.KV_DEV_ERR_TABLE


# ------------------------------------------------------------------- append

def run_append(w, Q, dtype, rot, *, layer=1, kernel_facing=False, strided=0, seed=0, bad=None):
    g = torch.Generator().manual_seed(seed + 5)
    n = w.n_rows
    width = (Q + 2 * w.H) * w.D
    fused = torch.randn(n, width + strided, generator=g).to(T[dtype])
    if bad is not None:
        bad(fused)
    f = fused.cuda()
    q, k, v = (x.unflatten(1, (-1, w.D)) for x in f[:, :width].split([Q * w.D, w.H * w.D, w.H * w.D], 1))
    qc, kc, vc = (x.unflatten(1, (-1, w.D)) for x in fused[:, :width].split([Q * w.D, w.H * w.D, w.H * w.D], 1))
    d = Dev(w, kernel_facing)
    q_out = torch.full(q.shape, 7.0, dtype=T[dtype], device="cuda")
    r = None
    if rot is not None:
        r = gt.kv_rotary(rot.table.cuda(), None if rot.positions is None else rot.positions.cuda(), rot.axis_pairs,
                         rot.interleaved)
    gt.kv_append_layer(d.pool, layer, d.batch, k, v, rotary=r, q=q, q_out=q_out, scales=d.scales)
    assert d.error() == 0
    raw, scales = ref.append(w, layer, kc, vc, rot)
    assert torch.equal(d.raw.cpu(), raw), "pool bytes"
    if scales is not None:
        assert torch.equal(d.scales.cpu(), scales)
    want = torch.full(q.shape, 7.0, dtype=T[dtype])
    for row, s, j in w.rows():
        want[row] = ref.rotate(rot, qc[row], row, j, torch.float32).to(T[dtype])
    assert torch.equal(q_out.cpu().view(torch.uint8), want.view(torch.uint8))
    # and against 64 bits: one rounding of the output, and 32-bit products
    for row, s, j in w.rows():
        x = ref.rotate(rot, qc[row], row, j, torch.float64)
        u = U.get(T[dtype], 2.0 ** -24)
        fin = x.isfinite()
        assert ((want[row].double() - x).abs()[fin] <= (u + 2.0 ** -22) * 2 * qc[row].double().abs().max() + 2.0 ** -24).all()
    return d, raw, scales


APPENDS = [  # D, rotary_dim, H, Q, ps
    (128, 128, 2, 4, 16), (64, 64, 8, 8, 32), (64, 32, 2, 2, 4), (128, 64, 1, 3, 64), (16, 16, 3, 1, 1),
    (80, 48, 2, 4, 16), (256, 256, 1, 2, 16), (8, 8, 4, 2, 4), (24, 10, 2, 1, 7), (128, 0, 2, 2, 16), (96, 96, 1, 1, 256),
]


@pytest.mark.parametrize("D,rd,H,Q,ps", APPENDS)
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("e4m3", "bf16"),
                                         ("e4m3", "fp16"), ("e4m3", "fp32")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(D, rd, H, Q, ps, cache, dtype, interleaved):
    for i, (lens, news) in enumerate([([9, 30, 1, 65], [1, 1, 1, 1]), ([70, 33, 0, 40], [41, 33, 0, 2])]):
        w = ref.world(D + i, lens, news, D=D, H=H, ps=ps, cache=cache, gap=i == 1, tombs=i)
        rot = ref.rotation(i, rd, 80, w.n_rows, interleaved=interleaved, given=i == 1) if rd else None
        run_append(w, Q, dtype, rot, kernel_facing=i == 1, strided=0 if i else 16)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("strided", [0, 3])
def test_append_several_axes(axes, cache, dtype, strided):
    w = ref.world(axes, [50, 20], [37, 3], D=64, H=2, cache=cache)
    for k in range(3):
        rot = ref.rotation(k, 64, 100, w.n_rows, axes=axes, interleaved=k == 1)
        run_append(w, 3, dtype, rot, strided=strided)


@pytest.mark.parametrize("D,ps", [(64, 16), (24, 16), (64, 256)])
def test_append_codes_stand_for_the_values(D, ps):
    """Codes times scales against 64 bits, over appends that grow the scale of a partly filled page."""
    w = ref.world(6, [5, 3], [5, 3], D=D, H=2, ps=ps, cache="e4m3", spare=4)
    w.table[:, 0] = [1, 2]
    w.table = np.concatenate([w.table[:, :1], np.array([[3], [4]], dtype=np.int32)], 1)
    truth = {}
    for step, (grow, news) in enumerate([(1e-3, [5, 3]), (1.0, [4, 1]), (0.01, [1, 9]), (3e4, [2, 1])]):
        if step:
            w.lens = [a + b for a, b in zip(w.lens, news)]
            w.news = news
        if max(w.lens) > ps * 2:
            break
        rot = ref.rotation(step, D, 64, w.n_rows)
        g = torch.Generator().manual_seed(step)
        k, v = (torch.randn(w.n_rows, 2, D, generator=g) * grow for _ in range(2))
        d = Dev(w)
        gt.kv_append_layer(d.pool, 1, d.batch, k.cuda(), v.cuda(),
                           rotary=gt.kv_rotary(rot.table.cuda()), scales=d.scales)
        assert d.error() == 0
        w.raw, w.scales = d.raw.cpu(), d.scales.cpu()
        for r, s, j in w.rows():
            truth[s, j] = (ref.rotate(rot, k[r], r, j, torch.float64), v[r].double())
        got = w.values()
        for (s, j), both in truth.items():
            for which in (0, 1):
                pg = ref.page_of(w, s, j)
                x, y = both[which], got[pg, 1, which, j % ps]
                S = w.scales[pg, 1, which].double()[:, None]
                # half a step of e4m3's 4 significant bits and of its subnormals; each rescaling
                # of a page (at most 3 here) may add half a subnormal step
                assert ((x - y).abs() <= 2.0 ** -4 * x.abs() * (1 + 2.0 ** -20) + 4 * 2.0 ** -10 * S).all()


def test_append_non_finite_and_zero_values():
    def bad(x):
        x[0] = 0
        x[3, 5::7] = float("nan")
        x[4, 2::5] = float("inf")
        x[5, ::3] = -float("inf")
        x[6] = float("nan")

    for D in (64, 24):
        w = ref.world(7, [1, 40, 33, 20], [1, 8, 1, 4], D=D, H=2, cache="e4m3")
        w.scales[int(w.table[2, 2])] = float("nan")
        w.scales[int(w.table[3, 1])] = -1.0
        rot = None

        def bytes_equal(a, b):
            return torch.equal(a.view(torch.uint8) & 0x7F, b.view(torch.uint8) & 0x7F)

        g = torch.Generator().manual_seed(5)
        x = torch.randn(w.n_rows, 4 * D, generator=g)
        bad(x)
        k, v = x.cuda().split([2 * D, 2 * D], 1)
        d = Dev(w)
        gt.kv_append_layer(d.pool, 1, d.batch, k.unflatten(1, (2, D)), v.unflatten(1, (2, D)), scales=d.scales)
        kc, vc = x.split([2 * D, 2 * D], 1)
        raw, scales = ref.append(w, 1, kc.unflatten(1, (2, D)), vc.unflatten(1, (2, D)), rot)
        got = d.raw.cpu()
        diff = got != raw
        assert ((got[diff] & 0x7F) == (raw[diff] & 0x7F)).all()  # only a NaN's sign may differ
        assert ((got[diff] & 0x7F) == 0x7F).all() or not diff.any()
        assert torch.equal(d.scales.cpu().nan_to_num(-5.0), scales.nan_to_num(-5.0))


def test_append_then_attend_then_gather_as_a_step():
    """The three calls in a row, kernel-facing, captured in a graph."""
    w = ref.world(9, [100, 33, 70], [1, 33, 4], D=128, H=2, cache="e4m3")
    rot = ref.rotation(1, 128, 128, w.n_rows)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(w.n_rows, h, 128, generator=g).to(torch.bfloat16) for h in (8, 2, 2))
    d = Dev(w, kernel_facing=True)
    r = gt.kv_rotary(rot.table.cuda())
    dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    out = torch.empty_like(dq)
    ok, ov = torch.empty_like(dk), torch.empty_like(dv)
    q_in = dq.clone()
    ws = torch.empty(gt.kv_attend_workspace_bytes(d.pool, 8, w.S, w.n_rows), dtype=torch.uint8, device="cuda")
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        gt.kv_append_layer(d.pool, 1, d.batch, dk, dv, rotary=r, q=q_in, q_out=dq, scales=d.scales)
        gt.kv_attend_layer(d.pool, 1, d.batch, dq, out, 0.09, ws, scales=d.scales)
        gt.kv_gather_layer_scaled(d.pool, 1, d.batch, d.scales, ok, ov)
    gr.replay()
    torch.cuda.synchronize()
    assert d.error() == 0
    w.raw, w.scales = ref.append(w, 1, k, v, rot)
    assert torch.equal(d.raw.cpu(), w.raw) and torch.equal(d.scales.cpu(), w.scales)
    qr = torch.stack([ref.rotate(rot, q[r_], r_, j, torch.float32).to(q.dtype) for r_, _, j in w.rows()])
    want, _, size = ref.attend(w, 1, qr, 0.09)
    u = 2.0 ** -8
    assert ((out.cpu().double() - want).abs() <= u * want.abs() + (u + 2.0 ** -12) * size).all()
    val = w.values()
    for r_, s, j in w.rows():
        pg = ref.page_of(w, s, j)
        assert torch.equal(ok[r_].cpu(), val[pg, 1, 0, j % w.ps].to(torch.bfloat16))
        assert torch.equal(ov[r_].cpu(), val[pg, 1, 1, j % w.ps].to(torch.bfloat16))


def test_append_queries_in_place_and_bad_positions():
    w = ref.world(15, [30, 40], [5, 2], D=64, H=2)
    d = Dev(w)
    rot = ref.rotation(0, 64, 64, w.n_rows, given=True)
    x = torch.randn(w.n_rows, 6, 64).to(torch.bfloat16)
    q = x[:, :2].contiguous().cuda()
    k, v = x[:, 2:4].cuda(), x[:, 4:].cuda()
    gt.kv_append_layer(d.pool, 1, d.batch, k.contiguous(), v.contiguous(), q=q, q_out=q,
                       rotary=gt.kv_rotary(rot.table.cuda(), rot.positions.cuda()))
    for r, s, j in w.rows():
        assert torch.equal(q[r].cpu(), ref.rotate(rot, x[r, :2], r, j, torch.float32).to(q.dtype))
    # a position outside the table: that row alone is left out
    for cache in ("bf16", "e4m3"):
        for D in (64, 24):
            w = ref.world(16, [30, 40], [5, 2], D=D, H=2, cache=cache)
            w.table[0, 1] = 0 if D == 24 else w.table[0, 1]
            d = Dev(w)
            rot = ref.rotation(0, D, 64, w.n_rows, given=True)
            pos = rot.positions.clone()
            pos[0, 3], pos[0, 6] = 64, -1
            x = torch.randn(w.n_rows, 3, D).to(torch.bfloat16)
            out = torch.full((w.n_rows, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
            k = x[:, :2].contiguous()
            gt.kv_append_layer(d.pool, 1, d.batch, k.cuda(), k.cuda(), q=x[:, 2:].contiguous().cuda(), q_out=out,
                               rotary=gt.kv_rotary(rot.table.cuda(), pos.cuda()), scales=d.scales)
            assert d.error() == gt.KV_DEV_ERR_POSITION
            o = out.cpu()
            assert (o[[3, 6]] == 7.0).all() and (o[[0, 1, 2, 4, 5]] != 7.0).any(-1).all()
            got, was = w.view(d.raw.cpu()), w.view()
            for r, s, j in w.rows():
                pg = ref.page_of(w, s, j)
                same = torch.equal(got[pg, 1, 1, j % w.ps].view(torch.uint8), was[pg, 1, 1, j % w.ps].view(torch.uint8))
                assert same == (r in (3, 6) or pg == 0)


# ------------------------------------------------------------------- gather

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,H,ps", [(64, 8, 32), (128, 2, 16), (24, 2, 4), (16, 1, 1), (80, 3, 7)])
def test_gather_scaled(dtype, D, H, ps):
    for odd, (lens, news) in enumerate([([40, 1, 90], [1, 1, 1]), ([40, 0, 90, 33], [40, 0, 57, 12])]):
        w = ref.world(D, lens, news, D=D, H=H, ps=ps, cache="e4m3", tombs=3, gap=bool(odd), odd_scales=bool(odd))
        d = Dev(w, kernel_facing=bool(odd))
        outs = [torch.full((w.n_rows, H, D), 7.0, dtype=T[dtype], device="cuda") for _ in range(2)]
        gt.kv_gather_layer_scaled(d.pool, 1, d.batch, d.scales, *outs)
        assert d.error() == 0
        val = w.view().float() * w.scales[:, :, :, None, :, None]
        for which in (0, 1):
            want = torch.full((w.n_rows, H, D), 7.0)
            for r, s, j in w.rows():
                pg = ref.page_of(w, s, j)
                want[r] = val[pg, 1, which, j % ps] if pg else 0.0
            assert torch.equal(outs[which].cpu(), want.to(T[dtype]))


# ------------------------------------------------------------------ refusals

def test_refusals():
    w = ref.world(1, [20], [2], D=64, H=2)
    d = Dev(w)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(gt.kv_attend_workspace_bytes(d.pool, 4, 1, 2), dtype=torch.uint8, device="cuda")

    def refused(code, call):
        with pytest.raises(gt.KVError) as e:
            call()
        assert e.value.code == code, e.value

    at = lambda **kw: gt.kv_attend_layer(d.pool, kw.pop("layer", 1), kw.pop("batch", d.batch), kw.pop("q", q),  # noqa: E731
                                         kw.pop("out", out), kw.pop("scale", 1.0), kw.pop("ws", ws), **kw)
    refused(-1, lambda: at(layer=2))
    refused(-1, lambda: at(layer=-1))
    refused(-1, lambda: at(window=-1))
    refused(-1, lambda: at(sinks=-1))
    refused(-1, lambda: at(scale=float("nan")))
    refused(-1, lambda: at(scale=float("inf")))
    refused(-1, lambda: at(ws=ws[: ws.numel() - 16]))
    refused(-5, lambda: at(ws=torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")[1:]))
    refused(-1, lambda: at(q=q.float(), out=out.float()))
    q3 = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    refused(-1, lambda: at(q=q3, out=q3.clone()))
    with pytest.raises(ValueError):
        at(q=q.cpu())
    with pytest.raises(ValueError):
        at(q=q[:1])
    with pytest.raises(ValueError):
        at(out=out.half())
    with pytest.raises(ValueError):
        at(scales=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        at(lse=torch.zeros(2, 3, device="cuda"))
    with pytest.raises(ValueError):
        at(q=q.transpose(1, 2).contiguous().transpose(1, 2))
    ap = lambda k_=k, v_=k, **kw: gt.kv_append_layer(d.pool, kw.pop("layer", 0), d.batch, k_, v_, **kw)  # noqa: E731
    refused(-1, lambda: ap(k.float(), k.float()))  # another size than the pool's elements
    refused(-1, lambda: ap(layer=7))
    table = torch.zeros(64, 64, device="cuda")
    refused(-1, lambda: ap(rotary=gt.kv_rotary(torch.zeros(4, 66, device="cuda"))))  # past the head
    refused(-1, lambda: ap(rotary=gt.kv_rotary(torch.zeros(4, 63, device="cuda"))))
    refused(-1, lambda: ap(rotary=gt.kv_rotary(table, torch.zeros(2, 2, dtype=torch.int32, device="cuda"), (20, 13))))
    wide = torch.zeros(2, 6, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        ap(q=wide[:, :4], q_out=wide[:, :4])
    with pytest.raises(ValueError):
        ap(k[:, :1], k[:, :1])
    with pytest.raises(ValueError):
        gt.kv_rotary(table, torch.zeros(2, 2, dtype=torch.int32, device="cuda"))
    refused(-1, lambda: gt.kv_scale_bytes(d.pool))
    with pytest.raises(ValueError):
        gt.kv_gather_layer_scaled(d.pool, 0, d.batch, torch.zeros(4, device="cuda"), k, k)
    # an 8-bit pool without scales, an MLA pool
    w8 = Dev(ref.world(1, [20], [2], D=64, H=2, cache="e4m3"))
    with pytest.raises(ValueError):
        gt.kv_append_layer(w8.pool, 0, w8.batch, k, k)
    mla = gt.kv_pool_create(gt.make_desc(2, 2, 64, 2, 16, 8, latent_only=True))
    refused(-1, lambda: gt.kv_append_layer(mla, 0, d.batch, k, k))
    refused(-1, lambda: gt.kv_attend_layer(mla, 0, d.batch, q, out, 1.0, ws))
    # nothing to do
    empty = gt.kv_batch(torch.zeros(0, 4, dtype=torch.int32, device="cuda"),
                        torch.zeros(0, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int64, device="cuda"), 0)
    none = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    gt.kv_attend_layer(d.pool, 0, empty, none, none.clone(), 1.0, ws)
    gt.kv_append_layer(d.pool, 0, empty, none[:, :2], none[:, :2])
    assert d.error() == 0
