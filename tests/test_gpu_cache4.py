"""Pools of 4-bit values (KV_FORMAT_E2M1) on the GPU: append, gather and
attention against the plain forms of cache4_ref.py and attention_ref.py.

Bounds. Appended bytes and gathered values are exact: the formulas round where
they say. Attention: u is the unit roundoff of the 16-bit output type (2^-8
for bf16, 2^-11 for fp16). The cache's values are exact in 16 bits. An output is rounded once
(u |out|); weights may meet the values rounded to 16 bits (u * A, A the
weighted mean of |v|); scores are 32-bit sums of at most 256 products, scaled
by D^-0.5, so that a weight's relative error stays below 2^-12 (2^-12 * A);
fp16's subnormal step is 2^-24. The log-sum-exp carries the scores' error
alone: 2^-12.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as ref
import cache4_ref as ref4
import gather_translate_kv_gb300 as gt
from test_gpu_attention import APPENDS, LENGTHS, T, U, Dev, _built  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


class Dev4(Dev):
    """A World4's pool and batch on the device."""

    def __init__(self, w, kernel_facing=False):
        self.w = w
        self.raw = w.raw.cuda()
        self.pool = gt.kv_pool_create(gt.make_desc(w.L, w.H, w.D, 1, w.ps, w.P, format=gt.KV_FORMAT_E2M1), self.raw)
        assert self.pool.row_bytes == w.R
        self.scales = None
        table = w.table.copy()
        if kernel_facing:
            live = (table > 0) & (table < w.P)
            table[live] *= 2 * w.L
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.batch = gt.kv_batch(torch.from_numpy(table).cuda(), i32(w.lens), torch.from_numpy(w.cu).cuda(), w.n_rows,
                                 seq_start=i32([a - b for a, b in zip(w.lens, w.news)]), kernel_facing=kernel_facing)


def check_attend(w, Q, dtype, *, layer=1, window=0, sinks=0, seed=0, kernel_facing=False, scale=None, qmul=1.0):
    d = Dev4(w, kernel_facing)
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
    e, wl = lse.cpu().double()[rows], wlse[rows]
    assert torch.equal(e.isinf(), wl.isinf())
    fin = ~wl.isinf()
    assert ((e - wl).abs()[fin] <= 2.0 ** -12 * wl.abs().clamp(min=1)[fin]).all()
    return out


# ---------------------------------------------------------------------- append

def run_append(w, Q, dtype, rot, *, layer=1, kernel_facing=False, strided=0, seed=0, change=None):
    g = torch.Generator().manual_seed(seed + 5)
    width = (Q + 2 * w.H) * w.D
    fused = torch.randn(w.n_rows, width + strided, generator=g).to(T[dtype])
    if change is not None:
        change(fused)
    f = fused.cuda()
    sizes = [Q * w.D, w.H * w.D, w.H * w.D]
    q, k, v = (x.unflatten(1, (-1, w.D)) for x in f[:, :width].split(sizes, 1))
    qc, kc, vc = (x.unflatten(1, (-1, w.D)) for x in fused[:, :width].split(sizes, 1))
    d = Dev4(w, kernel_facing)
    q_out = torch.full(q.shape, 7.0, dtype=T[dtype], device="cuda")
    r = None
    if rot is not None:
        r = gt.kv_rotary(rot.table.cuda(), None if rot.positions is None else rot.positions.cuda(), rot.axis_pairs,
                         rot.interleaved)
    gt.kv_append_layer(d.pool, layer, d.batch, k, v, rotary=r, q=q, q_out=q_out)
    assert d.error() == 0
    raw, free = ref4.append(w, layer, kc, vc, rot)
    assert torch.equal(d.raw.cpu()[~free], raw[~free]), "pool bytes"
    want = torch.full(q.shape, 7.0, dtype=T[dtype])
    for row, s, j in w.rows():
        want[row] = ref.rotate(rot, qc[row], row, j, torch.float32).to(T[dtype])
    assert torch.equal(q_out.cpu().nan_to_num(5.0), want.nan_to_num(5.0))
    return d, raw


SHAPES = [c for c in APPENDS if c[0] % 16 == 0] + [(128, 32, 8, 8, 16), (32, 32, 1, 1, 4), (48, 40, 2, 2, 7)]


@pytest.mark.parametrize("D,rd,H,Q,ps", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(D, rd, H, Q, ps, dtype, interleaved):
    for i, (lens, news) in enumerate([([9, 30, 1, 65], [1, 1, 1, 1]), ([70, 33, 0, 40], [41, 33, 0, 2])]):
        w = ref4.world(D + i, lens, news, D=D, H=H, ps=ps, gap=i == 1, tombs=i)
        rot = ref.rotation(i, rd, 80, w.n_rows, interleaved=interleaved, given=i == 1) if rd else None
        run_append(w, Q, dtype, rot, kernel_facing=i == 1, strided=0 if i else 16)


# Head sizes that leave lanes without a head, and heads of which a warp holds queries and keys.
LANES = [(96, 96, 32, 32), (96, 64, 3, 21), (160, 160, 2, 13), (192, 64, 2, 16), (224, 224, 1, 5), (128, 128, 2, 10),
         (64, 32, 3, 11)]


@pytest.mark.parametrize("D,rd,H,Q", LANES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cleared", ["none", "some", "all"])
def test_append_rounds_without_a_head_to_code(D, rd, H, Q, dtype, cleared):
    """Rounds in which lanes of a warp have queries, lanes have no head and no lane has one to code, before rounds
    in which some do; new rows of live and of cleared pages: bytes and queries as the formula has them."""
    for lens, news in (([9, 30, 1, 65], [1, 1, 1, 1]), ([70, 33, 0, 40], [41, 33, 0, 2])):
        w = ref4.world(D + Q, lens, news, D=D, H=H, ps=8)
        for s, j in ((s, j) for _, s, j in w.rows()):
            if cleared == "all" or (cleared == "some" and (s + j // 8) % 2):
                w.table[s, j // 8] = -1
        run_append(w, Q, dtype, ref.rotation(1, rd, 80, w.n_rows))


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("strided", [0, 3])
def test_append_several_axes(axes, strided):
    w = ref4.world(axes, [50, 20], [37, 3], D=64, H=2)
    for k in range(3):
        rot = ref.rotation(k, 64, 100, w.n_rows, axes=axes, interleaved=k == 1)
        run_append(w, 3, "fp16", rot, strided=strided)


@pytest.mark.parametrize("D", [64, 48])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_of_every_magnitude_and_of_values_that_are_not_finite(D, dtype):
    """Blocks of zeros, from the smallest scale to values past the largest one, borders
    between codes, NaN and infinities."""
    def change(x):
        n = x.shape[1] // 16 * 16
        b = x[:, :n].unflatten(1, (-1, 16))
        b[0] = 0
        b[1] *= torch.exp2(torch.linspace(-40, 20, b.shape[1]))[:, None].to(x.dtype)
        b[2] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0.0])
        b[3] = b[2] * torch.exp2(torch.arange(b.shape[1]) % 18 - 17.0)[:, None].to(x.dtype)
        b[4, ::3, 5] = float("nan")
        b[5, ::2, 0] = float("inf")
        b[6, 1::2, 15] = -float("inf")
        b[7, :, 3:5] = torch.tensor([-0.0, 1e-30])
        b[8] = 6e4 if dtype == "bf16" else 3e38

    w = ref4.world(3, [20, 3], [9, 3], D=D, H=2)
    run_append(w, 2, dtype, None, change=change)


def test_appended_values_against_64_bits():
    """A value is off by at most half a step: a block's scale is its largest magnitude over 6 to 3 bits, 2^-4 off at
    most and 2^-11 by its first rounding, so steps of the largest codes are 2 S <= amax / 3 * (1 + 2^-4 + 2^-10)."""
    w = ref4.world(5, [40], [40], D=128, H=2)
    rot = ref.rotation(0, 128, 64, w.n_rows)
    d, raw = run_append(w, 1, "fp32", rot)
    got = ref4.decode(w.rows_view(d.raw.cpu()).numpy(), w.H, w.D)
    x = torch.randn(w.n_rows, 5 * 128, generator=torch.Generator().manual_seed(5))
    k, v = x[:, 128:384].unflatten(1, (2, 128)), x[:, 384:].unflatten(1, (2, 128))
    for r, s, j in w.rows():
        for which, y in ((0, ref.rotate(rot, k[r], r, j, torch.float64)), (1, v[r].double())):
            b = y.view(2, -1, 16)
            amax = b.abs().amax(-1, keepdim=True)
            off = (got[ref.page_of(w, s, j), 1, which, j % 16].view(2, -1, 16) - b).abs()
            S = amax / 6 * (1 + 2.0 ** -4 + 2.0 ** -10)
            step = torch.where(b.abs() < 2 * S, 0.5, torch.where(b.abs() < 4 * S, 1.0, 2.0)) * S
            assert (off <= step / 2 * (1 + 2.0 ** -20)).all()


def test_append_queries_in_place_and_bad_positions():
    for D, strided in ((64, 0), (64, 1), (48, 0)):
        w = ref4.world(15, [30, 40], [5, 2], D=D, H=2)
        d = Dev4(w)
        rot = ref.rotation(0, D, 64, w.n_rows, given=True)
        x = torch.randn(w.n_rows, 6, D).to(torch.bfloat16)
        q = x[:, :2].contiguous().cuda()
        kv = torch.empty(w.n_rows, 4 * D + strided, dtype=torch.bfloat16, device="cuda")[:, :4 * D].unflatten(1, (4, D))
        kv.copy_(x[:, 2:])
        pos = rot.positions.clone()
        pos[0, 3], pos[0, 6] = 64, -1
        gt.kv_append_layer(d.pool, 1, d.batch, kv[:, :2], kv[:, 2:], q=q, q_out=q,
                           rotary=gt.kv_rotary(rot.table.cuda(), pos.cuda()))
        assert d.error() == gt.KV_DEV_ERR_POSITION
        raw, _ = ref4.append(w, 1, x[:, 2:4], x[:, 4:], rot)
        want, got, was = (w.rows_view(y) for y in (raw, d.raw.cpu(), w.raw))
        for r, s, j in w.rows():
            at = ref.page_of(w, s, j), 1, slice(None), j % w.ps
            out = r in (3, 6)  # that row alone is left out
            assert torch.equal(got[at], was[at] if out else want[at])
            assert torch.equal(q[r].cpu(), x[r, :2] if out else
                               ref.rotate(rot, x[r, :2], r, j, torch.float32).to(q.dtype))


# ---------------------------------------------------------------------- gather

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,H,ps", [(64, 8, 32), (128, 2, 16), (48, 2, 4), (16, 1, 1), (80, 3, 7), (128, 1, 256)])
def test_gather(dtype, D, H, ps):
    for odd, (lens, news) in enumerate([([40, 1, 90], [1, 1, 1]), ([40, 0, 90, 33], [40, 0, 57, 12])]):
        w = ref4.world(D, lens, news, D=D, H=H, ps=ps, lo=0, hi=0xFF if odd else 0xE0, tombs=3, gap=bool(odd))
        d = Dev4(w, kernel_facing=bool(odd))
        outs = [torch.full((w.n_rows, H, D), 7.0, dtype=T[dtype], device="cuda") for _ in range(2)]
        gt.kv_gather_layer_scaled(d.pool, 1, d.batch, None, *outs)
        assert d.error() == 0
        n = outs[0].numel()
        off = 16 // outs[0].element_size()  # outputs that start on 16 bytes, not on 32
        shifted = [torch.full((n + off,), 7.0, dtype=T[dtype], device="cuda")[off:].view(outs[0].shape) for _ in range(2)]
        gt.kv_gather_layer_scaled(d.pool, 1, d.batch, None, *shifted)
        assert all(torch.equal(x.nan_to_num(3.0), y.nan_to_num(3.0)) for x, y in zip(outs, shifted))
        val = w.values()
        for which in (0, 1):
            want = torch.full((w.n_rows, H, D), 7.0, dtype=torch.float64)
            for r, s, j in w.rows():
                pg = ref.page_of(w, s, j)
                want[r] = val[pg, 1, which, j % ps] if pg else 0.0
            assert (want.to(T[dtype]).double().nan_to_num(1.0) == want.nan_to_num(1.0)).all()  # six bits fit any type
            assert torch.equal(outs[which].cpu().double().nan_to_num(-9.0), want.nan_to_num(-9.0))


def test_moves_and_gathers_of_rows_carry_the_scales():
    """The byte movers of kv_pool.h on 4-bit rows: a moved token reads the same values."""
    w = ref4.world(2, [40], [40], D=128, H=1, L=2)
    d = Dev4(w)
    ids = torch.empty(2, dtype=torch.int32, device="cuda")
    src, dst = int(w.table[0, 1]) * 16 + 3, int(w.table[0, 0]) * 16 + 9
    gt.kv_translate(d.pool, torch.tensor([src, dst], device="cuda"), ids)
    gt.kv_move(d.pool, ids[:1], ids[1:])
    outs = [torch.empty(w.n_rows, 1, 128, device="cuda") for _ in range(2)]
    for layer in range(2):
        gt.kv_gather_layer_scaled(d.pool, layer, d.batch, None, *outs)
        for which in (0, 1):
            assert torch.equal(outs[which][9], outs[which][19])
            assert torch.equal(outs[which][9].cpu().double(), w.values()[int(w.table[0, 1]), layer, which, 3])
    rows = torch.empty(w.n_rows, w.R, dtype=torch.uint8, device="cuda")
    gt.kv_gather_layer(d.pool, 1, d.batch.tensors[0], d.batch.tensors[1], d.batch.tensors[2], rows, rows.clone())
    assert torch.equal(ref4.decode(rows.cpu().numpy(), 1, 128)[9], w.values()[int(w.table[0, 1]), 1, 0, 3])
    assert d.error() == 0


# ------------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("D", [64, 128])
def test_attend(dtype, lengths, D):
    w = ref4.world(len(lengths) * 7 + D, *LENGTHS[lengths], D=D, gap=lengths == "mixed")
    check_attend(w, 8, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ps", [1, 4, 7, 16, 24, 64, 256])
@pytest.mark.parametrize("lengths", ["decode", "drafts", "chunks"])
def test_attend_page_sizes(dtype, ps, lengths):
    w = ref4.world(ps, *LENGTHS[lengths], ps=ps)
    check_attend(w, 6, dtype, kernel_facing=ps % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,G", [(1, 1), (1, 71), (2, 1), (3, 5), (4, 2), (8, 8), (5, 16), (2, 17)])
def test_attend_head_layouts(dtype, H, G):
    w = ref4.world(H * 100 + G, [40, 130, 9], [1, 3, 9], H=H)
    check_attend(w, H * G, dtype)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (33, 4), (64, 70), (100, 16), (1000, 3), (5, 1000)])
@pytest.mark.parametrize("lengths", ["decode", "chunks", "drafts"])
def test_attend_window_and_sinks(window, sinks, lengths):
    w = ref4.world(window + sinks, *LENGTHS[lengths])
    check_attend(w, 4, "fp16", window=window, sinks=sinks)


@pytest.mark.parametrize("lengths", ["decode", "chunks", "drafts"])
@pytest.mark.parametrize("ps", [4, 16, 32])
def test_attend_tombstones_and_empty_rows(lengths, ps):
    w = ref4.world(5, *LENGTHS[lengths], ps=ps, tombs=12)
    w.table[0, :] = -1  # a sequence with nothing left
    check_attend(w, 4, "bf16")
    check_attend(w, 4, "bf16", window=9, sinks=2)


@pytest.mark.parametrize("D,H", [(16, 1), (48, 2), (80, 2), (96, 1), (112, 2), (192, 1), (256, 1)])
def test_attend_other_head_sizes(D, H):
    w = ref4.world(D, [1, 37, 90], [1, 2, 20], D=D, H=H)
    check_attend(w, 2 * H, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lo,hi", [(0, 8), (0, 0x30), (0xA0, 0xB0), (0x20, 0x98)])
@pytest.mark.parametrize("lengths", ["decode", "chunks"])
def test_attend_scales_far_from_one(dtype, lo, hi, lengths):
    """The smallest scale bytes (subnormal ones and zero), large ones, and a wide mix; scores kept in range by the
    queries, so that the bound on weights holds."""
    w = ref4.world(hi, *LENGTHS[lengths], lo=lo, hi=hi)
    top = float(ref4.scale_value(hi))
    check_attend(w, 4, dtype, qmul=min(1.0, 0.5 / top))


@pytest.mark.parametrize("lengths", ["decode", "chunks", "drafts"])
@pytest.mark.parametrize("byte", [0xFF, 0xE1, 0xF7])
def test_what_is_not_seen_changes_nothing(lengths, byte):
    """Blocks that read as NaN past a sequence's end, before its window, in the sink page and in cleared pages."""
    w = ref4.world(11, *LENGTHS[lengths], tombs=2)
    kw = dict(window=40, sinks=3)
    clean = check_attend(w, 4, "fp16", **kw)
    seen = torch.zeros(w.P, w.ps, dtype=torch.bool)
    for r, s, i in w.rows():
        for j in range(i + 1):
            if i - j < 40 or j < 3:
                seen[ref.page_of(w, s, j), j % w.ps] = True
    seen[0] = False
    w.scale_bytes().masked_fill_(~seen[:, None, None, :, None, None], byte)
    again = check_attend(w, 4, "fp16", **kw)
    rows = [r for r, _, _ in w.rows()]
    assert torch.equal(again[rows], clean[rows])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("news", [5, 60, 300, 700])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("byte", [0xFF, 0xE1])
def test_a_block_that_is_not_finite_reaches_every_row_that_sees_it(dtype, news, window, byte):
    """One scale of one value: NaN in its 16 elements of the rows that see it, and nowhere else."""
    n = news + 20
    w = ref4.world(13, [n], [news], D=64)
    q = torch.randn(w.n_rows, w.H, w.D, generator=torch.Generator().manual_seed(3)).to(T[dtype])
    clean = Dev4(w).attend(1, q.cuda(), 0.125, window=window)
    for at in (n - 1, n - news, n - news // 2, 7):
        bad = ref4.World4(**{**w.__dict__, "raw": w.raw.clone()})
        bad.scale_bytes()[ref.page_of(w, 0, at), 1, 1, at % w.ps, 0, 2] = byte
        out = Dev4(bad).attend(1, q.cuda(), 0.125, window=window)
        pos = torch.arange(news) + n - news
        sees = (pos >= at) & ((window == 0) | (pos - at < window))
        want = torch.zeros(out.shape, dtype=torch.bool)
        want[:news, 0, 32:48] = sees[:, None]
        assert torch.equal(out.isnan().cpu(), want)
        assert torch.equal(out[:news][~sees], clean[:news][~sees])


@pytest.mark.parametrize("news", [3, 40, 150])
def test_a_later_token_does_not_change_an_earlier_row(news):
    n = 200
    w = ref4.world(12, [n], [news], D=64)
    q = torch.randn(w.n_rows, 4, w.D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    clean = Dev4(w).attend(1, q.cuda(), 0.125)
    at = n - news // 2 - 1
    for which in (0, 1):
        bad = ref4.World4(**{**w.__dict__, "raw": w.raw.clone()})
        bad.scale_bytes()[ref.page_of(w, 0, at), 1, which, at % w.ps] = 0xFF
        out = Dev4(bad).attend(1, q.cuda(), 0.125)
        before = at - (n - news)
        assert torch.equal(out[:before], clean[:before])
        assert not out[before:].isfinite().all(-1).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attend_many_splits_and_repeatability(dtype):
    w = ref4.world(21, [5003], [1], H=1, D=128, L=1)
    out = check_attend(w, 4, dtype, layer=0)
    d = Dev4(w)
    q = torch.randn(w.n_rows, 4, 128, generator=torch.Generator().manual_seed(77)).to(T[dtype]).cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for i in range(5):
        again = d.attend(0, q, 128 ** -0.5, stream=st if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(again, out)


@pytest.mark.parametrize("lengths", ["decode", "drafts", "long", "chunks", "prompt"])
@pytest.mark.parametrize("D,ps", [(64, 16), (128, 64), (64, 24)])
def test_weights_keep_more_than_sixteen_bits(lengths, D, ps):
    """As for the other caches: two kinds of keys, values 1 and -c, balanced so
    that an error which the weights' rounding leaves shows (fp16 output).
    Half a unit of |out|, 2^-15 of the mean of |v|."""
    w = ref4.world(23, *LENGTHS[lengths], D=D, ps=ps)
    g = torch.Generator().manual_seed(4)
    kinds = torch.randn(2, w.H, D, generator=g).numpy()
    c = np.repeat(np.exp2(np.arange(D // 16) / 2.0 - 2), 16)
    pair = np.stack([np.ones(D, np.float32), -c.astype(np.float32)])
    rows = w.rows_view()
    a, nb = w.H * D // 2, w.H * D // 16
    for which, x in ((0, kinds), (1, np.broadcast_to(pair[:, None], (2, w.H, D)))):
        for kind in (0, 1):
            codes, scales, _ = ref4.encode(x[kind])
            rows[:, :, which, kind::2, :a] = torch.from_numpy(codes.reshape(-1))
            rows[:, :, which, kind::2, a:a + nb] = torch.from_numpy(scales.reshape(-1))
    d = Dev4(w)
    q = torch.randn(w.n_rows, 4 * w.H, D, generator=g).half()
    out = d.attend(1, q.cuda(), D ** -0.5).cpu().double()
    assert d.error() == 0
    want, _, size = ref.attend(w, 1, q, D ** -0.5)
    rows = [r for r, _, _ in w.rows()]
    tol = 2.0 ** -11 * want.abs() + 2.0 ** -15 * size + 2.0 ** -25
    assert (want.abs() < size / 8)[rows].any()  # some are balanced
    over = ((out - want).abs() / tol)[rows].max()
    assert over <= 1, float(over)


def test_offsets_past_32_bits():
    """A pool of 5 GiB: rows past 2^32 bytes, written, gathered and attended to."""
    w = ref4.world(4, [100, 70], [1, 40], D=128, H=8, L=2, ps=16, spare=0)
    d0 = Dev4(w)
    q = torch.randn(w.n_rows, 16, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    want = d0.attend(1, q, 0.1)
    page = 4 * 16 * w.R
    P = 5 * 2 ** 30 // page
    raw = torch.zeros((P + 1) * page, dtype=torch.uint8, device="cuda")
    pool = gt.kv_pool_create(gt.make_desc(2, 8, 128, 1, 16, P, format=gt.KV_FORMAT_E2M1), raw)
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
    back = [torch.empty_like(k) for _ in range(4)]
    gt.kv_append_layer(pool, 1, b, k, k)
    gt.kv_gather_layer_scaled(pool, 1, b, None, *back[:2])
    gt.kv_append_layer(d0.pool, 1, d0.batch, k, k)
    gt.kv_gather_layer_scaled(d0.pool, 1, d0.batch, None, *back[2:])
    assert gt.kv_pool_last_error(pool) == 0
    rows = [r for r, _, _ in w.rows()]
    for i in (0, 1):
        assert torch.equal(back[i][rows], back[i + 2][rows])


def test_device_errors_are_reported_and_harmless():
    w = ref4.world(41, [40, 50, 60], [2, 3, 20], D=64)
    q = torch.zeros(w.n_rows, 2, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.randn(w.n_rows, 2, 64, device="cuda").to(torch.bfloat16)
    back = [torch.empty_like(k) for _ in range(2)]
    calls = [lambda d: d.attend(1, q, 1.0), lambda d: gt.kv_append_layer(d.pool, 1, d.batch, k, k),
             lambda d: gt.kv_append_layer(d.pool, 1, d.batch, k.float()[:, :, :].contiguous(), k.float()),
             lambda d: gt.kv_gather_layer_scaled(d.pool, 1, d.batch, None, *back)]
    for call in calls:
        bad = ref4.World4(**{**w.__dict__, "table": w.table.copy()})
        bad.table[0, 2] = w.P + 5  # the page of the new tokens
        d = Dev4(bad)
        call(d)
        assert d.error() == gt.KV_DEV_ERR_ROW
        d = Dev4(w, kernel_facing=True)
        d.batch.tensors[0][1, 3] += 1
        call(d)
        assert d.error() == gt.KV_DEV_ERR_FORM
        for which, value in ((1, 10 ** 6), (3, -4)):
            d = Dev4(w)
            d.batch.tensors[which][1] = value
            call(d)
            assert d.error() == gt.KV_DEV_ERR_TABLE


def test_step_in_a_graph_and_on_two_streams():
    """Append, attention and gather as a step, kernel-facing; captured in a graph, and two steps with pages of
    their own on two streams at once: the same bits."""
    w = ref4.world(9, [100, 33, 70], [1, 33, 4], D=128, H=2)
    rot = ref.rotation(1, 128, 128, w.n_rows)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(w.n_rows, h, 128, generator=g).to(torch.bfloat16) for h in (8, 2, 2))
    r = gt.kv_rotary(rot.table.cuda())
    dq, dk, dv = q.cuda(), k.cuda(), v.cuda()

    class Step:
        def __init__(self):
            self.d = Dev4(w, kernel_facing=True)
            self.q, self.out = torch.empty_like(dq), torch.empty_like(dq)
            self.k, self.v = torch.empty_like(dk), torch.empty_like(dv)
            self.ws = torch.empty(gt.kv_attend_workspace_bytes(self.d.pool, 8, w.S, w.n_rows), dtype=torch.uint8,
                                  device="cuda")

        def run(self, stream=None):
            d = self.d
            gt.kv_append_layer(d.pool, 1, d.batch, dk, dv, rotary=r, q=dq, q_out=self.q, stream=stream)
            gt.kv_attend_layer(d.pool, 1, d.batch, self.q, self.out, 0.09, self.ws, stream=stream)
            gt.kv_gather_layer_scaled(d.pool, 1, d.batch, None, self.k, self.v, stream=stream)

    a = Step()
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        a.run()
    gr.replay()
    torch.cuda.synchronize()
    assert a.d.error() == 0
    raw, _ = ref4.append(w, 1, k, v, rot)
    assert torch.equal(a.d.raw.cpu(), raw)
    after = ref4.World4(**{**w.__dict__, "raw": raw})
    qr = torch.stack([ref.rotate(rot, q[r_], r_, j, torch.float32).to(q.dtype) for r_, _, j in w.rows()])
    want, _, size = ref.attend(after, 1, qr, 0.09)
    u = 2.0 ** -8
    assert ((a.out.cpu().double() - want).abs() <= u * want.abs() + (u + 2.0 ** -12) * size).all()
    val = after.values()
    for r_, s, j in w.rows():
        pg = ref.page_of(w, s, j)
        assert torch.equal(a.k[r_].cpu(), val[pg, 1, 0, j % w.ps].to(torch.bfloat16))
        assert torch.equal(a.v[r_].cpu(), val[pg, 1, 1, j % w.ps].to(torch.bfloat16))
    two = [(Step(), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for step, st in two:
            step.run(st)
    torch.cuda.synchronize()
    for step, _ in two:
        assert step.d.error() == 0
        for x, y in zip((step.q, step.out, step.k, step.v, step.d.raw), (a.q, a.out, a.k, a.v, a.d.raw)):
            assert torch.equal(x, y)


def test_refusals():
    w = ref4.world(1, [20], [2], D=64, H=4)
    d = Dev4(w)
    k = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    scales = torch.zeros(w.P * w.L * 2 * w.H, device="cuda")
    with pytest.raises(gt.KVError):
        gt.kv_scale_bytes(d.pool)  # scales lie in the rows
    with pytest.raises(ValueError):
        gt.kv_append_layer(d.pool, 0, d.batch, k, k, scales=scales)
    with pytest.raises(ValueError):
        gt.kv_gather_layer_scaled(d.pool, 0, d.batch, scales, k, k.clone())
    with pytest.raises(ValueError):
        d.scales = scales
        d.attend(0, k, 1.0)
    # the library's own checks
    p = d.batch.ptr
    x, s = k.data_ptr(), scales.data_ptr()
    L = gt.lib()
    assert L.kv_append_layer(d.pool.handle, 0, p, 1, x, 256, x, 256, None, None, 0, 0, None, s, None) == -1
    assert L.kv_gather_layer_scaled(d.pool.handle, 0, p, s, 1, x, x, None) == -1
    assert L.kv_append_layer(d.pool.handle, 0, p, 1, x + 1, 256, x, 256, None, None, 0, 0, None, None, None) == -5
    assert L.kv_gather_layer_scaled(d.pool.handle, 0, p, None, 1, x + 8, x, None) == -5
    assert d.error() == 0
