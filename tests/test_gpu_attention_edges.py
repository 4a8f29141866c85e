"""Edges of the operators of kv_attention.h on the GPU: metadata that is
inconsistent, pages that nobody sees, the ends of the scales' range, the bits
that weights keep, pools of one geometry alone, calls on two streams at once. Plain forms: attention_ref.py.
"""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_ref as ref
import gather_translate_kv_gb300 as gt
from test_gpu_attention import CACHES, LENGTHS, T, Dev, _built, check_attend  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("lengths", ["decode", "chunks", "drafts"])
@pytest.mark.parametrize("ps", [4, 16, 24, 64])
@pytest.mark.parametrize("window,sinks", [(40, 3), (7, 1), (33, 20)])
def test_pages_that_no_row_sees_are_not_read(cache, dtype, lengths, ps, window, sinks):
    """Stale entries and scales before the window and behind the first tokens:
    no error, and not a bit of the output changes."""
    w = ref.world(17 + ps, *LENGTHS[lengths], ps=ps, cache=cache)
    kf = ps % 16 == 0
    kw = dict(window=window, sinks=sinks, kernel_facing=kf)
    clean = check_attend(w, 4, dtype, **kw)
    seen = np.zeros(w.table.shape, dtype=bool)
    for _, s, i in w.rows():
        for j in range(i + 1):
            if i - j < window or j < sinks:
                seen[s, j // ps] = True
    held = np.arange(w.table.shape[1])[None] < [[-(-n // ps)] for n in w.lens]
    rows = [r for r, _, _ in w.rows()]
    if cache == "e4m3":
        for k, scale in enumerate((0.0, float("nan"))):
            was = w.scales.clone()
            w.scales[torch.from_numpy(w.table[held & ~seen]).long()] = scale
            assert torch.equal(check_attend(w, 4, dtype, **kw)[rows], clean[rows]), scale
            w.scales = was
    w.table[held & ~seen] = 0x7FFFFFF1  # past the pool, and off the kernel-facing grid
    again = check_attend(w, 4, dtype, **kw)
    assert torch.equal(again[rows], clean[rows])


# ------------------------------------------------- metadata that is inconsistent

# lens, news of three sequences whose runs are numbered by row, and by page
BY = {"row": ([40, 70, 33], [1, 1, 1]), "page": ([40, 70, 33], [25, 30, 20])}


def broken(kind, by, *, D=64, cache="bf16", seed=1):
    """A batch with one inconsistent sequence, the World of what is left of it
    (that sequence without new tokens), and the error bit that it has to set."""
    lens, news = BY[by]
    lost = {"no span": 1, "outside": 2, "short span": 0, "start": 1, "len": 1, "backwards": 2}[kind]
    kept = [0 if s == lost else n for s, n in enumerate(news)]
    w = ref.world(seed, lens, kept, D=D, cache=cache)
    d = Dev(w)
    start = [n - m for n, m in zip(lens, news)]
    lens = list(lens)
    if kind in ("short span", "start", "len"):  # its rows are there
        w.gap[lost] = news[lost]
    cu = w.cu.tolist()
    if kind == "short span":
        start[0] -= 1
    elif kind == "start":
        start[1] = -2
    elif kind == "len":
        lens[1] = w.table.shape[1] * w.ps + 1
    elif kind == "outside":  # all rows past the tensors
        cu[3] = w.n_rows + news[2]
    elif kind == "backwards":  # the span ends before it begins
        cu[3] = w.n_rows - 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    d.batch = gt.kv_batch(torch.from_numpy(w.table).cuda(), i32(lens), torch.tensor(cu, device="cuda"), w.n_rows,
                          seq_start=i32(start))
    return w, d


KINDS = ["no span", "outside", "short span", "start", "len", "backwards"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("by", list(BY))
@pytest.mark.parametrize("D", [64, 24])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_append_reports_an_inconsistent_sequence(kind, by, D, cache):
    """KV_DEV_ERR_TABLE is set, nothing of that sequence is written, and the others are stored."""
    w, d = broken(kind, by, D=D, cache=cache)
    g = torch.Generator().manual_seed(2)
    k, v, q = (torch.randn(w.n_rows, w.H, D, generator=g).to(torch.bfloat16) for _ in range(3))
    q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    gt.kv_append_layer(d.pool, 1, d.batch, k.cuda(), v.cuda(), q=q.cuda(), q_out=q_out, scales=d.scales)
    assert d.error() == gt.KV_DEV_ERR_TABLE
    raw, scales = ref.append(w, 1, k, v, None)
    assert torch.equal(d.raw.cpu(), raw)
    if scales is not None:
        assert torch.equal(d.scales.cpu(), scales)
    want = torch.full(q.shape, 7.0, dtype=torch.bfloat16)
    for r, _, _ in w.rows():
        want[r] = q[r]
    assert torch.equal(q_out.cpu(), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("by", list(BY))
def test_scaled_gather_reports_an_inconsistent_sequence(kind, by):
    w, d = broken(kind, by, cache="e4m3")
    outs = [torch.full((w.n_rows, w.H, w.D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gt.kv_gather_layer_scaled(d.pool, 1, d.batch, d.scales, *outs)
    assert d.error() == gt.KV_DEV_ERR_TABLE
    val = w.values()
    for which in (0, 1):
        want = torch.full(outs[0].shape, 7.0, dtype=torch.bfloat16)
        for r, s, j in w.rows():
            want[r] = val[ref.page_of(w, s, j), 1, which, j % w.ps].to(torch.bfloat16)
        assert torch.equal(outs[which].cpu(), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("by", list(BY))
@pytest.mark.parametrize("D", [64, 80])
def test_attention_reports_an_inconsistent_sequence(kind, by, D):
    w, d = broken(kind, by, D=D)
    q = torch.randn(w.n_rows, 4, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out = d.attend(1, q.cuda(), 0.125).cpu().double()
    assert d.error() == gt.KV_DEV_ERR_TABLE
    want, _, size = ref.attend(w, 1, q, 0.125)
    rows = [r for r, _, _ in w.rows()]
    rest = sorted(set(range(w.n_rows)) - set(rows))
    assert (out[rest] == 7.0).all()
    u = 2.0 ** -8
    assert ((out - want).abs() <= u * want.abs() + (u + 2.0 ** -12) * size)[rows].all()


@pytest.mark.parametrize("by", list(BY))
@pytest.mark.parametrize("D", [64, 24])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("entry", ["past the pool", "off the grid"])
def test_append_and_gather_report_bad_entries(by, D, cache, entry):
    """A bad entry counts as a tombstone: its tokens alone are not stored, and are read as zeros."""
    lens, news = BY[by]
    w = ref.world(3, lens, news, D=D, cache=cache)
    kf = entry == "off the grid"
    d = Dev(w, kernel_facing=kf)
    page = (lens[1] - 1) // w.ps
    d.batch.tensors[0][1, page] = int(w.table[1, page]) * 2 * w.L + 1 if kf else w.P
    bit = gt.KV_DEV_ERR_FORM if kf else gt.KV_DEV_ERR_ROW
    w.table[1, page] = 0
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(w.n_rows, w.H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    gt.kv_append_layer(d.pool, 1, d.batch, k.cuda(), v.cuda(), scales=d.scales)
    assert d.error() == bit
    raw, scales = ref.append(w, 1, k, v, None)
    assert torch.equal(d.raw.cpu(), raw)
    if cache != "e4m3":
        return
    assert torch.equal(d.scales.cpu(), scales)
    outs = [torch.full(k.shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gt.kv_gather_layer_scaled(d.pool, 1, d.batch, d.scales, *outs)
    assert d.error() == bit
    val = w.values(raw, scales)
    for which in (0, 1):
        for r, s, j in w.rows():
            pg = ref.page_of(w, s, j)
            want = val[pg, 1, which, j % w.ps] if pg else torch.zeros(w.H, D, dtype=torch.float64)
            assert torch.equal(outs[which][r].cpu(), want.to(torch.bfloat16))


@pytest.mark.parametrize("lengths", ["decode", "chunks", "long"])
@pytest.mark.parametrize("ps", [16, 24])
@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -122, 2.0 ** -118, 2.0 ** -115, 2.0 ** -112, 1.5 * 2.0 ** 126])
def test_value_scales_at_the_ends_of_their_range(lengths, ps, scale):
    """Denominators (weights over scales) and 1 / scale near both ends of the 32-bit range."""
    w = ref.world(19, *LENGTHS[lengths], ps=ps, cache="e4m3")
    w.scales[:, :, 1] = scale
    if scale > 1:  # codes of 1, 1/2 and their negatives, so that the values are finite
        codes = torch.tensor([0x38, 0x30, 0xB8, 0xB0], dtype=torch.uint8)
        v = w.view().view(torch.uint8)[:, :, 1]
        v.copy_(codes[(v & 3).long()])
    check_attend(w, 4, "bf16")


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("lengths", ["decode", "drafts", "long", "chunks", "prompt"])
@pytest.mark.parametrize("D,ps", [(64, 16), (128, 64), (64, 24)])
def test_weights_keep_more_than_sixteen_bits(cache, dtype, lengths, D, ps):
    """Two kinds of keys, a and b, with values 1 and -c: where c balances the
    two, what is left is small beside the values, and an error that the
    rounding of the weights leaves is not hidden by the output's own rounding.

    Bounds. Half a unit of the output (2^-8 bf16, 2^-11 fp16) of |out|; the
    weights meet the values as two 16-bit parts, 2^-16 relative at most; the
    exponents are sums of 32-bit products of total magnitude below 16, in
    steps of 16, and leave 2^-16 at most: 2^-15 of the mean of |v|.
    """
    w = ref.world(23, *LENGTHS[lengths], D=D, ps=ps, cache=cache)
    g = torch.Generator().manual_seed(4)
    kinds = torch.randn(2, w.H, D, generator=g)
    c = 2.0 ** (torch.arange(D) / (D / 8) - 4.0)  # a factor of 256 in steps of 2^(8 / D)
    v = w.view()
    first = torch.arange(w.ps) % 2 == 0
    pair = torch.stack([torch.ones(D), -c])  # values of the two kinds
    scale = 1.0
    if cache == "e4m3":
        w.scales[:] = 2.0 ** -4
        scale = 2.0 ** 4
    for which, x in ((0, kinds), (1, pair[:, None].expand(2, w.H, D))):
        v[:, :, which] = torch.where(first[:, None, None], x[0] * scale, x[1] * scale).to(v.dtype)
    d = Dev(w)
    q = torch.randn(w.n_rows, 4 * w.H, D, generator=g).to(T[dtype])
    out = d.attend(1, q.cuda(), D ** -0.5).cpu().double()
    assert d.error() == 0
    want, _, size = ref.attend(w, 1, q, D ** -0.5)
    rows = [r for r, _, _ in w.rows()]
    u = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[dtype]
    tol = u * want.abs() + 2.0 ** -15 * size + 2.0 ** -25
    assert (want.abs() < size / 8)[rows].any()  # some are balanced
    over = ((out - want).abs() / tol)[rows].max()
    assert over <= 1, float(over)


STEP = """
import sys, torch
sys.path[:0] = sys.argv[1:3]
import attention_ref as ref
from test_gpu_attention import check_attend, run_append
D, ps, cache, dtype = int(sys.argv[3]), int(sys.argv[4]), sys.argv[5], sys.argv[6]
w = ref.world(1, [40, 150], [1, 100], D=D, ps=ps, cache=cache)
if dtype != "fp32":  # attention takes 16-bit rows
    check_attend(w, 8, dtype)
    check_attend(ref.world(2, [40, 150], [1, 2], D=D, ps=ps, cache=cache), 32, dtype)
run_append(w, 4, dtype, None)
print("done")
"""


def test_a_pool_prepares_the_kernels_of_its_own_geometry():
    """A process whose only pool is of one geometry can call everything on it."""
    here = os.path.dirname(os.path.abspath(__file__))
    cases = [(D, ps, c, t) for D in (64, 128) for ps in (16, 24) for c, t in (("e4m3", "bf16"), ("e4m3", "fp16"))]
    cases += [(D, 16, c, c) for D in (64, 128) for c in ("bf16", "fp16", "fp32")] + [(16, 16, "e4m3", "fp32")]
    for at in range(0, len(cases), 5):
        run = [(c, subprocess.Popen([sys.executable, "-c", STEP, here, os.path.dirname(here), *map(str, c)],
                                    stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
               for c in cases[at:at + 5]]
        for c, p in run:
            out, _ = p.communicate(timeout=300)
            assert p.returncode == 0 and out.endswith("done\n"), (c, out)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_two_streams_at_once(cache):
    """Steps on two streams with pages, tensors and workspaces of their own,
    nothing awaited in between: the same bits as one after the other."""
    lens, news = [900, 64, 300, 1300], [1, 40, 300, 3]
    w = ref.world(29, lens, news, D=128, cache=cache)
    rot = ref.rotation(1, 128, 2048, w.n_rows)
    g = torch.Generator().manual_seed(3)
    rows = [(int(w.cu[s]), int(w.cu[s + 1])) for s in range(4)]
    x = torch.randn(w.n_rows, 12, 128, generator=g).to(torch.bfloat16).cuda()
    both = ((0, 1), (2, 3))

    def run(streams):
        d = Dev(w)
        r = gt.kv_rotary(rot.table.cuda())
        parts = []
        for seqs in both:
            a, b = rows[seqs[0]][0], rows[seqs[1]][1]
            n = b - a
            i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
            ls = [w.lens[s] for s in seqs]
            ns = [w.news[s] for s in seqs]
            batch = gt.kv_batch(torch.from_numpy(w.table[list(seqs)]).cuda(), i32(ls),
                                torch.tensor([0, ns[0], n], device="cuda"), n,
                                seq_start=i32([p - m for p, m in zip(ls, ns)]))
            ws = torch.empty(gt.kv_attend_workspace_bytes(d.pool, 8, 2, n), dtype=torch.uint8, device="cuda")
            q, k, v = (y.contiguous() for y in x[a:b].split([8, 2, 2], 1))
            q_out, out = torch.empty_like(q), torch.empty_like(q)
            back = [torch.empty(n, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            parts.append((batch, ws, q, k, v, q_out, out, back))
        torch.cuda.synchronize()
        for layer in (0, 1) * 8:
            for (batch, ws, q, k, v, q_out, out, back), st in zip(parts, streams):
                gt.kv_append_layer(d.pool, layer, batch, k, v, rotary=r, q=q, q_out=q_out, scales=d.scales, stream=st)
                gt.kv_attend_layer(d.pool, layer, batch, q_out, out, 0.09, ws, scales=d.scales, stream=st)
                if cache == "e4m3":
                    gt.kv_gather_layer_scaled(d.pool, layer, batch, d.scales, *back, stream=st)
                if streams[0] is streams[1]:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert d.error() == 0
        done = [t.clone() for p in parts for t in (p[5], p[6], *(p[7] if cache == "e4m3" else ()))]
        return done + [d.raw] + ([d.scales] if cache == "e4m3" else [])

    one = torch.cuda.Stream()
    want = run((one, one))
    for _ in range(3):
        got = run((torch.cuda.Stream(), torch.cuda.Stream()))
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
