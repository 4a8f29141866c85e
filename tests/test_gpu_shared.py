"""Attention of sequences that share prefixes (kv_attend_shared_layer) on the
GPU, against the plain 64-bit form of attention_ref.py, which knows of no
sharing. Bounds as for kv_attend_layer (test_gpu_attention.py, test_gpu_cache4.py): joining
two sums in 32 bits adds 2^-22 of the mean of |v|, which the 2^-12 of the scores cover.
"""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_ref as ref
import cache4_ref as ref4
import gather_translate_kv_gb300 as gt
from test_gpu_attention import T, U, Dev, _built  # noqa: F401 (fixture)
from test_gpu_cache4 import Dev4

pytestmark = pytest.mark.gpu

CACHES = [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16"), ("e2m1", "bf16"), ("e2m1", "fp16")]

# groups: (prefix, [(own tokens, new tokens), ...])
GROUPS = {
    "one": [(64, [(1, 1), (1, 1)])],
    "decode": [(200, [(1, 1), (17, 1), (64, 1), (5, 1)]), (0, [(40, 1)]), (33, [(3, 1), (9, 1), (1, 1)])],
    "long": [(1500, [(3, 1), (40, 1)])],
    "drafts": [(130, [(5, 3), (9, 4), (2, 1), (30, 5)]), (16, [(9, 2), (4, 4)])],
    "many": [(300, [(1 + 7 * i % 50, 1 + i % 2) for i in range(40)]), (150, [(4, 1)] * 9)],
    "mixed": [(100, [(30, 1), (0, 0), (3, 3)]), (50, [(0, 0), (7, 7)]), (48, [(0, 0), (0, 0)]), (15, [(4, 1), (4, 2)])],
    "alone": [(100, [(5, 1)]), (70, [(6, 2)]), (0, [(3, 1)])],
    "chunks": [(260, [(40, 40), (70, 33), (90, 20)])],
}


class Shared:
    """A World whose groups share their first tokens: whole pages by the table, the
    rest of the last one by its contents."""

    def __init__(self, seed, groups, cache, *, gap=False, wide=True, **kw):
        lens = [p + a for p, members in groups for a, _ in members]
        news = [n for _, members in groups for _, n in members]
        w = ref4.world(seed, lens, news, gap=gap, **kw) if cache == "e2m1" else ref.world(seed, lens, news, cache=cache,
                                                                                        gap=gap, **kw)
        self.w, self.cache = w, cache
        self.group, self.prefix = [0], []
        for p, members in groups:
            s0 = self.group[-1]
            full = p // w.ps
            for s in range(s0 + 1, s0 + len(members)):
                w.table[s, :full] = w.table[s0, :full]
                if p % w.ps:
                    a, b = int(w.table[s0, full]), int(w.table[s, full])
                    view = w.rows_view() if cache == "e2m1" else w.view()
                    view[b, :, :, : p % w.ps] = view[a, :, :, : p % w.ps]
                    if w.scales is not None:
                        w.scales[b] = w.scales[a]
            self.group.append(s0 + len(members))
            self.prefix.append(p)
        if wide and w.S > len(groups):
            # tables so wide that the batch may be far larger than the caches: sharing pays, as far as the host can tell
            pages = -(-2 ** 28 // ((w.S - len(groups)) * w.H * w.D * 2 * w.ps))
            if pages > w.table.shape[1]:
                fill = np.full((w.S, pages - w.table.shape[1]), 0x7ffffff0, dtype=np.int32)  # never read
                w.table = np.concatenate([w.table, fill], 1)

    def dev(self, kernel_facing=False):
        return (Dev4 if self.cache == "e2m1" else Dev)(self.w, kernel_facing)

    def groups(self, group=None, prefix=None):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return gt.kv_prefix_groups(i32(self.group if group is None else group),
                                   i32(self.prefix if prefix is None else prefix))


def attend(d, groups, layer, q, scale, lse=None, stream=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    ws = torch.full((gt.kv_attend_shared_workspace_bytes(d.pool, q.shape[1], d.w.S, d.w.n_rows),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    gt.kv_attend_shared_layer(d.pool, layer, d.batch, groups, q, out, scale, ws, scales=d.scales, lse=lse, stream=stream)
    return out


def queries(w, Q, dtype, seed=0):
    return torch.randn(w.n_rows, Q, w.D, generator=torch.Generator().manual_seed(seed + 77)).to(T[dtype])


def check(sh, Q, dtype, *, layer=1, kernel_facing=False, group=None, prefix=None, error=0):
    w = sh.w
    d = sh.dev(kernel_facing)
    q = queries(w, Q, dtype)
    lse = torch.full((w.n_rows, Q), 7.0, device="cuda")
    out = attend(d, sh.groups(group, prefix), layer, q.cuda(), w.D ** -0.5, lse=lse)
    assert d.error() == error
    want, wlse, size = ref.attend(w, layer, q, w.D ** -0.5)
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


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("D", [64, 128])
def test_shared(cache, dtype, groups, D):
    check(Shared(len(groups) + D, GROUPS[groups], cache, D=D, gap=groups in ("mixed", "many")), 8, dtype)


@pytest.mark.parametrize("cache,dtype", CACHES[:5:2])
@pytest.mark.parametrize("groups", list(GROUPS))
def test_shared_in_narrow_tables(cache, dtype, groups):
    """Batches that are too small for sharing to pay."""
    check(Shared(3, GROUPS[groups], cache, wide=False), 8, dtype)


@pytest.mark.parametrize("cache,dtype", CACHES[1::2])
@pytest.mark.parametrize("ps", [1, 4, 7, 16, 24, 64, 256])
@pytest.mark.parametrize("groups", ["decode", "drafts", "many"])
def test_shared_page_sizes(cache, dtype, ps, groups):
    check(Shared(ps, GROUPS[groups], cache, ps=ps), 6, dtype, kernel_facing=ps % 2 == 0)


@pytest.mark.parametrize("cache,dtype", [CACHES[0], CACHES[3], CACHES[4]])
@pytest.mark.parametrize("H,G", [(1, 1), (1, 71), (2, 1), (3, 5), (4, 2), (8, 8), (5, 16), (2, 17)])
def test_shared_head_layouts(cache, dtype, H, G):
    D = 128 if cache == "e2m1" and H % 2 else 64
    check(Shared(H * 100 + G, [(70, [(4, 1), (9, 2), (3, 3)]), (20, [(5, 1), (1, 1)])], cache, H=H, D=D), H * G, dtype)


@pytest.mark.parametrize("cache,dtype", [CACHES[0], CACHES[2], CACHES[5]])
@pytest.mark.parametrize("D", [16, 48, 80, 256])
def test_shared_other_head_sizes(cache, dtype, D):
    check(Shared(D, GROUPS["drafts"], cache, D=D, H=1), 2, dtype)


@pytest.mark.parametrize("cache,dtype", CACHES[::2])
def test_shared_tombstones(cache, dtype):
    """Cleared pages in a prefix, a prefix that is cleared whole, own pages that are."""
    sh = Shared(5, [(200, [(9, 1), (40, 3), (3, 1)]), (64, [(5, 1), (4, 4)]), (96, [(9, 1), (20, 2)])], cache)
    w = sh.w
    w.table[0:3, 3] = -1
    w.table[0:3, 7] = 0
    w.table[3:5, :4] = -1
    w.table[5, 6] = -1   # nothing of its own
    check(sh, 4, dtype)
    w.table[5:7, :8] = -1  # nothing at all
    check(sh, 4, dtype)


def test_shared_prefixes_that_reach_into_new_tokens():
    """A prefix counts up to the members' first new token, in steps of 16 tokens; a negative one shares nothing."""
    sh = Shared(6, GROUPS["drafts"], "bf16")
    check(sh, 4, "bf16", prefix=[1000, 2 ** 31 - 1])
    check(sh, 4, "bf16", prefix=[-5, 0])
    check(sh, 4, "bf16", prefix=[17, 15])
    check(sh, 4, "bf16", group=[0, 0, 4, 4, 6], prefix=[7, 130, 9, 16])  # empty groups


@pytest.mark.parametrize("group", [[0, 4, 5], [1, 4, 6], [0, 7, 6], [0, -1, 6], [0, 4, 2 ** 31 - 1]])
def test_shared_groups_that_are_no_groups(group):
    """An error bit, and the answer of a batch that shares nothing."""
    sh = Shared(7, GROUPS["drafts"], "bf16")
    check(sh, 4, "bf16", group=group, error=gt.KV_DEV_ERR_TABLE)


@pytest.mark.parametrize("cache,dtype", [CACHES[0], CACHES[2], CACHES[4]])
@pytest.mark.parametrize("group", [[0, 4, 5], [1, 4, 6], [0, 7, 6], [0, -1, 6], [0, 4, 2 ** 31 - 1], [0, 1, 2, 3, 4, 5, 5]])
@pytest.mark.parametrize("D,H,Q", [(64, 2, 4), (128, 1, 17), (128, 1, 33), (80, 2, 4)])
@pytest.mark.parametrize("most", [32, 130])
def test_shared_groups_that_are_no_groups_where_nothing_is_shared(cache, dtype, group, D, H, Q, most):
    """Batches that are too small for sharing to pay, and head sizes that never share: the error bit all the same, whichever
    kernels take the rows (few rows of 2 heads, in one piece or cut; too many rows of one head's 17 or 33 query heads; row
    by row)."""
    news = 1 if D == 64 else 9
    sh = Shared(7, [(most, [(9, news), (10, news), (11, news), (30, news)]), (16, [(9, news), (14, news)])], cache, D=D, H=H,
                wide=False)
    check(sh, Q, dtype, group=group, prefix=[16] * (len(group) - 1), error=gt.KV_DEV_ERR_TABLE)
    check(sh, Q, dtype, group=[0, 0, 1, 6], prefix=[16, 16, 0])


@pytest.mark.parametrize("cache,dtype", [CACHES[0], CACHES[2], CACHES[4]])
@pytest.mark.parametrize("members", [3, 40])
def test_shared_value_that_is_not_finite(cache, dtype, members):
    """One element (or block) of one value of a prefix: NaN for every row of its group, there and nowhere else."""
    sh = Shared(13, [(150, [(5, 1)] * members), (64, [(4, 2), (6, 1)])], cache)
    w = sh.w
    q = queries(w, w.H, dtype)
    clean = attend(sh.dev(), sh.groups(), 1, q.cuda(), 0.125)
    for at in (0, 77, 143, 149):  # the last: the tokens past a multiple of 16
        keep = w.raw.clone()
        for s in {0} if at < 144 else range(members):
            pg, off = int(w.table[s, at // w.ps]), at % w.ps
            if cache == "e4m3":
                w.view().view(torch.uint8)[pg, 1, 1, off, 0, 9] = 0x7F
            elif cache == "e2m1":
                w.scale_bytes()[pg, 1, 1, off, 0, 0] = 0xFF
            else:
                w.view()[pg, 1, 1, off, 0, 9] = float("nan")
        out = attend(sh.dev(), sh.groups(), 1, q.cuda(), 0.125)
        want = torch.zeros(out.shape, dtype=torch.bool)
        want[:members, 0, slice(0, 16) if cache == "e2m1" else 9] = True
        assert torch.equal(out.isnan().cpu(), want)
        rest = ~want.any(-1).cuda()
        assert torch.equal(out[rest], clean[rest])
        w.raw = keep


@pytest.mark.parametrize("cache,dtype", [CACHES[0], CACHES[3], CACHES[4]])
@pytest.mark.parametrize("which", [0, 1])
def test_shared_infinite_keys_and_values(cache, dtype, which):
    """Whatever is not finite in a prefix gives what kv_attend_layer gives."""
    sh = Shared(14, [(160, [(5, 1)] * 5)], cache)
    w = sh.w
    pg = int(w.table[0, 3])
    if cache == "e4m3":
        w.view().view(torch.uint8)[pg, 1, which, 5] = 0x7F
    elif cache == "e2m1":
        w.scale_bytes()[pg, 1, which, 5] = 0xE1
    else:
        w.view()[pg, 1, which, 5] = float("inf")
    q = queries(w, 4, dtype).cuda()
    d = sh.dev()
    got, want = attend(d, sh.groups(), 1, q, 0.125), d.attend(1, q, 0.125)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    assert got.isfinite().logical_not().any()


def test_shared_inconsistent_members():
    """A member whose metadata is inconsistent takes no part; the others keep their prefix."""
    for which, at, value in ((1, 1, 10 ** 6), (3, 1, -4), (3, 0, -1), (1, 3, -1)):
        sh = Shared(8, [(80, [(4, 2)] * 4), (32, [(5, 1), (7, 2)])], "bf16")
        w = sh.w
        d = sh.dev()
        q = queries(w, 4, "bf16")
        d.batch.tensors[which][at] = value
        out = attend(d, sh.groups(), 1, q.cuda(), 0.125).cpu().double()
        assert d.error() == (gt.KV_DEV_ERR_TABLE if value != -1 or which == 3 else 0)
        want, _, size = ref.attend(w, 1, q, 0.125)
        gone = list(range(2 * at, 2 * at + 2))
        rows = [r for r, _, _ in w.rows() if r not in gone]
        assert (out[gone] == 7.0).all()
        assert ((out - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * size)[rows].all()


@pytest.mark.parametrize("cache,dtype", [CACHES[0], CACHES[2], CACHES[4]])
@pytest.mark.parametrize("entry,value", [(4, 10), (5, 50), (6, 20), (7, 30)])
def test_shared_rows_that_step_back(cache, dtype, entry, value):
    """One entry of the rows' offsets that decreases, so that the next sequence's rows lie between those of another
    group: the sequence before it takes no part, every other one keeps its own answer."""
    sh = Shared(18, [(96, [(9, 4), (20, 4), (5, 4)]), (48, [(7, 4), (4, 4), (30, 4)]), (64, [(4, 4), (33, 4), (5, 4)])],
                cache)
    w = sh.w
    w.gap = [0, 92, 0] + [0] * 6
    cu = w.cu
    cu[entry] = value
    d = sh.dev()
    d.batch.tensors[2].copy_(torch.from_numpy(cu))
    q = queries(w, 4, dtype)
    u = U[T[dtype]]
    for _ in range(3):
        out = attend(d, sh.groups(), 1, q.cuda(), 0.125).cpu().double()
        assert d.error() == gt.KV_DEV_ERR_TABLE
        tokens = set()
        for s in range(w.S):
            a, b = int(cu[s]), int(cu[s]) + w.news[s]
            if cu[s + 1] < b:
                assert s == entry - 1
                continue
            tokens |= set(range(a, b))
            one = type(w)(**{**w.__dict__, "lens": [w.lens[s]], "news": [w.news[s]], "gap": [0],
                             "table": w.table[s:s + 1]})
            want, _, size = ref.attend(one, 1, q[a:b], 0.125)
            assert ((out[a:b] - want).abs() <= u * want.abs() + (u + 2.0 ** -12) * size).all(), s
        assert (out[sorted(set(range(w.n_rows)) - tokens)] == 7.0).all()


def test_shared_bad_entries():
    sh = Shared(9, [(80, [(4, 2)] * 4), (32, [(5, 1), (7, 2)])], "bf16")
    w = sh.w
    w.table[0:4, 2] = w.P + 9  # a page of the prefix past the pool: its tokens drop out
    d = sh.dev()
    q = queries(w, 4, "bf16")
    out = attend(d, sh.groups(), 1, q.cuda(), 0.125).cpu().double()
    assert d.error() == gt.KV_DEV_ERR_ROW
    w.table[0:4, 2] = 0
    want, _, size = ref.attend(w, 1, q, 0.125)
    assert ((out - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * size).all()
    d = sh.dev(kernel_facing=True)
    d.batch.tensors[0][0:4, 1] += 1
    attend(d, sh.groups(), 1, q.cuda(), 0.125)
    assert d.error() == gt.KV_DEV_ERR_FORM


@pytest.mark.parametrize("cache,dtype", [CACHES[0], CACHES[2], CACHES[4]])
def test_shared_repeats_bit_for_bit(cache, dtype):
    """Long prefixes that are cut over the whole GPU, in both kernels; twice on one
    workspace, in a graph, and two calls at once on two streams: the same bits."""
    sh = Shared(10, [(3007, [(9 + i, 1) for i in range(50)]), (2005, [(40, 1), (3, 1), (700, 2)])], cache, D=128, H=2,
                L=2)
    w = sh.w
    want = check(sh, 8, dtype)
    d, groups = sh.dev(), sh.groups()
    q = queries(w, 8, dtype).cuda()
    size = gt.kv_attend_shared_workspace_bytes(d.pool, 8, w.S, w.n_rows)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.full_like(q, 7.0) for _ in range(2)]
    call = lambda i, st=None: gt.kv_attend_shared_layer(d.pool, 1, d.batch, groups, q, outs[i], 128 ** -0.5,  # noqa: E731
                                                        ws[i], scales=d.scales, stream=st)
    for _ in range(3):
        call(0)
    assert torch.equal(outs[0], want)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call(1)
        call(1)
    for _ in range(3):
        outs[1].fill_(7.0)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[1], want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for o in outs:
        o.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(10):
        for i in (0, 1):
            call(i, streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert d.error() == 0


def test_shared_workspace_on_sixteen_bytes():
    sh = Shared(11, GROUPS["many"], "bf16", D=128)
    d, w = sh.dev(), sh.w
    q = queries(w, 8, "bf16").cuda()
    want = attend(d, sh.groups(), 1, q, 0.1)
    size = gt.kv_attend_shared_workspace_bytes(d.pool, 8, w.S, w.n_rows)
    for off in (16, 48, 240):
        ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")[off:off + size]
        assert ws.data_ptr() % 32 == off % 32
        out = torch.empty_like(q)
        gt.kv_attend_shared_layer(d.pool, 1, d.batch, sh.groups(), q, out, 0.1, ws)
        rows = [r for r, _, _ in w.rows()]
        assert torch.equal(out[rows], want[rows])
    assert d.error() == 0


@pytest.mark.parametrize("cache,dtype", [CACHES[0], CACHES[4]])
def test_shared_by_thousands(cache, dtype):
    """A group of thousands of sequences and groups of two, in tables so narrow that units are not cut: against
    kv_attend_layer, twice that one's bound."""
    g = [(128, [(1 + 7 * i % 90, 1) for i in range(3000)])] + [(16 + 16 * (i % 5), [(3, 1), (40, 2)]) for i in range(700)]
    sh = Shared(17, g, cache, wide=False, H=2, D=128, L=2)
    w = sh.w
    assert (w.S - len(g)) * w.table.shape[1] * w.ps * w.H * w.D * 2 >= 2 ** 28
    d = sh.dev()
    q = queries(w, 4, dtype).cuda()
    got, want = attend(d, sh.groups(), 1, q, 128 ** -0.5), d.attend(1, q, 128 ** -0.5)
    assert d.error() == 0
    top = {"bf16": 6.0, "fp16": 6.0, "e4m3": 448 * 2.0 ** -5, "e2m1": 6.0}[cache]  # of |v|: the bound's mean is below it
    u = U[T[dtype]]
    assert ((got.double() - want.double()).abs() <= 2 * (u * want.double().abs() + (u + 2.0 ** -12) * top)).all()
    # and a few rows against the formula
    for s in (0, 1501, 2999, 3000, 4399):
        one = type(w)(**{**w.__dict__, "lens": [w.lens[s]], "news": [w.news[s]], "gap": [0], "table": w.table[s:s + 1]})
        a, b = int(w.cu[s]), int(w.cu[s]) + w.news[s]
        ref_out, _, size = ref.attend(one, 1, q[a:b].cpu(), 128 ** -0.5)
        assert ((got[a:b].cpu().double() - ref_out).abs() <= u * ref_out.abs() + (u + 2.0 ** -12) * size + 2.0 ** -24).all()


FIRST = """
import sys
sys.path[:0] = {path!r}
import threading
import torch
import gather_translate_kv_gb300 as gt
from test_gpu_shared import GROUPS, Shared, attend, check, queries
sh = Shared(19, GROUPS["many"], {cache!r}, D=128)
w, q = sh.w, queries(sh.w, 8, "bf16").cuda()
first = sh.dev()
size = gt.kv_attend_workspace_bytes(first.pool, 8, w.S, w.n_rows) + (64 << 20) + w.n_rows * 8 * 130 * 4
ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
outs = [torch.full_like(q, 7.0) for _ in range(3)]
groups, devs = sh.groups(), [sh.dev() for _ in range(3)]
call = lambda i, st=None: gt.kv_attend_shared_layer(devs[i].pool, 1, devs[i].batch, groups, q, outs[i], 128 ** -0.5, ws[i],
                                                    scales=devs[i].scales, stream=st)
torch.cuda.synchronize()
if {how!r} == "captured":
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
        call(1)
        call(2)
    assert all((o == 7.0).all() for o in outs)
    graph.replay()
else:
    streams = [torch.cuda.Stream() for _ in range(3)]
    at = [threading.Thread(target=call, args=(i, streams[i])) for i in range(3)]
    [x.start() for x in at]
    [x.join() for x in at]
torch.cuda.synchronize()
want = check(sh, 8, "bf16")
assert all(torch.equal(o, want) for o in outs) and all(d.error() == 0 for d in devs)
print("done")
"""


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("how", ["captured", "threads"])
def test_shared_first_calls_of_a_process(cache, how):
    """A pool sets up its kernels at its first shared call, or when it is asked for the workspace: without having been
    asked, the first calls of a process while a stream is captured, and from three threads at once."""
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST.format(path=[os.path.dirname(here), here], cache=cache, how=how)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stdout[-2000:] + r.stderr[-2000:]


def test_shared_strided_queries():
    sh = Shared(11, GROUPS["many"], "bf16", D=128)
    d, w = sh.dev(), sh.w
    wide = torch.randn(w.n_rows, 4 * 128 + 41, device="cuda").to(torch.bfloat16)
    for x in (wide[:, 8:520], wide[:, 3:515]):
        q = x.unflatten(1, (4, 128))
        assert torch.equal(attend(d, sh.groups(), 1, q, 0.1), attend(d, sh.groups(), 1, q.contiguous(), 0.1))


def test_shared_step():
    """Decode steps behind a shared prompt as a serving loop runs them, in a 4-bit pool: append, shared attention."""
    sh = Shared(12, [(96, [(1 + i, 1) for i in range(6)])], "e2m1", D=128, H=2)
    w = sh.w
    rot = ref.rotation(1, 128, 128, w.n_rows)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(w.n_rows, h, 128, generator=g).to(torch.bfloat16) for h in (8, 2, 2))
    d = sh.dev(kernel_facing=True)
    dq = torch.empty_like(q, device="cuda")
    gt.kv_append_layer(d.pool, 1, d.batch, k.cuda(), v.cuda(), rotary=gt.kv_rotary(rot.table.cuda()), q=q.cuda(), q_out=dq)
    out = attend(d, sh.groups(), 1, dq, 0.09).cpu().double()
    assert d.error() == 0
    w.raw, _ = ref4.append(w, 1, k, v, rot)
    assert torch.equal(d.raw.cpu(), w.raw)
    want, _, size = ref.attend(w, 1, dq.cpu(), 0.09)
    assert ((out - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * size).all()


def test_refusals():
    sh = Shared(1, [(32, [(4, 1), (5, 1)])], "bf16")
    d, groups = sh.dev(), sh.groups()
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    size = gt.kv_attend_shared_workspace_bytes(d.pool, 4, 2, 2)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    at = lambda **kw: gt.kv_attend_shared_layer(d.pool, kw.pop("layer", 1), d.batch, kw.pop("groups", groups),  # noqa: E731
                                                kw.pop("q", q), kw.pop("out", out), kw.pop("scale", 1.0),
                                                kw.pop("ws", ws), **kw)

    def refused(code, **kw):
        with pytest.raises(gt.KVError) as e:
            at(**kw)
        assert e.value.code == code, e.value

    refused(-1, layer=2)
    refused(-1, scale=float("nan"))
    refused(-1, ws=ws[: size - 16])
    refused(-5, ws=torch.empty(size + 16, dtype=torch.uint8, device="cuda")[1:])
    refused(-1, q=q.float(), out=out.float())
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    refused(-1, groups=gt.kv_prefix_groups(i32([0]), i32([])))
    for bad in ((i32([0, 2]), i32([1, 2])), (i32([[0, 2]]), i32([1])), (torch.tensor([0, 2], device="cuda"), i32([1])),
                (i32([0, 2]).cpu(), i32([1]))):
        with pytest.raises(ValueError):
            gt.kv_prefix_groups(*bad)
    with pytest.raises(ValueError):
        at(scales=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        at(q=q[:1])
    g = gt.kv_prefix_groups(i32([0, 2]), i32([32]))
    g.struct.reserved = 1
    refused(-1, groups=g)
    g.struct.reserved, g.struct.n_groups = 0, -1
    refused(-1, groups=g)
    g.struct.n_groups, was = 1, g.struct.group_dev
    g.struct.group_dev = None
    refused(-1, groups=g)
    g.struct.group_dev = was + 2
    refused(-5, groups=g)
    with pytest.raises(gt.KVError):
        gt.kv_attend_shared_workspace_bytes(d.pool, 3, 2, 2)
    with pytest.raises(gt.KVError):
        gt.kv_attend_shared_workspace_bytes(d.pool, 4, 2, 1 << 50)
    empty = gt.kv_batch(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), i32([]),
                        torch.zeros(1, dtype=torch.int64, device="cuda"), 0)
    none = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    gt.kv_attend_shared_layer(d.pool, 0, empty, gt.kv_prefix_groups(i32([0]), i32([])), none, none.clone(), 1.0, ws)
    assert d.error() == 0
