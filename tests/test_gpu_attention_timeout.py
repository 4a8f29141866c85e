"""The bounded waits of the tensor-core attention kernel, made to run out on purpose.

k_attend_tile's warps hand tiles to one another through mbarriers and wait at
most about a second for each. A build with GTKV_TEST_EXTRA_ARRIVALS=1 makes
the barriers of finished weights expect one arrival more than they get: all
copies and products that were started complete, but the next product never
starts. Every block must then give up, raise KV_DEV_ERR_TIMEOUT, write none of its rows
and return, leaving the context usable. Nothing faults, traps or hangs; the
library itself is never built with that flag.
"""
from __future__ import annotations

import os
import time

import pytest
import torch

import attention_ref as ref
import gather_translate_kv_gb300 as gt
from gather_translate_kv_gb300 import build
from test_gpu_attention import Dev

pytestmark = pytest.mark.gpu

VARIANT_DIR = os.path.join(build.BUILD, "attention_timeout_test")
VARIANT_LIB = os.path.join(VARIANT_DIR, "libgtkv_attention_timeout_test.so")


@pytest.fixture(scope="module")
def variant():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    path = build.build(force=True, extra_flags=["-DGTKV_TEST_EXTRA_ARRIVALS=1"], lib=VARIANT_LIB,
                       build_dir=VARIANT_DIR)
    return gt.load(path)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_attention_wait_runs_out_cleanly(variant, monkeypatch, cache):
    monkeypatch.setattr(gt, "_lib", variant)
    # a decode step and two prompts, one of them cut over many blocks
    w = ref.world(1, [40, 150, 1200], [1, 150, 600], D=128, cache=cache)
    d = Dev(w)
    q = torch.randn(w.n_rows, 8, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    t0 = time.time()
    out = d.attend(1, q.cuda(), 0.1).cpu().double()
    assert time.time() - t0 < 60
    assert d.error() == gt.KV_DEV_ERR_TIMEOUT
    assert (out[1:] == 7.0).all()  # no row of the prompts was written
    # the decode step is the other kernel's, and the context is still usable
    one = ref.World(**{**w.__dict__, "lens": [40], "news": [1], "gap": [0], "table": w.table[:1]})
    want, _, size = ref.attend(one, 1, q[:1], 0.1)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * size
    assert ((out[:1] - want).abs() <= tol).all()
    d1 = Dev(one)
    again = d1.attend(1, q[:1].cuda(), 0.1).cpu().double()
    assert d1.error() == 0
    assert ((again - want).abs() <= tol).all()
    for x in (d, d1):
        gt.kv_pool_destroy(x.pool)
