"""The bounded waits of the tile kernel in its pass over prefixes, made to run
out on purpose, in the build of test_gpu_attention_timeout.py (the barriers of
finished weights expect one arrival more than they get): the pass gives up, the one over the
sequences' own tokens runs to its end all the same, the error word says so, and the
context stays usable. Nothing faults, traps or hangs.
"""
from __future__ import annotations

import time

import pytest
import torch

import gather_translate_kv_gb300 as gt
from test_gpu_attention_timeout import variant  # noqa: F401 (fixture)
from test_gpu_shared import Shared, attend, check, queries

pytestmark = pytest.mark.gpu

LARGE = [(1200, [(9, 1)] * 40), (700, [(4, 2)] * 30)]


@pytest.mark.parametrize("cache", ["bf16", "e2m1"])
def test_wait_in_a_prefix_runs_out_cleanly(variant, monkeypatch, cache):  # noqa: F811
    with monkeypatch.context() as m:
        m.setattr(gt, "_lib", variant)
        sh = Shared(1, LARGE, cache, D=128)
        d = sh.dev()
        q = queries(sh.w, 8, "bf16").cuda()
        t0 = time.time()
        attend(d, sh.groups(), 1, q, 0.1)
        assert d.error() == gt.KV_DEV_ERR_TIMEOUT
        assert time.time() - t0 < 60
        gt.kv_pool_destroy(d.pool)
    check(Shared(1, LARGE, cache, D=128), 8, "bf16")
