"""Edges of the operators of kv_attention.h on the GPU: metadata that is
inconsistent, pages that nobody sees, the ends of the scales' range, the bits
that weights keep, calls on two streams at once. Plain forms: attention_ref.py.
"""
from __future__ import annotations

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
