"""Host side of 4-bit pools (KV_FORMAT_E2M1): sizes and gates, constants, and
the plain form of the codes itself (no GPU here)."""
import re

import numpy as np
import pytest

import cache4_ref as ref4
import gather_translate_kv_gb300 as gt


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gather_translate_kv_gb300 import build

    build.build()


def test_format_constants_match_the_header():
    src = open(gt.HEADER).read()
    got = {k: int(v) for k, v in re.findall(r"(KV_FORMAT_\w+) = (\d+)", src)}
    assert got == {"KV_FORMAT_ELEMENTS": gt.KV_FORMAT_ELEMENTS, "KV_FORMAT_E2M1": gt.KV_FORMAT_E2M1}


@pytest.mark.parametrize("H,D,R", [(8, 128, 576), (8, 64, 288), (1, 128, 80), (1, 16, 16), (3, 80, 144), (2, 256, 288)])
def test_sizes(H, D, R):
    assert ref4.row_bytes(H, D) == R
    desc = gt.make_desc(3, H, D, 1, 16, 10, format=gt.KV_FORMAT_E2M1)
    assert gt.kv_pool_required_bytes(desc) == (10 * 6 * 16 * R, 6 * 16 * R)


@pytest.mark.parametrize("change,code", [
    (dict(head_dim=72), -1), (dict(itemsize=2), -1), (dict(itemsize=4), -1), (dict(latent_only=True), -1),
    (dict(format=2), -1), (dict(format=-1), -1), (dict(v_head_dim=64), -2), (dict(num_pages=1 << 28), -3)])
def test_gates(change, code):
    d = dict(layer_num=2, head_num=2, head_dim=128, itemsize=1, page_size=16, num_pages=8, format=gt.KV_FORMAT_E2M1)
    gt.kv_pool_required_bytes(gt.make_desc(**d))
    with pytest.raises(gt.KVError) as e:
        gt.kv_pool_required_bytes(gt.make_desc(**{**d, **change}))
    assert e.value.code == code


def test_plain_codes():
    """By hand: every step, the borders between steps, scale bytes at the ends of their range."""
    y = np.array([0, .25, .26, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.1, 6, 9, -.25, -.3, -6.4], np.float32)
    want = [0, 0, 1, 1, 2, 2, 2, 3, 4, 4, 4, 5, 6, 6, 6, 7, 7, 7, 8, 9, 15]
    assert ref4.nearest(y).tolist() == want
    assert ref4.scale_value([0, 1, 7, 8, 0x78, 0x7C, 0xE0, 0xE1, 0xFF])[:7].tolist() == [
        0, 2.0 ** -17, 7 * 2.0 ** -17, 2.0 ** -14, 1, 1.5, 8192]
    assert np.isnan(ref4.scale_value([0xE1, 0xFF])).all()
    x = np.zeros((1, 16), np.float32)
    x[0, :4] = [6, -3, 1.24, 0.25]
    codes, scales, bad = ref4.encode(x)
    assert scales.tolist() == [[0x78]] and codes[0, :2].tolist() == [0xD7, 0x02] and not bad.any()
    assert ref4.encode(np.full((1, 16), 1e9, np.float32))[1].tolist() == [[0xE0]]
    assert ref4.encode(np.zeros((1, 16), np.float32))[1].tolist() == [[0]]


def test_prefix_groups_match_the_header(tmp_path):
    import ctypes
    import subprocess

    from gather_translate_kv_gb300 import build

    fields = [f for f, _ in gt.kv_prefix_groups_t._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kv_attention.h"\nint main(void) {' +
                   "".join(f'printf("%zu\\n", offsetof(kv_prefix_groups, {f}));' for f in fields) +
                   'printf("%zu\\n", sizeof(kv_prefix_groups));return 0;}\n')
    exe = tmp_path / "t"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", build.INCLUDE, str(src), "-o", str(exe)])
    got = list(map(int, subprocess.check_output([str(exe)], text=True).split()))
    assert got == [getattr(gt.kv_prefix_groups_t, f).offset for f in fields] + [ctypes.sizeof(gt.kv_prefix_groups_t)]


def test_shared_calls_without_a_pool_are_refused():
    import ctypes

    L, n = gt.lib(), ctypes.c_int64()
    vp = ctypes.c_void_p
    g = gt.kv_prefix_groups_t(16, 16, 1, 0)
    b = gt.kv_batch_t()
    assert L.kv_attend_shared_workspace_bytes(None, 1, 1, 1, ctypes.byref(n)) == -1
    assert L.kv_attend_shared_layer(None, 0, ctypes.addressof(b), ctypes.addressof(g), 1, vp(16), 1, 1, vp(16), None, 1.0,
                                    None, vp(16), 1, None) == -1
    assert L.kv_attend_shared_layer(None, 0, ctypes.addressof(b), None, 1, vp(16), 1, 1, vp(16), None, 1.0, None, vp(16),
                                    1, None) == -1
