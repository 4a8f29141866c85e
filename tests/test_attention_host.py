"""Host-side checks of include/kv_attention.h: its constants and structures
agree with the binding, it compiles as C99, and calls without a pool are
refused (no GPU here)."""
import ctypes
import re
import subprocess

import pytest
import torch

import gather_translate_kv_gb300 as gt


@pytest.fixture(scope="module")
def lib():
    from gather_translate_kv_gb300 import build

    build.build()
    return gt.lib()


def test_constants_match_the_header():
    src = open(gt.ATTENTION_HEADER).read()
    defs = dict(re.findall(r"^#define (KV_DEV_ERR_\w+) (\d+)", src, flags=re.M))
    assert defs == {"KV_DEV_ERR_POSITION": str(gt.KV_DEV_ERR_POSITION)}
    types = dict(re.findall(r"(KV_TYPE_\w+) = (\d+)", src))
    assert {k: int(v) for k, v in types.items()} == {
        "KV_TYPE_BF16": gt.KV_TYPE[torch.bfloat16], "KV_TYPE_F16": gt.KV_TYPE[torch.float16],
        "KV_TYPE_F32": gt.KV_TYPE[torch.float32]}


def test_structures_match_the_header(tmp_path):
    """Offsets as a C99 compiler lays them out."""
    fields = {"kv_batch": gt.kv_batch_t, "kv_rotary": gt.kv_rotary_t}
    body = "".join(f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for c, s in fields.items() for f, _ in s._fields_)
    body += "".join(f'printf("{c} %zu\\n", sizeof({c}));' for c in fields)
    src = tmp_path / "t.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"kv_attention.h\"\nint main(void) {" + body +
                   "return 0;}\n")
    from gather_translate_kv_gb300 import build

    exe = tmp_path / "t"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", build.INCLUDE, str(src), "-o",
                           str(exe)])
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
        name, n = line.split()
        c, _, f = name.partition(".")
        assert (getattr(fields[c], f).offset if f else ctypes.sizeof(fields[c])) == int(n), name


def test_calls_without_a_pool_are_refused(lib):
    b = gt.kv_batch_t()
    n = ctypes.c_int64()
    assert lib.kv_scale_bytes(None, ctypes.byref(n)) == -1
    assert lib.kv_attend_workspace_bytes(None, 1, 1, 1, ctypes.byref(n)) == -1
    vp = ctypes.c_void_p
    p = ctypes.addressof(b)
    assert lib.kv_append_layer(None, 0, p, 1, vp(16), 1, vp(16), 1, None, None, 0, 0, None, None, None) == -1
    assert lib.kv_attend_layer(None, 0, p, 1, vp(16), 1, 1, vp(16), None, 1.0, 0, 0, None, vp(16), 1, None) == -1
    assert lib.kv_gather_layer_scaled(None, 0, p, vp(16), 1, vp(16), vp(16), None) == -1


def test_tensors_are_checked_before_the_library_is_called():
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        gt.kv_batch(t, torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), 1)  # not on a GPU
    with pytest.raises(ValueError):
        gt.kv_batch(t[0], torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), 1)
    with pytest.raises(ValueError):
        gt.kv_batch(t, torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), 1)
    with pytest.raises(ValueError):
        gt.kv_rotary(torch.zeros(4))
