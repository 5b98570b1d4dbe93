"""The sizes of kv_forms reach the forms that they are named for, on 256 compute units."""

import ctypes
import os

import pytest

import fp8_dynamic_quant_amd as wq
import kv_forms as kf

pytestmark = pytest.mark.skipif(not os.path.exists(wq.LIB_PATH), reason="libwq.so not built")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", sorted(kf.FORMS))
def test_sizes_reach_their_form(name, D):
    c = ctypes.create_string_buffer(4096)
    ctypes.memmove(ctypes.addressof(c) + 4, ctypes.byref(ctypes.c_int(256)), 4)
    f = kf.form(name, D)
    d = wq.KvCacheDesc(1, 9, f["H"], f["P"], D, None, None, None, None, None, f["width"], f["width"])
    T = int(f["offsets"][-1]) + 2
    assert wq.lib().wq_kv_attention_path(c, ctypes.byref(d), T, f["H"] * f["R"], len(f["ns"])) == f["path"]
