"""pkv_prompt_attention refuses an output in place of an input (a row that is
done again reads its inputs again): on the host, before anything is enqueued
(the pointers are never dereferenced)."""
import ctypes

import pytest

from paged_attention_kv_gb300 import binding as pkv

vp = ctypes.c_void_p


@pytest.mark.parametrize("out", [0x10000, 0x20000, 0x30000])
def test_an_output_in_place_of_an_input(out):
    assert pkv.LIB.pkv_prompt_attention(vp(0x10000), 1024, vp(0x20000), 256, vp(0x30000), 256, 40, 8, 2, 128,
                                        vp(0x40000), 2, ctypes.c_float(0.1), vp(out), None, None) == pkv.PKV_E_DIMS
