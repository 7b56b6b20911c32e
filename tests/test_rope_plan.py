"""How the norm and rotation kernel shares a token's heads among warps: the
rule's values, by the warps that the device runs at once."""
import ctypes
import os
import subprocess

import pytest

from conftest import REPO

CSRC = os.path.join(REPO, "paged_attention_kv_gb300", "csrc")


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cpp", d / "plan.so"
    src.write_text('#include "rope_plan.h"\nextern "C" int parts(long long t, int s, long long w) '
                   "{ return pkv::rope_parts(t, s, w); }\n")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    fn = ctypes.CDLL(str(lib)).parts
    fn.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong]
    return fn


def warps(sms):
    return sms * 24


@pytest.mark.parametrize("sms", [1, 76, 148, 152])
@pytest.mark.parametrize("steps", [1, 2, 6, 10, 65])
def test_the_parts_of_least_cost(parts, sms, steps):
    w = warps(sms)
    for tokens in [1, 2, 37, 256, 512, 521, 1300, 2240, 2500, 3000, 4000, 7000, 7500, 14593, 32768, 2 ** 31 - 1]:
        cost = {p: -(-tokens * p // w) * (-(-steps // p) + 1) for p in range(1, steps + 1)
                if p == 1 or tokens * p <= 4 * w}
        assert parts(tokens, steps, w) == max(p for p in cost if cost[p] == min(cost.values()))


def test_a_batch_that_just_fills_one_round_of_more_sms_takes_fewer_warps_on_less(parts):
    assert parts(521, 10, warps(152)) == 7
    assert parts(521, 10, warps(148)) == 6


def test_one_warp_takes_a_whole_token_of_a_large_batch(parts):
    """Past twice the warps that run at once; the GPU tests of large batches
    rely on it."""
    for steps in (2, 5, 10, 24):
        assert parts(7500, steps, warps(152)) == 1
        assert parts(14593, steps, warps(152)) == 1
        assert 1 < parts(700, max(steps, 5), warps(152))


def test_several_warps_take_several_steps_each_in_between(parts):
    assert parts(4000, 4, warps(152)) == 2
    assert parts(2240, 12, warps(152)) == 3
