"""CPU tests of the attention plan at the ends of its ranges."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import heterogeneous_adapter_batching_amd as hl
from test_attn_plan import REPO, _attn, _kv, _launch, _read, _write, check_plan, make_table, shape

LAST = 2 ** 31 - 1
# new tokens and cached tokens with them, rows before the first token among them
MIXED = ([40, 1, 3, 300, 5], [35, 70, 0, 290, 5])


@pytest.mark.parametrize("window", [2 ** 30 - 1, 2 ** 30, 2 ** 30 + 1, LAST - 40, LAST])
@pytest.mark.parametrize("sinks", [0, 5, 2 ** 30 + 1, LAST])
def test_a_window_longer_than_any_sequence_is_none(window, sinks):
    """Such a window hides nothing: the plan is that of no window."""
    q_len, kv_len = MIXED
    tab = make_table(np.random.default_rng(3), kv_len, 16, 1000)
    staging, info = hl.lora_attn_plan(shape(window=window, sinks=sinks), q_len, kv_len, tab)
    check_plan(shape(), q_len, kv_len, tab, staging, info)
    assert np.array_equal(staging, hl.lora_attn_plan(shape(), q_len, kv_len, tab)[0])
    # what the kernels subtract from positions of -2^30 and more
    assert info.shape.window == min(window, 2 ** 30) and info.shape.sinks == min(sinks, 2 ** 30)


@pytest.mark.parametrize("sinks", [64, 2 ** 30, LAST - 63, LAST])
@pytest.mark.parametrize("window", [1, 100])
def test_more_sinks_than_any_sequence_has_tokens(window, sinks):
    q_len, kv_len = MIXED
    tab = make_table(np.random.default_rng(4), kv_len, 16, 1000)
    staging, info = hl.lora_attn_plan(shape(window=window, sinks=sinks), q_len, kv_len, tab)
    check_plan(shape(window=window, sinks=sinks), q_len, kv_len, tab, staging, info)


@pytest.mark.parametrize("q_len,kv_len,capacity,code", [
    ([3, 3], [20, 20], 40, hl.LORA_ECAPACITY), ([3], [20000], 4000, hl.LORA_EINVAL), ([3], [33], 4000, hl.LORA_EPAGE)])
def test_a_launch_holds_no_plan_after_an_error(q_len, kv_len, capacity, code):
    """Not the new batch's numbers with the old one's places either."""
    L = _launch()
    tab = np.array([[0, 1, 5000]] * len(q_len), np.int32)
    lens = [np.array(x, np.int32) for x in (q_len, kv_len)]
    staging, s = np.zeros(4000, np.int32), shape()
    assert _attn(L, _kv(), scale=0.0) == hl.LORA_EINVAL and L.meta  # a plan, refused for the scale alone
    st = hl._lib.lora_attn_prepare(ctypes.byref(s), len(q_len), lens[0].ctypes.data, lens[1].ctypes.data, tab.ctypes.data,
                                   tab.shape[1], staging.ctypes.data, capacity, 0x1000, None, ctypes.byref(L))
    assert st == code
    assert not L.meta
    assert _attn(L, _kv()) == hl.LORA_EINVAL and _write(L, _kv()) == hl.LORA_EINVAL and _read(L, _kv()) == hl.LORA_EINVAL


def _sanitize(tmp_path, planner):
    exe = tmp_path / "attn_sanitize_edges"
    csrc = os.path.join(REPO, "heterogeneous_adapter_batching_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(REPO, "include"), "-I", csrc, planner,
                    os.path.join(REPO, "tests", "attn_sanitize_edges.cpp"), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_planner_over_its_ranges_under_sanitizers(tmp_path):
    r = _sanitize(tmp_path, os.path.join(REPO, "heterogeneous_adapter_batching_amd", "csrc", "attn_plan.cpp"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert "attention planner ok over its ranges" in r.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_that_test_fails_for_a_planner_that_refuses_everything(tmp_path):
    stub = tmp_path / "refuses.cpp"
    stub.write_text('#include "hetlora.h"\nextern "C" int32_t lora_attn_plan(const lora_attn_shape_t*, int32_t, const int32_t*, '
                    'const int32_t*, const int32_t*, int64_t, int32_t*, int64_t, lora_attn_info_t*) { return LORA_EINVAL; }\n')
    assert _sanitize(tmp_path, str(stub)).returncode == 1


def test_attn_refuses_a_scale_that_overflows_in_base_2():
    """Scores are multiplied by scale * log2 e, and zero by infinity is not zero."""
    for scale in (2.4e38, 3.4e38):
        assert _attn(_launch(), _kv(), scale=scale) == hl.LORA_EINVAL


def test_status_of_a_shape_says_so():
    assert "shape" in hl.lora_status_string(hl.LORA_ESHAPE)
