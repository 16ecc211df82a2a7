"""Host checks of the token cache: csrc/cache_args.cpp and the index helpers of
csrc/cache.h, built by the host compiler with AddressSanitizer and
UndefinedBehaviorSanitizer and driven by tests/native/cache_args_check.cpp;
sizes through the C ABI; and the helper class's own refusals."""
import os
import shutil
import subprocess

import pytest

from kv_cache_compression_jolt_amd import binding as jb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kv_cache_compression_jolt_amd", "csrc")


@pytest.mark.timeout(300)
def test_checks_and_indexes_under_asan_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "cache_args_check")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, os.path.join(CSRC, "cache_args.cpp"),
           os.path.join(ROOT, "tests", "native", "cache_args_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=240)
    assert r.returncode == 0 and "cache args: 0 failures" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])


def _cache(**kw):
    c = jb.jolt_cache(8, 128, 4, 64, 10, 3, 1, 0, 1, 0, 0, 4096, 1 << 30, 4096, 4096)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_pool_bytes():
    # K and V codes and scales of 64 tokens, 8 heads, 10 pages
    assert jb.jolt_cache_pool_bytes(_cache()) == 10 * 8 * 64 * 2 * (64 + 4)
    assert jb.jolt_cache_pool_bytes(_cache(d=64, bits=8, page_tokens=32)) == 10 * 8 * 32 * 2 * (64 + 2)
    assert jb.jolt_cache_pool_bytes(_cache(pages=0)) == 0
    for kw in (dict(d=80), dict(bits=5), dict(page_tokens=96)):
        with pytest.raises(jb.JoltError) as e:
            jb.jolt_cache_pool_bytes(_cache(**kw))
        assert e.value.status == jb.JOLT_E_UNSUPPORTED


def test_attention_workspace_size():
    c = _cache()
    # few rows over a long cache are split: the workspace holds m, l and d sums per split and row
    b = jb.jolt_cache_attention_workspace_size(c, 1, 1, 1, 65535, 32)
    assert b > 0 and b % 4 == 0
    # grows with the rows, none for a call without rows
    assert jb.jolt_cache_attention_workspace_size(c, 2, 2, 1, 65535, 32) > 0
    assert jb.jolt_cache_attention_workspace_size(c, 1, 0, 0, 65535, 32) == 0
    assert jb.jolt_cache_attention_workspace_size(c, 0, 0, 0, 0, 32) == 0
    with pytest.raises(jb.JoltError) as e:
        jb.jolt_cache_attention_workspace_size(c, 1, 1, 1, 100, 12)
    assert e.value.status == jb.JOLT_E_INVALID


def test_a_cache_lies_on_a_gpu():
    import torch
    i32 = torch.int32
    with pytest.raises(ValueError):
        jb.JoltCache(1, 64, 4, torch.zeros(4096, dtype=torch.uint8), torch.zeros(1, 1, dtype=i32),
                     torch.zeros(1, dtype=i32))
