"""Refusals and messages of the serving calls at the edge of what their documentation allows, without a GPU."""
import os
import shutil
import subprocess

import pytest

from padding_free_varlen_b200 import build as pbuild
from padding_free_varlen_b200 import capi
from test_serving_host import INVALID, O, Q, cache, refused

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    pbuild.build()
    return capi.load()


@pytest.mark.parametrize("code,change", [
    (INVALID, dict(max_len=0x7c000001)), (INVALID, dict(max_len=0x7fffffff)),
    (INVALID, dict(budget=0x7fffffff, new_max_pages=1 << 27)), (INVALID, dict(budget=0x7c000001, new_max_pages=1 << 27)),
    (capi.ENERGON_ERR_WORKSPACE_TOO_SMALL, dict(budget=0x7c000000, new_max_pages=1 << 27)),
])
def test_evict_refuses_sizes_at_the_end_of_32_bits(code, change):
    a = dict(cache=cache(), table=4096, max_pages=1 << 27, lens=8192, new_table=4096, new_max_pages=2, new_lens=8192, batch=2,
             max_len=64, budget=20, recent=4, status=0, ws=1 << 24, ws_bytes=1 << 20)
    refused(code, capi.energon_cache_evict, *dict(a, **change).values())


@pytest.mark.parametrize("max_len", [0x7c000001, 0x7fffff00, 0x7fffffff])
def test_cache_attention_refuses_lengths_at_the_end_of_32_bits(max_len):
    refused(INVALID, capi.energon_cache_attention, cache(), 4096, 1 << 27, 8192, 2, max_len, Q, 256, 4, capi.ENERGON_F16, 0.1, O, 256,
            0, 0, 0, 1 << 24, 1 << 20)


def test_scales_beyond_what_the_kernels_can_hold_are_refused():
    for scale in (2.4e38, 2.9e38):
        refused(INVALID, capi.energon_prompt_attention, Q, 512, Q, 512, Q, 512, Q, 2, 8, 4, 4, 128, capi.ENERGON_F16, scale, O, 512)
        refused(INVALID, capi.energon_cache_attention, cache(), 4096, 4, 8192, 2, 64, Q, 256, 4, capi.ENERGON_F16, scale, O, 256, 0, 0, 0,
                1 << 24, 1 << 20)


OUT_OF_MEMORY = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include "energon_rce.h"

static bool none_left = false;
void* operator new(std::size_t n) {
    void* p = none_left ? nullptr : std::malloc(n);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

static int call(int head_dim) {
    char* at = nullptr;  // addresses that are never followed: there is no device
    return energon_prompt_attention(at + 4096, 512, at + 8192, 512, at + 12288, 512, (const int32_t*)(at + 16384), 1, 8, 4, 4,
                                    head_dim, ENERGON_F32, 0.1f, at + 20480, 512, nullptr, nullptr, nullptr);
}
int main() {
    const int no_device = call(64);
    std::printf("%d [%s]\n", no_device, energon_last_error());
    none_left = true;
    const int code = call(128);  // (its kernel is not known yet)
    none_left = false;
    std::printf("%d [%s]\n", code, energon_last_error());
    none_left = true;
    const int refused = energon_prompt_attention(nullptr, 1, nullptr, 1, nullptr, 1, nullptr, 1, 8, 4, 3, 64, ENERGON_F32, 0.1f, nullptr, 1,
                                                 nullptr, nullptr, nullptr);
    none_left = false;
    std::printf("%d [%s]\n", refused, energon_last_error());
    return 0;
}
"""


def test_no_memory_on_the_host_is_an_error_with_a_message(tmp_path):
    """An allocation that fails inside a call leaves no exception, but the code and a message; a refusal needs none."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "memory.cpp", tmp_path / "memory"
    src.write_text(OUT_OF_MEMORY)
    libdir = os.path.dirname(pbuild.LIB_PATH)
    subprocess.run(["g++", "-std=c++17", "-rdynamic", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe), pbuild.LIB_PATH,
                    f"-Wl,-rpath,{libdir}"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, env=dict(os.environ, CUDA_VISIBLE_DEVICES="-1")).stdout
    first, second, third = out.splitlines()
    assert first.startswith(f"{capi.ENERGON_ERR_CUDA} [prompt attention: ")
    assert second == f"{capi.ENERGON_ERR_CUDA} [prompt attention: std::bad_alloc]"
    assert third == f"{INVALID} [prompt attention: n_heads 4 is not a multiple of n_kv_heads 3]"
