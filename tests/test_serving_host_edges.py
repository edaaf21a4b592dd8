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
