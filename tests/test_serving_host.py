"""The serving operators without a GPU: refusals on the host before any launch, workspace sizes,
the struct's layout, and pins of the plain 64-bit implementations that the GPU tests use."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import serving_ref as ref
from padding_free_varlen_b200 import build as pbuild
from padding_free_varlen_b200 import capi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, MISALIGNED = (capi.ENERGON_ERR_INVALID_ARGUMENT, capi.ENERGON_ERR_UNSUPPORTED,
                                    capi.ENERGON_ERR_MISALIGNED)


@pytest.fixture(scope="module", autouse=True)
def lib():
    pbuild.build()
    return capi.load()


def refused(code, fn, *args):
    with pytest.raises(capi.EnergonError) as e:
        fn(*args, stream=0)
    assert e.value.code == code, str(e.value)


# addresses that are never followed: every call below is refused by the host-side checks
Q, K, V, O, CU = 4096, 8192, 12288, 16384, 20480
PROMPT = dict(q=Q, ld_q=512, k=K, ld_k=256, v=V, ld_v=256, cu=CU, batch=2, rows=8, n_heads=4, n_kv=2, d=128,
              dtype=capi.ENERGON_F16, scale=0.1, o=O, ld_o=512)


@pytest.mark.parametrize("code,change", [
    (INVALID, dict(q=0)), (INVALID, dict(k=0)), (INVALID, dict(v=0)), (INVALID, dict(o=0)), (INVALID, dict(cu=0)),
    (INVALID, dict(batch=-1)), (INVALID, dict(rows=-1)), (INVALID, dict(rows=0x7fffffff)), (INVALID, dict(n_heads=0)),
    (INVALID, dict(n_heads=3)), (INVALID, dict(n_kv=0)), (UNSUPPORTED, dict(d=96)), (INVALID, dict(dtype=9)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-1.0)), (INVALID, dict(scale=float("nan"))),
    (INVALID, dict(scale=float("inf"))), (INVALID, dict(ld_q=511)), (INVALID, dict(ld_k=128)), (INVALID, dict(ld_o=0)),
    (MISALIGNED, dict(ld_v=260)), (MISALIGNED, dict(q=4104)), (MISALIGNED, dict(o=16386)), (INVALID, dict(o=Q)),
    (INVALID, dict(o=V)), (UNSUPPORTED, dict(n_heads=65536, ld_q=1 << 23, ld_o=1 << 23)),
])
def test_prompt_attention_refusals(code, change):
    a = dict(PROMPT, **change)
    refused(code, capi.energon_prompt_attention, *a.values())


@pytest.mark.parametrize("code,change", [
    (INVALID, dict(lse=0)), (INVALID, dict(weights=0)), (INVALID, dict(window=0)), (INVALID, dict(window=-3)),
    (UNSUPPORTED, dict(d=32)), (MISALIGNED, dict(ld_k=257)), (INVALID, dict(q=0)),
])
def test_key_weights_refusals(code, change):
    a = dict(q=Q, ld_q=512, k=K, ld_k=256, lse=V, cu=CU, batch=2, rows=8, n_heads=4, n_kv=2, d=128,
             dtype=capi.ENERGON_BF16, scale=0.1, window=4, weights=O)
    refused(code, capi.energon_prompt_key_weights, *dict(a, **change).values())


def cache(**change):
    a = dict(k_codes=1 << 20, v_codes=1 << 21, k_scale=4096, v_scale=8192, weight=12288, n_pages=10, n_kv_heads=2,
             page_len=16, head_dim=64)
    return capi.energon_kv_cache(*dict(a, **change).values())


BAD_CACHES = [(INVALID, dict(k_codes=0)), (INVALID, dict(v_scale=0)), (INVALID, dict(n_pages=0)),
              (INVALID, dict(n_kv_heads=0)), (UNSUPPORTED, dict(page_len=24)), (UNSUPPORTED, dict(page_len=256)),
              (UNSUPPORTED, dict(head_dim=80)), (MISALIGNED, dict(k_codes=(1 << 20) + 8))]


@pytest.mark.parametrize("code,bad,change", [(c, b, {}) for c, b in BAD_CACHES] + [
    (INVALID, {}, dict(table=0)), (INVALID, {}, dict(lens=0)), (INVALID, {}, dict(max_pages=0)),
    (INVALID, {}, dict(k=0)), (INVALID, {}, dict(cu=0)), (INVALID, {}, dict(batch=-1)), (INVALID, {}, dict(dtype=5)),
    (INVALID, {}, dict(ld_k=64)), (MISALIGNED, {}, dict(ld_v=130)), (UNSUPPORTED, {}, dict(batch=65536)),
])
def test_append_refusals(code, bad, change):
    a = dict(cache=cache(**bad), table=4096, max_pages=4, lens=8192, k=K, ld_k=128, v=V, ld_v=128, weights=0, cu=CU,
             batch=2, rows=5, dtype=capi.ENERGON_F32)
    refused(code, capi.energon_kv_append, *dict(a, **change).values())


@pytest.mark.parametrize("code,bad,change", [(c, b, {}) for c, b in BAD_CACHES] + [
    (INVALID, dict(weight=0), {}), (INVALID, {}, dict(q=0)), (INVALID, {}, dict(o=Q)), (INVALID, {}, dict(n_heads=3)),
    (INVALID, {}, dict(max_len=-1)), (INVALID, {}, dict(scale=0.0)), (MISALIGNED, {}, dict(ws=4097)),
    (capi.ENERGON_ERR_WORKSPACE_TOO_SMALL, {}, dict(ws_bytes=3)), (INVALID, {}, dict(ld_o=128)),
    (capi.ENERGON_ERR_WORKSPACE_TOO_SMALL, {}, dict(ws=0, ws_bytes=0)),
])
def test_cache_attention_refusals(code, bad, change):
    a = dict(cache=cache(**bad), table=4096, max_pages=4, lens=8192, batch=2, max_len=64, q=Q, ld_q=256, n_heads=4,
             dtype=capi.ENERGON_F16, scale=0.1, o=O, ld_o=256, lse=0, accumulate=1, status=0, ws=1 << 24,
             ws_bytes=1 << 20)
    refused(code, capi.energon_cache_attention, *dict(a, **change).values())


@pytest.mark.parametrize("code,bad,change", [(c, b, {}) for c, b in BAD_CACHES] + [
    (INVALID, dict(weight=0), {}), (INVALID, {}, dict(new_table=0)), (INVALID, {}, dict(new_lens=0)),
    (INVALID, {}, dict(budget=0)), (INVALID, {}, dict(recent=-1)), (INVALID, {}, dict(recent=21)),
    (INVALID, {}, dict(new_max_pages=1)), (INVALID, {}, dict(max_len=-1)), (MISALIGNED, {}, dict(ws=4100)),
    (capi.ENERGON_ERR_WORKSPACE_TOO_SMALL, {}, dict(ws_bytes=64)),
])
def test_evict_refusals(code, bad, change):
    a = dict(cache=cache(**bad), table=4096, max_pages=4, lens=8192, new_table=4096, new_max_pages=2, new_lens=8192,
             batch=2, max_len=64, budget=20, recent=4, status=0, ws=1 << 24, ws_bytes=1 << 20)
    refused(code, capi.energon_cache_evict, *dict(a, **change).values())


def test_nothing_to_do_needs_no_memory():
    """No rows or no sequences: nothing is launched, and empty tensors' NULL addresses are fine."""
    f16 = capi.ENERGON_F16
    capi.energon_prompt_attention(0, 512, 0, 256, 0, 256, CU, 1, 0, 4, 2, 128, f16, 0.1, 0, 512, stream=0)
    capi.energon_prompt_key_weights(0, 512, 0, 256, 0, CU, 1, 0, 4, 2, 128, f16, 0.1, 4, 0, stream=0)
    capi.energon_kv_append(cache(), 4096, 4, 8192, 0, 128, 0, 128, 0, CU, 2, 0, f16, stream=0)
    capi.energon_cache_attention(cache(), 0, 4, 0, 0, 64, 0, 256, 4, f16, 0.1, 0, 256, stream=0)
    capi.energon_cache_evict(cache(), 0, 4, 0, 0, 2, 0, 0, 64, 20, 4, stream=0)


def test_binding_checks_tensors():
    cpu = torch.zeros(8, 4, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        capi.energon_prompt_attention(cpu, 512, K, 256, V, 256, CU, 2, 8, 4, 2, 128, capi.ENERGON_F16, 0.1, O, 512, stream=0)
    with pytest.raises(ValueError):
        capi.make_kv_cache(torch.zeros(2, 1, 16, 64, dtype=torch.int8), torch.zeros(2, 1, 16, 64, dtype=torch.int8),
                           torch.zeros(2, 1), torch.zeros(2, 1))
    with pytest.raises(ValueError):
        capi.make_kv_cache(torch.zeros(2, 1, 16, 64, dtype=torch.int8), torch.zeros(2, 1, 16, 128, dtype=torch.int8),
                           torch.zeros(2, 1), torch.zeros(2, 1))


def test_workspace_sizes():
    c = cache()
    a = capi.energon_cache_attention_workspace_bytes(c, 4, 100, 8, 0)
    b = capi.energon_cache_attention_workspace_bytes(c, 4, 100, 8, 1)
    assert 0 < a < b and b >= a + 4 * 4 * 8 * 100          # a score per (sequence, head, token)
    assert capi.energon_cache_attention_workspace_bytes(c, -1, 100, 8, 0) == 0
    assert capi.energon_cache_evict_workspace_bytes(c, 4, 50) >= 4 * 2 * 50 * 12
    assert capi.energon_cache_evict_workspace_bytes(c, 4, 0) == 0
    big = capi.energon_cache_attention_workspace_bytes(c, 60000, 1 << 20, 1024, 1)   # no 32-bit wrap
    assert big > 60000 * (1 << 20) * 1024 * 4


def test_cache_struct_layout(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    fields = [n for n, _ in capi.energon_kv_cache._fields_]
    src = tmp_path / "layout.c"
    body = "".join(f'printf("%zu\\n", offsetof(energon_kv_cache, {f}));' for f in fields)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "energon_rce.h"\nint main(void) {'
                   f'printf("%zu\\n", sizeof(energon_kv_cache));{body} return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    out = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert out == [ctypes.sizeof(capi.energon_kv_cache)] + [getattr(capi.energon_kv_cache, f).offset for f in fields]


# ------------------------------------------------------------------ the plain implementations, pinned


def test_ref_prompt_against_torch():
    rng = np.random.default_rng(1)
    lens, H, kv, d = [5, 0, 1, 9], 4, 2, 8
    T = sum(lens)
    q, k, v = rng.standard_normal((T, H, d)), rng.standard_normal((T, kv, d)), rng.standard_normal((T, kv, d))
    o, lse, _, _ = ref.prompt(q, k, v, lens, 0.3)
    w = ref.key_weights(q, k, lse, lens, 0.3, 1 << 30)
    for a, b in ref.spans(lens):
        if a == b:
            continue
        tq, tk, tv = (torch.from_numpy(np.ascontiguousarray(x[a:b].transpose(1, 0, 2))) for x in (q, k, v))
        tk, tv = tk.repeat_interleave(H // kv, 0), tv.repeat_interleave(H // kv, 0)
        t = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, is_causal=True, scale=0.3)
        assert np.allclose(t.numpy().transpose(1, 0, 2), o[a:b], rtol=0, atol=1e-12)
        assert np.isclose(w[:, a:b].sum(), H * (b - a))     # every query gives away weight 1 per head
    last = ref.key_weights(q, k, lse, lens, 0.3, 1)
    assert np.allclose([last[:, a:b].sum() for a, b in ref.spans(lens)], [H if b > a else 0 for a, b in ref.spans(lens)])


def empty_cache(n_pages, kv, P, d, weight=True):
    z = lambda *s: np.zeros(s, np.float32)  # noqa: E731
    return ref.Cache(np.zeros((n_pages, kv, P, d), np.int8), np.zeros((n_pages, kv, P, d), np.int8), z(n_pages, kv),
                     z(n_pages, kv), z(n_pages, kv, P) if weight else None)


def test_ref_append_hand_case_and_bound():
    c = empty_cache(2, 1, 16, 4)
    table = np.array([[1, 0]])
    x = np.array([[[127.0, -63.5, 0.4, 0.0]]], np.float32)
    ref.append(c, table, [1], x, x, None, [1])
    s = c.scale["k"][1, 0]
    assert np.isclose(s, 1.0, rtol=1e-6) and c.codes["k"][1, 0, 0, 0] == 127 and c.codes["k"][1, 0, 0, 2] == 0
    ref.append(c, table, [2], 3 * x, x, None, [1])                       # needs 3: the scale doubles twice
    assert c.scale["k"][1, 0] == 4 * s and c.codes["k"][1, 0, 0, 0] == 32 and c.codes["k"][1, 0, 1, 0] == 95
    assert c.scale["v"][1, 0] == s
    # token by token, no element is ever off by a final scale or more
    rng = np.random.default_rng(2)
    for seed in range(20):
        c = empty_cache(1, 1, 16, 64)
        rows = (rng.standard_normal((16, 1, 64)) * np.exp(rng.uniform(-3, 3, (16, 1, 1)))).astype(np.float32)
        for t in range(16):
            ref.append(c, np.array([[0]]), [t + 1], rows[t:t + 1], rows[t:t + 1], None, [1])
        off = np.abs(c.held("k", [0], 0, 16) - rows[:, 0])
        assert off.max() < c.scale["k"][0, 0]


def test_ref_evict_hand_case():
    c = empty_cache(4, 1, 16, 4)
    c.codes["k"][0, 0, :, 0] = np.arange(16)
    c.codes["k"][1, 0, :, 0] = 100
    c.scale["k"][:] = np.array([[1.0], [0.5], [0], [0]])
    c.scale["v"][:] = 1.0
    c.weight[0, 0] = [5, 1, 7, 7, 2, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, np.nan]
    c.weight[1, 0] = 9
    assert ref.evict(c, np.array([[0, 1]]), [18], np.array([[3]]), 5, 2) == [5]
    # 0, 2, 3 (of the others) and the last two, 16 and 17, halved into page 0's scale
    assert list(c.codes["k"][3, 0, :6, 0]) == [0, 2, 3, 50, 50, 0] and c.scale["k"][3, 0] == 1.0
    assert list(c.weight[3, 0, :5]) == [5, 7, 7, 9, 9]


def test_ref_decode_agrees_with_prompt():
    """The last row of a prompt equals a decode step over a cache that holds its tokens exactly."""
    rng = np.random.default_rng(3)
    n, H, kv, d, P = 21, 4, 2, 8, 16
    k, v = rng.integers(-127, 128, (2, n, kv, d)).astype(np.float32) / 64
    q = rng.standard_normal((n, H, d))
    c = empty_cache(3, kv, P, d)
    table = np.array([[2, 0]])
    for t in range(n):
        c.scale["k"][:] = c.scale["v"][:] = 1 / 64
        for name, x in (("k", k), ("v", v)):
            c.codes[name][table[0, t // P], :, t % P] = np.rint(x[t] * 64)
    o, lse, probs, _, _ = ref.decode(c, table, [n], q[-1:], 0.2)
    po, plse, _, _ = ref.prompt(q, k.astype(np.float64), v.astype(np.float64), [n], 0.2)
    assert np.allclose(o[0], po[-1]) and np.allclose(lse[0], plse[:, -1])
    assert np.isclose(sum(p.sum() for p in probs.values()), H)
