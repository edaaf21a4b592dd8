"""The serving operators on calls at the edge of what their documentation allows: queries and scales that
are not finite, offsets that step back, value scales and probabilities far apart, one status word for
layers and serving calls, waits that run out.  Tolerances as in test_gpu_serving.py unless derived here."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from padding_free_varlen_b200 import capi, synth
from helpers import SYNTH_TO_ENERGON, TORCH_OF_SYNTH, gpu_layer_weights
from test_gpu_serving import (DT, OK, call_append, call_decode, call_prompt, f64, gen, half_step, host, ints, make, randn, same,
                              score_error, starts, status, tables)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from padding_free_varlen_b200 import build
    build.build()
    capi.load()


# ------------------------------------------------------------------ queries and scales that are not finite


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("lens", [[1, 40, 0], [700, 33, 700], [5000]], ids=str)
@pytest.mark.parametrize("acc", [0, 1])
def test_cache_attention_query_not_finite(dt, bad, lens, acc):
    """It shows in its own head's output and log sum (and in the weights its head adds to), like in a plain
    softmax, and nowhere else; an empty sequence stays empty."""
    H, kv, d, P = 6, 2, 64, 16
    pages = sum(-(-n // P) for n in lens)
    t = make(pages, kv, P, d, seed=3)
    t[0][:, :, 0] = -t[0][:, :, 0].abs()                  # (one sign alone among some tokens' codes)
    table = tables(lens, P, pages, 1)
    q = randn(gen(2), len(lens), H, d, dt=DT[dt])
    clean = [x.clone() for x in t]
    want, wl = call_decode(clean, table, lens, q, 0.1, accumulate=acc)
    q2 = q.clone()
    q2[:, 4, 9] = bad
    o, lse = call_decode(t, table, lens, q2, 0.1, accumulate=acc)
    rest = [0, 1, 2, 3, 5]
    assert torch.equal(o[:, rest], want[:, rest]) and torch.equal(lse[:, rest], wl[:, rest])
    for b, n in enumerate(lens):
        if n:
            assert bool(torch.isnan(o[b, 4]).all()) and bool(torch.isnan(lse[b, 4]))
        else:
            assert bool((o[b] == 0).all()) and bool((lse[b] == float("-inf")).all())
    assert torch.equal(t[4][:, 0], clean[4][:, 0])
    if acc:
        for b, n in enumerate(lens):
            for i in (0, n - 1)[:min(n, 2)]:
                assert bool(torch.isnan(t[4][int(table[b, i // P]), 1, i % P]))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("n", [32, 128, 900, 5000])
@pytest.mark.parametrize("which", [2, 3])
def test_cache_attention_scale_not_a_number(dt, n, which):
    """A page whose scale is NaN, in every place that a page can have in the work: all outputs of its head are NaN."""
    H, kv, d, P = 4, 2, 128, 32
    pages = -(-n // P)
    t = make(pages, kv, P, d, seed=4)
    q = randn(gen(5), 1, H, d, dt=DT[dt])
    table = np.arange(pages, dtype=np.int32)[None]
    want, wl = call_decode(t, table, [n], q, 0.1)
    for p in {0, 1 % pages, pages // 2, pages - 1}:
        u = [x.clone() for x in t]
        u[which][p, 1] = float("nan")
        o, lse = call_decode(u, table, [n], q, 0.1)
        assert torch.equal(o[:, :2], want[:, :2]) and torch.equal(lse[:, :2], wl[:, :2])
        assert bool(torch.isnan(o[:, 2:]).all()), p
        assert bool(torch.isnan(lse[:, 2:]).all()) if which == 2 else torch.equal(lse, wl), p
