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

# ------------------------------------------------------------------ offsets that step back


def accepted(cu, rows):
    """Which sequences are computed: rows inside [0, rows], and none between the first and the last row of those before."""
    lo, hi, good = None, None, []
    for a, b in zip(cu, cu[1:]):
        inside = 0 <= a <= b <= rows
        good.append(inside and (a == b or lo is None or a >= hi or b <= lo))
        if inside and a < b:
            lo, hi = (a, b) if lo is None else (min(lo, a), max(hi, b))
    return good


def stepping(seed, batch, rows):
    """Offsets of `batch` sequences with some steps back and some outside the rows."""
    r = np.random.default_rng(seed)
    cu, at = [], int(r.integers(0, rows // 2))
    for _ in range(batch + 1):
        cu.append(at)
        at += int(r.choice([0, 1, 40, 130, 300]))
        kind = r.random()
        if kind < 0.08:
            at = int(r.integers(0, rows))
        elif kind < 0.11:
            at = int(r.choice([-5, rows + 9, 1 << 30]))
        at = at if at < rows or kind >= 0.08 else rows
        if at > rows and kind >= 0.11:
            at = int(r.integers(0, rows // 2))
    return cu


STEPS = [([0, 1000, 10, 2000, 3000, 4000], 4000), ([5, 5, -1, 0, 10, 400, 399, 700], 700), ([600, 900, 0, 300, 600, 650], 900),
         ([0, 128, 0, 128, 0, 128, 0, 128, 256], 256)] + [(stepping(s, n, 2500), 2500) for s, n in ((1, 20), (2, 70), (3, 200))]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("case", range(len(STEPS)))
def test_prompts_offsets_that_step_back(dt, case):
    """Sequences whose rows belong to others too are left out; all the others are computed, none twice."""
    cu, rows = STEPS[case]
    H, kv, d, B = 2, 1, 64, len(cu) - 1
    g = gen(case)
    q, k, v = (randn(g, rows, h, d, dt=DT[dt]) for h in (H, kv, kv))
    o, lse = torch.full((rows, H, d), 7.0, dtype=DT[dt], device="cuda"), torch.full((H, rows), 7.0, device="cuda")
    w, want_w = (torch.full((kv, rows), 7.0, device="cuda") for _ in range(2))
    want, want_l, good = o.clone(), lse.clone(), accepted(cu, rows)
    code, st, st2 = capi.DTYPE_OF[DT[dt]], status(), status()
    capi.energon_prompt_attention(q, H * d, k, kv * d, v, kv * d, ints(cu), B, rows, H, kv, d, code, 0.2, o, H * d, lse, st)
    assert int(st) == (OK if all(good) else capi.ENERGON_DEVICE_BAD_LENGTH) and not all(good)
    for a, b, ok in zip(cu, cu[1:], good):
        if ok and a < b:
            x, l = call_prompt(q[a:b], k[a:b], v[a:b], [b - a], 0.2)
            want[a:b], want_l[:, a:b] = x, l
            part = torch.empty(kv, b - a, device="cuda")
            capi.energon_prompt_key_weights(q[a:b], H * d, k[a:b], kv * d, l.contiguous(), starts([b - a]), 1, b - a, H, kv, d,
                                            code, 0.2, 33, part)
            want_w[:, a:b] = part
    assert torch.equal(o, want) and torch.equal(lse, want_l)
    capi.energon_prompt_key_weights(q, H * d, k, kv * d, want_l, ints(cu), B, rows, H, kv, d, code, 0.2, 33, w, st2)
    assert torch.equal(w, want_w) and int(st2) == capi.ENERGON_DEVICE_BAD_LENGTH


@pytest.mark.parametrize("case", range(len(STEPS)))
def test_append_offsets_that_step_back(case):
    cu, rows = STEPS[case]
    kv, d, P, B = 1, 64, 16, len(cu) - 1
    good = accepted(cu, rows)
    lens = [min(max(b - a, 0), rows) + 3 for a, b in zip(cu, cu[1:])]
    pages = sum(-(-n // P) for n in lens)
    t, x = make(pages, kv, P, d, seed=case), randn(gen(case), rows, kv, d)
    table, h, st = tables(lens, P, pages, 2), host(make(pages, kv, P, d, seed=case)), status()
    xs = f64(x).astype(np.float32)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        if good[i]:
            ref.append(h, table[i:i + 1], [lens[i]], xs[a:b], xs[a:b], None, [b - a])
    c = capi.make_kv_cache(*t)
    capi.energon_kv_append(c, ints(table), table.shape[1], ints(lens), x, kv * d, x.clone(), kv * d, None, ints(cu), B, rows,
                           capi.ENERGON_F32, st)
    assert int(st) == capi.ENERGON_DEVICE_BAD_LENGTH
    same(t, h)

# ------------------------------------------------------------------ value scales far apart


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("small", [1e-3, 1e-6, 1e-10, 1e-30])
@pytest.mark.parametrize("big", ["first", "last", "between", "every other"])
@pytest.mark.parametrize("pages", [40, 400])
def test_cache_attention_large_scale_without_weight(dt, P, small, big, pages):
    """Pages of value scale 1 whose tokens have next to no probability beside pages of small scales that have
    all of it: the error is relative to what the output is made of."""
    H, kv, d, n = 6, 2, 64, pages * P - 5
    t, g = make(pages, kv, P, d, seed=P), gen(P)
    t[0][:] = torch.randint(1, 4, t[0].shape, device="cuda", generator=g, dtype=torch.int8)
    t[2][:], t[3][:] = 0.01, small
    at = {"first": [0], "last": [pages - 1], "between": [pages // 2, pages // 2 + 3], "every other": list(range(0, pages, 2))}[big]
    for p in at:                                           # 60 and more below the others' scores, in units of log2 87
        t[0][p], t[2][p], t[3][p] = -100, 0.01, 1.0
    if small == 1e-3:
        t[2][at] = 0.0025                                  # 15 below: their part of the output counts a little
    q = torch.ones(1, H, d, device="cuda", dtype=DT[dt]) + randn(g, 1, H, d, dt=DT[dt]) / 16
    table = np.arange(pages, dtype=np.int32)[None]
    o, lse = call_decode(t, table, [n], q, 1.0)
    ro, rlse, probs, mag, smag = ref.decode(host(t), table, [n], f64(q), 1.0)
    # (the pages without weight have larger scores, whose errors do not count: less than 2^-28 of the output)
    smag = ref.decode(host(t), table, [n], f64(q), 1.0, good=lambda b, i: i // P not in at)[4]
    ds, u = score_error(d, smag) * (4 if dt == "f32" else 1), half_step(DT[dt])
    scale = np.repeat(t[3].cpu().numpy().astype(np.float64), P, 0)[:n]        # [n, kv]
    top = np.array([[(probs[0, h] * scale[:, h // 3]).max() for h in range(H)]])
    # a probability times its scale: half a step of fp16 (2^-22 in two terms), but not finer than 2^-25 of a unit
    # that the largest of them reaches 2^5 of
    rel = 2 * ds[..., None] + n * 2.0 ** -24 + 2.0 ** -19 + (u if dt != "f32" else 0.0) + (2.0 ** -11 if dt != "f32" else 2.0 ** -22)
    tol = mag * rel + u * np.abs(ro) + n * 2.0 ** -30 * 127 * top[..., None]
    if dt == "f16":
        tol = tol + 2.0 ** -25
    err = np.abs(f64(o) - ro)
    assert (err <= tol).all(), float((err / tol).max())
    lerr = np.abs(f64(lse) - rlse)
    assert (lerr <= ds + n * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(rlse))).all()

# ------------------------------------------------------------------ probabilities below the normal range of fp16


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("below", [14.5, 20.5, 23.4375, 27.0])
def test_prompt_many_small_probabilities(dt, d, below):
    """One key takes nearly all the weight and its value is 0; the others, `below` powers of two less each,
    make the output: it is as exact as their own rounding."""
    H, kv, lens = 2, 1, [900, 70]
    T, g = sum(lens), gen(d)
    q, k = torch.zeros(T, H, d, device="cuda", dtype=DT[dt]), torch.zeros(T, kv, d, device="cuda", dtype=DT[dt])
    q[:, :, 0] = 1
    v = (torch.rand(T, kv, d, device="cuda", generator=g) + 1).to(DT[dt]) * 2 ** 10
    for first in (0, 900):
        k[first, 0, 0], v[first] = below, 0
    scale = float(np.log(2.0))
    o, lse = call_prompt(q, k, v, lens, scale)
    ro, rlse, mag, smag = ref.prompt(f64(q), f64(k), f64(v), lens, scale)
    ds, u = score_error(d, smag), half_step(DT[dt])
    tol = mag * (2 * ds.T[..., None] + 900 * 2.0 ** -24 + 2.0 ** -20 + u) + u * np.abs(ro)
    if dt == "f16":
        # 2^-25 of a unit in which a probability of 1 is 2^7; the output's own smallest half step
        tol = tol + 900 * 2.0 ** -32 * 2.0 ** 11 + 2.0 ** -25
    err = np.abs(f64(o) - ro)
    assert (err <= tol).all(), float((err / tol).max())
    lerr = np.abs(f64(lse) - rlse)
    assert (lerr <= ds + 900 * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(rlse))).all()

# ------------------------------------------------------------------ one status word for all calls


@pytest.mark.parametrize("dtype", [synth.F32, synth.F16])
def test_a_notice_of_the_cache_does_not_stop_the_layers(dtype):
    """A layer and the cache's calls share a status word: what an append says about a value or a page leaves
    the layer's work alone; a wait that ran out and a bad length still stop it."""
    shape = synth.LayerShape(256, 4, 1024)
    lens, S = [5, 9], 16
    T, tdt = sum(lens), TORCH_OF_SYNTH[dtype]
    _, dev_w = gpu_layer_weights(shape, 0, 7, dtype, synth.WeightRecipe(w_std=0.02, bias_std=0.1, gamma_std=0.2, beta_std=0.1))
    cfg = capi.make_config(shape.hidden, shape.n_heads, shape.ffn, SYNTH_TO_ENERGON[dtype])
    n = capi.energon_workspace_bytes(cfg, len(lens), S)
    ws, w = torch.empty(n, dtype=torch.uint8, device="cuda"), capi.make_weights(dev_w)
    x = randn(gen(1), len(lens) * S, shape.hidden, dt=tdt)

    def layer(st):
        y = torch.full_like(x, 7.0)
        capi.energon_layer_forward(cfg, w, x, starts(lens), len(lens), S, y, st, ws, n)
        return y
    st = status()
    want = layer(st)
    assert int(st) == OK and not bool((want[:T] == 7).all(1).any())
    # the layer's keys and values go to a cache, one of them infinite
    t = make(2, 4, 16, 64)
    kv = want[:T].view(T, 4, 64).clone()
    kv[3, 1, 5] = float("inf")
    call_append(t, np.array([[0], [1]], np.int32), lens, kv, kv.clone(), lens, st=st)
    assert int(st) == capi.ENERGON_DEVICE_NONFINITE
    assert torch.equal(layer(st)[:T], want[:T]) and int(st) == capi.ENERGON_DEVICE_NONFINITE
    call_append(t, np.array([[0], [9]], np.int32), lens, kv, kv.clone(), lens, st=st)
    assert int(st) == capi.ENERGON_DEVICE_NONFINITE | capi.ENERGON_DEVICE_BAD_PAGE
    assert torch.equal(layer(st)[:T], want[:T])
    for bit in (capi.ENERGON_DEVICE_BAD_LENGTH, capi.ENERGON_DEVICE_TIMEOUT):
        st = status() + bit
        assert bool((layer(st) == 7).all()) and int(st) == bit

# ------------------------------------------------------------------ waits that run out


@pytest.fixture
def short_waits():
    capi.energon_set_wait_timeout_us(1)
    yield
    capi.energon_set_wait_timeout_us(2000000)


def busy(stream, n=6):
    """Memory traffic beside the call, so that its loads take longer than the limit."""
    a = torch.empty(1 << 28, dtype=torch.int32, device="cuda")
    a.record_stream(stream)
    with torch.cuda.stream(stream):
        for _ in range(n):
            a.copy_(a.roll(1))


def test_waits_that_run_out(short_waits):
    """A limit of a microsecond: a call ends, in far less than the second that it grants copies in flight, and
    says that a wait ran out or has computed everything; a call with its limit back, on the same buffers, has the
    usual bits.  What ran out stops the calls behind it."""
    g, side, ran_out = gen(1), torch.cuda.Stream(), 0
    P, lens, ctx = 64, [1500, 700, 130, 64] * 4, [9000, 3000, 500, 70]
    for dt, H, kv, d in ((torch.bfloat16, 16, 4, 128), (torch.float16, 8, 8, 64), (torch.float16, 24, 2, 128)):
        T, code, scale = sum(lens), capi.DTYPE_OF[dt], d ** -0.5
        q, k, v = (randn(g, T, h, d, dt=dt) for h in (H, kv, kv))
        cu, B = starts(lens), len(lens)
        t = make(220, kv, P, d, seed=2)
        table, one = tables(ctx, P, 220, 3), randn(g, len(ctx), H, d, dt=dt)
        cache, tab, ctx_lens = capi.make_kv_cache(*t), ints(table), ints(ctx)
        ws = torch.empty(capi.energon_cache_attention_workspace_bytes(cache, len(ctx), max(ctx), H, 1), dtype=torch.uint8, device="cuda")
        held = t[4].clone()

        def prompt(out, st):
            capi.energon_prompt_attention(q, H * d, k, kv * d, v, kv * d, cu, B, T, H, kv, d, code, scale, out[0], H * d, out[1], st)

        def weights(window):
            def call(out, st):
                capi.energon_prompt_key_weights(q, H * d, k, kv * d, lse, cu, B, T, H, kv, d, code, scale, window, out[0], st)
            return call

        def decode(out, st):
            t[4].copy_(held)
            capi.energon_cache_attention(cache, tab, table.shape[1], ctx_lens, len(ctx), max(ctx), one, H * d, H, code, scale, out[0],
                                         H * d, out[1], 1, st, ws, ws.numel())
            out[2].copy_(t[4])
        new = lambda *s, dt=torch.float32: torch.full(s, 7.0, dtype=dt, device="cuda")  # noqa: E731
        shapes = {prompt: lambda: [new(T, H, d, dt=dt), new(H, T)], weights(40): lambda: [new(kv, T)],
                  weights(1 << 30): lambda: [new(kv, T)],
                  decode: lambda: [new(len(ctx), H, d, dt=dt), new(len(ctx), H), torch.empty_like(held)]}
        capi.energon_set_wait_timeout_us(2000000)
        want = prompt_out = shapes[prompt]()
        prompt(want, status())
        lse = prompt_out[1]
        for call, outs in shapes.items():
            capi.energon_set_wait_timeout_us(2000000)
            want, st = outs(), status()
            call(want, st)
            assert int(st) == OK
            for i in range(6):
                capi.energon_set_wait_timeout_us(1)
                out, st = outs(), status()
                a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                torch.cuda.synchronize()
                if i % 2:
                    busy(side)
                a.record()
                call(out, st)
                b.record()
                torch.cuda.synchronize()
                assert a.elapsed_time(b) < 500.0
                assert int(st) in (OK, capi.ENERGON_DEVICE_TIMEOUT)
                if int(st) == OK:
                    assert all(torch.equal(x, y) for x, y in zip(out, want))
                else:
                    ran_out += 1
                    behind = outs()
                    capi.energon_set_wait_timeout_us(2000000)
                    call(behind, st)
                    assert all(bool((x == 7).all()) for x in behind[:2])
                capi.energon_set_wait_timeout_us(2000000)
                again, st = outs(), status()
                call(again, st)
                assert int(st) == OK and all(torch.equal(x, y) for x, y in zip(again, want))
    assert ran_out
