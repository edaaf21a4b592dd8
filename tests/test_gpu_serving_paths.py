"""The serving operators where their kernels change course: many work items per block, maxima that
grow from block to block, values that are not finite in several items, groups of every size, scales
far apart, codes at the middle of two steps, and contexts longer than a block holds in registers or in
shared memory.  Against plain implementations in 64 bits; tolerances as in test_gpu_serving.py."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from padding_free_varlen_b200 import capi
from test_gpu_serving import (DT, OK, call_append, call_decode, call_evict, call_prompt, check_decode, gen, half_step, host, make,
                              randn, same, score_error, starts, status, tables)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from padding_free_varlen_b200 import build
    build.build()
    capi.load()


def plain_prompt(q, k, v, lens, scale):
    """o, log sums, sums of p |v|, largest sum |q||k| per row, in 64 bits on the GPU."""
    T, H, d = q.shape
    g = H // k.shape[1]
    o, mag = (torch.zeros(T, H, d, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, smag = (torch.zeros(H, T, dtype=torch.float64, device="cuda") for _ in range(2))
    at = 0
    for n in lens:
        a, b = at, at + n
        at = b
        if n == 0:
            continue
        later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for j in range(H):
            kk, vv = k[a:b, j // g].double(), v[a:b, j // g].double()
            x = (q[a:b, j].double() @ kk.t() * scale).masked_fill(later, float("-inf"))
            p = torch.softmax(x, 1)
            o[a:b, j], mag[a:b, j], lse[j, a:b] = p @ vv, p @ vv.abs(), torch.logsumexp(x, 1)
            smag[j, a:b] = (q[a:b, j].double().abs() @ kk.abs().t() * scale).masked_fill(later, 0).amax(1)
    return o, lse, mag, smag


def check_plain(q, k, v, lens, scale, o, lse):
    T, d, dt, n = sum(lens), q.shape[2], q.dtype, max(lens)
    ro, rlse, mag, smag = plain_prompt(q[:T], k[:T], v[:T], lens, scale)
    ds, u = score_error(d, smag), half_step(dt)
    tol = mag * (2 * ds.t()[..., None] + n * 2.0 ** -24 + 2.0 ** -20 + u) + u * ro.abs()
    tol = tol + (n * 2.0 ** -25 * float(v[:T].double().abs().max()) + 2.0 ** -25 if dt == torch.float16 else 2.0 ** -60)
    err = (o[:T].double() - ro).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    lerr = (lse[:, :T].double() - rlse).abs()
    assert bool((lerr <= ds + n * 2.0 ** -24 + 2.0 ** -22 * (1 + rlse.abs())).all())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("H,kv,d", [(48, 6, 128), (40, 40, 64), (15, 3, 128)])
def test_prompt_many_items_per_block(dt, H, kv, d):
    """More tiles than the GPU holds at once, of 1 to 5 blocks of keys and none, so that a block goes on
    from item to item: lengths around the tile's and the block's edges among them."""
    r = np.random.default_rng(H)
    lens = [int(x) for x in r.integers(0, 310, 40)] + [0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 0, 0, 320] * 2
    T, g = sum(lens), gen(H + d)
    q, k, v = (randn(g, T + 3, h, d, dt=DT[dt]) for h in (H, kv, kv))
    q[T:] = k[T:] = v[T:] = float("nan")
    st = status()
    o, lse = call_prompt(q, k, v, lens, 1.5 / d ** 0.5, st=st)
    assert int(st) == OK and (o[T:] == 7).all()
    check_plain(q, k, v, lens, 1.5 / d ** 0.5, o, lse)
    for _ in range(5):                                   # whichever block takes an item
        again, l2 = call_prompt(q, k, v, lens, 1.5 / d ** 0.5)
        assert torch.equal(o, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_maxima_that_grow(dt, d):
    """Scores that rise by hundreds from block to block (the output is rescaled each time), fall, and jump
    once by a little less and a little more than the growth that is left standing."""
    H, kv, lens = 8, 2, [700, 130, 64, 500] * 8
    T, g = sum(lens), gen(d)
    v = randn(g, T, kv, d, dt=DT[dt])
    q = torch.ones(T, H, d, device="cuda", dtype=DT[dt])
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens]).float()
    for f in (lambda p: p / 64, lambda p: -p / 64, lambda p: (p >= 64).float() * 0.25 * 64 / d, lambda p: (p // 64 % 2) * 8,
              lambda p: torch.floor(p / 64) * 5.5 * 64 / d):
        k = (torch.zeros(T, kv, d, device="cuda") + f(pos)[:, None, None]).to(DT[dt])
        o, lse = call_prompt(q, k, v, lens, 0.35)
        check_plain(q, k, v, lens, 0.35, o, lse)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prompt_values_not_finite_in_many_items(dt):
    """Every third sequence has values that are not finite, of every kind, at different places of its
    blocks: the other sequences and the rows before them do not change, the rows behind show them."""
    H, kv, d, lens = 32, 4, 128, [200, 90, 300, 64, 65, 129] * 7
    T, g = sum(lens), gen(5)
    q, k, v = (randn(g, T, h, d, dt=DT[dt]) for h in (H, kv, kv))
    want, wl = call_prompt(q, k, v, lens, 0.1)
    bad = v.clone()
    ends = np.cumsum([0] + lens)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    spots = []
    for s in range(0, len(lens), 3):
        t = (s * 37) % lens[s]
        kind = [float("inf"), float("-inf"), float("nan")][s // 3 % 3]
        row = int(ends[s]) + t
        bad[row, s % kv, s % d] = kind
        keep[row:int(ends[s + 1])] = False
        spots.append((row, int(ends[s + 1]), s % kv, s % d, kind))
    o, lse = call_prompt(q, k, bad, lens, 0.1)
    assert torch.equal(o[keep], want[keep]) and torch.equal(lse, wl)
    for row, end, j, col, kind in spots:
        got = o[row:end, j * (H // kv):(j + 1) * (H // kv), col].float()
        assert bool((torch.isnan(got) if kind != kind else (got == kind)).all())
        rest = torch.ones(d, dtype=torch.bool, device="cuda")
        rest[col] = False
        assert torch.equal(o[row:end][..., rest], want[row:end][..., rest])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("H,kv,d", [(14, 2, 128), (5, 1, 64), (16, 1, 128), (22, 2, 64), (12, 12, 128)])
@pytest.mark.parametrize("window", [1, 32, 37, 64, 65, 300, 1 << 30])
def test_key_weights_groups(dt, H, kv, d, window):
    """Groups of 1, 5, 7, 8, 11 and 16 heads, shared by clusters of every size; steps over several tiles."""
    lens = [700, 0, 129, 1, 384, 511]
    T, g = sum(lens), gen(H)
    q, k, v = (randn(g, T, h, d, dt=DT[dt]) for h in (H, kv, kv))
    scale = 1.2 / d ** 0.5
    _, rlse, _, smag = plain_prompt(q, k, v, lens, scale)
    lse = rlse.float()
    w, st = torch.full((kv, T), 7.0, device="cuda"), status()
    capi.energon_prompt_key_weights(q, H * d, k, kv * d, lse, starts(lens), len(lens), T, H, kv, d, capi.DTYPE_OF[DT[dt]], scale,
                                    window, w, st)
    assert int(st) == OK
    want, at = torch.zeros(kv, T, dtype=torch.float64, device="cuda"), 0
    for n in lens:
        a, b = at, at + n
        at = b
        w0 = max(0, n - window)
        for j in range(H if n else 0):
            x = q[a + w0:b, j].double() @ k[a:b, j // (H // kv)].double().t() * scale
            p = torch.exp(x - lse[j, a + w0:b].double()[:, None])
            seen = torch.arange(n, device="cuda")[None, :] <= torch.arange(w0, n, device="cuda")[:, None]
            want[j // (H // kv), a:b] += torch.where(seen, p, torch.zeros_like(p)).sum(0)
    # 2^-22 of each exponential beside the errors of its exponent and the sum's
    rel = score_error(d, smag.max()) + 2.0 ** -22 * (rlse.abs().max() + 5) + max(lens) * (H // kv) * 2.0 ** -24
    assert bool(((w.double() - want).abs() <= want * rel + 1e-30).all())


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("P", [16, 64])
def test_cache_attention_scales_far_apart(dt, P):
    """Value scales from 1e-30 to 1e3 and 0 over the pages of one sequence, in rising and falling order;
    key scales over six orders of magnitude."""
    H, kv, d, n = 8, 2, 128, 40 * P + 5
    g = gen(P)
    for order in (1, -1):
        t = make(42, kv, P, d, seed=2)
        table = np.arange(41, dtype=np.int32)[None, ::order].copy()
        s = torch.logspace(-30, 3, 42, device="cuda")
        t[3][:] = s[:, None]
        t[3][7] = 0
        t[2][:] = torch.logspace(-8, -2, 42, device="cuda")[torch.randperm(42, device="cuda", generator=g)][:, None]
        q = randn(g, 1, H, d, dt=DT[dt])
        before = [x.clone() for x in t]
        o, lse = call_decode(t, table, [n], q, 0.02, accumulate=1)
        check_decode(before, table, [n], q, 0.02, o, lse, t[4])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("H,kv", [(3, 1), (10, 2), (7, 1), (24, 8), (33, 1), (17, 1)])
def test_cache_attention_groups_with_weights(dt, H, kv):
    """Groups that are no multiple of 4, odd, and larger than a tile of queries; one and several splits."""
    d, P, lens = 64, 32, [700, 33, 1, 0, 320]
    t = make(60, kv, P, d, seed=H)
    table = tables(lens, P, 60, 2)
    q = randn(gen(H), len(lens), H, d, dt=DT[dt])
    before = [x.clone() for x in t]
    o, lse = call_decode(t, table, lens, q, 0.1, accumulate=1)
    check_decode(before, table, lens, q, 0.1, o, lse, t[4])


def test_cache_attention_scores_that_grow():
    """Scores that rise by more than the growth left standing from step to step, in one warp's and in
    other warps' steps."""
    H, kv, d, P, n = 4, 1, 128, 64, 2500
    t = make(40, kv, P, d, seed=1)
    t[0][:] = 1
    table = np.arange(40, dtype=np.int32)[None]
    for s in (torch.arange(40) * 0.3, 12 - torch.arange(40) * 0.3, (torch.arange(40) % 5) * 2.0):
        t[2][:] = s.cuda()[:, None] + 1e-3
        q = torch.ones(1, H, d, device="cuda")
        for dt in DT.values():
            o, lse = call_decode(t, table, [n], q.to(dt), 0.1)
            check_decode(t, table, [n], q.to(dt), 0.1, o, lse)


@pytest.mark.parametrize("dt", DT)
def test_append_between_two_codes(dt):
    """Elements whose quotient lies exactly or nearly in the middle of two codes: halves of whole numbers
    over a largest element of 127, and all 16-bit mantissas over others."""
    kv, d, P = 1, 128, 64
    halves = torch.arange(-127, 127.5, 0.5, device="cuda")
    for top in (127.0, 127.0 * 2.0 ** -20, 3.0, 251.0, 1.0 / 3):
        x = torch.zeros(P * d, device="cuda")
        x[:halves.numel()] = halves / 127 * top
        x[1000:1256] = (128 + torch.arange(256, device="cuda")) / 256 * top
        x[2000:4000] = torch.rand(2000, device="cuda", generator=gen(3)) * 2 * top - top
        x[-1] = top
        x = x.view(P, kv, d).to(DT[dt])
        t = make(2, kv, P, d)
        h = host(t)
        xs = x.double().cpu().numpy().astype(np.float32)
        ref.append(h, np.array([[1]]), [P], xs, xs, None, [P])
        call_append(t, np.array([[1]], np.int32), [P], x, x.clone(), [P])
        same(t, h)


@pytest.mark.parametrize("top", [3e38, 1e36, 1e-25, 1e-30, 2e-36, 1e-37])
def test_append_scales_at_the_ends_of_the_range(top):
    kv, d, P = 2, 64, 16
    x = randn(gen(1), 5, kv, d).clamp(-3, 3) / 3 * top
    for dt in (torch.float32, torch.bfloat16):
        y = x.to(dt)
        t = make(3, kv, P, d)
        h = host(t)
        ys = y.double().cpu().numpy().astype(np.float32)
        for i in range(5):                               # one by one: scales that double
            z = (y[i:i + 1] * (1 if i == 4 else 0.01)).to(dt)
            zs = z.double().cpu().numpy().astype(np.float32)
            ref.append(h, np.array([[2]]), [i + 1], zs, zs, None, [1])
            call_append(t, np.array([[2]], np.int32), [i + 1], z, z.clone(), [1])
        same(t, h)
        ref.append(h, np.array([[1]]), [5], ys, ys, None, [5])
        call_append(t, np.array([[1]], np.int32), [5], y, y.clone(), [5])
        same(t, h)


@pytest.mark.parametrize("n", [8192, 8193, 16500, 58000])
@pytest.mark.parametrize("kind", ["random", "ties"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long_contexts(n, kind, in_place):
    """Weights in registers, in shared memory and (the last) in the cache alone."""
    kv, d, P, budget, recent = 1, 64, 128, 700, 65
    lens = [n, 900]
    n_pages = sum(-(-x // P) for x in lens)
    per = -(-budget // P)
    t = make(n_pages + 2 * per, kv, P, d, seed=n)
    if kind == "ties":
        t[4] = (t[4] * 8).round() - 4
    table = tables(lens, P, n_pages, 9)
    new_table = table if in_place else (np.arange(2 * per).reshape(2, per).astype(np.int32) + n_pages)
    h, st = host(t), status()
    want = ref.evict(h, table, lens, new_table, budget, recent)
    assert call_evict(t, table, lens, new_table, budget, recent, st) == want
    assert int(st) == OK
    same(t, h)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_between_two_codes(in_place):
    """Ratios of scales that put the fp32 product of a code into the middle of two, where the exact
    product lies beside it: every code times several such ratios."""
    kv, d, P = 1, 64, 16
    ratios = [1.0, 0.65, 0.55, 0.85, 0.35, 0.15, 0.95, 0.05, 0.7, 0.9, 0.1, 0.3]
    n = len(ratios) * P
    t = make(2 * len(ratios), kv, P, d, seed=1)
    for i, r in enumerate(ratios):
        t[2][i] = t[3][i] = float(np.float32(r) * np.float32(0.0173))
    for c in t[:2]:
        c[:len(ratios)] = ((torch.arange(P * d, device="cuda") * 7) % 255 - 127).to(torch.int8).view(1, 1, P, d)
    t[4][:] = torch.rand(t[4].shape, device="cuda", generator=gen(2))
    t[4][0] = 2                                          # the page of the largest scale is met by all
    table = np.arange(len(ratios), dtype=np.int32)[None]
    new_table = table if in_place else table + len(ratios)
    for budget in (n - 1, 3 * P, P):
        u = [x.clone() for x in t]
        h = host(u)
        want = ref.evict(h, table, [n], new_table, budget, 3)
        assert call_evict(u, table, [n], new_table, budget, 3) == want
        same(u, h)


def test_calls_on_two_streams_at_once():
    """Two long calls of each operator, on two streams with outputs and workspaces of their own."""
    H, kv, d, P = 16, 4, 128, 64
    lens = [900, 300, 1500]
    T, g = sum(lens), gen(3)
    q, k, v = (randn(g, T, h, d, dt=torch.bfloat16) for h in (H, kv, kv))
    t = make(64, kv, P, d, seed=4)
    table = tables(lens, P, 64, 4)
    one = randn(g, len(lens), H, d, dt=torch.bfloat16)
    want, wl = call_prompt(q, k, v, lens, 0.1)
    wd, wdl = call_decode(t, table, lens, one, 0.1)
    torch.cuda.synchronize()
    got = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((call_prompt(q, k, v, lens, 0.1), call_decode(t, table, lens, one, 0.1)))
    torch.cuda.synchronize()
    for (o, lse), (x, xl) in got:
        assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(x, wd) and torch.equal(xl, wdl)
