"""The serving operators on the GPU against plain implementations in 64 bits.

Tolerances are sums of the roundings an operator may make, each at most half a step:
u = eps / 2 of the 16-bit type for the probabilities of the product with V (against sum p |v|)
and for the output; a score's error ds from fp32 sums of head_dim products, which moves a
probability by the factor exp(ds); fp32 sums over n tokens.  Codes, scales, selections and
moved weights are exact."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from padding_free_varlen_b200 import capi

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OK = capi.ENERGON_DEVICE_OK


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from padding_free_varlen_b200 import build
    build.build()
    capi.load()


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dt):
    return torch.finfo(dt).eps / 2


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dt=torch.float32):
    return torch.randn(*shape, device="cuda", generator=g).to(dt)


def starts(lens):
    return ints([0] + list(np.cumsum(lens)))


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ prompts

LENGTHS = [[1], [0, 1, 2, 3], [127, 128, 129, 0, 255], [64, 1, 200, 63, 65], [513]]
HEADS = [(4, 4, 128), (8, 2, 128), (6, 2, 64), (3, 1, 128), (5, 5, 64)]


def call_prompt(q, k, v, lens, scale, rows=None, lse=True, st=None, o=None, stream=None):
    rows = q.shape[0] if rows is None else rows
    H, kv, d = q.shape[1], k.shape[1], q.shape[2]
    o = torch.full((rows, H, d), 7.0, dtype=q.dtype, device="cuda") if o is None else o
    out_lse = torch.full((H, rows), 7.0, device="cuda") if lse else None
    capi.energon_prompt_attention(q, q.stride(0), k, k.stride(0), v, v.stride(0), starts(lens), len(lens), rows, H, kv,
                                  d, capi.DTYPE_OF[q.dtype], scale, o, o.stride(0), out_lse, st, stream=stream)
    return o, out_lse


def score_error(d, smag):
    return (d + 16) * 2.0 ** -23 * smag + 2.0 ** -21


def check_prompt(q, k, v, lens, scale, o, lse):
    T, d, dt, n = sum(lens), q.shape[2], q.dtype, max(lens)
    ro, rlse, mag, smag = ref.prompt(f64(q[:T]), f64(k[:T]), f64(v[:T]), lens, scale)
    ds = score_error(d, smag)
    u = half_step(dt)
    rel = 2 * ds.T[..., None] + n * 2.0 ** -24 + 2.0 ** -20 + (u if dt != torch.float32 else 0.0)
    vmax = float(v[:T].double().abs().max()) if T else 0.0
    # probabilities below the normal range of fp16 lose up to 2^-25 each
    tol = mag * rel + u * np.abs(ro) + (n * 2.0 ** -25 * vmax + 2.0 ** -25 if dt == torch.float16 else 2.0 ** -60)
    err = np.abs(f64(o[:T]) - ro)
    assert np.isfinite(err).all() and (err <= tol).all(), float((err / tol).max())
    ltol = ds + n * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(rlse))
    lerr = np.abs(f64(lse[:, :T]) - rlse)
    assert (lerr <= ltol).all(), float((lerr / ltol).max())
    return float((err / tol).max()) if T else 0.0


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("H,kv,d", HEADS)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_prompt_attention(dt, H, kv, d, lens):
    g = gen(sum(lens) + H * d)
    T, extra = sum(lens), 5
    q, k, v = (randn(g, T + extra, h, d, dt=DT[dt]) for h in (H, kv, kv))
    for x in (q, k, v):
        x[T:] = float("nan")                       # rows behind the last sequence
    st = status()
    scale = 1.7 / d ** 0.5
    o, lse = call_prompt(q, k, v, lens, scale, st=st)
    assert int(st) == OK and (o[T:] == 7).all() and (lse[:, T:] == 7).all()
    check_prompt(q, k, v, lens, scale, o, lse)
    o2, _ = call_prompt(q, k, v, lens, scale, lse=False)
    assert torch.equal(o, o2)                      # run to run, and without the log sums


@pytest.mark.parametrize("dt", DT)
def test_prompt_attention_views_of_fused_rows(dt):
    """Q, K and V as parts of one fused row, in the layer's order, and o inside wider rows."""
    H, kv, d, lens = 4, 2, 128, [70, 131]
    T = sum(lens)
    fused = randn(gen(1), T, (H + 2 * kv) * d + 16, dt=DT[dt])
    q = fused[:, :H * d].view(T, H, d)
    k = fused[:, H * d:(H + kv) * d].view(T, kv, d)
    v = fused[:, (H + kv) * d:(H + 2 * kv) * d].view(T, kv, d)
    wide = torch.full((T, H * d + 8), 3.0, dtype=DT[dt], device="cuda")
    o, lse = call_prompt(q, k, v, lens, 0.1, o=wide[:, :H * d].view(T, H, d))
    check_prompt(q, k, v, lens, 0.1, o, lse)
    assert (wide[:, H * d:] == 3).all()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_attention_sharp_and_flat_scores(dt, d):
    """Scores of hundreds (one key takes all the weight), all equal, and rising along the sequence
    (every block brings a new maximum)."""
    lens, H, kv = [300, 140], 4, 2
    T, g = sum(lens), gen(2)
    q, k, v = (randn(g, T, h, d, dt=DT[dt]) for h in (H, kv, kv))
    o, lse = call_prompt(q, k, v, lens, 4.0)
    check_prompt(q, k, v, lens, 4.0, o, lse)
    o, lse = call_prompt(torch.zeros_like(q), k, v, lens, 1.0)
    check_prompt(torch.zeros_like(q), k, v, lens, 1.0, o, lse)
    rise = torch.arange(T, device="cuda", dtype=torch.float32)[:, None, None] / 32
    for sign in (1, -1):
        kr, qr = (torch.ones_like(k).float() * rise * sign).to(DT[dt]), torch.ones_like(q)
        o, lse = call_prompt(qr, kr, v, lens, 0.25)
        check_prompt(qr, kr, v, lens, 0.25, o, lse)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("H,kv,d", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v", "q"])
def test_prompt_attention_later_values_do_not_reach_earlier_rows(dt, H, kv, d, bad, where):
    """A value that is not finite at position t changes no output before t, wherever t lies in a
    tile, and no other sequence."""
    lens, g = [140, 290, 33], gen(3)
    T = sum(lens)
    q, k, v = (randn(g, T, h, d, dt=DT[dt]) for h in (H, kv, kv))
    want, wl = call_prompt(q, k, v, lens, 0.2)
    for t in (0, 1, 17, 63, 64, 127, 128, 200, 289):
        x = {"q": q.clone(), "k": k.clone(), "v": v.clone()}
        x[where][140 + t, -1, 5] = bad
        o, lse = call_prompt(x["q"], x["k"], x["v"], lens, 0.2)
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[140 + t:430] = False
        if where == "q":
            keep[140 + t + 1:430] = True
        assert torch.equal(o[keep], want[keep]), t
        assert torch.equal(lse[:, keep], wl[:, keep]), t
        if where == "v":
            sees = o[140 + t:430, -1, 5].float()
            assert (torch.isnan(sees) if bad != bad else torch.isnan(sees) | (sees == bad)).all(), t
            rest = torch.ones(d, dtype=torch.bool, device="cuda")
            rest[5] = False
            assert torch.equal(o[140 + t:430, :, rest], want[140 + t:430, :, rest])


@pytest.mark.parametrize("dt", DT)
def test_prompt_attention_bad_lengths_and_status(dt):
    H, kv, d = 4, 2, 64
    g = gen(4)
    q, k, v = (randn(g, 50, h, d, dt=DT[dt]) for h in (H, kv, kv))
    for cu in ([10, 20, 0, 10], [0, 20, 51, 50], [-3, 20, 30, 50], [0, 1 << 30, 30, 50]):
        o = torch.full((50, H, d), 7.0, dtype=DT[dt], device="cuda")
        st = status()
        capi.energon_prompt_attention(q, H * d, k, kv * d, v, kv * d, ints(cu), 3, 50, H, kv, d, capi.DTYPE_OF[DT[dt]],
                                      0.2, o, H * d, None, st)
        assert int(st) == capi.ENERGON_DEVICE_BAD_LENGTH
        for a, b in zip(cu, cu[1:]):               # the good sequences are computed all the same
            if 0 <= a <= b <= 50:
                want, _ = call_prompt(q[a:b], k[a:b], v[a:b], [b - a], 0.2)
                assert torch.equal(o[a:b], want)
    st = status() + 2
    o = torch.full((50, H, d), 7.0, dtype=DT[dt], device="cuda")
    call_prompt(q, k, v, [50], 0.2, st=st, o=o)
    assert int(st) == 2 and (o == 7).all()         # a wait ran out before: no work
    call_prompt(q, k, v, [0, 0], 0.2, o=o)
    call_prompt(q[:0], k[:0], v[:0], [0], 0.2)
    capi.energon_prompt_attention(q, H * d, k, kv * d, v, kv * d, starts([]), 0, 50, H, kv, d, capi.DTYPE_OF[DT[dt]], 0.2,
                                  o, H * d)
    assert (o == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_prompt_attention_many_sequences(dt):
    """More sequences than a warp looks at in one step, most of them short or empty."""
    lens = [(i * 37) % 11 for i in range(300)] + [400] + [0] * 40
    H, kv, d = 2, 1, 64
    T, g = sum(lens), gen(5)
    q, k, v = (randn(g, T, h, d, dt=DT[dt]) for h in (H, kv, kv))
    o, lse = call_prompt(q, k, v, lens, 0.2)
    check_prompt(q, k, v, lens, 0.2, o, lse)


# ------------------------------------------------------------------ key weights


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("H,kv,d", HEADS)
@pytest.mark.parametrize("window", [1, 5, 64, 200, 1 << 40])
def test_key_weights(dt, H, kv, d, window):
    lens = [129, 0, 1, 64, 300, 2]
    T, g = sum(lens), gen(H + d)
    q, k, v = (randn(g, T + 3, h, d, dt=DT[dt]) for h in (H, kv, kv))
    q[T:] = k[T:] = float("nan")
    scale = 1.3 / d ** 0.5
    _, rlse, _, smag = ref.prompt(f64(q[:T]), f64(k[:T]), f64(v[:T]), lens, scale)
    lse = torch.full((H, T + 3), float("nan"), device="cuda")
    lse[:, :T] = torch.from_numpy(rlse).float()
    w, st = torch.full((kv, T + 3), 7.0, device="cuda"), status()

    def call(out):
        capi.energon_prompt_key_weights(q, H * d, k, kv * d, lse, starts(lens), len(lens), T + 3, H, kv, d,
                                        capi.DTYPE_OF[DT[dt]], scale, window, out, st)
    call(w)
    assert int(st) == OK and (w[:, T:] == 7).all()
    rw = ref.key_weights(f64(q[:T]), f64(k[:T]), f64(lse[:, :T]), lens, scale, window)
    # each term's exponent is off by ds and by the roundings of the sum and of the product with log2(e)
    rel = score_error(d, smag.max()) + 2.0 ** -22 * (np.abs(rlse).max() + 4) + max(lens) * (H // kv) * 2.0 ** -24
    err = np.abs(f64(w[:, :T]) - rw)
    assert (err <= rw * rel + 1e-30).all(), float((err / (rw * rel + 1e-30)).max())
    again = torch.empty_like(w)
    call(again)
    assert torch.equal(w[:, :T], again[:, :T])


def test_key_weights_bad_lengths():
    H, kv, d = 4, 2, 64
    q, k = randn(gen(1), 40, H, d, dt=torch.float16), randn(gen(2), 40, kv, d, dt=torch.float16)
    lse = torch.zeros(H, 40, device="cuda")
    w, st = torch.full((kv, 40), 7.0, device="cuda"), status()
    capi.energon_prompt_key_weights(q, H * d, k, kv * d, lse, ints([0, 50, 40]), 2, 40, H, kv, d, capi.ENERGON_F16, 0.1,
                                    8, w, st)
    assert int(st) == capi.ENERGON_DEVICE_BAD_LENGTH and (w == 7).all()


# ------------------------------------------------------------------ the cache


def make(n_pages, kv, P, d, seed=None, weight=True):
    """A cache on the GPU, filled with codes in use or empty, and its tensors."""
    if seed is None:
        t = [torch.zeros(n_pages, kv, P, d, dtype=torch.int8, device="cuda") for _ in range(2)]
        t += [torch.zeros(n_pages, kv, device="cuda") for _ in range(2)]
        t += [torch.zeros(n_pages, kv, P, device="cuda") if weight else None]
    else:
        g = gen(seed)
        t = [torch.randint(-127, 128, (n_pages, kv, P, d), device="cuda", generator=g, dtype=torch.int8) for _ in range(2)]
        t += [torch.rand(n_pages, kv, device="cuda", generator=g) * 0.02 + 0.001 for _ in range(2)]
        t += [torch.rand(n_pages, kv, P, device="cuda", generator=g) if weight else None]
    return t


def host(t):
    return ref.Cache(*[None if x is None else x.cpu().numpy() for x in t])


def tables(lens, P, n_pages, seed, room=0):
    """Shuffled distinct pages; entries behind the last used one are poison (never read)."""
    need = [-(-n // P) for n in lens]
    most = max(1, max(need) + room)
    t = np.full((len(lens), most), 1 << 30, np.int32)
    order = np.random.default_rng(seed).permutation(n_pages)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    assert at <= n_pages
    return t


def same(t, h):
    for name, codes, scale in (("k", t[0], t[2]), ("v", t[1], t[3])):
        assert np.array_equal(scale.cpu().numpy(), h.scale[name]), name
        assert np.array_equal(codes.cpu().numpy(), h.codes[name]), name
    if t[4] is not None:
        assert np.array_equal(t[4].cpu().numpy(), h.weight, equal_nan=True)


def call_append(t, table, lens, k, v, new, weights=None, st=None):
    c = capi.make_kv_cache(*t)
    capi.energon_kv_append(c, ints(table), table.shape[1], ints(lens), k, k.stride(0), v, v.stride(0), weights, starts(new),
                           len(lens), k.shape[0], capi.DTYPE_OF[k.dtype], st)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("kv,d,P", [(2, 128, 64), (3, 64, 16), (1, 128, 128), (2, 64, 32)])
@pytest.mark.parametrize("new", [None, 1, 7, 40], ids=str)
@pytest.mark.parametrize("given", [False, True])
def test_append(dt, kv, d, P, new, given):
    """Whole prompts, single tokens and chunks that begin inside a page, bit for bit."""
    lens = [1, P, P + 1, 3 * P - 1, 0, 41]
    news = [min(n, new) if new else n for n in lens]
    t = make(14, kv, P, d, seed=P + d)
    table = tables(lens, P, 14, 1, room=2)
    T = sum(news)
    g = gen(T + kv)
    k = (randn(g, T + 2, kv, d) * torch.exp(torch.randn(T + 2, 1, 1, device="cuda", generator=g))).to(DT[dt])
    v = randn(g, T + 2, kv, d, dt=DT[dt])
    w = torch.rand(kv, T + 2, device="cuda", generator=g) if given else None
    h, st = host(t), status()
    ref.append(h, table, lens, f64(k).astype(np.float32), f64(v).astype(np.float32), None if w is None else w.cpu().numpy(), news)
    call_append(t, table, lens, k, v, news, w, st)
    assert int(st) == OK
    same(t, h)
    call_append(t, table, lens, k, v, news, w, st)      # the same rows again change nothing
    same(t, h)


@pytest.mark.parametrize("dt", DT)
def test_append_token_by_token(dt):
    """40 steps that grow the scales; every element stays within one final scale."""
    kv, d, P, B, n = 2, 64, 16, 3, 40
    t = make(9, kv, P, d)
    table = tables([n] * B, P, 9, 2)
    h, g = host(t), gen(6)
    rows = []
    for i in range(n):
        k = (randn(g, B, kv, d) * (1 + i % 7) ** 2).to(DT[dt])
        v = randn(g, B, kv, d, dt=DT[dt])
        call_append(t, table, [i + 1] * B, k, v, [1] * B)
        ref.append(h, table, [i + 1] * B, f64(k).astype(np.float32), f64(v).astype(np.float32), None, [1] * B)
        rows.append(f64(k))
    same(t, h)
    rows = np.stack(rows)                                # [n, B, kv, d]
    for b in range(B):
        for j in range(kv):
            off = np.abs(host(t).held("k", table[b], j, n) - rows[:, b, j])
            step = np.repeat([t[2][int(p), j].item() for p in table[b]], P)[:n, None]
            assert (off < step).all()


def test_append_views_zero_rows_and_extremes():
    kv, d, P = 2, 64, 16
    for dt in DT.values():
        t = make(6, kv, P, d, seed=1)
        lens = [20, 5]
        table, T = tables(lens, P, 6, 3), 25
        fused = randn(gen(7), T, 3 * kv * d, dt=dt)
        fused[3] = 0
        fused[20:, :kv * d] = 0                              # a page of zeros: scale 0
        if dt == torch.float32:
            fused[0, :] = 1e-41                              # below the normal range
            fused[21, kv * d] = 3e38
        k, v = fused[:, :kv * d].view(T, kv, d), fused[:, kv * d:2 * kv * d].view(T, kv, d)
        h = host(t)
        ref.append(h, table, lens, f64(k).astype(np.float32), f64(v).astype(np.float32), None, lens)
        call_append(t, table, lens, k, v, lens)
        same(t, h)
        t = make(2, kv, P, d)                                # only values below the normal range
        x = torch.full((1, kv, d), 1e-39, device="cuda").to(dt)
        h = host(t)
        ref.append(h, np.array([[1]]), [1], f64(x).astype(np.float32), f64(x).astype(np.float32), None, [1])
        call_append(t, np.array([[1]], np.int32), [1], x, x.clone(), [1])
        same(t, h)


@pytest.mark.parametrize("dt", DT)
def test_append_not_finite(dt):
    kv, d, P = 1, 64, 16
    t = make(2, kv, P, d)
    x = randn(gen(8), 3, kv, d, dt=DT[dt])
    x[0, 0, 0], x[1, 0, 1], x[2, 0, 2] = float("nan"), float("inf"), float("-inf")
    h, st = host(t), status()
    ref.append(h, np.array([[1]]), [3], f64(x).astype(np.float32), f64(x).astype(np.float32), None, [3])
    call_append(t, np.array([[1]], np.int32), [3], x, x.clone(), [3], st=st)
    assert int(st) == capi.ENERGON_DEVICE_NONFINITE
    same(t, h)
    assert t[0][1, 0, 0, 0] == 0 and t[0][1, 0, 1, 1] == 127 and t[0][1, 0, 2, 2] == -127


def test_append_bad_pages_and_lengths():
    kv, d, P, dt = 2, 64, 16, torch.float16
    x = randn(gen(9), 40, kv, d, dt=dt)
    for page in (-1, 6, 1 << 30):
        t = make(6, kv, P, d, seed=2)
        h, st = host(t), status()
        table = np.array([[0, page], [1, 2]], np.int32)
        call_append(t, table, [20, 20], x, x.clone(), [20, 20], st=st)
        assert int(st) == capi.ENERGON_DEVICE_BAD_PAGE
        xs = f64(x).astype(np.float32)
        ref.append(h, table, [16], xs[:16], xs[:16], None, [16])            # all but the page that is not there
        ref.append(h, table[1:], [20], xs[20:], xs[20:], None, [20])
        same(t, h)
    for lens, new in (([33, 20], [20, 20]), ([19, 20], [20, 20]), ([-1, 20], [20, 20])):
        t = make(6, kv, P, d, seed=2)
        h, st = host(t), status()
        table = np.array([[3, 0], [1, 2]], np.int32)
        call_append(t, table, lens, x, x.clone(), new, st=st)
        assert int(st) == capi.ENERGON_DEVICE_BAD_LENGTH
        ref.append(h, table[1:], [20], xs[20:], xs[20:], None, [20])
        same(t, h)
    t = make(6, kv, P, d, seed=2)
    h, st = host(t), status() + 2
    call_append(t, np.array([[0, 1], [2, 3]], np.int32), [20, 20], x, x.clone(), [20, 20], st=st)
    same(t, h)


# ------------------------------------------------------------------ attention over the cache


def call_decode(t, table, lens, q, scale, max_len=None, accumulate=0, st=None, lse=True):
    c = capi.make_kv_cache(*t)
    B, H, d = q.shape
    max_len = max(max(lens), 0) if max_len is None else max_len
    n = capi.energon_cache_attention_workspace_bytes(c, B, max_len, H, accumulate)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full((B, H, d), 7.0, dtype=q.dtype, device="cuda")
    out = torch.full((B, H), 7.0, device="cuda") if lse else None
    capi.energon_cache_attention(c, ints(table), table.shape[1], ints(lens), B, max_len, q, q.stride(0), H,
                                 capi.DTYPE_OF[q.dtype], scale, o, H * d, out, accumulate, st, ws, n)
    return o, out


def check_decode(t0, table, lens, q, scale, o, lse, weight=None, good=None):
    h = host(t0)
    ro, rlse, probs, mag, smag = ref.decode(h, table, lens, f64(q), scale, good)
    B, H, d = q.shape
    n, u = max(max(lens), 1), half_step(q.dtype)
    # q is held to 2^-22 of its largest element (fp32) or exactly (16-bit) beside the fp32 sums
    ds = score_error(d, smag) * (4 if q.dtype == torch.float32 else 1)
    rel = 2 * ds[..., None] + n * 2.0 ** -24 + 2.0 ** -19 + (u if q.dtype != torch.float32 else 0.0)
    vmax = 127 * max(float(t0[3].max()), 0.0)
    # probabilities below the normal range of fp16 lose up to 2^-25 each
    tol = mag * rel + u * np.abs(ro) + n * 2.0 ** -25 * vmax * (1.0 if q.dtype != torch.float32 else 2.0 ** -11) + 2.0 ** -60
    if q.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = np.abs(f64(o) - ro)
    assert np.isfinite(err).all() and (err <= tol).all(), float((err / tol).max())
    if lse is not None:
        fin = np.isfinite(rlse)
        got = f64(lse)
        assert np.array_equal(np.isneginf(got), ~fin)
        ltol = ds + n * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(np.where(fin, rlse, 0)))
        lerr = np.abs(got[fin] - rlse[fin])
        assert (lerr <= ltol[fin]).all(), float((lerr / ltol[fin]).max())
    if weight is not None:
        want, got = h.weight.astype(np.float64), f64(weight)
        g, bound = H // h.kv, np.zeros_like(want)
        for b, m in enumerate(lens):
            for i in range(max(int(m), 0)):
                p = int(table[b, i // h.P])
                if not 0 <= p < h.n_pages:
                    continue
                for j in range(h.kv):
                    add = sum(probs[b, x][i] for x in range(j * g, (j + 1) * g))
                    want[p, j, i % h.P] += add
                    bound[p, j, i % h.P] += add * (2 * ds[b].max() + n * 2.0 ** -24 + 2.0 ** -19) + 1e-38
        werr = np.abs(got - want)
        assert (werr <= bound + 2.0 ** -23 * want).all()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("H,kv,d,P", [(4, 4, 128, 16), (8, 2, 128, 64), (14, 2, 64, 32), (8, 1, 128, 128), (32, 2, 64, 16),
                                      (40, 2, 128, 64)])
@pytest.mark.parametrize("acc", [0, 1])
def test_cache_attention(dt, H, kv, d, P, acc):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 129, 300, 2]
    t = make(64, kv, P, d, seed=H + d)
    table = tables(lens, P, 64, 4, room=1)
    q = randn(gen(H), len(lens), H, d, dt=DT[dt])
    before = [x.clone() for x in t]
    st = status()
    scale = 2.0 / d ** 0.5
    o, lse = call_decode(t, table, lens, q, scale, accumulate=acc, st=st)
    assert int(st) == OK and (o[0] == 0).all()
    check_decode(before, table, lens, q, scale, o, lse, t[4])if acc else check_decode(before, table, lens, q, scale, o, lse)
    for a, b in zip(t[:4] + ([] if acc else [t[4]]), before):
        assert torch.equal(a, b)
    o2, _ = call_decode(before, table, lens, q, scale, lse=False)     # run to run
    assert torch.equal(o, o2)
    o3, lse3 = call_decode(before, table, lens, q, scale, max_len=table.shape[1] * P, accumulate=0)
    check_decode(before, table, lens, q, scale, o3, lse3)             # a looser bound on the lengths


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("B,H,kv,d,P,n", [(1, 8, 2, 128, 64, 5001), (2, 4, 1, 64, 16, 3001), (1, 2, 2, 128, 128, 9000)])
def test_cache_attention_long(dt, B, H, kv, d, P, n):
    """A long axis with few rows: the work is split over it and joined."""
    lens = [n - 17 * b for b in range(B)]
    pages = sum(-(-x // P) for x in lens) + 1
    t = make(pages, kv, P, d, seed=9)
    table = tables(lens, P, pages, 5)
    q = randn(gen(n), B, H, d, dt=DT[dt])
    before = [x.clone() for x in t]
    o, lse = call_decode(t, table, lens, q, 0.05, accumulate=1)
    check_decode(before, table, lens, q, 0.05, o, lse, t[4])
    o2, _ = call_decode(before, table, lens, q, 0.05)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("dt", DT)
def test_cache_attention_extreme_values(dt):
    """Queries of very large and very small magnitude, a few dominant elements, zero scales, flat scores."""
    H, kv, d, P, lens = 4, 2, 128, 16, [50, 33, 16, 70]
    t = make(16, kv, P, d, seed=3)
    table = tables(lens, P, 16, 6)
    t[2][int(table[0, 1])] = 0                      # a page of zero keys
    t[3][int(table[0, 2])] = 0                      # and one of zero values
    q = randn(gen(4), 4, H, d, dt=torch.float32)
    q[1] *= 1e-6 if dt == "f16" else 1e-20
    q[2] = 0
    q[3, :, 7] = 3000.0
    q = q.to(DT[dt])
    for scale in (1e-4, 0.02, 3.0):
        o, lse = call_decode(t, table, lens, q, scale)
        check_decode(t, table, lens, q, scale, o, lse)


@pytest.mark.parametrize("page", [-1, 20, 1 << 30])
@pytest.mark.parametrize("acc", [0, 1])
def test_cache_attention_bad_pages(page, acc):
    """Tokens of a page that is not there count as masked; a sequence of such pages alone is empty."""
    H, kv, d, P, lens = 4, 2, 64, 32, [70, 20, 64]
    t = make(20, kv, P, d, seed=3)
    table = tables(lens, P, 20, 7)
    table[0, 1] = page
    table[1, 0] = page
    q = randn(gen(5), 3, H, d, dt=torch.bfloat16)
    before = [x.clone() for x in t]
    st = status()
    o, lse = call_decode(t, table, lens, q, 0.2, accumulate=acc, st=st)
    assert int(st) == capi.ENERGON_DEVICE_BAD_PAGE and (o[1] == 0).all()
    check_decode(before, table, lens, q, 0.2, o, lse, t[4] if acc else None,
                 good=lambda b, i: 0 <= table[b, i // P] < 20)


def test_cache_attention_bad_lengths_and_status():
    H, kv, d, P = 4, 2, 64, 16
    t = make(20, kv, P, d, seed=3)
    table = tables([40, 40, 40], P, 20, 8)
    q = randn(gen(5), 3, H, d, dt=torch.float16)
    want, wl = call_decode(t, table, [40, 0, 40], q, 0.2, max_len=48)
    for bad in (-1, 49, 1 << 30):
        st = status()
        o, lse = call_decode(t, table, [40, bad, 40], q, 0.2, max_len=48, st=st)
        assert int(st) == capi.ENERGON_DEVICE_BAD_LENGTH
        assert torch.equal(o, want) and torch.equal(lse, wl) and (o[1] == 0).all()
    st = status() + 2
    before = t[4].clone()
    o, lse = call_decode(t, table, [40, 40, 40], q, 0.2, accumulate=1, st=st)
    assert (o == 7).all() and (lse == 7).all() and torch.equal(before, t[4])
    o, _ = call_decode(t, table, [0, 0, 0], q, 0.2, accumulate=1)      # max_len 0
    assert (o == 0).all() and torch.equal(before, t[4])


def test_cache_attention_shared_pages():
    """Two sequences with a common prefix read the same pages, and both add to their weights."""
    H, kv, d, P, lens = 4, 2, 128, 16, [40, 44]
    t = make(8, kv, P, d, seed=3)
    table = np.array([[5, 1, 2], [5, 1, 6]], np.int32)
    q = randn(gen(5), 2, H, d, dt=torch.bfloat16)
    before = [x.clone() for x in t]
    o, lse = call_decode(t, table, lens, q, 0.2, accumulate=1)
    check_decode(before, table, lens, q, 0.2, o, lse, t[4])


def test_cache_attention_offsets_beyond_32_bits():
    """Codes behind 2^31 and 2^32 bytes of the pool."""
    kv, d, P = 8, 128, 128
    n_pages = (1 << 32) // (kv * d * P) + 40
    codes = [torch.empty(n_pages, kv, P, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    t = codes + [torch.full((n_pages, kv), 0.01, device="cuda") for _ in range(2)] + [torch.zeros(n_pages, kv, P, device="cuda")]
    pages = np.array([[n_pages - 1, (1 << 31) // (kv * d * P), 3, n_pages // 2 + 1]], np.int32)
    g = gen(11)
    for p in pages[0]:
        for c in codes:
            c[int(p)] = torch.randint(-127, 128, (kv, P, d), device="cuda", generator=g, dtype=torch.int8)
    q = randn(g, 1, kv, d, dt=torch.bfloat16)
    lens = [4 * P - 5]
    o, lse = call_decode(t, pages, lens, q, 0.05, accumulate=1)
    # the same pages in a small pool
    idx = torch.from_numpy(pages[0]).long().cuda()
    small = [x[idx].contiguous() for x in t[:4]] + [torch.zeros(4, kv, P, device="cuda")]
    o2, lse2 = call_decode(small, np.array([[0, 1, 2, 3]], np.int32), lens, q, 0.05, accumulate=1)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(t[4][idx], small[4])
    x = randn(g, 3, kv, d, dt=torch.bfloat16)
    call_append(t, pages, [3 * P + 3], x, x.clone(), [3])
    call_append(small, np.array([[0, 1, 2, 3]], np.int32), [3 * P + 3], x, x.clone(), [3])
    assert torch.equal(t[0][idx], small[0]) and torch.equal(t[2][idx], small[2])


# ------------------------------------------------------------------ eviction


def call_evict(t, table, lens, new_table, budget, recent, st=None, max_len=None, in_place_lens=False):
    c = capi.make_kv_cache(*t)
    B = len(lens)
    n = capi.energon_cache_evict_workspace_bytes(c, B, budget)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    d_lens = ints(lens)
    out = d_lens if in_place_lens else torch.full((B,), -9, dtype=torch.int32, device="cuda")
    capi.energon_cache_evict(c, ints(table), table.shape[1], d_lens, ints(new_table), new_table.shape[1], out, B,
                             max(max(lens), 0) if max_len is None else max_len, budget, recent, st, ws, n)
    return out.tolist()


@pytest.mark.parametrize("kv,d,P", [(2, 128, 64), (3, 64, 16), (1, 128, 128), (2, 64, 32)])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (50, 0), (50, 50), (64, 7), (129, 30), (400, 100)])
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(kv, d, P, budget, recent, kind, in_place):
    lens = [0, 1, 50, 51, 200, 385]
    n_pages = sum(-(-n // P) for n in lens)
    per = -(-budget // P)
    t = make(n_pages + len(lens) * per, kv, P, d, seed=P + budget)
    table = tables(lens, P, n_pages, 9)
    if kind == "ties":
        t[4] = (t[4] * 4).round()
    elif kind == "equal":
        t[4] = torch.zeros_like(t[4])
    elif kind == "odd":
        t[4] = torch.where(t[4] < 0.2, float("nan"), torch.where(t[4] < 0.3, float("inf"), torch.where(
            t[4] < 0.4, -0.0, torch.where(t[4] < 0.5, 0.0, torch.where(t[4] < 0.6, float("-inf"), t[4] - 0.8)))))
    if in_place:
        new_table = np.full((len(lens), max(per, table.shape[1])), 1 << 30, np.int32)
        new_table[:, :table.shape[1]] = table
    else:
        new_table = np.random.default_rng(1).permutation(len(lens) * per).reshape(len(lens), per).astype(np.int32) + n_pages
    h, st = host(t), status()
    want = ref.evict(h, table, lens, new_table, budget, recent)
    got = call_evict(t, table, lens, new_table, budget, recent, st, in_place_lens=in_place)
    assert int(st) == OK and got == want
    same(t, h)
    if in_place:                                     # cut already: nothing more happens
        assert call_evict(t, table, want, new_table, budget, recent) == want
        same(t, h)


def test_evict_long():
    """More tokens than a block has threads, kept from all over a long sequence."""
    kv, d, P, lens, budget, recent = 2, 64, 64, [9001, 2500], 3000, 129
    n_pages = sum(-(-n // P) for n in lens)
    per = -(-budget // P)
    for in_place in (False, True):
        t = make(n_pages + 2 * per, kv, P, d, seed=12)
        t[4] = (t[4] * 1000).round() / 1000
        table = tables(lens, P, n_pages, 9)
        new_table = table if in_place else (np.arange(2 * per).reshape(2, per).astype(np.int32) + n_pages)
        h = host(t)
        want = ref.evict(h, table, lens, new_table, budget, recent)
        assert call_evict(t, table, lens, new_table, budget, recent) == want
        same(t, h)


def test_evict_bad_pages_lengths_and_status():
    kv, d, P = 2, 64, 16
    lens, budget = [60, 60, 60], 20
    base = tables(lens, P, 12, 3)
    new = np.arange(6).reshape(3, 2).astype(np.int32) + 12
    for page in (-1, 18, 1 << 30):
        for side in ("old", "new"):
            table, new_table = base.copy(), new.copy()
            (table if side == "old" else new_table)[1, 1] = page
            t = make(18, kv, P, d, seed=2)
            h, st = host(t), status()
            ref.evict(h, table[[0, 2]], [60, 60], new_table[[0, 2]], budget, 4)
            assert call_evict(t, table, lens, new_table, budget, 4, st) == [20, 0, 20]
            assert int(st) == capi.ENERGON_DEVICE_BAD_PAGE
            same(t, h)
    for bad in (-1, 65, 1 << 30):
        t = make(18, kv, P, d, seed=2)
        h, st = host(t), status()
        ref.evict(h, base[[0, 2]], [60, 60], new[[0, 2]], budget, 4)
        assert call_evict(t, base, [60, bad, 60], new, budget, 4, st, max_len=1 << 20) == [20, 0, 20]
        assert int(st) == capi.ENERGON_DEVICE_BAD_LENGTH
        same(t, h)
    t = make(18, kv, P, d, seed=2)
    h = host(t)
    assert call_evict(t, base, lens, new, budget, 4, status() + 2) == [-9, -9, -9]
    same(t, h)


# ------------------------------------------------------------------ together


class Session:
    """Prompts in, then single tokens: what a serving program does with the operators."""

    def __init__(self, dt, lens, H, kv, d, P, budget, recent, steps, seed):
        self.dt, self.lens, self.H, self.kv, self.d, self.P = dt, lens, H, kv, d, P
        self.budget, self.recent, self.steps = budget, recent, steps
        B, T = len(lens), sum(lens)
        self.B, self.T, self.scale = B, T, 1.0 / d ** 0.5
        g = gen(seed)
        self.q, self.k, self.v = (randn(g, T, h, d, dt=dt) for h in (H, kv, kv))
        self.tok = [tuple(randn(g, B, h, d, dt=dt) for h in (H, kv, kv)) for _ in range(steps)]
        self.max_pages = -(-(max(max(lens), budget) + steps) // P)
        self.table = ints(np.random.default_rng(seed).permutation(B * self.max_pages).reshape(B, self.max_pages))
        self.cap = self.max_pages * P
        self.status = status()
        self.t = make(B * self.max_pages, kv, P, d)
        self.cache = capi.make_kv_cache(*self.t)
        self.o, self.lse = torch.empty_like(self.q), torch.empty(H, T, device="cuda")
        self.w = torch.empty(kv, T, device="cuda")
        self.cu, self.ones = starts(lens), starts([1] * B)
        self.cache_lens = ints(lens)
        self.out = torch.empty(steps, B, H, d, dtype=dt, device="cuda")
        n = max(capi.energon_cache_attention_workspace_bytes(self.cache, B, self.cap, H, 1),
                capi.energon_cache_evict_workspace_bytes(self.cache, B, budget))
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def reset(self):
        for x in self.t:
            x.zero_()
        self.cache_lens.copy_(ints(self.lens))

    def run(self):
        H, kv, d, dt, B, st = self.H, self.kv, self.d, capi.DTYPE_OF[self.dt], self.B, self.status
        capi.energon_prompt_attention(self.q, H * d, self.k, kv * d, self.v, kv * d, self.cu, B, self.T, H, kv, d, dt,
                                      self.scale, self.o, H * d, self.lse, st)
        capi.energon_prompt_key_weights(self.q, H * d, self.k, kv * d, self.lse, self.cu, B, self.T, H, kv, d, dt,
                                        self.scale, 32, self.w, st)
        capi.energon_kv_append(self.cache, self.table, self.max_pages, self.cache_lens, self.k, kv * d, self.v, kv * d,
                               self.w, self.cu, B, self.T, dt, st)
        capi.energon_cache_evict(self.cache, self.table, self.max_pages, self.cache_lens, self.table, self.max_pages,
                                 self.cache_lens, B, self.cap, self.budget, self.recent, st, self.ws, self.ws.numel())
        for i, (q, k, v) in enumerate(self.tok):
            self.cache_lens.add_(1)
            capi.energon_kv_append(self.cache, self.table, self.max_pages, self.cache_lens, k, kv * d, v, kv * d, None,
                                   self.ones, B, B, dt, st)
            capi.energon_cache_attention(self.cache, self.table, self.max_pages, self.cache_lens, B, self.cap, q, H * d,
                                         H, dt, self.scale, self.out[i], H * d, None, 1, st, self.ws, self.ws.numel())
        return self.out


SESSION = dict(lens=[150, 7, 260, 64], H=8, kv=2, d=128, P=32, budget=90, recent=20, steps=9, seed=21)


@pytest.mark.parametrize("dt", DT)
def test_generate_step_by_step(dt):
    """The operators one after another; every decode step against the plain one on the cache's own state."""
    s = Session(DT[dt], **SESSION)
    out = s.run().clone()
    assert int(s.status) == OK
    check_prompt(s.q, s.k, s.v, s.lens, s.scale, s.o, s.lse)
    assert s.cache_lens.tolist() == [min(n, 90) + 9 for n in s.lens]
    # the plain run: append, evict and append are exact given the weights the library computed
    h = ref.Cache(*[np.zeros(x.shape, x.cpu().numpy().dtype) for x in s.t])
    table, lens = s.table.cpu().numpy(), list(s.lens)
    ref.append(h, table, lens, f64(s.k).astype(np.float32), f64(s.v).astype(np.float32), s.w.cpu().numpy(), lens)
    lens = ref.evict(h, table, lens, table, 90, 20)
    for i, (q, k, v) in enumerate(s.tok):
        lens = [n + 1 for n in lens]
        ref.append(h, table, lens, f64(k).astype(np.float32), f64(v).astype(np.float32), None, [1] * s.B)
        state = [torch.from_numpy(x) for x in (h.codes["k"], h.codes["v"], h.scale["k"], h.scale["v"], h.weight)]
        check_decode(state, table, lens, q, s.scale, out[i], None)
    for name, codes in (("k", s.t[0]), ("v", s.t[1])):
        assert np.array_equal(codes.cpu().numpy(), h.codes[name])


def test_generate_captured_and_replayed():
    """Two sessions captured into graphs, each with its own workspace, replayed at once on two streams
    with new inputs in the same buffers: the same bits as the calls made one by one."""
    ss = [Session(torch.bfloat16, **dict(SESSION, seed=30 + i)) for i in range(2)]
    want = []
    for s in ss:
        want.append(s.run().clone())
        s.reset()
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, stream in zip(ss, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=stream):
            s.run()
        graphs.append(gr)
    for _ in range(3):
        for s in ss:
            s.reset()
            s.out.fill_(9)
        torch.cuda.synchronize()
        for gr, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                gr.replay()
        torch.cuda.synchronize()
        for s, w in zip(ss, want):
            assert torch.equal(s.out, w) and int(s.status) == OK
    a, b = ss                                          # new inputs in the captured buffers
    for x, y in ((a.q, b.q), (a.k, b.k), (a.v, b.v)):
        x.copy_(y)
    for (x, y) in zip(a.tok, b.tok):
        for u, w in zip(x, y):
            u.copy_(w)
    a.table.copy_(b.table)
    a.reset()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[1])


def test_side_stream_and_explicit_handle():
    lens, H, kv, d = [130, 20], 4, 2, 128
    T, g = sum(lens), gen(13)
    q, k, v = (randn(g, T, h, d, dt=torch.float16) for h in (H, kv, kv))
    want, _ = call_prompt(q, k, v, lens, 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = call_prompt(q, k, v, lens, 0.1, stream=side)
    side.synchronize()
    got2, _ = call_prompt(q, k, v, lens, 0.1, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(want, got) and torch.equal(want, got2)


def test_binding_refuses_wrong_tensors():
    q = torch.zeros(8, 4, 128, dtype=torch.float16, device="cuda")
    args = (512, q, 512, q, 512, starts([8]), 1, 8, 4, 4, 128, capi.ENERGON_F16, 0.1)
    with pytest.raises(ValueError):
        capi.energon_prompt_attention(q[:7], *args, torch.empty_like(q), 512)            # too few rows
    with pytest.raises(ValueError):
        capi.energon_prompt_attention(q.bfloat16(), *args, torch.empty_like(q), 512)     # another type
    with pytest.raises(ValueError):
        capi.energon_prompt_attention(q.transpose(0, 1), *args, torch.empty_like(q), 512)
    with pytest.raises(ValueError):
        capi.energon_prompt_attention(q, *args, torch.empty_like(q), 512, torch.empty(3, device="cuda"))
    with pytest.raises(ValueError):
        capi.energon_prompt_attention(q, *args, torch.empty_like(q), 512, None, torch.zeros(1, device="cuda"))
    with pytest.raises(capi.EnergonError):
        capi.energon_prompt_attention(q, *args, q, 512)                                  # in place
