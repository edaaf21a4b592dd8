"""The serving operators around the key/value cache: cases, inputs and plain forms.

Five operators that a program calls one after another when it generates text with
grouped heads on packed prompts:

  prompt      causal attention of every token of a packed batch of prompts
  key_weight  the attention weight that each key of the prompts received
  append      keys and values written into a paged cache held in 8 bits
  decode      attention of one new token per sequence over that cache
  evict       the cache cut down to the tokens that received most weight

With ``own`` false ``run`` computes them with elementary torch operations in fp32, with
``own`` true through the library's entry points.  Both take what ``prepare`` gives.

Layouts: q [T, heads, d], k and v [T, kv_heads, d] packed by token; cache codes
[pages, kv_heads, page_len, d] int8 with one fp32 scale per page and kv head.  A held
value is code * scale.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # four short requests of the tiny fp32 configuration (4 heads of 64, lengths up to 32): launch latency
        dict(name="prompt_tiny_f32", op="prompt", dtype="f32", heads=4, kv_heads=4, d=64, batch=4, longest=32,
             ragged=True, mix=1),
        # the GPT-3 layer's attention on the dynamic batch: 64 requests of 1..256 tokens, 96 heads of 128
        dict(name="prompt_gpt3_dynbatch", op="prompt", dtype="f16", heads=96, kv_heads=96, d=128, batch=64,
             longest=256, ragged=True, mix=2),
        # a mixed batch of prompts of odd lengths with grouped heads
        dict(name="prompt_mixed", op="prompt", dtype="bf16", heads=32, kv_heads=8, d=128, batch=12, longest=1531,
             ragged=True, mix=3),
        # one long document: the largest call
        dict(name="prompt_long", op="prompt", dtype="bf16", heads=32, kv_heads=8, d=128, batch=1, longest=8192,
             ragged=False, mix=4),
        # the weights that the last 64 queries of each prompt give its keys (an observation window)
        dict(name="key_weight_window", op="key_weight", dtype="bf16", heads=32, kv_heads=8, d=128, batch=8,
             longest=2111, ragged=True, window=64, mix=5),
        # the weights over all queries of a long prompt
        dict(name="key_weight_all", op="key_weight", dtype="f16", heads=32, kv_heads=8, d=128, batch=1, longest=4096,
             ragged=False, window=1 << 30, mix=6),
        # one new token for each of 48 running requests: latency
        dict(name="append_token", op="append", dtype="f16", kv_heads=8, d=128, page_len=16, batch=48, longest=64,
             new=1, ragged=True, mix=7),
        # whole prompts written to the cache after the prompt pass
        dict(name="append_prompt", op="append", dtype="bf16", kv_heads=8, d=128, page_len=64, batch=16, longest=2000,
             new=0, ragged=True, mix=8),
        # one request with a context of a few thousand tokens: latency, few rows, a long axis
        dict(name="decode_single", op="decode", dtype="bf16", heads=32, kv_heads=8, d=128, page_len=64, batch=1,
             longest=4099, ragged=False, weight=False, mix=9),
        # a full batch of requests of different contexts, with the weights that eviction needs
        dict(name="decode_batch", op="decode", dtype="bf16", heads=64, kv_heads=8, d=128, page_len=64, batch=64,
             longest=8192, ragged=True, weight=True, mix=10),
        # four caches with 64-wide heads cut to 200 tokens
        dict(name="evict_small", op="evict", kv_heads=4, d=64, page_len=16, batch=4, longest=517, ragged=True,
             budget=200, recent=32, mix=11),
        # the caches of sixteen long prompts cut to a quarter
        dict(name="evict_prompts", op="evict", kv_heads=8, d=128, page_len=64, batch=16, longest=8192, ragged=True,
             budget=2048, recent=256, mix=12),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["prompt", "key_weight", "append", "decode", "evict"])
    heads, kv = rng.choice([(4, 4), (8, 1), (12, 4), (32, 8), (64, 8), (14, 2), (40, 8), (96, 96), (9, 3)])
    d = rng.choice([64, 128])
    c = dict(op=op, heads=heads, kv_heads=kv, d=d, ragged=rng.random() < 0.7, mix=rng.randrange(1 << 30))
    if op in ("prompt", "key_weight"):
        c["dtype"] = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
        c["batch"] = _spread(rng, 1, 64)
        most = 0.7e9 if c["dtype"] != "f32" else 0.05e9  # scores over the padded batch
        if op == "key_weight":
            most *= 0.4
        c["longest"] = _spread(rng, 1, max(1, min(8192, int(math.sqrt(most / (heads * c["batch"]))))))
        if op == "key_weight":
            c["window"] = rng.choice([1, 16, 32, 100, 1 << 30])
        return c
    c["page_len"] = rng.choice([16, 32, 64, 128])
    if op == "append":
        del c["heads"]
        c["dtype"] = rng.choice(["f16", "bf16", "f32"])
        c["batch"] = _spread(rng, 1, 64)
        c["new"] = rng.choice([0, 0, 1, 1, 5, 33])
        most = int(2e7 / (c["batch"] * kv * d))
        c["longest"] = _spread(rng, max(1, c["new"]), max(max(1, c["new"]), min(4000, most)))
    elif op == "decode":
        c["dtype"] = rng.choice(["f16", "bf16", "f32"])
        c["weight"] = rng.random() < 0.5
        c["batch"] = _spread(rng, 1, 64)
        c["longest"] = _spread(rng, 1, max(1, min(30000, int(2.5e8 / (c["batch"] * kv * d)))))
    else:
        del c["heads"]
        c["batch"] = _spread(rng, 1, 16)
        c["longest"] = _spread(rng, 2, max(2, min(20000, int(6e7 / (c["batch"] * kv * d)))))
        c["budget"] = _spread(rng, 1, c["longest"])
        c["recent"] = rng.randrange(0, c["budget"] + 1)
    return c


def _lens(case):
    """The sequences' lengths: a matter of the case, not of the seed."""
    r = np.random.RandomState(case["mix"] % (1 << 31))
    n = case["longest"]
    lens = np.full(case["batch"], n, np.int64)
    if case["ragged"]:
        lens = r.randint(max(1, case.get("new", 0)), n + 1, case["batch"])
        lens[0] = n
    return [int(x) for x in lens]


def _new(case, lens):
    """Tokens of each sequence that an append brings: all of them, or the last few."""
    return [min(x, case["new"]) if case["new"] else x for x in lens]


def work(case):
    lens = _lens(case)
    kv, d, op = case["kv_heads"], case["d"], case["op"]
    if op in ("prompt", "key_weight"):
        h, e, T = case["heads"], SIZES[case["dtype"]], sum(lens)
        if op == "prompt":
            pairs = sum(n * (n + 1) // 2 for n in lens)
            return {"bytes": T * d * e * (2 * h + 2 * kv) + 4 * h * T, "flops": 4 * d * h * pairs}
        win = [min(n, case["window"]) for n in lens]
        pairs = sum(n * (n + 1) // 2 - (n - w) * (n - w + 1) // 2 for n, w in zip(lens, win))
        return {"bytes": T * kv * d * e + sum(win) * h * (d * e + 4) + 4 * kv * T, "flops": 2 * d * h * pairs}
    if op == "append":
        T, pool = sum(_new(case, lens)), sum(-(-n // case["page_len"]) for n in lens) + 1
        # rows read, codes written, and the pool's held values as the outputs
        return {"bytes": 2 * T * kv * d * (SIZES[case["dtype"]] + 1) + 2 * pool * kv * case["page_len"] * d * 4, "flops": 0}
    S = sum(lens)
    if op == "decode":
        h, e = case["heads"], SIZES[case["dtype"]]
        by = 2 * S * kv * d + 2 * case["batch"] * h * d * e + 4 * case["batch"] * h
        by += 8 * S * kv if case["weight"] else 0
        return {"bytes": by, "flops": 4 * d * h * S}
    kept = sum(min(n, case["budget"]) for n in lens)
    pool = case["batch"] * -(-case["budget"] // case["page_len"])
    # weights read, kept codes read and written, the new pages' held values and weights as the outputs
    return {"bytes": 4 * S * kv + kept * kv * (4 * d + 4) + pool * kv * case["page_len"] * (8 * d + 4), "flops": 0}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _keys(g, rows, kv, d, dt):
    """Key-like rows: a few channels much larger than the rest, as trained models have them."""
    gain = 1.0 + 4.0 * (torch.rand(kv, d, device="cuda", generator=g) < 0.03).float()
    return (_randn(g, rows, kv, d) * gain).to(dt)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(lens):
    return _ints([0] + [int(x) for x in np.cumsum(lens)])


def _tables(case, lens, g, extra=0):
    """(page table [batch, max_pages], pages used): pages handed out in a shuffled order."""
    P = case["page_len"]
    need = [-(-n // P) for n in lens]
    most, total = max(1, max(need)), sum(need)
    order = torch.randperm(total + extra, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros(len(lens), most, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, most, total


def _filled(case, pages, g):
    """Codes and scales of a cache in use, and the weights its tokens received so far."""
    kv, P, d = case["kv_heads"], case["page_len"], case["d"]
    st = {}
    for n in ("k", "v"):
        codes = torch.empty(pages, kv, P, d, dtype=torch.int8, device="cuda")
        for at in range(0, pages, 512):
            part = codes[at:at + 512]
            part.copy_((_randn(g, *part.shape) * 34.0).round_().clamp_(-127, 127))
        st[n + "_codes"] = codes
        st[n + "_scale"] = (0.5 + torch.rand(pages, kv, device="cuda", generator=g)) * 0.03
    w = torch.rand(pages, kv, P, device="cuda", generator=g)
    st["weight"] = (w * w * w * w * 4.0).contiguous()  # few tokens carry most of the weight
    return st


def prepare(case, seed):
    g = _gen(seed)
    lens, op, kv, d = _lens(case), case["op"], case["kv_heads"], case["d"]
    s = dict(case=dict(case), lens=lens, longest=max(lens), scale=1.0 / math.sqrt(d))
    B = len(lens)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op in ("prompt", "key_weight"):
        h, dt, T = case["heads"], DTYPES[case["dtype"]], sum(lens)
        s["cu"], s["rows"] = _starts(lens), T
        s["q"] = _randn(g, T, h, d).to(dt)
        s["k"] = _keys(g, T, kv, d, dt)
        if op == "prompt":
            s["v"] = _randn(g, T, kv, d).to(dt)
            s["o"] = torch.empty(T, h, d, dtype=dt, device="cuda")
            s["lse"] = torch.empty(h, T, device="cuda")
        else:
            s["lse"] = torch.cat([_log_sums(s["q"][a:b], s["k"][a:b], s["scale"]) for a, b in _spans(lens)], 1).contiguous()
            s["window"] = case["window"]
            s["weights"] = torch.empty(kv, T, device="cuda")
        return s
    P = case["page_len"]
    if op == "append":
        new, dt = _new(case, lens), DTYPES[case["dtype"]]
        s["table"], s["max_pages"], pages = _tables(case, lens, g, extra=1)
        s.update(_filled(case, pages + 1, g))
        T = sum(new)
        s["cu"], s["rows"], s["cache_lens"] = _starts(new), T, _ints(lens)
        s["k"], s["v"] = _keys(g, T, kv, d, dt), _randn(g, T, kv, d).to(dt)
        s["given"] = torch.rand(kv, T, device="cuda", generator=g)
    elif op == "decode":
        h, dt = case["heads"], DTYPES[case["dtype"]]
        s["table"], s["max_pages"], pages = _tables(case, lens, g, extra=1)
        s.update(_filled(case, pages + 1, g))
        s["cache_lens"] = _ints(lens)
        s["q"] = _randn(g, B, h, d).to(dt)
        s["o"] = torch.empty(B, h, d, dtype=dt, device="cuda")
        s["lse"] = torch.empty(B, h, device="cuda")
    else:
        s["table"], s["max_pages"], pages = _tables(case, lens, g)
        per = -(-case["budget"] // P)
        s["first_new"] = pages  # the new pages follow the old ones in the pool
        s.update(_filled(case, pages + B * per, g))
        s["new_table"] = (torch.randperm(B * per, device="cuda", generator=g).to(torch.int32) + pages).view(B, per)
        s["new_max_pages"] = per
        s["cache_lens"], s["new_lens"] = _ints(lens), torch.zeros(B, dtype=torch.int32, device="cuda")
    if op != "append":
        s["workspace"] = torch.empty(_workspace_bytes(case, lens), dtype=torch.uint8, device="cuda")
    return s


def _workspace_bytes(case, lens):
    """Room for what a call keeps between its launches, as its documentation bounds it."""
    S, kv, B = max(lens), case["kv_heads"], len(lens)
    if case["op"] == "decode":
        h = case["heads"]
        return 4 * B * h * (S + 64) + 64 * B * h * (case["d"] + 2) * 4 + (1 << 20)
    return B * kv * (16 * (case["budget"] + 128) + 64) + (1 << 20)


def _spans(lens):
    ends = np.cumsum(lens)
    return [(int(e - n), int(e)) for n, e in zip(lens, ends)]


def _log_sums(q, k, scale):
    """log sum_t exp(scale q_s . k_t) over t <= s, for one sequence: [heads, n] fp32."""
    n, h, d = q.shape
    kv = k.shape[1]
    rep = h // kv
    out = []
    for j in range(kv):
        x = torch.einsum("sgd,td->gst", q[:, j * rep:(j + 1) * rep].float(), k[:, j].float()) * scale
        x.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=q.device).triu_(1), -math.inf)
        out.append(torch.logsumexp(x, -1))
    return torch.cat(out, 0)


# ------------------------------------------------------------------ one pass


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from padding_free_varlen_b200 import capi
    c = s["case"]
    op, kv, d, B = c["op"], c["kv_heads"], c["d"], c["batch"]
    if op in ("prompt", "key_weight"):
        h, dt = c["heads"], capi.DTYPE_OF[s["q"].dtype]
        if op == "prompt":
            capi.energon_prompt_attention(s["q"], h * d, s["k"], kv * d, s["v"], kv * d, s["cu"], B, s["rows"], h, kv,
                                          d, dt, s["scale"], s["o"], h * d, s["lse"], s["status"])
            return {"o": s["o"], "lse": s["lse"]}
        capi.energon_prompt_key_weights(s["q"], h * d, s["k"], kv * d, s["lse"], s["cu"], B, s["rows"], h, kv, d, dt,
                                        s["scale"], s["window"], s["weights"], s["status"])
        return {"weights": s["weights"]}
    cache = capi.make_kv_cache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["weight"])
    if op == "append":
        capi.energon_kv_append(cache, s["table"], s["max_pages"], s["cache_lens"], s["k"], kv * d, s["v"], kv * d,
                               s["given"], s["cu"], B, s["rows"], capi.DTYPE_OF[s["k"].dtype], s["status"])
        return _held(s, 0)
    if op == "decode":
        h = c["heads"]
        capi.energon_cache_attention(cache, s["table"], s["max_pages"], s["cache_lens"], B, s["longest"], s["q"],
                                     h * d, h, capi.DTYPE_OF[s["q"].dtype], s["scale"], s["o"], h * d, s["lse"],
                                     int(c["weight"]), s["status"], s["workspace"], s["workspace"].numel())
        return {"o": s["o"], "lse": s["lse"], "weight": s["weight"] if c["weight"] else None}
    capi.energon_cache_evict(cache, s["table"], s["max_pages"], s["cache_lens"], s["new_table"], s["new_max_pages"],
                             s["new_lens"], B, s["longest"], c["budget"], c["recent"], s["status"], s["workspace"],
                             s["workspace"].numel())
    return dict(_held(s, s["first_new"]), lens=s["new_lens"])


def _held(s, first):
    """The values that the pool's pages from `first` on stand for, and their tokens' weights."""
    return {"k": s["k_codes"][first:] * s["k_scale"][first:, :, None, None],
            "v": s["v_codes"][first:] * s["v_scale"][first:, :, None, None], "weight": s["weight"][first:]}


def _run_plain(s):
    return {"prompt": _prompt, "key_weight": _key_weight, "append": _append, "decode": _decode, "evict": _evict}[s["case"]["op"]](s)


def _padded(s):
    """Positions of the padded batch in the packed rows, and which of them hold a token."""
    cu, S = s["cu"].long(), s["longest"]
    n = cu[1:] - cu[:-1]
    at = torch.arange(S, device="cuda")
    ok = at[None, :] < n[:, None]
    return torch.where(ok, cu[:-1, None] + at[None, :], cu[:-1, None]), ok


def _packed_at(s):
    """For each packed row its place (sequence * S + position) in the padded batch."""
    cu = s["cu"].long()
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(cu, r, right=True) - 1
    return b * s["longest"] + (r - cu[b])


def _scores(s, rows, at, idx):
    """scale q . k of the queries at `rows` (their positions: `at`, [batch, Q]) over the padded batch's keys:
    [batch, kv, group, Q, S] fp32, -inf where the key is after the query."""
    c, S, Q = s["case"], s["longest"], rows.shape[1]
    B, h, kv, d = c["batch"], c["heads"], c["kv_heads"], c["d"]
    q = s["q"][rows].float().view(B, Q, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(B, kv, h // kv * Q, d)
    k = s["k"][idx].float().permute(0, 2, 3, 1)
    x = torch.matmul(q, k).view(B, kv, h // kv, Q, S).mul_(s["scale"])
    after = torch.arange(S, device="cuda")[None, None, :] > at[:, :, None]
    return x.masked_fill_(after[:, None, None], -math.inf)


def _prompt(s):
    c, S = s["case"], s["longest"]
    B, h, kv, d = c["batch"], c["heads"], c["kv_heads"], c["d"]
    idx, _ = _padded(s)
    x = _scores(s, idx, torch.arange(S, device="cuda").expand(B, S), idx)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    v = s["v"][idx].float().permute(0, 2, 1, 3)
    o = torch.matmul(x.view(B, kv, -1, S), v).view(B, kv, h // kv, S, d) / l
    at = _packed_at(s)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * S, h, d)[at]
    lse = (m + l.log()).view(B, h, S).permute(1, 0, 2).reshape(h, B * S)[:, at]
    return {"o": o.to(s["q"].dtype), "lse": lse}


def _key_weight(s):
    c, S, Q = s["case"], s["longest"], min(s["window"], s["longest"])
    B, h, kv = c["batch"], c["heads"], c["kv_heads"]
    idx, _ = _padded(s)
    cu = s["cu"].long()
    at = (cu[1:] - cu[:-1] - Q)[:, None] + torch.arange(Q, device="cuda")  # the queries that count, where not negative
    seen, at = at >= 0, at.clamp(min=0)
    rows = cu[:-1, None] + at
    x = _scores(s, rows, at, idx)
    lse = s["lse"][:, rows].view(kv, h // kv, B, Q).permute(2, 0, 1, 3)
    x.sub_(lse[..., None]).exp_().mul_(seen[:, None, None, :, None])
    w = x.sum((2, 3))
    return {"weights": w.permute(1, 0, 2).reshape(kv, B * S)[:, _packed_at(s)]}


def _pow2(k):
    """2^k in fp32, exactly, for whole k within the normal range."""
    return ((k.clamp(-126, 127) + 127).to(torch.int32) << 23).view(torch.float32)


def _append(s):
    c = s["case"]
    kv, d, P, B = c["kv_heads"], c["d"], c["page_len"], c["batch"]
    cu, lens, pages = s["cu"].long(), s["cache_lens"].long(), s["k_scale"].shape[0]
    n = cu[1:] - cu[:-1]
    start = lens - n
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(cu, r, right=True) - 1
    pos = start[b] + r - cu[b]
    page, slot = s["table"].long()[b, pos // P], pos % P
    first = s["table"].long().gather(1, (start // P).clamp_(max=s["max_pages"] - 1)[:, None])[:, 0]
    part = (start % P > 0) & (n > 0)  # the sequence's first page already holds tokens
    share = torch.full((1,), 1.0 / 127.0, dtype=torch.float32, device="cuda")
    for name in ("k", "v"):
        codes, scale, x = s[name + "_codes"], s[name + "_scale"], s[name].float()
        need = torch.zeros(pages, kv, device="cuda").index_reduce_(0, page, x.abs().amax(-1) * share, "amax")
        # a page that already holds tokens keeps its scale or takes it times a power of two
        old, want = scale[first], need[first]
        ms, es = torch.frexp(old)
        mn, en = torch.frexp(want)
        up = (en - es + (mn > ms).int()).clamp_(min=0)
        up = torch.where(part[:, None] & (old > 0) & (want > 0), up, torch.zeros_like(up))
        grown = torch.where(old > 0, old * _pow2(up), want)
        kept = torch.where(part[:, None, None, None], torch.round(codes[first].float() * _pow2(-up)[:, :, None, None]), codes[first].float())
        codes.index_copy_(0, first, kept.to(torch.int8))
        # pages that begin with a new token take the scale that their tokens need
        fresh = torch.zeros(pages, dtype=torch.bool, device="cuda").index_fill_(0, page, True)
        scale.copy_(torch.where(fresh[:, None], need, scale))
        scale.index_copy_(0, first, torch.where(part[:, None], grown, scale[first]))
        now = scale[page]
        q = torch.where(now[..., None] > 0, torch.round(x / now[..., None]), torch.zeros_like(x)).clamp_(-127, 127)
        codes.view(pages, kv, P, d).permute(0, 2, 1, 3)[page, slot] = q.to(torch.int8)
    s["weight"].permute(0, 2, 1)[page, slot] = s["given"].t()
    return _held(s, 0)


def _decode(s):
    c = s["case"]
    B, h, kv, d, P, n_p = c["batch"], c["heads"], c["kv_heads"], c["d"], c["page_len"], s["max_pages"]
    table, S = s["table"].long(), s["max_pages"] * c["page_len"]

    def rows(codes, scale):
        x = codes[table].float() * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, kv, S, d)

    x = torch.matmul(s["q"].float().view(B, kv, h // kv, d), rows(s["k_codes"], s["k_scale"]).transpose(2, 3)).mul_(s["scale"])
    x.masked_fill_((torch.arange(S, device="cuda")[None, :] >= s["cache_lens"][:, None])[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    x.div_(l)
    o = torch.matmul(x, rows(s["v_codes"], s["v_scale"])).view(B, h, d).to(s["q"].dtype)
    lse = (m + l.log()).view(B, h)
    if c["weight"]:
        w = x.sum(2).view(B, kv, n_p, P).permute(0, 2, 1, 3).reshape(B * n_p, kv, P)
        s["weight"].index_add_(0, table.view(-1), w)
    return {"o": o, "lse": lse, "weight": s["weight"] if c["weight"] else None}


def _evict(s):
    c = s["case"]
    B, kv, d, P, n_p, budget = c["batch"], c["kv_heads"], c["d"], c["page_len"], s["max_pages"], c["budget"]
    table, to, lens, S, new_p = s["table"].long(), s["new_table"].long(), s["cache_lens"].long(), s["max_pages"] * c["page_len"], s["new_max_pages"]
    w = s["weight"][table].permute(0, 2, 1, 3).reshape(B, kv, S)
    at = torch.arange(S, device="cuda")
    last = lens - torch.minimum(lens, torch.full_like(lens, c["recent"]))
    rank = torch.where((at[None, :] >= last[:, None])[:, None], torch.full_like(w, math.inf), w)
    rank = torch.where((at[None, :] >= lens[:, None])[:, None], torch.full_like(w, -math.inf), rank)
    keep = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    new_lens = lens.clamp(max=budget)
    room = torch.arange(budget, device="cuda")
    used = (room[None, :] < new_lens[:, None])[:, None]  # slots that hold a token afterwards
    keep = torch.where(used, keep, torch.full_like(keep, S)).sort(-1).values.clamp_(max=S - 1)
    src = table[:, None, :].expand(B, kv, n_p).gather(2, keep // P)
    head = torch.arange(kv, device="cuda")[None, :, None]
    dst, slot = to[:, None, :].expand(B, kv, new_p).gather(2, (room // P).expand(B, kv, budget)), (room % P).expand(B, kv, budget)
    used = used.expand(B, kv, budget)[..., None]
    for name in ("k", "v"):
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        sc = torch.where(used[..., 0], scale[src, head], torch.zeros_like(keep, dtype=torch.float32))
        most = torch.zeros(B, kv, new_p * P, device="cuda")
        most[..., :budget] = sc
        most = most.view(B, kv, new_p, P).amax(-1)
        ratio = sc / most.gather(2, (room // P).expand(B, kv, budget))
        got = torch.where(sc[..., None] > 0, torch.round(codes[src, head, keep % P].float() * ratio[..., None]), torch.zeros((), device="cuda"))
        codes[dst, head, slot] = torch.where(used, got.to(torch.int8), codes[dst, head, slot])
        old = scale[to].permute(0, 2, 1)
        scale[to] = torch.where((torch.arange(new_p, device="cuda")[None, :] * P < new_lens[:, None])[:, None], most, old).permute(0, 2, 1)
    s["weight"][dst, head, slot] = torch.where(used[..., 0], w.gather(2, keep), s["weight"][dst, head, slot])
    s["new_lens"].copy_(new_lens)
    return dict(_held(s, s["first_new"]), lens=s["new_lens"])


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "key_weight": _exact_key_weight, "append": _exact_append,
            "decode": _exact_decode, "evict": _exact_evict}[case["op"]](s)


def _exact_weights(s, a, b, j, w0=0):
    """Probabilities and log sums of head j's queries a + w0 .. b-1 over the keys a .. b-1, one sequence."""
    g = s["case"]["heads"] // s["case"]["kv_heads"]
    x = (s["q"][a + w0:b, j].double() @ s["k"][a:b, j // g].double().t()) * s["scale"]
    n = b - a
    x = x + torch.full((n, n), -math.inf, dtype=torch.float64, device="cuda").triu(1)[w0:]
    return x


def _exact_prompt(s):
    c = s["case"]
    g = c["heads"] // c["kv_heads"]
    o = torch.empty(s["rows"], c["heads"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.empty(c["heads"], s["rows"], dtype=torch.float64, device="cuda")
    for a, b in _spans(s["lens"]):
        for j in range(c["heads"]):
            x = _exact_weights(s, a, b, j)
            lse[j, a:b] = torch.logsumexp(x, 1)
            o[a:b, j] = torch.softmax(x, 1) @ s["v"][a:b, j // g].double()
    return {"o": o, "lse": lse}


def _exact_key_weight(s):
    c = s["case"]
    g = c["heads"] // c["kv_heads"]
    w = torch.zeros(c["kv_heads"], s["rows"], dtype=torch.float64, device="cuda")
    for a, b in _spans(s["lens"]):
        w0 = max(0, b - a - s["window"])
        for j in range(c["heads"]):
            # the sums as given (fp32) are an input: a weight is exp(score - sum)
            x = _exact_weights(s, a, b, j, w0)
            w[j // g, a:b] += torch.exp(x - s["lse"][j, a + w0:b].double()[:, None]).sum(0)
    return {"weights": w}


def _exact_append(s):
    c = s["case"]
    P, new = c["page_len"], _new(c, s["lens"])
    table, cu = s["table"].tolist(), s["cu"].tolist()
    out = {}
    for name in ("k", "v"):
        codes, scale = s[name + "_codes"].double(), s[name + "_scale"].double()
        x = s[name].double()
        for b, n in enumerate(s["lens"]):
            at, row = n - new[b], cu[b]
            while at < n:
                take = min(n, (at // P + 1) * P) - at
                p, y = table[b][at // P], x[row:row + take]
                # scales are held in fp32: the largest magnitude times the fp32 value of 1/127
                need = (y.abs().amax((0, 2)).float() * torch.tensor(1.0 / 127.0, device="cuda")).double()
                if at % P:
                    old = scale[p]
                    # the scale doubles until it covers the new tokens
                    times = torch.ones_like(old)
                    while bool(((old > 0) & (old * times < need)).any()):
                        times = torch.where((old > 0) & (old * times < need), times * 2, times)
                    codes[p] = torch.round(codes[p] / times[:, None, None])
                    scale[p] = torch.where(old > 0, old * times, need)
                else:
                    scale[p] = need
                # a code is the nearest whole number to the quotient in fp32
                q = torch.round((y / scale[p][None, :, None]).float()).double()
                codes[p][:, at % P:at % P + take] = torch.nan_to_num(q).clamp(-127, 127).permute(1, 0, 2)
                at, row = at + take, row + take
        out[name] = codes * scale[:, :, None, None]
    w = s["weight"].clone()
    for b, n in enumerate(s["lens"]):
        pos = torch.arange(n - new[b], n, device="cuda")
        p = s["table"][b].long()[pos // P]
        w[p, :, pos % P] = s["given"][:, cu[b]:cu[b + 1]].t()
    return dict(out, weight=w.double())


def _exact_decode(s):
    c = s["case"]
    B, h, kv, d, P = c["batch"], c["heads"], c["kv_heads"], c["d"], c["page_len"]
    o = torch.empty(B, h, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, h, dtype=torch.float64, device="cuda")
    weight = s["weight"].double()
    for b, n in enumerate(s["lens"]):
        pages = s["table"][b, :-(-n // P)].long()

        def held(codes, scale):
            x = codes[pages].double() * scale[pages].double()[:, :, None, None]
            return x.transpose(0, 1).reshape(kv, -1, d)[:, :n]

        x = torch.einsum("jgd,jtd->jgt", s["q"][b].double().view(kv, h // kv, d), held(s["k_codes"], s["k_scale"])) * s["scale"]
        lse[b] = torch.logsumexp(x, -1).view(h)
        p = torch.softmax(x, -1)
        o[b] = torch.einsum("jgt,jtd->jgd", p, held(s["v_codes"], s["v_scale"])).reshape(h, d)
        w = torch.nn.functional.pad(p.sum(1), (0, len(pages) * P - n)).view(kv, len(pages), P).transpose(0, 1)
        weight[pages] += w
    return {"o": o, "lse": lse, "weight": weight if c["weight"] else None}


def _exact_evict(s):
    c = s["case"]
    kv, P, budget, first = c["kv_heads"], c["page_len"], c["budget"], s["first_new"]
    out = {n: s[n + "_codes"][first:].double() for n in ("k", "v")}
    scales = {n: s[n + "_scale"][first:].double() for n in ("k", "v")}
    weight = s["weight"][first:].double()
    new_lens = []
    for b, n in enumerate(s["lens"]):
        pages, to = s["table"][b].long(), (s["new_table"][b].long() - first).tolist()
        tail = min(c["recent"], n)
        new_lens.append(min(n, budget))
        for j in range(kv):
            pos = torch.arange(n, device="cuda")
            w = s["weight"][pages[pos // P], j, pos % P]
            if n > budget:
                best = torch.sort(-w[:n - tail].double(), stable=True).indices[:budget - tail]
                pos = torch.cat([best, pos[n - tail:]]).sort().values
                w = w[pos]
            for at in range(0, len(pos), P):
                p, part = to[at // P], pos[at:at + P]
                weight[p, j, :len(part)] = w[at:at + P].double()
                for name in ("k", "v"):
                    src = s[name + "_scale"][pages[part // P], j]
                    big = src.max()
                    # ratios are fp32 quotients, a code the nearest whole number to the fp32 product
                    ratio = (src.double() / big.double()).float().double()
                    q = s[name + "_codes"][pages[part // P], j, part % P].double() * ratio[:, None]
                    out[name][p, j, :len(part)] = torch.round(q.float()).double()
                    scales[name][p, j] = big.double()
    held = {n: out[n] * scales[n][:, :, None, None] for n in ("k", "v")}
    return dict(held, weight=weight, lens=torch.tensor(new_lens, dtype=torch.int32, device="cuda"))
