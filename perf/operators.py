"""The verification pass between two drafting calls, measured operator by operator.

A drafting call leaves 0..k draft ids per row; the target model then runs the row's last token and its
drafts (1..k+1 positions) over its cache, and the drafts are verified against the probabilities it gives:

  write   the new tokens' keys and values into a paged cache held in 8 bits (e4m3, one power-of-two scale
          per block of tokens and head), then the blocks that changed read back as the values they stand for;
  read    whole contexts of the cache, back as bf16 or f16;
  attend  attention of the 1..k+1 new tokens of each row over the cache, optionally with a sliding window
          and a few first tokens that stay visible;
  verify  the drafts against the target's logits, from given random numbers: the accepted ids and one more.

`run` computes them in plain torch, in 32 bits, or (own) through the framework's public entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
F8_MAX = 448.0
EXP_MIN, EXP_MAX = -48, 48       # the range of a block scale's exponent
GREEDY_BELOW = 1e-5              # temperatures below this take the largest logit
NOISE_MIN = 2.0 ** -60


# ---- the cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # one small batch of the smallest workload (B=4, k=8, V=32000): latency of a serving step with few requests
        dict(name="verify small", op="verify", B=4, k=8, V=32000, dtype="bf16", q=False, greedy=0.25),
        # the serving workload's batch (B=256, k=16, V=151936) with the drafter's own drafts
        dict(name="verify serving", op="verify", B=256, k=16, V=151936, dtype="bf16", q=False, greedy=0.25),
        # drafts of a draft model: its probabilities are compared with the target's, logits kept in 32 bits
        dict(name="verify draft model", op="verify", B=48, k=5, V=128256, dtype="f32", q=True, greedy=0.0),
        # one request's next token and its drafts enter the cache
        dict(name="write one", op="write", B=1, k=4, n_lo=500, n_hi=500, Hkv=8, D=128, P=64, dtype="bf16"),
        # the serving batch's step: 1..17 new tokens per row
        dict(name="write step", op="write", B=256, k=16, n_lo=1024, n_hi=4096, Hkv=8, D=128, P=64, dtype="bf16"),
        # prompts of up to 8192 tokens enter the cache at once
        dict(name="write prompts", op="write", B=8, k=8191, n_lo=8192, n_hi=8192, Hkv=8, D=128, P=64, dtype="f16"),
        # one short context read back
        dict(name="read one", op="read", B=1, n_lo=777, n_hi=777, Hkv=4, D=64, P=32, dtype="f16"),
        # a batch's contexts read back (handed to another engine, or to a kernel that takes 16 bits)
        dict(name="read batch", op="read", B=64, n_lo=1024, n_hi=8192, Hkv=8, D=128, P=64, dtype="bf16"),
        # one request, one token: the latency of a decode step without drafts
        dict(name="attend one", op="attend", B=1, k=0, n_lo=2000, n_hi=2000, Hkv=8, G=4, D=128, P=64, dtype="bf16", window=0, sinks=0),
        # the serving batch's verification pass: 1..17 new tokens per row over 1024..4096 cached
        dict(name="attend serving", op="attend", B=256, k=16, n_lo=1024, n_hi=4096, Hkv=8, G=4, D=128, P=64, dtype="bf16", window=0, sinks=0),
        # long contexts of the agentic workload (8192..32768 tokens, k=32)
        dict(name="attend long", op="attend", B=32, k=32, n_lo=8192, n_hi=32768, Hkv=8, G=4, D=128, P=128, dtype="bf16", window=0, sinks=0),
        # single tokens over long contexts with a window of 2048 and 4 first tokens, small heads, small pages
        dict(name="attend window", op="attend", B=128, k=0, n_lo=2048, n_hi=16384, Hkv=8, G=8, D=64, P=16, dtype="f16", window=2048, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["verify", "write", "read", "attend", "attend"])
    if op == "verify":
        while True:
            c = dict(op=op, B=_log_int(rng, 1, 1024), k=_log_int(rng, 1, 32), V=_log_int(rng, 1000, 160000),
                     dtype=rng.choice(["bf16", "f16", "f32"]), q=rng.random() < 0.3, greedy=rng.choice([0.0, 0.3, 1.0]))
            if work(c)["bytes"] <= 9e8:
                return c
    kv = dict(Hkv=rng.choice([1, 2, 4, 5, 8, 16]), D=rng.choice([64, 128]), P=rng.choice([16, 32, 64, 128]),
              dtype=rng.choice(["bf16", "f16"]))
    while True:
        n_hi = _log_int(rng, 1, 32768)
        n_lo = _log_int(rng, 1, n_hi)
        B = _log_int(rng, 1, 512)
        if op == "attend":
            c = dict(op=op, B=B, k=rng.choice([0, 0, _log_int(rng, 1, 32)]), n_lo=n_lo, n_hi=n_hi, G=rng.choice([1, 2, 3, 4, 6, 8]),
                     window=0, sinks=0, **kv)
            if rng.random() < 0.4:
                c["window"], c["sinks"] = _log_int(rng, 1, 8192), rng.choice([0, 1, 4, 70])
        elif op == "write":
            c = dict(op=op, B=B, k=rng.choice([0, _log_int(rng, 1, 32), _log_int(rng, 1, n_hi)]), n_lo=n_lo, n_hi=n_hi, **kv)
        else:
            c = dict(op=op, B=B, n_lo=n_lo, n_hi=n_hi, **kv)
        w = work(c)
        if B * n_hi * kv["Hkv"] * kv["D"] <= 1.1e9 and (op != "attend" or B * kv["Hkv"] * c["G"] * (c["k"] + 1) * n_hi <= 1.2e9) \
                and w["bytes"] <= 1.4e9 and w["flops"] <= 3e11:
            return c


# ---- lengths: the same multiset for every seed, in an order that the seed gives ---------------------

def _spread(lo, hi, B, phase):
    f = np.mod((np.arange(B) + 0.5) * 0.6180339887498949 + phase, 1.0)
    return (lo + np.floor(f * (hi - lo + 1))).astype(np.int64)


def _lengths(case):
    """(cached tokens with the new ones, new tokens) of every row."""
    n = _spread(case["n_lo"], case["n_hi"], case["B"], 0.0)
    if case["op"] == "read":
        return n, np.zeros_like(n)
    return n, np.minimum(_spread(1, case["k"] + 1, case["B"], 0.37), n)


def _drafted(case):
    nv = _spread(0, case["k"], case["B"], 0.21)
    greedy = np.arange(case["B"]) < int(round(case["greedy"] * case["B"]))
    return nv, greedy


def _visible(case, n, ql):
    """Pairs (new token, position it sees), and positions that any of a row's new tokens sees."""
    pairs = seen = 0
    w, s = case["window"], case["sinks"]
    for nb, qb in zip(n.tolist(), ql.tolist()):
        p = np.arange(nb - qb, nb)
        first = np.maximum(0, p - w + 1) if w else np.zeros_like(p)
        pairs += int((p - first + 1 + np.minimum(first, s)).sum())
        seen += int(nb - first[0] + min(first[0], s))
    return pairs, seen


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"] == "verify":
        nv, greedy = _drafted(case)
        R, V, B = int((nv + 1).sum()), case["V"], case["B"]
        draws = B - int(greedy.sum())
        b = R * V * es + draws * V * 4 + (draws * V * 4 if case["q"] else 0) + B * (4 * case["k"] + 8) * 3
        return {"bytes": b, "flops": 6 * R * V}
    n, ql = _lengths(case)
    H, D, P = case["Hkv"], case["D"], case["P"]
    blocks = lambda x: int((-(-x // P)).sum())  # noqa: E731
    if case["op"] == "read":
        return {"bytes": int(n.sum()) * H * D * 2 * (1 + es) + blocks(n) * (8 * H + 4), "flops": int(n.sum()) * H * D * 2}
    if case["op"] == "write":
        first = (n - ql) // P * P
        new, touched = int(ql.sum()), int((n - first).sum())
        old = touched - new
        b = new * H * D * 2 * (es + 1) + old * H * D * 2 + blocks(n - first) * (16 * H + 4)   # the write
        b += touched * H * D * 2 * (1 + es) + blocks(n - first) * 8 * H                       # the read back
        return {"bytes": b, "flops": touched * H * D * 2 * 3}
    pairs, seen = _visible(case, n, ql)
    b = seen * H * D * 2 + seen // P * (8 * H + 4) + int(ql.sum()) * H * case["G"] * D * 2 * es
    return {"bytes": b, "flops": 4 * D * pairs * H * case["G"]}


# ---- inputs ------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g, np.random.default_rng(seed)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _inputs_verify(case, seed):
    g, rng = _gen(seed)
    B, k, V, dt = case["B"], case["k"], case["V"], DT[case["dtype"]]
    nv, greedy = _drafted(case)
    order = rng.permutation(B)
    nv, greedy = nv[order], greedy[order]
    at = _starts(nv + 1)
    R = int(at[-1])
    row = np.repeat(np.arange(B), nv + 1)
    pos = np.arange(R) - at[row]
    is_draft = _i32(pos < nv[row]).bool()
    # logits as a language model's: a broad bulk, and at a drafted id what makes it likely or not
    logits = torch.empty(R, V, device=DEV, dtype=dt)
    step = max(1, (1 << 28) // V)
    for a in range(0, R, step):
        logits[a:a + step] = (torch.randn(min(step, R - a), V, generator=g, device=DEV) * 2.5).to(dt)
    drafts = torch.full((B, k), -1, dtype=torch.int32, device=DEV)
    q = None
    if case["q"]:
        q = torch.empty(R, V, device=DEV)
        ids = torch.empty(R, dtype=torch.int64, device=DEV)
        for a in range(0, R, step):
            m = min(step, R - a)
            q[a:a + m] = torch.softmax(logits[a:a + m].float() * 0.9 + torch.randn(m, V, generator=g, device=DEV) * 0.5, -1)
            ids[a:a + m] = (q[a:a + m] / torch.empty(m, V, device=DEV).exponential_(generator=g)).argmax(-1)
    else:
        ids = torch.randint(0, V, (R,), generator=g, device=DEV)
        p = torch.where(torch.rand(R, generator=g, device=DEV) < 0.75, 0.85, 0.1)
        lse = math.log(V) + 2.5 ** 2 / 2
        boost = (lse + torch.log(p / (1 - p))).to(dt)
        r = torch.arange(R, device=DEV)
        logits[r, ids] = torch.where(is_draft, boost, logits[r, ids])
    # one row in eight comes from a sampler that has left only its likeliest ids
    cut = (torch.arange(R, device=DEV) % 8 == 3)[:, None]
    for a in range(0, R, step):
        x = logits[a:a + step]
        x.masked_fill_(cut[a:a + step] & (x < 4.0), float("-inf"))
    r, ps = torch.from_numpy(row).to(DEV), torch.from_numpy(pos).to(DEV)
    slot = torch.where(is_draft, ps, k)
    padded = torch.full((B, k + 1), -1, dtype=torch.int32, device=DEV)
    padded[r, slot] = ids.int()
    drafts.copy_(padded[:, :k])
    temp = torch.rand(B, generator=g, device=DEV) * 0.6 + 0.6
    temp = torch.where(_i32(greedy).bool(), 0.0, temp)
    return dict(logits=logits, drafts=drafts, num_valid=_i32(nv), row_start=_i32(at), temperature=temp, q=q,
                uniform=torch.rand(B, k, generator=g, device=DEV),
                noise=torch.empty(B, V, device=DEV).exponential_(generator=g))


def _inputs_cache(case, seed):
    g, rng = _gen(seed)
    B, H, D, P, dt = case["B"], case["Hkv"], case["D"], case["P"], DT[case["dtype"]]
    n, ql = _lengths(case)
    order = rng.permutation(B)
    n, ql = n[order], ql[order]
    pages = -(-n // P)
    total = int(pages.sum()) + 3
    width = int(pages.max())
    table = np.full((B, width), -1, np.int64)
    free = rng.permutation(total)
    used = 0
    for b in range(B):
        table[b, :pages[b]] = free[used:used + pages[b]]
        used += pages[b]
    s = dict(table=_i32(table), seq_lens=_i32(n), q_start=_i32(_starts(ql)), n=n, ql=ql, width=width)
    # what earlier steps left in the cache: channels and blocks of unequal size
    channel = torch.ones(D, device=DEV)
    channel[rng.integers(0, D, 3)] = 4.0
    for name in ("k", "v"):
        cache = torch.empty(total, H, P, D, device=DEV, dtype=torch.uint8)
        scale = torch.empty(total, H, device=DEV)
        step = max(1, (1 << 27) // (H * P * D))
        for a in range(0, total, step):
            m = min(step, total - a)
            x = torch.randn(m, H, P, D, generator=g, device=DEV)
            if name == "k":
                x *= channel
            x *= torch.exp2(torch.rand(m, H, 1, 1, generator=g, device=DEV) * 2 - 1)
            sc = _scale_of(x.abs().amax((2, 3)))
            scale[a:a + m] = sc
            cache[a:a + m] = _encode(x, sc[:, :, None, None])
        s[name + "_cache"], s[name + "_scale"] = cache, scale
    return s, g, rng


def _handle(case, s):
    """The cache object that a user's program keeps, over the state's own tensors."""
    from model_free_suffix_gb300 import KVCache
    f8 = torch.float8_e4m3fn
    return KVCache(num_pages=s["k_cache"].shape[0], page_size=case["P"], kv_heads=case["Hkv"], head_dim=case["D"],
                   q_heads=case["Hkv"] * case.get("G", 1), max_batch=case["B"], max_pages_per_row=s["width"],
                   storage=(s["k_cache"][None].view(f8), s["v_cache"][None].view(f8), s["k_scale"][None], s["v_scale"][None]))


_drafters = {}


def _drafter(B, k, V):
    """The drafter that a user's program keeps, one per geometry."""
    from model_free_suffix_gb300 import SuffixDrafter
    if (B, k, V) not in _drafters:
        _drafters.clear()
        _drafters[B, k, V] = SuffixDrafter(max_batch=B, seq_capacity=256, vocab_size=V, k=k)
    return _drafters[B, k, V]


def prepare(case, seed):
    if case["op"] == "verify":
        s = dict(case, **_inputs_verify(case, seed))
        if own:
            s["drafter"] = _drafter(case["B"], case["k"], case["V"])
            s["verdict"] = s["drafter"].new_verdict(case["B"])
        return s
    s, g, rng = _inputs_cache(case, seed)
    B, H, D, P, dt = case["B"], case["Hkv"], case["D"], case["P"], DT[case["dtype"]]
    n, ql = s["n"], s["ql"]
    N = int(ql.sum())
    s.update(case, max_q=int(ql.max()))
    if case["op"] == "write":
        # keys and values as a model's projection leaves them: side by side in one row per token
        x = torch.randn(N, 2, H, D, generator=g, device=DEV)
        x *= torch.exp2(torch.randn(N, 1, H, 1, generator=g, device=DEV))
        x = x.to(dt)
        s["k_new"], s["v_new"] = x[:, 0], x[:, 1]
        s["from"] = (n - ql) // P * P
    elif case["op"] == "read":
        s["from"] = np.zeros_like(n)
    else:
        s["q"] = (torch.randn(N, H * case["G"], D, generator=g, device=DEV) * 1.5).to(dt)
        s["scale"] = D ** -0.5
        s["out"] = torch.empty_like(s["q"])
    if case["op"] != "attend":
        s["touched"] = int((n - s["from"]).sum())
        s["out_start"] = _i32(_starts(n - s["from"]))
        s["from_dev"] = _i32(s["from"])
        s["blocks"] = int((-(-(n - s["from"]) // P)).max())
        s["k_out"] = torch.empty(s["touched"], H, D, device=DEV, dtype=dt)
        s["v_out"] = torch.empty_like(s["k_out"])
    if own:
        s["cache"] = _handle(case, s)
    return s


# ---- the plain forms ---------------------------------------------------------------------------------

def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, its exponent held in [-48, 48]."""
    f, e = torch.frexp(amax)
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, EXP_MIN).clamp(EXP_MIN, EXP_MAX)
    return torch.ldexp(torch.ones_like(amax), e)


def _encode(x, scale):
    """e4m3 bytes of x / scale (round to nearest even, saturated)."""
    return (x / scale).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(b):
    return b.view(torch.float8_e4m3fn).float()


def _rows_of(start, N):
    """Of each packed token: its row, and its place within the row."""
    i = torch.arange(N, device=DEV)
    b = torch.searchsorted(start[1:].long(), i, right=True)
    return b, i - start.long()[b]


def _plain_verify(s):
    B, k, V = s["B"], s["k"], s["V"]
    x = s["logits"].float()
    R = x.shape[0]
    row, pos = _rows_of(s["row_start"], R)
    nv, temp = s["num_valid"].long(), s["temperature"]
    greedy = temp < GREEDY_BELOW
    inv = (1.0 / torch.where(greedy, 1.0, temp))[row][:, None]
    m = x.amax(-1, keepdim=True)
    ids = torch.arange(V, device=DEV)
    best = torch.where(x == m, ids, V).amin(-1)
    x = (x - m) * inv
    Z = torch.exp(x).sum(-1)
    slot = s["row_start"].long()[:B, None] + torch.arange(k + 1, device=DEV)[None]          # [B, k+1]
    inside = torch.arange(k, device=DEV)[None] < nv[:, None]
    slot = torch.where(torch.arange(k + 1, device=DEV)[None] <= nv[:, None], slot, s["row_start"].long()[:B, None])
    d = torch.where(inside, s["drafts"].long(), 0)
    at = slot[:, :k]
    p = torch.exp(x[at, d]) / Z[at]
    u = s["uniform"]
    if s["q"] is not None:
        u = u * s["q"][at, d]
    ok = torch.where(greedy[:, None], best[at] == d, u < p) & inside
    acc = torch.cumprod(ok.long(), -1).sum(-1)                                            # accepted drafts
    last = slot.gather(1, acc[:, None])[:, 0]                                             # the row that a token is drawn from
    rejected = acc < nv
    xd = d.gather(1, acc.clamp(max=k - 1)[:, None])
    w = torch.exp(x[last])
    if s["q"] is not None:
        w = w / Z[last][:, None]
        w = torch.where(rejected[:, None], torch.clamp(w - s["q"][last], min=0.0), w)
    else:
        w = torch.where(rejected[:, None] & (ids[None] == xd), 0.0, w)
    w = w / s["noise"].clamp(min=NOISE_MIN)
    drawn = torch.where(w == w.amax(-1, keepdim=True), ids, V).amin(-1)
    token = torch.where(greedy, best[last], drawn)
    places = torch.arange(k + 1, device=DEV)[None]
    out = torch.where(places == acc[:, None], token[:, None], torch.nn.functional.pad(d, (0, 1)))
    used = places <= acc[:, None]
    logp = torch.where(used, x[slot, out] - torch.log(Z)[slot], 0.0)
    return {"sampled": torch.where(used, out, -1).int(), "num_accepted": acc.int(), "logprobs": logp}


def _plain_write(s):
    B, H, P, J = s["B"], s["Hkv"], s["P"], s["blocks"]
    q_start, n = s["q_start"].long(), s["seq_lens"].long()
    ql = q_start[1:] - q_start[:-1]
    start = n - ql
    N = s["k_new"].shape[0]
    b, t = _rows_of(s["q_start"], N)
    first = start // P
    last = (n - 1) // P
    j = torch.arange(J, device=DEV)[None]
    block = torch.minimum(first[:, None] + j, last[:, None])                              # [B, J], the last one repeated
    page = s["table"].long().gather(1, block)
    place = block[:, :, None] * P + torch.arange(P, device=DEV)                           # [B, J, P]
    src = (place - start[:, None, None] + q_start[:-1, None, None]).clamp(0, N - 1)
    fresh = (place >= start[:, None, None]) & (place < n[:, None, None])
    valid = place < n[:, None, None]
    for name in ("k", "v"):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        old = cache[page]                                                                 # [B, J, H, P, D]
        was = _decode(old) * scale[page][..., None, None]
        new = s[name + "_new"].float()[src].transpose(2, 3)
        x = torch.where(fresh[:, :, None, :, None], new, was)
        x = torch.where(valid[:, :, None, :, None], x, 0.0)
        sc = _scale_of(x.abs().amax((3, 4)))
        cache[page] = torch.where(valid[:, :, None, :, None], _encode(x, sc[..., None, None]), old)
        scale[page] = sc


def _plain_read(s):
    b, t = _rows_of(s["out_start"], s["touched"])
    place = s["from_dev"].long()[b] + t
    page, slot = s["table"].long()[b, place // s["P"]], place % s["P"]
    one = lambda name: (_decode(s[name + "_cache"][page, :, slot]) * s[name + "_scale"][page][..., None]).to(s["k_out"].dtype)  # noqa: E731
    return one("k"), one("v")


def _plain_attend(s):
    B, H, G, D, P, T = s["B"], s["Hkv"], s["G"], s["D"], s["P"], s["max_q"]
    q_start, n = s["q_start"].long(), s["seq_lens"].long()
    ql = q_start[1:] - q_start[:-1]
    N, L = s["q"].shape[0], s["width"] * P
    page = s["table"].long().clamp(min=0)
    k, v = ((_decode(s[x + "_cache"][page]) * s[x + "_scale"][page][..., None, None]).transpose(1, 2).reshape(B, H, L, D) for x in ("k", "v"))
    t = torch.arange(T, device=DEV)[None]
    src = (q_start[:-1, None] + t).clamp(max=N - 1)                                       # [B, T]
    q = s["q"].float()[src].reshape(B, T, H, G, D).transpose(1, 2).reshape(B, H, T * G, D)
    z = (q @ k.transpose(-1, -2)).reshape(B, H, T, G, L) * s["scale"]
    p = ((n - ql)[:, None] + t)[:, :, None]                                               # [B, T, 1]
    at = torch.arange(L, device=DEV)[None, None]
    see = at <= p
    if s["window"]:
        see = see & ((at > p - s["window"]) | (at < s["sinks"]))
    z.masked_fill_(~see[:, None, :, None], float("-inf"))
    z = torch.exp(z - z.amax(-1, keepdim=True))
    z = z / z.sum(-1, keepdim=True)
    o = (z.reshape(B, H, T * G, L) @ v).reshape(B, H, T, G, D).transpose(1, 2).reshape(B, T, H * G, D)
    b, i = _rows_of(s["q_start"], N)
    return o[b, i].to(s["q"].dtype)


def run(state):
    s, op = state, state["op"]
    if op == "verify":
        if not own:
            return _plain_verify(s)
        r = s["drafter"].verify(s["logits"], s["drafts"], s["num_valid"], s["uniform"], s["noise"], row_start=s["row_start"],
                                temperature=s["temperature"], draft_probs=s["q"], out=s["verdict"])
        return {"sampled": r.sampled, "num_accepted": r.num_accepted, "logprobs": r.logprobs}
    if op == "attend":
        if not own:
            return _plain_attend(s)
        return s["cache"].attend(s["q"], s["table"], s["seq_lens"], s["q_start"], s["max_q"], scale=s["scale"],
                                 window=s["window"], sinks=s["sinks"], out=s["out"])
    if op == "write":
        if own:
            s["cache"].write(s["k_new"], s["v_new"], s["table"], s["seq_lens"], s["q_start"])
        else:
            _plain_write(s)
    if own:
        k, v = s["cache"].read(s["table"], s["from_dev"], s["out_start"], out=(s["k_out"], s["v_out"]))
    else:
        k, v = _plain_read(s)
    return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]} if op == "write" else {"k": k, "v": v}


# ---- the same from the definitions, in 64 bits -------------------------------------------------------

def _to_e4m3(y):
    """The nearest e4m3 value (ties to the even one, saturated): steps of 2^(e-3), e >= -6."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    u = torch.exp2(e - 3)
    return (torch.round(y / u) * u).clamp(-F8_MAX, F8_MAX)


def _e4m3_values():
    c = np.arange(256)
    e, m, sign = (c >> 3) & 15, c & 7, np.where(c > 127, -1.0, 1.0)
    v = sign * np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[[127, 255]] = np.nan
    return torch.from_numpy(v).to(DEV)


def _exact_blocks(s, case, b, first, last, values):
    """Row b's blocks first..last of the cache: their pages, and for keys and values [tokens, H, D] in 64 bits."""
    ids = s["table"][b, first:last + 1].long()
    both = []
    for name in ("k", "v"):
        x = values[s[name + "_cache"][ids].long()] * s[name + "_scale"][ids].double()[:, :, None, None]
        both.append(x.transpose(1, 2).reshape(-1, case["Hkv"], case["D"]))
    return ids, both


def _exact_cache(case, seed):
    plain = prepare(case, seed)
    values, P, H, D = _e4m3_values(), case["P"], case["Hkv"], case["D"]
    starts = np.concatenate([[0], np.cumsum(plain["ql"])])
    out = {"k": [], "v": []}
    for b, (n, ql) in enumerate(zip(plain["n"].tolist(), plain["ql"].tolist())):
        first, last = int(plain["from"][b]) // P, (n - 1) // P
        ids, both = _exact_blocks(plain, case, b, first, last, values)
        for name, x in zip("kv", both):
            x = x[:n - first * P].clone()
            if case["op"] == "write":
                x[n - ql - first * P:] = plain[name + "_new"][starts[b]:starts[b + 1]].double()
                full = torch.zeros(len(ids) * P, H, D, device=DEV, dtype=torch.float64)
                full[:x.shape[0]] = x
                full = full.view(len(ids), P, H, D)
                # (log2 may be an ulp above the whole number that it should be)
                e = torch.ceil(torch.log2(full.abs().amax((1, 3)) / F8_MAX) - 1e-12).clamp(EXP_MIN, EXP_MAX)
                sc = torch.exp2(e)
                plain[name + "_scale"][ids] = sc.float()
                x = (_to_e4m3(full / sc[:, None, :, None]) * sc[:, None, :, None]).view(-1, H, D)[:x.shape[0]]
            out[name].append(x)
    out = {name: torch.cat(x) for name, x in out.items()}
    if case["op"] == "write":
        out["k_scale"], out["v_scale"] = plain["k_scale"].double(), plain["v_scale"].double()
    return out


def _exact_attend(case, seed):
    s = prepare(case, seed)
    values, P, H, G, D = _e4m3_values(), case["P"], case["Hkv"], case["G"], case["D"]
    starts = np.concatenate([[0], np.cumsum(s["ql"])])
    out = torch.empty(s["q"].shape, device=DEV, dtype=torch.float64)
    for b, (n, ql) in enumerate(zip(s["n"].tolist(), s["ql"].tolist())):
        _, (k, v) = _exact_blocks(s, case, b, 0, (n - 1) // P, values)
        q = s["q"][starts[b]:starts[b + 1]].double().view(ql, H, G, D)
        z = torch.einsum("thgd,jhd->htgj", q, k[:n]) / math.sqrt(D)
        i = torch.arange(n - ql, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        hidden = j > i
        if case["window"]:
            hidden = hidden | ((i - j >= case["window"]) & (j >= case["sinks"]))
        z = z.masked_fill(hidden[None, :, None, :], -math.inf)
        out[starts[b]:starts[b + 1]] = torch.einsum("htgj,jhd->thgd", torch.softmax(z, -1), v[:n]).reshape(ql, H * G, D)
    return out


def _exact_verify(case, seed):
    s = prepare(case, seed)
    start, nv = s["row_start"].cpu().numpy(), s["num_valid"].cpu().numpy()
    drafts, u, temp = s["drafts"].cpu().numpy(), s["uniform"].double().cpu().numpy(), s["temperature"].double().cpu().numpy()
    logp = np.zeros((case["B"], case["k"] + 1))
    for b in range(case["B"]):
        greedy = temp[b] < GREEDY_BELOW
        for i in range(nv[b] + 1):
            x = s["logits"][start[b] + i].double()
            lp = torch.log_softmax(x / (1.0 if greedy else temp[b]), -1)
            if i < nv[b]:
                d = int(drafts[b, i])
                q = float(s["q"][start[b] + i, d]) if s["q"] is not None else 1.0
                value = float(lp[d])
                if (int(torch.nonzero(x == x.max())[0]) == d) if greedy else (u[b, i] * q < math.exp(value)):
                    logp[b, i] = value
                    continue
            if greedy:
                token = int(torch.nonzero(x == x.max())[0])
            else:
                w = torch.exp(lp)
                if i < nv[b]:
                    if s["q"] is not None:
                        w = (w - s["q"][start[b] + i].double()).clamp(min=0)
                    else:
                        w[d] = 0
                token = int((w / s["noise"][b].double()).argmax())
            logp[b, i] = float(lp[token])
            break
    return {"sampled": None, "num_accepted": None, "logprobs": logp}


def exact(case, seed):
    if case["op"] == "verify":
        return _exact_verify(case, seed) if work(case)["bytes"] < 2e9 else None
    with torch.no_grad():
        return _exact_attend(case, seed) if case["op"] == "attend" else _exact_cache(case, seed)
