"""How prompts enter the cache and a step's tokens find their place in it, measured operator by operator.

  assign  the pages of every row for its next tokens, on the device: from how many tokens each row keeps and how many
          new ones it gets, pages given back and handed out, the block tables, and for the packed new tokens their rows,
          positions and slots;
  prompt  attention over whole prompts: causal, heads of queries in groups, packed sequences of different lengths,
          optionally with a sliding window and a few first tokens that stay visible;
  chunk   attention of a chunk of new tokens of each row (keys and values as the model gave them, in 16 bits) over the
          row's earlier tokens in the paged 8-bit cache and over the chunk itself.

`run` computes them in plain torch, in 32 bits, or (own) through the framework's public entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
F8_MAX = 448.0
EXP_MIN, EXP_MAX = -48, 48       # the range of a block scale's exponent
PIECE = 1 << 29                  # scores that the plain attention holds at a time


# ---- the cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # the step of a server with few requests: latency
        dict(name="assign few", op="assign", B=4, k=8, n_lo=400, n_hi=900, P=64, turnover=0.25),
        # the serving batch (256 rows of 1024..4096 tokens, k=16): 5% of its rows finish, as many prompts come in
        dict(name="assign serving", op="assign", B=256, k=16, n_lo=1024, n_hi=4096, P=64, turnover=0.05),
        # a large batch over small pages, a quarter of it replaced at once: prompts of up to 8192 tokens
        dict(name="assign turnover", op="assign", B=1024, k=32, n_lo=1, n_hi=8192, P=16, turnover=0.25),
        # one short prompt: the time to a first token with nothing else to do
        dict(name="prompt one", op="prompt", B=1, n_lo=200, n_hi=200, Hkv=8, G=4, D=128, dtype="bf16", window=0, sinks=0),
        # the serving workload's prompts (1024..8192 tokens), as many as a step takes at once
        dict(name="prompt serving", op="prompt", B=8, n_lo=1024, n_hi=8192, Hkv=8, G=4, D=128, dtype="bf16", window=0, sinks=0),
        # many short ragged prompts, small heads, groups of three
        dict(name="prompt short", op="prompt", B=201, n_lo=1, n_hi=700, Hkv=5, G=3, D=64, dtype="f16", window=0, sinks=0),
        # one long context of the agentic workload (its longest: 32768)
        dict(name="prompt long", op="prompt", B=1, n_lo=32768, n_hi=32768, Hkv=8, G=4, D=128, dtype="bf16", window=0, sinks=0),
        # the same workload with a window of 2048 and 4 first tokens
        dict(name="prompt window", op="prompt", B=5, n_lo=8192, n_hi=32767, Hkv=8, G=8, D=64, dtype="f16", window=2048, sinks=4),
        # one request's last piece of a prompt: latency
        dict(name="chunk one", op="chunk", B=1, k=99, n_lo=2100, n_hi=2100, Hkv=8, G=4, D=128, P=64, dtype="bf16", window=0, sinks=0),
        # a step that mixes rows with one new token and rows with up to 1024, over 1024..8192 tokens
        dict(name="chunk serving", op="chunk", B=24, k=1023, n_lo=1024, n_hi=8192, Hkv=8, G=4, D=128, P=64, dtype="bf16", window=0, sinks=0),
        # a long context goes in by chunks of 2048: the last of them
        dict(name="chunk long", op="chunk", B=1, k=2047, n_lo=32768, n_hi=32768, Hkv=8, G=4, D=128, P=128, dtype="bf16", window=0, sinks=0),
        # chunks of up to 512 with a window of 2048 and 4 first tokens, small heads, small pages
        dict(name="chunk window", op="chunk", B=24, k=511, n_lo=2048, n_hi=16384, Hkv=8, G=8, D=64, P=16, dtype="f16", window=2048, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["assign", "prompt", "prompt", "chunk", "chunk"])
    while True:
        n_hi = _log_int(rng, 1, 32768)
        n_lo = _log_int(rng, 1, n_hi)
        if op == "assign":
            c = dict(op=op, B=_log_int(rng, 1, 2048), k=_log_int(rng, 1, 32), n_lo=n_lo, n_hi=n_hi, P=rng.choice([16, 32, 64, 128]),
                     turnover=rng.choice([0.0, 0.05, 0.25, 1.0]))
            w = work(c)
            if w["bytes"] <= 3e7 and c["B"] * (n_hi + c["k"]) <= 2e7:
                return c
            continue
        c = dict(op=op, B=_log_int(rng, 1, 256), n_lo=n_lo, n_hi=n_hi, Hkv=rng.choice([1, 2, 4, 5, 8, 16]), G=rng.choice([1, 2, 3, 4, 6, 8]),
                 D=rng.choice([64, 128]), dtype=rng.choice(["bf16", "f16"]), window=0, sinks=0)
        if op == "chunk":
            c["k"], c["P"] = _log_int(rng, 1, 4096) - 1, rng.choice([16, 32, 64, 128])
        if rng.random() < 0.4:
            c["window"], c["sinks"] = _log_int(rng, 1, 8192), rng.choice([0, 1, 4, 70])
        n, ql = _lengths(c)
        plain = int((n * ql).sum()) * c["Hkv"] * c["G"]           # the scores that the plain form makes
        w = work(c)
        if plain <= 3e10 and w["flops"] <= 6e12 and int(ql.sum()) * c["Hkv"] * (c["G"] + 2) * c["D"] <= 8e8 \
                and int(n.sum()) * c["Hkv"] * c["D"] <= 8e8:
            return c


# ---- lengths: the same multiset for every seed, in an order that the seed gives ---------------------

def _spread(lo, hi, B, phase):
    f = np.mod((np.arange(B) + 0.5) * 0.6180339887498949 + phase, 1.0)
    return (lo + np.floor(f * (hi - lo + 1))).astype(np.int64)


def _lengths(case):
    """(tokens with the new ones, new tokens) of every row."""
    n = _spread(case["n_lo"], case["n_hi"], case["B"], 0.0)
    return n, n.copy() if case["op"] == "prompt" else np.minimum(_spread(1, case["k"] + 1, case["B"], 0.37), n)


def _steps(case):
    """Two steps of a server that follow one another for ever: (keep, new) of every row, twice.

    Rows that decode keep n in the first step; in the second what was accepted of its 1..k+1 tokens.  The others
    finish in the first (all pages are given back), and a prompt takes their place in the second."""
    B, k = case["B"], case["k"]
    n, x, y = _spread(case["n_lo"], case["n_hi"], B, 0.0), _spread(1, k + 1, B, 0.37), _spread(1, k + 1, B, 0.71)
    kept = n + 1 + np.mod(np.arange(B) * 7, x)
    over = np.arange(B) < int(round(case["turnover"] * B))
    over = over[np.argsort(_spread(0, 1 << 20, B, 0.11), kind="stable")]
    zero = np.zeros_like(n)
    return (np.where(over, zero, n), np.where(over, zero, x)), (np.where(over, zero, kept), np.where(over, n, y))


def _visible(case, n, ql):
    """Pairs (new token, position it sees), and positions that any of a row's new tokens sees, new ones left out."""
    pairs = seen = 0
    w, s = case["window"], case["sinks"]
    for nb, qb in zip(n.tolist(), ql.tolist()):
        p = np.arange(nb - qb, nb)
        first = np.maximum(0, p - w + 1) if w else np.zeros_like(p)
        pairs += int((p - first + 1 + np.minimum(first, s)).sum())
        old = nb - qb
        seen += max(0, old - int(first[0])) + min(int(first[0]), s, old)
    return pairs, seen


def work(case):
    if case["op"] == "assign":
        P, total, held = case["P"], 0, None
        two = _steps(case)
        held = -(-(two[1][0] + two[1][1]) // P)                                         # pages after the step before
        for keep, new in two:
            need = -(-(keep + new) // P)
            give, want = np.maximum(held - need, 0).sum(), np.maximum(need - held, 0).sum()
            touched = np.where(new > 0, need - keep // P, 0).sum()
            total += int(24 * case["B"] + 12 * new.sum() + 12 * give + 8 * want + 4 * touched)
            held = need
        return {"bytes": total, "flops": int(sum(new.sum() for _, new in two))}
    n, ql = _lengths(case)
    H, G, D = case["Hkv"], case["G"], case["D"]
    pairs, seen = _visible(case, n, ql)
    b = int(ql.sum()) * H * D * 2 * (2 * G + 2)                                         # q, k, v and the result, 16 bits
    if case["op"] == "chunk":
        b += seen * H * D * 2 + seen // case["P"] * (8 * H + 4)
    return {"bytes": b, "flops": 4 * D * pairs * H * G}


# ---- inputs ------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g, np.random.default_rng(seed)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _inputs_assign(case, seed):
    _, rng = _gen(seed)
    B, P = case["B"], case["P"]
    order = rng.permutation(B)
    two = [(keep[order], new[order]) for keep, new in _steps(case)]
    held = -(-(two[1][0] + two[1][1]) // P)
    most = int(max((keep + new).max() for keep, new in two))
    width = -(-most // P) + 1
    need = sum(-(-(keep + new) // P) for keep, new in two)                               # enough for either step, and some left
    total = int(need.sum()) + 3
    pages = rng.permutation(total)
    table = np.full((B, width), -1, np.int64)
    at = _starts(held)
    for b in range(B):
        table[b, :held[b]] = pages[at[b]:at[b + 1]]
    free = np.full(total, -1, np.int64)
    count = total - int(at[-1])
    free[:count] = pages[at[-1]:]
    N = int(max(new.sum() for _, new in two))
    return dict(table=_i32(table), held=_i32(held), free=_i32(free), count=_i32([count]), width=width, total=total, N=max(N, 1),
                steps=[(_i32(keep), _i32(new)) for keep, new in two],
                outs=[dict(seq_lens=torch.empty(B, dtype=torch.int32, device=DEV), q_start=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                           **{x: torch.empty(max(N, 1), dtype=torch.int32, device=DEV) for x in ("positions", "slots", "rows")}) for _ in two])


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, its exponent held in [-48, 48]."""
    f, e = torch.frexp(amax)
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, EXP_MIN).clamp(EXP_MIN, EXP_MAX)
    return torch.ldexp(torch.ones_like(amax), e)


def _inputs_attention(case, seed):
    g, rng = _gen(seed)
    B, H, G, D, dt = case["B"], case["Hkv"], case["G"], case["D"], DT[case["dtype"]]
    n, ql = _lengths(case)
    order = rng.permutation(B)
    n, ql = n[order], ql[order]
    at, N = _starts(ql), int(ql.sum())
    s = dict(n=n, ql=ql, q_start=_i32(at), seq_lens=_i32(n), scale=D ** -0.5)
    # queries, keys and values as a model's projection leaves them: side by side in one row per token, a few channels
    # of the keys larger than the others
    channel = torch.ones(H * (G + 2), D, device=DEV)
    channel[H * G:H * (G + 1), rng.integers(0, D, 3)] = 4.0
    channel[:H * G] = 1.5
    x = torch.empty(N, H * (G + 2), D, device=DEV, dtype=dt)
    step = max(1, (1 << 27) // (H * (G + 2) * D))
    for a in range(0, N, step):
        x[a:a + step] = (torch.randn(min(step, N - a), H * (G + 2), D, generator=g, device=DEV) * channel).to(dt)
    s["q"], s["k"], s["v"] = x[:, :H * G], x[:, H * G:H * (G + 1)], x[:, H * (G + 1):]
    s["out"] = torch.empty(N, H * G, D, device=DEV, dtype=dt)
    # what the plain form takes at a time: (row, its new tokens from .. to)
    s["pieces"] = []
    for b in range(B):
        most = max(1, PIECE // (H * G * int(n[b])))
        s["pieces"] += [(b, t, min(t + most, int(ql[b]))) for t in range(0, int(ql[b]), most)]
    if case["op"] == "prompt":
        return s
    P = case["P"]
    pages = -(-n // P)
    total, width = int(pages.sum()) + 3, int(pages.max())
    table = np.full((B, width), -1, np.int64)
    free, used = rng.permutation(total), _starts(pages)
    for b in range(B):
        table[b, :pages[b]] = free[used[b]:used[b + 1]]
    s.update(table=_i32(table), width=width)
    # what earlier chunks left in the cache: blocks of unequal size
    for name in ("k", "v"):
        cache = torch.empty(total, H, P, D, device=DEV, dtype=torch.uint8)
        scale = torch.empty(total, H, device=DEV)
        step = max(1, (1 << 27) // (H * P * D))
        for a in range(0, total, step):
            m = min(step, total - a)
            y = torch.randn(m, H, P, D, generator=g, device=DEV)
            if name == "k":
                y *= channel[H * G]
            y *= torch.exp2(torch.rand(m, H, 1, 1, generator=g, device=DEV) * 2 - 1)
            sc = _scale_of(y.abs().amax((2, 3)))
            scale[a:a + m] = sc
            cache[a:a + m] = (y / sc[:, :, None, None]).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_cache"], s[name + "_scale"] = cache, scale
    return s


def prepare(case, seed):
    s = dict(case, **(_inputs_assign(case, seed) if case["op"] == "assign" else _inputs_attention(case, seed)))
    if own:
        from model_free_suffix_gb300 import KVCache, KVPages, PagePlan
        if case["op"] == "assign":
            s["cache"] = KVCache(num_pages=s["total"], page_size=case["P"], kv_heads=1, head_dim=64, max_batch=case["B"],
                                 max_pages_per_row=s["width"])
            s["pages"] = KVPages(s["table"], s["held"], s["free"], s["count"])
            s["plans"] = [PagePlan(**o) for o in s["outs"]]
        elif case["op"] == "prompt":
            s["cache"] = KVCache(num_pages=1, page_size=64, kv_heads=case["Hkv"], head_dim=case["D"], q_heads=case["Hkv"] * case["G"],
                                 max_batch=case["B"], max_pages_per_row=1)
        else:
            f8 = torch.float8_e4m3fn
            s["cache"] = KVCache(num_pages=s["k_cache"].shape[0], page_size=case["P"], kv_heads=case["Hkv"], head_dim=case["D"],
                                 q_heads=case["Hkv"] * case["G"], max_batch=case["B"], max_pages_per_row=s["width"],
                                 storage=(s["k_cache"][None].view(f8), s["v_cache"][None].view(f8), s["k_scale"][None], s["v_scale"][None]))
    return s


# ---- the plain forms ---------------------------------------------------------------------------------

def _plain_assign(s, keep, new, out):
    """Rows whose keep or new makes no sense hold what they have and get nothing; then, row by row, what does not fit
    the packed tokens or the free pages.  Pages given back go on the free list first, in the order of the rows;
    those handed out come from its end."""
    P, N = s["P"], s["N"]
    B, W = s["table"].shape
    table, held, free = s["table"].long(), s["held"].long(), s["free"].long()
    keep, new, count = keep.long(), new.long(), s["count"].long()
    j = torch.arange(W, device=DEV)[None]
    good = (keep >= 0) & (new >= 0) & (keep <= held * P) & (keep + new <= W * P)
    new = torch.where(good, new, 0)
    new = torch.where(torch.cumsum(new, 0) <= N, new, 0)
    need = torch.where(good, (keep + new + P - 1) // P, held)
    back = (j >= need[:, None]) & (j < held[:, None])
    place = torch.where(back, count + torch.cumsum(back.flatten(), 0).view(B, W) - 1, s["total"])
    free = torch.cat([free, free[:1]]).scatter(0, place.flatten(), table.flatten())[:-1]
    count = count + back.sum()
    want = (need - held).clamp(min=0)
    served = (torch.cumsum(want, 0) <= count) | (want == 0)
    new, need = torch.where(served, new, 0), torch.where(served, need, held)
    take = (j >= held[:, None]) & (j < need[:, None])
    at = count - torch.cumsum(take.flatten(), 0).view(B, W)
    table = torch.where(take, free[at.clamp(0, s["total"] - 1)], torch.where(back, -1, table))
    s["table"].copy_(table)
    s["held"].copy_(need)
    s["free"].copy_(free)
    s["count"].copy_(count - take.sum())
    q_start = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    out["seq_lens"].copy_(torch.where(good, keep + new, 0))
    out["q_start"].copy_(q_start)
    i = torch.arange(N, device=DEV)
    row = torch.searchsorted(q_start[1:], i, right=True).clamp(max=B - 1)
    live = i < q_start[B]
    position = torch.where(live, keep[row] + i - q_start[row], 0)
    out["rows"].copy_(torch.where(live, row, -1))
    out["positions"].copy_(position)
    out["slots"].copy_(torch.where(live, table[row, position // P] * P + position % P, -1))


def _cached(s, name, b, m):
    """Positions 0 .. m - 1 of row b: [m, H, D]."""
    page = s["table"][b, :-(-m // s["P"])].long()
    x = s[name + "_cache"][page].view(torch.float8_e4m3fn).float() * s[name + "_scale"][page][:, :, None, None]
    return x.transpose(1, 2).reshape(-1, s["Hkv"], s["D"])[:m]


def _plain_attention(s):
    H, G, D = s["Hkv"], s["G"], s["D"]
    starts = _starts(s["ql"])
    for b, t0, t1 in s["pieces"]:
        old, at, T = int(s["n"][b] - s["ql"][b]), int(starts[b]), t1 - t0
        k, v = s["k"][at:at + t1].float(), s["v"][at:at + t1].float()
        if s["op"] == "chunk":
            k, v = torch.cat([_cached(s, "k", b, old), k]), torch.cat([_cached(s, "v", b, old), v])
        q = s["q"][at + t0:at + t1].float().reshape(T, H, G, D).permute(1, 0, 2, 3).reshape(H, T * G, D)
        z = torch.matmul(q, k.permute(1, 2, 0)).view(H, T, G, old + t1).mul_(s["scale"])
        p, j = torch.arange(old + t0, old + t1, device=DEV)[:, None], torch.arange(old + t1, device=DEV)[None]
        hidden = j > p
        if s["window"]:
            hidden |= (j <= p - s["window"]) & (j >= s["sinks"])
        z.masked_fill_(hidden[None, :, None], float("-inf"))
        z = z.sub_(z.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(z.view(H, T * G, -1), v.transpose(0, 1)).view(H, T, G, D) / z.sum(-1, keepdim=True)
        s["out"][at + t0:at + t1] = o.transpose(0, 1).reshape(T, H * G, D).to(s["out"].dtype)
    return s["out"]


def run(state):
    s = state
    if s["op"] == "assign":
        if own:
            for (keep, new), plan in zip(s["steps"], s["plans"]):
                s["cache"].assign(s["pages"], keep, new, out=plan)
        else:
            for (keep, new), out in zip(s["steps"], s["outs"]):
                _plain_assign(s, keep, new, out)
        return {"steps": s["outs"], "table": s["table"], "held": s["held"], "free": s["free"], "count": s["count"]}
    if not own:
        return _plain_attention(s)
    if s["op"] == "prompt":
        return s["cache"].attend_prompt(s["q"], s["k"], s["v"], s["q_start"], scale=s["scale"], window=s["window"], sinks=s["sinks"],
                                        out=s["out"])
    return s["cache"].attend_chunk(s["q"], s["k"], s["v"], s["table"], s["seq_lens"], s["q_start"], scale=s["scale"],
                                   window=s["window"], sinks=s["sinks"], out=s["out"])


# ---- the same from the definitions, in 64 bits (whole numbers: one at a time) ------------------------

def _exact_assign(case, seed):
    s = prepare(case, seed)
    P, N = case["P"], s["N"]
    table, free = s["table"].tolist(), s["free"].tolist()
    held, top = s["held"].tolist(), int(s["count"])
    steps = []
    for keep, new in s["steps"]:
        keep, new = keep.tolist(), new.tolist()
        # given back in the order of a row's table, rows in theirs
        for b in range(case["B"]):
            need = -(-(keep[b] + new[b]) // P)
            for j in range(need, held[b]):
                free[top], table[b][j] = table[b][j], -1
                top += 1
            held[b] = min(held[b], need)
        rows, positions, slots, starts = [], [], [], [0]
        for b in range(case["B"]):
            while held[b] * P < keep[b] + new[b]:
                top -= 1
                table[b][held[b]] = free[top]
                held[b] += 1
            for p in range(keep[b], keep[b] + new[b]):
                rows.append(b)
                positions.append(p)
                slots.append(table[b][p // P] * P + p % P)
            starts.append(len(rows))
        empty = N - len(rows)
        steps.append(dict(seq_lens=[a + c for a, c in zip(keep, new)], q_start=starts, positions=positions + [0] * empty,
                          slots=slots + [-1] * empty, rows=rows + [-1] * empty))
    as_array = lambda x: np.asarray(x, dtype=np.int64)  # noqa: E731
    return {"steps": [{k: as_array(v) for k, v in st.items()} for st in steps], "table": as_array(table), "held": as_array(held),
            "free": as_array(free), "count": as_array([top])}


def _e4m3_values():
    c = np.arange(256)
    e, m, sign = (c >> 3) & 15, c & 7, np.where(c > 127, -1.0, 1.0)
    v = sign * np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[[127, 255]] = np.nan
    return torch.from_numpy(v).to(DEV)


def _exact_attention(case, seed):
    s = prepare(case, seed)
    H, G, D, values = case["Hkv"], case["G"], case["D"], _e4m3_values()
    out = torch.empty(s["q"].shape, device=DEV, dtype=torch.float64)
    first = 0
    for b, (n, ql) in enumerate(zip(s["n"].tolist(), s["ql"].tolist())):
        old = n - ql
        both = []
        for name in ("k", "v"):
            x = s[name][first:first + ql].double()
            if old:
                page = s["table"][b, :(old - 1) // case["P"] + 1].long()
                y = values[s[name + "_cache"][page].long()] * s[name + "_scale"][page].double()[:, :, None, None]
                x = torch.cat([y.permute(0, 2, 1, 3).reshape(-1, H, D)[:old], x])
            both.append(x)
        k, v = both
        i = torch.arange(old, n, device=DEV)
        step = max(1, (1 << 27) // (G * n))
        for h in range(H):
            for t in range(0, ql, step):
                p = i[t:t + step, None]
                low = max(0, int(p[0]) - case["window"] + 1) if case["window"] else 0
                at = torch.cat([torch.arange(min(low, case["sinks"]), device=DEV), torch.arange(low, int(p[-1]) + 1, device=DEV)])
                j = at[None]
                seen = j <= p
                if case["window"]:
                    seen &= (p - j < case["window"]) | (j < case["sinks"])
                q = s["q"][first + t:first + t + len(p), h * G:(h + 1) * G].double()
                z = torch.einsum("tgd,jd->tgj", q, k[at, h]) / math.sqrt(D)
                w = torch.softmax(torch.where(seen[:, None], z, -math.inf), -1)
                out[first + t:first + t + len(p), h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", w, v[at, h])
        first += ql
    return out


def exact(case, seed):
    if case["op"] == "assign":
        return _exact_assign(case, seed)
    # (products in 64 bits: about a TFLOP/s)
    if work(case)["flops"] > 6e12:
        return None
    with torch.no_grad():
        return _exact_attention(case, seed)
