"""What a serving step does with attention weights and logits, as measured cases.

Three operators:

* ``score``  -- the attention weight that every cached token has drawn so far,
  brought up to date with a step's rows (``ddl_kv8_score``);
* ``evict``  -- the 8-bit paged cache of a request cut to its heaviest tokens
  by that weight, each K/V head by its own, and moved to new pages
  (``ddl_kv8_evict``);
* ``sample`` -- the next tokens from logits, each row with its own temperature,
  top-k, top-p and min-p, from given random numbers (``ddl_sample``).

``run`` computes them with elementary torch operations, or with the
framework's entry points where ``own`` is set.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16  # tokens that share one scale
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def listed():
    return [
        # The small layer at batch 1: the smallest scoring call.
        {"name": "score small b1", "op": "score", "R": 1, "rows": 1, "H_q": 8, "H_kv": 2, "hd": 64, "page": 16,
         "max_len": 129, "codes": "e4m3", "dtype": "bf16", "softcap": 0.0, "window": 0, "slopes": False, "decay": 1.0},
        # Batch 1 of a 70B-class layer, cache 32768, 8-bit integers, fp32 rows as the layer stack has them.
        {"name": "score b1 32k int8", "op": "score", "R": 1, "rows": 1, "H_q": 64, "H_kv": 8, "hd": 128, "page": 256,
         "max_len": 32769, "codes": "int8", "dtype": "f32", "softcap": 0.0, "window": 0, "slopes": False,
         "decay": 1.0},
        # A full batch at ragged lengths up to 8192: the ordinary serving step, memory-bound.
        {"name": "score b64 8k", "op": "score", "R": 64, "rows": 1, "H_q": 64, "H_kv": 8, "hd": 128, "page": 64,
         "max_len": 8192, "codes": "e4m3", "dtype": "bf16", "softcap": 0.0, "window": 0, "slopes": False,
         "decay": 0.99},
        # 64 prompt rows each of two requests, groups of 7 heads, capped scores: compute counts here.
        {"name": "score chunk 64 rows", "op": "score", "R": 2, "rows": 64, "H_q": 28, "H_kv": 4, "hd": 128, "page": 32,
         "max_len": 8192, "codes": "e4m3", "dtype": "f16", "softcap": 30.0, "window": 0, "slopes": False,
         "decay": 1.0},
        # One short sequence cut to half: latency counts.
        {"name": "evict small b1", "op": "evict", "R": 1, "H_kv": 2, "hd": 64, "page": 16, "max_len": 129, "keep": 65,
         "sinks": 4, "recent": 16, "codes": "e4m3"},
        # A long sequence of 8-bit integers cut to a quarter: few heads, a long axis to choose from.
        {"name": "evict b1 32k int8", "op": "evict", "R": 1, "H_kv": 8, "hd": 128, "page": 256, "max_len": 32769,
         "keep": 8193, "sinks": 4, "recent": 512, "codes": "int8"},
        # Several ragged sequences, some of them short enough to stay as they are, an odd budget.
        {"name": "evict b9 4k", "op": "evict", "R": 9, "H_kv": 4, "hd": 128, "page": 32, "max_len": 4097, "keep": 1531,
         "sinks": 0, "recent": 33, "codes": "e4m3"},
        # A full batch that has outgrown its pool: memory-bound.
        {"name": "evict b32 8k", "op": "evict", "R": 32, "H_kv": 8, "hd": 128, "page": 64, "max_len": 8192,
         "keep": 2048, "sinks": 16, "recent": 256, "codes": "e4m3"},
        # One sequence over the framework's vocabulary: latency counts.
        {"name": "sample b1 152k", "op": "sample", "B": 1, "V": 152064, "dtype": "f32", "how": "top_p", "masked": 0.0},
        # A full batch, every row with settings of its own (one greedy, one without any filter), banned tokens.
        {"name": "sample b64 152k mixed", "op": "sample", "B": 64, "V": 152064, "dtype": "f32", "how": "mixed",
         "masked": 0.1},
        # An odd vocabulary in fp16 (rows are not aligned), min-p.
        {"name": "sample b17 50257 min-p", "op": "sample", "B": 17, "V": 50257, "dtype": "f16", "how": "min_p",
         "masked": 0.0},
        # Many rows of bf16 logits (whose values repeat), top-k and top-p.
        {"name": "sample b256 bf16", "op": "sample", "B": 256, "V": 128256, "dtype": "bf16", "how": "top_kp",
         "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["score", "evict", "sample"])
    page, hd, codes = rng.choice([16, 32, 64, 256]), rng.choice([64, 128]), rng.choice(["e4m3", "int8"])
    if op == "sample":
        B = _log(rng, 1, 256)
        V = _log(rng, 200, min(262144, 256 * 128256 // B))
        return {"op": op, "B": B, "V": V, "dtype": rng.choice(["f32", "f32", "bf16", "f16"]),
                "how": rng.choice(["plain", "top_k", "top_p", "min_p", "top_kp", "mixed"]),
                "masked": rng.choice([0.0, 0.0, 0.1, 0.9])}
    H_kv = rng.choice([1, 2, 4, 8])
    if op == "evict":
        R = _log(rng, 1, 32)
        max_len = _log(rng, 2, min(32769, 32 * 8192 // R))
        keep = _log(rng, 1, max(1, min(max_len - 1, 32 * 2048 // R)))
        return {"op": op, "R": R, "H_kv": H_kv, "hd": hd, "page": page, "max_len": max_len, "keep": keep,
                "sinks": rng.choice([0, 4, 17]), "recent": rng.choice([0, 1, 1 + keep // 4]), "codes": codes}
    R, rows = _log(rng, 1, 64), rng.choice([1, 1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 64)])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    most = min(32769, 64 * 8192 // (R * max(1, rows // 2)))
    max_len = _log(rng, rows, max(rows, most))
    return {"op": op, "R": R, "rows": rows, "H_q": H_kv * group, "H_kv": H_kv, "hd": hd, "page": page,
            "max_len": max_len, "codes": codes, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
            "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]), "window": rng.choice([0, 0, 1 + max_len // 3]),
            "slopes": rng.choice([False, False, True]), "decay": rng.choice([1.0, 0.9, 0.99])}


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Per request: tokens in the cache and the step's rows among them (score), or tokens and how many of them stay
    (evict); host arrays of the case alone: the work and the plain form's sizes follow from them, whatever the seed."""
    g = np.random.RandomState(4321)
    R, most = case["R"], case["max_len"]
    if case["op"] == "evict":
        total = 1 + (g.rand(R) * most).astype(np.int64)
        total[0] = most
        return total, np.minimum(total, case["keep"])
    rows = case["rows"]
    add = np.full(R, rows)
    if R > 1 and rows > 1:
        add[1:] = g.randint(1, rows + 1, R - 1)
    total = add + (g.rand(R) * (most - add + 1)).astype(np.int64)
    total[0] = most
    return total, add.astype(np.int64)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _table(need, ids, per):
    table = np.full((len(need), per), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    return table


def _pool(s, case, pages, g):
    # what quantized rows of about N(0, 1) look like: codes spread over the type's range, scales near 2^-7 (e4m3)
    # or 2^-5 (int8), differing by head and block
    H, P, hd = case["H_kv"], case["page"], case["hd"]
    codes = CODES[case["codes"]]
    width, e0 = (128.0, -7) if codes == torch.float8_e4m3fn else (32.0, -5)
    for name in ("k", "v"):
        pool = torch.empty((pages, H, P, hd), dtype=codes, device="cuda")
        step = max(1, (1 << 26) // (H * P * hd))
        for i in range(0, pages, step):
            n = min(step, pages - i)
            x = torch.randn((n, H, P, hd), generator=g, device="cuda", dtype=torch.float32) * width
            pool[i:i + n] = (x if codes == torch.float8_e4m3fn else x.round()).clamp(-127, 127).to(codes)
        e = torch.randint(-1, 2, (pages, H, P // BLOCK), generator=g, device="cuda", dtype=torch.int32)
        s[name] = pool
        s[name + "_scale"] = ((e + (e0 + 127)) << 23).view(torch.float32)


def _settings(case, rng):
    """Per row: temperature (0: greedy), top_k (0: all), top_p and min_p (1 and 0: all)."""
    B, how = case["B"], case["how"]
    t, k, p, m = np.ones(B), np.zeros(B, np.int64), np.ones(B), np.zeros(B)
    t[:] = rng.choice([0.6, 0.8, 1.0, 1.3], B)
    if how in ("top_k", "top_kp"):
        k[:] = rng.choice([1, 20, 50, 1000, 5000], B)
    if how in ("top_p", "top_kp"):
        p[:] = rng.choice([0.5, 0.9, 0.95, 0.99], B)
    if how == "min_p":
        m[:] = rng.choice([0.02, 0.05, 0.1], B)
    if how == "mixed":
        kind = (np.arange(B) + rng.randint(0, 6)) % 6
        t[kind == 0] = 0.0
        k[(kind == 2) | (kind == 5)] = 40
        p[(kind == 3) | (kind == 5)] = 0.9
        m[(kind == 4) | (kind == 5)] = 0.05
    return t, k, p, m


def _prepare_sample(case, seed):
    rng = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, V = case["B"], case["V"]
    # the bulk of a vocabulary at about N(0, 2), a few tokens well above it, as a model's logits have them
    x = torch.randn((B, V), generator=g, device="cuda") * 2.0
    n = min(V, 32)
    at = torch.randint(0, V, (B, n), generator=g, device="cuda")
    x.scatter_add_(1, at, torch.rand((B, n), generator=g, device="cuda") * 10.0)
    if case["masked"]:
        x.masked_fill_(torch.rand((B, V), generator=g, device="cuda") < case["masked"], -math.inf)
    t, k, p, m = _settings(case, rng)
    f32 = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    return {"case": case, "logits": x.to(DTYPES[case["dtype"]]), "temperature": f32(t), "top_k": _dev(k), "top_p": f32(p),
            "min_p": f32(m), "u": torch.rand(B, generator=g, device="cuda"),
            "tokens": torch.zeros(B, dtype=torch.int32, device="cuda"), "logp": torch.zeros(B, device="cuda")}


def prepare(case, seed):
    if case["op"] == "sample":
        return _prepare_sample(case, seed)
    rng = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device="cuda").manual_seed(seed)
    R, H, P, L = case["R"], case["H_kv"], case["page"], case["max_len"]
    total, second = _lengths(case)
    s = {"case": case, "kv_len": _dev(total)}
    held = -(-total // P)
    # what earlier steps have left: most tokens have drawn little, a few much, many of an old decaying one nothing
    score = torch.exp(2.0 * torch.randn((R, H, L), generator=g, device="cuda") - 4.0)
    score.masked_fill_(torch.rand((R, H, L), generator=g, device="cuda") < 0.05, 0.0)
    s["score"] = score
    if case["op"] == "evict":
        new = np.where(second < total, -(-second // P), 0)
        pages = int(held.sum() + new.sum()) + 3
        ids = rng.permutation(pages).astype(np.int32)
        s["page_table"] = _dev(_table(held, ids, int(held.max()) + 1))
        s["new_table"] = _dev(_table(new, ids[int(held.sum()):], -(-case["keep"] // P)))
        s["keep_len"] = _dev(np.full(R, case["keep"]))
        s["kept"] = torch.full((R, H, case["keep"]), -1, dtype=torch.int32, device="cuda")
        s["score_out"] = torch.zeros_like(score)
        _pool(s, case, pages, g)
        return s
    pages = int(held.sum()) + 3
    table = _table(held, rng.permutation(pages).astype(np.int32), int(held.max()) + 1)
    s["page_table"] = _dev(table)
    _pool(s, case, pages, g)
    T = int(second.sum())
    s["q"] = torch.randn((T, case["H_q"], case["hd"]), generator=g, device="cuda").to(DTYPES[case["dtype"]])
    s["q_off"] = None if case["rows"] == 1 else _dev(np.concatenate([[0], np.cumsum(second)]))
    s["slopes"] = None
    if case["slopes"]:  # one slope per head, a geometric sequence
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["H_q"] + 1, device="cuda").float() / case["H_q"])
    # the log-sum-exp that the attention of the same rows has returned
    lse = torch.empty((T, case["H_q"]), device="cuda")
    at = 0
    for r in range(R):
        n = int(second[r])
        w = _scores_64(case, s, table[r], int(total[r]), n, at)
        lse[at:at + n] = torch.logsumexp(w, -1).permute(2, 0, 1).reshape(n, -1).float()
        at += n
    s["lse"] = lse
    return s


def _scores_64(case, s, pages, L, n, at):
    """Scores of a request's rows in 64 bits: [H_kv][group][n][L], -inf where a row does not see a token."""
    H_q, H, hd, P = case["H_q"], case["H_kv"], case["hd"], case["page"]
    ids = torch.from_numpy(pages[:-(-L // P)].astype(np.int64)).cuda()
    k = s["k"].view(torch.uint8)[ids].view(s["k"].dtype).double().transpose(0, 1)
    f = s["k_scale"][ids].double().transpose(0, 1)
    k = (k.reshape(H, -1, BLOCK, hd) * f.reshape(H, -1, 1, 1)).reshape(H, -1, hd)[:, :L]
    q = s["q"][at:at + n].double().view(n, H, H_q // H, hd).permute(1, 2, 0, 3)
    w = torch.einsum("hgnd,hkd->hgnk", q, k) / math.sqrt(hd)
    if case["softcap"]:
        w = torch.tanh(w / case["softcap"]) * case["softcap"]
    dist = torch.arange(L - n, L, device="cuda")[:, None] - torch.arange(L, device="cuda")[None, :]
    if case["slopes"]:
        w = w - s["slopes"].double().view(H, -1, 1, 1) * dist
    hidden = (dist < 0) | (dist >= case["window"]) if case["window"] else dist < 0
    return w.masked_fill(hidden, -math.inf)


# ------------------------------------------------------------------ the operators

def _score_plain(s):
    case = s["case"]
    R, S, H_q, H, hd, L, P = (case[n] for n in ("R", "rows", "H_q", "H_kv", "hd", "max_len", "page"))
    q, G = s["q"], H_q // H
    dev = q.device
    lens = s["kv_len"].long()
    if s["q_off"] is None:
        start, rows = torch.arange(R, device=dev), torch.ones(R, device=dev, dtype=torch.long)
    else:
        start, rows = s["q_off"][:-1].long(), (s["q_off"][1:] - s["q_off"][:-1]).long()
    i = torch.arange(S, device=dev)[None, :]
    at = (start[:, None] + i).clamp(max=q.shape[0] - 1)
    n = -(-L // P)
    ids = s["page_table"][:, :n].long().clamp(min=0)
    k = s["k"].view(torch.uint8)[ids].view(s["k"].dtype).float()
    k = k * s["k_scale"][ids].repeat_interleave(BLOCK, -1)[..., None]
    k = k.transpose(1, 2).reshape(R, H, n * P, hd)[:, :, :L]
    qp = q[at].float().view(R, S, H, G, hd).permute(0, 2, 3, 1, 4).reshape(R, H, G * S, hd)
    w = (qp @ k.transpose(-1, -2)).view(R, H, G, S, L) * (1.0 / math.sqrt(hd))
    if case["softcap"]:
        w = case["softcap"] * torch.tanh(w / case["softcap"])
    far = (lens - rows)[:, None, None] + i[..., None] - torch.arange(L, device=dev)
    if s["slopes"] is not None:
        w = w - s["slopes"].view(1, H, G, 1, 1) * far[:, None, None].float()
    seen = (far >= 0) & (i < rows[:, None])[..., None]
    if case["window"]:
        seen = seen & (far < case["window"])
    lse = s["lse"][at].view(R, S, H, G).permute(0, 2, 3, 1)[..., None]
    p = torch.where(seen[:, None, None], torch.exp(w - lse), 0.0)
    j = torch.arange(L, device=dev)
    old = (j < (lens - rows)[:, None])[:, None]  # tokens that were there before the step; the step's begin at zero
    fresh = torch.where(old, case["decay"] * s["score"], 0.0) + p.sum((2, 3))
    s["score"].copy_(torch.where((j < lens[:, None])[:, None], fresh, s["score"]))
    return s["score"]


def _evict_plain(s):
    case = s["case"]
    R, H, hd, L, P, keep = (case[n] for n in ("R", "H_kv", "hd", "max_len", "page", "keep"))
    int8 = case["codes"] == "int8"
    lens, score = s["kv_len"].long(), s["score"]
    dev = score.device
    cut = lens > keep
    j = torch.arange(L, device=dev)
    recent = min(case["recent"], keep)
    sinks = min(case["sinks"], keep - recent)
    here = j < lens[:, None]
    sure = ((j < sinks) | (j >= lens[:, None] - recent)) & here
    rank = torch.where(sure[:, None], math.inf, torch.where(here[:, None], score, -math.inf))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    chosen = order.sort(-1).values  # ascending, [R][H][keep]
    s["kept"].copy_(torch.where(cut[:, None, None], chosen, s["kept"].long()))
    moved = torch.zeros_like(score)
    moved[..., :keep] = score.gather(-1, chosen)
    stays = torch.where(cut[:, None], j < keep, here)
    s["score_out"].copy_(torch.where(stays[:, None], torch.where(cut[:, None, None], moved, score), s["score_out"]))
    # blocks of 16 kept tokens with a scale of their own; what the last one lacks is zero
    nb = -(-keep // BLOCK)
    pad = nb * BLOCK - keep
    idx = torch.nn.functional.pad(chosen, (0, pad)).view(R, H, nb, BLOCK)
    there = torch.nn.functional.pad(torch.ones_like(chosen, dtype=torch.bool), (0, pad)).view(R, H, nb, BLOCK)
    page = torch.take_along_dim(s["page_table"].long()[:, None], (idx // P).view(R, H, -1), -1).view_as(idx).clamp(min=0)
    head = torch.arange(H, device=dev)[None, :, None, None]
    r = torch.nonzero(cut)[:, 0]
    to = s["new_table"].long()[:, torch.arange(nb, device=dev) * BLOCK // P]  # [R][nb]
    sub = (torch.arange(nb, device=dev) * BLOCK % P // BLOCK).expand(R, nb)
    outs = []
    for name in ("k", "v"):
        pool, scale = s[name], s[name + "_scale"]
        raw = pool.view(torch.uint8)
        x = raw[page[r], head, idx[r] % P].view(pool.dtype).float()
        x = x * scale[page[r], head, idx[r] % P // BLOCK][..., None]
        x = torch.where(there[r][..., None], x, 0.0)
        amax = x.abs().amax((-1, -2))
        # the smallest power of two with amax / scale <= 448 = 0.875 * 2^9, or 127 = 0.9921875 * 2^7
        f, e = torch.frexp(amax)
        e = torch.where(f <= (0.9921875 if int8 else 0.875), e - (7 if int8 else 9), e - (6 if int8 else 8)).clamp(min=-126)
        now = torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), 0.0)
        y = torch.where(now[..., None, None] > 0, x / now[..., None, None], 0.0)
        code = y.round().clamp(-127, 127).to(torch.int8) if int8 else y.clamp(-448, 448).to(torch.float8_e4m3fn)
        view = raw.view(raw.shape[0], H, P // BLOCK, BLOCK, hd)
        view[to[r][:, None], head[..., 0], sub[r][:, None]] = code.view(torch.uint8)
        scale[to[r][:, None], head[..., 0], sub[r][:, None]] = now
        outs += [pool, scale]
    return outs + [s["kept"], s["score_out"]]


def _sample_plain(s):
    x, u = s["logits"].float(), s["u"].double()
    B, V = x.shape
    t = s["temperature"].double()[:, None]
    greedy = ~(t > 0)
    top = x.amax(-1, keepdim=True)
    w = torch.exp((x.double() - top.double()) / torch.where(greedy, 1.0, t))
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    w_sorted = w.gather(-1, order)
    rank = torch.arange(V, device=x.device)[None, :]
    k = s["top_k"].long()[:, None]
    keep = (rank < torch.where(k > 0, k, V)) & torch.isfinite(x).gather(-1, order)
    keep = keep & ~(greedy & (rank > 0))
    inside = torch.where(keep, w_sorted, 0.0)
    before = inside.cumsum(-1) - inside
    p = s["top_p"].double()[:, None]
    keep_p = keep & ((before < p * inside.sum(-1, keepdim=True)) | (p >= 1)) & (w_sorted >= s["min_p"].double()[:, None])
    keep_p = keep_p | (keep & (rank == 0))
    mass = torch.zeros_like(w).scatter_(-1, order, torch.where(keep_p, w_sorted, 0.0))
    total = mass.sum(-1, keepdim=True)
    token = (mass.cumsum(-1) > u[:, None] * total).to(torch.uint8).argmax(-1, keepdim=True)
    logp = torch.log(mass.gather(-1, token) / total)[:, 0]
    s["tokens"].copy_(token[:, 0])
    s["logp"].copy_(logp)
    return s["tokens"], s["logp"]


def _run_own(s):
    from memory_bound_transformer_decode_gb300 import ddl

    case = s["case"]
    if case["op"] == "sample":
        ddl.ddl_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                       min_p=s["min_p"], tokens=s["tokens"], logp=s["logp"])
        return s["tokens"], s["logp"]
    pool = (s["k"], s["v"], s["k_scale"], s["v_scale"])
    if case["op"] == "score":
        ddl.ddl_kv8_score(pool, s["q"], s["lse"], s["kv_len"], s["page_table"], case["max_len"], s["score"],
                          q_off=s["q_off"], max_rows=case["rows"], decay=case["decay"], softcap=case["softcap"],
                          window=case["window"], slopes=s["slopes"])
        return s["score"]
    ddl.ddl_kv8_evict(pool, s["score"], s["kv_len"], s["keep_len"], s["page_table"], s["new_table"], case["max_len"],
                      kept=s["kept"], score_out=s["score_out"], sinks=case["sinks"], recent=case["recent"])
    return [s["k"], s["k_scale"], s["v"], s["v_scale"], s["kept"], s["score_out"]]


def run(s):
    if own:
        return _run_own(s)
    return {"score": _score_plain, "evict": _evict_plain, "sample": _sample_plain}[s["case"]["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "f32" else 2
        # a difference, a product, an exponential and a sum for each logit
        return {"bytes": float(case["B"] * (case["V"] * size + 5 * 4 + 8)), "flops": 4.0 * case["B"] * case["V"]}
    total, second = _lengths(case)
    R, P, H, hd = case["R"], case["page"], case["H_kv"], case["hd"]
    if case["op"] == "evict":
        cut = second < total
        n = second[cut]
        blocks = int((-(-n // BLOCK)).sum())
        # scores in; codes in and out with their scales (at least as many blocks in); indices out, scores out
        moved = int(n.sum()) * H * (2 * 2 * hd + 4) + blocks * H * 2 * 2 * 4
        return {"bytes": float(int(total.sum()) * H * 4 + moved + int(second.sum()) * H * 4
                               + 4 * (2 * R + int((-(-total // P)).sum()) + int((-(-n // P)).sum()))), "flops": 0.0}
    size = 4 if case["dtype"] == "f32" else 2
    old, T = total - second, int(second.sum())
    lo = np.maximum(0, old - case["window"] + 1) if case["window"] else np.zeros_like(old)
    keys = total - lo
    pairs = 0.0
    for o, n in zip(old.tolist(), second.tolist()):
        seen = np.arange(o + 1, o + n + 1)
        pairs += float((np.minimum(seen, case["window"]) if case["window"] else seen).sum())
    blocks = -(-total // BLOCK) - lo // BLOCK
    touched = total if case["decay"] != 1.0 else keys  # scores that change
    read = int(keys.sum()) * H * hd + int(blocks.sum()) * H * 4 + int((-(-total // P) - lo // P).sum()) * 4
    return {"bytes": float(read + T * case["H_q"] * (hd * size + 4) + int(touched.sum()) * H * 8 + 4 * R),
            "flops": 2.0 * pairs * case["H_q"] * hd}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_score(case, s):
    total, add = _lengths(case)
    table = s["page_table"].cpu().numpy()
    out = s["score"].double()
    at = 0
    for r in range(case["R"]):
        L, n = int(total[r]), int(add[r])
        lse = s["lse"][at:at + n].double().view(n, case["H_kv"], -1).permute(1, 2, 0)[..., None]
        p = torch.exp(_scores_64(case, s, table[r], L, n, at) - lse).sum((1, 2))
        out[r, :, :L - n] *= case["decay"]
        out[r, :, L - n:L] = 0
        out[r, :, :L] += p
        at += n
    return out


def _nearest_e4m3(x):
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6)
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, torch.where(torch.exp2(e) > a, (e - 1).clamp(min=-6), e))
    step = torch.exp2(e - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_evict(case, s):
    H, P, keep, int8 = case["H_kv"], case["page"], case["keep"], case["codes"] == "int8"
    total, _ = _lengths(case)
    src, dst = s["page_table"].cpu().numpy(), s["new_table"].cpu().numpy()
    score = s["score"].cpu().numpy()
    kept, score_out = s["kept"].cpu().numpy(), s["score_out"].cpu().numpy().astype(np.float64)
    pools = {n: (s[n].double() if not int8 else s[n].clone(), s[n + "_scale"].double()) for n in ("k", "v")}
    top = 127.0 if int8 else 448.0
    for r in range(case["R"]):
        L = int(total[r])
        if L <= keep:
            score_out[r, :, :L] = score[r, :, :L]
            continue
        recent = min(case["recent"], keep)
        sinks = min(case["sinks"], keep - recent)
        for h in range(H):
            middle = np.arange(sinks, L - recent)
            best = middle[np.lexsort((middle, -score[r, h, middle].astype(np.float64)))][:keep - sinks - recent]
            t = np.concatenate([np.arange(sinks), np.sort(best), np.arange(L - recent, L)])
            kept[r, h] = t
            score_out[r, h, :keep] = score[r, h, t]
            at = torch.from_numpy(src[r, t // P].astype(np.int64) * P + t % P).cuda()
            to = torch.from_numpy(dst[r, np.arange(0, keep, BLOCK) // P].astype(np.int64)).cuda()
            sub = torch.arange(0, keep, BLOCK, device="cuda") % P // BLOCK
            for name in ("k", "v"):
                pool, scale = pools[name]
                x = s[name].view(torch.uint8)[at // P, h, at % P].view(s[name].dtype).double()
                x = x * s[name + "_scale"].double()[at // P, h, at % P // BLOCK][:, None]
                x = torch.cat([x, x.new_zeros(-keep % BLOCK, x.shape[1])]).view(-1, BLOCK, x.shape[1])
                amax = x.abs().amax((1, 2))
                now = torch.exp2(torch.ceil(torch.log2(amax / top)))
                now = torch.where(top * now < amax, 2 * now, torch.where(top / 2 * now >= amax, now / 2, now))
                y = x / now[:, None, None]
                y = torch.round(y).to(torch.int8) if int8 else _nearest_e4m3(y)
                pool.view(pool.shape[0], H, P // BLOCK, BLOCK, -1)[to, h, sub] = y
                scale[to, h, sub] = now
    return [*pools["k"], *pools["v"], kept, score_out]


def _exact_sample(case, s):
    x = s["logits"].double().cpu().numpy()
    u, t, k, p, m = (s[n].cpu().numpy().astype(np.float64) for n in ("u", "temperature", "top_k", "top_p", "min_p"))
    B, V = x.shape
    tokens, logp = np.zeros(B, np.int32), np.zeros(B)
    for b in range(B):
        if not t[b] > 0:
            tokens[b] = np.argmax(x[b])
            continue
        ids = np.argsort(-x[b], kind="stable")
        ids = ids[np.isfinite(x[b, ids])]
        if 0 < k[b] < len(ids):
            ids = ids[:int(k[b])]
        w = np.exp((x[b, ids] - x[b, ids[0]]) / t[b])
        ahead = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        stay = w >= m[b]
        if p[b] < 1:
            stay &= ahead < p[b] * w.sum()
        stay[0] = True
        n = len(ids) if stay.all() else int(np.argmin(stay))  # both filters keep the largest ones
        ids, w = ids[:n], w[:n]
        by_id = np.argsort(ids)
        c = np.cumsum(w[by_id])
        i = by_id[min(n - 1, int(np.searchsorted(c, u[b] * c[-1], side="right")))]
        tokens[b], logp[b] = ids[i], math.log(w[i] / w.sum())
    return tokens, logp


def exact(case, seed):
    s = prepare(case, seed)
    return {"score": _exact_score, "evict": _exact_evict, "sample": _exact_sample}[case["op"]](case, s)
