"""The 8-bit paged KV cache's operators as measured cases.

Three operators that a serving step runs one after the other:

* ``plan``   -- page tables, row positions and slot maps of a step, built on
  the GPU from the requests' lengths (``ddl_page_plan``);
* ``append`` -- new K/V rows quantized into the paged 8-bit cache, one
  power-of-two scale per 16 tokens and head (``ddl_kv8_append``);
* ``attn``   -- attention of each request's newest rows over that cache
  (``ddl_kv8_attention``), with capped scores, a distance bias and a window.

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
        # One decode step of a full batch: every request gets one token; latency counts.
        {"name": "plan decode b64", "op": "plan", "R": 64, "page": 64, "max_len": 4096, "max_add": 1, "T": 64},
        # A step that mixes decoding requests with prompt chunks, idle requests among them.
        {"name": "plan mixed r1000", "op": "plan", "R": 1000, "page": 16, "max_len": 8192, "max_add": 128, "T": 65536},
        # One token of one sequence of the 27B-class stack's layer: the smallest append.
        {"name": "append b1", "op": "append", "R": 1, "rows": 1, "H_kv": 8, "hd": 128, "page": 64, "max_len": 8192,
         "dtype": "bf16"},
        # One token of each of 64 sequences at their own places inside a block.
        {"name": "append b64", "op": "append", "R": 64, "rows": 1, "H_kv": 8, "hd": 128, "page": 64, "max_len": 4096,
         "dtype": "bf16"},
        # Prompt chunks of several sequences, odd lengths.
        {"name": "append prompt", "op": "append", "R": 5, "rows": 1633, "H_kv": 4, "hd": 128, "page": 16,
         "max_len": 4096, "dtype": "f32"},
        # The small layer at batch 1: the smallest attention call.
        {"name": "attn small b1", "op": "attn", "R": 1, "rows": 1, "H_q": 8, "H_kv": 2, "hd": 64, "page": 16,
         "max_len": 129, "codes": "e4m3", "dtype": "bf16", "softcap": 0.0, "window": 0, "slopes": False},
        # Batch 1 of the 27B-class layer, cache 8192: the long axis has to be split.
        {"name": "attn b1 8k", "op": "attn", "R": 1, "rows": 1, "H_q": 64, "H_kv": 8, "hd": 128, "page": 64,
         "max_len": 8193, "codes": "e4m3", "dtype": "f32", "softcap": 0.0, "window": 0, "slopes": False},
        # Batch 1 of a 70B-class layer, cache 32768, 8-bit integers.
        {"name": "attn b1 32k int8", "op": "attn", "R": 1, "rows": 1, "H_q": 64, "H_kv": 8, "hd": 128, "page": 256,
         "max_len": 32769, "codes": "int8", "dtype": "bf16", "softcap": 0.0, "window": 0, "slopes": False},
        # A full batch at ragged lengths up to 8192: the ordinary serving step, memory-bound.
        {"name": "attn b64 8k", "op": "attn", "R": 64, "rows": 1, "H_q": 64, "H_kv": 8, "hd": 128, "page": 64,
         "max_len": 8192, "codes": "e4m3", "dtype": "bf16", "softcap": 0.0, "window": 0, "slopes": False},
        # Groups of 7 heads, capped scores and a sliding window over longer caches.
        {"name": "attn b16 capped window", "op": "attn", "R": 16, "rows": 1, "H_q": 28, "H_kv": 4, "hd": 128,
         "page": 32, "max_len": 4097, "codes": "int8", "dtype": "f16", "softcap": 30.0, "window": 2049,
         "slopes": False},
        # Checking 4 drafted tokens of each of 16 sequences, distance bias.
        {"name": "attn verify 4 rows", "op": "attn", "R": 16, "rows": 4, "H_q": 64, "H_kv": 8, "hd": 128, "page": 64,
         "max_len": 4096, "codes": "e4m3", "dtype": "bf16", "softcap": 0.0, "window": 0, "slopes": True},
        # A prompt chunk of 64 rows on an 8192-token cache: compute counts here.
        {"name": "attn chunk 64 rows", "op": "attn", "R": 1, "rows": 64, "H_q": 64, "H_kv": 8, "hd": 128, "page": 64,
         "max_len": 8192, "codes": "e4m3", "dtype": "bf16", "softcap": 0.0, "window": 0, "slopes": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 256])
    if op == "plan":
        R, add = _log(rng, 1, 2000), _log(rng, 1, 300)
        T = min(131072, R * add)
        return {"op": op, "R": R, "page": page, "max_len": _log(rng, 1, 16384), "max_add": add, "T": T}
    if op == "append":
        R = _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, 8165 // R))
        return {"op": op, "R": R, "rows": rows, "H_kv": rng.choice([1, 2, 4, 8]), "hd": rng.choice([64, 128]),
                "page": page, "max_len": rows + _log(rng, 1, 8192), "dtype": rng.choice(["bf16", "f16", "f32"])}
    R, rows = _log(rng, 1, 64), rng.choice([1, 1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 64)])
    H_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    most = min(32769, 64 * 8192 // (R * max(1, rows // 2)))
    max_len = _log(rng, rows, max(rows, most))
    return {"op": op, "R": R, "rows": rows, "H_q": H_kv * group, "H_kv": H_kv, "hd": rng.choice([64, 128]),
            "page": page, "max_len": max_len, "codes": rng.choice(["e4m3", "int8"]),
            "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]),
            "window": rng.choice([0, 0, 1 + max_len // 3]), "slopes": rng.choice([False, False, True])}


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Per request: tokens in the cache before the step and rows that the step adds (host arrays of the case alone:
    the work and the plain form's sizes follow from them, whatever the seed)."""
    g = np.random.RandomState(1234)
    R, most = case["R"], case["max_len"]
    if case["op"] == "plan":
        add = g.randint(0 if R > 1 and case["max_add"] > 1 else 1, case["max_add"] + 1, R)
        old = g.randint(0, most + 1, R)
        old[g.rand(R) < 0.1] = 0
        over = np.cumsum(add) > case["T"]
        add[over] = 0
        return old.astype(np.int64), add.astype(np.int64)
    rows = case["rows"]
    add = np.full(R, rows)
    if R > 1 and rows > 1:
        add[1:] = g.randint(1, rows + 1, R - 1)
    total = add + (g.rand(R) * (most - add + 1)).astype(np.int64)
    total[0] = most
    return (total - add).astype(np.int64), add.astype(np.int64)


def _pages(case, total, rng):
    """A page table [R][pages_per_seq] of distinct pages in random order, and the pool's page count."""
    P = case["page"]
    need = -(-total // P)
    per = max(1, int(need.max()) + 1)
    pages = int(need.sum()) + 3
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((case["R"], per), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, pages


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    rng = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device="cuda").manual_seed(seed)
    old, add = _lengths(case)
    P, R = case["page"], case["R"]
    total = old + add
    s = {"case": case}
    if case["op"] == "plan":
        held = -(-old // P)
        per = int((-(-total // P)).max()) + 2
        need = int((-(-total // P) - held).sum())
        pages = int(held.sum()) + need + 5
        ids = rng.permutation(pages).astype(np.int32)
        table = np.full((R, per), -1, np.int32)
        table[np.arange(per)[None, :] < held[:, None]] = ids[:int(held.sum())]
        s["old_len"], s["add_len"] = _dev(old), _dev(add)
        s["page_table"] = _dev(table)
        # the last requests find no page left, where there are several
        s["free_pages"] = _dev(ids[int(held.sum()):][:need if R < 8 else max(1, int(0.97 * need))])
        T = case["T"]
        for name, n in (("row_off", R + 1), ("kv_len", R), ("row_pos", T), ("slot", T), ("used", 1), ("status", R)):
            s[name] = torch.zeros(n, dtype=torch.int32, device="cuda")
        return s
    table, pages = _pages(case, total, rng)
    H, hd = case["H_kv"], case["hd"]
    codes = CODES[case.get("codes", "e4m3")]
    # what quantized rows of about N(0, 1) look like: codes spread over the type's range, scales near 2^-7 (e4m3)
    # or 2^-5 (int8), differing by head and block
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
    s["page_table"], s["kv_len"] = _dev(table), _dev(total)
    T = int(add.sum())
    if case["op"] == "append":
        seq = np.repeat(np.arange(R), add)
        pos = np.concatenate([np.arange(o, t) for o, t in zip(old, total)])
        s["slot"] = _dev(table[seq, pos // P].astype(np.int64) * P + pos % P)
        # rows of one projection's output: k and v lie side by side, heads of different magnitude
        mag = torch.exp2(torch.randint(-2, 3, (1, 2 * H, 1), generator=g, device="cuda").float())
        kv = (torch.randn((T, 2 * H, hd), generator=g, device="cuda") * mag).to(DTYPES[case["dtype"]])
        s["k_new"], s["v_new"] = kv[:, :H], kv[:, H:]
        return s
    s["q"] = torch.randn((T, case["H_q"], hd), generator=g, device="cuda").to(DTYPES[case["dtype"]])
    s["out"] = torch.zeros_like(s["q"])
    s["q_off"] = None if case["rows"] == 1 else _dev(np.concatenate([[0], np.cumsum(add)]))
    s["slopes"] = None
    if case["slopes"]:  # one slope per head, a geometric sequence
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["H_q"] + 1, device="cuda").float() / case["H_q"])
    return s


# ------------------------------------------------------------------ the operators

def _plan_plain(s):
    P, T = s["case"]["page"], s["case"]["T"]
    old, add, table, free = s["old_len"].long(), s["add_len"].long(), s["page_table"], s["free_pages"]
    R, per = table.shape
    held, total = (old + P - 1) // P, old + add
    fits = (old >= 0) & (add >= 0) & (total <= per * P)
    need = torch.where(fits, (total + P - 1) // P - held, 0)
    rows = torch.where(fits, add, 0)
    no_page = fits & (need > 0) & (need.cumsum(0) > free.numel())
    no_row = fits & ~no_page & (rows > 0) & (rows.cumsum(0) > T)
    ok = fits & ~no_page & ~no_row
    status = torch.where(fits, torch.where(no_page, 2, torch.where(no_row, 3, 0)), 1)
    need, rows = torch.where(ok, need, 0), torch.where(ok, add, 0)
    end_p, end_r = need.cumsum(0), rows.cumsum(0)
    j = torch.arange(per, device=table.device)[None, :]
    at = (end_p - need)[:, None] + j - held[:, None]
    new = (j >= held[:, None]) & (j < (held + need)[:, None])
    s["page_table"] = table = torch.where(new, free[at.clamp(0, free.numel() - 1)], table)
    i = torch.arange(T, device=table.device)
    live = i < end_r[-1]
    r = torch.searchsorted(end_r, i, right=True).clamp(max=R - 1)
    pos = torch.where(live, old[r] + i - (end_r - rows)[r], -1)
    slot = torch.where(live, table[r, (pos // P).clamp(min=0)] * P + pos % P, -1)
    row_off = torch.cat([end_r.new_zeros(1), end_r])
    kv_len = torch.where(fits, old + rows, old.clamp(min=0).clamp(max=per * P))
    return [x.to(torch.int32) for x in (table, row_off, kv_len, pos, slot, end_p[-1:], status)]


def _blocks(pool):
    pages, H, P, hd = pool.shape
    return pool.view(pages, H, P // BLOCK, BLOCK, hd)


def _append_plain(s):
    slot = s["slot"].long()
    P = s["case"]["page"]
    page, sub, off = slot // P, slot % P // BLOCK, slot % BLOCK
    outs = []
    for name in ("k", "v"):
        pool, scale, x = s[name], s[name + "_scale"], s[name + "_new"].float()
        H = x.shape[1]
        heads = torch.arange(H, device=x.device)[None, :]
        block = slot // BLOCK  # of the pool's 16-token blocks
        n_blocks = pool.shape[0] * (P // BLOCK)
        first = torch.full((n_blocks,), BLOCK, device=x.device, dtype=off.dtype).scatter_reduce(0, block, off, "amin")
        amax = torch.zeros((n_blocks, H), device=x.device)
        amax = amax.scatter_reduce(0, block[:, None].expand(-1, H), x.abs().amax(-1), "amax")[block]
        # the smallest power of two with amax / scale <= 448 = 0.875 * 2^9
        m, e = torch.frexp(amax)
        e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
        fresh = torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), 0.0)
        held = (first[block] > 0)[:, None]
        was = torch.where(held, scale[page[:, None], heads, sub[:, None]], 0.0)
        now = torch.maximum(was, fresh)
        ratio = torch.where(now > 0, was / now, 0.0)
        view = _blocks(pool.view(torch.uint8))
        at = (page[:, None], heads, sub[:, None])
        old = view[at].view(torch.float8_e4m3fn).float() * ratio[..., None, None]
        old = old.to(torch.float8_e4m3fn).view(torch.uint8)
        kept = (torch.arange(BLOCK, device=x.device)[None, :] < first[block][:, None])[:, None, :, None]
        view[at] = torch.where(kept, old, view[at])
        code = torch.where(now[..., None] > 0, x / now[..., None], 0.0).clamp(-448, 448).to(torch.float8_e4m3fn)
        view[page[:, None], heads, sub[:, None], off[:, None]] = code.view(torch.uint8)
        scale[at] = now
        outs += [pool, scale]
    return outs


def _gathered(s, name, dtype):
    """Every request's rows of a pool as values: [R][H_kv][max_len][hd]."""
    case, pool, scale = s["case"], s[name], s[name + "_scale"]
    P, L = case["page"], case["max_len"]
    n = -(-L // P)
    ids = s["page_table"][:, :n].long().clamp(min=0)
    x = pool.view(torch.uint8)[ids].view(pool.dtype).to(dtype)
    x = x * scale[ids].to(dtype).repeat_interleave(BLOCK, -1)[..., None]
    R, n, H, P, hd = x.shape
    return x.transpose(1, 2).reshape(R, H, n * P, hd)[:, :, :L]


def _attn_plain(s):
    case = s["case"]
    R, S, H_q, H, hd, L = case["R"], case["rows"], case["H_q"], case["H_kv"], case["hd"], case["max_len"]
    q, G = s["q"], H_q // H
    dev = q.device
    lens = s["kv_len"].long()
    if s["q_off"] is None:
        start, rows = torch.arange(R, device=dev), torch.ones(R, device=dev, dtype=torch.long)
    else:
        start, rows = s["q_off"][:-1].long(), (s["q_off"][1:] - s["q_off"][:-1]).long()
    i = torch.arange(S, device=dev)[None, :]
    at = (start[:, None] + i).clamp(max=q.shape[0] - 1)
    qp = q[at].float().view(R, S, H, G, hd).permute(0, 2, 3, 1, 4).reshape(R, H, G * S, hd)
    score = (qp @ _gathered(s, "k", torch.float32).transpose(-1, -2)).view(R, H, G, S, L) * (1.0 / math.sqrt(hd))
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    far = (lens - rows)[:, None, None] + i[..., None] - torch.arange(L, device=dev)
    if s["slopes"] is not None:
        score = score - s["slopes"].view(1, H, G, 1, 1) * far[:, None, None].float()
    seen = (far >= 0) & (i < rows[:, None])[..., None]
    if case["window"]:
        seen = seen & (far < case["window"])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    o = p.view(R, H, G * S, L) @ _gathered(s, "v", torch.float32)
    o = o.view(R, H, G, S, hd).permute(0, 3, 1, 2, 4).reshape(R * S, H_q, hd)
    live = (i < rows[:, None]).reshape(-1)
    # rows of a request that has fewer than S are written to a spare last row
    to = torch.where(live, at.reshape(-1), q.shape[0])
    out = torch.empty((q.shape[0] + 1, H_q, hd), device=dev, dtype=q.dtype)
    out[to] = o.to(q.dtype)
    return out[:-1]


def _run_own(s):
    from memory_bound_transformer_decode_gb300 import ddl

    case = s["case"]
    if case["op"] == "plan":
        ddl.ddl_page_plan(s["old_len"], s["add_len"], s["free_pages"], s["page_table"], case["page"],
                          row_off=s["row_off"], kv_len=s["kv_len"], row_pos=s["row_pos"], slot=s["slot"],
                          used=s["used"], status=s["status"])
        return [s[n] for n in ("page_table", "row_off", "kv_len", "row_pos", "slot", "used", "status")]
    pool = (s["k"], s["v"], s["k_scale"], s["v_scale"])
    if case["op"] == "append":
        ddl.ddl_kv8_append(pool, s["k_new"], s["v_new"], s["slot"])
        return [s["k"], s["k_scale"], s["v"], s["v_scale"]]
    if "workspace" not in s:
        n = ddl.ddl_kv8_attention_workspace_bytes(case["H_q"], case["H_kv"], case["hd"], case["R"], s["q"].shape[0],
                                                  case["rows"], case["max_len"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    ddl.ddl_kv8_attention(pool, s["q"], s["kv_len"], s["page_table"], case["max_len"], q_off=s["q_off"],
                          max_rows=case["rows"], softcap=case["softcap"], window=case["window"], slopes=s["slopes"],
                          out=s["out"], workspace=s["workspace"])
    return s["out"]


def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plan_plain, "append": _append_plain, "attn": _attn_plain}[s["case"]["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    old, add = _lengths(case)
    R, P = case["R"], case["page"]
    total, T = old + add, int(add.sum())
    if case["op"] == "plan":
        new = int((-(-total // P) - -(-old // P)).sum())
        # lengths in; offsets, lengths and status out; free pages in, table entries out; the page of each row's first
        # slot in; positions and slots out
        return {"bytes": 4.0 * (2 * R + 3 * R + 2 + 2 * new + R + 2 * case["T"]), "flops": 0.0}
    H, hd = case["H_kv"], case["hd"]
    if case["op"] == "append":
        size = 4 if case["dtype"] == "f32" else 2
        blocks = int((-(-total // BLOCK) - old // BLOCK).sum())
        return {"bytes": float(2 * (T * H * hd * (size + 1) + blocks * H * 8) + 4 * T), "flops": 0.0}
    size = 4 if case["dtype"] == "f32" else 2
    lo = np.maximum(0, old - case["window"] + 1) if case["window"] else np.zeros_like(old)
    keys = total - lo
    pairs = 0.0
    for o, n in zip(old.tolist(), add.tolist()):
        seen = np.arange(o + 1, o + n + 1)
        pairs += float((np.minimum(seen, case["window"]) if case["window"] else seen).sum())
    blocks = -(-total // BLOCK) - lo // BLOCK
    read = int(keys.sum()) * 2 * H * hd + int(blocks.sum()) * 2 * H * 4 + int((-(-total // P) - lo // P).sum()) * 4
    return {"bytes": float(read + 2 * T * case["H_q"] * hd * size + 4 * R),
            "flops": 4.0 * pairs * case["H_q"] * hd}


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3_64(x):
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6)
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, torch.where(torch.exp2(e) > a, (e - 1).clamp(min=-6), e))
    step = torch.exp2(e - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_append(case, s):
    slot = s["slot"].cpu().numpy()
    P = case["page"]
    runs, i = [], 0  # the rows of one block follow one another
    while i < len(slot):
        j = i + 1
        while j < len(slot) and slot[j] // BLOCK == slot[i] // BLOCK:
            j += 1
        runs.append((i, j))
        i = j
    if len(runs) > 4000:
        return None
    outs = []
    for name in ("k", "v"):
        pool, scale, x = s[name].double(), s[name + "_scale"].double(), s[name + "_new"].double()
        for i, j in runs:
            page, sub, off = slot[i] // P, slot[i] % P // BLOCK, slot[i] % BLOCK
            rows = pool[page, :, sub * BLOCK:(sub + 1) * BLOCK]
            amax = x[i:j].abs().amax((0, 2))
            fresh = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
            fresh = torch.where(448.0 * fresh < amax, 2 * fresh, torch.where(224.0 * fresh >= amax, fresh / 2, fresh))
            was = scale[page, :, sub] if off else torch.zeros_like(amax)
            now = torch.maximum(was, fresh)
            rows[:, :off] = _e4m3_64(rows[:, :off] * (was / now)[:, None, None])
            rows[:, off:off + j - i] = _e4m3_64(x[i:j].transpose(0, 1) / now[:, None, None])
            scale[page, :, sub] = now
        outs += [pool, scale]
    return outs


def _exact_attn(case, s):
    R, H_q, H, hd, P = case["R"], case["H_q"], case["H_kv"], case["hd"], case["page"]
    old, add = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for r in range(R):
        L, n = int(old[r] + add[r]), int(add[r])
        ids = s["page_table"][r, :-(-L // P)].long()
        vals = []
        for name in ("k", "v"):
            x = s[name].view(torch.uint8)[ids].view(s[name].dtype).double().transpose(0, 1)
            f = s[name + "_scale"][ids].double().transpose(0, 1)
            x = (x.reshape(H, -1, BLOCK, hd) * f.reshape(H, -1, 1, 1)).reshape(H, -1, hd)[:, :L]
            vals.append(x)
        k, v = vals
        q = s["q"][at:at + n].double().view(n, H, H_q // H, hd).permute(1, 2, 0, 3)
        w = torch.einsum("hgnd,hkd->hgnk", q, k) / math.sqrt(hd)
        if case["softcap"]:
            w = torch.tanh(w / case["softcap"]) * case["softcap"]
        dist = torch.arange(L - n, L, device="cuda")[:, None] - torch.arange(L, device="cuda")[None, :]
        if case["slopes"]:
            w = w - s["slopes"].double().view(H, -1, 1, 1) * dist
        bad = (dist < 0) | (dist >= case["window"]) if case["window"] else dist < 0
        w = torch.softmax(w.masked_fill(bad, -math.inf), -1)
        out[at:at + n] = torch.einsum("hgnk,hkd->nhgd", w, v).reshape(n, H_q, hd)
        at += n
    return out


def exact(case, seed):
    if case["op"] == "plan":  # whole numbers only: they have to be equal
        return None
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attn(case, s)
