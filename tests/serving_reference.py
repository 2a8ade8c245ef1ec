"""64-bit references of the cache scores, the eviction by them and the draw of
the next tokens, written from their definitions in ddl.h.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import kv8_reference as ref

BLOCK = 16


def score(pool, q, lse, q_off, kv_len, table, old, decay, scale, softcap=0.0, window=0, slopes=None):
    """(score, tolerance) in float64, both [R, H, S], after the step.

    A weight is exp(s - lse): an error d of s - lse moves it by at most w (e^d - 1).
    d: hd products added in fp32, each addition within 2^-23 of the partial sum
    of magnitudes (tensor cores truncate); q of fp32 rows held to 2^-22 of an
    element; elements of q held no finer than 2^-25 of the row's largest (fp32
    2^-29); the score's factor, cap, bias and the difference with lse rounded in
    fp32 (2^-24 of each, three roundings: 2^-22 of |s|, |lse| and the bias; the cap's
    tanh 2^-21 of the cap); e^x within 2^-21.  The sum of N weights is within
    N 2^-24 of itself, decay * old + sum adds two roundings."""
    k, _, ks, _ = pool
    T, H_q, hd = q.shape
    H, P = k.shape[1], k.shape[2]
    G = H_q // H
    dev = q.device
    out, tol = old.double().clone(), torch.zeros_like(old, dtype=torch.float64)
    table = np.asarray(table)
    fine = 2.0 ** -29 if q.dtype == torch.float32 else 2.0 ** -25
    for r in range(len(kv_len)):
        a, b = int(q_off[r]), int(q_off[r + 1])
        n, L = b - a, int(kv_len[r])
        if n <= 0 or L <= 0:
            continue
        kk = ref.gather(k, ks, table[r, :-(-L // P)].tolist(), L)
        qq = q[a:b].double().view(n, H, G, hd).permute(1, 2, 0, 3)
        s = torch.einsum("hgnd,hkd->hgnk", qq, kk) * scale
        mag = torch.einsum("hgnd,hkd->hgnk", qq.abs(), kk.abs()) * abs(scale)
        least = qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)[:, None, None] * abs(scale) * fine
        d = mag * (hd * 2.0 ** -23 + 2.0 ** -22) + least + s.abs() * 2.0 ** -22
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            d = d + softcap * 2.0 ** -21 + s.abs() * 2.0 ** -22
        dist = torch.arange(L - n, L, device=dev)[:, None] - torch.arange(L, device=dev)
        if slopes is not None:
            bias = slopes.double().view(H, G, 1, 1) * dist
            s = s - bias
            d = d + (bias.abs() + s.abs()) * 2.0 ** -22
        ll = lse[a:b].double().view(n, H, G).permute(1, 2, 0)[..., None]
        d = d + ll.abs().nan_to_num(posinf=0.0) * 2.0 ** -22 + 2.0 ** -21
        seen = dist >= 0
        if window:
            seen = seen & (dist < window)
        w = torch.where(seen & (ll != -math.inf), torch.exp(s - ll), 0.0)
        e = torch.where(seen, w * torch.expm1(d), 0.0)
        total = w.sum((1, 2))
        was = old[r, :, :L].double() * decay if decay else torch.zeros_like(total)
        was[:, max(0, L - n):] = 0
        out[r, :, :L] = was + total
        tol[r, :, :L] = e.sum((1, 2)) + total * (n * G * 2.0 ** -24) + (was.abs() + total) * 2.0 ** -22 + 1e-37
    return out, tol


def evict(codes, scales, score, kv_len, keep_len, table, new_table, sinks, recent, page, int8, kept, score_out):
    """codes: (k, v) uint8 [pages, H, page, hd], scales: (k, v) float64; everything after the call."""
    codes, scales = [c.copy() for c in codes], [s.copy() for s in scales]
    src_c, src_s = [c.copy() for c in codes], [s.copy() for s in scales]
    kept, score_out = kept.copy(), score_out.copy()
    top = 127.0 if int8 else 448.0
    enc = ref.encode_int8 if int8 else ref.encode_e4m3
    for r in range(len(kv_len)):
        L, keep = int(kv_len[r]), int(keep_len[r])
        if keep < 0 or keep >= L:
            score_out[r, :, :L] = score[r, :, :L]
            continue
        rc = min(recent, keep)
        sc = min(sinks, keep - rc)
        for h in range(score.shape[1]):
            mid = list(range(sc, L - rc))
            s = score[r, h]
            key = lambda i: (0 if s[i] == s[i] else 1, -s[i] if s[i] == s[i] else 0.0, i)  # noqa: E731
            best = sorted(mid, key=key)[:keep - rc - sc]
            t = np.array(sorted(list(range(sc)) + best + list(range(L - rc, L))), dtype=int)
            kept[r, h, :keep] = t
            score_out[r, h, :keep] = s[t]
            for b in range(-(-keep // BLOCK)):
                tt = t[b * BLOCK:(b + 1) * BLOCK]
                pg, sub = new_table[r, b * BLOCK // page], b * BLOCK % page // BLOCK
                if pg < 0 or pg >= codes[0].shape[0]:
                    continue
                for i in range(2):
                    x = np.zeros((BLOCK, codes[i].shape[-1]))
                    raw = np.zeros((BLOCK, codes[i].shape[-1]), np.uint8)
                    f = np.zeros(BLOCK)
                    for j, tok in enumerate(tt):
                        p = table[r, tok // page]
                        if 0 <= p < codes[i].shape[0]:
                            raw[j] = src_c[i][p, h, tok % page]
                            f[j] = src_s[i][p, h, tok % page // BLOCK]
                    with np.errstate(invalid="ignore", over="ignore"):
                        x = (ref.decode(raw, int8) * f[:, None]).astype(np.float32).astype(np.float64)
                    if not np.all((f >= 0) & np.isfinite(f)):
                        scales[i][pg, h, sub] = np.nan
                        codes[i][pg, h, sub * BLOCK:(sub + 1) * BLOCK] = 0  # (no defined content)
                        continue
                    a = np.abs(x)
                    a = a[~np.isnan(a)]
                    amax = a.max() if a.size else 0.0
                    now = 0.0
                    if amax > 0:
                        e = math.frexp(amax / top)[1]
                        while 2.0 ** (e - 1) * top >= amax:
                            e -= 1
                        while 2.0 ** e * top < amax:
                            e += 1
                        now = 2.0 ** max(e, -126)
                    with np.errstate(invalid="ignore"):
                        new = enc(x / now if now else x)
                    same = (f == now)[:, None]
                    codes[i][pg, h, sub * BLOCK:(sub + 1) * BLOCK] = np.where(same, raw, new)
                    scales[i][pg, h, sub] = now
    return codes, scales, kept, score_out


def draw(x, t, k, p, m, u):
    """{token: its possible logp} over the tokens that a draw within the stated precision may give, for one row of
    logits in float64.

    Weights are held to 2^-33 of themselves and 2^-43 of the largest, so borders of
    their sums lie within 2^-32 of the exact ones: a border (top-p's, the draw's) nearer
    than that to its number may fall on either side."""
    live = np.flatnonzero(~np.isnan(x) & (x > -np.inf))
    if live.size == 0:
        return {-1: {-math.inf}}
    top = x[live].max()
    if not t >= 2.0 ** -60:
        i = int(live[np.argmax(x[live])])
        return {i: {0.0}}
    order = live[np.lexsort((live, -x[live]))]
    if 0 < k < len(order):
        order = order[:k]
    with np.errstate(invalid="ignore"):
        w = np.where(x[order] == top, 1.0, np.exp((x[order] - top) / t))
    w = np.nan_to_num(w, nan=0.0)
    ahead = np.concatenate([[0.0], np.cumsum(w)[:-1]])
    total = w.sum()
    tokens = {}
    u = min(max(u if u == u else 0.0, 0.0), 1 - 2.0 ** -24)
    d = 2.0 ** -32
    sizes = set()
    for pp in (p - d, p, p + d) if p < 1 else (p,):
        stay = np.ones(len(order), bool)
        if m > 0:
            stay &= w >= m
        if p < 1:
            stay &= ahead < pp * total
        stay[0] = True
        sizes.add(len(stay) if stay.all() else int(np.argmin(stay)))
    for n in sizes:
        ids = np.argsort(order[:n])
        c = np.cumsum(w[:n][ids])
        for uu in (u - d, u, u + d):
            i = min(n - 1, int(np.searchsorted(c, max(uu, 0.0) * c[-1], side="right")))
            tok = int(order[ids[i]])
            with np.errstate(divide="ignore"):
                tokens.setdefault(tok, set()).add(float(np.log(w[ids[i]] / c[-1])))
    return tokens
