"""64-bit references of the 8-bit paged cache's operators, written from their
definitions in ddl.h: the page plan and the quantizing append in numpy, the
attention in torch float64 with a bound on what fp32 arithmetic may lose.
"""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 16
E4M3 = np.array([(-1.0) ** (c >> 7) * ((c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0
                                       else (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7))
                 if c & 127 != 127 else np.nan for c in range(256)])
_POS = E4M3[:127]  # 0 .. 448, increasing


def encode_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even code, saturating; NaN 0x7F."""
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(a), 0.0, a)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(_POS[hi] == a, hi, code)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def encode_int8(x: np.ndarray) -> np.ndarray:
    c = np.rint(np.clip(np.where(np.isnan(x), 0.0, x), -127, 127))
    return c.astype(np.int8).view(np.uint8)


def decode(codes: np.ndarray, int8: bool) -> np.ndarray:
    return codes.view(np.int8).astype(np.float64) if int8 else E4M3[codes]


def plan(old, add, free, table, page, T):
    """(table, row_off, kv_len, row_pos, slot, used, status), one request after the other."""
    R, per = table.shape
    table = table.copy()
    status, kv_len, row_off = np.zeros(R, int), np.zeros(R, int), np.zeros(R + 1, int)
    pos, slot = np.full(T, -1), np.full(T, -1)
    sum_need = sum_add = used = rows = 0
    for r in range(R):
        o, a = int(old[r]), int(add[r])
        ok = o >= 0 and a >= 0 and o + a <= per * page
        need = -(-(o + a) // page) - -(-o // page) if ok else 0
        if ok:
            sum_need += need
            sum_add += a
        if not ok:
            status[r] = 1
        elif need > 0 and sum_need > len(free):
            status[r] = 2
        elif a > 0 and sum_add > T:
            status[r] = 3
        kv_len[r] = min(max(o, 0), per * page)
        row_off[r] = rows
        if status[r] == 0:
            kv_len[r] = o + a
            held = -(-o // page)
            table[r, held:held + need] = free[used:used + need]
            used += need
            for i in range(a):
                p = o + i
                pos[rows + i] = p
                slot[rows + i] = table[r, p // page] * page + p % page
            rows += a
    row_off[R] = rows
    return table, row_off, kv_len, pos, slot, np.array([used]), status


def append(codes, scale, x, slot, page, int8):
    """codes [pages, H, page, hd] uint8 and scale [pages, H, page / 16] after
    storing rows x [T, H, hd] (float64) at slot [T]."""
    codes, scale = codes.copy(), scale.astype(np.float64).copy()
    top = 127.0 if int8 else 448.0
    enc = encode_int8 if int8 else encode_e4m3
    total = codes.shape[0] * page
    i = 0
    while i < len(slot):
        s = int(slot[i])
        if s < 0 or s >= total:
            i += 1
            continue
        j = i
        while j < len(slot) and slot[j] >= 0 and slot[j] // BLOCK == s // BLOCK:
            j += 1
        pg, sub = s // page, s % page // BLOCK
        offs = np.asarray(slot[i:j]) % BLOCK
        low = int(offs.min())
        rows = codes[pg, :, sub * BLOCK:(sub + 1) * BLOCK]
        for h in range(codes.shape[1]):
            a = np.abs(x[i:j, h])
            a = a[np.isfinite(a)]
            amax = a.max() if a.size else 0.0
            fresh = 0.0
            if amax > 0:
                e = math.frexp(amax / top)[1]
                while 2.0 ** (e - 1) * top >= amax:
                    e -= 1
                while 2.0 ** e * top < amax:
                    e += 1
                fresh = 2.0 ** max(e, -126)
            was = scale[pg, h, sub] if low > 0 else 0.0
            now = max(was, fresh)
            if low > 0 and now != was:
                rows[h, :low] = enc(decode(rows[h, :low], int8) * (was / now))
            for k in range(i, j):
                with np.errstate(invalid="ignore"):
                    rows[h, slot[k] % BLOCK] = enc(x[k, h] / now if now > 0 else x[k, h])
            scale[pg, h, sub] = now
        i = j
    return codes, scale


def gather(codes: torch.Tensor, scale: torch.Tensor, ids, n: int) -> torch.Tensor:
    """The first n rows of the pages `ids` as values: [H, n, hd] float64."""
    ids = torch.as_tensor(ids, device=codes.device, dtype=torch.long)
    x = codes.view(torch.uint8)[ids].view(codes.dtype).double()        # [p, H, P, hd]
    f = scale[ids].double().repeat_interleave(BLOCK, -1)[..., None]
    x = (x * f).transpose(0, 1)
    return x.reshape(x.shape[0], -1, x.shape[-1])[:, :n]


def attention(pool, q, q_off, kv_len, table, scale, softcap=0.0, window=0, slopes=None):
    """(out, lse, tol_out, tol_lse) in float64 for q [T, H_q, hd]: the
    definition, and a bound on |error| of an fp32 evaluation whose products,
    exponentials and sums each lose at most a few fp32 roundings.  Rows of no
    request are NaN.

    With weights w_j = p_j / sum p, an error d_j of score j moves out by at
    most sum w_j d_j (|v_j| + |out|) (first order; d << 1).  d_j: hd products
    added in fp32, each addition within 2^-23 of the partial sum of
    magnitudes (tensor cores truncate), q held to 2^-21; the score's scaling,
    cap (tanh from exp within 2^-21 of the cap) and bias rounded in fp32; e^s
    within 2^-21 and the running maximum's rescaling within another 2^-21.
    The weights are rounded to at least 2^-11 of themselves for 16-bit outputs,
    2^-21 for fp32 ones, but no finer than an absolute F = 2^-23 (fp32: 2^-27)
    of the largest weight, in units of the largest V scale: that is half the
    smallest e4m3 step, 2^-10, over the weights' scale 2^5 and the last limbs'
    2^8 (2^12).  Such a weight p_j changes by at most min(p_j, F vmax / vs_j).
    (p_j relative to the running maximum: at most twice that to the true one;
    the sum of weights is at least 1.)  The sums over n keys are within n 2^-23
    of their magnitudes, and the output once to its type: half a step, eps / 2 of the
    value, or of the smallest normal number where the value lies below it
    (the steps stop shrinking there: fp16's are 2^-24)."""
    k, v, ks, vs = pool
    T, H_q, hd = q.shape
    H = k.shape[1]
    G = H_q // H
    dev = q.device
    out = torch.full((T, H_q, hd), math.nan, dtype=torch.float64, device=dev)
    lse = torch.full((T, H_q), math.nan, dtype=torch.float64, device=dev)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    p_round = 2.0 ** -21 if q.dtype == torch.float32 else 2.0 ** -11
    floor = 2.0 ** -27 if q.dtype == torch.float32 else 2.0 ** -23
    eps = torch.finfo(q.dtype).eps / 2
    P = k.shape[2]
    table = np.asarray(table)
    for r in range(len(kv_len)):
        a, b = int(q_off[r]), int(q_off[r + 1])
        n, L = b - a, int(kv_len[r])
        if n <= 0:
            continue
        if L <= 0:
            out[a:b], lse[a:b] = 0, -math.inf
            continue
        ids = table[r, :-(-L // P)].tolist()
        kk, vv = gather(k, ks, ids, L), gather(v, vs, ids, L)
        qq = q[a:b].double().view(n, H, G, hd).permute(1, 2, 0, 3)
        s = torch.einsum("hgnd,hkd->hgnk", qq, kk) * scale
        mag = torch.einsum("hgnd,hkd->hgnk", qq.abs(), kk.abs()) * abs(scale)
        d = mag * (hd * 2.0 ** -23 + 2.0 ** -21) + s.abs() * 2.0 ** -21
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            d = d + softcap * 2.0 ** -20
        dist = torch.arange(L - n, L, device=dev)[:, None] - torch.arange(L, device=dev)
        if slopes is not None:
            bias = slopes.double().view(H, G, 1, 1) * dist
            s = s - bias
            d = d + bias.abs() * 2.0 ** -21 + s.abs() * 2.0 ** -21
        d = d + 2.0 ** -20
        seen = dist >= 0
        if window:
            seen = seen & (dist < window)
        s = s.masked_fill(~seen, -math.inf)
        none = ~seen.any(-1)
        top = s.amax(-1, keepdim=True)
        w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
        top_w = w
        l = w.sum(-1, keepdim=True)
        w = w / torch.where(l == 0, 1.0, l)
        o = torch.einsum("hgnk,hkd->hgnd", w, vv)
        A = torch.einsum("hgnk,hkd->hgnd", w, vv.abs())
        wd = w * torch.where(seen, d, 0.0)
        E = torch.einsum("hgnk,hkd->hgnd", wd, vv.abs()) + o.abs() * wd.sum(-1, keepdim=True)
        sv = vs[torch.as_tensor(ids, device=dev)].double().transpose(0, 1)
        sv = sv.reshape(H, -1).repeat_interleave(BLOCK, -1)[:, :L]
        tiny = floor * sv.amax(-1, keepdim=True) / sv.clamp(min=1e-300)
        least = torch.minimum(2 * top_w, tiny[:, None, None, :])
        E = E + A * (p_round + (L + 64) * 2.0 ** -23) + torch.einsum("hgnk,hkd->hgnd", least, vv.abs())
        ll = (top + torch.log(l))[..., 0]
        dl = wd.sum(-1) + (L + 64) * 2.0 ** -23 + ll.abs().nan_to_num(posinf=0.0) * 2.0 ** -21 + 2.0 ** -21
        o = torch.where(none[:, None], 0.0, o) if none.ndim == 1 else o
        back = lambda x: x.permute(2, 0, 1, 3).reshape(n, H_q, hd)  # noqa: E731
        out[a:b] = back(o)
        tol[a:b] = back(E * (1 + eps) + eps * o.abs().clamp(min=torch.finfo(q.dtype).smallest_normal) + 1e-30)
        lse[a:b] = ll.permute(2, 0, 1).reshape(n, H_q)
        tol_l[a:b] = dl.permute(2, 0, 1).reshape(n, H_q)
        if none.any():
            rows = torch.nonzero(none)[:, 0] + a
            out[rows], lse[rows] = 0, -math.inf
            tol[rows], tol_l[rows] = 0, 0
    return out, lse, tol, tol_l
