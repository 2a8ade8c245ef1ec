"""A bound on the error of the 8-bit cache's attention that takes nothing from
keys a row does not see, and measures the weights' rounding by the row's own
largest product of weight and V scale."""
from __future__ import annotations

import math

import numpy as np
import torch

import kv8_reference as ref

# The weights w_j = p_j vs_j of a row are rounded to 2^-11 (16-bit rows: fp16) or 2^-22 (fp32 rows: two fp16 parts)
# of themselves, but to no finer step than the types reach below the largest of them: fp16's half step 2^-25 over a
# largest weight of 2^5 is 2^-30 for 16-bit rows, over 2^11 2^-36 for fp32 rows. Twice that here (the reference of
# the weights is the largest product so far, up to its own rounding).
FLOOR = {torch.float32: 2.0 ** -35, torch.bfloat16: 2.0 ** -29, torch.float16: 2.0 ** -29}
STEP = {torch.float32: 2.0 ** -22, torch.bfloat16: 2.0 ** -11, torch.float16: 2.0 ** -11}


def attention(pool, q, q_off, lens, table, scale, softcap=0.0, window=0, slopes=None):
    """(out, lse, tol_out, tol_lse) in float64; rows of no request are NaN.

    First order in the errors: with weights w_j = p_j / sum p over the seen keys
    - score j is off by d_j: hd products added in fp32 (each addition within 2^-23 of the magnitudes so far), q held to
      2^-21, the scaling, cap (tanh within 2^-22 of itself) and bias rounded a few times in fp32, e^s within 2^-21, and its argument, s
      less the reference, rounded once: 2^-24 of it. The reference is off the largest score by no more than the
      spread of the V scales seen, in powers of two;
    - w_j is rounded as above, so p_j changes by min(2 p_j, FLOOR max_i(p_i vs_i) / vs_j);
    - the sums over n keys are within (n + 64) 2^-23 of their magnitudes, and the output is rounded once."""
    k, v, ks, vs = pool
    T, H_q, hd = q.shape
    H = k.shape[1]
    G = H_q // H
    dev, P = q.device, k.shape[2]
    out = torch.full((T, H_q, hd), math.nan, dtype=torch.float64, device=dev)
    lse = torch.full((T, H_q), math.nan, dtype=torch.float64, device=dev)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    eps = torch.finfo(q.dtype).eps / 2
    floor, step = FLOOR[q.dtype], STEP[q.dtype]
    table = np.asarray(table)
    for r in range(len(lens)):
        a, b, L = int(q_off[r]), int(q_off[r + 1]), int(lens[r])
        n = b - a
        if n <= 0:
            continue
        if L <= 0:
            out[a:b], lse[a:b] = 0, -math.inf
            continue
        ids = table[r, :-(-L // P)].tolist()
        one = torch.ones_like(vs)
        kk, code = ref.gather(k, ks, ids, L), ref.gather(v, one, ids, L).abs()
        vv = ref.gather(v, vs, ids, L)
        sv = vs[torch.as_tensor(ids, device=dev)].double().transpose(0, 1)
        sv = sv.reshape(H, -1).repeat_interleave(ref.BLOCK, -1)[:, None, None, :L]
        qq = q[a:b].double().view(n, H, G, hd).permute(1, 2, 0, 3)
        s = torch.einsum("hgnd,hkd->hgnk", qq, kk) * scale
        mag = torch.einsum("hgnd,hkd->hgnk", qq.abs(), kk.abs()) * abs(scale)
        d = mag * (hd * 2.0 ** -23 + 2.0 ** -21) + s.abs() * 2.0 ** -21
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            d = d + s.abs() * 2.0 ** -21
        dist = torch.arange(L - n, L, device=dev)[:, None] - torch.arange(L, device=dev)
        if slopes is not None:
            bias = slopes.double().view(H, G, 1, 1) * dist
            s = s - bias
            d = d + bias.abs() * 2.0 ** -21 + s.abs() * 2.0 ** -21
        seen = (dist >= 0) & ((dist < window) if window else True)
        s = s.masked_fill(~seen, -math.inf)
        none = ~seen.any(-1)
        top = s.amax(-1, keepdim=True)
        away = s - torch.where(top == -math.inf, 0.0, top)
        lv = torch.where(seen & (sv > 0), torch.log2(sv.clamp(min=1e-300)), math.nan)
        spread = (lv.nan_to_num(nan=-1e9).amax(-1, keepdim=True) - lv.nan_to_num(nan=1e9).amin(-1, keepdim=True)).clamp(0, 90)
        d = d + 2.0 ** -20 + (away.abs().nan_to_num(posinf=0.0) + spread) * 2.0 ** -23
        p = torch.exp(away)
        l = p.sum(-1, keepdim=True)
        l1 = torch.where(l == 0, 1.0, l)
        w = p / l1
        o = torch.einsum("hgnk,hkd->hgnd", w, vv)
        A = torch.einsum("hgnk,hkd->hgnd", w, vv.abs())
        wd = torch.where(seen, w * d, 0.0)
        E = torch.einsum("hgnk,hkd->hgnd", wd, vv.abs()) + o.abs() * wd.sum(-1, keepdim=True)
        prod = p * sv
        lost = torch.minimum(2 * prod, floor * prod.amax(-1, keepdim=True)).masked_fill(~seen, 0.0) / l1
        E = E + A * (step + (L + 64) * 2.0 ** -23) + torch.einsum("hgnk,hkd->hgnd", lost, code)
        ll = (top + torch.log(l))[..., 0]
        dl = wd.sum(-1) + (L + 64) * 2.0 ** -23 + ll.abs().nan_to_num(posinf=0.0) * 2.0 ** -21 + 2.0 ** -21 + \
            spread[..., 0] * 2.0 ** -23
        o = torch.where(none[:, None], 0.0, o)
        back = lambda x: x.permute(2, 0, 1, 3).reshape(n, H_q, hd)  # noqa: E731
        out[a:b] = back(o)
        tol[a:b] = back(E * (1 + eps) + eps * o.abs().clamp(min=torch.finfo(q.dtype).smallest_normal) + 1e-30)
        lse[a:b] = ll.permute(2, 0, 1).reshape(n, H_q)
        tol_l[a:b] = dl.permute(2, 0, 1).reshape(n, H_q)
        rows = torch.nonzero(none)[:, 0] + a
        out[rows], lse[rows], tol[rows], tol_l[rows] = 0, -math.inf, 0, 0
    return out, lse, tol, tol_l
