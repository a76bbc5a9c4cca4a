"""Bounds on each element of fa_fwd_paged's O from that row's own weights."""
import math

import numpy as np
import torch

import paged_util as pu


def attention(q, k, v, lens, new, seen, scale, dtype, drop=None):
    """(o, lse, bound on |o - kernel's|) in 64 bits, arguments as paged_util.attention's; drop: key positions
    that a planted mistake leaves out of P V.

    With weights w_j = p_j / l, the kernel's result is sum_j P(p_j) v_j / l, rounded:
     * P, rounded to the input type, is off by at most u = eps / 2 of p_j; in fp16 also by half a subnormal
       step, 2^-25, and l >= 1, because the reference of the exponentials is a score of the row (of each part
       of it: the parts' errors are weighed together with weights that add to 1);
     * the score of p_j is a sum of D products that are exact in fp32, off by (D + 2) 2^-24 sum |q k| |scale|
       at most, and the exponential by 2^-22 relative: together d; O moves by at most 2 d sum w |v|, since
       numerator and denominator move alike;
     * fp32 sums: the products add up in steps of at least 8 positions, each off by 2^-23 of a partial sum
       (the tensor core may truncate), l in fewer; rescaling, 1 / l and joining parts: 2^-20;
     * the last rounding: u |o|, in fp16 also 2^-25."""
    Z, Hq, T, D = q.shape
    u = torch.finfo(pu.DT[dtype]).eps / 2
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    o, lse, bound = np.zeros((Z, Hq, T, D)), np.full((Z, Hq, T), -math.inf), np.zeros((Z, Hq, T, D))
    for z in range(Z):
        n = int(lens[z]) + int(new[z])
        for h in range(Hq):
            kk, vv = k[z][h * k[z].shape[0] // Hq], v[z][h * k[z].shape[0] // Hq]
            for t in range(int(new[z])):
                keep = np.ones(n, dtype=bool)
                keep[int(lens[z]):] = np.arange(int(new[z])) <= t if seen is None else seen[z, t, :int(new[z])]
                if not keep.any():
                    continue
                s = scale * (kk[keep] @ q[z, h, t])
                m = s.max()
                p = np.exp(s - m)
                w = p / p.sum()
                lse[z, h, t] = m + math.log(p.sum())
                far = np.zeros(n, dtype=bool) if drop is None else np.isin(np.arange(n), drop)
                o[z, h, t] = np.where(far[keep], 0.0, w) @ vv[keep]
                size = w @ np.abs(vv[keep])
                d = (D + 2) * 2.0 ** -24 * abs(scale) * float((np.abs(kk[keep]) @ np.abs(q[z, h, t])).max()) + 2.0 ** -22
                d += int(keep.sum()) / 8 * 2.0 ** -23 + 2.0 ** -20
                bound[z, h, t] = size * (u + 2 * d) + u * np.abs(o[z, h, t]) + tiny * (1 + np.abs(vv[keep]).sum(0))
    return o, lse, bound
