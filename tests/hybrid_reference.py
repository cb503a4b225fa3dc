"""Plain fp64 forms of the hybrid step's operators (state pool, paged append, paged attention),
token by token on the CPU, with the bounds that the kernels' roundings allow."""
from __future__ import annotations

import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}   # half a step
U = 2.0 ** -24   # half a step of fp32


def pool_step(q, k, v, g, beta, pool, slots_in, slots_out, lens, normalize=False, g_logits=False,
              beta_logits=False):
    """Returns (out fp64 [T, Hv, D], pool fp64, bound on |out|'s arithmetic error [T, Hv, D])."""
    q, k, v, g, beta, pool = (x.double().cpu() for x in (q, k, v, g, beta, pool))
    pool = pool.clone()
    T, Hk, D = q.shape
    Hv = v.shape[1]
    if normalize:
        q = q / q.norm(dim=-1, keepdim=True).clamp_min(1e-12)
        k = k / k.norm(dim=-1, keepdim=True).clamp_min(1e-12)
    q, k = q.repeat_interleave(Hv // Hk, 1), k.repeat_interleave(Hv // Hk, 1)
    a = torch.sigmoid(g) if g_logits else torch.exp(g)
    a = a[..., None] if a.dim() == 2 else a
    b = torch.sigmoid(beta) if beta_logits else beta
    out, bound = torch.zeros(T, Hv, D, dtype=torch.float64), torch.zeros(T, Hv, D, dtype=torch.float64)
    t = 0
    for n, length in enumerate(lens):
        if length == 0:
            continue
        slot = int(slots_in[n])
        S = pool[slot].clone() if slot >= 0 else torch.zeros(Hv, D, D, dtype=torch.float64)
        err = torch.zeros_like(S)   # bound of the state's error so far, elementwise
        for _ in range(length):
            S, err = a[t][..., None] * S, a[t][..., None] * err + 8 * U * (a[t][..., None] * S).abs()
            read = torch.einsum("hcv,hc->hv", S, k[t])
            eread = torch.einsum("hcv,hc->hv", err + (D + 8) * U * S.abs(), k[t].abs())
            u = b[t][:, None] * (v[t] - read)
            eu = b[t][:, None] * eread + 8 * U * (b[t][:, None] * (v[t].abs() + read.abs()))
            S = S + k[t][..., None] * u[:, None, :]
            err = err + k[t].abs()[..., None] * eu[:, None, :] + 8 * U * (S.abs() + (k[t][..., None] * u[:, None, :]).abs())
            out[t] = torch.einsum("hcv,hc->hv", S, q[t])
            kq = (k[t] * q[t]).abs().sum(-1, keepdim=True)
            bound[t] = torch.einsum("hcv,hc->hv", err + (D + 8) * U * S.abs(), q[t].abs()) + 2 * D * U * kq * u.abs()
            if int(slots_out[t]) >= 0:
                pool[int(slots_out[t])] = S
            t += 1
    return out, pool, bound


def rotate(x, positions, inv_freq, axis_pairs, adjacent):
    """x [T, H, D] fp64 rotated by positions [axes, T]; returns (y, |x1| + |x2| of each output)."""
    x = x.double().cpu()
    pos, freq = positions.double().cpu(), inv_freq.double().cpu()
    angle = torch.cat([pos[a][:, None] * freq[None, sum(axis_pairs[:a]):sum(axis_pairs[:a + 1])]
                       for a in range(len(axis_pairs))], 1)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    half = freq.shape[0]
    i1 = torch.arange(0, 2 * half, 2) if adjacent else torch.arange(half)
    i2 = i1 + 1 if adjacent else i1 + half
    y, size = x.clone(), torch.zeros_like(x)
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    size[..., i1] = size[..., i2] = x[..., i1].abs() + x[..., i2].abs()
    return y, size


def rotation_bound(y, size, dtype):
    """The angle is exact to 2^-25 turns (2^-22.3 rad), sine and cosine to 2^-23, each of the two
    products and the sum to 2^-24: 2^-21 of |x1| + |x2|; then one rounding to the type (e4m3 steps
    are 2^-9 below its smallest normal)."""
    b = HALF[dtype] * y.abs() + 2.0 ** -21 * size
    if dtype == torch.bfloat16:
        b = b * (1 + 2.0 ** -7)
    return b


def attend(q, k_cache, v_cache, table, seq_lens, lens, scale, softcap=0.0, window=0, slopes=None, start=None,
           k_scale=None, v_scale=None):
    """Returns (out, lse, bound on out, bound on lse), fp64 [T, Hq, D] and [T, Hq].

    Score errors: the products of bf16 and e4m3 inputs are exact in fp32, fp32 inputs are split in
    two parts of 11 bits each (2^-22 each, and the product of the low parts is dropped: 3 * 2^-22);
    D additions of 2^-24; scale, cap and bias a few 2^-24 of |s| and of the bias.  A weight then is
    off by the score's error and by e^x's (2^-21), and by half a step of the type that multiplies v."""
    T, Hq, D = q.shape
    ps, Hkv = k_cache.shape[2], k_cache.shape[1]
    ty = q.dtype
    fp8 = k_cache.dtype == torch.float8_e4m3fn
    q = q.double().cpu()
    kc, vc = k_cache.float().cpu().double(), v_cache.float().cpu().double()
    table, seq_lens = table.cpu(), seq_lens.cpu()
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    # half a step of the type in which weights multiply values (fp16 over an e4m3 cache)
    wide = 3 * 2.0 ** -22 if ty == torch.float32 else (2.0 ** -11 if fp8 else 2.0 ** -8)
    t = 0
    for n, length in enumerate(lens):
        L = int(seq_lens[n])
        for i in range(length):
            pos = L - length + i
            lo = max(0, int(start[n]) if start is not None else 0, pos - window + 1 if window else 0)
            js = [j for j in range(lo, pos + 1) if j // ps < table.shape[1] and 0 <= int(table[n, j // ps]) < kc.shape[0]]
            if js:
                j = torch.tensor(js)
                pages = table[n].long()[j // ps]
                K, V = kc[pages, :, j % ps], vc[pages, :, j % ps]   # [len, Hkv, D]
                if k_scale is not None:
                    K = K * k_scale.double().cpu()[:, None]
                if v_scale is not None:
                    V = V * v_scale.double().cpu()[:, None]
                K, V = (x.repeat_interleave(Hq // Hkv, 1) for x in (K, V))
                s = scale * torch.einsum("hd,jhd->hj", q[t], K)
                es = abs(scale) * torch.einsum("hd,jhd->hj", q[t].abs(), K.abs()) * (D * U + (3 * 2.0 ** -22 if ty == torch.float32 else 0)) + 6 * U * s.abs()
                if softcap:
                    es = es + 2.0 ** -21 * softcap * torch.tanh(s / softcap).abs()
                    s = softcap * torch.tanh(s / softcap)
                if slopes is not None:
                    bias = slopes.double().cpu()[:, None] * (j - pos).double()[None]
                    s, es = s + bias, es + 2 * U * (bias.abs() + s.abs())
                p = torch.softmax(s, -1)
                # the bias keeps far keys at weights of nothing: their errors weigh nothing either
                off = (p * (2 * es + 2.0 ** -20)).sum(-1)
                size = torch.einsum("hj,jhd->hd", p, V.abs())
                out[t] = torch.einsum("hj,jhd->hd", p, V)
                lse[t] = torch.logsumexp(s, -1)
                ob[t] = torch.einsum("hj,jhd->hd", p * (2 * es + 2.0 ** -20 + wide), V.abs()) + off[:, None] * size
                ob[t] += len(js) * U * size
                if ty != torch.float32:   # weights below the type's smallest normal (fp16: 2^-14)
                    ob[t] += (2.0 ** -25 if fp8 else 0.0) * V.abs().sum(0)
                ob[t] = ob[t] * (1 + HALF[ty]) + HALF[ty] * out[t].abs()
                lb[t] = off + 4 * U * lse[t].abs() + len(js) * U
            t += 1
    return out, lse, ob, lb
