"""Plain 64-bit models of the decoder serving calls, from their definitions (CPU tensors)."""
import math

import torch

G = 32
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f32(x):
    """The fp32 rounding of a 64-bit tensor."""
    return x.to(torch.float32).double()


def kv_codes(x):
    """(values -8..7 [..., dim], scales [..., dim / 32], both 64 bits) of rows of keys or values."""
    x = torch.nan_to_num(x.double(), nan=0.0, posinf=float("inf"), neginf=float("-inf")).unflatten(-1, (-1, G))
    s = f32(x.abs().amax(-1) / 7).clamp(max=8188.0).half().double()
    inv = f32(1 / torch.where(s > 0, s, torch.ones_like(s))).unsqueeze(-1)
    # an infinity saturates; rint is half to even
    c = torch.round(f32(x * inv)).clamp(-8, 7)
    c = torch.where(s.unsqueeze(-1) > 0, c, torch.zeros_like(c))
    return c.flatten(-2), s


def kv_values(x):
    c, s = kv_codes(x)
    return (c.unflatten(-1, (-1, G)) * s.unsqueeze(-1)).flatten(-2)


def attention(q, keys, values, lens, news, window=0, cap=0.0, seen=None):
    """(out, bound) for q [tokens, hq, d]: keys / values lists of [ctx, hkv, d] (64 bits, as stored).

    bound is the error the call may make, element by element: scores carry the keys' rounding to
    fp16 (2^-11; fp32 queries once more) and fp32 products over code + 1032 (33 roundings of sums of
    at most 1039 |q| scale a channel); a score off by e changes a weight by at most e^(2 e); weights
    and values each round to fp16; the sums are fp32; the output rounds once to its type.
    seen[b] (bool [ctx]) hides places without a page."""
    dt = q.dtype
    q = q.double()
    out = torch.zeros_like(q)
    bound = torch.zeros_like(q)
    hq, d = q.shape[1], q.shape[2]
    at = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        k, v = keys[b], values[b]
        group = hq // k.shape[1]
        place = torch.arange(n - m, n)
        t = torch.arange(n)
        mask = t[None] <= place[:, None]
        if window:
            mask &= t[None] > place[:, None] - window
        if seen is not None:
            mask &= seen[b][None]
        scale_of = k.abs().unflatten(-1, (-1, G)).amax(-1, keepdim=True).expand(*k.shape[:2], d // G, G).flatten(-2)
        for h in range(hq):
            kk, vv, ss = k[:, h // group], v[:, h // group], scale_of[:, h // group]
            qq = q[at:at + m, h]
            x = qq @ kk.T / math.sqrt(d)
            if cap:
                x = cap * torch.tanh(x / cap)
            x = x.masked_fill(~mask, float("-inf"))
            p = torch.softmax(x, -1)
            p = torch.where(mask.any(1, keepdim=True), p, torch.zeros_like(p))
            out[at:at + m, h] = p @ vv
            # scale_of is at least the scale (the largest value of a run is 7 or 8 scales, or less)
            rounds = 2.0 ** -11 * (2 if dt == torch.float32 else 1)
            e = (rounds * (qq.abs() @ kk.abs().T) + 33 * 1039 * 2.0 ** -24 * (qq.abs() @ ss.T)) / math.sqrt(d)
            e = torch.where(mask, e, torch.zeros_like(e)).amax(1, keepdim=True) if n else torch.zeros(m, 1).double()
            rel = torch.expm1(2 * (e + 2.0 ** -20)) + 2 * 2.0 ** -11 + n * 2.0 ** -23
            bound[at:at + m, h] = rel * (p @ vv.abs()) + U[dt] * out[at:at + m, h].abs() + 1e-7
        at += m
    return out, bound


def norm_rows(x, residual, weight, eps):
    """(h, codes, zero, row scale, values) of rmsnorm_dq8ca; the codes' steps in fp32 as defined."""
    dt = weight.dtype
    h = x.float().double() if residual is None else f32(x.double() + residual.double())
    h = h.to(torch.float32).to(dt).double()
    t = f32(h * weight.double())
    lo, hi = t.amin(1, keepdim=True).clamp(max=0), t.amax(1, keepdim=True).clamp(min=0)
    step = f32(f32(hi - lo) / 255).clamp(min=2.0 ** -126)
    inv = f32(1 / step)
    zero = (-128 - torch.round(f32(lo * inv))).clamp(-128, 127)
    codes = (torch.round(f32(t * inv)) + zero).clamp(-128, 127)
    row = step / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, codes, zero, row, (codes - zero) * row
