"""Plain models of trees of drafted tokens, from their definition (CPU tensors)."""
import math
import random

import torch

from tests.serving_model import G, U, kv_values  # noqa: F401


def ancestors(parents):
    """Per node the list root .. node; a parent that is not an earlier node makes a root."""
    paths = []
    for i, p in enumerate(parents):
        paths.append((paths[p] if 0 <= p < i else []) + [i])
    return paths


def forest(n, kind, seed=0):
    """Parents of n nodes: "chain", "star" (all behind node 0), "roots" (no edges), "far" (parents anywhere
    before), "wild" (values that name no earlier node among them), "near" (a few nodes back)."""
    r = random.Random(f"{n} {kind} {seed}")
    one = {
        "chain": lambda i: i - 1,
        "star": lambda i: 0 if i else -1,
        "roots": lambda i: -1,
        "far": lambda i: r.randrange(i) if i else -1,
        "wild": lambda i: r.choice([i, i + 1, -1, -7, 2 ** 31 - 1, -2 ** 31, r.randrange(i + 1)]),
        "near": lambda i: max(-1, i - r.randint(1, 4)),
    }[kind]
    return [one(i) for i in range(n)]


def seen(parents, n, window):
    """bool [m, n]: the places of a sequence of n tokens that each node sees."""
    m = len(parents)
    paths = ancestors(parents)
    p0 = n - m
    out = torch.zeros(m, n, dtype=torch.bool)
    for i, path in enumerate(paths):
        position = p0 + len(path) - 1
        for depth, j in enumerate(path):
            if p0 + j >= 0 and (not window or p0 + depth > position - window):
                out[i, p0 + j] = True
        first = max(0, position - window + 1) if window else 0
        out[i, min(first, max(p0, 0)):max(p0, 0)] = True
    return out


def tree_attention(q, keys, values, parents, lens, window=0, cap=0.0, paged=None):
    """(out, bound) for q [tokens, hq, d], as serving_model.attention; parents: a list per sequence;
    paged[b] (bool [ctx]) hides places without a page."""
    dt = q.dtype
    q = q.double()
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    hq, d = q.shape[1], q.shape[2]
    at = 0
    for b, (n, tree) in enumerate(zip(lens, parents)):
        k, v, m = keys[b], values[b], len(tree)
        group = hq // k.shape[1]
        mask = seen(tree, n, window)
        if paged is not None:
            mask &= paged[b][None]
        scale = k.abs().unflatten(-1, (-1, G)).amax(-1, keepdim=True).expand(*k.shape[:2], d // G, G).flatten(-2)
        for h in range(hq):
            kk, vv, ss, qq = k[:, h // group], v[:, h // group], scale[:, h // group], q[at:at + m, h]
            x = qq @ kk.T / math.sqrt(d)
            if cap:
                x = cap * torch.tanh(x / cap)
            x = x.masked_fill(~mask, float("-inf"))
            p = torch.where(mask.any(1, keepdim=True), torch.softmax(x, -1), torch.zeros_like(x))
            out[at:at + m, h] = p @ vv
            # the errors of serving_model.attention
            rounds = 2.0 ** -11 * (2 if dt == torch.float32 else 1)
            e = (rounds * (qq.abs() @ kk.abs().T) + 33 * 1039 * 2.0 ** -24 * (qq.abs() @ ss.T)) / math.sqrt(d)
            e = torch.where(mask, e, torch.zeros_like(e)).amax(1, keepdim=True) if n else torch.zeros(m, 1).double()
            rel = torch.expm1(2 * (e + 2.0 ** -20)) + 2 * 2.0 ** -11 + n * 2.0 ** -23
            bound[at:at + m, h] = rel * (p @ vv.abs()) + U[dt] * out[at:at + m, h].abs() + 1e-7
        at += m
    return out, bound
