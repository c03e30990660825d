"""Serving operators around the 4-bit linear layer, as cases to time and compare.

Three operators of a decoder layer whose weights and cache are held in 4 bits:

  norm    residual addition, root-mean-square norm and per-row int8 codes in one pass
          h = round(x + residual),  t = h * weight,  codes and zero point of the row t as the
          int8-activation linear defines them (range [min(0, min t), max(0, max t)] over 255 steps,
          every step in fp32), row scale = step / sqrt(mean(h^2) + eps).  The norm's factor is one
          number per row, so it goes into the row's scale and the codes do not depend on it.
  append  keys and values of new tokens into a paged cache of 4-bit codes: per token, head and run
          of 32 channels, scale = fp16(min(max|x| / 7, 8188)), code - 8 = clamp(rint(x * (1 / scale)),
          -8, 7), 0 where the scale is 0 or x is NaN; then the same rows read back.
  attend  causal attention of the newest tokens of each sequence over that cache: grouped heads,
          one token (decoding), a few (verification of drafts) or many (a prompt), optionally a
          sliding window and scores capped by cap * tanh(score / cap).

`run` takes plain torch operations where `own` is false and the package's calls where it is true.
"""
import random

import torch

own = False

P = 64                      # tokens per cache page
G = 32                      # channels per scale
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FLT_MIN = 2.0 ** -126
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------------------
def _attend(name, batch, new, ctx, hq, hkv, dim, dtype, ragged=False, window=0, cap=0.0):
    return dict(name=name, op="attend", batch=batch, new=new, ctx=ctx, hq=hq, hkv=hkv, dim=dim, dtype=dtype,
                ragged=ragged, window=window, cap=cap)


def _append(name, batch, new, ctx, hkv, dim, dtype, ragged=False):
    return dict(name=name, op="append", batch=batch, new=new, ctx=ctx, hkv=hkv, dim=dim, dtype=dtype, ragged=ragged)


def _norm(name, rows, cols, xtype, rtype):
    return dict(name=name, op="norm", rows=rows, cols=cols, xtype=xtype, rtype=rtype)


def listed():
    return [
        # one user, one token, a short conversation, in the geometry of the QKV triple 2048 / 512 / 512:
        # the latency of a call
        _attend("decode_one", 1, 1, 509, 32, 8, 64, "bf16"),
        # a server's batch of unlike lengths, one token each
        _attend("decode_batch", 32, 1, 4096, 32, 8, 128, "fp16", ragged=True),
        # two long documents: few rows, so the cache's length has to be split
        _attend("decode_long", 2, 1, 131072, 32, 8, 128, "bf16"),
        # the largest serving batch: the cache's bytes are all that counts
        _attend("decode_large", 64, 1, 16384, 32, 8, 128, "bf16", ragged=True),
        # wide heads, a sliding window and capped scores
        _attend("decode_window", 16, 1, 8191, 16, 4, 256, "bf16", ragged=True, window=1024, cap=50.0),
        # five drafted tokens of each sequence checked at once
        _attend("verify", 8, 5, 3001, 64, 8, 128, "bf16", ragged=True),
        # one prompt of 512 tokens from its beginning, in the geometry of decode_one
        _attend("prompt_512", 1, 512, 512, 32, 8, 64, "fp16"),
        # chunks of 2048 prompt tokens behind unlike parts already in the cache
        _attend("prompt_chunk", 3, 2048, 8192, 32, 8, 128, "bf16", ragged=True),
        # one decoding step's keys and values of a batch
        _append("append_step", 64, 1, 4099, 8, 128, "bf16", ragged=True),
        # a prompt's keys and values, from the middle of pages on
        _append("append_prompt", 4, 4099, 8200, 8, 128, "fp16", ragged=True),
        # one decoding step of a small batch: the linear layer's fp32 output on an fp32 stream
        _norm("norm_step", 4, 2048, "fp32", "fp32"),
        # a prompt's rows at the widest layer
        _norm("norm_prompt", 4096, 8192, "bf16", "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    kind = rng.choice(["decode", "decode", "decode", "verify", "prompt", "prompt", "append", "norm", "norm"])
    dtype = rng.choice(["bf16", "fp16"])
    hkv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 64, 96, 128, 128, 128, 256])
    group = rng.choice([1, 2, 3, 4, 4, 6, 8])
    window = rng.choice([0, 0, 0, _spread(rng, 16, 4096)])
    cap = rng.choice([0.0, 0.0, 0.0, 30.0, 50.0])
    ragged = rng.random() < 0.7
    if kind == "norm":
        rows = _spread(rng, 1, 4096)
        cols = _spread(rng, 300, 16384)
        if rng.random() < 0.75:
            cols = (cols + 63) // 64 * 64
        if rows * cols > 4096 * 8192:
            rows = 4096 * 8192 // cols
        return _norm("", rows, cols, rng.choice(["fp32", "bf16", "fp16"]), rng.choice(["fp32", "bf16", "fp16"]))
    if kind == "append":
        new = _spread(rng, 1, 4096)
        batch = _spread(rng, 1, max(1, min(64, 16384 // new)))
        return _append("", batch, new, new + _spread(rng, 1, 8192) - 1, hkv, dim, dtype, ragged)
    if kind == "prompt":
        new = _spread(rng, 65, 3000)
        batch = _spread(rng, 1, max(1, min(8, 4096 // new)))
        ctx = new + rng.choice([0, _spread(rng, 1, 6000)])
        # heads x rows x keys x width at most a quarter of prompt_chunk's
        while batch * hkv * group * new * ctx * dim > 3 * 32 * 2048 * 8192 * 128 // 4:
            new, ctx = max(1, new // 2), max(1, ctx // 2)
        return _attend("", batch, new, ctx, hkv * group, hkv, dim, dtype, ragged, window, cap)
    new = 1 if kind == "decode" else rng.randint(2, 9)
    ctx = new + _spread(rng, 1, 131072) - 1
    most = 64 * 8192 * 8 * 128
    batch = _spread(rng, 1, max(1, min(64, most // (ctx * hkv * dim))))
    return _attend("", batch, new, ctx, hkv * group, hkv, dim, dtype, ragged, window, cap)


def _lens(case):
    """(new tokens, tokens in the cache with them) of every sequence: all alike, or unlike with
    the first as long as the case says."""
    new, ctx = [case["new"]] * case["batch"], [case["ctx"]] * case["batch"]
    if case["ragged"]:
        r = random.Random(f"{case['batch']} {case['new']} {case['ctx']}")
        for b in range(1, case["batch"]):
            if case["new"] > 9:
                new[b] = r.randint((case["new"] + 1) // 2, case["new"])
            ctx[b] = r.randint(max(new[b], case["ctx"] // 4), case["ctx"])
    return new, ctx


def _first(pos, window):
    """The first key that the token at `pos` sees."""
    return max(0, pos - window + 1) if window else 0


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        x, r = size[case["xtype"]], size[case["rtype"]]
        # x, the residual and the weight; h, the int8 codes and the values; a scale and a zero point a row
        return {"bytes": n * (x + 2 * r + 1 + 4) + case["cols"] * r + 8 * case["rows"], "flops": 10 * n}
    new, ctx = _lens(case)
    row = case["hkv"] * case["dim"] * 2           # elements of one token's keys and values
    if case["op"] == "append":
        n = sum(new) * row
        # the new rows, their codes and scales, and the values they stand for in fp32
        return {"bytes": int(n * (size[case["dtype"]] + 0.5 + 2 / G + 4)), "flops": 6 * n}
    keys = pairs = 0
    for m, n in zip(new, ctx):
        keys += n - _first(n - m, case["window"])
        pairs += sum(p + 1 - _first(p, case["window"]) for p in range(n - m, n))
    io = 2 * sum(new) * case["hq"] * case["dim"] * size[case["dtype"]]
    return {"bytes": int(keys * row * (0.5 + 2 / G)) + io, "flops": 4 * pairs * case["hq"] * case["dim"]}


# ---- inputs ----------------------------------------------------------------------------------
def _gen(seed, b):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 7919 * b + 1)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _keys_values(case, seed, b, n):
    """n tokens of keys (a few channels larger than the others, as keys have them) and values."""
    g = _gen(seed, b)
    h, d = case["hkv"], case["dim"]
    channel = 0.5 + torch.rand(h, d, generator=g, device="cuda")
    channel = torch.where(torch.rand(h, d, generator=g, device="cuda") < 0.03, 5 * channel, channel)
    k = (_randn(g, n, h, d) * channel).to(DT[case["dtype"]])
    return k, _randn(g, n, h, d).to(DT[case["dtype"]])


def _quantise(x):
    """(code - 8 as int8 [.., dim], scale fp16 [.., dim / 32]) of rows of keys or values."""
    g = x.float().unflatten(-1, (-1, G))
    g = torch.where(g.isnan(), torch.zeros_like(g), g)
    amax = g.abs().amax(-1)
    s = (amax / torch.full_like(amax, 7.0)).clamp(max=8188.0).half()
    inv = (1.0 / s.float()).unsqueeze(-1)
    c = torch.where(s.unsqueeze(-1) > 0, (g * inv).round().clamp(-8, 7), torch.zeros_like(g))
    return c.to(torch.int8).flatten(-2), s


def _values(codes, scale):
    return (codes.unflatten(-1, (-1, G)).float() * scale.float().unsqueeze(-1)).flatten(-2)


class _Pool:
    """The plain form's cache: int8 code - 8 and scales of every page's tokens."""

    def __init__(self, pages, h, d):
        self.k, self.v = (torch.zeros(pages, P, h, d, dtype=torch.int8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.zeros(pages, P, h, d // G, dtype=torch.float16, device="cuda") for _ in range(2))

    def store(self, k, v, page, slot):
        self.k[page, slot], self.ks[page, slot] = _quantise(k)
        self.v[page, slot], self.vs[page, slot] = _quantise(v)


def prepare(case, seed):
    if case["op"] == "norm":
        g = _gen(seed, 0)
        m, k = case["rows"], case["cols"]
        r = DT[case["rtype"]]
        s = dict(case=case, x=_randn(g, m, k).to(DT[case["xtype"]]), residual=(3 * _randn(g, m, k)).to(r),
                 weight=(1 + 0.2 * _randn(g, k)).to(r))
        if own:
            import bit_group_quantized_q4gsw_amd as q4
            s.update(q4=q4, rows=q4.dq8ca_rows(m, k, "cuda"), h=torch.empty(m, k, dtype=r, device="cuda"),
                     values=torch.empty(m, k, dtype=torch.float32, device="cuda"))
        return s

    new, ctx = _lens(case)
    h, d = case["hkv"], case["dim"]
    need = [(n + P - 1) // P for n in ctx]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 1)).tolist()
    table = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
        order = order[n:]
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
    s = dict(case=case, new=new, ctx=ctx, tokens=sum(new), pages=pages, table=table.cuda(), cu=cu.cuda(),
             lens=torch.tensor(ctx, dtype=torch.int32).cuda())
    if own:
        import bit_group_quantized_q4gsw_amd as q4
        s.update(q4=q4, cache=q4.kv_cache(pages, P, h, d, "cuda"))
    else:
        s.update(pool=_Pool(pages, h, d))

    if case["op"] == "append":
        kv = [_keys_values(case, seed, b, m) for b, m in enumerate(new)]
        s.update(k=torch.cat([k for k, _ in kv]), v=torch.cat([v for _, v in kv]))
        return s

    g = _gen(seed, -1)
    # scores of a spread of two to three, as trained heads have them
    s["q"] = (1.6 * _randn(g, sum(new), case["hq"], d)).to(DT[case["dtype"]])
    for b, n in enumerate(ctx):
        k, v = _keys_values(case, seed, b, n)
        if own:
            one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            s["q4"].kv_append(s["cache"], k, v, s["table"][b:b + 1], one, s["lens"][b:b + 1])
        else:
            s["pool"].store(k, v, *_slots(s, b, 0, n))
    if own:
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = torch.empty(
            q4.kv_attention_workspace_bytes(s["cache"], len(ctx), sum(new), case["hq"], max(new), max(ctx)),
            dtype=torch.uint8, device="cuda")
    return s


def _slots(s, b, first, last):
    """Pages and places in them of the tokens first .. last - 1 of sequence b."""
    t = torch.arange(first, last, device="cuda")
    return s["table"][b].long()[t // P], t % P


# ---- the operators ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _own_norm, "append": _own_append, "attend": _own_attend}[op](s)
    return {"norm": _plain_norm, "append": _plain_append, "attend": _plain_attend}[op](s)


def _own_norm(s):
    _, h, values = s["q4"].rmsnorm_dq8ca(s["x"], s["weight"], EPS, residual=s["residual"], rows=s["rows"], h=s["h"],
                                         values=s["values"])
    return h, values


def _own_append(s):
    s["q4"].kv_append(s["cache"], s["k"], s["v"], s["table"], s["cu"], s["lens"])
    return s["q4"].kv_read(s["cache"], s["table"], s["cu"], s["lens"], s["tokens"])


def _own_attend(s):
    c = s["case"]
    return s["q4"].kv_attention(s["cache"], s["q"], s["table"], s["cu"], s["lens"], max(s["new"]), max(s["ctx"]),
                                window=c["window"], softcap=c["cap"], out=s["out"], workspace=s["workspace"])


def _plain_norm(s):
    h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    t = h.float() * s["weight"].float()
    lo = t.amin(1, keepdim=True).clamp(max=0.0)
    hi = t.amax(1, keepdim=True).clamp(min=0.0)
    step = ((hi - lo) / torch.full_like(hi, 255.0)).clamp(min=FLT_MIN)
    inv = 1.0 / step
    zero = (-128 - (lo * inv).round()).clamp(-128, 127)
    codes = ((t * inv).round() + zero).clamp(-128, 127)
    factor = (1.0 / (h.double().square().mean(1, keepdim=True) + EPS).sqrt()).float()
    return h, (factor * step) * (codes - zero)


def _plain_append(s):
    token = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    pos = s["lens"][seq] - (s["cu"][seq + 1] - token)
    page, slot, pool = s["table"][seq, pos // P].long(), pos % P, s["pool"]
    pool.store(s["k"], s["v"], page, slot)
    return _values(pool.k[page, slot], pool.ks[page, slot]), _values(pool.v[page, slot], pool.vs[page, slot])


def _plain_attend(s):
    c, pool = s["case"], s["pool"]
    hkv, d, group = c["hkv"], c["dim"], c["hq"] // c["hkv"]
    out, at = torch.empty_like(s["q"]), 0
    for b, (m, n) in enumerate(zip(s["new"], s["ctx"])):
        first = _first(n - m, c["window"])
        page, slot = _slots(s, b, first, n)
        k = _values(pool.k[page, slot], pool.ks[page, slot]).permute(1, 2, 0).contiguous()
        v = _values(pool.v[page, slot], pool.vs[page, slot]).transpose(0, 1).contiguous()
        q = s["q"][at:at + m].float().view(m, hkv, group, d).permute(1, 2, 0, 3).reshape(hkv, group * m, d)
        x = torch.matmul(q, k) * d ** -0.5
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        if m > 1 or c["window"]:
            i = torch.arange(n - m, n, device="cuda").repeat(group)[:, None]
            j = torch.arange(first, n, device="cuda")[None]
            seen = (j <= i) & (j > i - c["window"]) if c["window"] else j <= i
            x = x.masked_fill(~seen, float("-inf"))
        p = torch.exp(x - x.amax(-1, keepdim=True))
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        out[at:at + m] = o.view(hkv, group, m, d).permute(2, 0, 1, 3).reshape(m, c["hq"], d).to(out.dtype)
        at += m
    return out


# ---- the definitions in 64 bits --------------------------------------------------------------
def _f32(x):
    return x.to(torch.float32).double()


def _stored(x):
    """What the cache stands for, in 64 bits; the definition's roundings to 16 and 32 bits kept."""
    n, h, d = x.shape
    x = torch.nan_to_num(x.double(), nan=0.0, posinf=float("inf"), neginf=float("-inf")).view(n, h, d // G, G)
    step = _f32(x.abs().max(dim=-1, keepdim=True).values / 7).clamp(max=8188.0).to(torch.float16).double()
    code = torch.round(_f32(x * _f32(1 / step.clamp(min=2.0 ** -24)))).clamp(-8, 7)
    return (code * step).view(n, h, d)


def exact(case, seed):
    if case["op"] == "norm":
        g = _gen(seed, 0)
        m, k = case["rows"], case["cols"]
        r = DT[case["rtype"]]
        x = _randn(g, m, k).to(DT[case["xtype"]])
        res = (3 * _randn(g, m, k)).to(r)
        w = (1 + 0.2 * _randn(g, k)).to(r).double()
        h = _f32(x.double() + res.double()).to(r).double()
        t = _f32(h * w)
        lo, hi = t.min(1).values.clamp(max=0)[:, None], t.max(1).values.clamp(min=0)[:, None]
        step = _f32(_f32(hi - lo) / 255).clamp(min=FLT_MIN)
        inv = _f32(1 / step)
        zero = (-128 - torch.round(_f32(lo * inv))).clamp(-128, 127)
        code = (torch.round(_f32(t * inv)) + zero).clamp(-128, 127)
        return h, (code - zero) * step * torch.rsqrt((h * h).sum(1, keepdim=True) / k + EPS)

    new, ctx = _lens(case)
    if case["op"] == "append":
        kv = [_keys_values(case, seed, b, m) for b, m in enumerate(new)]
        return torch.cat([_stored(k) for k, _ in kv]), torch.cat([_stored(v) for _, v in kv])

    group, win, cap = case["hq"] // case["hkv"], case["window"], case["cap"]
    q = (1.6 * _randn(_gen(seed, -1), sum(new), case["hq"], case["dim"])).to(DT[case["dtype"]]).double()
    out, at = torch.zeros_like(q), 0
    for b, (m, n) in enumerate(zip(new, ctx)):
        k, v = _keys_values(case, seed, b, n)
        pos = torch.arange(n, device="cuda")
        lag = pos[n - m:, None] - pos[None]
        gone = (lag < 0) | (lag >= win) if win else lag < 0
        for kvh in range(case["hkv"]):
            ks, vs = _stored(k[:, kvh:kvh + 1])[:, 0], _stored(v[:, kvh:kvh + 1])[:, 0]
            for hq in range(kvh * group, (kvh + 1) * group):
                x = q[at:at + m, hq] @ ks.T / case["dim"] ** 0.5
                if cap:
                    x = cap * torch.tanh(x / cap)
                x[gone] = -float("inf")
                out[at:at + m, hq] = torch.softmax(x, dim=1) @ vs
        at += m
    return out
