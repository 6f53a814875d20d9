"""Serving operators beside the W4A4 layer, as measured cases.

Four operators of quantized LLM serving, each in its plain form (elementary torch operations in
32 bits, rounded once at the end) and as a call of this package:

* ``linear``     int8 x int8 linear layer: per-token activation scales, per-output-channel weight
                 scales, optional bias.
* ``append``     keys and values of new tokens into a paged cache of 4-bit codes, and those tokens
                 read back as the values they stand for.
* ``attention``  causal attention of each sequence's last tokens over its pages of that cache: one
                 query token (a decode step), a few (draft tokens to verify), or whole prompts.

Cache layout (page p, kv head h, token t of the page, channel d): keys k[p, h, t, d // 2] hold the
even channel in the low nibble; values v[p, h, t // 4, d // 4, 4 * (t % 4 // 2) + 2 * (t % 2) + d % 4 // 2]
likewise (tokens interleaved by four); k_par / v_par[p, h, t] = (zero point, scale) in fp16.  A code q
stands for scale * (q - zero point).
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    """Cases: sizes of the Llama-7B and Llama-70B layers that this repository measures, a tiny
    one, and odd ones."""
    lin = dict(op="linear", bias=False)
    app = dict(op="append", page=64)
    att = dict(op="attention", page=64, empty=False)
    return [
        # one token through an attention projection: latency
        dict(lin, name="linear_1x4096x4096", m=1, k=4096, n=4096, dtype="fp16"),
        # a decode batch through the MLP's gate: the weights' bytes
        dict(lin, name="linear_16x4096x11008", m=16, k=4096, n=11008, dtype="bf16"),
        # odd sizes, with a bias: rows that no vector load fits
        dict(lin, name="linear_333x1155x777_bias", m=333, k=1155, n=777, dtype="fp16", bias=True),
        # the MLP's second product for a batch of prompts: the matrix cores
        dict(lin, name="linear_2048x11008x4096", m=2048, k=11008, n=4096, dtype="fp16"),
        # the largest: a Llama-70B MLP
        dict(lin, name="linear_4096x8192x28672", m=4096, k=8192, n=28672, dtype="bf16"),
        # a decode step's new tokens: latency
        dict(app, name="append_64_tokens_8_heads", tokens=64, heads=8, dim=128, dtype="bf16", pad=3),
        # a batch of prompts: the bytes
        dict(app, name="append_8192_tokens_32_heads", tokens=8192, heads=32, dim=128, dtype="fp16", pad=0),
        # one short sequence, small heads: latency
        dict(att, name="decode_1x700_dim64", batch=1, q=1, heads=16, kv_heads=16, dim=64, length=700,
             spread=0.0, dtype="fp16", page=16),
        # a decode batch of ragged lengths, one key head for each query head
        dict(att, name="decode_16x2048_32_heads", batch=16, q=1, heads=32, kv_heads=32, dim=128, length=2048,
             spread=0.6, dtype="fp16"),
        # few long sequences, eight query heads to a key head: the long axis has to be split
        dict(att, name="decode_4x32768_64_8_heads", batch=4, q=1, heads=64, kv_heads=8, dim=128, length=32768,
             spread=0.3, dtype="bf16"),
        # a few drafted tokens a sequence over ragged lengths, one sequence empty
        dict(att, name="verify_8x5x4001_64_8_heads", batch=8, q=5, heads=64, kv_heads=8, dim=128, length=4001,
             spread=0.9, dtype="bf16", page=32, empty=True),
        # two prompts: the matrix cores
        dict(att, name="prefill_2x4096_32_heads", batch=2, q=4096, heads=32, kv_heads=32, dim=128, length=4096,
             spread=0.25, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes over the listed cases' ranges, odd ones among them."""
    dtype = rng.choice(["fp16", "bf16"])
    op = rng.choice(["linear", "linear", "append", "attention", "attention"])
    if op == "linear":
        m, k, n = _log(rng, 1, 4096), _log(rng, 64, 11008), _log(rng, 64, 28672)
        if rng.random() < 0.5:
            k = max(128, k // 128 * 128)
        while m * k * n > 4e11:
            m = (m + 1) // 2
        return dict(op=op, m=m, k=k, n=n, dtype=dtype, bias=rng.random() < 0.5)
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    if op == "append":
        heads = rng.choice([1, 2, 4, 8, 12, 32])
        tokens = _log(rng, 1, 8192 * 32 * 128 // (heads * dim) if heads * dim > 4096 else 8192)
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, page=page, dtype=dtype,
                    pad=rng.randrange(0, 4) if tokens > 8 else 0)
    kv_heads, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4, 5, 8])
    q = rng.choice([1, 1, rng.randrange(2, 9), _log(rng, 9, 2048)])
    length = max(q, _log(rng, 1, 32768 if q < 9 else 4096))
    batch = _log(rng, 1, 32)
    while batch > 1 and (batch * kv_heads * length * dim > 1 << 27 or batch * kv_heads * group * q * length > 1 << 29):
        batch //= 2
    while kv_heads * group * q * length > 1 << 29:
        q //= 2
    return dict(op=op, batch=batch, q=q, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page,
                length=length, spread=rng.choice([0.0, 0.3, 0.9]), dtype=dtype, empty=batch > 2 and rng.random() < 0.3)


def _sequences(case):
    """(key lengths, query tokens) of each sequence: whole numbers spread below the largest."""
    b = case["batch"]
    lens = [max(1, int(case["length"] * (1 - case["spread"] * i / b))) for i in range(b)]
    count = [max(1, int(case["q"] * (1 - case["spread"] * i / b))) for i in range(b)]
    count = [min(c, n) for c, n in zip(count, lens)]
    if case["empty"]:
        lens[-1] = 0
    return lens, count


# ----------------------------------------------------------------------------- inputs
def _spread_slots(g, tokens, page, pages):
    """Slots of consecutive tokens that start inside a page, over shuffled pages."""
    order = torch.randperm(pages, generator=g, device="cuda")
    at = torch.arange(tokens, device="cuda") + page // 2 + 1
    return order[at // page] * page + at % page


def _quantize_heads(x):
    """Codes, zero points and scales (fp32 values) of x [..., dim], one scale a row."""
    lo, hi = x.amin(-1, keepdim=True).clamp(max=0.0), x.amax(-1, keepdim=True).clamp(min=0.0)
    s = ((hi - lo) / torch.full_like(lo, 15.0)).clamp(max=65504.0).half().float()
    safe = torch.where(s > 0, s, torch.ones_like(s))
    zero = torch.round(-lo / safe).clamp(0, 15)
    q = (torch.round(x / safe) + zero).clamp(0, 15)
    return torch.where(s > 0, q, 0.0), torch.where(s > 0, zero, 0.0), s


def _pack_pairs(q):
    """[..., 2n] codes -> [..., n] bytes, the even code in the low nibble."""
    q = q.to(torch.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4)


def _store(cache, q, zero, s, slots, values):
    """Codes [tokens, heads, dim] and parameters into the slots of one side of the cache."""
    codes, par = cache
    page = par.shape[2]
    ok = slots >= 0
    p, t = slots[ok] // page, slots[ok] % page
    rows = _pack_pairs(q[ok])                               # [n, heads, dim / 2]
    if values:                                              # [P, H, T / 4, D / 4, 2, 2, 2 bytes]
        at = codes.view(*codes.shape[:4], 4, 2)
        at[p, :, t // 4, :, t % 4] = rows.view(rows.shape[0], rows.shape[1], -1, 2)
    else:
        codes[p, :, t] = rows
    par[p, :, t] = torch.cat([zero[ok], s[ok]], -1).half()


def _empty_cache(g, pages, page, heads, dim):
    """Pages as a pool holds them: what earlier sequences left, here any bits at all."""
    def raw(*shape):
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)

    k, v = raw(pages, heads, page, dim // 2), raw(pages, heads, page // 4, dim // 4, 8)
    kp = raw(pages, heads, page, 4).view(torch.float16)
    vp = raw(pages, heads, page, 4).view(torch.float16)
    return k, kp, v, vp


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        x = normal(m, k)
        x[:, torch.randint(0, k, (max(1, k // 100),), generator=g, device="cuda")] *= 20.0   # outlier channels
        w = normal(n, k).mul_(0.02)
        s = (w.abs().amax(1, keepdim=True) / torch.full((n, 1), 127.0, device="cuda"))
        codes = torch.zeros(n, -(-k // 128) * 128, dtype=torch.int8, device="cuda")          # rows padded with zeros
        codes[:, :k] = torch.round(w.div_(s)).clamp_(-127, 127)
        return dict(case=case, x=x.to(dtype), w=codes, sw=s[:, 0].contiguous(),
                    bias=normal(n).to(dtype) if case["bias"] else None)
    dim, page = case["dim"], case["page"]
    if case["op"] == "append":
        tokens, heads = case["tokens"], case["heads"]
        pages = tokens // page + 4
        slots = _spread_slots(g, tokens, page, pages)
        slots[tokens - case["pad"]:] = -1                                                    # a padded batch's tail
        # keys carry a few large channels, values do not
        gain = 1.0 + 7.0 * (torch.rand(heads, dim, generator=g, device="cuda") < 0.04)
        qkv = torch.cat([normal(tokens, heads * dim) * gain.view(-1), normal(tokens, heads * dim)], 1).to(dtype)
        key, value = (t.view(tokens, heads, dim) for t in qkv.split(heads * dim, 1))         # views of one projection
        return dict(case=case, key=key, value=value, slots=slots, cache=_empty_cache(g, pages, page, heads, dim))
    lens, count = _sequences(case)
    b, kv = case["batch"], case["kv_heads"]
    width = -(-max(case["length"], 1) // page)
    pages = b * width
    table = torch.randperm(pages, generator=g, device="cuda").view(b, width).int()
    cache = _empty_cache(g, pages, page, kv, dim)
    gain = 1.0 + 7.0 * (torch.rand(kv, dim, generator=g, device="cuda") < 0.04)
    for i in range(b):
        if lens[i]:
            at = torch.arange(lens[i], device="cuda")
            slots = table[i].long()[at // page] * page + at % page
            for side, x in ((0, normal(lens[i], kv, dim) * gain), (2, normal(lens[i], kv, dim))):
                _store(cache[side:side + 2], *_quantize_heads(x), slots, side == 2)
    total = sum(count)
    start = torch.tensor([sum(count[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
    q = (normal(total, case["heads"], dim) / gain.repeat_interleave(case["heads"] // kv, 0)).to(dtype)
    return dict(case=case, q=q, cache=cache, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                start=start, max_q=max(count), max_len=max(max(lens), 1), total=total)


# ----------------------------------------------------------------------------- plain forms
def _codes(cache, values):
    """Codes [P, H, T, D] of one side as integers."""
    c = cache[0]
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    if not values:
        return c
    p, h, blocks, quads, _ = c.shape                        # [P, H, T / 4, D / 4, 16]
    return c.view(p, h, blocks, quads, 4, 4).transpose(3, 4).reshape(p, h, blocks * 4, quads * 4)


def _linear(s):
    x = s["x"].float()
    a = x.abs().amax(1, keepdim=True)
    sx = a / torch.full_like(a, 127.0)
    q = torch.round(x / torch.where(sx > 0, sx, torch.ones_like(sx))).clamp(-127, 127)
    y = (q @ s["w"][:, :x.shape[1]].float().t()) * sx * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


def _append(s):
    out = []
    ok = (s["slots"] >= 0).view(-1, 1, 1)
    for side, x in ((0, s["key"]), (2, s["value"])):
        q, zero, scale = _quantize_heads(x.float())
        _store(s["cache"][side:side + 2], q, zero, scale, s["slots"], side == 2)
        out.append(torch.where(ok, (q - zero) * scale, 0.0).to(x.dtype))
    return out


def _dense(cache, table, values):
    """One side of the cache as fp32 [B, H, L, D], by the sequences' pages."""
    par = cache[1][table].float()                           # [B, W, H, T, 2]
    c = _codes((cache[0][table].flatten(0, 1),), values).view(*par.shape[:4], -1)
    x = (c.float() - par[..., :1]) * par[..., 1:]
    return x.transpose(1, 2).flatten(2, 3)


def _attention(s):
    c, table, lens, start = s["case"], s["table"].long(), s["lens"].long(), s["start"].long()
    b, kv, dim, most = c["batch"], c["kv_heads"], c["dim"], s["max_q"]
    group = c["heads"] // kv
    # queries padded to [B, kv, most * group, dim]
    at = start[:-1, None] + torch.arange(most, device="cuda")
    real = at < start[1:, None]
    q = s["q"].float()[at.clamp(max=s["total"] - 1)].view(b, most, kv, group, dim).permute(0, 2, 1, 3, 4)
    key, value = _dense(s["cache"][:2], table, False), _dense(s["cache"][2:], table, True)
    t = torch.arange(key.shape[2], device="cuda")
    inside = t < lens[:, None]                              # what lies behind a sequence's end is no number
    key = torch.where(inside[:, None, :, None], key, 0.0)
    value = torch.where(inside[:, None, :, None], value, 0.0)
    score = (q.reshape(b, kv, most * group, dim) @ key.transpose(2, 3)).mul_(dim ** -0.5).view(b, kv, most, group, -1)
    place = lens[:, None] - (start[1:] - start[:-1])[:, None] + torch.arange(most, device="cuda")
    seen = t <= place[:, :, None]                           # [B, most, L]
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    w = score.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    out = (w.view(b, kv, most * group, -1) @ value).view(b, kv, most, group, dim) / total.clamp(min=1e-30)
    return out.permute(0, 2, 1, 3, 4).reshape(b, most, c["heads"], dim)[real].to(s["q"].dtype)


def run(state):
    op = state["case"]["op"]
    if own:
        import bit_quantized_gemm_amd as bq

        if op == "linear":
            return bq.linear_w8a8(state["x"], state["w"], state["sw"], bias=state["bias"])
        if op == "append":
            bq.atom_kv4_append(state["key"], state["value"], state["slots"], state["cache"])
            return bq.atom_kv4_read(state["cache"], state["slots"], dtype=state["key"].dtype)
        return bq.atom_kv4_attention(state["q"], state["cache"], state["table"], state["lens"], state["start"],
                                     max_len=state["max_len"], max_q=state["max_q"])
    return {"linear": _linear, "append": _append, "attention": _attention}[op](state)


def work(case):
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * k + n * k + 4 * n + 2 * m * n + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    dim = case["dim"]
    if case["op"] == "append":
        rows = case["tokens"] * case["heads"] * 2           # key and value rows
        # read as fp16, write codes and parameters, read them, write the values
        return {"bytes": rows * (2 * dim + 2 * (dim // 2 + 4) + 2 * dim) + 16 * case["tokens"], "flops": 0}
    lens, count = _sequences(case)
    cache = sum(lens) * case["kv_heads"] * 2 * (dim // 2 + 4)
    rows = 2 * 2 * sum(count) * case["heads"] * dim
    pairs = sum(sum(max(0, n - c + i + 1) for i in range(c)) for n, c in zip(lens, count)) * case["heads"]
    return {"bytes": cache + rows, "flops": 4 * pairs * dim}


# ----------------------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x = s["x"].double()
        sx = (x.abs().max(1).values.float() / torch.tensor(127.0, device="cuda").expand(case["m"])).double()
        q = torch.where(sx[:, None] > 0, x / sx[:, None], 0.0).round()
        y = torch.mm(q, s["w"][:, :case["k"]].double().mT)
        y *= torch.outer(sx, s["sw"].double())
        return y if s["bias"] is None else y + s["bias"].double()[None]
    if case["op"] == "append":
        out = []
        for x in (s["key"].double(), s["value"].double()):
            least = torch.minimum(x.min(2).values, torch.zeros((), dtype=x.dtype, device="cuda"))
            step = (torch.maximum(x.max(2).values, torch.zeros_like(least)) - least) / 15
            step = step.half().double()[..., None]
            z = torch.nan_to_num(-least[..., None] / step, 0.0).round().clamp(0, 15)
            code = torch.nan_to_num(x / step, 0.0).round() + z
            v = (code.clamp(0, 15) - z) * step
            v[s["slots"] < 0] = 0
            out.append(v)
        return out
    lens, count = _sequences(case)
    k, kp, v, vp = s["cache"]
    page, dim, group = case["page"], case["dim"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s["total"], case["heads"], dim, dtype=torch.float64, device="cuda")
    d = torch.arange(dim, device="cuda")
    first = 0
    for i, (n, c) in enumerate(zip(lens, count)):
        if n:
            t = torch.arange(n, device="cuda")
            p, r = s["table"][i].long()[t // page], t % page
            for h in range(case["kv_heads"]):
                byte = k[p, h, r].long()
                code = (byte[:, d // 2] >> (4 * (d % 2))) & 15
                par = kp[p, h, r].double()
                key = (code - par[:, :1]) * par[:, 1:]
                byte = v[p, h, r // 4].long()               # [n, dim / 4, 8]
                at = (2 * (r % 4))[:, None] + (d % 4) // 2
                code = (byte[t[:, None], (d // 4)[None], at] >> (4 * (d % 2))) & 15
                par = vp[p, h, r].double()
                value = (code - par[:, :1]) * par[:, 1:]
                q = s["q"][first:first + c, h * group:(h + 1) * group].double()
                a = torch.tensordot(q, key, ([2], [1])) / math.sqrt(dim)                     # [c, group, n]
                hidden = t[None] > (n - c + torch.arange(c, device="cuda"))[:, None]
                a = torch.softmax(a.masked_fill(hidden[:, None], -math.inf), -1)
                a = torch.nan_to_num(a, 0.0)
                out[first:first + c, h * group:(h + 1) * group] = torch.tensordot(a, value, ([2], [0]))
        first += c
    return out
