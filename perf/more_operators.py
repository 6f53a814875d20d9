"""More serving operators, as measured cases.

Operators of quantized LLM serving that stand around the W4A4 and W8A8 layers and the 4-bit KV cache, each in its
plain form (elementary torch operations in 32 bits, in 64 where a value next to the border of two codes decides, rounded once at
the end) and as a call of this package:

* ``linear``   linear layer in microscaled 4-bit floating point (MXFP4) on both sides, optional bias.
* ``norm``     root-mean-square norm, with the residual's addition in front and the rows quantized behind it: to int8
               with one scale a row (``w8``), the W8A8 layer's operand, or to MXFP4 (``mx``), the layer above's.
* ``extend``   the tokens that a step adds to each sequence: pages taken from a pool, the block table continued, and the
               slot of each token.
* ``release``  the pages of finished sequences given back to the pool.

MXFP4: blocks of 32 values of a row share a scale 2^e, e = floor(log2(max |x|)) - 2; a value is the nearest of 0, 0.5, 1, 1.5,
2, 3, 4, 6 times the scale (ties to the even code, larger ones 6), with its sign in bit 3 of a 4-bit code.  Rows are
padded with zeros to whole groups of 256; two codes a byte, the even one in the low nibble; scales are bytes e + 127, in an
array [groups, rows, 8].
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    """Cases: sizes of the Llama-7B and Llama-70B layers that this repository measures, a tiny one, and odd ones."""
    lin = dict(op="linear", bias=False)
    norm = dict(op="norm", residual=True)
    return [
        # one token through an attention projection: latency
        dict(lin, name="linear_1x4096x4096", m=1, k=4096, n=4096, dtype="fp16"),
        # a decode batch through the MLP's gate: the weights' bytes
        dict(lin, name="linear_16x4096x11008", m=16, k=4096, n=11008, dtype="bf16"),
        # odd sizes, with a bias: rows that no vector load fits, a block that ends inside a row
        dict(lin, name="linear_333x1155x777_bias", m=333, k=1155, n=777, dtype="fp16", bias=True),
        # the MLP's second product for a batch of prompts: the matrix cores
        dict(lin, name="linear_2048x11008x4096", m=2048, k=11008, n=4096, dtype="fp16"),
        # the largest: a Llama-70B MLP
        dict(lin, name="linear_4096x8192x28672", m=4096, k=8192, n=28672, dtype="bf16"),
        # a decode batch between two layers: latency
        dict(norm, name="norm_16x4096_w8", m=16, k=4096, to="w8", dtype="fp16"),
        # the first norm of a model (nothing to add yet), odd rows
        dict(norm, name="norm_333x1155_mx", m=333, k=1155, to="mx", dtype="fp16", residual=False),
        # a batch of prompts: the bytes
        dict(norm, name="norm_8192x8192_mx", m=8192, k=8192, to="mx", dtype="bf16"),
        # a decode step: one token for each sequence, latency
        dict(op="extend", name="extend_64_decode", batch=64, page=64, width=64, length=4000, most=1, pad=0, short=False),
        # ragged prompts for sequences that hold some tokens already, a padded batch
        dict(op="extend", name="extend_256_prompts", batch=256, page=16, width=256, length=2000, most=1800, pad=1000,
             short=False),
        # a few sequences of a decode batch end
        dict(op="release", name="release_64", batch=64, page=64, width=64, length=4000, done=0.1),
        # a large batch of long sequences is cleared out, small pages
        dict(op="release", name="release_1024", batch=1024, page=16, width=512, length=8000, done=0.7),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes over the listed cases' ranges, odd ones among them."""
    op = rng.choice(["linear", "linear", "linear", "norm", "norm", "extend", "release"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "linear":
        m, k, n = _log(rng, 1, 4096), _log(rng, 32, 11008), _log(rng, 32, 28672)
        if rng.random() < 0.5:
            k = max(128, k // 128 * 128)
        while m * k * n > 9e11:
            m = (m + 1) // 2
        return dict(op=op, m=m, k=k, n=n, dtype=dtype, bias=rng.random() < 0.5)
    if op == "norm":
        m, k = _log(rng, 1, 8192), _log(rng, 32, 16384)
        if rng.random() < 0.5:
            k = max(128, k // 128 * 128)
        while m * k > 8192 * 8192:
            m = (m + 1) // 2
        return dict(op=op, m=m, k=k, to=rng.choice(["w8", "mx"]), dtype=dtype, residual=rng.random() < 0.7)
    batch, page = _log(rng, 1, 1024), rng.choice([16, 32, 64, 128, 256])
    length = _log(rng, 1, 8000)
    if op == "release":
        while batch * length > 1 << 23:
            batch //= 2
        return dict(op=op, batch=batch, page=page, width=length // page + rng.randrange(1, 9), length=length,
                    done=rng.choice([0.1, 0.5, 1.0]))
    most = rng.choice([1, rng.randrange(2, 9), _log(rng, 9, 2000)])
    while batch * most > 1 << 19:
        batch //= 2
    return dict(op=op, batch=batch, page=page, width=(length + most) // page + rng.randrange(1, 9), length=length, most=most,
                pad=rng.choice([0, rng.randrange(1, 500)]), short=rng.random() < 0.1)


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] in ("linear", "norm"):
        dtype, m, k = DTYPES[case["dtype"]], case["m"], case["k"]
        x = normal(m, k)
        x[:, torch.randint(0, k, (max(1, k // 100),), generator=g, device="cuda")] *= 20.0       # outlier channels
        s = dict(case=case, x=x.to(dtype))
        if case["op"] == "linear":
            s["w"], s["sw"] = _pack(*_blocks(normal(case["n"], k).mul_(0.02)))
            s["bias"] = normal(case["n"]).to(dtype) if case["bias"] else None
        else:
            s["weight"] = normal(k).mul_(0.3).add_(1.0).to(dtype)
            s["residual"] = normal(m, k).mul_(3.0).to(dtype) if case["residual"] else None
        return s
    batch, page, width, length = (case[n] for n in ("batch", "page", "width", "length"))

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)

    lens = whole(0, length, batch)
    held = (lens + page - 1) // page                                   # pages of each sequence
    pages = batch * width + 64
    order = torch.randperm(pages, generator=g, device="cuda").int()
    inside = torch.arange(width, device="cuda") < held[:, None]
    # behind a sequence's pages the table holds what earlier ones left
    table = torch.where(inside, order[:batch * width].view(batch, width), whole(-9, pages, batch, width)).contiguous()
    free = torch.cat([order[batch * width:], order[:batch * width][~inside.view(-1)]])
    state = torch.zeros(2, dtype=torch.int32, device="cuda")
    state[0] = free.numel()
    free = torch.cat([free, torch.full((pages - free.numel(),), -1, dtype=torch.int32, device="cuda")])
    s = dict(case=case, lens=lens, table=table, free=free, state=state)
    if case["op"] == "release":
        s["done"] = torch.rand(batch, generator=g, device="cuda") < case["done"]
        return s
    tokens = batch * (case["most"] + 1) // 2
    end = torch.cumsum(whole(1, case["most"], batch), 0).double()
    end = (end * tokens / end[-1].clone()).floor().int()                # shares of the step's tokens
    s["new"] = torch.diff(end, prepend=end.new_zeros(1))
    s["total"] = tokens + case["pad"]
    if case["short"]:
        state[0] = 0
    return s


# ----------------------------------------------------------------------------- plain forms
def _power(e, dtype):
    """2^e exactly, for whole numbers e of normal results."""
    if dtype is torch.float64:
        return ((e.long() + 1023) << 52).view(torch.float64)
    return ((e.int() + 127) << 23).view(torch.float32)


def _blocks(x):
    """(values with their signs in units of the scale [rows, blocks, 32], exponents [rows, blocks]) of rows."""
    rows, k = x.shape
    x = torch.nn.functional.pad(x, (0, -k % 256)).view(rows, -1, 32)
    top = x.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 125)
    u = x * _power(-e, x.dtype)[..., None]
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(x.dtype)
    return torch.copysign(((a / step).round() * step).clamp(max=6.0), u), e


def _pack(v, e):
    """Codes [rows, bytes] and scales [groups, rows, 8] of what _blocks gives."""
    rows = v.shape[0]
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.view(rows, -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8).view(rows, -1, 8).transpose(0, 1).contiguous()


def _values(codes, scales):
    """What packed rows stand for, in fp32 (with the zeros behind their ends)."""
    rows = codes.shape[0]
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()].view(rows, -1, 32)
    e = scales.transpose(0, 1).reshape(rows, -1).int() - 127
    return (v * _power(e.clamp(min=-126), torch.float32)[..., None]).view(rows, -1)


def _linear(s):
    v, e = _blocks(s["x"].float())
    x = (v * _power(e.clamp(min=-126), torch.float32)[..., None]).flatten(1)
    y = x @ _values(s["w"], s["sw"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


def _norm(s):
    c, dtype = s["case"], s["x"].dtype
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dtype)
    # in 64 bits: a value's code and a block's exponent turn over at borders that 32 bits put on either side
    d = h.double()
    y = d * s["weight"].double() / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)
    if c["to"] == "w8":
        scale = (y.abs().amax(1, keepdim=True) / 127).float()
        safe = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
        q = torch.round(y / safe).clamp(-127, 127)
        out = [(q.float() * scale).to(dtype), scale[:, 0]]
    else:
        v, e = _blocks(y)
        out = [(v * _power(e, torch.float64)[..., None]).flatten(1)[:, :c["k"]].to(dtype)]
    return out if s["residual"] is None else out + [h]


def _exclusive(n):
    """Sums in front of each entry, and the sum of all."""
    c = torch.cumsum(n, 0)
    return c - n, c[-1]


def _extend(s):
    c, table, free = s["case"], s["table"], s["free"]
    page, width, total = c["page"], c["width"], s["total"]
    most = width * page
    lens = s["lens"].long().clamp(0, most)
    end = torch.cumsum(s["new"].long().clamp(min=0), 0).clamp(max=total)
    start = torch.nn.functional.pad(end, (1, 0))
    after = (lens + start[1:] - start[:-1]).clamp(max=most)
    have, want = (lens + page - 1) // page, (after + page - 1) // page
    first, needed = _exclusive(want - have)
    pool = s["state"][0].long().clamp(0, free.numel())
    fits = needed <= pool
    col = torch.arange(width, device=table.device)
    fresh = (col >= have[:, None]) & (col < want[:, None]) & fits
    at = pool - 1 - (first[:, None] + col - have[:, None])
    table.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table))
    row = torch.arange(total, device=table.device)
    b = torch.searchsorted(end, row, right=True).clamp(max=c["batch"] - 1)
    t = lens[b] + row - start[b]
    p = table[b, (t // page).clamp(0, width - 1)].long()
    slots = torch.where((row < end[-1]) & (t < most) & fits & (p >= 0), p * page + t % page, -1)
    state = torch.stack([torch.where(fits, pool - needed, pool), torch.where(fits, 0, needed - pool)])
    return [slots, start.int(), torch.where(fits, after, lens).int(), state.int(), table]


def _release(s):
    c, table, free = s["case"], s["table"], s["free"]
    page, width = c["page"], c["width"]
    lens = s["lens"].long().clamp(0, width * page)
    n = torch.where(s["done"], (lens + page - 1) // page, 0)
    first, given = _exclusive(n)
    pool = s["state"][0].long().clamp(0, free.numel())
    col = torch.arange(width, device=table.device)
    to = pool + first[:, None] + col
    to = torch.where((col < n[:, None]) & (to < free.numel()), to, free.numel())       # the others: one place behind the end
    grown = torch.nn.functional.pad(free, (0, 1))
    grown[to.view(-1)] = table.view(-1)
    free.copy_(grown[:-1])
    state = torch.stack([(pool + given).clamp(max=free.numel()), torch.zeros_like(pool)])
    return [torch.where(s["done"], 0, lens).int(), state.int(), free]


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import bit_quantized_gemm_amd as bq

        if op == "linear":
            return bq.linear_mxfp4(state["x"], state["w"], state["sw"], bias=state["bias"])
        if op == "norm":
            call, read = ((bq.atom_rmsnorm_w8a8, bq.atom_dequantize_w8a8) if c["to"] == "w8" else
                          (bq.atom_rmsnorm_mxfp4, bq.atom_dequantize_mxfp4))
            xq, sx, h = call(state["x"], state["weight"], EPS, residual=state["residual"])
            out = [read(xq, sx, c["k"], dtype=state["x"].dtype)] + ([sx] if c["to"] == "w8" else [])
            return out if h is None else out + [h]
        pool = bq.KV4Pool(state["free"], state["state"])
        if op == "extend":
            return [*bq.atom_kv4_extend(state["lens"], state["new"], state["table"], pool, c["page"], state["total"]),
                    state["table"]]
        return [*bq.atom_kv4_release(state["done"], state["lens"], state["table"], pool, c["page"]), state["free"]]
    return {"linear": _linear, "norm": _norm, "extend": _extend, "release": _release}[op](state)


def work(case):
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * k + n * k // 2 + n * -(-k // 32) + 2 * m * n + (2 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        codes = m * k + 4 * m if case["to"] == "w8" else m * (k // 2) + m * -(-k // 32)
        # the row (and the residual, and their sum out), the codes out, read again, their values out
        return {"bytes": 2 * m * k * (3 if case["residual"] else 1) + 2 * k + 2 * codes + 2 * m * k, "flops": 0}
    batch, page = case["batch"], case["page"]
    if case["op"] == "extend":
        tokens = batch * (case["most"] + 1) // 2
        # the lengths in and out, the new counts, the starts; a page out of the pool and into the table; the slots
        return {"bytes": 16 * batch + 8 * (tokens // page) + 4 * batch + 8 * (tokens + case["pad"]), "flops": 0}
    return {"bytes": 9 * batch + 8 * int(case["done"] * batch * (case["length"] / 2 / page)) + 16, "flops": 0}


# ----------------------------------------------------------------------------- definitions in 64 bits
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _microscaled(x):
    """fp64 rows [rows, k] to the values that their MXFP4 codes stand for."""
    rows, k = x.shape
    pad = torch.zeros(rows, -(-k // 32) * 32, dtype=torch.float64, device=x.device)
    pad[:, :k] = x
    b = pad.view(rows, -1, 32)
    top = b.abs().max(2, keepdim=True).values
    e = torch.floor(torch.log2(top.clamp(min=1e-300)))
    e += (torch.exp2(e + 1) <= top).double() - (torch.exp2(e) > top).double()      # log2 next to a power of two
    scale = torch.exp2((e - 2).clamp(-127, 125))
    u = b / scale
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    a = u.abs()
    up, down = torch.bucketize(a, middle, right=True), torch.bucketize(a, middle)   # these differ on a border alone
    code = torch.where(up % 2 == 0, up, down)
    return (grid[code] * torch.sign(u) * scale).view(rows, -1)[:, :k]


def exact(case, seed):
    if case["op"] not in ("linear", "norm"):
        return None
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "linear":
        byte = s["w"].long()
        code = torch.stack([byte % 16, byte // 16], 2).flatten(1)[:, :case["k"]]
        e = s["sw"].permute(1, 0, 2).flatten(1).double() - 127
        grid = torch.tensor(_GRID, dtype=torch.float64, device="cuda")
        w = grid[code % 8] * (1 - 2 * (code // 8)) * torch.exp2(e).repeat_interleave(32, 1)[:, :case["k"]]
        y = torch.mm(_microscaled(x), w.t().contiguous())
        return y if s["bias"] is None else y + s["bias"].double()[None]
    total = x if s["residual"] is None else x + s["residual"].double()
    h = total.to(s["x"].dtype).double()
    y = h * torch.rsqrt((h * h).sum(1) / case["k"] + EPS)[:, None] * s["weight"].double()
    if case["to"] == "w8":
        step = (y.abs().max(1).values / 127.0).float().double()
        out = [torch.nan_to_num(y / step[:, None], 0.0).round() * step[:, None], step]
    else:
        out = [_microscaled(y)]
    return out if s["residual"] is None else out + [total]
