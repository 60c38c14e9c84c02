"""Operators around the sparse MLA attention's cache: cases and plain forms for measuring.

Four operators, as a serving program that prefills with this library uses them:

  rope   ds4sp_rope: rotary positions of part of each head (interleaved or half layout,
         linear / NTK / YaRN scaling for long contexts), and the transposed rotation, its
         gradient;
  cache  ds4sp_cache_write then ds4sp_cache_read: latent rows rotated, quantized and written
         to a cache as they are produced, and the rows of the blocks it touched read back;
  read   ds4sp_cache_read: rows of a cache gathered by index and dequantized;
  attn   ds4sp_sparse_attn over a cache of 8-bit rows with a scale for each block of 64
         tokens (kv_format 5): a prefill, and the calls of one token or a few.

``listed()`` and ``draw()`` give cases, ``prepare()`` the inputs a program has in hand,
``run()`` one pass: with ``own`` false the plain form in elementary torch operations, with
``own`` true the library's calls. ``exact()`` is the same result in 64 bits, from the
definitions. ``work()`` is what a pass has to read, write and compute.
"""
import math

import torch

own = False

D_QK, D_V, D_ROPE, HEADS = 576, 512, 64, 16   # a latent row: 512 latent + 64 rotary dims
BLOCK = 64                                    # rows that share a scale in kv_format 5
F16, Q8, Q4, Q8Q4, E4M3 = 0, 1, 2, 3, 5       # kv_format of a cache
CONTEXT = 122880                              # the long-context workload
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
NONE, LINEAR, NTK, YARN = 0, 1, 2, 3          # scaling of the rotary frequencies


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The rotary part of the queries of a 5-token verify step at a 122,880-token
        # context: read from the query projection, written beside the absorbed part.
        _rope("rope_verify", n=5, heads=16, width=192, head=64, into=576, scaling=YARN, factor=32.0,
              pos0=CONTEXT - 5),
        # The same of a whole 10,240-token prefill.
        _rope("rope_prefill", n=10240, heads=16, width=192, head=64, into=576, layout=1, scaling=YARN,
              factor=32.0),
        # Gradient of the indexer queries' rotation (64 of 128 dims, 64 heads), bf16.
        _rope("rope_index_grad", n=10240, heads=64, width=128, head=128, offset=64, dtype="bf16",
              scaling=NTK, factor=8.0, transpose=True),
        # One decoded token's row appended inside a block at a long context.
        _cache("append_token", fmt=E4M3, n=1, row0=122843),
        # A ragged chunk of compressed rows (every fourth position) that starts inside a block.
        _cache("write_ragged", fmt=E4M3, n=1777, row0=1003, dtype="fp32", pos_step=4),
        # The raw rows of a whole long context, bf16 from the projection.
        _cache("write_context", fmt=E4M3, n=CONTEXT, row0=0, dtype="bf16"),
        # The rows that five verify tokens select, gathered from a long cache as fp16.
        _read("read_selected", fmt=E4M3, rows=30720, n=5 * 512, gather=True),
        # A whole 10K prefill's Q8 K / Q4 V cache, read back as bf16.
        _read("read_cache", fmt=Q8Q4, rows=10240, n=10240, gather=False, dtype="bf16"),
        # One decoded token, five verified ones, one 2,048-token band, a 10,240-token prefill.
        _attn("attn_token", n=1, t0=CONTEXT - 1, k=512, n_swa=128),
        _attn("attn_verify", n=5, t0=CONTEXT - 5, k=512, n_swa=128),
        _attn("attn_band", n=2048, t0=0, k=128, n_swa=128),
        _attn("attn_prefill", n=10240, t0=0, k=512, n_swa=128),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    op = rng.choice(("rope", "cache", "read", "attn"))
    if op == "rope":
        dims = 2 * rng.randint(2, 64)
        offset = rng.choice((0, rng.randint(0, 70)))
        head = dims + offset + rng.choice((0, rng.randint(0, 64)))
        heads = rng.choice((1, 16, 64, rng.randint(1, 64)))
        n = min(log(1, 16384), max(1, 10240 * 64 * 128 // (heads * head)))
        scaling = rng.choice((NONE, LINEAR, NTK, YARN))
        return _rope(None, n=n, heads=heads, width=head + rng.choice((0, 64, rng.randint(0, 99))), head=head,
                     into=rng.choice((0, head + 8 * rng.randint(0, 64))), dims=dims, offset=offset,
                     layout=rng.randint(0, 1), dtype=rng.choice(("fp16", "bf16", "fp32")), scaling=scaling,
                     factor=1.0 if scaling == NONE else rng.uniform(1.5, 40.0), pos0=rng.randint(0, 1 << 20),
                     listed_positions=rng.random() < 0.5, transpose=rng.random() < 0.4)
    if op == "cache":
        fmt = rng.choice((F16, Q8, Q4, Q8Q4, E4M3, E4M3))
        n = log(1, CONTEXT)
        return _cache(None, fmt=fmt, n=n, row0=rng.randint(0, CONTEXT - n), rope=fmt != Q4,
                      dtype=rng.choice(("fp16", "bf16", "fp32")) if n <= CONTEXT // 2 else "fp16",
                      pos_step=rng.choice((1, 4)))
    if op == "read":
        rows = log(1, CONTEXT)
        gather = rng.random() < 0.6
        return _read(None, fmt=rng.choice((F16, Q8, Q4, Q8Q4, E4M3, E4M3)), rows=rows, gather=gather,
                     n=log(1, 40000) if gather else rows, dtype=rng.choice(("fp16", "bf16", "fp32")))
    n = log(1, 10240)
    k, n_swa = rng.choice((0, 512, rng.randint(1, 1200))), rng.choice((1, 128, rng.randint(2, 300)))
    n = max(1, min(n, 10240 * 640 // (k + n_swa)))
    return _attn(None, n=n, t0=rng.choice((0, rng.randint(0, CONTEXT - n))), k=k, n_swa=n_swa)


def _case(name, **kw):
    return kw if name is None else dict(name=name, **kw)


def _rope(name, n, heads, width, head, into=0, dims=64, offset=0, layout=0, dtype="fp16", scaling=NONE,
          factor=1.0, pos0=0, listed_positions=False, transpose=False):
    """n tokens x heads of `head` values (the last of `width` in the source), of which
    [offset, offset + dims) are rotated; into: width of a head of the tensor whose last
    `head` values they are written to, or 0 for a tensor of their own."""
    return _case(name, op="rope", n=n, heads=heads, width=width, head=head, into=into, dims=dims, offset=offset,
                 layout=layout, dtype=dtype, scaling=scaling, factor=factor, pos0=pos0,
                 listed_positions=listed_positions, transpose=transpose)


def _cache(name, fmt, n, row0, dtype="fp16", rope=True, pos_step=1):
    return _case(name, op="cache", fmt=fmt, n=n, row0=row0, dtype=dtype, rope=rope, pos_step=pos_step)


def _read(name, fmt, rows, n, gather, dtype="fp16"):
    return _case(name, op="read", fmt=fmt, rows=rows, n=n, gather=gather, dtype=dtype)


def _attn(name, n, t0, k, n_swa):
    return _case(name, op="attn", n=n, t0=t0, k=k, n_swa=n_swa)


def _rope_of(case):
    """The rotary settings of a case (ds4sp_rope_config's fields)."""
    if case["op"] == "rope":
        return dict(dims=case["dims"], offset=case["offset"], layout=case["layout"], base=10000.0,
                    scaling=case["scaling"], factor=case["factor"], orig_len=4096)
    return dict(dims=D_ROPE, offset=D_QK - D_ROPE, layout=0, base=10000.0, scaling=YARN, factor=32.0,
                orig_len=4096)


# ------------------------------------------------------------------ cache formats

def _cache_row(fmt):
    """Bytes of a stored row of 576 values."""
    return {F16: 1152, Q8: 624, Q4: 336, Q8Q4: 912, E4M3: 576}[fmt]


def _place(rows):
    """kv_format 5: the stored place of a row; each 64 rows are followed by their scale's record."""
    return rows + rows // BLOCK


def _quant_blocks(x, fmt):
    """fp32 [..., 32 m] -> codes and fp16 scales of each block of 32."""
    v = x.reshape(*x.shape[:-1], -1, 32)
    if fmt == Q8:
        d = (v.abs().amax(-1) / torch.full((), 127.0, device=x.device)).half()
    else:
        at = torch.arange(32, device=x.device)              # the first of equal extremes
        first = torch.where(v.abs() == v.abs().amax(-1, keepdim=True), at, 32).amin(-1, keepdim=True)
        d = (v.gather(-1, first).squeeze(-1) / torch.full((), -8.0, device=x.device)).half()
        d = torch.where(d == 0, torch.zeros_like(d), d)
    dd = d.float().unsqueeze(-1)
    q = torch.where(dd == 0, torch.zeros_like(v), torch.round(v / torch.where(dd == 0, torch.ones_like(dd), dd)))
    return (q.clamp(-127, 127) if fmt == Q8 else q.clamp(-8, 7)), d


def _power_of_two(e):
    """2^e in fp32 for whole e, from its bits."""
    return ((e + 127).int() << 23).view(torch.float32)


def _block_exponents(x):
    """kv_format 5: the smallest e with max|x| <= 448 * 2^e over each block (dims -2, -1), -40 <= e <= 40."""
    top = x.abs().nan_to_num(0.0, 0.0, 0.0).amax((-2, -1))
    m, e = torch.frexp(top / torch.full((), 448.0, device=x.device))
    # top / 448 = m * 2^e, 0.5 <= m < 1: e, or e - 1 where top is exactly 448 * 2^(e-1)
    e = torch.where(448.0 * _power_of_two((e - 1).clamp(-126, 127)) >= top, e - 1, e)
    return torch.where(top == 0, torch.full_like(e, -40), e).clamp(-40, 40)


def _to_e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _encode(x, fmt, rows=None):
    """Cache bytes of fp32 rows x [n, 576], for `rows` rows of room (what an earlier write left)."""
    n, rows = x.shape[0], x.shape[0] if rows is None else rows
    if fmt == F16:
        return x.half().view(torch.uint8).reshape(-1)
    if fmt == E4M3:
        blocks = (rows + BLOCK - 1) // BLOCK
        full = torch.zeros(blocks, BLOCK, D_QK, device=x.device)
        full.view(-1, D_QK)[:n] = x
        scale = _power_of_two(_block_exponents(full))
        out = torch.zeros(blocks, BLOCK + 1, D_QK, dtype=torch.uint8, device=x.device)
        out[:, :BLOCK] = _to_e4m3(full / scale[:, None, None]).view(torch.uint8)
        out[:, BLOCK, :4] = scale.view(torch.uint8).view(blocks, 4)
        return out.view(-1)
    parts = []
    for part, f in ((x, Q8 if fmt == Q8Q4 else fmt),) + (((x[:, :D_V], Q4),) if fmt == Q8Q4 else ()):
        q, d = _quant_blocks(part, f)
        if f == Q8:
            codes = q.to(torch.int8).view(n, -1).view(torch.uint8)
        else:
            c = (q + 8).to(torch.uint8)
            codes = (c[..., :16] | (c[..., 16:] << 4)).view(n, -1)
        parts += [codes, d.contiguous().view(torch.uint8).view(n, -1)]
        pad = -(parts[-2].shape[1] + parts[-1].shape[1]) % 16
        parts.append(torch.zeros(n, pad, dtype=torch.uint8, device=x.device))
    return torch.cat(parts, 1).reshape(-1)


def _decode_q(b, fmt, dims, real=torch.float32):
    """Values of stored Q8_0 / Q4_0 rows b [n, bytes]."""
    if fmt == Q8:
        q = b[:, :dims].contiguous().view(torch.int8).to(real)
        d = b[:, dims:dims + dims // 16]
    else:
        c = b[:, :dims // 2].reshape(b.shape[0], -1, 16)
        q = torch.cat((c & 15, c >> 4), -1).reshape(b.shape[0], dims).to(real) - 8
        d = b[:, dims // 2:dims // 2 + dims // 16]
    d = d.contiguous().view(torch.float16).to(real)
    return (q.view(b.shape[0], -1, 32) * d[..., None]).view(b.shape[0], dims)


def _decode(cache, fmt, index, real=torch.float32):
    """Values of the rows `index` (int64, any shape) of a cache, or a pair of key and value rows."""
    if fmt == F16:
        return cache.view(torch.float16).view(-1, D_QK)[index].to(real)
    if fmt == E4M3:
        rows = cache.view(-1, D_QK)
        scale = rows[BLOCK::BLOCK + 1, :4].contiguous().view(torch.float32).view(-1)
        return rows[_place(index)].view(torch.float8_e4m3fn).to(real) * scale[index // BLOCK].to(real)[..., None]
    b = cache.view(-1, _cache_row(fmt))[index]
    if fmt == Q8Q4:
        return _decode_q(b[:, :624], Q8, D_QK, real), _decode_q(b[:, 624:], Q4, D_V, real)
    return _decode_q(b, fmt, D_QK, real)


# ------------------------------------------------------------------ prepare

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def latent(n):
        # normalised latents, rotary keys of larger spread, and rows of uneven size
        x = normal(n, D_QK) * torch.exp(0.5 * normal(n, 1))
        x[:, D_V:] *= 4.0
        return x

    op = case["op"]
    s = {"case": case}
    if op == "rope":
        dt = DTYPES[case["dtype"]]
        s["x"] = normal(case["n"], case["heads"], case["width"]).to(dt)[..., case["width"] - case["head"]:]
        if case["into"]:
            s["out"] = normal(case["n"], case["heads"], case["into"]).to(dt)[..., case["into"] - case["head"]:]
        if case["listed_positions"]:
            s["positions"] = torch.randint(0, case["pos0"] + 1, (case["n"],), generator=g, device=dev).int()
    elif op == "cache":
        n, row0, fmt = case["n"], case["row0"], case["fmt"]
        s["x"] = latent(n).to(DTYPES[case["dtype"]])
        if fmt == E4M3:
            blocks = (row0 + n + BLOCK - 1) // BLOCK
            s["cache"] = torch.zeros(blocks * (BLOCK + 1) * D_QK, dtype=torch.uint8, device=dev)
            if row0 % BLOCK:                                   # the block's rows of earlier tokens
                at, size = row0 // BLOCK * (BLOCK + 1) * D_QK, (BLOCK + 1) * D_QK
                s["cache"][at:at + size] = _encode(latent(row0 % BLOCK), E4M3, BLOCK)
        else:
            s["cache"] = torch.zeros((row0 + n) * _cache_row(fmt), dtype=torch.uint8, device=dev)
    elif op == "read":
        s["cache"] = _encode(latent(case["rows"]), case["fmt"])
        if case["gather"]:
            s["rows"] = torch.randint(0, case["rows"], (case["n"],), generator=g, device=dev).int()
    else:
        n, t0, k = case["n"], case["t0"], case["k"]
        T, n_c = t0 + n, (t0 + n) // 4
        s["q"] = normal(n, HEADS, D_QK).half()
        s["kv_raw"] = _encode(latent(T), E4M3)
        s["kv_cmp"] = _encode(latent(max(n_c, 1)), E4M3)
        if k:
            # the indexer's choice: min(k, n_vis(t)) visible rows, ascending, then -1
            vis = (torch.arange(t0, T, device=dev) + 1) // 4
            top = torch.full((n, k), max(n_c, 1), dtype=torch.int64, device=dev)
            if n_c:
                score = torch.rand(n, n_c, generator=g, device=dev)
                score.masked_fill_(torch.arange(n_c, device=dev) >= vis[:, None], -1.0)
                v, i = score.topk(min(k, n_c), dim=1)
                top[:, :min(k, n_c)] = torch.where(v < 0, torch.full_like(i, n_c), i)
            top = top.sort(dim=1).values
            s["topk"] = torch.where(top >= n_c, torch.full_like(top, -1), top).int().contiguous()
        else:
            s["topk"] = None
        if own:
            from sparse_mla_prefill_b200 import ds4sp as D
            s["handle"] = D.ds4sp_create(D.make_config(n_idx_heads=64, d_idx=128, top_k=k, n_swa=case["n_swa"],
                                                       max_tokens=T, kv_format=E4M3, pv_mode=1))
    return s


# ------------------------------------------------------------------ run

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from sparse_mla_prefill_b200 import ds4sp as D
    c = s["case"]
    op = c["op"]
    if op == "rope":
        return D.ds4sp_rope(s["x"], D.make_rope(**_rope_of(c)), out=s.get("out"), positions=s.get("positions"),
                            pos0=c["pos0"], transpose=c["transpose"])
    if op == "cache":
        fmt, row0, n = c["fmt"], c["row0"], c["n"]
        D.ds4sp_cache_write(s["cache"], fmt, s["x"], row0, rope=D.make_rope(**_rope_of(c)) if c["rope"] else None,
                            pos0=row0 * c["pos_step"], pos_step=c["pos_step"])
        first = _first_read(c)
        key = D.ds4sp_cache_read(s["cache"], fmt, D_QK, row0=first, n=row0 + n - first)
        if fmt == Q8Q4:
            return key, D.ds4sp_cache_read(s["cache"], fmt, D_QK, row0=first, n=row0 + n - first, part=1)
        return key
    if op == "read":
        args = dict(rows=s["rows"]) if c["gather"] else dict(row0=0, n=c["n"])
        key = D.ds4sp_cache_read(s["cache"], c["fmt"], D_QK, dtype=DTYPES[c["dtype"]], **args)
        if c["fmt"] == Q8Q4:
            return key, D.ds4sp_cache_read(s["cache"], c["fmt"], D_QK, part=1, dtype=DTYPES[c["dtype"]], **args)
        return key
    out = torch.empty(c["n"], HEADS, D_V, device="cuda")
    D.ds4sp_sparse_attn(s["handle"], s["q"], s["kv_raw"], s["kv_cmp"], s["topk"], c["t0"], c["n"], out)
    return out


def _first_read(c):
    """First row read back: the start of the first block the write touched."""
    return c["row0"] // BLOCK * BLOCK if c["fmt"] == E4M3 else c["row0"]


def _inverse_frequencies(r, device):
    """Radians per position of each pair, 64 bits, and the factor of cos and sin."""
    d, s = r["dims"], r["factor"]
    i = torch.arange(0, d, 2, dtype=torch.float64, device=device)
    base = r["base"] * s ** (d / (d - 2)) if r["scaling"] == NTK else r["base"]
    f = base ** (-i / d)
    if r["scaling"] == LINEAR:
        return f / s, 1.0
    if r["scaling"] != YARN:
        return f, 1.0

    def turns_at(b):                         # the pair index that turns b times over orig_len
        return d * math.log(r["orig_len"] / (b * 2 * math.pi)) / (2 * math.log(r["base"]))
    low, high = max(math.floor(turns_at(32.0)), 0), min(math.ceil(turns_at(1.0)), d - 1)
    ramp = ((i / 2 - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0 if s > 1 else 1.0


def _rotate(x, positions, r, transpose=False):
    """fp32 x [n, heads, head]: pairs of [offset, offset + dims) turned by position * frequency."""
    f, m = _inverse_frequencies(r, x.device)
    angle = positions.double()[:, None] * f
    cos, sin = ((t * m).float()[:, None] for t in (angle.cos(), angle.sin()))
    if transpose:
        sin = -sin
    o, d = r["offset"], r["dims"]
    part = x[..., o:o + d]
    a, b = (part[..., 0::2], part[..., 1::2]) if r["layout"] == 0 else (part[..., :d // 2], part[..., d // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, v), -1).flatten(-2) if r["layout"] == 0 else torch.cat((u, v), -1)
    return torch.cat((x[..., :o], turned, x[..., o + d:]), -1)


def _positions(s):
    c = s["case"]
    if "positions" in s:
        return s["positions"]
    step = c.get("pos_step", 1)
    first = c["pos0"] if c["op"] == "rope" else c["row0"] * step
    return first + step * torch.arange(c["n"], device="cuda")


def _plain_rope(s):
    c = s["case"]
    y = _rotate(s["x"].float(), _positions(s), _rope_of(c), c["transpose"]).to(s["x"].dtype)
    return s["out"].copy_(y) if "out" in s else y


def _plain_cache(s):
    c = s["case"]
    x = s["x"].float()
    if c["rope"]:
        x = _rotate(x[:, None], _positions(s), _rope_of(c))[:, 0]
    if c["fmt"] == F16:
        return x.half()
    if c["fmt"] != E4M3:
        def values(part, f):
            q, d = _quant_blocks(part, f)
            return (q * d.float()[..., None]).view(part.shape).half()
        if c["fmt"] == Q8Q4:
            return values(x, Q8), values(x[:, :D_V], Q4)
        return values(x, c["fmt"])
    # Blocks of 64 rows: earlier rows of the first block keep their scale unless a new row
    # needs a larger one; they are then rounded again to it.
    first, last = _first_read(c), c["row0"] + c["n"]
    old = c["row0"] - first
    blocks = (last - first + BLOCK - 1) // BLOCK
    full = torch.zeros(blocks, BLOCK, D_QK, device=x.device)
    full.view(-1, D_QK)[old:last - first] = x
    e = _block_exponents(full)
    if old:
        kept = s["cache"].view(-1, BLOCK + 1, D_QK)[first // BLOCK]
        scale = kept[BLOCK, :4].contiguous().view(torch.float32)
        e[0] = torch.maximum(e[0], torch.frexp(scale).exponent[0] - 1)
        full.view(-1, D_QK)[:old] = kept[:old].view(torch.float8_e4m3fn).float() * scale
    scale = _power_of_two(e)[:, None, None]
    return (_to_e4m3(full / scale).float() * scale).view(-1, D_QK)[:last - first].half()


def _plain_read(s):
    c = s["case"]
    index = s["rows"].long() if c["gather"] else torch.arange(c["n"], device="cuda")
    v = _decode(s["cache"], c["fmt"], index)
    dt = DTYPES[c["dtype"]]
    return tuple(p.to(dt) for p in v) if isinstance(v, tuple) else v.to(dt)


def _plain_attn(s):
    c = s["case"]
    t = torch.arange(c["t0"], c["t0"] + c["n"], device="cuda")
    at = t[:, None] - torch.arange(c["n_swa"] - 1, -1, -1, device="cuda")
    rows, seen = _decode(s["kv_raw"], E4M3, at.clamp(min=0)), at >= 0
    if s["topk"] is not None:
        top = s["topk"].long()
        rows = torch.cat((_decode(s["kv_cmp"], E4M3, top.clamp(min=0)), rows), 1)
        seen = torch.cat((top >= 0, seen), 1)
    logits = torch.matmul(s["q"].float(), rows.transpose(1, 2)) / math.sqrt(D_QK)
    logits = torch.where(seen[:, None], logits, torch.full((), -math.inf, device="cuda"))
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    return torch.matmul(p / p.sum(-1, keepdim=True), rows[..., :D_V])


_PLAIN = {"rope": _plain_rope, "cache": _plain_cache, "read": _plain_read, "attn": _plain_attn}


# ------------------------------------------------------------------ exact

def _exact_turned(x, positions, r, transpose=False):
    """64-bit x [n, heads, head] times exp(i * angle), pair by pair, as complex numbers."""
    d, o, s = r["dims"], r["offset"], float(r["factor"])
    speed, size = [], 1.0
    for i in range(d // 2):
        w = r["base"] ** (-2.0 * i / d)
        if r["scaling"] == LINEAR:
            w /= s
        elif r["scaling"] == NTK:
            w = (r["base"] * s ** (d / (d - 2.0))) ** (-2.0 * i / d)
        elif r["scaling"] == YARN:
            size = 0.1 * math.log(s) + 1.0 if s > 1 else 1.0
            at = [d * math.log(r["orig_len"] / (b * 2 * math.pi)) / (2 * math.log(r["base"])) for b in (32, 1)]
            low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
            far = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            w = w * (1 - far) + w / s * far
        speed.append(w)
    angle = positions.to(torch.float64)[:, None, None] * torch.tensor(speed, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(angle, size), -angle if transpose else angle)
    y = x.clone()
    first = slice(o, o + d, 2) if r["layout"] == 0 else slice(o, o + d // 2)
    second = slice(o + 1, o + d, 2) if r["layout"] == 0 else slice(o + d // 2, o + d)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_e4m3(x):
    """64-bit x rounded to four significant bits, at least 2^-9 apart, half to even, up to 448."""
    e = torch.frexp(x).exponent.double() - 1
    step = _exact_power(e.clamp(min=-6.0) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_blocks(x, fmt):
    v = x.unflatten(-1, (-1, 32))
    if fmt == Q8:
        d = (v.abs().amax(-1) / 127).half().double()[..., None]
        low, high = -127, 127
    else:
        big, small = v.amax(-1), v.amin(-1)
        at = torch.arange(32, device=x.device)
        up = torch.where(v == big[..., None], at, 32).amin(-1)
        down = torch.where(v == small[..., None], at, 32).amin(-1)
        m = torch.where((big > -small) | ((big == -small) & (up < down)), big, small)
        d = (m / -8).half().double()[..., None]
        low, high = -8, 7
    q = torch.where(d == 0, 0.0, torch.round(v / torch.where(d == 0, 1.0, d))).clamp(low, high)
    return (q * d).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "rope":
        return _exact_turned(s["x"].double(), _positions(s), _rope_of(c), c["transpose"])
    if op == "cache":
        x = s["x"].double()
        if c["rope"]:
            x = _exact_turned(x[:, None], _positions(s), _rope_of(c))[:, 0]
        if c["fmt"] == F16:
            return x
        if c["fmt"] == Q8Q4:
            return _exact_blocks(x, Q8), _exact_blocks(x[:, :D_V], Q4)
        if c["fmt"] != E4M3:
            return _exact_blocks(x, c["fmt"])
        out, first = [], _first_read(c)
        old = _decode(s["cache"], E4M3, torch.arange(first, c["row0"], device="cuda"), torch.float64)
        x = torch.cat((old, x))
        x = torch.cat((x, torch.zeros(-x.shape[0] % BLOCK, D_QK, dtype=x.dtype, device=x.device)))
        x = x.unflatten(0, (-1, BLOCK))
        top = x.abs().amax((1, 2))
        if old.shape[0]:                                   # the first block's scale never shrinks
            kept = s["cache"].view(-1, D_QK)[int(_place(torch.tensor(first))) + BLOCK, :4]
            top[0] = torch.maximum(top[0], kept.clone().view(torch.float32)[0].double() * 448)
        m, e = torch.frexp(top.clamp(min=1e-30) / 448)
        size = _exact_power(torch.where(m == 0.5, e - 1, e).clamp(-40, 40))[:, None, None]
        return (_exact_e4m3(x / size) * size).flatten(0, 1)[:c["row0"] + c["n"] - first]
    if op == "read":
        index = s["rows"].long() if c["gather"] else torch.arange(c["n"], device="cuda")
        return _decode(s["cache"], c["fmt"], index, torch.float64)
    outs = []
    raw = _decode(s["kv_raw"], E4M3, torch.arange(c["t0"] + c["n"], device="cuda"), torch.float64)
    cmp_ = _decode(s["kv_cmp"], E4M3, torch.arange(max((c["t0"] + c["n"]) // 4, 1), device="cuda"), torch.float64)
    for i in range(0, c["n"], 256):
        t = torch.arange(c["t0"] + i, c["t0"] + min(i + 256, c["n"]), device="cuda")
        at = t[:, None] - torch.arange(c["n_swa"], device="cuda")
        rows, hidden = raw[at.clamp(min=0)], at < 0
        if s["topk"] is not None:
            top = s["topk"][i:i + 256].long()
            rows, hidden = torch.cat((rows, cmp_[top.clamp(min=0)]), 1), torch.cat((hidden, top < 0), 1)
        z = torch.einsum("nhd,nrd->nhr", s["q"][i:i + 256].double(), rows) / 24.0
        z.masked_fill_(hidden[:, None], -math.inf)
        outs.append(torch.einsum("nhr,nrd->nhd", torch.softmax(z, -1), rows[..., :D_V]))
    return torch.cat(outs)


# ------------------------------------------------------------------ work

def work(case):
    c, op = case, case["op"]
    if op == "rope":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * size * c["n"] * c["heads"] * c["head"],
                "flops": 3 * c["n"] * c["heads"] * c["dims"]}
    if op == "cache":
        back = c["row0"] + c["n"] - _first_read(c)
        size = 4 if c["dtype"] == "fp32" else 2
        values = D_QK + (D_V if c["fmt"] == Q8Q4 else 0)
        return {"bytes": c["n"] * (D_QK * size + _cache_row(c["fmt"])) + back * (_cache_row(c["fmt"]) + 2 * values),
                "flops": 2 * (c["n"] + back) * D_QK}
    if op == "read":
        size = 4 if c["dtype"] == "fp32" else 2
        values = D_QK + (D_V if c["fmt"] == Q8Q4 else 0)
        return {"bytes": c["n"] * (_cache_row(c["fmt"]) + size * values + (4 if c["gather"] else 0)),
                "flops": c["n"] * values}
    n, t0, k, w = c["n"], c["t0"], c["k"], c["n_swa"]
    attended = sum(min(k, (t + 1) // 4) + min(w, t + 1) for t in range(t0, t0 + n))
    unique = min((t0 + n) // 4, n * k) + t0 + n - max(0, t0 - w + 1)
    return {"bytes": n * (HEADS * D_QK * 2 + HEADS * D_V * 4 + 4 * k) + unique * _cache_row(E4M3),
            "flops": 2 * HEADS * (D_QK + D_V) * attended}
