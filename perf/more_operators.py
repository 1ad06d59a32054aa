"""The operators around a 4-bit latent cache, as measured: norms of queries and
keys with the position rotation in the same pass, the append of latent rows to
a paged cache of 4-bit rows, reading such rows back, and attention of new
tokens over them.

`run` computes each operator in its plain form (elementary torch operations in
32 bits, angles in 64) or, with `own` set, through mla_ragged_paged_gb300.binding.
`exact` restates the definitions in 64 bits.

A cached row of W elements: W / 2 bytes of e2m1 codes (the lower of two
elements in the low half of a byte), a byte with the row's exponent E, W / 64
bytes with the shift of each block of 32 elements (the lower of two blocks in
the low half), zeros up to a multiple of 16 bytes.  An element is
e2m1(code) * 2^(E - 127 - shift).
"""
import math

import torch

own = False

LATENT, ROPE = 512, 64
WIDTH = LATENT + ROPE  # one latent row: [c_kv 512 | k_rope 64]
BLOCK = 32             # elements that share a shift
ROW = 304              # bytes of a cached row of WIDTH elements
USED = WIDTH // 2 + WIDTH // 64 + 1  # of them, those that hold something
LEAST, MOST, DEEPEST = -100, 125, 14  # a row's exponent, and its blocks' shifts
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One new token of one sequence, 128 heads: rope dims of the queries and
        # the latent row (norm of its 512, rotation of its 64).  Latency.
        dict(name="rope_token", op="rope", tokens=1, heads=128, kind="mla", interleaved=True, far=4000),
        # One new token for each of 256 sequences.
        dict(name="rope_step", op="rope", tokens=256, heads=128, kind="mla", interleaved=True, far=131072),
        # A long prompt.
        dict(name="rope_prompt", op="rope", tokens=16384, heads=128, kind="mla", interleaved=True, far=16384),
        # Queries and keys normalised whole, head by head, rotated by halves; an odd
        # number of tokens far into a context.
        dict(name="rope_heads", op="rope", tokens=5003, heads=32, kind="heads", kheads=8, dim=128, rot=128,
             interleaved=False, far=1000000),
        # One token for each of 256 sequences into the cache, and back as it is stored.
        dict(name="append_step", op="append", batch=256, new=1, spread=False, prior=500, page=64, seed=1),
        # Prompts of uneven lengths into the cache, and back as they are stored.
        dict(name="append_prompts", op="append", batch=16, new=2048, spread=True, prior=300, page=128, seed=2),
        # A short context in 8 bits, for a product with 8-bit weights.
        dict(name="read_short", op="read", batch=1, length=1000, spread=False, to="e4m3", page=64, seed=3),
        # A buffer row of cached contexts in bf16, for prefill.
        dict(name="read_row", op="read", batch=24, length=2700, spread=True, to="bf16", page=64, seed=4),
        # A short chat's next token on a 16-head shard: latency.
        dict(name="decode_one", op="decode", batch=1, heads=16, new=1, length=1000, spread=False, page=64, seed=5),
        # Drafted tokens of a middling batch, 24 heads, pages that no power of two fills.
        dict(name="decode_drafts", op="decode", batch=40, heads=24, new=3, length=2000, spread=True, page=24,
             seed=6),
        # The next token of 64 sequences, 128 heads.
        dict(name="decode_batch", op="decode", batch=64, heads=128, new=1, length=4500, spread=True, page=128,
             seed=7),
        # Two tokens a sequence (one of them drafted) over very long contexts, 16 heads.
        dict(name="decode_long", op="decode", batch=4, heads=16, new=2, length=131072, spread=False, page=64,
             seed=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "read", "decode", "decode"])
    seed = rng.randrange(1 << 30)
    if op == "rope":
        far, interleaved = _log(rng, 100, 1000000), rng.random() < 0.5
        if rng.random() < 0.5:
            heads = rng.choice([1, 8, 16, 24, 64, 128])
            return dict(op=op, tokens=_log(rng, 1, 16384), heads=heads, kind="mla", interleaved=interleaved, far=far)
        dim = rng.choice([64, 80, 96, 128, 192, 256, 576, 50])
        heads, kheads = rng.choice([(32, 8), (16, 16), (12, 1), (7, 3), (64, 4)])
        tokens = max(1, min(_log(rng, 1, 16384), 16384 * 8192 // (dim * (heads + kheads))))
        return dict(op=op, tokens=tokens, heads=heads, kind="heads", kheads=kheads, dim=dim,
                    rot=rng.choice([dim, dim // 4 * 2, 32]), interleaved=interleaved, far=far)
    page = rng.choice([16, 64, 128, 256, 12, 24, 1])
    if op == "append":
        new = _log(rng, 1, 4096)
        return dict(op=op, batch=max(1, min(_log(rng, 1, 256), 32768 // new)), new=new, spread=rng.random() < 0.5,
                    prior=_log(rng, 1, 2000), page=page, seed=seed)
    if op == "read":
        length = _log(rng, 4, 65536)
        return dict(op=op, batch=max(1, min(_log(rng, 1, 128), 65536 // length)), length=length,
                    spread=rng.random() < 0.5, to=rng.choice(["bf16", "e4m3"]), page=page, seed=seed)
    length = _log(rng, 4, 131072)
    heads = rng.choice([1, 4, 8, 16, 24, 32, 64, 128])
    new = rng.choice([1, 1, 1, 2, 4])
    cap = max(1, min(262144 // length, 64 * 4500 * 128 // (length * heads * new)))
    return dict(op=op, batch=min(_log(rng, 1, 128), cap), heads=heads, new=new, length=length,
                spread=rng.random() < 0.6, page=page, seed=seed)


def _lengths(case):
    """(new, prior) of each sequence, on the host: part of the case, so that
    `work` knows them."""
    g = torch.Generator().manual_seed(case["seed"])
    B = case["batch"]

    def pick(mean, least):
        if not case["spread"]:
            return [mean] * B
        lo, hi = max(least, mean // 4), max(least, mean * 7 // 4)
        return torch.randint(lo, hi + 1, (B,), generator=g).tolist()

    if case["op"] == "append":
        new = pick(case["new"], 1)
        prior = torch.randint(0, case["prior"] + 1, (B,), generator=g).tolist()
    elif case["op"] == "read":      # a window of each context, from `prior` on
        new = pick(case["length"], 1)
        prior = torch.randint(0, 200, (B,), generator=g).tolist()
    else:
        new = [case["new"]] * B
        prior = [max(0, n - case["new"]) for n in pick(case["length"], case["new"])]
    return new, prior


def work(case):
    if case["op"] == "rope":
        t = case["tokens"]
        if case["kind"] == "mla":
            n, weights, rot = t * (case["heads"] * ROPE + WIDTH), 2 * LATENT, ROPE
        else:
            n, weights, rot = t * (case["heads"] + case["kheads"]) * case["dim"], 4 * case["dim"], case["rot"]
        return dict(bytes=4 * n + 4 * t + weights + 2 * rot, flops=6 * n)
    new, prior = _lengths(case)
    t = sum(new)
    if case["op"] == "append":
        return dict(bytes=t * (2 * WIDTH + USED + 2 * WIDTH), flops=3 * t * WIDTH)
    if case["op"] == "read":
        return dict(bytes=t * (USED + (2 * WIDTH if case["to"] == "bf16" else WIDTH + 4)), flops=t * WIDTH)
    ctx = sum(n + p for n, p in zip(new, prior))
    pairs = sum(p * n + n * (n + 1) // 2 for n, p in zip(new, prior)) * case["heads"]
    rows = t * case["heads"]
    return dict(bytes=ctx * USED + rows * 2 * (WIDTH + LATENT) + 4 * rows, flops=2 * pairs * (WIDTH + LATENT))


# ------------------------------------------------------------------ 4-bit rows

def _power(e):
    """2^e in fp32, exactly (a device's pow and exp2 need not be); e in -126 .. 128 (infinity)."""
    return (e + 127 << 23).view(torch.float32)


def _encode(x):
    """Cached rows [n, ROW] (bytes) of fp32 rows x [n, WIDTH]."""
    n, blocks = x.shape[0], WIDTH // BLOCK
    x = x.reshape(n, blocks, BLOCK)
    amax = x.abs().amax(dim=2)
    # The least e with amax <= 7 * 2^e, from the bits of amax.
    e = ((amax.view(torch.int32) + 0x1FFFFF) >> 23) - 129
    base = e.amax(dim=1).clamp(LEAST, MOST)
    shift = (base[:, None] - e).clamp(0, DEEPEST)
    y = x.abs() * _power(shift - base[:, None])[:, :, None]
    code = torch.signbit(x).to(torch.uint8) * 8
    for at, tie_up in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        code += (y >= at) if tie_up else (y > at)
    code = code.view(n, WIDTH // 2, 2)
    shift = shift.to(torch.uint8).view(n, WIDTH // 64, 2)
    exponent = base + 127
    bad = ~torch.isfinite(amax).all(dim=1)
    rows = torch.zeros((n, ROW), dtype=torch.uint8, device=x.device)
    rows[:, :WIDTH // 2] = code[:, :, 0] | code[:, :, 1] << 4
    rows[:, WIDTH // 2] = exponent.to(torch.uint8)
    rows[:, WIDTH // 2 + 1:USED] = shift[:, :, 0] | shift[:, :, 1] << 4
    rows[bad] = 0
    rows[:, WIDTH // 2].masked_fill_(bad, 255)
    return rows


def _units(rows):
    """Of cached rows [..., ROW] (bytes): the elements as fp32 in units of
    2^(E - 133), [..., WIDTH], and that unit, [..., 1]."""
    lead = rows.shape[:-1]
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=rows.device)
    codes = rows[..., :WIDTH // 2]
    v = table[torch.stack([codes & 15, codes >> 4], dim=-1).int()].view(*lead, WIDTH // BLOCK, BLOCK)
    shifts = rows[..., WIDTH // 2 + 1:USED]
    shift = torch.stack([shifts & 15, shifts >> 4], dim=-1).int().view(*lead, WIDTH // BLOCK, 1)
    unit = _power(rows[..., WIDTH // 2:WIDTH // 2 + 1].int() - 133)
    return (v * _power(6 - shift)).view(*lead, WIDTH), unit


# ------------------------------------------------------------------ the inputs

def _page_table(lengths, page, gen):
    cols = [-(-n // page) for n in lengths]
    total = sum(cols) + 1
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(lengths), max(max(cols), 1)), dtype=torch.int32, device="cuda")
    counts = torch.tensor(cols, device="cuda")
    held = torch.arange(table.shape[1], device="cuda")[None, :] < counts[:, None]
    table[held] = order[:total - 1]
    return table, total


def _ragged(case, s):
    new, prior = _lengths(case)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["new"], s["prior"], s["starts"] = new, prior, starts
    s["row_offsets"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["cache_lens"] = torch.tensor(prior, dtype=torch.int32, device="cuda")
    return [n + p for n, p in zip(new, prior)], starts[-1]


def _latent_rows(n, gen):
    """Normalised c_kv and rotated rope dims: bell-shaped, the rows of uneven size."""
    x = torch.randn((n, WIDTH), generator=gen, device="cuda")
    x *= torch.exp(0.3 * torch.randn((n, 1), generator=gen, device="cuda"))
    return x.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    bf16 = lambda *shape: randn(*shape).to(torch.bfloat16)
    empty = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    if case["op"] == "rope":
        t, heads = case["tokens"], case["heads"]
        s["positions"] = torch.randint(0, case["far"], (t,), generator=gen, device="cuda").to(torch.int32)
        s["eps"] = 1e-6
        if case["kind"] == "mla":
            rot = ROPE
            # The queries' rope dims lie in the projection's [T, H, 192] rows and go
            # where the absorbed queries [T, H, 576] have them.
            s["q"] = bf16(t, heads, 128 + ROPE)[:, :, 128:]
            s["q_out"] = torch.zeros((t, heads, WIDTH), dtype=torch.bfloat16, device="cuda")[:, :, LATENT:]
            s["q_weight"] = None
            s["k"], s["k_out"] = bf16(t, 1, WIDTH), empty(t, 1, WIDTH)
            s["k_weight"] = (1 + 0.1 * randn(LATENT)).to(torch.bfloat16)
        else:
            rot, dim, kheads = case["rot"], case["dim"], case["kheads"]
            s["q"], s["q_out"] = bf16(t, heads, dim), empty(t, heads, dim)
            s["k"], s["k_out"] = bf16(t, kheads, dim), empty(t, kheads, dim)
            s["q_weight"] = (1 + 0.1 * randn(dim)).to(torch.bfloat16)
            s["k_weight"] = (1 + 0.1 * randn(dim)).to(torch.bfloat16)
        powers = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot
        s["inv_freq"] = (10000.0 ** -powers).float()
        s["rope_scale"] = 1.0
        return s
    lengths, total = _ragged(case, s)
    s["table"], pages = _page_table(lengths, case["page"], gen)
    slots = pages * case["page"]
    s["cache"] = _encode(_latent_rows(slots, gen).float()).view(pages, case["page"], ROW)
    if case["op"] == "append":
        s["rows"], s["back"] = _latent_rows(total, gen), empty(total, WIDTH)
    elif case["op"] == "read":
        s["back"] = torch.empty((total, WIDTH), dtype=torch.bfloat16 if case["to"] == "bf16" else E4M3, device="cuda")
        s["back_scales"] = None if case["to"] == "bf16" else torch.empty(total, device="cuda")
    else:
        s["q"] = bf16(total, case["heads"], WIDTH)
        s["softmax_scale"] = 1 / math.sqrt(192)
        s["out_t"] = empty(total, case["heads"], LATENT)
        s["lse"] = torch.empty((total, case["heads"]), dtype=torch.float32, device="cuda")
        if own:
            from mla_ragged_paged_gb300 import binding
            s["workspace"] = binding.alloc_decode_workspace()
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return dict(rope=_plain_rope, append=_plain_append, read=_plain_read, decode=_plain_decode)[s["op"]](s)


def _run_own(s):
    from mla_ragged_paged_gb300 import binding
    if s["op"] == "rope":
        binding.norm_rope(s["positions"], s["inv_freq"], q=s["q"], q_out=s["q_out"], q_weight=s["q_weight"],
                          k=s["k"], k_out=s["k_out"], k_weight=s["k_weight"], eps=s["eps"],
                          rope_scale=s["rope_scale"], interleaved=s["interleaved"])
        return [s["q_out"], s["k_out"]]
    if s["op"] == "append":
        binding.append_latent_fp4(s["cache"], s["rows"], s["table"], s["row_offsets"], s["cache_lens"])
        binding.gather_latent_fp4(s["back"], s["cache"], s["table"], s["row_offsets"], s["cache_lens"])
        return [s["back"]]
    if s["op"] == "read":
        binding.gather_latent_fp4(s["back"], s["cache"], s["table"], s["row_offsets"], s["cache_lens"],
                                  dst_scales=s["back_scales"])
        return [s["back"]] if s["back_scales"] is None else [s["back"], s["back_scales"]]
    binding.decode_latent_fp4(s["out_t"], s["q"], s["cache"], s["table"], s["row_offsets"], s["cache_lens"],
                              s["softmax_scale"], workspace=s["workspace"], lse=s["lse"])
    return [s["out_t"], s["lse"]]


def _plain_rotated(s, x, weight):
    y = x.float()
    rot = 2 * s["inv_freq"].numel()
    if weight is not None:
        n = weight.numel()
        a = y[:, :, :n]
        a = a * torch.rsqrt((a * a).mean(dim=2, keepdim=True) + s["eps"]) * weight.float()
        y = torch.cat([a, y[:, :, n:]], dim=2)
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    tail = y[:, :, y.shape[2] - rot:]
    if s["interleaved"]:
        u, v = tail[:, :, 0::2], tail[:, :, 1::2]
    else:
        u, v = tail[:, :, :rot // 2], tail[:, :, rot // 2:]
    turned = [(u * cos - v * sin) * s["rope_scale"], (u * sin + v * cos) * s["rope_scale"]]
    tail = torch.stack(turned, dim=3).flatten(2) if s["interleaved"] else torch.cat(turned, dim=2)
    return torch.cat([y[:, :, :y.shape[2] - rot], tail], dim=2).to(torch.bfloat16)


def _plain_rope(s):
    return [_plain_rotated(s, s["q"], s["q_weight"]), _plain_rotated(s, s["k"], s["k_weight"])]


def _slots(s, total):
    """The cache slots of rows row_offsets[b] + i, at context positions cache_lens[b] + i."""
    page = s["cache"].shape[1]
    starts = s["row_offsets"].long()
    b = torch.repeat_interleave(starts[1:] - starts[:-1], output_size=total)
    pos = s["cache_lens"][b].long() + torch.arange(total, device="cuda") - starts[b]
    return s["table"][b, pos // page].long() * page + pos % page


def _plain_append(s):
    slots = _slots(s, len(s["rows"]))
    rows = s["cache"].view(-1, ROW)
    rows[slots] = _encode(s["rows"].float())
    units, unit = _units(rows[slots])
    return [(units * unit).to(torch.bfloat16)]


def _plain_read(s):
    units, unit = _units(s["cache"].view(-1, ROW)[_slots(s, len(s["back"]))])
    if s["back_scales"] is None:
        return [(units * unit).to(torch.bfloat16)]
    return [units.to(E4M3), unit[:, 0]]


def _plain_decode(s):
    heads, new, page = s["heads"], s["new"][0], s["cache"].shape[1]
    batch = len(s["new"])
    longest = max(s["prior"]) + new
    pos = torch.arange(longest, device="cuda")
    columns = (pos // page)[None, :].expand(batch, -1)
    slots = torch.gather(s["table"].long(), 1, columns) * page + pos % page
    units, unit = _units(s["cache"].view(-1, ROW)[slots])
    k = units.mul_(unit)
    x = torch.bmm(s["q"].float().view(batch, new * heads, WIDTH), k.transpose(1, 2)) * s["softmax_scale"]
    seen = s["cache_lens"].long()[:, None] + torch.arange(new, device="cuda")
    hidden = pos[None, None, :] > seen[:, :, None]
    x = x.view(batch, new, heads, longest).masked_fill(hidden[:, :, None, :], float("-inf"))
    top = x.amax(dim=3, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(dim=3, keepdim=True)
    out = torch.bmm((e / total).view(batch, new * heads, longest), k[:, :, :LATENT])
    lse = (top + torch.log(total))[:, :, :, 0]
    return [out.view(batch * new, heads, LATENT).to(torch.bfloat16), lse.reshape(batch * new, heads)]


# ------------------------------------------------------------------ in 64 bits

def _power64(e):
    return (e.long() + 1023 << 52).view(torch.float64)


def _values64(rows):
    """The elements of cached rows [n, ROW] in 64 bits."""
    n = rows.shape[0]
    nibbles = torch.empty((n, WIDTH), dtype=torch.int64, device="cuda")
    nibbles[:, 0::2] = rows[:, :WIDTH // 2] % 16
    nibbles[:, 1::2] = rows[:, :WIDTH // 2] // 16
    magnitude = nibbles % 8
    # Two exponent bits and one mantissa bit; the lowest exponent has no leading one.
    exponent, mantissa = magnitude // 2, (magnitude % 2).double()
    v = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * _power64(exponent - 1))
    v = torch.where(nibbles >= 8, -v, v)
    shifts = torch.empty((n, WIDTH // BLOCK), dtype=torch.int64, device="cuda")
    shifts[:, 0::2] = rows[:, WIDTH // 2 + 1:USED] % 16
    shifts[:, 1::2] = rows[:, WIDTH // 2 + 1:USED] // 16
    power = rows[:, WIDTH // 2].long()[:, None] - 127 - shifts
    return v * torch.repeat_interleave(_power64(power), BLOCK, dim=1)


def _stored64(x):
    """What rows x (64-bit) read back as once they are stored."""
    n = x.shape[0]
    blocks = x.view(n, WIDTH // BLOCK, BLOCK)
    mantissa, e = torch.frexp(blocks.abs().amax(dim=2).clamp_min(1e-38))  # mantissa 2^e, 1/2 <= mantissa < 1
    e = e.long() - torch.where(mantissa <= 0.875, 3, 2)
    top = e.max(dim=1, keepdim=True).values.clamp(LEAST, MOST)
    step = _power64(torch.maximum(torch.minimum(e, top), top - DEEPEST))[:, :, None]
    y = (blocks / step).abs()
    # To the nearest even multiple of the spacing there: 1/2 below 2, 1 below 4, then 2.
    spacing = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    q = torch.clamp(torch.round(y / spacing) * spacing, max=6.0)
    return (torch.sign(blocks) * q * step).view(n, WIDTH)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None, :]
        half = turn.shape[2]
        outs = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            y = x.double()
            if w is not None:
                n = len(w)
                rms = torch.linalg.vector_norm(y[:, :, :n], dim=2, keepdim=True) / math.sqrt(n)
                y[:, :, :n] *= w.double() / torch.hypot(rms, torch.full_like(rms, math.sqrt(s["eps"])))
            first = y.shape[2] - 2 * half
            even = slice(first, None, 2) if s["interleaved"] else slice(first, first + half)
            odd = slice(first + 1, None, 2) if s["interleaved"] else slice(first + half, None)
            z = torch.complex(y[:, :, even].contiguous(), y[:, :, odd].contiguous()) * turn * s["rope_scale"]
            y[:, :, even], y[:, :, odd] = z.real, z.imag
            outs.append(y)
        return outs
    page = case["page"]
    flat = s["cache"].view(-1, ROW)
    if case["op"] == "append":
        return [_stored64(s["rows"].double())]
    table = s["table"].cpu()
    slots = []
    for b, (n, p) in enumerate(zip(s["new"], s["prior"])):
        first = 0 if case["op"] == "decode" else p
        pos = torch.arange(first, p + n)
        slots.append((table[b, pos // page].long() * page + pos % page).to("cuda"))
    if case["op"] == "read":
        rows = flat[torch.cat(slots)]
        v = _values64(rows)
        if case["to"] == "bf16":
            return [v]
        unit = _power64(rows[:, WIDTH // 2].long() - 133)
        return [v / unit[:, None], unit]
    out = torch.empty((s["starts"][-1], case["heads"], LATENT), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["starts"][-1], case["heads"]), dtype=torch.float64, device="cuda")
    for b, (n, p) in enumerate(zip(s["new"], s["prior"])):
        k = _values64(flat[slots[b]])
        for i in range(n):
            seen = k[:p + i + 1]
            x = torch.einsum("hd,jd->hj", s["q"][s["starts"][b] + i].double(), seen) * s["softmax_scale"]
            z = torch.logsumexp(x, dim=1)
            lse[s["starts"][b] + i] = z
            out[s["starts"][b] + i] = torch.exp(x - z[:, None]) @ seen[:, :LATENT]
    return [out, lse]
