"""The operators of a serving step with 8-bit weights and an 8-bit latent
cache, as measured: a root-mean-square norm with the residual's addition and
8-bit output, the block-scaled 8-bit matrix product, the append of latent rows
to a paged 8-bit cache, and attention of new tokens over that cache.

`run` computes each operator in its plain form (elementary torch operations in
32 bits) or, with `own` set, through mla_ragged_paged_gb300.binding.
`exact` restates the definitions in 64 bits.
"""
import math

import torch

own = False

GROUP = 128            # columns that share one scale of a row, and the side of a weight block
LATENT, ROPE = 512, 64
WIDTH = LATENT + ROPE  # one cached latent row: [c_kv 512 | k_rope 64]
FP8_MAX = 448.0
FP8_TINY = 1e-30       # the least amax a scale is formed from
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One new token of one sequence through a norm of the hidden state: latency.
        dict(name="norm_token", op="norm", rows=1, dim=8192, stride=8192, residual=True, fp8=True),
        # A long prompt's hidden states before a projection with 8-bit weights.
        dict(name="norm_prompt", op="norm", rows=16384, dim=8192, stride=8192, residual=True, fp8=True),
        # The latent part of 576-wide rows, normalised in bf16 before it is cached.
        dict(name="norm_latent", op="norm", rows=5003, dim=512, stride=576, residual=False, fp8=False),
        # A projection for one new token: all weight bytes for one row.
        dict(name="matmul_token", op="matmul", m=1, n=8192, k=4096, out="bf16", row_scale=False),
        # The output projection of 128 heads x 128 for a batch of 64 new tokens.
        dict(name="matmul_batch", op="matmul", m=64, n=8192, k=16384, out="bf16", row_scale=False),
        # K_nope of a 4096-token buffer row from gathered rows of the 8-bit
        # latent cache (one scale a row), 128 heads x 128.
        dict(name="matmul_latent", op="matmul", m=4096, n=16384, k=512, out="bf16", row_scale=True),
        # A prompt's projection with sizes that fill no tile, 32-bit output.
        dict(name="matmul_ragged", op="matmul", m=5001, n=8200, k=4112, out="f32", row_scale=False),
        # One token for each of 256 sequences into the cache.
        dict(name="append_step", op="append", batch=256, new=1, spread=False, prior=500, page=64, seed=1),
        # Prompts of uneven lengths into the cache.
        dict(name="append_prompts", op="append", batch=16, new=2048, spread=True, prior=300, page=128, seed=2),
        # A short chat's next token on a 16-head shard: latency.
        dict(name="decode_one", op="decode", batch=1, heads=16, new=1, length=1000, spread=False, page=64, seed=3),
        # The next token of 64 sequences, 128 heads.
        dict(name="decode_batch", op="decode", batch=64, heads=128, new=1, length=4500, spread=True, page=128,
             seed=4),
        # Two tokens a sequence (one of them drafted) over very long contexts, 16 heads.
        dict(name="decode_long", op="decode", batch=4, heads=16, new=2, length=131072, spread=False, page=64,
             seed=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "matmul", "append", "decode", "matmul", "decode"])
    seed = rng.randrange(1 << 30)
    if op == "norm":
        dim = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            dim = max(8, dim // 8 * 8)
        rows = _log(rng, 1, max(2, min(16384, 16384 * 8192 // dim)))
        return dict(op=op, rows=rows, dim=dim, stride=dim + rng.choice([0, 0, 64, 8]),
                    residual=rng.random() < 0.6, fp8=rng.random() < 0.7)
    if op == "matmul":
        k = max(16, _log(rng, 128, 16384) // 16 * 16)
        n = _log(rng, 64, 16384)
        m = _log(rng, 1, 8192)
        while 2 * m * n * k > 3.3e11 or n * k > 16384 * 8192:
            m, n = max(1, m // 2), max(64, n * 3 // 4)
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(["bf16", "bf16", "f32"]), row_scale=rng.random() < 0.3)
    page = rng.choice([16, 64, 128, 256, 12, 24])
    if op == "append":
        new = _log(rng, 1, 4096)
        return dict(op=op, batch=max(1, min(_log(rng, 1, 256), 32768 // new)), new=new, spread=rng.random() < 0.5,
                    prior=_log(rng, 1, 2000), page=page, seed=seed)
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
    else:
        new = [case["new"]] * B
        prior = [max(0, n - case["new"]) for n in pick(case["length"], case["new"])]
    return new, prior


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        scales = case["rows"] * -(-case["dim"] // GROUP) * 4
        b = 2 * n + (4 * n if case["residual"] else 0) + (n + scales if case["fp8"] else 2 * n) + 2 * case["dim"]
        return dict(bytes=b, flops=6 * n)
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // GROUP)
        b = m * k + n * k + m * n * (2 if case["out"] == "bf16" else 4)
        b += 4 * (m if case["row_scale"] else m * kb) + 4 * -(-n // GROUP) * kb
        return dict(bytes=b, flops=2 * m * n * k)
    new, prior = _lengths(case)
    t = sum(new)
    if case["op"] == "append":
        return dict(bytes=t * (2 * WIDTH + WIDTH + 4), flops=3 * t * WIDTH)
    ctx = sum(n + p for n, p in zip(new, prior))
    pairs = sum(p * n + n * (n + 1) // 2 for n, p in zip(new, prior)) * case["heads"]
    rows = t * case["heads"]
    return dict(bytes=ctx * (WIDTH + 4) + rows * 2 * (WIDTH + LATENT) + 4 * rows,
                flops=2 * pairs * (WIDTH + LATENT))


# ------------------------------------------------------------------ the inputs

def _quantise(x, amax):
    """e4m3 codes and scales of fp32 x; amax broadcasts over what shares a scale."""
    scale = amax.clamp_min(FP8_TINY) / FP8_MAX
    return (x / scale).to(E4M3), scale


def _page_table(lengths, page, gen):
    cols = [-(-n // page) for n in lengths]
    total = sum(cols) + 1
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(lengths), max(max(cols), 1)), dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(cols):
        table[b, :c] = order[at:at + c]
        at += c
    return table, total


def _ragged(case, s):
    new, prior = _lengths(case)
    ro = [0]
    for n in new:
        ro.append(ro[-1] + n)
    s["new"], s["prior"], s["starts"] = new, prior, ro
    s["row_offsets"] = torch.tensor(ro, dtype=torch.int32, device="cuda")
    s["cache_lens"] = torch.tensor(prior, dtype=torch.int32, device="cuda")
    return [n + p for n, p in zip(new, prior)], ro[-1]


def _latent_rows(n, gen):
    """Normalised c_kv and rotated rope dims: bell-shaped, the rows of uneven size."""
    x = torch.randn((n, WIDTH), generator=gen, device="cuda")
    x *= torch.exp(0.3 * torch.randn((n, 1), generator=gen, device="cuda"))
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    if case["op"] == "norm":
        rows, dim = case["rows"], case["dim"]
        s["x"] = randn(rows, case["stride"]).to(torch.bfloat16)[:, :dim]
        s["weight"] = (1 + 0.1 * randn(dim)).to(torch.bfloat16)
        s["eps"] = 1e-6
        s["res"] = (2 * randn(rows, dim)).to(torch.bfloat16) if case["residual"] else None
        s["res_out"] = torch.empty_like(s["res"]) if case["residual"] else None
        if case["fp8"]:
            s["y"] = torch.empty((rows, dim), dtype=E4M3, device="cuda")
            s["y_scales"] = torch.empty((rows, -(-dim // GROUP)), dtype=torch.float32, device="cuda")
        else:
            s["y"] = torch.empty((rows, dim), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // GROUP), -(-n // GROUP)
        x = torch.nn.functional.pad(randn(m, k), (0, kb * GROUP - k)).view(m, kb, GROUP)
        amax = x.abs().amax(dim=(1, 2) if case["row_scale"] else 2, keepdim=True)
        codes, scale = _quantise(x, amax)
        s["x"] = codes.view(m, kb * GROUP)[:, :k].contiguous()
        s["x_scales"] = scale.view(m, 1).expand(m, kb) if case["row_scale"] else scale.view(m, kb).contiguous()
        del x, codes
        w = torch.nn.functional.pad(randn(n, k) / math.sqrt(k), (0, kb * GROUP - k, 0, nb * GROUP - n))
        w = w.view(nb, GROUP, kb, GROUP)
        codes, scale = _quantise(w, w.abs().amax(dim=(1, 3), keepdim=True))
        s["w"] = codes.view(nb * GROUP, kb * GROUP)[:n, :k].contiguous()
        s["w_scales"] = scale.view(nb, kb).contiguous()
        s["out_t"] = torch.empty((m, n), dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32,
                                 device="cuda")
    else:
        lengths, tq = _ragged(case, s)
        s["table"], pages = _page_table(lengths, case["page"], gen)
        rows = _latent_rows(pages * case["page"], gen)
        rows = rows.to(torch.bfloat16).float()
        codes, scale = _quantise(rows, rows.abs().amax(dim=1, keepdim=True))
        del rows
        s["cache"] = codes.view(pages, case["page"], WIDTH)
        s["scales"] = scale.view(pages, case["page"])
        if case["op"] == "append":
            s["rows"] = _latent_rows(tq, gen).to(torch.bfloat16)
        else:
            s["q"] = randn(tq, case["heads"], WIDTH).to(torch.bfloat16)
            s["softmax_scale"] = 1 / math.sqrt(192)
            s["out_t"] = torch.empty((tq, case["heads"], LATENT), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty((tq, case["heads"]), dtype=torch.float32, device="cuda")
            if own:
                from mla_ragged_paged_gb300 import binding
                s["workspace"] = binding.alloc_decode_workspace()
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return dict(norm=_plain_norm, matmul=_plain_matmul, append=_plain_append, decode=_plain_decode)[s["op"]](s)


def _run_own(s):
    from mla_ragged_paged_gb300 import binding
    if s["op"] == "norm":
        if s["fp8"]:
            binding.rms_norm(s["x"], s["weight"], s["eps"], residual=s["res"], residual_out=s["res_out"],
                             out_fp8=s["y"], out_scales=s["y_scales"])
            out = [s["y"], s["y_scales"]]
        else:
            binding.rms_norm(s["x"], s["weight"], s["eps"], residual=s["res"], residual_out=s["res_out"],
                             out=s["y"])
            out = [s["y"]]
        return out + [s["res_out"]] if s["residual"] else out
    if s["op"] == "matmul":
        binding.matmul_fp8(s["out_t"], s["x"], s["x_scales"], s["w"], s["w_scales"])
        return [s["out_t"]]
    if s["op"] == "append":
        binding.append_latent(s["cache"], s["scales"], s["rows"], s["table"], s["row_offsets"], s["cache_lens"])
        return [s["cache"], s["scales"]]
    binding.decode_latent(s["out_t"], s["q"], s["cache"], s["scales"], s["table"], s["row_offsets"],
                          s["cache_lens"], s["softmax_scale"], workspace=s["workspace"], lse=s["lse"])
    return [s["out_t"], s["lse"]]


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"]:
        h = h + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + s["eps"]) * s["weight"].float()
    if s["fp8"]:
        rows, dim = y.shape
        groups = -(-dim // GROUP)
        g = torch.nn.functional.pad(y, (0, groups * GROUP - dim)).view(rows, groups, GROUP)
        codes, scale = _quantise(g, g.abs().amax(dim=2, keepdim=True))
        out = [codes.view(rows, -1)[:, :dim], scale.view(rows, groups)]
    else:
        out = [y.to(torch.bfloat16)]
    return out + [h.to(torch.bfloat16)] if s["residual"] else out


def _plain_matmul(s):
    m, k = s["x"].shape
    n = s["w"].shape[0]
    x = s["x"].float() * s["x_scales"].repeat_interleave(GROUP, dim=1)[:, :k]
    w = s["w"].float() * s["w_scales"].repeat_interleave(GROUP, dim=1)[:, :k].repeat_interleave(GROUP, dim=0)[:n]
    return [(x @ w.t()).to(s["out_t"].dtype)]


def _slots(s, b, first, count):
    """Cache slots of context positions first .. first + count - 1 of sequence b."""
    page = s["cache"].shape[1]
    pos = torch.arange(first, first + count, device="cuda")
    return s["table"][b, pos // page].long() * page + pos % page


def _plain_append(s):
    rows = s["rows"].float()
    codes, scale = _quantise(rows, rows.abs().amax(dim=1, keepdim=True))
    starts = s["row_offsets"].long()
    b = torch.repeat_interleave(starts[1:] - starts[:-1], output_size=len(rows))
    pos = s["cache_lens"][b].long() + torch.arange(len(rows), device="cuda") - starts[b]
    page = s["cache"].shape[1]
    slots = s["table"][b, pos // page].long() * page + pos % page
    s["cache"].view(torch.uint8).view(-1, WIDTH)[slots] = codes.view(torch.uint8)
    s["scales"].view(-1)[slots] = scale[:, 0]
    return [s["cache"], s["scales"]]


def _plain_decode(s):
    heads = s["heads"]
    codes, scales = s["cache"].view(torch.uint8).view(-1, WIDTH), s["scales"].view(-1)
    outs, lses = [], []
    for b, (n, p) in enumerate(zip(s["new"], s["prior"])):
        slots = _slots(s, b, 0, n + p)
        k = codes[slots].view(E4M3).float() * scales[slots][:, None]
        q = s["q"][s["starts"][b]:s["starts"][b + 1]].float().reshape(n * heads, WIDTH)
        x = (q @ k.t() * s["softmax_scale"]).view(n, heads, n + p)
        i = torch.arange(n, device="cuda")
        hidden = torch.arange(n + p, device="cuda")[None, :] > p + i[:, None]
        x = x.masked_fill(hidden[:, None, :], float("-inf"))
        top = x.amax(dim=2, keepdim=True)
        e = torch.exp(x - top)
        total = e.sum(dim=2, keepdim=True)
        outs.append(((e / total).view(n * heads, n + p) @ k[:, :LATENT]).view(n, heads, LATENT))
        lses.append((top + torch.log(total))[:, :, 0])
    return [torch.cat(outs).to(torch.bfloat16), torch.cat(lses)]


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:
            h += s["res"].double()
        norm = torch.linalg.vector_norm(h, dim=1) / math.sqrt(case["dim"])
        y = h / torch.hypot(norm, torch.full_like(norm, math.sqrt(s["eps"])))[:, None]
        y *= s["weight"].double()
        tail = [h] if case["residual"] else []
        if not case["fp8"]:
            return [y] + tail
        scales = torch.stack([c.abs().max(dim=1).values for c in y.split(GROUP, dim=1)], dim=1)
        scales = scales.clamp(min=FP8_TINY) / FP8_MAX
        for j, c in enumerate(y.split(GROUP, dim=1)):
            c /= scales[:, j:j + 1]
        return [y, scales] + tail
    if case["op"] == "matmul":
        out = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        w = s["w"].double()
        for j in range(s["w_scales"].shape[1]):
            cols = slice(j * GROUP, min((j + 1) * GROUP, case["k"]))
            column = torch.repeat_interleave(s["w_scales"][:, j].double(), GROUP)[:case["n"]]
            out += (s["x"][:, cols].double() @ w[:, cols].t()) * s["x_scales"][:, j:j + 1].double() * column
        return [out]
    page = case["page"]
    if case["op"] == "append":
        cache = s["cache"].double()
        scales = s["scales"].double()
        t = 0
        table = s["table"].tolist()
        b_of, pos = [], []
        for b, (n, p) in enumerate(zip(s["new"], s["prior"])):
            b_of += [b] * n
            pos += range(p, p + n)
        for t0 in range(0, len(pos), 4096):
            part = range(t0, min(t0 + 4096, len(pos)))
            pg = torch.tensor([table[b_of[t]][pos[t] // page] for t in part], device="cuda")
            sl = torch.tensor([pos[t] % page for t in part], device="cuda")
            x = s["rows"][t0:t0 + 4096].double()
            sc = x.abs().max(dim=1).values.clamp(min=FP8_TINY) / FP8_MAX
            cache[pg, sl] = x / sc[:, None]
            scales[pg, sl] = sc
        return [cache, scales]
    out = torch.empty((s["starts"][-1], case["heads"], LATENT), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["starts"][-1], case["heads"]), dtype=torch.float64, device="cuda")
    flat = s["cache"].view(torch.uint8).view(-1, WIDTH)
    for b, (n, p) in enumerate(zip(s["new"], s["prior"])):
        pages = s["table"][b, :-(-(n + p) // page)].long()
        slots = (pages[:, None] * page + torch.arange(page, device="cuda")).view(-1)[:n + p]
        k = flat[slots].view(E4M3).double()
        k *= s["scales"].view(-1)[slots].double()[:, None]
        for i in range(n):
            seen = k[:p + i + 1]
            x = torch.einsum("hd,jd->hj", s["q"][s["starts"][b] + i].double(), seen) * s["softmax_scale"]
            z = torch.logsumexp(x, dim=1)
            lse[s["starts"][b] + i] = z
            out[s["starts"][b] + i] = torch.exp(x - z[:, None]) @ seen[:, :LATENT]
    return [out, lse]
