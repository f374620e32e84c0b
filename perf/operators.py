"""Measured cases of the paged-cache operators: the head norm with rotary
embedding, the paged append (with the read-back of what it stored) and paged
attention of new tokens.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, where ``own`` is set, through the library.  Shapes are the ones of
the library's synthetic workloads: GPT-2-small (12 heads, head_dim 64),
Llama-2-13B (40 heads, head_dim 128), the serving mix (32 query heads over 8,
head_dim 128) and the wide-GQA model (16 query heads over 2, head_dim 256).
"""
import math
import random

import torch

own = False

PAIRS, HALVES = 0, 1
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of the serving mix: 64 tokens, norm and rotation before the cache
        dict(name="norm_rope_step", op="norm_rope", tokens=64, q_heads=32, kv_heads=8, head_dim=128, dtype="bf16",
             rope_dim=128, style=HALVES, rows=32768),
        # a long prompt of the wide-GQA model: its keys pass a norm before the cache, a quarter of the channels turn
        dict(name="norm_rope_prompt", op="norm_rope", tokens=65521, q_heads=16, kv_heads=2, head_dim=256, dtype="f16",
             rope_dim=64, style=PAIRS, rows=131072),
        # one decode step of the serving mix into 4-bit pages
        dict(name="append_step", op="append", batch=64, new_lo=1, new_hi=1, past_lo=1023, past_hi=32767, kv_heads=8,
             head_dim=128, dtype="bf16", page_tokens=16, k_bits=4, v_bits=4, group=64, rope_dim=128, style=HALVES,
             shape=1),
        # ragged prompts of the Llama-2-13B shape into fp16 pages
        dict(name="append_prompts", op="append", batch=16, new_lo=1, new_hi=4113, past_lo=0, past_hi=0, kv_heads=40,
             head_dim=128, dtype="f16", page_tokens=64, k_bits=16, v_bits=16, group=32, rope_dim=128, style=PAIRS,
             shape=2),
        # GPT-2-small prompts (learned positions, no rotation) into 8-bit keys and 4-bit values
        dict(name="append_prompts_8_4", op="append", batch=8, new_lo=1900, new_hi=2048, past_lo=0, past_hi=0,
             kv_heads=12, head_dim=64, dtype="f16", page_tokens=32, k_bits=8, v_bits=4, group=32, rope_dim=0,
             style=PAIRS, shape=3),
        # single tokens, few heads: where the launch and the join of the splits count
        dict(name="attn_step_small", op="attn", batch=8, new_lo=1, new_hi=1, past_lo=2047, past_hi=2047, q_heads=12,
             kv_heads=12, head_dim=64, dtype="f16", page_tokens=32, k_bits=16, v_bits=16, group=32, window=0, pad=0,
             shape=4),
        # single tokens of the serving mix over 4-bit pages: 64 sequences of 1k to 32k tokens
        dict(name="attn_step_mix_4bit", op="attn", batch=64, new_lo=1, new_hi=1, past_lo=1023, past_hi=32767,
             q_heads=32, kv_heads=8, head_dim=128, dtype="bf16", page_tokens=16, k_bits=4, v_bits=4, group=64,
             window=0, pad=0, shape=5),
        # single tokens of the Llama-2-13B shape over bf16 pages
        dict(name="attn_step_bf16", op="attn", batch=16, new_lo=1, new_hi=1, past_lo=4112, past_hi=4112, q_heads=40,
             kv_heads=40, head_dim=128, dtype="bf16", page_tokens=64, k_bits=16, v_bits=16, group=32, window=0, pad=0,
             shape=6),
        # drafted tokens to be verified: five a sequence, a batch padded behind its last token
        dict(name="attn_drafts_8bit", op="attn", batch=16, new_lo=5, new_hi=5, past_lo=1000, past_hi=16384,
             q_heads=32, kv_heads=8, head_dim=128, dtype="bf16", page_tokens=64, k_bits=8, v_bits=8, group=32,
             window=0, pad=7, shape=7),
        # a chunk of a long prompt
        dict(name="attn_chunk_bf16", op="attn", batch=1, new_lo=2048, new_hi=2048, past_lo=30720, past_hi=30720,
             q_heads=32, kv_heads=8, head_dim=128, dtype="bf16", page_tokens=128, k_bits=16, v_bits=16, group=32,
             window=0, pad=0, shape=8),
        # a short chunk at the end of the wide-GQA model's context, 4-bit keys and 8-bit values
        dict(name="attn_chunk_wide_4_8", op="attn", batch=1, new_lo=509, new_hi=509, past_lo=130563, past_hi=130563,
             q_heads=16, kv_heads=2, head_dim=256, dtype="f16", page_tokens=64, k_bits=4, v_bits=8, group=32,
             window=0, pad=0, shape=9),
        # ragged first prompts of the Llama-2-13B shape, each token seeing the last 1024
        dict(name="attn_prompts_window", op="attn", batch=8, new_lo=1, new_hi=2048, past_lo=0, past_hi=0, q_heads=40,
             kv_heads=40, head_dim=128, dtype="f16", page_tokens=16, k_bits=16, v_bits=16, group=32, window=1024,
             pad=0, shape=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(12, 12, 64), (8, 8, 64), (40, 40, 128), (32, 8, 128), (16, 16, 128), (16, 2, 256)]


def _format(rng, head_dim):
    k_bits, v_bits = rng.choice([(16, 16), (16, 16), (8, 8), (4, 4), (8, 4), (4, 8)])
    return dict(page_tokens=rng.choice([16, 32, 64, 128]), k_bits=k_bits, v_bits=v_bits,
                group=rng.choice([g for g in (32, 64, 128, 256) if g <= head_dim]))


def draw(rng):
    q_heads, kv_heads, head_dim = rng.choice(HEADS)
    heads = dict(q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim)
    op = rng.choice(["norm_rope", "append", "attn", "attn", "attn"])
    rope = dict(rope_dim=rng.choice([d for d in (32, 64, 128, 256) if d <= head_dim]), style=rng.choice([PAIRS, HALVES]))
    shape = rng.randrange(1 << 30)
    if op == "norm_rope":
        most = 65521 * 18 * 256 // ((q_heads + kv_heads) * head_dim)
        tokens = _log(rng, 1, most)
        return dict(op=op, tokens=tokens, dtype=rng.choice(["f16", "bf16", "f32"]), rows=rng.choice([8192, 32768]),
                    **heads, **rope)
    if op == "append":
        batch = _log(rng, 1, 64)
        most = max(1, 32768 * 40 * 128 // (batch * kv_heads * head_dim))
        hi = _log(rng, 1, min(8192, most))
        past = rng.choice([0, _log(rng, 1, 16384)])
        if rng.random() < 0.25:
            rope["rope_dim"] = 0
        return dict(op=op, batch=batch, new_lo=rng.choice([0, 1, hi]), new_hi=hi, past_lo=past // 2, past_hi=past,
                    kv_heads=kv_heads, head_dim=head_dim, dtype=rng.choice(["f16", "bf16", "f32"]), shape=shape,
                    **_format(rng, head_dim), **rope)
    kind = rng.choice(["step", "drafts", "chunk", "prompts"])
    if kind in ("step", "drafts"):
        batch, new_hi = _log(rng, 1, 64), 1 if kind == "step" else rng.randint(2, 16)
        past_hi = _log(rng, 1, max(2, min(65536, 10**9 // (batch * kv_heads * head_dim))))
    elif kind == "chunk":
        batch, new_hi = rng.randint(1, 4), _log(rng, 17, 2048)
        past_hi = _log(rng, 16, 65536)
    else:
        batch, new_hi, past_hi = rng.randint(1, 12), _log(rng, 17, 2048), 0
    # scores of the plain form, and the cache, stay within the largest listed case's
    past_hi = min(past_hi, max(0, 10**9 // (batch * q_heads * new_hi) - new_hi),
                  max(0, 10**9 // (batch * kv_heads * head_dim) - new_hi))
    window = rng.choice([0, 0, _log(rng, 16, 8192)])
    return dict(op=op, batch=batch, new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi, past_lo=past_hi // 4,
                past_hi=past_hi, dtype=rng.choice(["f16", "bf16"]), window=window, pad=rng.choice([0, 0, 5]),
                shape=shape, **heads, **_format(rng, head_dim))


def sequences(case):
    """[(new tokens, length with them)] of the case's sequences; one of them at least has a token."""
    r = random.Random(case["shape"])
    got = []
    for _ in range(case["batch"]):
        n = r.randint(case["new_lo"], case["new_hi"])
        got.append([n, n + r.randint(case["past_lo"], case["past_hi"])])
    if not any(n for n, _ in got):
        got[0] = [1, got[0][1] + 1]
    return got


def _row_bytes(case, bits):
    d = case["head_dim"]
    return 2.0 * d if bits == 16 else d * bits / 8 + 4.0 * d / case["group"]


def work(case):
    d = case["head_dim"]
    size = {"f16": 2, "bf16": 2, "f32": 4}[case["dtype"]]
    if case["op"] == "norm_rope":
        values = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * d
        return {"bytes": 2.0 * size * values + 4.0 * case["rope_dim"] * case["tokens"], "flops": 7.0 * values}
    seqs, h = sequences(case), case["kv_heads"]
    held = _row_bytes(case, case["k_bits"]) + _row_bytes(case, case["v_bits"])
    if case["op"] == "append":
        n = sum(s[0] for s in seqs)
        # the rows in, what the pages hold of them, the rows read back, the table of angles
        return {"bytes": n * h * (2.0 * d * size + held + 4.0 * d) + 4.0 * case["rope_dim"] * n, "flops": 10.0 * n * h * d}
    w, seen, rows, pairs = case["window"], 0, 0, 0
    for n, ln in seqs:
        rows += n
        if n:
            seen += ln if not w else min(ln, w + n - 1)
        for i in range(n):
            p = ln - n + i + 1
            pairs += min(p, w) if w else p
    return {"bytes": seen * h * held + 4.0 * rows * case["q_heads"] * d, "flops": 4.0 * pairs * case["q_heads"] * d}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _angles(rows, dim):
    """[rows][dim / 2][2] cosines and sines of position * 10000^(-2i / dim), from 64-bit angles."""
    f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()


def _offsets(counts):
    return torch.tensor([0] + counts, dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)


def _table(lens, page_tokens, g):
    """(table [batch][longest], pages): every sequence's pages, dealt at random from the pool."""
    counts = [-(-n // page_tokens) for n in lens]
    pages = sum(counts) + 3
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int64).int()
    table = torch.full((len(lens), max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    return table, pages


def _keys_values(case, n, g, dtype):
    """[n][kv_heads][head_dim] keys (four large channels a head) and values, as two slices of one projection."""
    h, d = case["kv_heads"], case["head_dim"]
    kv = _normal(g, n, 2, h, d)
    big = torch.rand(h, d, generator=g, device="cuda").argsort(dim=-1)[:, :4]
    kv[:, 0] *= torch.ones(h, d, device="cuda").scatter_(1, big, 6.0)
    kv = kv.to(dtype)
    return kv[:, 0], kv[:, 1]


def _inputs(case, seed):
    g = _gen(seed)
    s = {"op": case["op"], "case": case}
    d = case["head_dim"]
    if case["op"] == "norm_rope":
        n, hq, h, t = case["tokens"], case["q_heads"], case["kv_heads"], TYPES[case["dtype"]]
        qkv = (_normal(g, n, hq + 2 * h, d) * 1.7).to(t)  # one row of the query, key and value projections a token
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + h]
        s["qw"], s["kw"] = ((1.0 + 0.3 * _normal(g, d)).to(t) for _ in range(2))
        s["positions"] = torch.randint(0, case["rows"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["angles"] = _angles(case["rows"], case["rope_dim"])
        return s
    seqs = sequences(case)
    news, lens = [x[0] for x in seqs], [x[1] for x in seqs]
    s["n"], s["most_new"], s["longest"] = sum(news), max(news), max(lens)
    s["q_start"] = _offsets(news)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["table"], s["pages"] = _table(lens, case["page_tokens"], g)
    if case["op"] == "append":
        s["k"], s["v"] = _keys_values(case, s["n"], g, TYPES[case["dtype"]])
        s["angles"] = _angles(max(lens), case["rope_dim"]) if case["rope_dim"] else None
        return s
    # the cache's contents, all tokens of all sequences in order; what pages hold is 16-bit or made from fp16 rows
    held = torch.float16 if case["k_bits"] < 16 else TYPES[case["dtype"]]
    s["k"], s["v"] = _keys_values(case, sum(lens), g, held)
    s["k_start"] = _offsets(lens)
    s["q"] = _normal(g, s["n"] + case["pad"], case["q_heads"], d).to(TYPES[case["dtype"]])
    s["out"] = torch.zeros_like(s["q"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm_rope":
        if own:
            from bit_quantized_kv_02_gb300 import kvq
            s["kvq"], s["rope"] = kvq, kvq.Rope(s["angles"], case["style"], s["positions"])
        return s
    h, d, pt = case["kv_heads"], case["head_dim"], case["page_tokens"]
    quantized = case["k_bits"] < 16
    if own:
        from bit_quantized_kv_02_gb300 import kvq
        fmt = [None if b == 16 else (b, case["group"], kvq.PER_TOKEN, kvq.ASYM) for b in (case["k_bits"], case["v_bits"])]
        dtype = kvq.BF16 if case["dtype"] == "bf16" and not quantized else kvq.F16
        cfg = kvq.make_pages_config(1, s["pages"], pt, case.get("q_heads", h), h, d, *fmt, dtype=dtype)
        s["cache"] = kvq.KVQPages(cfg)
        s["batch"] = kvq.PagesBatch(s["q_start"], s["lens"], s["table"], s["n"] + case.get("pad", 0), s["most_new"])
        if case["op"] == "append":
            s["rope"] = kvq.Rope(s["angles"], case["style"]) if case["rope_dim"] else None
        else:
            s["cache"].kvq_pages_append(0, s.pop("k"), s.pop("v"),
                                        kvq.PagesBatch(s["k_start"], s["lens"], s["table"], int(s["k_start"][-1])))
        return s
    if quantized:
        for name in ("k", "v"):
            s["pool_" + name] = [torch.zeros((s["pages"], pt, h, d), dtype=torch.uint8, device="cuda")] + [
                torch.zeros((s["pages"], pt, h, d // case["group"]), dtype=torch.float16, device="cuda") for _ in range(2)]
    else:
        held = torch.float16 if case["dtype"] != "bf16" else torch.bfloat16
        for name in ("k", "v"):
            s["pool_" + name] = [torch.zeros((s["pages"], pt, h, d), dtype=held, device="cuda")]
    if case["op"] == "attn":
        page, slot, _ = _slots(s["k_start"], s["lens"], s["table"], pt, s["k"].shape[0])
        for name in ("k", "v"):
            _store(s["pool_" + name], page, slot, s.pop(name), case[name + "_bits"], case["group"])
    return s


# ------------------------------------------------------------- plain form --

def _rotate(x, cs, dim, style):
    """x [n][heads][d] in 32 bits; cs [n][dim / 2][2]."""
    c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
    y = x.clone()
    if style == PAIRS:
        a, b = x[..., 0:dim:2], x[..., 1:dim:2]
        y[..., 0:dim:2], y[..., 1:dim:2] = a * c - b * sn, b * c + a * sn
    else:
        a, b = x[..., :dim // 2], x[..., dim // 2:dim]
        y[..., :dim // 2], y[..., dim // 2:dim] = a * c - b * sn, b * c + a * sn
    return y


def _norm_rope(x, weight, cs, dim, style, eps):
    f = x.float()
    f = f * torch.rsqrt((f * f).mean(dim=-1, keepdim=True) + eps) * weight.float()
    return _rotate(f, cs, dim, style).to(x.dtype)


def _next16(h, up):
    """The next fp16 value above (below) h."""
    i = h.view(torch.int16)
    away = (i >= 0) == up  # further from zero
    step = torch.where(i == 0, torch.full_like(i, 1 if up else -32767), torch.where(away, i + 1, i - 1))
    return step.view(torch.float16)


def _round16(x, up):
    """x in fp16, rounded up (down)."""
    h = x.half()
    off = (h.float() < x) if up else (h.float() > x)
    return torch.where(off, _next16(h, up), h)


def _codes(x, bits, group):
    """(codes, zero points, steps) of x [n][heads][d], groups of `group` channels."""
    n, h, d = x.shape
    g = x.float().reshape(n, h, d // group, group)
    lo, hi = g.amin(dim=-1), g.amax(dim=-1)
    zero = _round16(lo + 0.0, False)
    levels = torch.full_like(hi, float(2 ** bits - 1))
    step = _round16((hi - zero.float()) / levels, True)
    z, st = zero.float()[..., None], step.float()[..., None]
    c = torch.where(st == 0, torch.zeros_like(g), ((g - z) / st).round().clamp(0, 2 ** bits - 1))
    return c.to(torch.uint8).reshape(n, h, d), zero, step


def _slots(start, lens, table, page_tokens, n):
    """(page, slot, position) of n rows of new tokens: row i of sequence b is token lens[b] - new + i."""
    row = torch.arange(n, device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), row, right=True)
    pos = lens[b].long() - start[b + 1].long() + row
    return table[b, pos // page_tokens].long(), pos % page_tokens, pos


def _store(pool, page, slot, x, bits, group):
    if bits == 16:
        pool[0][page, slot] = x.to(pool[0].dtype)
    else:
        for p, y in zip(pool, _codes(x, bits, group)):
            p[page, slot] = y


def _held(pool, page, slot, group):
    """What the pool holds at (page, slot): 16-bit values, or zero point + code * step rounded to fp16."""
    if len(pool) == 1:
        return pool[0][page, slot]
    c, zero, step = (p[page, slot] for p in pool)
    g = c.float().unflatten(-1, (-1, group))
    return torch.addcmul(zero.float()[..., None], g, step.float()[..., None]).flatten(-2).half()


def _append(s):
    case = s["case"]
    page, slot, pos = _slots(s["q_start"], s["lens"], s["table"], case["page_tokens"], s["n"])
    k, v = s["k"].float(), s["v"].float()
    if case["rope_dim"]:
        k = _rotate(k, s["angles"][pos], case["rope_dim"], case["style"])
    _store(s["pool_k"], page, slot, k, case["k_bits"], case["group"])
    _store(s["pool_v"], page, slot, v, case["v_bits"], case["group"])
    return _held(s["pool_k"], page, slot, case["group"]), _held(s["pool_v"], page, slot, case["group"])


def _attn(s):
    case = s["case"]
    batch, hq, h, d = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"]
    rep, n, t = hq // h, s["most_new"], s["longest"]
    lens, start, q = s["lens"].long(), s["q_start"].long(), s["q"]
    at = torch.arange(t, device="cuda")
    page = s["table"][:, at // case["page_tokens"]].clamp_min(0).long()
    slot = (at % case["page_tokens"]).expand_as(page)
    k = _held(s["pool_k"], page, slot, case["group"]).permute(0, 2, 3, 1).float()  # [batch][h][d][t]
    v = _held(s["pool_v"], page, slot, case["group"]).permute(0, 2, 1, 3).float()  # [batch][h][t][d]
    i = torch.arange(n, device="cuda")
    new = start[1:] - start[:-1]
    row = (start[:-1, None] + i).clamp_max(q.shape[0] - 1)  # [batch][n]
    x = (q[row].float() * (1.0 / math.sqrt(d))).reshape(batch, n, h, rep, d).permute(0, 2, 3, 1, 4)
    score = (x.reshape(batch, h, rep * n, d) @ k).reshape(batch, h, rep, n, t)
    del k
    pos = (lens - new)[:, None] + i
    hide = at[None, None, :] > pos[..., None]
    if case["window"]:
        hide |= at[None, None, :] <= pos[..., None] - case["window"]
    score.masked_fill_(hide[:, None, None], float("-inf"))
    top = score.amax(dim=-1, keepdim=True).clamp_min(-3.0e38)
    score.sub_(top).exp_()
    total = score.sum(dim=-1, keepdim=True)
    o = score.reshape(batch, h, rep * n, t) @ v
    o = o.reshape(batch, h, rep, n, d) / total.clamp_min(1e-38)
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, n, hq, d).to(q.dtype)
    is_new = i[None, :] < new[:, None]
    s["out"][row[is_new]] = o[is_new]
    return s["out"]


def run(s):
    case = s["case"]
    if s["op"] == "norm_rope":
        if own:
            return s["kvq"].kvq_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], eps=1e-6, rope=s["rope"])
        cs = s["angles"][s["positions"].long()]
        return tuple(_norm_rope(x, w, cs, case["rope_dim"], case["style"], 1e-6)
                     for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    if s["op"] == "append":
        if own:
            s["cache"].kvq_pages_append(0, s["k"], s["v"], s["batch"], rope=s["rope"])
            return s["cache"].kvq_pages_read(0, s["batch"])
        return _append(s)
    if own:
        return s["cache"].kvq_pages_attn(0, s["q"], s["batch"], out=s["out"], window=case["window"])
    return _attn(s)


# ------------------------------------------------------------------ exact --

def _turned(x, angles, dim, style):
    """x [n][heads][d] in 64 bits as complex numbers times e^(i angle)."""
    w = torch.view_as_complex(angles.double().contiguous())[:, None]
    head, rest = x[..., :dim], x[..., dim:]
    if style == PAIRS:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], dim // 2, 2).contiguous()) * w
        head = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(head[..., :dim // 2].contiguous(), head[..., dim // 2:].contiguous()) * w
        head = torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([head, rest], dim=-1)


def _grid16(x, rounding):
    """x on the fp16 grid, by `rounding` (torch.floor or torch.ceil) of its multiple of the grid's spacing."""
    unit = torch.exp2(torch.frexp(x)[1].double().sub(1).clamp_min(-14) - 10)
    return rounding(x / unit) * unit


def _as_held(x, bits, group, dtype):
    """What pages hold of x (64 bits), in 64 bits."""
    if bits == 16:
        return x if dtype is None else x.to(dtype).double()
    y = x.unflatten(-1, (-1, group))
    zero = _grid16(y.amin(dim=-1, keepdim=True), torch.floor)
    step = ((y.amax(dim=-1, keepdim=True) - zero) / (2 ** bits - 1)).float().double()
    step = _grid16(step, torch.ceil)
    code = torch.where(step > 0, (y - zero) / step, torch.zeros_like(y)).round().clamp(0, 2 ** bits - 1)
    return (zero + code * step).flatten(-2).half().double()


def exact(case, seed):
    s = _inputs(case, seed)
    d = case["head_dim"]
    if case["op"] == "norm_rope":
        got = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for a in range(0, x.shape[0], 8192):
                f = x[a:a + 8192].double()
                f = f / (f.square().sum(dim=-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
                y[a:a + 8192] = _turned(f, s["angles"][s["positions"][a:a + 8192].long()], case["rope_dim"], case["style"])
            got.append(y)
        return tuple(got)
    seqs = sequences(case)
    if case["op"] == "append":
        pos = torch.cat([torch.arange(ln - n, ln, device="cuda") for n, ln in seqs])
        ks, vs = [], []
        for a in range(0, s["n"], 4096):
            k, v = s["k"][a:a + 4096].double(), s["v"][a:a + 4096].double()
            if case["rope_dim"]:
                k = _turned(k, s["angles"][pos[a:a + 4096]], case["rope_dim"], case["style"])
            ks.append(_as_held(k, case["k_bits"], case["group"], None))
            vs.append(_as_held(v, case["v_bits"], case["group"], None))
        return torch.cat(ks), torch.cat(vs)
    hq, h = case["q_heads"], case["kv_heads"]
    rep = hq // h
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    a = b = 0
    for n, ln in seqs:
        if n:
            key = torch.arange(ln, device="cuda")
            query = torch.arange(ln - n, ln, device="cuda")[:, None]
            see = key <= query
            if case["window"]:
                see &= key > query - case["window"]
            k = _as_held(s["k"][b:b + ln].double(), case["k_bits"], case["group"], None)
            v = _as_held(s["v"][b:b + ln].double(), case["v_bits"], case["group"], None)
            for j in range(hq):
                p = s["q"][a:a + n, j].double() @ k[:, j // rep].T / math.sqrt(d)
                p = torch.softmax(p.masked_fill(~see, float("-inf")), dim=-1)
                out[a:a + n, j] = p @ v[:, j // rep]
        a, b = a + n, b + ln
    return out
