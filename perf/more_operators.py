"""Measured cases of the paged cache's branching operators: attention of drafted
trees and cross attention, keeping some of a sequence's tokens, copying pages, and
forking sequences with the pages their next tokens need.

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

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --

def listed():
    small = dict(q_heads=12, kv_heads=12, head_dim=64)
    llama = dict(q_heads=40, kv_heads=40, head_dim=128)
    mix = dict(q_heads=32, kv_heads=8, head_dim=128)
    wide = dict(q_heads=16, kv_heads=2, head_dim=256)
    return [
        # one stream with a small drafted tree: the tree and four layers, where launches and joins count
        dict(name="tree_small", op="tree", batch=1, new_lo=13, new_hi=13, past_lo=1000, past_hi=1000, words=1, layers=4,
             window=0, pad=0, dtype="f16", page_tokens=32, k_bits=16, v_bits=16, group=32, shape=1, **small),
        # the serving mix verifies 64 drafted tokens a sequence over bf16 pages
        dict(name="tree_mix_bf16", op="tree", batch=16, new_lo=64, new_hi=64, past_lo=1000, past_hi=16384, words=1,
             layers=1, window=0, pad=0, dtype="bf16", page_tokens=64, k_bits=16, v_bits=16, group=32, shape=2, **mix),
        # ragged trees over 4-bit pages, a batch padded behind its last token
        dict(name="tree_ragged_4bit", op="tree", batch=32, new_lo=1, new_hi=31, past_lo=500, past_hi=8192, words=1,
             layers=1, window=0, pad=7, dtype="bf16", page_tokens=16, k_bits=4, v_bits=4, group=64, shape=3, **mix),
        # a wide tree at the end of the wide-GQA model's context, 4-bit keys and 8-bit values
        dict(name="tree_long_wide", op="tree", batch=1, new_lo=125, new_hi=125, past_lo=130900, past_hi=130900, words=2,
             layers=1, window=0, pad=0, dtype="f16", page_tokens=64, k_bits=4, v_bits=8, group=32, shape=4, **wide),
        # single decoder tokens over encoder states of up to 1500 positions
        dict(name="cross_step", op="cross", batch=64, new_lo=1, new_hi=1, past_lo=100, past_hi=1500, layers=1, pad=0,
             dtype="f16", page_tokens=32, k_bits=16, v_bits=16, group=32, shape=5, **small),
        # ragged decoder prompts over longer encoder states in 8-bit pages
        dict(name="cross_prompts_8bit", op="cross", batch=8, new_lo=1, new_hi=448, past_lo=1, past_hi=8190, layers=1,
             pad=0, dtype="bf16", page_tokens=64, k_bits=8, v_bits=8, group=64, shape=6, **mix),
        # the drafted tokens that were accepted, 64 drafted a sequence, four layers at once
        dict(name="keep_drafts", op="keep", batch=16, new_lo=64, new_hi=64, past_lo=1000, past_hi=16384, sinks=1,
             most=0.1, layers=4, dtype="bf16", page_tokens=64, k_bits=16, v_bits=16, group=32, shape=7, **mix),
        # long sequences cut to their first tokens and the better half of the later ones, 4-bit pages
        dict(name="keep_half_4bit", op="keep", batch=8, new_lo=9000, new_hi=16400, past_lo=0, past_hi=0, sinks=4,
             most=0.45, layers=4, dtype="f16", page_tokens=16, k_bits=4, v_bits=4, group=64, shape=8, **mix),
        # a few pages of all of GPT-2-small's layers
        dict(name="copy_few", op="copy", copies=5, pages=300, layers=12, dtype="f16", page_tokens=16, k_bits=16, v_bits=16,
             group=32, shape=9, **small),
        # many pages of the Llama-2-13B shape, 8-bit keys and 4-bit values
        dict(name="copy_many_8_4", op="copy", copies=509, pages=1100, layers=4, dtype="f16", page_tokens=64, k_bits=8,
             v_bits=4, group=64, shape=10, **llama),
        # a step of beam search: 16 prompts with 4 beams each, one token more
        dict(name="branch_beams", op="branch", groups=16, beams=4, prompt_lo=100, prompt_hi=4000, tail=30, new_lo=1,
             new_hi=1, layers=4, dtype="bf16", page_tokens=16, k_bits=16, v_bits=16, group=32, spare=1000, shape=11, **mix),
        # many samples of few long prompts with drafted chunks of up to 600 tokens, a pool of 60000 pages
        dict(name="branch_samples", op="branch", groups=8, beams=32, prompt_lo=2000, prompt_hi=30000, tail=200, new_lo=1,
             new_hi=600, layers=1, dtype="f16", page_tokens=16, k_bits=4, v_bits=4, group=64, spare=42000, shape=12, **wide),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(12, 12, 64), (8, 8, 64), (40, 40, 128), (32, 8, 128), (16, 16, 128), (16, 2, 256)]


def draw(rng):
    q_heads, kv_heads, head_dim = rng.choice(HEADS)
    k_bits, v_bits = rng.choice([(16, 16), (16, 16), (8, 8), (4, 4), (8, 4), (4, 8)])
    c = dict(op=rng.choice(["tree", "tree", "cross", "keep", "copy", "branch"]), q_heads=q_heads, kv_heads=kv_heads,
             head_dim=head_dim, dtype=rng.choice(["f16", "bf16"]), page_tokens=rng.choice([16, 32, 64, 128]),
             k_bits=k_bits, v_bits=v_bits, group=rng.choice([g for g in (32, 64, 128, 256) if g <= head_dim]),
             layers=rng.choice([1, 2, 4]), shape=rng.randrange(1 << 30))
    row = kv_heads * head_dim * c["layers"]  # channels of a token in all layers
    if c["op"] in ("tree", "cross"):
        if c["op"] == "tree":
            c["words"] = rng.choice([1, 1, 1, 2, 4])
            new_hi, batch = _log(rng, 2, 64 * c["words"]), _log(rng, 1, 64)
            c["window"] = rng.choice([0, 0, _log(rng, 64 * c["words"], 8192)])
        else:
            new_hi, batch = rng.choice([1, _log(rng, 2, 512)]), _log(rng, 1, 64)
        most = min(6 * 10**8 // (batch * q_heads * new_hi * c["layers"]), 2 * 10**8 // (batch * row))
        past_hi = _log(rng, 1, max(2, min(65536, most)))
        return dict(c, batch=batch, new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi,
                    past_lo=rng.choice([0, past_hi // 4, past_hi]), past_hi=past_hi, pad=rng.choice([0, 0, 5]))
    if c["op"] == "keep":
        batch = _log(rng, 1, 32)
        new_hi = _log(rng, 2, max(4, min(16000, 10**8 // (batch * row))))
        past_hi = rng.choice([0, _log(rng, 1, max(2, min(8000, 10**8 // (batch * row))))])
        return dict(c, batch=batch, new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi, past_lo=past_hi // 3,
                    past_hi=past_hi, sinks=rng.choice([0, 1, 4]), most=rng.uniform(0.02, 0.5))
    page = row * c["page_tokens"]
    if c["op"] == "copy":
        copies = _log(rng, 1, max(2, min(800, 2 * 10**8 // page)))
        return dict(c, copies=copies, pages=2 * copies + rng.randint(1, 9 + copies // 4))
    groups, beams = _log(rng, 1, 16), rng.randint(1, 16)
    tokens = max(40, min(30000, 10**8 // (row * (groups + beams))))
    prompt_hi, new_hi = _log(rng, 20, tokens), rng.choice([1, _log(rng, 2, max(3, min(600, tokens // beams)))])
    tail = rng.randint(0, max(1, min(200, tokens // beams)))
    need = groups * beams * (2 + (tail + new_hi) // c["page_tokens"])
    return dict(c, groups=groups, beams=beams, prompt_lo=prompt_hi // 3 + 1, prompt_hi=prompt_hi, tail=tail,
                new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi,
                spare=need + _log(rng, 1, max(2, 2 * 10**8 // page)))


def sequences(case):
    """[(new tokens, length)] of the case's sequences (cross: the encoder's length); one of them at least has a token."""
    r = random.Random(case["shape"])
    got = []
    for _ in range(case["batch"]):
        n = r.randint(case["new_lo"], case["new_hi"])
        got.append([n, (0 if case["op"] == "cross" else n) + r.randint(case["past_lo"], case["past_hi"])])
    if not any(n for n, _ in got):
        got[0] = [1, got[0][1] + 1]
    return got


def keeps(case):
    """Rows to keep of each sequence's new tokens: the first ones, then some of those behind the place where the last kept one goes."""
    r = random.Random(case["shape"] + 1)
    got = []
    for n, _ in sequences(case):
        m = min(n, max(1, int(n * case["most"])))
        a = min(m, case["sinks"])
        got.append(list(range(a)) + sorted(r.sample(range(m, n), min(m - a, n - m))))
    return got


def branches(case):
    """(lengths, new tokens, prompts) of the case's sequences, groups of beams of one length over a shared prompt."""
    r = random.Random(case["shape"])
    prompts = [r.randint(case["prompt_lo"], case["prompt_hi"]) for _ in range(case["groups"])]
    lens = [x for x in (p + r.randint(0, case["tail"]) for p in prompts) for _ in range(case["beams"])]
    return lens, [r.randint(case["new_lo"], case["new_hi"]) for _ in lens], prompts


def _row_bytes(case, bits):
    d = case["head_dim"]
    return 2.0 * d if bits == 16 else d * bits / 8 + 4.0 * d / case["group"]


def work(case):
    d, h, layers, pt = case["head_dim"], case["kv_heads"], case["layers"], case["page_tokens"]
    held = h * (_row_bytes(case, case["k_bits"]) + _row_bytes(case, case["v_bits"]))  # of a token in a layer
    read = h * 4.0 * d  # a token's key and value rows as they are read back
    if case["op"] == "copy":
        n = case["copies"] * pt * layers
        return {"bytes": n * (3.0 * held + read), "flops": 0.0}  # read and written once, then what was stored is read
    if case["op"] == "branch":
        lens, news, _ = branches(case)
        parts = sum(x % pt for x in lens) * layers
        entries = sum(-(-x // pt) for x in lens)
        return {"bytes": parts * (3.0 * held + read) + 8.0 * entries + 4.0 * sum(-(-n // pt) for n in news), "flops": 0.0}
    seqs = sequences(case)
    if case["op"] == "keep":
        moved = sum(sum(i != j for j, i in enumerate(k)) for k in keeps(case)) * layers
        n = sum(s[0] for s in seqs)
        return {"bytes": 2.0 * moved * held + n * (layers * (held + read) + 1), "flops": 0.0}
    seen = rows = pairs = 0
    w = case.get("window", 0)
    for n, ln in seqs:
        rows += n
        if n:
            past = ln if case["op"] == "cross" else ln - n
            sees = min(past, w) if w else past
            seen += sees + (ln - past)
            pairs += n * (sees + (math.log(n) + 1 if case["op"] == "tree" else 0))
    tree = rows * (8.0 + 8 * case["words"]) if case["op"] == "tree" else 0.0
    return {"bytes": layers * (seen * held + 4.0 * rows * case["q_heads"] * d) + tree,
            "flops": 4.0 * layers * pairs * case["q_heads"] * d}


# ----------------------------------------------------------------- inputs --

def _offsets(counts):
    return torch.tensor([0] + list(counts), dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(lens, page_tokens, r):
    """(table, pages): every sequence's pages, dealt at random from the pool."""
    counts = [-(-n // page_tokens) for n in lens]
    pages = sum(counts) + 3
    perm = r.sample(range(pages), pages)
    width, at, rows = max(1, max(counts)), 0, []
    for c in counts:
        rows.append(perm[at:at + c] + [-1] * (width - c))
        at += c
    return _ints(rows), pages


def _shared_table(case, r):
    """(table, references, pages): the beams of a group share their prompt's full pages."""
    lens, news, prompts = branches(case)
    pt = case["page_tokens"]
    rows, at = [], 0
    for g, p in enumerate(prompts):
        shared = list(range(at, at + p // pt))
        at += p // pt
        for b in range(case["beams"]):
            more = -(-lens[g * case["beams"] + b] // pt) - p // pt
            rows.append(shared + list(range(at, at + more)))
            at += more
    pages = at + case["spare"]
    perm = r.sample(range(pages), pages)
    width = max(-(-(a + b) // pt) for a, b in zip(lens, news)) + 1
    refs = [0] * pages
    for i, row in enumerate(rows):
        rows[i] = [perm[x] for x in row] + [-1] * (width - len(row))
        for x in row:
            refs[perm[x]] += 1
    return _ints(rows), _ints(refs), pages


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    r = random.Random(int(seed))
    s = {"op": case["op"], "case": case}
    h, d, pt, op = case["kv_heads"], case["head_dim"], case["page_tokens"], case["op"]
    held = TYPES[case["dtype"]] if case["k_bits"] == 16 else torch.float16  # (codes are made from fp16 rows)
    if op == "copy":
        s["pages"] = case["pages"]
        pair = r.sample(range(s["pages"]), 2 * case["copies"])
        s["src"], s["dst"] = _ints(pair[::2]), _ints(pair[1::2])
        s["rows"] = case["copies"] * pt  # the copies, as one sequence's tokens
        s["q_start"], s["lens"], s["table"] = _ints([0, s["rows"]]), _ints([s["rows"]]), s["dst"][None]
    elif op == "branch":
        lens, news, _ = branches(case)
        s["table"], s["refs"], s["pages"] = _shared_table(case, r)
        s["lens"], s["q_start"] = _ints(lens), _offsets(news)
        k = case["beams"]
        s["parent"] = _ints([b - b % k + r.randrange(k) for b in range(len(lens))])
        s["parts"], s["rows"] = _offsets([x % pt for x in lens]), sum(x % pt for x in lens)
    else:
        seqs = sequences(case)
        news, lens = [x[0] for x in seqs], [x[1] for x in seqs]
        s["rows"], s["most_new"], s["longest"] = sum(news) + case.get("pad", 0), max(news), max(max(lens), 1)
        s["q_start"], s["lens"] = _offsets(news), _ints(lens)
        s["table"], s["pages"] = _table(lens, pt, r)
        if op == "keep":
            keep = torch.zeros(s["rows"], dtype=torch.bool)
            at = 0
            for n, rows in zip(news, keeps(case)):
                keep[[at + i for i in rows]] = True
                at += n
            s["keep"] = keep.cuda()
        else:
            s["q"] = [torch.randn((s["rows"], case["q_heads"], d), generator=g, device="cuda").to(TYPES[case["dtype"]])
                      for _ in range(case["layers"])]
            s["out"] = [torch.zeros_like(q) for q in s["q"]]
        if op == "tree":
            # a drafted token hangs on any earlier one, one in twenty on the past
            i = torch.arange(s["rows"], device="cuda") - torch.repeat_interleave(
                s["q_start"][:-1].long(), torch.tensor(news[:-1] + [news[-1] + case["pad"]], device="cuda"))
            u = torch.rand((2, s["rows"]), generator=g, device="cuda")
            s["parents"] = torch.where((i == 0) | (u[1] < 0.05), torch.full_like(i, -1), (u[0] * i).long()).int()
            s["seen"] = torch.zeros((s["rows"], case["words"]), dtype=torch.int64, device="cuda")
            s["positions"] = torch.zeros(s["rows"], dtype=torch.int32, device="cuda")
    # every slot of the pool holds a token: keys with four large channels a head
    s["k"], s["v"] = [], []
    for _ in range(case["layers"]):
        kv = torch.randn((2, s["pages"] * pt, h, d), generator=g, device="cuda", dtype=held)
        big = torch.rand(h, d, generator=g, device="cuda").argsort(dim=-1)[:, :4]
        kv[0] *= torch.ones(h, d, device="cuda").scatter_(1, big, 6.0).to(held)
        s["k"].append(kv[0])
        s["v"].append(kv[1])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    h, d, pt, group = case["kv_heads"], case["head_dim"], case["page_tokens"], case["group"]
    if own:
        from bit_quantized_kv_02_gb300 import kvq
        fmt = [None if b == 16 else (b, group, kvq.PER_TOKEN, kvq.ASYM) for b in (case["k_bits"], case["v_bits"])]
        dtype = kvq.BF16 if case["dtype"] == "bf16" and case["k_bits"] == 16 else kvq.F16
        cache = s["cache"] = kvq.KVQPages(kvq.make_pages_config(case["layers"], s["pages"], pt, case["q_heads"], h, d,
                                                                *fmt, dtype=dtype))
        slots = s["pages"] * pt
        whole = kvq.PagesBatch(_ints([0, slots]), _ints([slots]), torch.arange(s["pages"], dtype=torch.int32,
                                                                              device="cuda")[None], slots)
        for i in range(case["layers"]):
            cache.kvq_pages_append(i, s["k"][i], s["v"][i], whole)
        if case["op"] == "branch":
            s["kvq"] = kvq
        else:
            s["batch"] = kvq.PagesBatch(s["q_start"], s["lens"], s["table"], s["rows"], s.get("most_new", 0))
        if case["op"] == "tree":
            s["tree"] = kvq.PagesTree(s["seen"], s["positions"])
    else:
        for name in ("k", "v"):
            s["pool_" + name] = [_stored(x.unflatten(0, (s["pages"], pt)), case[name + "_bits"], group) for x in s[name]]
    del s["k"], s["v"]
    return s


# ------------------------------------------------------------- plain form --

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


def _stored(x, bits, group):
    """What a pool holds of x [pages][tokens][heads][d]: the values, or codes, zero points and steps."""
    if bits == 16:
        return [x.clone()]
    g = x.float().unflatten(-1, (-1, group))
    lo, hi = g.amin(dim=-1), g.amax(dim=-1)
    zero = _round16(lo + 0.0, False)
    step = _round16((hi - zero.float()) / torch.full_like(hi, float(2 ** bits - 1)), True)
    z, st = zero.float()[..., None], step.float()[..., None]
    c = torch.where(st == 0, torch.zeros_like(g), ((g - z) / st).round().clamp(0, 2 ** bits - 1))
    return [c.to(torch.uint8).flatten(-2), zero, step]


def _held(pool, page, slot, group):
    """What the pool holds at (page, slot): 16-bit values, or zero point + code * step rounded to fp16."""
    if len(pool) == 1:
        return pool[0][page, slot]
    c, zero, step = (p[page, slot] for p in pool)
    g = c.float().unflatten(-1, (-1, group))
    return torch.addcmul(zero.float()[..., None], g, step.float()[..., None]).flatten(-2).half()


def _pools(s):
    return [(s["pool_k"][i], s["pool_v"][i]) for i in range(s["case"]["layers"])]


def _places(start, lens, table, page_tokens, n):
    """(page, slot, sequence, position) of n rows: row i of a sequence's last tokens."""
    row = torch.arange(n, device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), row, right=True)
    pos = lens[b].long() - start[b + 1].long() + row
    return table[b, pos // page_tokens].long(), pos % page_tokens, b, pos


def _read(s, start, lens, table, n):
    """Keys and values that the layers hold for n rows."""
    page, slot, _, _ = _places(start, lens, table, s["case"]["page_tokens"], n)
    return [tuple(_held(p, page, slot, s["case"]["group"]) for p in pair) for pair in _pools(s)]


def _rows(s):
    """(row, is a new token) of [batch][most new tokens] rows."""
    start = s["q_start"].long()
    i = torch.arange(s["most_new"], device="cuda")
    return (start[:-1, None] + i).clamp_max(s["rows"] - 1), i < (start[1:] - start[:-1])[:, None]


def _ancestors(s):
    """[batch][row][token]: whether the row is the token or descends from it."""
    row, is_new = _rows(s)
    n = s["most_new"]
    parent = s["parents"].long()[row]
    j = torch.arange(n, device="cuda")
    up = ((parent[..., None] == j) & is_new[..., None]).float() + torch.eye(n, device="cuda")
    for _ in range(max(1, (n - 1).bit_length())):  # ancestors at twice the distance
        up = (up @ up).clamp_max(1.0)
    return up > 0


def _attend(s, q, pair, out, see):
    """out = softmax(q k / sqrt(d)) v of the rows, over the tokens that `see` [batch][row][token] shows."""
    case = s["case"]
    batch, hq, h, d = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"]
    rep, n, t = hq // h, s["most_new"], s["longest"]
    at = torch.arange(t, device="cuda")
    page = s["table"][:, (at // case["page_tokens"]).clamp_max(s["table"].shape[1] - 1)].clamp_min(0).long()
    slot = (at % case["page_tokens"]).expand_as(page)
    k = _held(pair[0], page, slot, case["group"]).permute(0, 2, 3, 1).float()  # [batch][h][d][t]
    v = _held(pair[1], page, slot, case["group"]).permute(0, 2, 1, 3).float()  # [batch][h][t][d]
    row, is_new = _rows(s)
    x = (q[row].float() * (1.0 / math.sqrt(d))).reshape(batch, n, h, rep, d).permute(0, 2, 3, 1, 4)
    score = (x.reshape(batch, h, rep * n, d) @ k).reshape(batch, h, rep, n, t)
    del k
    score.masked_fill_(~see[:, None, None], float("-inf"))
    top = score.amax(dim=-1, keepdim=True).clamp_min(-3.0e38)
    score.sub_(top).exp_()
    total = score.sum(dim=-1, keepdim=True)
    o = (score.reshape(batch, h, rep * n, t) @ v).reshape(batch, h, rep, n, d) / total.clamp_min(1e-38)
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, n, hq, d).to(q.dtype)
    out[row[is_new]] = o[is_new]
    return out


def _tree(s):
    case = s["case"]
    row, is_new = _rows(s)
    n, w = s["most_new"], case["words"]
    up = _ancestors(s)
    new = is_new.sum(dim=-1)
    past = (s["lens"].long() - new)[:, None]
    pos = past + up.sum(dim=-1) - 1
    s["positions"][row[is_new]] = pos[is_new].int()
    bits = torch.zeros(up.shape[:2] + (64 * w,), dtype=torch.int64, device="cuda")
    bits[..., :n] = up.long()
    seen = (bits.unflatten(-1, (w, 64)) << torch.arange(64, device="cuda")).sum(dim=-1)
    s["seen"][row[is_new]] = seen[is_new]
    at = torch.arange(s["longest"], device="cuda")
    see = at < past[..., None]
    if case["window"]:
        see = see & (at > pos[..., None] - case["window"])
    j = (at - past).clamp(0, n - 1)[:, None].expand(-1, n, -1)
    see = see | ((at >= past)[:, None] & (at < s["lens"][:, None])[:, None] & up.gather(2, j))
    outs = [_attend(s, q, pair, out, see) for q, pair, out in zip(s["q"], _pools(s), s["out"])]
    return [s["seen"], s["positions"]] + outs


def _keep(s):
    case = s["case"]
    n = s["rows"]
    start, keep = s["q_start"].long(), s["keep"]
    page, slot, b, pos = _places(s["q_start"], s["lens"], s["table"], case["page_tokens"], n)
    before = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), keep.long().cumsum(0)])
    to = s["lens"].long()[b] - (start[1:] - start[:-1])[b] + before[:-1] - before[start[b]]
    to = to[keep]
    to_page, to_slot = s["table"][b[keep], to // case["page_tokens"]].long(), to % case["page_tokens"]
    for pair in _pools(s):
        for p in pair[0] + pair[1]:
            p[to_page, to_slot] = p[page[keep], slot[keep]]
    count = before[start[1:]] - before[start[:-1]]
    lens = (s["lens"].long() - (start[1:] - start[:-1]) + count).int()
    return [lens] + _read(s, s["q_start"], s["lens"], s["table"], n)


def _copy(s):
    for pair in _pools(s):
        for p in pair[0] + pair[1]:
            p[s["dst"].long()] = p[s["src"].long()]
    return _read(s, s["q_start"], s["lens"], s["table"], s["rows"])


def _count(table, pages):
    x = table[table >= 0].long()
    return torch.zeros(pages, dtype=torch.int32, device="cuda").scatter_add_(0, x, torch.ones_like(x, dtype=torch.int32))


def _branch(s):
    pt, pages = s["case"]["page_tokens"], s["pages"]
    parent = s["parent"].long()
    lens = s["lens"][parent].long()
    at = torch.arange(s["table"].shape[1], device="cuda")
    table = torch.where(at < (-(-lens // pt))[:, None], s["table"][parent], -1)
    refs = s["refs"] - _count(s["table"], pages) + _count(table, pages)
    # pages for the new tokens: a last page that others name too is copied, but by the last who grows into it
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    first = lens // pt
    grows = (new > 0) & (lens % pt > 0)
    last = table.gather(1, first[:, None])[:, 0].clamp_min(0).long()
    same = (last[:, None] == last) & grows[:, None] & grows
    copies = grows & (same.tril(-1).sum(dim=1) < refs[last] - 1)
    need = (at >= first[:, None]) & (at <= ((lens + new - 1) // pt)[:, None]) & (new > 0)[:, None]
    need &= (table < 0) | (copies[:, None] & (at == first[:, None]))
    fresh = (refs == 0).nonzero()[:, 0][:int(need.sum())].int()
    table[need] = fresh
    refs[fresh.long()] = 1
    refs.scatter_add_(0, last[copies], torch.full_like(last[copies], -1, dtype=torch.int32))
    to = table.gather(1, first[:, None])[:, 0].long()
    for pair in _pools(s):
        for p in pair[0] + pair[1]:
            p[to[copies]] = p[last[copies]]
    got = _read(s, s["parts"], lens.int(), table, s["rows"])
    return [table, (lens + new).int(), refs] + got


def run(s):
    case, op = s["case"], s["op"]
    if not own:
        if op == "cross":
            see = (torch.arange(s["longest"], device="cuda") < s["lens"][:, None])[:, None]
            return [_attend(s, q, pair, out, see) for q, pair, out in zip(s["q"], _pools(s), s["out"])]
        return {"tree": _tree, "keep": _keep, "copy": _copy, "branch": _branch}[op](s)
    cache, layers = s["cache"], range(case["layers"])
    if op == "tree":
        cache.kvq_pages_tree(s["parents"], s["batch"], tree=s["tree"])
        return [s["seen"], s["positions"]] + [
            cache.kvq_pages_tree_attn(i, s["q"][i], s["batch"], s["tree"], out=s["out"][i], window=case["window"])
            for i in layers]
    if op == "cross":
        return [cache.kvq_pages_cross_attn(i, s["q"][i], s["batch"], out=s["out"][i]) for i in layers]
    if op == "keep":
        return [cache.kvq_pages_keep(s["keep"], s["batch"])] + [cache.kvq_pages_read(i, s["batch"]) for i in layers]
    if op == "copy":
        cache.kvq_pages_copy(s["src"], s["dst"])
        return [cache.kvq_pages_read(i, s["batch"]) for i in layers]
    table, lens, refs = cache.kvq_pages_fork(s["parent"], s["table"], s["lens"], s["refs"])
    grown = cache.kvq_pages_grow(s["q_start"], table, lens, refs)
    parts = s["kvq"].PagesBatch(s["parts"], lens, table, s["rows"])
    return [table, grown, refs] + [cache.kvq_pages_read(i, parts) for i in layers]


# ------------------------------------------------------------------ exact --

def _grid16(x, rounding):
    """x on the fp16 grid, by `rounding` (torch.floor or torch.ceil) of its multiple of the grid's spacing."""
    unit = torch.exp2(torch.frexp(x)[1].double().sub(1).clamp_min(-14) - 10)
    return rounding(x / unit) * unit


def _as_held(x, bits, group):
    """What pages hold of x, in 64 bits."""
    x = x.double()
    if bits == 16:
        return x
    y = x.unflatten(-1, (-1, group))
    zero = _grid16(y.amin(dim=-1, keepdim=True), torch.floor)
    step = ((y.amax(dim=-1, keepdim=True) - zero) / (2 ** bits - 1)).float().double()
    step = _grid16(step, torch.ceil)
    code = torch.where(step > 0, (y - zero) / step, torch.zeros_like(y)).round().clamp(0, 2 ** bits - 1)
    return (zero + code * step).flatten(-2).half().double()


def _slots_of(table, page_tokens, n):
    """Rows of the pool that hold a sequence's first n tokens."""
    at = torch.arange(n, device="cuda")
    return table[at // page_tokens].long() * page_tokens + at % page_tokens


def exact(case, seed):
    s = _inputs(case, seed)
    pt, group, d = case["page_tokens"], case["group"], case["head_dim"]

    def pick(rows):
        got = []
        for i in range(case["layers"]):
            sides = []
            for name in ("k", "v"):
                sides.append(torch.cat([_as_held(s[name][i][x], case[name + "_bits"], group) for x in rows.split(1 << 15)])
                             if rows.numel() else s[name][i][rows].double())
            got.append(tuple(sides))
        return got

    if case["op"] == "copy":
        return pick((s["src"].long()[:, None] * pt + torch.arange(pt, device="cuda")).flatten())
    if case["op"] == "branch":
        lens = s["lens"].tolist()
        rows = [_slots_of(s["table"][p], pt, lens[p])[lens[p] // pt * pt:] for p in s["parent"].tolist()]
        return [None, None, None] + pick(torch.cat(rows))
    seqs = sequences(case)
    if case["op"] == "keep":
        rows = []
        for b, (n, ln) in enumerate(seqs):
            at = _slots_of(s["table"][b], pt, ln)[ln - n:]
            kept = at[torch.tensor(keeps(case)[b], dtype=torch.int64, device="cuda")]
            rows.append(torch.cat([kept, at[len(kept):]]))
        return [None] + pick(torch.cat(rows))
    hq, h = case["q_heads"], case["kv_heads"]
    outs = [torch.zeros(s["q"][0].shape, dtype=torch.float64, device="cuda") for _ in range(case["layers"])]
    parents, w = s["parents"].tolist() if case["op"] == "tree" else None, case.get("window", 0)
    a = 0
    for b, (n, ln) in enumerate(seqs):
        if n and ln:
            see = torch.ones((n, ln), dtype=torch.bool)
            if case["op"] == "tree":
                past, depth = ln - n, []
                see[:, past:] = False
                for i in range(n):
                    p = parents[a + i]
                    if p >= 0:
                        see[i, past:] = see[p, past:]
                    see[i, past + i] = True
                    depth.append(depth[p] + 1 if p >= 0 else 0)
                    if w:
                        see[i, :max(0, min(past, past + depth[i] - w + 1))] = False
            see = see.cuda()
            for i, (k, v) in enumerate(pick(_slots_of(s["table"][b], pt, ln))):
                for j in range(hq):
                    p = s["q"][i][a:a + n, j].double() @ k[:, j // (hq // h)].T / math.sqrt(d)
                    p = torch.softmax(p.masked_fill(~see, float("-inf")), dim=-1)
                    outs[i][a:a + n, j] = p @ v[:, j // (hq // h)]
        a += n
    return ([None, None] if case["op"] == "tree" else []) + outs
