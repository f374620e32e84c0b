"""The paged cache: host-side refusals (CPU), and on the GPU append, read-back,
norm with rotary embedding and attention against plain 64-bit forms."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from bit_quantized_kv_02_gb300 import build, kvq
from tests.pages_ref import FORMATS, HALF_STEP, HALVES, PAIRS, Case, angles, attention, held, rotate

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(kvq.LIB_PATH):
        build.build()
    return kvq.lib()


def config(**kw):
    base = dict(layers=1, pages=4, page_tokens=16, q_heads=8, kv_heads=2, head_dim=64, k=None, v=None, dtype=kvq.F16)
    base.update(kw)
    return kvq.make_pages_config(**base)


# ----------------------------------------------------------------- refusals --

@pytest.mark.parametrize("kw,status", [
    (dict(layers=0), 1), (dict(pages=0), 1), (dict(kv_heads=0), 1), (dict(q_heads=7), 1), (dict(page_tokens=0), 1),
    (dict(page_tokens=48), 2), (dict(head_dim=96), 2), (dict(q_heads=130, kv_heads=2), 2), (dict(dtype=1), 1),
    (dict(dtype=7), 1), (dict(k=(8, 32, 0, 0)), 2), (dict(v=(4, 32, 0, 0)), 2),
    (dict(k=(8, 32, 0, 0), v=(1, 32, 0, 0)), 1), (dict(k=(8, 32, 0, 0), v=(2, 32, 0, 0)), 2),
    (dict(k=(8, 32, 1, 0), v=(8, 32, 0, 0)), 2), (dict(k=(8, 32, 0, 1), v=(8, 32, 0, 0)), 2),
    (dict(k=(8, 48, 0, 0), v=(8, 32, 0, 0)), 2), (dict(k=(8, 128, 0, 0), v=(8, 32, 0, 0)), 2),
    (dict(k=(8, -1, 0, 0), v=(8, 32, 0, 0)), 2), (dict(k=(8, 0, 0, 0), v=(8, 32, 0, 0)), 1),
    (dict(k=(8, 32, 2, 0), v=(8, 32, 0, 0)), 1), (dict(k=(8, 32, 0, 3), v=(8, 32, 0, 0)), 1),
    (dict(k=(8, 32, 0, 0), v=(8, 32, 0, 0), dtype=kvq.BF16), 1),
    (dict(layers=2 ** 30, pages=2 ** 30, page_tokens=128), 2),
])
def test_config_refusals(kw, status):
    with pytest.raises(kvq.KVQError) as e:
        kvq.kvq_pages_bytes(config(**kw))
    assert e.value.status == status


@pytest.mark.parametrize("name", FORMATS)
def test_sizes(name):
    k, v, dtype = FORMATS[name]
    b = kvq.kvq_pages_bytes(config(layers=3, pages=5, page_tokens=32, kv_heads=4, head_dim=128, k=k, v=v, dtype=dtype))
    tokens = 3 * 5 * 32 * 4
    bits = [16 if t is None else t[0] for t in (k, v)]
    meta = 0 if k is None else sum(4 * 128 // t[1] for t in (k, v))
    assert b.packed == tokens * 128 * sum(bits) / 8
    assert b.metadata == tokens * meta
    assert b.elements == 2 * tokens * 128
    assert b.alloc >= b.total and b.alloc % 256 == 0


def test_create_refusals(L):
    cfg = config()
    need = kvq.kvq_pages_bytes(cfg).alloc
    h = ctypes.c_void_p()
    ref = ctypes.byref
    assert L.kvq_pages_create(ref(cfg), None, need, None, ref(h)) == 1
    assert L.kvq_pages_create(ref(cfg), ctypes.c_void_p((1 << 20) + 16), need, None, ref(h)) == 1
    assert L.kvq_pages_create(ref(cfg), ctypes.c_void_p(1 << 20), need - 1, None, ref(h)) == 4
    assert L.kvq_pages_create(ref(cfg), ctypes.c_void_p(1 << 20), need, None, None) == 1
    assert L.kvq_pages_bytes(ref(cfg), None) == 1
    assert L.kvq_pages_bytes(None, None) == 1
    assert L.kvq_pages_destroy(None) == 1
    assert L.kvq_pages_append(None, 0, None, None, 0, 0, 0, None, None, None) == 1
    assert L.kvq_pages_attn(None, 0, None, 0, 0, None, 0.0, 0, None, None) == 1
    assert L.kvq_pages_read(None, 0, None, None, None, None) == 1
    assert L.kvq_pages_set_kernel(None, 0) == 1
    assert L.kvq_pages_status(None, None) == 1
    assert L.kvq_pages_last_error(None) == b""


def test_status_string_of_a_bad_index():
    assert "out of range" in kvq.kvq_status_string(7)


@pytest.mark.parametrize("kw,rope,status", [
    (dict(tokens=-1), None, 1), (dict(head_dim=96), None, 2), (dict(dtype=5), None, 1), (dict(eps=float("nan")), None, 1),
    (dict(eps=-1.0), None, 1), (dict(weight_dtype=2, q_weight=64), None, 1), (dict(q_stride=8 * 64 - 1), None, 1),
    (dict(k_out_stride=0), None, 1), (dict(q=0), None, 1), (dict(k_out=0), None, 1), (dict(q_heads=-1), None, 1),
    ({}, dict(table=0), 1), ({}, dict(table=72), 1), ({}, dict(rows=0), 1), ({}, dict(dim=8), 1), ({}, dict(dim=72), 1),
    ({}, dict(dim=80), 1), ({}, dict(style=2), 1), ({}, dict(positions=0), 1), (dict(tokens=0), None, 0),
    (dict(q=65), None, 1), (dict(dtype=1, k=66), None, 1), (dict(q_out=67), None, 1), (dict(k_weight=65), None, 1),
    (dict(q_weight=66, weight_dtype=1), None, 1), ({}, dict(positions=66), 1),
    (dict(q_heads=0, kv_heads=0), None, 0),
])
def test_norm_rope_refusals(L, kw, rope, status):
    """Nothing here reaches CUDA: the pointers are never followed."""
    f = dict(tokens=3, q_heads=8, kv_heads=2, head_dim=64, dtype=0, q=64, k=64, q_out=64, k_out=64, q_stride=512,
             k_stride=128, q_out_stride=512, k_out_stride=128, norm=1, eps=1e-6, q_weight=0, k_weight=0, weight_dtype=0)
    f.update(kw)
    a = kvq._NormRopeArgs(**{k: (v or None) if k in ("q", "k", "q_out", "k_out", "q_weight", "k_weight") else v
                             for k, v in f.items()})
    r = None
    if rope is not None:
        g = dict(table=64, rows=10, dim=64, style=0, positions=64)
        g.update(rope)
        r = ctypes.byref(kvq._Rope(g["table"] or None, g["rows"], g["dim"], g["style"], g["positions"] or None))
    assert L.kvq_qk_norm_rope(ctypes.byref(a), r, None) == status
    assert L.kvq_qk_norm_rope(None, None, None) == 1


def test_wrapper_refuses_cpu_tensors_and_wrong_shapes():
    z = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        kvq.PagesBatch(z, z[:2], z[:2, None], 1)
    with pytest.raises(ValueError):
        kvq.Rope(angles(4, 16))
    with pytest.raises(ValueError):
        kvq.kvq_qk_norm_rope(torch.zeros(2, 3, 64), None)


# --------------------------------------------------------------- norm + rope --

def norm_bound(x, w, cs, dim, style, eps):
    """(value, bound without the last rounding) in 64 bits.  In fp32 the mean square
    of d terms rounds at most 13 times on any path through its tree (8 in a lane,
    5 between lanes) and the root halves that; eps, the root, the quotient, the two
    products and the rotation's product and sum round once each: fewer than 24
    half steps of 2^-24 of the magnitudes that are added."""
    f = x.double()
    if w is not None:
        f = f / ((f * f).mean(dim=-1, keepdim=True) + eps).sqrt() * w.double()
    if cs is None:
        return f, f.abs() * 24 * 2.0 ** -24
    return rotate(f, cs.double(), dim, style), rotate_size(f, cs, dim, style) * 24 * 2.0 ** -24


def rotate_size(f, cs, dim, style):
    """|a c| + |b s| of each rotated channel, |a| of the others."""
    a, c, s = f.abs(), cs[:, None, :, 0].abs().double(), cs[:, None, :, 1].abs().double()
    y = a.clone()
    if style == PAIRS:
        y[..., 0:dim:2] = a[..., 0:dim:2] * c + a[..., 1:dim:2] * s
        y[..., 1:dim:2] = a[..., 1:dim:2] * c + a[..., 0:dim:2] * s
    else:
        h = dim // 2
        y[..., :h] = a[..., :h] * c + a[..., h:dim] * s
        y[..., h:dim] = a[..., h:dim] * c + a[..., :h] * s
    return y


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,hq,h,dim,style", [(64, 5, 1, 64, PAIRS), (64, 12, 12, 32, HALVES), (128, 32, 8, 128, HALVES),
                                              (128, 7, 3, 48, HALVES), (256, 16, 2, 64, PAIRS), (256, 3, 1, 256, HALVES),
                                              (128, 4, 4, 16, PAIRS), (128, 2, 2, 0, PAIRS)])
@pytest.mark.parametrize("tokens", [1, 37, 2500])
def test_norm_rope(dtype, d, hq, h, dim, style, tokens):
    g = torch.Generator().manual_seed(d + tokens)
    qkv = (torch.randn((tokens, hq + 2 * h, d), generator=g) * 3).to(dtype)
    qw, kw = (torch.rand(d, generator=g) + 0.5).to(dtype), None
    pos = torch.randint(0, 300, (tokens,), generator=g).int()
    tab = angles(300, dim) if dim else None
    dev = qkv.cuda()
    rope = kvq.Rope(tab.cuda(), style, pos.cuda()) if dim else None
    yq, yk = kvq.kvq_qk_norm_rope(dev[:, :hq], dev[:, hq:hq + h], qw.cuda(), kw, eps=1e-5, rope=rope)
    cs = tab[pos.long()] if dim else None
    for got, x, w in ((yq, qkv[:, :hq], qw), (yk, qkv[:, hq:hq + h], torch.ones(d))):
        ref, tol = norm_bound(x, w, cs, dim, style, 1e-5)
        tol = tol + ref.abs() * HALF_STEP[dtype] * (1 + 2.0 ** -10) + 2.0 ** -25  # fp16 results below its normal range
        assert ((got.cpu().double() - ref).abs() <= tol).all()
    # rotation alone, in place, with a slice that starts off 16 bytes and an odd stride
    flat = torch.zeros(tokens * ((hq + h) * d + 3) + 5, dtype=dtype, device="cuda")
    view = flat[5:].view(tokens, -1)[:, :(hq + h) * d].unflatten(1, (hq + h, d))
    view.copy_(dev[:, :hq + h])
    kvq.kvq_qk_norm_rope(view[:, :hq], view[:, hq:], rope=rope, q_out=view[:, :hq], k_out=view[:, hq:], norm=False)
    ref, tol = norm_bound(qkv[:, :hq + h], None, cs, dim, style, 0)
    tol = tol + ref.abs() * HALF_STEP[dtype] * (1 + 2.0 ** -10) + 2.0 ** -25
    assert ((view.cpu().double() - ref).abs() <= tol).all()
    assert not flat[:5].any() and not flat[5:].view(tokens, -1)[:, (hq + h) * d:].any()


@gpu
def test_norm_rope_one_side_fp32_weights_and_bad_positions():
    g = torch.Generator().manual_seed(1)
    k = torch.randn((4, 2, 128), generator=g).bfloat16()
    w = torch.rand(128, generator=g) + 0.5
    pos = torch.tensor([0, 9, 10, -1], dtype=torch.int32)
    rope = kvq.Rope(angles(10, 128).cuda(), HALVES, pos.cuda())
    none, y = kvq.kvq_qk_norm_rope(None, k.cuda(), None, w.cuda(), rope=rope)
    assert none is None
    ref, tol = norm_bound(k[:2], w, angles(10, 128)[pos[:2].long()], 128, HALVES, 1e-6)
    tol = tol + ref.abs() * HALF_STEP[torch.bfloat16] * (1 + 2.0 ** -10)
    assert ((y[:2].cpu().double() - ref).abs() <= tol).all()
    assert y[2:].isnan().all()
    q, none = kvq.kvq_qk_norm_rope(k.cuda(), None, norm=False)
    assert none is None and torch.equal(q.cpu(), k)
    # zero rows: nothing to divide by but eps; zero tokens
    z, _ = kvq.kvq_qk_norm_rope(torch.zeros((3, 2, 64), device="cuda", dtype=torch.float16), None)
    assert not z.any()
    assert kvq.kvq_qk_norm_rope(torch.zeros((0, 2, 64), device="cuda"), None)[0].shape == (0, 2, 64)


# ------------------------------------------------------------ append + read --

BATCHES = {
    "ones": ([1, 1, 1], [1, 40, 17]),
    "ragged": ([5, 0, 33, 1, 70], [5, 9, 50, 300, 129]),
    "short": ([3, 4, 2], [1, 4, 0]),   # more new tokens than the sequence holds: the first ones have no place
}


def make(name, page_tokens, fmt, heads=(4, 2), d=64, seed=0, layers=1, pad=0):
    news, lens = BATCHES[name] if isinstance(name, str) else name
    c = Case(news, lens, page_tokens, seed, pad=pad)
    k, v, dtype = FORMATS[fmt]
    c.cache = kvq.KVQPages(kvq.make_pages_config(layers, c.pages, page_tokens, heads[0], heads[1], d, k, v, dtype))
    c.bits = [16 if t is None else t[0] for t in (k, v)]
    c.group = [32 if t is None else t[1] for t in (k, v)]
    c.dtype = torch.bfloat16 if dtype == kvq.BF16 else torch.float16
    return c


def positions(c):
    return torch.cat([torch.arange(ln - n, ln) for n, ln in zip(c.news, c.lens)])


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name,page_tokens,d,h,rope,in_dtype", [
    ("ones", 16, 128, 8, (128, HALVES), torch.bfloat16), ("ragged", 32, 64, 3, (32, PAIRS), torch.float16),
    ("ragged", 128, 256, 2, (64, HALVES), torch.float32), ("ragged", 64, 128, 1, None, torch.float32),
    ("short", 16, 64, 5, (64, PAIRS), torch.float16)])
def test_append_and_read(fmt, name, page_tokens, d, h, rope, in_dtype):
    c = make(name, page_tokens, fmt, (h, h), d, layers=2, pad=2)
    kv = c.normal(c.rows, 2, h, d)
    kv[:, 0, :, 3] *= 9.0
    kv = kv.to(in_dtype)
    k, v = kv.cuda()[:, 0], kv.cuda()[:, 1]
    pos = positions(c)
    r, keys = None, kv[:c.n, 0].float()
    if rope:
        tab = angles(400, rope[0])
        r = kvq.Rope(tab.cuda(), rope[1])
        keys = rotate(keys, tab[pos.clamp_min(0)], *rope)
    c.cache.kvq_pages_append(1, k, v, c.batch(), rope=r)
    fill = torch.full((c.rows, h, d), 7.0, dtype=c.dtype, device="cuda")
    ko, vo = c.cache.kvq_pages_read(1, c.batch(), fill.clone(), fill.clone())
    assert c.cache.kvq_pages_status() == 0
    has = pos >= 0
    for got, x, i in ((ko, keys, 0), (vo, kv[:c.n, 1].float(), 1)):
        want = held(x, c.bits[i], c.group[i], c.dtype)
        assert torch.equal(got[:c.n].cpu()[has], want[has])
        assert (got[:c.n].cpu()[~has] == 7).all() and (got[c.n:] == 7).all()
    # the other layer and the spare pages are as they were
    per = c.cache.bytes.packed + c.cache.bytes.metadata
    assert not c.cache.buffer[:int(per) // 2].any()
    layer = c.cache.buffer[int(per) // 2:int(per)].view(c.pages, -1) if int(per) // 2 % 256 == 0 else None
    if layer is not None:
        assert not layer[c.free.long().cuda()].any()


@gpu
def test_append_positions_and_unaligned_rows():
    c = make("ragged", 16, "f16", (2, 2), 64)
    flat = torch.randn(c.rows * (2 * 128 + 1) + 3, generator=c.g)
    kv = flat[3:].view(c.rows, 257)[:, :256].unflatten(1, (2, 2, 64))
    dev = flat.half().cuda()[3:].view(c.rows, 257)[:, :256].unflatten(1, (2, 2, 64))
    tab, at = angles(50, 64), torch.randint(0, 50, (c.rows,), generator=c.g).int()
    c.cache.kvq_pages_append(0, dev[:, 0], dev[:, 1], c.batch(), rope=kvq.Rope(tab.cuda(), HALVES, at.cuda()))
    ko, vo = c.cache.kvq_pages_read(0, c.batch())
    assert torch.equal(ko.cpu(), rotate(kv[:, 0].half().float(), tab[at.long()], 64, HALVES).half())
    assert torch.equal(vo.cpu(), kv[:, 1].half())


@gpu
def test_append_grows_token_by_token_like_a_prompt():
    """A prompt and the same tokens one by one leave the same bytes."""
    for fmt in ("bf16", "8_4"):
        a, b = (make(([75], [75]), 32, fmt, (2, 2), 128, seed=5) for _ in range(2))
        k, v = (a.normal(75, 2, 128).cuda() for _ in range(2))
        r = kvq.Rope(angles(80, 128).cuda(), HALVES)
        a.cache.kvq_pages_append(0, k, v, a.batch(), rope=r)
        table = b.table.cuda()
        for i in range(75):
            one = kvq.PagesBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(),
                                 torch.tensor([i + 1], dtype=torch.int32).cuda(), table, 1)
            b.cache.kvq_pages_append(0, k[i:i + 1], v[i:i + 1], one, rope=r)
        per = int(a.cache.bytes.packed + a.cache.bytes.metadata)
        assert torch.equal(a.cache.buffer[:per], b.cache.buffer[:per])


# ---------------------------------------------------------------- attention --

def fill(c, h, d, layer=0):
    """Gives the cache random contents; returns what the pages hold, per sequence."""
    t = int(c.k_start[-1])
    k, v = c.normal(t, h, d), c.normal(t, h, d)
    k[:, :, 5] *= 6.0
    if t:
        c.cache.kvq_pages_append(layer, k.cuda(), v.cuda(), c.whole())
    ko, vo = (x.cpu() for x in c.cache.kvq_pages_read(layer, c.whole()))
    s = c.k_start.tolist()
    return [(ko[a:b], vo[a:b]) for a, b in zip(s, s[1:])]


def check_attention(c, q, got, data, window=0, scale=None):
    d = q.shape[2]
    scale = scale or 1.0 / math.sqrt(d)
    p_step = HALF_STEP[torch.float16 if c.bits[0] < 16 else c.dtype]
    s, worst = c.q_start.tolist(), 0.0
    for b, (k, v) in enumerate(data):
        rows = slice(s[b], s[b + 1])
        pos = torch.arange(c.lens[b] - c.news[b], c.lens[b])
        ref, tol = attention(q[rows], k, v, pos, window, scale, p_step)
        tol = tol + ref.abs() * HALF_STEP[q.dtype] + 2.0 ** -25
        off = (got[rows].double() - ref).abs()
        assert (off <= tol).all(), (b, float((off / tol).max()))
        worst = max(worst, float((off / tol).max()) if off.numel() else 0.0)
    return worst


ATTN_BATCHES = {
    "steps": ([1, 1, 1, 1], [1, 2, 333, 1500]),
    "drafts": ([5, 3, 0, 8], [700, 3, 20, 129]),
    "mixed": ([1, 60, 0, 17, 200], [2000, 60, 0, 500, 450]),
    "negative": ([4, 3, 40], [2, 0, 33]),
    "long": ([2], [9000]),
    "prompt": ([700], [700]),
}


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name,page_tokens,d,heads,window", [
    ("steps", 16, 64, (12, 12), 0), ("steps", 64, 128, (8, 2), 0), ("steps", 128, 256, (16, 2), 70),
    ("drafts", 32, 128, (8, 1), 0), ("drafts", 16, 64, (3, 1), 33), ("mixed", 64, 128, (4, 4), 0),
    ("mixed", 32, 256, (5, 1), 100), ("negative", 16, 128, (4, 2), 0), ("negative", 64, 64, (64, 1), 5),
    ("long", 128, 64, (2, 1), 0), ("long", 16, 128, (8, 1), 4000), ("prompt", 32, 64, (6, 2), 0),
    ("prompt", 128, 256, (2, 1), 129)])
def test_attention(which, fmt, name, page_tokens, d, heads, window):
    c = make(ATTN_BATCHES[name], page_tokens, fmt, heads, d, seed=3, pad=3)
    data = fill(c, heads[1], d)
    types = [c.dtype] if c.bits[0] == 16 else [torch.float16, torch.bfloat16]
    c.cache.kvq_pages_set_kernel(which)
    for dtype in types:
        q = c.normal(c.rows, heads[0], d).to(dtype)
        out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
        got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(), out=out, window=window)
        assert c.cache.kvq_pages_status() == 0
        assert (got[c.n:] == 5).all()
        check_attention(c, q, got.cpu(), data, window)
        # the default choice, with and without the hint
        c.cache.kvq_pages_set_kernel(0)
        for hint in (0, max(c.news)):
            check_attention(c, q, c.cache.kvq_pages_attn(0, q.cuda(), c.batch(hint), window=window).cpu(), data, window)
        c.cache.kvq_pages_set_kernel(which)


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_does_not_see_what_pages_held_before(which, fmt):
    """NaN and infinities of an earlier owner of the pages, behind the sequence's end."""
    c = make(([1, 20, 40, 129], [5, 50, 40, 200]), 64, fmt, (4, 2), 128, seed=9)
    # all bytes of the pool to NaN patterns, codes and metadata alike
    per = int(c.cache.bytes.packed + c.cache.bytes.metadata)
    c.cache.buffer[:per].fill_(0xFF)
    data = fill(c, 2, 128)
    q = c.normal(c.rows, 4, 128).to(c.dtype)
    c.cache.kvq_pages_set_kernel(which)
    got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch())
    assert c.cache.kvq_pages_status() == 0
    check_attention(c, q, got.cpu(), data)


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", ["f16", "bf16", "4_8"])
def test_attention_scale_strides_and_magnitudes(which, fmt):
    """A given scale, queries that are an unaligned slice, and bf16 queries far
    outside the range of fp16 over quantized pages."""
    c = make(([3, 30], [90, 30]), 16, fmt, (4, 2), 64, seed=2)
    data = fill(c, 2, 64)
    dtype = torch.bfloat16 if c.bits[0] < 16 else c.dtype
    c.cache.kvq_pages_set_kernel(which)
    flat = c.normal(c.rows * 259 + 1).to(dtype)
    q = flat[1:].view(c.rows, 259)[:, :256].unflatten(1, (4, 64))
    dev = flat.cuda()[1:].view(c.rows, 259)[:, :256].unflatten(1, (4, 64))
    got = c.cache.kvq_pages_attn(0, dev, c.batch(), scale=0.31)
    check_attention(c, q, got.cpu(), data, scale=0.31)
    if dtype == torch.bfloat16:
        big = (c.normal(c.rows, 4, 64) * 1e30).to(dtype)
        got = c.cache.kvq_pages_attn(0, big.cuda(), c.batch(), scale=1e-31)
        check_attention(c, big, got.cpu(), data, scale=1e-31)
        small = (c.normal(c.rows, 4, 64) * 1e-30).to(dtype)
        got = c.cache.kvq_pages_attn(0, small.cuda(), c.batch(), scale=1e30)
        check_attention(c, small, got.cpu(), data, scale=1e30)


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", ["f16", "bf16", "4_8"])
def test_attention_of_vanishing_scores(which, fmt):
    """A scale and queries whose product is below every float: all visible weights
    are equal, and hidden tokens stay hidden."""
    c = make(([3, 40], [90, 40]), 16, fmt, (4, 2), 64, seed=2)
    data = fill(c, 2, 64)
    dtype = torch.bfloat16 if c.bits[0] < 16 else c.dtype
    c.cache.kvq_pages_set_kernel(which)
    small = 1e-30 if dtype == torch.bfloat16 else 2.0 ** -14
    for scale in (1e-30, 1e-45):
        q = (c.normal(c.rows, 4, 64) * small).to(dtype)
        for window in (0, 7):
            got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(), scale=scale, window=window)
            check_attention(c, q, got.cpu(), data, window, scale=scale)


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", ["bf16", "4_4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages_before_the_window_may_leave(which, fmt, d):
    """Table entries of pages whose 128-token block lies before the window are not read."""
    c = make(([1, 30, 4], [700, 600, 130]), 16, fmt, (4, 2), d, seed=5)
    data = fill(c, 2, d)
    window = 150
    for b, (n, ln) in enumerate(zip(c.news, c.lens)):
        first = max(ln - n + 1 - window, 0) // 128 * 128
        c.table[b, :first // 16] = -1
    q = c.normal(c.rows, 4, d).to(c.dtype)
    c.cache.kvq_pages_set_kernel(which)
    got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(), window=window)
    assert c.cache.kvq_pages_status() == 0
    check_attention(c, q, got.cpu(), data, window)


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
def test_two_caches_on_two_streams(which):
    """Calls of two handles at the same time, outputs made on the calls' own streams."""
    cases = []
    for i, fmt in enumerate(("bf16", "4_8")):
        c = make(([1, 200, 8], [1500, 400, 30]), 32, fmt, (8, 2), 128, seed=20 + i)
        data = fill(c, 2, 128)
        c.cache.kvq_pages_set_kernel(which)
        q = c.normal(c.rows, 8, 128).to(c.dtype)
        cases.append((c, data, q, q.cuda(), c.batch(), torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for _ in range(8):
        for c, _, _, dev, batch, stream, outs in cases:
            turned, _ = kvq.kvq_qk_norm_rope(dev, None, norm=False, stream=stream)
            outs.append(c.cache.kvq_pages_attn(0, turned, batch, stream=stream))
            del turned
            outs.append(c.cache.kvq_pages_read(0, c.whole(), stream=stream)[0])
    torch.cuda.synchronize()
    for c, data, q, _, _, _, outs in cases:
        held_keys = torch.cat([k for k, _ in data])
        for i in range(0, len(outs), 2):
            check_attention(c, q, outs[i].cpu(), data)
            assert torch.equal(outs[i + 1].cpu(), held_keys)
        assert c.cache.kvq_pages_status() == 0


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", ["8_8", "4_8"])
def test_largest_batch_with_the_largest_records(which, fmt):
    news = [1] * 1024
    lens = [1 + (i * 29) % 60 for i in range(1024)]
    c = make((news, lens), 16, fmt, (2, 1), 256, seed=8)
    data = fill(c, 1, 256)
    q = c.normal(c.rows, 2, 256).bfloat16()
    c.cache.kvq_pages_set_kernel(which)
    got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(1)).cpu()
    assert c.cache.kvq_pages_status() == 0
    check_attention(c, q, got, data)


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
def test_attention_of_a_peaked_softmax(which):
    """Scores that grow along the sequence move the maximum in every tile."""
    c = make(([2, 64], [2000, 1000]), 32, "f16", (2, 1), 64, seed=4)
    t = int(c.k_start[-1])
    k, v = torch.zeros(t, 1, 64), c.normal(t, 1, 64)
    k[:, 0, 0] = torch.cat([torch.arange(2000), torch.arange(1000).flip(0)]) * 0.125
    c.cache.kvq_pages_append(0, k.cuda(), v.cuda(), c.whole())
    q = torch.zeros(c.rows, 2, 64)
    q[:, 0, 0], q[:, 1, 0] = 8.0, 1.0
    q = q.half()
    c.cache.kvq_pages_set_kernel(which)
    got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch()).cpu()
    check_attention(c, q, got, [(k[:2000].half(), v[:2000].half()), (k[2000:].half(), v[2000:].half())])


@gpu
@pytest.mark.parametrize("which", [0, 1, 2])
def test_attention_large_batch(which):
    """1024 sequences, most without new tokens, one of them long."""
    news = [(i * 7) % 3 if i % 5 == 0 else 0 for i in range(1024)]
    lens = [news[i] + (i * 13) % 50 for i in range(1024)]
    news[500], lens[500] = 90, 3000
    c = make((news, lens), 16, "bf16", (4, 2), 64, seed=8)
    data = fill(c, 2, 64)
    q = c.normal(c.rows, 4, 64).bfloat16()
    c.cache.kvq_pages_set_kernel(which)
    got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(90)).cpu()
    assert c.cache.kvq_pages_status() == 0
    check_attention(c, q, got, data)


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", ["f16", "8_8"])
def test_shared_pages(which, fmt):
    """Two sequences that share the pages of their prefix."""
    c = make(([6, 4], [70, 68]), 32, fmt, (4, 2), 64, seed=6)
    c.table[1, :2] = c.table[0, :2]
    k, v = c.normal(138, 2, 64), c.normal(138, 2, 64)
    k[70:134], v[70:134] = k[:64], v[:64]
    c.cache.kvq_pages_append(0, k[:70].cuda(), v[:70].cuda(), kvq.PagesBatch(
        torch.tensor([0, 70], dtype=torch.int32).cuda(), torch.tensor([70], dtype=torch.int32).cuda(), c.table[:1].cuda(), 70))
    c.cache.kvq_pages_append(0, k[134:].cuda(), v[134:].cuda(), kvq.PagesBatch(
        torch.tensor([0, 4], dtype=torch.int32).cuda(), torch.tensor([68], dtype=torch.int32).cuda(), c.table[1:].cuda(), 4))
    ko, vo = (x.cpu() for x in c.cache.kvq_pages_read(0, c.whole()))
    q = c.normal(c.rows, 4, 64).half()
    c.cache.kvq_pages_set_kernel(which)
    got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch()).cpu()
    check_attention(c, q, got, [(ko[:70], vo[:70]), (ko[70:], vo[70:])])


@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_repeats_bit_for_bit(which, fmt, d):
    """Short pieces of items, one behind the other in a CTA, many times over: a slot
    or a column given back too early shows as a run that differs."""
    for batch, heads, window in ((([200], [450]), (5, 1), 0), (([1, 60, 0, 17, 200], [2000, 60, 0, 500, 450]), (5, 1), 100)):
        c = make(batch, 32, fmt, heads, d, seed=3)
        data = fill(c, 1, d)
        q = c.normal(c.rows, heads[0], d).to(c.dtype)
        c.cache.kvq_pages_set_kernel(which)
        dev, b = q.cuda(), c.batch()
        first = c.cache.kvq_pages_attn(0, dev, b, window=window).clone()
        check_attention(c, q, first.cpu(), data, window)
        out = torch.zeros_like(first)
        differ = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(60):
            c.cache.kvq_pages_attn(0, dev, b, out=out, window=window)
            differ += (out != first).sum()
        assert int(differ) == 0 and c.cache.kvq_pages_status() == 0


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "4_8"])
def test_no_window_is_an_endless_one(fmt):
    c = make(([4, 3, 40, 200], [2, 50, 33, 300]), 16, fmt, (4, 2), 64, seed=4)
    data = fill(c, 2, 64)
    q = c.normal(c.rows, 4, 64).to(c.dtype)
    for which in (1, 2):
        c.cache.kvq_pages_set_kernel(which)
        a = c.cache.kvq_pages_attn(0, q.cuda(), c.batch())
        check_attention(c, q, a.cpu(), data)
        for window in (2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1):
            b = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(), window=window)
            check_attention(c, q, b.cpu(), data)


@gpu
def test_two_graphs_of_one_cache_take_turns():
    """Two captured calls over the same handle (they share its workspace), replayed
    alternately on one stream, and layers that do not touch one another."""
    c = make(([3, 90], [700, 600]), 32, "bf16", (8, 2), 128, seed=12, layers=2)
    layers = [fill(c, 2, 128, layer) for layer in (0, 1)]
    q = c.normal(c.rows, 8, 128).bfloat16()
    dev, b, outs, graphs = q.cuda(), c.batch(), [], []
    for layer in (0, 1):
        outs.append(c.cache.kvq_pages_attn(layer, dev, b))
    for layer in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.cache.kvq_pages_attn(layer, dev, b, out=outs[layer])
        graphs.append(g)
    for i in range(6):
        for o in outs:
            o.zero_()
        for layer in ((0, 1), (1, 0))[i % 2]:
            graphs[layer].replay()
        for layer in (0, 1):
            check_attention(c, q, outs[layer].cpu(), layers[layer])


@gpu
def test_far_offsets():
    """A pool beyond 4 GiB and 2^31 values: the sequence lives in its last pages."""
    pages = 18000  # 18000 * 128 tokens * 4 heads * 512 bytes = 4.7 GB
    cfg = kvq.make_pages_config(1, pages, 128, 4, 4, 128, dtype=kvq.BF16)
    cache = kvq.KVQPages(cfg)
    c = Case([2], [300], 128, 1)
    c.table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32)
    c.cache, c.bits, c.dtype = cache, [16, 16], torch.bfloat16
    data = fill(c, 4, 128)
    q = c.normal(c.rows, 4, 128).bfloat16()
    for which in (1, 2):
        cache.kvq_pages_set_kernel(which)
        check_attention(c, q, cache.kvq_pages_attn(0, q.cuda(), c.batch()).cpu(), data)


# ------------------------------------------------------ bad indexes, streams --

@gpu
def test_bad_indexes_are_reported_and_not_followed():
    c = make(([2, 2, 40], [40, 20, 60]), 16, "f16", (2, 2), 64, seed=1)
    data = fill(c, 2, 64)
    k = c.normal(c.rows, 2, 64).half().cuda()
    q = c.normal(c.rows, 2, 64).half()
    for entry in (c.pages, -1, 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[0, 2] = entry
        batch = kvq.PagesBatch(c.q_start.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda(), table.cuda(), c.rows)
        for which in (1, 2):
            c.cache.kvq_pages_set_kernel(which)
            got = c.cache.kvq_pages_attn(0, q.cuda(), batch).cpu()
            assert c.cache.kvq_pages_status() == 7
            assert c.cache.kvq_pages_status() == 0
            s = c.q_start.tolist()
            for b in (1, 2):  # the other sequences are right
                ref, tol = attention(q[s[b]:s[b + 1]], *data[b], torch.arange(c.lens[b] - c.news[b], c.lens[b]), 0, 0.125,
                                     HALF_STEP[torch.float16])
                assert ((got[s[b]:s[b + 1]].double() - ref).abs() <= tol + ref.abs() * 2.0 ** -11 + 2.0 ** -25).all()
        before = c.cache.buffer.clone()
        one = kvq.PagesBatch(torch.tensor([0, 2], dtype=torch.int32).cuda(), torch.tensor([40], dtype=torch.int32).cuda(),
                             table[:1].cuda(), 2)
        c.cache.kvq_pages_append(0, k[:2], k[:2], one)
        assert c.cache.kvq_pages_status() == 7
        assert torch.equal(before, c.cache.buffer)
        out = torch.full((2, 2, 64), 3.0, dtype=torch.float16, device="cuda")
        c.cache.kvq_pages_read(0, one, out, out.clone())
        assert c.cache.kvq_pages_status() == 7 and (out == 3).all()


@gpu
@pytest.mark.parametrize("q_start,lens", [([0, 2, 4], [40, 1000000]), ([0, 2, 4], [40, -5]), ([0, 3, 2], [40, 20]),
                                          ([-1, 2, 4], [40, 20]), ([0, 2, 9], [40, 20])])
def test_bad_lengths_are_reported(q_start, lens):
    c = make(([2, 2], [40, 20]), 16, "8_8", (2, 2), 64, seed=1)
    fill(c, 2, 64)
    batch = kvq.PagesBatch(torch.tensor(q_start, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           c.table.cuda(), 4)
    q = c.normal(4, 2, 64).half().cuda()
    for which in (1, 2):
        c.cache.kvq_pages_set_kernel(which)
        c.cache.kvq_pages_attn(0, q, batch)
        assert c.cache.kvq_pages_status() == 7
    c.cache.kvq_pages_append(0, q, q, batch)
    assert c.cache.kvq_pages_status() == 7


@gpu
@pytest.mark.parametrize("q_start,lens,bad", [([0, 2, 4], [49, 20], [0]), ([0, 2, 4], [40, -5], [1]),
                                              ([0, 3, 2], [40, 20], [1]), ([-1, 2, 4], [40, 20], [0]),
                                              ([0, 2, 9], [40, 20], [1])])
@pytest.mark.parametrize("fmt", ["f16", "8_8"])
def test_sequences_out_of_range_keep_what_they_hold(fmt, q_start, lens, bad):
    """A length or rows that do not fit: the sequence is neither written nor read back."""
    c = make(([2, 2], [40, 20]), 16, fmt, (2, 2), 64, seed=1)
    data = fill(c, 2, 64)
    batch = kvq.PagesBatch(torch.tensor(q_start, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           c.table.cuda(), 4)
    x = c.normal(4, 2, 64).half().cuda()
    c.cache.kvq_pages_append(0, x, x, batch)
    assert c.cache.kvq_pages_status() == 7
    ko, vo = (y.cpu() for y in c.cache.kvq_pages_read(0, c.whole()))
    s = c.k_start.tolist()
    for b in range(2):
        same = torch.equal(ko[s[b]:s[b + 1]], data[b][0]) and torch.equal(vo[s[b]:s[b + 1]], data[b][1])
        assert same == (b in bad)
    out = torch.full((4, 2, 64), 3.0, dtype=torch.float16, device="cuda")
    got, _ = c.cache.kvq_pages_read(0, batch, out, out.clone())
    assert c.cache.kvq_pages_status() == 7
    kept = [bool((row == 3).all()) for row in got]
    good = [t for b in range(2) if b not in bad for t in range(q_start[b], q_start[b + 1])]
    assert kept == [t not in good for t in range(4)]


@gpu
def test_rope_rows_too_few_are_reported():
    c = make("ones", 16, "f16", (2, 2), 64)
    x = c.normal(c.rows, 2, 64).half().cuda()
    c.cache.kvq_pages_append(0, x, x, c.batch(), rope=kvq.Rope(angles(17, 64).cuda(), PAIRS))
    assert c.cache.kvq_pages_status() == 7  # positions 0 and 16 have rows, 39 has none
    fill = torch.full((3, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    _, vo = c.cache.kvq_pages_read(0, c.batch(), fill.clone(), fill.clone())
    assert torch.equal(vo[0], x[0]) and torch.equal(vo[2], x[2]) and not vo[1].any()


@gpu
def test_call_refusals(L):
    c = make("ones", 16, "f16", (4, 2), 64, layers=2)
    x = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    q = torch.zeros((3, 4, 64), dtype=torch.float16, device="cuda")
    b, cache = c.batch(), c.cache
    for layer in (-1, 2):
        with pytest.raises(kvq.KVQError) as e:
            cache.kvq_pages_append(layer, x, x, b)
        assert e.value.status == 1
        with pytest.raises(kvq.KVQError):
            cache.kvq_pages_attn(layer, q, b)
        with pytest.raises(kvq.KVQError):
            cache.kvq_pages_read(layer, b)
    for bad in (dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=3e38)):
        with pytest.raises(kvq.KVQError):
            cache.kvq_pages_attn(0, q, b, **bad)
    with pytest.raises(kvq.KVQError):
        cache.kvq_pages_attn(0, q.bfloat16(), b)
    for call in (lambda: cache.kvq_pages_attn(0, q.float(), b), lambda: cache.kvq_pages_attn(0, q[:2], b),
                 lambda: cache.kvq_pages_attn(0, q.cpu(), b), lambda: cache.kvq_pages_attn(0, x, b),
                 lambda: cache.kvq_pages_attn(0, q, b, out=q.bfloat16()), lambda: cache.kvq_pages_append(0, x, x[:2], b),
                 lambda: cache.kvq_pages_append(0, x, x.float(), b), lambda: cache.kvq_pages_append(0, x.int(), x.int(), b),
                 lambda: cache.kvq_pages_append(0, x.transpose(1, 2), x, b), lambda: cache.kvq_pages_read(0, b, x[:2])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(kvq.KVQError):
        cache.kvq_pages_set_kernel(3)
    for n, bt in ((-1, 1), (3, 0), (3, 1025)):
        r = kvq._PagesBatch(bt, n, 0, b.q_start.data_ptr(), b.lens.data_ptr(), b.table.data_ptr(), b.table.shape[1])
        assert L.kvq_pages_read(cache.handle, 0, ctypes.byref(r), None, None, None) == 1
    assert b"batch" in L.kvq_pages_last_error(cache.handle)
    r = kvq._PagesBatch(3, 2 ** 31 - 1, 0, b.q_start.data_ptr(), b.lens.data_ptr(), b.table.data_ptr(), 3)
    assert L.kvq_pages_read(cache.handle, 0, ctypes.byref(r), None, None, None) == 2
    # pointers that do not fit their elements are refused on the host
    r, odd = ctypes.byref(b.c), lambda t, by=1: t.data_ptr() + by
    assert L.kvq_pages_attn(cache.handle, 0, odd(q), 0, 256, r, 0.0, 0, q.data_ptr(), None) == 1
    assert L.kvq_pages_append(cache.handle, 0, odd(x), x.data_ptr(), 0, 128, 128, r, None, None) == 1
    assert L.kvq_pages_append(cache.handle, 0, x.data_ptr(), odd(x, 2), 1, 128, 128, r, None, None) == 1
    for i in range(3):
        ptrs = [t.data_ptr() + 2 * (i == j) for j, t in enumerate((b.q_start, b.lens, b.table))]
        shifted = kvq._PagesBatch(3, 3, 0, *ptrs, b.table.shape[1])
        assert L.kvq_pages_read(cache.handle, 0, ctypes.byref(shifted), None, None, None) == 1
    rope = kvq._Rope(x.data_ptr(), 3, 64, 0, b.lens.data_ptr() + 2)
    assert L.kvq_pages_append(cache.handle, 0, x.data_ptr(), x.data_ptr(), 0, 128, 128, r, ctypes.byref(rope), None) == 1
    # no rows: nothing to do
    empty = kvq.PagesBatch(torch.zeros(2, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                           torch.zeros((1, 1), dtype=torch.int32).cuda(), 0)
    cache.kvq_pages_append(0, x[:0], x[:0], empty)
    assert cache.kvq_pages_attn(0, q[:0], empty).shape == (0, 4, 64)
    assert cache.kvq_pages_status() == 0


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "4_4"])
def test_captured_step_replayed_with_other_lengths(fmt):
    """Norm with rotation, append and attention of one step, captured once and
    replayed while the sequences grow, against the same steps run eagerly; on a
    stream of its own."""
    d, hq, h, steps = 128, 8, 2, 20
    start, news = [30, 0, 100], [1, 1, 1]
    a, b = (make((news, [n + steps for n in start]), 16, fmt, (hq, h), d, seed=7) for _ in range(2))
    tab = angles(200, d).cuda()
    g = torch.Generator().manual_seed(3)
    x = torch.randn((steps, 3, hq + 2 * h, d), generator=g).to(a.dtype).cuda()
    w = torch.rand(d, generator=g).to(a.dtype).cuda()
    pk = torch.randn((130, 2, h, d), generator=g).cuda()
    for c in (a, b):
        pre = kvq.PagesBatch(torch.tensor([0, 30, 30, 130], dtype=torch.int32).cuda(),
                             torch.tensor(start, dtype=torch.int32).cuda(), c.table.cuda(), 130)
        c.cache.kvq_pages_append(0, pk[:, 0], pk[:, 1], pre)

    def step(c, row, batch, rope, out):
        q, k = kvq.kvq_qk_norm_rope(row[:, :hq], row[:, hq:hq + h], w, w, rope=rope)
        c.cache.kvq_pages_append(0, k, row[:, hq + h:], batch)
        return c.cache.kvq_pages_attn(0, q, batch, out=out)

    def state(c):
        lens = torch.tensor(start, dtype=torch.int32).cuda()
        pos = lens.clone()
        batch = kvq.PagesBatch(torch.tensor([0, 1, 2, 3], dtype=torch.int32).cuda(), lens, c.table.cuda(), 3, 1)
        return lens, pos, batch, kvq.Rope(tab, HALVES, pos), torch.zeros((3, hq, d), dtype=a.dtype, device="cuda")

    lens, pos, batch, rope, out = state(a)
    want = []
    for i in range(steps):
        pos.copy_(lens)
        lens += 1
        want.append(step(a, x[i], batch, rope, out).clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lens, pos, batch, rope, out = state(b)
        row = torch.zeros_like(x[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pos.copy_(lens)
            lens += 1
            step(b, row, batch, rope, out)
        for i in range(steps):
            row.copy_(x[i])
            graph.replay()
            assert torch.equal(out, want[i])
    torch.cuda.synchronize()
    assert a.cache.kvq_pages_status() == 0 and b.cache.kvq_pages_status() == 0
    per = int(a.cache.bytes.packed + a.cache.bytes.metadata)
    assert torch.equal(a.cache.buffer[:per], b.cache.buffer[:per])


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_chunks_of_a_prompt_agree_with_the_whole(fmt):
    """A prompt in one call and in chunks (some of one token): the same bytes in the
    pages, and outputs that are each within the bound of the 64-bit form."""
    d, hq, h, t = 128, 8, 2, 300
    whole = make(([t], [t]), 32, fmt, (hq, h), d, seed=11)
    parts = make(([t], [t]), 32, fmt, (hq, h), d, seed=11)
    k, v = whole.normal(t, h, d).cuda(), whole.normal(t, h, d).cuda()
    q = whole.normal(t, hq, d).to(whole.dtype)
    whole.cache.kvq_pages_append(0, k, v, whole.batch())
    data = [tuple(x.cpu() for x in whole.cache.kvq_pages_read(0, whole.batch()))]
    check_attention(whole, q, whole.cache.kvq_pages_attn(0, q.cuda(), whole.batch()).cpu(), data)
    got, at = torch.zeros(q.shape, dtype=q.dtype), 0
    for n in (1, 16, 100, 1, 7, 175):
        b = kvq.PagesBatch(torch.tensor([0, n], dtype=torch.int32).cuda(),
                           torch.tensor([at + n], dtype=torch.int32).cuda(), parts.table.cuda(), n)
        parts.cache.kvq_pages_append(0, k[at:at + n], v[at:at + n], b)
        got[at:at + n] = parts.cache.kvq_pages_attn(0, q[at:at + n].cuda(), b).cpu()
        at += n
    assert at == t
    check_attention(parts, q, got, data)
    per = int(whole.cache.bytes.packed + whole.cache.bytes.metadata)
    assert torch.equal(whole.cache.buffer[:per], parts.cache.buffer[:per])
