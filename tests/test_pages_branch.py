"""Branching sequences on the paged cache: trees of drafted tokens, cross attention,
keeping some of the tokens, copying pages, and tables whose rows share pages, against
plain forms (64 bits for attention, step by step for tables)."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from bit_quantized_kv_02_gb300 import build, kvq
from tests.pages_ref import FORMATS, HALF_STEP, HALVES, Case, angles
from tests.test_pages import fill, make

gpu = pytest.mark.gpu
WHICH = pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(kvq.LIB_PATH):
        build.build()
    return kvq.lib()


def ints(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


# ----------------------------------------------------------------- refusals --

def test_calls_without_a_handle(L):
    assert L.kvq_pages_tree(None, None, None, 1, None, None, None) == 1
    assert L.kvq_pages_tree_attn(None, 0, None, 0, 0, None, None, 0.0, 0, None, None) == 1
    assert L.kvq_pages_cross_attn(None, 0, None, 0, 0, None, 0.0, None, None) == 1
    assert L.kvq_pages_keep(None, 0, None, None, None, None) == 1
    assert L.kvq_pages_copy(None, 0, None, None, 0, None) == 1
    assert L.kvq_pages_fork(None, None, None) == 1
    assert L.kvq_pages_grow(None, None, None) == 1
    assert "free pages" in kvq.kvq_status_string(8)


def test_wrapper_refuses_cpu_tensors():
    with pytest.raises(ValueError):
        kvq.PagesTree(torch.zeros((3, 1), dtype=torch.int64))


@gpu
def test_call_refusals(L):
    """Each call refuses what it cannot use before it launches anything."""
    cache = kvq.KVQPages(kvq.make_pages_config(2, 6, 16, 4, 2, 64))
    z = torch.zeros(64, dtype=torch.int64, device="cuda")
    p = z.data_ptr()
    ref = ctypes.byref
    batch = kvq._PagesBatch(1, 3, 0, p, p, p, 1)
    none = kvq._PagesBatch(0, 3, 0, p, p, p, 1)
    out = torch.zeros((3, 4, 64), dtype=torch.float16, device="cuda")
    q = torch.zeros_like(out)

    def tree(seen=p, words=1, positions=p):
        return ref(kvq._Tree(seen, words, positions))

    def attn(t=None, window=0, layer=0, b=batch, dtype=0, stride=256, o=out.data_ptr()):
        return L.kvq_pages_tree_attn(cache.handle, layer, q.data_ptr(), dtype, stride, ref(b), t, 0.0, window, o, None)

    assert attn(None) == 1 and attn(tree(seen=None)) == 1 and attn(tree(words=0)) == 1 and attn(tree(words=5)) == 1
    assert attn(tree(seen=p + 4)) == 1 and attn(tree(positions=p + 2)) == 1
    assert attn(tree(), window=-1) == 1 and attn(tree(), window=63) == 2 and attn(tree(words=2), window=127) == 2
    assert attn(tree(positions=None), window=64) == 1
    assert attn(tree(), layer=2) == 1 and attn(tree(), layer=-1) == 1 and attn(tree(), b=none) == 1
    assert attn(tree(), dtype=2) == 1 and attn(tree(), stride=255) == 1 and attn(tree(), o=out.data_ptr() + 2) == 1
    assert attn(tree(), o=q.data_ptr()) == 1 and attn(tree(), o=None) == 1
    cross = L.kvq_pages_cross_attn
    assert cross(cache.handle, 2, q.data_ptr(), 0, 256, ref(batch), 0.0, out.data_ptr(), None) == 1
    assert cross(cache.handle, 0, q.data_ptr(), 0, 256, None, 0.0, out.data_ptr(), None) == 1
    assert cross(cache.handle, 0, q.data_ptr(), 0, 256, ref(batch), float("nan"), out.data_ptr(), None) == 1
    make_tree = L.kvq_pages_tree
    assert make_tree(cache.handle, None, p, 1, p, p, None) == 1
    for words in (0, 5):
        assert make_tree(cache.handle, ref(batch), p, words, p, p, None) == 1
    assert make_tree(cache.handle, ref(batch), None, 1, p, p, None) == 1
    assert make_tree(cache.handle, ref(batch), p, 1, None, p, None) == 1
    assert make_tree(cache.handle, ref(batch), p, 1, p + 4, p, None) == 1
    keep = L.kvq_pages_keep
    assert keep(cache.handle, 2, ref(batch), p, None, None) == 1 and keep(cache.handle, -2, ref(batch), p, None, None) == 1
    assert keep(cache.handle, 0, None, p, None, None) == 1 and keep(cache.handle, 0, ref(batch), None, None, None) == 1
    assert keep(cache.handle, 0, ref(batch), p, p, None) == 1 and keep(cache.handle, 0, ref(batch), p, p + 6, None) == 1
    copy = L.kvq_pages_copy
    assert copy(cache.handle, 2, p, p, 1, None) == 1 and copy(cache.handle, 0, p, p, -1, None) == 1
    assert copy(cache.handle, 0, None, p, 1, None) == 1 and copy(cache.handle, 0, p, p + 2, 1, None) == 1
    assert copy(cache.handle, 0, None, None, 0, None) == 0

    def fork(**kw):
        f = dict(rows_in=2, rows_out=2, parent=p, table_in=p + 16, stride_in=2, lens_in=p + 40, refs_in=p + 64,
                 table_out=p + 96, stride_out=2, lens_out=p + 128, refs_out=p + 160)
        f.update(kw)
        return L.kvq_pages_fork(cache.handle, ref(kvq._ForkArgs(**f)), None)

    for name in ("parent", "table_in", "lens_in", "refs_in", "table_out", "lens_out", "refs_out"):
        assert fork(**{name: None}) == 1 and fork(**{name: p + 202}) == 1, name
    assert L.kvq_pages_fork(cache.handle, None, None) == 1
    assert fork(rows_in=0) == 1 and fork(rows_out=1025) == 1 and fork(stride_in=0) == 1 and fork(stride_out=0) == 1
    assert fork(table_out=p + 28) == 1 and fork(lens_out=p + 4) == 1 and fork(refs_out=p + 60) == 1
    assert fork(refs_out=p + 68) == 1 and fork(lens_out=p + 100) == 1 and fork(table_out=p + 172) == 1

    def grow(**kw):
        f = dict(sequences=2, q_start=p, lens=p + 16, table=p + 32, table_stride=2, refs=p + 64, lens_out=p + 96)
        f.update(kw)
        return L.kvq_pages_grow(cache.handle, ref(kvq._GrowArgs(**f)), None)

    for name in ("q_start", "lens", "table", "refs", "lens_out"):
        assert grow(**{name: None}) == 1 and grow(**{name: p + 202}) == 1, name
    assert L.kvq_pages_grow(cache.handle, None, None) == 1
    assert grow(sequences=0) == 1 and grow(sequences=1025) == 1 and grow(table_stride=0) == 1
    assert grow(sequences=1024, table_stride=1 << 21) == 2
    assert grow(lens_out=p + 20) == 1 and grow(lens_out=p + 8) == 1 and grow(table=p + 60) == 1 and grow(table=p + 12) == 1
    assert grow(refs=p + 4) == 1 and grow(lens_out=p + 84) == 1
    assert cache.kvq_pages_status() == 0
    # the wrapper's own
    b = kvq.PagesBatch(ints([0, 3]), ints([20]), ints([[0, 1]]), 3)
    t = kvq.PagesTree(torch.zeros((2, 1), dtype=torch.int64, device="cuda"))
    for call in (lambda: cache.kvq_pages_tree_attn(0, q, b, t), lambda: cache.kvq_pages_tree(ints([0, 0]), b),
                 lambda: cache.kvq_pages_tree(ints([0, 0, 0]), b, tree=t),
                 lambda: cache.kvq_pages_keep(torch.ones(3, device="cuda"), b),
                 lambda: cache.kvq_pages_keep(torch.ones(2, dtype=torch.bool, device="cuda"), b),
                 lambda: cache.kvq_pages_copy(ints([0, 1]), ints([2])),
                 lambda: cache.kvq_pages_fork(ints([0]), ints([[0, 1]]), ints([20]), ints([1])),
                 lambda: cache.kvq_pages_grow(ints([0]), ints([[0, 1]]), ints([20]), ints([1] * 6)),
                 lambda: cache.kvq_pages_cross_attn(0, q[:2], b)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cache.kvq_pages_tree(ints([0, 0, 0]), b, words=5),
                 lambda: cache.kvq_pages_keep(torch.ones(3, dtype=torch.bool, device="cuda"), b, layer=7)):
        with pytest.raises(kvq.KVQError):
            call()


# --------------------------------------------------------------------- trees --

def drafted(n, g, roots=0.1):
    """Parents of n drafted tokens."""
    return [-1 if i == 0 or float(torch.rand((), generator=g)) < roots else int(torch.randint(0, i, (), generator=g))
            for i in range(n)]


def ancestors(parents):
    """see [n][n]: row i's ancestors and itself."""
    n = len(parents)
    see = torch.zeros((n, n), dtype=torch.bool)
    for i, p in enumerate(parents):
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
    return see


def pack(see, words):
    """[n][n] truth values as [n][words] int64."""
    out = np.zeros((see.shape[0], words), np.uint64)
    for i, j in see.nonzero().tolist():
        out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(out.view(np.int64))


@gpu
@pytest.mark.parametrize("words,news", [(1, [1, 0, 64, 7, 33]), (2, [65, 128, 1]), (3, [150, 192]), (4, [256, 2, 255])])
def test_tree_masks_and_positions(words, news):
    c = make((news, [n + 5 * i for i, n in enumerate(news)]), 16, "f16", pad=3)
    kinds = [lambda n: drafted(n, c.g), lambda n: list(range(-1, n - 1)), lambda n: [-1] * n, lambda n: [-1] + [0] * (n - 1)]
    for kind in kinds:
        parents = [kind(n) if n else [] for n in news]
        seen = torch.full((c.rows, words), 9, dtype=torch.int64, device="cuda")
        pos = torch.full((c.rows,), 9, dtype=torch.int32, device="cuda")
        flat = ints(sum(parents, []) + [77] * 3)
        t = c.cache.kvq_pages_tree(flat, c.batch(), tree=kvq.PagesTree(seen, pos))
        assert t.seen is seen and c.cache.kvq_pages_status() == 0
        at = 0
        for b, p in enumerate(parents):
            see = ancestors(p)
            assert torch.equal(seen[at:at + len(p)].cpu(), pack(see, words))
            assert pos[at:at + len(p)].tolist() == (c.lens[b] - len(p) + see.sum(dim=1) - 1).tolist()
            at += len(p)
        assert (seen[at:] == 9).all() and (pos[at:] == 9).all()
        new = c.cache.kvq_pages_tree(flat, c.batch(), words=words)
        assert torch.equal(new.seen[:at], seen[:at]) and torch.equal(new.positions[:at], pos[:at])
        assert not new.seen[at:].any() and not new.positions[at:].any()
        c.cache.kvq_pages_tree(flat, c.batch(), tree=kvq.PagesTree(seen.zero_()))  # masks alone
        assert torch.equal(new.seen[:at], seen[:at])


@gpu
def test_tree_of_bad_parents_and_sequences():
    c = make(([4, 65, 2, 3], [10, 70, 2, 40]), 16, "f16")
    parents = [1, 0, 2, -2] + [-1] * 65 + [-1, 0] + [-1, 0, 0]
    t = c.cache.kvq_pages_tree(ints(parents), c.batch())
    assert c.cache.kvq_pages_status() == 7 and c.cache.kvq_pages_status() == 0
    # (1 and 2 are no earlier tokens, -2 is none at all)
    assert t.seen[:4, 0].tolist() == [1, 3, 4, 8] and t.positions[:4].tolist() == [6, 7, 6, 6]
    assert not t.seen[4:69].any() and not t.positions[4:69].any()  # more than 64 tokens: left as they were
    assert t.seen[69:, 0].tolist() == [1, 3, 1, 3, 5] and t.positions[69:].tolist() == [0, 1, 37, 38, 38]
    bad = kvq.PagesBatch(c.q_start.cuda(), ints([10, 70, -1, 40]), c.table.cuda(), c.rows)
    t = c.cache.kvq_pages_tree(ints(parents), bad, words=2)
    assert c.cache.kvq_pages_status() == 7
    assert t.seen[4:69, 0].any() and not t.seen[69:71].any() and t.seen[71:, 0].tolist() == [1, 3, 5]


def attention_of(q, k, v, see, scale, p_half_step):
    """One sequence, rows of q seeing `see` [n][t]: (out, bound) in 64 bits, the bound counted as in
    tests/pages_ref.py's attention."""
    n, hq, d = q.shape
    t, h = k.shape[0], k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, bound = torch.zeros(n, hq, d, dtype=torch.float64), torch.zeros(n, hq, d, dtype=torch.float64)
    if t == 0 or n == 0:
        return out, bound
    for j in range(hq):
        kk, vv = k[:, j // (hq // h)], v[:, j // (hq // h)]
        s = ((q[:, j] @ kk.T) * scale).masked_fill(~see, -math.inf)
        size = (q[:, j].abs() @ kk.abs().T) * scale
        e = torch.exp(s - s.amax(dim=-1, keepdim=True).clamp_min(-1e300))
        tot = e.sum(dim=-1, keepdim=True)
        p = torch.where(tot > 0, e / tot, torch.zeros_like(e))
        out[:, j] = p @ vv
        off = 2.0 * (size * see).amax(dim=-1, keepdim=True) * (d + 4) * 2.0 ** -23 + 2.0 ** -20
        sums = (t / 16 + 64) * 2.0 ** -23
        bound[:, j] = (p_half_step + 2 * off + 2 * sums) * (p @ vv.abs()) + t * 2.0 ** -31 * vv.abs().max()
    return out, bound


def check(c, q, got, data, sees, scale=None):
    scale = scale or 1.0 / math.sqrt(q.shape[2])
    p_step = HALF_STEP[torch.float16 if c.bits[0] < 16 else c.dtype]
    s = c.q_start.tolist()
    for b, (k, v) in enumerate(data):
        rows = slice(s[b], s[b + 1])
        ref, tol = attention_of(q[rows], k, v, sees[b], scale, p_step)
        tol = tol + ref.abs() * HALF_STEP[q.dtype] + 2.0 ** -25
        off = (got[rows].double() - ref).abs()
        assert (off <= tol).all(), (b, float((off / tol).max()))


def tree_sees(c, masks, depths, window):
    """What each row of each sequence sees: the past (inside the window), and its mask among the new tokens."""
    sees = []
    for n, ln, m, depth in zip(c.news, c.lens, masks, depths):
        past = ln - n
        see = torch.zeros((n, ln), dtype=torch.bool)
        if past > 0:
            at = torch.arange(past)[None, :]
            see[:, :past] = (at > past + depth[:, None] - window) if window else True
        see[:, max(past, 0):] = m[:, max(-past, 0):]
        sees.append(see)
    return sees


TREES = {
    "one": ([1, 1, 1], [1, 40, 700], 1),
    "drafts": ([5, 3, 0, 8, 16], [700, 3, 20, 129, 16], 1),
    "mixed": ([1, 60, 0, 17, 64], [2000, 60, 0, 500, 450], 1),
    "wide": ([200, 3, 129], [500, 140, 129], 4),
    "two": ([65, 128], [1100, 128], 2),
    "negative": ([4, 3, 40], [2, 0, 33], 1),
    "long": ([21], [9000], 1),
}


@gpu
@WHICH
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name,page_tokens,d,heads,window", [
    ("one", 16, 64, (12, 12), 0), ("drafts", 32, 128, (8, 1), 0), ("drafts", 16, 64, (3, 1), 64),
    ("mixed", 64, 128, (4, 4), 0), ("mixed", 32, 256, (5, 1), 100), ("wide", 128, 64, (4, 2), 300),
    ("two", 16, 256, (4, 2), 0), ("negative", 16, 128, (4, 2), 0), ("negative", 64, 64, (64, 1), 70),
    ("long", 128, 64, (2, 1), 0), ("long", 16, 128, (8, 1), 4000)])
def test_tree_attention(which, fmt, name, page_tokens, d, heads, window):
    news, lens, words = TREES[name]
    c = make((news, lens), page_tokens, fmt, heads, d, seed=4, pad=3)
    data = fill(c, heads[1], d)
    parents = [drafted(n, c.g) for n in news]
    tree = c.cache.kvq_pages_tree(ints(sum(parents, []) + [0] * 3), c.batch(), words=words)
    masks = [ancestors(p) for p in parents]
    sees = tree_sees(c, masks, [m.sum(dim=1) - 1 for m in masks], window)
    for dtype in [c.dtype] if c.bits[0] == 16 else [torch.float16, torch.bfloat16]:
        q = c.normal(c.rows, heads[0], d).to(dtype)
        out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
        c.cache.kvq_pages_set_kernel(which)
        got = c.cache.kvq_pages_tree_attn(0, q.cuda(), c.batch(), tree, out=out, window=window)
        assert c.cache.kvq_pages_status() == 0
        assert (got[c.n:] == 5).all()
        check(c, q, got.cpu(), data, sees)
        again = c.cache.kvq_pages_tree_attn(0, q.cuda(), c.batch(), tree, window=window)
        assert torch.equal(again[:c.n], got[:c.n])
        c.cache.kvq_pages_set_kernel(0)
        for hint in (0, max(news)):
            check(c, q, c.cache.kvq_pages_tree_attn(0, q.cuda(), c.batch(hint), tree, window=window).cpu(), data, sees)


@gpu
@WHICH
@pytest.mark.parametrize("fmt", ["f16", "4_8"])
@pytest.mark.parametrize("past", [0, 37, 128, 250])
def test_any_mask_of_the_new_tokens(which, fmt, past):
    """Masks that are no trees: later tokens seen, nothing seen (zeros where there is no past
    either), bits behind the last token, and a first block without a visible token."""
    n = 150
    c = make(([n, 64], [past + n, 64]), 32, fmt, (6, 2), 64, seed=past)
    data = fill(c, 2, 64)
    masks = [torch.rand((n, n), generator=c.g) < 0.3, torch.zeros((64, 64), dtype=torch.bool)]
    masks[0][3] = False
    masks[0][7] = True
    masks[0][9] = False
    masks[0][9, n - 1] = True
    masks[1][5, 63] = True
    seen = torch.cat([pack(m, 3) for m in masks])
    seen[:n, 2] |= torch.tensor(-1 << (n - 128), dtype=torch.int64)
    seen[n:, 1:] = -1
    tree = kvq.PagesTree(seen.cuda())
    sees = tree_sees(c, masks, [None, None], 0)
    c.cache.kvq_pages_set_kernel(which)
    q = c.normal(c.rows, 6, 64).to(c.dtype)
    got = c.cache.kvq_pages_tree_attn(0, q.cuda(), c.batch(), tree)
    assert c.cache.kvq_pages_status() == 0
    check(c, q, got.cpu(), data, sees)
    assert not got[n:n + 5].any() and not got[n + 6:].any()


@gpu
@WHICH
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_tree_of_one_token_is_plain_attention(which, fmt, d):
    """Bit for bit by the kernel for few rows.  The masked kernel for many rows sums the even and the odd
    blocks of few rows apart, so there both are held to the same value in 64 bits."""
    c = make(([1, 1, 1], [200, 1, 1333]), 64, fmt, (4, 2), d, seed=1)
    data = fill(c, 2, d)
    c.cache.kvq_pages_set_kernel(which)
    q = c.normal(c.rows, 4, d).to(c.dtype)
    tree = c.cache.kvq_pages_tree(ints([-1] * 3), c.batch())
    one = [torch.ones((1, 1), dtype=torch.bool)] * 3
    for window in (0, 100):
        got = c.cache.kvq_pages_tree_attn(0, q.cuda(), c.batch(), tree, window=window)
        plain = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(), window=window)
        sees = tree_sees(c, one, [torch.zeros(1, dtype=torch.int64)] * 3, window)
        check(c, q, got.cpu(), data, sees)
        check(c, q, plain.cpu(), data, sees)
        if which == 1:
            assert torch.equal(got, plain)


@gpu
@WHICH
@pytest.mark.parametrize("fmt", FORMATS)
def test_tree_and_cross_do_not_see_what_pages_held_before(which, fmt):
    """NaN and infinities of an earlier owner of the pages, behind the sequence's end."""
    c = make(([1, 20, 40, 64], [5, 50, 40, 200]), 64, fmt, (4, 2), 128, seed=9)
    per = int(c.cache.bytes.packed + c.cache.bytes.metadata)
    c.cache.buffer[:per].fill_(0xFF)
    data = fill(c, 2, 128)
    q = c.normal(c.rows, 4, 128).to(c.dtype)
    parents = [drafted(n, c.g) for n in c.news]
    masks = [ancestors(p) for p in parents]
    c.cache.kvq_pages_set_kernel(which)
    tree = c.cache.kvq_pages_tree(ints(sum(parents, [])), c.batch())
    got = c.cache.kvq_pages_tree_attn(0, q.cuda(), c.batch(), tree)
    check(c, q, got.cpu(), data, tree_sees(c, masks, [None] * 4, 0))
    got = c.cache.kvq_pages_cross_attn(0, q.cuda(), c.batch())
    assert c.cache.kvq_pages_status() == 0
    check(c, q, got.cpu(), data, [torch.ones((n, ln), dtype=torch.bool) for n, ln in zip(c.news, c.lens)])


@gpu
def test_bad_sequences_of_a_tree_are_reported():
    c = make(([70, 3], [100, 50]), 16, "bf16", (4, 2), 64)
    data = fill(c, 2, 64)
    q = c.normal(c.rows, 4, 64).to(c.dtype)
    parents = drafted(3, c.g)
    tree = kvq.PagesTree(torch.cat([torch.zeros((70, 1), dtype=torch.int64), pack(ancestors(parents), 1)]).cuda(),
                         ints([-2 ** 31] * 35 + [2 ** 31 - 1] * 35 + [47, 48, 49]))
    for which in (0, 1, 2):
        c.cache.kvq_pages_set_kernel(which)
        got = c.cache.kvq_pages_tree_attn(0, q.cuda(), c.batch(), tree, window=64).cpu()
        assert c.cache.kvq_pages_status() == 7  # more than 64 tokens in the first sequence
        see = torch.ones((3, 50), dtype=torch.bool)
        see[:, 47:] = ancestors(parents)
        ref, tol = attention_of(q[70:], *data[1], see, 1 / 8, HALF_STEP[c.dtype])
        assert ((got[70:].double() - ref).abs() <= tol + ref.abs() * HALF_STEP[c.dtype] + 2.0 ** -25).all()


# --------------------------------------------------------------------- cross --

CROSS = {
    "steps": ([1, 1, 1, 1, 1], [1, 0, 333, 1500, 128]),
    "prompts": ([5, 200, 0, 33, 7], [700, 3, 20, 0, 129]),
    "long": ([3], [9000]),
    "many": ([150, 100], [500, 1]),
}


@gpu
@WHICH
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name,page_tokens,d,heads", [
    ("steps", 16, 64, (12, 12)), ("steps", 64, 128, (8, 2)), ("steps", 128, 256, (16, 2)), ("prompts", 32, 128, (8, 1)),
    ("prompts", 16, 256, (3, 1)), ("long", 64, 64, (4, 4)), ("many", 128, 64, (64, 1)), ("many", 16, 128, (6, 2))])
def test_cross_attention(which, fmt, name, page_tokens, d, heads):
    c = make(CROSS[name], page_tokens, fmt, heads, d, seed=6, pad=2)
    data = fill(c, heads[1], d)
    sees = [torch.ones((n, ln), dtype=torch.bool) for n, ln in zip(c.news, c.lens)]
    for dtype in [c.dtype] if c.bits[0] == 16 else [torch.float16, torch.bfloat16]:
        q = c.normal(c.rows, heads[0], d).to(dtype)
        out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
        c.cache.kvq_pages_set_kernel(which)
        got = c.cache.kvq_pages_cross_attn(0, q.cuda(), c.batch(), out=out)
        assert c.cache.kvq_pages_status() == 0
        assert (got[c.n:] == 5).all()
        check(c, q, got.cpu(), data, sees)
        c.cache.kvq_pages_set_kernel(0)
        for hint in (0, max(c.news)):
            check(c, q, c.cache.kvq_pages_cross_attn(0, q.cuda(), c.batch(hint), scale=0.2).cpu(), data, sees, scale=0.2)


# ---------------------------------------------------------------------- keep --

def layers_of(c, layers):
    """What each layer holds: [(keys, values)] of all tokens of all sequences."""
    return [tuple(x.cpu() for x in c.cache.kvq_pages_read(i, c.whole())) for i in range(layers)]


def kept(c, keep, before):
    """The rows of all sequences' tokens after the kept ones closed up, and the lengths."""
    after, lens, row, at = [x.clone() for x in before], [], 0, 0
    for n, ln in zip(c.news, c.lens):
        first = max(ln - n, 0)
        src = [ln - n + i for i in range(n) if keep[row + i] and ln - n + i >= 0]
        for x, y in zip(after, before):
            x[at + first:at + first + len(src)] = y[at:at + ln][src]
        lens.append(first + len(src))
        row += n
        at += ln
    return after, lens


KEEPS = {
    "drafts": ([5, 1, 0, 64, 3], [705, 1, 9, 130, 40]),
    "negative": ([4, 3, 40], [2, 0, 33]),
    "whole": ([300, 17, 2000], [300, 17, 2000]),
    "tail": ([513, 256], [700, 1000]),
}


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name,page_tokens,d,h", [("drafts", 16, 64, 12), ("drafts", 64, 128, 3), ("negative", 32, 64, 2),
                                                  ("whole", 16, 256, 2), ("whole", 128, 64, 1), ("tail", 32, 128, 5)])
def test_keep(fmt, name, page_tokens, d, h):
    layers = 3
    c = make(KEEPS[name], page_tokens, fmt, (h, h), d, layers=layers, seed=8, pad=2)
    for i in range(layers):
        fill(c, h, d, layer=i)
    for share in (0.0, 0.1, 0.5, 0.95, 1.0):
        keep = torch.rand(c.rows, generator=c.g) < share
        for layer in (kvq.ALL_LAYERS, 1):
            before, buf = layers_of(c, layers), c.cache.buffer.clone()
            marks = keep.cuda() if layer == 1 else (keep.to(torch.uint8) * 200).cuda()
            lens = c.cache.kvq_pages_keep(marks, c.batch(), layer=layer)
            assert c.cache.kvq_pages_status() == 0
            for i, (x, y) in enumerate(zip(layers_of(c, layers), before)):
                want, new = kept(c, keep.tolist(), y)
                if layer in (kvq.ALL_LAYERS, i):
                    assert all(torch.equal(a, b) for a, b in zip(x, want))
                else:
                    assert all(torch.equal(a, b) for a, b in zip(x, y))
            assert lens.tolist() == new
            # pages of no sequence, and the other layers, have not changed by a byte
            size = c.cache.buffer.numel()
            per = (int(c.cache.bytes.packed + c.cache.bytes.metadata) // layers + 255) // 256 * 256
            assert per * layers <= size
            pages = [x[:per * layers].view(layers, per)[:, :per // c.pages * c.pages].view(layers, c.pages, -1)
                     for x in (buf, c.cache.buffer)] if per % c.pages == 0 else None
            if pages is not None:
                assert torch.equal(pages[0][:, c.free.long().cuda()], pages[1][:, c.free.long().cuda()])


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "4_4"])
@pytest.mark.parametrize("share", [0.03, 0.5, 0.9, 0.999])
def test_keep_of_long_sequences(fmt, share):
    """Tens of thousands of tokens in segments that many CTAs move: few and many places between a token's
    old place and its new one; a hint that is wrong changes nothing."""
    c = make(([20011, 129, 3, 6000], [20011, 500, 3, 6000]), 32, fmt, (3, 3), 64, layers=2, seed=4, pad=1)
    for trial in range(3):
        for i in range(2):
            fill(c, 3, 64, layer=i)
        keep = torch.rand(c.rows, generator=c.g) < share
        before = layers_of(c, 2)
        lens = c.cache.kvq_pages_keep(keep.cuda(), c.batch(max_new=5 if trial == 2 else 0))
        assert c.cache.kvq_pages_status() == 0
        for x, y in zip(layers_of(c, 2), before):
            want, new = kept(c, keep.tolist(), y)
            assert all(torch.equal(a, b) for a, b in zip(x, want))
        assert lens.tolist() == new


@gpu
def test_keep_of_more_rows_than_its_workspace_counts():
    """Sequences that name the same rows, twice as many as the segments there is room for."""
    n = 16400 * 128
    cache = kvq.KVQPages(kvq.make_pages_config(1, 2, 128, 1, 1, 64))
    table = torch.zeros((4, 16400), dtype=torch.int32, device="cuda")
    batch = kvq.PagesBatch(ints([0, n, 0, n, n]), ints([n, 7, n, 5]), table, n)
    lens = cache.kvq_pages_keep(torch.zeros(n, dtype=torch.bool, device="cuda"), batch)
    assert cache.kvq_pages_status() == 7
    assert lens.tolist() == [0, 7, n, 5]


@gpu
def test_keep_where_indices_are_bad():
    """A bad page leaves its tokens, a bad sequence all of its own; both are reported, the others are right."""
    c = make(([40, 5, 6], [40, 20, 30]), 16, "f16", (2, 2), 64, layers=1)
    fill(c, 2, 64)
    before = layers_of(c, 1)[0]
    keep = torch.ones(c.rows, dtype=torch.bool)
    keep[0] = False
    keep[42] = False
    keep[46] = False
    table = c.table.clone()
    table[0, 1] = c.pages + 5
    bad = kvq.PagesBatch(c.q_start.cuda(), ints([40, 1 << 20, 30]), table.cuda(), c.rows)
    lens = c.cache.kvq_pages_keep(keep.cuda(), bad)
    assert c.cache.kvq_pages_status() == 7
    assert lens.tolist() == [39, 1 << 20, 29]
    after = layers_of(c, 1)[0]
    for x, y in zip(after, before):
        # (tokens 1 .. 15 and 33 .. 39 move inside their pages, those that page 1 holds or would hold do not)
        assert torch.equal(x[:15], y[1:16]) and torch.equal(x[15:32], y[15:32]) and torch.equal(x[32:39], y[33:40])
        assert torch.equal(x[40:60], y[40:60])
        want = y[60:90].clone()
        want[25:29] = y[86:90]  # (row 46, token 25, is dropped)
        assert torch.equal(x[60:90], want)


@gpu
def test_keep_without_lengths_and_without_rows(L):
    c = make(([0, 0], [20, 3]), 16, "f16", (2, 2), 64)
    b = c.batch()
    assert c.cache.kvq_pages_keep(torch.ones(0, dtype=torch.bool, device="cuda"), b).tolist() == [20, 3]
    assert L.kvq_pages_keep(c.cache.handle, -1, b.ref, None, None, None) == 0


# ---------------------------------------------------------------------- copy --

@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page_tokens,d,h", [(16, 64, 1), (64, 128, 5), (128, 256, 2)])
def test_copy(fmt, page_tokens, d, h):
    k, v, dtype = FORMATS[fmt]
    pages, layers = 16, 3  # (a layer of 16 pages is a multiple of 256 bytes, so pages lie side by side)
    cache = kvq.KVQPages(kvq.make_pages_config(layers, pages, page_tokens, h, h, d, k, v, dtype))
    per = int(cache.bytes.packed + cache.bytes.metadata)
    g = torch.Generator().manual_seed(3)
    for layer in (kvq.ALL_LAYERS, 2):
        cache.buffer[:per].copy_(torch.randint(0, 256, (per,), generator=g).to(torch.uint8))
        rest = cache.buffer[per:].clone()
        want = cache.buffer[:per].clone().view(layers, pages, -1)
        src, dst = [3, 0, -1, 15, 3, 7, pages, 2], [9, 1, 4, 8, 10, -5, 5, pages + 3]
        for s, t in list(zip(src, dst))[:2] + [(15, 8), (3, 10)]:
            for i in range(layers):
                if layer in (kvq.ALL_LAYERS, i):
                    want[i, t] = want[i, s]
        cache.kvq_pages_copy(ints(src), ints(dst), layer=layer)
        assert cache.kvq_pages_status() == 7  # (the pairs outside the pool)
        assert torch.equal(cache.buffer[:per].view(layers, pages, -1), want)
        assert torch.equal(cache.buffer[per:], rest)
    cache.kvq_pages_copy(ints([1, 2]), ints([3, -1]))
    assert cache.kvq_pages_status() == 0
    cache.kvq_pages_copy(ints([]), ints([]))


# ------------------------------------------------------------- fork and grow --

class Pool:
    """Tables and reference counts, one sequence after the other."""

    def __init__(self, pages, page_tokens, rows, width):
        self.pages, self.pt, self.width = pages, page_tokens, width
        self.table = [[-1] * width for _ in range(rows)]
        self.lens = [0] * rows
        self.refs = [0] * pages

    def fork(self, parent):
        table, lens = [], []
        for p in parent:
            ln = self.lens[p] if p >= 0 else 0
            held = -(-(ln if ln >= 0 else -1 - ln) // self.pt)
            table.append([self.table[p][i] if i < held else -1 for i in range(self.width)] if p >= 0 else [-1] * self.width)
            lens.append(ln)
        for row in self.table:
            for x in row:
                if x >= 0:
                    self.refs[x] -= 1
        for row in table:
            for x in row:
                if x >= 0:
                    self.refs[x] += 1
        self.table, self.lens = table, lens

    def grow(self, news):
        """Returns the pages to copy."""
        free = [i for i, r in enumerate(self.refs) if r == 0]
        before, copies, full = list(self.refs), [], False
        done = {}  # sequences that have grown into a page
        for b, n in enumerate(news):
            ln = self.lens[b]
            if ln < 0:
                continue
            if n < 0 or ln + n > self.width * self.pt:
                self.lens[b] = -1 - ln
                continue
            if n == 0:
                continue
            fresh = []
            for i in range(ln // self.pt, (ln + n - 1) // self.pt + 1):
                x = self.table[b][i]
                if x < 0:
                    fresh.append((i, -1, False))
                elif i == ln // self.pt and ln % self.pt:
                    if done.get(x, 0) < before[x] - 1:
                        fresh.append((i, x, True))
                    done[x] = done.get(x, 0) + 1
                elif before[x] > 1:
                    fresh.append((i, x, False))
            if full or len(fresh) > len(free):
                full = True
                self.lens[b] = -1 - ln
                continue
            for i, x, copy in fresh:
                f = free.pop(0)
                self.table[b][i], self.refs[f] = f, 1
                if x >= 0:
                    self.refs[x] -= 1
                if copy:
                    copies.append((x, f))
            self.lens[b] = ln + n
        return copies

    def tensors(self):
        return ints(self.table), ints(self.lens), ints(self.refs)

    def same(self, table, lens, refs):
        assert lens.tolist() == self.lens
        assert table.tolist() == self.table
        assert refs.tolist() == self.refs

    def sound(self):
        count = [0] * self.pages
        for row in self.table:
            for x in row:
                if x >= 0:
                    count[x] += 1
        assert count == self.refs


def starts(news):
    return ints([0] + list(np.cumsum(news)))


@gpu
@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("pages,page_tokens,rows,width,most", [
    (60, 16, 6, 12, 20), (40, 32, 9, 5, 40), (700, 16, 33, 30, 90), (40000, 16, 7, 900, 5000), (3000, 128, 1024, 4, 130),
    (5, 64, 3, 4, 200)])
def test_fork_and_grow(pages, page_tokens, rows, width, most, seed):
    """Steps of a random life of sequences: tables, lengths and counts as dealt out one by one, and the
    copied pages' bytes."""
    r = np.random.RandomState(seed + pages)
    cache = kvq.KVQPages(kvq.make_pages_config(2, pages, page_tokens, 1, 1, 64))
    per = int(cache.bytes.packed) // 2
    cache.buffer[:2 * per].copy_(torch.from_numpy(r.randint(0, 256, 2 * per, dtype=np.uint8)))
    pool = Pool(pages, page_tokens, rows, width)
    # some pages are the caller's
    mine = r.permutation(pages)[:pages // 7]
    for x in mine:
        pool.refs[x] += 1
    table, lens, refs = pool.tensors()
    lowest = 0
    for step in range(6):
        parent = [int(r.randint(0, rows)) if r.rand() < 0.5 else (b if r.rand() < 0.8 else -1) for b in range(rows)]
        old = (table.clone(), lens.clone(), refs.clone())
        inplace = step % 2 == 1
        table2, lens2, refs2 = cache.kvq_pages_fork(ints(parent), table, lens, refs, refs_out=refs if inplace else None)
        pool.fork(parent)
        assert cache.kvq_pages_status() == 0
        pool.same(table2, lens2, refs2)
        assert torch.equal(table, old[0]) and torch.equal(lens, old[1])
        assert inplace or torch.equal(refs, old[2])
        table, lens, refs = table2, lens2, refs2
        news = [int(r.randint(0, most)) if r.rand() < 0.7 else 0 for _ in range(rows)]
        before = cache.buffer[:2 * per].clone().view(2, pages, -1)
        copies = pool.grow(news)
        grown = cache.kvq_pages_grow(starts(news), table, lens, refs, lens_out=lens if inplace else None)
        status = cache.kvq_pages_status()
        lowest = min([lowest] + pool.lens)
        assert status in ((0, 7, 8) if min(pool.lens) < 0 else (0,))
        pool.same(table, grown, refs)
        lens = grown
        for x, y in copies:
            before[:, y] = before[:, x]
        assert torch.equal(cache.buffer[:2 * per].view(2, pages, -1), before)
        for x in mine:
            pool.refs[x] -= 1
        pool.sound()
        for x in mine:
            pool.refs[x] += 1
    if pages == 5:
        assert lowest < 0  # it ran out


@gpu
def test_grow_reports_what_it_cannot_do():
    """Out of pages: the sequence and the growing ones behind it stay; an index out of range: that
    sequence alone; negative lengths are handed on."""
    cache = kvq.KVQPages(kvq.make_pages_config(1, 8, 16, 1, 1, 64))
    table = ints([[0, 1, -1], [2, -1, -1], [3, -1, -1], [4, -1, -1], [5, -1, -1]])
    refs = ints([1, 1, 1, 1, 1, 1, 0, 0])
    lens = ints([30, 16, 16, 10, 16])
    out = cache.kvq_pages_grow(starts([2, 33, 1, 3, 0]), table, lens, refs)
    assert cache.kvq_pages_status() == 7  # 49 tokens do not fit the table
    assert out.tolist() == [32, -17, 17, 13, 16]
    assert table.tolist() == [[0, 1, -1], [2, -1, -1], [3, 6, -1], [4, -1, -1], [5, -1, -1]]
    again = cache.kvq_pages_grow(starts([1, 1, 0, 17, 1]), table, out, refs)
    assert cache.kvq_pages_status() == 8
    # one page is left: the first takes it, the fourth finds none, the fifth stands behind it
    assert again.tolist() == [33, -17, 17, -14, -17]
    assert table.tolist() == [[0, 1, 7], [2, -1, -1], [3, 6, -1], [4, -1, -1], [5, -1, -1]]
    assert refs.tolist() == [1] * 8
    # what stays counts: freeing by a fork whose rows have negative lengths
    t2, l2, r2 = cache.kvq_pages_fork(ints([-1, 1, -1, 3, 4]), table, again, refs)
    assert l2.tolist() == [0, -17, 0, -14, -17] and cache.kvq_pages_status() == 0
    assert t2.tolist() == [[-1] * 3, [2, -1, -1], [-1] * 3, [4, -1, -1], [5, -1, -1]]
    assert r2.tolist() == [0, 0, 1, 0, 1, 1, 0, 0]
    # a table whose last page is none, q_start that decreases
    out = cache.kvq_pages_grow(ints([0, 1, 2, 1, 1, 2]), ints([[9, -1]] * 5), ints([5, 16, 16, 16, 16]), ints([0] * 8))
    assert cache.kvq_pages_status() == 7
    assert out.tolist() == [-6, 17, -17, 16, 17]


@gpu
def test_a_step_of_sequences_without_pages_touches_nothing():
    """The lengths that a refused growth leaves are skipped by every other call of the step."""
    cache = kvq.KVQPages(kvq.make_pages_config(2, 2, 16, 2, 2, 64))
    per = int(cache.bytes.packed)
    cache.buffer[:per].random_(0, 256)
    table, refs = ints([[0, -1], [1, -1]]), ints([1, 1])
    lens = cache.kvq_pages_grow(starts([1, 1]), table, ints([16, 10]), refs)
    # (the second has room in its page, but stands behind the first, which has none)
    assert lens.tolist() == [-17, -11] and table.tolist() == [[0, -1], [1, -1]] and refs.tolist() == [1, 1]
    before = cache.buffer[:per].clone()
    batch = kvq.PagesBatch(starts([1, 1]), lens, table, 2, 1)
    x = torch.randn((2, 2, 64), device="cuda").half()
    fill_ = torch.full_like(x, 7.0)
    tree = cache.kvq_pages_tree(ints([-1, -1]), batch)
    for i in range(2):
        cache.kvq_pages_append(i, x, x, batch)
        cache.kvq_pages_tree_attn(i, x, batch, tree)  # (values of no meaning)
        cache.kvq_pages_cross_attn(i, x, batch)
        ko, vo = cache.kvq_pages_read(i, batch, fill_.clone(), fill_.clone())
        assert (ko == 7).all() and (vo == 7).all()
    kept_lens = cache.kvq_pages_keep(torch.ones(2, dtype=torch.bool, device="cuda"), batch)
    assert cache.kvq_pages_status() == 8 and cache.kvq_pages_status() == 0
    assert not tree.seen.any() and not tree.positions.any()
    assert kept_lens.tolist() == [-17, -11]
    assert torch.equal(cache.buffer[:per], before)
    # the first gives its page back, the second grows into its own
    table, lens, refs = cache.kvq_pages_fork(ints([-1, 1]), table, lens, refs)
    again = ints([0, -1 - int(lens[1])])
    assert cache.kvq_pages_grow(starts([0, 1]), table, again, refs).tolist() == [0, 11]
    assert cache.kvq_pages_status() == 0 and refs.tolist() == [0, 1]


@gpu
def test_tree_and_cross_in_two_graphs_that_take_turns():
    """Two captured attention calls of one cache share its workspace; replayed in turn on one stream, each
    gives what it gives alone."""
    c = make(([9, 40, 1], [900, 300, 2500]), 32, "bf16", (8, 2), 64, seed=11)
    fill(c, 2, 64)
    q = c.normal(c.rows, 8, 64).to(c.dtype).cuda()
    batch = c.batch()
    tree = c.cache.kvq_pages_tree(ints(sum([drafted(n, c.g) for n in c.news], [])), batch)
    outs = [torch.zeros_like(q) for _ in range(2)]
    calls = [lambda: c.cache.kvq_pages_tree_attn(0, q, batch, tree, out=outs[0]),
             lambda: c.cache.kvq_pages_cross_attn(0, q, batch, out=outs[1])]
    want = [call().clone() for call in calls]
    graphs = []
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for turn in range(6):
        outs[turn % 2].zero_()
        graphs[turn % 2].replay()
        graphs[1 - turn % 2].replay()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@gpu
def test_fork_of_bad_rows():
    cache = kvq.KVQPages(kvq.make_pages_config(1, 8, 16, 1, 1, 64))
    table = ints([[0, 1, 2], [3, 99, -1]])
    refs = ints([1, 1, 1, 1, 0, 0, 0, 0])
    t, n, r = cache.kvq_pages_fork(ints([0, 2, -7, 1, 0]), table, ints([40, 32]), refs)
    assert cache.kvq_pages_status() == 7
    assert t.tolist() == [[0, 1, 2], [-1] * 3, [-1] * 3, [3, -1, -1], [0, 1, 2]]
    assert n.tolist() == [40, 0, 0, 32, 40] and r.tolist() == [2, 2, 2, 1, 0, 0, 0, 0]
    narrow = torch.empty((1, 2), dtype=torch.int32, device="cuda")
    t, n, r = cache.kvq_pages_fork(ints([0]), table[:1], ints([40]), refs, table_out=narrow)
    assert cache.kvq_pages_status() == 7 and t.tolist() == [[-1, -1]] and n.tolist() == [0] and r.tolist()[:3] == [0, 0, 0]
    t, n, r = cache.kvq_pages_fork(ints([0, 0]), table[:1], ints([20]), refs, table_out=torch.empty((2, 2), dtype=torch.int32, device="cuda"))
    assert t.tolist() == [[0, 1], [0, 1]] and r.tolist()[:3] == [2, 2, 0] and cache.kvq_pages_status() == 0


# ------------------------------------------------------------------ together --

class Life:
    """Two samples of one prompt that draft, verify and keep."""

    def __init__(self, fmt, d=64, heads=(4, 2), pt=16, prompt=37):
        k, v, dtype = FORMATS[fmt]
        self.heads, self.d, self.pt = heads, d, pt
        self.cache = kvq.KVQPages(kvq.make_pages_config(2, 40, pt, *heads, d, k, v, dtype))
        self.type = torch.bfloat16 if dtype == kvq.BF16 else torch.float16
        self.g = torch.Generator().manual_seed(1)
        self.tab = angles(200, d).cuda()
        self.table, self.lens, self.refs = torch.full((2, 12), -1, dtype=torch.int32, device="cuda"), ints([0, 0]), ints([0] * 40)
        self.held = [[], []]  # tokens of each sample: (position, keys, values) a layer

    def rows(self, n):
        return [tuple(torch.randn((n, h, self.d), generator=self.g).to(self.type).cuda() for h in (self.heads[0], self.heads[1], self.heads[1]))
                for _ in range(2)]


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_run_of_the_operators_together(fmt):
    """A prompt, forked into two samples; each step drafts a tree a sample, attends, keeps one branch.
    What the caches hold and the attention over it are those of a cache that was given the kept
    tokens alone, at their positions."""
    s = Life(fmt)
    cache, n0 = s.cache, 37
    q_start = starts([n0, 0])
    s.lens = cache.kvq_pages_grow(q_start, s.table, s.lens, s.refs)
    rope = lambda pos: kvq.Rope(s.tab, HALVES, pos)  # noqa: E731
    told = [[], []]  # (keys, values) a layer, of each sample's tokens, as appended
    prompt = s.rows(n0)
    batch = kvq.PagesBatch(q_start, s.lens, s.table, n0)
    for i, (q, k, v) in enumerate(prompt):
        cache.kvq_pages_append(i, k, v, batch, rope=rope(torch.arange(n0, dtype=torch.int32, device="cuda")))
    told[0] = [[(j, [(k[j], v[j]) for _, k, v in prompt]) for j in range(n0)]][0]
    s.table, s.lens, s.refs = cache.kvq_pages_fork(ints([0, 0]), s.table, s.lens, s.refs)
    told[1] = list(told[0])
    for step, news in enumerate([[7, 5], [3, 9], [1, 12]]):
        q_start = starts(news)
        rows = sum(news)
        s.lens = cache.kvq_pages_grow(q_start, s.table, s.lens, s.refs)
        batch = kvq.PagesBatch(q_start, s.lens, s.table, rows, max(news))
        parents = [drafted(n, s.g, roots=0.0) for n in news]
        tree = cache.kvq_pages_tree(ints(sum(parents, [])), batch)
        new = s.rows(rows)
        outs = []
        for i, (q, k, v) in enumerate(new):
            cache.kvq_pages_append(i, k, v, batch, rope=rope(tree.positions))
            outs.append(cache.kvq_pages_tree_attn(i, q, batch, tree))
        # the branch of a random token is kept
        keep, at = torch.zeros(rows, dtype=torch.bool), 0
        for b, n in enumerate(news):
            leaf = int(torch.randint(0, n, (), generator=s.g))
            path = ancestors(parents[b])[leaf].nonzero()[:, 0].tolist()
            base = len(told[b])
            # a plain cache that holds the kept tokens alone sees them alike
            for depth, j in enumerate(path):
                told[b].append((base + depth, [(k[at + j], v[at + j]) for _, k, v in new]))
                keep[at + j] = True
            plain = kvq.KVQPages(s.cache.cfg)
            count = len(told[b])
            one = kvq.PagesBatch(ints([0, count]), ints([count]), torch.arange(12, dtype=torch.int32, device="cuda")[None], count)
            last = kvq.PagesBatch(ints([0, 1]), ints([count]), one.table, 1, 1)
            for i in range(2):
                plain.kvq_pages_append(i, *(torch.stack([t[1][i][x] for t in told[b]]) for x in (0, 1)), one,
                                       rope=rope(ints([t[0] for t in told[b]])))
                got, want = outs[i][at + leaf].float(), plain.kvq_pages_attn(i, new[i][0][at + leaf:at + leaf + 1], last)[0].float()
                # (both are within a weight's and an output's rounding of the same value, values are below 6)
                assert (got - want).abs().max() <= 6 * 4 * HALF_STEP[s.type]
            told_k = [plain.kvq_pages_read(i, one) for i in range(2)]
            if b == 0:
                first = told_k
            at += n
        s.lens = cache.kvq_pages_keep(keep.cuda(), batch)
        assert s.lens.tolist() == [len(t) for t in told] and cache.kvq_pages_status() == 0
        whole = kvq.PagesBatch(starts(s.lens.tolist()), s.lens, s.table, int(s.lens.sum()))
        for i in range(2):
            for x in (0, 1):
                assert torch.equal(cache.kvq_pages_read(i, whole)[x], torch.cat([first[i][x], told_k[i][x]]))
        # pages behind the end go back
        s.table, s.lens, s.refs = cache.kvq_pages_fork(ints([0, 1]), s.table, s.lens, s.refs)
        assert int((s.table >= 0).sum()) == sum(-(-len(t) // s.pt) for t in told) == int(s.refs.sum())
    assert cache.kvq_pages_status() == 0


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "4_4"])
def test_a_captured_step_with_other_trees_and_lengths(fmt):
    """Tree, append, attention and keep captured once; replayed for other trees, lengths, pages and marks."""
    layers = 2
    news, a, b = [9, 4], [120, 33], [64, 300]
    cs = [make((news, lens), 16, fmt, (4, 2), 64, layers=layers, seed=i) for i, lens in enumerate((a, b))]
    pages = max(c.pages for c in cs)
    k, v, dtype = FORMATS[fmt]
    cache = kvq.KVQPages(kvq.make_pages_config(layers, pages, 16, 4, 2, 64, k, v, dtype))
    width = max(c.table.shape[1] for c in cs)
    n = sum(news)
    lens, table, q_start = ints([0, 0]), ints([[0] * width] * 2), starts(news)
    parents, keep = ints([-1] * n), torch.zeros(n, dtype=torch.bool, device="cuda")
    batch = kvq.PagesBatch(q_start, lens, table, n, max(news))
    q, kk, vv = (torch.zeros((n, h, 64), dtype=cs[0].dtype, device="cuda") for h in (4, 2, 2))
    tree = kvq.PagesTree(torch.zeros((n, 1), dtype=torch.int64, device="cuda"), ints([0] * n))
    outs, new = [torch.zeros_like(q) for _ in range(layers)], ints([0, 0])

    def step():
        cache.kvq_pages_tree(parents, batch, tree=tree)
        for i in range(layers):
            cache.kvq_pages_append(i, kk, vv, batch)
            cache.kvq_pages_tree_attn(i, q, batch, tree, out=outs[i])
        cache.kvq_pages_keep(keep, batch, lens_out=new)

    lens.copy_(ints(a))
    table[:, :cs[0].table.shape[1]].copy_(cs[0].table.clamp_min(0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for c, ln in zip(cs, (a, b)):
        full = torch.full((2, width), -1, dtype=torch.int32)
        full[:, :c.table.shape[1]] = c.table
        c.table = full
        c.cache.close()
        c.cache = cache
        cache.buffer.zero_()
        for i in range(layers):
            fill(c, 2, 64, layer=i)
        for trial in range(2):
            ps = [drafted(m, c.g) for m in news]
            lens.copy_(ints(ln))
            table.copy_(full.cuda())
            parents.copy_(ints(sum(ps, [])))
            keep.copy_(torch.rand(n, generator=c.g) < 0.5)
            for x in (q, kk, vv):
                x.copy_(c.normal(*x.shape))
            graph.replay()
            assert cache.kvq_pages_status() == 0
            got = [o.clone() for o in outs]
            kept_lens, after = new.tolist(), layers_of(c, layers)
            # the same by calls
            for i in range(layers):
                cache.kvq_pages_append(i, kk, vv, batch)
            whole = layers_of(c, layers)
            masks = [ancestors(p) for p in ps]
            s = c.k_start.tolist()
            for i in range(layers):
                data = [tuple(x[s[j]:s[j + 1]] for x in whole[i]) for j in range(2)]
                check(c, q.cpu(), got[i].cpu(), data, tree_sees(c, masks, [None] * 2, 0))
                want, want_lens = kept(c, keep.tolist(), whole[i])
                assert kept_lens == want_lens
                assert all(torch.equal(x, y) for x, y in zip(after[i], want))


@gpu
def test_a_captured_fork_and_growth():
    """Fork and grow captured once over two tables that take turns."""
    pool = Pool(200, 16, 5, 20)
    cache = kvq.KVQPages(kvq.make_pages_config(1, 200, 16, 1, 1, 64))
    (table, lens, refs), q_start, parent = pool.tensors(), ints([0] * 6), ints([0] * 5)
    table2, lens2 = torch.empty_like(table), torch.empty_like(lens)
    graphs = []
    for t, n, t2, n2 in ((table, lens, table2, lens2), (table2, lens2, table, lens)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.kvq_pages_fork(parent, t, n, refs, table_out=t2, lens_out=n2, refs_out=refs)
            cache.kvq_pages_grow(q_start, t2, n2, refs, lens_out=n2)
        graphs.append((g, t2, n2))
    r = np.random.RandomState(0)
    for step in range(8):
        ps, news = r.randint(-1, 5, 5).tolist(), r.randint(0, 40, 5).tolist()
        parent.copy_(ints(ps))
        q_start.copy_(starts(news))
        g, t2, n2 = graphs[step % 2]
        g.replay()
        pool.fork(ps)
        pool.grow(news)
        pool.same(t2, n2, refs)
        pool.sound()


@gpu
def test_on_a_stream_of_the_users():
    """All calls on a side stream, with the tensors that they make there."""
    c = make(([5, 9], [40, 60]), 16, "bf16", (4, 2), 64, seed=2)
    data = fill(c, 2, 64)
    q = c.normal(c.rows, 4, 64).to(c.dtype)
    dev, parents = q.cuda(), [drafted(n, c.g) for n in c.news]
    flat, batch, keep = ints(sum(parents, [])), c.batch(), (torch.arange(c.rows) % 2 == 0).cuda()
    refs = ints([0] * c.pages)
    refs[c.table[c.table >= 0].long().cuda()] = 1
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tree = c.cache.kvq_pages_tree(flat, batch, stream=side)
    out = c.cache.kvq_pages_tree_attn(0, dev, batch, tree, stream=side)
    cross = c.cache.kvq_pages_cross_attn(0, dev, batch, stream=side)
    lens = c.cache.kvq_pages_keep(keep, batch, stream=side)
    table, lens2, refs2 = c.cache.kvq_pages_fork(ints([1, 0, 1]), batch.table, lens, refs, stream=side)
    side.synchronize()
    masks = [ancestors(p) for p in parents]
    check(c, q, out.cpu(), data, tree_sees(c, masks, [None] * 2, 0))
    check(c, q, cross.cpu(), data, [torch.ones((n, ln), dtype=torch.bool) for n, ln in zip(c.news, c.lens)])
    assert lens.tolist() == [38, 55] and lens2.tolist() == [55, 38, 55]
    assert c.cache.kvq_pages_status(stream=side) == 0


@gpu
def test_far_offsets():
    """Pages whose bytes lie beyond 32 bits, in a layer of its own."""
    cfg = kvq.make_pages_config(2, 20000, 64, 8, 8, 128, dtype=kvq.BF16)  # 2 x 5.2 GB
    if torch.cuda.mem_get_info()[0] < 2 * kvq.kvq_pages_bytes(cfg).alloc:
        pytest.skip("not enough memory")
    cache = kvq.KVQPages(cfg)
    g = torch.Generator().manual_seed(0)
    table = torch.tensor([[19999, 3, 19990]], dtype=torch.int32, device="cuda")
    n = 150
    batch = kvq.PagesBatch(ints([0, n]), ints([n]), table, n)
    rows = [[torch.randn((n, 8, 128), generator=g).bfloat16() for _ in range(2)] for _ in range(2)]
    for i in range(2):
        cache.kvq_pages_append(i, rows[i][0].cuda(), rows[i][1].cuda(), batch)
    cache.kvq_pages_copy(ints([19999, 19990]), ints([19998, 5]))
    keep = torch.rand(n, generator=g) < 0.5
    lens = cache.kvq_pages_keep(keep.cuda(), batch)
    m = int(keep.sum())
    assert lens.tolist() == [m]
    kept_batch = kvq.PagesBatch(ints([0, m]), lens, table, m)
    for i in range(2):
        for x, y in zip(cache.kvq_pages_read(i, kept_batch), rows[i]):
            assert torch.equal(x.cpu(), y[keep])
    copies = kvq.PagesBatch(ints([0, 86]), ints([86]), ints([[19998, 5]]), 86)
    for i in range(2):
        for x, y in zip(cache.kvq_pages_read(i, copies), rows[i]):
            assert torch.equal(x[:64].cpu(), y[:64]) and torch.equal(x[64:].cpu(), y[128:])
    q = torch.randn((3, 8, 128), generator=g).bfloat16()
    cross = kvq.PagesBatch(ints([0, 3]), lens, table, 3)
    got = cache.kvq_pages_cross_attn(1, q.cuda(), cross).cpu()
    ref, tol = attention_of(q, rows[1][0][keep], rows[1][1][keep], torch.ones((3, m), dtype=torch.bool), 128 ** -0.5,
                            HALF_STEP[torch.bfloat16])
    assert ((got.double() - ref).abs() <= tol + ref.abs() * HALF_STEP[torch.bfloat16] + 2.0 ** -25).all()
    assert cache.kvq_pages_status() == 0
