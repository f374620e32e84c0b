"""Branching sequences on the paged cache where tables, lengths and arguments are not as they should be."""
import ctypes
import os

import pytest
import torch

from bit_quantized_kv_02_gb300 import build, kvq
from tests.test_pages import fill, make
from tests.test_pages_branch import ints, kept, layers_of, starts

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(kvq.LIB_PATH):
        build.build()
    return kvq.lib()


def said(cache):
    return cache._lib.kvq_pages_last_error(cache.handle).decode()


# ---------------------------------------------------------------------- grow --

@gpu
@pytest.mark.parametrize("bad_first", [True, False])
@pytest.mark.parametrize("entry", [8, 99, 2 ** 31 - 1])
def test_grow_leaves_a_sequence_that_needs_an_entry_outside_the_pool(entry, bad_first):
    """Such a sequence stays as it was, table and length, wherever among the needed entries the bad one stands; the
    others grow, and one that shares its last page copies it, as the sequence that stayed still holds it."""
    cache = kvq.KVQPages(kvq.make_pages_config(2, 8, 16, 1, 1, 64))
    per = int(cache.bytes.packed) // 2
    cache.buffer[:2 * per].copy_(torch.randint(0, 256, (2 * per,), generator=torch.Generator().manual_seed(0)).to(torch.uint8))
    pages = cache.buffer[:2 * per].clone().view(2, 8, -1)
    rows = [([2, entry, -1], 5, 15),   # shares page 2; needs entries 0 and 1
            ([2, -1, -1], 5, 3),       # grows into page 2
            ([4, -1, entry], 16, 20),  # a free page, then the bad entry
            ([5, entry, -1], 16, 0),   # needs nothing
            ([6, -1, entry], 10, 10)]  # the bad entry stands behind what it needs
    if not bad_first:
        rows[0], rows[1] = rows[1], rows[0]
    table, lens, refs = ints([r[0] for r in rows]), ints([r[1] for r in rows]), ints([0, 0, 2, 0, 1, 1, 1, 0])
    out = cache.kvq_pages_grow(starts([r[2] for r in rows]), table, lens, refs)
    assert cache.kvq_pages_status() == 7
    want = [list(r[0]) for r in rows]
    grown = 1 if bad_first else 0
    want[grown][0], want[4][1] = 0, 1
    assert table.tolist() == want
    assert out.tolist() == [-6 if b != grown else 8 for b in range(2)] + [-17, 16, 20]
    assert refs.tolist() == [1, 1, 1, 0, 1, 1, 1, 0]
    pages[:, 0] = pages[:, 2]
    assert torch.equal(cache.buffer[:2 * per].view(2, 8, -1), pages)
    assert cache.kvq_pages_status() == 0


@gpu
def test_grow_without_pages_changes_no_entry():
    """Sequences that find no page keep their tables: any negative entry is none and stays what it was, shared pages
    and pages behind the tokens included."""
    cache = kvq.KVQPages(kvq.make_pages_config(1, 4, 16, 1, 1, 64))
    before = [[0, -5, -1], [1, 2, -7], [1, 2, -2147483648], [3, -3, -4]]
    table, refs = ints(before), ints([1, 2, 2, 1])
    lens = ints([16, 20, 12, 16])
    out = cache.kvq_pages_grow(starts([1, 20, 9, 0]), table, lens, refs)
    assert cache.kvq_pages_status() == 8
    assert out.tolist() == [-17, -21, -13, 16]
    assert table.tolist() == before and refs.tolist() == [1, 2, 2, 1]
    # with pages, the same entries are taken as none
    table, refs = ints([[0, -5, -1], [1, -7, -2147483648]]), ints([1, 1, 0, 0])
    out = cache.kvq_pages_grow(starts([3, 16]), table, ints([16, 8]), refs)
    assert cache.kvq_pages_status() == 0 and out.tolist() == [19, 24]
    assert table.tolist() == [[0, 2, -1], [1, 3, -2147483648]] and refs.tolist() == [1, 1, 1, 1]


# -------------------------------------------------------------------- status --

@gpu
def test_a_bad_page_is_reported_in_a_step_that_runs_out_of_pages():
    """Lengths tell that pages ran out; that a page was wrong shows in the status alone, so it comes first.  The
    lengths that such a growth leaves are no fault of their own beside it."""
    cache = kvq.KVQPages(kvq.make_pages_config(1, 2, 16, 2, 2, 64))
    x = torch.randn((2, 2, 64), device="cuda").half()

    def step(second_page):
        lens = cache.kvq_pages_grow(starts([1, 1]), ints([[0, -1], [1, -1]]), ints([16, 10]), ints([1, 1]))
        assert lens.tolist() == [-17, -11]
        cache.kvq_pages_append(0, x, x, kvq.PagesBatch(starts([1, 1]), lens, ints([[0, -1], [1, -1]]), 2, 1))
        cache.kvq_pages_append(0, x, x, kvq.PagesBatch(starts([1, 1]), ints([1, 1]), ints([[0], [second_page]]), 2, 1))

    step(1)
    assert cache.kvq_pages_status() == 8 and "free pages" in said(cache) and "range" not in said(cache)
    assert cache.kvq_pages_status() == 0
    step(9)
    assert cache.kvq_pages_status() == 7 and "range" in said(cache) and "free pages" in said(cache)
    assert cache.kvq_pages_status() == 0
    # a negative length alone is an index out of range
    batch = kvq.PagesBatch(starts([1, 1]), ints([-17, 1]), ints([[0], [1]]), 2, 1)
    tree = kvq.PagesTree(torch.ones((2, 1), dtype=torch.int64, device="cuda"), ints([0, 0]))
    for call in (lambda: cache.kvq_pages_append(0, x, x, batch), lambda: cache.kvq_pages_read(0, batch),
                 lambda: cache.kvq_pages_attn(0, x, batch), lambda: cache.kvq_pages_cross_attn(0, x, batch),
                 lambda: cache.kvq_pages_tree_attn(0, x, batch, tree),
                 lambda: cache.kvq_pages_tree(ints([-1, -1]), batch),
                 lambda: cache.kvq_pages_keep(torch.ones(2, dtype=torch.bool, device="cuda"), batch)):
        call()
        assert cache.kvq_pages_status() == 7 and "free pages" not in said(cache)


# ---------------------------------------------------------------------- keep --

KEPT = pytest.mark.parametrize("fmt,h,d", [("bf16", 3, 64), ("4_8", 2, 256), ("8_4", 5, 128)])


@gpu
@KEPT
@pytest.mark.parametrize("share", [0.1, 0.6, 0.99])
def test_keep_of_long_sequences_that_begin_before_their_first_token(fmt, h, d, share):
    """Rows with negative positions are no tokens, marked or not; segments are counted behind them."""
    c = make(([600, 5, 300, 2, 1000], [450, 5, 20, 0, 1000]), 32, fmt, (h, h), d, layers=2, seed=6, pad=3)
    for i in range(2):
        fill(c, h, d, layer=i)
    for layer in (kvq.ALL_LAYERS, 1):
        keep = torch.rand(c.rows, generator=c.g) < share
        before = layers_of(c, 2)
        lens = c.cache.kvq_pages_keep(keep.cuda(), c.batch(), layer=layer)
        assert c.cache.kvq_pages_status() == 0
        for i, (x, y) in enumerate(zip(layers_of(c, 2), before)):
            want, new = kept(c, keep.tolist(), y) if layer in (kvq.ALL_LAYERS, i) else (y, None)
            assert all(torch.equal(a, b) for a, b in zip(x, want))
        assert lens.tolist() == kept(c, keep.tolist(), before[0])[1]


@gpu
@KEPT
def test_keep_of_long_sequences_with_bad_pages_and_lengths(fmt, h, d):
    """A row that would leave or enter a page outside the pool stays, a sequence whose length does not fit is left
    alone; what stands before and behind them is right."""
    news, lens, pt = [700, 400, 1000, 900], [700, 400, 1000, 1300], 64
    c = make((news, lens), pt, fmt, (h, h), d, layers=1, seed=9)
    fill(c, h, d)
    before = layers_of(c, 1)[0]
    keep = torch.rand(c.rows, generator=c.g) < 0.7
    bad = {(0, 4), (0, 10), (2, 7), (3, 12)}  # (sequence, entry of its table)
    table = c.table.clone()
    for k, (b, e) in enumerate(sorted(bad)):
        table[b, e] = c.pages + 5 if k % 2 else -3
    told = [700, 1 << 20, 1000, 1300]
    got = c.cache.kvq_pages_keep(keep.cuda(), kvq.PagesBatch(c.q_start.cuda(), ints(told), table.cuda(), c.rows))
    assert c.cache.kvq_pages_status() == 7
    after = layers_of(c, 1)[0]
    row = at = 0
    for b, (n, ln) in enumerate(zip(news, lens)):
        first, to = ln - n, ln - n
        want = [x[at:at + ln].clone() for x in before]
        for i in range(n if b != 1 else 0):
            if not keep[row + i]:
                continue
            if (b, to // pt) not in bad and (b, (first + i) // pt) not in bad:
                for w, x in zip(want, before):
                    w[to] = x[at + first + i]
            to += 1
        assert got[b] == (told[1] if b == 1 else to)
        for w, x in zip(want, after):
            assert torch.equal(x[at:at + ln], w), b
        row += n
        at += ln


# ----------------------------------------------------- outputs over what is read --

class Room:
    """Arrays of a batch of two sequences with 70 new tokens in all, each in a kilobyte of its own."""

    def __init__(self):
        self.cache = kvq.KVQPages(kvq.make_pages_config(1, 8, 16, 4, 2, 64))
        self.memory = torch.zeros(64 << 10, dtype=torch.uint8, device="cuda")
        self.q_start, self.lens, self.table = (self.memory.data_ptr() + 1024 * i for i in range(1, 4))
        self.batch = kvq._PagesBatch(2, 70, 0, self.q_start, self.lens, self.table, 5)
        self.ref = ctypes.byref(self.batch)
        # (all lengths and sequences are empty: a call that is not refused has nothing to do)

    def at(self, kilobyte):
        return self.memory.data_ptr() + 1024 * kilobyte

    def over_the_batch(self, size, align=4):
        """Addresses of an array of `size` bytes that meets one of the batch's at its end or its beginning."""
        for a, n in ((self.q_start, 3), (self.lens, 2), (self.table, 10)):
            yield from (a + 4 * (n - 1) & -align, a - size + 4 + align - 1 & -align)


@gpu
def test_keep_refuses_lengths_over_the_marks(L):
    r = Room()
    for marks in (r.at(8), r.at(8) + 3):
        for lens_out in range(r.at(8) - 16, r.at(8) + 96, 4):
            meets = lens_out < marks + 70 and marks < lens_out + 8
            assert L.kvq_pages_keep(r.cache.handle, 0, r.ref, marks, lens_out, None) == int(meets), lens_out - marks
    assert L.kvq_pages_keep(r.cache.handle, 0, r.ref, r.at(8), None, None) == 0
    for lens_out in r.over_the_batch(8):
        assert L.kvq_pages_keep(r.cache.handle, 0, r.ref, r.at(8), lens_out, None) == 1
    assert r.cache.kvq_pages_status() == 0


@gpu
@pytest.mark.parametrize("words", [1, 3])
def test_tree_refuses_outputs_over_each_other_and_over_what_it_reads(L, words):
    r = Room()
    masks = 70 * 8 * words

    def tree(parents=r.at(8), seen=r.at(16), positions=r.at(24)):
        return L.kvq_pages_tree(r.cache.handle, r.ref, parents, words, seen, positions, None)

    assert tree() == 0 and tree(positions=None) == 0
    # parents end where the masks begin, the positions where parents do, and so on
    assert tree(parents=r.at(16) - 280) == 0 and tree(parents=r.at(16) + masks) == 0
    assert tree(positions=r.at(8) - 280) == 0 and tree(positions=r.at(8) + 280) == 0
    assert tree(positions=r.at(16) - 280) == 0 and tree(positions=r.at(16) + masks) == 0
    # one integer further
    assert tree(parents=r.at(16) - 276) == 1 and tree(parents=r.at(16) + masks - 4) == 1
    assert tree(positions=r.at(8)) == 1 and tree(positions=r.at(8) - 276) == 1 and tree(positions=r.at(8) + 276) == 1
    assert tree(positions=r.at(16) - 276) == 1 and tree(positions=r.at(16) + masks - 4) == 1
    assert tree(seen=r.at(8)) == 1 and tree(seen=r.at(8), positions=None) == 1
    for a in r.over_the_batch(masks, 8):
        assert tree(seen=a) == 1
    for a in r.over_the_batch(280):
        assert tree(positions=a) == 1
    assert r.cache.kvq_pages_status() == 0


@gpu
def test_attention_refuses_an_output_over_what_it_reads(L):
    r = Room()
    size = 70 * 4 * 64 * 2
    q = torch.zeros((70, 4, 64), dtype=torch.float16, device="cuda")
    free = r.at(12)
    assert size == 35 << 10

    def calls(out, seen=r.at(5), words=2, positions=r.at(8)):
        tree = ctypes.byref(kvq._Tree(seen, words, positions))
        return (L.kvq_pages_tree_attn(r.cache.handle, 0, q.data_ptr(), 0, 256, r.ref, tree, 0.0, 0, out, None),
                L.kvq_pages_attn(r.cache.handle, 0, q.data_ptr(), 0, 256, r.ref, 0.0, 0, out, None),
                L.kvq_pages_cross_attn(r.cache.handle, 0, q.data_ptr(), 0, 256, r.ref, 0.0, out, None))

    assert calls(free) == (0, 0, 0)
    for out in r.over_the_batch(size, 16):
        assert calls(out) == (1, 1, 1)
    # masks and positions that end where the output begins and begin where it ends, and ones that meet it
    assert calls(free, seen=free - 1120) == calls(free, positions=free - 280) == (0, 0, 0)
    assert calls(free, seen=free + size) == calls(free, positions=free + size) == (0, 0, 0)
    for kw in (dict(seen=free - 1112), dict(seen=free + size - 8), dict(positions=free - 276), dict(positions=free + size - 4)):
        assert calls(free, **kw) == (1, 0, 0), kw
    assert calls(free, positions=None) == (0, 0, 0)
    assert r.cache.kvq_pages_status() == 0
