"""Paged attention and append where a call's surroundings must not matter: the hint,
the other sequences of the batch, the magnitude of the queries."""
import math

import pytest
import torch

from bit_quantized_kv_02_gb300 import kvq
from tests.pages_ref import HALF_STEP, attention
from tests.test_pages import L, check_attention, fill, make  # noqa: F401  (L builds the library)

gpu = pytest.mark.gpu


# ----------------------------------------------------- rounding of the weights --

# (new tokens, lengths, rows behind them, hint): sequences of up to 16 query rows
# alone with the hint, without it, beside a prompt, and in a padded batch of one
SURROUNDINGS = {
    "hint": ([1, 1, 4, 1], [5, 33, 12, 1500], 0, 4),
    "no_hint": ([1] * 36 + [4], [3 + 2 * i for i in range(36)] + [700], 0, 0),
    "prompt": ([1, 4, 90, 1], [6, 40, 200, 1500], 0, 90),
    "padded": ([1], [9], 70, 0),
}


def cancelling_values(c, q, k, hq, h):
    """Values whose last visible one cancels the others in the first query head of
    each group: the output is then far below the terms it is made of, and an error of
    the weights shows beside the output's own rounding."""
    s, t = c.q_start.tolist(), c.k_start.tolist()
    v = c.normal(int(c.k_start[-1]), h, k.shape[2]).to(c.dtype)
    for b, n in enumerate(c.news):
        for j in range(h):
            x = q[s[b + 1] - 1, j * (hq // h)].double()
            p = torch.softmax(k[t[b]:t[b + 1], j].double() @ x / math.sqrt(k.shape[2]), dim=0)
            vb = v[t[b]:t[b + 1], j].double()
            v[t[b + 1] - 1, j] = (-(p[:-1] @ vb[:-1]) / p[-1]).to(c.dtype)
    return v


@gpu
@pytest.mark.parametrize("name", SURROUNDINGS)
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("d,heads", [(64, (4, 4)), (128, (8, 2)), (256, (4, 1))])
def test_weights_of_few_rows_keep_their_remainder(name, fmt, d, heads):
    """Up to 16 query rows over 16-bit pages: weights enter as operand and remainder,
    so their error is the square of the operand's half step, whatever else the batch
    holds and whether the hint is given."""
    news, lens, pad, hint = SURROUNDINGS[name]
    c = make((news, lens), 32, fmt, heads, d, seed=13, pad=pad)
    hq, h = heads
    q = (c.normal(c.rows, hq, d) * 0.3).to(c.dtype)
    k = (c.normal(int(c.k_start[-1]), h, d) * 0.3).to(c.dtype)
    v = cancelling_values(c, q, k, hq, h)
    c.cache.kvq_pages_append(0, k.cuda(), v.cuda(), c.whole())
    got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(hint)).cpu()
    assert c.cache.kvq_pages_status() == 0
    s, t = c.q_start.tolist(), c.k_start.tolist()
    for b, n in enumerate(news):
        few = n * (hq // h) <= 16
        step = HALF_STEP[c.dtype]
        ref, tol = attention(q[s[b]:s[b + 1]], k[t[b]:t[b + 1]], v[t[b]:t[b + 1]], torch.arange(lens[b] - n, lens[b]), 0,
                             1.0 / math.sqrt(d), step * step if few else step)
        tol = tol + ref.abs() * step + 2.0 ** -25
        off = (got[s[b]:s[b + 1]].double() - ref).abs()
        assert (off <= tol).all(), (b, float((off / tol).max()))


# ------------------------------------------------------- magnitude of the queries --

@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", ["8_8", "4_4", "4_8"])
@pytest.mark.parametrize("power", [-90, -112, -120, -130])
def test_smallest_queries_over_codes(which, fmt, power):
    """bf16 queries near the bottom of their range over codes, under a scale that
    brings the scores back: they count with all their bits."""
    c = make(([3, 40, 1], [90, 40, 700]), 16, fmt, (4, 2), 64, seed=2)
    data = fill(c, 2, 64)
    c.cache.kvq_pages_set_kernel(which)
    q = (c.normal(c.rows, 4, 64).double() * 2.0 ** power).to(torch.bfloat16)
    scale = 2.0 ** (min(-power, 126) - 3)
    got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(), scale=scale)
    check_attention(c, q, got.cpu(), data, scale=scale)


# ------------------------------------------------------------- reuse of the stages --

@gpu
@pytest.mark.parametrize("which", [1, 2], ids=["few", "many"])
@pytest.mark.parametrize("fmt", ["f16", "8_8", "4_4", "8_4", "4_8"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_copies_do_not_overtake_the_reads_before_them(which, fmt, d):
    """Long sequences that refill every stage many times, over and over: a copy that
    lands under a read shows as a run that differs."""
    c = make(([20, 30], [3000, 4100]), 32, fmt, (8, 2), d, seed=3)
    data = fill(c, 2, d)
    q = c.normal(c.rows, 8, d).to(c.dtype)
    c.cache.kvq_pages_set_kernel(which)
    dev, b = q.cuda(), c.batch()
    first = c.cache.kvq_pages_attn(0, dev, b).clone()
    check_attention(c, q, first.cpu(), data)
    out, differ = torch.zeros_like(first), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        c.cache.kvq_pages_attn(0, dev, b, out=out)
        differ += (out != first).sum()
    assert int(differ) == 0 and c.cache.kvq_pages_status() == 0


# ---------------------------------------------------------------- rows named twice --

@gpu
@pytest.mark.parametrize("fmt", ["f16", "8_8"])
def test_a_row_that_two_sequences_name(fmt):
    """q_start falls back at the second sequence, so the first and the third both name
    row 2: it goes with the first, the second is skipped, and no other token changes."""
    c = make(([3, 0, 1], [40, 20, 30]), 16, fmt, (2, 2), 64, seed=1)
    data = fill(c, 2, 64)
    batch = kvq.PagesBatch(torch.tensor([0, 3, 2, 4], dtype=torch.int32).cuda(),
                           torch.tensor(c.lens, dtype=torch.int32).cuda(), c.table.cuda(), 4)
    x = c.normal(4, 2, 64).half().cuda()
    # what the pages hold of the four rows
    alone = make(([4], [4]), 16, fmt, (2, 2), 64)
    alone.cache.kvq_pages_append(0, x, x, alone.batch())
    rows = [t.cpu() for t in alone.cache.kvq_pages_read(0, alone.batch())]
    for _ in range(200):
        c.cache.kvq_pages_append(0, x, x, batch)
    assert c.cache.kvq_pages_status() == 7
    s = c.k_start.tolist()
    for i, got in enumerate(t.cpu() for t in c.cache.kvq_pages_read(0, c.whole())):
        want = torch.cat([d[i] for d in data])
        want[s[0] + 37:s[0] + 40] = rows[i][:3]
        want[s[2] + 29] = rows[i][3]
        assert torch.equal(got, want)
    out = torch.full((4, 2, 64), 3.0, dtype=torch.float16, device="cuda")
    got, _ = c.cache.kvq_pages_read(0, batch, out, out.clone())
    assert c.cache.kvq_pages_status() == 7 and torch.equal(got.cpu(), rows[0])


# ------------------------------------------------------------------ memory of calls --

@gpu
def test_pool_belongs_to_the_stream_that_clears_it():
    """The buffer of a cache made on a stream comes from that stream's memory: what the
    current stream still writes to freed memory of its own cannot reach it."""
    cfg = kvq.make_pages_config(1, 500, 32, 4, 4, 64)
    size, stream = kvq.kvq_pages_bytes(cfg).alloc, torch.cuda.Stream()
    with torch.cuda.stream(stream):
        mine = torch.empty(size, dtype=torch.uint8, device="cuda")
    theirs = torch.empty(size, dtype=torch.uint8, device="cuda")
    at, other = mine.data_ptr(), theirs.data_ptr()
    del mine, theirs
    cache = kvq.KVQPages(cfg, stream=stream)
    assert cache.buffer.data_ptr() == at != other
    stream.synchronize()
    assert not cache.buffer.any() and cache.kvq_pages_status(stream) == 0


@gpu
def test_output_over_the_queries_is_refused():
    """Heads are read after others are written; an output beside the queries, or between
    two of their rows, is taken."""
    c = make(([3], [40]), 16, "f16", (4, 2), 64)
    data = fill(c, 2, 64)
    flat = torch.zeros(3 * 256 * 5, dtype=torch.float16, device="cuda")
    q = c.normal(3, 4, 64).half()

    def call(at, stride, out_at):
        dev = flat.as_strided((3, 4, 64), (stride, 64, 1), at)
        dev.copy_(q)
        return c.cache.kvq_pages_attn(0, dev, c.batch(), out=flat[out_at:out_at + 768].view(3, 4, 64))

    for at, stride, out_at in ((0, 256, 0), (0, 256, 760), (768, 256, 8), (0, 512, 512), (0, 1024, 264), (256, 1024, 520)):
        with pytest.raises(kvq.KVQError) as e:
            call(at, stride, out_at)
        assert e.value.status == 1 and "overlap" in str(e.value)
    for at, stride, out_at in ((0, 256, 768), (768, 256, 0), (0, 1024, 256), (256, 1024, 512), (768, 512, 0)):
        check_attention(c, q, call(at, stride, out_at).cpu(), data)


# --------------------------------------------------------- the choice of the kernel --

@gpu
@pytest.mark.parametrize("fmt", ["f16", "bf16", "8_8", "4_4"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hint", [True, False])
def test_rows_around_the_choice_of_the_kernel(fmt, d, hint):
    """Sequences with as many rows as the few-rows kernel takes by default, one fewer and
    one more, alone and in one batch."""
    few = 32 if fmt in ("f16", "bf16") else {64: 128, 128: 64, 256: 48}[d]
    for news in ([few - 1], [few], [few + 1], [few, 1, few + 1, 16, 17, few - 1]):
        c = make((news, [n + 75 for n in news]), 32, fmt, (1, 1), d, seed=17, pad=0 if hint else 40)
        data = fill(c, 1, d)
        q = c.normal(c.rows, 1, d).to(c.dtype)
        got = c.cache.kvq_pages_attn(0, q.cuda(), c.batch(max(news) if hint else 0))
        assert c.cache.kvq_pages_status() == 0 and not got[c.n:].any()
        check_attention(c, q, got.cpu(), data)
