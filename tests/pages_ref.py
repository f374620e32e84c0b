"""Plain 64-bit forms of the paged-cache operators, and bounds on how far a
kernel may be from them."""
import math

import numpy as np
import torch

import oracle
from bit_quantized_kv_02_gb300 import kvq

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
PAIRS, HALVES = kvq.ROPE_PAIRS, kvq.ROPE_HALVES


def angles(rows, dim, base=10000.0):
    """[rows][dim / 2][2] fp32 (cosine, sine) of position * base^(-2i / dim)."""
    f = base ** (-np.arange(0, dim, 2, dtype=np.float64) / dim)
    a = np.arange(rows, dtype=np.float64)[:, None] * f
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], axis=-1).astype(np.float32))


def rotate(x, cs, dim, style):
    """x [n][heads][d], cs [n][dim / 2][2]; in x's precision, an operation at a time."""
    c, s = cs[:, None, :, 0].to(x.dtype), cs[:, None, :, 1].to(x.dtype)
    y = x.clone()
    if style == PAIRS:
        a, b = x[..., 0:dim:2], x[..., 1:dim:2]
        y[..., 0:dim:2], y[..., 1:dim:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :dim // 2], x[..., dim // 2:dim]
        y[..., :dim // 2], y[..., dim // 2:dim] = a * c - b * s, b * c + a * s
    return y


def held(x, bits, group, dtype):
    """What pages hold of x [n][heads][d] (fp32): 16-bit values, or fp16(zero + code
    * step) with the oracle's codes and metadata."""
    if bits == 16:
        return x.to(dtype)
    n, h, d = x.shape
    if n == 0:
        return x.half()
    q = oracle.quantize_tensor(np.ascontiguousarray(x.numpy()[None]), np.array([n], np.int32), (n + 15) // 16 * 16, bits,
                               group, kvq.PER_TOKEN, sym=False)
    codes = q["codes"][0][:, :n].astype(np.float64)  # [h][n][d]
    meta = q["meta"].astype(np.float64).reshape(h, -1, d // group, 2)[:, :n]
    v = meta[..., 0].repeat(group, axis=-1) + codes * meta[..., 1].repeat(group, axis=-1)
    return torch.from_numpy(v.astype(np.float16)).permute(1, 0, 2).contiguous()


def attention(q, k, v, pos, window, scale, p_half_step):
    """One sequence: q [n][hq][d], k / v [t][h][d] (any type), pos [n] positions.
    Returns (out, bound) in 64 bits: the bound counts half a step of the output
    type's rounding elsewhere, and here the weights' rounding (p_half_step each),
    fp32 scores (products summed by the tensor core, at most one step of 2^-23
    of the running magnitude per term), and the fp32 sums over tokens (16 at a
    time, a step of 2^-23 each, and 64 more for the merges of warps and parts)."""
    n, hq, d = q.shape
    t, h = k.shape[0], k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, bound = torch.zeros(n, hq, d, dtype=torch.float64), torch.zeros(n, hq, d, dtype=torch.float64)
    if t == 0 or n == 0:
        return out, bound
    at = torch.arange(t)[None, :]
    see = at <= pos[:, None]
    if window:
        see &= at > pos[:, None] - window
    for j in range(hq):
        kk, vv = k[:, j // (hq // h)], v[:, j // (hq // h)]
        s = (q[:, j] @ kk.T) * scale
        size = (q[:, j].abs() @ kk.abs().T) * scale
        s = s.masked_fill(~see, -math.inf)
        top = s.amax(dim=-1, keepdim=True).clamp_min(-1e300)
        e = torch.exp(s - top)
        tot = e.sum(dim=-1, keepdim=True)
        p = torch.where(tot > 0, e / tot, torch.zeros_like(e))
        out[:, j] = p @ vv
        # a score off by x moves its weight by a factor e^x; the sum moves by as much again
        off = 2.0 * (size * see).amax(dim=-1, keepdim=True) * (d + 4) * 2.0 ** -23 + 2.0 ** -20
        sums = (t / 16 + 64) * 2.0 ** -23
        bound[:, j] = (p_half_step + 2 * off + 2 * sums) * (p @ vv.abs()) + t * 2.0 ** -31 * vv.abs().max()
    return out, bound


class Case:
    """A batch over a paged cache with its pages dealt at random."""

    def __init__(self, news, lens, page_tokens, seed=0, spare=3, pad=0):
        g = torch.Generator().manual_seed(seed)
        self.news, self.lens, self.pt, self.g = list(news), list(lens), page_tokens, g
        counts = [-(-max(n, 0) // page_tokens) for n in lens]
        self.pages = sum(counts) + spare
        perm = torch.randperm(self.pages, generator=g).int()
        self.table = torch.full((len(lens), max(1, max(counts))), -1, dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = perm[at:at + c]
            at += c
        self.free = perm[at:]
        self.n = sum(news)
        self.rows = self.n + pad
        self.q_start = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32)
        self.k_start = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)

    def batch(self, max_new=0):
        return kvq.PagesBatch(self.q_start.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.table.cuda(),
                              self.rows, max_new)

    def whole(self):
        """The batch whose new tokens are all tokens of all sequences."""
        return kvq.PagesBatch(self.k_start.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.table.cuda(),
                              int(self.k_start[-1]))

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g)


FORMATS = {"f16": (None, None, kvq.F16), "bf16": (None, None, kvq.BF16),
           "8_8": ((8, 32, 0, 0), (8, 64, 0, 0), kvq.F16), "4_4": ((4, 64, 0, 0), (4, 64, 0, 0), kvq.F16),
           "8_4": ((8, 64, 0, 0), (4, 32, 0, 0), kvq.F16), "4_8": ((4, 32, 0, 0), (8, 32, 0, 0), kvq.F16)}
