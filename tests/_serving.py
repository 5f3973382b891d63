"""Shared helpers of the serving tests: random caches and page tables, and the derived tolerances.

Tolerances, u the half step of the output type (fp16 2^-11, bf16 2^-8; subnormal fp16 2^-25):

* norm and rotation: the sum of d <= 256 squares in fp32 (8 per lane, then 5 shuffle steps) is off by at
  most 13 half steps of 2^-24, its root by half of that, rsqrtf by 2 steps, the products and the
  rotation by one half step each (about 5): under 16 * 2^-24 = 2^-20 of the terms' magnitudes; the bound
  takes 2^-19.  Then one rounding: u |y|.
* cache write without norm and rotation, and every read: IEEE float32 operations, bit for bit.
* cache write with norm and rotation: the value y is off by 2^-19 mag as above, so amax and the scale
  by as much relative to the row's largest magnitude M, and |code * ks - y| <= ks / 2 + 2^-17 M (half a
  step; the errors of y, of the scale over up to 127 steps, and of the product).
* decode: a score is off by at most (d + 8) half steps of its terms' magnitude delta, from the fp32
  sums, plus 2^-20 of itself for the scale products; ex2 and lg2 add 2^-21.  With e that error
  (natural units), weights are off by e relative to each other's, the output by 2 e sum p |v| (numerator and
  denominator).  P as fp16 adds 2^-11 sum p |v| for bf16 outputs, 2^-21 for fp16 (two terms).  fp32
  sums of n keys: n / 16 steps of accumulation at most, 2^-24 n / 8 sum p |v|.  Then u |out|.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import serving

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SUB = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}


def np32(t):
    return t.detach().float().cpu().numpy()


def heads(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def rope_table(n, rot, base=10000.0):
    ang = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def page_table(lens, page_size, seed, extra=0, spare_pages=3, behind=-7):
    """Random distinct pages for every sequence, `behind` in the entries after them; (table, num_pages)."""
    need = [-(-n // page_size) for n in lens]
    total = sum(need) + spare_pages
    order = np.random.RandomState(seed).permutation(total)
    table = np.full((len(lens), max(1, max(need) + extra)), behind, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table), total


def poison(lib, num_pages, Hkv, d, page_size):
    """A cache whose every byte would show if it were read: NaN codes and scales."""
    c = lib.sage_kv_cache(num_pages, Hkv, d, page_size)
    c["k8"].fill_(127), c["v8"].fill_(0x7F)
    c["ks"].fill_(math.nan), c["vs"].fill_(math.nan)
    return c


def fill(cache, table, lens, k8, ks, v8, vs, d):
    """Puts the sequences' codes (lists of (n, Hkv, ...) arrays) into their pages; channels behind d get code 0."""
    ps = cache["ks"].shape[2]
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pos = torch.arange(n)
        page, slot = table[b].long()[pos // ps].cuda(), (pos % ps).cuda()
        for name, x in (("k8", k8[b]), ("v8", v8[b])):
            full = np.zeros((*x.shape[:2], cache["k8"].shape[3]), x.dtype)
            full[..., :d] = x
            cache[name][page, :, slot] = torch.from_numpy(full).cuda()
        cache["ks"][page, :, slot] = torch.from_numpy(ks[b]).cuda()
        cache["vs"][page, :, slot] = torch.from_numpy(vs[b]).cuda()


def random_sequences(lens, Hkv, d, seed, k_amp=1.0, v_amp=1.0):
    """Codes and scales of N(0, 1) keys and values, per sequence."""
    out = ([], [], [], [])
    for b, n in enumerate(lens):
        r = np.random.RandomState(seed * 1000 + b)
        k8, ks = serving.k_codes((r.randn(n, Hkv, d) * k_amp).astype(np.float32))
        v8, vs = serving.v_codes((r.randn(n, Hkv, d) * v_amp).astype(np.float32))
        for o, x in zip(out, (k8, ks, v8, vs)):
            o.append(x)
    return out


def check_norm_rope(got, x, dtype, norm, eps, w, cos_sin, pos, interleaved, what=""):
    """got, x (tokens, heads, d)."""
    y, mag = serving.norm_rope(np32(x), norm, eps, None if w is None else np32(w), cos_sin, pos, interleaved)
    tol = U[dtype] * np.abs(y) + 2.0 ** -19 * mag + SUB[dtype]
    err = np.abs(np32(got).astype(np.float64) - y)
    assert (err <= tol).all(), f"{what}: {float((err - tol).max()):.3g} over the tolerance"


def check_decode(out, q, seqs, lens, scale, what=""):
    """out, q (B, Hq, d) tensors; seqs the codes and scales of every sequence."""
    dt = out.dtype
    for b, n in enumerate(lens):
        k8, ks, v8, vs = (x[b][:n] for x in seqs)
        k = k8.astype(np.float64) * ks.astype(np.float64)[..., None]
        v = serving.fp8.decode(v8) * vs.astype(np.float64)[..., None]
        d = q.shape[-1]
        ref, spread, delta = serving.decode(np32(q[b]).astype(np.float64), k, v, scale)
        e = ((d + 8) * 2.0 ** -24 + 2.0 ** -20) * delta + 2.0 ** -21
        p16 = 2.0 ** -11 if dt == torch.bfloat16 else 2.0 ** -21
        tol = U[dt] * np.abs(ref) + (2 * e + p16 + n / 8 * 2.0 ** -24) * spread * 1.01 + SUB[dt]
        err = np.abs(np32(out[b]).astype(np.float64) - ref)
        assert (err <= tol).all(), f"{what} sequence {b} ({n} keys): {float((err - tol).max()):.3g} over the tolerance " \
                                   f"(err {float(err.max()):.3g})"


def bits(t):
    return t.contiguous().view(torch.uint8).reshape(-1)
