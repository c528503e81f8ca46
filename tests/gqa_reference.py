"""Plain 64-bit forms of grouped-query attention and of the page pool's upkeep,
and the error bounds that its tests use.

Bounds.  With u_out the unit roundoff of the output's type, u_p that of the
type in which the weights p enter the second product (bf16 on the tensor
cores, f16 over an fp8 cache, else fp32), and A = sum_s softmax_s |v_s|:

    |out - ref| <= u_out |ref| + A (u_p + 2 d + e)        |lse - ref| <= d + e + 2^-22 |ref|

  d  error of a score: a dot product of `dim` terms in fp32 and the products
     with the scale, (dim + 8) 2^-24 scale max sum_i |q_i k_i|; twice, because
     numerator and denominator both carry it;
  e  the exponential (2^-21, and its argument's rounding: 2^-24 times the
     spread of the scores in base 2) and the fp32 sums of n terms (n 2^-24).
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attend(q, k, v, scale, mask):
    """q [H, m, D], k / v [Hkv, n, D], mask [m, n] bool: out [H, m, D], lse [H, m], A, score bound, spread (float64)."""
    H, m, D = q.shape
    g = H // k.shape[0]
    q, k, v = q.double(), k.double().repeat_interleave(g, 0), v.double().repeat_interleave(g, 0)
    z = (q @ k.transpose(1, 2)) * scale
    z = z.masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.where(mask, torch.exp(z - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[..., None]),
                    torch.zeros_like(z))
    mag = (q.abs() @ k.abs().transpose(1, 2)) * scale
    d = float(mag.max()) * (D + 8) * 2.0 ** -24 if mag.numel() else 0.0
    return p @ v, lse, p @ v.abs(), d


def check(out, lse, ref, ref_lse, A, d, n, u_p):
    """out / ref [..., D], lse / ref_lse [...]: asserts the bounds of this module."""
    e = 2.0 ** -21 + n * 2.0 ** -24 + 64 * 2.0 ** -24
    tol = U[out.dtype] * ref.abs() + A * (u_p + 2 * d + e) + 1e-30
    err = (out.double() - ref).abs()
    assert bool(torch.isfinite(out).all()), "out is not finite"
    worst = float((err / tol).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"output error {worst:.3g} times its bound"
    empty = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), empty)
    lerr = (lse.double() - ref_lse)[~empty].abs()
    ltol = d + e + 2.0 ** -22 * ref_lse[~empty].abs()
    worst = float((lerr / ltol).max()) if lerr.numel() else 0.0
    assert worst <= 1.0, f"lse error {worst:.3g} times its bound"


def e4m3_rows(x):
    """Rows of x [..., D] (fp32) in fp8: codes and scales by the cache's rule.  The
    quotients are formed in 64 bits and rounded to 32, which gives the correctly
    rounded binary32 quotient (torch divides by a number through its reciprocal)."""
    amax = x.abs().amax(-1).double()
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax)).float()
    quot = (x.double() / scale.double()[..., None]).float()
    return quot.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


class Pool:
    """The pool's books and caches kept entry by entry, in plain Python."""

    def __init__(self, batch, max_pages, page, num_pages):
        self.page, self.max_pages = page, max_pages
        self.table = [[-1] * max_pages for _ in range(batch)]
        self.length = [0] * batch
        self.count = [0] * num_pages

    def up(self, n):
        return -(-n // self.page)

    def free_ids(self):
        return [i for i, c in enumerate(self.count) if c == 0]

    def extend(self, seqs, add):
        free, asked, seen, ok = self.free_ids(), 0, set(), True
        first = list(self.length)
        for q, a in zip(seqs, add):
            if q == -1:
                continue
            if q in seen or not 0 <= q < len(self.length) or a < 0 or first[q] + a > self.max_pages * self.page:
                ok = False
                seen.add(q)
                continue
            seen.add(q)
            have, want = self.up(first[q]), self.up(first[q] + a)
            start, asked = asked, asked + want - have
            if want > have and asked > len(free):
                ok = False
                continue
            for j in range(have, want):
                self.table[q][j] = free[start + j - have]
                self.count[self.table[q][j]] = 1
            self.length[q] += a
        return ok

    def free(self, seqs):
        for q in seqs:
            if q == -1:
                continue
            for j in range(self.up(self.length[q])):
                self.count[self.table[q][j]] -= 1
                self.table[q][j] = -1
            self.length[q] = 0

    def fork(self, parents, children):
        """Returns the (src, dst) page copies."""
        free, asked, seen, pairs = self.free_ids(), 0, set(), []
        first = list(self.length)
        for p, c in zip(parents, children):
            if c == -1 or c in seen or first[c] != 0 or not 0 <= p < len(first):
                continue
            seen.add(c)
            full, ends = first[p] // self.page, first[p] % self.page > 0
            asked += ends
            if ends and asked > len(free):
                continue
            for j in range(full):
                self.table[c][j] = self.table[p][j]
                self.count[self.table[p][j]] += 1
            if ends:
                pairs.append((self.table[p][full], free[asked - 1]))
                self.table[c][full] = free[asked - 1]
                self.count[free[asked - 1]] = 1
            self.length[c] = first[p]
        return pairs

    def compact(self):
        live = sum(c > 0 for c in self.count)
        src = [i for i in range(live, len(self.count)) if self.count[i] > 0]
        dst = [i for i in range(live) if self.count[i] == 0]
        to = dict(zip(src, dst))
        for a, b in to.items():
            self.count[b], self.count[a] = self.count[a], 0
        self.table = [[to.get(x, x) for x in row] for row in self.table]
        return list(zip(src, dst))
