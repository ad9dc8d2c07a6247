"""Plain 64-bit references of the exact-attention calls and their error bounds (test infrastructure).

Bounds.  A rounding to bf16 is off by at most U = 2^-8 of the value, to fp32 by 2^-24.  For one query let
p_j = softmax weights, A = sum_j p_j |v_j| (per output dim), X = max_j scale sum_d |q_d k_d| and n the keys.
  - a score is an fp32 sum of 128 products (exact: bf16 x bf16); allowing one truncated step of 2^-23 per term,
    |ds| <= E = 130 * 2^-23 X, which moves out by at most 2 E A and lse by E;
  - 2^x has a relative error below 2^-22, the n-term fp32 sums (numerator and denominator) n 2^-24 each;
  - weights rounded to bf16 before the product (prompts) add U A, the rounding of out to bf16 U |out|;
  - weights as three bf16 parts (paged) add 2^-24 A.
"""
import math

import torch

SCALE = 1.0 / math.sqrt(128.0)
U_BF16 = 2.0 ** -8


def attend(q, k, v, n_seen):
    """Rows of one head in fp64: q [m, d], k / v [n, d]; row i sees keys 0 .. n_seen[i] - 1.
    Returns out, lse, A, X (see above)."""
    q, k, v = q.double(), k.double(), v.double()
    s = q @ k.T * SCALE
    hidden = torch.arange(k.shape[0])[None, :] >= n_seen[:, None]
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, dim=1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    x = (q.abs() @ k.abs().T * SCALE).masked_fill(hidden, 0.0).amax(1)
    return p @ v, lse, p @ v.abs(), x


def check_head(got_out, got_lse, ref, n_seen, bf16_weights):
    """Asserts one head's rows [m, d] / [m] against attend()'s `ref` by the bounds above."""
    out, lse, A, X = ref
    n = n_seen.double()[:, None]
    E = (130 * 2.0 ** -23 * X)[:, None]
    rel = 2 * E + 2 * 2.0 ** -22 + 2 * n * 2.0 ** -24
    if bf16_weights:
        tol = A * (rel + U_BF16) * (1 + U_BF16) + out.abs() * U_BF16 + 1e-30
    else:
        tol = A * (rel + 2.0 ** -24) + out.abs() * 2.0 ** -23 + 1e-30
    err = (got_out.double() - out).abs()
    assert torch.isfinite(got_out.double()).all()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, worst
    if got_lse is not None:
        seen = n_seen > 0
        assert torch.equal(got_lse[~seen].double(), torch.full((int((~seen).sum()),), -math.inf, dtype=torch.float64))
        tol = E[:, 0] + 2.0 ** -22 + n[:, 0] * 2.0 ** -24 + lse.abs() * 2.0 ** -22
        bad = ~((got_lse.double() - lse).abs() <= tol) & seen  # (NaN is not within it)
        assert not bad.any(), (got_lse[bad], lse[bad])
    return worst


def check_prompt(q, k, v, cu, out, lse):
    """Every sequence and head of a packed prompt call (CPU tensors)."""
    hq, hkv = q.shape[1], k.shape[1]
    for b in range(len(cu) - 1):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if hi <= lo:
            continue
        seen = torch.arange(1, hi - lo + 1)
        for h in range(hq):
            u = h // (hq // hkv)
            ref = attend(q[lo:hi, h], k[lo:hi, u], v[lo:hi, u], seen)
            check_head(out[lo:hi, h], None if lse is None else lse[lo:hi, h], ref, seen, True)


def gather(pool, row, n, u):
    """Tokens 0 .. n - 1 of kv head u of one sequence ([n, d]); None for tokens on pages outside the pool."""
    size = pool.shape[2]
    at = torch.arange(n)
    page = torch.as_tensor(row, dtype=torch.long)[at // size] if n else torch.zeros(0, dtype=torch.long)
    good = (page >= 0) & (page < pool.shape[0])
    return pool[page[good], u, (at % size)[good]]


def check_paged(q, k_pages, v_pages, table, lens, out, lse):
    hq, hkv = q.shape[1], k_pages.shape[1]
    g = hq // hkv
    for b in range(q.shape[0]):
        n = int(lens[b])
        for u in range(hkv):
            k, v = gather(k_pages, table[b], n, u), gather(v_pages, table[b], n, u)
            seen = torch.full((g,), k.shape[0])
            if k.shape[0] == 0:
                assert (out[b, u * g:(u + 1) * g] == 0).all() and torch.isinf(lse[b, u * g:(u + 1) * g]).all()
                assert (lse[b, u * g:(u + 1) * g] < 0).all()
                continue
            ref = attend(q[b, u * g:(u + 1) * g], k, v, seen)
            check_head(out[b, u * g:(u + 1) * g], lse[b, u * g:(u + 1) * g], ref, seen, False)
            err = (out[b, u * g:(u + 1) * g].double() - ref[0]).norm() / ref[0].norm()
            # rounding errors of random sign: 128-term fp32 scores give about sqrt(128) 2^-24 X relative per weight,
            # far below 2^-17, which one bf16 part (2^-9) would exceed
            assert err <= 2.0 ** -17, err


class Pages:
    """The page operations on Python lists (include/magicpig.h)."""

    def __init__(self, batch, n_pages, size, cols):
        self.size, self.cols = size, cols
        self.table = [[-1] * cols for _ in range(batch)]
        self.lens = [0] * batch
        self.refs = [0] * n_pages

    def held(self, b):
        return next((c for c, p in enumerate(self.table[b]) if p < 0), self.cols)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def pages_for(self, tokens):
        return -(-tokens // self.size)

    def reserve(self, new):
        need = [max(0, self.pages_for(n + m) - self.held(b)) if m > 0 else 0
                for b, (n, m) in enumerate(zip(self.lens, new))]
        free = self.free_pages()
        if sum(need) > len(free) or any(m > 0 and n + m > self.cols * self.size for n, m in zip(self.lens, new)):
            return False
        for b, k in enumerate(need):
            at = self.held(b)
            for c in range(at, at + k):
                self.table[b][c] = free.pop(0)
                self.refs[self.table[b][c]] = 1
        return True

    def fork(self, src, dst):
        """The list of copies, or None if refused."""
        batch = len(self.table)
        for a, b in zip(src, dst):
            if not (0 <= a < batch and 0 <= b < batch) or b in src or dst.count(b) > 1 or self.table[b][0] >= 0:
                return None
            if any(p < 0 or p >= len(self.refs) or self.refs[p] < 1
                   for p in self.table[a][:self.pages_for(self.lens[a])]):
                return None
        free, copies = self.free_pages(), []
        if sum(self.lens[a] % self.size > 0 for a in src) > len(free):
            return None
        for a, b in zip(src, dst):
            full, part = divmod(self.lens[a], self.size)
            row = self.table[a][:full]
            for p in row:
                self.refs[p] += 1
            if part:
                page = free.pop(0)
                self.refs[page] = 1
                copies.append((self.table[a][full], page, part))
                row = row + [page]
            self.table[b] = row + [-1] * (self.cols - len(row))
            self.lens[b] = self.lens[a]
        return copies

    def free(self, seqs):
        for b in seqs:
            for c, p in enumerate(self.table[b]):
                if p >= 0:
                    self.refs[p] -= 1
                    self.table[b][c] = -1
            self.lens[b] = 0

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        holes = [p for p in range(used) if self.refs[p] == 0]
        movers = [p for p in range(used, len(self.refs)) if self.refs[p] > 0]
        for to, of in zip(holes, movers):
            self.refs[to], self.refs[of] = self.refs[of], 0
        where = dict(zip(movers, holes))
        self.table = [[where.get(p, p) for p in row] for row in self.table]
        return [(of, to, self.size) for to, of in zip(holes, movers)]
