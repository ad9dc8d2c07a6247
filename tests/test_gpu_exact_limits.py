"""Exact attention and the paged cache on the GPU, at the limits of what the calls take: offsets out of order, many
groups of sequences, extreme scores and values, page numbers outside the pool, pools of many pages."""
import os
import random
import subprocess
import sys

import pytest
import torch

import lsh_sampled_sparse_simhash_b200 as mp
from exact_ref import Pages, check_paged, check_prompt
from test_gpu_exact import (  # noqa: F401
    D, Cache, _built, i32, paged_case, prompt_case, rand, run_paged, run_prompt, status_word)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ prompts ----

def attend_rows(q, k, v, cu):
    """One call over `cu`; out and lse hold 7 where nothing was written.  Returns out, lse, status."""
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    st = status_word()
    mp.prompt_attend(mp.PromptShape(len(cu) - 1, q.shape[1], k.shape[1], D, q.shape[0]), q.cuda(), k.cuda(), v.cuda(), i32(cu),
                     out, lse, status=st)
    return out.cpu(), lse.cpu(), st.item()


@pytest.mark.parametrize("total,hq,hkv,cu,good", [
    (8192, 4, 1, [0, 4096, 0, 4096, 8192], 1),         # overlapping sequences of more items than fit the grid of 8192 rows
    (2000, 4, 2, [0, 700, 700, 1000, 900, 1200, 2000], 3),
    (300, 2, 1, [0, 100, 301, 300], 1),                # past the rows
    (300, 2, 1, [-1, 100, 200, 300], 0),
    (300, 2, 1, [200, 100, 200, 300], 0),
    (2000, 2, 1, [20 * i for i in range(60)] + [5] + [20 * i for i in range(60, 100)], 59),  # more than 32 sequences
    (2000, 2, 1, [20 * i for i in range(33)] + [5] * 60, 32),
    (9000, 16, 16, [0, 1500, 3000, 4500, 6000, 7500, 7400, 9000], 5),  # in the second group of 4096 tokens
    (9000, 16, 16, [0, 1500, 7500, 7400, 9000], 2),    # behind a sequence that is a group of its own
])
def test_prompt_out_of_order_ends_the_list(total, hq, hkv, cu, good):
    """The sequences before the first one whose entries break the order are right, nothing else is written."""
    q, k, v, _ = prompt_case([total], hq, hkv, seed=200 + good)
    out, lse, status = attend_rows(q, k, v, cu)
    assert status == mp.MP_ERR_CAPACITY
    end = cu[good] if good else 0
    heads, g = (0, hkv - 1), hq // hkv
    for u in heads:
        at = slice(u * g, (u + 1) * g)
        check_prompt(q[:, at], k[:, u:u + 1], v[:, u:u + 1], cu[:good + 1], out[:, at], lse[:, at])
    assert (lse[:end] != 7.0).all() and (lse[end:] == 7.0).all() and (out[end:] == 7.0).all()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [5, 6, 9, 12, 20, 45])
def test_prompt_scores_of_any_size(power, sign):
    """Scores up to 2^100, so far apart that one key has all the weight: each row's result is the value of the visible
    key with the largest score.  (At power 6 a row's scores lie on both sides of 2^24.)"""
    n, hq, hkv = 512, 4, 2
    order = torch.randperm(n, generator=torch.Generator().manual_seed(power))
    w = (128 + torch.arange(n) % 128) * 2 ** (torch.arange(n) // 128)  # 512 different numbers of 8 bits
    w = w[order].double()
    q = torch.full((n, hq, D), sign * 2.0 ** power, dtype=torch.bfloat16)
    k = (w * 2.0 ** power).bfloat16()[:, None, None].expand(n, hkv, D).contiguous()
    v = rand(n, hkv, D, seed=300)
    s = sign * w * 2.0 ** (2 * power) * 128  # exact, in fp32 too
    out, lse = run_prompt(q, k, v, [0, n])
    best = torch.stack([s[:i + 1].argmax() for i in range(n)])
    want = v[best].repeat_interleave(hq // hkv, dim=1).double()
    # the weight is rounded to bf16 against an unrounded sum, and the result to bf16
    assert ((out.double() - want).abs() <= (2 * 2.0 ** -8 + 2.0 ** -16) * want.abs() + 1e-30).all()
    want = s[best][:, None] / 128 ** 0.5
    # one product, one multiply-add and the conversion to natural logarithms, with rounded constants; a logarithm of the sum
    assert ((lse.double() - want).abs() <= 6 * 2.0 ** -24 * want.abs() + 2.0 ** -22).all()


@pytest.mark.parametrize("lag", [0.0, 15.0])
def test_values_up_to_their_limit(lag):
    """Values of 2^78: the results of the same values without the factor, times it, exactly.  With a lag the rows' scores
    rise by that much (e^15 = 2^21.6) behind the first key tile that they meet."""
    n = 900
    q, k, v, cu = prompt_case([n], 4, 2, seed=310)
    q[:, :, 0], k[:, :, 0] = 1.0, 0.0
    k[:n - 200, :, 0] = lag * 128 ** 0.5
    want, want_lse = run_prompt(q, k, v, cu)
    out, lse = run_prompt(q, k, (v.float() * 2.0 ** 78).bfloat16(), cu)
    assert torch.equal(out.double(), want.double() * 2.0 ** 78) and torch.equal(lse, want_lse)
    check_prompt(q, k, v, cu, want, want_lse)
    q, k, v, table = paged_case([n, 5], 4, 2, 16, seed=311)
    want, want_lse = run_paged(q, k, v, table, [n, 5])
    out, lse = run_paged(q, k, (v.float() * 2.0 ** 78).bfloat16(), table, [n, 5])
    assert torch.equal(out.double(), want.double() * 2.0 ** 78) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("hq,hkv,lens", [
    (16, 16, [1500, 0, 1800, 700, 900, 3000, 1, 0, 2500, 40]),  # groups of up to 4096 tokens
    (16, 16, [300, 0, 5000, 1, 900, 0]),                        # one longer than a group: 13 kv heads, then 3
    (16, 8, [50] * 60 + [9000] + [20] * 40 + [0, 129]),         # more than 32 sequences to a group, before and behind it
    (32, 16, [4096, 4096, 4097, 1]),
])
def test_prompt_groups_of_sequences(hq, hkv, lens):
    """More keys and values than the blocks keep together: every row is written, with the result of a call for its sequence
    alone; the longest sequence and some heads against the 64-bit reference."""
    q, k, v, cu = prompt_case(lens, hq, hkv, pad=3, seed=320)
    out, lse, status = attend_rows(q, k, v, cu)
    assert status == 0 and (lse[:cu[-1]] != 7.0).all() and (lse[cu[-1]:] == 7.0).all() and (out[cu[-1]:] == 7.0).all()
    for lo, n in zip(cu, lens):
        if n:
            at = slice(lo, lo + n)
            alone, alone_lse, _ = attend_rows(q[at], k[at], v[at], [0, n])
            assert torch.equal(out[at], alone) and torch.equal(lse[at], alone_lse), (lo, n)
    g, lo = hq // hkv, cu[lens.index(max(lens))]
    at = slice(lo, lo + max(lens))
    for u in (0, hkv - 1):  # of the first part of the heads and of the second
        h = u * g
        check_prompt(q[at, h:h + 1], k[at, u:u + 1], v[at, u:u + 1], [0, max(lens)], out[at, h:h + 1], lse[at, h:h + 1])


def test_prompt_many_heads():
    """More heads than a group of sequences has room for tokens: 109 tokens a group, 300 kv heads of three query heads."""
    lens = [130, 1, 0, 77, 20]
    q, k, v, cu = prompt_case(lens, 900, 300, seed=325)
    out, lse, status = attend_rows(q, k, v, cu)
    assert status == 0 and (lse != 7.0).all()
    for u in (0, 150, 299):
        check_prompt(q[:, 3 * u:3 * u + 3], k[:, u:u + 1], v[:, u:u + 1], cu, out[:, 3 * u:3 * u + 3], lse[:, 3 * u:3 * u + 3])
    one = [x[:130].contiguous() for x in (q, k, v)]
    assert torch.equal(out[:130, 200:260], attend_rows(*one, [0, 130])[0][:, 200:260])


@pytest.mark.parametrize("threads", [1, 8])
def test_first_calls_of_threads(threads):
    """A process whose first call comes from a new host thread, or from eight at once."""
    code = f'''
import threading, torch
import lsh_sampled_sparse_simhash_b200 as mp
N = {threads}
q = torch.ones(8, 4, 128, dtype=torch.bfloat16, device="cuda")
cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
outs = [torch.zeros_like(q) for _ in range(N)]
torch.cuda.synchronize()
mp.library()
ready, failed = threading.Barrier(N), []
def call(i):
    ready.wait()
    try:
        mp.prompt_attend(mp.PromptShape(1, 4, 4, 128, 8), q, q, q, cu, outs[i])
    except Exception as e:
        failed.append(e)
threads = [threading.Thread(target=call, args=(i,)) for i in range(N)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not failed, failed
assert all((o == 1).all() for o in outs)
'''
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


# -------------------------------------------------------------------- paged ----

@pytest.mark.parametrize("size", [16, 24])
@pytest.mark.parametrize("bad", [-1, -2, -7, -(1 << 31), "P"])
def test_paged_reports_every_bad_page(size, bad):
    """Any number outside the pool within a length: left out and recorded; behind the length it does not matter."""
    lens = [100, 40]
    q, k, v, table = paged_case(lens, 4, 2, size, seed=330)
    bad = k.shape[0] if bad == "P" else bad
    table[1] = table[1][:2] + [bad] * (len(table[1]) - 2) if size == 24 else table[1][:3] + [bad] * (len(table[1]) - 3)
    out, lse = run_paged(q, k, v, table, lens)
    check_paged(q, k, v, table, lens, out, lse)
    table[0][1] = bad
    out, lse = run_paged(q, k, v, table, lens, want=mp.MP_ERR_CAPACITY)
    check_paged(q, k, v, table, lens, out, lse)


@pytest.mark.parametrize("batch,hkv", [(4096, 2), (4095, 16)])
def test_paged_largest_batches(batch, hkv):
    """As many sequences as a call takes, and as many (sequence, kv head) pairs; empty ones and a long one among them."""
    r = random.Random(batch)
    lens = [r.choice((0, 0, 1, 3, 17, 40)) for _ in range(batch)]
    lens[batch // 3] = 700
    q, k, v, table = paged_case(lens, hkv, hkv, 16, seed=345)
    out, lse = run_paged(q, k, v, table, lens)
    some = sorted(r.sample(range(batch), 60) + [0, batch // 3, batch - 1])
    check_paged(q[some], k, v, [table[b] for b in some], [lens[b] for b in some], out[some], lse[some])
    assert (out != 7.0).all() and (lse != 7.0).all() and torch.equal(torch.isfinite(lse[:, 0]), torch.tensor(lens) > 0)


def test_append_one_row_of_every_sequence():
    """The largest batch, one row each, step after step: every row in its place, every length one more."""
    batch, size, steps = 4096, 4, 6
    shape = mp.PagesShape(batch, 1, 1, D, 2 * batch, size, 2)
    table, lens, refs = i32([[-1] * 2] * batch), i32([0] * batch), i32([0] * 2 * batch)
    k, v = (torch.zeros(2 * batch, 1, size, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mp.pages_reserve(shape, i32([steps] * batch), table, lens, refs)
    rows = [(rand(batch, 1, D, seed=340 + t), rand(batch, 1, D, seed=360 + t)) for t in range(steps)]
    st = status_word()
    for a, b in rows:
        mp.paged_append(shape, a.cuda(), b.cuda(), table, lens, k, v, status=st)
    assert st.item() == 0 and (lens == steps).all()
    at = table.cpu().long()
    for t, (a, b) in enumerate(rows):
        assert torch.equal(k.cpu()[at[:, t // size], 0, t % size], a[:, 0])
        assert torch.equal(v.cpu()[at[:, t // size], 0, t % size], b[:, 0])


def test_plans_of_a_large_pool():
    """A pool whose runs are longer than the plans keep in registers (1024 pages a warp): reserve, fork, free and compact
    with used and free pages all over it, against the model."""
    P, batch, cols, size = 300000, 60, 3000, 4
    shape = mp.PagesShape(batch, 4, 1, D, P, size, cols)
    r = random.Random(1)
    m = Pages(batch, P, size, cols)
    order = r.sample(range(P), P)
    at = 0
    for b in range(40):
        n = r.randint(1, 2400 * size)
        h = -(-n // size)
        m.table[b] = order[at:at + h] + [-1] * (cols - h)
        m.lens[b] = n
        at += h
    for row in m.table:
        for p in row:
            if p >= 0:
                m.refs[p] = 1
    for p in order[at:at + 200000]:  # pages of nobody's here
        m.refs[p] = 2
    table, lens, refs = i32(m.table), i32(m.lens), i32(m.refs)
    st = status_word()

    def same():
        torch.cuda.synchronize()
        assert st.item() == 0 and lens.tolist() == m.lens and refs.tolist() == m.refs and table.tolist() == m.table

    def entries(copies, want):
        got = copies.tolist()
        assert got[0] == [len(want), 0, 0, 0] and [tuple(e[:3]) for e in got[1:1 + len(want)]] == want

    same()
    new = [r.choice((0, 1, 9, 2000)) if b < 40 else 0 for b in range(batch)]
    assert m.reserve(new)
    mp.pages_reserve(shape, i32(new), table, lens, refs, status=st)
    same()
    src, dst = [r.randrange(40) for _ in range(20)], list(range(40, 60))
    copies = torch.zeros(21, 4, dtype=torch.int32, device="cuda")
    mp.pages_fork(shape, i32(src), i32(dst), table, lens, refs, copies, status=st)
    entries(copies, m.fork(src, dst))
    same()
    ends = list(range(0, 60, 3))
    m.free(ends)
    mp.pages_free(shape, i32(ends), table, lens, refs, status=st)
    same()
    copies = torch.zeros(1 + P // 2, 4, dtype=torch.int32, device="cuda")
    mp.pages_compact(shape, table, refs, copies, status=st)
    entries(copies, m.compact())
    same()
    new = [4000 if t[0] < 0 else 0 for t in m.table]
    assert m.reserve(new)
    mp.pages_reserve(shape, i32(new), table, lens, refs, status=st)
    same()


def test_fork_with_too_few_pages_changes_nothing():
    c = Cache(6, 10, 4, 6)
    assert c.reserve([6, 0, 0, 3, 0, 0])
    c.append([6, 0, 0, 3, 0, 0])
    assert c.reserve([18, 0, 0, 9, 0, 0]) and len(c.m.free_pages()) == 1
    c.check()
    assert c.fork([0, 3], [1, 2]) == mp.MP_ERR_CAPACITY  # two partly filled pages; the list of copies is empty
    c.check()
    assert c.fork([0], [1]) == 0 and not c.m.free_pages()
    c.check()


def test_fork_of_empty_and_reserved_sequences():
    """A source without tokens gives one without; pages that a source holds past its length stay its own."""
    c = Cache(6, 20, 4, 5)
    assert c.reserve([8, 13, 0, 0, 0, 0])
    c.append([8, 2, 0, 0, 0, 0])
    assert c.fork([0, 1, 2], [3, 4, 5]) == 0
    c.check()
    assert c.reserve([1] * 6)
    c.append([1] * 6)
    c.check()


# ---------------------------------------------------------- the sampled decode ----

def test_prompt_into_the_contiguous_cache():
    """A prompt's rows stored by the append into the cache of the sampled decode, as one page a sequence: hashed and
    decoded like the same cache filled by hand, and like the paged decode over it."""
    B, Hq, Hkv, cap, n = 2, 8, 2, 512, [300, 411]
    q, k, v, cu = prompt_case(n, Hq, Hkv, seed=370)
    out, lse = run_prompt(q, k, v, cu)
    check_prompt(q, k, v, cu, out, lse)
    kc, vc, by_hand, by_hand_v = (torch.zeros(B, Hkv, cap, D, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    lens, table = i32([0, 0]), i32([[0], [1]])
    st = status_word()
    mp.paged_append(mp.PagesShape(B, Hq, Hkv, D, B, cap, 1), k.cuda(), v.cuda(), table, lens, kc, vc, cu_new=i32(cu), status=st)
    for b in range(B):
        by_hand[b, :, :n[b]] = k[cu[b]:cu[b + 1]].transpose(0, 1).cuda()
        by_hand_v[b, :, :n[b]] = v[cu[b]:cu[b + 1]].transpose(0, 1).cuda()
    assert st.item() == 0 and lens.tolist() == n and torch.equal(kc, by_hand) and torch.equal(vc, by_hand_v)
    W, q1 = rand(75 * 8, D, seed=380).cuda(), rand(B, Hq, D, seed=381)
    k1, v1 = rand(B, Hkv, D, seed=382).cuda(), rand(B, Hkv, D, seed=383).cuda()

    def decode(window, k_cache, v_cache):
        shape, at = mp.Shape(B, Hq, Hkv, D, cap, 8, 75, 4, window), i32(n)
        codes = torch.zeros(mp.codes_shape(shape)[1], dtype=torch.uint8, device="cuda")
        mp.hash_keys(shape, k_cache, W, max(n), codes)
        mp.append_token(shape, k1, v1, W, k_cache, v_cache, codes, at)
        out, lse, ns = torch.zeros(B, Hq, D, device="cuda"), torch.zeros(B, Hq, device="cuda"), i32([[0] * Hq] * B)
        ws = torch.empty(mp.decode_workspace_bytes(shape, max(n) + 1), dtype=torch.uint8, device="cuda")
        mp.decode_attend(shape, q1.cuda(), W, codes, k_cache, v_cache, at, max(n) + 1, out, lse, ns, ws)
        torch.cuda.synchronize()
        return codes, at, out.cpu(), lse.cpu(), ns

    for window in (64, cap):
        a, b = decode(window, kc.clone(), vc.clone()), decode(window, by_hand.clone(), by_hand_v.clone())
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    mp.append_token(mp.Shape(B, Hq, Hkv, D, cap, 8, 75, 4, cap), k1, v1, W, kc, vc, a[0], lens)
    got, got_lse = run_paged(q1, kc.cpu(), vc.cpu(), [[0], [1]], [x + 1 for x in n])
    # the sampled decode with every token in its exact set; its own bars: 2e-3 relative L2, 1e-3 on lse
    assert (got - a[2]).norm() / got.norm() <= 2e-3 and (got_lse - a[3]).abs().max() <= 1e-3
