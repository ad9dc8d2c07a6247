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
