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
