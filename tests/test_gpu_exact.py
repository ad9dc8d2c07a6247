"""Exact attention over prompts and over a paged cache, the append and the page operations, on the GPU, against the
64-bit references and bounds of exact_ref.py.  Page tables, counts and moved rows are compared exactly."""
import random

import pytest
import torch

import lsh_sampled_sparse_simhash_b200 as mp
from exact_ref import Pages, check_paged, check_prompt, gather

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def rand(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ prompts ----

def prompt_case(lens, hq, hkv, fused=False, pad=0, lead=0, seed=0):
    """CPU q, k, v and cu; `pad` / `lead` rows behind / before the sequences hold NaN."""
    total = lead + sum(lens) + pad
    q, k, v = rand(total, hq, D, seed=seed), rand(total, hkv, D, seed=seed + 1), rand(total, hkv, D, seed=seed + 2)
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    for x in (q, k, v):
        x[:lead] = float("nan")
        x[cu[-1]:] = float("nan")
    return q, k, v, cu


def run_prompt(q, k, v, cu, fused=False, with_lse=True):
    total, hq, hkv = q.shape[0], q.shape[1], k.shape[1]
    if fused:
        one = torch.cat((q, k, v), dim=1).cuda()
        dq, dk, dv = one[:, :hq], one[:, hq:hq + hkv], one[:, hq + hkv:]
    else:
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    out = torch.full((total, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, hq), 7.0, device="cuda") if with_lse else None
    st = status_word()
    mp.prompt_attend(mp.PromptShape(len(cu) - 1, hq, hkv, D, total), dq, dk, dv, i32(cu), out, lse, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    return out.cpu(), None if lse is None else lse.cpu()


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (3, 1), (8, 2), (5, 1), (6, 1), (7, 1), (8, 1)])
def test_prompt_groups(hq, hkv):
    """Every group size, lengths around the tiles' edges (16 to 256 tokens, 128 keys)."""
    q, k, v, cu = prompt_case([1, 37, 127, 128, 129, 0, 255, 300], hq, hkv, seed=hq)
    out, lse = run_prompt(q, k, v, cu)
    check_prompt(q, k, v, cu, out, lse)


@pytest.mark.parametrize("lens", [[1], [2], [16], [17], [63, 65], [64], [128], [256, 257], [1000], [1] * 70])
def test_prompt_lengths(lens):
    q, k, v, cu = prompt_case(lens, 4, 1, seed=len(lens) + lens[0])
    out, lse = run_prompt(q, k, v, cu)
    check_prompt(q, k, v, cu, out, lse)


@pytest.mark.parametrize("batch,hq,hkv", [(5000, 6, 2), (65536, 2, 1)])
def test_prompt_many_short_sequences(batch, hq, hkv):
    """One-token sequences (whose result is their value, exactly), empty ones and a few longer ones among them."""
    lens = [0 if i % 7 == 3 else 1 for i in range(batch)]
    longer = {11: 130, batch // 2: 300, batch - 1: 2}
    for i, n in longer.items():
        lens[i] = n
    q, k, v, cu = prompt_case(lens, hq, hkv, seed=160)
    out, lse = run_prompt(q, k, v, cu)
    ones = torch.tensor([cu[i] for i, n in enumerate(lens) if n == 1])
    assert torch.equal(out[ones], v[ones].repeat_interleave(hq // hkv, dim=1))
    for i, n in longer.items():
        at = slice(cu[i], cu[i] + n)
        check_prompt(q[at], k[at], v[at], [0, n], out[at], lse[at])


def test_prompt_long():
    """More key tiles than the ring has slots, many times over."""
    q, k, v, cu = prompt_case([2900], 2, 1, seed=5)
    out, lse = run_prompt(q, k, v, cu)
    check_prompt(q, k, v, cu, out, lse)


def test_prompt_fused_rows_with_nan_around():
    """Parts of a fused projection's rows; NaN in the rows before and behind the sequences, which stay as they are."""
    q, k, v, cu = prompt_case([50, 200, 3], 8, 2, pad=140, lead=9, seed=6)
    out, lse = run_prompt(q, k, v, cu, fused=True)
    check_prompt(q, k, v, cu, out, lse)
    for x in (out[:9], out[cu[-1]:], lse[:9], lse[cu[-1]:]):
        assert (x == 7.0).all()
    again, none = run_prompt(q, k, v, cu, fused=False, with_lse=False)
    assert none is None and torch.equal(again[9:cu[-1]], out[9:cu[-1]])


@pytest.mark.parametrize("order", ["up", "down", "spikes"])
def test_prompt_moving_maximum(order):
    """Scores whose maximum moves far from tile to tile (sums rescaled, weights that underflow)."""
    n = 700
    q, k, v, cu = prompt_case([n], 4, 2, seed=7)
    q = q.abs()
    i = torch.arange(n, dtype=torch.float32)
    f = {"up": i / n * 6, "down": 6 - i / n * 6, "spikes": (i % 97 == 5) * 9.0}[order]
    k = (k.float().abs() * f[:, None, None]).bfloat16()
    out, lse = run_prompt(q, k, v, cu)
    check_prompt(q, k, v, cu, out, lse)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (4, 1), (8, 2)])
def test_prompt_not_finite(hq, hkv):
    """A key that is not finite reaches the tokens from its own on; a value that is not, those whose key tiles have it:
    other kv heads, other sequences and the tokens of earlier tiles are as if they were not there."""
    lens, g = [300, 129, 200], hq // hkv
    q, k, v, cu = prompt_case(lens, hq, hkv, seed=140 + hq)
    want, want_lse = run_prompt(q, k, v, cu)
    for x in ("nan", "inf", "-inf"):
        bad = k.clone()
        bad[cu[0] + 150, 0, 3] = float(x)
        out, lse = run_prompt(q, bad, v, cu)
        assert torch.equal(out[:150], want[:150]) and torch.equal(lse[:150], want_lse[:150])
        assert torch.equal(out[300:], want[300:]) and torch.equal(out[:, g:], want[:, g:])
    assert not torch.isfinite(run_prompt(q, torch.where(torch.arange(629)[:, None, None] == 150, float("nan"), k.float()).bfloat16(),
                                         v, cu)[0][150:300].float()).any()
    bad = v.clone()
    bad[cu[2] + 128, 0, 9] = float("nan")
    out, lse = run_prompt(q, k, bad, cu)
    rest = torch.ones(629, hq, D, dtype=torch.bool)
    rest[cu[2] + 128:, :g, 9] = False
    first = 128 // g * 2  # tokens of an item; those whose item begins before the tile may have it as their last one
    rest[cu[2] + 128 // first * first:cu[2] + 128, :g, 9] = False
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse, want_lse)
    assert torch.isnan(out[cu[2] + 128:, :g, 9].float()).all()


def test_scores_all_minus_infinity():
    """Keys of score -inf have no weight; where a query sees no other, its result is that of no key."""
    lens = [3, 140]
    q, k, v, cu = prompt_case(lens, 4, 2, seed=150)
    q[:, :, 5] = 1.0
    k[cu[1]:cu[1] + 130, 1, 5] = float("-inf")  # of the second sequence's first 130 tokens
    out, lse = run_prompt(q, k, v, cu)
    assert (out[3:133, 2:] == 0).all() and (lse[3:133, 2:] == float("-inf")).all()
    check_prompt(q[133:, 2:], k[133:, 1:], v[133:, 1:], [0, 10], out[133:, 2:], lse[133:, 2:])
    q, k, v, table = paged_case([33, 2000], 4, 2, 16, seed=151)
    q[:, :, 5] = 1.0
    for p in table[1]:
        if p >= 0:
            k[p, 1, :, 5] = float("-inf")
    k[table[0][:2], 1, :, 5] = float("-inf")  # all but its last token
    out, lse = run_paged(q, k, v, table, [33, 2000])
    assert (out[1, 2:] == 0).all() and (lse[1, 2:] == float("-inf")).all() and torch.isfinite(out).all()
    want = v[table[0][2], 1, 0].double()
    assert ((out[0, 2:].double() - want).abs() <= 2.0 ** -22 * want.abs()).all()  # weight 1 exactly, up to its sum's division



def test_prompt_bad_lengths_skipped():
    """A sequence whose entries break the rules is skipped and recorded; the others are right."""
    q, k, v, _ = prompt_case([300], 4, 1, seed=8)
    cu = [0, 100, 90, 190, 400]  # the second decreases, the last ends past the rows
    out = torch.full((300, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    st = status_word()
    mp.prompt_attend(mp.PromptShape(4, 4, 1, D, 300), q.cuda(), k.cuda(), v.cuda(), i32(cu), out, status=st)
    torch.cuda.synchronize()
    assert st.item() == mp.MP_ERR_CAPACITY
    out = out.cpu()
    check_prompt(q, k, v, [0, 90], out[:90], None)   # rows 90 .. 99 belong to the first and the third
    assert (out[190:] == 7.0).all()


def test_prompt_captured_and_replayed_with_other_lengths():
    q, k, v, cu = prompt_case([100, 150], 4, 2, seed=9)
    dq, dk, dv, dcu = q.cuda(), k.cuda(), v.cuda(), i32(cu)
    out = torch.zeros(250, 4, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(250, 4, device="cuda")
    shape = mp.PromptShape(2, 4, 2, D, 250)
    mp.prompt_attend(shape, dq, dk, dv, dcu, out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mp.prompt_attend(shape, dq, dk, dv, dcu, out, lse)
    cu = [0, 201, 250]
    dcu.copy_(i32(cu))
    g.replay()
    torch.cuda.synchronize()
    check_prompt(q, k, v, cu, out.cpu(), lse.cpu())


def test_prompt_two_streams_at_once():
    """Two calls on two streams, again and again: each waits for the tensor memory that the other holds."""
    cases = [prompt_case([700 - 300 * j, 45, 300], 8, 2, seed=110 + j) for j in range(2)]
    runs = []
    for q, k, v, cu in cases:
        t = [x.cuda() for x in (q, k, v)]
        runs.append((t, i32(cu), torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda"),
                     torch.zeros(q.shape[:2], device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for t, cu, out, lse, st in runs:
            mp.prompt_attend(mp.PromptShape(3, 8, 2, D, out.shape[0]), *t, cu, out, lse, stream=st)
    torch.cuda.synchronize()
    for (q, k, v, cu), (_, _, out, lse, _) in zip(cases, runs):
        check_prompt(q, k, v, cu, out.cpu(), lse.cpu())


def test_prompt_rows_past_32_bits():
    """A short prompt at the end of row arrays of more than 2^31 elements (and 2^32 bytes)."""
    lead, n, hq, hkv = 560000, 150, 32, 4
    assert (lead + n) * hq * D > 1 << 31
    q, k, v, _ = prompt_case([n], hq, hkv, seed=120)
    with_lead = [torch.empty(lead + n, x.shape[1], D, dtype=torch.bfloat16, device="cuda") for x in (q, k, v)]
    for big, x in zip(with_lead, (q, k, v)):
        big[lead:] = x.cuda()
    out = torch.empty(lead + n, hq, D, dtype=torch.bfloat16, device="cuda")
    mp.prompt_attend(mp.PromptShape(1, hq, hkv, D, lead + n), *with_lead, i32([lead, lead + n]), out)
    check_prompt(q[:, :2], k[:, :1], v[:, :1], [0, n], out[lead:, :2].cpu(), None)
    check_prompt(q[:, 30:], k[:, 3:], v[:, 3:], [0, n], out[lead:, 30:].cpu(), None)


def test_prompt_same_result_every_time():
    q, k, v, cu = prompt_case([333, 20, 512], 8, 2, seed=10)
    a, b = run_prompt(q, k, v, cu), run_prompt(q, k, v, cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_binding_refuses_wrong_tensors():
    q, k, v, cu = prompt_case([20], 4, 2)
    dq, dk, dv, dcu = q.cuda(), k.cuda(), v.cuda(), i32(cu)
    out = torch.zeros(20, 4, D, dtype=torch.bfloat16, device="cuda")
    shape = mp.PromptShape(1, 4, 2, D, 20)
    for bad in ((dq.float(), dk, dv, dcu, out), (dq[:, :2], dk, dv, dcu, out), (dq, dk.transpose(0, 1), dv, dcu, out),
                (dq, dk, dv[:10], dcu, out), (dq, dk, dv, dcu.long(), out), (dq, dk, dv, dcu, out.float()),
                (dq, dk, v, dcu, out), (dq[:1].expand(20, 4, D), dk, dv, dcu, out)):
        with pytest.raises(ValueError):
            mp.prompt_attend(shape, *bad)
    with pytest.raises(mp.MagicPIGError) as e:
        mp.prompt_attend(mp.PromptShape(1, 4, 2, D, 20), torch.zeros(20, 4 * D + 4, dtype=torch.bfloat16,
                                                                    device="cuda")[:, :4 * D].view(20, 4, D), dk, dv, dcu, out)
    assert e.value.code == mp.MP_ERR_SHAPE


# -------------------------------------------------------------------- paged ----

def paged_case(lens, hq, hkv, size, seed=0, extra=3):
    """CPU q, pools, table (shuffled pages); rows past a sequence's length are NaN."""
    held = [-(-n // size) for n in lens]
    pages, cols = sum(held) + extra, max(1, max(held) + 1)
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    k, v = rand(pages, hkv, size, D, seed=seed), rand(pages, hkv, size, D, seed=seed + 1)
    table, at = [], 0
    for n, h in zip(lens, held):
        mine = order[at:at + h]
        at += h
        if n % size:
            k[mine[-1], :, n % size:] = float("nan")
            v[mine[-1], :, n % size:] = float("nan")
        table.append(mine + [-1] * (cols - h))
    for p in order[at:]:
        k[p], v[p] = float("nan"), float("nan")
    return rand(len(lens), hq, D, seed=seed + 2), k, v, table


def run_paged(q, k, v, table, lens, max_len=None, want=0):
    b, hq, _ = q.shape
    shape = mp.PagesShape(b, hq, k.shape[1], D, k.shape[0], k.shape[2], len(table[0]))
    max_len = max(lens) if max_len is None else max_len
    out = torch.full((b, hq, D), 7.0, device="cuda")
    lse = torch.full((b, hq), 7.0, device="cuda")
    ws = torch.full((max(16, mp.paged_workspace_bytes(shape, max_len)),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN words
    st = status_word()
    mp.paged_attend(shape, q.cuda(), k.cuda(), v.cuda(), i32(table), i32(lens), max_len, out, lse, ws, status=st)
    torch.cuda.synchronize()
    assert st.item() == want
    return out.cpu(), lse.cpu()


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (3, 1), (8, 2), (5, 1), (6, 1), (7, 1), (8, 1)])
def test_paged_groups(hq, hkv):
    lens = [0, 1, 15, 16, 17, 64, 65, 500]
    q, k, v, table = paged_case(lens, hq, hkv, 16, seed=20 + hq)
    out, lse = run_paged(q, k, v, table, lens)
    check_paged(q, k, v, table, lens, out, lse)


@pytest.mark.parametrize("size", [1, 3, 8, 16, 24, 64, 100, 700])
def test_paged_page_sizes(size):
    lens = [130, 0, 333, 1, 64, 699]
    q, k, v, table = paged_case(lens, 8, 2, size, seed=30 + size)
    out, lse = run_paged(q, k, v, table, lens)
    check_paged(q, k, v, table, lens, out, lse)


def test_paged_long_and_short_together():
    """One long sequence cut into many runs beside short and empty ones."""
    lens = [3, 0, 30011, 1, 0, 77]
    q, k, v, table = paged_case(lens, 4, 1, 32, seed=40)
    out, lse = run_paged(q, k, v, table, lens, max_len=30048)
    check_paged(q, k, v, table, lens, out, lse)


@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [0] * 40 + [1], [5] * 300])
def test_paged_few_tokens(lens):
    """No token at all, fewer blocks than runs, more sequences than a warp looks at in a step."""
    q, k, v, table = paged_case(lens, 2, 1, 16, seed=50 + len(lens))
    for max_len in (max(lens), max(16, max(lens))):
        out, lse = run_paged(q, k, v, table, lens, max_len=max_len)
        check_paged(q, k, v, table, lens, out, lse)


def test_paged_no_workspace_for_no_tokens():
    """max_len 0 needs no workspace: an empty tensor (null) does."""
    q, k, v, table = paged_case([0, 0], 4, 2, 16, seed=55)
    shape = mp.PagesShape(2, 4, 2, D, k.shape[0], 16, len(table[0]))
    assert mp.paged_workspace_bytes(shape, 0) == 0
    out, lse = torch.full((2, 4, D), 7.0, device="cuda"), torch.full((2, 4), 7.0, device="cuda")
    mp.paged_attend(shape, q.cuda(), k.cuda(), v.cuda(), i32(table), i32([0, 0]), 0, out, lse,
                    torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_paged_moving_maximum():
    n = 900
    q, k, v, table = paged_case([n], 4, 1, 16, seed=60)
    q = q.abs()
    for c, p in enumerate(table[0]):
        if p >= 0:
            k[p] = (k[p].float().abs() * (c * 16 / n * 8)).bfloat16()
    out, lse = run_paged(q, k, v, table, [n])
    check_paged(q, k, v, table, [n], out, lse)


def test_paged_bad_pages_left_out():
    """Page numbers outside the pool: their tokens do not count and the call says so; a length past max_len is cut."""
    lens = [100, 64, 33]
    q, k, v, table = paged_case(lens, 4, 2, 16, seed=70)
    table[0][2], table[1], table[2][1] = -1, [k.shape[0]] * len(table[1]), 1 << 30
    out, lse = run_paged(q, k, v, table, lens, want=mp.MP_ERR_CAPACITY)
    check_paged(q, k, v, table, lens, out, lse)
    q, k, v, table = paged_case([100, 20], 4, 2, 16, seed=71)
    out, lse = run_paged(q, k, v, table, [100, 20], max_len=50, want=mp.MP_ERR_CAPACITY)
    check_paged(q, k, v, table, [50, 20], out, lse)


@pytest.mark.parametrize("n", [1, 40, 5000])
def test_paged_not_finite(n):
    """What is not finite and seen reaches the results of its head, and of no other: a query of NaN, a key, a value."""
    lens = [n, 77]
    q, k, v, table = paged_case(lens, 4, 2, 16, seed=75)
    want, want_lse = run_paged(q, k, v, table, lens)
    bad = q.clone()
    bad[0, 1, 5] = float("nan")  # every score of the row
    out, lse = run_paged(bad, k, v, table, lens)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    rest = [0, 2, 3]
    assert torch.equal(out[0, rest], want[0, rest]) and torch.equal(out[1], want[1]) and torch.equal(lse[1], want_lse[1])
    page, row = table[0][(n - 1) // 16], (n - 1) % 16
    for x in ("nan", "inf"):
        bad = k.clone()
        bad[page, 1, row, 7] = float(x)
        bq = q.clone()
        bq[0, 2:, 7] = 1.0
        out, lse = run_paged(bq, bad, v, table, lens)
        assert torch.isnan(out[0, 2:]).all() and not torch.isfinite(lse[0, 2:]).any()
        assert torch.equal(out[0, :2], want[0, :2]) and torch.equal(out[1], want[1])
    bad = v.clone()
    bad[page, 0, row, 9] = float("nan")
    out, lse = run_paged(q, k, bad, table, lens)
    assert torch.isnan(out[0, :2, 9]).all() and torch.equal(lse, want_lse)
    out[0, :2, 9] = want[0, :2, 9]
    assert torch.equal(out, want)


def test_paged_reads_the_contiguous_cache():
    """The cache of the sampled decode, [B][Hkv][Ncap][d], as one page a sequence: with every token in the exact set
    D the two decodes are the same attention."""
    B, Hq, Hkv, cap, n = 2, 8, 2, 512, [300, 411]
    q, W = rand(B, Hq, D, seed=80), rand(75 * 8, D, seed=81).cuda()
    k, v = rand(B, Hkv, cap, D, seed=82), rand(B, Hkv, cap, D, seed=83)
    dk, dv, dq, lens = k.cuda(), v.cuda(), q.cuda(), i32(n)
    shape = mp.Shape(B, Hq, Hkv, D, cap, 8, 75, 4, cap)  # a window over everything
    codes = torch.zeros(mp.codes_shape(shape)[1], dtype=torch.uint8, device="cuda")
    out = torch.zeros(B, Hq, D, device="cuda")
    lse, ns = torch.zeros(B, Hq, device="cuda"), i32([[0] * Hq] * B)
    ws = torch.empty(mp.decode_workspace_bytes(shape, cap), dtype=torch.uint8, device="cuda")
    mp.decode_attend(shape, dq, W, codes, dk, dv, lens, cap, out, lse, ns, ws)
    torch.cuda.synchronize()
    table = [[0], [1]]
    got, got_lse = run_paged(q, k, v, table, n, max_len=cap)
    check_paged(q, k, v, table, n, got, got_lse)
    # decode_attend's own bars: 2e-3 relative L2, 1e-3 on lse
    assert (got - out.cpu()).norm() / got.norm() <= 2e-3 and (got_lse - lse.cpu()).abs().max() <= 1e-3


def test_paged_two_streams_and_graphs():
    """Two captured steps with a workspace each, replayed at the same time on two streams."""
    cases = []
    for j in range(2):
        lens = [700 + 300 * j, 65, 2000]
        q, k, v, table = paged_case(lens, 8, 2, 16, seed=90 + j)
        shape = mp.PagesShape(3, 8, 2, D, k.shape[0], 16, len(table[0]))
        t = dict(q=q.cuda(), k=k.cuda(), v=v.cuda(), table=i32(table), lens=i32(lens),
                 out=torch.zeros(3, 8, D, device="cuda"), lse=torch.zeros(3, 8, device="cuda"),
                 ws=torch.empty(mp.paged_workspace_bytes(shape, 2000), dtype=torch.uint8, device="cuda"))
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            mp.paged_attend(shape, t["q"], t["k"], t["v"], t["table"], t["lens"], 2000, t["out"], t["lse"], t["ws"])
        cases.append((q, k, v, table, lens, t, st, g))
    for _ in range(5):
        for *_, st, g in cases:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for q, k, v, table, lens, t, _, _ in cases:
        check_paged(q, k, v, table, lens, t["out"].cpu(), t["lse"].cpu())


# ------------------------------------------------------- pages and the append ----

class Cache:
    """A paged cache on the GPU beside its model, with every token's rows kept on the host."""

    def __init__(self, batch, n_pages, size, cols, hkv=2, hq=4):
        self.shape = mp.PagesShape(batch, hq, hkv, D, n_pages, size, cols)
        self.m = Pages(batch, n_pages, size, cols)
        self.table, self.lens, self.refs = i32(self.m.table), i32(self.m.lens), i32(self.m.refs)
        self.k = torch.full((n_pages, hkv, size, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.rows = [(torch.zeros(0, hkv, D, dtype=torch.bfloat16),) * 2 for _ in range(batch)]
        self.seed = 0

    def check(self):
        torch.cuda.synchronize()
        assert self.table.cpu().tolist() == self.m.table
        assert self.lens.cpu().tolist() == self.m.lens
        assert self.refs.cpu().tolist() == self.m.refs
        k, v = self.k.cpu(), self.v.cpu()
        for b, n in enumerate(self.m.lens):
            for u in range(self.shape.n_kv_heads):
                assert torch.equal(gather(k, self.m.table[b], n, u), self.rows[b][0][:, u]), b
                assert torch.equal(gather(v, self.m.table[b], n, u), self.rows[b][1][:, u]), b

    def reserve(self, new):
        st = status_word()
        mp.pages_reserve(self.shape, i32(new), self.table, self.lens, self.refs, status=st)
        ok = self.m.reserve(new)
        assert (st.item() == 0) == ok and (ok or st.item() == mp.MP_ERR_CAPACITY)
        return ok

    def append(self, new):
        self.seed += 1
        n, hkv = sum(new), self.shape.n_kv_heads
        k, v = rand(n, hkv, D, seed=self.seed), rand(n, hkv, D, seed=self.seed + 500)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        st = status_word()
        one = all(x == 1 for x in new)
        mp.paged_append(self.shape, k.cuda(), v.cuda(), self.table, self.lens, self.k, self.v,
                        cu_new=None if one else i32(cu), status=st)
        assert st.item() == 0
        for b, x in enumerate(new):
            self.rows[b] = tuple(torch.cat((old, t[cu[b]:cu[b + 1]])) for old, t in zip(self.rows[b], (k, v)))
            self.m.lens[b] += x

    def copy(self, copies, want):
        torch.cuda.synchronize()
        got = copies.cpu().tolist()
        assert got[0] == [len(want), 0, 0, 0] and [tuple(e[:3]) for e in got[1:1 + len(want)]] == want
        mp.pages_copy(self.shape, copies, self.k, self.v)

    def fork(self, src, dst):
        copies = torch.full((1 + len(src), 4), -5, dtype=torch.int32, device="cuda")
        st = status_word()
        mp.pages_fork(self.shape, i32(src), i32(dst), self.table, self.lens, self.refs, copies, status=st)
        want = self.m.fork(src, dst)
        assert (st.item() == 0) == (want is not None)
        self.copy(copies, want or [])
        if want is not None:
            for a, b in zip(src, dst):
                self.rows[b] = self.rows[a]
        return st.item()

    def free(self, seqs):
        st = status_word()
        mp.pages_free(self.shape, i32(seqs), self.table, self.lens, self.refs, status=st)
        self.m.free(seqs)
        assert st.item() == 0
        for b in seqs:
            self.rows[b] = tuple(t[:0] for t in self.rows[b])

    def compact(self):
        copies = torch.full((1 + self.shape.n_pages // 2, 4), -5, dtype=torch.int32, device="cuda")
        st = status_word()
        mp.pages_compact(self.shape, self.table, self.refs, copies, status=st)
        self.copy(copies, self.m.compact())
        assert st.item() == 0


@pytest.mark.parametrize("batch,n_pages,size,cols", [(4, 9, 4, 5), (7, 40, 1, 30), (40, 300, 16, 9), (9, 5000, 3, 700),
                                                     (300, 2000, 8, 40), (3, 64, 100, 33)])
def test_pages_random_life(batch, n_pages, size, cols):
    """Random turns of every operation, compared with the model after each."""
    c, r = Cache(batch, n_pages, size, cols), random.Random(batch * 1000 + size)
    for turn in range(14):
        what = r.choice(("grow", "grow", "step", "fork", "free", "compact")) if turn else "grow"
        empty = [b for b in range(batch) if c.m.table[b][0] < 0]
        full = [b for b in range(batch) if c.m.lens[b] > 0]
        if what in ("grow", "step"):
            most = max(1, min(cols * size, n_pages * size * 2 // batch) // 3)
            new = [1] * batch if what == "step" else [r.choice((0, 1, r.randint(0, most))) for _ in range(batch)]
            if c.reserve(new) and sum(new):
                c.append(new)
        elif what == "fork" and empty and full:
            dst = r.sample(empty, r.randint(1, len(empty)))
            c.fork([r.choice(full) for _ in dst], dst)
        elif what == "free" and full:
            gone = r.sample(full, r.randint(1, len(full)))
            c.free((gone + gone[:1])[:batch])
        else:
            c.compact()
        c.check()


def test_compact_of_a_large_pool():
    """Every other page free over many runs of the plan; and pools with nothing to move, all free, all used."""
    P = 20000
    shape = mp.PagesShape(100, 4, 1, D, P, 1, 200)
    for used in (lambda p: p % 2, lambda p: p < 777, lambda p: False, lambda p: True, lambda p: p == P - 1):
        m = Pages(100, P, 1, 200)
        m.refs = [int(bool(used(p))) * (1 + p % 3) for p in range(P)]
        pages = [p for p in range(P) if m.refs[p]][:20000]
        m.table = [(pages[b * 200:(b + 1) * 200] + [-1] * 200)[:200] for b in range(100)]
        table, refs = i32(m.table), i32(m.refs)
        copies = torch.zeros(1 + P // 2, 4, dtype=torch.int32, device="cuda")
        mp.pages_compact(shape, table, refs, copies)
        want = m.compact()
        assert table.cpu().tolist() == m.table and refs.cpu().tolist() == m.refs
        got = copies.cpu().tolist()
        assert got[0] == [len(want), 0, 0, 0] and [tuple(e[:3]) for e in got[1:1 + len(want)]] == want


def test_fork_refusals_change_nothing():
    c = Cache(6, 12, 4, 6)
    assert c.reserve([6, 0, 0, 3, 0, 0])
    c.append([6, 0, 0, 3, 0, 0])
    for src, dst in (([0], [6]), ([-1], [1]), ([0], [3]), ([0, 3], [1, 1]), ([0, 1], [1, 2]), ([0], [0])):
        assert c.fork(src, dst) == mp.MP_ERR_ARG
        c.check()
    assert c.reserve([18, 0, 0, 9, 0, 0])  # nothing left but one page
    assert c.fork([0, 3], [1, 2]) in (0, mp.MP_ERR_CAPACITY)
    c.check()


def test_free_and_copy_skip_what_is_wrong():
    c = Cache(3, 8, 4, 4)
    assert c.reserve([8, 4, 0])
    c.append([8, 4, 0])
    st = status_word()
    mp.pages_free(c.shape, i32([7, 1, -1]), c.table, c.lens, c.refs, status=st)
    c.m.free([1])
    c.rows[1] = tuple(t[:0] for t in c.rows[1])
    assert st.item() == mp.MP_ERR_ARG
    c.check()
    st = status_word()
    before = c.k.clone()
    copies = i32([[6, 0, 0, 0], [0, 8, 4, 0], [-1, 5, 4, 0], [0, 5, 5, 0], [0, 5, -1, 0], [0, 6, 3, 0]])  # count past the list
    mp.pages_copy(c.shape, copies, c.k, c.v, status=st)
    assert st.item() == mp.MP_ERR_ARG
    before[6, :, :3] = before[0, :, :3]
    assert torch.equal(c.k.view(torch.int16), before.view(torch.int16))


def test_append_without_pages():
    """Rows whose page is missing are not written, recorded, and the length stays; the other sequences' rows go in."""
    c = Cache(3, 6, 4, 3)
    assert c.reserve([4, 4, 0])
    k, v = rand(9, 2, D, seed=1), rand(9, 2, D, seed=2)
    st = status_word()
    mp.paged_append(c.shape, k.cuda(), v.cuda(), c.table, c.lens, c.k, c.v, cu_new=i32([0, 6, 9, 9]), status=st)
    assert st.item() == mp.MP_ERR_CAPACITY
    c.m.lens[1] = 3
    c.rows[1] = (k[6:9], v[6:9])
    c.check()
    st = status_word()
    mp.paged_append(c.shape, k[:3].cuda(), v[:3].cuda(), c.table, c.lens, c.k, c.v, status=st)  # one row each
    assert st.item() == mp.MP_ERR_CAPACITY  # the third sequence holds no page
    c.m.lens[0], c.m.lens[1] = 1, 4
    c.rows[0], c.rows[1] = (k[:1], v[:1]), tuple(torch.cat((x, y[1:2])) for x, y in zip(c.rows[1], (k, v)))
    c.check()


@pytest.mark.parametrize("cu", [[0, 6, 4, 9], [0, 6, 9, 10], [-1, 3, 6, 9]])
def test_append_with_entries_out_of_order(cu):
    """Rows that two sequences claim, or rows past the last one: recorded, and no sequence grows."""
    c = Cache(3, 12, 4, 3)
    assert c.reserve([9, 9, 9])
    k, v = rand(9, 2, D, seed=5), rand(9, 2, D, seed=6)
    st = status_word()
    mp.paged_append(c.shape, k.cuda(), v.cuda(), c.table, c.lens, c.k, c.v, cu_new=i32(cu), status=st)
    assert st.item() == mp.MP_ERR_CAPACITY and c.lens.tolist() == [0, 0, 0]
    c.check()


def test_append_for_several_layers():
    """advance=False leaves the lengths: two layers share table and lengths; rows come out of a fused projection."""
    c = Cache(2, 8, 16, 3, hkv=3, hq=6)
    assert c.reserve([20, 5])
    one = rand(25, 6, D, seed=3).cuda()
    k2, v2 = c.k.clone(), c.v.clone()
    cu = i32([0, 20, 25])
    mp.paged_append(c.shape, one[:, :3], one[:, 3:], c.table, c.lens, k2, v2, cu_new=cu, advance=False)
    mp.paged_append(c.shape, one[:, 3:], one[:, :3], c.table, c.lens, c.k, c.v, cu_new=cu)
    c.m.lens = [20, 5]
    h = one.cpu()
    c.rows = [(h[:20, 3:], h[:20, :3]), (h[20:, 3:], h[20:, :3])]
    c.check()
    c.k, c.v, c.rows = k2, v2, [(b, a) for a, b in c.rows]
    c.check()


def test_pages_past_32_bits():
    """Pools of more than 2^31 elements: append, decode, fork and copy on their last pages."""
    hkv, size, P = 8, 16, 131100
    assert (P - 9) * hkv * size * D > 1 << 31
    shape = mp.PagesShape(3, 16, hkv, D, P, size, 4)
    kp, vp = (torch.empty(P, hkv, size, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    refs = torch.ones(P, dtype=torch.int32, device="cuda")
    refs[-9:] = 0
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    lens = i32([0, 0, 0])
    mp.pages_reserve(shape, i32([40, 9, 0]), table, lens, refs)
    assert table.tolist()[0][:3] == [P - 9, P - 8, P - 7] and table.tolist()[1][0] == P - 6
    k, v, q = rand(49, hkv, D, seed=130), rand(49, hkv, D, seed=131), rand(3, 16, D, seed=132)
    mp.paged_append(shape, k.cuda(), v.cuda(), table, lens, kp, vp, cu_new=i32([0, 40, 49, 49]))
    copies = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    mp.pages_fork(shape, i32([0]), i32([2]), table, lens, refs, copies)
    mp.pages_copy(shape, copies, kp, vp)
    assert lens.tolist() == [40, 9, 40] and table.tolist()[2] == [P - 9, P - 8, P - 5, -1]
    out, lse = torch.empty(3, 16, D, device="cuda"), torch.empty(3, 16, device="cuda")
    ws = torch.empty(mp.paged_workspace_bytes(shape, 64), dtype=torch.uint8, device="cuda")
    mp.paged_attend(shape, q.cuda(), kp, vp, table, lens, 64, out, lse, ws)
    at = table.cpu()
    local = torch.where(at >= 0, at - (P - 9), at)  # the last 9 pages as a pool of their own
    check_paged(q, kp[-9:].cpu(), vp[-9:].cpu(), local.tolist(), [40, 9, 40], out.cpu(), lse.cpu())


# ------------------------------------------------------------- a run of all ----

def test_serving_run():
    """As a server uses them: prompts attended and stored, forked, decoded step by step, some ended, the pool brought
    together, decoding on; every result against the tokens that the sequences hold."""
    hq, hkv, size = 8, 2, 16
    c = Cache(6, 60, size, 12, hkv=hkv, hq=hq)
    new = [37, 100, 1, 0, 0, 0]
    assert c.reserve(new)
    q, k, v, cu = prompt_case(new, hq, hkv, seed=500)
    out, lse = run_prompt(q, k, v, cu, fused=True)
    check_prompt(q, k, v, cu, out, lse)
    mp.paged_append(c.shape, k.cuda(), v.cuda(), c.table, c.lens, c.k, c.v, cu_new=i32(cu))
    c.m.lens = list(new)
    c.rows = [(k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]) for b in range(6)]
    c.check()
    assert c.fork([1, 0], [3, 4]) == 0
    max_len = 12 * size
    ws = torch.empty(mp.paged_workspace_bytes(c.shape, max_len), dtype=torch.uint8, device="cuda")
    for step in range(24):
        if step == 10:
            c.free([1, 2])
            c.check()
        if step == 15:
            c.compact()
            c.check()
        new = [int(n > 0) for n in c.m.lens]
        assert c.reserve(new)
        c.append(new)
        q = rand(6, hq, D, seed=600 + step)
        out, lse = torch.empty(6, hq, D, device="cuda"), torch.empty(6, hq, device="cuda")
        mp.paged_attend(c.shape, q.cuda(), c.k, c.v, c.table, c.lens, max_len, out, lse, ws)
        torch.cuda.synchronize()
        check_paged(q, c.k.cpu(), c.v.cpu(), c.m.table, c.m.lens, out.cpu(), lse.cpu())
    c.check()


@pytest.mark.parametrize("packed", [False, True])
def test_serving_step_captured(packed):
    """A step of two layers (pages, rows and attention of each, lengths at the end) captured once and replayed without
    a pause: the tokens, pages and results are those of the same calls made one by one."""
    batch, hq, hkv, size, cols, steps = 5, 8, 2, 16, 9, 40
    layers, max_len = 2, cols * size
    shape = mp.PagesShape(batch, hq, hkv, D, batch * cols, size, cols)
    new = [1, 0, 1, 3, 1] if packed else [1] * batch  # tokens a step
    n = sum(new)
    cu = i32([sum(new[:b]) for b in range(batch + 1)]) if packed else None
    feed = [[rand(n, 2 * hkv, D, seed=700 + 10 * t + i).cuda() for i in range(layers)] for t in range(steps)]
    asks = [rand(batch, hq, D, seed=2000 + t).cuda() for t in range(steps)]

    def fresh():
        return dict(table=torch.full((batch, cols), -1, dtype=torch.int32, device="cuda"), lens=i32([0] * batch),
                    refs=i32([0] * batch * cols), new=i32(new), grown=i32([0] * batch), q=asks[0].clone(), kv=[x.clone() for x in feed[0]],
                    pools=[[torch.full((batch * cols, hkv, size, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                            for _ in range(2)] for _ in range(layers)],
                    out=torch.zeros(layers, batch, hq, D, device="cuda"), lse=torch.zeros(layers, batch, hq, device="cuda"),
                    ws=torch.empty(mp.paged_workspace_bytes(shape, max_len), dtype=torch.uint8, device="cuda"),
                    st=status_word())

    def step(c, pause):
        def then(f, *args, **kw):
            f(*args, **kw, status=c["st"])
            if pause:
                torch.cuda.synchronize()
        then(mp.pages_reserve, shape, c["new"], c["table"], c["lens"], c["refs"])
        torch.add(c["lens"], c["new"], out=c["grown"])  # what a layer attends to, its new rows with it
        for i, (k, v) in enumerate(c["pools"]):
            then(mp.paged_append, shape, c["kv"][i][:, :hkv], c["kv"][i][:, hkv:], c["table"], c["lens"], k, v, cu_new=cu,
                 advance=i == layers - 1)
            then(mp.paged_attend, shape, c["q"], k, v, c["table"], c["grown"], max_len, c["out"][i], c["lse"][i], c["ws"])

    def give(c, t):
        c["q"].copy_(asks[t])
        for x, y in zip(c["kv"], feed[t]):
            x.copy_(y)

    one, rep, results = fresh(), fresh(), []
    step(fresh(), False)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(rep, False)
    for t in range(steps):
        give(rep, t)
        g.replay()
        results.append((rep["out"].clone(), rep["lse"].clone(), rep["lens"].clone()))
    torch.cuda.synchronize()
    for t in range(steps):
        give(one, t)
        step(one, True)
        for x, y in zip(results[t], (one["out"], one["lse"], one["lens"])):
            assert torch.equal(x, y), t
    assert one["st"].item() == 0 and rep["st"].item() == 0
    lens = [x * steps for x in new]
    assert one["lens"].tolist() == lens and torch.equal(one["table"], rep["table"]) and torch.equal(one["refs"], rep["refs"])
    for i, (k, v) in enumerate(one["pools"]):
        assert torch.equal(torch.nan_to_num(k), torch.nan_to_num(rep["pools"][i][0]))
        assert torch.equal(torch.nan_to_num(v), torch.nan_to_num(rep["pools"][i][1]))
    for i, (k, v) in enumerate(one["pools"]):
        check_paged(asks[-1].cpu(), k.cpu(), v.cpu(), one["table"].tolist(), lens, one["out"][i].cpu(), one["lse"][i].cpu())
