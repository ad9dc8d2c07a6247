"""Cases of the exact-attention operators: causal attention over packed prompts, decode attention over a paged
key-value cache, the append of new rows into pages, and the operations on the pages themselves.

Each case is one pass of one of them as a serving program makes it.  With `own` false the pass is computed in its
plain form (elementary torch operations, 32-bit arithmetic, one rounding at the end), with `own` true by the
library's calls.  `exact` states the same results in 64 bits from the definitions, sequence by sequence.

Notation: T token rows, B sequences (rows of the page table), Hq query heads in groups of G = Hq / Hkv, head size 128,
pages of S tokens, pools [pages][Hkv][S][128].
"""
import math
import random

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
MU_NORM = 8.0      # keys share a mean of this norm per kv head, as in the ragged workloads
HEADS = ((32, 8), (32, 8), (16, 16), (16, 2), (12, 4), (8, 1))


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # a short chat turn: one prompt, all latency
        dict(name="prompt short", op="prompt", hq=32, hkv=8, batch=1, lo=37, hi=37, mix=0, fused=True, pad=0),
        # prompts of many users packed into one batch, read out of a fused projection, rows behind the last one unused
        dict(name="prompt packed", op="prompt", hq=32, hkv=8, batch=16, lo=64, hi=2048, mix=1, fused=True, pad=100),
        # many tiny prompts of odd lengths down to one token, three query heads to a kv head
        dict(name="prompt tiny g3", op="prompt", hq=12, hkv=4, batch=24, lo=1, hi=700, mix=2, fused=False, pad=0),
        # one long-context prompt (a 16k-token layer with 32 query and 8 kv heads)
        dict(name="prompt 16k", op="prompt", hq=32, hkv=8, batch=1, lo=16384, hi=16384, mix=0, fused=True, pad=0),
        # decode for one user with a 16k-token context: few rows, the length has to be split
        dict(name="paged one 16k", op="paged", hq=32, hkv=8, batch=1, lo=16384, hi=16384, page=64, mix=0),
        # decode for a batch of chats, some just started (length 0), one query head to a kv head
        dict(name="paged chats", op="paged", hq=16, hkv=16, batch=64, lo=0, hi=900, page=32, mix=3),
        # decode over long ragged contexts in small pages (16 sequences of 32k to 131k tokens)
        dict(name="paged ragged16", op="paged", hq=32, hkv=8, batch=16, lo=32768, hi=131072, page=16, mix=4),
        # one decode step's new rows
        dict(name="append step", op="append", hq=32, hkv=8, batch=64, lo=0, hi=2000, page=16, new_lo=1, new_hi=1, mix=5,
             fused=False),
        # packed prompts into their pages, read out of a fused projection
        dict(name="append prompts", op="append", hq=32, hkv=8, batch=12, lo=0, hi=500, page=64, new_lo=100, new_hi=4000,
             mix=6, fused=True),
        # parallel sampling: each of 8 prompts forked, half of the table's rows filled by it
        dict(name="fork samples", op="fork", hq=32, hkv=8, batch=64, lo=100, hi=8000, page=64, live=8, forks=32, mix=7),
        # a fragmented pool of 16-token pages brought together
        dict(name="compact pool", op="compact", hq=32, hkv=8, batch=128, lo=1, hi=600, page=16, live=96, mix=8),
        # finished sequences give their pages back and others take pages for their next tokens
        dict(name="turnover", op="turnover", hq=32, hkv=8, batch=256, lo=1, hi=16000, page=16, live=256, ends=40,
             new_lo=1, new_hi=64, mix=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "prompt", "paged", "paged", "paged", "append", "fork", "compact", "turnover"))
    hq, hkv = rng.choice(HEADS)
    c = dict(op=op, hq=hq, hkv=hkv, mix=rng.randrange(1 << 20))
    if op == "prompt":
        hi = _log(rng, 1, 12000)
        batch = max(1, min(_log(rng, 1, 32), 16384 // hi))
        c.update(batch=batch, lo=max(1, hi // rng.choice((1, 4, 40))), hi=hi, fused=rng.random() < 0.5,
                 pad=rng.choice((0, 0, 3, 130)))
    elif op == "paged":
        hi = _log(rng, 1, 120000)
        batch = max(1, min(_log(rng, 1, 64), (1 << 20) // hi))
        c.update(batch=batch, lo=max(0, hi // rng.choice((1, 3, 30)) - 1), hi=hi,
                 page=rng.choice((8, 16, 24, 32, 64, 128, 256)))
    elif op == "append":
        new_hi = rng.choice((1, 1, _log(rng, 2, 4000)))
        c.update(batch=_log(rng, 1, 128) if new_hi == 1 else _log(rng, 1, max(2, 32768 // new_hi // 4)), lo=0,
                 hi=_log(rng, 1, 3000), page=rng.choice((8, 16, 24, 32, 64, 128)), new_lo=min(new_hi, 1 + new_hi // 10),
                 new_hi=new_hi, fused=rng.random() < 0.5)
    elif op == "fork":
        live = _log(rng, 1, 16)
        forks = _log(rng, 1, 48)
        c.update(batch=live + forks + rng.randrange(8), lo=1, hi=_log(rng, 2, 8000),
                 page=rng.choice((8, 16, 24, 32, 64, 128)), live=live, forks=forks)
    elif op == "compact":
        batch = _log(rng, 4, 160)
        c.update(batch=batch, lo=1, hi=_log(rng, 2, 600), page=rng.choice((8, 16, 24, 32)), live=1 + batch * 3 // 4)
    else:
        batch = _log(rng, 4, 400)
        c.update(batch=batch, lo=1, hi=_log(rng, 2, 16000), page=rng.choice((8, 16, 24, 32, 64)), live=batch,
                 ends=1 + batch // rng.choice((3, 7, 20)), new_lo=1, new_hi=rng.choice((1, 8, 500)))
    return c


# ------------------------------------------------ what a case alone decides ----

def _ints(case, tag, n, lo, hi):
    """n whole numbers of [lo, hi], the same for every seed (so that the work of a case is known)."""
    r = random.Random("%s %s" % (case["mix"], tag))
    return [r.randint(lo, hi) for _ in range(n)]


def _lens(case):
    n = _ints(case, "lens", case["batch"], case["lo"], case["hi"])
    return [x if i < case.get("live", case["batch"]) else 0 for i, x in enumerate(n)]


def _new(case):
    return _ints(case, "new", case["batch"], case["new_lo"], case["new_hi"])


def _held(case):
    """Pages that each sequence holds before the pass."""
    s = case["page"]
    if case["op"] == "append":
        return [-(-(n + m) // s) for n, m in zip(_lens(case), _new(case))]
    return [-(-n // s) for n in _lens(case)]


def _sharers(case):
    """compact: every fourth sequence shares its first page with the next one."""
    return [i for i in range(0, case["live"] - 1, 4)] if case["op"] == "compact" else []


def _pairs(case):
    """fork: sources (the live sequences, over and over) and the empty rows that they go to."""
    return [i % case["live"] for i in range(case["forks"])], [case["live"] + i for i in range(case["forks"])]


def _ends(case):
    r = random.Random("%s ends" % case["mix"])
    return r.sample(range(case["batch"]), case["ends"])


def _pool(case):
    """(pages of the pool, columns of the page table)"""
    held, s = _held(case), case["page"]
    total = sum(held)
    if case["op"] == "paged":
        return total + 5, max(1, max(held))
    if case["op"] == "append":
        return total + 3, max(held) + 1
    if case["op"] == "fork":
        return total + case["forks"] + 9, max(held) + 2
    if case["op"] == "compact":
        return total * 3 // 2 + 4, max(held) + 2
    return total + sum(-(-x // s) + 1 for x in _new(case)), max(held) + -(-case["new_hi"] // s) + 1


def work(case):
    hq, hkv, op = case["hq"], case["hkv"], case["op"]
    row = 2 * hkv * D * 2   # K and V of one token
    lens = _lens(case)
    if op == "prompt":
        n = sum(lens)
        return {"bytes": n * (2 * hq * D * 2 + row + 4 * hq), "flops": sum(2 * D * hq * x * (x + 1) for x in lens)}
    if op == "paged":
        return {"bytes": sum(lens) * row + case["batch"] * hq * (2 * D + 4 * D + 4) + 4 * sum(_held(case)),
                "flops": 4 * D * hq * sum(lens)}
    if op == "append":
        return {"bytes": 2 * sum(_new(case)) * row, "flops": 0}
    pages, cols = _pool(case)
    if op == "fork":
        src, _ = _pairs(case)
        s = case["page"]
        return {"bytes": 2 * row * sum(lens[i] % s for i in src) + 4 * pages + sum(16 * -(-lens[i] // s) for i in src),
                "flops": 0}
    if op == "compact":
        table, refs = _tables(case)
        live = sum(r > 0 for r in refs)
        moved = sum(r > 0 for r in refs[live:])
        return {"bytes": 2 * row * case["page"] * moved + 8 * pages + 4 * sum(_held(case)), "flops": 0}
    return {"bytes": 8 * pages + 8 * sum(_held(case)), "flops": 0}


def _tables(case):
    """Page table rows (lists) and reference counts: pages handed out in a shuffled order, -1 behind them."""
    pages, cols = _pool(case)
    order = list(range(pages))
    random.Random("%s pages" % case["mix"]).shuffle(order)
    table, refs, at = [], [0] * pages, 0
    for n in _held(case):
        table.append(order[at:at + n])
        at += n
    for i in _sharers(case):
        if table[i] and table[i + 1]:
            table[i + 1][0] = table[i][0]
    for row in table:
        for p in row:
            refs[p] += 1
    return [row + [-1] * (cols - len(row)) for row in table], refs


# ------------------------------------------------------------------ inputs ----

def _rand(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _keys(gen, heads_at, *shape):
    """Keys N(0, 1) about a mean of norm MU_NORM per kv head (`heads_at`: the heads' place in shape)."""
    mu = torch.randn((shape[heads_at], D), generator=gen, device="cuda")
    mu = mu * (MU_NORM / mu.norm(dim=-1, keepdim=True))
    at = [1] * (len(shape) + 1)
    at[heads_at], at[-1] = shape[heads_at], D
    k = torch.empty(*shape, D, device="cuda", dtype=torch.bfloat16)
    part = max(1, (1 << 26) // max(1, k[0].numel()))
    mu = mu.view(at)
    for i in range(0, shape[0], part):
        k[i:i + part] = torch.randn(k[i:i + part].shape, generator=gen, device="cuda") + mu
    return k


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _rows(gen, case, total, with_q):
    """New tokens' (q,) k and v: views of one fused projection's output, or tensors of their own."""
    hq, hkv = case["hq"] if with_q else 0, case["hkv"]
    q = _rand(gen, total, hq, D)
    k = _keys(gen, 1, total, hkv)
    v = _rand(gen, total, hkv, D)
    if case["fused"]:
        one = torch.cat((q, k, v), dim=1)
        q, k, v = one[:, :hq], one[:, hq:hq + hkv], one[:, hq + hkv:]
    return q, k, v


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, hq, hkv = case["op"], case["hq"], case["hkv"]
    s = dict(case=case, op=op)
    lens = _lens(case)
    if op == "prompt":
        total = sum(lens) + case["pad"]
        q, k, v = _rows(gen, case, total, True)
        for x in (q, k, v):
            x[sum(lens):] = float("nan")   # rows behind the last sequence: memory nobody wrote
        s.update(q=q, k=k, v=v, lens=lens, cu=_i32(_cu(lens)),
                 out=torch.zeros(total, hq, D, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros(total, hq, dtype=torch.float32, device="cuda"))
    else:
        pages, cols = _pool(case)
        table, refs = _tables(case)
        s.update(table=_i32(table), refs=_i32(refs), lens=_i32(lens), max_len=max(lens))
        if op != "turnover":
            s.update(k_pages=_keys(gen, 1, pages, hkv, case["page"]), v_pages=_rand(gen, pages, hkv, case["page"], D))
        if op == "paged":
            s.update(q=_rand(gen, case["batch"], hq, D))
        elif op == "append":
            _, k, v = _rows(gen, case, sum(_new(case)), False)
            s.update(k=k, v=v, one=case["new_hi"] == 1, cu=_i32(_cu(_new(case))), new=_i32(_new(case)))
        elif op == "fork":
            src, dst = _pairs(case)
            s.update(src=_i32(src), dst=_i32(dst))
        elif op == "turnover":
            # which sequences end and how much the others grow differs from seed to seed
            shift = int(seed) % case["batch"]
            s.update(ends=_i32([(e + shift) % case["batch"] for e in _ends(case)]), new=_i32(_new(case)).roll(shift))
    return s


# ------------------------------------------------------------ the operators ----

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _plain_prompt(s):
    q, k, v, out, lse = s["q"], s["k"], s["v"], s["out"], s["lse"]
    hq, hkv = q.shape[1], k.shape[1]
    g = hq // hkv
    at = 0
    for n in s["lens"]:
        qf = q[at:at + n].float().view(n, hkv, g, D).permute(1, 2, 0, 3).reshape(hkv, g * n, D)
        kf = k[at:at + n].float().permute(1, 2, 0)
        vf = v[at:at + n].float().permute(1, 0, 2)
        p = torch.matmul(qf, kf).mul_(SCALE).view(hkv, g, n, n)
        i = torch.arange(n, device=q.device)
        p.masked_fill_(i[None, :] > i[:, None], float("-inf"))
        m = p.amax(-1, keepdim=True)
        p.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(hkv, g * n, n), vf).view(hkv, g, n, D) / l
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, hq, D).to(torch.bfloat16)
        lse[at:at + n] = (m + l.log())[..., 0].permute(2, 0, 1).reshape(n, hq)
        at += n
    return out, lse


def _plain_paged(s):
    q, table, lens = s["q"], s["table"], s["lens"]
    b, hq, _ = q.shape
    hkv = s["k_pages"].shape[1]
    at = table.clamp(min=0).long()
    k = s["k_pages"][at].permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, D).float()
    p = torch.matmul(q.float().view(b, hkv, hq // hkv, D), k.transpose(2, 3)).mul_(SCALE)
    del k
    unseen = torch.arange(p.shape[-1], device=q.device)[None] >= lens[:, None]
    p.masked_fill_(unseen[:, None, None], float("-inf"))
    m = p.amax(-1, keepdim=True)
    p.sub_(m.clamp(min=torch.finfo(torch.float32).min)).exp_()
    l = p.sum(-1, keepdim=True)
    v = s["v_pages"][at].permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, D).float()
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return o.view(b, hq, D), (m + l.log()).view(b, hq)


def _plain_append(s):
    size, n = s["k_pages"].shape[2], s["k"].shape[0]
    seq = torch.repeat_interleave(torch.arange(s["new"].numel(), device="cuda"), s["new"], output_size=n)
    pos = s["lens"].long()[seq] + torch.arange(n, device="cuda") - s["cu"].long()[seq]
    page = s["table"].long()[seq, pos // size]
    s["k_pages"][page, :, pos % size] = s["k"]
    s["v_pages"][page, :, pos % size] = s["v"]
    return s["k_pages"], s["v_pages"], s["lens"] + s["new"]


def _free_first(refs):
    """Page numbers, the free ones first, each kind in order."""
    return torch.argsort((refs != 0).to(torch.int32), stable=True)


def _plain_fork(s):
    table, lens, refs, size = s["table"].clone(), s["lens"].clone(), s["refs"].clone(), s["k_pages"].shape[2]
    src, dst = s["src"].long(), s["dst"].long()
    full, part = lens[src].long() // size, lens[src] % size
    need = part > 0
    fresh = _free_first(refs)[(torch.cumsum(need, 0) - 1).clamp(min=0)]
    cols = torch.arange(table.shape[1], device="cuda")[None]
    rows = table[src]
    last = torch.gather(rows, 1, full[:, None].clamp(max=rows.shape[1] - 1))[:, 0].long()
    shared = cols < full[:, None]
    refs.index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    table[dst] = torch.where(shared, rows, torch.where((cols == full[:, None]) & need[:, None], fresh[:, None].int(),
                                                       torch.full_like(rows, -1)))
    refs[fresh[need]] = 1
    lens[dst] = lens[src]
    to, of = fresh[need], last[need]
    taken = (torch.arange(size, device="cuda")[None] < part[need][:, None])[:, None, :, None]
    s["k_pages"][to] = torch.where(taken, s["k_pages"][of], s["k_pages"][to])
    s["v_pages"][to] = torch.where(taken, s["v_pages"][of], s["v_pages"][to])
    return s["k_pages"], s["v_pages"], table, lens, refs


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    index = torch.arange(refs.numel(), device="cuda")
    used = refs > 0
    live = used.sum()
    of = index[used & (index >= live)]
    to = index[~used & (index < live)]
    where = index.clone()
    where[of] = to
    moved = refs.clone()
    moved[to] = refs[of]
    moved[of] = 0
    s["k_pages"][to] = s["k_pages"][of]
    s["v_pages"][to] = s["v_pages"][of]
    return s["k_pages"], s["v_pages"], torch.where(table >= 0, where[table.clamp(min=0).long()].int(), table), moved


def _plain_turnover(s):
    table, lens, refs, size = s["table"].clone(), s["lens"].clone(), s["refs"].clone(), s["case"]["page"]
    ends = s["ends"].long()
    gone = table[ends]
    gone = gone[gone >= 0].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[ends] = -1
    lens[ends] = 0
    held = (table >= 0).sum(1)
    need = ((lens + s["new"] + size - 1) // size - held).clamp(min=0)
    first = torch.cumsum(need, 0) - need
    cols = torch.arange(table.shape[1], device="cuda")[None] - held[:, None]
    take = (cols >= 0) & (cols < need[:, None])
    page = _free_first(refs)[(first[:, None] + cols)[take]]
    table[take] = page.int()
    refs[page] = 1
    return table, lens, refs


_plain = dict(prompt=_plain_prompt, paged=_plain_paged, append=_plain_append, fork=_plain_fork, compact=_plain_compact,
              turnover=_plain_turnover)


def _shape(s):
    """The problem's shape, made once for the tensors at hand."""
    import lsh_sampled_sparse_simhash_b200 as mp
    c = s["case"]
    if "shape" not in s:
        if c["op"] == "prompt":
            s["shape"] = mp.PromptShape(c["batch"], c["hq"], c["hkv"], D, s["q"].shape[0])
        else:
            s["shape"] = mp.PagesShape(c["batch"], c["hq"], c["hkv"], D, s["refs"].numel(), c["page"], s["table"].shape[1])
    return s["shape"]


def _own_prompt(s):
    import lsh_sampled_sparse_simhash_b200 as mp
    mp.prompt_attend(_shape(s), s["q"], s["k"], s["v"], s["cu"], s["out"], s["lse"])
    return s["out"], s["lse"]


def _own_paged(s):
    import lsh_sampled_sparse_simhash_b200 as mp
    shape, q = _shape(s), s["q"]
    if "workspace" not in s:   # a serving loop keeps it from step to step
        s["workspace"] = torch.empty(mp.paged_workspace_bytes(shape, s["max_len"]), dtype=torch.uint8, device="cuda")
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    mp.paged_attend(shape, q, s["k_pages"], s["v_pages"], s["table"], s["lens"], s["max_len"], out, lse, s["workspace"])
    return out, lse


def _own_append(s):
    import lsh_sampled_sparse_simhash_b200 as mp
    lens = s["lens"].clone()
    mp.paged_append(_shape(s), s["k"], s["v"], s["table"], lens, s["k_pages"], s["v_pages"],
                    cu_new=None if s["one"] else s["cu"])
    return s["k_pages"], s["v_pages"], lens


def _own_fork(s):
    import lsh_sampled_sparse_simhash_b200 as mp
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    copies = torch.empty((1 + s["src"].numel(), 4), dtype=torch.int32, device="cuda")
    mp.pages_fork(_shape(s), s["src"], s["dst"], table, lens, refs, copies)
    mp.pages_copy(_shape(s), copies, s["k_pages"], s["v_pages"])
    return s["k_pages"], s["v_pages"], table, lens, refs


def _own_compact(s):
    import lsh_sampled_sparse_simhash_b200 as mp
    table, refs = s["table"].clone(), s["refs"].clone()
    copies = torch.empty((1 + refs.numel() // 2, 4), dtype=torch.int32, device="cuda")
    mp.pages_compact(_shape(s), table, refs, copies)
    mp.pages_copy(_shape(s), copies, s["k_pages"], s["v_pages"])
    return s["k_pages"], s["v_pages"], table, refs


def _own_turnover(s):
    import lsh_sampled_sparse_simhash_b200 as mp
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    mp.pages_free(_shape(s), s["ends"], table, lens, refs)
    mp.pages_reserve(_shape(s), s["new"], table, lens, refs)
    return table, lens, refs


_own = dict(prompt=_own_prompt, paged=_own_paged, append=_own_append, fork=_own_fork, compact=_own_compact,
            turnover=_own_turnover)


# ------------------------------------------------- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    return _exact[case["op"]](s)


def _exact_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    hq, g = q.shape[1], q.shape[1] // k.shape[1]
    out, lse = s["out"].double(), s["lse"].double()
    for lo, n in zip(_cu(s["lens"]), s["lens"]):
        for h in range(hq):
            kd, vd = k[lo:lo + n, h // g].double(), v[lo:lo + n, h // g].double()
            for a in range(0, n, 4096):
                z = min(n, a + 4096)
                x = q[lo + a:lo + z, h].double() @ kd[:z].T / math.sqrt(D)
                x = x.tril(diagonal=a) + torch.full_like(x, -math.inf).triu(diagonal=a + 1)
                norm = torch.logsumexp(x, dim=1)
                lse[lo + a:lo + z, h] = norm
                out[lo + a:lo + z, h] = torch.exp(x - norm[:, None]) @ vd[:z]
    return out, lse


def _exact_paged(s):
    q, lens, table = s["q"].double(), s["lens"].tolist(), s["table"].tolist()
    b, hq, _ = q.shape
    hkv, size = s["k_pages"].shape[1:3]
    out = torch.zeros(b, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        if n == 0:
            continue
        mine = torch.tensor(table[i][:-(-n // size)], device="cuda")
        for h in range(hkv):
            kd = s["k_pages"][mine, h].reshape(-1, D)[:n].double()
            vd = s["v_pages"][mine, h].reshape(-1, D)[:n].double()
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = q[i, heads] @ kd.T / math.sqrt(D)
            lse[i, heads] = torch.logsumexp(x, dim=1)
            out[i, heads] = torch.softmax(x, dim=1) @ vd
    return out, lse


def _exact_append(s):
    size, lens, new, table = s["case"]["page"], s["lens"].tolist(), s["new"].tolist(), s["table"].tolist()
    at = 0
    for i, n in enumerate(new):
        done = 0
        while done < n:   # run by run of rows inside one page
            off = (lens[i] + done) % size
            m = min(size - off, n - done)
            page = table[i][(lens[i] + done) // size]
            s["k_pages"][page, :, off:off + m] = s["k"][at:at + m].transpose(0, 1)
            s["v_pages"][page, :, off:off + m] = s["v"][at:at + m].transpose(0, 1)
            done += m
            at += m
    return s["k_pages"], s["v_pages"], None


def _exact_fork(s):
    size, lens, table, refs = s["case"]["page"], s["lens"].tolist(), s["table"].tolist(), s["refs"].tolist()
    for a in s["src"].tolist():
        if lens[a] % size:
            page, rows = refs.index(0), lens[a] % size
            refs[page] = 1
            for pool in (s["k_pages"], s["v_pages"]):
                pool[page, :, :rows] = pool[table[a][lens[a] // size], :, :rows]
    return s["k_pages"], s["v_pages"], None, None, None


def _exact_compact(s):
    refs = s["refs"].tolist()
    live = sum(r > 0 for r in refs)
    holes = [p for p in range(live) if refs[p] == 0]
    for to, of in zip(holes, (p for p in range(live, len(refs)) if refs[p] > 0)):
        for pool in (s["k_pages"], s["v_pages"]):
            pool[to] = pool[of]
    return s["k_pages"], s["v_pages"], None, None


_exact = dict(prompt=_exact_prompt, paged=_exact_paged, append=_exact_append, fork=_exact_fork, compact=_exact_compact,
              turnover=lambda s: None)
