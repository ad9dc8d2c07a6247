"""Exact attention and the paged cache, host side only: what the C entry points refuse before anything is launched,
the binding's checks of its tensors, and the references that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import lsh_sampled_sparse_simhash_b200 as mp
from lsh_sampled_sparse_simhash_b200 import _binding as B
from exact_ref import Pages, attend, check_head

A = 1 << 12  # aligned fake device pointers (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return mp.library()


def prompt_shape(**kw):
    d = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, total=100, q_stride=0, k_stride=0, v_stride=0)
    d.update(kw)
    return ctypes.byref(B._CPromptShape(*d.values()))


def pages_shape(**kw):
    d = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, n_pages=10, page_size=16, max_pages=5)
    d.update(kw)
    return ctypes.byref(B._CPagesShape(*d.values()))


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(head_dim=64), dict(n_q_heads=7), dict(n_q_heads=18), dict(n_kv_heads=0), dict(total=-1),
    dict(total=1 << 28), dict(q_stride=1000), dict(q_stride=1028), dict(k_stride=264 - 16), dict(v_stride=257),
    dict(q_stride=-8)])
def test_prompt_shapes_refused(lib, bad):
    assert lib.mp_prompt_attend(prompt_shape(**bad), A, A, A, A, A, A, None, None) == mp.MP_ERR_SHAPE


def test_prompt_batch_limit(lib):
    assert lib.mp_prompt_attend(prompt_shape(batch=65537), A, A, A, A, A, A, None, None) == mp.MP_ERR_SHAPE
    assert lib.mp_prompt_attend(prompt_shape(batch=65536, total=0), None, None, None, A, None, None, None, None) == mp.MP_OK


def test_prompt_pointers_refused(lib):
    good = [A, A, A, A, A, A, None, None]
    for i in (0, 1, 2, 3, 4):
        assert lib.mp_prompt_attend(prompt_shape(), *[None if j == i else x for j, x in enumerate(good)]) == mp.MP_ERR_ARG
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 2), (4, 8), (5, 2), (6, 2)):
        assert lib.mp_prompt_attend(prompt_shape(), *[(x or A) + off if j == i else x for j, x in enumerate(good)]) \
            == mp.MP_ERR_ALIGN, i
    assert lib.mp_prompt_attend(None, *good) == mp.MP_ERR_ARG
    assert lib.mp_prompt_attend(prompt_shape(total=0), None, None, None, A, None, None, None, None) == mp.MP_OK


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(batch=4097), dict(head_dim=256), dict(n_q_heads=9), dict(n_q_heads=20), dict(n_pages=0),
    dict(n_pages=(1 << 24) + 1), dict(page_size=0), dict(page_size=1 << 24), dict(max_pages=0),
    dict(max_pages=1 << 20, page_size=1 << 12), dict(batch=4096, n_q_heads=16, n_kv_heads=16)])
def test_pages_shapes_refused(lib, bad):
    n = ctypes.c_size_t()
    s = pages_shape(**bad)
    assert lib.mp_paged_workspace_bytes(s, 10, ctypes.byref(n)) == mp.MP_ERR_SHAPE
    assert lib.mp_paged_attend(s, A, A, A, A, A, 10, A, A, A, 1 << 30, None, None) == mp.MP_ERR_SHAPE
    assert lib.mp_paged_append(s, A, A, 0, 0, A, 10, 1, A, A, A, A, None, None) == mp.MP_ERR_SHAPE
    assert lib.mp_pages_reserve(s, A, A, A, A, None, None) == mp.MP_ERR_SHAPE
    assert lib.mp_pages_fork(s, A, A, 1, A, A, A, A, None, None) == mp.MP_ERR_SHAPE
    assert lib.mp_pages_free(s, A, 1, A, A, A, None, None) == mp.MP_ERR_SHAPE
    assert lib.mp_pages_compact(s, A, A, A, None, None) == mp.MP_ERR_SHAPE
    assert lib.mp_pages_copy(s, A, 1, A, A, None, None) == mp.MP_ERR_SHAPE


def test_paged_attend_refusals(lib):
    s, n = pages_shape(), ctypes.c_size_t()
    assert lib.mp_paged_workspace_bytes(s, 81, ctypes.byref(n)) == mp.MP_ERR_CAPACITY
    assert lib.mp_paged_workspace_bytes(s, -1, ctypes.byref(n)) == mp.MP_ERR_CAPACITY
    assert lib.mp_paged_workspace_bytes(s, 80, None) == mp.MP_ERR_ARG
    assert lib.mp_paged_workspace_bytes(s, 80, ctypes.byref(n)) == mp.MP_OK and n.value > 0
    need = n.value
    assert lib.mp_paged_workspace_bytes(s, 0, ctypes.byref(n)) == mp.MP_OK and n.value == 0
    f, good = lib.mp_paged_attend, [A, A, A, A, A, 80, A, A, A, need, None, None]
    for i in (0, 1, 2, 3, 4, 6, 7, 8):
        assert f(s, *[None if j == i else x for j, x in enumerate(good)]) == mp.MP_ERR_ARG, i
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 2), (4, 2), (6, 8), (7, 2), (8, 8), (10, 2)):
        assert f(s, *[(x or A) + off if j == i else x for j, x in enumerate(good)]) == mp.MP_ERR_ALIGN, i
    assert f(s, *[81 if j == 5 else x for j, x in enumerate(good)]) == mp.MP_ERR_CAPACITY
    assert f(s, *[need - 1 if j == 9 else x for j, x in enumerate(good)]) == mp.MP_ERR_WORKSPACE


def test_append_refusals(lib):
    s, f = pages_shape(), lib.mp_paged_append
    good = [A, A, 0, 0, A, 10, 1, A, A, A, A, None, None]
    for i in (0, 1, 7, 8, 9, 10):
        assert f(s, *[None if j == i else x for j, x in enumerate(good)]) == mp.MP_ERR_ARG, i
    for i, off in ((0, 8), (1, 8), (4, 2), (7, 2), (8, 2), (9, 8), (10, 8), (11, 2)):
        assert f(s, *[(x or A) + off if j == i else x for j, x in enumerate(good)]) == mp.MP_ERR_ALIGN, i
    assert f(s, *[None if j == 4 else x for j, x in enumerate(good)]) == mp.MP_ERR_ARG  # one row a sequence: n_rows == batch
    assert f(s, *[-1 if j == 5 else x for j, x in enumerate(good)]) == mp.MP_ERR_ARG
    assert f(s, *[0 if j == 5 else x for j, x in enumerate(good)]) == mp.MP_OK          # nothing to do
    assert f(s, *[128 if j == 2 else x for j, x in enumerate(good)]) == mp.MP_ERR_SHAPE  # shorter than a token
    assert f(s, *[260 if j == 3 else x for j, x in enumerate(good)]) == mp.MP_ERR_SHAPE  # not a multiple of 8


def test_page_operation_refusals(lib):
    s = pages_shape()
    assert lib.mp_pages_reserve(s, None, A, A, A, None, None) == mp.MP_ERR_ARG
    assert lib.mp_pages_reserve(s, A, A, A + 1, A, None, None) == mp.MP_ERR_ALIGN
    for n in (0, -1, 3):
        assert lib.mp_pages_fork(s, A, A, n, A, A, A, A, None, None) == mp.MP_ERR_ARG
        assert lib.mp_pages_free(s, A, n, A, A, A, None, None) == mp.MP_ERR_ARG
    assert lib.mp_pages_fork(s, A, A, 1, A, A, A, A + 8, None, None) == mp.MP_ERR_ALIGN
    assert lib.mp_pages_fork(s, A, A, 1, A, A, A, None, None, None) == mp.MP_ERR_ARG
    assert lib.mp_pages_free(s, None, 1, A, A, A, None, None) == mp.MP_ERR_ARG
    assert lib.mp_pages_compact(s, A, None, A, None, None) == mp.MP_ERR_ARG
    assert lib.mp_pages_compact(s, A, A, A + 4, None, None) == mp.MP_ERR_ALIGN
    assert lib.mp_pages_copy(s, A, -1, A, A, None, None) == mp.MP_ERR_ARG
    assert lib.mp_pages_copy(s, A + 4, 1, A, A, None, None) == mp.MP_ERR_ALIGN
    assert lib.mp_pages_copy(s, A, 0, A, A, None, None) == mp.MP_OK


def test_binding_refuses_host_tensors():
    """The binding raises before the library is called for tensors that are not on the GPU."""
    t = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B._rows_arg(t, "q", torch.bfloat16, (1, 8, 128), 0)
    with pytest.raises(ValueError):
        B._arg(t, "out", torch.bfloat16, (1, 8, 128), 0)


def test_reference_bounds_hold_for_rounded_weights():
    """The bounds of exact_ref accept bf16 weights and refuse a wrong mask."""
    torch.manual_seed(1)
    q, k, v = (torch.randn(40, 128).bfloat16() for _ in range(3))
    seen = torch.arange(1, 41)
    ref = attend(q, k, v, seen)
    s = (q.float() @ k.float().T / math.sqrt(128)).masked_fill(torch.arange(40)[None] >= seen[:, None], -math.inf)
    p = torch.exp(s - s.amax(1, keepdim=True))
    out = (p.bfloat16().float() @ v.float() / p.sum(1, keepdim=True)).bfloat16()
    check_head(out, torch.logsumexp(s, 1), ref, seen, True)
    with pytest.raises(AssertionError):
        check_head(out, None, attend(q, k, v, (seen - 1).clamp(min=1)), seen, True)


def test_pages_model():
    m = Pages(4, 8, 4, 4)
    assert m.reserve([6, 0, 1, 0]) and m.table[0][:3] == [0, 1, -1] and m.table[2][0] == 2
    m.lens = [6, 0, 1, 0]
    assert m.fork([0, 0], [1, 3]) == [(1, 3, 2), (1, 4, 2)] and m.refs == [3, 1, 1, 1, 1, 0, 0, 0]
    assert m.fork([0], [1]) is None
    m.free([0, 0, 2])
    assert m.refs == [2, 0, 0, 1, 1, 0, 0, 0]
    assert m.compact() == [(3, 1, 4), (4, 2, 4)] and m.refs == [2, 1, 1, 0, 0, 0, 0, 0]
    assert m.table[1] == [0, 1, -1, -1] and m.table[3] == [0, 2, -1, -1]
    assert not m.reserve([0, 40, 0, 0])
