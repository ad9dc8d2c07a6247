"""Exact attention and the paged cache, host side only: arguments at the limits of what the binding passes on."""
import copy
import pickle

import pytest
import torch

import lsh_sampled_sparse_simhash_b200 as mp
from exact_ref import attend, check_head, check_paged, check_prompt
from lsh_sampled_sparse_simhash_b200 import _binding as B

NO_DEVICE = -1  # what get_device() says of a tensor without memory


@pytest.mark.parametrize("stride", [1 << 31, 1 << 32, (1 << 32) + 1024, 1 << 40])
def test_token_strides_past_32_bits_refused(stride):
    """The library takes a 32-bit stride; the low bits of a larger one are another row's place (or 0, side by side)."""
    t = torch.empty_strided((2, 8, 128), (stride, 128, 1), dtype=torch.bfloat16, device="meta")
    assert t.get_device() == NO_DEVICE
    with pytest.raises(ValueError, match="token stride"):
        B._rows_arg(t, "k", torch.bfloat16, (2, 8, 128), NO_DEVICE)


def test_token_strides_of_32_bits_passed_on():
    for stride in (1024, 1032, (1 << 31) - 8):
        t = torch.empty_strided((2, 8, 128), (stride, 128, 1), dtype=torch.bfloat16, device="meta")
        assert B._rows_arg(t, "k", torch.bfloat16, (2, 8, 128), NO_DEVICE)[1] == stride
    one = torch.empty_strided((1, 8, 128), (1 << 32, 128, 1), dtype=torch.bfloat16, device="meta")
    assert B._rows_arg(one, "k", torch.bfloat16, (1, 8, 128), NO_DEVICE)[1] == 0  # one row has no stride


@pytest.mark.parametrize("max_len", [1 << 31, (1 << 32) + 10, -(1 << 32)])
def test_max_len_past_32_bits_refused(max_len):
    with pytest.raises(ValueError, match="max_len"):
        mp.paged_workspace_bytes(mp.PagesShape(2, 8, 2, 128, 10, 16, 5), max_len)


def test_shapes_past_32_bits_refused():
    good = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, n_pages=10, page_size=16, max_pages=5)
    for name in good:
        with pytest.raises(ValueError, match=name):
            mp.PagesShape(**{**good, name: (1 << 32) + good[name]})
    good = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, total=100)
    for name in good:
        with pytest.raises(ValueError, match=name):
            mp.PromptShape(**{**good, name: (1 << 32) + good[name]})


@pytest.mark.parametrize("shape", [mp.PromptShape(2, 8, 2, 128, 100), mp.PagesShape(2, 8, 2, 128, 10, 16, 5)])
def test_shapes_copied_and_pickled(shape):
    """A server sends its shapes to other processes."""
    for other in (copy.copy(shape), copy.deepcopy(shape), pickle.loads(pickle.dumps(shape))):
        assert other == shape and hash(other) == hash(shape)
    if isinstance(shape, mp.PagesShape):
        other = pickle.loads(pickle.dumps(shape))
        assert mp.paged_workspace_bytes(other, 80) == mp.paged_workspace_bytes(shape, 80) > 0


@pytest.mark.parametrize("wrong", [float("nan"), float("inf"), float("-inf"), 0.01, -0.01])
def test_checks_refuse_a_wrong_lse(wrong):
    """The checks that the GPU tests rely on accept the reference's own lse, and no other beside right results."""
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(20, 1, 128, generator=g).bfloat16() for _ in range(3))
    seen = torch.arange(1, 21)
    ref = attend(q[:, 0], k[:, 0], v[:, 0], seen)
    out, lse = ref[0].bfloat16()[:, None], ref[1].float()[:, None]
    bad = lse.clone()
    bad[7] += wrong
    check_head(out[:, 0], lse[:, 0], ref, seen, True)
    check_prompt(q, k, v, [0, 20], out, lse)
    with pytest.raises(AssertionError):
        check_head(out[:, 0], bad[:, 0], ref, seen, True)
    with pytest.raises(AssertionError):
        check_prompt(q, k, v, [0, 20], out, bad)
    pools = [x.transpose(0, 1)[None].contiguous() for x in (k, v)]  # one page of 20 tokens
    one = attend(q[:1, 0], k[:, 0], v[:, 0], torch.tensor([20]))
    out, lse = one[0].float()[None], one[1].float()[None]
    check_paged(q[:1], *pools, [[0]], [20], out, lse)
    with pytest.raises(AssertionError):
        check_paged(q[:1], *pools, [[0]], [20], out, lse + wrong)
