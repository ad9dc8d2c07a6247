"""Exact attention and the paged cache, host side only: arguments at the limits of what the binding passes on."""
import copy
import pickle

import pytest
import torch

import lsh_sampled_sparse_simhash_b200 as mp
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
