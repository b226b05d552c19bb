"""The weights of a HeadNorm: calls go by the addresses of its own tensors."""
import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa


@pytest.mark.parametrize("name", ["q_weight", "k_weight"])
def test_weights_change_in_place_only(name):
    norm = ssa.HeadNorm(torch.ones(128), torch.ones(128), device="cpu")
    was = getattr(norm, name)
    with pytest.raises(AttributeError, match="in place"):
        setattr(norm, name, torch.zeros(128))
    assert getattr(norm, name) is was
    was.fill_(2.0)
    assert norm._ptr == [norm.q_weight.data_ptr(), norm.k_weight.data_ptr()]


def test_the_rest_may_change():
    norm = ssa.HeadNorm(eps=1e-5, device="cpu")
    norm.eps = 1e-6
    assert norm.eps == 1e-6


def test_weights_are_copies():
    w = torch.ones(128)
    norm = ssa.HeadNorm(w, w, device="cpu")
    w.zero_()
    assert (norm.q_weight == 1).all() and (norm.k_weight == 1).all()
