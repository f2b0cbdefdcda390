"""The Python side of the paged calls on the CPU: whose memory they hand to the library."""
import pytest
import torch

import canvas_denoising_denoise_b200 as dg


def tensors(n_pages):
    pages = torch.zeros((n_pages, 2, 16, 64), dtype=torch.uint8)
    exps = torch.zeros((n_pages, 2), dtype=torch.uint8)
    return pages, pages.clone(), exps, exps.clone()


@pytest.mark.parametrize("name", ["k_pages", "v_pages", "k_exp", "v_exp"])
def test_a_caches_tensors_cannot_be_exchanged(name):
    """The calls hand over memory that the constructor has checked: no other tensor takes its place."""
    cache = dg.PagedCache(*tensors(4))
    with pytest.raises(AttributeError):
        setattr(cache, name, getattr(cache, name).clone())


@pytest.mark.parametrize("at", range(4))
def test_a_caches_pointers_follow_its_tensors(at):
    parts = tensors(4)
    cache = dg.PagedCache(*parts)
    assert cache.pointers == tuple(t.data_ptr() for t in parts)
    parts[at].set_(torch.zeros_like(parts[at]).clone())
    assert cache.pointers == tuple(t.data_ptr() for t in parts)
    parts[at].resize_(1 << 20)
    with pytest.raises(ValueError):
        cache.pointers
