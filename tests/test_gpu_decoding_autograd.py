"""What the decoding steps write in place, as autograd sees it: a tensor that a
backward pass needs as it was, and one that requires grad."""
from __future__ import annotations

import pytest

from lower_convex_hull_amd import iso
from tests.test_decoding_abi import _Fake


def test_an_array_that_requires_grad_is_refused():
    import torch

    leaf = torch.zeros(6, 4, 5, requires_grad=True)
    for t in (leaf, leaf * 2, leaf[1:]):
        with pytest.raises(ValueError, match="require grad"):
            iso._blocks(_Fake(), [torch.zeros(t.shape), t], 0, t.shape[0])
        with torch.no_grad():
            assert iso._blocks(_Fake(), t, 0, t.shape[0])[1] == 1
    assert iso._blocks(_Fake(), leaf.detach(), 0, 6)[1] == 1


@pytest.fixture(scope="module")
def torch():
    import torch as t

    assert t.cuda.is_available()
    iso.lib()
    return t


def calls(torch):
    """Each call over a state or pool of 6 rows of 4 x 5."""
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    yield lambda s: iso.beam_reorder(s, i(1, 0, 2, 3, 5, 4).view(2, 3))
    yield lambda s: iso.pages_fork(i(0).view(1, 1), i(3), i(1, 0, 0, 0, 0, 0), i(0, 0), page_size=4, pools=s)
    yield lambda s: iso.pages_compact(i(5), i(0, 0, 0, 0, 0, 1), pools=s)


@pytest.mark.gpu
@pytest.mark.parametrize("several", [False, True])
def test_a_backward_pass_that_saved_a_written_tensor_raises(torch, several):
    for call in calls(torch):
        state = torch.randn(6, 4, 5, device="cuda")
        weight = torch.ones(6, 4, 5, device="cuda", requires_grad=True)
        loss = (state * weight).sum()  # keeps the state for the weight's gradient
        before = state._version
        call([torch.zeros(6, 4, 5, device="cuda"), state] if several else state)
        assert state._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        # one that only reads it afterwards is right
        (state * weight).sum().backward()
        assert torch.equal(weight.grad, state)


@pytest.mark.gpu
def test_tensors_that_require_grad(torch):
    for call in calls(torch):
        leaf = torch.randn(6, 4, 5, device="cuda", requires_grad=True)
        keep = leaf.detach().clone()
        for t in (leaf, leaf * 1):
            with pytest.raises(ValueError, match="require grad"):
                call(t)
        assert torch.equal(leaf, keep)
        with torch.no_grad():
            call(leaf)
        assert not torch.equal(leaf, keep)
    with torch.inference_mode():
        state = torch.randn(6, 4, 5, device="cuda")
        for call in calls(torch):
            call(state)
