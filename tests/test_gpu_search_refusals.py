"""A search's step that is refused leaves the search as it was."""
import pytest
import torch

import rans_entropy_coding_b200 as rb

pytestmark = pytest.mark.gpu


def test_a_refused_step_changes_nothing():
    texts, beams, v = 2, 3, 50
    search = rb.BeamSearch(texts, beams, 5, ends=[1])
    x = torch.randn(texts * beams, v, device="cuda")
    search.step(x)
    kept = [p.clone() for p in search._parts]
    good = torch.zeros(texts * beams, 4, 3, device="cuda")
    odd = torch.zeros(texts * beams, 8, device="cuda")
    lengths = torch.zeros(texts, dtype=torch.int32, device="cuda")
    for kw in (dict(states=[good[:-1]]), dict(states=[good.cpu()]),
               dict(states=[good.transpose(1, 2)]),
               dict(states=[good], axis=3), dict(states=[good], lengths=lengths),
               dict(states=[good], lengths=lengths.long(), axis=1),
               dict(states=[good], axis=[1, 1]),
               dict(states=good, status=torch.zeros(2, device="cuda")),
               dict(states=[good, good]), dict(states=[odd[:, :5], odd[:, 4:]]),
               dict(states=[search.parents.view(-1, 1)]),
               dict(states=[lengths.repeat(3).view(-1, 1)[:, :0], good, good])):
        with pytest.raises((ValueError, rb.RansError)):
            search.step(x, **kw)
        for a, b in zip(kept, search._parts):
            assert torch.equal(a, b)
    search.step(x, states=[odd[:, :4], odd[:, 4:], good])
    assert search.lengths.tolist() == [2, 2]


def test_the_check_alone():
    parents = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    x = torch.arange(12.0, device="cuda").view(6, 2)
    assert rb.rans_reorder_states_check([x], parents, None, None, None) == rb.OK
    assert rb.rans_reorder_states_check([x, x], parents, None, None, None) == rb.ERR_ARG
    assert rb.rans_reorder_states_check([], parents, None, None, None) == rb.OK
    assert x.flatten().tolist() == list(range(12))
