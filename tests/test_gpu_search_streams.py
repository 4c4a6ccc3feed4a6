"""A search that is made on one stream and run on another."""
import pytest
import torch

import rans_entropy_coding_b200 as rb

pytestmark = pytest.mark.gpu


def test_a_search_made_behind_other_work_on_another_stream():
    texts, beams, v, steps = 4, 3, 500, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(steps, texts * beams, v, device="cuda", generator=g)
    plain = rb.BeamSearch(texts, beams, steps)
    for row in x:
        plain.step(row)
    want = plain.results(beams)
    a, out = torch.randn(4096, 4096, device="cuda"), torch.empty(4096, 4096, device="cuda")
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = [torch.full((texts, beams, steps), 7, dtype=torch.int32, device="cuda")
            for _ in range(8)]
    del junk  # (what the search's memory holds before it is written)
    torch.cuda.synchronize()
    for _ in range(20):  # some 30 ms on the stream on which the search is made
        torch.mm(a, a, out=out)
    search = rb.BeamSearch(texts, beams, steps)  # (ends would be copied, and waited for)
    for row in x:
        search.step(row, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    for p, q in zip(want, search.results(beams)):
        assert torch.equal(p, q)
