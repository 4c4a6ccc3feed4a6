"""Tokens under a model's logits on the GPU, where the two sides of a call
meet: numbers against rows that hold them, lists and logits at the ends of
float32, streams other than the tensors' own, rows of several tables and rings
that refill, and decoders under offsets that lie."""
import math

import numpy as np
import pytest
import torch

import rans_entropy_coding_b200 as rb
import token_oracle as TO
from test_gpu_tokens import (BF16, F16, F32, TYPES, U, check_adjusted, check_distill, coded,
                             make_adjust, make_logits, numpy_rows, status_ok, teacher)

pytestmark = pytest.mark.gpu


def rows32(n, x):
    return torch.full((n,), x, device="cuda", dtype=F32)


# ------------------------------------------------------------ adjustments --
@pytest.mark.parametrize("T", [0.55, 0.85, 1.1, 1.45, 1.95])
def test_texts_coded_under_a_number_decode_under_rows_of_it(T):
    """A server codes one text under its temperature and decodes it in a batch
    whose rows bring their own."""
    n, v, length = 3, 5000, 12
    x = make_logits(length, v, F32, seed=31)
    tok = torch.randint(0, v, (n, length), device="cuda",
                        generator=torch.Generator("cuda").manual_seed(31))
    c = rb.TokenCoder()
    one = rb.LogitAdjust(temperature=T, repetition=1.1, frequency=0.3, presence=0.2)
    for k in range(n):
        c.add(x, tok[k], one)
    data, offs = c.streams([length] * n)
    many = rb.LogitAdjust(temperature=rows32(n, T), repetition=rows32(n, 1.1),
                          frequency=0.3, presence=rows32(n, 0.2))
    assert torch.equal(rb.adjust_logits(x[:n], one), rb.adjust_logits(x[:n], many))
    every = torch.arange(v, dtype=torch.int32, device="cuda")
    row = x[:1].expand(v, v).contiguous()
    a = rb.token_intervals(row, every, one)
    b = rb.token_intervals(row, every, rb.LogitAdjust(temperature=rows32(v, T)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.begin(data, offs)
    for t in range(length):
        got = c.step(x[t:t + 1].expand(n, v).contiguous(), many)
        assert got.tolist() == tok[:, t].tolist()
    c.finish()
