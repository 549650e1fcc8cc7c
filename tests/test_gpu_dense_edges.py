"""Edges of the dense path on the GPU, each against the 64-bit oracle or exact arithmetic.

Bounds are those of test_gpu_dense (check_logprobs).
"""
import math

import pytest
import torch

import binary_rank_linear_lb_b200 as lb
from test_gpu_dense import BF16, F16, F32, check_logprobs, normal, random_tokens

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ alternatives of rows with NaN
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,vocab", [(9, 5), (9, 32), (9, 4001), (9, 70001), (170, 4099), (700, 2003),
                                        (2400, 1000)])
def test_nan_at_token_0(rows, vocab, dtype):
    """NaN comes before everything, token 0's first of all; no id is made up.  Split rows
    (few of them, long), and 64, 128 and 256 threads a row."""
    x = (normal((rows, vocab), 5) * 3).to(dtype)
    x[0, 0] = math.nan                                # alone
    x[1] = math.nan                                   # nothing else: ids 0, 1, 2, ...
    x[2, 0] = x[2, vocab - 1] = math.nan              # in the first and the last part of a row
    x[3] = -math.inf
    x[3, 0] = math.nan
    x[4] = math.inf
    x[4, 0] = math.nan
    x[5, vocab // 2:] = math.nan                      # not at 0, and parts of NaN only
    x[6, 0], x[6, 1] = math.inf, math.nan
    x[7, 0] = -math.nan                               # the other sign
    t = random_tokens(rows, vocab, 3)
    for top in {1, 2, min(5, vocab), min(32, vocab)}:
        r = lb.token_logprobs(x, t, top)
        assert (r.top_id >= 0).all() and (r.top_id < vocab).all()
        check_logprobs(r, x, t, top, (rows, vocab, dtype, top))


def test_a_token_whose_scale_is_nan_through_the_chain():
    """A stream with an infinity: NaN logits, alternatives 0, 1, 2, ... and NaN for them."""
    h, w = normal((3, 256), 1), normal((40, 256), 2)
    h[1, 7] = math.inf
    r = lb.Head(*lb.quantize_rows(w)).logprobs(h, random_tokens(3, 40, 3), top=32)
    assert torch.equal(r.top_id[1], torch.arange(32, device="cuda")) and r.top_logprob[1].isnan().all()
    assert r.top_logprob[[0, 2]].isfinite().all()
