"""Edges of the dense path on the GPU, each against the 64-bit oracle or exact arithmetic.

Bounds are those of test_gpu_dense (check_codes, check_linear, check_logprobs).
"""
import ctypes
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import binary_rank_linear_lb_b200 as lb
from oracle import dense
from test_gpu_dense import (BF16, F16, F32, check_codes, check_linear, check_logprobs, codes, f64, normal, pitched,
                            random_tokens, scales)

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


# ------------------------------------------------------------ codes on a border, 48-bit products
def exact_codes(s, w):
    """rint(127 s w / max|s w|) of whole numbers, ties to even, in integers."""
    v = [int(a) * int(b) for a, b in zip(s, w)]
    peak = max(abs(a) for a in v)
    out = []
    for a in v:
        k, rest = divmod(254 * abs(a) + peak, 2 * peak)       # floor(quotient + 1/2)
        k -= rest == 0 and k % 2                              # a tie: the even one
        out.append(k if a >= 0 else -k)
    return out


@pytest.mark.parametrize("cols", [7, 700, 5000, 40000])
def test_ties_of_fp32_products(cols):
    """v = (2 k + 1) peak / 254 exactly, with products of up to 48 bits: 127 v needs more
    than the 53 bits of a double.  And products one 2^-48 beside such a tie."""
    rng = np.random.default_rng(cols)
    for m in range(1, 254, 2 if cols < 5000 else 14):
        u = int(rng.integers(1 << 15, 66000)) | 1
        w0 = m * u + 2 if m > 126 else int(rng.integers(1 << 23, 1 << 24)) | 1
        s = np.zeros(cols, dtype=np.int64)
        w = np.full(cols, w0, dtype=np.int64)
        s[0] = 254 * u
        s[1:4] = m * u, -m * u, m * u + 1
        if m > 126:                                           # (m u + a)(w0 - a) = m u w0 + 2 a - a^2
            s[4:6] = m * u + 1, m * u + 3
            w[4:6] = w0 - 1, w0 - 3
        s[6] = m * u
        s[7:] = rng.integers(0, 127, max(cols - 7, 0)) * 2 * u   # (small: whole codes)
        s[cols - 1] = m * u
        x = torch.tensor(np.stack([s, -s]), dtype=F32, device="cuda") * 2.0 ** -24
        q, _, _ = lb.rmsnorm_quantize(x, torch.tensor(w, dtype=F32, device="cuda") * 2.0 ** -23)
        want = exact_codes(s, w)
        assert q[0].tolist() == want and q[1].tolist() == [-c for c in want], m


# ------------------------------------------------------------ head: batches, streams, types
def tiny_head(vocab=500, hidden=256, norm=True):
    return lb.Head(*lb.quantize_rows(normal((vocab, hidden), 71)),
                   normal((hidden,), 72, F16) if norm else None)


@pytest.mark.parametrize("norm", [True, False])
def test_head_of_a_batch_of_sequences(norm):
    """(batch, sequence, hidden) streams are batch * sequence tokens, in order."""
    head, h = tiny_head(norm=norm), normal((3, 5, 256), 73)
    t = random_tokens(15, 500, 74)
    want = head.logits(h.reshape(15, 256))
    assert torch.equal(head.logits(h), want) and want.shape == (15, 500)
    assert torch.equal(head.logits(h.transpose(0, 1)), head.logits(h.transpose(0, 1).reshape(15, 256)))
    for a, b in zip(head.logprobs(h, t.view(3, 5), 4), head.logprobs(h.reshape(15, 256), t, 4)):
        assert torch.equal(a, b)
    # one token in any shape, as ever
    assert torch.equal(head.logits(h[0, 0]), head.logits(h[0, :1]))
    assert torch.equal(head.logits(h[0, 0].view(1, 4, 64)), head.logits(h[0, :1]))
    for bad in (normal((2, 512), 1), normal((2, 3, 128), 1), normal((512,), 1), normal((3, 4, 1), 1)):
        with pytest.raises(ValueError):
            head.logits(bad)


def test_head_copies_what_it_reshapes_on_the_given_stream():
    """A strided token or batch, written on the stream that is given: read after that, not
    before."""
    head, side = tiny_head(), torch.cuda.Stream()
    src, t = normal((64, 256, 64), 75), random_tokens(64 * 64, 500, 78)
    slow = torch.empty(1 << 28, device="cuda")
    for pick in (lambda h: h[3:4, :16, :16].transpose(1, 2), lambda h: h[3, :, 5], lambda h: h.transpose(1, 2)):
        tokens = t[:1] if pick(src).numel() == 256 else t.view(64, 64).t()
        want = head.logprobs(pick(src).contiguous().view(-1, 256), tokens.reshape(-1), 3)
        for call in (lambda h: (head.logits(h, stream=side),), lambda h: head.logprobs(h, tokens, 3, side)):
            h = torch.zeros_like(src)
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                for _ in range(20):
                    slow.fill_(1.0)                   # some 3 ms before h is written
                h.copy_(src)
            got = call(pick(h))
            side.synchronize()
            if len(got) == 1:
                got = lb.token_logprobs(got[0], tokens.reshape(-1), 3)
            for a, b in zip(got, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_head_logprobs_of_logits_of_a_type(dtype):
    head, h, t = tiny_head(), normal((9, 256), 76), random_tokens(9, 500, 77)
    x = head.logits(h, dtype=dtype)
    r = head.logprobs(h, t, 5, dtype=dtype)
    check_logprobs(r, x, t, 5, dtype)
    for a, b in zip(r, lb.token_logprobs(x, t, 5)):
        assert torch.equal(a, b)


# ------------------------------------------------------------ a refused launch leaves no trace
def test_a_refused_launch_is_not_reported_by_the_next_call():
    """While a blocking stream is captured, CUDA refuses launches on the legacy stream with an
    error code.  The call returns it; calls after it do not."""
    rt = ctypes.CDLL("libcudart.so.12")               # (the one torch has loaded)
    x, latent = normal((4, 64), 1), normal((64, 64), 2)
    q, scale = torch.empty((4, 64), dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    words = lb.pack_signs(latent, axis=1)
    y, t = normal((4, 64), 3), torch.zeros(4, dtype=torch.int64, device="cuda")
    ent, out = torch.empty(4, device="cuda"), torch.empty((4, 4), device="cuda")
    L, p = lb.lib(), lambda a: a.data_ptr()
    calls = [
        lambda: L.lb_quantize_rows(p(x), lb.LB_F32, 4, 64, 64, p(q), 64, p(scale), None),
        lambda: L.lb_linear_int8(p(q), 64, p(scale), 4, p(q), 64, p(scale), 64, 4, p(out), lb.LB_F32, 4, None),
        lambda: L.lb_linear_int8(p(q), 64, p(scale), 1, p(q), 64, p(scale), 64, 4, p(out), lb.LB_F32, 4, None),
        lambda: L.lb_linear_int8(p(q) + 1, 65, p(scale), 3, p(q) + 1, 65, p(scale), 63, 3, p(out), lb.LB_F32, 4,
                                 None),
        lambda: L.lb_token_logprobs(p(y), lb.LB_F32, 4, 64, 64, None, None, p(ent), 0, None, None, None)]
    for call in calls:
        assert call() == lb.LB_OK
    for call in calls:
        torch.cuda.synchronize()
        s, g = ctypes.c_void_p(), ctypes.c_void_p()
        assert rt.cudaStreamCreate(ctypes.byref(s)) == 0
        assert rt.cudaStreamBeginCapture(s, 0) == 0   # global: other streams' unsafe calls fail
        try:
            status = call()
        finally:
            rt.cudaStreamEndCapture(s, ctypes.byref(g))   # (invalidated: no graph)
            rt.cudaGetLastError()                     # torch's own runtime is left as it was
            rt.cudaStreamDestroy(s)
        assert status == lb.LB_ERR_CUDA
        assert torch.equal(lb.pack_signs(latent, axis=1), words)


# ------------------------------------------------------------ the ends of the ranges
def test_the_widest_rows():
    """2^24 columns: quantised, and scored with 32 alternatives."""
    n = 1 << 24
    x = normal((2, n), 81)
    check_codes(*lb.quantize_rows(x), dense.quantize(f64(x)), "2^24")
    t = random_tokens(2, n, 82)
    check_logprobs(lb.token_logprobs(x, t, 32), x, t, 32, "2^24")


@pytest.mark.parametrize("M,k,n", [(1 << 20, 16, 3), (3, 16, 1 << 20), (1, 32, (1 << 20) + 1), (1 << 20, 16, 1),
                                   (1 << 18, 17, 5), (300, 131071, 260)])
def test_linear_of_many_tokens_or_channels(M, k, n):
    xq, wq = pitched(codes(M, k, 1), k if k == 17 else None), pitched(codes(n, k, 2), k if k == 17 else None)
    xs, ws = scales(M, 3), scales(n, 4)
    check_linear(lb.linear_int8(xq, xs, wq, ws), xq, xs, wq, ws, (M, k, n))


@pytest.mark.parametrize("M,k", [(1, 17), (2, 17), (5, 129), (300, 4097)])
def test_linear_of_one_channel_of_any_length(M, k):
    """A single channel's pitch is its length, off 16 bytes or not."""
    xq, wq = pitched(codes(M, k, 1)), codes(1, k, 2)
    xs, ws = scales(M, 3), scales(1, 4)
    check_linear(lb.linear_int8(xq, xs, wq, ws), xq, xs, wq, ws, (M, k))


def test_many_short_rows():
    x = normal((1 << 20, 5), 83, BF16)
    check_codes(*lb.quantize_rows(x), dense.quantize(f64(x)), "rows")
    t = random_tokens(1 << 17, 5, 84)
    check_logprobs(lb.token_logprobs(x[:1 << 17], t, 5), x[:1 << 17], t, 5, "rows")


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing has been loaded or asked for yet when the calls are captured."""
    code = '''
import torch, binary_rank_linear_lb_b200 as lb
h = torch.randn(24, 512, device="cuda")
w = torch.randint(-127, 128, (3000, 512), device="cuda").to(torch.int8)
ws, t = torch.rand(3000, device="cuda"), torch.zeros(24, dtype=torch.int64, device="cuda")
head, g = lb.Head(w, ws), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    r = head.logprobs(h, t, 5)
    one = head.logits(h[0])
g.replay()
torch.cuda.synchronize()
for a, b in zip(r, head.logprobs(h, t, 5)):
    assert torch.equal(a, b)
assert torch.equal(one, head.logits(h[0]))
print("done")
'''
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


def test_calls_of_several_threads_at_once():
    head, hs = tiny_head(), [normal((7 + i, 256), 90 + i) for i in range(4)]
    want = [head.logprobs(h, top=4) for h in hs]
    torch.cuda.synchronize()
    got = [[] for _ in hs]

    def work(i):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        for _ in range(50):
            got[i].append(head.logprobs(hs[i], top=4, stream=s))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for a, b in zip(want, got):
        assert len(b) == 50
        for r in b:
            assert all(torch.equal(u, v) for u, v in zip(a[1:], r[1:]))


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("cols", [5, 333, 777, 5001, 8192, 34567])
def test_one_buffer_as_x_residual_and_sum(dtype, cols):
    x, w = normal((5, cols), 95, dtype), normal((cols,), 96, F16)
    want = (x.double() * 2).to(dtype)
    q, s, total = lb.rmsnorm_quantize(x, w, x, sum_out=x)
    assert total is x and torch.equal(x, want)
    check_codes(q, s, dense.rmsnorm_quantize(f64(want), f64(w)), cols)


def test_default_stream_by_handle_and_from_a_side_stream():
    head, h, side = tiny_head(), normal((6, 256), 97), torch.cuda.Stream()
    want = head.logprobs(h, top=3)
    torch.cuda.synchronize()
    for arg in (0, torch.cuda.default_stream()):
        for here in (torch.cuda.default_stream(), side):
            with torch.cuda.stream(here):
                got = head.logprobs(h, top=3, stream=arg)
            torch.cuda.synchronize()
            for a, b in zip(got[1:], want[1:]):
                assert torch.equal(a, b)


def test_captured_with_a_stream_argument_that_is_joined():
    head, h, side = tiny_head(), normal((6, 256), 98), torch.cuda.Stream()
    head.logprobs(h, top=3)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        h2 = h * 2
        side.wait_stream(main)
        r = head.logprobs(h2, top=3, stream=side)
        main.wait_stream(side)
        out = [t.clone() for t in r[1:]]
    for seed in (1, 2):
        h.copy_(normal((6, 256), seed))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, head.logprobs(h * 2, top=3)[1:]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scales_past_the_range_of_fp32(dtype):
    """A norm of one value among 65536 is 256 times its weight; a row's peak can be fp32's
    smallest step."""
    x = torch.zeros((2, 65536), dtype=dtype, device="cuda")
    x[0, 5] = x[1, 9] = 1.0
    w = torch.ones(65536, device="cuda")
    w[5] = 3e38
    q, s, _ = lb.rmsnorm_quantize(x, w, eps=0.0)
    assert s[0] == math.inf and abs(float(s[1]) / (256 / 127) - 1) < 1e-6
    assert q[0, 5] == q[1, 9] == 127 and q.count_nonzero() == 2
    x = torch.zeros((1, 300), dtype=F32, device="cuda")
    x[0, 7] = 2.0 ** -149
    q, s = lb.quantize_rows(x)
    assert s[0] == 0 and q[0, 7] == 127 and q.count_nonzero() == 1
