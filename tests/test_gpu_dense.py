"""The dense path (8-bit rows, RMS norm, 8-bit linear, log probabilities) on the GPU.

Tolerances, u = 2^-24 (half a step of fp32, relative):
- codes: equal to the 64-bit oracle's (they are those of the exact quotient);
- scales: the mean of squares adds up to 64 squares a thread and 10 levels of a tree
  (under 80 u, halved by the root), then root, quotient and two products: under 64 u;
- y: the sum to fp32 and two products, 3 u, then half a step of y's own type;
- log probabilities: a sum of e^d over V / 256 terms an accumulator (V / 128 where V is at
  most 12288, under 96) and 13 levels, each term off by 4 u and by the rounding of d and of
  its product with log2 e (d up to 30 where e^d counts): (V / 256 + 128) u, and 4 u of the
  value itself; the entropy the same, times 1 + 2 H for its second sum.
"""
import math

import numpy as np
import pytest
import torch

import binary_rank_linear_lb_b200 as lb
from binary_rank_linear_lb_b200 import synth
from binary_rank_linear_lb_b200.configs import Model
from binary_rank_linear_lb_b200.model import build_head, build_stack
from oracle import dense

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
HALF_STEP = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: U}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, seed, dtype=F32):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


def in_pitch(t, ld, lead=0):
    """A copy of t inside a buffer of pitch ld whose other cells are NaN (codes: 77)."""
    fill = 77 if t.dtype == torch.int8 else math.nan     # (never read)
    buf = torch.full((t.shape[0] * ld + lead + 64,), fill, dtype=t.dtype, device="cuda")
    v = buf[lead:lead + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
    v.copy_(t)
    return v


# ------------------------------------------------------------------ quantise
def check_codes(q, scale, ref, what=""):
    rq, rs = ref
    assert np.array_equal(q.cpu().numpy(), rq), f"{what}: codes differ at " \
        f"{np.argwhere(q.cpu().numpy() != rq)[:4].tolist()}"
    got = f64(scale)
    assert np.array_equal(np.isnan(got), np.isnan(rs)), what
    # a scale below fp32's normal range is off by half of its smallest step instead
    ok = np.isnan(rs) | (np.abs(got - rs) <= 64 * U * np.abs(rs) + 2.0 ** -150)
    assert ok.all(), f"{what}: scale {got[~ok][:4]} for {rs[~ok][:4]}"


QSHAPES = [(1, 1), (1, 7), (3, 17), (2, 64), (5, 1000), (7, 2048), (33, 4096), (2, 8191), (1, 8192),
           (3, 28672), (2, 32768), (2, 40001), (1, 70000), (300, 129), (1000, 96), (150, 5120)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", QSHAPES)
def test_quantize_rows(rows, cols, dtype):
    x = normal((rows, cols), rows * 7 + cols, dtype)
    q, s = lb.quantize_rows(x)
    check_codes(q, s, dense.quantize(f64(x)), (rows, cols, dtype))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("ld,lead", [(1001, 0), (1008, 0), (1024, 3), (1007, 1), (1016, 8)])
def test_quantize_rows_pitches(dtype, ld, lead):
    x = in_pitch(normal((9, 1000), 5, dtype), ld, lead)
    buf = torch.full((9 * 1003 + 1,), 99, dtype=torch.int8, device="cuda")
    q = buf[1:].view(9, 1003)[:, :1000]
    scale = torch.empty(9, device="cuda")
    q2, s2 = lb.quantize_rows(x, q=q, scale=scale)
    assert q2 is q and s2 is scale
    check_codes(q, scale, dense.quantize(f64(x)), (ld, lead))
    assert (buf[1:].view(9, 1003)[:, 1000:] == 99).all() and buf[0] == 99


def test_quantize_rows_on_the_border_between_codes():
    """Values on, and one step to either side of, every border between two codes."""
    for peak in (1.0, 254.0, 0.3, 1e-3, 3.1e4):
        peak = float(np.float32(peak))
        v = []
        for k in range(127):
            b = np.float32((k + 0.5) * peak / 127.0)
            v += [b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(1e9)), -b]
        x = torch.tensor([[peak] + [float(f) for f in v]], device="cuda", dtype=F32)
        check_codes(*lb.quantize_rows(x), dense.quantize(f64(x)), f"peak {peak}")
        check_codes(*lb.rmsnorm_quantize(x)[:2], dense.rmsnorm_quantize(f64(x)), f"norm {peak}")
        w = normal((x.shape[1],), 3)
        w[0] = 4.0
        check_codes(*lb.rmsnorm_quantize(x, w)[:2], dense.rmsnorm_quantize(f64(x), f64(w)), f"w {peak}")
    # exact ties of 16-bit inputs: peak 254 puts every odd value on a border
    x = torch.arange(-254, 255, device="cuda").to(F16)[None, :].contiguous()
    check_codes(*lb.quantize_rows(x), dense.quantize(f64(x)), "ties")


def test_codes_of_many_random_quotients():
    """A few quotients in 10^5 lie nearer a border than fp32 can tell."""
    x, w = normal((512, 8192), 11), normal((8192,), 12)
    check_codes(*lb.rmsnorm_quantize(x, w)[:2], dense.rmsnorm_quantize(f64(x), f64(w)), "fp32")


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("cols", [3, 96, 1000, 8192, 40001])
def test_rows_with_nothing_or_too_much(dtype, cols):
    x = normal((8, cols), 3, dtype)
    x[0] = 0.0
    x[1] = -0.0
    x[2, cols // 2] = math.nan
    x[3, cols - 1] = math.inf
    x[4, 0] = -math.inf
    x[5] = 0.0
    x[5, cols - 1] = torch.finfo(dtype).tiny          # one value, the smallest normal one
    x[6] = torch.finfo(dtype).max
    check_codes(*lb.quantize_rows(x), dense.quantize(f64(x)), "rows")
    q, s, _ = lb.rmsnorm_quantize(x, eps=1e-5)
    check_codes(q, s, dense.rmsnorm_quantize(f64(x)), "norm")
    x = x[4:7].contiguous()
    q, s, _ = lb.rmsnorm_quantize(x, eps=0.0)
    check_codes(q, s, dense.rmsnorm_quantize(f64(x), eps=0.0), "norm, eps 0")


@pytest.mark.parametrize("wdtype", [None, F16, BF16, F32])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 8192), (3, 17), (333, 5120), (2, 28673), (1, 1), (4, 33000)])
def test_rmsnorm_quantize(rows, cols, dtype, wdtype):
    x, r = normal((rows, cols), 21, dtype), normal((rows, cols), 22, dtype)
    w = normal((cols,), 23, wdtype) if wdtype is not None else None
    wn = f64(w) if w is not None else None
    q, s, none = lb.rmsnorm_quantize(x, w)
    assert none is None
    check_codes(q, s, dense.rmsnorm_quantize(f64(x), wn), "no residual")
    q, s, total = lb.rmsnorm_quantize(x, w, r, 1e-6)
    assert torch.equal(total, (x.double() + r.double()).to(dtype))
    check_codes(q, s, dense.rmsnorm_quantize(f64(total), wn, 1e-6), "residual")


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("cols", [5, 333, 640, 1027, 5001, 8192, 12345, 34567])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_rmsnorm_quantize_in_place(dtype, cols, into):
    x, r, w = normal((5, cols), 31, dtype), normal((5, cols), 32, dtype), normal((cols,), 33, F16)
    want = (x.double() + r.double()).to(dtype)
    kept = (r if into == "x" else x).clone()
    q, s, total = lb.rmsnorm_quantize(x, w, r, sum_out=x if into == "x" else r)
    assert total is (x if into == "x" else r) and torch.equal(total, want)
    assert torch.equal(r if into == "x" else x, kept)
    check_codes(q, s, dense.rmsnorm_quantize(f64(want), f64(w)), into)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("cols", [7, 200, 777, 2500, 9001])
@pytest.mark.parametrize("lead", range(8))
def test_rmsnorm_quantize_pitches(dtype, cols, lead):
    """Three matrices off 16 bytes by different amounts; nothing beside them is written."""
    x = in_pitch(normal((6, cols), 41, dtype), cols + 2, lead)
    r = in_pitch(normal((6, cols), 42, dtype), cols + 23, 3)
    buf = torch.full((6 * (cols + 9) + 8,), 3.5, device="cuda", dtype=dtype)
    out = buf[5 * lead % 8:][:6 * (cols + 9)].view(6, cols + 9)[:, :cols]
    w = normal((cols + 1,), 43, F16)[1:]
    q, s, total = lb.rmsnorm_quantize(x, w, r, sum_out=out)
    want = (x.double() + r.double()).to(dtype)
    assert torch.equal(total, want)
    check_codes(q, s, dense.rmsnorm_quantize(f64(want), f64(w)), "pitch")
    out.fill_(3.5)
    assert (buf == 3.5).all()


def test_rmsnorm_of_values_whose_squares_leave_fp32():
    for a in (1e25, 1e-25, 3e37, 1e-38):
        x = normal((3, 2000), 51) * a
        for eps in (0.0, 1e-5):
            q, s, _ = lb.rmsnorm_quantize(x, eps=eps)
            check_codes(q, s, dense.rmsnorm_quantize(f64(x), eps=eps), (a, eps))
    x = normal((2, 300), 52) * 1e30
    w = normal((300,), 53) * 1e20                     # products past fp32, results inside it
    q, s, _ = lb.rmsnorm_quantize(x, w)
    check_codes(q, s, dense.rmsnorm_quantize(f64(x), f64(w)), "products")
    x, w = normal((2, 300), 54) * 1e-30, normal((300,), 55) * 1e-20     # and below it
    q, s, _ = lb.rmsnorm_quantize(x, w, eps=0.0)
    check_codes(q, s, dense.rmsnorm_quantize(f64(x), f64(w), eps=0.0), "small products")


# -------------------------------------------------------------------- linear
def codes(rows, cols, seed):
    return torch.randint(-128, 128, (rows, cols), generator=gen(seed), device="cuda",
                         dtype=torch.int64).to(torch.int8)


def pitched(t, ld=None, lead=0):
    return in_pitch(t, ld or (t.shape[1] + 15) // 16 * 16, lead)


def scales(n, seed, size=1.0):
    return (normal((n,), seed).abs() + 0.5) * size


def check_linear(y, xq, xs, wq, ws, what=""):
    ref = dense.linear_int8(f64(xq), f64(xs), f64(wq), f64(ws))
    got = f64(y)
    tol = (3 * U + HALF_STEP[y.dtype]) * np.abs(ref) * (1 + 4 * U)
    if y.dtype == F16:
        tol = tol + 2.0 ** -25                        # half the smallest step of fp16
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {got[bad][:3]} for {ref[bad][:3]} at {np.argwhere(bad)[:3].tolist()}"


LSHAPES = [(1, 1, 1), (1, 16, 128), (1, 4096, 1000), (2, 100, 130), (3, 17, 5), (4, 2048, 4097),
           (5, 333, 257), (7, 1024, 128), (8, 4095, 640), (13, 128, 129), (16, 8192, 300), (17, 64, 70),
           (31, 1000, 1000), (32, 512, 2048), (33, 129, 127), (64, 4096, 512), (65, 127, 300),
           (96, 640, 1111), (127, 256, 255), (128, 1024, 256), (129, 1025, 384), (200, 96, 1000),
           (256, 512, 640), (257, 384, 513), (300, 2048, 129), (333, 1000, 3000), (513, 272, 2049),
           (1000, 160, 1000), (1025, 4096, 300)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,k,n", LSHAPES)
def test_linear_int8(M, k, n, dtype):
    xq, wq = pitched(codes(M, k, M + k)), pitched(codes(n, k, n + k))
    # y of a size that fp16 holds: sums are at most about 2^13 sqrt(k) * 6
    xs, ws = scales(M, 1, 2.0 ** -8), scales(n, 2, 2.0 ** -8)
    y = lb.linear_int8(xq, xs, wq, ws, dtype=dtype)
    assert y.shape == (M, n) and y.dtype == dtype
    check_linear(y, xq, xs, wq, ws, (M, k, n, dtype))


@pytest.mark.parametrize("M", [1, 6, 40, 300])
@pytest.mark.parametrize("ldx,leadx,ldw,leadw", [(1001, 0, 1008, 0), (1008, 0, 1001, 0), (1008, 1, 1008, 0),
                                                 (1008, 0, 1008, 3), (1024, 16, 2048, 32), (1003, 2, 1007, 5)])
def test_linear_int8_pitches(M, ldx, leadx, ldw, leadw):
    xq, wq = in_pitch(codes(M, 1001, 3), ldx, leadx), in_pitch(codes(290, 1001, 4), ldw, leadw)
    xs, ws = scales(M, 5), scales(290, 6)
    buf = torch.full((M + 2, 293), 5.0, device="cuda")
    y = buf[1:M + 1, 1:291]
    assert lb.linear_int8(xq, xs, wq, ws, y=y) is y
    check_linear(y, xq, xs, wq, ws, (M, ldx, ldw))
    edge = buf.clone()
    edge[1:M + 1, 1:291] = 5.0
    assert (edge == 5.0).all()                        # nothing around y was written


@pytest.mark.parametrize("M", [1, 15, 16, 17, 64, 65])
@pytest.mark.parametrize("lead", [0, 1, 2, 3])
def test_linear_int8_off_words(M, lead):
    """Rows that start and end anywhere in a word, around a word's and a stage's end; the
    codes beside them are 77."""
    for k in (1, 2, 3, 4, 5, 63, 64, 65, 66, 127, 128, 129, 131):
        xq, wq = in_pitch(codes(M, k, k), k + 5, (lead + 1) % 4), in_pitch(codes(67, k, k + 1), k + 6, lead)
        xs, ws = scales(M, 5), scales(67, 6)
        check_linear(lb.linear_int8(xq, xs, wq, ws), xq, xs, wq, ws, (M, k, lead))


@pytest.mark.parametrize("M", [1, 4, 16, 130])
def test_linear_int8_largest_sums(M):
    """in = 131071 rows of -128: sums of 2147467264, the largest there are."""
    k = 131071
    xq = pitched(torch.full((M, k), -128, dtype=torch.int8, device="cuda"))
    wq = pitched(torch.full((140, k), -128, dtype=torch.int8, device="cuda"))
    wq[::2] = 127
    xs, ws = scales(M, 7, 2.0 ** -20), scales(140, 8)
    check_linear(lb.linear_int8(xq, xs, wq, ws), xq, xs, wq, ws, M)


@pytest.mark.parametrize("M", [1, 8, 64, 300])
def test_linear_int8_of_rows_without_a_value(M):
    """NaN scales (rows with a NaN or an infinity) give NaN rows and no other."""
    xq, wq, xs, ws = pitched(codes(M, 320, 1)), pitched(codes(200, 320, 2)), scales(M, 3), scales(200, 4)
    xs[M - 1] = math.nan
    ws[77] = math.inf
    y = f64(lb.linear_int8(xq, xs, wq, ws))
    assert np.isnan(y[M - 1]).all() and np.isfinite(np.delete(y[:M - 1], 77, axis=1)).all()
    assert not np.isfinite(y[:, 77]).any()


# -------------------------------------------------------------- logprobs
def check_logprobs(r, x, tokens, top, what=""):
    lp, h, ids, tlp = dense.token_logprobs(f64(x), tokens.cpu().numpy() if tokens is not None else None, top)
    base = (x.shape[1] / 256 + 128) * U

    def close(got, ref, tol, name):
        got = f64(got)
        same = (got == ref) | (np.isnan(got) & np.isnan(ref))
        with np.errstate(invalid="ignore"):
            bad = ~(same | (np.abs(got - ref) <= tol))
        assert not bad.any(), f"{what} {name}: {got[bad][:4]} for {ref[bad][:4]}"

    with np.errstate(invalid="ignore"):
        if tokens is not None:
            close(r.logprob, lp, base + 4 * U * np.abs(lp), "logprob")
        close(r.entropy, h, base * (1 + 2 * h) + 4 * U * h, "entropy")
        if top:
            assert np.array_equal(r.top_id.cpu().numpy(), ids), f"{what}: ids"
            close(r.top_logprob, tlp, base + 4 * U * np.abs(tlp), "top")


def random_tokens(rows, vocab, seed):
    return torch.randint(0, vocab, (rows,), generator=gen(seed), device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (2, 5, 5), (1, 33, 32), (3, 1000, 0), (7, 1001, 20),
                                            (1, 32000, 20), (5, 32000, 1), (160, 4099, 5), (700, 999, 3),
                                            (2, 50257, 32), (1, 128256, 5), (20, 131071, 7), (1, 300001, 32),
                                            (300, 32000, 4), (2500, 1211, 32), (3000, 700, 5), (2400, 31, 31),
                                            (700, 9000, 32), (2400, 5000, 3), (60, 9001, 32)])
def test_token_logprobs(rows, vocab, top, dtype):
    x = (normal((rows, vocab), vocab + rows) * 3).to(dtype)
    t = random_tokens(rows, vocab, 1)
    check_logprobs(lb.token_logprobs(x, t, top), x, t, top, (rows, vocab, top, dtype))


@pytest.mark.parametrize("rows", [1, 9, 400])
@pytest.mark.parametrize("ld,lead", [(5001, 0), (5008, 1), (5003, 7), (6000, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_token_logprobs_pitches(rows, ld, lead, dtype):
    x = in_pitch((normal((rows, 5000), 9) * 2).to(dtype), ld, lead)
    t = random_tokens(rows, 5000, 2)
    check_logprobs(lb.token_logprobs(x, t, 6), x, t, 6, (rows, ld, lead))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,vocab", [(12, 40), (12, 4000), (12, 70001), (200, 3001), (2400, 1000), (700, 2003)])
def test_token_logprobs_masks(rows, vocab, dtype):
    x = (normal((rows, vocab), 17) * 3).to(dtype)
    x[0] = -math.inf                                  # nothing left
    x[1] = torch.finfo(dtype).min                     # all at the lowest value: uniform
    x[2] = -math.inf
    x[2, vocab - 1] = -3.0                            # one token left
    x[3, : vocab - 2] = -math.inf                     # two left
    x[4, ::2] = torch.finfo(dtype).min                # masked with the lowest value
    x[5, vocab // 2] = math.nan
    x[6, 3] = math.inf
    x[7, 1] = math.nan
    x[7, vocab - 1] = math.nan
    x[8] = 0.0
    x[8, ::3] = -0.0                                  # equal: by rising token
    x[9, 1:] = -math.inf
    x[10, vocab // 3:] = -math.inf
    x[11, 5] = torch.finfo(dtype).max / 2             # one far above the rest
    t = random_tokens(rows, vocab, 3)
    t[2], t[3], t[6], t[9] = vocab - 1, 0, 3, -1
    t[10], t[11] = vocab, -100
    for top in (0, 1, 7, 32):
        check_logprobs(lb.token_logprobs(x, t, top), x, t, top, (vocab, dtype, top))


@pytest.mark.parametrize("rows", [1, 170, 2400])
@pytest.mark.parametrize("vocab", [500, 3001, 8192, 100003])
def test_token_logprobs_orders_that_defeat_a_threshold(rows, vocab):
    """Rising, falling, constant, few-valued and clustered rows."""
    i = torch.arange(vocab, device="cuda", dtype=F32)
    rowsets = [i / vocab, -i / vocab, torch.full_like(i, 2.5), (i % 3), (i * 7919 % vocab) / vocab,
               torch.where(i < 64, 5.0 + i / 64, -1.0), torch.where(i >= vocab - 64, 5.0 - i / vocab, -1.0),
               torch.where(i % 1024 == 5, 9.0, i / vocab)]
    if rows > 1000 and vocab > 3001:
        pytest.skip("many rows of these run the kernel that 170 rows run")
    for k, r in enumerate(rowsets):
        x = r.expand(rows, vocab).contiguous()
        for top in (1, 32):
            t = random_tokens(rows, vocab, k)
            check_logprobs(lb.token_logprobs(x, t, top), x, t, top, (k, rows, vocab, top))


def test_token_logprobs_without_tokens():
    x = normal((4, 777), 5)
    r = lb.token_logprobs(x, top=2)
    assert r.logprob is None
    check_logprobs(r, x, None, 2)


# ---------------------------------------------------- far offsets, streams, graphs
def far_rows(cols, dtype, fill):
    """Two rows more than 2^31 elements apart."""
    ld = (1 << 31) + 64
    buf = torch.empty(ld + cols, dtype=dtype, device="cuda")
    v = buf.as_strided((2, cols), (ld, 1))
    v.copy_(fill)
    return v


def test_offsets_past_32_bits():
    x = far_rows(1000, BF16, normal((2, 1000), 1, BF16))
    check_codes(*lb.quantize_rows(x), dense.quantize(f64(x)), "quantize")
    t = torch.tensor([3, 999], device="cuda")
    check_logprobs(lb.token_logprobs(x, t, 5), x, t, 5, "logprobs")
    del x
    for M in (2, 40):
        xq, wq = pitched(codes(M, 256, 1)), far_rows(256, torch.int8, codes(2, 256, 2))
        xs, ws = scales(M, 3), scales(2, 4)
        check_linear(lb.linear_int8(xq, xs, wq, ws), xq, xs, wq, ws, "w")
        xf = far_rows(256, torch.int8, codes(2, 256, 5))
        wq, ws = pitched(codes(200, 256, 6)), scales(200, 7)
        y = far_rows(200, F16, torch.zeros((2, 200)))
        lb.linear_int8(xf, xs[:2], wq, ws * 2.0 ** -8, y=y)
        check_linear(y, xf, xs[:2], wq, ws * 2.0 ** -8, "x, y")
        del wq, xf, y


def chain(x, r, w, wq, ws, t, stream=None):
    q, s, total = lb.rmsnorm_quantize(x, w, r, stream=stream)
    y = lb.linear_int8(q, s, wq, ws, stream=stream)
    out = lb.token_logprobs(y, t, 5, stream=stream)
    return q, s, total, y, *out


@pytest.mark.parametrize("M", [1, 24, 200])
def test_side_stream_and_stream_argument(M):
    x, r, w = normal((M, 512), 1, BF16), normal((M, 512), 2, BF16), normal((512,), 3, F16)
    wq, ws = lb.quantize_rows(normal((3000, 512), 4, F16))
    t = random_tokens(M, 3000, 5)
    want = chain(x, r, w, wq, ws, t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for arg in (side, side.cuda_stream):
        got = chain(x, r, w, wq, ws, t, stream=arg)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    with torch.cuda.stream(side):
        got = chain(x, r, w, wq, ws, t)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("M", [1, 3, 24, 200])
def test_calls_back_to_back_on_reused_buffers(M):
    """Each call may start while the one before it runs, and reads what that one writes:
    a long run without a wait, every buffer reused, gives what waited-for calls give."""
    n, k, steps = 4099, 776, 24
    xs = [normal((M, k), 70 + i, BF16) for i in range(steps)]
    w = normal((k,), 3, F16)
    wq, ws = lb.quantize_rows(normal((n, k), 4, F16))
    t = random_tokens(M, n, 5)

    def run(wait):
        r = normal((M, k), 1, BF16)
        q, s = pitched(codes(M, k, 2)), torch.empty(M, device="cuda")
        y = torch.empty((M, n), device="cuda")
        out = []
        for x in xs:
            lb.rmsnorm_quantize(x, w, r, sum_out=r, q=q, scale=s)
            if wait:
                torch.cuda.synchronize()
            lb.linear_int8(q, s, wq, ws, y=y)
            if wait:
                torch.cuda.synchronize()
            lp = lb.token_logprobs(y, t, 3)
            q2, s2 = lb.quantize_rows(y)
            if wait:
                torch.cuda.synchronize()
            out.append((r.clone(), q.clone(), y.clone(), *lp, q2, s2))
        torch.cuda.synchronize()
        return out

    for a, b in zip(run(True), run(False)):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("M", [1, 24, 200])
def test_two_captured_graphs_replayed_together(M):
    """The calls share no scratch: two graphs on two streams, with new inputs, give what
    plain calls give."""
    wq, ws = lb.quantize_rows(normal((5000, 1024), 4, F16))
    w = normal((1024,), 3, F16)
    sets, graphs, outs, streams = [], [], [], [torch.cuda.Stream() for _ in range(2)]
    chain(normal((M, 1024), 1, BF16), normal((M, 1024), 2, BF16), w, wq, ws, random_tokens(M, 5000, 5))
    torch.cuda.synchronize()
    for i in range(2):
        sets.append([normal((M, 1024), 10 + i, BF16), normal((M, 1024), 20 + i, BF16), w, wq, ws,
                     random_tokens(M, 5000, 30 + i)])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            outs.append(chain(*sets[i]))
        graphs.append(g)
    for rep in range(3):
        for i in range(2):
            sets[i][0].copy_(normal((M, 1024), 100 + 10 * rep + i, BF16))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], chain(*sets[i])))


@pytest.mark.parametrize("M", [1, 17, 150])
def test_captured_among_copies_and_joined_streams(M):
    """In a graph, a call that follows a copy or a memset and one that joins two streams
    wait for all of them."""
    k, n = 528, 640
    src, wsrc = normal((M, k), 1, F16), normal((n, k), 2, F16)
    buf, wbuf, junk = torch.empty_like(src), torch.empty_like(wsrc), torch.empty(1 << 20, device="cuda")
    t = random_tokens(M, n, 3)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def body(fork):
        buf.copy_(src)
        q, s = lb.quantize_rows(buf)
        if fork:
            side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side) if fork else torch.cuda.stream(torch.cuda.current_stream()):
            wbuf.copy_(wsrc)
            wq, ws = lb.quantize_rows(wbuf)
        if fork:
            torch.cuda.current_stream().wait_stream(side)
        y = lb.linear_int8(q, s, wq, ws)
        junk.zero_()
        r = lb.token_logprobs(y, t, 3)
        y2 = y * 2
        return (q, s, wq, ws, y, *r, y2, *lb.quantize_rows(y2))

    body(False)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        out = body(True)
    for rep in range(5):
        src.copy_(normal((M, k), 10 + rep, F16))
        wsrc.copy_(normal((n, k), 20 + rep, F16))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, body(False)))


# -------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("norm_weight", [True, False])
def test_stack_and_head_end_to_end(norm_weight):
    """One token through a stack and its head; a scored prompt of 40 residual streams."""
    model = Model("tiny", 512, 1024, 2, 4, 2)
    stack = build_stack(model, 1.0, base=60, ranks=[64] * 7)
    head = build_head(model, base=60, vocab=2000, norm_weight=norm_weight)
    # the head's codes are the oracle's of the same dense weight
    w = (synth.latent(2000, 512, synth.tensor_seed(60, 2, 0, 0, synth.KIND_HEAD), "cuda")
         * 512 ** -0.5).to(F16)
    check_codes(head.wq, head.ws, dense.quantize(f64(w)), "head")
    nw = f64(head.norm_weight) if norm_weight else None
    one = stack.forward(synth.activation(512, 61, BF16, "cuda"))
    prompt = normal((40, 512), 62) * one.abs().mean()
    for h in (one, prompt):
        h2 = h.reshape(-1, 512)
        xq, xs = dense.rmsnorm_quantize(f64(h2), nw)
        logits = head.logits(h)
        ref = dense.linear_int8(xq, xs, f64(head.wq), f64(head.ws))
        assert np.abs(f64(logits) - ref).max() <= 68 * U * np.abs(ref).max()   # scale 64 u, y 3 u
        # the logits are near those of the dense head: a code is off by half a step at most,
        # so a logit by half a scale times the other operand's 1-norm, on either side
        s = f64(h2)
        n = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + 1e-5) * (nw if nw is not None else 1.0)
        wd = f64(w)
        bound = 0.5 * xs[:, None] * np.abs(wd).sum(axis=1)[None, :] + \
            0.5 * f64(head.ws)[None, :] * np.abs(xq.astype(np.float64) * xs[:, None]).sum(axis=1)[:, None]
        assert (np.abs(ref - n @ wd.T) <= bound * (1 + 1e-6)).all()
        t = random_tokens(h2.shape[0], 2000, 63)
        r = head.logprobs(h, t, top=5)
        check_logprobs(r, logits, t, 5, "head")
    # a greedy continuation: the best alternative is the logits' argmax
    assert head.logprobs(one, top=1).top_id.item() == head.logits(one).argmax().item()


def test_calls_keep_nothing_between_them():
    """The same buffers with other contents give the other contents' results."""
    x, t = normal((3, 4000), 1), random_tokens(3, 4000, 2)
    first = lb.token_logprobs(x, t, 5)
    q1, s1 = lb.quantize_rows(x)
    x.copy_(normal((3, 4000), 7))
    check_logprobs(lb.token_logprobs(x, t, 5), x, t, 5, "again")
    check_codes(*lb.quantize_rows(x), dense.quantize(f64(x)), "again")
    assert not torch.equal(q1, lb.quantize_rows(x)[0]) and first.entropy.shape == (3,)


def test_refusals_on_the_gpu():
    x = normal((4, 64), 1)
    q, s = lb.quantize_rows(x)
    for call in (lambda: lb.quantize_rows(x[:0]), lambda: lb.quantize_rows(x[:, :0]),
                 lambda: lb.linear_int8(q[:0], s[:0], q, s), lambda: lb.token_logprobs(x[:0]),
                 lambda: lb.quantize_rows(x[:1].expand(3, 64)),
                 lambda: lb.rmsnorm_quantize(x, eps=-1.0)):
        with pytest.raises(lb.LbError):
            call()
    for call in (lambda: lb.linear_int8(q, s, q, s.cpu()), lambda: lb.rmsnorm_quantize(x, residual=x.cpu()),
                 lambda: lb.token_logprobs(x, torch.zeros(4, dtype=torch.int64)),
                 lambda: lb.linear_int8(q, s, q, s.cpu(), stream=torch.cuda.Stream()),
                 lambda: lb.token_logprobs(x.cpu(), stream=torch.cuda.Stream())):
        with pytest.raises(ValueError):
            call()
