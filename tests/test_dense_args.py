"""Refusals of the dense path (CPU): they return before any CUDA call, so the
"device" pointers here are plain numbers that nothing follows."""
import pytest
import torch

import binary_rank_linear_lb_b200 as lb
from binary_rank_linear_lb_b200 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return lb.lib()


BAD, ALIGN = lb.LB_ERR_INVALID_ARG, lb.LB_ERR_ALIGNMENT


def quantize(L, **kw):
    a = dict(x=64, dt=lb.LB_F32, rows=4, cols=8, ldx=8, q=64, ldq=8, scale=64)
    a.update(kw)
    return L.lb_quantize_rows(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(q=None), BAD), (dict(scale=None), BAD), (dict(dt=3), BAD),
    (dict(rows=0), BAD), (dict(cols=0), BAD), (dict(rows=-1), BAD), (dict(rows=1 << 31), BAD),
    (dict(cols=(1 << 24) + 1, ldx=1 << 25, ldq=1 << 25), BAD), (dict(ldx=7), BAD),
    (dict(ldq=7), BAD), (dict(ldx=(1 << 40) + 1), BAD), (dict(x=66), ALIGN), (dict(scale=66), ALIGN),
    (dict(x=65, dt=lb.LB_F16), ALIGN)])
def test_quantize_rows_refusals(L, kw, want):
    assert quantize(L, **kw) == want


def norm(L, **kw):
    a = dict(x=64, dt=lb.LB_BF16, rows=4, cols=8, ldx=8, r=64, ldr=8, s=64, lds=8, w=64,
             wdt=lb.LB_F16, eps=1e-5, q=64, ldq=8, scale=64)
    a.update(kw)
    return L.lb_rmsnorm_quantize(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(q=None), BAD), (dict(scale=None), BAD), (dict(dt=-1), BAD),
    (dict(wdt=9), BAD), (dict(r=None), BAD), (dict(s=None), BAD), (dict(rows=0), BAD),
    (dict(cols=0), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD), (dict(ldr=7), BAD), (dict(lds=7), BAD), (dict(ldx=0), BAD),
    (dict(ldq=0), BAD), (dict(r=65), ALIGN), (dict(s=65), ALIGN), (dict(w=65), ALIGN),
    (dict(w=66, wdt=lb.LB_F32), ALIGN), (dict(x=65), ALIGN), (dict(scale=65), ALIGN)])
def test_rmsnorm_quantize_refusals(L, kw, want):
    assert norm(L, **kw) == want


def linear(L, **kw):
    a = dict(xq=64, ldx=32, xs=64, M=4, wq=64, ldw=32, ws=64, k=32, n=8, y=64, dt=lb.LB_F32, ldy=8)
    a.update(kw)
    return L.lb_linear_int8(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(xq=None), BAD), (dict(xs=None), BAD), (dict(wq=None), BAD), (dict(ws=None), BAD),
    (dict(y=None), BAD), (dict(M=0), BAD), (dict(k=0), BAD), (dict(n=0), BAD), (dict(dt=5), BAD),
    (dict(M=(1 << 24) + 1), BAD), (dict(n=(1 << 24) + 1, ldy=1 << 25), BAD),
    (dict(k=131072, ldx=131072, ldw=131072), BAD), (dict(ldx=31), BAD), (dict(ldw=31), BAD),
    (dict(ldy=7), BAD), (dict(ldw=(1 << 32) + 1), BAD), (dict(xs=66), ALIGN), (dict(ws=66), ALIGN),
    (dict(y=66), ALIGN), (dict(y=65, dt=lb.LB_BF16), ALIGN)])
def test_linear_int8_refusals(L, kw, want):
    assert linear(L, **kw) == want


def logprobs(L, **kw):
    a = dict(x=64, dt=lb.LB_F32, rows=4, vocab=100, ld=100, tok=64, lp=64, h=64, top=5, ids=64, tlp=64)
    a.update(kw)
    return L.lb_token_logprobs(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(dt=3), BAD), (dict(rows=0), BAD), (dict(vocab=0), BAD),
    (dict(vocab=(1 << 24) + 1, ld=1 << 25), BAD), (dict(ld=99), BAD), (dict(tok=None), BAD),
    (dict(lp=None), BAD), (dict(top=-1), BAD), (dict(top=33), BAD), (dict(vocab=4, top=5), BAD),
    (dict(ids=None), BAD), (dict(tlp=None), BAD),
    (dict(tok=None, lp=None, h=None, top=0), BAD), (dict(x=66), ALIGN), (dict(tok=68), ALIGN),
    (dict(lp=66), ALIGN), (dict(h=66), ALIGN), (dict(ids=68), ALIGN), (dict(tlp=66), ALIGN)])
def test_token_logprobs_refusals(L, kw, want):
    assert logprobs(L, **kw) == want


def test_no_device_is_an_error_not_a_fallback(L):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    for st in (quantize(L), norm(L), linear(L), logprobs(L)):
        assert st in (lb.LB_ERR_CUDA, lb.LB_ERR_UNSUPPORTED)


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(4, 8)
    q, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: lb.quantize_rows(x), lambda: lb.rmsnorm_quantize(x),
                 lambda: lb.linear_int8(q, s, q, s), lambda: lb.token_logprobs(x),
                 lambda: lb.quantize_rows(x.reshape(-1)), lambda: lb.quantize_rows(x.t()),
                 lambda: lb.quantize_rows(x.double()), lambda: lb.rmsnorm_quantize(x, torch.ones(7)),
                 lambda: lb.rmsnorm_quantize(x, residual=x.half()),
                 lambda: lb.rmsnorm_quantize(x, residual=torch.zeros(3, 8)),
                 lambda: lb.rmsnorm_quantize(x, sum_out=x),
                 lambda: lb.linear_int8(q, s, q[:, :7], s), lambda: lb.linear_int8(q, s[:3], q, s),
                 lambda: lb.linear_int8(x, s, q, s), lambda: lb.linear_int8(q, s, q, s, y=x),
                 lambda: lb.token_logprobs(x, tokens=torch.zeros(4, dtype=torch.int32)),
                 lambda: lb.token_logprobs(x, tokens=torch.zeros(3, dtype=torch.int64)),
                 lambda: lb.token_logprobs(x, top=9), lambda: lb.token_logprobs(x, top=-1)):
        with pytest.raises(ValueError):
            call()
