"""Operators between a decoder stack and its answers, as cases to be timed.

A stack ends in a residual stream; what follows it is dense: the final norm, the
output head and the reading of its logits.  Four operators cover that path:

  norm       rmsnorm_quantize   s = x + residual, RMS norm of s, 8-bit rows with scales
  quantize   quantize_rows      8-bit rows with scales of a matrix (head weights, activations)
  linear     linear_int8        y = (xq wq^T) * token scale * channel scale
  logprobs   token_logprobs     log probabilities of given tokens, entropy, top alternatives

`run` computes a case in plain torch operations, or, with `own`, by the
package's entry points.  `exact` computes it in 64 bits from the definitions.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # the last norm of a 70B-shaped stack, one token, fp32 residual stream (latency)
        {"name": "norm_1x8192_f32", "op": "norm", "rows": 1, "cols": 8192, "dtype": "f32",
         "weight": "f16", "residual": True},
        # a ragged batch of 13B-shaped tokens
        {"name": "norm_333x5120_f16", "op": "norm", "rows": 333, "cols": 5120, "dtype": "f16",
         "weight": "f16", "residual": True},
        # a 70B-shaped prefill
        {"name": "norm_4096x8192_bf16", "op": "norm", "rows": 4096, "cols": 8192,
         "dtype": "bf16", "weight": "bf16", "residual": True},
        # the down projection's input of a small batch (fp32, as the gate product leaves it)
        {"name": "quantize_64x28672_f32", "op": "quantize", "rows": 64, "cols": 28672,
         "dtype": "f32"},
        # the head weight of a 7B-shaped model, quantised once at load time
        {"name": "quantize_32000x4096_bf16", "op": "quantize", "rows": 32000, "cols": 4096,
         "dtype": "bf16"},
        # 7B head, one token
        {"name": "linear_1x4096x32000_f32", "op": "linear", "rows": 1, "in": 4096, "out": 32000,
         "dtype": "f32"},
        # 70B gate projection kept dense, a decode batch
        {"name": "linear_16x8192x28672_bf16", "op": "linear", "rows": 16, "in": 8192,
         "out": 28672, "dtype": "bf16"},
        # 13B gate projection kept dense, a ragged batch
        {"name": "linear_333x5120x13824_f16", "op": "linear", "rows": 333, "in": 5120,
         "out": 13824, "dtype": "f16"},
        # 70B head over a whole prompt, as a perplexity evaluation runs it
        {"name": "linear_4096x8192x32000_f32", "op": "linear", "rows": 4096, "in": 8192,
         "out": 32000, "dtype": "f32"},
        # one decoded token with 20 alternatives (latency)
        {"name": "logprobs_1x32000_f32_top20", "op": "logprobs", "rows": 1, "vocab": 32000,
         "dtype": "f32", "top": 20, "masked": False},
        # constrained decoding of a ragged batch: part of the vocabulary masked
        {"name": "logprobs_77x32000_bf16_top5", "op": "logprobs", "rows": 77, "vocab": 32000,
         "dtype": "bf16", "top": 5, "masked": True},
        # scoring a whole prompt
        {"name": "logprobs_4096x32000_f32_top5", "op": "logprobs", "rows": 4096, "vocab": 32000,
         "dtype": "f32", "top": 5, "masked": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "logprobs"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "norm":
        return {"op": op, "rows": _spread(rng, 1, 4096), "cols": _spread(rng, 64, 8192),
                "dtype": dtype, "weight": rng.choice(["none", "f32", "f16", "bf16"]),
                "residual": rng.random() < 0.7}
    if op == "quantize":
        cols = _spread(rng, 64, 28672)
        return {"op": op, "rows": _spread(rng, 1, min(32000, (1 << 27) // cols)), "cols": cols,
                "dtype": dtype}
    if op == "linear":
        return {"op": op, "rows": _spread(rng, 1, 4096), "in": _spread(rng, 128, 8192),
                "out": _spread(rng, 128, 32000), "dtype": dtype}
    vocab = _spread(rng, 1000, 131072)
    return {"op": op, "rows": _spread(rng, 1, min(4096, (1 << 27) // vocab)), "vocab": vocab,
            "dtype": dtype, "top": rng.randint(0, 20), "masked": rng.random() < 0.4}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _stream(rows, cols, dtype, g):
    """A residual stream: unit normal, with a few channels that run far above the rest."""
    x = _normal((rows, cols), g)
    loud = torch.rand((cols,), generator=g, device="cuda") < 0.004
    x *= torch.where(loud, 20.0, 1.0)
    return x.to(DTYPES[dtype])


def _codes(rows, cols, g):
    """8-bit codes and scales of normal rows; the rows' pitch is a multiple of 16 bytes."""
    z = _normal((rows, cols), g)
    top = z.abs().amax(dim=1, keepdim=True)
    pitch = (cols + 15) // 16 * 16
    q = torch.zeros((rows, pitch), dtype=torch.int8, device="cuda")
    q[:, :cols] = torch.round(z * (127.0 / top)).to(torch.int8)
    return q[:, :cols], (top[:, 0] / 127.0).contiguous()


def prepare(case, seed):
    g = _generator(seed)
    op, rows = case["op"], case["rows"]
    if op == "norm":
        cols = case["cols"]
        weight = None
        if case["weight"] != "none":
            weight = (1.0 + 0.1 * _normal((cols,), g)).to(DTYPES[case["weight"]])
        return {"op": op, "x": _stream(rows, cols, case["dtype"], g), "weight": weight,
                "residual": _stream(rows, cols, case["dtype"], g) if case["residual"] else None}
    if op == "quantize":
        return {"op": op, "x": _stream(rows, case["cols"], case["dtype"], g)}
    if op == "linear":
        xq, xs = _codes(rows, case["in"], g)
        wq, ws = _codes(case["out"], case["in"], g)
        return {"op": op, "xq": xq, "xs": xs, "wq": wq, "ws": ws, "dtype": DTYPES[case["dtype"]]}
    vocab = case["vocab"]
    logits = 2.5 * _normal((rows, vocab), g)
    logits[:, :1] += 6.0 * torch.rand((rows, 1), generator=g, device="cuda")
    if case["masked"]:
        # each row keeps its own share of the vocabulary, the first row none of it
        share = torch.rand((rows, 1), generator=g, device="cuda")
        share[0] = 0.0 if rows > 1 else 0.5
        gone = torch.rand((rows, vocab), generator=g, device="cuda") >= share
        logits = logits.masked_fill(gone, -math.inf)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    if rows > 4:
        tokens[rows // 2] = -1                       # a padded position: no token given
    return {"op": op, "logits": logits.to(DTYPES[case["dtype"]]), "tokens": tokens,
            "top": case["top"]}


# ------------------------------------------------------------- plain forms
def _plain_quantize(v, size):
    """Codes and scales of v (64 bits, values next to a border between two codes):
    q = rint(127 v / max|v|), scale = size * max|v| / 127."""
    top = v.abs().amax(dim=1, keepdim=True)
    q = torch.where(top > 0, torch.round(v * 127.0 / top), 0.0).to(torch.int8)
    return q, (top[:, 0] * size / 127.0).to(torch.float32)


def _plain_norm(x, weight, residual):
    s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    v = s.double()
    size = 1.0 / torch.sqrt(v.square().mean(dim=1) + EPS)
    q, scale = _plain_quantize(v if weight is None else v * weight.double(), size)
    return (q, scale) if residual is None else (q, scale, s)


def _plain_linear(xq, xs, wq, ws, dtype):
    y = torch.matmul(xq.float(), wq.float().t())
    return (y * xs[:, None] * ws[None, :]).to(dtype)


def _plain_logprobs(logits, tokens, top):
    x = logits.float()
    best = x.amax(dim=1, keepdim=True)
    best = torch.where(torch.isinf(best), 0.0, best)
    d = x - best
    e = torch.exp(d)
    total = e.sum(dim=1, dtype=torch.float64)
    drop = torch.where(e > 0, e * d, 0.0).sum(dim=1, dtype=torch.float64)
    log_total = torch.log(total)
    some = total > 0
    entropy = torch.where(some, log_total - drop / total, 0.0).float()

    def logprob(picked):
        lp = picked - log_total[:, None]
        return torch.where(some[:, None], lp, -math.inf).float()

    given = logprob(d.gather(1, tokens.clamp(min=0)[:, None]).double())[:, 0]
    given = torch.where(tokens >= 0, given, 0.0)
    if top == 0:
        return given, entropy
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top].contiguous()
    return given, entropy, ids, logprob(d.gather(1, ids).double())


def run(state):
    op = state["op"]
    if own:
        import binary_rank_linear_lb_b200 as lb
        if op == "norm":
            q, scale, s = lb.rmsnorm_quantize(state["x"], state["weight"], state["residual"], EPS)
            return (q, scale) if s is None else (q, scale, s)
        if op == "quantize":
            return lb.quantize_rows(state["x"])
        if op == "linear":
            return lb.linear_int8(state["xq"], state["xs"], state["wq"], state["ws"],
                                  dtype=state["dtype"])
        r = lb.token_logprobs(state["logits"], state["tokens"], top=state["top"])
        if state["top"] == 0:
            return r.logprob, r.entropy
        return r.logprob, r.entropy, r.top_id, r.top_logprob
    if op == "norm":
        return _plain_norm(state["x"], state["weight"], state["residual"])
    if op == "quantize":
        return _plain_quantize(state["x"].double(), 1.0)
    if op == "linear":
        return _plain_linear(state["xq"], state["xs"], state["wq"], state["ws"], state["dtype"])
    return _plain_logprobs(state["logits"], state["tokens"], state["top"])


def work(case):
    op, rows = case["op"], case["rows"]
    size = SIZE[case["dtype"]]
    if op in ("norm", "quantize"):
        cells = rows * case["cols"]
        reads = cells * size
        if op == "norm":
            if case["residual"]:
                reads += 2 * cells * size
            if case["weight"] != "none":
                reads += case["cols"] * SIZE[case["weight"]]
        return {"bytes": reads + cells + 4 * rows, "flops": (6 if op == "norm" else 3) * cells}
    if op == "linear":
        k, n = case["in"], case["out"]
        return {"bytes": rows * k + n * k + 4 * (rows + n) + rows * n * size,
                "flops": 2 * rows * k * n}
    cells = rows * case["vocab"]
    return {"bytes": cells * size + rows * (8 + 4 + 4 + 12 * case["top"]), "flops": 5 * cells}


# ------------------------------------------------------------- 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        acc = state["xq"].double() @ state["wq"].double().t()
        acc *= torch.outer(state["xs"].double(), state["ws"].double())
        return acc
    if op == "logprobs":
        x = state["logits"].double()
        lse = torch.logsumexp(x, dim=1, keepdim=True)
        empty = torch.isinf(lse)
        lp = torch.where(empty, -math.inf, x - lse)
        entropy = torch.special.entr(lp.exp()).sum(dim=1)
        tokens = state["tokens"]
        given = torch.where(tokens < 0, 0.0, lp.gather(1, tokens.clamp(min=0)[:, None])[:, 0])
        if not case["top"]:
            return given, entropy
        # the values are all that 64 bits decide; the choice among equals is the callers'
        return given, entropy, None, torch.topk(lp, case["top"], dim=1).values
    x = state["x"]
    s, v, size = x, x.double(), torch.ones((), dtype=torch.float64, device=x.device)
    if op == "norm":
        if state["residual"] is not None:
            v = v + state["residual"].double()
            s = v.to(x.dtype)                        # the residual stream as it is stored
            v = s.double()
        size = torch.rsqrt(torch.sum(v * v, dim=1) / v.shape[1] + EPS)
        if state["weight"] is not None:
            v = state["weight"].double() * v
    peak = torch.linalg.vector_norm(v, ord=math.inf, dim=1)
    step = peak / 127.0
    codes = torch.round(v / step[:, None].clamp(min=1e-300))
    out = (codes.to(torch.int8), step * size)
    return out + (s,) if op == "norm" and state["residual"] is not None else out
