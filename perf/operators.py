"""Timed cases of the transformer-block operators around the W4A4 quantizer:
layer norm (forward and backward), the linear layer with bias, activation and
residual in its epilogue (MXFP4 and 16-bit operands), and attention over
packed prompts.

Shapes are those of the DiT layers this package is measured on (widths 1152 /
4608, 2240 / 5600 and 3072 / 12288 with 4096 or 4608 tokens, up to 65536 rows)
and generic ones.  ``own`` selects the library's kernels; otherwise ``run``
computes the same results with elementary torch operations in fp32.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # the norm of one token, the smallest call of a serving step
        dict(name="norm token", op="norm", m=1, d=1152, fmt="bf16", group_rows=0),
        # the norm of a whole sampling batch, modulated per image of 4096 tokens
        dict(name="norm batch", op="norm", m=65536, d=1152, fmt="bf16", group_rows=4096),
        # gradient of an odd-sized fp16 batch of short rows
        dict(name="norm grad odd", op="norm_grad", m=4095, d=1155, fmt="f16", group_rows=0),
        # gradient at the widest hidden size, the weight's sum over many rows
        dict(name="norm grad wide", op="norm_grad", m=18432, d=12288, fmt="bf16", group_rows=0),
        # one token through a W4A4 FFN-down layer: the weight's bytes and latency
        dict(name="w4a4 token", op="w4a4", m=1, n=3072, k=12288, act="none", residual=True,
             out="bf16"),
        # FFN-up of a 4096-token image, activation in the epilogue, short contraction
        dict(name="w4a4 ffn up", op="w4a4", m=4096, n=4608, k=1152, act="gelu_tanh", residual=False,
             out="bf16"),
        # FFN-down of a 4608-token image, residual added: the largest product
        dict(name="w4a4 ffn down", op="w4a4", m=4608, n=3072, k=12288, act="none", residual=True,
             out="bf16"),
        # a short text prompt through an unquantized projection (17 ragged rows)
        dict(name="linear prompt", op="linear", m=17, n=1152, k=4608, act="none", residual=True,
             fmt="bf16"),
        # an unquantized FFN-up layer on a whole image
        dict(name="linear image", op="linear", m=4096, n=5600, k=2240, act="silu", residual=False,
             fmt="bf16"),
        # one new token for each of 8 sequences with caches of up to 32768 tokens
        dict(name="attention token", op="attention", batch=8, max_q=1, max_k=32768, heads=32,
             kv_heads=8, dim=128, causal=True, fmt="bf16", ragged=True, lengths=3),
        # a packed batch of 16 prompts of different lengths, one of them empty
        dict(name="attention packed", op="attention", batch=16, max_q=2048, max_k=2048, heads=32,
             kv_heads=8, dim=128, causal=True, fmt="bf16", ragged=True, lengths=5),
        # one whole long prompt
        dict(name="attention long", op="attention", batch=1, max_q=16384, max_k=16384, heads=24,
             kv_heads=24, dim=128, causal=True, fmt="bf16", ragged=False, lengths=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "w4a4", "linear", "attention", "attention"])
    if op in ("norm", "norm_grad"):
        d = rng.choice([1152, 2240, 4608, 5600, _log(rng, 33, 12288), _log(rng, 33, 12288)])
        fmt = rng.choice(["bf16", "bf16", "f16", "f32"])
        m = _log(rng, 1, min(65536, 18432 * 12288 // d // (2 if fmt == "f32" else 1)))
        group = rng.choice([0, 0, _log(rng, max(1, m // 4096), m)])
        return dict(op=op, m=m, d=d, fmt=fmt, group_rows=group)
    if op in ("w4a4", "linear"):
        k = rng.choice([1152, 2240, 4608, 5600, 32 * _log(rng, 2, 384)])
        n = rng.choice([1152, 2240, 4608, 5600, _log(rng, 64, 12288)])
        most = max(1, 4608 * 3072 * 12288 // (n * k)) if op == "w4a4" else \
            max(1, 4096 * 5600 * 2240 * 4 // (n * k))
        c = dict(op=op, m=_log(rng, 1, min(8192, most)), n=n, k=k,
                 act=rng.choice(["none", "gelu", "gelu_tanh", "silu"]),
                 residual=rng.random() < 0.5)
        if op == "w4a4":
            c["out"] = rng.choice(["bf16", "bf16", "f16"])
        else:
            c["fmt"] = rng.choice(["bf16", "bf16", "f16"])
        return c
    dim = rng.choice([32, 64, 72, 128, 128])
    group = rng.choice([1, 2, 3, 4, 8])
    kv_heads = rng.choice([1, 2, 4, 8])
    kind = rng.choice(["prompt", "prompt", "chunk", "token"])
    max_k = _log(rng, 1, 8192)
    causal = rng.random() < 0.7
    max_q = max_k if kind == "prompt" else 1 if kind == "token" else _log(rng, 1, max_k)
    # at most as many pairs of rows and heads as the longest listed prompt has
    most = 16384 * 16384 * 24 // (max_q * max_k * kv_heads * group) // (1 if causal else 2)
    batch = min(_log(rng, 1, 32), max(1, most), max(1, 262144 // max_k))
    return dict(op="attention", batch=batch, max_q=max_q, max_k=max_k, heads=group * kv_heads,
                kv_heads=kv_heads, dim=dim, causal=causal,
                fmt=rng.choice(["bf16", "bf16", "f16"]), ragged=rng.random() < 0.7,
                lengths=rng.randrange(1 << 16))


# --- inputs --------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, m, d):
    """Gaussian entries, a lognormal size per token and 1 % outlier channels."""
    x = _randn(g, m, d)
    x *= torch.exp(0.5 * _randn(g, m, 1))
    ch = torch.randperm(d, generator=g, device="cuda")[:max(1, d // 100)]
    x[:, ch] *= 30.0
    return x


def _padded(x, dtype):
    """x in ``dtype`` as a view of rows whose pitch is a multiple of 16 bytes."""
    m, d = x.shape
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    buf = torch.zeros((m, d + (-d) % unit), dtype=dtype, device=x.device)
    buf[:, :d] = x
    return buf[:, :d]


def _quantized(x):
    """MXFP4 of fp32 rows: packed codes [m, k / 2] and 128x4 tiled E8M0 scales."""
    m, k = x.shape
    nb = k // 32
    b = x.reshape(m, nb, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.floor(torch.log2(amax)) - 2, torch.full_like(amax, -127.0))
    e = e.clamp(-127, 127)
    v = torch.ldexp(b, -e[..., None])
    a = v.abs()
    # the index of the nearest magnitude of 0, 0.5, 1, 1.5, 2, 3, 4, 6
    code = torch.zeros_like(a, dtype=torch.uint8)
    for edge in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += (a > edge).to(torch.uint8)
    code = code | ((v < 0).to(torch.uint8) << 3)
    code = code.reshape(m, k // 2, 2)
    q = code[..., 0] | (code[..., 1] << 4)
    ncb, nrt = (nb + 3) // 4, (m + 127) // 128
    tiles = torch.zeros((nrt * 128, ncb * 4), dtype=torch.uint8, device=x.device)
    tiles[:m, :nb] = (e + 127).to(torch.uint8)
    sf = tiles.reshape(nrt, 4, 32, ncb, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)
    return q.contiguous(), sf


def _lengths(case):
    """(query lengths, key lengths) of a packed batch."""
    b, mq, mk = case["batch"], case["max_q"], case["max_k"]
    if not case["ragged"]:
        return [mq] * b, [mk] * b
    rng = random.Random(case["lengths"])
    lk = [mk] + [rng.randint(1, mk) for _ in range(b - 1)]
    if mq == mk:
        lq = list(lk)
        if b > 2:
            lq[1] = lk[1] = 0                  # an empty sequence
    else:
        lq = [mq] + [rng.randint(1, mq) for _ in range(b - 1)]
        if b > 2:
            lk[1] = 0                          # rows that see no key
    order = list(range(b))
    rng.shuffle(order)
    return [lq[i] for i in order], [lk[i] for i in order]


def _groups(case):
    r = case["group_rows"]
    return 1 if r == 0 else -(-case["m"] // r)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(op=op, case=case)
    if op in ("norm", "norm_grad"):
        m, d, dt = case["m"], case["d"], DTYPE[case["fmt"]]
        groups = _groups(case)
        x = _activations(g, m, d) + 0.5 * _randn(g, 1, d)
        s["x"] = _padded(x, dt)
        s["weight"] = 1.0 + 0.3 * _randn(g, groups, d)
        s["bias"] = 0.2 * _randn(g, groups, d)
        if op == "norm_grad":
            xf = s["x"].float()
            s["mean"] = xf.mean(-1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(-1) + EPS)
            s["dy"] = _padded(_randn(g, m, d) * torch.exp(0.5 * _randn(g, m, 1)), dt)
        return s
    if op in ("w4a4", "linear"):
        m, n, k = case["m"], case["n"], case["k"]
        out = DTYPE[case["out"] if op == "w4a4" else case["fmt"]]
        a, w = _randn(g, m, k) * torch.exp(0.5 * _randn(g, m, 1)), _randn(g, n, k) / math.sqrt(k)
        if op == "w4a4":
            s["qa"], s["sfa"] = _quantized(a)
            s["qw"], s["sfw"] = _quantized(w)
        else:
            s["a"], s["w"] = a.to(out), w.to(out)
        s["bias"] = 0.5 * _randn(g, n)
        s["residual"] = _padded(_randn(g, m, n), out) if case["residual"] else None
        return s
    lq, lk = _lengths(case)
    dt, dim = DTYPE[case["fmt"]], case["dim"]
    tq, tk = sum(lq), sum(lk)
    s["q"] = (1.5 * _randn(g, tq, case["heads"], dim)).to(dt)
    s["k"] = _randn(g, tk, case["kv_heads"], dim).to(dt)
    s["v"] = (_randn(g, tk, case["kv_heads"], dim) + 0.5 * _randn(g, 1, case["kv_heads"], dim)).to(dt)
    s["cu_q"] = torch.tensor([0] + lq).cumsum(0).to(torch.int32).cuda()
    s["cu_k"] = torch.tensor([0] + lk).cumsum(0).to(torch.int32).cuda()
    s["max_q"], s["max_k"] = max(lq), max(lk)
    return s


# --- one pass ------------------------------------------------------------------

def run(s):
    op, case = s["op"], s["case"]
    if own:
        from w4a4_mxfp4_activation_gb300 import kq
        if op == "norm":
            y, mean, rstd = kq.kq_layer_norm(s["x"], s["weight"], s["bias"], EPS,
                                             group_rows=case["group_rows"], stats=True)
            return {"y": y, "mean": mean, "rstd": rstd}
        if op == "norm_grad":
            dx, dw, db = kq.kq_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"],
                                                   s["rstd"], group_rows=case["group_rows"])
            return {"dx": dx, "dweight": dw, "dbias": db}
        if op == "w4a4":
            return kq.kq_w4a4_linear(s["qa"], s["sfa"], s["qw"], s["sfw"], case["m"], case["n"],
                                     case["k"], bias=s["bias"], act=case["act"],
                                     residual=s["residual"], out_dtype=DTYPE[case["out"]])
        if op == "linear":
            return kq.kq_linear(s["a"], s["w"], bias=s["bias"], act=case["act"],
                                residual=s["residual"])
        out, lse = kq.kq_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"],
                                   s["max_k"], causal=case["causal"], lse=True)
        return {"out": out, "lse": lse}
    if op == "norm":
        return _plain_norm(s, case)
    if op == "norm_grad":
        return _plain_norm_grad(s, case)
    if op == "w4a4":
        a = _decode(s["qa"], s["sfa"], case["m"], case["k"])
        w = _decode(s["qw"], s["sfw"], case["n"], case["k"])
        return _plain_epilogue(a @ w.t(), s, case, DTYPE[case["out"]])
    if op == "linear":
        return _plain_epilogue(s["a"].float() @ s["w"].float().t(), s, case, s["a"].dtype)
    return _plain_attention(s, case)


def _row_groups(case, t):
    """The weight or bias rows [groups, d] for each of the m rows."""
    if case["group_rows"] == 0:
        return t
    rows = torch.arange(case["m"], device=t.device) // case["group_rows"]
    return t[rows]


def _plain_norm(s, case):
    x = s["x"].float()
    mean = x.mean(-1)
    c = x - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(-1) + EPS)
    y = c * rstd[:, None] * _row_groups(case, s["weight"]) + _row_groups(case, s["bias"])
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_grad(s, case):
    x, dy = s["x"].float(), s["dy"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gr = dy * _row_groups(case, s["weight"])
    dx = s["rstd"][:, None] * (gr - gr.mean(-1, keepdim=True)
                               - xhat * (gr * xhat).mean(-1, keepdim=True))
    dw = dy * xhat
    if case["group_rows"] == 0:
        return {"dx": dx.to(s["x"].dtype), "dweight": dw.sum(0, keepdim=True),
                "dbias": dy.sum(0, keepdim=True)}
    r, m, groups = case["group_rows"], case["m"], _groups(case)
    pad = (0, 0, 0, groups * r - m)
    dw = torch.nn.functional.pad(dw, pad).reshape(groups, r, -1).sum(1)
    db = torch.nn.functional.pad(dy, pad).reshape(groups, r, -1).sum(1)
    return {"dx": dx.to(s["x"].dtype), "dweight": dw, "dbias": db}


def _decode(q, sf, rows, k):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0,
                          -3.0, -4.0, -6.0], device=q.device)
    codes = torch.stack((q & 15, q >> 4), -1).reshape(rows, k)
    nb = k // 32
    ncb, nrt = (nb + 3) // 4, (rows + 127) // 128
    e = sf.reshape(nrt, ncb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(nrt * 128, ncb * 4)
    scale = torch.exp2(e[:rows, :nb].float() - 127.0)
    return (table[codes.int()].reshape(rows, nb, 32) * scale[..., None]).reshape(rows, k)


def _plain_act(x, act):
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _plain_epilogue(c, s, case, dtype):
    y = _plain_act(c + s["bias"], case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(dtype)


def _plain_attention(s, case):
    """Packed rows gathered into padded batches, scores with the masked keys at
    weight zero, and the rows gathered back."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    hk, dim, mq, mk = case["kv_heads"], case["dim"], s["max_q"], s["max_k"]
    grp = case["heads"] // hk
    dev = q.device
    iq, ik = torch.arange(mq, device=dev), torch.arange(mk, device=dev)
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    qp = q[(cu_q[:-1, None] + iq).clamp(max=q.shape[0] - 1)]
    kp = k[(cu_k[:-1, None] + ik).clamp(max=k.shape[0] - 1)]
    vp = v[(cu_k[:-1, None] + ik).clamp(max=k.shape[0] - 1)]
    b = qp.shape[0]
    qp = qp.reshape(b, mq, hk, grp, dim).permute(0, 2, 3, 1, 4).reshape(b, hk, grp * mq, dim)
    kp, vp = kp.permute(0, 2, 3, 1), vp.permute(0, 2, 1, 3)
    sc = (qp @ kp).reshape(b, hk, grp, mq, mk) / math.sqrt(dim)
    seen = (ik < lk[:, None])[:, None, :]
    if case["causal"]:
        seen = seen & (ik <= (iq[:, None] + (lk - lq)[:, None, None]))
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = (p.reshape(b, hk, grp * mq, mk) @ vp).reshape(b, hk, grp, mq, dim)
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total))[..., 0]
    tok = torch.arange(q.shape[0], device=dev)
    seq = torch.searchsorted(cu_q[1:].contiguous(), tok, right=True)
    pos = tok - cu_q[seq]
    out = out.permute(0, 3, 1, 2, 4)[seq, pos].reshape(q.shape)
    lse = lse.permute(0, 3, 1, 2)[seq, pos].reshape(q.shape[0], q.shape[1])
    return {"out": out.to(s["q"].dtype), "lse": lse}


# --- what a pass cannot do without -----------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        m, d, b, groups = case["m"], case["d"], 4 if case["fmt"] == "f32" else 2, _groups(case)
        if op == "norm":
            return {"bytes": 2 * m * d * b + 8 * groups * d + 8 * m, "flops": 8 * m * d}
        return {"bytes": 3 * m * d * b + 12 * groups * d + 8 * m, "flops": 14 * m * d}
    if op in ("w4a4", "linear"):
        m, n, k = case["m"], case["n"], case["k"]
        operands = (m + n) * (k // 2 + k // 32) if op == "w4a4" else 2 * (m + n) * k
        return {"bytes": operands + 4 * n + 2 * m * n * (2 if case["residual"] else 1),
                "flops": 2 * m * n * k}
    lq, lk = _lengths(case)
    pairs = 0
    for a, b in zip(lq, lk):
        if not case["causal"]:
            pairs += a * b
            continue
        # row i sees max(0, i + 1 + b - a) keys
        first = max(0, a - b)
        rows = a - first
        lo = first + 1 + b - a
        pairs += rows * lo + rows * (rows - 1) // 2 if rows > 0 else 0
    h, hk, dim = case["heads"], case["kv_heads"], case["dim"]
    return {"bytes": 2 * dim * (2 * sum(lq) * h + 2 * sum(lk) * hk) + 4 * sum(lq) * h,
            "flops": 4 * dim * h * pairs}


# --- the definitions in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s, case)
    if op in ("w4a4", "linear"):
        if op == "w4a4":
            a = _exact_mxfp4(s["qa"], s["sfa"], case["m"], case["k"])
            w = _exact_mxfp4(s["qw"], s["sfw"], case["n"], case["k"])
        else:
            a, w = s["a"].double(), s["w"].double()
        z = torch.mm(a, w.transpose(0, 1)).add_(s["bias"].double())
        if case["act"] == "gelu":                       # z times the normal distribution function
            z = z * torch.special.ndtr(z)
        elif case["act"] == "gelu_tanh":                # 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
            u = math.sqrt(2.0 / math.pi) * z * (1.0 + 0.044715 * z.square())
            z = z * torch.special.expit(2.0 * u)
        elif case["act"] == "silu":
            z = z * torch.special.expit(z)
        return z if s["residual"] is None else z + s["residual"].double()
    return _exact_attention(s, case)


def _exact_norm(s, case):
    m, d, r = case["m"], case["d"], case["group_rows"] or case["m"]
    groups = _groups(case)
    x = s["x"].double()
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        y = torch.empty_like(x)
        for i in range(groups) if groups <= 64 else ():
            rows = slice(i * r, min(m, (i + 1) * r))
            z = (x[rows] - mean[rows, None]) / torch.sqrt(var[rows, None] + EPS)
            y[rows] = torch.addcmul(s["bias"][i].double(), z, s["weight"][i].double())
        if groups > 64:
            at = torch.div(torch.arange(m, device=x.device), r, rounding_mode="floor")
            z = (x - mean[:, None]) / torch.sqrt(var[:, None] + EPS)
            y = torch.addcmul(s["bias"].double()[at], z, s["weight"].double()[at])
        return {"y": y, "mean": mean, "rstd": 1.0 / torch.sqrt(var + EPS)}
    at = torch.div(torch.arange(m, device=x.device), r, rounding_mode="floor")
    dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
    z = (x - s["mean"].double()[:, None]) * rstd
    gr = dy * s["weight"].double()[at]
    # the gradient with its projections on the constant row and on z removed
    along = torch.einsum("ij,ij->i", gr, z)[:, None] / d
    dx = (gr - gr.sum(1, keepdim=True) / d - along * z) * rstd
    dw = torch.zeros((groups, d), dtype=torch.float64, device=x.device).index_add_(0, at, dy * z)
    db = torch.zeros((groups, d), dtype=torch.float64, device=x.device).index_add_(0, at, dy)
    return {"dx": dx, "dweight": dw, "dbias": db}


def _exact_mxfp4(q, sf, rows, k):
    """E2M1 from its fields (2 exponent bits with bias 1, 1 mantissa bit) times
    2^(byte - 127), the byte at its place in the 128x4 tiles."""
    c = torch.empty((rows, k), dtype=torch.int32, device=q.device)
    c[:, 0::2], c[:, 1::2] = (q % 16).int(), (q // 16).int()
    ex, man = (c // 2) % 4, (c % 2).double()
    mag = torch.where(ex == 0, 0.5 * man, torch.ldexp(1.0 + 0.5 * man, ex - 1))
    i = torch.arange(rows, device=q.device)[:, None]
    b = torch.arange(k // 32, device=q.device)[None, :]
    tiles = (k // 32 + 3) // 4
    at = ((i // 128) * tiles + b // 4) * 512 + (i % 32) * 16 + ((i % 128) // 32) * 4 + b % 4
    e = sf[at].int() - 127
    v = torch.ldexp(torch.where(c >= 8, -mag, mag), e.repeat_interleave(32, dim=1))
    return v


def _exact_attention(s, case):
    lq, lk = _lengths(case)
    grp, dim = case["heads"] // case["kv_heads"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    rq = rk = 0
    for a, b in zip(lq, lk):
        for h in range(case["heads"] if a and b else 0):
            k, v = s["k"][rk:rk + b, h // grp].double(), s["v"][rk:rk + b, h // grp].double()
            for lo in range(0, a, 4096):
                hi = min(a, lo + 4096)
                z = torch.mm(s["q"][rq + lo:rq + hi, h].double(), k.t()) * dim ** -0.5
                if case["causal"]:
                    i = torch.arange(lo, hi, device="cuda")[:, None] + (b - a)
                    z[torch.arange(b, device="cuda")[None, :] > i] = -math.inf
                t = torch.logsumexp(z, 1)
                lse[rq + lo:rq + hi, h] = t
                w = torch.exp(z - torch.where(torch.isinf(t), torch.zeros_like(t), t)[:, None])
                out[rq + lo:rq + hi, h] = torch.mm(w, v)
        rq, rk = rq + a, rk + b
    return {"out": out, "lse": lse}
