"""The linear layers (bias, activation and residual in the epilogue): the CUDA
kernels against the formula in 64 bits, and the argument checks.

Tolerance of an element before the activation: the tensor cores add K products
in fp32, each addition off by at most 2^-23 of the partial sums (they may
truncate), so (K / 16 + 24) 2^-23 times the sum of the products' sizes bounds the
accumulator and the join of split contractions (the bound the W4A4 product is
tested with); the bias adds one rounding.  The activations' slopes are below
1.13, and they are computed to 8 roundings of fp32.  Then the residual and the
final rounding to the output type.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kq_oracle as O
from w4a4_mxfp4_activation_gb300 import kq

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from w4a4_mxfp4_activation_gb300 import build
    build.build()
    kq.lib()


def act64(x, act):
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(-x / math.sqrt(2))
    if act == "gelu_tanh":
        return x * torch.special.expit(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    if act == "silu":
        return x * torch.special.expit(x)
    return x


def check(out, a, w, bias, act, residual, dtype, k):
    z = a @ w.t() + (bias.double() if bias is not None else 0)
    off = (k / 16 + 24) * 2.0 ** -23 * (a.abs() @ w.abs().t()) + 2.0 ** -24 * z.abs()
    y = act64(z, act)
    off = (1.13 * off + 8 * 2.0 ** -24 * (y.abs() + z.abs())) if act != "none" else off
    ref = y + (residual.double() if residual is not None else 0)
    tol = off + 2.0 ** -24 * ref.abs() + UNIT[dtype] * 1.01 * (ref.abs() + off) + TINY[dtype]
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:4].tolist())


def rows(values, dtype, extra=0, fill=float("nan")):
    m, d = values.shape
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((m, d + (-d) % unit + extra * unit), fill, dtype=dtype, device="cuda")
    buf[:, :d] = values.to(dtype)
    return buf[:, :d]


def quantized(values, pad_byte=0xFF):
    """(codes, tiled scales, decoded fp64); the scale bytes of padding blocks
    are ``pad_byte`` (they must not be used)."""
    m, k = values.shape
    q, sf, _ = kq.kq_quantize_mxfp4(values.bfloat16(), k, layout=kq.KQ_SF_BLOCKED_128x4)
    dec = kq.kq_dequantize(q, sf, m, k, layout=kq.KQ_SF_BLOCKED_128x4).double()
    nb = k // 32
    if nb % 4:
        t = sf[:kq.kq_sf_bytes(m, k, 1)].view(-1, 32, 4, 4)
        ncb = (nb + 3) // 4
        t[ncb - 1::ncb, :, :, nb % 4:] = pad_byte
    return q, sf, dec


# (m, n, k): one token; split contractions of 2 to 8 parts with ragged stages;
# token tiles of 16 to 128 and more than one; ragged rows and columns; odd block
# counts; tiles of both widths on the products' kernel
SHAPES = [(1, 8, 32), (1, 3072, 12288), (3, 129, 96), (17, 1152, 4608), (64, 100, 1184),
          (100, 513, 2240), (128, 640, 1152), (129, 384, 256), (300, 257, 4640), (257, 1155, 1152),
          (1000, 4616, 1184), (1537, 2309, 2240), (4096, 1152, 288)]


@gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("act,bias,res,dtype", [
    ("none", False, False, torch.float32), ("gelu", True, False, torch.bfloat16),
    ("gelu_tanh", True, True, torch.float16), ("silu", False, True, torch.bfloat16),
    ("none", True, True, torch.float32)])
def test_w4a4_linear(m, n, k, act, bias, res, dtype):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    qa, sfa, a = quantized(rnd(m, k))
    qw, sfw, w = quantized(rnd(n, k) / math.sqrt(k))
    b = rnd(n) if bias else None
    r = rows(rnd(m, n), dtype, 1) if res else None
    out = kq.kq_w4a4_linear(qa, sfa, qw, sfw, m, n, k, b, act, r, out_dtype=dtype)
    check(out, a, w, b, act, r, dtype, k)


@gpu
@pytest.mark.parametrize("m,n,k", SHAPES + [(5, 40, 1), (33, 77, 1153), (2000, 1155, 333)])
@pytest.mark.parametrize("act,bias,res,dtype,out_dtype", [
    ("none", False, False, torch.bfloat16, torch.float32),
    ("gelu_tanh", True, True, torch.bfloat16, torch.bfloat16),
    ("silu", True, False, torch.float16, torch.float16),
    ("gelu", False, True, torch.float16, torch.bfloat16)])
def test_linear(m, n, k, act, bias, res, dtype, out_dtype):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    a, w = rows(rnd(m, k), dtype, 1), rows(rnd(n, k) / math.sqrt(k), dtype)
    b = rnd(n) if bias else None
    r = rows(rnd(m, n), out_dtype) if res else None
    out = kq.kq_linear(a, w, b, act, r, out_dtype=out_dtype)
    check(out, a.double(), w.double(), b, act, r, out_dtype, k)


@gpu
@pytest.mark.parametrize("m,n", [(7, 1155), (2000, 1155), (9, 64), (2000, 4616)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_residual_and_untouched_padding(m, n, dtype):
    """out may be the residual; columns past n and rows past m stay."""
    g = torch.Generator(device="cuda").manual_seed(m)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    a, w, b = rnd(m, 256).bfloat16(), rnd(n, 256).bfloat16() / 16, rnd(n)
    buf = torch.full((m + 1, n + (-n) % 8 + 16), 5.0, dtype=dtype, device="cuda")
    r = rnd(m, n).to(dtype)
    buf[:m, :n] = r
    view = buf[:m, :n]
    out = kq.kq_linear(a, w, b, "silu", residual=view, out=view)
    assert out.data_ptr() == buf.data_ptr()
    check(view, a.double(), w.double(), b, "silu", r, dtype, 256)
    assert (buf[:m, n:] == 5.0).all() and (buf[m] == 5.0).all()


@gpu
def test_same_result_as_the_product():
    """No bias, activation or residual, fp32: the bits of kq_w4a4_gemm."""
    m, n, k = 4096, 2240, 1152
    qa, sfa, _ = quantized(torch.randn(m, k, device="cuda"))
    qw, sfw, _ = quantized(torch.randn(n, k, device="cuda"))
    c = kq.kq_w4a4_gemm(qa, sfa, qw, sfw, m, n, k)
    out = kq.kq_w4a4_linear(qa, sfa, qw, sfw, m, n, k, out_dtype=torch.float32)
    assert torch.equal(c, out)


@gpu
@pytest.mark.parametrize("m", [2, 2048])
def test_nan_stays_in_its_row_and_column(m):
    a, w = torch.randn(m, 512, device="cuda").bfloat16(), torch.randn(1160, 512, device="cuda").bfloat16()
    a[1, 3] = float("nan")
    w[5, 511] = float("inf")
    out = kq.kq_linear(a, w, act="silu")
    assert torch.isnan(out[1]).all()
    bad = ~torch.isfinite(out)
    bad[1] = False
    assert not bad[:, :5].any() and not bad[:, 6:].any()


@gpu
def test_large_values_of_the_activations():
    """Both tails: x, and zero (not NaN) where exp overflows."""
    x = torch.tensor([-3e4, -200.0, -100.0, -20.0, -1e-3, 0.0, 1e-3, 20.0, 100.0, 3e4], device="cuda")
    a = x[:, None].bfloat16() * torch.ones(1, 32, device="cuda").bfloat16()
    w = torch.zeros(8, 32, device="cuda").bfloat16()
    w[:, 0] = 1
    for act in ("gelu", "gelu_tanh", "silu"):
        out = kq.kq_linear(a, w, act=act, out_dtype=torch.float32)
        z = a[:, :1].double()
        ref = act64(z, act).expand(-1, 8)
        assert torch.isfinite(out).all()
        assert ((out.double() - ref).abs() <= 9 * 2.0 ** -24 * (ref.abs() + z.abs()) + 1e-30).all()


@gpu
def test_empty_other_stream_and_repeatable():
    w = torch.randn(64, 96, device="cuda").bfloat16()
    assert kq.kq_linear(w[:0], w).shape == (0, 64)
    assert kq.kq_linear(w, w[:0]).shape == (64, 0)
    a = torch.randn(31, 4608, device="cuda").bfloat16()
    w = torch.randn(1152, 4608, device="cuda").bfloat16()
    first = kq.kq_linear(a, w, act="gelu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = [kq.kq_linear(a, w, act="gelu", stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(first, x) for x in again)


# --- argument checks (no GPU) ---------------------------------------------------------

FAKE = 1 << 20


def _w4a4(qa=FAKE, ldqa=32, sfa=FAKE, qw=FAKE, ldqw=32, sfw=FAKE, m=4, n=64, k=64, bias=None, act=0,
          res=None, ldr=0, out=FAKE, ldo=64, fmt=0):
    return kq.lib().kq_w4a4_linear(qa, ldqa, sfa, qw, ldqw, sfw, m, n, k, bias, act, res, ldr, out,
                                   ldo, fmt, None)


def test_w4a4_argument_checks():
    assert _w4a4(act=4) == 4 and _w4a4(act=-1) == 4 and _w4a4(fmt=3) == 4
    assert _w4a4(k=48) == 2 and _w4a4(k=0) == 2 and _w4a4(m=-1) == 2 and _w4a4(n=-1) == 2
    assert _w4a4(ldqa=16) == 2 and _w4a4(ldqw=16) == 2 and _w4a4(ldo=56) == 2
    assert _w4a4(res=FAKE, ldr=56) == 2 and _w4a4(n=(1 << 28) + 1, ldo=1 << 29) == 2
    assert _w4a4(qa=None) == 1 and _w4a4(sfa=None) == 1 and _w4a4(qw=None) == 1
    assert _w4a4(sfw=None) == 1 and _w4a4(out=None) == 1
    assert _w4a4(qa=FAKE + 8) == 3 and _w4a4(sfw=FAKE + 4) == 3 and _w4a4(out=FAKE + 2) == 3
    assert _w4a4(bias=FAKE + 4) == 3 and _w4a4(res=FAKE + 2, ldr=64) == 3
    assert _w4a4(ldqa=40) == 3 and _w4a4(ldo=68) == 3 and _w4a4(res=FAKE, ldr=68) == 3
    assert _w4a4(fmt=2, ldo=66) == 3
    assert _w4a4(m=0, qa=None) == 0 and _w4a4(n=0, ldo=0, qw=None) == 0


def _lin(a=FAKE, lda=64, w=FAKE, ldw=64, fmt_in=0, m=4, n=64, k=64, bias=None, act=0, res=None, ldr=0,
         out=FAKE, ldo=64, fmt=0):
    return kq.lib().kq_linear(a, lda, w, ldw, fmt_in, m, n, k, bias, act, res, ldr, out, ldo, fmt, None)


def test_linear_argument_checks():
    assert _lin(fmt_in=2) == 4 and _lin(act=9) == 4 and _lin(fmt=-1) == 4
    assert _lin(k=0) == 2 and _lin(lda=56) == 2 and _lin(ldw=56) == 2 and _lin(m=1 << 31) == 2
    assert _lin(a=None) == 1 and _lin(w=None) == 1 and _lin(out=None) == 1
    assert _lin(lda=68) == 3 and _lin(ldw=68) == 3 and _lin(a=FAKE + 2) == 3
    assert _lin(m=0, a=None, out=None) == 0


def test_binding_refusals():
    a, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kq.kq_linear(a, w[:, :32])
    with pytest.raises(ValueError):
        kq.kq_linear(a, w.half())
    with pytest.raises(KeyError):
        kq.kq_linear(a, w, act="relu6")
    with pytest.raises(ValueError):
        kq.kq_linear(a, w, bias=torch.zeros(7))
    with pytest.raises(ValueError):
        kq.kq_linear(a, w, residual=torch.zeros(4, 8))
    with pytest.raises(ValueError):
        kq.kq_linear(a, w, out=torch.zeros(4, 7, dtype=torch.bfloat16))
