"""Layer norm, forward and backward: the CUDA kernels against the formulas in
64 bits, against differences, and the argument checks.

Tolerances come from the arithmetic.  u32 = 2^-24 bounds one fp32 rounding and
u the final rounding to the storage type.  A sum over a row adds at most 32
elements per thread and then halves at most 10 times, and its terms and result
take a few roundings each, so a row sum is off by at most 64 u32 times the sum
of the terms' sizes.  A sum over R rows, in any order, is off by at most
(R + 8) u32 times the sum of the terms' sizes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from w4a4_mxfp4_activation_gb300 import kq

U32 = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
EPS = 1e-6
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from w4a4_mxfp4_activation_gb300 import build
    build.build()
    kq.lib()


def rows(values, dtype, extra=0, fill=float("nan")):
    """values [m, d] in rows of a pitch of a multiple of 16 bytes, ``extra``
    chunks longer than needed, with ``fill`` after the d columns."""
    m, d = values.shape
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((m, d + (-d) % unit + extra * unit), fill, dtype=dtype, device="cuda")
    buf[:, :d] = values.to(dtype)
    return buf[:, :d]


def inputs(m, d, dtype, group_rows, seed, extra=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    groups = 1 if group_rows == 0 else -(-m // group_rows)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = rnd(m, d) * torch.exp(0.5 * rnd(m, 1)) + 2.0 * rnd(m, 1)
    return (rows(x, dtype, extra), rows(rnd(m, d), dtype, extra), 1 + 0.3 * rnd(groups, d),
            0.2 * rnd(groups, d))


def per_row(t, m, group_rows):
    """[groups, d] parameters as fp64 rows [m, d]."""
    at = torch.zeros(m, dtype=torch.long, device=t.device) if group_rows == 0 else \
        torch.arange(m, device=t.device) // group_rows
    return t.double()[at]


def reference(x, w, b):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + EPS)
    z = (x - mean) * rstd
    return z * w + b, mean, rstd, z


def reference_grad(dy, z, rstd, w):
    g = dy.double() * w
    c1, c2 = g.mean(1, keepdim=True), (g * z).mean(1, keepdim=True)
    return rstd * (g - c1 - z * c2), dy.double() * z, g


def group_sum(t, m, group_rows):
    r = m if group_rows == 0 else group_rows
    return torch.stack([t[i:i + r].sum(0) for i in range(0, m, r)])


# one row and one column, ragged ends, every team size, row counts that leave
# teams and slices partly empty, groups that end inside a slice
SHAPES = [(1, 1, 0), (1, 1152, 0), (3, 7, 0), (5, 33, 2), (129, 511, 0), (130, 513, 40),
          (257, 1152, 64), (61, 1290, 0), (63, 2240, 1), (40, 4608, 7), (33, 5601, 0),
          (19, 12288, 19), (5, 16384, 3), (2000, 96, 1999)]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,d,group_rows", SHAPES)
def test_forward(m, d, group_rows, dtype):
    x, _, w, b = inputs(m, d, dtype, group_rows, 7 * m + d, extra=1)
    y, mean, rstd = kq.kq_layer_norm(x, w, b, EPS, group_rows=group_rows, stats=True)
    wr, br = per_row(w, m, group_rows), per_row(b, m, group_rows)
    ref, mean64, rstd64, z = reference(x, wr, br)
    size = x.double().abs().mean(1, keepdim=True)
    off_mean = 64 * U32 * size
    # the centred squares: 64 roundings, and the error of the mean twice over
    rel = 80 * U32 + off_mean * rstd64
    assert ((mean.double() - mean64[:, 0]).abs() <= off_mean[:, 0] + U32 * mean64[:, 0].abs()).all()
    assert ((rstd.double() - rstd64[:, 0]).abs() <= (rel * rstd64)[:, 0]).all()
    tol = (wr.abs() * (rstd64 * off_mean + z.abs() * rel) + 4 * U32 * (ref.abs() + br.abs())
           + UNIT[dtype] * ref.abs() * 1.01 + TINY[dtype])
    assert ((y.double() - ref).abs() <= tol).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,d,group_rows", SHAPES)
def test_backward(m, d, group_rows, dtype):
    x, dy, w, _ = inputs(m, d, dtype, group_rows, 11 * m + d, extra=2)
    wr = per_row(w, m, group_rows)
    _, mean, rstd, _ = reference(x, wr, torch.zeros_like(wr))
    mean, rstd = mean.float(), rstd.float()             # the gradient's own inputs
    z = (x.double() - mean.double()) * rstd.double()
    ref, ref_dw, g = reference_grad(dy, z, rstd.double(), wr)
    dx, dw, db = kq.kq_layer_norm_backward(dy, x, w, mean[:, 0], rstd[:, 0], group_rows=group_rows)
    # z takes two roundings: (x - mean) and the product with rstd
    sums = 64 * U32 * (g.abs().mean(1, keepdim=True)
                       + z.abs() * (g * z).abs().mean(1, keepdim=True))
    tol = (rstd.double() * (sums + 8 * U32 * (g.abs() + z.abs() * (g * z).abs().mean(1, keepdim=True)))
           + UNIT[dtype] * ref.abs() * 1.01 + TINY[dtype])
    assert ((dx.double() - ref).abs() <= tol).all()
    R = m if group_rows == 0 else min(m, group_rows)
    for got, terms in ((dw, ref_dw), (db, dy.double())):
        want = group_sum(terms, m, group_rows)
        tol = (R + 8) * U32 * group_sum(terms.abs(), m, group_rows)
        assert got.shape == want.shape
        assert ((got.double() - want).abs() <= tol + 2.0 ** -149).all()


@gpu
def test_backward_many_rows_few_columns():
    """Every slice of the column sums, and their sum over slices."""
    m, d = 70001, 40
    x, dy, w, _ = inputs(m, d, torch.bfloat16, 0, 3)
    _, mean, rstd, _ = reference(x, w.double(), torch.zeros_like(w).double())
    mean, rstd = mean.float(), rstd.float()
    _, dw, db = kq.kq_layer_norm_backward(dy, x, w, mean[:, 0], rstd[:, 0])
    z = (x.double() - mean.double()) * rstd.double()
    for got, terms in ((dw, dy.double() * z), (db, dy.double())):
        # chains of at most 58 rows a team, 4 teams, and the slices' sums
        tol = (58 + 4 + 304 + 8) * U32 * terms.abs().sum(0)
        assert ((got[0].double() - terms.sum(0)).abs() <= tol).all()


@gpu
def test_backward_against_differences():
    """<dx, v>, <dweight, v> and <dbias, v> against central differences of the
    loss sum(dy * y) in 64 bits."""
    m, d, group = 12, 200, 5
    x, dy, w, b = inputs(m, d, torch.float32, group, 21)
    _, mean, rstd = kq.kq_layer_norm(x, w, b, EPS, group_rows=group, stats=True)
    dx, dw, db = kq.kq_layer_norm_backward(dy, x, w, mean, rstd, group_rows=group)

    def loss(x, w, b):
        return (dy.double() * reference(x, per_row(w, m, group), per_row(b, m, group))[0]).sum()

    g = torch.Generator(device="cuda").manual_seed(5)
    args = [x.double(), w.double(), b.double()]
    for i, grad in enumerate((dx, dw, db)):
        v = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * v, args[i] - h * v
        diff = (loss(*up) - loss(*down)) / (2 * h)
        got = (grad.double() * v).sum()
        # fp32 gradients: 200 u32 of each term; h^2 of the third derivative
        tol = 200 * U32 * (grad.double().abs() * v.abs()).sum() + 1e-6 * diff.abs() + 1e-6
        assert (got - diff).abs() <= tol


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_parameters_and_columns_past_d_stay(dtype):
    m, d = 9, 1153
    x, dy, _, _ = inputs(m, d, dtype, 0, 4)
    out = torch.full((m, 1168), 7.0, dtype=dtype, device="cuda")
    y = out[:, :d]
    kq.kq_layer_norm(x, y=y)
    ref = reference(x, 1.0, 0.0)[0]
    assert ((y.double() - ref).abs() <= 2 * UNIT[dtype] * ref.abs() + 1e-5).all()
    assert (out[:, d:] == 7.0).all()
    mean, rstd = x.double().mean(1), reference(x, 1.0, 0.0)[2][:, 0]
    out.fill_(7.0)
    kq.kq_layer_norm_backward(dy, x, None, mean.float(), rstd.float(), dx=y)
    assert (out[:, d:] == 7.0).all() and torch.isfinite(y).all()


@gpu
def test_optional_outputs_of_the_backward_pass():
    m, d = 700, 320
    x, dy, w, _ = inputs(m, d, torch.bfloat16, 0, 8)
    _, mean, rstd = kq.kq_layer_norm(x, w, None, stats=True)
    dx, dw, db = kq.kq_layer_norm_backward(dy, x, w, mean, rstd)
    L, p = kq.lib(), lambda t: t.data_ptr()
    work = torch.empty(kq.lib().kq_layer_norm_backward_bytes(m, d, 0), dtype=torch.uint8,
                       device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    common = (p(dy), d, p(x), d, 0, m, d, p(w), 0, p(mean), p(rstd))
    only = torch.empty_like(dw)
    assert L.kq_layer_norm_backward(*common, None, 0, p(only), None, p(work), s) == 0
    assert torch.equal(only, dw)
    assert L.kq_layer_norm_backward(*common, None, 0, None, p(only), p(work), s) == 0
    assert torch.equal(only, db)
    alone = torch.empty_like(dx)
    assert L.kq_layer_norm_backward(*common, p(alone), d, None, None, None, s) == 0
    assert torch.equal(alone, dx)


@gpu
def test_empty_and_special_values():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert kq.kq_layer_norm(x).shape == (0, 64)
    z = torch.empty(0, device="cuda")
    dx, dw, db = kq.kq_layer_norm_backward(x, x, None, z, z)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    # a constant row has no spread: y is the bias; a NaN or an infinity stays in its row
    x = torch.randn(8, 1160, device="cuda").bfloat16()
    x[2] = 3.0
    x[4, 17] = float("inf")
    x[6, 1159] = float("nan")
    b = torch.randn(1160, device="cuda")
    y = kq.kq_layer_norm(x, None, b)
    assert torch.equal(y[2], b.bfloat16())
    assert torch.isnan(y[4]).any() and torch.isnan(y[6]).all()
    for i in (0, 1, 3, 5, 7):
        assert torch.isfinite(y[i]).all()


@gpu
def test_other_stream_and_repeatable():
    m, d = 3000, 1152
    x, dy, w, b = inputs(m, d, torch.bfloat16, 0, 12)
    y, mean, rstd = kq.kq_layer_norm(x, w, b, stats=True)
    first = kq.kq_layer_norm_backward(dy, x, w, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2 = kq.kq_layer_norm(x, w, b)
        again = kq.kq_layer_norm_backward(dy, x, w, mean, rstd)
    s.synchronize()
    assert torch.equal(y, y2)
    assert all(torch.equal(p, q) for p, q in zip(first, again))


# --- argument checks (no GPU) ---------------------------------------------------------

FAKE = 1 << 20


def _fwd(x=FAKE, ldx=64, fmt=0, m=4, d=64, w=FAKE, b=FAKE, group=0, eps=1e-6, y=FAKE, ldy=64,
         mean=None, rstd=None):
    return kq.lib().kq_layer_norm(x, ldx, fmt, m, d, w, b, group, eps, y, ldy, mean, rstd, None)


def test_forward_argument_checks():
    assert _fwd(fmt=3) == 4 and _fwd(fmt=-1) == 4
    assert _fwd(m=-1) == 2 and _fwd(d=0) == 2 and _fwd(d=16385, ldx=16392, ldy=16392) == 2
    assert _fwd(ldx=56) == 2 and _fwd(ldy=56) == 2 and _fwd(group=-1) == 2
    assert _fwd(eps=-1.0) == 2 and _fwd(eps=float("nan")) == 2
    assert _fwd(m=1 << 31) == 2
    assert _fwd(x=None) == 1 and _fwd(y=None) == 1
    assert _fwd(x=FAKE + 2) == 3 and _fwd(y=FAKE + 8) == 3 and _fwd(w=FAKE + 4) == 3
    assert _fwd(b=FAKE + 4) == 3 and _fwd(mean=FAKE + 2) == 3 and _fwd(rstd=FAKE + 1) == 3
    assert _fwd(ldx=66) == 3 and _fwd(ldy=68) == 3 and _fwd(fmt=2, ldx=66) == 3
    assert _fwd(m=0, x=None, y=None) == 0


def _bwd(dy=FAKE, lddy=64, x=FAKE, ldx=64, fmt=0, m=4, d=64, w=FAKE, group=0, mean=FAKE,
         rstd=FAKE, dx=FAKE, lddx=64, dw=FAKE, db=FAKE, work=FAKE):
    return kq.lib().kq_layer_norm_backward(dy, lddy, x, ldx, fmt, m, d, w, group, mean, rstd, dx,
                                           lddx, dw, db, work, None)


def test_backward_argument_checks():
    assert _bwd(fmt=7) == 4 and _bwd(m=-1) == 2 and _bwd(d=0) == 2 and _bwd(group=-2) == 2
    assert _bwd(ldx=32) == 2 and _bwd(lddy=32) == 2 and _bwd(lddx=32) == 2
    assert _bwd(dy=None) == 1 and _bwd(x=None) == 1 and _bwd(mean=None) == 1
    assert _bwd(rstd=None) == 1 and _bwd(m=64, work=None) == 1
    assert _bwd(dy=FAKE + 2) == 3 and _bwd(dx=FAKE + 2) == 3 and _bwd(dw=FAKE + 2) == 3
    assert _bwd(work=FAKE + 8) == 3 and _bwd(lddx=68) == 3
    assert _bwd(dx=None, dw=None, db=None, work=None) == 0
    assert _bwd(m=0, group=8, dy=None, x=None) == 0


def test_backward_workspace_bytes():
    size = kq.lib().kq_layer_norm_backward_bytes
    assert size(1, 64, 0) == 0 and size(0, 64, 0) == 0 and size(-1, 64, 0) == 0
    assert size(4, 0, 0) == 0 and size(4, 64, 1) == 0
    # at most 152 slices and one more per group, two fp32 rows of whole chunks each
    for m, d, group in ((4096, 1152, 0), (65536, 1150, 4096), (1000, 96, 100)):
        groups = 1 if group == 0 else -(-m // group)
        row = (d + 7) // 8 * 8
        assert 0 < size(m, d, group) <= (152 + groups) * 2 * row * 4
        assert size(m, d, group) % (groups * 2 * row * 4) == 0


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        kq.kq_layer_norm(x.to(torch.int32))
    with pytest.raises(ValueError):
        kq.kq_layer_norm(x.t())
    with pytest.raises(ValueError):
        kq.kq_layer_norm(x, torch.ones(63))
    with pytest.raises(TypeError):
        kq.kq_layer_norm(x, torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        kq.kq_layer_norm(x, y=torch.zeros(4, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        kq.kq_layer_norm_backward(x[:2], x, None, torch.zeros(4), torch.zeros(4))
