"""Attention over packed sequences: the CUDA kernel against the formula in 64
bits, and the argument checks.

Tolerances.  A score s = scale q.k is off by e = (d / 16 + 8) 2^-23 scale sum
|q||k| (fp32 accumulation in the tensor cores) and 2^-22 (|s| + |m|) from the
exponent's fp32 argument; 2^x is good to 2^-21.  A weight p is then off by r =
e + 2^-22 (|s| + |m|) + 2^-21 relatively, and by the rounding u of the storage
type (for float16 also 2^-25, its subnormal spacing, the largest weight being at
least 1).  The product with v adds (klen / 16 + 8) 2^-23, and the result is
rounded once.  lse: the largest r, and klen 2^-24 for the sum.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from w4a4_mxfp4_activation_gb300 import kq

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SUB = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from w4a4_mxfp4_activation_gb300 import build
    build.build()
    kq.lib()


def offsets(lengths, start=0):
    return torch.tensor([start] + [start + sum(lengths[:i + 1]) for i in range(len(lengths))],
                        dtype=torch.int32, device="cuda")


def make(lq, lk, heads, kv_heads, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda n, h: torch.randn(n, h, d, generator=g, device="cuda")
    return ((1.5 * rnd(sum(lq), heads)).to(dtype), rnd(sum(lk), kv_heads).to(dtype),
            (rnd(sum(lk), kv_heads) + 0.3).to(dtype))


def check(out, lse, q, k, v, lq, lk, causal, scale=None, q0=0, k0=0):
    heads, d = q.shape[1:]
    grp = heads // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    u, sub = UNIT[q.dtype], SUB[q.dtype]
    for a, b in zip(lq, lk):
        for h in range(heads if a else 0):
            o, L = out[q0:q0 + a, h].double(), lse[q0:q0 + a, h].double()
            if b == 0:
                assert (o == 0).all() and (L == -math.inf).all()
                continue
            qq, kk, vv = q[q0:q0 + a, h].double(), k[k0:k0 + b, h // grp].double(), v[k0:k0 + b, h // grp].double()
            s = scale * qq @ kk.t()
            e = (d / 16 + 8) * 2.0 ** -23 * scale * (qq.abs() @ kk.abs().t())
            if causal:
                i = torch.arange(a, device="cuda")[:, None] + (b - a)
                hide = torch.arange(b, device="cuda")[None] > i
                s, e = s.masked_fill(hide, -math.inf), e.masked_fill(hide, 0)
            want = torch.logsumexp(s, 1)
            empty = want == -math.inf
            assert (o[empty] == 0).all() and (L[empty] == -math.inf).all()
            p = torch.exp(s - want.masked_fill(empty, 0)[:, None])
            big = s.abs().masked_fill(s == -math.inf, 0)
            r = e + 2.0 ** -22 * (big + big.amax(1, keepdim=True)) + 2.0 ** -21
            pv = p @ vv
            size = p @ vv.abs()
            # the weights in units of their sum, which is at least the largest
            off = ((p * r) @ vv.abs() + (p * r).sum(1, keepdim=True) * pv.abs()
                   + (u + (b / 16 + 8) * 2.0 ** -23 + b * 2.0 ** -24) * size + sub * vv.abs().sum(0))
            tol = off + u * 1.01 * (pv.abs() + off) + sub
            assert ((o - pv).abs() <= tol)[~empty].all(), (a, b, h, float(((o - pv).abs() / tol).max()))
            ltol = r.amax(1) + b * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * want.abs()
            assert ((L - want).abs() <= ltol)[~empty].all()
        q0, k0 = q0 + a, k0 + b


def run(lq, lk, heads, kv_heads, d, dtype, causal, seed=0, **kw):
    q, k, v = make(lq, lk, heads, kv_heads, d, dtype, seed)
    out, lse = kq.kq_attention(q, k, v, offsets(lq), offsets(lk), max(lq + [1]), max(lk + [1]),
                               causal=causal, lse=True, **kw)
    check(out, lse, q, k, v, lq, lk, causal, kw.get("scale"))
    return out, lse


DTYPES = [torch.bfloat16, torch.float16]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [8, 32, 64, 72, 120, 128])
def test_one_sequence_of_each_width(d, causal, dtype):
    run([300], [300], 4, 2, d, dtype, causal, seed=d)


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 383, 1000])
def test_lengths(n, causal):
    run([n], [n], 2, 2, 64, torch.bfloat16, causal, seed=n)


@gpu
@pytest.mark.parametrize("group,kv_heads", [(1, 5), (2, 3), (3, 2), (5, 1), (6, 2), (7, 1), (8, 2), (12, 1),
                                            (40, 1), (96, 1), (130, 1), (131, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_groups(group, kv_heads, causal):
    """Tiles of 128 // group tokens, groups that do not divide 128, and groups
    larger than a tile."""
    run([37, 0, 150], [37, 5, 150], group * kv_heads, kv_heads, 32, torch.bfloat16, causal, seed=group)


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_packed_lengths(causal, dtype):
    """Empty sequences, sequences without keys or queries, fewer queries than
    keys and more (rows that see no key)."""
    lq = [5, 0, 300, 1, 17, 0, 129, 64, 2, 200]
    lk = [5, 7, 300, 40, 0, 0, 513, 64, 1000, 60]
    run(lq, lk, 8, 2, 64, dtype, causal, seed=9)


@gpu
@pytest.mark.parametrize("causal", [False, True])
def test_many_sequences(causal):
    """More sequences than one look of the scheduler holds, most of them short."""
    lq = [(7 * i) % 23 for i in range(150)]
    lk = [(11 * i) % 41 for i in range(150)]
    run(lq, lk, 4, 4, 32, torch.bfloat16, causal, seed=4)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lk", [[1], [127], [129], [2048], [5000, 3, 0, 777, 4096], [33000]])
def test_single_tokens_against_a_cache(lk, d):
    run([1] * len(lk), lk, 16, 2, d, torch.bfloat16, True, seed=len(lk))


@gpu
@pytest.mark.parametrize("lq", [[3, 9, 1], [70, 33, 128]])
def test_few_queries_against_a_cache(lq):
    run(lq, [1500, 9000, 257], 8, 1, 128, torch.float16, True, seed=2)


@gpu
@pytest.mark.parametrize("causal", [False, True])
def test_whole_items_on_every_sm(causal):
    """More items than SMs, several rounds, ragged ends."""
    run([1111, 900, 2050, 333], [1111, 900, 2050, 333], 24, 24, 128, torch.bfloat16, causal, seed=1)


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads,kv_heads,lq,lk", [
    (2, 2, [2000, 300, 0, 1500], [2000, 700, 9, 1500]),
    (2, 2, [9000], [9000]),                                 # shares of tile pairs
    (8, 2, [1000, 1, 129], [3000, 12500, 129]),
    (24, 24, [700], [700]),
    (1, 1, [2050], [2050])])
def test_shares_of_tile_pairs(heads, kv_heads, lq, lk, causal):
    """Fewer tile pairs than SMs, at both sides of the choice of single tiles."""
    run(lq, lk, heads, kv_heads, 64, torch.bfloat16, causal, seed=heads)


@gpu
def test_scale_and_growing_scores():
    """Scores that grow along the keys raise the running maximum in every tile,
    and a small scale leaves all weights alike."""
    q, k, v = make([200], [900], 2, 1, 64, torch.bfloat16, 3)
    k = (k.float() * torch.linspace(0.1, 12.0, 900, device="cuda")[:, None, None]).bfloat16()
    for scale in (0.001, 0.125, 1.0):
        out, lse = kq.kq_attention(q, k, v, offsets([200]), offsets([900]), 200, 900, causal=False,
                                   scale=scale, lse=True)
        check(out, lse, q, k, v, [200], [900], False, scale)


@gpu
def test_strides_and_offsets():
    """Views of a packed QKV tensor, head-major tensors, sequences that start
    past row 0, and rows of no sequence, which stay as they were."""
    lq, h, hk, d = [100, 60], 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    qkv = torch.randn(180, h + 2 * hk, d + 8, generator=g, device="cuda").bfloat16()[:, :, :d]
    q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    out = torch.full((180, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = offsets(lq, 10)
    res, lse = kq.kq_attention(q, k, v, cu, cu, 100, 100, lse=True, out=out)
    check(res, lse, q, k, v, lq, lq, True, q0=10, k0=10)
    assert (out[:10] == 7.0).all() and (out[170:] == 7.0).all()
    major = lambda t: t.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    again = torch.zeros(h, 180, d, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)
    kq.kq_attention(major(q), major(k), major(v), cu, cu, 100, 100, out=again)
    assert torch.equal(again[10:170], res[10:170])


@gpu
@pytest.mark.parametrize("causal", [False, True])
def test_non_finite_values_stay_in_their_sequence(causal):
    lens = [100, 77, 45, 300]
    q, k, v = make(lens, lens, 4, 2, 128, torch.bfloat16, 8)
    cu = offsets(lens)
    clean, _ = kq.kq_attention(q, k, v, cu, cu, 300, 300, causal=causal, lse=True)
    bad = slice(100, 177)
    k[bad], v[bad] = float("nan"), float("inf")
    out, lse = kq.kq_attention(q, k, v, cu, cu, 300, 300, causal=causal, lse=True)
    keep = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(out[keep], clean[keep])
    assert torch.isnan(out[bad]).all()


@gpu
def test_long_cache_offsets_past_31_bits():
    """Rows of k and v whose element offsets pass 2^31."""
    tk, hk, d = (1 << 31) // (128 * 8) + 3000, 8, 128
    k = torch.zeros(tk, hk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    q, kk, vv = make([3], [2900], 8, hk, d, torch.bfloat16, 5)
    k[-2900:], v[-2900:] = kk, vv
    cu_k = torch.tensor([0, tk - 2900, tk], dtype=torch.int32, device="cuda")
    cu_q = torch.tensor([0, 0, 3], dtype=torch.int32, device="cuda")
    out, lse = kq.kq_attention(q, k, v, cu_q, cu_k, 3, 2900, lse=True)
    check(out, lse, q, kk, vv, [3], [2900], True)


@gpu
def test_offsets_out_of_range_are_clamped():
    q, k, v = make([64], [64], 2, 2, 64, torch.bfloat16, 7)
    cu = torch.tensor([-5, 32, 1000], dtype=torch.int32, device="cuda")
    out, lse = kq.kq_attention(q, k, v, cu, cu, 32, 32, lse=True)
    check(out, lse, q, k, v, [32, 32], [32, 32], True)


@gpu
@pytest.mark.parametrize("tq,cu", [(64, [0, 64, 0, 64, 0, 64]), (3, [0, 3] * 60), (300, [300, 0, 300, 100])])
def test_falling_offsets_stay_in_range(tq, cu):
    """Offsets that fall are an error of the caller's: the result is not defined,
    but nothing outside the outputs is touched."""
    q, k, v = make([tq], [tq], 2, 2, 64, torch.bfloat16, 7)
    buf = torch.full((tq + 64, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kq.kq_attention(q, k, v, cu, cu, out=buf[:tq])
    torch.cuda.synchronize()
    assert (buf[tq:] == 7.0).all()


@gpu
def test_empty_bounds_stream_and_repeatable():
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert kq.kq_attention(e, e, e, offsets([0]), offsets([0]), 0).shape == (0, 4, 64)
    lq, lk = [1, 4, 300], [3000, 90, 300]
    q, k, v = make(lq, lk, 8, 2, 128, torch.bfloat16, 11)
    first, _ = run(lq, lk, 8, 2, 128, torch.bfloat16, True, seed=11)
    # a wrong bound of the key lengths changes the schedule only
    for max_k in (None, 1, 10 ** 6):
        out, lse = kq.kq_attention(q, k, v, offsets(lq), offsets(lk), 1, max_k, lse=True)
        check(out, lse, q, k, v, lq, lk, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = kq.kq_attention(q, k, v, offsets(lq), offsets(lk), 300)
    s.synchronize()
    assert torch.equal(first, again)


@gpu
def test_without_keys():
    q = torch.randn(5, 2, 64, device="cuda").bfloat16()
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = kq.kq_attention(q, k, k, offsets([5]), offsets([0]), 5, lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


# --- argument checks (no GPU) ---------------------------------------------------------

FAKE = 1 << 20


def _att(q=FAKE, qs=(256, 64), k=FAKE, ks=(128, 64), v=FAKE, vs=(128, 64), fmt=0, cu_q=FAKE, cu_k=FAKE,
         nseq=2, tq=8, tk=8, heads=4, kv=2, d=64, max_k=4096, causal=1, scale=0.125, out=FAKE, os=(256, 64),
         lse=None, work=FAKE):
    return kq.lib().kq_attention(q, *qs, k, *ks, v, *vs, fmt, cu_q, cu_k, nseq, tq, tk, heads, kv, d,
                                 max_k, causal, scale, out, *os, lse, work, None)


def test_argument_checks():
    assert _att(fmt=2) == 4 and _att(fmt=-1) == 4
    assert _att(d=60) == 2 and _att(d=0) == 2 and _att(d=136) == 2 and _att(heads=3) == 2
    assert _att(kv=0) == 2 and _att(tq=-1) == 2 and _att(tk=-1) == 2 and _att(nseq=-1) == 2
    assert _att(max_k=-1) == 2 and _att(tq=1 << 31) == 2 and _att(heads=1 << 17, kv=1 << 16) == 2
    assert _att(scale=0.0) == 2 and _att(scale=-1.0) == 2 and _att(scale=float("nan")) == 2
    assert _att(scale=float("inf")) == 2
    assert _att(qs=(256, 32)) == 2 and _att(ks=(32, 64)) == 2 and _att(os=(0, 64)) == 2
    assert _att(q=None) == 1 and _att(k=None) == 1 and _att(v=None) == 1 and _att(out=None) == 1
    assert _att(cu_q=None) == 1 and _att(cu_k=None) == 1 and _att(work=None) == 1
    assert _att(q=FAKE + 2) == 3 and _att(out=FAKE + 8) == 3 and _att(work=FAKE + 4) == 3
    assert _att(qs=(260, 64)) == 3 and _att(vs=(128, 68)) == 3 and _att(cu_q=FAKE + 2) == 3
    assert _att(lse=FAKE + 1) == 3
    assert _att(tq=0, q=None) == 0 and _att(nseq=0, cu_q=None) == 0


def test_workspace_bytes():
    size = kq.lib().kq_attention_bytes
    assert size(0, 2, 4, 2, 64, 4096) == 0 and size(8, 2, 4, 3, 64, 4096) == 0
    assert size(8, 2, 4, 2, 60, 4096) == 0
    assert size(8, 8, 32, 8, 128, 4096) > 0                  # few items: split
    assert size(8, 8, 32, 8, 128, 100) == 0                  # short keys: whole items
    assert size(16384, 1, 24, 24, 128, 16384) == 0           # whole items fill the SMs


def test_binding_refusals():
    q = torch.zeros(8, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    with pytest.raises(ValueError):
        kq.kq_attention(q, k, k[:4], cu, cu, 8)
    with pytest.raises(ValueError):
        kq.kq_attention(q, k.half(), k.half(), cu, cu, 8)
    with pytest.raises(TypeError):
        kq.kq_attention(q.float(), k.float(), k.float(), cu.long(), cu, 8)
    with pytest.raises(ValueError):
        kq.kq_attention(q, k, k, cu, torch.tensor([0, 4, 8], dtype=torch.int32), 8)
    with pytest.raises(ValueError):
        kq.kq_attention(q.transpose(1, 2), k.transpose(1, 2), k.transpose(1, 2), cu, cu, 8)
    with pytest.raises(ValueError):
        kq.kq_attention(q, k, k, cu, cu, 8, out=torch.zeros(8, 4, 32, dtype=torch.bfloat16))
