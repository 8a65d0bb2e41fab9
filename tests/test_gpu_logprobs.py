"""Token log-probabilities and their gradient on the GPU against the definitions in 64 bits.

Tolerances.  With d = scale (x - m) a term e = exp(d) is off by at most (|d| 2^-22 + 2^-22) of itself
(roundings of x - m and of two products, 2 ulp of the exponential), and a thread adds at most
vocab / 512 + 16 terms one after the other, each add 2^-24.  So S is off by at most
r = 2^-22 (E|d| + 1) + n 2^-24 of itself and lse, logp by r and a few roundings of themselves; W / S by
2^-22 (E d^2 + E|d|) + (n 2^-24 + r) E|d|.  Expectations are under the row's own distribution.
"""
import math

import pytest
import torch

import compressed_pseudo_gradient_gb300 as spl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = math.inf
LOW = torch.finfo(torch.float32).min
DTYPES = [torch.float32, torch.bfloat16]


def make(rows, vocab, dtype, seed, stride=None, offset=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    stride = stride or vocab
    buf = torch.full((rows * stride + offset,), 1e4, device=DEV).to(dtype)   # a stray read shows
    x = torch.as_strided(buf, (rows, vocab), (stride, 1), offset)
    x.copy_(torch.randn(rows, vocab, generator=g, device=DEV) * 3.0)
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    return x, t


def reference(x, t, scale):
    z = x.double() * scale
    m = z.max(1, keepdim=True).values
    lse = torch.logsumexp(z, 1)
    logq = z - lse[:, None]
    q = logq.exp()
    d = torch.where(q > 0, z - m, torch.zeros_like(z))
    ent = -(q * torch.where(q > 0, logq, torch.zeros_like(z))).sum(1)
    e1, e2 = (q * d.abs()).sum(1), (q * d * d).sum(1)
    logp = None if t is None else logq.gather(1, t.long()[:, None])[:, 0]
    return lse, ent, logp, logq, e1, e2


def order(x, k):
    """The k largest of each row, equal ones by ascending index."""
    return torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]


def check(x, t, scale=1.0, top=0):
    r = spl.token_logprobs(x, t, scale=scale, top=top)
    lse, ent, logp, logq, e1, e2 = reference(x, t, scale)
    n = x.shape[1] / 512 + 16
    rel = 2.0 ** -22 * (e1 + 1) + n * 2.0 ** -24
    own = 2.0 ** -22 * (1 + lse.abs())
    assert ((r.lse.double() - lse).abs() <= rel + own).all()
    tol = rel + 2.0 ** -22 * (e2 + e1) + (n * 2.0 ** -24 + rel) * e1 + 2.0 ** -22 * (1 + ent.abs() + e1)
    assert ((r.entropy.double() - ent).abs() <= tol).all()
    if t is not None:
        fin = torch.isfinite(logp)
        assert (torch.isneginf(r.logp) == ~fin).all()
        assert ((r.logp.double() - logp).abs() <= rel + 2.0 ** -22 * (1 + logp.abs()))[fin].all()
    if top:
        ids = order(x, top)
        assert torch.equal(r.top_ids, ids)
        want = logq.gather(1, ids)
        fin = torch.isfinite(want)
        assert (torch.isneginf(r.top_logp) == ~fin).all()
        assert ((r.top_logp.double() - want).abs() <= rel[:, None] + 2.0 ** -22 * (1 + want.abs()))[fin].all()
    return r


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 7), (2, 31), (4, 33), (7, 1000), (1, 4096),
                                        (2, 4097), (1, 65537), (3, 100003), (1, 262208), (700, 513),
                                        (33, 20000)])
def test_values_and_top(rows, vocab, dtype):
    x, t = make(rows, vocab, dtype, rows * 7 + vocab)
    for top in (0, 1, min(5, vocab), min(32, vocab)):
        check(x, t, scale=0.7 if top else 1.0, top=top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,extra", [(0, 1), (1, 0), (3, 5), (8, 8), (7, 3)])
def test_strides_and_alignments(offset, extra, dtype):
    for vocab in (5, 37, 2049, 9001):
        x, t = make(6, vocab, dtype, 3 + offset, stride=vocab + extra, offset=offset)
        check(x, t.int(), top=min(9, vocab))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_the_lower_id(dtype):
    g = torch.Generator(device=DEV).manual_seed(5)
    for rows, vocab in ((4, 50), (2, 5000), (1, 70000), (400, 3000)):
        x = torch.randint(-2, 3, (rows, vocab), generator=g, device=DEV).to(dtype)
        x[:, vocab // 2] = -0.0
        check(x, None, top=32)
    x = torch.zeros(3, 40000, device=DEV, dtype=dtype)
    assert torch.equal(check(x, None, top=32).top_ids[0].cpu(), torch.arange(32))
    # ascending rows: every value beats the list so far
    x = torch.arange(30000, device=DEV, dtype=torch.float32)[None].mul(1e-3).to(dtype)
    check(x, None, top=32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("low", [-INF, LOW])
def test_masked_logits(low, dtype):
    x, t = make(5, 6001, dtype, 11)
    low = max(low, torch.finfo(dtype).min) if low != -INF else low
    keep = x[4].clone()
    x[0, 1:] = low
    x[1, :-1] = low
    x[2, ::2] = low
    x[3, :4096] = low
    x[4] = keep
    t[0], t[1] = 0, 5
    r = check(x, t, top=3)
    assert abs(r.entropy[0].item()) == 0.0 and r.logp[0].item() == 0.0
    rep = spl.token_logprobs_grad(x, t, r.lse, torch.ones(5, device=DEV), entropy=r.entropy,
                                  d_entropy=torch.ones(5, device=DEV))
    assert torch.isfinite(rep.float()).all()
    masked = x == low
    masked[torch.arange(5), t] = False
    assert (rep[masked] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 9, 5000, 40001])
def test_a_row_of_nothing(vocab, dtype):
    x, t = make(3, vocab, dtype, 2)
    x[1] = -INF
    k = min(4, vocab)
    r = spl.token_logprobs(x, t, top=k)
    assert r.lse[1] == -INF and r.logp[1] == -INF and r.entropy[1] == 0 and (r.top_logp[1] == -INF).all()
    assert torch.equal(r.top_ids[1].cpu(), torch.arange(k))
    one = torch.ones(3, device=DEV)
    g = spl.token_logprobs_grad(x, t, r.lse, one, entropy=r.entropy, d_entropy=one)
    assert (g[1] == 0).all()
    check(x[::2], t[::2].contiguous(), top=k)
    # a row of the type's lowest value is uniform
    x[1] = torch.finfo(dtype).min
    r = spl.token_logprobs(x, t)
    assert abs(r.entropy[1].item() - math.log(vocab)) <= 2 ** -20 * (1 + math.log(vocab))


@pytest.mark.parametrize("bad", [math.nan, INF])
def test_nan_and_infinity_are_flagged(bad):
    x, t = make(4, 30001, torch.float32, 4)
    x[2, 12345] = bad
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = spl.token_logprobs(x, t, top=2, flags=flags)
    assert spl.flags_status(flags) == 4
    for v in (r.lse, r.entropy, r.logp, r.top_logp):
        assert torch.isnan(v[2]).all() and torch.isfinite(v[[0, 1, 3]]).all()
    assert r.top_ids[2, 0] == 12345


def test_targets_outside():
    x, t = make(4, 100, torch.float32, 4)
    t[0], t[1], t[2] = -100, -1, 100
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = spl.token_logprobs(x, t, flags=flags)
    assert r.logp[0] == 0 and r.logp[1] == 0 and torch.isnan(r.logp[2]) and torch.isfinite(r.logp[3])
    assert spl.flags_status(flags) == 7
    flags.zero_()
    g = spl.token_logprobs_grad(x, t, r.lse, torch.ones(4, device=DEV), flags=flags)
    assert spl.flags_status(flags) == 7 and (g[:3] == 0).all() and (g[3] != 0).any()


def grad_reference(x, t, lse, ent, g, h, scale):
    """The formula in 64 bits with the call's own lse and entropy, and each value's tolerance."""
    z, l, H = x.double() * scale, lse.double()[:, None], ent.double()[:, None]
    d = z - l
    p = d.exp()
    dead = p == 0
    d = d.masked_fill(dead, 0.0)
    z = z.masked_fill(dead, 0.0)
    w = (g.double() * (t >= 0))[:, None] if g is not None else torch.zeros_like(l)
    v = -w * p
    if g is not None:
        v.scatter_add_(1, t.clamp(min=0).long()[:, None], w)
    near = 2.0 ** -23 * (z.abs() + l.abs())                   # of d
    rel = near + d.abs() * 2.0 ** -22 + 2.0 ** -21            # of p
    tol = w.abs() * p * rel + 2.0 ** -22 * v.abs()
    if h is not None:
        hh = h.double()[:, None]
        v = v - hh * p * (d + H)
        tol = tol + hh.abs() * p * ((d + H).abs() * (rel + 2.0 ** -21) + near + 2.0 ** -22 * H.abs())
    return v * scale, tol * scale


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,extra,offset", [(1, 1, 0, 0), (4, 3, 0, 0), (3, 1000, 0, 0), (5, 4097, 0, 0),
                                                     (2, 9001, 7, 3), (3, 40000, 8, 0), (2, 100003, 0, 1)])
@pytest.mark.parametrize("terms", ["logp", "entropy", "both"])
def test_grad_formula(rows, vocab, extra, offset, dtype, terms):
    x, t = make(rows, vocab, dtype, vocab, stride=vocab + extra, offset=offset)
    t[0] = -100 if rows > 1 else t[0]
    g0 = torch.Generator(device=DEV).manual_seed(1)
    g = torch.randn(rows, generator=g0, device=DEV) if terms != "entropy" else None
    h = torch.randn(rows, generator=g0, device=DEV) if terms != "logp" else None
    r = spl.token_logprobs(x, t, scale=1.3)
    ref, tol = grad_reference(x, t, r.lse, r.entropy, g, h, 1.3)
    tol = tol + ref.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22) + 1e-38
    tt = None if g is None else t
    got = spl.token_logprobs_grad(x, tt, r.lse, g, entropy=r.entropy, d_entropy=h, scale=1.3)
    assert ((got.double() - ref).abs() <= tol).all()
    # rows that sit differently within 16 bytes, and in place: the same bits
    other = torch.empty(rows, vocab + 1, dtype=dtype, device=DEV)[:, 1:]
    spl.token_logprobs_grad(x, tt, r.lse, g, entropy=r.entropy, d_entropy=h, scale=1.3, out=other)
    assert torch.equal(other, got)
    spl.token_logprobs_grad(x, tt, r.lse, g, entropy=r.entropy, d_entropy=h, scale=1.3, out=x)
    assert torch.equal(x, got)


def test_grad_against_differences():
    """<gradient, direction> against central differences of the forward kernel: lse, logp and
    entropy are good to about 1e-6, the step is 2^-5, the third derivatives are of order 1."""
    x, t = make(6, 2000, torch.float32, 9)
    g0 = torch.Generator(device=DEV).manual_seed(2)
    g, h = (torch.randn(6, generator=g0, device=DEV) for _ in range(2))
    dirn = torch.randn(6, 2000, generator=g0, device=DEV)
    r = spl.token_logprobs(x, t, scale=0.9)
    grad = spl.token_logprobs_grad(x, t, r.lse, g, entropy=r.entropy, d_entropy=h, scale=0.9)
    step = 2.0 ** -5
    up, down = (spl.token_logprobs(x + s * step * dirn, t, scale=0.9) for s in (1, -1))
    per_row = lambda a, b: (a.double() - b.double()) / (2 * step)  # noqa: E731
    diff = g.double() * per_row(up.logp, down.logp) + h.double() * per_row(up.entropy, down.entropy)
    want = (grad.double() * dirn.double()).sum(1)
    assert ((diff - want).abs() <= 0.02 * (g.abs() + h.abs()).double() * (1 + want.abs())).all()


def test_side_stream_and_same_bits():
    x, t = make(40, 30000, torch.bfloat16, 6)
    a = spl.token_logprobs(x, t, top=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = x * 1
        b = spl.token_logprobs(y, t, top=8)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_empty_and_refusals():
    r = spl.token_logprobs(torch.empty(0, 10, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV))
    assert r.logp.shape == (0,)
    x, t = make(4, 10, torch.float32, 1)
    with pytest.raises(spl.SplError):
        spl.token_logprobs(x, t, top=11)
    with pytest.raises(spl.SplError):
        spl.token_logprobs(x, t, scale=0.0)
    with pytest.raises(ValueError):
        spl.token_logprobs(x, t[:3])
    with pytest.raises(ValueError):
        spl.token_logprobs(x.t(), t)
    with pytest.raises(TypeError):
        spl.token_logprobs(x.half(), t)
    with pytest.raises(TypeError):
        spl.token_logprobs(x, t.float())
    with pytest.raises(ValueError):
        spl.token_logprobs_grad(x, t, torch.zeros(4, device=DEV), None)
