"""Embedding lookup and its gradient on the GPU against the definitions in 64 bits."""
import math

import pytest
import torch

import compressed_pseudo_gradient_gb300 as spl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.bfloat16]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def padded(rows, cols, dtype, extra, offset, g):
    buf = torch.full((rows * (cols + extra) + offset,), 1e30, device=DEV).to(dtype)
    x = torch.as_strided(buf, (rows, cols), (cols + extra, 1), offset)
    x.copy_(torch.randn(rows, cols, generator=g, device=DEV))
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("count,vocab,width,extra,offset", [
    (1, 1, 1, 0, 0), (3, 10, 7, 0, 0), (100, 50, 64, 0, 0), (17, 33, 1001, 0, 0), (5, 9, 8192, 8, 0),
    (1000, 3000, 40, 24, 8), (7, 20, 100, 1, 3), (1, 5, 4096, 0, 0)])
def test_lookup_is_one_rounding(count, vocab, width, extra, offset, dtype):
    g = gen(count + width)
    table = padded(vocab, width, dtype, extra, offset, g)
    ids = torch.randint(0, vocab, (count,), generator=g, device=DEV)
    for scale in (1.0, math.sqrt(width)):
        want = (table[ids].float() * torch.tensor(scale, dtype=torch.float32)).to(dtype)
        for i in (ids, ids.int()):
            assert torch.equal(spl.embedding(i, table, scale=scale), want)
    wide = torch.full((count, width + 5), 3.0, device=DEV, dtype=dtype)
    spl.embedding(ids, table, out=wide[:, 2:2 + width])
    assert torch.equal(wide[:, 2:2 + width], table[ids])
    assert (wide[:, :2] == 3).all() and (wide[:, 2 + width:] == 3).all()


def test_lookup_shapes_and_bad_ids():
    table = torch.randn(10, 12, device=DEV)
    ids = torch.tensor([[0, 9, -1], [10, 3, 1 << 40]], device=DEV)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = spl.embedding(ids, table, flags=flags)
    assert out.shape == (2, 3, 12) and spl.flags_status(flags) == 7
    assert (out[0, 2] == 0).all() and (out[1, 0] == 0).all() and (out[1, 2] == 0).all()
    assert torch.equal(out[0, 0], table[0]) and torch.equal(out[1, 1], table[3])
    assert spl.embedding(ids[:0], table).shape == (0, 3, 12)


def reference(ids, d_out, vocab, scale):
    """The sums in 64 bits and a bound on any order of adding them in fp32."""
    width = d_out.shape[-1]
    ok = (ids >= 0) & (ids < vocab)
    x = d_out[ok].double()
    ref = torch.zeros(vocab, width, dtype=torch.float64, device=DEV).index_add_(0, ids[ok].long(), x)
    size = torch.zeros_like(ref).index_add_(0, ids[ok].long(), x.abs())
    n = torch.bincount(ids[ok].long(), minlength=vocab).double()[:, None]
    return ref * scale, abs(scale) * size * (n + 2) * 2.0 ** -24


CASES = [(1, 1, 1), (1, 100, 64), (5, 3, 7), (64, 10, 33), (65, 1, 128), (200, 4, 1000), (129, 70, 8),
         (1000, 2000, 300), (2048, 262208, 16), (2049, 5000, 24), (5000, 50, 96), (20000, 100000, 40),
         (9000, 9, 2050)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("count,vocab,width", CASES)
def test_grad_sums(count, vocab, width, dtype):
    g = gen(count * 3 + vocab)
    d_out = torch.randn(count, width, generator=g, device=DEV).to(dtype)
    u = torch.rand(count, generator=g, device=DEV)
    ids = (u.pow(4) * vocab).long().clamp(max=vocab - 1)
    ref, tol = reference(ids, d_out, vocab, 1.7)
    out = torch.full((vocab, width), math.nan, device=DEV)     # every row is written
    got = spl.embedding_grad(ids, d_out, vocab, scale=1.7, out=out)
    assert got is out and ((got.double() - ref).abs() <= tol).all()
    assert torch.equal(spl.embedding_grad(ids.int(), d_out, vocab, scale=1.7), got)
    base = torch.randn(vocab, width, generator=g, device=DEV)
    acc = base.clone()
    spl.embedding_grad(ids, d_out, vocab, scale=1.7, out=acc, accumulate=True)
    assert ((acc.double() - (base.double() + ref)).abs() <= tol + 2.0 ** -23 * (base.abs() + ref.abs())).all()
    untouched = torch.ones(vocab, dtype=torch.bool, device=DEV)
    untouched[ids] = False
    assert torch.equal(acc[untouched], base[untouched])


@pytest.mark.parametrize("width,lengths", [
    # sums are split every 16 tokens and again every 512 (every 32 and 1,024, 64 and 2,048 for the
    # last two): runs that end and begin there, beside it, and reach over many of them
    (33, [512, 512, 1, 511, 16, 496, 1024, 15, 497, 513, 3, 4096, 17]),
    (64, [4097, 15, 16, 1, 30000, 2, 510, 512, 1]),
    (520, [511, 1537, 16, 2048, 1, 1, 512 * 7 - 2, 600]),
    (1000, [1, 1023, 1024, 2047, 32, 33, 4096, 31, 20000]),
    (1000, [2048, 2047, 1, 1, 4095, 64, 65, 63, 40000, 4096, 20000])])
@pytest.mark.parametrize("dtype", DTYPES)
def test_grad_of_long_runs(width, lengths, dtype):
    g = gen(width + len(lengths))
    vocab = len(lengths) + 1
    ids = torch.arange(vocab - 1, device=DEV).repeat_interleave(torch.tensor(lengths, device=DEV))
    ids = ids[torch.randperm(ids.numel(), generator=g, device=DEV)]
    d_out = torch.randn(ids.numel(), width, generator=g, device=DEV).to(dtype)
    ref, tol = reference(ids, d_out, vocab, 0.7)
    got = spl.embedding_grad(ids, d_out, vocab, scale=0.7)
    assert ((got.double() - ref).abs() <= tol).all()
    assert torch.equal(spl.embedding_grad(ids, d_out, vocab, scale=0.7), got)
    base = torch.randn(vocab, width, generator=g, device=DEV)
    acc = base.clone()
    spl.embedding_grad(ids, d_out, vocab, scale=0.7, out=acc, accumulate=True)
    assert ((acc.double() - (base.double() + ref)).abs() <= tol + 2.0 ** -23 * (base.abs() + ref.abs())).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_grad_strides_padding_and_bad_ids(dtype):
    g = gen(1)
    count, vocab, width = 700, 40, 72
    d_out = padded(count, width, dtype, 5, 3, g)
    ids = torch.randint(-2, vocab + 2, (count,), generator=g, device=DEV)
    ids[100:300] = 7
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    ref, tol = reference(torch.where(ids == 7, -1, ids), d_out, vocab, 0.5)
    wide = torch.full((vocab, width + 3), 2.0, device=DEV)
    spl.embedding_grad(ids, d_out, vocab, scale=0.5, padding_id=7, out=wide[:, 1:1 + width], flags=flags)
    assert spl.flags_status(flags) == 7
    assert ((wide[:, 1:1 + width].double() - ref).abs() <= tol).all()
    assert (wide[7, 1:1 + width] == 0).all()
    assert (wide[:, 0] == 2).all() and (wide[:, 1 + width:] == 2).all()
    flags.zero_()
    ok = ids.clamp(0, vocab - 1)
    spl.embedding_grad(ok, d_out, vocab, padding_id=7, flags=flags)
    assert spl.flags_status(flags) == 0


def test_grad_of_nothing_and_of_only_padding():
    ids = torch.full((300,), 3, device=DEV)
    d = torch.randn(300, 20, device=DEV)
    out = torch.full((5, 20), 9.0, device=DEV)
    assert (spl.embedding_grad(ids, d, 5, padding_id=3, out=out) == 0).all()
    out.fill_(9.0)
    assert (spl.embedding_grad(ids[:0], d[:0], 5, out=out) == 0).all()
    out.fill_(9.0)
    assert (spl.embedding_grad(ids[:0], d[:0], 5, out=out, accumulate=True) == 9).all()


def test_grad_is_the_adjoint_of_the_lookup():
    """sum(d_out * lookup(table)) is linear in the table: its difference along a direction is
    sum(gradient * direction)."""
    g = gen(8)
    ids = torch.randint(0, 300, (900,), generator=g, device=DEV)
    d_out = torch.randn(900, 50, generator=g, device=DEV)
    dirn = torch.randn(300, 50, generator=g, device=DEV)
    grad = spl.embedding_grad(ids, d_out, 300, scale=3.0)
    lhs = (spl.embedding(ids, dirn, scale=3.0).double() * d_out.double()).sum()
    rhs = (grad.double() * dirn.double()).sum()
    size = (spl.embedding(ids, dirn.abs(), scale=3.0).double() * d_out.abs().double()).sum()
    assert abs(lhs - rhs) <= size * 30 * 2.0 ** -24


def test_same_bits_on_another_stream_with_a_kept_workspace():
    g = gen(4)
    ids = (torch.rand(30000, generator=g, device=DEV).pow(6) * 1000).long()
    d = torch.randn(30000, 64, generator=g, device=DEV).bfloat16()
    a = spl.embedding_grad(ids, d, 1000)
    ws = torch.full((spl.library().spl_embedding_grad_workspace(30000, 1000, 64),), 255,
                    dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            b = spl.embedding_grad(ids, d, 1000, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b)


def test_refusals():
    ids, d = torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, 6, device=DEV)
    for call in (lambda: spl.embedding_grad(ids[:3], d, 5), lambda: spl.embedding_grad(ids, d, 5, accumulate=True),
                 lambda: spl.embedding_grad(ids, d, 5, out=torch.zeros(4, 6, device=DEV)),
                 lambda: spl.embedding_grad(ids, d, 5, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)),
                 lambda: spl.embedding(ids, d.t()), lambda: spl.embedding(ids.cpu(), d)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        spl.embedding(ids, d.double())
    with pytest.raises(spl.SplError):
        spl.embedding(ids, d, scale=math.inf)
