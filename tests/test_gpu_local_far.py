"""Rows that lie more than 2^31 elements apart: each operator against itself on the rows side by side.

Alignments are alike in both, so the results are the same bits.
"""
import pytest
import torch

import compressed_pseudo_gradient_gb300 as spl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STRIDE = (1 << 27) + 8
ROWS = 18   # the last one starts beyond 2^31 elements
COLS = 1000
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", params=DTYPES)
def far(request):
    """Two sets of far rows, the first filled."""
    span = (ROWS - 1) * STRIDE + 2 * COLS
    if torch.cuda.mem_get_info()[0] < 2 * span * request.param.itemsize + (2 << 30):
        pytest.skip("needs 23 GB")
    sets = [torch.empty(span, dtype=request.param, device=DEV).as_strided((ROWS, COLS), (STRIDE, 1))
            for _ in range(2)]
    sets[0].copy_(torch.randn(ROWS, COLS, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV))
    yield sets
    del sets
    torch.cuda.empty_cache()


def test_token_logprobs(far):
    x, out = far
    near = x.contiguous()
    t = torch.arange(ROWS, device=DEV) * 55 % COLS
    a, b = spl.token_logprobs(x, t, top=3), spl.token_logprobs(near, t, top=3)
    for one, other in zip(a, b):
        assert torch.equal(one, other)
    g = torch.linspace(-1, 1, ROWS, device=DEV)
    spl.token_logprobs_grad(x, t, a.lse, g, entropy=a.entropy, d_entropy=g, out=out)
    assert torch.equal(out, spl.token_logprobs_grad(near, t, b.lse, g, entropy=b.entropy, d_entropy=g))


def test_embedding(far):
    table, out = far
    near = table.contiguous()
    ids = torch.tensor([17, 0, 16, 17, 3, 1, 2, 17, 5, 8, 13, 4, 4, 9, 10, 11, 12, 17], device=DEV)
    spl.embedding(ids, table, scale=0.5, out=out)
    assert torch.equal(out, spl.embedding(ids, near, scale=0.5))


def test_embedding_grad(far):
    d_out, out = far
    ids = torch.tensor([17, 0, 16, 17, 3, 1, 2, 17, 5, 8, 13, 4, 4, 9, 10, 11, 12, 17], device=DEV)
    if out.dtype != torch.float32:   # the table's gradient is fp32: half as many elements apart
        out = out.as_strided((ROWS, COLS * 2), (STRIDE, 1)).view(torch.float32)
    spl.embedding_grad(ids, d_out, ROWS, out=out)
    assert torch.equal(out, spl.embedding_grad(ids, d_out.contiguous(), ROWS))


def test_orthogonalize(far):
    x, _ = far
    assert torch.equal(spl.orthogonalize(x), spl.orthogonalize(x.contiguous()))
    stack = x.view(ROWS, 10, 100)   # the matrices far from each other
    assert torch.equal(spl.orthogonalize(stack), spl.orthogonalize(stack.contiguous()))
