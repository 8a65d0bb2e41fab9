"""The local step's C ABI on the host (CPU only): exported symbols, workspace sizes, and every
refusal that is decided before the GPU is touched."""
import ctypes
import os
import re

import pytest
import torch

import compressed_pseudo_gradient_gb300 as spl
from compressed_pseudo_gradient_gb300 import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, ALIGN = 0, 1, 2
F32, BF16 = 0, 1
A, B, C, D, E, F = (i << 40 for i in range(1, 7))   # device addresses that are never touched


@pytest.fixture(scope="module")
def lib():
    return spl.library()


def test_both_builds_export_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "spl_local.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(spl_[a-z_]+)\s*\(", text)))
    assert names == ["spl_embedding", "spl_embedding_grad", "spl_embedding_grad_workspace",
                     "spl_orthogonalize", "spl_orthogonalize_workspace", "spl_token_logprobs",
                     "spl_token_logprobs_grad"]
    for path in (lib_build.LIB_PATH, lib_build.CHECKED_LIB_PATH):
        for fn in names:
            assert hasattr(ctypes.CDLL(path), fn)


def test_bad_token_flag(lib):
    assert spl.flags_status(spl.FLAG_BAD_TOKEN) == 7
    assert spl.flags_status(spl.FLAG_BAD_TOKEN | spl.FLAG_NONFINITE) == 7
    assert spl.flags_status(spl.FLAG_BAD_TOKEN | spl.FLAG_TIMEOUT) == 6
    assert lib.spl_status_string(7) == b"token id out of range"


def logprobs(lib, **kw):
    a = dict(logits=A, dtype=F32, rows=4, vocab=100, stride=100, targets=B, bits=64, scale=1.0,
             top=2, logp=C, lse=C + 256, entropy=C + 512, ids=D, tlp=E, flags=F)
    a.update(kw)
    return lib.spl_token_logprobs(*a.values(), None)


def test_logprobs_refusals(lib):
    assert logprobs(lib, rows=0) == OK
    for kw in (dict(dtype=2), dict(bits=16), dict(vocab=0), dict(stride=99), dict(top=-1),
               dict(top=33), dict(vocab=1, top=2), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(logits=None),
               dict(logp=None), dict(ids=None), dict(tlp=None), dict(vocab=1 << 31, stride=1 << 31),
               dict(rows=1 << 31), dict(stride=1 << 60),
               # overlaps
               dict(lse=C), dict(lse=A), dict(logp=B), dict(entropy=A + 4), dict(ids=C),
               dict(tlp=D), dict(flags=A), dict(flags=C)):
        assert logprobs(lib, **kw) == INVALID, kw
    for kw in (dict(logits=A + 2), dict(targets=B + 4), dict(lse=C + 257), dict(ids=D + 4),
               dict(flags=F + 2)):
        assert logprobs(lib, **kw) == ALIGN, kw


def grad(lib, **kw):
    a = dict(logits=A, dtype=F32, rows=4, vocab=100, stride=100, targets=B, bits=64, scale=1.0,
             lse=C, d_logp=C + 256, entropy=C + 512, d_entropy=C + 1024, out=D, out_stride=100,
             flags=F)
    a.update(kw)
    return lib.spl_token_logprobs_grad(*a.values(), None)


def test_logprobs_grad_refusals(lib):
    assert grad(lib, rows=0) == OK
    for kw in (dict(dtype=-1), dict(bits=8), dict(vocab=0), dict(stride=99), dict(out_stride=99),
               dict(scale=0.0), dict(lse=None), dict(out=None), dict(logits=None),
               dict(targets=None), dict(d_logp=None), dict(entropy=None), dict(rows=1 << 31),
               # overlaps; in place only with the same stride
               dict(out=A, out_stride=101), dict(out=A + 4), dict(out=C), dict(out=B), dict(flags=D)):
        assert grad(lib, **kw) == INVALID, kw
    for kw in (dict(out=D + 1), dict(targets=B + 2), dict(d_logp=C + 258)):
        assert grad(lib, **kw) == ALIGN, kw


def embed(lib, **kw):
    a = dict(ids=A, bits=64, count=10, table=B, dtype=BF16, vocab=50, width=16, stride=16, scale=1.0,
             out=C, out_stride=16, flags=F)
    a.update(kw)
    return lib.spl_embedding(*a.values(), None)


def test_embedding_refusals(lib):
    assert embed(lib, count=0) == OK
    for kw in (dict(bits=0), dict(dtype=5), dict(vocab=0), dict(width=0), dict(stride=15),
               dict(out_stride=15), dict(scale=float("inf")), dict(ids=None), dict(table=None),
               dict(out=None), dict(out=B), dict(out=A), dict(flags=C)):
        assert embed(lib, **kw) == INVALID, kw
    for kw in (dict(ids=A + 4), dict(table=B + 1), dict(out=C + 1)):
        assert embed(lib, **kw) == ALIGN, kw


def embed_grad(lib, **kw):
    a = dict(ids=A, bits=64, count=10, d_out=B, dtype=BF16, width=16, d_stride=16, vocab=50,
             scale=1.0, pad=-1, acc=0, table=C, stride=16, ws=D, ws_bytes=1 << 20, flags=F)
    a.update(kw)
    return lib.spl_embedding_grad(*a.values(), None)


def test_embedding_grad_refusals(lib):
    assert embed_grad(lib, count=0, acc=1) == OK
    need = lib.spl_embedding_grad_workspace(10, 50, 16)
    assert need > 0 and lib.spl_embedding_grad_workspace(10, 0, 16) == 0
    for kw in (dict(bits=1), dict(dtype=2), dict(width=0), dict(vocab=0), dict(d_stride=15),
               dict(stride=15), dict(scale=float("nan")), dict(ids=None), dict(d_out=None),
               dict(table=None), dict(ws=None), dict(ws_bytes=need - 1), dict(table=B),
               dict(table=D), dict(ws=A), dict(flags=C), dict(count=1 << 32)):
        assert embed_grad(lib, **kw) == INVALID, kw
    for kw in (dict(ids=A + 2), dict(d_out=B + 1), dict(table=C + 2), dict(ws=D + 16)):
        assert embed_grad(lib, **kw) == ALIGN, kw


def orth(lib, **kw):
    coef = (ctypes.c_float * 3)(*kw.pop("coef", (3.4445, -4.775, 2.0315)))
    a = dict(update=A, dtype=F32, batch=2, rows=10, cols=20, stride=20, bstride=200, momentum=B,
             mu=0.95, nesterov=1, steps=5, coef=coef, eps=1e-7, out=C, ws=D, ws_bytes=1 << 20,
             flags=F)
    a.update(kw)
    return lib.spl_orthogonalize(*a.values(), None)


def test_orthogonalize_refusals(lib):
    need = lib.spl_orthogonalize_workspace(2, 10, 20)
    assert need > 0
    for bad in ((0, 10, 20), (2, 0, 20), (2, 10, 0), (65536, 10, 20), (1, 10, 1 << 21)):
        assert lib.spl_orthogonalize_workspace(*bad) == 0
    for kw in (dict(dtype=3), dict(batch=0), dict(rows=0), dict(cols=0), dict(stride=19),
               dict(bstride=199), dict(steps=0), dict(steps=33), dict(coef=(9.0, 0.0, 0.0)),
               dict(coef=(1.0, float("nan"), 0.0)), dict(eps=-1.0), dict(eps=float("inf")),
               dict(mu=float("nan")), dict(update=None), dict(out=None), dict(ws=None),
               dict(ws_bytes=need - 1), dict(out=A), dict(out=B), dict(momentum=A), dict(ws=C),
               dict(flags=C), dict(batch=1 << 40)):
        assert orth(lib, **kw) == INVALID, kw
    for kw in (dict(update=A + 2), dict(momentum=B + 2), dict(out=C + 2), dict(ws=D + 128)):
        assert orth(lib, **kw) == ALIGN, kw


def test_workspaces_grow_with_the_sizes(lib):
    """The state's four fp16 planes and the two square ones; the sorted tokens and the partials."""
    assert lib.spl_orthogonalize_workspace(1, 1024, 8192) >= 4 * 2 * 1024 * 8192 + 2 * 2 * 1024 ** 2
    assert lib.spl_orthogonalize_workspace(1, 8192, 1024) == lib.spl_orthogonalize_workspace(1, 1024, 8192)
    assert lib.spl_embedding_grad_workspace(65536, 262208, 8192) >= 4 * 4 * 65536 + 2 * 1024 * 8192 * 4


def test_binding_rejects_cpu_tensors_and_bad_types():
    x = torch.zeros(4, 8)
    for call in (lambda: spl.token_logprobs(x), lambda: spl.token_logprobs_grad(x, None, x, None),
                 lambda: spl.embedding(torch.zeros(3, dtype=torch.int64), x),
                 lambda: spl.embedding_grad(torch.zeros(4, dtype=torch.int64), x, 10),
                 lambda: spl.orthogonalize(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        spl.orthogonalize([[1.0]])
