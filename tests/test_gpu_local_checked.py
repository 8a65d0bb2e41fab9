"""The local step's operators through the checked build: the same results, and no memory index
out of range on ragged, strided, masked and tied cases."""
import pytest
import torch

import compressed_pseudo_gradient_gb300 as spl
import test_gpu_embedding as emb
import test_gpu_logprobs as lp
import test_gpu_orthogonalize as orth

pytestmark = pytest.mark.gpu


@pytest.fixture()
def checked():
    torch.cuda.synchronize()
    prev = spl.use_library(spl.checked_library_path())
    spl.debug_words(reset=True)
    try:
        yield
        torch.cuda.synchronize()
        d = spl.debug_words(reset=True)
        assert d["failures"] == 0 and d["sites"] == 0, f"failed checks {d}"
    finally:
        spl.use_library(prev)


def test_checked_build_is_the_one_loaded(checked):
    assert hasattr(spl.library(), "spl_debug_read")


@pytest.mark.parametrize("dtype", lp.DTYPES)
def test_logprobs(checked, dtype):
    for rows, vocab in ((1, 1), (4, 33), (2, 4097), (1, 65537), (700, 513)):
        lp.test_values_and_top(rows, vocab, dtype)
    lp.test_strides_and_alignments(7, 3, dtype)
    lp.test_ties_go_to_the_lower_id(dtype)
    lp.test_masked_logits(-lp.INF, dtype)
    lp.test_a_row_of_nothing(40001, dtype)
    for terms in ("logp", "both"):
        lp.test_grad_formula(2, 9001, 7, 3, dtype, terms)
        lp.test_grad_formula(2, 100003, 0, 1, dtype, terms)
    lp.test_targets_outside()


@pytest.mark.parametrize("dtype", emb.DTYPES)
def test_embedding(checked, dtype):
    for case in ((1, 1, 1, 0, 0), (17, 33, 1001, 0, 0), (1000, 3000, 40, 24, 8), (7, 20, 100, 1, 3)):
        emb.test_lookup_is_one_rounding(*case, dtype)
    emb.test_lookup_shapes_and_bad_ids()
    for case in emb.CASES:
        emb.test_grad_sums(*case, dtype)
    emb.test_grad_strides_padding_and_bad_ids(dtype)
    emb.test_grad_of_nothing_and_of_only_padding()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize(checked, dtype):
    for m, n in ((1, 1), (9, 1), (17, 33), (129, 127), (200, 1000), (513, 700)):
        orth.test_matrix(m, n, dtype)
    orth.test_stack_of_strided_matrices(5, 130, 50, 6)
    orth.test_momentum(True, dtype)
