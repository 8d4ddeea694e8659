"""Penalties on batches large enough for the kernel that takes more logits a
workgroup (512 parts of rows and more), in each of its instances; against the
definition in 64 bits, with the tolerances derived where `check` is defined."""
import pytest

from tests.test_gpu_penalty import DTYPES, case, check

pytestmark = pytest.mark.gpu


def batch(dtype):
    """Rows and logits: 5 parts of 16384 logits of 16 bits a row, 9 of 8192 of 32 bits."""
    return (70 if dtype == "fp32" else 130), 65600


@pytest.mark.parametrize("grammars", [0, 5])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_without_biases(dtype, packed, grammars):
    x, kw = case(*batch(dtype), 200, dtype, packed, grammars=grammars)
    check(x, dtype, **kw)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_with_biases_and_masks(dtype, packed):
    x, kw = case(*batch(dtype), 150, dtype, packed, biases=40, grammars=5, seed=1)
    check(x, dtype, **kw)


@pytest.mark.parametrize("biases", [0, 30])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_more_named_logits_than_slots(dtype, biases):
    # past tokens gather at the low ones: more than a thousand in a row's first part
    x, kw = case(*batch(dtype), 6000, dtype, True, biases=biases, seed=2)
    check(x, dtype, places=("out", "here"), **kw)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_a_mask_alone_or_nothing(dtype):
    x, kw = case(*batch(dtype), 1, dtype, False, grammars=4, seed=3)
    check(x, dtype, mask=kw["mask"], mask_slots=kw["mask_slots"])
    check(x, dtype)
