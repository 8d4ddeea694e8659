"""Sampling on the GPU at the sizes of top_k and vocabularies where the way a
row is cut changes."""
import numpy as np
import pytest

from tests.test_gpu_sample import DTYPES, check, logits, uniform

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab", [257, 2049, 16391, 20011, 140001])
def test_every_size_of_top_k(vocab, dtype):
    # Around powers of two: a bound by the lanes' maxima, a histogram, a list
    # that fits and one that does not, the whole row.
    ks = sorted({k + d for k in (1, 32, 64, 128, 256, 512, 1024, 2048, 8192) for d in (-1, 0, 1)}
                | {vocab - 1, vocab, vocab + 1})
    ks = np.array([k for k in ks if 0 < k <= vocab + 1], np.int32)
    x = logits(len(ks), vocab, dtype, vocab)
    check(x, uniform(len(ks), 31), top_k=ks)
    check(x, uniform(len(ks), 32), 0.8, ks, 0.9, 0.001)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_the_kept_lie_together(dtype):
    # All large logits in one stretch, or one lane's places: few of the
    # row's parts hold what is kept.
    x = logits(4, 30011, dtype, 33, 0.5)
    x[0, 7000:7300] += 9
    x[1, -200:] += 9
    x[2, ::512] += 9
    x[3, 8:30000:64] += 9
    for s in ({"top_k": 50}, {"top_k": 250}, {"top_k": 2000}, {"top_p": 0.9}, {"min_p": 0.01},
              {"top_k": 300, "top_p": 0.5, "temperature": 2.0}):
        check(x, uniform(4, 34), **s)
