"""The host definitions the GPU tests compare with, held to each other: the
recurrence against the sum over pairs of tokens, the gradient against
differences (the outputs are linear in each input, so a difference of any
size is exact), sampling against counts of drawn tokens."""
import numpy as np

from tests import linattn_ref as ref

H, DK, DV = 4, 5, 7
LENS = (6, 0, 1, 9)
G = np.array([-0.5, 0.0, -1e-3, -np.inf])


def inputs(rng, hk=2, hv=4):
    n = sum(LENS)
    return (rng.standard_normal((n, H, DK)), rng.standard_normal((n, hk, DK)),
            rng.standard_normal((n, hv, DV)), rng.standard_normal((len(LENS), H, DK, DV)))


def test_recurrence_is_the_sum_over_pairs():
    q, k, v, s0 = inputs(np.random.default_rng(1))
    out, last = ref.forward(q, k, v, G, 0.3, LENS, s0)
    power = lambda h, n: 1.0 if n == 0 else np.exp(G[h] * n)  # noqa: E731
    at = 0
    for s, n in enumerate(LENS):
        for h in range(H):
            for i in range(n):
                want = power(h, i + 1) * q[at + i, h] @ s0[s, h]
                for j in range(i + 1):
                    want = want + power(h, i - j) * (q[at + i, h] @ k[at + j, h // 2]) * v[at + j, h]
                assert np.allclose(out[at + i, h], 0.3 * want, rtol=1e-12, atol=1e-12)
            want = power(h, n) * s0[s, h]
            for j in range(n):
                want = want + power(h, n - 1 - j) * np.outer(k[at + j, h // 2], v[at + j, h])
            assert np.allclose(last[s, h], want, rtol=1e-12, atol=1e-12)
        at += n


def test_gradient_is_the_difference():
    rng = np.random.default_rng(2)
    x = list(inputs(rng, 2, 1))
    do = rng.standard_normal((sum(LENS), H, DV))
    dlast = rng.standard_normal(x[3].shape)

    def loss(a):
        out, last = ref.forward(a[0], a[1], a[2], G, 0.7, LENS, a[3])
        return (out * do).sum() + (last * dlast).sum()

    grads = ref.backward(do, x[0], x[1], x[2], G, 0.7, LENS, x[3], dlast)
    for i in range(4):
        d = rng.standard_normal(x[i].shape)
        moved = list(x)
        moved[i] = x[i] + d
        assert np.isclose((grads[i] * d).sum(), loss(moved) - loss(x), rtol=1e-10, atol=1e-10)


def test_sampling_draws_by_weight():
    x = np.log(np.array([1.0, 4.0, 2.0, 0.5, 2.5]))
    draws = [ref.sample(x, u, top_k=4, top_p=0.89)[0] for u in (np.arange(8500) + 0.5) / 8500]
    # 0.5 is past top_k; of the others' 9.5, 4 + 2.5 + 2 reach 0.89
    assert ref.sample(x, 0.0, top_k=4, top_p=0.89)[2] == 3
    assert np.bincount(draws, minlength=5).tolist() == [0, 4000, 2000, 0, 2500]
    assert ref.sample(x, 0.99, min_p=0.6)[2] == 2
    assert ref.sample(x, 0.5, temperature=0.0) == (1, 0.0, 1)
    assert ref.sample([-np.inf, np.nan], 0.5)[0] == -1
    assert ref.sample([2.0, 3.0, 3.0, 3.0], 0.5, top_k=2)[0] == 2
