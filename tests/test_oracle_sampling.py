"""What pins oracle/sampling.py: torch's softmax, hand-worked sequences, and the
distribution that verification has to give."""
import numpy as np
import torch

from oracle import sampling


def test_target_is_the_softmax():
    z = np.random.default_rng(1).normal(size=50)
    np.testing.assert_allclose(sampling.target(z, 0.7), torch.softmax(torch.tensor(z) / 0.7, 0).numpy(), rtol=1e-13)
    z[[3, 9]] = np.nan, -np.inf
    p = sampling.target(z, 2.0)
    assert p[3] == 0 and p[9] == 0 and abs(p.sum() - 1) < 1e-12
    assert sampling.target([1.0, 5.0, 5.0], 0.0).tolist() == [0, 1, 0]
    assert sampling.target([1.0, np.inf, 3e38, np.inf], 1.0).tolist() == [0, 0.5, 0, 0.5]


def test_infinity_counts_as_the_largest_finite_number_in_greedy_rows_too():
    top = float(np.finfo(np.float32).max)
    assert sampling.target([1.0, top, np.inf], 0.0).tolist() == [0, 1, 0]
    assert sampling.target([1.0, np.inf, top], 0.0).tolist() == [0, 1, 0]
    assert sampling.target([np.nan, 3e38, np.inf], 0.0).tolist() == [0, 0, 1]


def test_draw_by_hand():
    w = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    assert [sampling.draw(w, u) for u in (0.0, 0.2499, 0.25, 0.7499, 0.75, 0.9999)] == [1, 1, 3, 3, 4, 4]


def test_verify_by_hand():
    log = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.2, 0.7], [0.6, 0.3, 0.1]]))
    q = np.array([[0.25, 0.5, 0.25], [0.1, 0.8, 0.1], [9, 9, 9]], np.float32)
    tokens, off = [7, 1, 1], [0, 3]

    def run(u1, u2, un, probs=q):
        return [x[0] for x in sampling.verify(log, tokens, off, [0.9, u1, u2], [un], probs)[:3]]
    # p/q of the drafted tokens: 0.5, 0.25
    assert run(0.49, 0.24, 0.95) == [2, 2, 0]      # both taken, the next by the last row
    assert run(0.49, 0.26, 0.0) == [1, 2, 1]       # max(p - q, 0) = 0, 0, 0.6
    assert run(0.51, 0.0, 0.99) == [0, 0, 2]       # 0.25, 0, 0
    # certain drafts: u < p, the rest is p without the token
    assert run(0.24, 0.19, 0.0, None) == [2, 0, 0]
    assert run(0.26, 0.0, 0.7, None) == [0, 2, 2]
    assert sampling.verify(log, [7, 5, 1], off, [0, 0, 0], [0.6], q)[0] == [0]
    assert sampling.verify(log, tokens, [0, 0, 3], [0, 0, 0], [0.6, 0.6], q)[1][0] == -1


def test_verified_tokens_are_distributed_as_the_target():
    """Over drafts by q, the first token behind a prefix is distributed by p."""
    rng = np.random.default_rng(2)
    V, N = 5, 20000
    log = rng.normal(size=(2, V))
    p, q = sampling.target(log[0], 1.0), sampling.target(rng.normal(size=V), 1.0).astype(np.float32)
    count = np.zeros(V)
    probs = np.stack([q, q])
    for _ in range(N):
        x = sampling.draw(q.astype(np.float64), rng.random())
        a, t, _, _, _ = sampling.verify(log, [0, x], [0, 2], rng.random(2), rng.random(1), probs)
        count[x if a[0] else t[0]] += 1
    # five deviations of a binomial count
    assert (np.abs(count / N - p) <= 5 * np.sqrt(p * (1 - p) / N)).all()
