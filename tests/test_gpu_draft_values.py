"""Draft verification on rows with negative and NaN entries, which count as 0 in both rows: in the test of a
drafted token, in the weights after a refusal and in the weights of the target's row alone."""
import numpy as np
import pytest
import torch

import dense_reference as ref
import gather_qsa_pool_gb300 as qsa

pytestmark = pytest.mark.gpu

DEV = "cuda"


def spoil(rng, x, share):
    """A copy of x with some entries negative and some NaN, and what those rows stand for."""
    y = x.copy()
    at = rng.random(x.shape)
    y[at < share] = np.nan
    y[(at >= share) & (at < 2 * share)] *= -1
    y[(at >= 2 * share) & (at < 3 * share)] = -3.0
    return y, np.where(y > 0, y, 0).astype(np.float32)


def run(p, q, tokens, u):
    n, D = tokens.shape
    out = torch.full((n, D + 1), -9, dtype=torch.int32, device=DEV)
    acc = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    dev = [None if x is None else torch.from_numpy(x).to(DEV) for x in (p, q, tokens, u)]
    qsa.draft_verify(*dev, out, acc)
    return out.cpu().numpy(), acc.cpu().numpy()


# (one CTA a sequence; odd rows; a cluster a sequence; more chunks a warp than one)
@pytest.mark.parametrize("n,D,V", [(90, 3, 64), (40, 2, 131), (6, 4, 8192), (160, 1, 40000)])
@pytest.mark.parametrize("greedy", [False, True])
def test_negative_and_nan_count_as_zero(n, D, V, greedy):
    rng = np.random.default_rng(V + D)
    for share in (0.02, 0.3):
        # weights that are multiples of 2^-12: every sum is exact, whatever its order
        p = rng.integers(0, 64, (n, D + 1, V)).astype(np.float32) / 4096
        q = rng.integers(0, 64, (n, D, V)).astype(np.float32) / 4096
        tokens = rng.integers(0, V, (n, D)).astype(np.int32)
        u = (rng.integers(0, 256, (n, D + 1)) / 256).astype(np.float32)
        u[:, :D] *= 2.0 ** -4  # some tokens are taken
        (p, p0), (q, q0) = spoil(rng, p, share), spoil(rng, q, share)
        got, acc = run(p, None if greedy else q, tokens, u)
        for s in range(n):
            want, a = ref.verify(p0[s], None if greedy else q0[s], tokens[s], D, u[s])
            assert acc[s] == a
            np.testing.assert_array_equal(got[s], want)


def test_a_drafts_entry_that_is_no_number():
    """Token 1 of a row whose draft entry is NaN, or below zero, is taken where the target has any weight
    there, refused where it has none; and the residual keeps the target's weight."""
    p = np.zeros((4, 2, 6), np.float32)
    q = np.zeros((4, 1, 6), np.float32)
    q[0, 0, 1], q[1, 0, 1], q[2, 0, 1], q[3, 0, 1] = np.nan, -1.0, np.nan, -1.0
    p[:2, 0, 1] = 0.25          # taken
    p[:, 1, 5] = 1.0
    p[2:, 0, 3] = 0.5           # refused: 0 < 0 does not hold
    q[2:, 0, 4] = 0.5
    tokens = np.ones((4, 1), np.int32)
    u = np.full((4, 2), 0.5, np.float32)
    got, acc = run(p, q, tokens, u)
    assert acc.tolist() == [1, 1, 0, 0]
    assert got.tolist() == [[1, 5], [1, 5], [3, -1], [3, -1]]
