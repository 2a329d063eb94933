"""Draft verification where a warp's slice of the row has many chunks: more sequences than clusters of two
run at once, a vocabulary above sixteen chunks a warp."""
import numpy as np
import pytest
import torch

import gather_qsa_pool_gb300 as qsa
import test_gpu_dense

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("V", [40001, 70000])
def test_long_slices(V):
    test_gpu_dense.test_draft_verify(160, 1, V, False)


@pytest.mark.parametrize("V", [40001, 65536, 5])
def test_few_weights_at_the_ends_of_chunks(V):
    """Rows of zeros but for a few equal weights (sums are exact): the drawn index is known for every u."""
    n = 160
    rng = np.random.default_rng(V)
    places = np.unique(np.minimum([0, 1, 127, 128, 2047, 2048, 2049, 32767, 32768, V - 2, V - 1], V - 1))
    p = np.zeros((n, 1, V), np.float32)
    u = rng.integers(0, 1 << 20, (n, 1)).astype(np.float32) / (1 << 20)
    want = np.zeros(n, np.int64)
    for s in range(n):
        at = np.sort(rng.choice(places, rng.integers(1, min(len(places), 8) + 1), replace=False))
        w = rng.integers(1, 4, len(at)).astype(np.float32)
        p[s, 0, at] = w
        if s % 4 == 0:  # a point on a weight's edge belongs to the next
            k = rng.integers(0, len(at))
            edge = w[:k].sum() / w.sum()
            u[s, 0] = edge if float(np.float32(edge)) == float(edge) and (w.sum() in (1, 2, 4, 8)) else u[s, 0]
        run = np.cumsum(w.astype(np.float64))
        want[s] = at[np.argmax(run > float(u[s, 0]) * run[-1])]
    out = torch.full((n, 1), -9, dtype=torch.int32, device=DEV)
    acc = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    tokens = torch.zeros((n, 0), dtype=torch.int32, device=DEV)
    qsa.draft_verify(torch.from_numpy(p).to(DEV), None, tokens, torch.from_numpy(u).to(DEV), out, acc)
    np.testing.assert_array_equal(out[:, 0].cpu().numpy(), want)
    assert (acc == 0).all()
