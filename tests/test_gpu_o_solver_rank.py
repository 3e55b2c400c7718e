"""The multi-launch calibration solve on statistics of fewer non-zero eigenvalues than
rows asked for: the rows beyond them have no direction of their own, and still
complete an orthonormal set on every call."""

import numpy as np
import pytest

from gpu_util import rng, to_dev, to_np, torch_or_skip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,rank,R", [(200, 1, 3), (700, 1, 8), (700, 4, 12), (300, 1, 16), (1500, 2, 8), (2500, 3, 12)])
def test_rows_of_a_rank_deficient_statistic(monkeypatch, L, rank, R):
    """Bounds of the solver's other tests: 1e-4 for orthonormality, 1e-3 for vectors whose
    eigenvalues are a factor of two apart."""
    torch = torch_or_skip()
    from rank_compressed_backprop_gb300 import api

    monkeypatch.setenv("INSTANT_SOLVER_MULTI", "1")
    for seed in range(12):
        v = np.linalg.qr(rng(seed * 7 + L).standard_normal((L, rank)))[0]
        lam = 3.0 * 0.5 ** np.arange(rank)
        C = to_dev((16 * (v * lam) @ v.T).astype(np.float32))
        rows = torch.full((R, L), 9.0, dtype=torch.float32, device="cuda")
        res = api.calib_solve(C, 16, rows, eps=0.95, r_override=R, scale_on=False)
        assert np.abs(np.array(res.eigenvalues[:rank]) - lam).max() <= 3e-4
        got = to_np(rows)
        assert np.abs(got @ got.T - np.eye(R)).max() <= 1e-4, seed
        assert np.abs(np.abs(got[:rank] @ v) - np.eye(rank)).max() <= 1e-3, seed
        assert np.abs(got[rank:] @ v).max() <= 1e-3, seed
    assert api.device_status() == 0
