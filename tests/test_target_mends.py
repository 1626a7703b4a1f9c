"""Further cases of the target's verification pass: each test holds one behaviour that went wrong before, against
oracle/target.py or a plain 64-bit computation."""
import numpy as np
import pytest

from oracle import target as O

gpu = pytest.mark.gpu


def _dfl():
    import block_speculative_drafting_gb300 as dfl
    return dfl


def _torch():
    return pytest.importorskip("torch")


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _i32(torch, x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


# --------------------------------------------------------------------------- verification
@gpu
def test_verify_of_many_short_sequences_in_clusters_that_start_late():
    """Thousands of clusters with next to nothing to read, behind work on another stream that keeps the SMs: a cluster's
    CTAs then start at different times, and none may be written to before it runs."""
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    n, V = 3000, 40
    t = torch.from_numpy(rng.standard_normal((n, V)).astype(np.float32)).cuda()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    su = torch.from_numpy(rng.random(n).astype(np.float32)).cuda()
    temps = torch.from_numpy(np.where(np.arange(n) % 3 == 0, 0.0, 0.9).astype(np.float32)).cuda()  # greedy ones between
    res, _ = O.verify(f64(t), [], [], f64(su), None, None, temps.tolist())
    side, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    for _ in range(5):
        with torch.cuda.stream(side):
            for _ in range(4):
                busy = busy @ busy * 1e-3
        acc, nxt, _ = dfl.verify_drafts(t, none, torch.empty(0, device="cuda"), su, temperature=temps)
        got = nxt.tolist()
        assert acc.tolist() == [0] * n
        assert all(g == x for g, (_, x, margin) in zip(got, res) if margin > 1e-5)
        torch.cuda.synchronize()
