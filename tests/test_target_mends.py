"""Further cases of the target's verification pass: each test holds one behaviour that went wrong before, against
oracle/target.py or a plain 64-bit computation."""
import numpy as np
import pytest

from oracle import target as O
from test_paged_index import walk  # noqa: F401  (a fixture: the kernels' walk from rows to pages, on the host)

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


# --------------------------------------------------------------------------- starts out of order
BAD_STARTS = [[0, 5, 3, 8], [6, 0, 6, 2], [0, 99, 99, 99], [-5, 2, 4, 99], [3, 1, 2, 5], [8, 8, 0, 8], [0, 8, 8, 1],
              [2, -2 ** 31, 2 ** 31 - 1, 3]]


def test_rows_of_starts_out_of_order_have_one_owner(walk):  # noqa: F811
    """Every row has the sequence that the oracle's ascending starts give it, or none."""
    text = ""
    for start in BAD_STARTS:
        text += f"3 8 1 16 4 0\n{' '.join(map(str, start))}\n9 9 9\n0 1 2\n"
    lines = iter(walk(text + "-1 0 0 0 0 0\n"))
    for start in BAD_STARTS:
        owner = {r: s for s, a, n in O.rows_of(3, 8, start) for r in range(a, a + n)}
        for r in range(8):
            assert int(next(lines).split()[0]) == owner.get(r, -1), (start, r)
        assert next(lines) == "end"


@gpu
@pytest.mark.parametrize("start", BAD_STARTS)
@pytest.mark.parametrize("heads", [4, 40])  # the warps' kernel, and the tensor memory's
def test_paged_calls_with_starts_out_of_order(start, heads):
    torch, dfl = _torch(), _dfl()
    rng = np.random.default_rng(0)
    R = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
    kc, vc, q, k, v = R(6, 16, 2, 64), R(6, 16, 2, 64), R(8, heads, 64), R(8, 2, 64), R(8, 2, 64)
    table, lens = [[0, 1], [2, 3], [4, 5]], [20, 31, 9]
    args = (_i32(torch, table), _i32(torch, lens))
    k64, v64 = f64(kc), f64(vc)
    q_out = torch.full_like(q, 7.0)
    dfl.paged_append(kc, vc, k, v, *args, row_start=_i32(torch, start), q=q, q_out=q_out)
    slots, _, touched = O.paged_append(f64(k), f64(v), f64(q), table, lens, 16, 6, start)
    for at, (kk, vv) in slots.items():
        k64[at], v64[at] = kk, vv
    assert np.array_equal(f64(kc), k64) and np.array_equal(f64(vc), v64)
    rest = [r for r in range(8) if r not in touched]
    assert np.array_equal(f64(q_out)[touched], f64(q)[touched]) and (f64(q_out)[rest] == 7.0).all()
    ref, _, mag, touched = O.paged_attention(f64(q), k64, v64, table, lens, start)
    out = torch.full_like(q, 7.0)
    dfl.paged_attention(q, kc, vc, *args, row_start=_i32(torch, start), out=out)
    # bf16 outputs: half a step; scores: 64 f32 products of up to |q| |k| = 100, times the scale
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 64 * 2.0 ** -24 * 100 * mag)[touched].all()
    assert (f64(out)[[r for r in range(8) if r not in touched]] == 7.0).all()


@gpu
@pytest.mark.parametrize("start", BAD_STARTS)
@pytest.mark.parametrize("drawn", [False, True])
def test_verify_with_starts_out_of_order(start, drawn):
    """What the oracle's ascending starts give, whatever the workspace held before: every output, and nothing else."""
    torch, dfl = _torch(), _dfl()
    for seed, temps in enumerate(([0.0, 0.0, 0.0], [0.9, 0.0, 1.4], [0.7, 1.0, 0.8])):
        rng = np.random.default_rng(seed)
        n, d, V = 3, 8, 100
        t = torch.from_numpy(rng.standard_normal((n + d, V)).astype(np.float32)).cuda()
        dl = torch.from_numpy(rng.standard_normal((d, V)).astype(np.float32)).cuda()
        tok = rng.integers(0, V, d)
        au, su = (torch.from_numpy(rng.random(m).astype(np.float32)).cuda() for m in (d, n))
        res, pref = O.verify(f64(t), tok, f64(au), f64(su), f64(dl) if drawn else None, start, temps)
        at = O.rows_of(n, d, start)
        owned = [j for _, a, m in at for j in range(a, a + m)]
        need = dfl.verify_workspace(n, d, V)
        for fill in (0x00, 0x7f, 0xff, 0x41):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            prob = torch.full((d,), 7.0, device="cuda")
            acc, nxt, _ = dfl.verify_drafts(t, _i32(torch, tok), au, su, draft_logits=dl if drawn else None,
                                            draft_start=_i32(torch, start), prob=prob, workspace=ws,
                                            temperature=torch.tensor(temps, device="cuda"))
            for s, (a, x, margin) in enumerate(res):
                if margin > 1e-5:
                    assert (acc[s].item(), nxt[s].item()) == (a, x), (start, s, fill)
                assert -1 <= nxt[s].item() < V and 0 <= acc[s].item() <= at[s][2]
            p = f64(prob)
            assert (np.abs(p[owned] - pref[owned]) <= 2e-6 * np.abs(pref[owned])).all()
            assert all(p[j] == 7.0 for j in range(d) if j not in owned)


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
