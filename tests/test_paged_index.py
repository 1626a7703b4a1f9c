"""The walk of the paged calls' kernels from a row to its sequence, position, page and slot, run on the host (the same
functions, compiled for it) against oracle/target.py: rows of no sequence, row starts out of order and out of range,
lengths below 0 and past the table, bad page ids, any page size.  Every table and start is allocated to its size, so a
read outside it would be seen by an address sanitizer; what is checked here is that no page or slot outside the cache
comes out."""
import os
import random
import subprocess

import pytest

from oracle import target as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    from block_speculative_drafting_gb300.csrc.build import nvcc
    exe = str(tmp_path_factory.mktemp("paged") / "paged_index")
    r = subprocess.run([nvcc(), "-std=c++17", "-O1", "-Xcompiler", "-fsanitize=address", "-Xcompiler", "-static-libasan",
                        "-I", os.path.join(ROOT, "include"), "-o", exe, os.path.join(ROOT, "tests", "paged_index.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(text):
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120,
                             env={**os.environ, "ASAN_OPTIONS": "protect_shadow_gap=0:detect_leaks=0"})
        assert out.returncode == 0, out.stderr[-2000:]
        return out.stdout.split("\n")
    return run


def _case(rng):
    ns, page = rng.randint(1, 6), rng.choice((1, 2, 3, 7, 16, 48, 64, 1000, 65536))
    mp, np_ = rng.randint(0, 6), rng.randint(0, 9)
    uniform = rng.random() < 0.3
    nr = ns * rng.randint(0, 5) if uniform else rng.randint(0, 20)
    start = None
    if not uniform:
        start = sorted(rng.randint(0, nr) for _ in range(ns + 1))
        if rng.random() < 0.5:  # anything else
            start = [rng.choice((rng.randint(-3, nr + 3), -2 ** 31, 2 ** 31 - 1, nr)) for _ in range(ns + 1)]
    lens = [rng.choice((rng.randint(-3, mp * page + 5), 0, -2 ** 31, 2 ** 31 - 1)) for _ in range(ns)]
    table = [[rng.choice((rng.randint(0, max(np_ - 1, 0)), -1, np_, 2 ** 31 - 1, -2 ** 31)) for _ in range(mp)]
             for _ in range(ns)]
    return ns, nr, mp, page, np_, start, lens, table


def test_rows_find_their_pages(walk):
    rng = random.Random(7)
    cases = [_case(rng) for _ in range(400)]
    text = ""
    for ns, nr, mp, page, np_, start, lens, table in cases:
        text += f"{ns} {nr} {mp} {page} {np_} {int(start is None)}\n"
        text += " ".join(map(str, (start or []) + lens + [x for row in table for x in row])) + "\n"
    lines = iter(walk(text + "-1 0 0 0 0 0\n"))
    ordered = 0
    for ns, nr, mp, page, np_, start, lens, table in cases:
        rows = O.rows_of(ns, nr, start)
        well = start is None or all(a <= b for a, b in zip(start, start[1:])) and start[0] >= 0 and start[-1] <= nr
        ordered += well
        for r in range(nr):
            s, pos, pg, slot = map(int, next(lines).split())
            if s >= 0:
                assert rows[s][1] <= r < rows[s][1] + rows[s][2]
                want = O.slot_of(table[s], page, np_, lens[s] - rows[s][2] + r - rows[s][1])
                assert pos == lens[s] - rows[s][2] + r - rows[s][1]
                assert ((pg, slot) if pg >= 0 else None) == want
                assert pg < np_ and 0 <= slot < page
            elif well:
                assert not any(a <= r < a + n for _, a, n in rows)
        assert next(lines) == "end"
    assert ordered > 100


def test_division_by_any_page_size(walk):
    rng = random.Random(1)
    pairs = [(n, d) for d in (1, 2, 3, 5, 7, 48, 100, 127, 1000, 4095, 65535, 65536)
             for n in (0, 1, d - 1, d, d + 1, 2 ** 31 - 1, 2 ** 31 - d, *(rng.randrange(2 ** 31) for _ in range(40)))]
    got = walk("-1 0 0 0 0 0\n" + "\n".join(f"{n} {d}" for n, d in pairs) + "\n")
    assert [int(x) for x in got if x] == [n // d for n, d in pairs]
