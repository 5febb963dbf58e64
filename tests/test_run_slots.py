"""The schedule of balanced runs, restated: which slot each piece of a job leaves its softmax
statistics in, and where the second launch of the accumulated weights looks for them."""
import numpy as np
import pytest

SETUP = 5                                   # list entries a job counts besides its pages


def runs(lens, heads, workers, min_share):
    """[(worker, job, first page, pages, second)] of all pieces, as the warps walk their runs."""
    pages = [-(-n // 16) for n in lens]
    jobs = [(b * heads + h, p) for b, p in enumerate(pages) if p for h in range(heads)]
    total = sum(p + SETUP for _, p in jobs)
    share = max(min_share, -(-total // workers))
    starts = np.cumsum([0] + [p + SETUP for _, p in jobs])
    out = []
    for i, (job, p) in enumerate(jobs):
        f, end = int(starts[i]), int(starts[i + 1])
        while f < end:
            w = f // share
            upto = min(end, (w + 1) * share)
            entry = f - int(starts[i])
            page = max(0, entry - SETUP)
            n = max(0, entry + upto - f - SETUP) - page
            if n > 0:
                out.append((w, job, page, n, f != w * share))
            f = upto
    return out, share, dict(zip((j for j, _ in jobs), starts)), dict(jobs)


def written(piece, pages, workers):
    w, job, _, n, second = piece
    return 2 * workers + job if n == pages[job] else 2 * w + second


def read(job, start, pages, share, workers):
    """The slots of a job's pieces in page order."""
    w0, w1 = (start + SETUP) // share, (start + pages + SETUP - 1) // share
    if w0 == w1:
        return [2 * workers + job]
    return [2 * w + (w == w0 and start > w0 * share) for w in range(w0, w1 + 1)]


@pytest.mark.parametrize("seed", range(60))
def test_no_two_pieces_share_a_slot(seed):
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 300))
    hi = int(rng.choice([20, 64, 400, 4096]))
    lens = rng.integers(0, hi + 1, B)
    if seed % 3 == 0:
        lens[rng.integers(0, B)] = 20000
    heads = int(rng.choice([1, 2, 8, 16]))
    workers = int(rng.choice([7, 100, 1216, 2432]))
    pieces, share, start, pages = runs(lens.tolist(), heads, workers, 8)
    assert all(w < workers for w, *_ in pieces)
    slots = [written(x, pages, workers) for x in pieces]
    assert len(set(slots)) == len(slots)
    by_job = {}
    for x, s in zip(pieces, slots):
        by_job.setdefault(x[1], []).append(s)
    assert set(by_job) == set(pages)
    for job, s in by_job.items():
        assert s == read(job, int(start[job]), pages[job], share, workers)
    # without slots of their own, whole jobs of one run would meet in the worker's second one
    if seed == 0:
        lens = [64] * 512
        pieces, _, _, pages = runs(lens, 8, 2432, 8)
        shared = [2 * x[0] + x[4] for x in pieces]
        assert len(set(shared)) < len(shared)
