"""CPU check of the two ends of the blocked cache attention kernel's work (cache_sparse_kernel): the first item's rows are split
before any tile record is there, and the reader writes end records until both softmax pairs, which look at every second
record only, have one. The model of tests/test_pipeline_cache.py with these roles as the kernel has them."""
import random

import pytest

from tests.pipeline_model import Model
from tests.test_pipeline_cache import BATCH, BATCHES, DENS, FAC, TOPS, cache_sparse_model


def with_ends(m, counts, seed=0, bugs=()):
    cache_sparse_model(m, counts, seed=seed)
    tiles = [(k, t, c) for k, c in enumerate(counts) for t in range(c)]
    N = len(tiles)
    first = [t == 0 for _, t, _ in tiles]
    last = [t == c - 1 for _, t, c in tiles]
    pre = [t == c - 2 for _, t, c in tiles]
    item = [k for k, _, _ in tiles]
    rng = random.Random(seed)
    rescale = {n: not first[n] and rng.random() < 0.4 for n in range(N)}

    def reader():
        k, seen, ended = 0, False, False
        while not seen:
            sl = k % BATCHES
            yield ("wait", f"REC_EMPTY{sl}", k // BATCHES - 1)
            seen = ended
            for i in range(BATCH):
                if not ended and k * BATCH + i == N:
                    ended = True
                    seen = i < BATCH - 1 or "one_end" in bugs
                yield ("put", f"REC{sl}.{i}", k * BATCH + i)
            yield ("arrive", f"REC_FULL{sl}")
            k += 1

    def split(k, of):  # the k-th split, of item `of`
        yield ("wait", f"Q_EMPTY{k & 1}", (k >> 1) - 1)
        yield ("write", f"Q{k & 1}")
        yield ("put", f"FAC{k % FAC}", of)
        yield ("arrive", f"Q_FULL{k & 1}")

    def q_warps():
        k = 1
        yield from split(0, 0)
        for n in range(N + 1):
            b = n // BATCH
            if n % BATCH == 0:
                yield ("wait", f"REC_FULL{b % BATCHES}", b // BATCHES)
            yield ("get", f"REC{b % BATCHES}.{n % BATCH}", n)
            if n == N:
                return
            if n % BATCH == BATCH - 1:
                yield ("arrive", f"REC_EMPTY{b % BATCHES}")
            if first[n] and (item[n] > 0 or "first_twice" in bugs):
                yield from split(k, item[n])
                k += 1

    def softmax(pair, half):
        grp, n = 2 * pair + half, pair
        while True:
            b = n // BATCH
            if n % BATCH < 2:
                yield ("wait", f"REC_FULL{b % BATCHES}", b // BATCHES)
            yield ("get", f"REC{b % BATCHES}.{n % BATCH}", n)
            if n >= N:
                return
            k = item[n]
            if n % BATCH >= BATCH - 2:
                yield ("arrive", f"REC_EMPTY{b % BATCHES}")
            yield ("wait", f"S_FULL{pair}", n >> 1)
            yield ("read", f"S{pair}h{half}")
            yield ("get", f"FAC{k % FAC}", k)
            yield ("arrive", f"S_FREE{pair}")
            if n > 0:
                yield ("wait", f"M_READY{pair ^ 1}", (n - 1) >> 1)
            yield ("put", f"T{n % TOPS}h{half}", n)
            yield ("arrive", f"M_READY{pair}")
            if not first[n]:
                yield ("get", f"T{(n - 1) % TOPS}h0", n - 1)
                yield ("get", f"T{(n - 1) % TOPS}h1", n - 1)
            yield ("wait", f"M_READY{pair}", n >> 1)
            yield ("get", f"T{n % TOPS}h{half ^ 1}", n)
            if n >= 2:
                yield ("wait", f"PV_DONE{pair}", (n - 2) >> 1)
            yield ("write", f"P{pair}h{half}")
            if rescale[n]:
                yield ("wait", f"PV_DONE{pair ^ 1}", (n - 1) >> 1)
                yield ("read", "O")
                yield ("write", "O")
            if pre[n] or last[n]:
                yield ("put", f"D{k % DENS}g{grp}", k)
            yield ("arrive", f"P_FULL{pair}")
            if last[n]:
                yield ("wait", f"PV_DONE{pair}", n >> 1)
                yield ("get", f"D{k % DENS}g{grp ^ 1}", k)
                if not first[n]:
                    yield ("get", f"D{k % DENS}g{2 * (pair ^ 1)}", k)
                    yield ("get", f"D{k % DENS}g{2 * (pair ^ 1) + 1}", k)
                yield ("read", "O")
                yield ("arrive", "O_FREE")
                yield ("write", f"VF{pair}")
                yield ("arrive", f"STAGED{pair}")
            n += 2

    m.roles["reader"] = reader()
    m.roles["q"] = q_warps()
    m.roles.update({f"softmax{p}{h}": softmax(p, h) for p in range(2) for h in range(2)})


def some_counts(rng, total=None):
    """Tiles of each item; with a total, exactly that many together."""
    counts = [rng.choice([1, 1, 1, 2, 3, 5, 9]) for _ in range(rng.randint(1, 9))]
    if total:
        while sum(counts) < total:
            counts.append(rng.randint(1, 4))
        while sum(counts) > total:
            counts[-1] -= sum(counts) - total
            if counts[-1] <= 0:
                counts.pop()
    return counts


@pytest.mark.parametrize("total", [None, 1, 7, 8, 9, 15, 16, 23, 24, 31])
def test_both_ends(total):
    rng = random.Random(total or 0)
    for seed in range(250 if total is None else 30):
        counts = some_counts(rng, total)
        m = Model(seed, pipe_overlap=False)
        with_ends(m, counts, seed=seed)
        m.run()
        assert not m.errors, (counts, m.errors[:3])


@pytest.mark.parametrize("bug,total", [("one_end", 15), ("one_end", 23), ("first_twice", None)])
def test_planted_mistakes_at_the_ends_are_caught(bug, total):
    rng = random.Random(5)
    for seed in range(100):
        m = Model(seed, stall_p=0.1)
        with_ends(m, some_counts(rng, total), seed=seed, bugs=(bug,))
        m.run(max_steps=200_000)
        if m.errors:
            return
    raise AssertionError("not caught")
