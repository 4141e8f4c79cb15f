"""CPU check of the blocked cache attention kernel's synchronisation (cache_sparse_kernel), with the discrete-event model
of tests/pipeline_model.py: many random interleavings with random stalls must finish without a deadlock, a barrier phase
passed with the wrong number of completions, a region reused while a copy or tensor operation may still touch it, or a
value (tile record, row factor, row maximum, denominator share) read after another step overwrote it. Planted mistakes
must be caught."""
import random

import pytest

from tests.pipeline_model import Model

BATCH, BATCHES, KST = 8, 3, 3
FAC, TOPS, DENS = 4, 4, 2  # slots of the row factors (items), maxima (tiles), denominator shares (items)


def cache_sparse_model(m, counts, seed=0, bugs=()):
    tiles = [(k, t, c) for k, c in enumerate(counts) for t in range(c)]
    N = len(tiles)
    first = [t == 0 for _, t, _ in tiles]
    last = [t == c - 1 for _, t, c in tiles]
    pre = [t == c - 2 for _, t, c in tiles]
    item = [k for k, _, _ in tiles]
    rng = random.Random(seed)
    rescale = {n: not first[n] and rng.random() < 0.4 for n in range(N)}
    consumers = 9
    for s in range(2):
        for b in ("Q_FULL", "Q_EMPTY", "V8_FULL", "V8_EMPTY", "VF_FULL", "S_FULL", "PV_DONE", "FLUSHED"):
            m.bar(f"{b}{s}")
        for b in ("P_FULL", "STAGED", "S_FREE", "M_READY"):
            m.bar(f"{b}{s}", 2)  # both halves of a pair
    m.bar("O_FREE", 2)
    m.bar("MMA_DONE")
    for s in range(KST):
        m.bar(f"K_FULL{s}")
        m.bar(f"K_EMPTY{s}")
    for s in range(BATCHES):
        m.bar(f"REC_FULL{s}")
        m.bar(f"REC_EMPTY{s}", consumers)

    def reader():
        k = 0
        while True:
            sl = k % BATCHES
            yield ("wait", f"REC_EMPTY{sl}", k // BATCHES - 1)
            for i in range(BATCH):
                yield ("put", f"REC{sl}.{i}", k * BATCH + i)
            yield ("arrive", f"REC_FULL{sl}")
            k += 1
            if k * BATCH > N:  # the end record was in this batch
                return

    def record(n):
        k = n // BATCH
        if n % BATCH == 0:
            yield ("wait", f"REC_FULL{k % BATCHES}", k // BATCHES)
        yield ("get", f"REC{k % BATCHES}.{n % BATCH}", n)

    def release(n):
        if n % BATCH == BATCH - 1:
            yield ("arrive", f"REC_EMPTY{(n // BATCH) % BATCHES}")

    def tma(full, empty, region, stages):
        for n in range(N + 1):
            yield from record(n)
            if n == N:
                return
            s = n % stages
            yield ("wait", f"{empty}{s}", n // stages - 1)
            yield ("expect", f"{full}{s}", 1)
            yield ("tma", f"{full}{s}", 1, f"{region}{s}")
            yield from release(n)

    def q_warps():
        k = 0
        for n in range(N + 1):
            yield from record(n)
            if n == N:
                return
            yield from release(n)
            if not first[n]:
                continue
            if "no_q_empty_wait" not in bugs:
                yield ("wait", f"Q_EMPTY{k & 1}", (k >> 1) - 1)
            yield ("write", f"Q{k & 1}")
            yield ("put", f"FAC{k % (2 if 'short_fac' in bugs else FAC)}", k)
            yield ("arrive", f"Q_FULL{k & 1}")
            k += 1

    def v_warps():
        fin, staged, flushed = [False, False], [0, 0], [0, 0]

        def flush(sl):
            yield ("wait", f"STAGED{sl}", staged[sl])
            staged[sl] += 1
            yield ("store", f"FLUSHED{sl}", f"VF{sl}")
            yield ("wait", f"FLUSHED{sl}", flushed[sl])
            flushed[sl] += 1
            fin[sl] = False

        for n in range(N + 1):
            yield from record(n)
            if n == N:
                break
            yield from release(n)
            b = n & 1
            if n >= 2:
                if fin[b] and "no_flush" not in bugs:
                    yield from flush(b)
                else:
                    yield ("wait", f"PV_DONE{b}", (n - 2) >> 1)
            yield ("wait", f"V8_FULL{b}", n >> 1)
            yield ("read", f"V8{b}")
            yield ("write", f"VF{b}")
            yield ("arrive", f"V8_EMPTY{b}")
            yield ("arrive", f"VF_FULL{b}")
            fin[b] = last[n]
        for x in range(2):
            if fin[(N + x) & 1]:
                yield from flush((N + x) & 1)

    def mma():
        st = {"pv": 0, "pv_items": 0}

        def issue_pv():
            pv = st["pv"]
            b = pv & 1
            yield ("wait", f"P_FULL{b}", pv >> 1)
            yield ("wait", f"VF_FULL{b}", pv >> 1)
            if first[pv]:
                if st["pv_items"] > 0 and "no_o_free_wait" not in bugs:
                    yield ("wait", "O_FREE", st["pv_items"] - 1)
                st["pv_items"] += 1
            yield ("mma", [f"P{b}h0", f"P{b}h1", f"VF{b}"], ["O"])
            yield ("commit", f"PV_DONE{b}")
            st["pv"] += 1

        items = 0
        for n in range(N + 1):
            yield from record(n)
            if n == N:
                break
            yield from release(n)
            if first[n]:
                items += 1
                yield ("wait", f"Q_FULL{(items - 1) & 1}", (items - 1) >> 1)
            qs, ks, b = (items - 1) & 1, n % KST, n & 1
            yield ("wait", f"K_FULL{ks}", n // KST)
            if "no_s_free_wait" not in bugs:
                yield ("wait", f"S_FREE{b}", (n >> 1) - 1)
            yield ("mma", [f"Q{qs}", f"K{ks}"], [f"S{b}h0", f"S{b}h1"])
            yield ("commit", f"S_FULL{b}")
            yield ("commit", f"K_EMPTY{ks}")
            if last[n] or ("early_q_release" in bugs and first[n]):
                if not ("early_q_release" in bugs and not first[n]):
                    yield ("commit", f"Q_EMPTY{qs}")
            if n >= 2:
                yield from issue_pv()
        while st["pv"] < N:
            yield from issue_pv()
        yield ("commit", "MMA_DONE")
        yield ("wait", "MMA_DONE", 0)

    def softmax(pair, half):
        grp = 2 * pair + half
        for n in range(N + 1):
            yield from record(n)
            if n == N:
                return
            yield from release(n)
            if n & 1 != pair:
                continue
            k = item[n]
            yield ("wait", f"S_FULL{pair}", n >> 1)
            yield ("read", f"S{pair}h{half}")
            yield ("get", f"FAC{k % (2 if 'short_fac' in bugs else FAC)}", k)
            yield ("arrive", f"S_FREE{pair}")
            late = "publish_first" in bugs
            if n > 0 and not late:
                yield ("wait", f"M_READY{pair ^ 1}", (n - 1) >> 1)
            yield ("put", f"T{n % TOPS}h{half}", n)
            yield ("arrive", f"M_READY{pair}")
            if n > 0 and late:
                yield ("wait", f"M_READY{pair ^ 1}", (n - 1) >> 1)
            if not first[n]:
                yield ("get", f"T{(n - 1) % TOPS}h0", n - 1)
                yield ("get", f"T{(n - 1) % TOPS}h1", n - 1)
            yield ("wait", f"M_READY{pair}", n >> 1)
            yield ("get", f"T{n % TOPS}h{half ^ 1}", n)
            if n >= 2 and "no_p_free_wait" not in bugs:
                yield ("wait", f"PV_DONE{pair}", (n - 2) >> 1)
            yield ("write", f"P{pair}h{half}")
            if rescale[n]:
                if "no_rescale_wait" not in bugs:
                    yield ("wait", f"PV_DONE{pair ^ 1}", (n - 1) >> 1)
                yield ("read", "O")
                yield ("write", "O")
            if pre[n] or last[n]:
                yield ("put", f"D{k % DENS}g{grp}", k)
            yield ("arrive", f"P_FULL{pair}")
            if not last[n]:
                continue
            if "no_epilogue_pv_wait" not in bugs:
                yield ("wait", f"PV_DONE{pair}", n >> 1)
            yield ("get", f"D{k % DENS}g{grp ^ 1}", k)
            if not first[n]:
                yield ("get", f"D{k % DENS}g{2 * (pair ^ 1)}", k)
                yield ("get", f"D{k % DENS}g{2 * (pair ^ 1) + 1}", k)
            yield ("read", "O")
            yield ("arrive", "O_FREE")
            yield ("write", f"VF{pair}")
            yield ("arrive", f"STAGED{pair}")

    m.roles = {"reader": reader(), "tma_k": tma("K_FULL", "K_EMPTY", "K", KST), "tma_v": tma("V8_FULL", "V8_EMPTY", "V8", 2),
               "q": q_warps(), "v": v_warps(), "mma": mma()}
    m.roles.update({f"softmax{p}{h}": softmax(p, h) for p in range(2) for h in range(2)})


def test_protocol():
    rng = random.Random(7)
    for seed in range(250):
        counts = [rng.choice([1, 1, 1, 2, 3, 5, 9]) for _ in range(rng.randint(1, 9))]
        m = Model(seed, pipe_overlap=False)
        cache_sparse_model(m, counts, seed=seed)
        m.run()
        assert not m.errors, (counts, m.errors[:3])


@pytest.mark.parametrize("bug", ["no_q_empty_wait", "early_q_release", "no_flush", "no_o_free_wait", "no_s_free_wait",
                                 "no_p_free_wait", "no_rescale_wait", "no_epilogue_pv_wait", "short_fac", "publish_first"])
def test_planted_mistakes_are_caught(bug):
    rng = random.Random(3)
    caught = 0
    for seed in range(200):
        counts = [rng.choice([1, 1, 2, 3, 5]) for _ in range(rng.randint(2, 8))]
        m = Model(seed, stall_p=0.1)
        cache_sparse_model(m, counts, seed=seed, bugs=(bug,))
        m.run(max_steps=200_000)
        caught += bool(m.errors)
        if caught:
            return
    assert caught > 0
