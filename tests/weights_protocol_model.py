"""Model of the attention-weight kernel's mbarrier pipeline (csrc/fa_weights.cu: weights_kernel), on
the checker of protocol_model.py: a warp that hands pieces of work to the other roles through a
ring, a TMA producer, which takes a piece when it issues the last tile of the one before, an MMA
issuer and 2 x 4 warps of weights, which load the queries of the job after the next one and write
those of the next one before they turn to this one's key tiles.  It restates the kernel's waits, arrivals and commits
and must change with it."""

from __future__ import annotations

from protocol_model import Bar, Buf, Sim


def weights(pieces, S, seed, ring=4, stats=4, bug=None, abort_at=None, groups=2):
    """pieces: (key tiles, jobs) of each piece, both at least 1.  `bug` plants a protocol error:
    "mma_no_s_wait", "no_q_wait", "early_k_release", "early_piece_release".  `stats`: places for the
    jobs' statistics.  `abort_at`: the abort_at-th spin of a bounded wait times out.  Returns the Sim."""
    sim = Sim(seed, abort_at)
    wait_ok = sim.wait_ok
    k_full, k_empty = ([Bar(1, f"{n}{s}") for s in range(S)] for n in ("k_full", "k_empty"))
    q_full, q_empty = ([Bar(c, f"{n}{t}") for t in range(2)] for n, c in (("q_full", 4 * groups), ("q_empty", 1)))
    s_full, s_empty = ([Bar(c, f"{n}{t}") for t in range(groups)] for n, c in (("s_full", 1), ("s_empty", 4)))
    mma_done = Bar(1, "mma_done")
    piece_full = [Bar(1, f"piece_full{i}") for i in range(ring)]
    piece_empty = [Bar(2 + 4 * groups, f"piece_empty{i}") for i in range(ring)]
    slots = [Buf(f"piece{i}") for i in range(ring)]
    Kst = [Buf(f"K{s}") for s in range(S)]
    Qt = [[Buf(f"Q{t}w{w}") for w in range(4 * groups)] for t in range(2)]
    stat = [[Buf(f"stats{i}w{w}") for w in range(4 * groups)] for i in range(stats)]
    Sreg = [[Buf(f"S{t}q{q}") for q in range(4)] for t in range(groups)]
    done = []
    first = [0]  # number of the first job of each piece
    for _, jobs in pieces:
        first.append(first[-1] + jobs)

    def walker():
        for i, n in enumerate(pieces + [None]):
            if not (yield from wait_ok(piece_empty[i % ring], ((i // ring) & 1) ^ 1, i // ring)):
                return
            slots[i % ring].write((i, n), readers=2 + 4 * groups if n is not None else 0)
            piece_full[i % ring].arrive()

    def take(i):
        if not (yield from wait_ok(piece_full[i % ring], (i // ring) & 1, i // ring + 1)):
            return None
        n = pieces[i] if i < len(pieces) else None
        slots[i % ring].read((i, n))
        return n if n is not None else ()

    def release(i):
        slots[i % ring].read((i, pieces[i]), consume=True)
        piece_empty[i % ring].arrive()

    def load(buf, val, bar):
        def fn():
            buf.write(val, readers=1)
            bar.arrive()
        sim.copy(fn)

    def producer():
        jk, i, ok = 0, 1, True
        got = yield from take(0)
        if got:
            release(0)
        while ok and got:
            tiles = got[0] * got[1]
            for x in range(tiles):
                if x == tiles - 1:
                    got = yield from take(i)
                    if got is None:
                        ok = False
                        break
                    if got:
                        release(i)
                    i += 1
                ok = yield from wait_ok(k_empty[jk % S], ((jk // S) & 1) ^ 1, jk // S)
                if not ok:
                    break
                load(Kst[jk % S], jk, k_full[jk % S])
                jk += 1
        for c in range(max(0, jk - S), jk):
            yield from sim.drain(k_full[c % S], (c // S) & 1)

    def op_S(job, j, c):
        def fn():
            for w in range(4 * groups):
                Qt[job & 1][w].read(job, consume=True)
            for q in range(4):
                Sreg[j % groups][q].write((job, j), readers=1)
            Kst[c % S].read(c, consume=True)
        sim.issue(fn)

    def commit(bar):
        sim.issue(bar.arrive)

    def mma():
        jk = job = i = 0
        issued = [0] * groups
        ok = True
        while ok:
            got = yield from take(i)
            if not got:
                break
            release(i)
            i += 1
            n, jobs = got
            for _ in range(jobs):
                if bug != "no_q_wait":
                    ok = yield from wait_ok(q_full[job & 1], (job >> 1) & 1, (job >> 1) + 1)
                for j in range(n if ok else 0):
                    t = j % groups
                    ok = yield from wait_ok(k_full[jk % S], (jk // S) & 1, jk // S + 1)
                    if ok and bug != "mma_no_s_wait":
                        ok = yield from wait_ok(s_empty[t], (issued[t] & 1) ^ 1, issued[t])
                    if not ok:
                        break
                    if bug == "early_k_release":
                        commit(k_empty[jk % S])
                    op_S(job, j, jk)
                    commit(s_full[t])
                    if bug != "early_k_release":
                        commit(k_empty[jk % S])
                    issued[t] += 1
                    jk += 1
                if not ok:
                    break
                commit(q_empty[job & 1])
                job += 1
        commit(mma_done)
        yield from sim.drain(mma_done, 0)

    def put(w, at, job):
        """Generator: False when the wait gives up."""
        if not (yield from wait_ok(q_empty[job & 1], ((job >> 1) & 1) ^ 1, job >> 1)):
            return False
        Qt[job & 1][w].write(job, readers=pieces[at][0])
        stat[job % stats][w].write(job, readers=4 * groups)
        q_full[job & 1].arrive()
        return True

    def warp(t, q):
        w, job, seen, i, r = 4 * t + q, 0, 0, 0, 0

        def following(at, k):
            """Generator: the job behind (piece, job of it); None when the wait gives up."""
            if at == len(pieces):
                return at, k
            if k + 1 < pieces[at][1]:
                return at, k + 1
            got = yield from take(at + 1)
            return None if got is None else (at + 1, 0)

        got = yield from take(0)
        if not got or not (yield from put(w, 0, 0)):
            return
        after = yield from following(0, 0)
        if after is None:
            return
        while True:
            n, jobs = pieces[i]
            ni, nr = after
            if ni < len(pieces):
                if not (yield from put(w, ni, job + 1)):
                    return
                after = yield from following(ni, nr)
                if after is None:
                    return
                if after[0] < len(pieces):  # its queries are loaded
                    slots[after[0] % ring].read((after[0], pieces[after[0]]))
            if bug == "early_piece_release" and ni != i:
                release(i)
            if not (yield from wait_ok(q_full[job & 1], (job >> 1) & 1, (job >> 1) + 1)):
                return
            for j in range(t, n, groups):
                seen += 1
                if not (yield from wait_ok(s_full[t], (seen - 1) & 1, seen)):
                    return
                slots[i % ring].read((i, pieces[i]))
                for x in range(4 * groups):
                    stat[job % stats][x].read(job)
                Sreg[t][q].read((job, j), consume=True)
                s_empty[t].arrive()
                yield
                done.append((job, j, q))
            for x in range(4 * groups):  # the job's statistics are free once all warps are through with it
                stat[job % stats][x].read(job, consume=True)
            job += 1
            if ni != i and bug != "early_piece_release":
                release(i)
            i, r = ni, nr
            if i == len(pieces):
                return

    sim.run([walker(), producer()] + [warp(t, q) for t in range(groups) for q in range(4)], mma())
    assert sim.exit_ops == 0, f"CTA exits with {sim.exit_ops} MMA operations queued"
    if not sim.abort:
        assert sim.exit_copies == 0, f"CTA exits with {sim.exit_copies} copies in flight"
        want = [(first[p] + r, j, q) for p, (n, jobs) in enumerate(pieces) for r in range(jobs)
                for j in range(n) for q in range(4)]
        assert sorted(done) == sorted(want)
    return sim
