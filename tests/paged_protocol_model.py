"""Model of the paged tensor-core kernel's mbarrier pipeline (csrc/fa_paged_mma.cu:
paged_mma_kernel), on the checker of protocol_model.py: a warp that hands pieces of work to the
other roles through a ring, a TMA producer, an MMA issuer and 2 x 4 softmax warps, which also write
the query tiles; with `twin`, both tile slots on one query tile at alternate key tiles.  It
restates the kernel's waits, arrivals and commits and must change with it."""

from __future__ import annotations

from protocol_model import Bar, Buf, Sim


def paged(pieces, S, seed, twin=False, ring=4, bug=None, abort_at=None):
    """pieces: (n0, n1), the key tiles of each query tile of a piece; with `twin` their number
    instead.  `bug` plants a protocol error: "mma_no_q_wait", "twin_no_wait", "early_v_release",
    "early_piece_release".  `abort_at`: the abort_at-th spin of a bounded wait times out.  Returns
    the Sim."""
    tiles = [((n + 1) // 2, n // 2) if twin else n for n in pieces]
    positions = [sum(n) if twin else max(n) for n in tiles]
    sim = Sim(seed, abort_at)
    wait_ok = sim.wait_ok
    q_full, mma_done, twin_full = Bar(8, "q_full"), Bar(1, "mma_done"), Bar(4, "twin_full")
    k_full, k_empty, v_full, v_empty = ([Bar(1, f"{n}{s}") for s in range(S)]
                                        for n in ("k_full", "k_empty", "v_full", "v_empty"))
    s_full, o_full = ([Bar(1, f"{n}{t}") for t in range(2)] for n in ("s_full", "o_full"))
    p_full = [Bar(4, f"p_full{t}") for t in range(2)]
    piece_full = [Bar(1, f"piece_full{i}") for i in range(ring)]
    piece_empty = [Bar(10, f"piece_empty{i}") for i in range(ring)]
    slots = [Buf(f"piece{i}") for i in range(ring)]
    Kst, Vst = ([Buf(f"{n}{s}") for s in range(S)] for n in "KV")
    Qt = [[Buf(f"Q{t}w{q}") for q in range(4)] for t in range(2)]
    Sreg = [[Buf(f"S{t}q{q}") for q in range(4)] for t in range(2)]
    Oreg = [[Buf(f"O{t}q{q}") for q in range(4)] for t in range(2)]
    stats = [Buf(f"stats q{q}") for q in range(4)]
    done = []

    def walker():
        for i, n in enumerate(tiles + [None]):
            if not (yield from wait_ok(piece_empty[i % ring], ((i // ring) & 1) ^ 1, i // ring)):
                return
            slots[i % ring].write((i, n), readers=10 if n is not None else 0)
            piece_full[i % ring].arrive()

    def take(i):
        """Generator: the i-th piece's (key tiles, positions); None when the wait gives up, and
        positions -1 behind the last piece."""
        if not (yield from wait_ok(piece_full[i % ring], (i // ring) & 1, i // ring + 1)):
            return None
        n = tiles[i] if i < len(tiles) else None
        slots[i % ring].read((i, n))
        return (n, positions[i] if n is not None else -1)

    def release(i):
        if i < len(tiles):
            slots[i % ring].read((i, tiles[i]), consume=True)
        piece_empty[i % ring].arrive()

    def readers_of(n, j):
        return 1 if twin else sum(1 for t in range(2) if j < n[t])

    def load(buf, val, readers, bar):
        def fn():
            buf.write(val, readers=readers)
            bar.arrive()
        sim.copy(fn)

    def producer():
        jk = jv = base = i = 0
        while True:
            got = yield from take(i)
            if got is None:
                break
            n, npos = got
            release(i)
            i += 1
            if npos < 0:
                break
            # (K or V, position) in the order of issue: with twin K runs one position ahead
            order = [x for j in range(npos) for x in (("K", j), ("V", j))]
            if twin and npos:
                order = [("K", 0)] + [x for j in range(npos)
                                      for x in ([("K", j + 1)] if j + 1 < npos else []) + [("V", j)]]
            ok = True
            for kind, j in order:
                c = jk if kind == "K" else jv
                assert c == base + j
                full, empty, st = (k_full, k_empty, Kst) if kind == "K" else (v_full, v_empty, Vst)
                ok = yield from wait_ok(empty[c % S], ((c // S) & 1) ^ 1, c // S)
                if not ok:
                    break
                load(st[c % S], c, readers_of(n, j), full[c % S])
                if kind == "K":
                    jk += 1
                else:
                    jv += 1
            if not ok:
                break
            base += npos
        for full, count in ((k_full, jk), (v_full, jv)):
            for c in range(max(0, count - S), count):
                yield from sim.drain(full[c % S], (c // S) & 1)

    def op_S(t, q_tile, piece, step, c):
        def fn():
            for q in range(4):
                Qt[q_tile][q].read(("Q", piece), consume=True)
                Sreg[t][q].write(("S", piece, step), readers=1)
            Kst[c % S].read(c, consume=True)
        sim.issue(fn)

    def op_PV(t, piece, step, c, last):
        def fn():
            for q in range(4):
                Sreg[t][q].read(("P", piece, step), consume=True)
                if step:
                    Oreg[t][q].read(("O", piece, step))
                Oreg[t][q].write(("O", piece, step + 1), readers=1 if last else 0)
            Vst[c % S].read(c, consume=True)
        sim.issue(fn)

    def commit(bar):
        sim.issue(bar.arrive)

    def mma():
        issued, base, segs, i = [0, 0], 0, 0, 0
        ok = True
        while ok:
            got = yield from take(i)
            if got is None:
                break
            n, npos = got
            release(i)
            piece, i = i, i + 1
            if npos < 0:
                break
            if npos == 0:
                continue
            if bug != "mma_no_q_wait":
                ok = yield from wait_ok(q_full, segs & 1, segs + 1)
                if not ok:
                    break
            segs += 1
            lag = 2 if twin else 1
            for j in range(npos + lag):
                c, cp, jp = base + j, base + j - lag, j - lag
                if not twin and j < npos:
                    ok = yield from wait_ok(k_full[c % S], (c // S) & 1, c // S + 1)
                if ok and jp >= 0:
                    ok = yield from wait_ok(v_full[cp % S], (cp // S) & 1, cp // S + 1)
                if not ok:
                    break
                if bug == "early_v_release" and jp >= 0:
                    commit(v_empty[cp % S])
                for t in ([j & 1] if twin else [0, 1]):
                    pv = jp >= 0 if twin else 0 <= jp < n[t]
                    if pv:
                        ok = yield from wait_ok(p_full[t], (issued[t] - 1) & 1, issued[t])
                        if not ok:
                            break
                        step = jp // 2 if twin else jp
                        last = step + 1 == n[t]
                        op_PV(t, piece, step, cp, last)
                        if last:
                            commit(o_full[t])
                        if twin and bug != "early_v_release":
                            commit(v_empty[cp % S])
                    if (j < npos) if twin else (j < n[t]):
                        if twin:
                            ok = yield from wait_ok(k_full[c % S], (c // S) & 1, c // S + 1)
                            if not ok:
                                break
                        op_S(t, 0 if twin else t, piece, j // 2 if twin else j, c)
                        commit(s_full[t])
                        if twin:
                            commit(k_empty[c % S])
                        issued[t] += 1
                if not ok:
                    break
                if not twin:
                    if j < npos:
                        commit(k_empty[c % S])
                    if jp >= 0 and bug != "early_v_release":
                        commit(v_empty[cp % S])
            base += npos
        commit(mma_done)
        yield from sim.drain(mma_done, 0)

    def softmax(t, q):
        segs = seen = outs = twins = i = 0
        while True:
            got = yield from take(i)
            if got is None:
                return
            n, npos = got
            piece, i = i, i + 1
            if npos < 0:
                return
            if bug == "early_piece_release":
                release(piece)
            if npos > 0:
                if n[t] > 0 and not (twin and t == 1):
                    Qt[t][q].write(("Q", piece), readers=npos if twin else n[t])
                q_full.arrive()
                if not (yield from wait_ok(q_full, segs & 1, segs + 1)):
                    return
                segs += 1
            for j in range(n[t]):
                if not (yield from wait_ok(s_full[t], (seen + j) & 1, seen + j + 1)):
                    return
                slots[piece % ring].read((piece, n))  # its fields are read until the piece is done
                Sreg[t][q].read(("S", piece, j), consume=True)
                if j:  # rescaling O~ needs every earlier P V of the slot to have completed
                    Oreg[t][q].read(("O", piece, j))
                Sreg[t][q].write(("P", piece, j), readers=1)
                p_full[t].arrive()
            seen += n[t]
            if n[t] > 0:
                outs += 1
                if not (yield from wait_ok(o_full[t], (outs - 1) & 1, outs)):
                    return
            both = twin and npos >= 2
            if both and t == 1:
                stats[q].write(piece, readers=1)
                twin_full.arrive()
            else:
                if both:
                    if bug != "twin_no_wait":
                        if not (yield from wait_ok(twin_full, twins & 1, twins + 1)):
                            return
                    twins += 1
                    yield
                    stats[q].read(piece, consume=True)
                    Oreg[1][q].read(("O", piece, n[1]), consume=True)
                if n[t] > 0:
                    Oreg[t][q].read(("O", piece, n[t]), consume=True)
                if not (twin and t == 1):
                    done.append((piece, t, q))
            if bug != "early_piece_release":
                release(piece)

    sim.run([walker(), producer()] + [softmax(t, q) for t in range(2) for q in range(4)], mma())
    assert sim.exit_ops == 0, f"CTA exits with {sim.exit_ops} MMA operations queued"
    if not sim.abort:
        assert sim.exit_copies == 0, f"CTA exits with {sim.exit_copies} copies in flight"
        want = [(p, t, q) for p in range(len(tiles)) for t in range(1 if twin else 2) for q in range(4)]
        assert sorted(done) == want
    return sim
