"""The end of the projections' blocks (k_tile, k_few) modelled on the host: what is asynchronous arrives
later than it is issued, and nothing may arrive at a CTA's barriers once its block may have ended.

Copies and commits are kept in flight and delivered in any order (a commit's arrivals at a pair's two
CTAs apart from one another); a block ends when all the roles of its cluster have.  A delivery after
that is the fault looked for."""
import random

import pytest


def run(roles, counts, seed):
    """None, or a description of the failure.  Operations: ("wait", barrier, k) for its k-th phase,
    ("arrive", barrier), ("later", barrier) for an arrival that comes at some time afterwards."""
    rng = random.Random(seed)
    gens = [r() for r in roles]
    cur = [next(g, None) for g in gens]
    arrivals, flying = {}, []
    done = lambda b: arrivals.get(b, 0) // counts.get(b, 1)
    # some runs deliver only when no role can go on, and one kind of arrival only when nothing else flies
    eager, slow = rng.choice((0.3, 0.0)), rng.choice(("full", "empty", "acc_full", None))
    while any(c is not None for c in cur):
        ready = []
        for i, c in enumerate(cur):
            if c is None:
                continue
            if c[0] != "wait":
                ready.append(i)
                continue
            if done(c[1]) >= c[2] + 2:
                return f"role {i} waits for phase {c[2]} of {c[1]} after {done(c[1])} completions"
            if done(c[1]) == c[2] + 1:
                ready.append(i)
        if not ready and not flying:
            return f"deadlock at {cur}"
        if flying and (not ready or rng.random() < eager):
            first = [i for i, b in enumerate(flying) if b[0] != slow] or range(len(flying))
            b = flying.pop(rng.choice(first))
            arrivals[b] = arrivals.get(b, 0) + 1
            continue
        i = rng.choice(ready)
        op = cur[i]
        if op[0] == "arrive":
            arrivals[op[1]] = arrivals.get(op[1], 0) + 1
        elif op[0] == "later":
            flying.append(op[1])
        cur[i] = next(gens[i], None)
    return f"after the blocks' end: {sorted(set(flying))}" if flying else None


def roles(cg, stages, epi, tiles, nk, chunk, drain=True, pieces=0):
    """`drain` False leaves out the producers' last wait for the stages' `empty` barriers.  `pieces`: a
    tile's pieces of residual, the first asked for before the chunks, each waited for after them."""
    nch = -(-nk // chunk)
    sizes = [nk * (c + 1) // nch - nk * c // nch for c in range(nch)]
    total = tiles * nk

    def producer(cta):
        for it in range(total):
            s = it % stages
            if it >= stages:
                yield ("wait", ("empty", cta, s), it // stages - 1)
            yield ("later", ("full", s))
        for i in range(stages):
            uses = total // stages + (i < total % stages)
            if uses and cta == 0:
                yield ("wait", ("full", i), uses - 1)
            if uses and drain:
                yield ("wait", ("empty", cta, i), uses - 1)

    def issuer():
        it = ac = 0
        for _ in range(tiles):
            for n in sizes:
                buf = ac & 1
                if ac >= 2:
                    yield ("wait", ("acc_empty", buf), ac // 2 - 1)
                for _ in range(n):
                    yield ("wait", ("full", it % stages), it // stages)
                    for cta in range(cg):
                        yield ("later", ("empty", cta, it % stages))
                    it += 1
                for cta in range(cg):
                    yield ("later", ("acc_full", cta, buf))
                ac += 1

    def warp(cta, i):
        for t in range(tiles):
            if pieces:
                yield ("later", ("res", cta, i))
            for ac in range(t * nch, (t + 1) * nch):
                yield ("wait", ("acc_full", cta, ac & 1), ac // 2)
                yield ("arrive", ("acc_empty", ac & 1))
            for k in range(pieces):
                if k:
                    yield ("later", ("res", cta, i))
                yield ("wait", ("res", cta, i), t * pieces + k)

    rs = [issuer] + [(lambda c=c: producer(c)) for c in range(cg)]
    rs += [(lambda c=c, i=i: warp(c, i)) for c in range(cg) for i in range(epi)]
    counts = {("full", s): cg for s in range(stages)}
    counts.update({("acc_empty", b): epi * cg for b in range(2)})
    return rs, counts


SIZES = [(1, 1, 12), (1, 13, 4), (3, 1, 12), (4, 7, 3), (5, 12, 12), (2, 25, 12)]


@pytest.mark.parametrize("cg,stages,epi", [(1, 3, 2), (1, 6, 8), (2, 5, 2), (2, 6, 3)])
@pytest.mark.parametrize("tiles,nk,chunk", SIZES)
@pytest.mark.parametrize("pieces", [0, 1, 2])
def test_nothing_arrives_after_the_end(cg, stages, epi, tiles, nk, chunk, pieces):
    for seed in range(12):
        assert run(*roles(cg, stages, epi, tiles, nk, chunk, pieces=pieces), seed) is None


@pytest.mark.parametrize("cg,stages,epi", [(1, 6, 8), (2, 5, 2)])
@pytest.mark.parametrize("tiles,nk,chunk", SIZES)
def test_without_the_last_wait_something_does(cg, stages, epi, tiles, nk, chunk):
    found = [run(*roles(cg, stages, epi, tiles, nk, chunk, drain=False), seed) for seed in range(24)]
    assert any(f is not None and f.startswith("after the blocks' end") for f in found)
