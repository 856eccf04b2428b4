"""The projections' mbarrier protocol (k_tile, k_few) modelled on the host: a TMA producer per CTA,
one MMA issuer, the epilogue warps, for single CTAs and pairs, in the order and with the phases of
the kernel source.  As in test_barrier_protocols: no interleaving deadlocks, no wait is two phases
behind, and a planted wrong phase is found."""
import pytest

from test_barrier_protocols import run


def roles(cg, stages, epi, tiles, nk, chunk, late=0):
    """nk stages per tile in chunks of at most `chunk`; `late` shifts the issuer's wait for a free
    accumulator (0 is the kernel's)."""
    nch = -(-nk // chunk)
    sizes = [nk * (c + 1) // nch - nk * c // nch for c in range(nch)]
    total = tiles * nk

    def producer(cta):
        for it in range(total):
            s = it % stages
            if it >= stages:
                yield ("wait", ("empty", cta, s), it // stages - 1)
            yield ("arrive", ("full", s))                 # the CTA's copies of the stage
        if cta == 0:                                      # every copy has landed
            for i in range(stages):
                uses = total // stages + (i < total % stages)
                if uses:
                    yield ("wait", ("full", i), uses - 1)

    def issuer():
        it = ac = 0
        for _ in range(tiles):
            for n in sizes:
                buf = ac & 1
                if ac >= 2:
                    yield ("wait", ("acc_empty", buf), ac // 2 - 1 + late)
                for i in range(n):
                    s = it % stages
                    yield ("wait", ("full", s), it // stages)
                    for cta in range(cg):
                        yield ("arrive", ("empty", cta, s))
                    it += 1
                for cta in range(cg):
                    yield ("arrive", ("acc_full", cta, buf))
                ac += 1

    def warp(cta):
        for ac in range(tiles * nch):
            buf = ac & 1
            yield ("wait", ("acc_full", cta, buf), ac // 2)
            yield ("arrive", ("acc_empty", buf))

    rs = [issuer] + [(lambda c=c: producer(c)) for c in range(cg)]
    rs += [(lambda c=c: warp(c)) for c in range(cg) for _ in range(epi)]
    counts = {("full", s): cg for s in range(stages)}
    counts.update({("acc_empty", b): epi * cg for b in range(2)})
    return rs, counts


@pytest.mark.parametrize("cg,stages,epi", [(1, 3, 2), (1, 6, 8), (2, 5, 2), (2, 6, 3)])
@pytest.mark.parametrize("tiles,nk,chunk", [(1, 1, 12), (1, 13, 4), (3, 1, 12), (4, 7, 3), (5, 12, 12), (2, 25, 12)])
def test_protocol_completes(cg, stages, epi, tiles, nk, chunk):
    for seed in range(8):
        rs, counts = roles(cg, stages, epi, tiles, nk, chunk)
        assert run(rs, counts, seed) is None


def test_wrong_phase_is_found():
    found = [run(*roles(2, 5, 2, 4, 7, 3, late=1), seed) for seed in range(8)]
    assert all(f is not None for f in found)
