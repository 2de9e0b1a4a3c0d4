"""CPU model of the paged kernel's key/value ring for fp16: barriers whose
phases are told by parity, the copying warp, the product warp and the two
warps that look at V tiles, taken in random order.  The kernel's rule (a V
stage is filled again only when all three have let it go) never lets a wait
take another phase for its own; with the product warp's release alone, one
does as soon as a V warp falls behind."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        """try_wait.parity: the phase of that parity is not the current one."""
        return self.phase & 1 != parity


class Mistaken(Exception):
    pass


def ring(stages, tiles, ragged, v_count, rng, slow):
    """One run over `tiles` key tiles; `ragged`: those whose V rows are fixed;
    slow: one of the V warps moves once in a while only."""
    full = [Barrier(1) for _ in range(stages)]
    empty = [Barrier(v_count if s % 2 else 1) for s in range(stages)]
    ready = [Barrier(2) for _ in range(stages)]

    def wait(bar, fill, parity):
        while not bar.passed(parity):
            yield
        if bar.phase != fill + 1:
            raise Mistaken("phase %d taken for %d" % (bar.phase - 1, fill))

    def load():
        for at in range(2 * tiles):
            s, n = at % stages, at // stages
            if n:
                yield from wait(empty[s], n - 1, (n - 1) & 1)
            full[s].arrive()
            yield

    def products():
        for j in range(tiles):
            for at in (2 * j, 2 * j + 1):
                s, n = at % stages, at // stages
                yield from wait(full[s], n, n & 1)
                if at % 2 and j in ragged:
                    while ready[s].phase == ready_seen[s]:
                        yield
                    ready_seen[s] += 1
                empty[s].arrive()
                yield

    def v_warp():
        for j in range(tiles):
            at = 2 * j + 1
            s, n = at % stages, at // stages
            yield from wait(full[s], n, n & 1)
            if v_count == 3:
                empty[s].arrive()
            if j in ragged:
                yield
                ready[s].arrive()
            yield

    ready_seen = [0] * stages
    late = v_warp()
    roles = [load(), products(), v_warp(), late]
    steps = 0
    while roles:
        steps += 1
        assert steps < 100000, "no role moves"
        r = rng.choice(roles)
        if slow and r is late and rng.random() > 0.02:
            continue
        try:
            next(r)
        except StopIteration:
            roles.remove(r)


@pytest.mark.parametrize("stages", [4, 8])
@pytest.mark.parametrize("seed", range(30))
def test_no_wait_takes_another_phase_for_its_own(stages, seed):
    rng = random.Random(seed)
    tiles = rng.randint(1, 60)
    ragged = {j for j in range(tiles) if rng.random() < 0.1} | {tiles - 1}
    ring(stages, tiles, ragged, 3, rng, slow=rng.random() < 0.5)


def test_the_products_release_alone_is_not_enough():
    with pytest.raises((Mistaken, AssertionError)):
        for seed in range(20):
            ring(4, 40, {39}, 1, random.Random(seed), slow=True)
