"""When a CTA of the linear layer's kernel may leave, as a timing model of csrc/linear.cu.

A pair of CTAs runs one ring of slices. Each CTA's producer loads its share of a slice when the commit of
the MMA that read the slot before has arrived in that CTA; all copies count on rank 0's barriers. One thread
of rank 0 issues MMAs, a commit per slice, one per tile, one at the end; each commit arrives in both CTAs, at
delays of its own, so commits to different barriers may arrive in another order than they were issued in.
The first arrivals of a run are as they come; a run may lose one copy (its barrier never completes, and waits
for it give up), or have another role stop rank 0 early.

Shared memory is released when both CTAs have met at the last cluster barrier. Nothing may be on its way
into it then. The leave rules: "counts", the kernel's (each CTA waits for the last phase of each of its
barriers, rank 1 by the number of commits that rank 0 sends it, and rank 0 for all copies that rank 1 says it
has issued); "drain" (rank 1 waits for the last commit alone); "armed" (rank 0 waits only for slices that it
has announced itself).
"""
import random

import pytest

NS, LIMIT = 6, 1e6


def leaves_safely(rng, rule, lost=False, stop=False):
    """One run; True if nothing lands after the cluster barrier."""
    n = rng.randint(1, 30)

    def delay():
        return rng.expovariate(1.0) * rng.choice([0.1, 1.0, 5.0])
    lost_copy = (rng.randrange(n), rng.randrange(2)) if lost else None
    stop_at = rng.uniform(0.0, 25.0) if stop else float("inf")  # rank 0's roles give up once they wait longer than this
    loads = ([], [])   # of each CTA: when the copies of its slices land
    commits = []       # (arrival in CTA 0, in CTA 1) of each slice's commit
    at = [0.0, 0.0]    # the producers' clocks
    live = [True, True]
    mma, mma_live = 0.0, True
    for i in range(n):
        for r in (0, 1):
            if not live[r]:
                continue
            free = 0.0 if i < NS else commits[i - NS][r] if i - NS < len(commits) else float("inf")
            if max(free, at[r]) > (stop_at if r == 0 else LIMIT) and free > at[r]:  # a blocked wait ends
                at[r] = max(at[r], stop_at) if r == 0 and stop else at[r] + LIMIT
                live[r] = False
                continue
            at[r] = max(at[r], free)
            loads[r].append(at[r] + delay() if lost_copy != (i, r) else None)
        if mma_live:
            full = max((loads[r][i] if i < len(loads[r]) and loads[r][i] is not None else float("inf")) for r in (0, 1))
            if full > mma and full > min(mma + LIMIT, stop_at):
                mma = max(mma, stop_at) if stop else mma + LIMIT
                mma_live = False
            else:
                mma = max(mma, full) + rng.uniform(0.0, 0.5)
                commits.append((mma + delay(), mma + delay()))
    tile = [(mma + delay(), mma + delay())] if mma_live else []
    last = (mma + delay(), mma + delay())
    arrivals = [[c[r] for c in commits + tile] + [last[r]] for r in (0, 1)]
    lands = [[t for t in loads[r] if t is not None] for r in (0, 1)]
    leave0 = max(arrivals[0] + [mma, at[0]])  # the MMA thread's own barriers
    if rule == "armed":
        seen = len(loads[0])
        leave0 = max([leave0] + lands[0] + [t for t in loads[1][:seen] if t is not None])
    else:
        leave0 = max([leave0, at[1] + delay()] + lands[0] + lands[1])
    leave1 = max(at[1], last[1]) if rule == "drain" else max([at[1], mma + delay()] + arrivals[1])
    leave = max(leave0, leave1)
    return max(arrivals[0] + arrivals[1] + lands[0] + lands[1]) <= leave


@pytest.mark.parametrize("lost,stop", [(False, False), (True, False), (False, True)])
def test_nothing_lands_after_the_last_barrier(lost, stop):
    rng = random.Random(7)
    for _ in range(4000):
        assert leaves_safely(rng, "counts", lost, stop)


def test_the_last_commit_alone_is_not_enough():
    rng = random.Random(7)
    assert not all(leaves_safely(rng, "drain") for _ in range(4000))


def test_slices_that_only_the_other_cta_has_loaded_count():
    rng = random.Random(7)
    assert not all(leaves_safely(rng, "armed", stop=True) for _ in range(4000))
