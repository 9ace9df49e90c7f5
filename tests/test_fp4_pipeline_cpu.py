"""The pipeline protocol of the 4-bit grouped product (gemm_fp4.cu), modelled on the CPU with
pipeline_model.py, for one SM and for SM pairs.

Codes and scales come by producers of their own into rings of their own.  A turning warp rewrites a
window of scales when its copy has landed and reports it: in a pair the leader's arms the leader's
`turned` barrier and the follower's completes it by an asynchronous copy, so that it may land before
the leader's arrives.  The MMA warp waits for a stage's codes and scales, and its commits free both.
Eight epilogue warps a CTA free an accumulator.  A window of MXFP4 is copied for each of its two
stages, as one of NVFP4 is for its one.

Every wait must pass on the phase it means, every arrival land in its phase, and every schedule run
to its end."""

import os
import random
import re

import pytest

import pipeline_model as model
from pipeline_model import Barrier, ring, wait_full

SOURCE = open(os.path.join(os.path.dirname(__file__), "..", "moe_grouped_matrix_gb300", "csrc", "gemm_fp4.cu")).read()


def depths(pair):
    """(stages of codes, windows of scales, turning warps) as the kernel has them."""
    def pick(name):
        m = re.search(rf"static constexpr int {name} = kPair \? (\d+) : (\d+);", SOURCE)
        return int(m.group(1 if pair else 2))

    return pick("kStages"), pick("kScales"), int(re.search(r"constexpr int kTurners = (\d+);", SOURCE).group(1))


def roles(tiles, pair, turner_of=None):
    n_codes, n_scales, turners = depths(pair)
    ctas = range(2 if pair else 1)
    total = sum(tiles)
    # the leader's: its arm and each CTA's bytes; its turning warp and, in a pair, the follower's signal
    full = [Barrier(f"full{s}", 1 + len(ctas)) for s in range(n_codes)]
    turned = [Barrier(f"turned{s}", len(ctas)) for s in range(n_scales)]
    empty = [ring(f"empty[cta{c}]", n_codes, 1) for c in ctas]
    sempty = [ring(f"sempty[cta{c}]", n_scales, 1) for c in ctas]
    sfull = [ring(f"sfull[cta{c}]", n_scales, 2) for c in ctas]  # the arm, and the bytes
    accf = [ring(f"accf[cta{c}]", 2, 1) for c in ctas]
    acce = ring("acce", 2, 8 * len(ctas))

    def codes(cta):
        for s in range(total):
            yield wait_full(empty[cta][s % n_codes], s // n_codes - 1)
            if cta == 0:
                yield ("arrive", full[s % n_codes], s // n_codes)
            yield ("async", None, full[s % n_codes], s // n_codes)

    def scales(cta):
        for s in range(total):
            yield wait_full(sempty[cta][s % n_scales], s // n_scales - 1)
            yield ("arrive", sfull[cta][s % n_scales], s // n_scales)
            yield ("async", None, sfull[cta][s % n_scales], s // n_scales)

    def turner(cta, which):
        for s in range(total):
            mine = (s % n_scales) % turners if turner_of is None else turner_of(s)
            if mine == which:
                yield wait_full(sfull[cta][s % n_scales], s // n_scales)
                if cta == 0:
                    yield ("arrive", turned[s % n_scales], s // n_scales)
                else:
                    yield ("async", None, turned[s % n_scales], s // n_scales)

    def mma():
        s = 0
        for t, stages in enumerate(tiles):
            yield wait_full(acce[t % 2], t // 2 - 1)
            for kb in range(stages):
                yield wait_full(turned[s % n_scales], s // n_scales)
                yield wait_full(full[s % n_codes], s // n_codes)
                for c in ctas:
                    yield ("async", "mma", empty[c][s % n_codes], s // n_codes)
                for c in ctas:
                    yield ("async", "mma", sempty[c][s % n_scales], s // n_scales)
                if kb == stages - 1:
                    for c in ctas:
                        yield ("async", "mma", accf[c][t % 2], t // 2)
                s += 1

    def epilogue(cta):
        for t in range(len(tiles)):
            yield wait_full(accf[cta][t % 2], t // 2)
            yield ("arrive", acce[t % 2], t // 2)

    return ([codes(c) for c in ctas] + [scales(c) for c in ctas] + [turner(c, w) for c in ctas for w in range(turners)]
            + [mma()] + [epilogue(c) for c in ctas for _ in range(8)])


def tiles(seed, n=12):
    rng = random.Random(seed)
    return [rng.choice((1, 2, 3, 8, 16)) for _ in range(n)]


@pytest.mark.parametrize("pair", [False, True])
def test_every_schedule_runs_to_its_end(pair):
    for seed in range(25):
        errors = model.run(roles(tiles(seed), pair), seed)
        assert not errors, (pair, seed, errors[:3])


@pytest.mark.parametrize("pair", [False, True])
def test_turning_warps_without_slots_of_their_own_are_caught(pair):
    """A control: turning warps that take every n-th window, whatever its slot, wait on barriers of which
    they have not seen every phase, and pass on the phase before."""
    _, n_scales, turners = depths(pair)
    assert n_scales % turners
    for seed in range(400):
        if any("passed at" in e for e in model.run(roles([16] * 6, pair, turner_of=lambda s: s % turners), seed)):
            return
    pytest.fail("no schedule showed it")
