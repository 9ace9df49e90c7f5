"""The 4-bit grouped product's protocol (test_fp4_pipeline_cpu.py's roles) with the MMA warp's commits in
the kernel's order: a window of scales is released once it has been copied to tensor memory, before the
stage's MMAs, its codes after them.  So a window may be filled and turned again while the MMAs that use the
one before in its slot are still to come."""

import pytest

import pipeline_model as model
from test_fp4_pipeline_cpu import SOURCE, depths, roles, tiles

ORDER = ("sempty", "empty", "accf")


def mma_last(pair):
    return -1 - 8 * (2 if pair else 1)  # the MMA warp's place in roles(): before the epilogue warps


def in_kernel_order(gen):
    """The same operations, each run of commits in the kernel's order."""
    commits = []
    for op in gen:
        if op[0] == "async":
            commits.append(op)
            continue
        yield from sorted(commits, key=lambda c: [c[2].name.startswith(n) for n in ORDER].index(True))
        commits = []
        yield op
    yield from sorted(commits, key=lambda c: [c[2].name.startswith(n) for n in ORDER].index(True))


def test_the_kernel_commits_in_this_order():
    at = [SOURCE.index(f"commit<kPair>({bar}_bar(") for bar in ORDER]
    first_mma = SOURCE.index("mma_fp4<kPair, kNv>(d_tmem")
    assert at == sorted(at) and at[0] < first_mma < at[1]


@pytest.mark.parametrize("pair", [False, True])
def test_every_schedule_runs_to_its_end(pair):
    for seed in range(40):
        gens = roles(tiles(seed), pair)
        gens[mma_last(pair)] = in_kernel_order(gens[mma_last(pair)])
        errors = model.run(gens, seed)
        assert not errors, (pair, seed, errors[:3])


@pytest.mark.parametrize("pair", [False, True])
def test_a_window_is_filled_again_while_its_stage_waits_for_its_mmas(pair):
    """The schedules that the order allows, and only it, are among those played: a window's next filling is
    armed before the codes of the stage that used it are released."""
    n_codes, n_scales, _ = depths(pair)

    def ahead(reorder):
        seen = False
        for seed in range(40):
            gens = roles([16] * 4, pair)
            if reorder:
                gens[mma_last(pair)] = in_kernel_order(gens[mma_last(pair)])
            scales = 2 if pair else 1  # the leader's copies of scales, after the copies of codes
            inner, codes = gens[scales], []

            def watched():
                nonlocal seen
                s = 0
                for op in inner:
                    if op[0] == "arrive":
                        old = s - n_scales
                        if old >= 0 and codes[0][old % n_codes].done <= old // n_codes:
                            seen = True
                        s += 1
                    yield op

            codes.append([None] * n_codes)
            first = gens[0]

            def noted():
                for op in first:
                    if op[0] == "wait":
                        codes[0][int(op[1].name.split("]")[1])] = op[1]
                    yield op

            gens[scales], gens[0] = watched(), noted()
            assert not model.run(gens, seed)
        return seen

    assert ahead(True) and not ahead(False)
