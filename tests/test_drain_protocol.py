"""The barriers of the tcgen05 products and attention gradient on host-side models (no GPU): copies that land late, and
how the kernels end: usual ends, waits that run out early and waits that run out after the producer has left, with
its last copies still on their way."""
import random

import pytest

import attn_protocol_model as A
import drain_protocol_model as M

WAYS = {"usual": dict(), "early": dict(timeout_p=0.02), "late": dict(timeout_p=0.3, late=True)}


def outcomes(run, trials, seed):
    rng = random.Random(seed)
    seen = {"ok": 0, "aborted": 0, "hazard": 0}
    for _ in range(trials):
        try:
            seen[run(rng)] += 1
        except M.Hazard:
            seen["hazard"] += 1
    return seen


@pytest.mark.parametrize("way", sorted(WAYS))
def test_products_end_with_nothing_in_flight(way):
    def run(rng):
        kblocks, stages = M.random_gemm(rng)
        return M.gemm(kblocks, stages, rng, **WAYS[way])
    seen = outcomes(run, 300, 1)
    assert seen["hazard"] == 0 and (seen["ok"] == 300) == (way == "usual"), seen


def test_products_that_are_held_run_into_the_limit():
    assert outcomes(lambda rng: M.gemm(*M.random_gemm(rng), rng, hold=True), 100, 2) == {"ok": 0, "aborted": 100, "hazard": 0}


def test_a_producer_that_asks_the_flag_leaves_copies_behind():
    """What the model is for: the flag is not up yet when the producer leaves, and the copies outlive the CTA."""
    run = lambda drain: outcomes(lambda rng: M.gemm(*M.random_gemm(rng), rng, drain=drain, **WAYS["late"]), 200, 3)
    assert run("flag")["hazard"] > 0 and run("never")["hazard"] > 0


PASSES = [(d, key) for d in (64, 128) for key in (False, True)]


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("d,key", PASSES)
def test_attention_gradient_reads_its_own_tiles(d, key, late):
    """Key and query passes, items without partners among them; late: copies land when nothing else can move, in any
    order, so that an earlier load of a slot may still be on its way when a later one is waited for."""
    assert outcomes(lambda rng: M.bwd_pass(d, key, M.random_items(rng), rng, late=late), 200, 4)["ok"] == 200


def test_waiting_for_the_tile_before_the_buffer_reads_another_tile():
    """Key pass at d = 128, five slots that X and Y share: a wait for Y of pair g passes on the parity of a phase two
    back while X of pair g - 2 is on its way, so the buffer's release (which implies that load) comes first."""
    run = lambda late: outcomes(lambda rng: M.bwd_pass(128, True, M.random_items(rng), rng, late=late, first="full"), 300, 4)
    assert run(False)["hazard"] > 0 and run(True)["hazard"] > 0



@pytest.mark.parametrize("way", sorted(WAYS))
@pytest.mark.parametrize("d,key", PASSES)
def test_attention_gradient_ends_with_nothing_in_flight(d, key, way):
    """Key and query passes, items without partners among them."""
    seen = outcomes(lambda rng: M.bwd_pass(d, key, M.random_items(rng), rng, **WAYS[way]), 120, 4)
    assert seen["hazard"] == 0 and (way != "usual" or seen["ok"] == 120) and (way == "usual" or seen["aborted"] > 0), seen


@pytest.mark.parametrize("d,key", PASSES)
def test_attention_gradient_that_is_held_runs_into_the_limit(d, key):
    seen = outcomes(lambda rng: M.bwd_pass(d, key, [1] + M.random_items(rng), rng, hold=True), 40, 5)
    assert seen == {"ok": 0, "aborted": 40, "hazard": 0}


@pytest.mark.parametrize("d,key", PASSES)
def test_an_attention_gradient_that_asks_the_flag_leaves_copies_behind(d, key):
    for drain, way in (("flag", "late"), ("never", "late"), ("never", "early")):
        run = lambda rng: M.bwd_pass(d, key, M.random_items(rng), rng, drain=drain, **WAYS[way])
        assert outcomes(run, 200, 6)["hazard"] > 0, (drain, way)


@pytest.mark.parametrize("d,key", [(128, False), (128, True)])
def test_draining_a_slot_used_again_waits_for_nothing(d, key):
    """The flag form's other fault: the parity of an earlier use of a slot, which does not come round again."""
    for seed in range(400):
        rng = random.Random(seed)
        try:
            M.bwd_pass(d, key, [8, 8], rng, drain="flag", timeout_p=0.02)
        except M.Hazard as e:
            if "waits for nothing" in str(e):
                return
    raise AssertionError("not met")


def attention(rng, fault=None):
    """The forward with copies that land when nothing else can move, and waits that run out meanwhile."""
    items = A.random_items(rng, allow_empty=True)
    try:
        r = A.run(items, rng, starve=("tmaK", "tmaV"), timeout_p=0.01, faults=(fault,) if fault else ())
    except A.Hazard as e:
        raise M.Hazard(str(e)) from None
    return r.split(":")[0]


def test_attention_ends_with_nothing_in_flight_when_a_role_gives_up_late():
    seen = outcomes(attention, 300, 7)
    assert seen["hazard"] == 0 and seen["aborted"] > 0, seen


def test_an_attention_that_asks_the_flag_leaves_copies_behind():
    assert outcomes(lambda rng: attention(rng, "tma_asks_flag"), 300, 8)["hazard"] > 0


@pytest.mark.parametrize("hold", [False, True])
@pytest.mark.parametrize("way", sorted(WAYS))
def test_pairs_of_ctas(way, hold):
    """Products on CTA pairs, an abort flag in each CTA."""
    def run(rng):
        kblocks, stages = M.random_gemm(rng)
        return M.gemm_pair(kblocks, rng, stages, hold=hold, **WAYS[way])
    seen = outcomes(run, 300, 9)
    assert seen["hazard"] == 0 and (seen["ok"] == 300) == (way == "usual" and not hold), seen
