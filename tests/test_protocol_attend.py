"""The cache attention tile kernel's mbarrier protocol, checked on the CPU under
random schedules (tests/protocol_model_attend.py mirrors the kernel's roles); each
planted mistake is caught."""

import pytest

import protocol_model_attend as pa


@pytest.mark.parametrize("nt", [0, 1, 2, 3, 4, 7])
def test_protocol_holds_under_random_schedules(nt):
    for seed in range(120):
        pa.run_schedule(nt, seed)
        pa.run_schedule(nt, seed, pa.Variant(raises=(0, 1, nt - 1)))


@pytest.mark.parametrize("nt", [1, 2, 5])
def test_protocol_holds_in_issue_order(nt):
    for seed in range(20):
        pa.run_schedule(nt, seed, pa.Variant(raises=(1, 3)), in_order=True)


def caught(n=300, nt=6, **kw):
    hits = 0
    for seed in range(n):
        try:
            pa.run_schedule(nt, seed, pa.Variant(**kw))
        except pa.ProtocolError:
            hits += 1
    return hits


@pytest.mark.parametrize("wait", ["kf", "s_free", "qf", "pf", "vf", "k_free", "v_free", "sf", "last_od"])
def test_waits_are_needed(wait):
    assert caught(skip=[wait]) > 0, wait


def test_moving_a_reference_waits_for_the_last_product():
    assert caught(skip=["raise_od"], raises=(3,)) > 0


def test_mistakes_are_caught():
    assert caught(one_pf=True) > 0
    assert caught(two_ks=True) > 0
