"""The decayed linear-attention kernel's mbarrier protocol, checked on the CPU under
random schedules (tests/protocol_model_decay.py mirrors the kernel's roles): every
barrier test in the phase it is for or the next, every arrival in its phase, every
read of the version it needs, no deadlock; and each planted mistake is caught."""

import pytest

import protocol_model_decay as pd


@pytest.mark.parametrize("own_o", [False, True])
@pytest.mark.parametrize("nc", [1, 2, 3, 4, 7])
def test_protocol_holds_under_random_schedules(nc, own_o):
    for seed in range(80):
        pd.run_schedule(nc, seed, pd.Variant(own_o=own_o))
        # a step that is not full: the last forwards, the first backwards
        pd.run_schedule(nc, seed, pd.Variant(own_o=own_o, partial=nc - 1))
        pd.run_schedule(nc, seed, pd.Variant(own_o=own_o, partial=0))


@pytest.mark.parametrize("nc", [1, 2, 3, 6])
def test_state_only_form_holds(nc):
    for seed in range(80):
        pd.run_schedule(nc, seed, pd.Variant(state_only=True))
        pd.run_schedule(nc, seed, pd.Variant(state_only=True, partial=nc - 1))


@pytest.mark.parametrize("own_o", [False, True])
@pytest.mark.parametrize("nc", [1, 2, 5])
def test_protocol_holds_in_issue_order(nc, own_o):
    for seed in range(20):
        pd.run_schedule(nc, seed, pd.Variant(own_o=own_o, partial=nc - 1), in_order=True)


def caught(n=300, **kw):
    hits = 0
    for seed in range(n):
        try:
            pd.run_schedule(6, seed, pd.Variant(**kw))
        except pd.ProtocolError:
            hits += 1
    return hits


@pytest.mark.parametrize("wait", ["y_free", "x_free", "z_free", "xf", "zh", "kve", "ssf", "oe", "pf", "ow",
                                  "af", "qsd", "od", "state_kvf", "s_free", "zf", "zh_free"])
def test_waits_are_needed(wait):
    """Each wait of the kernel, left out, is caught."""
    assert caught(skip=[wait]) > 0, wait


def test_waits_of_single_cases_are_needed():
    assert caught(skip=["stage_free"], own_o=True) > 0
    assert caught(skip=["a_cleared"], partial=5) > 0
    assert caught(skip=["zh_yf"], partial=0) > 0
    assert caught(skip=["yf"], state_only=True) > 0


def test_one_wait_is_implied():
    """A of a step waits for the P Z of two steps back that read the same buffer; the
    X S issued before it has waited for that product's output to be read.  The wait
    stays as a guard against a reordering."""
    assert caught(n=150, skip=["a_free"]) == 0


def test_one_completion_barrier_for_both_stages_is_caught():
    """The producer waits for a product two steps back while the last one may have
    completed too: with one barrier that wait would never end.  The same for the
    store thread, which rows may outrun by two steps."""
    assert caught(one_kvf=True) > 0
    assert caught(one_ow=True) > 0
