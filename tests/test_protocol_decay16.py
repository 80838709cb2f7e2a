"""The fp16 form of the decayed linear-attention kernel's mbarrier protocol, checked on the
CPU under random schedules (tests/protocol_model_decay16.py), and planted mistakes."""

import pytest

import protocol_model_decay16 as pd


@pytest.mark.parametrize("nc", [0, 1, 2, 3, 4, 7])
def test_protocol_holds_under_random_schedules(nc):
    for seed in range(80):
        pd.run_schedule(nc, seed, pd.Variant16())
        pd.run_schedule(nc, seed, pd.Variant16(partial=nc - 1))
        pd.run_schedule(nc, seed, pd.Variant16(partial=0))
        pd.run_schedule(nc, seed, pd.Variant16(partial=nc - 1), in_order=True)


@pytest.mark.parametrize("nc", [1, 2, 3, 6])
def test_state_only_form_holds(nc):
    for seed in range(80):
        pd.run_schedule(nc, seed, pd.Variant16(state_only=True))
        pd.run_schedule(nc, seed, pd.Variant16(state_only=True, partial=nc - 1))


def caught(n=300, **kw):
    hits = 0
    for seed in range(n):
        try:
            pd.run_schedule(6, seed, pd.Variant16(**kw))
        except pd.ProtocolError:
            hits += 1
    return hits


@pytest.mark.parametrize("wait", ["af", "sv", "sm", "qsd", "od", "state_kvf", "s_free", "zf", "zh_free",
                                  "stage_free", "pf", "oe", "kve", "ssf", "zh", "sv_xf", "sv_yf"])
def test_waits_are_needed(wait):
    assert caught(skip=[wait]) > 0, wait


def test_fewer_slots_are_caught():
    assert caught(zd_slots=2) > 0
    assert caught(sd_slots=1) > 0
    assert caught(sx_slots=1) > 0
    assert caught(clear_ahead=1) > 0 and caught(clear_ahead=3) > 0
