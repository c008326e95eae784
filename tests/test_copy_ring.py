"""What the kernels' rings of copies do once a wait has run out, on a model of the barriers (no GPU)."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "microscaling_fp4_quantization_mxfp4_b200", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("copy_ring") / "copy_ring.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, os.path.join(HERE, "host", "copy_ring.cpp"),
                    "-o", out], check=True)
    return ctypes.CDLL(out)


@pytest.mark.parametrize("rows_at_once", [1, 2])
def test_a_late_reader_asks_for_no_more(model, rows_at_once):
    """No second arrival in an open phase, no copy into a slot with one in flight, none in flight at the end."""
    caught = 0
    for slots in (2, 3, 4, 8, 16):
        if rows_at_once == 2 and slots < 8:
            continue
        for count in (1, 2, 3, 7, 16, 17, 40, 41):
            for stuck in range(count + 1):
                for lag in (1, 3, 1000):
                    case = (slots, count, rows_at_once, stuck, lag)
                    assert model.ring_faults(*case, 0) == 0, case
                    caught += model.ring_faults(*case, 1) > 0
    assert caught                                       # the model sees the faults of a reader that goes on asking


def test_a_pair_that_stops_waits_for_what_either_asked_for(model):
    """Whatever each CTA of an SM pair has asked for, and whatever of it is in flight: all of it has landed at the end."""
    for slots in (2, 3, 4, 7):
        for done in (0, 1, slots, 2 * slots + 1):
            for mine in range(done, done + slots + 1):
                for peers in range(done, done + slots + 1):
                    masks = range(1 << slots) if slots < 5 else (0, 1, 5, 64, 85, 127)
                    for own in masks:
                        for peer in masks:
                            case = (slots, done, mine, peers, own, peer)
                            assert model.pair_faults(*case) == 0, case


def test_a_producer_counts_the_copies_it_asked_for(model):
    """One count too many, from before the wait that ran out, looks for a phase that never opens and misses the slot's own."""
    for slots in (2, 4, 7):
        for asked in range(1, 5 * slots):
            assert model.copies_missed(slots, asked, asked) == 0
            if asked >= slots:
                assert model.copies_missed(slots, asked, asked + 1) == 1
