"""How far a checkpoint's values may be off, as the header states it, on the tests' own description
of the format: half a step, and no more than 1/127.5 of the run's largest magnitude unless the step
is the smallest, 2^-126."""
import numpy as np

import act_reference as R


def test_half_a_step_and_its_share_of_the_largest_value():
    rng = np.random.default_rng(0)
    tops = np.concatenate([np.linspace(1, 2, 257)[:-1], [127.5 / 64, np.nextafter(127.5 / 64, 0)]])
    for e in (-100, -3, 0, 40, 120):
        top = np.ldexp(tops, e)[:, None]
        x = rng.uniform(-1, 1, (tops.size, 32)) * top
        x[:, 4] = top[:, 0]
        x[:, 8:24] = top / 128 * (np.arange(16) + 0.5)                # halves of a step, where it is top / 64
        _, p = R.quantise(x)
        off = np.abs(R.held(x) - x)
        assert (off <= np.ldexp(0.5, p)).all() and (off <= top / 127.5).all()
        assert (np.ldexp(63.75, p) <= top).all() and (top < np.ldexp(127.5, p)).all()


def test_a_largest_value_that_rounds_up_to_64_steps():
    """127.5 would round to 128, so the step doubles: 1 is half of it and goes to 0, 1/127.5 off."""
    x = np.zeros((1, 32))
    x[0, :3] = 127.5, 3, 1
    off = np.abs(R.held(x) - x).max()
    assert off == 1.0 and off > 127.5 / 128


def test_runs_below_the_smallest_step():
    """No step is below 2^-126: such a run keeps what is above half of that."""
    x = np.zeros((1, 32))
    x[0, :4] = np.ldexp([0.25, 0.5, 0.75, -1.25], -126)
    assert np.array_equal(R.held(x)[0, :4], np.ldexp([0.0, 0.0, 1.0, -1.0], -126))
