"""The workspace of the whole-vocabulary log probabilities (host logic, CPU only): a call of more than 8192
rows is several launches over one workspace, the last of them with a plan of its own.  So the size given out
has to hold every launch of the call, whatever the GPU's SM count, and the launches of a shorter call too."""
import itertools
import random

import pytest

from shared_prefix_question_gb300 import blink, build

SMS = (2, 3, 76, 108, 132, 141, 142, 146, 148, 150, 152, 154, 158, 160, 170, 300, 400)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return blink.lib()


def plan(n, H, V, top, sms):
    return blink.blink_token_logprobs_workspace_plan(n, H, V, top, sms)


def test_every_launch_fits(lib):
    rng = random.Random(1)
    rows = [1, 128, 129, 256, 257, 512, 513, 8191, 8192, 8193, 8192 + 7936, 9000, 16384, 16385, 131072]
    rows += [rng.randint(1, 131072) for _ in range(60)]
    for sms, n, (H, V, top) in itertools.product(SMS, rows, ((8, 20000, 32), (8, 1000, 1), (152, 151936, 32),
                                                             (2560, 151936, 20), (64, 5, 0), (64, 257, 5))):
        given, used = plan(n, H, V, top, sms)
        assert used <= given, (n, H, V, top, sms, used - given)


def test_a_longer_calls_workspace_serves_shorter_ones(lib):
    for sms, (H, V, top) in itertools.product(SMS, ((8, 20000, 32), (2560, 151936, 20), (64, 700, 3), (64, 40000, 0))):
        last = 0
        for n in (*range(1, 1400, 9), 512, 513, *range(1400, 8193, 97), 8192, 8193, 16128, 100000):
            size = plan(n, H, V, top, sms)[0]
            if n > 1 and n not in (512, 513):
                assert size >= last, (n, H, V, top, sms)
                last = size
        assert plan(512, H, V, top, sms)[0] <= plan(513, H, V, top, sms)[0]


def test_the_query_is_bounded_by_rows_and_alternatives(lib):
    """A launch has at most 8192 rows: 16 KB per unit of H of gathered rows, the rest does not depend on H."""
    base = plan(8192, 8, 151936, 32, 152)[0] - 16384 * 8
    for n, H in ((8192, 2560), (131072, 5120), (131072, 32768)):
        assert plan(n, H, 151936, 32, 152)[0] <= base + 16384 * H
    assert base <= 90 << 20


def test_refusals(lib):
    for bad in ((0, 8, 9, 0, 152), (131073, 8, 9, 0, 152), (1, 0, 9, 0, 152), (1, 8, 0, 0, 152), (1, 8, 9, 33, 152),
                (1, 8, 9, -1, 152), (1, 8, 9, 0, 1)):
        with pytest.raises(blink.BlinkError):
            plan(*bad)
    assert lib.blink_token_logprobs_workspace_plan(1, 8, 9, 0, 152, None, None) == blink.BLINK_INVALID_ARG
