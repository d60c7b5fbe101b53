"""The barrier protocol of the feed-forward block's tensor-core kernels, on a model (rows_protocol): right
data under any schedule, an end and a report when a wait runs out."""
import random

import pytest

import rows_protocol as Q


def test_any_schedule_gives_right_data():
    R = random.Random(1)
    for seed in range(600):
        assert not Q.Cta(Q.random_plan(R), seed).run()


def test_late_copies_end_and_are_reported():
    """One copy or product, any of them, is later than waits last: the CTA ends with nothing in
    flight, and reports it unless every result is right."""
    R = random.Random(2)
    reported = 0
    for seed in range(600):
        plan = Q.random_plan(R)
        things = Q.Cta(plan, seed)
        things.run()
        late = (R.randrange(things.started),
                R.choice([Q.LIMIT + R.randint(-200, 2000),
                          R.randint(Q.LIMIT // 2, Q.LIMIT * 9 // 5)]))
        reported += Q.Cta(plan, seed, late).run()
    assert reported > 300


@pytest.mark.parametrize("mistakes", [("meet", "silent"), ("apart",), ("silent",), ("go on",),
                                      ("trust",), ("count skipped",)], ids="-".join)
def test_planted_mistakes_are_seen(mistakes):
    R = random.Random(3)
    for seed in range(4000):
        plan = Q.random_plan(R)
        first = Q.Cta(plan, seed)
        first.run()
        late = (R.randrange(first.started), Q.LIMIT + R.randint(-200, 2000))
        try:
            Q.Cta(plan, seed, late, mistakes).run()
        except (Q.Hang, Q.Wrong):
            return
    pytest.fail(f"the model does not see {mistakes}")
