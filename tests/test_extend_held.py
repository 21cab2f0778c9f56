"""Sequence extension with held pages: the refusals, and the plain form at cases worked by hand
(no GPU)."""
import pytest

from tests import loop_ref as R
from tests.held_ref import Held

FAKE = 0x10000


def test_extend_held_refuses(lib):
    names = (("bt", FAKE), ("mb", 8), ("sl", FAKE), ("nl", FAKE + 64), ("held", FAKE + 128),
             ("free", FAKE), ("cap", 64), ("count", FAKE), ("B", 2), ("T", 5), ("nb", 64),
             ("window", 0), ("sinks", 0), ("qsl", FAKE), ("slots", FAKE), ("pos", FAKE),
             ("ol", FAKE), ("oc", FAKE), ("s", None))

    def f(**kw):
        return lib.ps_extend_held_sequences(*[kw.get(n, d) for n, d in names])

    assert f(held=None) == -1
    for same in ("sl", "nl", "ol"):  # the pages are written while the lengths are read
        assert f(**{same: FAKE + 4096, "held": FAKE + 4096}) == -1
    assert f(ol=2 * FAKE, nl=2 * FAKE) == -1
    assert f(B=-1) == -1 and f(T=-1) == -1 and f(mb=0) == -1 and f(cap=-1) == -1
    assert f(nb=0) == -1 and f(nb=1 << 28) == -1 and f(window=-1) == -1 and f(sinks=-1) == -1
    assert f(B=8193) == -2 and f(B=8192, mb=1 << 18) == -2 and f(T=2 ** 31 - 1) == -2
    for name in ("bt", "sl", "nl", "free", "count", "qsl", "slots", "pos", "ol", "oc"):
        assert f(**{name: None}) == -1


def test_a_page_of_rejected_tokens_is_kept():
    """15 tokens and 5 drafts take a second page; one draft stays, and the page with it."""
    c = Held([15], 4, 3, 4)
    offsets, slots, positions, errors = c.step([5], 5)
    assert (offsets, positions, errors) == ([0, 5], [15, 16, 17, 18, 19], set())
    second = c.tables[0][1]
    c.shorten([4])
    offsets, slots, _, _ = c.step([3], 4)
    assert c.tables[0][1] == second and slots == [16 * second + i for i in range(3)] + [-1]
    assert c.held == [2] and c.lens == [19]
    c.check_blocks()
    c.step([-1], 0)
    assert sorted(c.stack) == [0, 1, 2, 3] and c.held == [0]


def test_without_held_pages_it_is_lost():
    """The same by lengths alone, as the header says of them."""
    bt, lens, stack, count = [[3, -1, -1, -1]], [15], [0, 1, 2, -1], 3
    bt, lens, stack, count, *_ = R.extend(bt, lens, [5], stack, count, 5, 4)
    bt, lens, stack, count, *_ = R.extend(bt, [16], [3], stack, count, 3, 4)
    assert len([e for e in bt[0] if e >= 0] + stack[:count]) == 3  # of four


@pytest.mark.parametrize("seed", range(3))
def test_both_forms_agree_where_lengths_only_grow(seed):
    import random
    r = random.Random(seed)
    lens = [r.randint(0, 60) for _ in range(6)]
    c = Held(lens, 12, 20, 50)
    bt, count = [list(t) for t in c.tables], len(c.stack)
    stack = c.stack + [-1] * 60
    for _ in range(25):
        news = [r.choice([-1, 0, 1, 1, 2, 20]) for _ in lens]
        T, window, sinks = r.randint(0, 40), r.choice([0, 20]), r.randint(0, 20)
        bt, lens, stack, count, *rest = R.extend(bt, lens, news, stack, count, T, c.nb, window,
                                                 sinks)
        offsets, slots, positions, errors = c.step(news, T, window, sinks)
        assert rest == [offsets, slots, positions, errors]
        assert (c.lens, c.tables, c.stack) == (lens, bt, stack[:count])
        c.check_blocks()
