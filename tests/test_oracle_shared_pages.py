"""Pages that several rows name, and the plan, which does not know of them, in the oracle."""

from oracle import serving as S
from tests import shared_pages as P


def plan(table, stack, held, ctx, new):
    out = S.cache_plan(P.PAGE, table, stack + [-1] * (P.N_PAGES - len(stack)), len(stack), held, ctx, new, P.N_PAGES, 100)
    assert out["status"] == 0
    return out["table"], out["stack"], out["used"]


def start():
    return [P.PREFIX + [-1] * (P.COLS - len(P.PREFIX)) for _ in range(P.ROWS)], [p for p in range(P.N_PAGES) if p not in P.PREFIX]


def test_requests_that_end_at_the_shared_pages_lose_none():
    table, stack = start()
    for n, step in enumerate(P.STEPS):
        table, stack, used = plan(table, stack, *P.tokens(step))
        P.check([row[:u] for row, u in zip(table, used)], stack, shared=n < 6)


def test_dropping_shared_pages_gives_them_away_while_others_use_them():
    """What the header warns of."""
    table, stack = start()
    table, stack, _ = plan(table, stack, [P.S] * 3, [P.S] * 3, [0, 0, 70])
    _, stack, _ = plan(table, stack, [P.S, P.S, P.S + 70], [0, 0, P.S + 70], [0, 0, 0])
    assert [stack.count(p) for p in P.PREFIX] == [2, 2, 2]
