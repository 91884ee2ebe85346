"""The life of a batch behind one prompt, for the tests of the plan: its whole pages stand in every row."""

PAGE, ROWS, COLS, N_PAGES, PREFIX = 16, 3, 8, 24, [5, 9, 2]
S = PAGE * len(PREFIX)  # tokens of the whole shared pages

# (held_len, ctx_len, new_len) of each step's requests, in tokens past S where >= 0; None: 0 tokens at all
STEPS = [
    ([0, 0, 0], [0, 0, 0], [20, 7, 1]),
    ([20, 7, 1], [20, 7, 1], [1, 16, 1]),
    ([21, 23, 2], [21, 9, 2], [1, 1, 40]),     # rejected drafts are dropped
    ([22, 10, 42], [0, 10, 0], [0, 1, 33]),    # the first ends, the last starts over
    ([0, 11, 33], [0, 11, 33], [5, 1, 1]),     # another request in the first row
    ([5, 12, 34], [0, 0, 0], [0, 0, 0]),       # all end
    ([0, None, None], [None] * 3, [None] * 3),  # the prefix is over: one row gives it back
    ([None] * 3, [None] * 3, [17, 3, None]),   # and all start again, without it
]


def tokens(step):
    held, ctx, new = step
    return [S + h if h is not None else 0 for h in held], [S + c if c is not None else 0 for c in ctx], [n or 0 for n in new]


def check(pages_of, stack, shared):
    """No page is held by two requests, or by one and the stack, but the prefix's by every row; none is lost."""
    own = [p for row in pages_of for p in row[len(PREFIX):]] if shared else [p for row in pages_of for p in row]
    every = own + list(stack) + (PREFIX if shared else [])
    assert sorted(every) == list(range(N_PAGES)), (pages_of, stack)
    if shared:
        assert all(row[:len(PREFIX)] == PREFIX for row in pages_of), pages_of
