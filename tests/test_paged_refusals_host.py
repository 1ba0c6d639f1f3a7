"""More refusals of the paged cache's entry points, before anything touches a device."""
import pytest

from exact_io_aware_32_gb300 import build, fa

A = 1 << 30  # fake addresses, aligned and far apart; never dereferenced because validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


def plan(**args):
    kw = dict(R=4, page_size=16, n_free=8, max_pages=9, T=4)
    kw.update((n, (2 + i) * A) for i, n in enumerate(("ctx_lens", "new_lens", "free_pages", "free_head", "block_table",
                                                      "query_start", "seq_lens", "slots", "pages_taken")))
    kw.update(args)
    return fa.fa_paged_plan(**kw, stream=0)


@pytest.mark.parametrize("R", [2 ** 30 + 1, 2 ** 31 - 256, 2 ** 31 - 1])
def test_plan_refuses_more_requests_than_it_counts(R):
    """Places of requests, a few hundred past the last one, must fit 32 bits."""
    assert plan(R=R) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("args", [
    dict(seq_lens=2 * A),               # the lengths advanced in place
    dict(seq_lens=3 * A),
    dict(query_start=2 * A + 12),       # R + 1 entries: the last of ctx_lens
    dict(query_start=2 * A - 16),       # and from below
    dict(pages_taken=5 * A),            # the free list's head counted up in place
    dict(pages_taken=4 * A + 28),       # its last entry
    dict(slots=4 * A + 28),
    dict(block_table=4 * A),
    dict(block_table=2 * A - 4 * 4 * 9 + 4),
    dict(slots=7 * A, query_start=7 * A),
    dict(pages_taken=6 * A + 4 * 4 * 9 - 4),
])
def test_plan_refuses_outputs_that_are_read_or_written_elsewhere(args):
    assert plan(**args) == fa.FA_ERR_INVALID_ARG


def test_plan_takes_neighbours_and_inputs_that_are_one():
    """Arrays side by side, an empty free list, one array as both lengths: not refused. (Without a GPU the call then stops
    at the device; it is not made where there is one, since the addresses are not real.)"""
    import torch

    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not real")
    for args in (dict(), dict(new_lens=2 * A), dict(query_start=2 * A + 16), dict(query_start=2 * A - 20),
                 dict(pages_taken=4 * A + 32), dict(n_free=0, free_pages=10 * A), dict(free_head=None, pages_taken=5 * A)):
        assert plan(**args) == fa.FA_ERR_LAUNCH, args
