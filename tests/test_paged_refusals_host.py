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
