"""Sizes whose products pass 64 bits, and scores that are written before they are
read, are refused before any launch (no GPU
needed; the addresses are never read)."""
import pytest

pytest.importorskip("torch")

from test_attn_abi_cpu import P  # noqa: E402


@pytest.mark.parametrize("groups,beams,pages,page", [
    (1 << 62, 4, 3, 16), (1 << 58, 64, 3, 16), (1 << 61, 8, 0, 1), (2, 16, 1 << 60, 16), (2, 64, 1 << 58, 64), (1, 1, 1 << 62, 65536),
    ((1 << 62) + 1, 4, 3, 16)])
def test_beam_pages(lq, groups, beams, pages, page):
    assert lq.lib().lq_beam_pages(P, groups, beams, P, pages, P, page, 2 * P, P, 0) == lq.LQ_ERR_UNSUPPORTED


def test_scores_that_would_be_written_before_they_are_read(lq):
    """Results in the place of other groups' scores: as many as beams, in their own
    place, or none."""
    def select(s, a, groups, beams, k):
        return lq.lib().lq_beam_select(16 * P, 100, s, groups, beams, 100, k, 0, 0, a, 32 * P, 64 * P, 128 * P, 0)

    for s, a, groups, beams, k in ((P, P, 4, 4, 3), (P, P, 4, 4, 8), (P, P + 4, 4, 4, 4), (P + 4, P, 4, 4, 4), (P, P + 60, 4, 4, 1), (P + 28, P, 4, 4, 2)):
        assert select(s, a, groups, beams, k) == lq.LQ_ERR_INVALID_ARG, (s, a, groups, beams, k)
