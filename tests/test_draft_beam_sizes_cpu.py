"""Sizes whose products pass 64 bits are refused before any launch (no GPU
needed; the addresses are never read)."""
import pytest

pytest.importorskip("torch")

from test_attn_abi_cpu import P  # noqa: E402


@pytest.mark.parametrize("groups,beams,pages,page", [
    (1 << 62, 4, 3, 16), (1 << 58, 64, 3, 16), (1 << 61, 8, 0, 1), (2, 16, 1 << 60, 16), (2, 64, 1 << 58, 64), (1, 1, 1 << 62, 65536),
    ((1 << 62) + 1, 4, 3, 16)])
def test_beam_pages(lq, groups, beams, pages, page):
    assert lq.lib().lq_beam_pages(P, groups, beams, P, pages, P, page, 2 * P, P, 0) == lq.LQ_ERR_UNSUPPORTED
