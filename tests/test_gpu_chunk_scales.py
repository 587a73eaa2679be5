"""Scales of an 8-bit cache and queries of extreme magnitudes, in every kernel that attends over windows and shared
prefixes."""
import pytest

from chunk_util import make
from test_gpu_window import check_chunk_shared, check_chunk_window, ts  # noqa: F401
from window_util import make_shared

pytestmark = pytest.mark.gpu
kernels = pytest.mark.parametrize("kernel", [0, 5, 1], ids=["auto", "units", "simt"])


@kernels
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 30, 2]], ids=["decoded", "chunks"])
def test_keys_of_zeros_score_zero_whatever_their_scale(ts, cuda_device, new, kernel):  # noqa: F811
    """q and K's scale are large enough that their product passes float32's range, and K's codes are zeros: every score is
    0 and every token that a row sees weighs the same."""
    p, go, sl = make_shared(cuda_device, [(128, [100, 30, 5])], new, 8, 2, 128, "bf16", True, seed=63)
    p.q.fill_(2.0 ** 100)
    for b, (S, n) in enumerate(zip(p.prefix, p.new)):
        for i in range((S + n + 15) // 16):
            page = int(p.page_table[b, i])
            p.k_pages.view(p.k_pages.dtype)[page] = 0
            p.k_scales[page] = 2.0 ** 50
    assert check_chunk_window(ts, p, 70, 3, kernel) == 0
    assert check_chunk_shared(ts, p, go, sl, kernel) == 0


@kernels
def test_scores_keep_their_ratio_at_both_ends_of_the_range(ts, cuda_device, kernel):  # noqa: F811
    """The same scores from large queries over small scales, and from small ones over large."""
    for up in (2.0 ** 90, 2.0 ** -90):
        p = make(cuda_device, [300, 77], [1, 1], 8, 2, 128, "bf16", True, seed=65)
        p.q *= up
        p.k_scales /= up
        assert check_chunk_window(ts, p, 130, 3, kernel) == 0
