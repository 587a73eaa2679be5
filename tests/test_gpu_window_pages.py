"""Pages that a window has passed: not read, whatever their table entries name and whatever stands there."""
import math

import pytest
import torch

from chunk_util import make
from test_gpu_window import run_chunk_window, run_tree_window, tree_problem, ts  # noqa: F401

pytestmark = pytest.mark.gpu
kernels = pytest.mark.parametrize("kernel", [5, 0, 1], ids=["units", "auto", "simt"])


def page_of(p, b, i):
    return int(p.page_table[b, i])


@kernels
@pytest.mark.parametrize("kind", ["chunk", "tree"])
def test_a_page_given_back_counts_for_no_row_that_is_not_finite(ts, cuda_device, kind, kernel):  # noqa: F811
    """Every row sees an infinity in one column of V, which spoils that column and nothing else.  The page before the
    window, in the window's first tile, now belongs to someone else who writes to it: no bit may depend on it."""
    prefix, n, window = 500, 40, 100                           # the window begins at token 401, its tile at 384
    if kind == "chunk":
        p = make(cuda_device, [prefix], [n], 8, 2, 128, "bf16", seed=61)
        run = lambda: run_chunk_window(ts, p, window, 0, kernel)  # noqa: E731
    else:
        p, q, parents = tree_problem(cuda_device, [prefix], [n], n, 8, 2, 128, "bf16", False, 61)
        run = lambda: run_tree_window(ts, p, q, parents, window, 0, kernel)  # noqa: E731
    p.v_pages[page_of(p, 0, prefix // 16), prefix % 16, :, 5] = math.inf   # the first new token: all rows see it
    outs = []
    for what in (0.0, math.nan, math.inf):
        p.k_pages[page_of(p, 0, 24)] = p.v_pages[page_of(p, 0, 24)] = what
        out, status = run()
        assert status == 0
        outs.append(out)
    others = [d for d in range(128) if d != 5]
    assert torch.isfinite(outs[0][..., others]).all() and not torch.isfinite(outs[0][..., 5]).any()
    assert all(torch.equal(out[..., others], outs[0][..., others]) for out in outs[1:])
