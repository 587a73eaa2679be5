"""Pages that a window has passed: not read, whatever their table entries name and whatever stands there."""
import math

import pytest
import torch

from chunk_util import make
from test_gpu_window import run_chunk_shared, run_chunk_window, run_tree_window, tree_problem, ts  # noqa: F401
from window_util import make_shared

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


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[9, 1], [1, 1], [90, 3]], ids=["few", "decoded", "chunks"])
def test_no_page_is_flagged_at_the_end_of_a_large_pool(ts, cuda_device, new, e4m3):  # noqa: F811
    """Pages whose offsets pass 32 bits, up to the pool's last; entries of the table that no row sees name none."""
    pages = 300_000 if e4m3 else 280_000
    p, go, sl = make_shared(cuda_device, [(64, [100, 31])], new, 16, 8, 128, "bf16", e4m3, seed=67)
    calls = lambda: (run_chunk_window(ts, p, 80, 3), run_chunk_shared(ts, p, go, sl))  # noqa: E731
    want = calls()
    small = p.k_pages.shape[0]
    p.page_table += pages - small
    for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
        old = getattr(p, name)
        if old is not None:
            big = torch.empty((pages,) + tuple(old.shape[1:]), dtype=old.dtype, device=cuda_device)
            (big[pages - small:].view(torch.uint8) if old.element_size() == 1 else big[pages - small:]).copy_(
                old.view(torch.uint8) if old.element_size() == 1 else old)
            setattr(p, name, big)
    for (got, status), (ref, _) in zip(calls(), want):
        assert status == 0 and torch.equal(got, ref)
