"""What the key/value cache's binding refuses by itself (no GPU needed)."""

import pytest

torch = pytest.importorskip("torch")

import nvfp4_router_gate_gb300 as R  # noqa: E402
from test_abi_cpu import _lib  # noqa: E402


@pytest.mark.parametrize("nbytes,D", [(1200, 64), (1151, 64), (1152, 96), (1152, 128), (36864, 128), (0, 64)])
def test_pages_of_no_page_size_are_refused(nbytes, D):
    """A cache whose pages are larger than a page of its tokens would be walked with the wrong step."""
    _lib()
    cache, g = torch.zeros(2, 3, nbytes, dtype=torch.uint8), torch.ones(3)
    with pytest.raises(ValueError, match="page_size"):
        R.nvfp4_kv_gather(cache, torch.zeros(1, dtype=torch.int32), g, g, D)
    with pytest.raises(ValueError, match="page_size"):
        R.nvfp4_kv_append(None, torch.zeros(1, 3, D), torch.zeros(1, 3, D), None, torch.zeros(1, dtype=torch.int32),
                          None, None, cache, g, g)


def test_heads_that_do_not_share_the_kv_heads_are_refused():
    _lib()
    assert R.Nvfp4KVCache(2, 2, 64, page_size=16, n_heads=6, device="cpu").n_heads == 6
    with pytest.raises(ValueError, match="heads"):
        R.Nvfp4KVCache(2, 2, 64, page_size=16, n_heads=7, device="cpu")
