"""A commit whose new lengths would overwrite what other CTAs of the row still read is refused
before anything is launched."""
import numpy as np
import pytest
import torch

from packed_cache_decode_b200 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("use_pages", [False, True])
@pytest.mark.parametrize("which", ["path", "path_end", "count", "nodes", "lens", "overlap"])
def test_new_lengths_may_not_overlap_inputs(which, use_pages):
    lay = B.Layout(np.full(64, 2), 2, 0).upload(0)
    b, n, h_kv, cap = 2, 4, 2, 64
    ints = torch.full((64,), 2, dtype=torch.int32, device="cuda")
    path, count, nodes, lens, spare = ints[:8].view(b, n), ints[8:10], ints[10:12], ints[12:14], ints[20:22]
    new = {"path": ints[0:2], "path_end": ints[7:9], "count": count, "nodes": nodes, "lens": lens, "overlap": ints[9:11]}[which]
    if use_pages:
        pool = torch.full((lay.tile_bytes * h_kv * b,), 3, dtype=torch.uint8, device="cuda")
        pages = B.PagedCache(pool, torch.arange(b, dtype=torch.int32, device="cuda").view(b, 1))
        call = lambda new: B.tree_commit_paged(lay, path, count, n, pages, lens, new, h_kv, n_nodes=nodes)  # noqa: E731
    else:
        pool = torch.full((lay.cache_bytes(b, h_kv, cap),), 3, dtype=torch.uint8, device="cuda")
        call = lambda new: B.tree_commit(lay, path, count, n, pool, lens, new, cap, h_kv, n_nodes=nodes)  # noqa: E731
    with pytest.raises(B.BgtqError):
        call(new)
    torch.cuda.synchronize()
    assert (ints == 2).all() and (pool == 3).all() and lay.status() == 0
    path.zero_()                                   # (nodes 0 and 0 of 2: the row keeps its first node twice)
    call(spare)
    assert lay.status() == 0 and (spare == 2).all()
