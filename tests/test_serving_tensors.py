"""Tensors that the tree, commit, mass and eviction calls cannot take as they are (row counts
spaced apart or repeated, the wrong type or length, host memory) are refused before the library
is called."""
import numpy as np
import pytest
import torch

from packed_cache_decode_b200 import binding as B

N, B_ROWS, H_Q, H_KV = 4, 2, 8, 2


class OnGpu(torch.Tensor):
    """A host tensor that says it is on the GPU (nothing is launched here)."""
    is_cuda = True


def gpu(t):
    return t.as_subclass(OnGpu)


def ints(n=B_ROWS):
    return gpu(torch.ones(n, dtype=torch.int32))


BAD_ROWS = {
    "strided": lambda: gpu(torch.ones(2 * B_ROWS, dtype=torch.int32)[::2]),
    "repeated": lambda: gpu(torch.ones(1, dtype=torch.int32).expand(B_ROWS)),
    "int64": lambda: gpu(torch.ones(B_ROWS, dtype=torch.int64)),
    "short": lambda: ints(B_ROWS - 1),
    "host": lambda: torch.ones(B_ROWS, dtype=torch.int32),
}


class Refused(Exception):
    pass


@pytest.fixture
def layout(monkeypatch):
    """A layout of the real library; a call that got as far as the library raises Refused."""
    lay = B.Layout(np.full(64, 2), 2, 0)

    def check(status, what):
        if status:
            raise Refused(what)

    monkeypatch.setattr(B, "_check", check)
    monkeypatch.setattr(B, "_raw_stream", lambda stream: 0)
    return lay


def calls(lay):
    """name -> (call, its tensors by name); the tensors as given are taken (the library then says
    that the layout is not on a device)."""
    f = lambda *shape: gpu(torch.zeros(*shape))  # noqa: E731
    cache = gpu(torch.zeros(16, dtype=torch.uint8))
    pages = B.PagedCache(gpu(torch.zeros(16, dtype=torch.uint8)), gpu(torch.zeros(B_ROWS, 1, dtype=torch.int32)))
    tree = {"q": f(B_ROWS, N, H_Q, 128), "mask": gpu(torch.ones(B_ROWS, N, dtype=torch.int64)), "lens": ints(), "nodes": ints(),
            "out": f(B_ROWS, N, H_Q, 128)}
    commit = {"path": gpu(torch.zeros(B_ROWS, N, dtype=torch.int32)), "count": ints(), "lens": ints(), "new": ints(), "nodes": ints()}
    mass = {"q": f(B_ROWS, H_Q, 128), "lens": ints(), "mass": f(B_ROWS, H_KV, 64), "out": f(B_ROWS, H_Q, 128)}
    evict = {"lens": ints(), "mass": f(B_ROWS, H_KV, 64), "mass_out": f(B_ROWS, H_KV, 8),
             "kept": gpu(torch.zeros(B_ROWS, H_KV, 8, dtype=torch.int32)), "new": ints()}
    return {
        "tree": (lambda q, mask, lens, nodes, out: B.tree_attention(lay, q, mask, cache, lens, 64, 64, out, cache, H_KV, nodes), tree),
        "tree_paged": (lambda q, mask, lens, nodes, out: B.tree_attention_paged(lay, q, mask, pages, lens, 64, out, cache, H_KV,
                                                                                nodes), tree),
        "commit": (lambda path, count, lens, new, nodes: B.tree_commit(lay, path, count, N, cache, lens, new, 64, H_KV, nodes), commit),
        "commit_paged": (lambda path, count, lens, new, nodes: B.tree_commit_paged(lay, path, count, N, pages, lens, new, H_KV, nodes),
                         commit),
        "mass": (lambda q, lens, mass, out: B.decode_attention_mass(lay, q, cache, lens, 64, 64, mass, out, cache, H_KV), mass),
        "mass_paged": (lambda q, lens, mass, out: B.decode_attention_mass_paged(lay, q, pages, lens, 64, mass, out, cache, H_KV), mass),
        "evict": (lambda lens, mass, mass_out, kept, new: B.cache_evict(lay, cache, lens, 64, 64, mass, 8, 1, 1, cache, 64, mass_out,
                                                                         kept, new, H_KV), evict),
        "evict_paged": (lambda lens, mass, mass_out, kept, new: B.cache_evict_paged(lay, pages, lens, 64, mass, 8, 1, 1, pages, mass_out,
                                                                                     kept, new, H_KV), evict),
    }


NAMES = ["tree", "tree_paged", "commit", "commit_paged", "mass", "mass_paged", "evict", "evict_paged"]


@pytest.mark.parametrize("name", NAMES)
def test_good_tensors_reach_the_library(layout, name):
    call, tensors = calls(layout)[name]
    with pytest.raises(Refused):
        call(**tensors)


@pytest.mark.parametrize("kind", list(BAD_ROWS))
@pytest.mark.parametrize("name", NAMES)
def test_row_counts_are_checked(layout, name, kind):
    call, tensors = calls(layout)[name]
    for which in ("lens", "nodes", "count", "new"):
        if which in tensors:
            with pytest.raises(AssertionError):
                call(**{**tensors, which: BAD_ROWS[kind]()})


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors_are_refused(layout, name):
    call, tensors = calls(layout)[name]
    for which, t in tensors.items():
        with pytest.raises(AssertionError):
            call(**{**tensors, which: t.as_subclass(torch.Tensor)})
