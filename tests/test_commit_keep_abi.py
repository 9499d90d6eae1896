"""Refusals of pa_commit_tree_keep: made on the host, before any CUDA call (no GPU)."""
import ctypes

import pytest

P = ctypes.c_void_p
NULL = P(0)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_04_gb300 import _build
    _build.ensure_built()
    import paged_kv_cache_04_gb300 as pa
    return pa.library()


def at(i, off=0):
    """An aligned address of its own; never dereferenced, as the calls fail on the host."""
    return P(0x10000000 * (i + 1) + off)


def commit(lib, **kw):
    k, v = (P * 2)(0x10000, 0x20000), (P * 2)(0x4000000, 0x8000000)
    a = dict(k=k, v=v, layers=2, bt=at(0), max_blocks=64, ctx=at(1), before=at(6), qs=at(2), mask=at(3), words=1,
             acc=at(4), out=at(5), S=2, N=16, G=8, d=128, B=16, layout=0, nb=1000, dt=2)
    a.update(kw)
    return lib.pa_commit_tree_keep(*a.values(), NULL)


@pytest.mark.parametrize("change,status", [
    (dict(S=0), 0), (dict(layers=0), 1), (dict(ctx=NULL), 1), (dict(out=NULL), 1), (dict(before=at(6, 2)), 1),
    (dict(out=at(6, 4)), 1), (dict(before=at(5, 4)), 1), (dict(out=at(1)), 1), (dict(before=at(1), out=at(1)), 1),
    (dict(words=5), 2), (dict(d=4), 2),
    # the old lengths' own array is no overlap, nor is none at all: what refuses these calls comes behind that check
    (dict(before=at(5), d=4), 2), (dict(before=NULL, d=4), 2),
])
def test_commit_tree_keep_refuses(lib, change, status):
    assert commit(lib, **change) == status


def test_binding_refuses(lib):
    import torch

    import paged_kv_cache_04_gb300 as pa
    z, c = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 8, 16, 64)
    with pytest.raises(pa.PAError):
        pa.pa_commit_tree([c], [c], z.view(2, 2), z[:2], z[:3], None, z[:2], z[:2], context_lens_before=3)
