"""A plan's C struct keeps what it points to, without the object it came from."""
import gc
import weakref

import pytest


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    return d


@pytest.mark.parametrize("in_place", [False, True])
def test_grad_plan_struct_keeps_its_list(lib, in_place):
    import torch
    grads = [torch.empty(0) for _ in range(3)]          # without elements: no device needed
    outs = grads if in_place else [torch.empty(0) for _ in range(3)]
    alive = [weakref.ref(t) for t in grads + outs]
    c = lib.GradPlan(grads, outs).c
    del grads, outs
    gc.collect()
    assert all(r() is not None for r in alive)
    assert c.count == 3 and [c.tensors[i].n for i in range(3)] == [0, 0, 0]
    c2, array = lib.disco_grad_plan([r() for r in alive], None)
    array = weakref.ref(array)
    gc.collect()
    assert array() is not None and c2.count == 6
    del c, c2
    gc.collect()
    assert array() is None and all(r() is None for r in alive)


@pytest.mark.gpu
def test_psi_struct_keeps_its_buffer(lib):
    grid = (9, 16, 1)
    psi = lib.Psi(grid, grid, 1, 3, 0.5)
    buffer, c = weakref.ref(psi.buffer), psi.c
    del psi
    gc.collect()
    assert buffer() is not None and buffer().data_ptr() <= c.row_ptr < buffer().data_ptr() + buffer().nbytes
    del c
    gc.collect()
    assert buffer() is None
