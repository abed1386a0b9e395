"""Calls of several host threads at once, each thread on its own stream: calls
whose kernels are the same and whose shared memory differs are all taken."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

CALLS, THREADS = 5000, 4


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    d.disco_device_status(clear=True)
    return d


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _together(lib, make):
    """CALLS calls of make(thread) -> (function, arguments but the stream), from each thread; their failures."""
    failed, start = [], threading.Barrier(THREADS)

    def work(k):
        s = torch.cuda.Stream()
        fn, args, _keep = make(k)
        args = (*args, ctypes.c_void_p(s.cuda_stream))
        torch.cuda.synchronize()
        start.wait()
        for _ in range(CALLS):
            if fn(*args) != 0:
                failed.append(lib.disco_last_error())
        s.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return failed


def test_gradient_of_rows_with_and_without_dh(lib):
    B, C = 1, 8000                                     # 64 KB of shared memory without dh, 96 with it
    so = lib.load_library()
    results = [None] * THREADS
    ins = [torch.randn((B, C, 1), generator=torch.Generator().manual_seed(k)).bfloat16().cuda() for k in range(4)]

    def make(k):
        dx = torch.empty_like(ins[0])
        results[k] = dx
        args = (_ptr(ins[0]), _ptr(ins[1]), None, _ptr(ins[2]) if k % 2 else None, ctypes.c_float(1e-5), _ptr(dx), None,
                B, C, 1, lib.DISCO_BF16, None, 0)
        return so.disco_rms_norm_bwd, args, dx

    failed = _together(lib, make)
    assert not failed, (len(failed), failed[0])
    for k in range(2):
        want = torch.empty_like(ins[0])
        lib.disco_rms_norm_bwd(ins[0], ins[1], None, ins[2] if k else None, 1e-5, want, None, B, C, 1)
        assert all(torch.equal(results[j], want) for j in range(k, THREADS, 2))


def test_norm_of_tiles_with_two_group_sizes(lib):
    B, C, P = 1, 128, 40000                            # 16-byte words of 512 threads: 64 KB, and the groups' maxima
    so = lib.load_library()
    results, groups = [None] * THREADS, (0, 16)
    x = torch.randn((B, C, P), generator=torch.Generator().manual_seed(9)).bfloat16().cuda()

    def outputs(group):
        return [torch.empty((B, C, P), dtype=torch.uint8, device="cuda"),
                torch.empty((B, C // group if group else 1, P), device="cuda")]

    def make(k):
        q, s = results[k] = outputs(groups[k % 2])
        args = (_ptr(x), None, None, ctypes.c_float(1e-5), None, None, _ptr(q), _ptr(s), groups[k % 2], B, C, P, lib.DISCO_BF16)
        return so.disco_rms_norm, args, (q, s)

    failed = _together(lib, make)
    assert not failed, (len(failed), failed[0])
    for k in range(2):
        q, s = outputs(groups[k])
        lib.disco_rms_norm(x, None, None, 1e-5, None, None, B, C, P, q=q, scale=s, group=groups[k])
        assert all(torch.equal(results[j][0], q) and torch.equal(results[j][1], s) for j in range(k, THREADS, 2))


def test_contractions_of_two_grids(lib):
    """Two threads, each waiting for its own call before the next."""
    C, grids = 128, [(9, 64, 1), (9, 128, 1)]           # table rows of the forward: 80 and 144 entries
    psis = [lib.Psi(g, g, 1, 3, 0.8) for g in grids]
    failed, start, results, ins = [], threading.Barrier(2), [None, None], []
    for k, (nlat, nlon, _) in enumerate(grids):
        ins.append(torch.randn((1, C, nlat, nlon), generator=torch.Generator().manual_seed(k)).bfloat16().cuda())

    def work(k):
        s, c = torch.cuda.Stream(), psis[k].c
        nlat, nlon, _ = grids[k]
        X = results[k] = torch.empty((1, C, c.K, nlat, nlon), dtype=torch.bfloat16, device="cuda")
        args = (ctypes.byref(c), _ptr(ins[k]), _ptr(X), 1, C, lib.DISCO_BF16, ctypes.c_void_p(s.cuda_stream))
        fn = lib.load_library().disco_fwd
        torch.cuda.synchronize()
        start.wait()
        for _ in range(CALLS):
            if fn(*args) != 0:
                failed.append(lib.disco_last_error())
            s.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, (len(failed), failed[0])
    for k in range(2):
        want = torch.empty_like(results[k])
        lib.disco_fwd(psis[k].c, ins[k], want, 1, C)
        assert torch.equal(results[k], want)
    assert lib.disco_device_status() == 0
