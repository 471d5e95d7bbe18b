"""Calls from several host threads, and what they hold meanwhile."""
import ctypes
import threading

import pytest
import torch

from mixture_experts_projections_b200 import rom

BF16 = torch.bfloat16
gpu = pytest.mark.gpu


@gpu
def test_norm_gradients_of_two_widths_from_two_threads():
    """A launch's shared memory may not depend on what another thread's launch
    of another width asked for in between. (The C calls with prepared arguments:
    they release the interpreter lock and take longer than what Python does
    between them, so that the two threads' calls do overlap.)"""
    lib, T, results = rom.load_library(), 3, {}
    code, null = rom.ROM_BF16, None
    runs = {}
    for D in (8200, 16384):
        g = torch.Generator().manual_seed(D)
        dy, s = (torch.randn(T, D, generator=g).to(BF16).cuda() for _ in range(2))
        w, rstd = torch.ones(D, device="cuda"), torch.ones(T, device="cuda")
        dx, ref, st = torch.zeros_like(dy), torch.empty_like(dy), torch.cuda.Stream()
        rom.rom_add_rmsnorm_bwd(dy, None, s, w, rstd, ref, None, None, None)
        p = [ctypes.c_void_p(t.data_ptr()) for t in (dy, s, w, rstd, dx)]
        call = (p[0], code, null, p[1], code, T, D, p[2], p[3], p[4], null, null, null, 0,
                ctypes.c_void_p(st.cuda_stream))
        runs[D] = call, st, dx, ref, (dy, s, w, rstd)
    torch.cuda.synchronize()
    go = threading.Barrier(len(runs))

    def work(D):
        call, f = runs[D][0], lib.rom_add_rmsnorm_bwd
        go.wait(60)
        results[D] = {f(*call) for _ in range(20000)}

    threads = [threading.Thread(target=work, args=(D,)) for D in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert results == {D: {rom.ROM_OK} for D in runs}
    assert all(torch.equal(dx, ref) for _, _, dx, ref, _ in runs.values())


@gpu
def test_checked_calls_release_the_interpreter_lock():
    """A launch may block (a full queue) until a host function ran that needs the
    lock. PyGILState_Check stands in for the library's function: its status says
    whether the caller holds the lock."""
    lib = rom.load_library()
    if rom._fast is None:
        pytest.skip("the checked calls are not built")
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    x = torch.zeros(4, 64, device="cuda")
    q, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(4, device="cuda")
    try:
        rom._fast.bind(*[held] * 5)
        assert rom._fast.quant_rows(x, q, s) == 0
    finally:
        rom._load_fast_calls(lib)
    assert rom._fast.quant_rows(x, q, s) == 0
