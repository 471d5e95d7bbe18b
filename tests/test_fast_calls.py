"""The binding's checked calls (binding/fast_calls.cpp): built, loaded with the
library, and refusing what is not theirs."""
import pytest
import torch

from mixture_experts_projections_b200 import rom

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def fast():
    from mixture_experts_projections_b200.build import build
    build()
    rom.load_library()
    assert rom._fast is not None
    return rom._fast


def test_refuses_cpu_tensors_and_other_objects(fast):
    x, w = torch.zeros(4, 64, dtype=BF16), torch.ones(64)
    assert fast.add_rmsnorm(x, None, w, 1e-5, None, x, None, None, None) is None
    assert fast.add_rmsnorm(None, None, w, 1e-5, None, x, None, None, None) is None
    assert fast.add_rmsnorm() is None and fast.quant_rows(1, 2, 3) is None
    assert fast.add_rmsnorm_bwd(*[x] * 9) is None and fast.quant_rows(x, x, w) is None
    assert fast.expert_proj_q8(*[x] * 12) is None and fast.expert_proj_w4(*[x] * 11) is None
    assert fast.expert_proj_q8(0, x, w, x, w, None, None, "1", None, None, None, x) is None


@gpu
def test_each_wrong_tensor_is_left_to_the_checks_that_name_it(fast):
    """One argument at a time is of another type, shape, layout or device: the
    call is not made."""
    c = "cuda"
    T, D, E, N, k = 8, 128, 2, 128, 1
    z = torch.zeros
    q = z(E, 8, 1, 2, 8, 4, 16, dtype=torch.uint8, device=c)
    calls = {
        fast.add_rmsnorm: [z(T, D, dtype=BF16, device=c), z(T, D, device=c), z(D, device=c), 1e-5, z(T, D, device=c),
                           z(T, D, dtype=BF16, device=c), z(T, D, dtype=E4M3, device=c), z(T, device=c), z(T, device=c)],
        fast.add_rmsnorm_bwd: [z(T, D, dtype=BF16, device=c), z(T, D, device=c), z(T, D, device=c), z(D, device=c), z(T, device=c),
                               z(T, D, dtype=BF16, device=c), z(T, D, device=c), z(D, device=c), z(T * D, device=c)],
        fast.quant_rows: [z(T, D, device=c), z(T, D, dtype=E4M3, device=c), z(T, device=c)],
        fast.expert_proj_q8: [rom.ROM_PROJ_OUT, z(T, D, dtype=E4M3, device=c), z(T, device=c), z(E, N, D, dtype=E4M3, device=c),
                              z(E, N, device=c), None, None, k, z(E + 1, dtype=torch.int32, device=c),
                              z(T, dtype=torch.int32, device=c), z(T, k, device=c), z(T, N, dtype=BF16, device=c)],
        fast.expert_proj_w4: [rom.ROM_PROJ_OUT, z(T, D, dtype=BF16, device=c), q, z(E, 8, 1, 16, 2, dtype=BF16, device=c), None, None,
                              N, k, z(T, k, dtype=torch.int32, device=c), z(T, k, device=c), z(T, N, dtype=BF16, device=c)],
    }
    for f, args in calls.items():
        assert f(*args) == rom.ROM_OK, f.__name__
        for i, a in enumerate(args):
            if not isinstance(a, torch.Tensor):
                continue
            wrong = [a.cpu(), a.to(torch.float64) if a.dtype != torch.uint8 else a.int(), 3]
            if not (f is fast.add_rmsnorm_bwd and i == 8):  # a workspace may have any shape and type
                wrong.append(a[:-1] if a.shape[0] > 1 else a[:0])
            else:
                wrong = [a.cpu(), 3]
            if a.dim() > 1:
                wrong.append(a.transpose(0, 1).contiguous().transpose(0, 1))
            for b in wrong:
                if torch.is_tensor(b) and b.is_cuda and b.dtype == a.dtype and b.shape == a.shape and b.is_contiguous():
                    continue  # a transposition that changes nothing
                assert f(*args[:i], b, *args[i + 1:]) is None, (f.__name__, i)
    torch.cuda.synchronize()
    assert rom.rom_get_status() == rom.ROM_OK


@gpu
def test_fast_and_python_checks_make_the_same_call(fast, monkeypatch):
    x = torch.randn(40, 256, generator=torch.Generator().manual_seed(0)).to(BF16).cuda()
    w = torch.ones(256, device="cuda")
    a = rom.add_rmsnorm(x, None, w, q8=True)
    monkeypatch.setattr(rom, "_fast", None)
    b = rom.add_rmsnorm(x, None, w, q8=True)
    assert torch.equal(a.y, b.y) and torch.equal(a.y8.view(torch.uint8), b.y8.view(torch.uint8))
