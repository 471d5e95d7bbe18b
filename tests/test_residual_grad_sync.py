"""Data-parallel training of a pre-norm block: which tensors
residual_block_backward(grad_sync=...) exchanges between the ranks, when and in
which order. Two gloo ranks on CPU, stand-ins for the kernels."""
import contextlib
import os
import socket
import sys

import torch
import torch.multiprocessing as mp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, DM, DE, E, K = 6, 64, 256, 2, 2


def _rank_main(rank, world, port):
    import torch.distributed as dist

    sys.path.insert(0, ROOT)
    from mixture_experts_projections_b200 import rom

    log = []
    value = lambda n: float((rank + 1) * n)  # noqa: E731

    def kernel(name, outputs):
        """A stand-in that writes (rank + 1) * n into argument i, for each i: n."""
        def run(*args, **kw):
            log.append(name)
            for i, n in outputs.items():
                if args[i] is not None:
                    args[i].fill_(value(n))
        return run

    for name, outputs in (("rom_bwd_gather", {4: 1}), ("rom_bwd_dgrad_out", {6: 1}), ("rom_bwd_gate", {6: 1}),
                          ("rom_bwd_dgrad_in", {6: 1}), ("rom_route_probs", {3: 1}), ("rom_route_bwd", {10: 1, 11: 2}),
                          ("rom_route_wgrad", {2: 5, 3: 7}), ("rom_bwd_wgrad", {5: 11, 6: 13}),
                          ("rom_add_rmsnorm_bwd", {5: 17, 7: 19})):
        assert hasattr(rom, name)
        setattr(rom, name, kernel(name, outputs))
    rom._scope = lambda t, stream: contextlib.nullcontext()

    os.environ["MASTER_ADDR"], os.environ["MASTER_PORT"] = "127.0.0.1", str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        exchanged, real = [], dist.all_reduce

        def all_reduce(t, **kw):
            log.append("all_reduce")
            exchanged.append(t)
            return real(t, **kw)

        dist.all_reduce = all_reduce
        fwd = rom.BlockBuffers(T, DM, DE, E, K, torch.bfloat16, "cpu")
        norm = rom.NormBuffers(T, DM, torch.bfloat16, torch.float32, "cpu")
        fwd.out = norm.y
        sync = rom.GradientAllReduce()
        w_r, w = torch.zeros(DM, E), torch.zeros(E, DE, DM, dtype=torch.bfloat16)
        w_out = torch.zeros(E, DM, DE, dtype=torch.bfloat16)
        for renorm in (True, False):
            log.clear(), exchanged.clear()
            bwd, g = rom.residual_block_backward(rom.ResidualBlock(norm, fwd, renorm), torch.zeros(T, DM, dtype=torch.bfloat16),
                                                 torch.ones(DM), w_r, w, w, w_out, grad_sync=sync)
            order = [bwd.dw_out, bwd.dw_r, bwd.dbias, bwd.dw_conv, bwd.dw_gate, g.dw]
            assert [t.data_ptr() for t in exchanged] == [t.data_ptr() for t in order]
            assert sync.pending == []
            # the sums over both ranks, of what the kernels had written by then
            for t, n in zip(order, (11, 5, 7, 11, 13, 19)):
                assert torch.all(t == 3 * n), (rank, n)
            # the gradients of the tokens stay the rank's own
            assert torch.all(bwd.dx == value(2)) and torch.all(g.dx == value(17))
            # dW_out leaves before the rest of the backward runs, dw after the norm's
            assert log.index("all_reduce") < log.index("rom_bwd_gate")
            assert log[-2:] == ["rom_add_rmsnorm_bwd", "all_reduce"]
            # without an exchange: the same kernels, nothing sent
            log.clear(), exchanged.clear()
            _, g = rom.residual_block_backward(rom.ResidualBlock(norm, fwd, renorm), torch.zeros(T, DM, dtype=torch.bfloat16),
                                               torch.ones(DM), w_r, w, w, w_out)
            assert not exchanged and torch.all(g.dw == value(19))
        dist.barrier()
    finally:
        dist.destroy_process_group()


def test_residual_block_gradients_over_two_gloo_ranks():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    mp.start_processes(_rank_main, args=(2, port), nprocs=2, start_method="spawn", join=True)
