"""The 8-bit cache's calls and sample_rows with every output and workspace given: no device memory is taken, by torch
or by the library."""
import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd
from test_gpu_q8_attn import call, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,Hq,d,dt", [(3, 8, 128, "bf16"), (60, 16, 128, "bf16"), (5, 6, 64, "bf16"), (5, 4, 64, "f32")])
def test_nothing_is_allocated(N, Hq, d, dt):
    s = setup(2, N, Hq, 2, d, 16, [900, 333], True, dt, "chain" if N < 10 else "rand", cap=1400)
    c, t = s["cache"], dict(dtype=s["q"].dtype, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse, ws = torch.empty_like(s["q"]), torch.empty(2, N, Hq, device="cuda"), tsd.tree_verify_attn_q8_workspace(s["q"], c)
    status, acc, n = i32(0, 0), i32(1, 2), i32(7, 0)
    path = torch.ones(2, s["D"] + 1, dtype=torch.int32, device="cuda")
    rows = [torch.randn(2, 9, 2, d, device="cuda").to(s["q"].dtype) for _ in range(2)]
    back = [torch.empty(2, 50, 2, d, **t) for _ in range(2)]
    z, u, par = torch.randn(3, 50257, **t), torch.rand(3, device="cuda"), torch.full((3,), 0.9, device="cuda")
    k, tok, pr = i32(40, 0, 3000), i32(0, 0, 0), torch.empty(3, device="cuda")

    def everything():
        call(s, out=out, lse=lse, workspace=ws, status=status)
        tsd.kv_q8_commit(c, s["kt"], s["vt"], path, acc, s["nn"], s["D"], status=status)
        tsd.kv_q8_append(c, rows[0], rows[1], n, status=status)
        tsd.kv_q8_read(c, k_out=back[0], v_out=back[1], status=status)
        tsd.sample_rows(z, u, par, k, par, par, tokens=tok, probs=pr)

    everything()                                                   # (loads the kernels)
    torch.cuda.synchronize()
    free, taken = torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        everything()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == taken
    assert torch.cuda.mem_get_info()[0] == free
    assert not status.any()
