"""Calls from host threads of their own."""
import threading

import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd
from test_gpu_q8_attn import call, setup

pytestmark = pytest.mark.gpu


def in_a_new_thread(f):
    got = []

    def work():
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


@pytest.mark.parametrize("N", [3, 60])
def test_a_threads_first_call(N):
    """An attention call as the first CUDA work of a host thread, outputs and workspace given."""
    s = setup(2, N, 8, 2, 128, 16, [300, 70], True, "bf16")
    out, status = torch.empty_like(s["q"]), torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = tsd.tree_verify_attn_q8_workspace(s["q"], s["cache"])
    want = call(s, workspace=ws)[0]
    in_a_new_thread(lambda: call(s, out=out, workspace=ws, status=status))
    assert torch.equal(out, want)
    k = torch.randn(2, 2, 400, 128, device="cuda").bfloat16()
    args = (s["q"], k, k, s["cache"].prefix_len, s["kt"], s["vt"], s["ps"], s["nn"], s["D"])
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    want = tsd.tree_verify_attn(*args, workspace=ws)[0]
    in_a_new_thread(lambda: tsd.tree_verify_attn(*args, out=out, workspace=ws, status=status))
    assert torch.equal(out, want)
