"""Calls from host threads of their own, each on its own stream: none disturbs another's launch."""
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


def together(calls, n=1500):
    """Runs every call n times in a thread of its own; then its result once more against its result alone."""
    want = [[t.clone() for t in f()] for f in calls]
    torch.cuda.synchronize()
    go, errors = threading.Barrier(len(calls)), []

    def work(f, want):
        try:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                go.wait()
                for i in range(n):
                    got = f()
                    if i % 100 == 0:
                        side.synchronize()
                side.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(calls, want)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_sampling_of_several_vocabularies(dt):
    def one(V):
        z, u = torch.randn(2, V, device="cuda").to(dt), torch.rand(2, device="cuda")
        out = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda")
        return lambda: list(tsd.sample_rows(z, u, tokens=out[0], probs=out[1]).values())
    together([one(V) for V in (128256, 3000, 100000, 5000)])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_c_calls_in_tight_loops(dt):
    """The C calls alone, next to no Python between them: the threads' launches come within a microsecond."""
    f, failed = tsd.lib().tsd_sample_rows, []

    def work(V):
        z, u, tok = torch.randn(1, V, device="cuda").to(dt), torch.rand(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        args = (z.data_ptr(), int(dt == torch.bfloat16), 1, V, u.data_ptr(), None, None, None, None, tok.data_ptr(), None,
                side.cuda_stream)
        failed.append(sum(f(*args) != 0 for _ in range(20000)))
        side.synchronize()

    threads = [threading.Thread(target=work, args=(V,)) for V in (128256, 3000, 100000, 5000)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert failed == [0, 0, 0, 0]


@pytest.mark.parametrize("d,dt", [(128, "bf16"), (64, "bf16"), (64, "f32")])
def test_attention_of_small_and_large_trees(d, dt):
    def one(N):
        s = setup(1, N, 4, 2, d, 16, [70], True, dt, "star")
        out, ws = torch.empty_like(s["q"]), tsd.tree_verify_attn_q8_workspace(s["q"], s["cache"])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return lambda: [call(s, out=out, workspace=ws, status=status)[0]]
    together([one(N) for N in (1, 600, 5, 900)])


def test_attention_and_acceptance_over_a_bf16_cache():
    def one(N):
        t = lambda *s: torch.randn(s, device="cuda").bfloat16()  # noqa: E731
        q, k, v, kt, vt = t(1, N, 8, 128), t(1, 2, 128, 128), t(1, 2, 128, 128), t(1, N, 2, 128), t(1, N, 2, 128)
        parent = torch.zeros(1, N, dtype=torch.int32, device="cuda")
        parent[0, 0] = -1
        ps, L = tsd.tree_prepare(parent, None, 8)["parent_s"], torch.tensor([100], dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return lambda: [tsd.tree_verify_attn(q, k, v, L, kt, vt, ps, None, 8, out=out, workspace=ws, status=status)[0]]
    together([one(N) for N in (1, 500, 9, 700)])
