"""Calls on a given stream while the current one is busy: what a call makes for itself (status words, workspaces,
zeroed outputs) belongs to the stream it runs on."""
import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd
from test_gpu_q8_attn import call, setup

pytestmark = pytest.mark.gpu

BUSY = 300_000_000     # cycles: 0.15 s of work already on a stream


def on_side(run):
    """run(stream) on a side stream while the current stream is busy; the results as they are when the side stream
    is done, and as they are later."""
    side = torch.cuda.Stream()
    run(side)                                                      # (a kernel's first launch loads it, which waits)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    out = run(side)
    with torch.cuda.stream(side):
        first = [t.clone() for t in out]
    side.synchronize()
    assert not torch.cuda.current_stream().query()                 # still busy: nothing waited for it
    torch.cuda.synchronize()
    return first, out


def behind_a_busy_side(run):
    """run(stream) on a side stream that is busy; meanwhile the current stream fills what the allocator gives it."""
    fill = lambda: [torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
                    for n in (512, 4096, 1 << 16, 1 << 20, 1 << 22) for _ in range(8)]
    side = torch.cuda.Stream()
    run(side), fill()                                              # (so is the allocator's memory there)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    out = run(side)
    junk = fill()
    torch.cuda.current_stream().synchronize()
    assert not side.query()
    torch.cuda.synchronize()
    del junk
    return out, out


@pytest.mark.parametrize("how", [on_side, behind_a_busy_side])
@pytest.mark.parametrize("paged", [True, False])
def test_cache_calls_on_a_given_stream(how, paged):
    s = setup(2, 5, 16, 2, 128, 16, [300, 70], paged, "bf16", "chain")
    c = s["cache"]
    want = tsd.kv_q8_read(c, S=70)
    for got in how(lambda st: tsd.kv_q8_read(c, S=70, stream=st)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    acc = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    for got in how(lambda st: [tsd.kv_q8_commit(c, s["kt"], s["vt"], None, acc, Dmax=s["D"], mode="length", advance=False, stream=st)]):
        assert not got[0].any()
    bad = torch.tensor([c.capacity, 1], dtype=torch.int32, device="cuda")
    rows = torch.zeros(2, c.capacity, 2, 128, dtype=torch.bfloat16, device="cuda")
    for got in how(lambda st: [tsd.kv_q8_append(c, rows, rows, bad, advance=False, stream=st)]):
        assert [x & 255 for x in got[0].tolist()] == [6, 0]
    again = tsd.kv_q8_read(c, S=64)
    assert torch.equal(again[0], want[0][:, :64])                  # (the block of row 70 may have been requantised)


@pytest.mark.parametrize("how", [on_side, behind_a_busy_side])
@pytest.mark.parametrize("B,N,Hq,L", [(1, 3, 8, 900), (16, 60, 8, 800)])
def test_attention_on_a_given_stream(how, B, N, Hq, L):
    """A workspace of its own, split and merged in a second kernel and in the kernel."""
    s = setup(B, N, Hq, 2, 128, 16, [L - b for b in range(B)], True, "bf16")
    assert tsd.tree_verify_attn_q8_workspace(s["q"], s["cache"]).numel() > 16
    want = call(s, want_lse=True)
    for got in how(lambda st: call(s, want_lse=True, stream=st)):
        assert torch.equal(got[0][:, :N], want[0][:, :N]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("how", [on_side, behind_a_busy_side])
def test_sampling_on_a_given_stream(how):
    z = torch.randn(4, 32000, device="cuda").bfloat16()
    u = torch.rand(4, device="cuda")
    want = tsd.sample_rows(z, u)
    for got in how(lambda st: list(tsd.sample_rows(z, u, stream=st).values())):
        assert torch.equal(got[0], want["tokens"]) and torch.equal(got[1], want["probs"])


def test_results_outlive_the_callers_reference():
    """A result that the caller's stream still reads is not handed out again when its last reference goes."""
    s = setup(1, 5, 16, 2, 128, 16, [300], True, "bf16")
    want = tsd.kv_q8_read(s["cache"], S=300)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    k, v = tsd.kv_q8_read(s["cache"], S=300, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    got = k.clone()                                                # reads it after the sleep
    del k, v
    with torch.cuda.stream(side):
        for _ in range(4):
            torch.full_like(want, 7.0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
