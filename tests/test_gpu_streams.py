"""Calls on a given stream while the current one is busy: what a call makes for itself (status words, workspaces,
zeroed outputs) belongs to the stream it runs on."""
import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd
import workloads as W
from test_gpu_q8_attn import call, setup
from tree_speculative_decoding_06_b200.step import to_device

pytestmark = pytest.mark.gpu

BUSY = 600_000_000     # cycles: 0.3 s of work already on a stream


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


def flat(r):
    return [t for t in (r.values() if isinstance(r, dict) else r if isinstance(r, tuple) else [r]) if t is not None]


@pytest.mark.parametrize("how", [on_side, behind_a_busy_side])
@pytest.mark.parametrize("name", ["tree26", "eagle60"])
def test_verify_calls_on_a_given_stream(how, name):
    """The calls over a cache of the call's type: prepare, attention, every acceptance, commit."""
    w = W.WORKLOADS[name]
    w = w.scaled(L=900, V=2048) if name == "tree26" else w.scaled(B=3, L=850, L_lo=300, V=2048)
    x = to_device(W.make_inputs(w, nan_guard=False))
    D, nodes = int(x["Dmax"]), x["num_nodes"]
    prep = tsd.tree_prepare(x["parent"], nodes, D)
    ps, B, N = prep["parent_s"], *x["parent"].shape
    u = torch.rand(B, N, device="cuda")
    draft = torch.randn_like(x["logits"].float()).to(x["logits"].dtype)
    acc = tsd.tree_accept_greedy(x["logits"], x["tokens"], ps, nodes, Dmax=D)
    paged = "k_pages" in x
    prefix = x["prefix_len"].clone()

    def attn(st=None):
        if paged:
            return tsd.tree_verify_attn_paged(x["q"], x["k_pages"], x["v_pages"], x["block_table"], x["prefix_len"], x["k_tree"],
                                              x["v_tree"], ps, nodes, D, want_lse=True, stream=st)
        return tsd.tree_verify_attn(x["q"], x["k_cache"], x["v_cache"], x["prefix_len"], x["k_tree"], x["v_tree"], ps, nodes, D,
                                    want_lse=True, stream=st)

    def commit(st=None):
        with torch.cuda.stream(st or torch.cuda.current_stream()):
            p = prefix.clone()
        if paged:
            return tsd.kv_commit_paged(x["k_pages"], x["v_pages"], x["block_table"], p, x["k_tree"], x["v_tree"], acc["path"],
                                       acc["accept_len"], nodes, D, stream=st)
        return tsd.kv_commit(x["k_cache"], x["v_cache"], p, x["k_tree"], x["v_tree"], acc["path"], acc["accept_len"], nodes, D,
                             stream=st)

    calls = [attn, commit,
             lambda st=None: tsd.tree_prepare(x["parent"], nodes, D, stream=st),
             lambda st=None: tsd.tree_accept_greedy(x["logits"], x["tokens"], ps, nodes, Dmax=D, stream=st),
             lambda st=None: tsd.tree_accept_greedy_noalloc(x["logits"], x["tokens"], ps, nodes, Dmax=D, stream=st),
             lambda st=None: tsd.tree_accept_threshold(x["logits"], x["tokens"], ps, 0.1, 0.8, nodes, Dmax=D, stream=st),
             lambda st=None: tsd.tree_accept_sample(x["logits"], draft, x["tokens"], ps, u, 0.8, nodes, D, stream=st)]
    live = torch.arange(N, device="cuda")[None] < nodes[:, None]   # (rows of nodes past N_b are not written)
    for f in calls:
        want = flat(f())
        torch.cuda.synchronize()
        for got in how(lambda st: flat(f(st))):
            for a, b in zip(got, want):
                ok = torch.equal(a[live], b[live]) if f is attn else torch.equal(a, b)
                assert ok, f


def test_a_stream_may_be_given_by_position():
    z, u = torch.randn(3, 5000, device="cuda"), torch.rand(3, device="cuda")
    want = tsd.sample_rows(z, u)["tokens"]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = tsd.sample_rows(z, u, None, None, None, None, None, None, side)["tokens"]
    side.synchronize()
    assert torch.equal(got, want)
    tree, other = tsd.DraftTree(1, 4, 20), tsd.DraftTree(1, 4, 20)
    root, logits = torch.tensor([7], dtype=torch.int32, device="cuda"), torch.randn(1, 4, 5000, device="cuda")
    torch.cuda.synchronize()
    tree.init(root, side), tree.expand(logits, 4, side)
    a = tree.finalize(5, None, None, None, side)
    side.synchronize()
    other.init(root), other.expand(logits, 4)
    b = other.finalize(5)
    for k in a:
        assert torch.equal(a[k], b[k])
