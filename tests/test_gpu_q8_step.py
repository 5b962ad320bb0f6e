"""The 8-bit cache, the attention over it and the sampler together, as a serving loop uses them: prompts
appended, the first token drawn, verify steps, rows read back."""
import numpy as np
import pytest
import torch

import oracle
import tree_speculative_decoding_06_b200 as tsd
import workloads as W
from q8_ref import sample
from test_gpu_q8_attn import check
from test_gpu_q8_cache import check_cache, make, rows_np, to_gpu
from tree_speculative_decoding_06_b200.step import VerifyStep, to_device

pytestmark = pytest.mark.gpu


def prompts(inp, paged, bs, steps):
    """An empty reference cache and its Q8Cache with room for the workload's prefixes and some steps, the
    prompts (the workload's own bf16 prefix rows) appended to both through the library and the reference."""
    B, Hkv, d = inp["parent"].shape[0], inp["k_tree"].shape[2], inp["k_tree"].shape[3]
    L = [int(x) for x in inp["prefix_len"]]
    cap = max(L) + steps * (int(inp["Dmax"]) + 1) + 3
    ref = make(B, Hkv, d, bs, [0] * B, cap, paged, junk=True)
    cache = to_gpu(ref, paged, cap)
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = [torch.randn(B, max(L), Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    status = tsd.kv_q8_append(cache, rows[0], rows[1], torch.tensor(L, dtype=torch.int32, device="cuda"))
    assert not status.any()
    for b in range(B):
        ref.write(b, rows_np(rows[0][b, :L[b]]), rows_np(rows[1][b, :L[b]]))
    ref.prefix = np.array(L)
    return ref, cache, cap


def step_inputs(inp, seed):
    """The workload's tree with new queries, tree K/V and logits."""
    x = to_device(inp)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for k in ("q", "k_tree", "v_tree"):
        x[k] = torch.randn(x[k].shape, generator=g, device="cuda").to(x[k].dtype)
    return x


@pytest.mark.parametrize("paged,bs", [(True, 16), (False, 64)])
@pytest.mark.parametrize("schedule", ["overlap", "serial"])
@pytest.mark.parametrize("name", ["tree26", "eagle60"])
def test_serving_loop(name, paged, bs, schedule):
    w = W.WORKLOADS[name]
    w = w.scaled(L=200, V=2048) if name == "tree26" else w.scaled(B=3, L=250, L_lo=100, V=2048)
    inp = W.make_inputs(w, nan_guard=False)
    ref, cache, cap = prompts(inp, paged, bs, 3)
    B = len(ref.prefix)
    # the first token of every sequence
    z = torch.randn(B, 2048, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    u = torch.full((B,), 0.4, device="cuda")
    T, k, P = torch.full((B,), 0.7, device="cuda"), torch.full((B,), 40, dtype=torch.int32, device="cuda"), torch.full((B,), 0.9, device="cuda")
    first = tsd.sample_rows(z, u, T, k, P)["tokens"].tolist()
    assert first == [sample(rows_np(z[b]), np.float32(0.7), 40, np.float32(0.9), 0.0, np.float32(0.4))[0] for b in range(B)]
    x = step_inputs(inp, 0)
    step = VerifyStep.for_inputs(x, q8=cache, schedule=schedule)
    acc = oracle.accept_greedy(inp)
    for n in range(3):
        x = step_inputs(inp, n)
        L = [int(p) for p in ref.prefix]
        res = step.run(x)
        torch.cuda.synchronize()
        assert not res["status"].any()
        # attention of the step, acceptance, then the commit of the accepted rows
        s = dict(ref=ref, q=x["q"], kt=x["k_tree"], vt=x["v_tree"], par=inp["parent"], nodes=[int(c) for c in inp["num_nodes"]],
                 L=L, dt="bf16")
        check(s, res["out"], None)
        assert np.array_equal(res["accept_len"].cpu().numpy(), acc["accept_len"])
        assert np.array_equal(res["out_tokens"].cpu().numpy(), acc["out_tokens"])
        for b in range(B):
            src = [int(p) - 1 for p in acc["path"][b][:acc["accept_len"][b] + 1]]
            ref.write(b, rows_np(x["k_tree"][b, src]), rows_np(x["v_tree"][b, src]))
        ref.prefix = ref.prefix + acc["accept_len"] + 1
        assert cache.prefix_len.tolist() == ref.prefix.tolist()
    check_cache(cache, ref, paged, cap)
    # the last rows read back are the values the next attention attends
    S = 20
    start = torch.tensor([int(p) - S for p in ref.prefix], dtype=torch.int32, device="cuda")
    kk, vv = tsd.kv_q8_read(cache, start, S=S)
    for b in range(B):
        rk, rv = ref.rows(b, int(start[b]), int(start[b]) + S)
        assert np.array_equal(rows_np(kk[b]), rk) and np.array_equal(rows_np(vv[b]), rv)


def test_captured_step_and_shared_prefix_len():
    """A captured two-layer step: the layers share prefix_len, the last one's commit advances it; replays
    give what eager runs give."""
    w = W.WORKLOADS["tree26"].scaled(L=100, V=2048)
    inp = W.make_inputs(w, nan_guard=False)
    _, c0, _ = prompts(inp, True, 16, 4)
    twin = lambda c, pl: tsd.Q8Cache.wrap(c.k.clone(), c.v.clone(), c.k_scale.clone(), c.v_scale.clone(), pl, 16, c.block_table)  # noqa: E731
    x = step_inputs(inp, 1)
    D = int(x["Dmax"])
    prep = tsd.tree_prepare(x["parent"], x["num_nodes"], D)
    acc = tsd.tree_accept_greedy(x["logits"], x["tokens"], prep["parent_s"], x["num_nodes"], Dmax=D)

    def layers(caches, outs, ws, status):
        for i, c in enumerate(caches):
            tsd.tree_verify_attn_q8(x["q"], c, x["k_tree"], x["v_tree"], prep["parent_s"], x["num_nodes"], D, out=outs[i],
                                    workspace=ws, status=status)
            tsd.kv_q8_commit(c, x["k_tree"], x["v_tree"], acc["path"], acc["accept_len"], x["num_nodes"], D,
                             advance=i == len(caches) - 1, status=status)

    def state():
        pl = c0.prefix_len.clone()
        caches = [twin(c0, pl), twin(c0, pl)]
        return caches, [torch.zeros_like(x["q"]) for _ in caches], tsd.tree_verify_attn_q8_workspace(x["q"], c0), \
            torch.zeros(x["q"].shape[0], dtype=torch.int32, device="cuda")

    eager, graph = state(), state()
    for _ in range(3):
        layers(*eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layers(*graph)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    rows = int(acc["accept_len"][0]) + 1
    for caches, outs, _, status in (eager, graph):
        assert not status.any() and caches[0].prefix_len.tolist() == [100 + 3 * rows]
    for a, b in zip(eager[0] , graph[0]):
        assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and torch.equal(a.v_scale, b.v_scale)
    for a, b in zip(eager[1], graph[1]):
        assert torch.equal(a, b)


def test_step_refusals():
    cache = tsd.Q8Cache(1, 8, 128, Lmax=64, block_size=16)
    kw = dict(B=1, Nmax=26, Hq=32, Hkv=8, d=128, Dmax=6, V=1000, dtype=torch.bfloat16)
    for bad in (dict(schedule="fused"), dict(history_cap=8), dict(Hkv=4)):
        with pytest.raises(ValueError):
            VerifyStep(**{**kw, **bad}, q8=cache)
    step = VerifyStep(**kw, q8=cache)
    assert step.launches_per_step() == 1 + step.attn_launches() + 1 + 3
