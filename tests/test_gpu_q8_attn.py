"""Tree attention over the 8-bit cache against the 64-bit reference on the cache's own values.

Tolerance.  The reference attends the values code * scale, which the kernels hold exactly.  A kernel's
result differs by: scores summed in fp32 (error E of the reference, the largest over the row's keys; it
also covers a query held as two 8-bit pieces), which changes each weight by e^(2E) - 1 < 3E; weights and
their sums in fp32, (L + N) 2^-24 relative at most; weights rounded to bf16, 2^-8 relative; and the
output's rounding, 2^-8 (bf16) or 2^-24 (fp32) relative.  All but the last apply to the attention of |V|."""
import os

import numpy as np
import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd
from q8_ref import attention
from test_gpu_q8_cache import DT, make, rows_np, to_gpu

pytestmark = pytest.mark.gpu


def tree(B, N, kind, rng):
    if kind == "chain":
        p = np.arange(N) - 1
    elif kind == "star":
        p = np.where(np.arange(N) > 0, 0, -1)
    elif kind == "forest":
        p = np.where(np.arange(N) % 5 == 0, -1, np.arange(N) - 1)
    else:
        p = np.array([-1] + [int(rng.integers(max(0, i - 9), i)) for i in range(1, N)])
    return np.tile(p.astype(np.int32), (B, 1))


def depth(par):
    d = []
    for p in par:
        d.append(0 if p < 0 else d[p] + 1)
    return max(d)


def setup(B, N, Hq, Hkv, d, bs, L, paged, dt, kind="rand", nodes=None, cap=None, seed=0):
    rng = np.random.default_rng(seed)
    cap = max(L) + 3 if cap is None else cap
    ref = make(B, Hkv, d, bs, L, cap, paged, seed)
    cache = to_gpu(ref, paged, cap)
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dt])  # noqa: E731
    q, kt, vt = t(B, N, Hq, d), t(B, N, Hkv, d), t(B, N, Hkv, d)
    par = tree(B, N, kind, rng)
    nodes = [N] * B if nodes is None else nodes
    for b in range(B):                              # rows of nodes past N_b are never read
        kt[b, nodes[b]:], vt[b, nodes[b]:], q[b, nodes[b]:] = float("nan"), float("nan"), float("nan")
    D = max(1, depth(par[0]))
    nn = torch.tensor(nodes, dtype=torch.int32, device="cuda")
    prep = tsd.tree_prepare(torch.from_numpy(par).cuda(), nn, D, kind == "forest")
    return dict(ref=ref, cache=cache, q=q, kt=kt, vt=vt, par=par, nodes=nodes, nn=nn, D=D, ps=prep["parent_s"], L=L, dt=dt)


def call(s, **kw):
    return tsd.tree_verify_attn_q8(s["q"], s["cache"], s["kt"], s["vt"], s["ps"], s["nn"], s["D"], **kw)


def check(s, out, lse, skip=(), scale=None):
    d = s["q"].shape[3]
    half = 2.0 ** -8 if s["dt"] == "bf16" else 2.0 ** -24
    for b, n in enumerate(s["nodes"]):
        if b in skip or n == 0:
            continue
        K, V = s["ref"].rows(b, 0, s["L"][b])
        o, l, a, e = attention(rows_np(s["q"][b, :n]), K, V, rows_np(s["kt"][b, :n]), rows_np(s["vt"][b, :n]),
                               s["par"][b], d ** -0.5 if scale is None else scale)
        rel = 3 * e + (s["L"][b] + n) * 2.0 ** -24 + (half if s["dt"] == "bf16" else 0.0)
        tol = rel[..., None] * a + half * np.abs(o) + 1e-30
        got = rows_np(out[b, :n])
        bad = ~(np.abs(got - o) <= tol)
        assert not bad.any(), (b, int(bad.sum()), float(np.nanmax(np.abs(got - o) / tol)), np.argwhere(bad)[:3].tolist())
        if lse is not None:
            gl = lse[b, :n].double().cpu().numpy()
            assert (np.abs(gl - l) <= 3 * e + (s["L"][b] + n + 16) * 2.0 ** -24 + np.abs(l) * 2.0 ** -22).all(), b


CASES = [
    # B, N, Hq, Hkv, d, bs, lengths, paged, type, tree
    (1, 1, 8, 8, 128, 16, [0], True, "bf16", "chain"),
    (1, 1, 32, 8, 128, 16, [1], True, "bf16", "chain"),
    (2, 1, 32, 8, 128, 16, [63, 64], True, "bf16", "chain"),
    (3, 6, 16, 2, 128, 64, [65, 0, 640], False, "bf16", "chain"),
    (1, 26, 32, 8, 128, 32, [1031], False, "bf16", "rand"),
    (2, 60, 8, 2, 128, 16, [700, 129], True, "bf16", "rand"),
    (2, 70, 16, 4, 128, 8, [255, 257], True, "bf16", "forest"),
    (1, 130, 8, 2, 128, 128, [513], True, "bf16", "star"),
    (1, 3, 4, 4, 128, 256, [777], False, "bf16", "rand"),
    (2, 9, 128, 1, 128, 16, [200, 90], True, "bf16", "rand"),
    (2, 5, 6, 2, 128, 16, [100, 333], True, "bf16", "rand"),       # three query heads a KV head
    (2, 9, 14, 2, 64, 8, [77, 5], True, "bf16", "rand"),
    (1, 33, 4, 1, 64, 64, [500], False, "bf16", "rand"),
    (3, 7, 12, 4, 64, 32, [301, 0, 64], True, "f32", "rand"),
    (1, 20, 2, 1, 128, 16, [210], False, "f32", "forest"),
    (2, 1, 8, 2, 128, 8, [9, 1000], True, "f32", "chain"),
]


@pytest.mark.parametrize("B,N,Hq,Hkv,d,bs,L,paged,dt,kind", CASES)
def test_against_the_reference(B, N, Hq, Hkv, d, bs, L, paged, dt, kind):
    s = setup(B, N, Hq, Hkv, d, bs, L, paged, dt, kind, nodes=[max(1, N - 2 * b) for b in range(B)])
    out = torch.full_like(s["q"], 5.0)
    out, lse = call(s, out=out, want_lse=True)
    check(s, out, lse)
    for b, n in enumerate(s["nodes"]):
        assert (out[b, n:] == 5).all()                             # rows of nodes past N_b stay


@pytest.mark.parametrize("splits", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("N,Hq", [(6, 16), (40, 16)])
def test_any_number_of_key_splits(splits, N, Hq, monkeypatch):
    """Splits with no keys, one key tile, and many; one and two query tiles per CTA."""
    s = setup(3, N, Hq, 2, 128, 16, [400, 3, 0], True, "bf16")
    monkeypatch.setenv("TSD_ATTN_SPLITS", str(splits))
    ws = torch.zeros(tsd.tree_verify_attn_ticket_bytes() + 3 * 2 * 8 * 8 * N * 130 * 4, dtype=torch.uint8, device="cuda")
    for _ in range(2):                                             # the ticket words come back to zero
        out, lse = call(s, want_lse=True, workspace=ws)
        check(s, out, lse)
    assert not ws[:tsd.tree_verify_attn_ticket_bytes()].any()


@pytest.mark.parametrize("dt,d,Hq", [("bf16", 128, 8), ("bf16", 64, 8), ("f32", 64, 6)])
def test_scales_far_apart(dt, d, Hq):
    """Blocks whose K and V differ by many powers of two, zero blocks, and large queries."""
    B, N, Hkv, bs, L = 2, 4, 2, 16, [150, 97]
    s = setup(B, N, Hq, Hkv, d, bs, L, True, dt)
    rng = np.random.default_rng(3)
    ref = make(B, Hkv, d, bs, [0, 0], max(L) + 3, True)
    for b in range(B):
        k = rng.normal(size=(L[b], Hkv, d)) * 2.0 ** (-(np.arange(L[b]) // bs % 9) * 3.0)[:, None, None]
        v = rng.normal(size=(L[b], Hkv, d)) * 2.0 ** ((np.arange(L[b]) // bs % 7) * 6.0 - 20)[:, None, None]
        v[bs:2 * bs] = 0
        k[3 * bs:4 * bs] = 0
        ref.write(b, k, v)
    ref.prefix = np.array(L)
    s["ref"], s["cache"] = ref, to_gpu(ref, True, max(L) + 3)
    s["q"] *= 30.0
    out, lse = call(s, want_lse=True)
    check(s, out, lse)
    s["q"] *= 2.0 ** -60                                           # scores of (almost) zero: an average
    out, lse = call(s, want_lse=True)
    check(s, out, lse)
    out, lse = call(s, want_lse=True, scale=0.5)
    check(s, out, lse, scale=0.5)


@pytest.mark.parametrize("N,Hq", [(5, 16), (40, 16), (5, 6)])
def test_flagged_and_bad_sequences_are_zero(N, Hq):
    """A sequence flagged on entry, one past its capacity and one with a bad block id give zero rows and
    their status; an idle one (no nodes) writes nothing; the others are right."""
    L = [100, 100, 100, 200, 333]
    s = setup(5, N, Hq, 2, 128, 16, L, True, "bf16", nodes=[N, N, N, 0, N])
    s["cache"].prefix_len[1] = s["cache"].capacity + 1
    s["cache"].block_table[2, 3] = s["cache"].k.shape[0]
    status = torch.tensor([9, 0, 0, 0, 0], dtype=torch.int32, device="cuda")
    out = torch.full_like(s["q"], 5.0)
    for _ in range(2):
        call(s, out=out, status=status)
        assert [x & 255 for x in status.tolist()] == [9, 6, 6, 0, 0]
        assert not out[:3].any() and (out[3] == 5).all()
        check(s, out, None, skip=(0, 1, 2, 3))


def test_captured_and_on_another_stream():
    s = setup(2, 6, 16, 2, 128, 16, [300, 70], True, "bf16")
    want, _ = call(s)
    out, ws = torch.zeros_like(want), tsd.tree_verify_attn_q8_workspace(s["q"], s["cache"])
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        call(s, out=out, workspace=ws, status=status)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.stream(side):
        again, _ = call(s)
    side.synchronize()
    assert torch.equal(again, want)


def test_binding_refusals():
    s = setup(2, 6, 16, 2, 128, 16, [30, 70], True, "bf16")
    for bad in (dict(q=s["q"][:1]), dict(kt=s["kt"][:, :3]), dict(vt=s["vt"].float()), dict(ps=s["ps"][:, :3]),
                dict(nn=s["nn"].long()), dict(q=s["q"].half()), dict(q=s["q"].transpose(1, 2))):
        with pytest.raises(tsd.TsdError):
            call({**s, **bad})
    with pytest.raises(tsd.TsdError):
        call(s, out=s["q"].float())
    with pytest.raises(tsd.TsdError):
        call(s, status=torch.zeros(2, device="cuda"))


@pytest.mark.parametrize("N,Hq", [(6, 16), (40, 16)])
@pytest.mark.parametrize("tile", [0, 2, 5])
def test_time_out_is_reported(N, Hq, tile, monkeypatch):
    """A key tile that never arrives: the bounded waits give up, the sequence is flagged and zero, and the
    next call on the same workspace is right."""
    s = setup(2, N, Hq, 2, 128, 16, [310, 310], True, "bf16")
    ws = tsd.tree_verify_attn_q8_workspace(s["q"], s["cache"])
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("TSD_TEST_WITHHOLD_TILE", str(tile))
    out, _ = call(s, workspace=ws, status=status)
    torch.cuda.synchronize()
    assert [x & 255 for x in status.tolist()] == [7, 7] and not torch.isnan(out).any()
    monkeypatch.delenv("TSD_TEST_WITHHOLD_TILE")
    out, lse = call(s, workspace=ws, want_lse=True)
    check(s, out, lse)


def test_many_seeds():
    """Random shapes of the whole range."""
    rng = np.random.default_rng(int(os.environ.get("TSD_TEST_SEED", "11")))
    for i in range(16):
        Hkv, G = int(rng.choice([1, 2, 4])), int(rng.choice([1, 2, 3, 4, 8, 16]))
        B, N, bs = int(rng.integers(1, 5)), int(rng.integers(1, 50)), int(2 ** rng.integers(3, 9))
        L = [int(2 ** rng.uniform(0, 9.5)) - 1 for _ in range(B)]
        s = setup(B, N, G * Hkv, Hkv, int(rng.choice([64, 128, 128, 128])), bs, L, bool(rng.random() < 0.6),
                  str(rng.choice(["bf16", "bf16", "f32"])), str(rng.choice(["rand", "chain", "forest", "star"])), seed=i)
        out, lse = call(s, want_lse=True)
        check(s, out, lse)


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("N,Hq,d,dt,kind", [(5, 16, 128, "bf16", "star"), (12, 4, 128, "bf16", "forest"),
                                            (40, 16, 128, "bf16", "forest"), (130, 8, 128, "bf16", "forest"),
                                            (70, 2, 128, "bf16", "forest"), (12, 6, 128, "bf16", "forest"),
                                            (70, 8, 64, "bf16", "forest"), (12, 6, 64, "f32", "forest"),
                                            (70, 2, 128, "f32", "star")])
def test_infinities_and_nan_reach_only_the_rows_that_see_them(N, Hq, d, dt, kind, splits, monkeypatch):
    """A node's infinite or NaN keys, values and queries show in its own and its descendants' rows (as the
    formula has them) and in no other; NaN in the cache reaches every row of its heads."""
    if splits > 1:
        monkeypatch.setenv("TSD_ATTN_SPLITS", str(splits))
    L, Hkv = [300, 20], 2
    s = setup(2, N, Hq, Hkv, d, 16, L, True, dt, kind)
    nan, inf = float("nan"), float("inf")
    s["vt"][0, N - 1, 0, 5], s["vt"][0, 1, 0, 9], s["vt"][0, 1, 1, d - 1] = nan, inf, -inf
    s["vt"][1, 2, 1], s["kt"][1, 3, 0] = inf, nan
    s["kt"][1, 1, 1, 2] = nan
    s["q"][0, 3, 0, 1] = nan
    ws = torch.zeros(tsd.tree_verify_attn_ticket_bytes() + 2 * 2 * 64 * 8 * N * 130 * 4, dtype=torch.uint8, device="cuda")
    out, lse = call(s, want_lse=True, workspace=ws)
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    for b in range(2):
        K, V = s["ref"].rows(b, 0, L[b])
        with np.errstate(invalid="ignore"):
            o, l, a, e = attention(rows_np(s["q"][b]), K, V, rows_np(s["kt"][b]), rows_np(s["vt"][b]), s["par"][b], d ** -0.5)
            tol = (3 * e + (L[b] + N) * 2.0 ** -24 + (half if dt == "bf16" else 0.0))[..., None] * a + half * np.abs(o)
            got = rows_np(out[b])
            good = np.where(np.isfinite(o), np.abs(got - o) <= tol + 1e-30, np.where(np.isnan(o), np.isnan(got), got == o))
        assert not np.isfinite(o).all() and good.all(), (b, np.argwhere(~good)[:4].tolist())
        assert (np.isnan(l) == np.isnan(lse[b].cpu().numpy())).all()
    c = s["cache"]
    c.k.view(torch.uint8)[c.block_table[0, 7], 0, 3, 4] = 127
    c.v.view(torch.uint8)[c.block_table[1, 0], 1, 2, 6] = 255
    clean = setup(2, N, Hq, Hkv, d, 16, L, True, dt, kind)
    got = call({**clean, "cache": c}, workspace=ws)[0].isnan()
    G = Hq // Hkv
    assert got[0, :, :G].all() and not got[0, :, G:].any()
    assert got[1, :, G:, 6].all() and int(got[1].sum()) == N * G


@pytest.mark.parametrize("B,N,Hq,Hkv,d,dt,L", [(600, 2, 4, 2, 128, "bf16", 40), (600, 3, 3, 1, 64, "f32", 9),
                                               (1, 4096, 1, 1, 128, "bf16", 70), (1, 4096, 4, 1, 64, "bf16", 33),
                                               (1, 4096, 2, 1, 128, "f32", 5)])
def test_large_batches_and_trees(B, N, Hq, Hkv, d, dt, L):
    """More sequences than the longest-first order takes, and the largest tree."""
    s = setup(B, N, Hq, Hkv, d, 16, [L - b % 5 for b in range(B)], True, dt, "star")
    out, lse = call(s, want_lse=True)
    check(s, out, lse)


@pytest.mark.parametrize("dt,d,Hq", [("bf16", 128, 8), ("bf16", 64, 6), ("f32", 64, 4)])
def test_a_cache_of_no_capacity(dt, d, Hq):
    """Lmax = 0: the tree attends to itself."""
    s = setup(2, 7, Hq, 2, d, 16, [0, 0], False, dt)
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    s["cache"] = tsd.Q8Cache(2, 2, d, Lmax=0, prefix_len=z)
    out, lse = call(s, want_lse=True)
    check(s, out, lse)


@pytest.mark.parametrize("N,Hq", [(1, 4), (5, 32), (13, 32), (20, 32), (14, 12)])
def test_the_last_wave_alone_is_split(N, Hq):
    """More row blocks than SMs: only the blocks of the shortest sequences are split and merged."""
    B, Hkv = 40, 4                                                 # 160 blocks on 148 SMs
    L = [int(x) for x in np.random.default_rng(4).integers(0, 900, B)]
    L[3], L[7] = 0, 1
    s = setup(B, N, Hq, Hkv, 128, 16, L, True, "bf16", cap=2000)
    launches, ctas = tsd.tree_verify_attn_q8_launches(s["cache"], N, Hq, 1 if s["q"].dtype == torch.bfloat16 else 0)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert launches == 1 and (sms >= B * Hkv or ctas > B * Hkv)
    ws = tsd.tree_verify_attn_q8_workspace(s["q"], s["cache"])
    for _ in range(2):
        out, lse = call(s, want_lse=True, workspace=ws)
        check(s, out, lse)
    assert not ws[:tsd.tree_verify_attn_ticket_bytes()].any()
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    status[3] = 9
    s["cache"].prefix_len[7] = s["cache"].capacity + 1             # both among the split ones
    out, _ = call(s, workspace=ws, status=status)
    assert not out[3].any() and not out[7].any() and (status[7].item() & 255) == 6
    check(s, out, None, skip=(3, 7))
    assert not ws[:tsd.tree_verify_attn_ticket_bytes()].any()


@pytest.mark.parametrize("merge", ["f", "k"])
@pytest.mark.parametrize("N,Hq,splits", [(6, 16, 3), (1, 8, 2), (40, 16, 2), (40, 16, 5)])
def test_either_merge_of_the_splits(N, Hq, splits, merge, monkeypatch):
    """Merged by the last CTA of a row block (f) or by the merge kernel (k)."""
    monkeypatch.setenv("TSD_ATTN_MERGE", merge)
    monkeypatch.setenv("TSD_ATTN_SPLITS", str(splits))
    s = setup(3, N, Hq, 2, 128, 16, [400, 3, 131], True, "bf16")
    ws = torch.zeros(tsd.tree_verify_attn_ticket_bytes() + 3 * 2 * 8 * 8 * N * 130 * 4, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        out, lse = call(s, want_lse=True, workspace=ws)
        check(s, out, lse)
    assert not ws[:tsd.tree_verify_attn_ticket_bytes()].any()


@pytest.mark.parametrize("B,N,Hq,Hkv,L,paged,kind", [
    (2, 1, 3, 1, [200, 65], True, "chain"), (2, 9, 14, 2, [129, 700], True, "rand"), (1, 4, 14, 2, [0], False, "rand"),
    (3, 50, 6, 2, [64, 0, 333], True, "forest"), (2, 40, 7, 1, [500, 31], False, "rand"), (1, 130, 6, 2, [77], True, "star"),
    (2, 21, 12, 2, [90, 256], True, "rand"), (1, 3, 100, 1, [150], True, "chain"), (2, 2, 127, 1, [64, 63], True, "chain"),
    (1, 5, 48, 1, [513], True, "chain"), (1, 512, 3, 1, [300], True, "star"), (2, 60, 10, 2, [1000, 999], True, "forest")])
@pytest.mark.parametrize("splits", [0, 3])
def test_any_group_size(B, N, Hq, Hkv, L, paged, kind, splits, monkeypatch):
    """Groups that do not divide a query tile: its last rows stay empty."""
    s = setup(B, N, Hq, Hkv, 128, 16, L, paged, "bf16", kind, nodes=[max(1, N - 3 * b) for b in range(B)])
    ws = torch.zeros(tsd.tree_verify_attn_ticket_bytes() + B * Hkv * 32 * (Hq // Hkv) * N * 130 * 4, dtype=torch.uint8,
                     device="cuda")
    if splits:
        monkeypatch.setenv("TSD_ATTN_SPLITS", str(splits))
    for merge in ("k", "f"):
        monkeypatch.setenv("TSD_ATTN_MERGE", merge)
        out, lse = call(s, out=torch.full_like(s["q"], 5.0), want_lse=True, workspace=ws)
        check(s, out, lse)
        for b, n in enumerate(s["nodes"]):
            assert (out[b, n:] == 5).all()


@pytest.mark.parametrize("N,Hq,d,dt", [(5, 16, 128, "bf16"), (40, 16, 128, "bf16"), (12, 6, 64, "bf16"), (5, 4, 64, "f32")])
def test_an_infinite_query_gives_nan(N, Hq, d, dt):
    """Scores of both infinities: the row is NaN, as in the formula, and no other is touched."""
    s = setup(2, N, Hq, 2, d, 16, [300, 90], True, dt)
    want, _ = call(s)
    s["q"][0, 1, 0, 3], s["q"][1, 2, 1, 0] = float("inf"), -float("inf")
    out, _ = call(s)
    assert out[0, 1, 0].isnan().all() and out[1, 2, 1].isnan().all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[0, 1, 0] = keep[1, 2, 1] = False
    assert torch.equal(out[keep], want[keep])


@pytest.mark.parametrize("N,Hq,d,dt", [(5, 16, 128, "bf16"), (40, 16, 128, "bf16"), (1, 4, 128, "bf16"), (12, 6, 64, "bf16"),
                                       (5, 4, 64, "f32")])
def test_scores_that_underflow(N, Hq, d, dt):
    """All-zero query rows, all-zero K blocks and tiny scales: every visible key has the same weight, and a masked
    one none (its score is -inf, never -inf times a factor that underflowed)."""
    B, Hkv, bs, L = 2, 2, 16, [150, 70]
    s = setup(B, N, Hq, Hkv, d, bs, L, True, dt)
    ref = make(B, Hkv, d, bs, [0, 0], max(L) + 3, True)
    rng = np.random.default_rng(8)
    for b in range(B):
        k = rng.normal(size=(L[b], Hkv, d))
        k[64:] = 0                                                 # the last, partly filled tile
        ref.write(b, k, rng.normal(size=(L[b], Hkv, d)))
    ref.prefix = np.array(L)
    s["ref"], s["cache"] = ref, to_gpu(ref, True, max(L) + 3)
    s["q"][:, :, ::2] = 0
    for scale in (0.1, 1e-4, 1e-12, 1e-38):
        out, lse = call(s, want_lse=True, scale=scale)
        check(s, out, lse, scale=scale)
