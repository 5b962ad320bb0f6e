"""8-bit cache on the GPU: append, commit and read against the 64-bit reference.  Codes and scales are
compared exactly: every step of the format (a power-of-two scale, one rounding to e4m3) is defined to
the bit, so there is no tolerance."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd
from q8_ref import Cache, TABLE

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(B, Hkv, d, bs, L, cap, paged, seed=0, junk=True):
    """A cache with rows already committed (through the reference) and junk behind them."""
    rng = np.random.default_rng(seed)
    nb = -(-cap // bs)
    pages = B * nb + 3
    table = rng.permutation(pages)[:B * nb].reshape(B, nb).astype(np.int32)
    if not paged:
        table, pages = np.arange(B * nb, dtype=np.int32).reshape(B, nb), B * nb
    shape = (pages, Hkv, bs, d)
    code = [np.full(shape, 0x7f, np.uint8) if junk else np.zeros(shape, np.uint8) for _ in range(2)]
    sc = [np.full(shape[:2], 255, np.uint8) for _ in range(2)]
    ref = Cache(code[0], code[1], sc[0], sc[1], table, np.zeros(B, np.int64), bs)
    for b in range(B):
        if L[b]:
            ref.write(b, rng.normal(size=(L[b], Hkv, d)) * 0.3, rng.normal(size=(L[b], Hkv, d)) * 5)
    ref.prefix = np.array(L)
    return ref


def to_gpu(ref, paged, cap, device="cuda"):
    """The reference cache as a Q8Cache (the contiguous layout holds cap positions of each sequence)."""
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    pl = t(ref.prefix.astype(np.int32))
    if paged:
        return tsd.Q8Cache.wrap(t(ref.code["k"]), t(ref.code["v"]), t(ref.scale["k"]), t(ref.scale["v"]), pl, ref.bs,
                                t(ref.table))
    B, nb = ref.table.shape
    def lay(c):
        P, H, bs, d = c.shape
        return t(c.reshape(B, nb, H, bs, d).transpose(0, 2, 1, 3, 4).reshape(B, H, nb * bs, d)[:, :, :cap])
    def scl(s):
        return t(s.reshape(B, nb, -1).transpose(0, 2, 1))
    return tsd.Q8Cache.wrap(lay(ref.code["k"]), lay(ref.code["v"]), scl(ref.scale["k"]), scl(ref.scale["v"]), pl, ref.bs)


def check_cache(cache, ref, paged, cap):
    for name, code, sc in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        c, s = ref.code[name], ref.scale[name]
        if not paged:
            B, nb = ref.table.shape
            P, H, bs, d = c.shape
            c = c.reshape(B, nb, H, bs, d).transpose(0, 2, 1, 3, 4).reshape(B, H, nb * bs, d)[:, :, :cap]
            s = s.reshape(B, nb, H).transpose(0, 2, 1)
        got = code.view(torch.uint8).cpu().numpy()
        assert np.array_equal(sc.cpu().numpy(), s), name
        assert np.array_equal(TABLE[got], TABLE[c], equal_nan=True), name


SHAPES = [
    # B, Hkv, d, bs, S, lengths, paged, type
    (1, 1, 64, 8, 1, [0], True, "bf16"),
    (1, 8, 128, 16, 1, [15], True, "bf16"),
    (2, 3, 128, 16, 5, [13, 32], False, "bf16"),
    (3, 2, 64, 32, 33, [0, 31, 64], True, "f32"),
    (2, 2, 128, 64, 130, [1, 63], True, "bf16"),
    (2, 1, 128, 256, 300, [255, 17], False, "f32"),
    (2, 4, 128, 256, 600, [3, 256], True, "bf16"),
    (4, 8, 128, 16, 97, [0, 7, 16, 33], True, "bf16"),
]


def rows_np(x):
    return x.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("B,Hkv,d,bs,S,L,paged,dt", SHAPES)
def test_append(B, Hkv, d, bs, S, L, paged, dt):
    cap = max(L) + S + 5
    ref = make(B, Hkv, d, bs, L, cap, paged)
    cap = ref.table.shape[1] * bs if paged else cap
    cache = to_gpu(ref, paged, cap)
    g = torch.Generator(device="cuda").manual_seed(1)
    # tokens of unlike sizes: scales grow inside a block and from call to call
    size = torch.exp2(torch.randint(-12, 13, (B, S, Hkv, 1), generator=g, device="cuda").float())
    k, v = ((torch.randn(B, S, Hkv, d, generator=g, device="cuda") * size).to(DT[dt]) for _ in range(2))
    n = torch.tensor([max(0, S - 3 * b) for b in range(B)], dtype=torch.int32, device="cuda")
    status = tsd.kv_q8_append(cache, k, v, n, advance=False)
    assert not status.any() and cache.prefix_len.tolist() == L
    for b in range(B):
        ref.write(b, rows_np(k[b, :n[b]]), rows_np(v[b, :n[b]]))
    check_cache(cache, ref, paged, cap)
    # a second call that advances: the same rows again give the same cache (scales never shrink)
    tsd.kv_q8_append(cache, k, v, n, advance=True)
    assert cache.prefix_len.tolist() == [a + c for a, c in zip(L, n.tolist())]
    check_cache(cache, ref, paged, cap)


def test_append_special_values():
    """Infinities saturate, NaN stays NaN, neither sets the scale; an all-zero block has the smallest
    scale; fp32 values at the ends of the range; ties go to the even code."""
    d, bs = 64, 8
    cache = tsd.Q8Cache(1, 1, d, Lmax=64, block_size=bs)
    ref = make(1, 1, d, bs, [0], 64, False, junk=False)
    x = torch.zeros(1, 40, 1, d, device="cuda")
    x[0, 0, 0, 0], x[0, 1, 0, 1], x[0, 2, 0, 2], x[0, 3, 0, 3] = float("inf"), float("-inf"), float("nan"), 1.75
    x[0, 8:16] = 0.0
    x[0, 16, 0, 0], x[0, 17, 0, 1] = 3.0e38, -1.0e-38
    x[0, 24:32, 0] = torch.arange(8 * d, device="cuda").view(8, d) / 16.0       # many ties
    x[0, 32:, 0] = 1e-30
    tsd.kv_q8_append(cache, x, -x)
    ref.write(0, rows_np(x[0]), rows_np(-x[0]))
    ref.scale["k"][5:], ref.scale["v"][5:] = 127, 127                           # blocks not written
    check_cache(cache, ref, False, 64)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["path", "length"])
def test_commit(paged, dt, mode):
    B, Hkv, d, bs, N, D, cap = 6, 2, 128, 16, 9, 4, 96
    L = [0, 15, 16, 31, 40, 90]
    ref = make(B, Hkv, d, bs, L, cap, paged)
    cache = to_gpu(ref, paged, cap)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = ((torch.randn(B, N, Hkv, d, generator=g, device="cuda") * 9).to(DT[dt]) for _ in range(2))
    path = torch.tensor([[1, 2, 4, 7, 9], [1, 3, 5, 0, 0], [1, 0, 0, 0, 0], [1, 2, 6, 8, 0], [7, 7, 7, 0, 0],
                         [1, 2, 3, 4, 5]], dtype=torch.int32, device="cuda")
    acc = torch.tensor([4, 2, 0, 3, 2, -1], dtype=torch.int32, device="cuda")   # the last: a miss
    status = tsd.kv_q8_commit(cache, k, v, path if mode == "path" else None, acc, Dmax=D, mode=mode)
    assert not status.any()
    for b in range(B):
        n = int(acc[b]) + 1
        src = [int(path[b, j]) - 1 if mode == "path" else j for j in range(n)]
        ref.write(b, rows_np(k[b, src]), rows_np(v[b, src]))
    check_cache(cache, ref, paged, cap)
    assert cache.prefix_len.tolist() == [a + int(c) + 1 for a, c in zip(L, acc.tolist())]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d,bs", [(64, 8), (128, 16), (128, 256)])
def test_read(paged, dt, d, bs):
    B, Hkv, S = 4, 3, 40
    L = [0, 40, 77, 300]
    ref = make(B, Hkv, d, bs, L, 300, paged)
    cache = to_gpu(ref, paged, 300)
    start = torch.tensor([0, 0, 37, 255], dtype=torch.int32, device="cuda")
    n = torch.tensor([0, 40, 39, 40], dtype=torch.int32, device="cuda")
    k, v = (torch.full((B, S, Hkv, d), 7.0, dtype=DT[dt], device="cuda") for _ in range(2))
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    tsd.kv_q8_read(cache, start, n, k_out=k, v_out=v, status=status)
    assert not status.any()
    for b in range(B):
        rk, rv = ref.rows(b, int(start[b]), int(start[b] + n[b]))
        m = int(n[b])
        assert np.array_equal(rows_np(k[b, :m]), rk) and np.array_equal(rows_np(v[b, :m]), rv)
        assert (k[b, m:] == 7).all() and (v[b, m:] == 7).all()                  # rows behind stay
    k2, _ = tsd.kv_q8_read(cache, S=0)
    assert k2.shape == (B, 0, Hkv, d)


def test_errors_leave_the_cache_untouched():
    B, Hkv, d, bs, S = 5, 2, 64, 16, 20
    L = [10, 10, 10, 10, 10]
    ref = make(B, Hkv, d, bs, L, 48, True)
    ref.table[1, 1] = ref.code["k"].shape[0]        # a block id past the pool
    ref.prefix[2] = 30                              # 30 + 20 > 48
    cache = to_gpu(ref, True, 48)
    before = [t.view(torch.uint8).clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    x = torch.randn(B, S, Hkv, d, device="cuda").bfloat16()
    n = torch.tensor([-1, S, S, S + 1, S], dtype=torch.int32, device="cuda")
    status = torch.tensor([0, 0, 0, 0, 3], dtype=torch.int32, device="cuda")    # the last: flagged on entry
    tsd.kv_q8_append(cache, x, x, n, status=status)
    assert [s & 255 for s in status.tolist()] == [1, 6, 6, 1, 3]
    for t, w in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        assert torch.equal(t.view(torch.uint8), w)
    assert cache.prefix_len.tolist() == [10, 10, 30, 10, 10]
    # commit: a path entry of 0 and past the nodes, accept_len past Dmax and past the nodes
    path = torch.tensor([[1, 0, 0], [1, 2, 9], [1, 2, 3], [1, 2, 3], [1, 2, 3]], dtype=torch.int32, device="cuda")
    acc = torch.tensor([1, 2, 3, 2, 1], dtype=torch.int32, device="cuda")
    nodes = torch.tensor([8, 8, 8, 2, 8], dtype=torch.int32, device="cuda")
    status.zero_()
    ref.table[1, 1] = 0
    cache.block_table.copy_(torch.from_numpy(ref.table))
    status[4] = 7
    tsd.kv_q8_commit(cache, x[:, :8].contiguous(), x[:, :8].contiguous(), path, acc, nodes, Dmax=2, status=status)
    assert [s & 255 for s in status.tolist()] == [1, 1, 1, 1, 7]
    for t, w in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        assert torch.equal(t.view(torch.uint8), w)
    # read: rows past the prefix, a negative start, a bad block; flagged rows are zero
    status.zero_()
    cache.block_table[3, 0] = -1
    start = torch.tensor([0, -1, 20, 0, 0], dtype=torch.int32, device="cuda")
    rows = torch.tensor([11, 4, 10, 10, 10], dtype=torch.int32, device="cuda")
    k, v = (torch.ones(B, S, Hkv, d, device="cuda") for _ in range(2))
    tsd.kv_q8_read(cache, start, rows, k_out=k, v_out=v, status=status)
    assert [s & 255 for s in status.tolist()] == [6, 1, 0, 6, 0]
    for b, m in ((0, 11), (1, 4), (3, 10)):
        assert not k[b, :m].any() and not v[b, :m].any() and (k[b, m:] == 1).all()


def test_captured_append_follows_prefix_len():
    """A decode loop captured once: every replay appends behind the rows the last one wrote."""
    B, Hkv, d, bs = 2, 2, 128, 16
    ref = make(B, Hkv, d, bs, [0, 11], 64, True)
    cache = to_gpu(ref, True, 64)
    x = torch.zeros(B, 1, Hkv, d, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            tsd.kv_q8_append(cache, x, x, status=status)
    torch.cuda.synchronize()
    for step in range(20):
        x.copy_(torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(step)) * (step + 1))
        g.replay()
        torch.cuda.synchronize()
        for b in range(B):
            ref.write(b, rows_np(x[b]), rows_np(x[b]))
        ref.prefix = ref.prefix + 1
    assert not status.any() and cache.prefix_len.tolist() == [20, 31]
    check_cache(cache, ref, True, 64)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bs", [16, 64])
def test_the_largest_floats_stay_finite(dt, bs):
    """Rows up to the type's largest value: the nearest finite multiple of the scale comes back, also beside
    infinities and as committed rows of a block whose scale grows to the largest."""
    d, big = 128, torch.finfo(DT[dt]).max
    cache = tsd.Q8Cache(1, 1, d, Lmax=2 * bs, block_size=bs)
    x = torch.zeros(1, 3, 1, d)
    x[0, 0, 0, :4] = torch.tensor([2.0 ** 119, -1.5 * 2.0 ** 119, 448 * 2.0 ** 110, 1.0])
    x[0, 1, 0, :9] = torch.tensor([big, -big, 1.75 * 2.0 ** 127, 1.8125 * 2.0 ** 127, 1.9 * 2.0 ** 127, float("inf"),
                                   float("-inf"), float("nan"), -2.0 ** 126])
    x[0, 2, 0, :2] = torch.tensor([1.9375 * 2.0 ** 127, 2.0 ** 120])
    x = x.to(DT[dt]).cuda()
    tsd.kv_q8_append(cache, x[:, :1].contiguous(), x[:, :1].contiguous())
    assert cache.k_scale[0, 0, 0] < 247
    tsd.kv_q8_append(cache, x[:, 1:].contiguous(), x[:, 1:].contiguous())
    assert cache.k_scale[0, 0, 0] == 247 and cache.v_scale[0, 0, 0] == 247
    top, u = 240.0, 2.0 ** 120
    want = torch.zeros(3, d, dtype=torch.float64)
    want[0, :3] = torch.tensor([0.5, -0.75, 448 * 2.0 ** -10]) * u     # (the third and fourth: e4m3's own steps)
    want[1, :9] = torch.tensor([top, -top, 224, 224, 240, top, -top, float("nan"), -64]).double() * u
    want[2, :2] = torch.tensor([top, 1.0]).double() * u
    for out_dt in (torch.bfloat16, torch.float32):
        for got in tsd.kv_q8_read(cache, S=3, dtype=out_dt):
            got = got[0, :, 0].double().cpu()
            assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0)), (got[:, :9] / u, want[:, :9] / u)
