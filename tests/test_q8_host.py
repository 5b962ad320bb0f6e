"""8-bit cache and sampling without a GPU: the reference's format against torch's float8, and every
host-side refusal of the C calls and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd
from q8_ref import TABLE, encode, sample, scale_byte


def test_reference_format_is_torch_e4m3():
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(vals, TABLE, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 100, rng.normal(size=4000) * 2.0 ** -8,
                        np.arange(-448, 449, 0.5), [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = np.clip(x, -448, 448)
    want = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(TABLE[encode(x)], TABLE[want])
    assert np.isnan(TABLE[encode(np.array([np.nan]))]).all()
    assert np.array_equal(TABLE[encode(np.array([np.inf, -np.inf]))], [448.0, -448.0])


def test_reference_scale():
    assert scale_byte(np.zeros(3)) == 87
    assert scale_byte(np.array([448.0])) == 127 and scale_byte(np.array([448.01])) == 128
    assert scale_byte(np.array([224.0, -225.0])) == 127 and scale_byte(np.array([np.inf, 1.75, np.nan])) == 119


def test_reference_sampler():
    z = np.array([1.0, 3.0, 3.0, 2.0])
    assert sample(z, 0.0, 0, 1.0, 0.0, 0.9)[0] == 1                  # greedy: lowest id of the maximum
    assert sample(z, 1.0, 1, 1.0, 0.0, 0.99)[0] == 1                 # top-1 breaks the tie downward
    assert sample(z, 1.0, 0, 1e-9, 0.0, 0.99)[0] == 1
    assert sample(z, 1.0, 0, 1.0, 1.0, 0.99)[0] == 2                 # min-p 1 keeps both maxima
    assert sample(np.array([np.nan, -np.inf]), 1.0, 0, 1.0, 0.0, 0.3)[:2] == (0, 0.0)


def _desc(**kw):
    f = dict(k=None, v=None, k_scale=None, v_scale=None, prefix_len=None, Lmax=64, block_table=None, max_blocks=0,
             block_size=16, num_blocks=0)
    f.update(kw)
    return tsd.Q8CacheDesc(*[f[n] for n, _ in tsd.Q8CacheDesc._fields_])


@pytest.fixture
def mem():
    buf = ctypes.create_string_buffer(1 << 12)
    base = (ctypes.addressof(buf) + 255) & ~255
    yield base, buf


def test_cache_calls_refuse_bad_arguments_before_any_launch(mem):
    L, p, R = tsd.lib(), ctypes.c_void_p(mem[0]), ctypes.byref
    full = dict(k=p, v=p, k_scale=p, v_scale=p, prefix_len=p)
    ok = _desc(**full)

    def append(c=ok, k=p, v=p, n=None, B=1, S=4, H=2, d=64, dt=1, adv=1, st=p):
        return L.tsd_kv_q8_append(R(c) if c else None, k, v, n, B, S, H, d, dt, adv, st, None)

    def commit(c=ok, k=p, path=p, acc=p, B=1, N=4, H=2, d=64, D=3, dt=1, mode=0, adv=1, st=p):
        return L.tsd_kv_q8_commit(R(c) if c else None, k, p, path, acc, None, B, N, H, d, D, dt, mode, adv, st, None)

    def read(c=ok, ko=p, B=1, S=4, H=2, d=64, dt=1, st=p):
        return L.tsd_kv_q8_read(R(c) if c else None, None, None, ko, p, B, S, H, d, dt, st, None)

    odd = ctypes.c_void_p(mem[0] + 4)
    for call in (append, commit, read):
        assert call(c=None) == 1
        assert call(dt=5) == 2
        assert call(d=96) == 1 and call(H=0) == 1 and call(B=-1) == 1 and call(B=70000) == 1
        assert call(B=0) == 0                                                     # an empty batch
        assert call(st=None) == 1
        for bs in (0, 4, 12, 512):
            assert call(c=_desc(**full, block_size=bs)) == 1
        assert call(c=_desc(**{**full, "k": odd})) == 1 and call(c=_desc(**{**full, "k_scale": None})) == 1
        assert call(c=_desc(**{**full, "prefix_len": None})) == 1 and call(c=_desc(**full | {"Lmax": -1})) == 1
        assert call(c=_desc(**full, block_table=p, max_blocks=1 << 28, num_blocks=4)) == 1   # over 2^31 positions
    assert append(k=odd) == 1 and append(k=None) == 1 and append(S=-1) == 1 and append(S=0) == 0 and append(adv=2) == 1
    assert commit(k=odd) == 1 and commit(path=None) == 1 and commit(acc=None) == 1 and commit(D=256) == 1
    assert commit(mode=2) == 1                                                    # no in-place mode
    assert read(ko=odd) == 1 and read(ko=None) == 1 and read(S=-1) == 1


def test_attention_refuses_bad_arguments_before_any_launch(mem):
    L, p, R = tsd.lib(), ctypes.c_void_p(mem[0]), ctypes.byref
    odd = ctypes.c_void_p(mem[0] + 4)
    full = dict(k=p, v=p, k_scale=p, v_scale=p, prefix_len=p)

    def call(c=_desc(**full), q=p, kt=p, vt=p, ps=p, B=1, N=4, Hq=8, H=2, d=64, D=3, dt=1, out=p, ws=p, nb=1 << 30,
             st=p, scale=0.1):
        return L.tsd_tree_verify_attn_q8(q, R(c) if c else None, kt, vt, ps, None, B, N, Hq, H, d, D, dt, scale, out,
                                         None, ws, nb, st, None)

    assert call(c=None) == 1 and call(dt=3) == 2 and call(d=32) == 1 and call(Hq=9) == 1 and call(N=5000) == 1
    assert call(B=0) == 0 and call(N=0) == 0
    assert call(q=None) == 1 and call(q=odd) == 1 and call(out=odd) == 1 and call(ps=None) == 1 and call(st=None) == 1
    assert call(kt=None, vt=None) == 1 and call(vt=None) == 1     # the tree K/V are required
    assert call(c=_desc(**{**full, "v_scale": None})) == 1 and call(c=_desc(**{**full, "v": odd})) == 1
    assert call(scale=0.0) == 1 and call(scale=-1.0) == 1 and call(scale=float("nan")) == 1
    long = _desc(**full | {"Lmax": 8192})
    need = L.tsd_tree_verify_attn_q8_workspace_size(R(long), 1, 26, 32, 8, 128, 1)
    assert need > 65536
    assert call(c=long, N=26, Hq=32, H=8, d=128, nb=need - 1) == 9
    assert call(c=long, N=26, Hq=32, H=8, d=128, ws=odd) == 9 and call(c=long, N=26, Hq=32, H=8, d=128, ws=None) == 9
    for bad in ((0, 26, 32, 8), (1, 0, 32, 8), (1, 26, 33, 8), (1, 26, 32, 0)):
        assert L.tsd_tree_verify_attn_q8_workspace_size(R(long), *bad, 128, 1) == 0
    assert L.tsd_tree_verify_attn_q8_workspace_size(None, 1, 26, 32, 8, 128, 1) == 0


def test_sampler_refuses_bad_arguments_before_any_launch(mem):
    L, p = tsd.lib(), ctypes.c_void_p(mem[0])

    def call(z=p, dt=1, R=2, V=100, u=p, tok=p):
        return L.tsd_sample_rows(z, dt, R, V, u, None, None, None, None, tok, None, None)

    assert call(dt=9) == 2 and call(R=-1) == 1 and call(V=0) == 1 and call(R=0) == 0
    assert call(z=None) == 1 and call(u=None) == 1 and call(tok=None) == 1
    assert call(V=8 * 81920 + 8) == 1 and call(dt=0, V=8 * 40960 + 8) == 1        # a slice over 160 KiB


def test_binding_checks_shapes_and_types():
    z8 = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    sc = torch.zeros(4, 2, dtype=torch.uint8)
    pl = torch.zeros(2, dtype=torch.int32)
    bt = torch.zeros(2, 3, dtype=torch.int32)
    W = tsd.Q8Cache.wrap
    for bad in (lambda: W(z8.float(), z8.float(), sc, sc, pl, 16, bt), lambda: W(z8, z8[:, :1], sc, sc, pl, 16, bt),
                lambda: W(z8, z8, sc.int(), sc, pl, 16, bt), lambda: W(z8, z8, sc[:, :1], sc, pl, 16, bt),
                lambda: W(z8, z8, sc, sc, pl, 32, bt), lambda: W(z8, z8, sc, sc, pl, 16, bt[:1]),
                lambda: W(z8, z8, sc, sc, pl, 16), lambda: tsd.Q8Cache(2, 2, 64, Lmax=8, num_blocks=3),
                lambda: tsd.Q8Cache(2, 2, 64), lambda: tsd.Q8Cache(2, 2, 64, num_blocks=3, device="cpu"),
                lambda: W(z8, z8, sc, sc, pl, 16, bt)):            # CPU tensors reach no kernel
        with pytest.raises(tsd.TsdError):
            bad()


def test_binding_refuses_block_sizes():
    for bs in (0, -16, 4, 12, 24, 512):
        with pytest.raises(tsd.TsdError):
            tsd.Q8Cache(2, 2, 64, Lmax=64, block_size=bs, device="cpu")
        with pytest.raises(tsd.TsdError):
            tsd.Q8Cache.wrap(None, None, None, None, torch.zeros(2, dtype=torch.int32), bs)
