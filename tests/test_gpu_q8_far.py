"""Pages and rows behind the first 2^32 bytes of a cache: the same bits as in a small one."""
import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def serve(cache, rows, q, kt, vt, ps, D, acc):
    """Prompt, verify, commit, verify, read back."""
    assert not tsd.kv_q8_append(cache, rows, -rows).any()
    out0, lse0 = tsd.tree_verify_attn_q8(q, cache, kt, vt, ps, None, D, want_lse=True)
    assert not tsd.kv_q8_commit(cache, kt, vt, None, acc, Dmax=D, mode="length").any()
    out1, lse1 = tsd.tree_verify_attn_q8(q, cache, kt, vt, ps, None, D, want_lse=True)
    k, v = tsd.kv_q8_read(cache, num_rows=cache.prefix_len.clone(), S=int(cache.prefix_len.max()), dtype=rows.dtype)
    return [out0, lse0, out1, lse1, k, v, cache.prefix_len.clone()]


def inputs(d, dt, N):
    g = torch.Generator(device="cuda").manual_seed(d + N)
    t = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dt])  # noqa: E731
    parent = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").clamp(max=3).repeat(2, 1)
    ps = tsd.tree_prepare(parent, None, 5)["parent_s"]
    return t(2, 333, 8, d), t(2, N, 16, d), t(2, N, 8, d), t(2, N, 8, d), ps, 5, torch.tensor([2, 0], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,dt,N", [(128, "bf16", 5), (128, "bf16", 80), (64, "bf16", 5), (128, "f32", 5)])
def test_far_pages(d, dt, N):
    bs, Hkv, per = 16, 8, 24
    pages = (1 << 32) // (Hkv * bs * d) + 3 * per
    near = torch.arange(2 * per, dtype=torch.int32, device="cuda").view(2, per)
    far = pages - 1 - near.flip(1)
    x = inputs(d, dt, N)
    want = serve(tsd.Q8Cache(2, Hkv, d, num_blocks=2 * per, block_table=near, block_size=bs), *x)
    got = serve(tsd.Q8Cache(2, Hkv, d, num_blocks=pages, block_table=far, block_size=bs), *x)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,dt,N", [(128, "bf16", 5), (64, "bf16", 5), (128, "f32", 5)])
def test_far_sequences(d, dt, N):
    """Contiguous: the second sequence starts past 2^31 codes (the splits are planned for the capacity, so each
    element is held to the rounding of its type)."""
    Hkv, L = 8, (1 << 31) // (8 * d) + 7
    x = inputs(d, dt, N)
    want = serve(tsd.Q8Cache(2, Hkv, d, Lmax=512, block_size=16), *x)
    got = serve(tsd.Q8Cache(2, Hkv, d, Lmax=L, block_size=16), *x)
    for a, b in zip(got[4:], want[4:]):
        assert torch.equal(a, b)
    for a, b in zip(got[:4], want[:4]):
        # (the same values summed in other groups: P to 8 bits and the output's rounding in bf16, sums in fp32)
        half = 2.0 ** -24 * 512 if a.dtype == torch.float32 else 2.0 ** -8
        assert ((a.float() - b.float()).abs() <= 4 * half * b.float().abs().clamp(min=0.25)).all()
