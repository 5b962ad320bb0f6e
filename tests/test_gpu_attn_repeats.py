"""An attention call repeats itself bit for bit, also where the last CTA of a row block merges its splits: the
order in which they arrive is not the order of the sum."""
import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd
from test_gpu_q8_attn import call, check, setup

pytestmark = pytest.mark.gpu


def _repeat(run, n=25):
    out, lse = run()
    want, want_lse = out.clone(), lse.clone()
    for _ in range(n):
        out, lse = run()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)
    return want, want_lse


@pytest.mark.parametrize("B,N,Hq,Hkv,L,splits", [(16, 60, 32, 8, 900, 0), (16, 60, 32, 8, 900, 5), (4, 6, 32, 4, 700, 4),
                                                 (5, 1, 8, 8, 600, 3), (40, 5, 32, 4, 900, 0)])
def test_q8_attention_repeats(B, N, Hq, Hkv, L, splits, monkeypatch):
    s = setup(B, N, Hq, Hkv, 128, 16, [L - 17 * (b % 7) for b in range(B)], True, "bf16", cap=2 * L)
    ws = tsd.tree_verify_attn_q8_workspace(s["q"], s["cache"])
    if splits:
        monkeypatch.setenv("TSD_ATTN_SPLITS", str(splits))
        monkeypatch.setenv("TSD_ATTN_MERGE", "f")
        need = tsd.tree_verify_attn_ticket_bytes() + B * Hkv * splits * (Hq // Hkv) * N * 130 * 4
        ws = torch.zeros(max(need, ws.numel()), dtype=torch.uint8, device="cuda")
    out, lse = _repeat(lambda: call(s, want_lse=True, workspace=ws))
    check(s, out, lse, skip=range(2, B))


@pytest.mark.parametrize("splits", [2, 3, 5])
@pytest.mark.parametrize("N,Hq,Hkv", [(60, 32, 8), (6, 32, 8), (26, 16, 4)])
def test_attention_repeats(N, Hq, Hkv, splits, monkeypatch):
    B, d, L = 16, 128, 900
    monkeypatch.setenv("TSD_ATTN_SPLITS", str(splits))
    monkeypatch.setenv("TSD_ATTN_MERGE", "f")
    t = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(N)
    q, k, v, kt, vt = t(B, N, Hq, d), t(B, Hkv, L, d), t(B, Hkv, L, d), t(B, N, Hkv, d), t(B, N, Hkv, d)
    parent = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").clamp(max=5).repeat(B, 1)
    prep = tsd.tree_prepare(parent, None, 8)
    assert not prep["status"].any()
    L_b = torch.full((B,), L, dtype=torch.int32, device="cuda")
    ws = torch.zeros(tsd.tree_verify_attn_ticket_bytes() + B * Hkv * splits * (Hq // Hkv) * N * 130 * 4,
                     dtype=torch.uint8, device="cuda")
    _repeat(lambda: tsd.tree_verify_attn(q, k, v, L_b, kt, vt, prep["parent_s"], None, 8, workspace=ws, want_lse=True))
    assert not ws[:tsd.tree_verify_attn_ticket_bytes()].any()
