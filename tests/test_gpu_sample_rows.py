"""tsd_sample_rows against the 64-bit reference.

Tolerances.  A weight is held in units of 2^-sh, sh = min(51, 62 - ceil(log2 V)), so it is off by at most
2^-(sh+1), and by its polynomial's 2^-48 relative, and a sum of V of them by V 2^-(sh+1) + Z 2^-48.  A draw whose u Z lies nearer than that to a border may go to
either side; every other token has to be equal.  A probability w / Z is then off by the same over w, plus
one fp32 rounding (2^-24 relative)."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_06_b200 as tsd
from q8_ref import sample

pytestmark = pytest.mark.gpu


def run_and_check(z, u, T=None, k=None, P=None, m=None):
    R, V = z.shape
    dev = lambda a, t: None if a is None else torch.tensor(np.asarray(a), dtype=t, device="cuda")  # noqa: E731
    r = tsd.sample_rows(z, dev(u, torch.float32), dev(T, torch.float32), dev(k, torch.int32), dev(P, torch.float32),
                        dev(m, torch.float32))
    tok, pr = r["tokens"].cpu().numpy(), r["probs"].cpu().numpy()
    zz = z.float().cpu().numpy()
    f = lambda a, i, d: d if a is None else np.float32(a[i])  # noqa: E731
    off = V * 2.0 ** -(1 + min(51, 62 - math.ceil(math.log2(V)))) + 2.0 ** -47
    for i in range(R):
        t, p, margin = sample(zz[i], f(T, i, 1.0), 0 if k is None else k[i], f(P, i, 1.0), f(m, i, 0.0),
                              np.float32(u[i]))
        if margin > 2 * off:
            assert tok[i] == t, (i, tok[i], t, margin)
            assert abs(pr[i] - p) <= p * 2.0 ** -24 + 2 * off, (i, pr[i], p)
    return tok, pr


@pytest.mark.parametrize("V", [1, 2, 31, 100, 1000, 32000, 50257, 128256])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_every_filter(V, dt):
    R = 24
    rng = np.random.default_rng(V)
    z = torch.tensor(rng.normal(size=(R, V)) * 2.5, dtype=torch.float32, device="cuda").to(dt)
    T = rng.uniform(0.3, 1.6, R)
    k = np.where(rng.random(R) < 0.5, 0, rng.integers(1, 2 * V + 1, R) % 5000)
    P = np.where(rng.random(R) < 0.4, 1.0, rng.uniform(0.05, 0.999, R))
    m = np.where(rng.random(R) < 0.6, 0.0, rng.uniform(0, 0.3, R))
    u = rng.random(R).astype(np.float32)
    u[0], u[1] = 0.0, np.float32(1 - 2.0 ** -24)
    T[2], T[3] = 0.0, -1.0
    run_and_check(z, u, T, k, P, m)
    run_and_check(z, u)                              # no parameters: the plain softmax
    run_and_check(z, u, T=T)
    run_and_check(z, u, k=np.full(R, min(V, 7)))
    run_and_check(z, u, P=np.full(R, 0.9))
    run_and_check(z, u, m=np.full(R, 0.05))


def test_ties_and_flat_rows():
    """Equal logits: borders inside a run of ties keep the lowest ids; a flat row spreads evenly."""
    V = 4099
    rng = np.random.default_rng(5)
    z = np.zeros((8, V), np.float32)
    z[1] = rng.integers(0, 3, V)
    z[2] = rng.integers(0, 40, V) / 4
    z[3, 17] = z[3, 4000] = 5.0
    z[4:] = rng.integers(0, 2, (4, V))
    zt = torch.tensor(z, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        for k, P in ((0, 0.5), (1, 1.0), (100, 1.0), (2050, 0.31), (2050, 0.999), (3, 0.2)):
            for u in (0.0, 0.37, 0.999999):
                run_and_check(zt.to(dt), np.full(8, u, np.float32), k=np.full(8, k), P=np.full(8, P), T=np.full(8, 0.7))


def test_masked_vocabularies():
    """-inf and NaN logits are never drawn, rows of nothing else give token 0, +inf shares the mass, and
    temperatures at both ends of the range stay finite."""
    V = 1000
    rng = np.random.default_rng(6)
    z = rng.normal(size=(9, V)).astype(np.float32) * 3
    z[0, rng.random(V) < 0.9] = -np.inf
    z[1, rng.random(V) < 0.9] = np.nan
    z[2] = -np.inf
    z[3] = np.nan
    z[4, [3, 700]] = np.inf
    z[5] = -3.3e38
    z[6] *= 1e37
    z[7, 1:] = -np.inf
    z[8] = np.where(rng.random(V) < 0.5, -3.38e38, z[8])
    for dt in (torch.float32, torch.bfloat16):
        zt = torch.tensor(z, device="cuda").to(dt)
        for T in (1.0, 1e-6, 1e-30, 1e4, 1e30):
            for k, P, m in ((0, 1.0, 0.0), (5, 0.9, 0.0), (0, 0.7, 0.02), (999, 0.99999, 0.0)):
                tok, pr = run_and_check(zt, rng.random(9), T=np.full(9, T), k=np.full(9, k), P=np.full(9, P), m=np.full(9, m))
                assert tok[2] == tok[3] == 0 and pr[2] == pr[3] == 0 and tok[7] == 0
                assert tok[4] in (3, 700)


def test_bad_uniforms_and_parameters_are_clamped():
    z = torch.randn(6, 333, device="cuda")
    nan = float("nan")
    u = torch.tensor([nan, -1.0, 2.0, 0.5, 0.5, 0.5], device="cuda")
    r = tsd.sample_rows(z, u, top_p=torch.tensor([1.0, 1, 1, 0, -3, 1], device="cuda"),
                        min_p=torch.tensor([0.0, 0, 0, 0, 0, 9], device="cuda"))
    top = z.argmax(1).tolist()
    tok = r["tokens"].tolist()
    assert tok[:3] == [0, 0, 332] and tok[3:] == top[3:]


def test_odd_row_starts():
    """A view that starts off a 16-byte boundary, and odd vocabularies, take the scalar loads."""
    for dt in (torch.bfloat16, torch.float32):
        base = torch.randn(3 * 5001 + 1, device="cuda").to(dt)
        run_and_check(base[1:].view(3, 5001), [0.2, 0.6, 0.9], T=[1.0, 0.5, 0.7], k=[0, 50, 0], P=[0.9, 1.0, 0.8])


def test_captured_and_on_another_stream():
    z = torch.randn(5, 32000, device="cuda").bfloat16()
    u = torch.rand(5, device="cuda")
    T = torch.full((5,), 0.8, device="cuda")
    want = tsd.sample_rows(z, u, T)
    tok, pr = torch.zeros_like(want["tokens"]), torch.zeros_like(want["probs"])
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        tsd.sample_rows(z, u, T, tokens=tok, probs=pr)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(tok, want["tokens"]) and torch.equal(pr, want["probs"])
    z.copy_(torch.randn(5, 32000, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    again = tsd.sample_rows(z, u, T, stream=torch.cuda.current_stream())
    assert torch.equal(tok, again["tokens"])


def border_margin(z, T, k, P):
    """Distance of top-p's border to the nearest sum of masses, over the mass: nearer than the weights' own error,
    the border token may go to either side."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, np.float64))
    M = z.max()
    if not T > 0 or not P < 1 or M == -np.inf:
        return 1.0
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(z == M, 0.0, z - M) / np.float64(T))
    w = w[np.lexsort((np.arange(len(z)), -z))][:k if 0 < k < len(z) else len(z)]
    cum = np.cumsum(w)
    return float(np.abs(np.append(cum[:-1], 0.0) - np.float64(P) * cum[-1]).min() / cum[-1])


def check_clear_borders(z, u, T, k, P, m=None):
    """run_and_check of the rows whose top-p border is clear (all but a few)."""
    V = z.shape[1]
    off = V * 2.0 ** -(1 + min(51, 62 - math.ceil(math.log2(V)))) + 2.0 ** -47
    zz = z.float().cpu().numpy()
    ok = [i for i in range(len(zz)) if border_margin(zz[i], np.float32(T[i]), k[i], np.float32(P[i])) > 2 * off]
    assert len(ok) >= len(zz) - 1
    pick = lambda a: None if a is None else np.asarray(a)[ok]  # noqa: E731
    return run_and_check(z[ok].contiguous(), pick(u), pick(T), pick(k), pick(P), pick(m))


@pytest.mark.parametrize("V", [1000, 2049, 4099, 20000, 50257, 128256])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_masked_vocabularies_of_every_size(V, dt):
    """Masks of -inf, NaN and the type's lowest value, infinities and large logits, on both sides of the sizes
    that one CTA finishes and that one CTA holds; top-p over the whole row and behind a large top-k.  A masked
    token is drawn only when its row has nothing else."""
    rng = np.random.default_rng(V)
    low = torch.finfo(dt).min
    z = rng.normal(size=(9, V)) * 3
    z[0, rng.random(V) < 0.9] = -np.inf
    z[1, rng.random(V) < 0.9] = np.nan
    z[2, rng.random(V) < 0.5] = low
    z[3, 5:] = low
    z[4, [3, V - 7]] = np.inf
    z[5] = low
    z[6] *= 1e37
    z[7, 1:] = low
    z[8, rng.random(V) < 0.3] = -1e38
    masked = z <= -1e38
    masked[5], masked[6] = False, False
    zt = torch.tensor(z, device="cuda").to(dt)
    for T in (0.7, 1.0, 25.0, 40.0, 1e-6, 1e4):
        for k, P, m in ((0, 0.9, 0.0), (0, 0.25, 0.02), (2500, 0.9999, 0.0), (0, 1.0, 0.0), (7, 0.9, 0.0)):
            tok, pr = check_clear_borders(zt, rng.random(9).astype(np.float32), np.full(9, T), np.full(9, k), np.full(9, P),
                                          np.full(9, m))
            if len(tok) == 9:
                assert not masked[np.arange(9), tok].any() and not np.isnan(z[1, tok[1]])
                assert tok[4] in (3, V - 7) and tok[7] == 0 and (pr > 0).all()


@pytest.mark.parametrize("V", [64, 4099, 50257])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_zeros_of_either_sign_are_ties(V, dt):
    """-0 and +0 are one value: the lowest id wins the maximum, and borders of top-k and top-p inside a run of
    zeros keep the lowest ids, at temperatures down to the smallest differences of floats."""
    rng = np.random.default_rng(V)
    z = np.where(rng.random((5, V)) < 0.5, -0.0, 0.0)      # 0: zeros only
    z[1] = -1.0
    z[1, [3, 7, V - 2]] = -0.0, 0.0, -0.0                  # the maximum
    z[2, :20] = 2.0                                        # the zeros are where a top-k ends
    z[3] = np.where(rng.random(V) < 0.2, z[3], -6.0)       # and where top-p does
    z[4, rng.random(V) < 0.5] = -3.0
    zt = torch.tensor(z, device="cuda").to(dt)
    assert torch.signbit(zt[0]).any() and not torch.signbit(zt[0]).all()
    tok, _ = run_and_check(zt, np.full(5, 0.3, np.float32), T=np.zeros(5))
    assert tok.tolist() == [0, 3, 0, int(np.argmax(z[3])), int(np.argmax(z[4]))]
    for k, P in ((1, 1.0), (2, 1.0), (30, 1.0), (30, 0.9), (0, 0.31), (0, 0.05), (2060, 0.77), (0, 1.0)):
        for T in (1.0, 1e-3, 1e-38):
            for u in (0.0, 0.41, 0.93, 0.999999):
                check_clear_borders(zt, np.full(5, u, np.float32), np.full(5, T), np.full(5, k), np.full(5, P))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kb", [16, 64, 66, 67, 72, 131, 133])
def test_a_row_does_not_depend_on_its_batch(kb, dt):
    """However many CTAs a row gets (a large batch: fewer), its token and probability are the same bits."""
    V, R = kb * 1024 // (2 if dt == torch.bfloat16 else 4) + 3, 600
    g = torch.Generator(device="cuda").manual_seed(kb)
    r = lambda lo, hi: torch.rand(R, generator=g, device="cuda") * (hi - lo) + lo  # noqa: E731
    z = (torch.randn(R, V, generator=g, device="cuda") * 2.5).to(dt)
    u, T, P, m = r(0, 1), r(0.4, 1.5), r(0.3, 1.1), r(-0.1, 0.1)
    k = torch.randint(-3000, 5000, (R,), generator=g, device="cuda", dtype=torch.int32)
    all_ = tsd.sample_rows(z, u, T, k, P, m)
    for i in range(0, R, 67):
        few = tsd.sample_rows(z[i:i + 2], *(x[i:i + 2] for x in (u, T, k, P, m)))
        assert torch.equal(few["tokens"], all_["tokens"][i:i + 2]) and torch.equal(few["probs"], all_["probs"][i:i + 2])


@pytest.mark.parametrize("V", [1000, 4099, 50257])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_differences_past_the_largest_float(V, dt):
    """Logits whose distance overflows fp32, at temperatures that bring it back, up to infinity (a flat row)."""
    rng = np.random.default_rng(V)
    z = rng.uniform(-3.3e38, 3.3e38, (4, V))
    z[1] = rng.choice([-3.3e38, 0.0, 3.3e38], V)
    z[2] = np.where(rng.random(V) < 0.9, -3.3e38, 3.3e38)
    z[3] = rng.normal(size=V)
    zt = torch.tensor(z, device="cuda").to(dt)
    for T in (1e37, 1e38, 3.4e38, float("inf")):
        for k, P in ((0, 1.0), (50, 1.0), (0, 0.9), (0, 0.3), (2500, 0.95)):
            check_clear_borders(zt, rng.random(4).astype(np.float32), np.full(4, T), np.full(4, k), np.full(4, P))


def test_the_smallest_temperatures():
    """A temperature of (0, 2^-100) counts as 2^-100; logits of that size are told apart by it."""
    V, rng = 4099, np.random.default_rng(1)
    z = (rng.normal(size=(6, V)) * 2.0 ** -99).astype(np.float32)
    zt = torch.tensor(z, device="cuda")
    for k, P in ((0, 1.0), (50, 0.9), (0, 0.9)):
        u = rng.random(6).astype(np.float32)
        want = check_clear_borders(zt, u, np.full(6, 2.0 ** -100), np.full(6, k), np.full(6, P))
        r = tsd.sample_rows(zt, torch.tensor(u, device="cuda"), torch.tensor([2.0 ** -100, 2.0 ** -101, 1e-36, 1e-38, 1e-40, 1e-45],
                                                                            device="cuda"),
                            torch.full((6,), k, dtype=torch.int32, device="cuda"), torch.full((6,), P, device="cuda"))
        assert np.array_equal(r["tokens"].cpu().numpy(), want[0]) and np.array_equal(r["probs"].cpu().numpy(), want[1])
