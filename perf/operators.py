"""Cases, plain forms and work of the 8-bit KV cache operators (append, commit, read, tree attention) and of
sampling under temperature, top-k, top-p and min-p."""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E_MIN = 87            # the smallest scale byte: 2^-40


# --------------------------------------------------------------------------- cases
def _attn(name, **k):
    c = dict(op="attn", B=1, N=1, Hq=32, Hkv=8, d=128, Lmin=1024, Lmax=1024, bs=16, paged=True, dtype="bf16", tree="heap",
             ragged=False)
    c.update(k, name=name)
    return c


def listed():
    return [
        # one token of one sequence: the decode call of a single chat
        _attn("attn decode b1", Lmin=1000, Lmax=1000),
        # one sequence's 26-node static tree over a contiguous cache
        _attn("attn tree26 b1", N=26, Lmin=2048, Lmax=2048, paged=False, bs=64),
        # a batch of 60-node dynamic trees over ragged paged prefixes
        _attn("attn eagle60 b16", B=16, N=60, Lmin=1024, Lmax=8192, ragged=True),
        # a full batch of 5-token chains over long prefixes: bound by the cache's bytes
        _attn("attn chain5 b64", B=64, Hq=64, N=6, Lmin=8192, Lmax=8192, paged=False, bs=64, tree="chain"),
        # 512 pre-drafted nodes of one long sequence: bound by the products
        _attn("attn forest b1", N=512, Lmin=32768, Lmax=32768),
        # fp32, head size 64, three query heads a KV head, odd lengths
        _attn("attn fp32 d64", B=3, N=7, Hq=12, Hkv=4, d=64, Lmin=301, Lmax=777, bs=32, dtype="f32", ragged=True),
        # a batch of prompts written into fresh pages
        dict(name="append prompts b8", op="append", B=8, S=4096, Hkv=8, d=128, Lmin=0, Lmax=37, bs=16, dtype="bf16",
             ragged=True),
        # the accepted paths of a batch, a few rows each, into partly filled pages
        dict(name="commit path b64", op="commit", B=64, N=26, D=6, Hkv=8, d=128, Lmin=1024, Lmax=2048, bs=16,
             dtype="bf16", mode="path"),
        # long prefixes read back into a bf16 cache
        dict(name="read b8", op="read", B=8, S=8192, Hkv=8, d=128, start=0, bs=16, dtype="bf16", ragged=True),
        # a short odd piece of one sequence in fp32
        dict(name="read fp32 d64 b1", op="read", B=1, S=301, Hkv=4, d=64, start=77, bs=32, dtype="f32", ragged=False),
        # the first token of one request
        dict(name="sample b1", op="sample", R=1, V=128256, dtype="bf16", greedy=False),
        # a mixed batch of requests, each with parameters of its own
        dict(name="sample b64", op="sample", R=64, V=128256, dtype="bf16", greedy=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "commit", "read", "sample", "sample"])
    if op == "attn":
        while True:
            Hkv = rng.choice([1, 2, 4, 8])
            G = rng.choice([1, 2, 3, 4, 7, 8])
            L = _log(rng, 1, 32768)
            c = dict(op=op, B=_log(rng, 1, 64), N=_log(rng, 1, 512), Hq=G * Hkv, Hkv=Hkv, d=rng.choice([64, 128, 128]),
                     Lmin=max(1, L // rng.choice([1, 2, 5])), Lmax=L, bs=rng.choice([8, 16, 32, 64, 128, 256]),
                     paged=rng.random() < 0.6, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
                     tree=rng.choice(["heap", "chain"]), ragged=rng.random() < 0.5)
            if c["tree"] == "chain":
                c["N"] = min(c["N"], 40)
            w = work(c)
            # fp32 runs on the FMA pipes, for which the largest listed case would be too large
            if w["bytes"] < 5e8 and w["flops"] < (6e10 if c["dtype"] == "bf16" else 4e9):
                return c
    if op == "append":
        while True:
            c = dict(op=op, B=_log(rng, 1, 32), S=_log(rng, 1, 8192), Hkv=rng.choice([1, 2, 4, 8]),
                     d=rng.choice([64, 128]), Lmin=0, Lmax=rng.choice([0, 1, 37, 700]),
                     bs=rng.choice([8, 16, 32, 64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "f32"]), ragged=True)
            if work(c)["bytes"] < 2.4e8:
                return c
    if op == "commit":
        return dict(op=op, B=_log(rng, 1, 128), N=rng.randint(8, 60), D=rng.randint(1, 7), Hkv=rng.choice([1, 2, 4, 8]),
                    d=rng.choice([64, 128]), Lmin=rng.randint(0, 300), Lmax=rng.randint(300, 2048),
                    bs=rng.choice([8, 16, 32, 64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    mode=rng.choice(["path", "length"]))
    if op == "read":
        while True:
            c = dict(op=op, B=_log(rng, 1, 32), S=_log(rng, 1, 16384), Hkv=rng.choice([1, 2, 4, 8]),
                     d=rng.choice([64, 128]), start=rng.choice([0, 1, 77, 1000]), bs=rng.choice([8, 16, 32, 64, 128, 256]),
                     dtype=rng.choice(["bf16", "bf16", "f32"]), ragged=rng.random() < 0.7)
            if work(c)["bytes"] < 4e8:
                return c
    while True:
        c = dict(op=op, R=_log(rng, 1, 512), V=rng.choice([1000, 32000, 50257, 128256, 151936, _log(rng, 100, 200000)]),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), greedy=rng.random() < 0.5)
        if c["R"] * c["V"] <= 64 * 128256:
            return c


# --------------------------------------------------------------------------- sizes that a case fixes
def _lens(c):
    """The prefix lengths of the batch: spread over [Lmin, Lmax], the first the longest."""
    B, lo, hi = c["B"], c["Lmin"], c["Lmax"]
    return [hi if b == 0 else lo + (b * 7919) % (hi - lo + 1) for b in range(B)]


def _nodes(c):
    return [max(1, c["N"] - b % 3) if c["ragged"] else c["N"] for b in range(c["B"])]


def _rows(c):
    """Rows of each sequence to append or read: the first has all of them, the others fewer where ragged."""
    return [max(1, c["S"] - (b * 31 * c["S"]) // (64 * c["B"])) if c["ragged"] else c["S"] for b in range(c["B"])]


def _parents(c):
    return [i - 1 if c["tree"] == "chain" else (i - 1) // 3 if i else -1 for i in range(c["N"])]


def _depths(c):
    d = []
    for p in _parents(c):
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _accepted(c):
    """Committed rows less one of each sequence: every length from 0 to the largest that the tree and D allow."""
    most = min(c["D"], _path_depth(c["N"])) if c["mode"] == "path" else min(c["D"], c["N"] - 1)
    return [(b * 5 + most) % (most + 1) for b in range(c["B"])]


def _path_depth(N):
    i, d = N - 1, 0
    while i > 0:
        i, d = (i - 1) // 3, d + 1
    return d


def work(case):
    c = case
    if c["op"] == "attn":
        es = 2 if c["dtype"] == "bf16" else 4
        G, dep = c["Hq"] // c["Hkv"], _depths(c)
        by = fl = 0
        for L, N in zip(_lens(c), _nodes(c)):
            by += 2 * L * c["Hkv"] * c["d"] + 2 * -(-L // c["bs"]) * c["Hkv"]
            by += 2 * N * c["Hkv"] * c["d"] * es + 2 * N * c["Hq"] * c["d"] * es
            fl += 4 * c["d"] * c["Hkv"] * G * (N * L + sum(dep[:N]) + N)
        return {"bytes": by, "flops": fl}
    if c["op"] == "sample":
        n = c["R"] * c["V"]
        return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + 28 * c["R"], "flops": 4 * n}
    es = 2 if c["dtype"] == "bf16" else 4
    rows = sum(_rows(c)) if c["op"] in ("append", "read") else sum(a + 1 for a in _accepted(c))
    n = 2 * rows * c["Hkv"] * c["d"]
    return {"bytes": n * (es + 1) + 2 * c["Hkv"] * -(-rows // c["bs"]), "flops": 3 * n}


# --------------------------------------------------------------------------- the format
def _scale_byte(amax):
    """The byte of the smallest power of two that keeps amax (fp32, finite) within 448 of its units."""
    m, e = torch.frexp(amax)                                   # amax = m 2^e, m in [1/2, 1)
    k = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, k + 127, torch.zeros_like(k)).clamp(min=E_MIN)


def _two_to(byte):
    return (byte.to(torch.int32) << 23).view(torch.float32)    # the byte is an fp32 exponent field


def _code(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _value(code):
    return code.view(torch.float8_e4m3fn).to(torch.float32)


def _filled(gen, shape, bs_dim, spread):
    """Random codes and scale bytes of whole blocks: normal values whose size differs between blocks."""
    x = torch.randn(shape, generator=gen, device=DEV)
    sc = list(shape)
    sc[bs_dim] = sc[-1] = 1
    x *= torch.exp(spread * torch.randn(sc, generator=gen, device=DEV))
    byte = _scale_byte(x.abs().amax((bs_dim, -1), keepdim=True))
    x /= _two_to(byte)
    return _code(x), byte.to(torch.uint8).squeeze(-1).squeeze(bs_dim)


# --------------------------------------------------------------------------- inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pool(c, gen, longest, filled):
    """A page pool with page 0 kept free, and the pages of every sequence in random order."""
    B, bs = c["B"], c["bs"]
    mb = -(-longest // bs)
    nblk = B * mb + 1
    table = (torch.randperm(nblk - 1, generator=gen, device=DEV)[: B * mb] + 1).to(torch.int32).reshape(B, mb)
    shape = (nblk, c["Hkv"], bs, c["d"])
    if filled:
        (k, ks), (v, vs) = _filled(gen, shape, 2, 0.5), _filled(gen, shape, 2, 0.5)
    else:
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
        ks, vs = (torch.full(shape[:2], 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    return dict(k=k, v=v, k_scale=ks, v_scale=vs, table=table, num_blocks=nblk)


def prepare(case, seed):
    c, gen = case, torch.Generator(device=DEV).manual_seed(int(seed))
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    s = dict(c)
    if c["op"] == "sample":
        R, V = c["R"], c["V"]
        s["logits"] = (2.5 * rnd(R, V)).to(DT[c["dtype"]])
        u = torch.rand(5, R, generator=gen, device=DEV)
        s["T"] = 0.4 + u[0]
        if c["greedy"]:
            s["T"][3::8] = 0.0                      # some requests of the batch are greedy
        i = torch.arange(R, device=DEV)
        s["top_k"] = torch.where(i % 4 == 1, 0, (2.0 ** (1 + 7 * u[1])).to(torch.int32) + 1).to(torch.int32)
        s["top_k"] = torch.where(i % 4 == 2, 2000, s["top_k"]).to(torch.int32)
        s["top_p"] = torch.where(i % 3 == 2, 1.0, 0.6 + 0.39 * u[2])
        s["min_p"] = torch.where(i % 2 == 0, 0.0, 0.1 * u[3])
        s["u"] = u[4]
        return s
    if c["op"] == "attn":
        B, N, dt = c["B"], c["N"], DT[c["dtype"]]
        s["q"] = rnd(B, N, c["Hq"], c["d"]).to(dt)
        s["k_tree"], s["v_tree"] = rnd(B, N, c["Hkv"], c["d"]).to(dt), rnd(B, N, c["Hkv"], c["d"]).to(dt)
        par = _i32([_parents(c)] * B)
        s["parent_s"] = torch.cat([torch.zeros(B, 1, dtype=torch.int32, device=DEV), par + 1], 1).contiguous()
        s["num_nodes"], s["D"] = _i32(_nodes(c)), max(_depths(c))
        s["prefix_len"] = _i32(_lens(c))
        if c["paged"]:
            s.update(_pool(c, gen, max(_lens(c)), True))
        else:
            nb = -(-c["Lmax"] // c["bs"])
            (k, s["k_scale"]), (v, s["v_scale"]) = (_filled(gen, (B, c["Hkv"], nb, c["bs"], c["d"]), 3, 0.5) for _ in range(2))
            s["k"], s["v"] = (t.reshape(B, c["Hkv"], nb * c["bs"], c["d"]) for t in (k, v))
        s["out"] = torch.zeros_like(s["q"])
        return s
    B, dt = c["B"], DT[c["dtype"]]
    if c["op"] == "read":
        s.update(_pool(c, gen, c["start"] + c["S"], True))
        s["start"], s["rows"] = _i32([c["start"]] * B), _i32(_rows(c))
        s["prefix_len"] = _i32([c["start"] + c["S"]] * B)
        s["k_out"], s["v_out"] = (torch.zeros(B, c["S"], c["Hkv"], c["d"], dtype=dt, device=DEV) for _ in range(2))
        return s
    R = c["S"] if c["op"] == "append" else c["D"] + 1
    s.update(_pool(c, gen, c["Lmax"] + R, True))
    s["prefix_len"] = _i32(_lens(c))
    M = c["S"] if c["op"] == "append" else c["N"]
    wide = torch.exp(0.7 * rnd(2, B, M, c["Hkv"], 1))     # tokens of unlike sizes, so that scales grow
    s["k_new"], s["v_new"] = ((rnd(B, M, c["Hkv"], c["d"]) * w).to(dt) for w in wide)
    if c["op"] == "append":
        s["rows"] = _i32(_rows(c))
        return s
    s["accept_len"] = _i32(_accepted(c))
    path = []
    for a in _accepted(c):                          # the path from the root to a node of depth a, as slots
        i = sum(3 ** k for k in range(a))           # the first node of depth a
        p = [i]
        while i:
            i = (i - 1) // 3
            p.append(i)
        path.append([n + 1 for n in reversed(p)] + [0] * (c["D"] - a))
    s["path"] = _i32(path)
    return s


# --------------------------------------------------------------------------- plain forms
def _gather(s, what):
    """The cache as values [B, Hkv, positions, d] in 32 bits."""
    code, sc = s[what], s[what + "_scale"]
    if not s.get("paged", True):
        B, H, L, d = code.shape
        return (_value(code).view(B, H, L // s["bs"], s["bs"], d) * _two_to(sc)[..., None, None]).view(B, H, L, d)
    t = s["table"].long()
    x = _value(code[t]) * _two_to(sc[t])[..., None, None]              # [B, blocks, Hkv, bs, d]
    return x.transpose(1, 2).flatten(2, 3)


def _attn_plain(s):
    B, N, Hq, d = s["q"].shape
    Hkv, G = s["Hkv"], Hq // s["Hkv"]
    K, V = _gather(s, "k"), _gather(s, "v")
    q = s["q"].float().view(B, N, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, d)
    kt, vt = (s[n].float().transpose(1, 2) for n in ("k_tree", "v_tree"))
    pos = torch.arange(K.shape[2], device=DEV)
    sp = torch.matmul(q, K.transpose(2, 3)) / math.sqrt(d)
    sp.masked_fill_((pos >= s["prefix_len"][:, None])[:, None, None], -math.inf)
    node = torch.arange(N, device=DEV)
    one = (s["parent_s"][:, 1:, None] - 1 == node) | (node[:, None] == node)
    anc = torch.linalg.matrix_power(one.float(), max(1, s["D"])) > 0
    anc &= node < s["num_nodes"][:, None, None]
    st = torch.matmul(q, kt.transpose(2, 3)) / math.sqrt(d)
    st = st.view(B, Hkv, N, G, N).masked_fill(~anc[:, None, :, None], -math.inf).view(B, Hkv, N * G, N)
    m = torch.maximum(sp.amax(-1, keepdim=True), st.amax(-1, keepdim=True)).clamp(min=-1e30)
    sp, st = sp.sub_(m).exp_(), (st - m).exp()
    o = (torch.matmul(sp, V) + torch.matmul(st, vt)) / (sp.sum(-1, keepdim=True) + st.sum(-1, keepdim=True))
    o = o.view(B, Hkv, N, G, d).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, d)
    return torch.where((node < s["num_nodes"][:, None])[..., None, None], o, 0.0).to(s["q"].dtype)


def _write_plain(s, rows, n):
    """Rows [B, R, Hkv, d] (K, V) into the blocks from prefix_len on; n of them count in each sequence."""
    L, bs, R = s["prefix_len"].long(), s["bs"], rows[0].shape[1]
    nb = (R + bs - 2) // bs + 1
    blk = L[:, None] // bs + torch.arange(nb, device=DEV)
    pos = blk[..., None] * bs + torch.arange(bs, device=DEV)            # [B, nb, bs]
    rel = pos - L[:, None, None]
    new, old = (rel >= 0) & (rel < n[:, None, None]), rel < 0
    hit = new.any(-1)
    page = torch.where(hit, s["table"].long().gather(1, blk.clamp(max=s["table"].shape[1] - 1)), 0)   # page 0 is free
    had, put = (old.any(-1) & hit)[..., None], hit[..., None, None, None]
    bi = torch.arange(L.shape[0], device=DEV)[:, None, None]
    for name, x in zip(("k", "v"), rows):
        code, sc = s[name][page], s[name + "_scale"][page].int()         # [B, nb, Hkv, bs, d], [B, nb, Hkv]
        x = x[bi, rel.clamp(0, R - 1)].float().permute(0, 1, 3, 2, 4)
        isnew, isold = new[:, :, None, :, None], (old & hit[..., None])[:, :, None, :, None]
        byte = _scale_byte(torch.where(isnew, x, 0.0).abs().amax((-1, -2)))
        byte = torch.where(had, torch.maximum(byte, sc), byte)
        unit = _two_to(byte)[..., None, None]
        c_old = _code(_value(code) * (_two_to(sc)[..., None, None] / unit))
        code = torch.where(isnew & put, _code(torch.where(isnew, x, 0.0) / unit), torch.where(isold, c_old, code))
        s[name].index_put_((page,), code)
        s[name + "_scale"].index_put_((page,), torch.where(hit[..., None], byte, sc).to(torch.uint8))
    return _written(s)


def _written(s):
    return {n: s[n].view(torch.float8_e4m3fn) if n in "kv" else s[n] for n in ("k", "v", "k_scale", "v_scale")}


def _read_plain(s):
    S, bs = s["k_out"].shape[1], s["bs"]
    i = torch.arange(S, device=DEV)
    ok = (i < s["rows"][:, None])[..., None, None]
    pos = torch.where(ok[..., 0, 0], s["start"][:, None] + i, 0).long()
    page, row = s["table"].long().gather(1, pos // bs), pos % bs
    for n in ("k", "v"):
        x = _value(s[n][page, :, row]) * _two_to(s[n + "_scale"][page])[..., None]
        s[n + "_out"].copy_(torch.where(ok, x.to(s["k_out"].dtype), s[n + "_out"]))
    return s["k_out"], s["v_out"]


def _sample_plain(s):
    z = s["logits"].double()                      # 64 bits: the draw is decided next to borders of the sums
    R, V = z.shape
    T, P, m, u = (s[n].double()[:, None] for n in ("T", "top_p", "min_p", "u"))
    k = s["top_k"].long()[:, None]
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    w = torch.exp((zs - zs[:, :1]) / torch.where(T > 0, T, 1.0))
    rank = torch.arange(V, device=DEV)
    keep = (rank < torch.where((k <= 0) | (k > V), V, k)) & ((rank < 1) | (T > 0))
    cum = (w * keep).cumsum(1)
    keep &= (cum - w < P * cum[:, -1:]) | (P >= 1) | (rank < 1)
    keep &= w >= m.clamp(max=1.0)
    w = torch.zeros_like(w).scatter_(1, order, w * keep)
    cdf = w.cumsum(1)
    Z = cdf[:, -1:]
    last = torch.where(w > 0, rank, 0).amax(1, keepdim=True)
    tok = torch.minimum((cdf <= u * Z).sum(1, keepdim=True), last)
    return tok[:, 0].to(torch.int32), (w.gather(1, tok) / Z)[:, 0].float()


# --------------------------------------------------------------------------- the library's calls
def _cache(tsd, s):
    if "cache" not in s:
        f8 = {n: s[n].view(torch.float8_e4m3fn) for n in ("k", "v")}
        s["cache"] = tsd.Q8Cache.wrap(f8["k"], f8["v"], s["k_scale"], s["v_scale"], s["prefix_len"], s["bs"],
                                      s["table"] if s.get("paged", True) else None)
    return s["cache"]


def _own(s):
    import tree_speculative_decoding_06_b200 as tsd
    if s["op"] == "sample":
        r = tsd.sample_rows(s["logits"], s["u"], s["T"], s["top_k"], s["top_p"], s["min_p"])
        return r["tokens"], r["probs"]
    cache = _cache(tsd, s)
    if s["op"] == "attn":
        if "ws" not in s:
            s["ws"] = tsd.tree_verify_attn_q8_workspace(s["q"], cache)
            s["status"] = torch.zeros(s["B"], dtype=torch.int32, device=DEV)
        return tsd.tree_verify_attn_q8(s["q"], cache, s["k_tree"], s["v_tree"], s["parent_s"], s["num_nodes"], s["D"],
                                       out=s["out"], workspace=s["ws"], status=s["status"])[0]
    if "status" not in s:
        s["status"] = torch.zeros(s["B"], dtype=torch.int32, device=DEV)
    if s["op"] == "read":
        return tsd.kv_q8_read(cache, s["start"], s["rows"], k_out=s["k_out"], v_out=s["v_out"], status=s["status"])
    if s["op"] == "append":
        tsd.kv_q8_append(cache, s["k_new"], s["v_new"], s["rows"], advance=False, status=s["status"])
    else:
        tsd.kv_q8_commit(cache, s["k_new"], s["v_new"], s["path"] if s["mode"] == "path" else None, s["accept_len"],
                         Dmax=s["D"], mode=s["mode"], advance=False, status=s["status"])
    return _written(s)


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "attn":
        return _attn_plain(s)
    if s["op"] == "sample":
        return _sample_plain(s)
    if s["op"] == "read":
        return _read_plain(s)
    if s["op"] == "append":
        return _write_plain(s, (s["k_new"], s["v_new"]), s["rows"])
    b = torch.arange(s["B"], device=DEV)[:, None]
    node = (s["path"] - 1).clamp(min=0).long() if s["mode"] == "path" else \
        torch.arange(s["D"] + 1, device=DEV).clamp(max=s["N"] - 1).expand(s["B"], -1)
    return _write_plain(s, (s["k_new"][b, node], s["v_new"][b, node]), s["accept_len"] + 1)


# --------------------------------------------------------------------------- in 64 bits
_E4M3 = [(-1.0 if i & 128 else 1.0) * ((i & 7) / 512.0 if not i & 120 else (8 + (i & 7)) * 2.0 ** ((i >> 3 & 15) - 10))
         for i in range(256)]


def _p2(e):
    """2^e in 64 bits, exact, for whole e (torch.pow may be an ulp off on the GPU, which would break ties)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _positions(s, what, b, lo, hi):
    """Positions lo..hi-1 of sequence b in 64 bits, [positions, Hkv, d]."""
    tab = torch.tensor(_E4M3, dtype=torch.float64, device=DEV)
    p = torch.arange(lo, hi, device=DEV)
    if s.get("paged", True):
        page = s["table"][b].long()[p // s["bs"]]
        code, byte = s[what][page, :, p % s["bs"]], s[what + "_scale"][page]
    else:
        code, byte = s[what][b][:, p].transpose(0, 1), s[what + "_scale"][b][:, p // s["bs"]].T
    return tab[code.long()] * _p2(byte.long() - 127)[..., None]


def _round_e4m3(x):
    """Nearest e4m3 value, ties to even, of |x| <= 448 in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(_p2(e) > x.abs().clamp(min=2.0 ** -6), e - 1, e)
    e = torch.where(_p2(e + 1) <= x.abs(), e + 1, e)
    step = _p2(e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "sample":
        z, probs = s["logits"].to(f64), []
        for r in range(s["R"]):
            T, k, P, m, u = (float(s[n][r]) for n in ("T", "top_k", "top_p", "min_p", "u"))
            if T <= 0:
                probs.append(1.0)
                continue
            ids = torch.argsort(z[r], descending=True, stable=True)
            p = torch.softmax(z[r] / T, 0)
            a = p[ids]
            n = s["V"] if k <= 0 else min(int(k), s["V"])
            if P < 1:
                n = min(n, 1 + int((a[:n].cumsum(0)[:-1] < P * a[:n].sum()).sum()))
            if m > 0:
                n = min(n, max(1, int((a >= min(m, 1.0) * a[0]).sum())))
            kept, _ = torch.sort(ids[:n])
            q = p[kept] / p[kept].sum()
            j = min(int(torch.searchsorted(q.cumsum(0), torch.tensor(u, dtype=f64, device=DEV), right=True)), n - 1)
            probs.append(float(q[j]))
        return None, torch.tensor(probs, dtype=f64)
    if s["op"] == "attn":
        out = torch.zeros(s["q"].shape, dtype=f64, device=DEV)
        G, par = s["Hq"] // s["Hkv"], _parents(s)
        anc = torch.zeros(s["N"], s["N"], dtype=torch.bool)
        for i in range(s["N"]):
            j = i
            while j >= 0:
                anc[i, j] = True
                j = par[j]
        anc = anc.to(DEV)
        for b, (L, N) in enumerate(zip(_lens(s), _nodes(s))):
            K = torch.cat([_positions(s, "k", b, 0, L), s["k_tree"][b, :N].to(f64)])
            V = torch.cat([_positions(s, "v", b, 0, L), s["v_tree"][b, :N].to(f64)])
            see = torch.cat([torch.ones(N, L, dtype=torch.bool, device=DEV), anc[:N, :N]], 1)
            for h in range(s["Hq"]):
                a = (s["q"][b, :N, h].to(f64) @ K[:, h // G].T) * s["d"] ** -0.5
                out[b, :N, h] = torch.softmax(a.masked_fill(~see, -math.inf), 1) @ V[:, h // G]
        return out
    if s["op"] == "read":
        outs = [t.to(f64) for t in (s["k_out"], s["v_out"])]
        for b, n in enumerate(_rows(s)):
            for o, what in zip(outs, "kv"):
                o[b, :n] = _positions(s, what, b, s["start"][b].item(), s["start"][b].item() + n)
        return tuple(outs)
    tab = torch.tensor(_E4M3, dtype=f64, device=DEV)
    done = {w: tab[s[w].long()] for w in "kv"}
    for b, L in enumerate(_lens(s)):
        n = _rows(s)[b] if s["op"] == "append" else _accepted(s)[b] + 1
        src = torch.arange(n, device=DEV) if s.get("mode") != "path" else s["path"][b, :n].long() - 1
        for what in "kv":
            x = s[what + "_new"][b].to(f64)[src]                          # [n, Hkv, d]
            for j in range(L // s["bs"], (L + n - 1) // s["bs"] + 1):
                lo, hi = max(L, j * s["bs"]), min(L + n, (j + 1) * s["bs"])
                page = int(s["table"][b, j])
                y = x[lo - L: hi - L].transpose(0, 1)                     # [Hkv, rows, d]
                top = y.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top / 448))
                e = e + (top > 448 * _p2(e)).to(f64) - (top <= 448 * _p2(e - 1)).to(f64)
                e = torch.where(top > 0, e, torch.full_like(e, -40.0)).clamp(min=-40)
                was = s[what + "_scale"][page].to(f64) - 127
                if L > j * s["bs"]:
                    e = torch.maximum(e, was)
                    cut = L - j * s["bs"]
                    done[what][page, :, :cut] = _round_e4m3(done[what][page, :, :cut] * _p2(was - e)[:, None, None])
                at = lo - j * s["bs"]
                done[what][page, :, at: at + hi - lo] = _round_e4m3(y / _p2(e)[:, None, None])
    return {"k": done["k"], "v": done["v"], "k_scale": None, "v_scale": None}
