"""The 8-bit KV cache and filtered sampling: binding of tsd_kv_q8_append / _commit / _read,
tsd_tree_verify_attn_q8 and tsd_sample_rows.

``Q8Cache`` holds one layer's committed K/V as float8_e4m3fn codes with one power-of-two scale byte
per (block of tokens, KV head); the functions carry the C names without the ``tsd_`` prefix.  The
format, every argument and every error are documented in include/tsd.h.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import COMMIT_MODES, Q8CacheDesc, TsdError, _check, _dt, _empty, _i32, _nbytes, _ptr, _under, lib

_raw_stream = torch._C._cuda_getCurrentRawStream


def _need(ok: bool, what: str):
    if not ok:
        raise TsdError(what)


def _on(dev: int, f, args):
    """f(*args, stream) on the current stream of device `dev`, that device current: launches go by it."""
    raw = _raw_stream(dev)
    if torch.cuda.current_device() == dev:
        return f(*args, raw)
    with torch.cuda.device(dev):
        return f(*args, raw)


def _at(t: Optional[torch.Tensor], dev: int, name: str, dtype=None, shape=None):
    """Address of a tensor (None: null), checked: contiguous, on device `dev`, of this type and shape."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise TsdError(f"{name} is on another device than the call's" if t.is_cuda else f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise TsdError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TsdError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise TsdError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _shape(t: Optional[torch.Tensor], shape, name: str):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise TsdError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


I32, F32 = torch.int32, torch.float32
BLOCK_SIZES = (8, 16, 32, 64, 128, 256)


class Q8Cache:
    """One layer's 8-bit K/V cache.

    ``Q8Cache(B, Hkv, d, Lmax=...)`` allocates the contiguous layout [B, Hkv, Lmax, d] (block_size
    consecutive positions share a scale); ``Q8Cache(B, Hkv, d, num_blocks=..., block_table=...)`` a pool
    of pages [num_blocks, Hkv, block_size, d].  ``prefix_len`` may be shared between layers (pass the
    same tensor; only the last layer's append / commit advances it).  ``wrap`` takes tensors that
    exist already.  Codes of rows at or past prefix_len are never read."""

    def __init__(self, B: int, Hkv: int, d: int, *, Lmax: Optional[int] = None, num_blocks: Optional[int] = None,
                 block_table: Optional[torch.Tensor] = None, block_size: int = 16,
                 prefix_len: Optional[torch.Tensor] = None, device="cuda"):
        _need((Lmax is None) != (num_blocks is None), "give either Lmax (contiguous) or num_blocks (paged)")
        _need(block_size in BLOCK_SIZES, "block_size must be a power of two in [8, 256]")
        dev = torch.device(device) if block_table is None else block_table.device
        if Lmax is not None:
            shape, sc = (B, Hkv, Lmax, d), (B, Hkv, -(-Lmax // block_size))
        else:
            _need(block_table is not None, "a paged cache needs its block_table")
            shape, sc = (num_blocks, Hkv, block_size, d), (num_blocks, Hkv)
        if prefix_len is None:
            prefix_len = torch.zeros(B, dtype=torch.int32, device=dev)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.full(sc, 127, dtype=torch.uint8, device=dev) for _ in range(2))
        self._set(k, v, ks, vs, prefix_len, block_size, block_table)

    @classmethod
    def wrap(cls, k, v, k_scale, v_scale, prefix_len, block_size: int, block_table=None) -> "Q8Cache":
        """A cache over existing tensors: codes (float8_e4m3fn or uint8), scale bytes (uint8), prefix_len
        [B] int32 and, for pages, block_table [B, max_blocks] int32."""
        self = cls.__new__(cls)
        self._set(k, v, k_scale, v_scale, prefix_len, block_size, block_table)
        return self

    def _set(self, k, v, k_scale, v_scale, prefix_len, block_size, block_table):
        B = prefix_len.shape[0]
        _need(block_size in BLOCK_SIZES, "block_size must be a power of two in [8, 256]")
        _need(k.dim() == 4 and k.shape == v.shape, "k and v must be [B, Hkv, Lmax, d] or [num_blocks, Hkv, block, d]")
        for t in (k, v):
            _need(t.dtype in (torch.float8_e4m3fn, torch.uint8), "codes must be float8_e4m3fn (or their bytes, uint8)")
        for t in (k_scale, v_scale):
            _need(t.dtype == torch.uint8, "scales must be uint8")
        for t in (v, k_scale, v_scale, prefix_len, block_table):
            _need(t is None or t.device == k.device, "the tensors of a cache must be on one device")
        if block_table is None:
            _need(k.shape[0] == B, "prefix_len and the codes disagree on the number of sequences")
            want = (B, k.shape[1], -(-k.shape[2] // block_size))
        else:
            _need(k.shape[2] == block_size, "a page holds block_size rows")
            _need(block_table.dim() == 2 and block_table.shape[0] == B, "block_table must be [B, max_blocks]")
            want = (k.shape[0], k.shape[1])
        _shape(k_scale, want, "k_scale")
        _shape(v_scale, want, "v_scale")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.prefix_len, self.block_table, self.block_size = prefix_len, block_table, block_size
        self.B, self.Hkv, self.d = B, k.shape[1], k.shape[3]
        paged = block_table is not None
        self.desc = Q8CacheDesc(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _i32(prefix_len, "prefix_len"),
                                0 if paged else k.shape[2], _i32(block_table, "block_table"),
                                block_table.shape[1] if paged else 0, block_size, k.shape[0] if paged else 0)
        self.ref = C.byref(self.desc)
        self.dev = k.get_device()

    @property
    def capacity(self) -> int:
        """Positions a sequence can hold."""
        return self.k.shape[2] if self.block_table is None else self.block_table.shape[1] * self.block_size


def _status(cache: Q8Cache, status):
    return torch.zeros(cache.B, dtype=I32, device=cache.k.device) if status is None else status


def _rows_of(cache: Q8Cache, k, v, what: str):
    if not (k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.shape[0] == cache.B and
            k.shape[2] == cache.Hkv and k.shape[3] == cache.d):
        raise TsdError(f"{what} must be two [B, rows, Hkv, d] tensors of one type that fit the cache")
    return k.shape[1]


def kv_q8_append(cache: Q8Cache, k_new, v_new, num_rows=None, advance: bool = True, status=None, stream=None):
    """Quantise rows [B, S, Hkv, d] into the cache from prefix_len on (num_rows [B] of them, default S).
    Returns status."""
    if stream is not None:
        return _under(kv_q8_append, locals())
    S, B, dev = _rows_of(cache, k_new, v_new, "k_new and v_new"), cache.B, cache.dev
    status = _status(cache, status)
    rc = _on(dev, lib().tsd_kv_q8_append,
             (cache.ref, _at(k_new, dev, "k_new"), _at(v_new, dev, "v_new"), _at(num_rows, dev, "num_rows", I32, (B,)), B, S,
              cache.Hkv, cache.d, _dt(k_new), int(advance), _at(status, dev, "status", I32, (B,))))
    _check(rc, "tsd_kv_q8_append")
    return status


def kv_q8_commit(cache: Q8Cache, k_tree, v_tree, path, accept_len, num_nodes=None, Dmax: int = 8,
                 mode: str = "path", advance: bool = True, status=None, stream=None):
    """Quantise the accepted rows of the tree K/V [B, Nmax, Hkv, d] into the cache (mode "path" or
    "length").  Returns status."""
    if stream is not None:
        return _under(kv_q8_commit, locals())
    Nmax, B, dev = _rows_of(cache, k_tree, v_tree, "k_tree and v_tree"), cache.B, cache.dev
    status = _status(cache, status)
    rc = _on(dev, lib().tsd_kv_q8_commit,
             (cache.ref, _at(k_tree, dev, "k_tree"), _at(v_tree, dev, "v_tree"), _at(path, dev, "path", I32, (B, Dmax + 1)),
              _at(accept_len, dev, "accept_len", I32, (B,)), _at(num_nodes, dev, "num_nodes", I32, (B,)), B, Nmax, cache.Hkv,
              cache.d, Dmax, _dt(k_tree), COMMIT_MODES[mode], int(advance), _at(status, dev, "status", I32, (B,))))
    _check(rc, "tsd_kv_q8_commit")
    return status


def kv_q8_read(cache: Q8Cache, start=None, num_rows=None, S: Optional[int] = None, dtype=torch.bfloat16,
               k_out=None, v_out=None, status=None, stream=None):
    """Read rows start[b] .. start[b] + num_rows[b] - 1 back as values.  Returns (k, v), each
    [B, S, Hkv, d] (rows at or past num_rows are not written; new outputs start as zeros)."""
    if stream is not None:
        return _under(kv_q8_read, locals())
    B, dev = cache.B, cache.dev
    if k_out is None or v_out is None:
        _need(k_out is None and v_out is None, "give both outputs or neither")
        _need(S is not None, "S is needed when the outputs are not given")
        k_out, v_out = (torch.zeros(B, S, cache.Hkv, cache.d, dtype=dtype, device=cache.k.device) for _ in range(2))
    S = _rows_of(cache, k_out, v_out, "k_out and v_out")
    status = _status(cache, status)
    rc = _on(dev, lib().tsd_kv_q8_read,
             (cache.ref, _at(start, dev, "start", I32, (B,)), _at(num_rows, dev, "num_rows", I32, (B,)),
              _at(k_out, dev, "k_out"), _at(v_out, dev, "v_out"), B, S, cache.Hkv, cache.d, _dt(k_out),
              _at(status, dev, "status", I32, (B,))))
    _check(rc, "tsd_kv_q8_read")
    return k_out, v_out


def tree_verify_attn_q8_workspace_size(cache: Q8Cache, Nmax: int, Hq: int, dtype: int) -> int:
    """Bytes of workspace tree_verify_attn_q8 needs for these sizes."""
    return int(lib().tsd_tree_verify_attn_q8_workspace_size(cache.ref, cache.B, Nmax, Hq, cache.Hkv, cache.d, dtype))


def tree_verify_attn_q8_workspace(q, cache: Q8Cache) -> torch.Tensor:
    """A workspace for calls of q's shape over this cache (zeroed: its ticket words start at zero)."""
    n = tree_verify_attn_q8_workspace_size(cache, q.shape[1], q.shape[2], _dt(q))
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=q.device)


def tree_verify_attn_q8_launches(cache: Q8Cache, Nmax: int, Hq: int, dtype: int):
    """(kernels, CTAs of the split kernel) of one tree_verify_attn_q8 call for these sizes."""
    ctas = C.c_longlong(0)
    n = lib().tsd_tree_verify_attn_q8_kernels(cache.ref, cache.B, Nmax, Hq, cache.Hkv, cache.d, dtype, C.byref(ctas))
    return int(n), int(ctas.value)


def tree_verify_attn_q8(q, cache: Q8Cache, k_tree, v_tree, parent_s, num_nodes=None, Dmax: int = 8,
                        scale: Optional[float] = None, out=None, lse=None, workspace=None, status=None,
                        want_lse: bool = False, stream=None):
    """Tree-masked GQA attention of q [B, N, Hq, d] over the 8-bit cache and the tree's own K/V
    [B, N, Hkv, d] (tsd_tree_verify_attn_q8).  workspace: from tree_verify_attn_q8_workspace, kept by the
    caller (None: a new one).  Returns (out, lse)."""
    if stream is not None:
        return _under(tree_verify_attn_q8, locals())
    B, Nmax, Hq, d = q.shape
    dev, dtype = cache.dev, q.dtype
    if B != cache.B or d != cache.d:
        raise TsdError("q must be [B, N, Hq, d] of the cache's B and d")
    if k_tree.dtype != dtype or _rows_of(cache, k_tree, v_tree, "k_tree and v_tree") != Nmax:
        raise TsdError("the tree K/V must have q's type and node count")
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = _empty((B, Nmax, Hq), F32, q)
    status = _status(cache, status)
    if workspace is None:
        workspace = tree_verify_attn_q8_workspace(q, cache)
    rc = _on(dev, lib().tsd_tree_verify_attn_q8,
             (_at(q, dev, "q"), cache.ref, _at(k_tree, dev, "k_tree"), _at(v_tree, dev, "v_tree"),
              _at(parent_s, dev, "parent_s", I32, (B, Nmax + 1)), _at(num_nodes, dev, "num_nodes", I32, (B,)), B, Nmax, Hq,
              cache.Hkv, d, Dmax, _dt(q), d ** -0.5 if scale is None else float(scale), _at(out, dev, "out", dtype, q.shape),
              _at(lse, dev, "lse", F32, (B, Nmax, Hq)), _at(workspace, dev, "workspace"), _nbytes(workspace),
              _at(status, dev, "status", I32, (B,))))
    _check(rc, "tsd_tree_verify_attn_q8")
    return out, lse


def sample_rows(logits, uniforms, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, probs=None,
                stream=None):
    """Draw one token per row of logits [R, V] under per-row temperature, top_k (int32), top_p and min_p
    (each a tensor [R], or None for 1 / off) from uniforms [R] (tsd_sample_rows).  Returns tokens [R]
    int32 and probs [R] fp32, the drawn tokens' probabilities in the filtered distributions."""
    if stream is not None:
        return _under(sample_rows, locals())
    R, V = logits.shape
    dev = logits.get_device()
    _need(dev >= 0, "logits must be a CUDA tensor")
    if tokens is None:
        tokens = _empty((R,), I32, logits)
    if probs is None:
        probs = _empty((R,), F32, logits)
    _need(uniforms is not None, "uniforms are needed")
    rc = _on(dev, lib().tsd_sample_rows,
             (_at(logits, dev, "logits"), _dt(logits), R, V, _at(uniforms, dev, "uniforms", F32, (R,)),
              _at(temperature, dev, "temperature", F32, (R,)), _at(top_k, dev, "top_k", I32, (R,)),
              _at(top_p, dev, "top_p", F32, (R,)), _at(min_p, dev, "min_p", F32, (R,)), _at(tokens, dev, "tokens", I32, (R,)),
              _at(probs, dev, "probs", F32, (R,))))
    _check(rc, "tsd_sample_rows")
    return {"tokens": tokens, "probs": probs}
