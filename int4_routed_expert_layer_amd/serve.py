"""Thin ctypes layer over the serving operators of include/coli_moe.h: the
paged latent cache, latent attention (absorbed and expanded) and the
verification of drafted tokens.

The pages' engine keeps 576 values a token in place of 32,768 (README "Come
funziona", compressed attention state) and drafts tokens that the main model
verifies in one batched forward; the operators are that step's attention and
acceptance, next to the expert layer of ``binding``.

Tensors are checked here (device, type, shape, innermost stride), because the
C ABI sees addresses; sizes and alignment are checked there.  Work goes to
torch's current stream of the handle's device.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import binding as B

LATENT, ROPE = 512, 64
ROW = LATENT + ROPE
HALF = {"bf16": (0, torch.bfloat16), "f16": (1, torch.float16)}
PROBS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class ServeDims(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_heads", "latent", "rope", "nope", "v_dim", "page_size", "max_tokens", "max_seqs", "half")]


class Serve:
    """The serving operators of one model on one device (owns their plan and scratch).

    One handle serves every layer of a step: ``plan`` once, then ``append``
    and ``decode`` per layer.  Calls on one handle must not overlap in time.
    """

    def __init__(self, n_heads, max_tokens, max_seqs, page_size=64, nope=192, v_dim=256, dtype="bf16", device=0, latent=LATENT, rope=ROPE):
        if dtype not in HALF:
            raise ValueError(f"dtype {dtype!r} must be one of {sorted(HALF)}")
        code, self.dtype = HALF[dtype]
        self.dims = ServeDims(n_heads, latent, rope, nope, v_dim, page_size, max_tokens, max_seqs, code)
        self.device = torch.device("cuda", device)
        self.handle = None
        h = C.c_void_p()
        st = B.lib.coli_serve_create(C.byref(self.dims), device, C.byref(h))
        if st != B.OK:
            raise B.ColiError(st, B.lib.coli_serve_last_error(None).decode())
        self.handle = h
        self._planned = None    # sequences and tokens of the plan

    def close(self):
        if getattr(self, "handle", None):
            B.lib.coli_serve_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- checks ------------------------------------------------------------
    def _call(self, name, *args):
        if not self.handle:
            raise ValueError("the handle is closed")
        stream = C.c_void_p(torch.cuda.current_stream(self.device).cuda_stream)
        st = getattr(B.lib, name)(self.handle, *args, stream)
        if st != B.OK:
            raise B.ColiError(st, B.lib.coli_serve_last_error(self.handle).decode())

    def _tensor(self, name, t, dtype, *shape, dense=False):
        """Checks a tensor: device, type, shape (None: any size), innermost
        stride 1, and with ``dense`` no gaps at all."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the handle on {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} is {t.dtype}, must be {dtype}")
        if t.dim() != len(shape) or any(w is not None and w != s for w, s in zip(shape, t.shape)):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, must be {tuple('any' if w is None else w for w in shape)}")
        if t.numel() and ((dense and not t.is_contiguous()) or (t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1)):
            raise ValueError(f"{name} must be contiguous" + ("" if dense else " in its last dimension"))
        return t

    def _cache(self, cache):
        page = self.dims.page_size
        self._tensor("cache", cache, self.dtype, None, page, ROW)
        if cache.stride(1) != ROW:
            raise ValueError("the rows of a cache page must be contiguous")
        return B._dptr(cache), cache.stride(0), cache.shape[0]

    def _out(self, name, out, shape, dtype):
        if out is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        return self._tensor(name, out, dtype, *shape, dense=True)

    def _starts(self, name, q_start):
        self._tensor(name, q_start, torch.int32, None, dense=True)
        if q_start.shape[0] < 1:
            raise ValueError(f"{name} needs n_seq + 1 entries")
        return q_start.shape[0] - 1

    # -- operators ---------------------------------------------------------
    def append(self, c, norm_weight, eps, cos, sin, positions, slots, cache, q_pe=None, q_out=None, interleaved=True):
        """Write the latent rows of new tokens into the cache (coli_latent_append).

        c [T, 576], norm_weight [512], cos and sin fp32 [n_positions, 32],
        positions int32 [T], slots int64 [T] (negative: not cached), cache
        [n_pages, page_size, 576].  Returns the turned q_pe [T, n_heads, 64], or
        None without q_pe."""
        n = self._tensor("c", c, self.dtype, None, ROW).shape[0]
        self._tensor("norm_weight", norm_weight, self.dtype, LATENT, dense=True)
        n_pos = self._tensor("cos", cos, torch.float32, None, ROPE // 2, dense=True).shape[0]
        self._tensor("sin", sin, torch.float32, n_pos, ROPE // 2, dense=True)
        self._tensor("positions", positions, torch.int32, n, dense=True)
        self._tensor("slots", slots, torch.int64, n, dense=True)
        base, stride, pages = self._cache(cache)
        q = (None, 0, 0, None)
        if q_pe is not None:
            self._tensor("q_pe", q_pe, self.dtype, n, self.dims.n_heads, ROPE)
            q_out = self._out("q_out", q_out, (n, self.dims.n_heads, ROPE), self.dtype)
            q = (B._dptr(q_pe), q_pe.stride(0), q_pe.stride(1), B._dptr(q_out))
        elif q_out is not None:
            raise ValueError("q_out without q_pe")
        self._call("coli_latent_append", B._dptr(c), c.stride(0), B._dptr(norm_weight), float(eps), B._dptr(cos), B._dptr(sin), n_pos,
                   int(bool(interleaved)), B._dptr(positions), B._dptr(slots), n, base, stride, pages, *q)
        return q_out

    def plan(self, q_start, kv_len, n_tok=None):
        """Plan the absorbed attention of a step (coli_latent_plan): q_start
        int32 [B + 1], kv_len int32 [B].  n_tok is the number of tokens of the
        step; if not given it is read from q_start, a synchronising copy."""
        n_seq = self._starts("q_start", q_start)
        self._tensor("kv_len", kv_len, torch.int32, n_seq, dense=True)
        if n_tok is None:
            n_tok = int(q_start[-1])
        self._call("coli_latent_plan", B._dptr(q_start), B._dptr(kv_len), n_seq, n_tok)
        self._planned = (n_seq, n_tok)

    def decode(self, q_lat, q_pe, cache, block_table, scale, tree_mask=None, return_lse=False, out=None, lse=None):
        """Absorbed attention of the planned step (coli_latent_decode).

        q_lat [T, n_heads, 512], q_pe [T, n_heads, 64], cache [n_pages,
        page_size, 576], block_table int32 [B, max_pages], tree_mask int64
        [T, words] of ancestor bits or None for chains.  Returns out [T,
        n_heads, 512], or (out, lse fp32 [T, n_heads])."""
        if self._planned is None:
            raise B.ColiError(B.E_STATE, "no plan: plan() comes first")
        n_seq, n = self._planned
        h = self.dims.n_heads
        self._tensor("q_lat", q_lat, self.dtype, n, h, LATENT)
        self._tensor("q_pe", q_pe, self.dtype, n, h, ROPE)
        base, stride, pages = self._cache(cache)
        self._tensor("block_table", block_table, torch.int32, n_seq, None)
        words = 0
        if tree_mask is not None:
            words = self._tensor("tree_mask", tree_mask, torch.int64, n, None, dense=True).shape[1]
        out = self._out("out", out, (n, h, LATENT), self.dtype)
        if return_lse or lse is not None:
            lse = self._out("lse", lse, (n, h), torch.float32)
        self._call("coli_latent_decode", B._dptr(q_lat), q_lat.stride(0), q_lat.stride(1), B._dptr(q_pe), q_pe.stride(0), q_pe.stride(1),
                   base, stride, pages, B._dptr(block_table), block_table.stride(0), block_table.shape[1],
                   None if tree_mask is None else B._dptr(tree_mask), words, float(scale), n, B._dptr(out),
                   None if lse is None else B._dptr(lse))
        return (out, lse) if lse is not None else out

    def prompt(self, q, kv, k_pe, q_start, k_start, scale, causal=True, return_lse=False, out=None, lse=None):
        """Expanded attention of whole prompts (coli_latent_prompt).

        q [Tq, n_heads, nope + 64], kv [Tk, n_heads, nope + v_dim], k_pe [Tk,
        64], q_start and k_start int32 [B + 1].  Returns out [Tq, n_heads,
        v_dim], or (out, lse)."""
        d = self.dims
        n_q = self._tensor("q", q, self.dtype, None, d.n_heads, d.nope + d.rope).shape[0]
        n_k = self._tensor("kv", kv, self.dtype, None, d.n_heads, d.nope + d.v_dim).shape[0]
        self._tensor("k_pe", k_pe, self.dtype, n_k, d.rope)
        n_seq = self._starts("q_start", q_start)
        self._tensor("k_start", k_start, torch.int32, n_seq + 1, dense=True)
        out = self._out("out", out, (n_q, d.n_heads, d.v_dim), self.dtype)
        if return_lse or lse is not None:
            lse = self._out("lse", lse, (n_q, d.n_heads), torch.float32)
        self._call("coli_latent_prompt", B._dptr(q), q.stride(0), q.stride(1), B._dptr(kv), kv.stride(0), kv.stride(1), B._dptr(k_pe),
                   k_pe.stride(0), B._dptr(q_start), B._dptr(k_start), n_seq, n_q, n_k, int(bool(causal)), float(scale), B._dptr(out),
                   None if lse is None else B._dptr(lse))
        return (out, lse) if lse is not None else out

    def verify(self, probs, tokens, q_start, u, race, draft_probs=None, parents=None, max_path=None):
        """Accept drafted tokens and sample the next one (coli_draft_verify).

        probs [T, vocab] (fp32, bf16 or f16), draft_probs the same or None,
        tokens and parents int32 [T] (parents None: chains), u fp32 [T], race fp32
        [B, vocab].  Returns path int32 [B, max_path], count int32 [B] and
        next_tokens int32 [B, max_path]; max_path (default T) bounds the nodes
        of a path, node 0 among them."""
        if not isinstance(probs, torch.Tensor) or probs.dtype not in PROBS:
            raise TypeError(f"probs must be a tensor of {sorted(map(str, PROBS))}")
        n, vocab = self._tensor("probs", probs, probs.dtype, None, None).shape
        n_seq = self._starts("q_start", q_start)
        self._tensor("tokens", tokens, torch.int32, n, dense=True)
        self._tensor("u", u, torch.float32, n, dense=True)
        self._tensor("race", race, torch.float32, n_seq, vocab)
        if draft_probs is not None:
            self._tensor("draft_probs", draft_probs, probs.dtype, n, vocab)
        if parents is not None:
            self._tensor("parents", parents, torch.int32, n, dense=True)
        cols = max(n, 1) if max_path is None else int(max_path)
        path = torch.empty((n_seq, max(cols, 0)), dtype=torch.int32, device=self.device)
        count = torch.empty((n_seq,), dtype=torch.int32, device=self.device)
        nxt = torch.empty_like(path)

        def rows(t):   # a row stride of one row's tensor may be anything
            return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), vocab)

        self._call("coli_draft_verify", B._dptr(probs), rows(probs), None if draft_probs is None else B._dptr(draft_probs),
                   0 if draft_probs is None else rows(draft_probs), PROBS[probs.dtype], vocab, B._dptr(tokens),
                   None if parents is None else B._dptr(parents), B._dptr(q_start), n_seq, n, B._dptr(u), B._dptr(race), rows(race),
                   B._dptr(path), cols, B._dptr(count), B._dptr(nxt))
        return path, count, nxt

    def keep(self, cache, block_table, q_start, kv_len, path, n_tok=None):
        """Move the accepted nodes' cache rows together (coli_latent_keep), in
        place: cache [n_pages, page_size, 576], or [n_layers, ...] for every
        layer in one launch; path int32 [B, cols] as ``verify`` returns it."""
        layers, layer_stride = 1, 0
        if isinstance(cache, torch.Tensor) and cache.dim() == 4:
            layers, layer_stride = cache.shape[0], cache.stride(0)
            if layers == 0:
                return
            cache = cache[0]
        base, stride, pages = self._cache(cache)
        n_seq = self._starts("q_start", q_start)
        self._tensor("kv_len", kv_len, torch.int32, n_seq, dense=True)
        self._tensor("block_table", block_table, torch.int32, n_seq, None)
        self._tensor("path", path, torch.int32, n_seq, None)
        self._call("coli_latent_keep", base, stride, pages, layers, layer_stride, B._dptr(block_table), block_table.stride(0),
                   block_table.shape[1], B._dptr(q_start), B._dptr(kv_len), n_seq, self.dims.max_tokens if n_tok is None else n_tok,
                   B._dptr(path), path.stride(0), path.shape[1])

    def device_errors(self) -> int:
        """Read and clear the device error flags (synchronises the device)."""
        f = C.c_int32()
        st = B.lib.coli_serve_device_errors(self.handle, C.byref(f))
        if st != B.OK:
            raise B.ColiError(st, B.lib.coli_serve_last_error(self.handle).decode())
        return f.value
