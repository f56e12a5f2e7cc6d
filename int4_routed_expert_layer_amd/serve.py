"""Thin ctypes layer over the serving operators of include/coli_moe.h: the
paged latent cache (in 16 or 8 bits), latent attention (absorbed and expanded),
the verification of drafted tokens and beam search.

The pages' engine keeps 576 values a token in place of 32,768 (README "Come
funziona", compressed attention state) and drafts tokens that the main model
verifies in one batched forward; the operators are that step's attention and
acceptance, next to the expert layer of ``binding``.

A cache of the handle's 16-bit type has rows of 576 values, one of torch.uint8
rows of 656 bytes (``ROW8``: 512 e4m3 values, 64 16-bit rotary ones, 16 scale
exponents); every call that takes a cache takes either.

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
GROUP = 32                                    # latent values of an 8-bit row that share a scale
ROW8 = LATENT + 2 * ROPE + LATENT // GROUP    # bytes of an 8-bit row
HALF = {"bf16": (0, torch.bfloat16), "f16": (1, torch.float16)}
PROBS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

_append, _plan, _decode = B.lib.coli_latent_append, B.lib.coli_latent_plan, B.lib.coli_latent_decode
_prompt, _verify, _keep = B.lib.coli_latent_prompt, B.lib.coli_draft_verify, B.lib.coli_latent_keep
_append8, _decode8, _keep8 = B.lib.coli_latent8_append, B.lib.coli_latent8_decode, B.lib.coli_latent8_keep
_read, _plan_shared = B.lib.coli_latent_read, B.lib.coli_latent_plan_shared
_select, _reorder = B.lib.coli_beam_select, B.lib.coli_beam_reorder


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle without a stream object, where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


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
        self.index = device
        self.page_size = page_size
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
    # The calls of a decode step take a few microseconds on the device, so the
    # checks look at a tensor in one pass and only a failure is taken apart.
    def _call(self, call, *args):
        if not self.handle:
            raise ValueError("the handle is closed")
        st = call(self.handle, *args, _raw_stream(self.index))
        if st != B.OK:
            raise B.ColiError(st, B.lib.coli_serve_last_error(self.handle).decode())

    def _dense(self, name, t, dtype, shape):
        """Address of a contiguous tensor of exactly this type and shape."""
        try:
            if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == self.index:
                return t.data_ptr()
        except AttributeError:
            pass
        self._refuse(name, t, dtype, shape, True)
        return t.data_ptr()

    def _rows(self, name, t, dtype, shape):
        """Address of a tensor of this type and shape whose last dimension is contiguous."""
        try:
            if t.dtype is dtype and t.shape == shape and t.get_device() == self.index and (t.stride()[-1] == 1 or t.shape[-1] <= 1):
                return t.data_ptr()
        except (AttributeError, IndexError):
            pass
        self._refuse(name, t, dtype, shape, False)
        return t.data_ptr()

    def _refuse(self, name, t, dtype, shape, dense):
        """Raises what is wrong with the tensor; returns if nothing is (an empty one)."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the handle on {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} is {t.dtype}, must be {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, must be {tuple(shape)}")
        if t.numel() and (not t.is_contiguous() if dense else t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1):
            raise ValueError(f"{name} must be contiguous" + ("" if dense else " in its last dimension"))

    def _sizes(self, name, t, dims):
        """Shape of a tensor of this many dimensions."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.dim() != dims:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, must have {dims} dimensions")
        return t.shape

    def _cache(self, cache, layers=()):
        """Address, page stride, pages and whether it is of 8 bits; `layers` is () or the leading (n_layers,)."""
        try:
            kind, shape, strides = cache.dtype, cache.shape, cache.stride()
            width = ROW8 if kind is torch.uint8 else ROW if kind is self.dtype else 0
            if len(shape) == 3 + len(layers) and shape[-1] == width == strides[-2] and shape[-2] == self.page_size and strides[-1] == 1 and shape[-3] > 1 and cache.get_device() == self.index:
                return cache.data_ptr(), strides[-3], shape[-3], width == ROW8
        except (AttributeError, IndexError):
            pass
        pages = self._sizes("cache", cache, 3 + len(layers))[-3]
        eight = cache.dtype is torch.uint8
        width = ROW8 if eight else ROW
        at = self._rows("cache", cache, torch.uint8 if eight else self.dtype, (*layers, pages, self.page_size, width))
        page, row = cache.stride()[-3:-1]
        if row != width and self.page_size > 1:
            raise ValueError("the rows of a cache page must be contiguous")
        return at, page if pages > 1 else max(page, self.page_size * width), pages, eight

    def _layers(self, cache):
        """The same of a cache with or without a leading dimension of layers, and their number and stride."""
        if isinstance(cache, torch.Tensor) and cache.dim() == 4:
            n = cache.shape[0]
            return *self._cache(cache, (n,)), n, cache.stride()[0]
        return *self._cache(cache), 1, 0

    def _table(self, block_table, n_seq):
        try:
            rows, cols = block_table.shape
            row, step = block_table.stride()
            if rows == n_seq and step == 1 and block_table.dtype is torch.int32 and block_table.get_device() == self.index:
                return block_table.data_ptr(), row, cols
        except (AttributeError, ValueError):
            pass
        cols = self._sizes("block_table", block_table, 2)[1]
        return self._rows("block_table", block_table, torch.int32, (n_seq, cols)), block_table.stride()[0], cols

    def _out(self, name, out, shape, dtype):
        """An output tensor and its address."""
        if out is None:
            out = torch.empty(*shape, dtype=dtype, device=self.device)
            return out, out.data_ptr()
        return out, self._dense(name, out, dtype, shape)

    def _starts(self, name, q_start):
        n = self._sizes(name, q_start, 1)[0]
        if n < 1:
            raise ValueError(f"{name} needs n_seq + 1 entries")
        return self._dense(name, q_start, torch.int32, (n,)), n - 1

    # -- operators ---------------------------------------------------------
    def append(self, c, norm_weight, eps, cos, sin, positions, slots, cache, q_pe=None, q_out=None, interleaved=True):
        """Write the latent rows of new tokens into the cache (coli_latent_append).

        c [T, 576], norm_weight [512], cos and sin fp32 [n_positions, 32],
        positions int32 [T], slots int64 [T] (negative: not cached), cache
        [n_pages, page_size, 576], or 656 bytes a row.  Returns the turned q_pe [T, n_heads, 64], or
        None without q_pe."""
        n = self._sizes("c", c, 2)[0]
        n_pos = self._sizes("cos", cos, 2)[0]
        pc = self._rows("c", c, self.dtype, (n, ROW))
        pw = self._dense("norm_weight", norm_weight, self.dtype, (LATENT,))
        pcos = self._dense("cos", cos, torch.float32, (n_pos, ROPE // 2))
        psin = self._dense("sin", sin, torch.float32, (n_pos, ROPE // 2))
        ppos = self._dense("positions", positions, torch.int32, (n,))
        pslot = self._dense("slots", slots, torch.int64, (n,))
        base, page, pages, eight = self._cache(cache)
        pq = po = None
        qt = qh = 0
        if q_pe is not None:
            shape = (n, self.dims.n_heads, ROPE)
            pq = self._rows("q_pe", q_pe, self.dtype, shape)
            qt, qh, _ = q_pe.stride()
            q_out, po = self._out("q_out", q_out, shape, self.dtype)
        elif q_out is not None:
            raise ValueError("q_out without q_pe")
        self._call(_append8 if eight else _append, pc, c.stride()[0], pw, eps, pcos, psin, n_pos, 1 if interleaved else 0, ppos, pslot, n, base, page, pages, pq, qt, qh, po)
        return q_out

    def plan(self, q_start, kv_len, n_tok=None, group_start=None, prefix_len=None):
        """Plan the absorbed attention of a step (coli_latent_plan): q_start
        int32 [B + 1], kv_len int32 [B].  n_tok is the number of tokens of the
        step; if not given it is read from q_start, a synchronising copy.

        With group_start int32 [G + 1] and prefix_len int32 [G] the sequences
        group_start[g] .. group_start[g + 1] - 1 begin with the same prefix_len[g]
        cached tokens, which are attended to once for all of them
        (coli_latent_plan_shared, which says where that is the faster)."""
        ps, n_seq = self._starts("q_start", q_start)
        pl = self._dense("kv_len", kv_len, torch.int32, (n_seq,))
        if (group_start is None) != (prefix_len is None):
            raise ValueError("group_start and prefix_len go together")
        if group_start is not None:
            pg, groups = self._starts("group_start", group_start)
            pp = self._dense("prefix_len", prefix_len, torch.int32, (groups,))
        if n_tok is None:
            n_tok = int(q_start[-1])
        if group_start is None:
            self._call(_plan, ps, pl, n_seq, n_tok)
        else:
            self._call(_plan_shared, ps, pl, n_seq, n_tok, pg, pp, groups)
        self._planned = (n_seq, n_tok)

    def decode(self, q_lat, q_pe, cache, block_table, scale, tree_mask=None, return_lse=False, out=None, lse=None):
        """Absorbed attention of the planned step (coli_latent_decode).

        q_lat [T, n_heads, 512], q_pe [T, n_heads, 64], cache [n_pages,
        page_size, 576] or [..., 656] bytes, block_table int32 [B, max_pages], tree_mask int64
        [T, words] of ancestor bits or None for chains.  Returns out [T,
        n_heads, 512], or (out, lse fp32 [T, n_heads])."""
        if self._planned is None:
            raise B.ColiError(B.E_STATE, "no plan: plan() comes first")
        n_seq, n = self._planned
        h = self.dims.n_heads
        pl = self._rows("q_lat", q_lat, self.dtype, (n, h, LATENT))
        pp = self._rows("q_pe", q_pe, self.dtype, (n, h, ROPE))
        base, page, pages, eight = self._cache(cache)
        table, row, cols = self._table(block_table, n_seq)
        words, pm = 0, None
        if tree_mask is not None:
            words = self._sizes("tree_mask", tree_mask, 2)[1]
            pm = self._dense("tree_mask", tree_mask, torch.int64, (n, words))
        out, po = self._out("out", out, (n, h, LATENT), self.dtype)
        pe = None
        if return_lse or lse is not None:
            lse, pe = self._out("lse", lse, (n, h), torch.float32)
        lt, lh, _ = q_lat.stride()
        qt, qh, _ = q_pe.stride()
        self._call(_decode8 if eight else _decode, pl, lt, lh, pp, qt, qh, base, page, pages, table, row, cols, pm, words, scale, n, po, pe)
        return out if pe is None else (out, lse)

    def prompt(self, q, kv, k_pe, q_start, k_start, scale, causal=True, return_lse=False, out=None, lse=None):
        """Expanded attention of whole prompts (coli_latent_prompt).

        q [Tq, n_heads, nope + 64], kv [Tk, n_heads, nope + v_dim], k_pe [Tk,
        64], q_start and k_start int32 [B + 1].  Returns out [Tq, n_heads,
        v_dim], or (out, lse)."""
        d = self.dims
        h = d.n_heads
        n_q, n_k = self._sizes("q", q, 3)[0], self._sizes("kv", kv, 3)[0]
        pq = self._rows("q", q, self.dtype, (n_q, h, d.nope + ROPE))
        pkv = self._rows("kv", kv, self.dtype, (n_k, h, d.nope + d.v_dim))
        pk = self._rows("k_pe", k_pe, self.dtype, (n_k, ROPE))
        ps, n_seq = self._starts("q_start", q_start)
        pks = self._dense("k_start", k_start, torch.int32, (n_seq + 1,))
        out, po = self._out("out", out, (n_q, h, d.v_dim), self.dtype)
        pe = None
        if return_lse or lse is not None:
            lse, pe = self._out("lse", lse, (n_q, h), torch.float32)
        qt, qh, _ = q.stride()
        kt, kh, _ = kv.stride()
        self._call(_prompt, pq, qt, qh, pkv, kt, kh, pk, k_pe.stride()[0], ps, pks, n_seq, n_q, n_k, 1 if causal else 0, scale, po, pe)
        return out if pe is None else (out, lse)

    def verify(self, probs, tokens, q_start, u, race, draft_probs=None, parents=None, max_path=None):
        """Accept drafted tokens and sample the next one (coli_draft_verify).

        probs [T, vocab] (fp32, bf16 or f16), draft_probs the same or None,
        tokens and parents int32 [T] (parents None: chains), u fp32 [T], race fp32
        [B, vocab].  Returns path int32 [B, max_path], count int32 [B] and
        next_tokens int32 [B, max_path]; max_path (default T) bounds the nodes
        of a path, node 0 among them."""
        n, vocab = self._sizes("probs", probs, 2)
        kind = PROBS.get(probs.dtype)
        if kind is None:
            raise TypeError(f"probs is {probs.dtype}, must be one of {sorted(map(str, PROBS))}")
        pp = self._rows("probs", probs, probs.dtype, (n, vocab))
        ps, n_seq = self._starts("q_start", q_start)
        pt = self._dense("tokens", tokens, torch.int32, (n,))
        pu = self._dense("u", u, torch.float32, (n,))
        pr = self._rows("race", race, torch.float32, (n_seq, vocab))
        pd = pa = None
        if draft_probs is not None:
            pd = self._rows("draft_probs", draft_probs, probs.dtype, (n, vocab))
        if parents is not None:
            pa = self._dense("parents", parents, torch.int32, (n,))
        cols = max(n, 1) if max_path is None else max_path
        if cols < 1:
            raise ValueError(f"max_path {cols} must be >= 1")
        path = torch.empty(n_seq, cols, dtype=torch.int32, device=self.device)
        nxt = torch.empty_like(path)
        count = torch.empty(n_seq, dtype=torch.int32, device=self.device)

        def rows(t):   # a tensor of one row may have any row stride
            return t.stride()[0] if t.shape[0] > 1 else vocab

        self._call(_verify, pp, rows(probs), pd, 0 if pd is None else rows(draft_probs), kind, vocab, pt, pa, ps, n_seq, n, pu, pr, rows(race),
                   path.data_ptr(), cols, count.data_ptr(), nxt.data_ptr())
        return path, count, nxt

    def keep(self, cache, block_table, q_start, kv_len, path, n_tok=None):
        """Move the accepted nodes' cache rows together (coli_latent_keep), in
        place: cache [n_pages, page_size, 576] (or 656 bytes a row), or [n_layers, ...]
        for every layer in one launch; path int32 [B, cols] as ``verify`` returns it."""
        if isinstance(cache, torch.Tensor) and cache.dim() == 4 and cache.shape[0] == 0:
            return
        base, page, pages, eight, layers, layer_stride = self._layers(cache)
        ps, n_seq = self._starts("q_start", q_start)
        pl = self._dense("kv_len", kv_len, torch.int32, (n_seq,))
        table, row, cols = self._table(block_table, n_seq)
        most = self._sizes("path", path, 2)[1]
        pp = self._rows("path", path, torch.int32, (n_seq, most))
        self._call(_keep8 if eight else _keep, base, page, pages, layers, layer_stride, table, row, cols, ps, pl, n_seq, self.dims.max_tokens if n_tok is None else n_tok,
                   pp, path.stride()[0], most)

    def read(self, cache, block_table, k_start, n_rows=None, first=None, out=None):
        """Cached rows as 16-bit values, one sequence behind the other (coli_latent_read).

        Row k_start[b] + i of the result [n_rows, 576] is position first[b] + i of
        sequence b (first None: from position 0); k_start int32 [B + 1], first int32
        [B].  n_rows, if neither it nor out is given, is read from k_start, a
        synchronising copy.  Rows of out that no sequence covers stay as they are
        (those of a new tensor are unspecified)."""
        base, page, pages, eight = self._cache(cache)
        ps, n_seq = self._starts("k_start", k_start)
        table, row, cols = self._table(block_table, n_seq)
        pf = None if first is None else self._dense("first", first, torch.int32, (n_seq,))
        if n_rows is None:
            n_rows = int(k_start[-1]) if out is None else self._sizes("out", out, 2)[0]
        if n_rows < 0:
            raise ValueError(f"n_rows {n_rows} must be >= 0")
        if out is None:
            out = torch.empty(n_rows, ROW, dtype=self.dtype, device=self.device)
        po = self._rows("out", out, self.dtype, (n_rows, ROW))
        self._call(_read, 1 if eight else 0, base, page, pages, table, row, cols, pf, ps, n_seq, n_rows, po, out.stride()[0] if n_rows > 1 else ROW)
        return out

    def beam_select(self, logits, scores, keep):
        """The best continuations of each group's beams (coli_beam_select).

        logits [n_groups * beams, vocab] (fp32, bf16 or f16), scores fp32 [n_groups,
        beams].  Returns scores fp32, parents (the beam within the group) and tokens,
        int32, [n_groups, keep] each, from the best down; -inf, -1, -1 where there
        are fewer."""
        n, vocab = self._sizes("logits", logits, 2)
        groups, beams = self._sizes("scores", scores, 2)
        kind = PROBS.get(logits.dtype)
        if kind is None:
            raise TypeError(f"logits is {logits.dtype}, must be one of {sorted(map(str, PROBS))}")
        if n != groups * beams:
            raise ValueError(f"logits has {n} rows, must have one for each of the {groups * beams} scores")
        pl = self._rows("logits", logits, logits.dtype, (n, vocab))
        ps = self._dense("scores", scores, torch.float32, (groups, beams))
        if keep < 1:
            raise ValueError(f"keep {keep} must be >= 1")
        best, parents, tokens = torch.empty(3, groups, keep, dtype=torch.int32, device=self.device).unbind()
        best = best.view(torch.float32)
        self._call(_select, pl, logits.stride()[0] if n > 1 else vocab, kind, vocab, ps, groups, beams, keep, best.data_ptr(), parents.data_ptr(), tokens.data_ptr())
        return best, parents, tokens

    def beam_reorder(self, cache, block_table, kv_len, parents, out=None):
        """The cache and block tables of the beams that go on (coli_beam_reorder).

        parents int32 [n_groups, beams]: the beam of its group that each place
        continues, -1 for none; kv_len int32 [n_groups * beams], equal within a
        group; block_table [n_groups * beams, cols].  Rows of shared last pages are
        copied within cache ([n_pages, page_size, ...] or [n_layers, ...], all layers
        in one launch).  Returns the new block table; of whole pages that then stand in
        none of its rows the caller may dispose."""
        groups, beams = self._sizes("parents", parents, 2)
        pp = self._dense("parents", parents, torch.int32, (groups, beams))
        n = groups * beams
        table, row, cols = self._table(block_table, n)
        pl = self._dense("kv_len", kv_len, torch.int32, (n,))
        base, page, pages, eight, layers, layer_stride = self._layers(cache)
        if out is None:
            out = torch.empty(n, cols, dtype=torch.int32, device=self.device)
        po = self._rows("out", out, torch.int32, (n, cols))
        self._call(_reorder, 1 if eight else 0, base, page, pages, layers, layer_stride, table, row if n > 1 else cols, cols, pl, pp, groups, beams, po,
                   out.stride()[0] if n > 1 else cols)
        return out

    def device_errors(self) -> int:
        """Read and clear the device error flags (synchronises the device)."""
        if not self.handle:
            raise ValueError("the handle is closed")
        f = C.c_int32()
        st = B.lib.coli_serve_device_errors(self.handle, C.byref(f))
        if st != B.OK:
            raise B.ColiError(st, B.lib.coli_serve_last_error(self.handle).decode())
        return f.value
