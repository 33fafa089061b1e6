"""Python binding of libkvq with the C ABI's names (include/kvq.h).

Marshalling only: tensors become device pointers, structs are passed by
reference, a non-zero status raises KvqError.  Device memory comes from
PyTorch (caller-owned); the library never allocates.

Helpers:
  LayerCache -- allocates one layer's pool arrays as torch tensors and holds
                the kvq_layout / kvq_pool descriptors;
  Batch      -- block table + sequence lengths (kvq_seqs);
  Workspace  -- a zero-filled, 256-byte aligned device buffer;
  Allocator  -- the host page allocator (free list + reference counts);
  RopeTable  -- rotary frequencies on the device (kvq_rope);
  AttnMod    -- score forms of the new tokens' attention (kvq_attn_mod).
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._abi import (BITS_E4M3, BLOCK_TOKENS, HEAD_DIM, K_GROUP_TOKENS, V_SYMMETRIC, KvqError, Layout, Pool,  # noqa: F401
                   Seqs, check, lib)


def _p(x):
    """Device/host pointer of a tensor (None stays NULL; ints pass through)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _s(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ref(x):
    return ctypes.byref(x.c if hasattr(x, "c") else x)


# ------------------------------------------------------------------ descriptors

def make_layout(n_q_heads, n_kv_heads, bits, v_group_dims=64):
    return Layout(HEAD_DIM, n_q_heads, n_kv_heads, BLOCK_TOKENS, bits, K_GROUP_TOKENS, v_group_dims)


class LayerCache:
    """Device storage of one layer (torch tensors) plus its kvq_layout/kvq_pool."""

    def __init__(self, n_q_heads, n_kv_heads, bits, num_blocks, max_seqs, v_group_dims=64, t_cap=0,
                 device="cuda"):
        self.layout = make_layout(n_q_heads, n_kv_heads, bits, v_group_dims)
        H, d, P = n_kv_heads, HEAD_DIM, BLOCK_TOKENS
        self.bits, self.H, self.num_blocks, self.max_seqs, self.t_cap = bits, H, num_blocks, max_seqs, t_cap
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)  # noqa: E731
        self.k_codes = self.v_codes = self.k_sz = self.v_sz = self.k_tail = None
        self.k16 = self.v16 = self.kT = self.k_absmax = None
        if bits == _abi.BITS_E4M3:
            self.k_codes = z((num_blocks, H, P, d), torch.uint8)
            self.v_codes = z((num_blocks, H, P, d), torch.uint8)
        elif bits == 16:
            self.k16 = z((num_blocks, H, P, d), torch.float16)
            self.v16 = z((num_blocks, H, P, d), torch.float16)
            if t_cap:
                self.kT = z((max_seqs, H, d, t_cap), torch.float16)
                self.k_absmax = z((max_seqs, H, d), torch.float32)
        else:
            R = d * (bits & 0xFF) // 8
            self.k_codes = z((num_blocks, H, P, R), torch.uint8)
            self.v_codes = z((num_blocks, H, P, R), torch.uint8)
            self.k_sz = z((num_blocks, H, d, 2), torch.float16)
            self.v_sz = z((num_blocks, H, P, d // v_group_dims, 2), torch.float16)
            self.k_tail = z((max_seqs, H, K_GROUP_TOKENS, d), torch.float16)
        self.c = Pool(num_blocks, max_seqs, t_cap, _p(self.k_codes), _p(self.v_codes), _p(self.k_sz),
                      _p(self.v_sz), _p(self.k_tail), _p(self.k16), _p(self.v16), _p(self.kT),
                      _p(self.k_absmax))


class Batch:
    """Block table + sequence lengths of a batch (kvq_seqs)."""

    def __init__(self, block_table, seq_lens, max_len):
        assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32
        self.block_table = block_table.contiguous()
        self.seq_lens = seq_lens.contiguous()
        self.max_len = int(max_len)
        B, mb = self.block_table.shape
        self.c = Seqs(_p(self.block_table), _p(self.seq_lens), B, mb, self.max_len, 0)

    @property
    def batch(self):
        return self.c.batch


class Workspace:
    """Zero-filled device workspace of `nbytes` (rounded to 256)."""

    def __init__(self, nbytes, device="cuda"):
        n = max(256, (int(nbytes) + 255) // 256 * 256)
        self.t = torch.zeros(n + 256, dtype=torch.uint8, device=device)
        off = (-self.t.data_ptr()) % 256
        self.ptr = self.t.data_ptr() + off
        self.nbytes = n


class Allocator:
    """Host page allocator (free list, reference counts for shared pages)."""

    def __init__(self, num_blocks, seed=0):
        self.h = lib().kvq_alloc_create(int(num_blocks), int(seed))
        if not self.h:
            raise KvqError(_abi.KVQ_ERR_INVALID_ARG, "kvq_alloc_create", _abi.last_error())
        self.num_blocks = int(num_blocks)

    def alloc(self, n):
        ids = (ctypes.c_int32 * max(n, 1))()
        check(lib().kvq_block_alloc(self.h, int(n), ids), "kvq_block_alloc")
        return [ids[i] for i in range(n)]

    def ref(self, page):
        check(lib().kvq_block_ref(self.h, int(page)), "kvq_block_ref")

    def free(self, page):
        check(lib().kvq_block_free(self.h, int(page)), "kvq_block_free")

    def free_n(self, pages):
        """free() for a list of pages; nothing changes when one of them is refused."""
        ids = _i32s(pages)
        check(lib().kvq_block_free_n(self.h, len(pages), ids), "kvq_block_free_n")

    def fork(self, cache, n_tokens, pages):
        """(pages, pairs) of a fork of a sequence of n_tokens on `pages`: the fork's own pages and the
        (source, destination) pairs that kv_pages_copy has to copy."""
        n = (int(n_tokens) + BLOCK_TOKENS - 1) // BLOCK_TOKENS
        if len(pages) < n:
            raise KvqError(_abi.KVQ_ERR_INVALID_ARG, "kvq_block_fork", f"{len(pages)} pages for {n_tokens} tokens")
        dst, pairs, m = (ctypes.c_int32 * max(n, 1))(), (ctypes.c_int32 * 8)(), ctypes.c_int32(0)
        check(lib().kvq_block_fork(self.h, ctypes.byref(_layout_of(cache)), int(n_tokens), _i32s(pages), dst, pairs,
                                   ctypes.byref(m)), "kvq_block_fork")
        return list(dst[:n]), [(pairs[2 * i], pairs[2 * i + 1]) for i in range(m.value)]

    def compact(self, max_moves=None):
        """(pairs, map): the moves that bring the used pages to the lowest ids (at most max_moves of them),
        for kv_pages_copy, and the new id of every page, for kvq_table_remap."""
        n = self.num_blocks if max_moves is None else int(max_moves)
        pairs, m = (ctypes.c_int32 * max(2 * n, 1))(), ctypes.c_int32(0)
        new_id = (ctypes.c_int32 * self.num_blocks)()
        check(lib().kvq_block_compact(self.h, n, pairs, new_id, ctypes.byref(m)), "kvq_block_compact")
        return [(pairs[2 * i], pairs[2 * i + 1]) for i in range(m.value)], list(new_id)

    def refcount(self, page):
        r = lib().kvq_block_refcount(self.h, int(page))
        if r < 0:
            raise KvqError(r, "kvq_block_refcount", _abi.last_error())
        return r

    def num_free(self):
        return lib().kvq_alloc_num_free(self.h)

    def __del__(self):
        h = getattr(self, "h", None)
        if h:
            lib().kvq_alloc_destroy(h)
            self.h = None


class RopeTable:
    """Rotary frequencies of kv_qk_norm_rope, laid out once: kvq_rope plus its device steps and mscale.

    scaling: "plain", "linear", "ntk", "yarn" (low > high: fast and slow turns, 32 and 1 by default) or
    "knees" (low < high turns, 1 and 4 by default), as KVQ_ROPE_* in kvq.h."""

    def __init__(self, rot_dim=HEAD_DIM, base=10000.0, interleaved=False, scaling="plain", factor=1.0, original_len=0,
                 low=None, high=None, device="cuda"):
        if scaling not in _abi.ROPE_SCALINGS:
            raise KvqError(_abi.KVQ_ERR_UNSUPPORTED, "kvq_rope_steps", f"scaling {scaling!r}")
        d_low, d_high = (32.0, 1.0) if scaling == "yarn" else (1.0, 4.0)
        self.c = _abi.Rope(int(rot_dim), int(bool(interleaved)), _abi.ROPE_SCALINGS[scaling], int(original_len),
                           float(base), float(factor), d_low if low is None else float(low),
                           d_high if high is None else float(high))
        steps, m = (ctypes.c_uint64 * max(1, int(rot_dim) // 2))(), ctypes.c_float(0)
        check(lib().kvq_rope_steps(ctypes.byref(self.c), steps, ctypes.byref(m)), "kvq_rope_steps")
        self.mscale = m.value
        signed = [x - (1 << 64) if x >> 63 else x for x in steps]
        self.steps = torch.tensor(signed, dtype=torch.int64, device=device)
        self.at, self.gpu = self.steps.data_ptr(), self.steps.get_device()


class AttnMod:
    """Score forms of kv_decode_attn and kv_chunk_attn (kvq_attn_mod); keeps its tensors alive."""

    def __init__(self, scale=0.0, softcap=0.0, window=0, n_sink=0, slopes=None, prefix_len=None, doc_start=None):
        gpu = _gpu() if any(x is not None for x in (slopes, prefix_len, doc_start)) else -1
        at = [_dev(x, dt, None, gpu, "kvq_attn_mod", name)
              for x, dt, name in ((slopes, torch.float32, "slopes"), (prefix_len, torch.int32, "prefix_len"),
                                  (doc_start, torch.int32, "doc_start"))]
        self.slopes, self.prefix_len, self.doc_start = slopes, prefix_len, doc_start
        self.gpu = gpu
        self.c = _abi.AttnModStruct(float(scale), float(softcap), int(window), int(n_sink), *at)


_ROW = (HEAD_DIM,)


def _i32s(xs):
    return (ctypes.c_int32 * max(len(xs), 1))(*[int(x) for x in xs])


def _gpu():
    return torch._C._cuda_getDevice()


def _raw(stream, gpu):
    """The cudaStream_t of `stream`, or of the current stream of GPU `gpu`."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(gpu)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dev(x, dtype, shape, gpu, fn, name):
    """Address of x, or None for None.  Refuses what would be read or written wrongly through a bare
    pointer: a tensor that is not on GPU `gpu`, of another type, with gaps, or not of `shape` (None: any)."""
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        if x.dtype is dtype and (shape is None or x.shape == shape) and x.is_contiguous() and x.get_device() == gpu:
            return x.data_ptr()
        have = f"{x.dtype} {tuple(x.shape)} on {x.device}" + ("" if x.is_contiguous() else ", not contiguous")
    else:
        have = f"{type(x).__name__}"
    raise KvqError(_abi.KVQ_ERR_INVALID_ARG, fn, f"{name}: {have} instead of a contiguous {dtype} tensor"
                   f"{'' if shape is None else ' ' + str(tuple(shape))} on GPU {gpu}")


def _need(x, fn, name):
    if x is None:
        raise KvqError(_abi.KVQ_ERR_INVALID_ARG, fn, f"{name} is missing")
    return x


def _mod(mod, fn, layout, batch, rows, gpu):
    """kvq_attn_mod by reference, its tensors' sizes checked against the call's."""
    if mod is None:
        return None
    if mod.gpu >= 0:
        for x, n, name in ((mod.slopes, layout.n_q_heads, "slopes"), (mod.prefix_len, batch, "prefix_len"),
                           (mod.doc_start, rows, "doc_start")):
            if x is not None and (x.numel() < n or mod.gpu != gpu):
                raise KvqError(_abi.KVQ_ERR_INVALID_ARG, fn, f"{name}: {x.numel()} entries on GPU {mod.gpu} for {n} on {gpu}")
    return ctypes.byref(mod.c)


# ------------------------------------------------------------------ the C ABI, same names

def kv_quant_pack(cache, seqs, seq, t_start, n_tokens, k, v, stride_t=None, stream=None):
    if stride_t is None:
        stride_t = cache.H * HEAD_DIM
    return check(lib().kv_quant_pack(_ref(cache.layout), _ref(cache), _ref(seqs), int(seq), int(t_start),
                                      int(n_tokens), _p(k), _p(v), int(stride_t), _s(stream)), "kv_quant_pack")


def kv_page_append_ws():
    return lib().kv_page_append_ws()


def kv_page_append(cache, seqs, k_new, v_new, ws, stream=None):
    return check(lib().kv_page_append(_ref(cache.layout), _ref(cache), _ref(seqs), _p(k_new), _p(v_new), ws.ptr,
                                      ws.nbytes, _s(stream)), "kv_page_append")


def kv_decode_attn_quant_ws(cache, seqs):
    return lib().kv_decode_attn_quant_ws(_ref(cache.layout), _ref(seqs))


def kv_decode_attn_quant(cache, seqs, q, out, ws, stream=None):
    return check(lib().kv_decode_attn_quant(_ref(cache.layout), _ref(cache), _ref(seqs), _p(q), _p(out), ws.ptr,
                                            ws.nbytes, _s(stream)), "kv_decode_attn_quant")


def kv_decode_attn_quant_noalloc(cache, seqs, q, out, stream=None):
    """kv_decode_attn_quant with the library's built-in scratch array instead of a
    workspace, for callers that may not allocate device memory."""
    return check(lib().kv_decode_attn_quant_noalloc(_ref(cache.layout), _ref(cache), _ref(seqs), _p(q), _p(out),
                                                    _s(stream)), "kv_decode_attn_quant_noalloc")


def kv_decode_attn_quant_noalloc_max_scratch():
    return lib().kv_decode_attn_quant_noalloc_max_scratch()


def kv_decode_attn_quant_plan(cache, seqs, noalloc=False):
    """(n_splits, groups_per_split) the quantized attention uses for this batch."""
    n, g = ctypes.c_int32(0), ctypes.c_int32(0)
    check(lib().kv_decode_attn_quant_plan(_ref(cache.layout), _ref(seqs), int(bool(noalloc)), ctypes.byref(n),
                                          ctypes.byref(g)), "kv_decode_attn_quant_plan")
    return n.value, g.value


def _layout_of(x):
    return x.layout if hasattr(x, "layout") else x


def kv_outlier_channels_ws(layout):
    """Workspace bytes of kv_outlier_channels (`layout`: a Layout or a cache)."""
    return lib().kv_outlier_channels_ws(ctypes.byref(_layout_of(layout)))


def kv_outlier_channels(layout, k, n_tokens, n_out, out_ch, ws, var=None, stride_t=None, stream=None):
    """The n_out largest-variance key channels per kv head of k [n_tokens][H_kv][d] (fp16)
    into out_ch [H_kv][n_out] (int32), optionally the variances into var [H_kv][d] (fp64)."""
    st = stride_t if stride_t is not None else k.stride(0)
    return check(lib().kv_outlier_channels(ctypes.byref(_layout_of(layout)), _p(k), n_tokens, st, n_out, _p(out_ch),
                                           _p(var), ws.ptr, ws.nbytes, _s(stream)), "kv_outlier_channels")


def kv_outlier_isolate(cache, seqs, seq, t_start, n_tokens, k, n_out, out_ch, k_out, stride_t=None, stream=None):
    st = stride_t if stride_t is not None else k.stride(0)
    return check(lib().kv_outlier_isolate(_ref(cache.layout), _ref(cache), _ref(seqs), seq, t_start, n_tokens, _p(k),
                                          st, n_out, _p(out_ch), _p(k_out), _s(stream)), "kv_outlier_isolate")


def kv_outlier_append_ws():
    return lib().kv_outlier_append_ws()


def kv_outlier_append(cache, seqs, n_out, out_ch, k_out, ws, stream=None):
    return check(lib().kv_outlier_append(_ref(cache.layout), _ref(cache), _ref(seqs), n_out, _p(out_ch), _p(k_out),
                                         ws.ptr, ws.nbytes, _s(stream)), "kv_outlier_append")


def kv_decode_attn_quant_outlier(cache, seqs, q, n_out, out_ch, k_out, out, ws, stream=None):
    return check(lib().kv_decode_attn_quant_outlier(_ref(cache.layout), _ref(cache), _ref(seqs), _p(q), n_out,
                                                    _p(out_ch), _p(k_out), _p(out), ws.ptr, ws.nbytes, _s(stream)),
                 "kv_decode_attn_quant_outlier")


def kv_critical_score(cache, seqs, q, n_crit, crit, scores, score_stride=None, stream=None):
    if score_stride is None:
        score_stride = scores.shape[-1]
    return check(lib().kv_critical_score(_ref(cache.layout), _ref(cache), _ref(seqs), _p(q), int(n_crit), _p(crit),
                                         _p(scores), int(score_stride), _s(stream)), "kv_critical_score")


def kv_group_critical_score(cache, seqs, q, n_crit, crit, scores, score_stride=None, stream=None):
    if score_stride is None:
        score_stride = scores.shape[-1]
    return check(lib().kv_group_critical_score(_ref(cache.layout), _ref(cache), _ref(seqs), _p(q), int(n_crit),
                                               _p(crit), _p(scores), int(score_stride), _s(stream)),
                 "kv_group_critical_score")


def kv_append_critical_score_ws():
    return lib().kv_append_critical_score_ws()


def kv_append_critical_score(cache, seqs, k_new, v_new, q, n_crit, crit, scores, hist, n_sink, window, ws,
                             score_stride=None, stream=None):
    if score_stride is None:
        score_stride = scores.shape[-1]
    return check(lib().kv_append_critical_score(_ref(cache.layout), _ref(cache), _ref(seqs), _p(k_new), _p(v_new),
                                                _p(q), int(n_crit), _p(crit), _p(scores), int(score_stride),
                                                _p(hist), int(n_sink), int(window), ws.ptr, ws.nbytes, _s(stream)),
                 "kv_append_critical_score")


def kv_select_sparse_attn_ws():
    return lib().kv_select_sparse_attn_ws()


def kv_select_sparse_attn(cache, seqs, q, scores, hist, k_fixed, ratio, n_sink, window, sel, sel_count, out, ws,
                          score_stride=None, stream=None):
    if score_stride is None:
        score_stride = scores.shape[-1]
    sel_cap = int(sel.shape[-1]) if sel is not None else 0
    return check(lib().kv_select_sparse_attn(_ref(cache.layout), _ref(cache), _ref(seqs), _p(q), _p(scores),
                                             int(score_stride), _p(hist), int(k_fixed), float(ratio), int(n_sink),
                                             int(window), _p(sel), sel_cap, _p(sel_count), _p(out), ws.ptr,
                                             ws.nbytes, _s(stream)), "kv_select_sparse_attn")


def kv_sparse_layer_decode_ws():
    return lib().kv_sparse_layer_decode_ws()


def kv_sparse_layer_decode(cache, seqs, k_new, v_new, q, n_crit, k_fixed, ratio, n_sink, window, out, ws,
                           scores=None, sel=None, sel_count=None, stream=None):
    stride = int(scores.shape[-1]) if scores is not None else 0
    sel_cap = int(sel.shape[-1]) if sel is not None else 0
    return check(lib().kv_sparse_layer_decode(_ref(cache.layout), _ref(cache), _ref(seqs), _p(k_new), _p(v_new),
                                              _p(q), int(n_crit), int(k_fixed), float(ratio), int(n_sink),
                                              int(window), _p(scores), stride, _p(sel), sel_cap, _p(sel_count),
                                              _p(out), ws.ptr, ws.nbytes, _s(stream)), "kv_sparse_layer_decode")


def kv_mixed_layer_decode_ws(cache, seqs):
    return lib().kv_mixed_layer_decode_ws(_ref(cache.layout), _ref(seqs))


def kv_mixed_layer_decode(cache, seqs, k_new, v_new, q, n_crit, k_fixed, ratio, n_sink, window, dense, out, ws,
                          sel=None, sel_count=None, stream=None):
    sel_cap = int(sel.shape[-1]) if sel is not None else 0
    return check(lib().kv_mixed_layer_decode(_ref(cache.layout), _ref(cache), _ref(seqs), _p(k_new), _p(v_new),
                                             _p(q), int(n_crit), int(k_fixed), float(ratio), int(n_sink), int(window),
                                             _p(dense), _p(sel), sel_cap, _p(sel_count), _p(out), ws.ptr, ws.nbytes,
                                             _s(stream)), "kv_mixed_layer_decode")


def kvq_classify_heads(P, n_q_heads, n_kv_heads, n_q, tau):
    """Per kv head: 1 if its q heads' mean dense-preference score over n_q exceeds tau."""
    Pa = (ctypes.c_float * n_q_heads)(*[float(x) for x in P])
    out = (ctypes.c_int32 * n_kv_heads)()
    r = lib().kvq_classify_heads(Pa, int(n_q_heads), int(n_kv_heads), int(n_q), float(tau), out)
    if r < 0:
        raise KvqError(r, "kvq_classify_heads", _abi.last_error())
    return [int(out[i]) for i in range(n_kv_heads)]


def kv_topk_select_ws():
    return lib().kv_topk_select_ws()


def kv_topk_select(seqs, n_heads, scores, k_fixed, ratio, n_sink, window, sel, sel_count, ws, score_stride=None,
                   stream=None):
    if score_stride is None:
        score_stride = scores.shape[-1]
    return check(lib().kv_topk_select(_ref(seqs), int(n_heads), _p(scores), int(score_stride), int(k_fixed),
                                      float(ratio), int(n_sink), int(window), _p(sel), int(sel.shape[-1]),
                                      _p(sel_count), ws.ptr, ws.nbytes, _s(stream)), "kv_topk_select")


def kv_block_select_ws(seqs, n_heads, block_tokens):
    return lib().kv_block_select_ws(_ref(seqs), int(n_heads), int(block_tokens))


def kv_block_select(seqs, n_heads, scores, n_keep_fixed, ratio, n_sink, window, block_tokens, sel, sel_count, ws,
                    score_stride=None, stream=None):
    if score_stride is None:
        score_stride = scores.shape[-1]
    return check(lib().kv_block_select(_ref(seqs), int(n_heads), _p(scores), int(score_stride), int(n_keep_fixed),
                                       float(ratio), int(n_sink), int(window), int(block_tokens), _p(sel),
                                       int(sel.shape[-1]), _p(sel_count), ws.ptr, ws.nbytes, _s(stream)),
                 "kv_block_select")


def kv_sparse_attn_ws(cache, seqs, sel_cap):
    return lib().kv_sparse_attn_ws(_ref(cache.layout), _ref(seqs), int(sel_cap))


def kv_sparse_attn(cache, seqs, q, sel, sel_count, sel_per_kv_head, out, probs, ws, stream=None):
    return check(lib().kv_sparse_attn(_ref(cache.layout), _ref(cache), _ref(seqs), _p(q), _p(sel),
                                      int(sel.shape[-1]), _p(sel_count), int(sel_per_kv_head), _p(out), _p(probs),
                                      ws.ptr, ws.nbytes, _s(stream)), "kv_sparse_attn")


def kv_h2o_accumulate_ws():
    return lib().kv_h2o_accumulate_ws()


def kv_h2o_accumulate(cache, seqs, probs, retained, retained_count, cum, budget, n_sink, window, new_pos, n_evicted,
                      ws, stream=None):
    return check(lib().kv_h2o_accumulate(_ref(cache.layout), _ref(seqs), _p(probs), _p(retained),
                                         _p(retained_count), _p(cum), int(retained.shape[-1]), int(budget),
                                         int(n_sink), int(window), _p(new_pos), _p(n_evicted), ws.ptr, ws.nbytes,
                                         _s(stream)), "kv_h2o_accumulate")


def kv_dense_pref_score_ws(cache, seqs, n_q):
    return lib().kv_dense_pref_score_ws(_ref(cache.layout), _ref(seqs), int(n_q))


def kv_dense_pref_score(cache, seqs, q_recent, n_q, topk, P, ws, stream=None):
    return check(lib().kv_dense_pref_score(_ref(cache.layout), _ref(cache), _ref(seqs), _p(q_recent), int(n_q),
                                           int(topk), _p(P), ws.ptr, ws.nbytes, _s(stream)), "kv_dense_pref_score")


def kv_offload_gather_ws():
    return lib().kv_offload_gather_ws()


def kv_offload_gather(src_k, src_v, src_stride_h, src_rows, n_heads, sel, sel_count, dst_k, dst_v, ws, stream=None):
    return check(lib().kv_offload_gather(_p(src_k), _p(src_v), int(src_stride_h), int(src_rows), int(n_heads),
                                         _p(sel), int(sel.shape[-1]), _p(sel_count), _p(dst_k), _p(dst_v), ws.ptr,
                                         ws.nbytes, _s(stream)), "kv_offload_gather")


def _head_rows(x, shape, dtype, gpu, fn, name):
    """(address, token stride) of x [n][heads][d], whose heads lie side by side (a slice of a wider row is fine)."""
    if x is None:
        return None, 0
    if not isinstance(x, torch.Tensor) or x.dtype is not dtype or x.shape != shape or x.get_device() != gpu:
        have = f"{x.dtype} {tuple(x.shape)} on {x.device}" if isinstance(x, torch.Tensor) else type(x).__name__
        raise KvqError(_abi.KVQ_ERR_INVALID_ARG, fn, f"{name}: {have} instead of {dtype} {shape} on GPU {gpu}")
    st = x.stride()
    if st[2] != 1 or (st[1] != HEAD_DIM and shape[1] > 1):
        raise KvqError(_abi.KVQ_ERR_INVALID_ARG, fn, f"{name}: a token's heads must lie side by side")
    return x.data_ptr(), st[0] if shape[0] > 1 else shape[1] * HEAD_DIM


def kv_qk_norm_rope(layout, rope, positions, q, k, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6, v=None,
                    v_out=None, stream=None):
    """Head norms (with a weight) and rotary positions of q [n][H_q][d] and k [n][H_kv][d], fp16 or bf16,
    into fp16 q_out and k_out; v is cast into v_out.  Each input may be None with its output.  `layout`: a
    Layout or a cache; `rope`: a RopeTable."""
    fn, gpu = "kv_qk_norm_rope", _gpu()
    L = _layout_of(layout)
    given = q if q is not None else k if k is not None else _need(v, fn, "q, k or v")
    n, dt = given.shape[0], given.dtype
    if dt is not torch.float16 and dt is not torch.bfloat16:
        raise KvqError(_abi.KVQ_ERR_UNSUPPORTED, fn, f"{dt}: float16 or bfloat16")
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (v is None) != (v_out is None):
        raise KvqError(_abi.KVQ_ERR_INVALID_ARG, fn, "an input and its output come together")
    if rope.gpu != gpu:
        raise KvqError(_abi.KVQ_ERR_INVALID_ARG, fn, f"the RopeTable is on GPU {rope.gpu}, not on {gpu}")
    sq, sk = (n, L.n_q_heads, HEAD_DIM), (n, L.n_kv_heads, HEAD_DIM)
    qa = ka = va = wq = wk = qo = ko = vo = None
    qs = ks = vs = 0
    if q is not None:
        qa, qs = _head_rows(q, sq, dt, gpu, fn, "q")
        qo = _dev(q_out, torch.float16, sq, gpu, fn, "q_out")
    if k is not None:
        ka, ks = _head_rows(k, sk, dt, gpu, fn, "k")
        ko = _dev(k_out, torch.float16, sk, gpu, fn, "k_out")
    if v is not None:
        va, vs = _head_rows(v, sk, dt, gpu, fn, "v")
        vo = _dev(v_out, torch.float16, sk, gpu, fn, "v_out")
    if q_weight is not None:
        wq = _dev(q_weight, torch.float32, _ROW, gpu, fn, "q_weight")
    if k_weight is not None:
        wk = _dev(k_weight, torch.float32, _ROW, gpu, fn, "k_weight")
    return check(lib().kv_qk_norm_rope(
        ctypes.byref(L), ctypes.byref(rope.c), rope.at, rope.mscale, _abi.F16 if dt is torch.float16 else _abi.BF16, n,
        _dev(positions, torch.int32, (n,), gpu, fn, "positions"), qa, qs, ka, ks, va, vs, wq, wk, float(eps), qo, ko, vo,
        _raw(stream, gpu)), fn)


def kv_decode_attn_ws(cache, seqs):
    return lib().kv_decode_attn_ws(_ref(cache.layout), _ref(seqs))


def kv_decode_attn(cache, seqs, q, out, ws, mod=None, lse=None, stream=None):
    """Attention of one new token per sequence over an fp16 layer; q [B][H_q][d] fp16, out fp32, `mod` an
    AttnMod, lse [B][H_q] fp32 (optional)."""
    fn, L, gpu = "kv_decode_attn", cache.layout, _gpu()
    B, H = seqs.c.batch, L.n_q_heads
    shape = (B, H, HEAD_DIM)
    return check(lib().kv_decode_attn(
        ctypes.byref(L), ctypes.byref(cache.c), ctypes.byref(seqs.c), _dev(_need(q, fn, "q"), torch.float16, shape, gpu, fn, "q"),
        _mod(mod, fn, L, B, B, gpu), _dev(_need(out, fn, "out"), torch.float32, shape, gpu, fn, "out"),
        _dev(lse, torch.float32, (B, H), gpu, fn, "lse"), ws.ptr, ws.nbytes, _raw(stream, gpu)), fn)


def kv_chunk_attn_ws(cache, seqs, n_rows, max_new):
    return lib().kv_chunk_attn_ws(_ref(cache.layout), _ref(seqs), int(n_rows), int(max_new))


def kv_chunk_attn(cache, seqs, q, q_starts, max_new, out, ws, mod=None, lse=None, stream=None):
    """Attention of the last q_starts[b+1] - q_starts[b] (at most max_new) tokens of every sequence over an
    fp16 layer; q and out [n_rows][H_q][d] fp16, lse [n_rows][H_q] fp32 (optional)."""
    fn, L, gpu = "kv_chunk_attn", cache.layout, _gpu()
    B, H, n = seqs.c.batch, L.n_q_heads, _need(q, fn, "q").shape[0]
    shape = (n, H, HEAD_DIM)
    return check(lib().kv_chunk_attn(
        ctypes.byref(L), ctypes.byref(cache.c), ctypes.byref(seqs.c), _dev(q, torch.float16, shape, gpu, fn, "q"),
        _dev(_need(q_starts, fn, "q_starts"), torch.int32, (B + 1,), gpu, fn, "q_starts"), n, int(max_new),
        _mod(mod, fn, L, B, n, gpu), _dev(_need(out, fn, "out"), torch.float16, shape, gpu, fn, "out"),
        _dev(lse, torch.float32, (n, H), gpu, fn, "lse"), ws.ptr, ws.nbytes, _raw(stream, gpu)), fn)


def _pairs(pairs, gpu, fn):
    """(address, count) of a device int32 [n][2] list."""
    n = _need(pairs, fn, "pairs").shape[0]
    return _dev(pairs, torch.int32, (n, 2), gpu, fn, "pairs"), n


def kv_pages_copy_ws():
    return lib().kv_pages_copy_ws()


def kv_pages_copy(cache, pairs, ws, stream=None):
    """Copies page pairs[i][0] to page pairs[i][1] (device int32 [n][2]) in every array of the layer."""
    gpu = _gpu()
    at, n = _pairs(pairs, gpu, "kv_pages_copy")
    return check(lib().kv_pages_copy(ctypes.byref(cache.layout), ctypes.byref(cache.c), at, n, ws.ptr, ws.nbytes,
                                     _raw(stream, gpu)), "kv_pages_copy")


def kv_slots_copy_ws():
    return lib().kv_slots_copy_ws()


def kv_slots_copy(cache, seqs, pairs, ws, stream=None):
    """Copies the per-sequence state (k_tail, or kT and k_absmax) of slot pairs[i][0] to slot pairs[i][1]."""
    gpu = _gpu()
    at, n = _pairs(pairs, gpu, "kv_slots_copy")
    return check(lib().kv_slots_copy(ctypes.byref(cache.layout), ctypes.byref(cache.c), ctypes.byref(seqs.c), at, n, ws.ptr,
                                     ws.nbytes, _raw(stream, gpu)), "kv_slots_copy")


def kvq_table_remap_ws():
    return lib().kvq_table_remap_ws()


def kvq_table_remap(block_table, new_id, ws, stream=None):
    """block_table[...] = new_id[block_table[...]], in place (device int32; negative entries stay)."""
    fn, gpu = "kvq_table_remap", _gpu()
    at = _dev(_need(block_table, fn, "block_table"), torch.int32, None, gpu, fn, "block_table")
    ids = _dev(_need(new_id, fn, "new_id"), torch.int32, None, gpu, fn, "new_id")
    return check(lib().kvq_table_remap(at, block_table.numel(), ids, new_id.numel(), ws.ptr, ws.nbytes, _raw(stream, gpu)), fn)


def kvq_seq_lens_add(seq_lens, delta, stream=None):
    return check(lib().kvq_seq_lens_add(_p(seq_lens), int(seq_lens.numel()), int(delta), _s(stream)),
                 "kvq_seq_lens_add")


def kv_page_copy(cache, src, dst, stream=None):
    return check(lib().kv_page_copy(_ref(cache.layout), _ref(cache), int(src), int(dst), _s(stream)),
                 "kv_page_copy")


def kvq_check(ws, stream=None):
    return check(lib().kvq_check(ws.ptr, _s(stream)), "kvq_check")


def kvq_selftest_bounded_wait(ws, stream=None):
    """Runs the library's bounded mbarrier wait on a barrier nothing completes (see kvq.h)."""
    return check(lib().kvq_selftest_bounded_wait(ws.ptr, ws.nbytes, _s(stream)), "kvq_selftest_bounded_wait")


def kvq_read_path_counters(ws, stream=None):
    """The workspace's diagnostic path counters (KVQ_PATH_*), read and cleared."""
    out = (ctypes.c_uint32 * _abi.N_PATH_COUNTERS)()
    check(lib().kvq_read_path_counters(ws.ptr, out, _s(stream)), "kvq_read_path_counters")
    return [int(out[i]) for i in range(_abi.N_PATH_COUNTERS)]
