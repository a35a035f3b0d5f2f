"""ctypes binding of libargus.so: argument marshalling only.

Every function here forwards to the C entry point of the same name declared in
include/argus.h; tensors are passed as raw device pointers (torch is used for
device memory and streams only).  A failing status raises ArgusError with the
library's one-line reason.  There is no fallback: if the library has not been
built, lib() raises.
"""

import ctypes
import os
import struct

import torch

FP16, BF16, FP8_E4M3, INT8, INT4_G32, INT2_G32, INT1_G32 = 0, 1, 2, 3, 4, 5, 6
CODEC_NAMES = {FP16: "fp16", BF16: "bf16", FP8_E4M3: "fp8_e4m3", INT8: "int8", INT4_G32: "int4_g32",
               INT2_G32: "int2_g32", INT1_G32: "int1_g32"}
DTYPE_CODEC = {torch.float16: FP16, torch.bfloat16: BF16}

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libargus.so")
_lib = None


class ArgusError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("argus status %d: %s" % (status, msg))
        self.status = status


class Geom(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32)]


PLACE_DEVICE, PLACE_HOST = 0, 1


class PoolDesc(ctypes.Structure):
    _fields_ = [("codec", ctypes.c_int32), ("placement", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("meta", ctypes.c_void_p),
                ("n_slots", ctypes.c_int64)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("g", Geom), ("batch", ctypes.c_int32), ("q_dtype", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("pools", ctypes.POINTER(PoolDesc)),
                ("n_pools", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_codec", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("sel_pages", ctypes.c_void_p),
                ("sel_count", ctypes.c_void_p), ("sel_width", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("out_dtype", ctypes.c_int32), ("out_f32", ctypes.c_void_p),
                ("lse2_out", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("num_splits", ctypes.c_int32), ("pdl", ctypes.c_int32),
                ("window_tokens", ctypes.c_int32), ("sink_tokens", ctypes.c_int32)]


class ExtendArgs(ctypes.Structure):
    _fields_ = [("g", Geom), ("batch", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("q_dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("q_start", ctypes.c_void_p),
                ("pools", ctypes.POINTER(PoolDesc)), ("n_pools", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("page_codec", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("lse2_out", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("softmax_scale", ctypes.c_float)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("g", Geom), ("batch", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("adjacent", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p), ("pair_axis", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("pool", ctypes.POINTER(PoolDesc)), ("page_codec", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int32),
                ("status", ctypes.c_void_p)]


EXPORTS = ["argus_quantize_pages", "argus_decode_workspace_bytes", "argus_paged_decode_attn",
           "argus_paged_decode_attn_noalloc",
           "argus_select_workspace_bytes", "argus_select_pages", "argus_fold_lse",
           "argus_window_prefill_workspace_bytes", "argus_window_prefill_attn",
           "argus_paged_window_prefill_workspace_bytes", "argus_paged_window_prefill_attn",
           "argus_staging_moves_less", "argus_extend_workspace_bytes", "argus_paged_extend_attn",
           "argus_rope_append", "argus_fork_workspace_bytes", "argus_fork_pages",
           "argus_compact_workspace_bytes", "argus_compact_pages", "argus_paged_window_extend_attn",
           "argus_paged_tree_attn", "argus_accept_tokens", "argus_norm_rope_append", "argus_attn_weights",
           "argus_evict_tokens", "argus_test_decode_stall",
           "argus_status_string", "argus_last_error"]


def lib_path():
    return _LIB_PATH


def lib():
    """Load libargus.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError("libargus.so is not built; run __graft_entry__.build() "
                           "(python -m mixed_precision_paged_argus_gb300.build)")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.argus_status_string.restype = ctypes.c_char_p
    L.argus_status_string.argtypes = [ctypes.c_int]
    L.argus_last_error.restype = ctypes.c_char_p
    L.argus_last_error.argtypes = []
    L.argus_quantize_pages.restype = ctypes.c_int
    L.argus_quantize_pages.argtypes = [ctypes.POINTER(Geom), i32, vp, i64, vp, ctypes.POINTER(PoolDesc),
                                       vp, i32, vp, vp, vp, vp]
    L.argus_decode_workspace_bytes.restype = ctypes.c_int
    L.argus_decode_workspace_bytes.argtypes = [ctypes.POINTER(DecodeArgs), ctypes.POINTER(sz)]
    L.argus_paged_decode_attn.restype = ctypes.c_int
    L.argus_paged_decode_attn.argtypes = [ctypes.POINTER(DecodeArgs), vp, sz, vp]
    L.argus_test_decode_stall.restype = ctypes.c_int
    L.argus_test_decode_stall.argtypes = [ctypes.POINTER(DecodeArgs), vp, sz, ctypes.c_uint32, i32, vp]
    L.argus_paged_decode_attn_noalloc.restype = ctypes.c_int
    L.argus_paged_decode_attn_noalloc.argtypes = [ctypes.POINTER(DecodeArgs), vp]
    L.argus_select_workspace_bytes.restype = ctypes.c_int
    L.argus_select_workspace_bytes.argtypes = [ctypes.POINTER(Geom), i32, i32, ctypes.POINTER(sz)]
    L.argus_select_pages.restype = ctypes.c_int
    L.argus_select_pages.argtypes = [ctypes.POINTER(Geom), i32, vp, i32, vp, vp, i32, i32, i32,
                                     vp, vp, i32, vp, vp, sz, vp]
    L.argus_fold_lse.restype = ctypes.c_int
    L.argus_fold_lse.argtypes = [i64, i32, vp, vp, vp, vp, vp]
    L.argus_window_prefill_attn.restype = ctypes.c_int
    L.argus_window_prefill_attn.argtypes = [ctypes.POINTER(Geom), i32, vp, vp, vp, i64, i64, i64, i64,
                                            ctypes.c_float, vp, vp, i32, i32, vp, sz, vp]
    L.argus_window_prefill_workspace_bytes.restype = ctypes.c_int
    L.argus_window_prefill_workspace_bytes.argtypes = [ctypes.POINTER(Geom), i32, i64, i32, ctypes.POINTER(sz)]
    L.argus_paged_window_prefill_workspace_bytes.restype = ctypes.c_int
    L.argus_paged_window_prefill_workspace_bytes.argtypes = [ctypes.POINTER(Geom), i32, i64, i32, ctypes.POINTER(sz)]
    L.argus_paged_window_prefill_attn.restype = ctypes.c_int
    L.argus_paged_window_prefill_attn.argtypes = [ctypes.POINTER(Geom), i32, vp, ctypes.POINTER(PoolDesc), i32, vp, vp,
                                                  i32, i64, i64, i64, ctypes.c_float, vp, vp, i32, i32, vp, sz, vp, vp]
    L.argus_staging_moves_less.restype = ctypes.c_int
    L.argus_staging_moves_less.argtypes = [ctypes.POINTER(ctypes.c_int64), i64, i64, ctypes.POINTER(i32)]
    L.argus_extend_workspace_bytes.restype = ctypes.c_int
    L.argus_extend_workspace_bytes.argtypes = [ctypes.POINTER(ExtendArgs), ctypes.POINTER(sz)]
    L.argus_paged_extend_attn.restype = ctypes.c_int
    L.argus_paged_extend_attn.argtypes = [ctypes.POINTER(ExtendArgs), vp, sz, vp]
    L.argus_rope_append.restype = ctypes.c_int
    L.argus_rope_append.argtypes = [ctypes.POINTER(RopeArgs), vp]
    L.argus_fork_workspace_bytes.restype = ctypes.c_int
    L.argus_fork_workspace_bytes.argtypes = [i32, ctypes.POINTER(PoolDesc), i32, ctypes.POINTER(sz)]
    L.argus_fork_pages.restype = ctypes.c_int
    L.argus_fork_pages.argtypes = [ctypes.POINTER(Geom), i32, vp, vp, i32, ctypes.POINTER(PoolDesc), i32,
                                   ctypes.POINTER(vp), ctypes.POINTER(vp), vp, vp, vp, vp, vp, vp, i32, vp, sz, vp, vp]
    L.argus_compact_workspace_bytes.restype = ctypes.c_int
    L.argus_compact_workspace_bytes.argtypes = [ctypes.POINTER(PoolDesc), ctypes.POINTER(sz)]
    L.argus_compact_pages.restype = ctypes.c_int
    L.argus_compact_pages.argtypes = [ctypes.POINTER(Geom), i32, ctypes.POINTER(PoolDesc), vp, vp, vp, vp, vp, vp, i32,
                                      vp, vp, sz, vp, vp]
    L.argus_paged_window_extend_attn.restype = ctypes.c_int
    L.argus_paged_window_extend_attn.argtypes = [ctypes.POINTER(ExtendArgs), i32, i32, vp, sz, vp]
    L.argus_paged_tree_attn.restype = ctypes.c_int
    L.argus_paged_tree_attn.argtypes = [ctypes.POINTER(ExtendArgs), vp, i32, vp, sz, vp]
    L.argus_accept_tokens.restype = ctypes.c_int
    L.argus_accept_tokens.argtypes = [ctypes.POINTER(Geom), i32, ctypes.POINTER(PoolDesc), vp, vp, i32, vp, vp, vp, i32, vp, vp, vp, vp]
    L.argus_norm_rope_append.restype = ctypes.c_int
    L.argus_norm_rope_append.argtypes = [ctypes.POINTER(RopeArgs), vp, vp, ctypes.c_float, vp]
    L.argus_attn_weights.restype = ctypes.c_int
    L.argus_attn_weights.argtypes = [ctypes.POINTER(ExtendArgs), vp, i64, ctypes.c_float, vp]
    L.argus_evict_tokens.restype = ctypes.c_int
    L.argus_evict_tokens.argtypes = [ctypes.POINTER(Geom), i32, ctypes.POINTER(PoolDesc), i32, vp, vp, vp, i32, vp, i64, i32, i32, i32,
                                     ctypes.POINTER(PoolDesc), vp, i32, vp, vp, vp, i64, vp, vp]
    _lib = L
    return L


def _check(status):
    if status != 0:
        L = lib()
        raise ArgusError(status, L.argus_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def geom(n_q_heads, n_kv_heads, head_dim, page_tokens):
    return Geom(n_q_heads, n_kv_heads, head_dim, page_tokens)


class Pool:
    """A physical page pool of one codec: codes (and meta) tensors, on the
    device, or in page-locked host memory (placement PLACE_HOST: read in place
    by decode over the host link)."""

    def __init__(self, codec, codes, meta, n_slots, placement=None):
        self.codec, self.codes, self.meta, self.n_slots = codec, codes, meta, int(n_slots)
        if placement is None:
            placement = PLACE_HOST if (codes is not None and not codes.is_cuda) else PLACE_DEVICE
        self.placement = placement

    def desc(self):
        return PoolDesc(self.codec, self.placement, _ptr(self.codes), _ptr(self.meta), self.n_slots)

    def to_host(self):
        """A copy of this pool in page-locked host memory (PLACE_HOST)."""
        codes = self.codes.cpu().pin_memory()
        meta = None if self.meta is None else self.meta.cpu().pin_memory()
        return Pool(self.codec, codes, meta, self.n_slots, PLACE_HOST)

    @staticmethod
    def empty(codec, n_slots, n_kv_heads, page_tokens, head_dim, device="cuda", zero=False):
        """Allocate a pool in the layout of include/argus.h (device="host":
        page-locked host memory)."""
        if str(device) == "host":
            p = Pool.empty(codec, n_slots, n_kv_heads, page_tokens, head_dim, device="cpu", zero=zero)
            return Pool(codec, p.codes.pin_memory(), None if p.meta is None else p.meta.pin_memory(), n_slots,
                        PLACE_HOST)
        alloc = torch.zeros if zero else torch.empty
        shape = (n_slots, 2, n_kv_heads, page_tokens)
        if codec in (FP16, BF16):
            codes = alloc(shape + (head_dim,), dtype=torch.float16 if codec == FP16 else torch.bfloat16,
                          device=device)
            meta = None
        elif codec in (FP8_E4M3, INT8):
            codes = alloc(shape + (head_dim,), dtype=torch.uint8, device=device)
            meta = alloc((n_slots, 2, n_kv_heads), dtype=torch.float32, device=device)
        elif codec in (INT4_G32, INT2_G32, INT1_G32):
            per_byte = {INT4_G32: 2, INT2_G32: 4, INT1_G32: 8}[codec]
            codes = alloc(shape + (head_dim // per_byte,), dtype=torch.uint8, device=device)
            meta = alloc(shape + (head_dim // 32, 2), dtype=torch.float16, device=device)
        else:
            raise ValueError(codec)
        return Pool(codec, codes, meta, n_slots)


def quantize_pages(g, src_dtype, src_codes, n_src_slots, src_slots, dst, dst_slots, n_pages,
                   valid_tokens=None, ckey_out=None, status=None, stream=None):
    d = dst.desc()
    _check(lib().argus_quantize_pages(ctypes.byref(g), src_dtype, _ptr(src_codes), int(n_src_slots),
                                      _ptr(src_slots), ctypes.byref(d), _ptr(dst_slots), int(n_pages),
                                      _ptr(valid_tokens), _ptr(ckey_out), _ptr(status), _stream(stream)))


def decode_args(g, batch, q, pools, page_codec, block_table, seq_lens, max_pages, softmax_scale,
                out=None, out_f32=None, lse2_out=None, sel_pages=None, sel_count=None, sel_width=0,
                status=None, num_splits=0, pdl=False, window_tokens=0, sink_tokens=0):
    """Build an argus_decode_args struct (keeps the pool array alive on the struct)."""
    arr = (PoolDesc * max(1, len(pools)))(*[p.desc() for p in pools])
    a = DecodeArgs()
    a.g = g
    a.batch = int(batch)
    a.q_dtype = DTYPE_CODEC[q.dtype]
    a.q = _ptr(q)
    a.pools = ctypes.cast(arr, ctypes.POINTER(PoolDesc))
    a.n_pools = len(pools)
    a.max_pages = int(max_pages)
    a.page_codec = _ptr(page_codec)
    a.block_table = _ptr(block_table)
    a.seq_lens = _ptr(seq_lens)
    a.sel_pages = _ptr(sel_pages)
    a.sel_count = _ptr(sel_count)
    a.sel_width = int(sel_width)
    a.softmax_scale = float(softmax_scale)
    a.out = _ptr(out)
    a.out_dtype = DTYPE_CODEC[out.dtype] if out is not None else FP16
    a.out_f32 = _ptr(out_f32)
    a.lse2_out = _ptr(lse2_out)
    a.status = _ptr(status)
    a.num_splits = int(num_splits)
    a.pdl = int(pdl)   # False / True / 2
    a.window_tokens = int(window_tokens)
    a.sink_tokens = int(sink_tokens)
    # the struct holds raw pointers: keep every tensor it points to alive with it
    a._keep = (arr, list(pools), q, page_codec, block_table, seq_lens, sel_pages, sel_count, out,
               out_f32, lse2_out, status)
    return a


def decode_workspace_bytes(args):
    n = ctypes.c_size_t(0)
    _check(lib().argus_decode_workspace_bytes(ctypes.byref(args), ctypes.byref(n)))
    return n.value


def paged_decode_attn(args, ws, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().argus_paged_decode_attn(ctypes.byref(args), _ptr(ws), int(ws_bytes), _stream(stream)))


STATUS_TIMEOUT_BIT = 0x80000000


def test_decode_stall(args, ws, wait_limit_us, stall_stage, stream=None):
    """Testing only: the decode with every device wait limited to wait_limit_us
    and stage stall_stage's arrival withheld, so that the waits run out."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().argus_test_decode_stall(ctypes.byref(args), _ptr(ws), nbytes, int(wait_limit_us),
                                         int(stall_stage), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 4 << 20


def paged_decode_attn_noalloc(args, stream=None):
    """Decode with the library's fixed device scratch instead of a workspace
    (for callers that cannot allocate; calls must not overlap on the GPU)."""
    _check(lib().argus_paged_decode_attn_noalloc(ctypes.byref(args), _stream(stream)))


def select_workspace_bytes(g, batch, max_pages):
    n = ctypes.c_size_t(0)
    _check(lib().argus_select_workspace_bytes(ctypes.byref(g), int(batch), int(max_pages), ctypes.byref(n)))
    return n.value


def select_pages(g, batch, q, ckeys, n_pages, max_pages, top_k, keep_newest, sel_pages, sel_count,
                 sel_width, drop_counter, ws, stream=None):
    _check(lib().argus_select_pages(ctypes.byref(g), int(batch), _ptr(q), DTYPE_CODEC[q.dtype], _ptr(ckeys),
                                    _ptr(n_pages), int(max_pages), int(top_k), int(bool(keep_newest)),
                                    _ptr(sel_pages), _ptr(sel_count), int(sel_width), _ptr(drop_counter),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def fold_lse(acc_o, acc_lse2, part_o, part_lse2, stream=None):
    n_rows = acc_lse2.numel()
    head_dim = acc_o.numel() // max(1, n_rows)
    _check(lib().argus_fold_lse(int(n_rows), int(head_dim), _ptr(acc_o), _ptr(acc_lse2), _ptr(part_o),
                                _ptr(part_lse2), _stream(stream)))


def window_prefill_workspace_bytes(g, n_q, win_len, num_splits=0):
    n = ctypes.c_size_t(0)
    _check(lib().argus_window_prefill_workspace_bytes(ctypes.byref(g), int(n_q), int(win_len), int(num_splits),
                                                      ctypes.byref(n)))
    return n.value


def staging_moves_less(row_read_bytes, cache_bytes):
    """Whether a prefill should stage the cache into device windows: the rows'
    in-place reads (host list of byte counts) together exceed cache_bytes."""
    vals = [int(x) for x in row_read_bytes] + [int(cache_bytes)]
    for x in vals:
        # ctypes wraps integers silently; a byte count outside int64 must not
        # turn into a small valid one
        if not (-2 ** 63 <= x < 2 ** 63):
            raise ValueError("staging_moves_less: byte count %d does not fit in int64" % x)
    rows = (ctypes.c_int64 * max(1, len(row_read_bytes)))(*vals[:-1])
    out = ctypes.c_int32(0)
    _check(lib().argus_staging_moves_less(rows, len(row_read_bytes), vals[-1], ctypes.byref(out)))
    return bool(out.value)


def window_prefill_attn(g, n_q, q, k, v, kv_head_stride, win_len, win_pos0, q_pos0, softmax_scale,
                        acc_o, acc_lse2, fold, num_splits=0, ws=None, stream=None):
    """num_splits / ws: key ranges per query tile and their partial-result
    workspace (window_prefill_workspace_bytes bytes); 0 with ws chooses the
    split count, 0 without ws is one CTA per tile."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().argus_window_prefill_attn(ctypes.byref(g), int(n_q), _ptr(q), _ptr(k), _ptr(v),
                                           int(kv_head_stride), int(win_len), int(win_pos0), int(q_pos0),
                                           float(softmax_scale), _ptr(acc_o), _ptr(acc_lse2), int(fold),
                                           int(num_splits), _ptr(ws), nbytes, _stream(stream)))


def paged_window_prefill_workspace_bytes(g, n_q, win_len, num_splits=0):
    n = ctypes.c_size_t(0)
    _check(lib().argus_paged_window_prefill_workspace_bytes(ctypes.byref(g), int(n_q), int(win_len), int(num_splits),
                                                            ctypes.byref(n)))
    return n.value


def paged_window_prefill_attn(g, n_q, q, pools, page_codec, block_table, max_pages, win_pos0, win_len, q_pos0,
                              softmax_scale, acc_o, acc_lse2, fold, ws, num_splits=0, status=None, stream=None):
    """Stage one window of the paged cache (block_table / page_codec rows of one
    sequence, pools of any codec) and attend the query chunk to it, folding
    into acc_o / acc_lse2; ws of paged_window_prefill_workspace_bytes bytes."""
    arr = (PoolDesc * max(1, len(pools)))(*[p.desc() for p in pools])
    _check(lib().argus_paged_window_prefill_attn(ctypes.byref(g), int(n_q), _ptr(q),
                                                 ctypes.cast(arr, ctypes.POINTER(PoolDesc)), len(pools),
                                                 _ptr(page_codec), _ptr(block_table), int(max_pages), int(win_pos0),
                                                 int(win_len), int(q_pos0), float(softmax_scale), _ptr(acc_o),
                                                 _ptr(acc_lse2), int(fold), int(num_splits), _ptr(ws),
                                                 ws.numel() * ws.element_size(), _ptr(status), _stream(stream)))


def _token_stride(name, t, heads, head_dim, device):
    """Elements between the tokens of t [tokens][heads][head_dim], whose tokens
    are dense and may lie apart (a slice of a fused projection's rows)."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim:
        raise ValueError("%s must be [tokens][%d][%d], not %s" % (name, heads, head_dim, list(shape)))
    if (stride[2] != 1 or (heads > 1 and stride[1] != head_dim)) and t.numel():
        raise ValueError("%s: the heads of a token must be dense" % name)
    if t.get_device() != device:
        raise ValueError("%s lies on another device" % name)
    if shape[0] <= 1:
        return heads * head_dim
    if stride[0] < heads * head_dim:     # 0 among them (a broadcast token), which the library reads as "dense"
        raise ValueError("%s: the tokens overlap in memory" % name)
    return stride[0]


def _at(name, t, dtype, numel, device):
    """Address of a dense tensor of at least numel elements on the device (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or not t.is_contiguous() or t.numel() < numel:
        raise ValueError("%s must be a dense %s tensor of %d elements or more" % (name, dtype, numel))
    if t.get_device() != device:
        raise ValueError("%s lies on another device" % name)
    return t.data_ptr()


def _status_at(t, device):
    if t is None:
        return None
    if t.element_size() != 4 or t.is_floating_point() or t.numel() < 1:
        raise ValueError("status must be a 32-bit integer tensor")
    if t.get_device() != device:
        raise ValueError("status lies on another device")
    return t.data_ptr()


def _stream_of(device, stream):
    """The stream to launch on: the given one, or the device's current one.  The
    library launches on the current device, so the tensors have to lie there."""
    if device >= 0:
        if device != torch._C._cuda_getDevice():
            raise ValueError("the tensors lie on cuda:%d, which is not the current device" % device)
    elif torch.cuda.is_available():
        raise ValueError("the tensors must lie on the GPU")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device) if device >= 0 else None
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ws_at(ws, device):
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError("ws must be a dense tensor on the tensors' device")
    return ws.data_ptr()


# the structs' layouts, field by field: packing takes a third of the time of building one by its fields
_POOL_DESC = struct.Struct("@iiPPq")
_EXTEND_ARGS = struct.Struct("@4i4iPqPPiiPPPPPPf0P")
_ROPE_ARGS = struct.Struct("@4i6i4P4q8PiP")
assert [x.size for x in (_POOL_DESC, _EXTEND_ARGS, _ROPE_ARGS)] == [ctypes.sizeof(x) for x in (PoolDesc, ExtendArgs, RopeArgs)]


_I32, _U8, _F32 = torch.int32, torch.uint8, torch.float32

# per codec: bits of a code, its float type if it has one, the meta's type
_LAYOUT = {FP16: (16, torch.float16, None), BF16: (16, torch.bfloat16, None), FP8_E4M3: (8, torch.float8_e4m3fn, _F32),
           INT8: (8, None, _F32), INT4_G32: (4, None, torch.float16), INT2_G32: (2, None, torch.float16), INT1_G32: (1, None, torch.float16)}


def _check_pool(p, units, values, device):
    """A device pool holds n_slots pages, dense, in its codec's types (or integers: their bits); a page has
    `units` units (a KV head's K or V) of `values` values together.  On the device a slot is compared with n_slots alone."""
    codec, codes, meta, n = p.codec, p.codes, p.meta, p.n_slots
    if codec not in _LAYOUT:
        return                               # the library refuses the codec
    bits, code_type, meta_type = _LAYOUT[codec]
    if codes is not None:
        if codes.get_device() != device:
            raise ValueError("a pool lies on another device")
        if codes.nbytes * 8 < n * values * bits or not codes.is_contiguous():
            raise ValueError("the pool of codec %d: codes must be a dense tensor of n_slots pages of this geometry" % codec)
        kind = codes.dtype
        if kind is not _U8 and kind is not code_type and kind.is_floating_point:
            raise ValueError("the pool of codec %d: codes of type %s" % (codec, kind))
    if meta is not None and meta_type is not None:
        if meta.get_device() != device:
            raise ValueError("a pool lies on another device")
        # a float per unit, or two halves per 32 values
        if meta.nbytes < n * (4 * units if meta_type is _F32 else values // 8) or not meta.is_contiguous():
            raise ValueError("the pool of codec %d: meta must be a dense tensor for n_slots pages of this geometry" % codec)
        kind = meta.dtype
        if kind is not meta_type and kind.is_floating_point:
            raise ValueError("the pool of codec %d: meta of type %s" % (codec, kind))


def _pool_array(pools, device=None, g=None):
    """The pools' descriptions; with a geometry, device pools are checked against it
    and the device (host pools are the library's to refuse)."""
    raw = []
    if g is not None:
        units = 2 * g.n_kv_heads
        values = units * g.page_tokens * g.head_dim
    for p in pools:
        codes, meta = p.codes, p.meta
        if g is not None and p.placement == PLACE_DEVICE:
            _check_pool(p, units, values, device)
        raw.append(_POOL_DESC.pack(p.codec, p.placement, 0 if codes is None else codes.data_ptr(),
                                   0 if meta is None else meta.data_ptr(), p.n_slots))
    if not raw:
        return (PoolDesc * 1)()
    return (PoolDesc * len(raw)).from_buffer_copy(b"".join(raw))


def extend_args(g, q, q_start, pools, page_codec, block_table, seq_lens, max_pages, softmax_scale, out,
                causal=True, lse2_out=None, status=None):
    """Build an argus_extend_args struct: q [total_q][Hq][D] (its tokens may lie
    apart), q_start [B + 1], seq_lens [B], out like q and dense (None for attn_weights, which
    reads lse2_out)."""
    batch, total, hq, dev = q_start.numel() - 1, q.shape[0], g.n_q_heads, q.get_device()
    arr = _pool_array(pools, dev, g)
    a = ExtendArgs.from_buffer_copy(_EXTEND_ARGS.pack(
        hq, g.n_kv_heads, g.head_dim, g.page_tokens, batch, total, DTYPE_CODEC[q.dtype], 1 if causal else 0, q.data_ptr(),
        _token_stride("q", q, hq, g.head_dim, dev), _at("q_start", q_start, _I32, 1, dev) or 0, ctypes.addressof(arr), len(pools),
        max_pages, _at("page_codec", page_codec, _U8, batch * max_pages, dev) or 0,
        _at("block_table", block_table, _I32, batch * max_pages, dev) or 0, _at("seq_lens", seq_lens, _I32, batch, dev) or 0,
        _at("out", out, q.dtype, q.numel(), dev) or 0, _at("lse2_out", lse2_out, _F32, total * hq, dev) or 0,
        _status_at(status, dev) or 0, softmax_scale))
    # the struct holds raw pointers: keep every tensor it points to alive with it
    a._keep = (arr, [(p.codes, p.meta) for p in pools], q, q_start, page_codec, block_table, seq_lens, out, lse2_out, status)
    a._device = dev
    return a


def extend_workspace_bytes(args):
    n = ctypes.c_size_t(0)
    _check(lib().argus_extend_workspace_bytes(ctypes.byref(args), ctypes.byref(n)))
    return n.value


def paged_extend_attn(args, ws, stream=None):
    """Attention of several query tokens per sequence over the paged cache;
    ws of extend_workspace_bytes bytes."""
    _check(lib().argus_paged_extend_attn(ctypes.byref(args), _ws_at(ws, args._device), ws.nbytes, _stream_of(args._device, stream)))


def _int32(name, x):
    """x as the library's 32-bit integer: ctypes would drop the bits above."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError("%s = %d does not fit in 32 bits" % (name, x))
    return x


def paged_window_extend_attn(args, ws, window_tokens, sink_tokens=0, stream=None):
    """paged_extend_attn where a token sees the newest window_tokens positions up
    to its own and the first sink_tokens; ws of extend_workspace_bytes bytes."""
    _check(lib().argus_paged_window_extend_attn(ctypes.byref(args), _int32("window_tokens", window_tokens), _int32("sink_tokens", sink_tokens),
                                                _ws_at(ws, args._device), ws.nbytes, _stream_of(args._device, stream)))


def paged_tree_attn(args, ws, tree_mask, stream=None):
    """paged_extend_attn for a tree of drafted tokens per sequence: tree_mask int32
    [tokens][words], bit x of a row: the sequence's drafted token x is seen (a row of
    no bits sees the cache in front of the tree); ws of extend_workspace_bytes bytes."""
    if tree_mask.dim() != 2 or tree_mask.shape[0] != args.total_q:
        raise ValueError("tree_mask must be [%d][words], not %s" % (args.total_q, list(tree_mask.shape)))
    _check(lib().argus_paged_tree_attn(ctypes.byref(args), _at("tree_mask", tree_mask, _I32, 0, args._device), tree_mask.shape[1],
                                       _ws_at(ws, args._device), ws.nbytes, _stream_of(args._device, stream)))


def accept_tokens(g, pool, page_codec, block_table, max_pages, q_start, seq_lens, path, n_path, seq_lens_out, status=None, stream=None):
    """Move the K and V rows of each sequence's accepted path (path int32 [B][width], the
    first n_path[b] entries: drafted tokens in ascending order) to where the sequence goes
    on; the new lengths go to seq_lens_out."""
    batch, dev = seq_lens.numel(), seq_lens.get_device()
    if path.dim() != 2 or path.shape[0] != batch:
        raise ValueError("path must be [%d][width], not %s" % (batch, list(path.shape)))
    entries = batch * _int32("max_pages", max_pages)
    _check(lib().argus_accept_tokens(
        ctypes.byref(g), batch, _pool_array((pool,), dev, g), _at("page_codec", page_codec, _U8, entries, dev),
        _at("block_table", block_table, _I32, entries, dev), max_pages, _at("q_start", q_start, _I32, batch + 1, dev),
        _at("seq_lens", seq_lens, _I32, 0, dev), _at("path", path, _I32, 0, dev), path.shape[1], _at("n_path", n_path, _I32, batch, dev),
        _at("seq_lens_out", seq_lens_out, _I32, batch, dev), _status_at(status, dev), _stream_of(dev, stream)))


def attn_weights(args, weights, decay=1.0, stream=None):
    """weights [B][Hkv][positions] (float32) become decay * weights plus the attention
    weights of the query tokens of args (extend_args; out may be None), whose log-sums
    args.lse2_out holds."""
    batch, hkv = args.batch, args.g.n_kv_heads
    if weights.dim() != 3 or weights.shape[0] != batch or weights.shape[1] != hkv:
        raise ValueError("weights must be [%d][%d][positions], not %s" % (batch, hkv, list(weights.shape)))
    _check(lib().argus_attn_weights(ctypes.byref(args), _at("weights", weights, _F32, 0, args._device), weights.shape[2], decay,
                                    _stream_of(args._device, stream)))


def evict_tokens(g, pools, page_codec, block_table, seq_lens, max_pages, weights, budget, sink_tokens, recent_tokens, dst, dst_table,
                 dst_pages, seq_lens_out, kept, weights_out, status=None, stream=None):
    """Bring every sequence to at most budget positions: each KV head keeps the first
    sink_tokens, the last recent_tokens and the heaviest between, gathered into the pages of
    dst that dst_table [B][dst_pages] names.  kept [B][Hkv][budget] takes the old positions,
    weights_out [B][Hkv][positions] their weights."""
    batch, dev, hkv = seq_lens.numel(), seq_lens.get_device(), g.n_kv_heads
    for name, t in (("weights", weights), ("weights_out", weights_out)):
        if t.dim() != 3 or t.shape[0] != batch or t.shape[1] != hkv:
            raise ValueError("%s must be [%d][%d][positions], not %s" % (name, batch, hkv, list(t.shape)))
    entries = batch * _int32("max_pages", max_pages)
    _check(lib().argus_evict_tokens(
        ctypes.byref(g), batch, _pool_array(pools, dev, g), len(pools), _at("page_codec", page_codec, _U8, entries, dev),
        _at("block_table", block_table, _I32, entries, dev), _at("seq_lens", seq_lens, _I32, 0, dev), max_pages,
        _at("weights", weights, _F32, 0, dev), weights.shape[2], _int32("budget", budget),
        _int32("sink_tokens", sink_tokens), _int32("recent_tokens", recent_tokens), _pool_array((dst,), dev, g),
        _at("dst_table", dst_table, _I32, batch * dst_pages, dev), _int32("dst_pages", dst_pages), _at("seq_lens_out", seq_lens_out, _I32, batch, dev),
        _at("kept", kept, _I32, batch * hkv * budget, dev), _at("weights_out", weights_out, _F32, 0, dev), weights_out.shape[2],
        _status_at(status, dev), _stream_of(dev, stream)))


def rope_append(g, q, k, v, q_out, q_start, seq_lens, positions, inv_freq, pool, page_codec, block_table, max_pages,
                pair_axis=None, adjacent=False, status=None, stream=None):
    """Turn q and k by their positions ([n_axes][tokens], one row per axis;
    inv_freq [rot_dim / 2] in float64, radians per position) into q_out and the
    cache, and store v: the tokens of sequence b become the last ones of its
    seq_lens[b] cached positions."""
    a, dev = _rope_args(g, q, k, v, q_out, q_start, seq_lens, positions, inv_freq, pool, page_codec, block_table, max_pages, pair_axis,
                        adjacent, status)
    _check(lib().argus_rope_append(ctypes.byref(a), _stream_of(dev, stream)))


def norm_rope_append(g, q, k, v, q_out, q_start, seq_lens, positions, inv_freq, pool, page_codec, block_table, max_pages, q_weight,
                     k_weight, eps, pair_axis=None, adjacent=False, status=None, stream=None):
    """rope_append whose queries and keys are normed first, each head by itself: divided by
    sqrt(mean(x^2) + eps), times q_weight or k_weight (float32 [head_dim], None: ones)."""
    a, dev = _rope_args(g, q, k, v, q_out, q_start, seq_lens, positions, inv_freq, pool, page_codec, block_table, max_pages, pair_axis,
                        adjacent, status)
    d = g.head_dim
    _check(lib().argus_norm_rope_append(ctypes.byref(a), _at("q_weight", q_weight, _F32, d, dev), _at("k_weight", k_weight, _F32, d, dev),
                                        eps, _stream_of(dev, stream)))


def _rope_args(g, q, k, v, q_out, q_start, seq_lens, positions, inv_freq, pool, page_codec, block_table, max_pages, pair_axis, adjacent,
               status):
    total, batch, dtype, dev = q.shape[0], q_start.numel() - 1, q.dtype, q.get_device()
    hq, hkv, d = g.n_q_heads, g.n_kv_heads, g.head_dim
    if k.shape[0] != total or v.shape[0] != total or q_out.shape[0] != total or positions.numel() % (total or 1):
        raise ValueError("rope_append: q, k, v, q_out and positions must have the same tokens")
    if k.dtype is not dtype or v.dtype is not dtype or q_out.dtype is not dtype:
        raise ValueError("rope_append: q, k, v and q_out must have the same type")
    half = inv_freq.numel()
    arr = _pool_array((pool,), dev, g)
    a = RopeArgs.from_buffer_copy(_ROPE_ARGS.pack(
        hq, hkv, d, g.page_tokens, batch, total, DTYPE_CODEC[dtype], 2 * half, 1 if adjacent else 0,
        positions.numel() // total if total else 1, q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(),
        _token_stride("q", q, hq, d, dev), _token_stride("k", k, hkv, d, dev), _token_stride("v", v, hkv, d, dev),
        _token_stride("q_out", q_out, hq, d, dev), _at("positions", positions, _I32, 0, dev) or 0,
        _at("inv_freq", inv_freq, torch.float64, 0, dev) or 0, _at("pair_axis", pair_axis, _U8, half, dev) or 0,
        _at("q_start", q_start, _I32, 1, dev) or 0, _at("seq_lens", seq_lens, _I32, batch, dev) or 0, ctypes.addressof(arr),
        _at("page_codec", page_codec, _U8, batch * max_pages, dev) or 0,
        _at("block_table", block_table, _I32, batch * max_pages, dev) or 0, max_pages, _status_at(status, dev) or 0))
    a._keep = arr
    return a, dev


def fork_workspace_bytes(batch, pools):
    n = ctypes.c_size_t(0)
    _check(lib().argus_fork_workspace_bytes(int(batch), _pool_array(pools), len(pools), ctypes.byref(n)))
    return n.value


def fork_pages(g, parents, n_new, new_codec, pools, ref_in, ref_out, page_codec, block_table, seq_lens, page_codec_out,
               block_table_out, seq_lens_out, max_pages, ws, status=None, stream=None):
    """One step of the page table: row b becomes row parents[b] (-1: freed),
    partial pages about to be written are copied where others hold them too, and
    pages of new_codec are added for n_new[b] tokens.  ref_in / ref_out: one
    int32 count per slot for each pool.  ws of fork_workspace_bytes bytes."""
    batch, n, dev = parents.numel(), len(pools), parents.get_device()
    if len(ref_in) != n or len(ref_out) != n:
        raise ValueError("fork_pages: one count tensor per pool")
    pointers = ctypes.c_void_p * (n or 1)
    rin = pointers(*[_at("ref_in", r, _I32, p.n_slots, dev) for p, r in zip(pools, ref_in)])
    rout = pointers(*[_at("ref_out", r, _I32, p.n_slots, dev) for p, r in zip(pools, ref_out)])
    entries = batch * max_pages
    _check(lib().argus_fork_pages(
        ctypes.byref(g), batch, _at("parents", parents, _I32, 0, dev), _at("n_new", n_new, _I32, batch, dev), new_codec,
        _pool_array(pools, dev, g), n, rin, rout, _at("page_codec", page_codec, _U8, entries, dev),
        _at("block_table", block_table, _I32, entries, dev), _at("seq_lens", seq_lens, _I32, batch, dev),
        _at("page_codec_out", page_codec_out, _U8, entries, dev), _at("block_table_out", block_table_out, _I32, entries, dev),
        _at("seq_lens_out", seq_lens_out, _I32, batch, dev), max_pages, _ws_at(ws, dev), ws.nbytes, _status_at(status, dev),
        _stream_of(dev, stream)))


def compact_workspace_bytes(pool):
    n = ctypes.c_size_t(0)
    _check(lib().argus_compact_workspace_bytes(_pool_array((pool,)), ctypes.byref(n)))
    return n.value


def compact_pages(g, pool, ref_in, ref_out, page_codec, block_table, seq_lens, block_table_out, max_pages, n_live, ws,
                  status=None, stream=None):
    """Move the live pages of a pool into its lowest slots; the new counts and
    table go to ref_out and block_table_out, the number of live slots to n_live.
    ws of compact_workspace_bytes bytes."""
    batch, dev = seq_lens.numel(), seq_lens.get_device()
    entries = batch * max_pages
    _check(lib().argus_compact_pages(
        ctypes.byref(g), batch, _pool_array((pool,), dev, g), _at("ref_in", ref_in, _I32, pool.n_slots, dev),
        _at("ref_out", ref_out, _I32, pool.n_slots, dev), _at("page_codec", page_codec, _U8, entries, dev),
        _at("block_table", block_table, _I32, entries, dev), _at("seq_lens", seq_lens, _I32, 0, dev),
        _at("block_table_out", block_table_out, _I32, entries, dev), max_pages, _at("n_live", n_live, _I32, 1, dev),
        _ws_at(ws, dev), ws.nbytes, _status_at(status, dev), _stream_of(dev, stream)))
