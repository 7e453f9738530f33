"""Thin Python binding of libkda.so (include/kda.h): one function per C entry point.

Argument marshalling only (ctypes, or a compiled module for the serving operators): tensors are
passed as raw device pointers with their sizes, on the current torch CUDA stream; every step of
the computation runs in the library's CUDA kernels. Outputs that the caller does not supply are
allocated with torch (plumbing).
Loading fails loudly if the library was not built: there is no fallback.
"""
import ctypes
import importlib.util
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkda.so")
NATIVE_PATH = os.path.join(_HERE, "_build", "_kda_native.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE, KDA_ERR_CUDA = range(5)
KDA_F32, KDA_BF16 = 0, 1
DECODE_BETA_LOGIT = 1
CONV_SILU = 1
MAX_WINDOW = 16
NORM_L2, ROPE_INTERLEAVED = 1, 2
PAGE = 64  # tokens of a page of the 8-bit cache
STATUS_BAD_SLOT, STATUS_BAD_OFFSETS, STATUS_TIMEOUT = 1, 4, 8
STATUS_BAD_PAGE, STATUS_BAD_TOKEN, STATUS_BAD_POSITION = 16, 32, 64

_lib = None


class KdaError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"[kda status {status}] {msg}")
        self.status = status


def lib():
    """The loaded libkda.so (ctypes). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libkda.so not found at {LIB_PATH}: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, F, Z, I64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                       ctypes.c_int64)
    L.kda_last_error.restype = ctypes.c_char_p
    L.kda_last_error.argtypes = []
    L.kda_version.restype = ctypes.c_char_p
    L.kda_version.argtypes = []
    L.kda_launch_count.restype = ctypes.c_uint64
    L.kda_launch_count.argtypes = []
    L.kda_chunk_workspace.restype = Z
    L.kda_chunk_workspace.argtypes = [I, I, I, I, I, I]
    L.kda_chunk_prefill.restype = I
    L.kda_chunk_prefill.argtypes = [I, I, I, P, I, I, I, I, F, P, P, P, P, P, P, P, P, P, Z, P,
                                    P]
    L.kda_segment_package.restype = I
    L.kda_segment_package.argtypes = [I, I, I, P, I, I, I, I, P, P, P, P, P, P, P, Z, P, P]
    L.kda_package_scan_workspace.restype = Z
    L.kda_package_scan_workspace.argtypes = [I, I, I, I, I]
    L.kda_package_scan.restype = I
    L.kda_package_scan.argtypes = [I, I, P, I, I, I, I, P, P, P, P, P, P, Z, P, P]
    L.kda_package_scan_noalloc.restype = I
    L.kda_package_scan_noalloc.argtypes = [I, I, P, I, I, I, I, P, P, P, P, P, P, P]
    L.kda_segment_replay.restype = I
    L.kda_segment_replay.argtypes = [I, I, I, P, I, I, I, I, F, P, P, P, P, P, P, P, P, P, Z, P,
                                     P]
    L.kda_chunk_prepare.restype = I
    L.kda_chunk_prepare.argtypes = [I, I, I, P, I, I, I, I, F, P, P, P, P, P, P, Z, P, P]
    L.kda_segment_package_prepared.restype = I
    L.kda_segment_package_prepared.argtypes = [I, I, I, P, I, I, I, I, P, P, P, Z, P, P]
    L.kda_segment_replay_prepared.restype = I
    L.kda_segment_replay_prepared.argtypes = [I, I, I, P, I, I, I, I, P, P, P, P, Z, P, P]
    L.kda_debug_flag_wait.restype = I
    L.kda_debug_flag_wait.argtypes = [I, I, I, P, I, I, I, I, P, P, P, P, Z, ctypes.c_uint64,
                                      P, P]
    L.kda_decode_step.restype = I
    L.kda_decode_step.argtypes = [I, I, I, I, I, F, P, P, P, P, P, P, P, I64, P, P, P]
    L.kda_decode_window.restype = I
    L.kda_decode_window.argtypes = [I, I, I, I, I, I, F, P, P, P, P, P, ctypes.c_uint, P, P, P,
                                    I64, P, P, P]
    L.kda_slot_zero.restype = I
    L.kda_slot_zero.argtypes = [I, P, P, I64, I64, P, P]
    L.kda_slot_copy.restype = I
    L.kda_slot_copy.argtypes = [I, P, P, I64, P, P, I64, I64, P, P]
    L.kda_short_conv.restype = I
    L.kda_short_conv.argtypes = [I, I, I, P, I, I, P, P, ctypes.c_uint, P, P, P, I64, P, P, P]
    L.kda_head_norm_rope.restype = I
    L.kda_head_norm_rope.argtypes = [I, I, I, I, I, P, I64, P, I64, P, P, F, ctypes.c_uint, P, I64,
                                     I, P, P, I64, P, I64, P, P]
    L.kda_cache_write.restype = I
    L.kda_cache_write.argtypes = [I, I, I, P, P, P, I, I, P, I64, P, I64, P, I, P, P, P, P, I64, P,
                                  P]
    L.kda_cache_read.restype = I
    L.kda_cache_read.argtypes = [I, I, I, P, P, I, I, P, I, P, P, P, P, I64, P, P, P, P]
    L.kda_cache_attention_workspace.restype = Z
    L.kda_cache_attention_workspace.argtypes = [I, I, I, I, I]
    L.kda_cache_attention.restype = I
    L.kda_cache_attention.argtypes = [I, I, I, I, I, I, F, P, P, P, P, I, P, P, P, P, I64, P, P, Z,
                                      P, P]
    L.kda_draft_verify.restype = I
    L.kda_draft_verify.argtypes = [I, I, I, I, P, I64, P, I64, P, P, P, P, P, P, P, P, P, P]
    L.kda_decay_prefill_workspace.restype = Z
    L.kda_decay_prefill_workspace.argtypes = [I, I, I, I, I]
    L.kda_decay_prefill.restype = I
    L.kda_decay_prefill.argtypes = [I, I, I, P, I, I, I, F, P, I64, P, I64, P, I64, P, I64, P, P, P,
                                    P, Z, P, P]
    L.kda_decay_window.restype = I
    L.kda_decay_window.argtypes = [I, I, I, I, I, I, F, P, I64, P, I64, P, I64, P, I64, P, P, P, I64,
                                   P, P, P]
    L.kda_cache_weigh.restype = I
    L.kda_cache_weigh.argtypes = [I, I, I, I, I, I, F, F, P, P, P, P, I, P, P, P, I64, P, Z, P, P]
    L.kda_cache_weigh_workspace.restype = Z
    L.kda_cache_weigh_workspace.argtypes = [I, I, I, I, I, I, I]
    L.kda_cache_evict.restype = I
    L.kda_cache_evict.argtypes = [I, I, I, P, P, I, P, I, P, P, P, P, P, I64, I, I, I, P, P, P, P]
    _lib = L
    return L


def version():
    return lib().kda_version().decode()


def launch_count():
    """Kernels launched through the library by this process so far."""
    return int(lib().kda_launch_count())


def last_error():
    return lib().kda_last_error().decode()


def _check(st):
    if st != KDA_OK:
        raise KdaError(st, last_error())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dt(t):
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _int32(*ts):
    for t in ts:
        if t is not None and t.dtype != torch.int32:
            raise TypeError("slot ids must be int32 tensors")


def chunk_workspace(dtype, n_ranges, total_tokens, H, dk, dv):
    """kda_chunk_workspace: scratch bytes of the chunked calls (0 if none is needed)."""
    dt = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_chunk_workspace(dt, n_ranges, total_tokens, H, dk, dv))


def _chunk_ws(workspace, dtype, n_ranges, T, H, dk, dv, device):
    need = chunk_workspace(dtype, n_ranges, T, H, dk, dv)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is None:
        return None, 0
    return workspace, workspace.numel() * workspace.element_size()


def chunk_prefill(q, k, v, g, beta, cu_seqlens=None, init_state=None, scale=1.0, o=None,
                  final_state=None, want_final=True, status=None, chunk=64, workspace=None,
                  stream=None):
    """kda_chunk_prefill. Returns (o, final_state). `workspace` (uint8 device tensor of at
    least chunk_workspace(...) bytes) is allocated here when not given."""
    _contig(q, k, v, g, beta, cu_seqlens, init_state, o, final_state)
    T, H, dk = k.shape
    dv = v.shape[2]
    n = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if o is None:
        o = torch.empty(T, H, dv, dtype=q.dtype, device=q.device)
    if final_state is None and want_final:
        final_state = torch.empty(n, H, dk, dv, dtype=torch.float32, device=q.device)
    ws, ws_bytes = _chunk_ws(workspace, q.dtype, n, T, H, dk, dv, q.device)
    _check(lib().kda_chunk_prefill(_dt(q), n, T, _ptr(cu_seqlens), H, dk, dv, chunk,
                                   float(scale), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                   _ptr(beta), _ptr(init_state), _ptr(o), _ptr(final_state),
                                   _ptr(ws), ws_bytes, _ptr(status), _stream(stream)))
    return o, final_state


def segment_package(k, v, g, beta, seg_offsets, M=None, D=None, status=None, chunk=64,
                    workspace=None, stream=None):
    """kda_segment_package. Returns (M, D)."""
    _contig(k, v, g, beta, seg_offsets, M, D)
    T, H, dk = k.shape
    dv = v.shape[2]
    P = seg_offsets.numel() - 1
    if M is None:
        M = torch.empty(P, H, dk, dk, dtype=torch.float32, device=k.device)
    if D is None:
        D = torch.empty(P, H, dk, dv, dtype=torch.float32, device=k.device)
    ws, ws_bytes = _chunk_ws(workspace, k.dtype, P, T, H, dk, dv, k.device)
    _check(lib().kda_segment_package(_dt(k), P, T, _ptr(seg_offsets), H, dk, dv, chunk,
                                     _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(M), _ptr(D),
                                     _ptr(ws), ws_bytes, _ptr(status), _stream(stream)))
    return M, D


def package_scan_workspace(n_seqs, max_segs_per_seq, H, dk, dv):
    return int(lib().kda_package_scan_workspace(n_seqs, max_segs_per_seq, H, dk, dv))


def package_scan(M, D, seq_seg_offsets, max_segs_per_seq, init_state=None, seg_init=None,
                 final_state=None, want_final=True, workspace=None, status=None, stream=None):
    """kda_package_scan. Returns (seg_init, final_state)."""
    _contig(M, D, seq_seg_offsets, init_state, seg_init, final_state)
    P, H, dk, dv = D.shape
    n = seq_seg_offsets.numel() - 1
    if seg_init is None:
        seg_init = torch.empty(P, H, dk, dv, dtype=torch.float32, device=D.device)
    if final_state is None and want_final:
        final_state = torch.empty(n, H, dk, dv, dtype=torch.float32, device=D.device)
    ws_bytes = package_scan_workspace(n, max_segs_per_seq, H, dk, dv)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=D.device)
    _check(lib().kda_package_scan(n, P, _ptr(seq_seg_offsets), int(max_segs_per_seq), H, dk,
                                  dv, _ptr(M), _ptr(D), _ptr(init_state), _ptr(seg_init),
                                  _ptr(final_state), _ptr(workspace), workspace.numel(),
                                  _ptr(status), _stream(stream)))
    return seg_init, final_state


def package_scan_noalloc(M, D, seq_seg_offsets, max_segs_per_seq, init_state=None,
                         seg_init=None, final_state=None, want_final=True, status=None,
                         stream=None):
    """kda_package_scan_noalloc: the scan with the library's built-in 64 MiB scratch, for
    callers that cannot allocate device memory (pass seg_init / final_state to allocate
    nothing here either). Returns (seg_init, final_state)."""
    _contig(M, D, seq_seg_offsets, init_state, seg_init, final_state)
    P, H, dk, dv = D.shape
    n = seq_seg_offsets.numel() - 1
    if seg_init is None:
        seg_init = torch.empty(P, H, dk, dv, dtype=torch.float32, device=D.device)
    if final_state is None and want_final:
        final_state = torch.empty(n, H, dk, dv, dtype=torch.float32, device=D.device)
    _check(lib().kda_package_scan_noalloc(n, P, _ptr(seq_seg_offsets), int(max_segs_per_seq),
                                          H, dk, dv, _ptr(M), _ptr(D), _ptr(init_state),
                                          _ptr(seg_init), _ptr(final_state), _ptr(status),
                                          _stream(stream)))
    return seg_init, final_state


def segment_replay(q, k, v, g, beta, seg_offsets, seg_init, scale=1.0, o=None,
                   seg_final=None, want_final=False, status=None, chunk=64, workspace=None,
                   stream=None):
    """kda_segment_replay. Returns (o, seg_final)."""
    _contig(q, k, v, g, beta, seg_offsets, seg_init, o, seg_final)
    T, H, dk = k.shape
    dv = v.shape[2]
    P = seg_offsets.numel() - 1
    if o is None:
        o = torch.empty(T, H, dv, dtype=q.dtype, device=q.device)
    if seg_final is None and want_final:
        seg_final = torch.empty(P, H, dk, dv, dtype=torch.float32, device=q.device)
    ws, ws_bytes = _chunk_ws(workspace, q.dtype, P, T, H, dk, dv, q.device)
    _check(lib().kda_segment_replay(_dt(q), P, T, _ptr(seg_offsets), H, dk, dv, chunk,
                                    float(scale), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                    _ptr(beta), _ptr(seg_init), _ptr(o), _ptr(seg_final),
                                    _ptr(ws), ws_bytes, _ptr(status), _stream(stream)))
    return o, seg_final


def chunk_prepare(q, k, v, g, beta, offsets=None, scale=1.0, workspace=None, status=None,
                  chunk=64, stream=None):
    """kda_chunk_prepare: per-chunk records of the ranges in `offsets` (q may be None when
    only packages will be built). Returns the workspace tensor holding them."""
    _contig(q, k, v, g, beta, offsets)
    T, H, dk = k.shape
    dv = v.shape[2]
    n = 1 if offsets is None else offsets.numel() - 1
    ws, ws_bytes = _chunk_ws(workspace, k.dtype, n, T, H, dk, dv, k.device)
    _check(lib().kda_chunk_prepare(_dt(k), n, T, _ptr(offsets), H, dk, dv, chunk, float(scale),
                                   _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(ws),
                                   ws_bytes, _ptr(status), _stream(stream)))
    return ws


def segment_package_prepared(workspace, seg_offsets, T, H, dk, dv, M=None, D=None,
                             dtype=torch.bfloat16, status=None, chunk=64, stream=None):
    """kda_segment_package_prepared over records from chunk_prepare. Returns (M, D)."""
    _contig(seg_offsets, M, D)
    P = seg_offsets.numel() - 1
    dev = workspace.device
    if M is None:
        M = torch.empty(P, H, dk, dk, dtype=torch.float32, device=dev)
    if D is None:
        D = torch.empty(P, H, dk, dv, dtype=torch.float32, device=dev)
    dt = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    _check(lib().kda_segment_package_prepared(dt, P, T, _ptr(seg_offsets), H, dk, dv, chunk,
                                              _ptr(M), _ptr(D), _ptr(workspace),
                                              workspace.numel(), _ptr(status), _stream(stream)))
    return M, D


def segment_replay_prepared(workspace, seg_offsets, seg_init, T, H, dk, dv, o=None,
                            seg_final=None, want_final=False, dtype=torch.bfloat16, status=None,
                            chunk=64, stream=None):
    """kda_segment_replay_prepared over records prepared with q. Returns (o, seg_final)."""
    _contig(seg_offsets, seg_init, o, seg_final)
    P = seg_offsets.numel() - 1
    dev = workspace.device
    if o is None:
        o = torch.empty(T, H, dv, dtype=dtype, device=dev)
    if seg_final is None and want_final:
        seg_final = torch.empty(P, H, dk, dv, dtype=torch.float32, device=dev)
    dt = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    _check(lib().kda_segment_replay_prepared(dt, P, T, _ptr(seg_offsets), H, dk, dv, chunk,
                                             _ptr(seg_init), _ptr(o), _ptr(seg_final),
                                             _ptr(workspace), workspace.numel(), _ptr(status),
                                             _stream(stream)))
    return o, seg_final


RECORD_BYTES = 147968  # one (64-token chunk, head) record of the tensor-core chunk path


def record_flags(workspace, n_ranges, T, H):
    """The ready flags after the records in a chunk workspace (an int32 view)."""
    R = (T // 64 + n_ranges) * H
    return workspace[R * RECORD_BYTES:R * RECORD_BYTES + 4 * R].view(torch.int32)


def debug_flag_wait(workspace, seg_offsets, seg_init, T, H, dk, dv, limit_ns, o=None,
                    seg_final=None, want_final=False, status=None, dtype=torch.bfloat16,
                    chunk=64, stream=None):
    """kda_debug_flag_wait: the prepared replay walk, each record gated by its ready flag
    (bounded by limit_ns). Returns (o, seg_final)."""
    _contig(seg_offsets, seg_init, o, seg_final)
    P = seg_offsets.numel() - 1
    dev = workspace.device
    if o is None:
        o = torch.zeros(T, H, dv, dtype=dtype, device=dev)
    if seg_final is None and want_final:
        seg_final = torch.empty(P, H, dk, dv, dtype=torch.float32, device=dev)
    dt = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    _check(lib().kda_debug_flag_wait(dt, P, T, _ptr(seg_offsets), H, dk, dv, chunk,
                                     _ptr(seg_init), _ptr(o), _ptr(seg_final), _ptr(workspace),
                                     workspace.numel(), int(limit_ns), _ptr(status),
                                     _stream(stream)))
    return o, seg_final


def decode_step(q, k, v, g, beta, slot_ids, state_pool, scale=1.0, o=None, status=None,
                stream=None):
    """kda_decode_step (state_pool updated in place). Returns o."""
    _contig(q, k, v, g, beta, slot_ids, state_pool, o)
    B, H, dk = k.shape
    dv = v.shape[2]
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    _check(lib().kda_decode_step(_dt(q), B, H, dk, dv, float(scale), _ptr(q), _ptr(k), _ptr(v),
                                 _ptr(g), _ptr(beta), _ptr(slot_ids), _ptr(state_pool),
                                 int(state_pool.shape[0]), _ptr(o), _ptr(status),
                                 _stream(stream)))
    return o


def decode_window(q, k, v, g, beta, read_slots, write_slots, state_pool, scale=1.0,
                  beta_is_logit=False, o=None, status=None, stream=None):
    """kda_decode_window: rows of `window` tokens (write_slots is [batch, window]; q, k, g are
    [batch*window, H, dk] or [batch, window, H, dk], likewise v and beta). Row b reads slot
    read_slots[b] and stores its state after token j into slot write_slots[b, j]. Returns o,
    shaped like v."""
    _contig(q, k, v, g, beta, read_slots, write_slots, state_pool, o)
    _int32(read_slots, write_slots)
    B = read_slots.numel()
    W = write_slots.numel() // B if B else 0
    if write_slots.numel() != B * W:
        raise ValueError("write_slots must hold batch x window ids")
    H, dk = k.shape[-2], k.shape[-1]
    dv = v.shape[-1]
    if k.numel() != B * W * H * dk:
        raise ValueError("k must hold batch x window tokens")
    if o is None:
        o = torch.empty(v.shape, dtype=q.dtype, device=q.device)
    _check(lib().kda_decode_window(_dt(q), B, W, H, dk, dv, float(scale), _ptr(q), _ptr(k),
                                   _ptr(v), _ptr(g), _ptr(beta),
                                   DECODE_BETA_LOGIT if beta_is_logit else 0, _ptr(read_slots),
                                   _ptr(write_slots), _ptr(state_pool),
                                   int(state_pool.shape[0]), _ptr(o), _ptr(status),
                                   _stream(stream)))
    return o


def slot_zero(state_pool, slot_ids=None, n=None, status=None, stream=None):
    """kda_slot_zero: zero the listed slots of state_pool (all of slots 0..n-1 when slot_ids
    is None)."""
    _contig(state_pool, slot_ids)
    _int32(slot_ids)
    if n is None:
        n = slot_ids.numel() if slot_ids is not None else state_pool.shape[0]
    _check(lib().kda_slot_zero(int(n), _ptr(slot_ids), _ptr(state_pool),
                               int(state_pool.shape[0]), int(state_pool[0].numel()),
                               _ptr(status), _stream(stream)))
    return state_pool


def slot_copy(src, src_ids, dst, dst_ids, n=None, status=None, stream=None):
    """kda_slot_copy: dst[dst_ids[i]] = src[src_ids[i]] (None ids mean 0..n-1)."""
    _contig(src, src_ids, dst, dst_ids)
    _int32(src_ids, dst_ids)
    if src[0].numel() != dst[0].numel():
        raise ValueError("src and dst slots differ in size")
    if n is None:
        n = src_ids.numel() if src_ids is not None else dst_ids.numel()
    _check(lib().kda_slot_copy(int(n), _ptr(src), _ptr(src_ids), int(src.shape[0]), _ptr(dst),
                               _ptr(dst_ids), int(dst.shape[0]), int(src[0].numel()),
                               _ptr(status), _stream(stream)))
    return dst


def short_conv(x, weight, cu_seqlens=None, silu=False, read_slots=None, write_slots=None,
               conv_state=None, out=None, status=None, stream=None):
    """kda_short_conv: causal depthwise convolution of x [T, C] with weight [C, W] over the
    packed sequences of cu_seqlens, each starting from the W - 1 inputs in conv_state
    [n_slots, W-1, C] at its read slot and leaving its last W - 1 inputs at its write slot.
    Returns out [T, C]."""
    _contig(x, weight, cu_seqlens, read_slots, write_slots, conv_state, out)
    _int32(cu_seqlens, read_slots, write_slots)
    T, C = x.shape
    W = weight.shape[1]
    n = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty_like(x)
    n_slots = 0 if conv_state is None else int(conv_state.shape[0])
    _check(lib().kda_short_conv(_dt(x), n, T, _ptr(cu_seqlens), C, W, _ptr(x), _ptr(weight),
                                CONV_SILU if silu else 0, _ptr(read_slots), _ptr(write_slots),
                                _ptr(conv_state), n_slots, _ptr(out), _ptr(status),
                                _stream(stream)))
    return out


# The serving operators are called once or more per layer and token, and a call's host time is
# what bounds it at small sizes: their checks and allocations run in a compiled module
# (csrc/kda_binding.cpp) that calls the same C entry points.

_native_module = None


def _native():
    """The compiled half of the binding. Raises if it has not been built."""
    global _native_module
    if _native_module is None:
        lib()
        if not os.path.exists(NATIVE_PATH):
            raise RuntimeError(f"_kda_native.so not found at {NATIVE_PATH}: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        spec = importlib.util.spec_from_file_location("_kda_native", NATIVE_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native_module = module
    return _native_module


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def head_norm_rope(q, k, q_weight=None, k_weight=None, eps=1e-6, l2=False, cos_sin=None,
                   positions=None, interleaved=False, q_out=None, k_out=None, status=None,
                   stream=None):
    """kda_head_norm_rope: RMS norm (2-norm with l2) of each head of q [T, Hq, d] and k [T, Hk, d]
    with per-channel weights, then the rotation by row `positions[t]` of cos_sin [n_pos, rot_dim]
    (none when cos_sin is None). q and k may be views of a fused projection's rows; either may be
    None. q_out = q (k_out = k) works in place. Returns (q_out, k_out)."""
    r = (_native_module or _native()).head_norm_rope(
        q, k, q_weight, k_weight, eps, l2, cos_sin, positions, interleaved, q_out, k_out, status,
        _handle(stream))
    if r.__class__ is int:
        _check(r)
    return r


def cache_write(k, v, start, page_table, k_cache, k_scale, v_cache, v_scale, cu_seqlens=None,
                lens=None, status=None, stream=None):
    """kda_cache_write: quantises k and v [T, Hkv, d] (views of a fused projection's rows are fine)
    into the paged cache [n_pages, Hkv, 64, d] with scales [n_pages, Hkv], token i of sequence s at
    position start[s] + i. The caches and scales are updated in place. A page's scale only grows
    while it keeps tokens, also for drafted tokens that are refused later."""
    r = (_native_module or _native()).cache_write(
        k, v, start, page_table, k_cache, k_scale, v_cache, v_scale, cu_seqlens, lens, status,
        _handle(stream))
    if r is not None:
        _check(r)


def cache_read(start, page_table, k_cache, k_scale, v_cache, v_scale, total_tokens,
               cu_seqlens=None, dtype=torch.bfloat16, k=None, v=None, status=None, stream=None):
    """kda_cache_read: cached keys and values of positions start[s] .. of each sequence, packed by
    cu_seqlens (total_tokens rows in all; rows that no sequence covers are not written). Returns
    (k, v), [total_tokens, Hkv, d] of `dtype`."""
    r = (_native_module or _native()).cache_read(
        start, page_table, k_cache, k_scale, v_cache, v_scale, total_tokens, cu_seqlens, dtype, k,
        v, status, _handle(stream))
    if r.__class__ is int:
        _check(r)
    return r


def cache_attention_workspace(batch, window, Hq, Hkv, d):
    """kda_cache_attention_workspace: scratch bytes of cache_attention."""
    return int(lib().kda_cache_attention_workspace(batch, window, Hq, Hkv, d))


def cache_attention(q, start, page_table, k_cache, k_scale, v_cache, v_scale, scale=1.0, lens=None,
                    o=None, workspace=None, status=None, stream=None):
    """kda_cache_attention: q [batch*window, Hq, d] or [batch, window, Hq, d], the window's token j
    of row b at position start[b] + j, seeing the cached positions 0 .. start[b] + j: one decoded
    token, a verify window, or a chunk of a prompt (any window up to 65536). `workspace`
    (uint8 device tensor of at least cache_attention_workspace(...) bytes) is allocated here when
    not given. Returns o, shaped like q. `status` (int32) tells of pages that were skipped, and of a
    wait inside the kernel that gave up, which leaves o undefined."""
    r = (_native_module or _native()).cache_attention(
        q, start, page_table, k_cache, k_scale, v_cache, v_scale, scale, lens, o, workspace, status,
        _handle(stream))
    if r.__class__ is int:
        _check(r)
    return r


def draft_verify(target_probs, draft_tokens, u_accept, u_sample, draft_probs=None, lens=None,
                 write_slots=None, tokens=None, n_accepted=None, resume_slots=None, status=None,
                 stream=None):
    """kda_draft_verify: takes the drafts [batch, window] in order while u * q(x) < p(x), then
    samples one token from the rest of p (target_probs [batch, window+1, vocab], draft_probs
    [batch, window, vocab] or None for drafts that were not sampled). Returns (n_accepted [batch],
    tokens [batch, window+1] padded with -1, resume_slots [batch]: write_slots[b, n_accepted[b]],
    the slot to resume the recurrent state from, or None without write_slots)."""
    r = (_native_module or _native()).draft_verify(
        target_probs, draft_tokens, u_accept, u_sample, draft_probs, lens, write_slots, tokens,
        n_accepted, resume_slots, status, _handle(stream))
    if r.__class__ is int:
        _check(r)
    return r


def decay_prefill_workspace(dtype, n_seqs, total_tokens, H, d):
    """kda_decay_prefill_workspace: scratch bytes of decay_prefill."""
    dt = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_decay_prefill_workspace(dt, n_seqs, total_tokens, H, d))


def decay_prefill(q, k, v, g, cu_seqlens=None, init_state=None, scale=1.0, o=None,
                  final_state=None, want_final=True, status=None, workspace=None, stream=None):
    """kda_decay_prefill: linear attention with one decay per head over packed prompts. q, k
    [T, Hk, d] and v [T, H, d] may be views of a fused projection's rows, each q and k head shared by
    H / Hk heads; g is [T, H] fp32 log-decays, or [H] for a constant decay per head. `workspace`
    (uint8 device tensor of at least decay_prefill_workspace(...) bytes) is allocated here when not
    given. Returns (o [T, H, d], final_state [n, H, d, d] or None)."""
    r = (_native_module or _native()).decay_prefill(
        q, k, v, g, cu_seqlens, init_state, scale, o, final_state, want_final, status, workspace,
        _handle(stream))
    if r.__class__ is int:
        _check(r)
    return r


def decay_window(q, k, v, g, read_slots, write_slots, state_pool, scale=1.0, o=None, status=None,
                 stream=None):
    """kda_decay_window: linear attention with one decay per head for rows of `window` tokens
    (write_slots is [batch, window]; q, k [batch*window, Hk, d], v [batch*window, H, d], g
    [batch*window, H] or [H]). Row b reads slot read_slots[b] of state_pool [n_slots, H, d, d] and
    stores its state after token j into slot write_slots[b, j]; one token with write_slots =
    read_slots is a decode step in place. Returns o, shaped like v."""
    r = (_native_module or _native()).decay_window(
        q, k, v, g, read_slots, write_slots, state_pool, scale, o, status, _handle(stream))
    if r.__class__ is int:
        _check(r)
    return r


def cache_weigh_workspace(dtype, batch, window, Hq, Hkv, d, max_pages):
    """kda_cache_weigh_workspace: scratch bytes of cache_weigh (0 where it needs none)."""
    dt = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_cache_weigh_workspace(dt, batch, window, Hq, Hkv, d, max_pages))


def cache_weigh(q, start, page_table, k_cache, k_scale, weights, scale=1.0, lens=None, keep=1.0,
                workspace=None, status=None, stream=None):
    """kda_cache_weigh: adds to weights [n_pages, Hkv, 64] the softmax weights with which the
    window's queries (as for cache_attention) see each cached token, summed over the window's
    tokens and the head's query heads; what the tokens before the window had counts `keep` times.
    `workspace` (uint8 device tensor of at least cache_weigh_workspace(...) bytes) is allocated here
    when not given. Returns weights, updated in place."""
    r = (_native_module or _native()).cache_weigh(
        q, start, page_table, k_cache, k_scale, weights, scale, lens, keep, workspace, status,
        _handle(stream))
    if r.__class__ is int:
        _check(r)
    return r


def cache_evict(length, page_table, new_table, k_cache, k_scale, v_cache, v_scale, weights, budget,
                sinks=0, recent=0, new_length=None, kept=None, status=None, stream=None):
    """kda_cache_evict: keeps `budget` of each row's length[b] cached tokens, per head: the first
    `sinks`, the last `recent`, and of the rest those of the largest weights. They move, in order,
    into the pages of new_table [n, pages], which hold no tokens of any row yet; the old pages can
    be reused after the call. Returns (new_length [n], kept [n, Hkv, budget]: the positions kept,
    then -1)."""
    r = (_native_module or _native()).cache_evict(
        length, page_table, new_table, k_cache, k_scale, v_cache, v_scale, weights, budget, sinks,
        recent, new_length, kept, status, _handle(stream))
    if r.__class__ is int:
        _check(r)
    return r
