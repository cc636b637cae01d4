"""ctypes binding of librk.so (include/rk.h), argument marshalling only.

The functions here carry the C ABI's names and arguments.  Every step of a
reduction runs in the library's HIP kernels; nothing here computes.  Loading
fails loudly when the library has not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librk.so")

# enums of include/rk.h
RK_OK, RK_ERR_INVALID_ARGUMENT, RK_ERR_UNSUPPORTED, RK_ERR_HIP, RK_ERR_TOO_LARGE = 0, 1, 2, 3, 4
RK_OP_SUM, RK_OP_MAX, RK_OP_MIN = 0, 1, 2
RK_MAP_IDENTITY, RK_MAP_SQUARE, RK_MAP_ABS = 0, 1, 2
RK_MAP2_MUL, RK_MAP2_SQDIFF, RK_MAP2_ABSDIFF = 0, 1, 2
RK_F32, RK_BF16, RK_F16, RK_F64, RK_I32, RK_I64 = 0, 1, 2, 3, 4, 5
RK_MODE_OVERWRITE, RK_MODE_FOLD, RK_MODE_HOST = 0, 1, 2
RK_GATE_VALUE, RK_GATE_LOG, RK_GATE_SIGMOID = 0, 1, 2
(RK_KERNEL_NONE, RK_KERNEL_ALL, RK_KERNEL_ALL_STRIDED, RK_KERNEL_THREAD, RK_KERNEL_TILED,
 RK_KERNEL_COLUMNS, RK_KERNEL_ROW, RK_KERNEL_GENERIC, RK_KERNEL_ALL2, RK_KERNEL_SCAN_TILE,
 RK_KERNEL_SCAN_ROWWAVE, RK_KERNEL_SCAN_LINES, RK_KERNEL_SCAN_COLUMNS, RK_KERNEL_SCAN_TRANSPOSE,
 RK_KERNEL_SOFTMAX_LINE, RK_KERNEL_SOFTMAX_SPLIT, RK_KERNEL_DRAFT_VERIFY) = range(17)
KERNEL_NAMES = {0: "none", 1: "all", 2: "all_strided", 3: "thread", 4: "tiled", 5: "columns",
                6: "row", 7: "generic", 8: "all2", 9: "scan_tile", 10: "scan_rowwave",
                11: "scan_lines", 12: "scan_columns", 13: "scan_transpose",
                14: "softmax_line", 15: "softmax_split", 16: "draft_verify"}

# every function include/rk.h declares
EXPORTS = ("rk_workspace_size", "rk_reduce_all", "rk_reduce_all2", "rk_reduce_dims", "rk_status_string",
           "rk_plan_all", "rk_plan_all2", "rk_plan_dims", "rk_debug_set_fused_finish",
           "rk_debug_set_launch_events", "rk_scan_workspace_size", "rk_scan", "rk_scan_dims",
           "rk_plan_scan", "rk_debug_stream_read", "rk_debug_device_info", "rk_debug_set_finish_tag",
           "rk_stream_timeouts", "rk_debug_force_wait_timeout", "rk_debug_fail_launches",
           "rk_reduce_dims_no_workspace",
           "rk_softmax_workspace_size", "rk_softmax", "rk_draft_verify_workspace_size", "rk_draft_verify",
           "rk_block_tables_workspace_size", "rk_block_tables", "rk_slot_map",
           "rk_plan_softmax", "rk_plan_draft_verify",
           "rk_beam_select_workspace_size", "rk_beam_select", "rk_fork_blocks_workspace_size", "rk_fork_blocks",
           "rk_compact_blocks_workspace_size", "rk_compact_blocks", "rk_copy_blocks",
           "rk_linear_recurrence_workspace_size", "rk_linear_recurrence", "rk_linear_recurrence_backward")


class rk_plan_info(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("launches", ctypes.c_int), ("grid", ctypes.c_int64),
                ("block", ctypes.c_int), ("split", ctypes.c_int), ("vec", ctypes.c_int),
                ("tile_outputs", ctypes.c_int), ("n_out", ctypes.c_int64),
                ("reduce_len", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t)]


class rk_block_cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("block_stride", ctypes.c_int64), ("block_bytes", ctypes.c_int64),
                ("n_blocks", ctypes.c_int64)]


class rk_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("seq_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


class RkError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})" if what
                         else f"{status_string(status)} (status {status})")


_lib = None


def load() -> ctypes.CDLL:
    """Load librk.so; raises when it is missing (build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"librk.so not found at {LIB_PATH}; build it with "
            "`python -m reduction_primitives_amd.build` (there is no fallback path)")
    # torch's HIP runtime must be the one the library binds to (same SONAME)
    import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint32,
                             ctypes.c_size_t)
    p64 = ctypes.POINTER(ctypes.c_int64)
    lib.rk_workspace_size.argtypes = [i32, i32, i32, p64, p64, u32]
    lib.rk_workspace_size.restype = sz
    lib.rk_reduce_all.argtypes = [i32, i32, i32, i32, i32, vp, i64, vp, i32, vp, vp, vp]
    lib.rk_reduce_all.restype = i32
    lib.rk_reduce_all2.argtypes = [i32, i32, i32, i32, i32, vp, vp, i64, vp, i32, vp, vp, vp]
    lib.rk_reduce_all2.restype = i32
    lib.rk_reduce_dims.argtypes = [i32, i32, i32, i32, i32, vp, i32, p64, p64, u32, vp, i32, vp, vp, vp]
    lib.rk_reduce_dims.restype = i32
    lib.rk_reduce_dims_no_workspace.argtypes = [i32, i32, i32, i32, i32, vp, i32, p64, p64, u32, vp, i32, vp, vp]
    lib.rk_reduce_dims_no_workspace.restype = i32
    lib.rk_scan_workspace_size.argtypes = [i32, i32, i32, p64, p64, i32]
    lib.rk_scan_workspace_size.restype = sz
    lib.rk_scan.argtypes = [i32, i32, i32, i32, vp, i64, vp, i32, vp, vp, vp]
    lib.rk_scan.restype = i32
    lib.rk_scan_dims.argtypes = [i32, i32, i32, i32, vp, i32, p64, p64, i32, vp, i32, vp, vp, vp]
    lib.rk_scan_dims.restype = i32
    lib.rk_plan_scan.argtypes = [i32, i32, i32, vp, vp, i32, p64, p64, i32, i32, ctypes.POINTER(rk_plan_info)]
    lib.rk_plan_scan.restype = i32
    lib.rk_status_string.argtypes = [i32]
    lib.rk_status_string.restype = ctypes.c_char_p
    lib.rk_plan_all.argtypes = [i32, i32, vp, i64, i32, ctypes.POINTER(rk_plan_info)]
    lib.rk_plan_all.restype = i32
    lib.rk_plan_all2.argtypes = [i32, i32, vp, vp, i64, i32, ctypes.POINTER(rk_plan_info)]
    lib.rk_plan_all2.restype = i32
    lib.rk_plan_dims.argtypes = [i32, i32, vp, i32, p64, p64, u32, i32, ctypes.POINTER(rk_plan_info)]
    lib.rk_plan_dims.restype = i32
    lib.rk_debug_set_fused_finish.argtypes = [i32]
    lib.rk_debug_set_fused_finish.restype = i32
    lib.rk_debug_set_launch_events.argtypes = [vp, vp]
    lib.rk_debug_set_launch_events.restype = i32
    lib.rk_debug_stream_read.argtypes = [vp, i64, i32, vp, vp]
    lib.rk_debug_stream_read.restype = i32
    lib.rk_debug_device_info.argtypes = [p64, p64, p64]
    lib.rk_debug_device_info.restype = i32
    lib.rk_debug_set_finish_tag.argtypes = [vp, u32]
    lib.rk_debug_set_finish_tag.restype = i32
    lib.rk_stream_timeouts.argtypes = [vp, ctypes.POINTER(ctypes.c_uint64)]
    lib.rk_stream_timeouts.restype = i32
    lib.rk_debug_force_wait_timeout.argtypes = [i64]
    lib.rk_debug_force_wait_timeout.restype = i32
    lib.rk_debug_fail_launches.argtypes = [i32]
    lib.rk_debug_fail_launches.restype = i32
    lib.rk_softmax_workspace_size.argtypes = [i32, i32, i64, i64]
    lib.rk_softmax_workspace_size.restype = sz
    lib.rk_softmax.argtypes = [i32, i32, vp, i64, i64, i64, vp, vp, i64, vp, sz, vp]
    lib.rk_softmax.restype = i32
    lib.rk_draft_verify_workspace_size.argtypes = [i32, i64, i64]
    lib.rk_draft_verify_workspace_size.restype = sz
    lib.rk_draft_verify.argtypes = [i32, i32, vp, i64, vp, i64, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.rk_draft_verify.restype = i32
    lib.rk_block_tables_workspace_size.argtypes = [i64]
    lib.rk_block_tables_workspace_size.restype = sz
    lib.rk_block_tables.argtypes = [vp, i64, i32, vp, vp, vp, i64, i32, vp, i64, vp, vp, vp, sz, vp]
    lib.rk_block_tables.restype = i32
    lib.rk_slot_map.argtypes = [vp, vp, i64, i32, vp, i64, i32, vp, i64, i32, i64, vp, vp, vp, vp, vp]
    lib.rk_slot_map.restype = i32
    lib.rk_plan_softmax.argtypes = [i32, i32, i64, i64, ctypes.POINTER(rk_plan_info)]
    lib.rk_plan_softmax.restype = i32
    lib.rk_plan_draft_verify.argtypes = [i32, i64, i64, i32, ctypes.POINTER(rk_plan_info)]
    lib.rk_plan_draft_verify.restype = i32
    lib.rk_beam_select_workspace_size.argtypes = [i32, i64, i64, i32, i32]
    lib.rk_beam_select_workspace_size.restype = sz
    lib.rk_beam_select.argtypes = [i32, i32, vp, i64, i64, i64, i32, vp, vp, i64, i32, vp, vp, vp, vp, sz, vp]
    lib.rk_beam_select.restype = i32
    lib.rk_fork_blocks_workspace_size.argtypes = [i64, i64, i32, i64]
    lib.rk_fork_blocks_workspace_size.restype = sz
    lib.rk_fork_blocks.argtypes = [vp, i64, vp, i64, i32, vp, vp, i64, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.rk_fork_blocks.restype = i32
    lib.rk_compact_blocks_workspace_size.argtypes = [i64]
    lib.rk_compact_blocks_workspace_size.restype = sz
    lib.rk_compact_blocks.argtypes = [vp, i64, vp, i64, i32, i64, vp, i64, vp, i64, vp, i64, vp, vp, sz, vp]
    lib.rk_compact_blocks.restype = i32
    lib.rk_copy_blocks.argtypes = [ctypes.POINTER(rk_block_cache), i32, vp, i64, vp]
    lib.rk_copy_blocks.restype = i32
    rows = ctypes.POINTER(rk_rows)
    lib.rk_linear_recurrence_workspace_size.argtypes = [i32, i32, i64, i64, i64, i32]
    lib.rk_linear_recurrence_workspace_size.restype = sz
    lib.rk_linear_recurrence.argtypes = [i32, i32, i32, i32, rows, rows, vp, i64, vp, vp, i64, i64, i64, rows, vp, vp, sz, vp]
    lib.rk_linear_recurrence.restype = i32
    lib.rk_linear_recurrence_backward.argtypes = [i32, i32, i32, i32, rows, rows, rows, rows, vp, vp, vp, i64, i64, i64, rows,
                                                  rows, vp, vp, sz, vp]
    lib.rk_linear_recurrence_backward.restype = i32
    _lib = lib
    return lib


def _i64_array(vals):
    vals = [int(v) for v in vals]
    return (ctypes.c_int64 * max(1, len(vals)))(*vals)


def status_string(status: int) -> str:
    return load().rk_status_string(int(status)).decode()


def rk_workspace_size(in_dtype, acc_dtype, ndim, shape, strides, reduce_mask) -> int:
    return int(load().rk_workspace_size(in_dtype, acc_dtype, ndim, _i64_array(shape),
                                        _i64_array(strides), reduce_mask))


def rk_reduce_all(op, map_, in_dtype, acc_dtype, out_dtype, ptr, n, init, mode, out, workspace,
                  stream) -> int:
    """Raw call; `init` and host-mode `out` are ctypes objects or None/addresses."""
    return int(load().rk_reduce_all(op, map_, in_dtype, acc_dtype, out_dtype, ptr, n, init, mode,
                                    out, workspace, stream))


def rk_reduce_all2(op, map2, in_dtype, acc_dtype, out_dtype, a, b, n, init, mode, out, workspace,
                   stream) -> int:
    return int(load().rk_reduce_all2(op, map2, in_dtype, acc_dtype, out_dtype, a, b, n, init, mode,
                                     out, workspace, stream))


def rk_reduce_dims(op, map_, in_dtype, acc_dtype, out_dtype, ptr, ndim, shape, strides,
                   reduce_mask, init, mode, out, workspace, stream) -> int:
    return int(load().rk_reduce_dims(op, map_, in_dtype, acc_dtype, out_dtype, ptr, ndim,
                                     _i64_array(shape), _i64_array(strides), reduce_mask, init,
                                     mode, out, workspace, stream))


def rk_reduce_dims_no_workspace(op, map_, in_dtype, acc_dtype, out_dtype, ptr, ndim, shape, strides,
                                reduce_mask, init, mode, out, stream) -> int:
    """rk_reduce_dims with the library's scratch in place of a workspace."""
    return int(load().rk_reduce_dims_no_workspace(op, map_, in_dtype, acc_dtype, out_dtype, ptr, ndim,
                                                  _i64_array(shape), _i64_array(strides), reduce_mask, init,
                                                  mode, out, stream))


def rk_plan_all(in_dtype, acc_dtype, ptr, n, num_cus=0) -> rk_plan_info:
    info = rk_plan_info()
    rc = load().rk_plan_all(in_dtype, acc_dtype, ptr, n, num_cus, ctypes.byref(info))
    if rc:
        raise RkError(rc, "rk_plan_all")
    return info


def rk_plan_all2(in_dtype, acc_dtype, a, b, n, num_cus=0) -> rk_plan_info:
    info = rk_plan_info()
    rc = load().rk_plan_all2(in_dtype, acc_dtype, a, b, n, num_cus, ctypes.byref(info))
    if rc:
        raise RkError(rc, "rk_plan_all2")
    return info


def rk_plan_dims(in_dtype, acc_dtype, ptr, ndim, shape, strides, reduce_mask, num_cus=0) -> rk_plan_info:
    info = rk_plan_info()
    rc = load().rk_plan_dims(in_dtype, acc_dtype, ptr, ndim, _i64_array(shape), _i64_array(strides),
                             reduce_mask, num_cus, ctypes.byref(info))
    if rc:
        raise RkError(rc, "rk_plan_dims")
    return info


def rk_scan_workspace_size(in_dtype, acc_dtype, ndim, shape, strides, dim) -> int:
    return int(load().rk_scan_workspace_size(in_dtype, acc_dtype, ndim, _i64_array(shape),
                                             _i64_array(strides), dim))


def rk_scan(op, in_dtype, acc_dtype, out_dtype, ptr, n, init, inclusive, out, workspace, stream) -> int:
    return int(load().rk_scan(op, in_dtype, acc_dtype, out_dtype, ptr, n, init, inclusive, out, workspace,
                              stream))


def rk_scan_dims(op, in_dtype, acc_dtype, out_dtype, ptr, ndim, shape, strides, dim, init, inclusive, out,
                 workspace, stream) -> int:
    return int(load().rk_scan_dims(op, in_dtype, acc_dtype, out_dtype, ptr, ndim, _i64_array(shape),
                                   _i64_array(strides), dim, init, inclusive, out, workspace, stream))


def rk_plan_scan(in_dtype, acc_dtype, out_dtype, ptr, out, ndim, shape, strides, dim, num_cus=0) -> rk_plan_info:
    info = rk_plan_info()
    rc = load().rk_plan_scan(in_dtype, acc_dtype, out_dtype, ptr, out, ndim, _i64_array(shape),
                             _i64_array(strides), dim, num_cus, ctypes.byref(info))
    if rc:
        raise RkError(rc, "rk_plan_scan")
    return info


def rk_softmax_workspace_size(in_dtype, out_dtype, n, lines) -> int:
    return int(load().rk_softmax_workspace_size(in_dtype, out_dtype, n, lines))


def rk_softmax(in_dtype, out_dtype, x, n, lines, x_stride, temperature, out, out_stride, workspace,
               workspace_bytes, stream) -> int:
    return load().rk_softmax(in_dtype, out_dtype, x, n, lines, x_stride, temperature, out, out_stride, workspace,
                             workspace_bytes, stream)


def rk_draft_verify_workspace_size(prob_dtype, vocab, n_req) -> int:
    return int(load().rk_draft_verify_workspace_size(prob_dtype, vocab, n_req))


def rk_draft_verify(prob_dtype, token_dtype, p, p_stride, q, q_stride, vocab, n_req, n_draft, max_draft, starts,
                    drafted, u, r, tokens, accepted, workspace, workspace_bytes, stream) -> int:
    return load().rk_draft_verify(prob_dtype, token_dtype, p, p_stride, q, q_stride, vocab, n_req, n_draft,
                                  max_draft, starts, drafted, u, r, tokens, accepted, workspace, workspace_bytes,
                                  stream)


def rk_block_tables_workspace_size(n_req) -> int:
    return int(load().rk_block_tables_workspace_size(n_req))


def rk_block_tables(lens, n_req, block_size, held, held_out, table, table_stride, max_blocks, ring, ring_size,
                    state, state_out, workspace, workspace_bytes, stream) -> int:
    return load().rk_block_tables(lens, n_req, block_size, held, held_out, table, table_stride, max_blocks, ring,
                                  ring_size, state, state_out, workspace, workspace_bytes, stream)


def rk_slot_map(lens, fresh, n_req, block_size, table, table_stride, max_blocks, held, n_blocks, slot_dtype,
                capacity, slots, positions, requests, starts, stream) -> int:
    return load().rk_slot_map(lens, fresh, n_req, block_size, table, table_stride, max_blocks, held, n_blocks,
                              slot_dtype, capacity, slots, positions, requests, starts, stream)


def rk_beam_select_workspace_size(dtype, vocab, n_req, beams, count) -> int:
    return int(load().rk_beam_select_workspace_size(dtype, vocab, n_req, beams, count))


def rk_beam_select(dtype, token_dtype, logits, stride, vocab, n_req, beams, scores, ended, end_token, count, best, tokens,
                   parents, workspace, workspace_bytes, stream) -> int:
    return load().rk_beam_select(dtype, token_dtype, logits, stride, vocab, n_req, beams, scores, ended, end_token, count, best,
                                 tokens, parents, workspace, workspace_bytes, stream)


def rk_fork_blocks_workspace_size(n_rows, n_out, max_blocks, n_blocks) -> int:
    return int(load().rk_fork_blocks_workspace_size(n_rows, n_out, max_blocks, n_blocks))


def rk_fork_blocks(parents, n_out, lens, n_rows, block_size, held, table, table_stride, max_blocks, ring, ring_size, state,
                   n_blocks, table_out, table_out_stride, held_out, lens_out, pairs, state_out, workspace, workspace_bytes,
                   stream) -> int:
    return load().rk_fork_blocks(parents, n_out, lens, n_rows, block_size, held, table, table_stride, max_blocks, ring,
                                 ring_size, state, n_blocks, table_out, table_out_stride, held_out, lens_out, pairs, state_out,
                                 workspace, workspace_bytes, stream)


def rk_compact_blocks_workspace_size(n_blocks) -> int:
    return int(load().rk_compact_blocks_workspace_size(n_blocks))


def rk_compact_blocks(held, n_rows, table, table_stride, max_blocks, n_blocks, table_out, table_out_stride, ring, ring_size,
                      pairs, max_pairs, state_out, workspace, workspace_bytes, stream) -> int:
    return load().rk_compact_blocks(held, n_rows, table, table_stride, max_blocks, n_blocks, table_out, table_out_stride, ring,
                                    ring_size, pairs, max_pairs, state_out, workspace, workspace_bytes, stream)


def rk_copy_blocks(caches, pairs, n_pairs, stream) -> int:
    """caches: (address, block_stride, block_bytes, n_blocks) each."""
    at = (rk_block_cache * max(len(caches), 1))(*(rk_block_cache(*c) for c in caches))
    return load().rk_copy_blocks(at, len(caches), pairs, n_pairs, stream)


def rk_linear_recurrence_workspace_size(x_dtype, gate_dtype, n_seq, tokens, channels, packed) -> int:
    return int(load().rk_linear_recurrence_workspace_size(x_dtype, gate_dtype, n_seq, tokens, channels, packed))


def _rows(r):
    return None if r is None else ctypes.byref(rk_rows(*r))


def rk_linear_recurrence(x_dtype, gate_dtype, kind, blend, gate, x, state, n_states, sources, starts, n_seq, tokens,
                         channels, out, state_out, workspace, workspace_bytes, stream) -> int:
    """gate, x, out: (address, seq_stride, token_stride) or None."""
    return load().rk_linear_recurrence(x_dtype, gate_dtype, kind, blend, _rows(gate), _rows(x), state, n_states, sources,
                                       starts, n_seq, tokens, channels, _rows(out), state_out, workspace, workspace_bytes,
                                       stream)


def rk_linear_recurrence_backward(x_dtype, gate_dtype, kind, blend, gate, x, out, dout, state, dstate_out, starts, n_seq,
                                  tokens, channels, dgate, dx, dstate, workspace, workspace_bytes, stream) -> int:
    """gate, x, out, dout, dgate, dx: (address, seq_stride, token_stride) or None."""
    return load().rk_linear_recurrence_backward(x_dtype, gate_dtype, kind, blend, _rows(gate), _rows(x), _rows(out),
                                                _rows(dout), state, dstate_out, starts, n_seq, tokens, channels,
                                                _rows(dgate), _rows(dx), dstate, workspace, workspace_bytes, stream)


def rk_plan_softmax(in_dtype, out_dtype, n, lines) -> rk_plan_info:
    info = rk_plan_info()
    rc = load().rk_plan_softmax(in_dtype, out_dtype, n, lines, ctypes.byref(info))
    if rc:
        raise RkError(rc, "rk_plan_softmax")
    return info


def rk_plan_draft_verify(prob_dtype, vocab, n_req, num_cus=0) -> rk_plan_info:
    info = rk_plan_info()
    rc = load().rk_plan_draft_verify(prob_dtype, vocab, n_req, num_cus, ctypes.byref(info))
    if rc:
        raise RkError(rc, "rk_plan_draft_verify")
    return info


def rk_debug_set_fused_finish(enable: int) -> int:
    return int(load().rk_debug_set_fused_finish(int(enable)))


def rk_debug_set_launch_events(begin, end) -> int:
    return int(load().rk_debug_set_launch_events(begin, end))


def rk_debug_set_finish_tag(stream, e: int) -> int:
    return int(load().rk_debug_set_finish_tag(stream, int(e)))


def rk_debug_stream_read(ptr, nbytes, grid, sink, stream) -> None:
    rc = load().rk_debug_stream_read(ptr, nbytes, grid, sink, stream)
    if rc:
        raise RkError(rc, "rk_debug_stream_read")


def rk_debug_device_info() -> dict:
    """The current device's compute units, memory clock (kHz) and memory bus
    width (bits)."""
    vals = [ctypes.c_int64() for _ in range(3)]
    rc = load().rk_debug_device_info(*(ctypes.byref(v) for v in vals))
    if rc:
        raise RkError(rc, "rk_debug_device_info")
    return dict(num_cus=vals[0].value, mem_clock_khz=vals[1].value, mem_bus_bits=vals[2].value)


def rk_stream_timeouts(stream) -> int:
    """Waits that gave up in calls on `stream` (a hipStream_t handle) since
    the last query; waits for the stream and clears the count."""
    n = ctypes.c_uint64()
    rc = load().rk_stream_timeouts(stream, ctypes.byref(n))
    if rc:
        raise RkError(rc, "rk_stream_timeouts")
    return int(n.value)


def rk_debug_force_wait_timeout(polls: int) -> int:
    return int(load().rk_debug_force_wait_timeout(int(polls)))


def rk_debug_fail_launches(count: int) -> int:
    return int(load().rk_debug_fail_launches(int(count)))
