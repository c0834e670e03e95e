"""Binding of the rows around an expert stage (the C ABI in include/moe_rows.h): tokens sorted by expert
for any router's choice, the way back with gates applied, and the gradients of both.

Argument marshalling only, as in ``fp8``: outputs and workspaces are the caller's tensors, every call enqueues
its kernels on the current stream (or ``stream``) and returns, and a wrong type, shape, layout or device
raises ValueError before the library is called; the library's own checks raise ``moe.MoEError``.

T tokens, k slots a token (at most 64), E experts (at most 1024), R rows of the buffers.  ``idx`` [T, k]
(int32 or int64) holds each slot's expert; any value outside [0, E) is a slot without a row.  ``slot_pos``
[T, k] (int32) holds each slot's row; where it is read, a value outside [0, R) is a slot without a row.
"""
import ctypes

import torch

from .fp8 import _check, _declare, _fp8

_I32, _I64, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_workspace = _declare("moe_rows_workspace", _I64, _I32, _I32, restype=ctypes.c_size_t)
_declare("moe_rows_sort", _P, _I32, _I64, _I32, _I32, _P, _P, _P, _P, ctypes.c_size_t, _P)
_declare("moe_rows_gather", _P, _I64, _I32, _P, _I32, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _P, _P)
_declare("moe_rows_dispatch", _P, _I32, _I64, _I32, _I32, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _P, _P,
         ctypes.c_size_t, _P)
_declare("moe_rows_combine", _P, _I32, _I64, _P, _P, _I64, _I32, _I64, _P, _P, _I32, _P)
_declare("moe_rows_combine_backward", _P, _I32, _P, _P, _I64, _I32, _I64, _I64, _P, _P, _I32, _P, _P)


def dispatch_workspace(T, k, E, device="cuda"):
    """The workspace of sort and dispatch for T tokens of k slots over E experts."""
    return torch.empty(max(1, int(_workspace(int(T), int(k), int(E)))), dtype=torch.uint8, device=device)


def sort(idx, counts, slot_pos, row_slot=None, workspace=None, stream=None):
    """counts [E], slot_pos [T, k] and row_slot [T k] (all int32) of the choice idx: expert e's rows lie
    behind those of the experts before it, in slot order (moe_rows_sort).  row_slot is -1 behind the last row."""
    _check(_fp8.rows_sort(idx, counts, slot_pos, row_slot, workspace, stream), "moe_rows_sort")


def gather(slot_pos, x, x_rows, x_scales=None, row_scales=None, gates=None, row_gates=None, stream=None):
    """x_rows[slot_pos[t, j]] = x[t] for x [T, d] (fp32, bf16 or e4m3; any row pitch) and x_rows [R, d]; with
    them the block factors of e4m3 rows ([T, scale_cols(d)] to [R, scale_cols(d)]) and gates [T, k] to
    row_gates [R], fp32 (moe_rows_gather).  Rows that no slot names are left as they were.  Its gradient
    is combine without gates."""
    _check(_fp8.rows_gather(slot_pos, x, x_rows, x_scales, row_scales, gates, row_gates, stream), "moe_rows_gather")


def dispatch(idx, x, counts, slot_pos, x_rows, workspace=None, row_slot=None, x_scales=None, row_scales=None, gates=None,
             row_gates=None, stream=None):
    """sort and gather in one call (moe_rows_dispatch): what Fp8ExpertPlan.forward and moe.ExpertPlan.forward take
    as seg_counts, rows and gates."""
    _check(_fp8.rows_dispatch(idx, x, counts, slot_pos, x_rows, workspace, row_slot, x_scales, row_scales, gates, row_gates, stream),
           "moe_rows_dispatch")


def combine(y_rows, slot_pos, out, gates=None, residual=None, stream=None):
    """out[t] = residual[t] + sum_j gates[t, j] y_rows[slot_pos[t, j]] (moe_rows_combine): y_rows [R, d] and out
    [T, d] fp32 or bf16, residual in out's type (it may be out itself), gates fp32 or None for ones."""
    _check(_fp8.rows_combine(y_rows, slot_pos, out, gates, residual, stream), "moe_rows_combine")


def combine_backward(dout, slot_pos, gates, y_rows=None, dy_rows=None, dgates=None, stream=None):
    """combine's gradients from dout [T, d] (moe_rows_combine_backward): dy_rows[slot_pos[t, j]] = gates[t, j]
    dout[t] in y_rows' type (it may be y_rows itself), and dgates[t, j] = <dout[t], y_rows[slot_pos[t, j]]>
    (fp32; 0 for a slot without a row), for which y_rows is needed.  The residual's gradient is dout."""
    _check(_fp8.rows_combine_backward(dout, slot_pos, gates, y_rows, dy_rows, dgates, stream), "moe_rows_combine_backward")
