"""ctypes binding of the context operators (include/pkv_context.h): windowed
and prompt attention, and the 4-bit cache.  Argument marshalling only, as in
``_lib``, whose library and errors it shares."""
from __future__ import annotations

import ctypes

from ._lib import LIB, _check, _ptr, _stream, pkv_problem

EXPORTED = ("pkv_kv4_page_bytes", "pkv_store_kv", "pkv_kv4_store", "pkv_kv4_load",
            "pkv_attend_workspace_bytes", "pkv_attend_window", "pkv_attend_kv4",
            "pkv_attend_splits", "pkv_prompt_workspace_bytes", "pkv_prompt_splits",
            "pkv_prompt_window", "pkv_prompt_kv4")


class pkv_view(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("sinks", ctypes.c_int32)]


def _prototypes() -> None:
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    prob, view = ctypes.POINTER(pkv_problem), ctypes.POINTER(pkv_view)
    for name, res, args in (
            ("pkv_kv4_page_bytes", sz, [i32]),
            ("pkv_store_kv", i32, [prob, vp, i32, vp, vp, i64, vp, i64, vp, vp, vp, vp]),
            ("pkv_kv4_store", i32, [prob, vp, i32, vp, vp, i64, vp, i64, vp, vp, vp]),
            ("pkv_kv4_load", i32, [prob, vp, i32, vp, vp, vp, vp, vp, vp]),
            ("pkv_attend_workspace_bytes", sz, [prob, i32]),
            ("pkv_attend_window", i32, [prob, view, vp, i32, vp, vp, vp, vp, vp, sz, vp, vp, vp]),
            ("pkv_attend_kv4", i32, [prob, view, vp, i32, vp, vp, vp, vp, sz, vp, vp, vp]),
            ("pkv_attend_splits", i32, [prob, view, i32]),
            ("pkv_prompt_workspace_bytes", sz, [prob, i32, i32, i32]),
            ("pkv_prompt_splits", i32, [prob, view, i32, i32, i32]),
            ("pkv_prompt_window", i32,
             [prob, view, vp, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp, vp, vp]),
            ("pkv_prompt_kv4", i32,
             [prob, view, vp, i32, vp, i32, vp, vp, vp, vp, sz, vp, vp, vp])):
        # A host-only build named by PKV_LIBRARY may hold the decode engine
        # alone; a call of a missing entry point then fails by its name.
        if hasattr(LIB, name):
            fn = getattr(LIB, name)
            fn.restype, fn.argtypes = res, args


_prototypes()


def make_view(window: int = 0, sinks: int = 0) -> pkv_view:
    return pkv_view(window, sinks)


def _byref(view):
    return None if view is None else ctypes.byref(view)


def pkv_kv4_page_bytes(head_dim: int) -> int:
    return LIB.pkv_kv4_page_bytes(head_dim)


def token_stride(x) -> int:
    """Elements between the tokens of [tokens][Hkv][d] with contiguous heads."""
    n, heads, d = x.shape
    token, head, one = x.stride()
    if one != 1 or (head != d and heads > 1):
        raise ValueError("new keys and values are [tokens][Hkv][d] with contiguous heads")
    # A single token's stride carries no meaning.
    return token if n > 1 else heads * d


def pkv_store_kv(prob, tok_offsets, num_tokens: int, seq_lens_dev, k_new, v_new, block_table,
                 k_pool, v_pool, stream=None) -> None:
    _check("pkv_store_kv", LIB.pkv_store_kv(
        ctypes.byref(prob), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev), k_new.data_ptr(),
        token_stride(k_new), v_new.data_ptr(), token_stride(v_new), _ptr(block_table),
        _ptr(k_pool), _ptr(v_pool), _stream(stream)))


def pkv_kv4_store(prob, tok_offsets, num_tokens: int, seq_lens_dev, k_new, v_new, block_table,
                  kv4_pool, stream=None) -> None:
    _check("pkv_kv4_store", LIB.pkv_kv4_store(
        ctypes.byref(prob), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev), k_new.data_ptr(),
        token_stride(k_new), v_new.data_ptr(), token_stride(v_new), _ptr(block_table),
        _ptr(kv4_pool), _stream(stream)))


def pkv_kv4_load(prob, tok_offsets, num_tokens: int, seq_lens_dev, block_table, kv4_pool, k_out,
                 v_out, stream=None) -> None:
    _check("pkv_kv4_load", LIB.pkv_kv4_load(
        ctypes.byref(prob), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev), _ptr(block_table),
        _ptr(kv4_pool), _ptr(k_out), _ptr(v_out), _stream(stream)))


def pkv_attend_workspace_bytes(prob, max_splits: int) -> int:
    return LIB.pkv_attend_workspace_bytes(ctypes.byref(prob), max_splits)


def pkv_attend_splits(prob, view, num_cus: int) -> int:
    return LIB.pkv_attend_splits(ctypes.byref(prob), _byref(view), num_cus)


def pkv_attend_window(prob, view, seq_lens_dev, max_splits: int, q, k_pool, v_pool, block_table,
                      workspace, out, lse=None, stream=None) -> None:
    _check("pkv_attend_window", LIB.pkv_attend_window(
        ctypes.byref(prob), _byref(view), _ptr(seq_lens_dev), max_splits, _ptr(q), _ptr(k_pool),
        _ptr(v_pool), _ptr(block_table), _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse),
        _stream(stream)))


def pkv_attend_kv4(prob, view, seq_lens_dev, max_splits: int, q, kv4_pool, block_table, workspace,
                   out, lse=None, stream=None) -> None:
    _check("pkv_attend_kv4", LIB.pkv_attend_kv4(
        ctypes.byref(prob), _byref(view), _ptr(seq_lens_dev), max_splits, _ptr(q), _ptr(kv4_pool),
        _ptr(block_table), _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse),
        _stream(stream)))


def pkv_prompt_workspace_bytes(prob, num_tokens: int, one_per_row: bool, max_splits: int) -> int:
    return LIB.pkv_prompt_workspace_bytes(ctypes.byref(prob), num_tokens, one_per_row, max_splits)


def pkv_prompt_splits(prob, view, num_tokens: int, one_per_row: bool, num_cus: int) -> int:
    return LIB.pkv_prompt_splits(ctypes.byref(prob), _byref(view), num_tokens, one_per_row,
                                 num_cus)


def pkv_prompt_window(prob, view, tok_offsets, num_tokens: int, seq_lens_dev, max_splits: int, q,
                      k_pool, v_pool, block_table, workspace, out, lse=None, stream=None) -> None:
    _check("pkv_prompt_window", LIB.pkv_prompt_window(
        ctypes.byref(prob), _byref(view), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev),
        max_splits, _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), _ptr(workspace),
        0 if workspace is None else workspace.numel(), _ptr(out), _ptr(lse), _stream(stream)))


def pkv_prompt_kv4(prob, view, tok_offsets, num_tokens: int, seq_lens_dev, max_splits: int, q,
                   kv4_pool, block_table, workspace, out, lse=None, stream=None) -> None:
    _check("pkv_prompt_kv4", LIB.pkv_prompt_kv4(
        ctypes.byref(prob), _byref(view), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev),
        max_splits, _ptr(q), _ptr(kv4_pool), _ptr(block_table), _ptr(workspace),
        0 if workspace is None else workspace.numel(), _ptr(out), _ptr(lse), _stream(stream)))
