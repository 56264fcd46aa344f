"""ctypes binding of the serving operators (include/pkv_serving.h): the 8-bit
cache, cross attention and page tables.  Argument marshalling only, as in
``_lib``, whose library and errors it shares."""
from __future__ import annotations

import ctypes

from ._context import _byref, token_stride
from ._lib import LIB, _check, _ptr, _stream, pkv_problem

EXPORTED = ("pkv_kv8_page_bytes", "pkv_kv8_store", "pkv_kv8_load", "pkv_attend_kv8",
            "pkv_prompt_kv8", "pkv_prompt_kv8_workspace_bytes", "pkv_prompt_kv8_splits",
            "pkv_cross_workspace_bytes", "pkv_cross_splits", "pkv_cross",
            "pkv_cross_kv4", "pkv_cross_kv8", "pkv_pages_take", "pkv_pages_release")


def _prototypes() -> None:
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    prob = ctypes.POINTER(pkv_problem)
    for name, res, args in (
            ("pkv_kv8_page_bytes", sz, [i32]),
            ("pkv_kv8_store", i32, [prob, vp, i32, vp, vp, i64, vp, i64, vp, vp, vp, vp]),
            ("pkv_kv8_load", i32, [prob, vp, i32, vp, vp, vp, vp, vp, vp, vp]),
            ("pkv_attend_kv8", i32, [prob, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp, vp, vp]),
            ("pkv_prompt_kv8", i32,
             [prob, vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp, vp, vp]),
            ("pkv_prompt_kv8_workspace_bytes", sz, [prob, i32, i32, i32]),
            ("pkv_prompt_kv8_splits", i32, [prob, vp, i32, i32, i32]),
            ("pkv_cross_workspace_bytes", sz, [prob, i32, i32, i32]),
            ("pkv_cross_splits", i32, [prob, i32, i32, i32]),
            ("pkv_cross", i32, [prob, vp, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp, vp, vp]),
            ("pkv_cross_kv4", i32, [prob, vp, i32, vp, i32, vp, vp, vp, vp, sz, vp, vp, vp]),
            ("pkv_cross_kv8", i32, [prob, vp, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp, vp, vp]),
            ("pkv_pages_take", i32, [prob, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            ("pkv_pages_release", i32, [prob, vp, vp, vp, vp, vp, vp])):
        # A host-only build named by PKV_LIBRARY may hold fewer operators; a call of
        # a missing entry point then fails by its name.
        if hasattr(LIB, name):
            fn = getattr(LIB, name)
            fn.restype, fn.argtypes = res, args


_prototypes()


def _workspace(ws) -> tuple:
    return _ptr(ws), 0 if ws is None else ws.numel()


def pkv_kv8_page_bytes(head_dim: int) -> int:
    return LIB.pkv_kv8_page_bytes(head_dim)


def pkv_kv8_store(prob, tok_offsets, num_tokens: int, seq_lens_dev, k_new, v_new, block_table,
                  kv8_pool, kv8_scales, stream=None) -> None:
    _check("pkv_kv8_store", LIB.pkv_kv8_store(
        ctypes.byref(prob), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev), k_new.data_ptr(),
        token_stride(k_new), v_new.data_ptr(), token_stride(v_new), _ptr(block_table),
        _ptr(kv8_pool), _ptr(kv8_scales), _stream(stream)))


def pkv_kv8_load(prob, tok_offsets, num_tokens: int, seq_lens_dev, block_table, kv8_pool,
                 kv8_scales, k_out, v_out, stream=None) -> None:
    _check("pkv_kv8_load", LIB.pkv_kv8_load(
        ctypes.byref(prob), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev), _ptr(block_table),
        _ptr(kv8_pool), _ptr(kv8_scales), _ptr(k_out), _ptr(v_out), _stream(stream)))


def pkv_attend_kv8(prob, view, seq_lens_dev, max_splits: int, q, kv8_pool, kv8_scales, block_table,
                   workspace, out, lse=None, stream=None) -> None:
    _check("pkv_attend_kv8", LIB.pkv_attend_kv8(
        ctypes.byref(prob), _byref(view), _ptr(seq_lens_dev), max_splits, _ptr(q), _ptr(kv8_pool),
        _ptr(kv8_scales), _ptr(block_table), *_workspace(workspace), _ptr(out), _ptr(lse),
        _stream(stream)))


def pkv_prompt_kv8(prob, view, tok_offsets, num_tokens: int, seq_lens_dev, max_splits: int, q,
                   kv8_pool, kv8_scales, block_table, workspace, out, lse=None,
                   stream=None) -> None:
    _check("pkv_prompt_kv8", LIB.pkv_prompt_kv8(
        ctypes.byref(prob), _byref(view), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev),
        max_splits, _ptr(q), _ptr(kv8_pool), _ptr(kv8_scales), _ptr(block_table),
        *_workspace(workspace), _ptr(out), _ptr(lse), _stream(stream)))


def pkv_prompt_kv8_workspace_bytes(prob, num_tokens: int, one_per_row: bool,
                                   max_splits: int) -> int:
    return LIB.pkv_prompt_kv8_workspace_bytes(ctypes.byref(prob), num_tokens, one_per_row,
                                              max_splits)


def pkv_prompt_kv8_splits(prob, view, num_tokens: int, one_per_row: bool, num_cus: int) -> int:
    return LIB.pkv_prompt_kv8_splits(ctypes.byref(prob), _byref(view), num_tokens, one_per_row,
                                     num_cus)


def pkv_cross_workspace_bytes(prob, num_tokens: int, one_per_row: bool, max_splits: int) -> int:
    return LIB.pkv_cross_workspace_bytes(ctypes.byref(prob), num_tokens, one_per_row, max_splits)


def pkv_cross_splits(prob, num_tokens: int, one_per_row: bool, num_cus: int) -> int:
    return LIB.pkv_cross_splits(ctypes.byref(prob), num_tokens, one_per_row, num_cus)


def pkv_cross(prob, tok_offsets, num_tokens: int, seq_lens_dev, max_splits: int, q, k_pool, v_pool,
              block_table, workspace, out, lse=None, stream=None) -> None:
    _check("pkv_cross", LIB.pkv_cross(
        ctypes.byref(prob), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev), max_splits, _ptr(q),
        _ptr(k_pool), _ptr(v_pool), _ptr(block_table), *_workspace(workspace), _ptr(out),
        _ptr(lse), _stream(stream)))


def pkv_cross_kv4(prob, tok_offsets, num_tokens: int, seq_lens_dev, max_splits: int, q, kv4_pool,
                  block_table, workspace, out, lse=None, stream=None) -> None:
    _check("pkv_cross_kv4", LIB.pkv_cross_kv4(
        ctypes.byref(prob), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev), max_splits, _ptr(q),
        _ptr(kv4_pool), _ptr(block_table), *_workspace(workspace), _ptr(out), _ptr(lse),
        _stream(stream)))


def pkv_cross_kv8(prob, tok_offsets, num_tokens: int, seq_lens_dev, max_splits: int, q, kv8_pool,
                  kv8_scales, block_table, workspace, out, lse=None, stream=None) -> None:
    _check("pkv_cross_kv8", LIB.pkv_cross_kv8(
        ctypes.byref(prob), _ptr(tok_offsets), num_tokens, _ptr(seq_lens_dev), max_splits, _ptr(q),
        _ptr(kv8_pool), _ptr(kv8_scales), _ptr(block_table), *_workspace(workspace), _ptr(out),
        _ptr(lse), _stream(stream)))


def pkv_pages_take(prob, counts, num_tokens: int, lens, block_table, free_pages, state, seq_lens,
                   tok_offsets, slots=None, positions=None, stream=None) -> None:
    _check("pkv_pages_take", LIB.pkv_pages_take(
        ctypes.byref(prob), _ptr(counts), num_tokens, _ptr(lens), _ptr(block_table),
        _ptr(free_pages), _ptr(state), _ptr(seq_lens), _ptr(tok_offsets), _ptr(slots),
        _ptr(positions), _stream(stream)))


def pkv_pages_release(prob, keep, lens, block_table, free_pages, state, stream=None) -> None:
    _check("pkv_pages_release", LIB.pkv_pages_release(
        ctypes.byref(prob), _ptr(keep), _ptr(lens), _ptr(block_table), _ptr(free_pages),
        _ptr(state), _stream(stream)))
