"""ctypes binding of the C ABI declared in ``include/pkv.h``.

Argument marshalling only: host arrays become int32 numpy buffers, device
buffers are torch tensors passed by pointer, streams are torch streams.  Every
step of the path runs in the CUDA library; there is no Python or CPU fallback.
If ``libpkv.so`` has not been built, every entry point raises.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libpkv.so")

MAX_GROUPS = 8
MAX_BATCH = 16384
STATIC_MAX_BATCH = 4096
ADVANCE = 1
LIVE_TABLES = 2
SCHEDULE_SETTLED = 4

OK = 0
ERR_INVALID_ARG = -1
ERR_FULL = -2
ERR_NOT_ACTIVE = -3
ERR_CAPACITY = -4
ERR_ALIGN = -5
ERR_CUDA = -6
ERR_DEVICE = -7

DEVERR_ROW = 1
DEVERR_COUNT = 2
DEVERR_POSITION = 4
DEVERR_BLOCK = 8
DEVERR_SLOT = 16
DEVERR_TIMEOUT = 32
DEVERR_TABLE_FULL = 64
DEVERR_OUTPUT_FULL = 128
DEVERR_DUP = 256

_NAMES = {OK: "PKV_OK", ERR_INVALID_ARG: "PKV_ERR_INVALID_ARG", ERR_FULL: "PKV_ERR_FULL",
          ERR_NOT_ACTIVE: "PKV_ERR_NOT_ACTIVE", ERR_CAPACITY: "PKV_ERR_CAPACITY",
          ERR_ALIGN: "PKV_ERR_ALIGN", ERR_CUDA: "PKV_ERR_CUDA", ERR_DEVICE: "PKV_ERR_DEVICE"}

# Every symbol the header declares.
EXPORTS = [
    "pkv_state_create", "pkv_state_destroy", "pkv_add_request", "pkv_update_request",
    "pkv_remove_request", "pkv_prepare_batch", "pkv_prepare_batch_device",
    "pkv_prepare_batch_static",
    "pkv_kv_cache_write", "pkv_kv_cache_write_layers", "pkv_kv_cache_write_step",
    "pkv_kv_indices", "pkv_apply_step", "pkv_block_keys", "pkv_prefix_cache_create", "pkv_prefix_cache_destroy",
    "pkv_prefix_cache_insert", "pkv_prefix_cache_match", "pkv_pool_reset", "pkv_pool_size",
    "pkv_pool_read", "pkv_allocate_slots", "pkv_release_blocks", "pkv_get_error",
    "pkv_state_error_word", "pkv_row_info", "pkv_read_row", "pkv_last_cuda_error",
    "pkv_version", "pkv_selftest_wait_timeout", "pkv_kv8_store", "pkv_kv8_attention_workspace",
    "pkv_kv8_attention", "pkv_kv8_evict", "pkv_rope_store", "pkv_kv4_store", "pkv_kv4_load",
    "pkv_kv4_attention_workspace", "pkv_kv4_attention", "pkv_verify_drafts",
]


class PkvError(RuntimeError):
    def __init__(self, code: int, call: str):
        extra = ""
        if code == ERR_CUDA and _LIB is not None:
            extra = f" (cudaError {_LIB.pkv_last_cuda_error()})"
        super().__init__(f"{call} failed: {_NAMES.get(code, code)}{extra}")
        self.code = code


class GroupSpec(C.Structure):
    _fields_ = [("block_size", C.c_int32), ("max_blocks_per_req", C.c_int32),
                ("num_blocks", C.c_int64)]


class BatchOut(C.Structure):
    _fields_ = [("index_mapping", C.c_void_p), ("query_start_loc", C.c_void_p),
                ("seq_lens", C.c_void_p), ("positions", C.c_void_p),
                ("input_ids", C.c_void_p), ("block_tables", C.c_void_p * MAX_GROUPS),
                ("slot_mapping", C.c_void_p * MAX_GROUPS)]


class StepDelta(C.Structure):
    _fields_ = [("num_finished", C.c_int32), ("finished_rows", C.c_void_p),
                ("num_new", C.c_int32), ("new_token_offsets", C.c_void_p),
                ("new_token_ids", C.c_void_p), ("new_num_computed", C.c_void_p),
                ("new_block_offsets", C.c_void_p * MAX_GROUPS),
                ("new_block_ids", C.c_void_p * MAX_GROUPS),
                ("num_cached", C.c_int32), ("cached_rows", C.c_void_p),
                ("cached_token_offsets", C.c_void_p), ("cached_token_ids", C.c_void_p),
                ("cached_num_computed", C.c_void_p),
                ("cached_block_offsets", C.c_void_p * MAX_GROUPS),
                ("cached_block_ids", C.c_void_p * MAX_GROUPS)]


class KvItem(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_cache", C.c_void_p),
                ("v_cache", C.c_void_p), ("slot_mapping", C.c_void_p), ("num_slots", C.c_int64)]


class Kv8CacheArgs(C.Structure):
    _fields_ = [("k_cache", C.c_void_p), ("v_cache", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("num_blocks", C.c_int64), ("block_size", C.c_int32),
                ("num_heads", C.c_int32), ("head_dim", C.c_int32)]


class Kv4CacheArgs(C.Structure):
    _fields_ = [("k_cache", C.c_void_p), ("v_cache", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("num_blocks", C.c_int64), ("block_size", C.c_int32),
                ("num_heads", C.c_int32), ("head_dim", C.c_int32), ("k_unit", C.c_float),
                ("v_unit", C.c_float)]


class RopeArgs(C.Structure):
    _fields_ = [("table", C.c_void_p), ("positions", C.c_void_p), ("pair_axes", C.c_char_p),
                ("axis_stride", C.c_int64), ("max_position", C.c_int32), ("rot_dim", C.c_int32),
                ("num_axes", C.c_int32), ("interleaved", C.c_int32)]


_P32 = C.POINTER(C.c_int32)
_VP = C.c_void_p
_LIB = None


def _declare(lib):
    i32, i64 = C.c_int32, C.c_int64
    sig = {
        "pkv_state_create": [C.POINTER(_VP), i32, i32, i32, C.POINTER(GroupSpec), i64, _VP],
        "pkv_state_destroy": [_VP],
        "pkv_add_request": [_VP, _P32, i32, i32, C.POINTER(_VP), _P32, _P32, _VP],
        "pkv_update_request": [_VP, i32, C.POINTER(_VP), _P32, _P32, i32, i32, _VP],
        "pkv_remove_request": [_VP, i32, _VP],
        "pkv_prepare_batch": [_VP, _P32, _P32, i32, i32, C.POINTER(BatchOut), _P32, _VP],
        "pkv_prepare_batch_device": [_VP, _VP, _VP, i32, i32, i32, C.POINTER(BatchOut), _VP],
        "pkv_prepare_batch_static": [_VP, _VP, i32, i32, i32, C.POINTER(GroupSpec),
                                     C.POINTER(_VP), _P32, _P32, i32, C.POINTER(BatchOut),
                                     _VP, _P32, _VP],
        "pkv_kv_cache_write": [_VP, _VP, i64, i64, _VP, _VP, i64, i32, _VP, i32, _VP, _VP],
        "pkv_kv_cache_write_layers": [i32, C.POINTER(_VP), C.POINTER(_VP), i64, i64,
                                      C.POINTER(_VP), C.POINTER(_VP), i64, i32, _VP, i32,
                                      _VP, _VP],
        "pkv_kv_cache_write_step": [i32, C.POINTER(KvItem), i64, i64, i32, i32, _VP, _VP],
        "pkv_apply_step": [_VP, C.POINTER(StepDelta), _P32, _VP],
        "pkv_kv_indices": [_VP, i32, _VP, _VP, i32, _VP, _VP, i64, _VP, _VP],
        "pkv_block_keys": [_VP, _P32, i32, i32, _P32, _VP, i64, _VP],
        "pkv_prefix_cache_create": [C.POINTER(_VP), i64, _VP],
        "pkv_prefix_cache_destroy": [_VP],
        "pkv_prefix_cache_insert": [_VP, _VP, _VP, i64, _VP, _VP],
        "pkv_prefix_cache_match": [_VP, _VP, _VP, _VP, i32, _VP, _VP, _VP],
        "pkv_pool_reset": [_VP, i32, _P32, i32, _VP],
        "pkv_pool_size": [_VP, i32, _P32],
        "pkv_pool_read": [_VP, i32, _P32, i32, _VP],
        "pkv_allocate_slots": [_VP, _P32, _P32, _P32, i32, _P32, i32, _P32, _P32, _VP],
        "pkv_release_blocks": [_VP, _P32, i32, _VP],
        "pkv_get_error": [_VP, _P32],
        "pkv_state_error_word": [_VP, C.POINTER(_VP)],
        "pkv_row_info": [_VP, i32, _P32, _P32, _P32, _P32],
        "pkv_read_row": [_VP, i32, _P32, _P32, i32, C.POINTER(_P32), _VP],
        "pkv_last_cuda_error": [],
        "pkv_version": [],
        "pkv_selftest_wait_timeout": [_VP, C.c_uint32, _VP],
        "pkv_kv8_store": [C.POINTER(Kv8CacheArgs), _VP, _VP, i64, i64, i32, _VP, i32, _VP, _VP],
        "pkv_kv8_attention_workspace": [i32, i32, i32, i32, C.POINTER(i64)],
        "pkv_kv8_attention": [C.POINTER(Kv8CacheArgs), _VP, i64, i32, i32, _VP, i32, _VP, _VP, i32,
                              i32, C.c_float, i32, _VP, i64, _VP, _VP, _VP, i64, _VP, _VP],
        "pkv_kv8_evict": [C.POINTER(Kv8CacheArgs), _VP, _VP, i32, _VP, i32, _VP, i32, i32, i32, i32,
                          _VP, _VP, _VP, _VP],
        "pkv_rope_store": [C.POINTER(RopeArgs), _VP, _VP, i64, i64, i32, i32, i32, _VP, i64, i32, _VP, i64,
                           _VP, _VP, i64, _VP, i32, _VP, _VP],
        "pkv_kv4_store": [C.POINTER(Kv4CacheArgs), C.POINTER(RopeArgs), _VP, _VP, i64, i64, i32, _VP, i64,
                          i32, _VP, i64, _VP, i32, _VP, _VP],
        "pkv_kv4_load": [C.POINTER(Kv4CacheArgs), _VP, i32, i32, _VP, _VP, _VP, _VP],
        "pkv_kv4_attention_workspace": [i32, C.POINTER(i64)],
        "pkv_kv4_attention": [C.POINTER(Kv4CacheArgs), _VP, i64, i32, i32, _VP, i32, _VP, _VP, i32, i32,
                              C.c_float, i32, _VP, i64, _VP, _VP, i64, _VP, _VP],
        "pkv_verify_drafts": [_VP, i64, _VP, i64, i32, i32, i32, _VP, _VP, i32, _VP, i32, _VP, _VP, _VP, _VP],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = C.c_int
    return lib


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIBRARY):
            raise RuntimeError(
                "paged_kv_prep_gb300: the CUDA library libpkv.so is not built "
                "(run paged_kv_prep_gb300.build.build() or __graft_entry__.build()); "
                "there is no fallback path")
        _LIB = _declare(C.CDLL(LIBRARY))
    return _LIB


def _check(rc, call):
    if rc != OK:
        raise PkvError(rc, call)


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _i32(a):
    return np.ascontiguousarray(a, dtype=np.int32)


def _p32(a):
    return a.ctypes.data_as(_P32)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr() if t.numel() else 0)


@dataclass
class Batch:
    """Device outputs of one prepare call (torch tensors)."""

    index_mapping: object
    query_start_loc: object
    seq_lens: object
    positions: object
    input_ids: object
    block_tables: list
    slot_mapping: list
    total_tokens: int

    def struct(self) -> BatchOut:
        o = BatchOut()
        o.index_mapping = self.index_mapping.data_ptr() if self.index_mapping.numel() else None
        o.query_start_loc = self.query_start_loc.data_ptr()
        o.seq_lens = self.seq_lens.data_ptr() if self.seq_lens.numel() else None
        o.positions = self.positions.data_ptr() if self.positions.numel() else None
        o.input_ids = self.input_ids.data_ptr() if self.input_ids.numel() else None
        for g, t in enumerate(self.block_tables):
            o.block_tables[g] = t.data_ptr() if t.numel() else None
        for g, t in enumerate(self.slot_mapping):
            o.slot_mapping[g] = t.data_ptr() if t.numel() else None
        return o


class State:
    """The worker's persistent request-state table on the current CUDA device
    (``pkv_state_create`` ... ``pkv_state_destroy``)."""

    def __init__(self, max_reqs, max_model_len, groups, ring_bytes=0, stream=None):
        """groups: sequence of (block_size, max_blocks_per_req, num_blocks)
        tuples, or objects with those attributes."""
        L = lib()
        specs = []
        for g in groups:
            if isinstance(g, (tuple, list)):
                specs.append(tuple(int(x) for x in g))
            else:
                specs.append((int(g.block_size), int(g.max_blocks_per_req), int(g.num_blocks)))
        self.G = len(specs)
        self.block_size = [s[0] for s in specs]
        self.W = [s[1] for s in specs]
        self.num_blocks = [s[2] for s in specs]
        self.max_reqs = int(max_reqs)
        self.max_model_len = int(max_model_len)
        arr = (GroupSpec * max(self.G, 1))(*[GroupSpec(*s) for s in specs])
        h = C.c_void_p()
        _check(L.pkv_state_create(C.byref(h), self.max_reqs, self.max_model_len, self.G, arr,
                                  int(ring_bytes), _stream(stream)), "pkv_state_create")
        self._h = h

    # -- lifecycle ----------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            _check(lib().pkv_state_destroy(self._h), "pkv_state_destroy")
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- request state ----------------------------------------------------------
    def _block_args(self, blocks):
        if blocks is None:
            blocks = [()] * self.G
        arrs = [_i32(b) for b in blocks]
        ptrs = (C.c_void_p * max(self.G, 1))(*[a.ctypes.data if a.size else None for a in arrs])
        counts = np.array([a.size for a in arrs], dtype=np.int32)
        return arrs, ptrs, counts

    def add_request(self, token_ids, num_computed, blocks, stream=None, check=True):
        tok = _i32(token_ids)
        arrs, ptrs, counts = self._block_args(blocks)
        row = C.c_int32(-1)
        rc = lib().pkv_add_request(self._h, _p32(tok) if tok.size else None, tok.size,
                                   int(num_computed), ptrs, _p32(counts), C.byref(row),
                                   _stream(stream))
        if check:
            _check(rc, "pkv_add_request")
            return row.value
        return row.value if rc == OK else rc

    def update_request(self, row, new_blocks=None, new_token_ids=(), num_computed=-1,
                       stream=None, check=True):
        tok = _i32(new_token_ids)
        arrs, ptrs, counts = self._block_args(new_blocks)
        rc = lib().pkv_update_request(self._h, int(row), ptrs, _p32(counts),
                                      _p32(tok) if tok.size else None, tok.size,
                                      int(num_computed), _stream(stream))
        if check:
            _check(rc, "pkv_update_request")
        return rc

    def remove_request(self, row, stream=None, check=True):
        rc = lib().pkv_remove_request(self._h, int(row), _stream(stream))
        if check:
            _check(rc, "pkv_remove_request")
        return rc

    def apply_step(self, finished=(), new=(), cached=(), stream=None, check=True):
        """Apply one step's scheduler output (``pkv_apply_step``).

        finished: rows to free; new: (token_ids, num_computed, blocks per
        group) per new request; cached: (row, new_token_ids, num_computed or
        -1, new blocks per group) per cached request.  Returns the new rows."""

        def csr(lists):
            lists = [_i32(x) for x in lists]
            off = np.zeros(len(lists) + 1, np.int32)
            if lists:
                off[1:] = np.cumsum([x.size for x in lists])
            flat = np.concatenate(lists) if lists and off[-1] else np.zeros(0, np.int32)
            return off, flat

        nt_off, nt_ids = csr([x[0] for x in new])
        ct_off, ct_ids = csr([x[1] for x in cached])
        nb = [csr([x[2][g] for x in new]) for g in range(self.G)]
        cb = [csr([x[3][g] for x in cached]) for g in range(self.G)]
        out = self.apply_step_arrays(
            list(finished), nt_off, nt_ids, [x[1] for x in new],
            [b[0] for b in nb], [b[1] for b in nb],
            [x[0] for x in cached], ct_off, ct_ids, [x[2] for x in cached],
            [b[0] for b in cb], [b[1] for b in cb], stream=stream, check=check)
        return out.tolist() if isinstance(out, np.ndarray) else out

    def apply_step_arrays(self, finished_rows, new_token_offsets, new_token_ids,
                          new_num_computed, new_block_offsets, new_block_ids, cached_rows,
                          cached_token_offsets, cached_token_ids, cached_num_computed,
                          cached_block_offsets, cached_block_ids, stream=None, check=True):
        """``pkv_apply_step`` from a scheduler output already packed as int32
        arrays: offsets are CSR ([count + 1], starting at 0) into the flat
        token / block id arrays, block arrays are one per KV-cache group.
        Returns the new requests' rows (int32 numpy array)."""
        keep = []

        def arr(a):
            a = _i32(a)
            keep.append(a)
            return a.ctypes.data if a.size else None

        d = StepDelta()
        fin = _i32(finished_rows)
        d.num_finished = int(fin.size)
        d.finished_rows = arr(fin)
        nnc = _i32(new_num_computed)
        d.num_new = int(nnc.size)
        d.new_token_offsets = arr(new_token_offsets)
        d.new_token_ids = arr(new_token_ids)
        d.new_num_computed = arr(nnc)
        cr = _i32(cached_rows)
        d.num_cached = int(cr.size)
        d.cached_rows = arr(cr)
        d.cached_token_offsets = arr(cached_token_offsets)
        d.cached_token_ids = arr(cached_token_ids)
        d.cached_num_computed = arr(cached_num_computed)
        for g in range(self.G):
            d.new_block_offsets[g] = arr(new_block_offsets[g])
            d.new_block_ids[g] = arr(new_block_ids[g])
            d.cached_block_offsets[g] = arr(cached_block_offsets[g])
            d.cached_block_ids[g] = arr(cached_block_ids[g])
        out = np.zeros(max(d.num_new, 1), np.int32)
        rc = lib().pkv_apply_step(self._h, C.byref(d), _p32(out), _stream(stream))
        if check:
            _check(rc, "pkv_apply_step")
            return out[:d.num_new]
        return rc if rc != OK else out[:d.num_new]

    def block_keys(self, rows, block_size, stream=None):
        """Prefix-cache keys of the full blocks of rows' known tokens
        (``pkv_block_keys``): (host int32 offsets [n+1], device int64 keys,
        the uint64 keys' bits)."""
        import torch

        r = _i32(rows)
        n = int(r.size)
        off = np.zeros(n + 1, np.int32)
        _check(lib().pkv_block_keys(self._h, _p32(r) if n else None, n, int(block_size),
                                    _p32(off), None, 0, _stream(stream)), "pkv_block_keys")
        keys = torch.empty(max(int(off[-1]), 1), dtype=torch.int64, device="cuda")
        _check(lib().pkv_block_keys(self._h, _p32(r) if n else None, n, int(block_size),
                                    _p32(off), C.c_void_p(keys.data_ptr()), int(keys.numel()),
                                    _stream(stream)), "pkv_block_keys")
        return off, keys[: int(off[-1])]

    def block_keys_into(self, rows, block_size, offsets, keys, stream=None):
        """``pkv_block_keys`` into preallocated outputs: rows and offsets
        (int32 numpy, n and n + 1), keys (int64 device tensor)."""
        _check(lib().pkv_block_keys(self._h, _p32(rows), int(rows.size), int(block_size),
                                    _p32(offsets), C.c_void_p(keys.data_ptr()),
                                    int(keys.numel()), _stream_handle(stream)), "pkv_block_keys")

    # -- free-block pools and allocate_slots ---------------------------------
    def pool_reset(self, group, free_ids, stream=None):
        ids = _i32(free_ids)
        _check(lib().pkv_pool_reset(self._h, int(group), _p32(ids) if ids.size else None,
                                    int(ids.size), _stream(stream)), "pkv_pool_reset")

    def pool_size(self, group):
        c = C.c_int32()
        _check(lib().pkv_pool_size(self._h, int(group), C.byref(c)), "pkv_pool_size")
        return c.value

    def pool(self, group, stream=None):
        n = self.pool_size(group)
        out = np.zeros(max(n, 1), np.int32)
        _check(lib().pkv_pool_read(self._h, int(group), _p32(out), n, _stream(stream)),
               "pkv_pool_read")
        return out[:n]

    def allocate_slots(self, rows, num_new, lookahead=None, windows=None, watermark=0,
                       stream=None, check=True):
        """Returns (admitted count, new blocks [n][G])."""
        r = _i32(rows)
        nn = _i32(num_new)
        n = int(r.size)
        la = None if lookahead is None else _i32(lookahead)
        win = None if windows is None else _i32(windows)
        adm = C.c_int32(0)
        nb = np.zeros(max(n * self.G, 1), np.int32)
        rc = lib().pkv_allocate_slots(self._h, _p32(r) if n else None, _p32(nn) if n else None,
                                      _p32(la) if la is not None and n else None, n,
                                      _p32(win) if win is not None else None, int(watermark),
                                      C.byref(adm), _p32(nb), _stream(stream))
        if rc != OK:
            if check:
                raise PkvError(rc, "pkv_allocate_slots")
            return rc
        return adm.value, nb[:n * self.G].reshape(n, self.G)

    def release_blocks(self, rows, stream=None):
        r = _i32(rows)
        _check(lib().pkv_release_blocks(self._h, _p32(r) if r.size else None, int(r.size),
                                        _stream(stream)), "pkv_release_blocks")

    def row_info(self, row):
        a, c, n = C.c_int32(), C.c_int32(), C.c_int32()
        nb = np.zeros(self.G, np.int32)
        _check(lib().pkv_row_info(self._h, int(row), C.byref(a), C.byref(c), C.byref(n),
                                  _p32(nb)), "pkv_row_info")
        return dict(active=bool(a.value), completed=c.value, n_tokens=n.value, num_blocks=nb)

    def read_row(self, row, n_tokens=None, stream=None):
        info = self.row_info(row)
        nt = info["n_tokens"] if n_tokens is None else int(n_tokens)
        tok = np.zeros(max(nt, 1), np.int32)
        tabs = [np.zeros(w, np.int32) for w in self.W]
        tptr = (_P32 * max(self.G, 1))(*[_p32(t) for t in tabs])
        comp = C.c_int32()
        _check(lib().pkv_read_row(self._h, int(row), C.byref(comp), _p32(tok), nt, tptr,
                                  _stream(stream)), "pkv_read_row")
        return dict(completed=comp.value, tokens=tok[:nt], block_table=tabs)

    # -- batch -----------------------------------------------------------------
    def alloc_batch(self, n, total_tokens, device="cuda"):
        import torch

        i32 = dict(dtype=torch.int32, device=device)
        return Batch(
            index_mapping=torch.empty(n, **i32),
            query_start_loc=torch.empty(n + 1, **i32),
            seq_lens=torch.empty(n, **i32),
            positions=torch.empty(total_tokens, **i32),
            input_ids=torch.empty(total_tokens, **i32),
            block_tables=[torch.empty(n, w, **i32) for w in self.W],
            slot_mapping=[torch.empty(total_tokens, dtype=torch.int64, device=device)
                          for _ in self.W],
            total_tokens=int(total_tokens))

    def prepare_batch(self, rows, num_sched, flags=0, out=None, stream=None, check=True):
        """Build the step's batch from host arrays (``pkv_prepare_batch``).
        Returns a Batch of device tensors (allocated unless ``out`` is given)."""
        r = _i32(rows)
        ns = _i32(num_sched)
        n = int(r.size)
        if out is None:
            out = self.alloc_batch(n, int(ns.sum(dtype=np.int64)) if n else 0)
        st = out.struct()
        total = C.c_int32(0)
        rc = lib().pkv_prepare_batch(self._h, _p32(r) if n else None, _p32(ns) if n else None,
                                     n, int(flags), C.byref(st), C.byref(total), _stream(stream))
        if check:
            _check(rc, "pkv_prepare_batch")
        elif rc != OK:
            return rc
        out.total_tokens = total.value
        return out

    def prepare_batch_device(self, d_rows, d_num_sched, total_tokens, out=None, stream=None,
                             check=True, flags=0):
        """Build the step's batch from a schedule already in device memory
        (``pkv_prepare_batch_device``); d_rows / d_num_sched are int32 tensors."""
        n = int(d_rows.numel())
        if out is None:
            out = self.alloc_batch(n, int(total_tokens), device=d_rows.device)
        st = out.struct()
        rc = lib().pkv_prepare_batch_device(self._h, _ptr(d_rows), _ptr(d_num_sched), n,
                                            int(total_tokens), int(flags), C.byref(st),
                                            _stream(stream))
        if check:
            _check(rc, "pkv_prepare_batch_device")
            return out
        return out if rc == OK else rc

    def kv_indices(self, group, index_mapping, seq_lens, capacity=None, out=None,
                   last_page_len=True, stream=None, check=True):
        """Paged (CSR) block table of a prepared batch (``pkv_kv_indices``):
        returns (kv_indptr [n+1], kv_indices [capacity], last_page_len [n] or
        None) as device tensors; the live entries are kv_indices[:kv_indptr[n]].
        ``index_mapping`` / ``seq_lens`` are the batch's int32 device tensors;
        ``out`` may supply the three buffers."""
        import torch

        n = int(index_mapping.numel())
        if capacity is None:
            capacity = n * self.W[group]
        if out is None:
            dev = index_mapping.device
            out = (torch.empty(n + 1, dtype=torch.int32, device=dev),
                   torch.empty(max(int(capacity), 1), dtype=torch.int32, device=dev),
                   torch.empty(max(n, 1), dtype=torch.int32, device=dev)
                   if last_page_len else None)
        indptr, indices, last = out
        rc = lib().pkv_kv_indices(self._h, int(group), _ptr(index_mapping), _ptr(seq_lens), n,
                                  _ptr(indptr), _ptr(indices), int(capacity),
                                  _ptr(last) if last is not None else None, _stream(stream))
        if check:
            _check(rc, "pkv_kv_indices")
            return out
        return out if rc == OK else rc

    # -- errors ----------------------------------------------------------------
    def get_error(self) -> int:
        code = C.c_int32(0)
        _check(lib().pkv_get_error(self._h, C.byref(code)), "pkv_get_error")
        return code.value

    @property
    def error_word(self) -> int:
        p = C.c_void_p()
        _check(lib().pkv_state_error_word(self._h, C.byref(p)), "pkv_state_error_word")
        return p.value


def _line_args(k, k_cache):
    line = k_cache[0].numel() * k_cache.element_size() if k_cache.shape[0] else 0
    if k_cache.numel() and not k_cache.is_contiguous():
        raise ValueError("the cache must be contiguous")
    ks = k.stride(0) * k.element_size() if k.dim() >= 1 and k.shape[0] else line
    return line, ks


def kv_cache_write(k, v, k_cache, v_cache, slot_mapping, num_tokens=None, d_error=None,
                   stream=None, check=True):
    """Store each token's K and V line at its slot (``pkv_kv_cache_write``).
    k, v: device tensors whose first dim is the token (row stride allowed, each
    row's line contiguous); k_cache, v_cache: contiguous [num_slots, ...];
    slot_mapping: int64 device tensor."""
    T = int(slot_mapping.numel()) if num_tokens is None else int(num_tokens)
    line, ks = _line_args(k, k_cache)
    _, vs = _line_args(v, v_cache)
    rc = lib().pkv_kv_cache_write(_ptr(k), _ptr(v), ks, vs, _ptr(k_cache), _ptr(v_cache),
                                  int(k_cache.shape[0]), int(line), _ptr(slot_mapping), T,
                                  C.c_void_p(d_error) if d_error else None, _stream(stream))
    if check:
        _check(rc, "pkv_kv_cache_write")
    return rc


def kv_cache_write_layers(ks, vs, k_caches, v_caches, slot_mapping, num_tokens=None,
                          d_error=None, stream=None, check=True):
    """The KV store for several layers sharing one slot_mapping, in one launch
    (``pkv_kv_cache_write_layers``).  Lists of same-shaped tensors."""
    L = len(ks)
    T = int(slot_mapping.numel()) if num_tokens is None else int(num_tokens)
    line, kst = _line_args(ks[0], k_caches[0])
    _, vst = _line_args(vs[0], v_caches[0])
    arr = lambda ts: (C.c_void_p * max(L, 1))(*[t.data_ptr() for t in ts])  # noqa: E731
    rc = lib().pkv_kv_cache_write_layers(L, arr(ks), arr(vs), kst, vst, arr(k_caches),
                                         arr(v_caches), int(k_caches[0].shape[0]), int(line),
                                         _ptr(slot_mapping), T,
                                         C.c_void_p(d_error) if d_error else None,
                                         _stream(stream))
    if check:
        _check(rc, "pkv_kv_cache_write_layers")
    return rc


def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


class KvStoreCall:
    """``pkv_kv_cache_write_layers`` with its arguments marshalled once.

    For a step that repeats with the same buffers (the same K/V sources,
    caches and slot_mapping tensors every step), building the pointer arrays
    each call costs more host time than the kernel takes on a small batch;
    this object builds them once and each call only passes the stream."""

    def __init__(self, ks, vs, k_caches, v_caches, slot_mapping, num_tokens=None,
                 d_error=None):
        self._keep = (list(ks), list(vs), list(k_caches), list(v_caches), slot_mapping)
        L = len(ks)
        T = int(slot_mapping.numel()) if num_tokens is None else int(num_tokens)
        line, kst = _line_args(ks[0], k_caches[0])
        _, vst = _line_args(vs[0], v_caches[0])
        arr = lambda ts: (C.c_void_p * max(L, 1))(*[t.data_ptr() for t in ts])  # noqa: E731
        self._args = (L, arr(ks), arr(vs), kst, vst, arr(k_caches), arr(v_caches),
                      int(k_caches[0].shape[0]), int(line), _ptr(slot_mapping), T,
                      C.c_void_p(d_error) if d_error else None)
        self._fn = lib().pkv_kv_cache_write_layers

    def __call__(self, stream=None):
        rc = self._fn(*self._args, _stream_handle(stream))
        if rc != OK:
            raise PkvError(rc, "pkv_kv_cache_write_layers")


class PrepareDeviceCall:
    """``pkv_prepare_batch_device`` with its arguments marshalled once (the
    schedule tensors and the output Batch are reused every call)."""

    def __init__(self, state, d_rows, d_num_sched, total_tokens, out, flags=0):
        self._keep = (state, d_rows, d_num_sched, out)
        self._st = out.struct()
        self._args = (state._h, _ptr(d_rows), _ptr(d_num_sched), int(d_rows.numel()),
                      int(total_tokens), int(flags), C.byref(self._st))
        self._fn = lib().pkv_prepare_batch_device

    def __call__(self, stream=None):
        rc = self._fn(*self._args, _stream_handle(stream))
        if rc != OK:
            raise PkvError(rc, "pkv_prepare_batch_device")


class PrepareHostCall:
    """``pkv_prepare_batch`` (host schedule) with the state and the output
    Batch marshalled once; each call passes only the schedule.  For a worker
    that reuses one set of output buffers every step, this takes the per-call
    Python cost from building the output struct and two pointer objects down
    to two address reads."""

    def __init__(self, state, out, flags=0):
        self._keep = (state, out)
        self._st = out.struct()
        self._total = C.c_int32(0)
        _VPT = C.c_void_p
        proto = C.CFUNCTYPE(C.c_int, _VPT, _VPT, _VPT, C.c_int32, C.c_int32, _VPT, _VPT, _VPT)
        self._fn = proto(("pkv_prepare_batch", lib()))
        self._h = state._h.value if isinstance(state._h, C.c_void_p) else state._h
        self._flags = int(flags)
        self._out_addr = C.addressof(self._st)
        self._total_addr = C.addressof(self._total)
        self._out = out
        # the buffers' capacity: requests and scheduled tokens
        self._cap_n = min(int(out.index_mapping.numel()), int(out.query_start_loc.numel()) - 1)
        self._cap_t = int(out.positions.numel())
        self._last = [None, None]

    def _addr(self, a, which):
        # an int32 contiguous array's address, remembered for the same array
        # object (held here, so it can be neither freed nor resized)
        last = self._last[which]
        if last is not None and last[0] is a:
            return last[1]
        addr = a.ctypes.data
        self._last[which] = (a, addr)
        return addr

    def __call__(self, rows, num_sched, stream=None):
        """Valid while the state is open; the schedule must fit the buffers."""
        r = np.ascontiguousarray(rows, dtype=np.int32)
        ns = np.ascontiguousarray(num_sched, dtype=np.int32)
        n = r.size
        if ns.size != n:
            raise ValueError("rows and num_sched differ in length")
        total = sum(ns.tolist()) if n <= 64 else int(ns.sum(dtype=np.int64))
        if n > self._cap_n or total > self._cap_t:
            raise ValueError("the schedule does not fit the output buffers")
        rp = self._addr(r, 0) if n else None
        np_ = self._addr(ns, 1) if n else None
        rc = self._fn(self._h, rp, np_, n, self._flags, self._out_addr, self._total_addr,
                      _stream_handle(stream))
        if rc != OK:
            raise PkvError(rc, "pkv_prepare_batch")
        self._out.total_tokens = self._total.value
        return self._out


def selftest_wait_timeout(d_error, polls=1000, stream=None):
    """``pkv_selftest_wait_timeout``: a kernel wait that nothing completes
    gives up after ``polls`` polls and ORs PKV_DEVERR_TIMEOUT into d_error
    (an int32 device tensor)."""
    _check(lib().pkv_selftest_wait_timeout(C.c_void_p(d_error.data_ptr()), int(polls),
                                           _stream_handle(stream)), "pkv_selftest_wait_timeout")


def _step_items(items):
    """items: sequence of (k, v, k_cache, v_cache, slot_mapping) tensors."""
    arr = (KvItem * max(len(items), 1))()
    line = kst = vst = None
    for i, (k, v, kc, vc, sm) in enumerate(items):
        ln, ks = _line_args(k, kc)
        _, vs = _line_args(v, vc)
        if line is None:
            line, kst, vst = ln, ks, vs
        elif (ln, ks, vs) != (line, kst, vst):
            raise ValueError("all items of a step share line size and source strides")
        arr[i] = KvItem(k.data_ptr(), v.data_ptr(), kc.data_ptr(), vc.data_ptr(),
                        sm.data_ptr() if sm.numel() else None, int(kc.shape[0]))
    return arr, int(line or 16), int(kst or 16), int(vst or 16)


def kv_cache_write_step(items, num_tokens=None, d_error=None, stream=None, check=True):
    """The step's KV store for several (layer, group) items, each with its own
    slot_mapping and caches, in one launch (``pkv_kv_cache_write_step``)."""
    arr, line, kst, vst = _step_items(items)
    T = int(items[0][4].numel()) if num_tokens is None and items else int(num_tokens or 0)
    rc = lib().pkv_kv_cache_write_step(len(items), arr, kst, vst, line, T,
                                       C.c_void_p(d_error) if d_error else None,
                                       _stream_handle(stream))
    if check and rc != OK:
        raise PkvError(rc, "pkv_kv_cache_write_step")
    return rc


class KvStepCall:
    """``pkv_kv_cache_write_step`` with its arguments marshalled once."""

    def __init__(self, items, num_tokens=None, d_error=None):
        self._keep = [tuple(it) for it in items]
        self._arr, line, kst, vst = _step_items(items)
        T = int(items[0][4].numel()) if num_tokens is None else int(num_tokens)
        self._args = (len(items), self._arr, kst, vst, line, T,
                      C.c_void_p(d_error) if d_error else None)
        self._fn = lib().pkv_kv_cache_write_step

    def __call__(self, stream=None):
        rc = self._fn(*self._args, _stream_handle(stream))
        if rc != OK:
            raise PkvError(rc, "pkv_kv_cache_write_step")


class PrefixCache:
    """Device index of cached blocks, key -> block id (``pkv_prefix_cache_*``)."""

    def __init__(self, capacity, stream=None):
        h = C.c_void_p()
        _check(lib().pkv_prefix_cache_create(C.byref(h), int(capacity), _stream_handle(stream)),
               "pkv_prefix_cache_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            _check(lib().pkv_prefix_cache_destroy(self._h), "pkv_prefix_cache_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def insert(self, keys, block_ids, d_error=None, stream=None):
        """keys: int64 device tensor (uint64 bits); block_ids: int32 device tensor."""
        _check(lib().pkv_prefix_cache_insert(self._h, _ptr(keys), _ptr(block_ids),
                                             int(keys.numel()),
                                             C.c_void_p(d_error) if d_error else None,
                                             _stream_handle(stream)), "pkv_prefix_cache_insert")

    def match_into(self, keys, offsets, max_hits, hits, ids, stream=None):
        """``pkv_prefix_cache_match`` into preallocated device tensors."""
        _check(lib().pkv_prefix_cache_match(self._h, _ptr(keys), _ptr(offsets), _ptr(max_hits),
                                            int(max_hits.numel()), _ptr(hits),
                                            C.c_void_p(ids.data_ptr()), _stream_handle(stream)),
               "pkv_prefix_cache_match")

    def match(self, keys, offsets, max_hits, stream=None):
        """Longest cached prefixes: offsets int32 [n+1], max_hits int32 [n]
        (device tensors). Returns (hit_blocks [n], hit_ids like keys)."""
        import torch

        n = int(max_hits.numel())
        hits = torch.empty(n, dtype=torch.int32, device=keys.device)
        ids = torch.empty(max(int(keys.numel()), 1), dtype=torch.int32, device=keys.device)
        _check(lib().pkv_prefix_cache_match(self._h, _ptr(keys), _ptr(offsets), _ptr(max_hits),
                                            n, _ptr(hits), C.c_void_p(ids.data_ptr()),
                                            _stream_handle(stream)), "pkv_prefix_cache_match")
        return hits, ids[: int(keys.numel())]


# -- the cache held in 8 bits -------------------------------------------------

_KV8 = None          # torch's types by what they are here (set on first use: torch loads late)


def _kv8_types():
    global _KV8
    if _KV8 is None:
        import torch

        _KV8 = (torch, {torch.bfloat16: 0, torch.float16: 1}, torch.float32, torch.int32, torch.int64,
                getattr(torch._C, "_cuda_getCurrentRawStream", None),
                getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device))
    return _KV8


def _kv8_cache(k_cache, v_cache, k_scale, v_scale):
    """The C view of an 8-bit cache: lines [num_slots, heads * head_dim] of one byte per element
    and scales [num_blocks, heads]."""
    f32 = _kv8_types()[2]       # a call's first use: from here on _KV8 is set
    shape, scales = k_cache.shape, k_scale.shape
    if not (len(scales) == 2 and v_scale.shape == scales and v_cache.shape == shape and len(shape) >= 1):
        raise ValueError("k_cache and v_cache, k_scale and v_scale have the same shapes; scales are [num_blocks, heads]")
    blocks, heads = scales
    slots, size = shape[0], k_cache.numel()
    if not (blocks > 0 and heads > 0 and slots > 0 and slots % blocks == 0 and size % (slots * heads) == 0):
        raise ValueError("the caches hold num_blocks * block_size lines of heads * head_dim bytes")
    if not (k_cache.itemsize == 1 and v_cache.itemsize == 1 and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("the caches are contiguous, one byte an element")
    if not (k_scale.dtype is f32 and v_scale.dtype is f32 and k_scale.is_contiguous() and v_scale.is_contiguous()):
        raise ValueError("the scales are contiguous float32")
    return Kv8CacheArgs(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                        blocks, slots // blocks, heads, size // (slots * heads))


def _kv8_int32(*tensors):
    i32 = _KV8[3]
    for t in tensors:
        if not (t.dtype is i32 and t.is_contiguous()):
            raise ValueError("tables, lengths and locations are contiguous int32")


def _kv8_rows(x, width, what):
    """Bytes between the tokens of x (two-byte elements): [tokens, width] or [tokens, heads,
    head_dim], each token's elements contiguous."""
    shape, stride = x.shape, x.stride()
    inner = 1
    for i in range(len(shape) - 1, 0, -1):
        if stride[i] != inner and shape[i] != 1:
            raise ValueError(f"{what}: a token's elements are contiguous")
        inner *= shape[i]
    if len(shape) < 2 or inner != width:
        raise ValueError(f"{what}: [tokens, heads, head_dim] of the cache's sizes")
    return stride[0] * 2 if shape[0] > 1 else width * 2


def _kv8_dtype(x):
    kind = _KV8[1].get(x.dtype)
    if kind is None:
        raise ValueError("bfloat16 or float16")
    return kind


def _kv8_size(x, what):
    """An integer argument as the library takes it; a larger one would be cut to its low 32 bits."""
    x = int(x)
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError(f"{what} is a 32-bit integer")
    return x


def _kv8_weights(weights, slots):
    if not (weights.dtype is _KV8[2] and weights.is_contiguous() and weights.numel() == slots):
        raise ValueError("weights is contiguous float32, one for each slot")


def _kv8_device(stream, *tensors):
    """The operands' device: one CUDA device, the stream's too (None: not given)."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("the tensors are on one device")
    if device < 0:
        raise ValueError("the tensors are on a CUDA device")
    if stream is not None and not isinstance(stream, int) and stream.device_index != device:
        raise ValueError("the stream is of the tensors' device")
    return device


def _kv8_elsewhere(device):
    """Whether another device than the operands' is the current one, by which the library launches."""
    return _KV8[6]() != device


def _kv8_stream(stream, device):
    """The stream's handle; without one the device's current stream (its raw handle where torch
    gives it: the stream object costs more than the rest of the marshalling)."""
    if stream is None:
        raw = _KV8[5]
        return raw(device) if raw is not None else _stream(None)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _kv8_make(shape, kind, device, stream, handle, returned=True):
    """A tensor that a call makes.  On another stream than the current one it is allocated there,
    behind the work that stream already has: a block of the current stream's pool may still be in use
    by the current stream's queue.  One that is returned is used, and freed, from the current stream."""
    torch = _KV8[0]
    if stream is None:
        return torch.empty(shape, dtype=kind, device=device)
    there = torch.cuda.ExternalStream(handle, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(there):
        made = torch.empty(shape, dtype=kind, device=device)
    if returned:
        made.record_stream(torch.cuda.current_stream(device))
    return made


def kv8_store(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, d_error=None, stream=None,
              check=True):
    """Quantise each token's K and V line into the 8-bit cache at its slot (``pkv_kv8_store``).

    k, v: bfloat16 or float16 [tokens, heads, head_dim] (or [tokens, heads * head_dim]), token
    stride allowed; k_cache, v_cache: one byte per element, [num_blocks * block_size, heads *
    head_dim]; k_scale, v_scale: float32 [num_blocks, heads]; slot_mapping: int64."""
    cache = _kv8_cache(k_cache, v_cache, k_scale, v_scale)
    T = slot_mapping.numel()
    if not (slot_mapping.dtype is _KV8[4] and slot_mapping.is_contiguous()):
        raise ValueError("slot_mapping is contiguous int64")
    if not (k.dtype is v.dtype and k.shape == v.shape and k.shape[0] >= T):
        raise ValueError("k and v have the same shape and type, a row for each slot")
    width = cache.num_heads * cache.head_dim
    k_stride, v_stride, kind = _kv8_rows(k, width, "k"), _kv8_rows(v, width, "v"), _kv8_dtype(k)
    device = _kv8_device(stream, k_cache, v_cache, k_scale, v_scale, k, v, slot_mapping)
    if _kv8_elsewhere(device):
        with _KV8[0].cuda.device(device):
            return kv8_store(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, d_error, stream, check)
    rc = lib().pkv_kv8_store(C.byref(cache), k.data_ptr(), v.data_ptr(), k_stride, v_stride, kind,
                             slot_mapping.data_ptr(), T, d_error or None, _kv8_stream(stream, device))
    if check and rc != OK:
        raise PkvError(rc, "pkv_kv8_store")
    return rc


def kv8_attention_workspace(num_tokens, num_q_heads, head_dim, with_weights=False):
    """Bytes of device workspace an attention call on the current device takes
    (``pkv_kv8_attention_workspace``)."""
    n = C.c_int64(0)
    rc = lib().pkv_kv8_attention_workspace(int(num_tokens), int(num_q_heads), int(head_dim),
                                           int(bool(with_weights)), C.byref(n))
    if rc != OK:
        raise PkvError(rc, "pkv_kv8_attention_workspace")
    return n.value


_KV8_WORKSPACE = {}      # bytes of calls without weights, which do not go by the number of tokens


def _kv8_workspace(device, num_tokens, num_q_heads, head_dim, with_weights):
    if with_weights:
        return kv8_attention_workspace(num_tokens, num_q_heads, head_dim, True)
    key = (device, num_q_heads, head_dim)        # by the device: its SMs
    found = _KV8_WORKSPACE.get(key)
    if found is None:
        found = _KV8_WORKSPACE[key] = kv8_attention_workspace(num_tokens, num_q_heads, head_dim)
    return found


def kv8_attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, query_start_loc, seq_lens,
                  softmax_scale=None, window=0, weights=None, out=None, lse=None, workspace=None,
                  d_error=None, stream=None, check=True):
    """Attention of a prepared batch's queries over the 8-bit cache (``pkv_kv8_attention``).

    q: bfloat16 or float16 [tokens, q_heads, head_dim], token stride allowed; block_tables [n, W],
    query_start_loc [n + 1] and seq_lens [n] as prepare_batch gives them.  window: a query sees
    that many positions, its own among them (0: all).  weights: float32 [num_slots], each token's
    softmax weight is added to it.  out, lse, workspace (uint8, kv8_attention_workspace bytes) are
    allocated when not given, on `stream` where one is.  Every tensor is on one CUDA device.  Returns
    (out, lse); lse is float32 [tokens, q_heads]."""
    cache = _kv8_cache(k_cache, v_cache, k_scale, v_scale)
    torch, _, f32 = _KV8[:3]
    _kv8_int32(block_tables, query_start_loc, seq_lens)
    n, table = seq_lens.numel(), block_tables.shape
    if not (len(table) == 2 and table[0] >= n and query_start_loc.numel() >= n + 1):
        raise ValueError("block_tables [n, W], query_start_loc [n + 1], seq_lens [n]")
    shape = q.shape
    if not (len(shape) == 3 and shape[2] == cache.head_dim):
        raise ValueError("q is [tokens, q_heads, head_dim]")
    T, hq, d = shape
    window = _kv8_size(window, "window")
    kind, q_stride = _kv8_dtype(q), _kv8_rows(q, hq * d, "q")
    if weights is not None:
        _kv8_weights(weights, k_cache.shape[0])
    if out is not None and not (out.shape == shape and out.dtype is q.dtype):
        raise ValueError("out has q's shape and type")
    out_stride = hq * d * 2 if out is None else _kv8_rows(out, hq * d, "out")
    if not (lse is None or lse.shape == (T, hq) and lse.dtype is f32 and lse.is_contiguous()):
        raise ValueError("lse is contiguous float32 [tokens, q_heads]")
    if not (workspace is None or workspace.is_contiguous()):
        raise ValueError("workspace is contiguous")
    device = _kv8_device(stream, k_cache, v_cache, k_scale, v_scale, q, block_tables, query_start_loc, seq_lens,
                         weights, out, lse, workspace)
    if _kv8_elsewhere(device):
        with torch.cuda.device(device):
            return kv8_attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, query_start_loc, seq_lens,
                                 softmax_scale, window, weights, out, lse, workspace, d_error, stream, check)
    handle = _kv8_stream(stream, device)
    if out is None:
        out = _kv8_make(shape, q.dtype, q.device, stream, handle)
    if lse is None:
        lse = _kv8_make((T, hq), f32, q.device, stream, handle)
    if workspace is None:
        size = _kv8_workspace(device, T, hq, d, weights is not None)
        workspace = _kv8_make(size, torch.uint8, q.device, stream, handle, returned=False)
    rc = lib().pkv_kv8_attention(C.byref(cache), q.data_ptr(), q_stride, kind, hq, block_tables.data_ptr(),
                                 table[1], query_start_loc.data_ptr(), seq_lens.data_ptr(), n, T,
                                 d ** -0.5 if softmax_scale is None else float(softmax_scale), window,
                                 out.data_ptr(), out_stride, lse.data_ptr(),
                                 None if weights is None else weights.data_ptr(), workspace.data_ptr(),
                                 workspace.numel() * workspace.itemsize, d_error or None, handle)
    if rc != OK:
        if check:
            raise PkvError(rc, "pkv_kv8_attention")
        return rc
    return out, lse


def kv8_evict(k_cache, v_cache, k_scale, v_scale, weights, block_tables, seq_lens,
              new_block_tables, budget, keep_first=0, keep_last=0, new_seq_lens=None, kept=None,
              d_error=None, stream=None, check=True):
    """Shrink requests to ``budget`` tokens by accumulated weight, into new blocks
    (``pkv_kv8_evict``).  Returns (new_seq_lens [n], kept [n, budget])."""
    cache = _kv8_cache(k_cache, v_cache, k_scale, v_scale)
    torch = _KV8[0]
    _kv8_int32(block_tables, new_block_tables, seq_lens)
    n, budget = seq_lens.numel(), _kv8_size(budget, "budget")
    keep_first, keep_last = _kv8_size(keep_first, "keep_first"), _kv8_size(keep_last, "keep_last")
    old, new = block_tables.shape, new_block_tables.shape
    if not (len(old) == 2 and len(new) == 2 and old[0] >= n and new[0] >= n):
        raise ValueError("block_tables and new_block_tables are [n, width]")
    _kv8_weights(weights, k_cache.shape[0])
    for t, size in ((new_seq_lens, n), (kept, n * max(budget, 0))):
        if t is not None:
            _kv8_int32(t)
            if t.numel() != size:
                raise ValueError("new_seq_lens [n], kept [n, budget]")
    device = _kv8_device(stream, k_cache, v_cache, k_scale, v_scale, weights, block_tables, seq_lens,
                         new_block_tables, new_seq_lens, kept)
    if _kv8_elsewhere(device):
        with torch.cuda.device(device):
            return kv8_evict(k_cache, v_cache, k_scale, v_scale, weights, block_tables, seq_lens, new_block_tables,
                             budget, keep_first, keep_last, new_seq_lens, kept, d_error, stream, check)
    handle = _kv8_stream(stream, device)
    if new_seq_lens is None:
        new_seq_lens = _kv8_make(n, torch.int32, seq_lens.device, stream, handle)
    if kept is None:
        kept = _kv8_make((n, max(budget, 0)), torch.int32, seq_lens.device, stream, handle)
    rc = lib().pkv_kv8_evict(C.byref(cache), weights.data_ptr(), block_tables.data_ptr(), old[1],
                             seq_lens.data_ptr(), n, new_block_tables.data_ptr(), new[1], budget,
                             keep_first, keep_last, new_seq_lens.data_ptr(), kept.data_ptr(), d_error or None,
                             handle)
    if rc != OK:
        if check:
            raise PkvError(rc, "pkv_kv8_evict")
        return rc
    return new_seq_lens, kept


# -- appending with the rotation by position ----------------------------------

_SHORT = None


def _short():
    """The calls from here on in C++ (csrc/pkv_marshal.cpp), with their operands in the common form.  They give
    NotImplemented, and have done nothing, for any other form; the functions below then check it.  Without
    _marshal.so they take every call, for 10 us and more of the host's time."""
    global _SHORT
    if _SHORT is None:
        import torch            # its libraries are there from here on

        from . import build

        try:
            if build.marshal_abi() != build.abi(torch.__version__):
                raise ImportError(f"built for {build.marshal_abi() or 'nothing that is known'}, not for {build.abi(torch.__version__)}")
            from . import _marshal
        except ImportError as e:
            import warnings

            warnings.warn("paged_kv_prep_gb300: _marshal.so is not built, or for another torch or Python; calls are marshalled in "
                          f"Python ({e}; paged_kv_prep_gb300.build.build() builds it)", RuntimeWarning, stacklevel=3)
            _marshal = _NoShort
        _SHORT = _marshal
    return _SHORT


class _NoShort:
    """In the place of _marshal.so: no call is of its common form."""
    rope_store = kv4_store = kv4_load = kv4_attention = verify_drafts = staticmethod(lambda *a: NotImplemented)


def _rope_args(positions, table, axes, interleaved, tokens):
    """The C view of a rotation, and what it points to."""
    f32, i32 = _KV8[2:4]
    shape, stride, rows = positions.shape, positions.stride(), table.shape
    if not (positions.dtype is i32 and len(shape) in (1, 2) and shape[-1] >= tokens):
        raise ValueError("positions is int32 [tokens] or [axes, tokens]")
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError("an axis's positions are contiguous")
    if not (table.dtype is f32 and len(rows) == 2 and table.is_contiguous()):
        raise ValueError("table is contiguous float32 [max_position, rot_dim]: cosines, then sines")
    count = shape[0] if len(shape) == 2 else 1
    if axes is not None:
        axes = bytes(axes)
        if len(axes) != rows[1] // 2:
            raise ValueError("axes has a row of positions for each of the rot_dim / 2 pairs")
    if rows[0] >= 1 << 31:
        raise ValueError("max_position is a 32-bit integer")
    return RopeArgs(table.data_ptr(), positions.data_ptr(), axes, stride[0] if count > 1 else 0,
                    rows[0], rows[1], count, 1 if interleaved else 0)


def _lines(x, shape, dim, what):
    """_kv8_rows of [tokens, heads, head_dim], the common case first."""
    stride = x.stride()
    if len(shape) == 3 and stride[2] == 1 and stride[1] == dim and shape[0] > 1:
        return stride[0] * 2
    return _kv8_rows(x, shape[1] * dim if len(shape) == 3 else shape[-1], what)


def _append_rows(k, v, q, q_out, slot_mapping, heads, dim):
    """Checks what a step appends; (tokens, type, strides of k, v, q and q_out in bytes, query heads)."""
    T, dtype, shape = slot_mapping.numel(), k.dtype, k.shape
    if not (slot_mapping.dtype is _KV8[4] and slot_mapping.is_contiguous()):
        raise ValueError("slot_mapping is contiguous int64")
    if not (dtype is v.dtype and shape == v.shape and shape[0] >= T):
        raise ValueError("k and v have the same shape and type, a row for each slot")
    kind = _KV8[1].get(dtype)
    if kind is None:
        raise ValueError("bfloat16 or float16")
    if not (len(shape) == 3 and shape[1] == heads and shape[2] == dim):
        _kv8_rows(k, heads * dim, "k")              # [tokens, heads * head_dim], or refused
    k_stride, v_stride = _lines(k, shape, dim, "k"), _lines(v, shape, dim, "v")
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        return T, kind, k_stride, v_stride, 0, 0, 0
    shape = q.shape
    if not (len(shape) == 3 and shape[2] == dim and shape[0] >= T and q.dtype is dtype):
        raise ValueError("q is [tokens, q_heads, head_dim] of k's type, a row for each slot")
    if q_out is None:
        return T, kind, k_stride, v_stride, _lines(q, shape, dim, "q"), shape[1] * dim * 2, shape[1]
    if not (q_out.shape == shape and q_out.dtype is dtype):
        raise ValueError("q_out has q's shape and type")
    return T, kind, k_stride, v_stride, _lines(q, shape, dim, "q"), _lines(q_out, shape, dim, "q_out"), shape[1]


def _make_like(x, stream, handle):
    """A contiguous tensor of x's shape and type that a call makes (see _kv8_make)."""
    if stream is None:
        torch = _KV8[0]
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return _kv8_make(x.shape, x.dtype, x.device, stream, handle)


def rope_store(k, v, k_cache, v_cache, slot_mapping, positions, table, axes=None, interleaved=False,
               q=None, q_out=None, d_error=None, stream=None, check=True):
    """Rotate a step's keys (and queries) by position and store K and V at their slots in a 16-bit
    paged cache (``pkv_rope_store``).

    k, v: bfloat16 or float16 [tokens, heads, head_dim], token stride allowed; k_cache, v_cache: the
    same type, contiguous [num_slots, heads, head_dim] (or [num_slots, heads * head_dim]);
    slot_mapping: int64, -1: not stored; positions: int32 [tokens] or [axes, tokens]; table: float32
    [max_position, rot_dim], cosines then sines; axes: the row of positions that each of the rot_dim /
    2 pairs goes by (None: the first); interleaved: pairs are neighbouring elements.  q: [tokens,
    q_heads, head_dim], rotated into q_out (may be q; allocated for the slots' tokens when not given).
    Returns q_out (None without q)."""
    made = (_SHORT or _short()).rope_store(k, v, k_cache, v_cache, slot_mapping, positions, table, axes, interleaved, q, q_out,
                                            d_error, stream, check)
    if made is not NotImplemented:
        return made
    torch = (_KV8 or _kv8_types())[0]
    if not (len(k.shape) == 3 and k_cache.shape == v_cache.shape and k_cache.dtype is k.dtype and
            v_cache.dtype is k.dtype and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k is [tokens, heads, head_dim], the caches contiguous and of its type")
    heads, dim = k.shape[1:]
    slots, size = k_cache.shape[0], k_cache.numel()
    if size != slots * heads * dim:
        raise ValueError("the caches hold num_slots lines of heads * head_dim elements")
    T, kind, ks, vs, qs, os_, hq = _append_rows(k, v, q, q_out, slot_mapping, heads, dim)
    rope = _rope_args(positions, table, axes, interleaved, T)
    device = _kv8_device(stream, k_cache, v_cache, k, v, slot_mapping, positions, table, q, q_out)
    if _kv8_elsewhere(device):
        with torch.cuda.device(device):
            return rope_store(k, v, k_cache, v_cache, slot_mapping, positions, table, axes, interleaved, q, q_out,
                              d_error, stream, check)
    handle = _kv8_stream(stream, device)
    if q is not None and q_out is None:
        q_out = _make_like(q if q.shape[0] == T else q[:T], stream, handle)
    rc = lib().pkv_rope_store(C.byref(rope), k.data_ptr(), v.data_ptr(), ks, vs, heads, dim, kind,
                              None if q is None else q.data_ptr(), qs, hq, None if q is None else q_out.data_ptr(), os_,
                              k_cache.data_ptr(), v_cache.data_ptr(), slots, slot_mapping.data_ptr(), T,
                              d_error or None, handle)
    if rc != OK:
        if check:
            raise PkvError(rc, "pkv_rope_store")
        return rc
    return q_out


# -- the cache held in 4 bits -------------------------------------------------


def _kv4_cache(k_cache, v_cache, k_scale, v_scale, k_unit, v_unit):
    """The C view of a 4-bit cache: codes [num_blocks, heads, block_size, head_dim / 2] and scales
    [num_blocks, heads, block_size, head_dim / 16], one byte an element."""
    if _KV8 is None:
        _kv8_types()            # a call's first use: from here on _KV8 is set
    shape, scales = k_cache.shape, k_scale.shape
    if not (len(shape) == 4 and v_cache.shape == shape and v_scale.shape == scales and len(scales) == 4):
        raise ValueError("the caches are [num_blocks, heads, block_size, head_dim / 2], the scales "
                         "[num_blocks, heads, block_size, head_dim / 16]")
    blocks, heads, size, half = shape
    if not (scales[0] == blocks and scales[1] == heads and scales[2] == size and 8 * scales[3] == half):
        raise ValueError("a scale for each 16 elements of each line")
    if not (k_cache.itemsize == 1 and v_cache.itemsize == 1 and k_scale.itemsize == 1 and v_scale.itemsize == 1 and
            k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous() and
            v_scale.is_contiguous()):
        raise ValueError("caches and scales are contiguous, one byte an element")
    return Kv4CacheArgs(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                        blocks, size, heads, 2 * half, k_unit, v_unit)


def kv4_store(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, positions=None, table=None, axes=None,
              interleaved=False, q=None, q_out=None, k_unit=1.0, v_unit=1.0, d_error=None, stream=None,
              check=True):
    """Quantise a step's K and V lines into the 4-bit cache, keys (and queries) rotated on the way
    (``pkv_kv4_store``; the rotation as in ``rope_store``, left out where positions and table are).

    k_cache, v_cache: one byte an element, [num_blocks, heads, block_size, head_dim / 2]; k_scale,
    v_scale: [num_blocks, heads, block_size, head_dim / 16] (uint8 or float8_e4m3fn); k_unit, v_unit:
    what all keys' and all values' scales are multiplied with.  Returns q_out (None without q)."""
    made = (_SHORT or _short()).kv4_store(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, positions, table, axes,
                                           interleaved, q, q_out, k_unit, v_unit, d_error, stream, check)
    if made is not NotImplemented:
        return made
    cache = _kv4_cache(k_cache, v_cache, k_scale, v_scale, k_unit, v_unit)
    heads, dim = k_cache.shape[1], 2 * k_cache.shape[3]
    T, kind, ks, vs, qs, os_, hq = _append_rows(k, v, q, q_out, slot_mapping, heads, dim)
    if (positions is None) != (table is None):
        raise ValueError("positions and table come together")
    if positions is None and (q is not None or axes is not None):
        raise ValueError("q and axes need positions and table")
    rope = None if positions is None else _rope_args(positions, table, axes, interleaved, T)
    device = _kv8_device(stream, k_cache, v_cache, k_scale, v_scale, k, v, slot_mapping, positions, table, q, q_out)
    if _kv8_elsewhere(device):
        with _KV8[0].cuda.device(device):
            return kv4_store(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, positions, table, axes,
                             interleaved, q, q_out, k_unit, v_unit, d_error, stream, check)
    handle = _kv8_stream(stream, device)
    if q is not None and q_out is None:
        q_out = _make_like(q if q.shape[0] == T else q[:T], stream, handle)
    rc = lib().pkv_kv4_store(C.byref(cache), None if rope is None else C.byref(rope), k.data_ptr(), v.data_ptr(),
                             ks, vs, kind, None if q is None else q.data_ptr(), qs, hq,
                             None if q is None else q_out.data_ptr(), os_, slot_mapping.data_ptr(), T,
                             d_error or None, handle)
    if rc != OK:
        if check:
            raise PkvError(rc, "pkv_kv4_store")
        return rc
    return q_out


def kv4_load(k_cache, v_cache, k_scale, v_scale, slots, dtype=None, k=None, v=None, k_unit=1.0, v_unit=1.0,
             d_error=None, stream=None, check=True):
    """Read the lines of ``slots`` (int64) of the 4-bit cache back as 16-bit values
    (``pkv_kv4_load``).  dtype: bfloat16 (the default) or float16; k, v: contiguous [slots, heads,
    head_dim], allocated when not given.  A negative slot gives zeros.  Returns (k, v)."""
    made = (_SHORT or _short()).kv4_load(k_cache, v_cache, k_scale, v_scale, slots, dtype, k, v, k_unit, v_unit, d_error, stream,
                                          check)
    if made is not NotImplemented:
        return made
    cache = _kv4_cache(k_cache, v_cache, k_scale, v_scale, k_unit, v_unit)
    torch = _KV8[0]
    n = slots.numel()
    if not (slots.dtype is _KV8[4] and slots.is_contiguous()):
        raise ValueError("slots is contiguous int64")
    given = k if k is not None else v
    if dtype is None:
        dtype = torch.bfloat16 if given is None else given.dtype
    kind, shape = _KV8[1].get(dtype), (n, k_cache.shape[1], 2 * k_cache.shape[3])
    if kind is None:
        raise ValueError("bfloat16 or float16")
    for t in (k, v):
        if t is not None and not (t.shape == shape and t.dtype is dtype and t.is_contiguous()):
            raise ValueError("k and v are contiguous [slots, heads, head_dim] of dtype")
    device = _kv8_device(stream, k_cache, v_cache, k_scale, v_scale, slots, k, v)
    if _kv8_elsewhere(device):
        with torch.cuda.device(device):
            return kv4_load(k_cache, v_cache, k_scale, v_scale, slots, dtype, k, v, k_unit, v_unit, d_error, stream,
                            check)
    handle = _kv8_stream(stream, device)
    if k is None:
        k = _kv8_make(shape, dtype, k_cache.device, stream, handle)
    if v is None:
        v = _kv8_make(shape, dtype, k_cache.device, stream, handle)
    rc = lib().pkv_kv4_load(C.byref(cache), slots.data_ptr(), _kv8_size(n, "slots"), kind, k.data_ptr(), v.data_ptr(),
                            d_error or None, handle)
    if rc != OK:
        if check:
            raise PkvError(rc, "pkv_kv4_load")
        return rc
    return k, v


def kv4_attention_workspace(head_dim):
    """Bytes of device workspace an attention call on the current device takes
    (``pkv_kv4_attention_workspace``)."""
    n = C.c_int64(0)
    rc = lib().pkv_kv4_attention_workspace(int(head_dim), C.byref(n))
    if rc != OK:
        raise PkvError(rc, "pkv_kv4_attention_workspace")
    return n.value


_KV4_WORKSPACE = {}      # bytes, by device (its SMs) and head_dim


def kv4_attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, query_start_loc, seq_lens,
                  softmax_scale=None, window=0, k_unit=1.0, v_unit=1.0, out=None, lse=None, workspace=None,
                  d_error=None, stream=None, check=True):
    """Attention of a prepared batch's queries over the 4-bit cache (``pkv_kv4_attention``).

    The cache as in ``kv4_store``; everything else as in ``kv8_attention``, which also adds up weights.
    workspace: uint8, kv4_attention_workspace bytes.  Returns (out, lse)."""
    made = (_SHORT or _short()).kv4_attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, query_start_loc, seq_lens,
                                               softmax_scale, window, k_unit, v_unit, out, lse, workspace, d_error, stream,
                                               check)
    if made is not NotImplemented:
        return made
    cache = _kv4_cache(k_cache, v_cache, k_scale, v_scale, k_unit, v_unit)
    torch, _, f32 = _KV8[:3]
    _kv8_int32(block_tables, query_start_loc, seq_lens)
    n, table = seq_lens.numel(), block_tables.shape
    if not (len(table) == 2 and table[0] >= n and query_start_loc.numel() >= n + 1):
        raise ValueError("block_tables [n, W], query_start_loc [n + 1], seq_lens [n]")
    shape = q.shape
    if not (len(shape) == 3 and shape[2] == 2 * k_cache.shape[3]):
        raise ValueError("q is [tokens, q_heads, head_dim]")
    T, hq, d = shape
    window = _kv8_size(window, "window")
    kind, q_stride = _kv8_dtype(q), _lines(q, shape, d, "q")
    if out is not None and not (out.shape == shape and out.dtype is q.dtype):
        raise ValueError("out has q's shape and type")
    out_stride = hq * d * 2 if out is None else _lines(out, shape, d, "out")
    if not (lse is None or lse.shape == (T, hq) and lse.dtype is f32 and lse.is_contiguous()):
        raise ValueError("lse is contiguous float32 [tokens, q_heads]")
    if not (workspace is None or workspace.is_contiguous()):
        raise ValueError("workspace is contiguous")
    device = _kv8_device(stream, k_cache, v_cache, k_scale, v_scale, q, block_tables, query_start_loc, seq_lens,
                         out, lse, workspace)
    if _kv8_elsewhere(device):
        with torch.cuda.device(device):
            return kv4_attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, query_start_loc, seq_lens,
                                 softmax_scale, window, k_unit, v_unit, out, lse, workspace, d_error, stream, check)
    handle = _kv8_stream(stream, device)
    if out is None:
        out = _make_like(q, stream, handle)
    if lse is None:
        lse = _kv8_make((T, hq), f32, q.device, stream, handle)
    if workspace is None:
        size = _KV4_WORKSPACE.get((device, d))
        if size is None:
            size = _KV4_WORKSPACE[device, d] = kv4_attention_workspace(d)
        workspace = _kv8_make(size, torch.uint8, q.device, stream, handle, returned=False)
    rc = lib().pkv_kv4_attention(C.byref(cache), q.data_ptr(), q_stride, kind, hq, block_tables.data_ptr(),
                                 table[1], query_start_loc.data_ptr(), seq_lens.data_ptr(), n, T,
                                 d ** -0.5 if softmax_scale is None else float(softmax_scale), window,
                                 out.data_ptr(), out_stride, lse.data_ptr(), workspace.data_ptr(),
                                 workspace.numel() * workspace.itemsize, d_error or None, handle)
    if rc != OK:
        if check:
            raise PkvError(rc, "pkv_kv4_attention")
        return rc
    return out, lse


# -- verification of drafted tokens -------------------------------------------


def verify_drafts(target_probs, draft_ids, query_start_loc, uniforms, max_drafts, draft_probs=None,
                  tokens=None, accepted=None, d_error=None, stream=None, check=True):
    """Which drafted tokens stand, and the token after them (``pkv_verify_drafts``).

    target_probs: float32, bfloat16 or float16 [rows, vocab], a row for each drafted token of a
    request and a last one for the token after them; draft_ids: int32, the token drafted at each row
    (input_ids[1:] of a prepared batch whose requests run one token and their drafts; not read for a
    request's last row, so rows - 1 entries do); query_start_loc: int32 [n + 1] of the rows; uniforms:
    float32 [rows] in [0, 1); draft_probs: like target_probs, the distributions the drafts were drawn
    from (None: drafts are certain).  Rows may be apart by a stride.  Returns (tokens int32 [n,
    max_drafts + 1]: the drafts that stand, the drawn token, then -1; accepted int32 [n])."""
    made = (_SHORT or _short()).verify_drafts(target_probs, draft_ids, query_start_loc, uniforms, max_drafts, draft_probs, tokens,
                                               accepted, d_error, stream, check)
    if made is not NotImplemented:
        return made
    torch, kinds, f32, i32 = _kv8_types()[:4]
    kind = 2 if target_probs.dtype is f32 else kinds.get(target_probs.dtype)
    if kind is None or target_probs.dim() != 2:
        raise ValueError("target_probs is float32, bfloat16 or float16 [rows, vocab]")
    rows, vocab = target_probs.shape
    for p in (target_probs, draft_probs):
        if p is not None and not (p.dtype is target_probs.dtype and p.shape == target_probs.shape and
                                  (p.stride(1) == 1 or vocab == 1)):
            raise ValueError("draft_probs has target_probs' shape and type, a row's elements are contiguous")
    _kv8_int32(draft_ids, query_start_loc)
    n, max_drafts = query_start_loc.numel() - 1, _kv8_size(max_drafts, "max_drafts")
    if n < 0 or max_drafts < 0 or draft_ids.numel() < rows - 1:
        raise ValueError("query_start_loc [n + 1], draft_ids a token for each row but the last")
    if not (uniforms.dtype is f32 and uniforms.is_contiguous() and uniforms.numel() >= rows):
        raise ValueError("uniforms is contiguous float32, one for each row")
    for t, shape in ((tokens, (n, max_drafts + 1)), (accepted, (n,))):
        if t is not None:
            _kv8_int32(t)
            if t.shape != shape:
                raise ValueError("tokens is [n, max_drafts + 1], accepted [n]")
    device = _kv8_device(stream, target_probs, draft_probs, draft_ids, query_start_loc, uniforms, tokens, accepted)
    if _kv8_elsewhere(device):
        with torch.cuda.device(device):
            return verify_drafts(target_probs, draft_ids, query_start_loc, uniforms, max_drafts, draft_probs, tokens,
                                 accepted, d_error, stream, check)
    handle = _kv8_stream(stream, device)
    if tokens is None:
        tokens = _kv8_make((n, max_drafts + 1), i32, target_probs.device, stream, handle)
    if accepted is None:
        accepted = _kv8_make(n, i32, target_probs.device, stream, handle)
    rc = lib().pkv_verify_drafts(target_probs.data_ptr(), target_probs.stride(0) if rows > 1 else vocab,
                                 None if draft_probs is None else draft_probs.data_ptr(),
                                 0 if draft_probs is None else draft_probs.stride(0) if rows > 1 else vocab, kind, vocab,
                                 rows, draft_ids.data_ptr(), query_start_loc.data_ptr(), n, uniforms.data_ptr(),
                                 max_drafts, tokens.data_ptr(), accepted.data_ptr(), d_error or None, handle)
    if rc != OK:
        if check:
            raise PkvError(rc, "pkv_verify_drafts")
        return rc
    return tokens, accepted
