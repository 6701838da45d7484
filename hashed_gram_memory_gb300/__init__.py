"""Engram hashed n-gram memory lookup for GB300 (sm_103a).

A thin Python binding over libengram.so, whose C ABI is include/engram.h.  The
functions carry the C names and only marshal arguments: torch tensors become
device pointers, the current torch CUDA stream becomes the cudaStream_t (or the one
that `stream` names, to which what a call allocates then belongs too), and a
non-zero status becomes an EngramError.  No call builds an autograd graph.  Every
step of the path runs in the library's CUDA kernels; there is no CPU or PyTorch
fallback, and importing this package fails if the library has not been built.
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libengram.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_OUT_OF_RANGE, ERR_TIMEOUT = range(6)
FLAG_BAD_TOKEN, FLAG_BAD_EID, FLAG_BAD_ROW, FLAG_TIMEOUT = 1, 2, 4, 8
TABLE_FP8_E4M3FN, TABLE_BF16, TABLE_FP8_E8M0, TABLE_FP8_E8M0_ROWS = 0, 1, 2, 3
EID_DEAD = ROW_DEAD = -1
LOOKUP_AUTO, LOOKUP_GATHER, LOOKUP_BULK = 0, 1, 2
PROJECTION_AUTO, PROJECTION_SINGLE, PROJECTION_PAIR = 0, 1, 2
MAX_HEADS, MAX_D = 32, 4096
DTYPE_BF16, DTYPE_F32 = 0, 1
MAX_EMBED_D = 16384
FP8_BLOCK = 128


class EngramError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(message)
        self.code = code


class engram_tables(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("D", C.c_int32), ("rows", C.c_int64 * 3),
                ("table", C.c_void_p * 3), ("scale", C.c_void_p * 3)]


class engram_layout(C.Structure):
    _fields_ = [("positions", C.c_void_p), ("dead", C.c_void_p),
                ("primes", C.POINTER(C.c_int64))]


def _layout(positions, dead, primes, host: bool):
    """The engram_layout struct for the whole-path calls (None when all three are
    None).  positions / dead are device tensors, or host tensors when `host`;
    primes is [3][n_heads] bucket sizes (host ints).  The struct keeps the
    primes array alive."""
    import torch
    if positions is None and dead is None and primes is None:
        return None
    for t, name, dts in ((positions, "positions", (torch.int32,)),
                         (dead, "dead", (torch.uint8, torch.bool))):
        if t is None:
            continue
        if t.is_cuda == host:
            where = "host" if host else "CUDA"
            raise EngramError(ERR_INVALID_ARG, f"{name} must be a {where} tensor here")
        if t.dtype not in dts or not t.is_contiguous():
            raise EngramError(ERR_INVALID_ARG, f"{name} must be contiguous {dts}")
    lay = engram_layout()
    lay.positions = None if positions is None else positions.data_ptr()
    lay.dead = None if dead is None else dead.data_ptr()
    if primes is not None:
        flat = [int(v) for order in primes for v in order]
        lay._primes = (C.c_int64 * len(flat))(*flat)
        lay.primes = C.cast(lay._primes, C.POINTER(C.c_int64))
    return lay


def _ref(lay):
    return None if lay is None else C.byref(lay)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the CUDA library first "
            "(python hashed_gram_memory_gb300/build.py, or __graft_entry__.build())")
    L = C.CDLL(LIB_PATH)
    vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    L.engram_compress.argtypes = [vp, i64, vp, i32, i32, vp, vp, vp]
    L.engram_compress_masked.argtypes = [vp, i64, vp, i32, i32, vp, vp, vp, vp]
    L.engram_hash.argtypes = [vp, i32, i32, vp, vp, i32, C.POINTER(C.c_int64), vp, vp, vp]
    L.engram_hash_packed.argtypes = [vp, i32, i32, vp, vp, vp, i32, C.POINTER(C.c_int64), vp, vp,
                                     vp]
    L.engram_hash_bucketed.argtypes = [vp, i32, i32, vp, vp, vp, i32, C.POINTER(C.c_int64), vp, vp,
                                       vp]
    L.engram_bucket_primes.argtypes = [i32, i32, i32, i64, C.POINTER(C.c_int64)]
    L.engram_compress_hash.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, i32,
                                       C.POINTER(C.c_int64), C.POINTER(engram_layout), vp, vp, vp,
                                       vp]
    L.engram_lookup_fused.argtypes = [vp, i64, i32, C.POINTER(engram_tables), vp, vp, vp,
                                      C.c_float, vp, vp, vp, vp]
    L.engram_read_status.argtypes = [vp, C.POINTER(C.c_int32), vp]
    for f in ("engram_compress", "engram_compress_masked", "engram_hash", "engram_hash_packed",
              "engram_hash_bucketed", "engram_bucket_primes", "engram_compress_hash",
              "engram_lookup_fused", "engram_read_status"):
        getattr(L, f).restype = C.c_int32
    L.engram_status_string.argtypes = [C.c_int32]
    L.engram_status_string.restype = C.c_char_p
    L.engram_last_error.argtypes = []
    L.engram_last_error.restype = C.c_char_p
    L.engram_abi_version.restype = C.c_int32
    L.engram_set_lookup_kernel.argtypes = [C.c_int32]
    L.engram_set_lookup_kernel.restype = C.c_int32
    L.engram_set_projection_kernel.argtypes = [C.c_int32]
    L.engram_set_projection_kernel.restype = C.c_int32
    L.engram_set_wait_limit_ns.argtypes = [C.c_int64]
    L.engram_set_wait_limit_ns.restype = C.c_int64
    L.engram_debug_withhold_copies.argtypes = [C.c_int32]
    L.engram_debug_withhold_copies.restype = None
    sz = C.c_size_t
    L.engram_forward_workspace_bytes.argtypes = [i32, i32, i32]
    L.engram_forward_workspace_bytes.restype = sz
    tabp, layp = C.POINTER(engram_tables), C.POINTER(engram_layout)
    L.engram_forward.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, i32, tabp, layp,
                                 vp, vp, vp, C.c_float, vp, sz, vp, vp]
    L.engram_forward.restype = i32
    L.engram_forward_host_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.engram_forward_host_workspace_bytes.restype = sz
    L.engram_forward_host.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, i32, tabp, layp,
                                      vp, vp, vp, C.c_float, i32, vp, sz, vp, vp]
    L.engram_forward_host.restype = i32
    L.engram_forward_static.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, i32, tabp, layp,
                                        vp, vp, vp, C.c_float, vp, vp]
    L.engram_forward_static.restype = i32
    L.engram_connection_host_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    L.engram_connection_host_workspace_bytes.restype = sz
    L.engram_connection_host.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, i32, tabp, layp,
                                         vp, i32, vp, vp, vp, C.c_float, i32, vp, sz, vp, vp]
    L.engram_connection_host.restype = i32
    L.engram_connection_workspace_bytes.argtypes = [i64, i32, i32, i32]
    L.engram_connection_workspace_bytes.restype = sz
    L.engram_connection.argtypes = [vp, i64, i32, C.POINTER(engram_tables), vp, i32, vp, vp, vp,
                                    C.c_float, vp, sz, vp, vp, vp, vp]
    L.engram_connection.restype = i32
    L.engram_concat_rows.argtypes = [vp, i64, i32, C.POINTER(engram_tables), vp, vp, vp, vp]
    L.engram_concat_rows.restype = i32
    L.engram_wkv_project.argtypes = [vp, i64, i32, vp, i32, vp, vp, vp]
    L.engram_wkv_project.restype = i32
    L.engram_gate_add.argtypes = [vp, vp, i64, i32, vp, vp, vp, C.c_float, vp, vp]
    L.engram_gate_add.restype = i32
    L.engram_pack_e8m0_rows.argtypes = [vp, vp, i64, i32, vp, vp]
    L.engram_pack_e8m0_rows.restype = i32
    L.engram_embed.argtypes = [vp, i64, i32, i64, vp, i32, i64, i32, i64, C.c_float, i32, vp, i32,
                               i64, i64, vp, vp]
    L.engram_embed.restype = i32
    L.engram_embed_grad_workspace_bytes.argtypes = [i64, i32, i32]
    L.engram_embed_grad_workspace_bytes.restype = sz
    L.engram_embed_grad.argtypes = [vp, i64, i32, i64, vp, i32, i64, i64, i64, i32, C.c_float, i32,
                                    vp, i32, i64, vp, sz, vp, vp]
    L.engram_embed_grad.restype = i32
    L.engram_embed_grad_rows.argtypes = [vp, i64, i32, i64, vp, i32, i64, i64, i64, i32, C.c_float,
                                         vp, vp, i32, i64, vp, vp, sz, vp, vp]
    L.engram_embed_grad_rows.restype = i32
    L.engram_fp8_quantise.argtypes = [vp, i32, i64, i64, i64, i32, vp, i64, vp, vp, i64, vp, vp,
                                      vp]
    L.engram_fp8_quantise.restype = i32
    L.engram_fp8_matmul.argtypes = [vp, i64, vp, i32, vp, i64, vp, i32, i64, i64, i64, vp, i32,
                                    i64, vp, vp]
    L.engram_fp8_matmul.restype = i32
    L.engram_gate_add_grad_workspace_bytes.argtypes = []
    L.engram_gate_add_grad_workspace_bytes.restype = sz
    L.engram_gate_add_grad.argtypes = [vp, vp, i64, i32, vp, vp, C.c_float, vp, vp, vp, i32, vp,
                                       vp, sz, vp]
    L.engram_gate_add_grad.restype = i32
    return L


lib = _load()


def _check(code: int, what: str):
    if code != OK:
        msg = lib.engram_last_error().decode() or lib.engram_status_string(code).decode()
        raise EngramError(code, f"{what}: {lib.engram_status_string(code).decode()}: {msg}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        try:  # the raw handle: a stream object costs several microseconds a call
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:
            return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _made(stream, make, *args, scratch=False, **kw):
    """make(*args, **kw), a tensor that a call makes for itself, in the pool of the stream that the
    call launches on: its memory is free for use there at once, and not handed out again before
    the launch is done with it.  Results (not scratch) also stay while the current stream reads
    them."""
    if stream is None or _stream(stream) == _stream(None):
        return make(*args, **kw)
    import torch
    if isinstance(stream, int):  # 0 and 1 name the default stream, which is not an external one
        stream = torch.cuda.ExternalStream(stream) if stream > 1 else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    if not scratch:
        t.record_stream(torch.cuda.current_stream())
    return t


def _need(t, dtypes, name, contiguous=True):
    if t is None:
        return
    if not t.is_cuda:
        raise EngramError(ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise EngramError(ERR_INVALID_ARG, f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if contiguous and not t.is_contiguous():
        raise EngramError(ERR_INVALID_ARG, f"{name} must be contiguous")


def e8m0_row_bytes(D: int) -> int:
    """Bytes of one row of a TABLE_FP8_E8M0_ROWS table of width D (the row, its
    D/32 exponents, zeros up to a multiple of 16)."""
    return (D + D // 32 + 15) // 16 * 16


@dataclasses.dataclass
class Tables:
    """The three device tables (orders 2, 3, 4) and their scales: fp32 [rows] for
    TABLE_FP8_E4M3FN, uint8 e8m0 exponents [rows, D/32] for TABLE_FP8_E8M0, none
    for TABLE_BF16.  TABLE_FP8_E8M0_ROWS tables are uint8 [rows,
    e8m0_row_bytes(D)] (engram_pack_e8m0_rows) with no scales; their D is the
    widest multiple of 32 whose packed row fills the table's row."""

    dtype: int
    tables: list
    scales: list | None = None

    @property
    def D(self) -> int:
        width = int(self.tables[0].shape[1])
        if self.dtype != TABLE_FP8_E8M0_ROWS:
            return width
        D = width * 32 // 33 // 32 * 32
        while D > 0 and e8m0_row_bytes(D) > width:
            D -= 32
        if D <= 0 or e8m0_row_bytes(D) != width:
            raise EngramError(ERR_INVALID_ARG, f"{width} bytes is no packed e8m0 row width")
        return D

    @property
    def rows(self):
        return [int(t.shape[0]) for t in self.tables]

    def struct(self) -> engram_tables:
        s = engram_tables()
        s.dtype = self.dtype
        s.D = self.D
        for n in range(3):
            s.rows[n] = int(self.tables[n].shape[0])
            s.table[n] = self.tables[n].data_ptr()
            sc = self.scales[n] if self.scales else None
            s.scale[n] = sc.data_ptr() if sc is not None else None
        return s


def engram_pack_e8m0_rows(table, exps, packed=None, stream=None):
    """A TABLE_FP8_E8M0_ROWS table from a TABLE_FP8_E8M0 one: table uint8 [rows, D],
    exps uint8 [rows, D/32] -> uint8 [rows, e8m0_row_bytes(D)] (each row, then its
    exponents, then zeros)."""
    import torch
    _need(table, (torch.uint8,), "table")
    _need(exps, (torch.uint8,), "exps")
    rows, D = table.shape
    if tuple(exps.shape) != (rows, D // 32):
        raise EngramError(ERR_INVALID_ARG, "exps must be [rows, D/32]")
    if packed is None:
        packed = _made(stream, torch.empty, (rows, e8m0_row_bytes(D)), dtype=torch.uint8,
                       device=table.device)
    _need(packed, (torch.uint8,), "packed")
    _check(lib.engram_pack_e8m0_rows(_ptr(table), _ptr(exps), rows, D, _ptr(packed),
                                     _stream(stream)), "engram_pack_e8m0_rows")
    return packed


def engram_compress(token_ids, tid2eid, n_eids: int, eids_out=None, status=None, stream=None,
                    dead=None):
    """eids_out[i] = tid2eid[token_ids[i]] (int32, same shape as token_ids); with a
    dead mask (uint8/bool, same shape) dead positions become EID_DEAD."""
    import torch
    _need(token_ids, (torch.int32,), "token_ids")
    _need(tid2eid, (torch.int32,), "tid2eid")
    _need(dead, (torch.uint8, torch.bool), "dead")
    if eids_out is None:
        eids_out = _made(stream, torch.empty_like, token_ids)
    _need(eids_out, (torch.int32,), "eids_out")
    _check(lib.engram_compress_masked(_ptr(token_ids), token_ids.numel(), _ptr(tid2eid),
                                      tid2eid.numel(), n_eids, _ptr(dead), _ptr(eids_out),
                                      _ptr(status), _stream(stream)),
           "engram_compress")
    return eids_out


def engram_bucket_primes(n_layers: int, max_ngram: int, n_heads: int, hash_vocab: int):
    """The released layout's bucket sizes, [n_layers][max_ngram - 1][n_heads] (host ints)."""
    n = n_layers * (max_ngram - 1) * n_heads
    out = (C.c_int64 * n)()
    _check(lib.engram_bucket_primes(n_layers, max_ngram, n_heads, hash_vocab, out),
           "engram_bucket_primes")
    flat = list(out)
    k = max_ngram - 1
    return [[flat[(l * k + i) * n_heads:(l * k + i + 1) * n_heads] for i in range(k)]
            for l in range(n_layers)]


def engram_hash(eids, n_heads: int, rows, history=None, history_out=None, row_ids_out=None,
                status=None, stream=None, positions=None, primes=None):
    """Row ids [B, S, 3, n_heads] int32 for eids [B, S]; history/history_out [B, 3];
    positions [B, S] (optional): each token's index within its packed sample.
    With primes ([3][n_heads] bucket sizes of one layer) the ids index one table
    cut into prime buckets (engram_hash_bucketed) and rows is not used."""
    import torch
    _need(eids, (torch.int32,), "eids")
    if eids.dim() != 2:
        raise EngramError(ERR_INVALID_ARG, "eids must be [batch, seq]")
    B, S = eids.shape
    if row_ids_out is None:
        row_ids_out = _made(stream, torch.empty, (B, S, 3, n_heads), dtype=torch.int32,
                            device=eids.device)
    _need(row_ids_out, (torch.int32,), "row_ids_out")
    _need(history, (torch.int32,), "history")
    _need(history_out, (torch.int32,), "history_out")
    _need(positions, (torch.int32,), "positions")
    if primes is not None:
        flat = [int(v) for order in primes for v in order]
        pr = (C.c_int64 * len(flat))(*flat)
        _check(lib.engram_hash_bucketed(_ptr(eids), B, S, _ptr(positions), _ptr(history),
                                        _ptr(history_out), n_heads, pr, _ptr(row_ids_out),
                                        _ptr(status), _stream(stream)), "engram_hash_bucketed")
        return row_ids_out
    r = (C.c_int64 * 3)(*[int(x) for x in rows])
    _check(lib.engram_hash_packed(_ptr(eids), B, S, _ptr(positions), _ptr(history),
                                  _ptr(history_out), n_heads, r, _ptr(row_ids_out), _ptr(status),
                                  _stream(stream)), "engram_hash")
    return row_ids_out


def engram_compress_hash(token_ids, tid2eid, n_eids: int, n_heads: int, rows, history=None,
                         history_out=None, row_ids_out=None, eids_out=None, status=None,
                         stream=None, positions=None, dead=None, primes=None):
    """Compression and hash in one launch: row ids [B, S, 3, n_heads] int32 for token
    ids [B, S]; positions / dead (device) and primes as for engram_forward;
    eids_out (optional, int32 [B, S]) receives the compressed ids."""
    import torch
    _need(token_ids, (torch.int32,), "token_ids")
    _need(tid2eid, (torch.int32,), "tid2eid")
    if token_ids.dim() != 2:
        raise EngramError(ERR_INVALID_ARG, "token_ids must be [batch, seq]")
    B, S = token_ids.shape
    if row_ids_out is None:
        row_ids_out = _made(stream, torch.empty, (B, S, 3, n_heads), dtype=torch.int32,
                            device=token_ids.device)
    _need(row_ids_out, (torch.int32,), "row_ids_out")
    _need(eids_out, (torch.int32,), "eids_out")
    _need(history, (torch.int32,), "history")
    _need(history_out, (torch.int32,), "history_out")
    r = None if rows is None else (C.c_int64 * 3)(*[int(x) for x in rows])  # unused with primes
    lay = _layout(positions, dead, primes, host=False)
    _check(lib.engram_compress_hash(_ptr(token_ids), B, S, _ptr(tid2eid), tid2eid.numel(), n_eids,
                                    _ptr(history), _ptr(history_out), n_heads, r, _ref(lay),
                                    _ptr(eids_out), _ptr(row_ids_out), _ptr(status),
                                    _stream(stream)), "engram_compress_hash")
    return row_ids_out


def engram_lookup_fused(row_ids, n_heads: int, tables: Tables, streams_in, alpha,
                        eps: float = 1e-6, streams_out=None, gate_out=None, mem_out=None,
                        status=None, stream=None):
    """The fused gather / mean / gate / add.  streams_in: bf16 [..., 4, D]; returns streams_out."""
    import torch
    _need(row_ids, (torch.int32,), "row_ids")
    bf = (torch.bfloat16, torch.int16)
    _need(streams_in, bf, "streams_in")
    _need(alpha, (torch.float32,), "alpha")
    D = tables.D
    if streams_in.shape[-2:] != (4, D):
        raise EngramError(ERR_INVALID_ARG, f"streams_in must be [..., 4, {D}]")
    T = streams_in.numel() // (4 * D)
    if row_ids.numel() != T * 3 * n_heads:
        raise EngramError(ERR_INVALID_ARG, "row_ids and streams disagree on the token count")
    if streams_out is None:
        streams_out = _made(stream, torch.empty_like, streams_in)
    _need(streams_out, bf, "streams_out")
    _need(gate_out, (torch.float32,), "gate_out")
    _need(mem_out, (torch.float32,), "mem_out")
    s = tables.struct()
    _check(lib.engram_lookup_fused(_ptr(row_ids), T, n_heads, C.byref(s), _ptr(streams_in),
                                   _ptr(streams_out), _ptr(alpha), float(eps), _ptr(gate_out),
                                   _ptr(mem_out), _ptr(status), _stream(stream)),
           "engram_lookup_fused")
    return streams_out


def engram_connection_workspace_bytes(n_tokens: int, n_heads: int, d: int, D: int) -> int:
    return int(lib.engram_connection_workspace_bytes(n_tokens, n_heads, d, D))


def engram_connection(row_ids, n_heads: int, tables: Tables, wkv, streams_in, alpha,
                      eps: float = 1e-6, streams_out=None, workspace=None, gate_out=None,
                      k_out=None, status=None, stream=None):
    """The connection with a wkv projection: rows concatenated, k = wkv e, gate, add.
    wkv: bf16 [D, 3*n_heads*d]; streams_in: bf16 [..., 4, D]; returns streams_out."""
    import torch
    _need(row_ids, (torch.int32,), "row_ids")
    bf = (torch.bfloat16, torch.int16)
    _need(streams_in, bf, "streams_in")
    _need(wkv, bf, "wkv")
    _need(alpha, (torch.float32,), "alpha")
    D = streams_in.shape[-1]
    if streams_in.shape[-2] != 4:
        raise EngramError(ERR_INVALID_ARG, "streams_in must be [..., 4, D]")
    T = streams_in.numel() // (4 * D)
    if row_ids.numel() != T * 3 * n_heads:
        raise EngramError(ERR_INVALID_ARG, "row_ids and streams disagree on the token count")
    if tuple(wkv.shape) != (D, 3 * n_heads * tables.D):
        raise EngramError(ERR_INVALID_ARG, f"wkv must be [{D}, {3 * n_heads * tables.D}]")
    if streams_out is None:
        streams_out = _made(stream, torch.empty_like, streams_in)
    _need(streams_out, bf, "streams_out")
    _need(gate_out, (torch.float32,), "gate_out")
    _need(k_out, (torch.float32,), "k_out")
    need = engram_connection_workspace_bytes(T, n_heads, tables.D, D)
    if workspace is None:
        workspace = _made(stream, torch.empty, max(need, 1), dtype=torch.uint8,
                          device=streams_in.device, scratch=True)
    s = tables.struct()
    _check(lib.engram_connection(_ptr(row_ids), T, n_heads, C.byref(s), _ptr(wkv), D,
                                 _ptr(streams_in), _ptr(streams_out), _ptr(alpha), float(eps),
                                 _ptr(workspace), workspace.numel(), _ptr(gate_out), _ptr(k_out),
                                 _ptr(status), _stream(stream)),
           "engram_connection")
    return streams_out


def engram_concat_rows(row_ids, n_heads: int, tables: Tables, e_out=None, state_out=None,
                       status=None, stream=None):
    """E = the tokens' concatenated rows (bf16 [T, 3*n_heads*d]) and their state
    (uint8 [T]: 0 live, 1 dead, 2 bad).  Returns (E, state)."""
    import torch
    _need(row_ids, (torch.int32,), "row_ids")
    T = row_ids.numel() // (3 * n_heads)
    K = 3 * n_heads * tables.D
    dev = row_ids.device
    if e_out is None:
        e_out = _made(stream, torch.empty, (T, K), dtype=torch.bfloat16, device=dev)
    if state_out is None:
        state_out = _made(stream, torch.empty, (T,), dtype=torch.uint8, device=dev)
    _need(e_out, (torch.bfloat16, torch.int16), "e_out")
    _need(state_out, (torch.uint8,), "state_out")
    if e_out.numel() != T * K or state_out.numel() != T:
        raise EngramError(ERR_INVALID_ARG, "e_out / state_out sizes")
    s = tables.struct()
    _check(lib.engram_concat_rows(_ptr(row_ids), T, n_heads, C.byref(s), _ptr(e_out),
                                  _ptr(state_out), _ptr(status), _stream(stream)),
           "engram_concat_rows")
    return e_out, state_out


def engram_wkv_project(e, wkv, k_out=None, status=None, stream=None):
    """k = E wkv^T on the tensor cores: e bf16 [T, K], wkv bf16 [D, K] -> k fp32 [T, D]."""
    import torch
    bf = (torch.bfloat16, torch.int16)
    _need(e, bf, "e")
    _need(wkv, bf, "wkv")
    T, K = e.shape
    D = wkv.shape[0]
    if wkv.shape[1] != K:
        raise EngramError(ERR_INVALID_ARG, "e and wkv disagree on K")
    if k_out is None:
        k_out = _made(stream, torch.empty, (T, D), dtype=torch.float32, device=e.device)
    _need(k_out, (torch.float32,), "k_out")
    if k_out.numel() != T * D:
        raise EngramError(ERR_INVALID_ARG, "k_out must be [T, D]")
    _check(lib.engram_wkv_project(_ptr(e), T, K, _ptr(wkv), D, _ptr(k_out), _ptr(status),
                                  _stream(stream)), "engram_wkv_project")
    return k_out


def engram_gate_add(k, state, streams_in, alpha, eps: float = 1e-6, streams_out=None,
                    gate_out=None, stream=None):
    """The gate of k against stream 0 and the gated add into the four streams."""
    import torch
    _need(k, (torch.float32,), "k")
    _need(state, (torch.uint8,), "state")
    bf = (torch.bfloat16, torch.int16)
    _need(streams_in, bf, "streams_in")
    _need(alpha, (torch.float32,), "alpha")
    D = streams_in.shape[-1]
    T = streams_in.numel() // (4 * D)
    if k.numel() != T * D or state.numel() != T:
        raise EngramError(ERR_INVALID_ARG, "k / state sizes disagree with the streams")
    if streams_out is None:
        streams_out = _made(stream, torch.empty_like, streams_in)
    _need(streams_out, bf, "streams_out")
    _need(gate_out, (torch.float32,), "gate_out")
    _check(lib.engram_gate_add(_ptr(k), _ptr(state), T, D, _ptr(streams_in), _ptr(streams_out),
                               _ptr(alpha), float(eps), _ptr(gate_out), _stream(stream)),
           "engram_gate_add")
    return streams_out


def engram_read_status(status, stream=None):
    """(code, flags): waits for the stream and reads the device status word."""
    v = C.c_int32(0)
    code = lib.engram_read_status(_ptr(status), C.byref(v), _stream(stream))
    if code not in (OK, ERR_OUT_OF_RANGE, ERR_TIMEOUT):
        _check(code, "engram_read_status")
    return code, int(v.value)


def engram_status_string(code: int) -> str:
    return lib.engram_status_string(code).decode()


def engram_abi_version() -> int:
    return int(lib.engram_abi_version())


def engram_set_projection_kernel(which: int) -> int:
    """PROJECTION_AUTO / PROJECTION_SINGLE / PROJECTION_PAIR for this process; returns the
    previous one."""
    prev = int(lib.engram_set_projection_kernel(which))
    if prev < 0:
        raise EngramError(ERR_INVALID_ARG, f"unknown projection kernel {which}")
    return prev


def engram_set_lookup_kernel(which: int) -> int:
    """LOOKUP_AUTO / LOOKUP_GATHER / LOOKUP_BULK for this process; returns the previous one."""
    prev = int(lib.engram_set_lookup_kernel(which))
    if prev < 0:
        raise EngramError(ERR_INVALID_ARG, f"unknown lookup kernel {which}")
    return prev


def engram_set_wait_limit_ns(ns: int) -> int:
    return int(lib.engram_set_wait_limit_ns(int(ns)))


def engram_debug_withhold_copies(launches: int) -> None:
    lib.engram_debug_withhold_copies(int(launches))


def engram_forward_workspace_bytes(batch: int, seq: int, n_heads: int) -> int:
    return int(lib.engram_forward_workspace_bytes(batch, seq, n_heads))


def engram_forward(token_ids, tid2eid, n_eids: int, n_heads: int, tables: Tables, streams_in,
                   alpha, eps: float = 1e-6, history=None, history_out=None, streams_out=None,
                   workspace=None, status=None, stream=None, positions=None, dead=None,
                   primes=None):
    """compress -> hash -> fused lookup in one call on device tensors; token_ids [B, S].
    positions [B, S] int32 and dead [B, S] uint8 (device) describe a packed batch;
    primes ([3][n_heads] bucket sizes) selects the prime-bucket table layout."""
    import torch
    _need(token_ids, (torch.int32,), "token_ids")
    B, S = token_ids.shape
    if streams_out is None:
        streams_out = _made(stream, torch.empty_like, streams_in)
    need = engram_forward_workspace_bytes(B, S, n_heads)
    if workspace is None:
        workspace = _made(stream, torch.empty, max(need, 16), dtype=torch.uint8,
                          device=token_ids.device, scratch=True)
    s = tables.struct()
    lay = _layout(positions, dead, primes, host=False)
    _check(lib.engram_forward(_ptr(token_ids), B, S, _ptr(tid2eid), tid2eid.numel(), n_eids,
                              _ptr(history), _ptr(history_out), n_heads, C.byref(s), _ref(lay),
                              _ptr(streams_in), _ptr(streams_out), _ptr(alpha), float(eps),
                              _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)),
           "engram_forward")
    return streams_out


def engram_forward_host_workspace_bytes(batch: int, seq: int, n_heads: int, D: int,
                                        chunk_tokens: int = 0) -> int:
    return int(lib.engram_forward_host_workspace_bytes(batch, seq, n_heads, D, chunk_tokens))


def engram_forward_host(token_ids_host, tid2eid, n_eids: int, n_heads: int, tables: Tables,
                        streams_in_host, streams_out_host, alpha, workspace, eps: float = 1e-6,
                        history=None, history_out=None, chunk_tokens: int = 0, status=None,
                        stream=None, positions=None, dead=None, primes=None):
    """The whole path with host (CPU, ideally pinned) token ids [B, S] and streams
    [B*S, 4, D]; positions / dead, when given, are host tensors too.  workspace is
    a device uint8 tensor of engram_forward_host_workspace_bytes(...) bytes.
    Asynchronous on `stream`."""
    B, S = token_ids_host.shape
    s = tables.struct()
    lay = _layout(positions, dead, primes, host=True)
    _check(lib.engram_forward_host(_ptr(token_ids_host), B, S, _ptr(tid2eid), tid2eid.numel(),
                                   n_eids, _ptr(history), _ptr(history_out), n_heads, C.byref(s),
                                   _ref(lay), _ptr(streams_in_host), _ptr(streams_out_host), _ptr(alpha),
                                   float(eps), chunk_tokens, _ptr(workspace), workspace.numel(),
                                   _ptr(status), _stream(stream)),
           "engram_forward_host")
    return streams_out_host


def engram_connection_host_workspace_bytes(batch: int, seq: int, n_heads: int, d: int, D: int,
                                           chunk_tokens: int = 0) -> int:
    return int(lib.engram_connection_host_workspace_bytes(batch, seq, n_heads, d, D, chunk_tokens))


def engram_connection_host(token_ids_host, tid2eid, n_eids: int, n_heads: int, tables: Tables,
                           wkv, streams_in_host, streams_out_host, alpha, workspace,
                           eps: float = 1e-6, history=None, history_out=None,
                           chunk_tokens: int = 0, status=None, stream=None, positions=None,
                           dead=None, primes=None):
    """The connection's whole path with host (ideally pinned) token ids [B, S] and
    streams [B*S, 4, D] (positions / dead host tensors too); wkv bf16 [D,
    3*n_heads*d] on the device; workspace a device uint8 tensor of
    engram_connection_host_workspace_bytes(...) bytes.  Asynchronous on `stream`."""
    B, S = token_ids_host.shape
    D = int(wkv.shape[0])
    s = tables.struct()
    lay = _layout(positions, dead, primes, host=True)
    _check(lib.engram_connection_host(_ptr(token_ids_host), B, S, _ptr(tid2eid), tid2eid.numel(),
                                      n_eids, _ptr(history), _ptr(history_out), n_heads,
                                      C.byref(s), _ref(lay), _ptr(wkv), D, _ptr(streams_in_host),
                                      _ptr(streams_out_host), _ptr(alpha), float(eps),
                                      chunk_tokens, _ptr(workspace), workspace.numel(),
                                      _ptr(status), _stream(stream)),
           "engram_connection_host")
    return streams_out_host


STATIC_WORKSPACE_BYTES = 16 << 20


def engram_forward_static(token_ids, tid2eid, n_eids: int, n_heads: int, tables: Tables,
                          streams_in, alpha, eps: float = 1e-6, history=None, history_out=None,
                          streams_out=None, status=None, stream=None, positions=None, dead=None,
                          primes=None):
    """engram_forward without a workspace: the library's fixed device array holds
    the ids (for callers that must not allocate device memory; see engram.h)."""
    import torch
    _need(token_ids, (torch.int32,), "token_ids")
    B, S = token_ids.shape
    if streams_out is None:
        streams_out = _made(stream, torch.empty_like, streams_in)
    s = tables.struct()
    lay = _layout(positions, dead, primes, host=False)
    _check(lib.engram_forward_static(_ptr(token_ids), B, S, _ptr(tid2eid), tid2eid.numel(), n_eids,
                                     _ptr(history), _ptr(history_out), n_heads, C.byref(s),
                                     _ref(lay), _ptr(streams_in), _ptr(streams_out), _ptr(alpha), float(eps),
                                     _ptr(status), _stream(stream)),
           "engram_forward_static")
    return streams_out


_dtype_codes: dict = {}


def _dtype(t, name):
    """The DTYPE_* of a bf16 (or bf16 bits) or fp32 CUDA tensor of any strides."""
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.bfloat16: DTYPE_BF16, torch.int16: DTYPE_BF16,
                             torch.float32: DTYPE_F32})
    code = _dtype_codes.get(t.dtype)
    if code is None or not t.is_cuda:
        _need(t, tuple(_dtype_codes), name, contiguous=False)
    return code


def _strides(t, name):
    """The strides of a tensor whose last dimension is dense."""
    st = t.stride()
    if st and st[-1] != 1 and t.shape[-1] > 1:
        raise EngramError(ERR_INVALID_ARG, f"the last dimension of {name} must be contiguous")
    return st


def _row_stride(t, name):
    """Elements between the rows of a two-dimensional tensor.  Under a row's width (broadcast or
    overlapping rows) the library refuses it; one row alone has no stride, whatever torch says."""
    stride = _strides(t, name)[0]
    return stride if t.shape[0] > 1 else max(stride, t.shape[1])


def _ids_view(ids):
    """ids [..., R] as (shape, tokens, R, stride between tokens)."""
    import torch
    if ids.dtype != torch.int32 or not ids.is_cuda:
        _need(ids, (torch.int32,), "ids", contiguous=False)
    shape = ids.shape
    if len(shape) == 2:
        return shape, shape[0], shape[1], _row_stride(ids, "ids")
    if not shape:
        raise EngramError(ERR_INVALID_ARG, "ids must have a dimension")
    if not ids.is_contiguous():
        raise EngramError(ERR_INVALID_ARG, "ids must be contiguous (or [tokens, ids] rows)")
    R = shape[-1] if len(shape) > 1 else 1
    return shape, (ids.numel() // R if R else 0), R, R


def _embed_rows(lead, t, D, pooled, name):
    """The strides (between tokens, between ids) of the rows of an output or gradient tensor
    that goes with ids of shape lead: [*lead, D], or [*lead[:-1], D] when pooled."""
    want = (*lead[:-1], D) if pooled else (*lead, D)
    if t.shape != want:
        raise EngramError(ERR_INVALID_ARG, f"{name} must be {list(want)}")
    st = _strides(t, name)
    if len(want) == 2:
        return (st[0], 0) if pooled else (st[0], D)
    if len(want) == 3 and not pooled:
        return st[0], st[1]
    if not t.is_contiguous():
        raise EngramError(ERR_INVALID_ARG, f"{name} must be contiguous beyond three dimensions")
    return (D, 0) if pooled else (lead[-1] * D, D)


def engram_embed(ids, table, scale: float = 1.0, pooled: bool = False, out=None, out_dtype=None,
                 status=None, stream=None):
    """out[..., :] = scale * table[ids]: ids int32 [T] or [T, R] (any leading dimensions when
    contiguous; rows of a wider id tensor when 2-D), table bf16 or fp32 [rows, D].  pooled
    sums over the last dimension of ids: [*ids.shape[:-1], D].  -1 reads as zeros."""
    td = _dtype(table, "table")
    if table.dim() != 2:
        raise EngramError(ERR_INVALID_ARG, "table must be [rows, D]")
    lead, T, R, ids_stride = _ids_view(ids)
    if pooled and len(lead) < 2:
        raise EngramError(ERR_INVALID_ARG, "pooled ids must be [..., ids]")
    rows, D = table.shape
    if out is None:
        import torch
        out = _made(stream, torch.empty, (*(lead[:-1] if pooled else lead), D),
                    dtype=out_dtype or table.dtype, device=table.device)
    od = _dtype(out, "out")
    tok, per = _embed_rows(lead, out, D, pooled, "out")
    _check(lib.engram_embed(ids.data_ptr(), T, R, ids_stride, table.data_ptr(), td, rows, D,
                            _row_stride(table, "table"), scale, pooled, out.data_ptr(), od,
                            tok, per, _ptr(status), _stream(stream)), "engram_embed")
    return out


def engram_embed_grad_workspace_bytes(n_tokens: int, n_ids: int, D: int) -> int:
    return int(lib.engram_embed_grad_workspace_bytes(n_tokens, n_ids, D))


def _grad_args(ids, dy, pooled, workspace, stream):
    """The arguments the two gradient calls share, from ids and dy ([*ids.shape, D], or
    [*ids.shape[:-1], D] when pooled; expanded dimensions may have stride 0)."""
    dd = _dtype(dy, "dy")
    lead, T, R, ids_stride = _ids_view(ids)
    if pooled and len(lead) < 2:
        raise EngramError(ERR_INVALID_ARG, "pooled ids must be [..., ids]")
    D = dy.shape[-1] if dy.dim() else 0
    tok, per = _embed_rows(lead, dy, D, pooled, "dy")
    if workspace is None:
        import torch
        workspace = _made(stream, torch.empty, max(engram_embed_grad_workspace_bytes(T, R, D), 16),
                          dtype=torch.uint8, device=dy.device, scratch=True)
    _need(workspace, (workspace.dtype,), "workspace")
    return D, T * R, (ids.data_ptr(), T, R, ids_stride, dy.data_ptr(), dd, tok, per), workspace


def engram_embed_grad(ids, dy, rows: int, scale: float = 1.0, pooled: bool = False, grad=None,
                      grad_dtype=None, accumulate: bool = False, workspace=None, status=None,
                      stream=None):
    """The gradient of engram_embed(ids, table [rows, D], scale, pooled)'s table for the output
    gradient dy: [rows, D], every row written (accumulate: added to grad, fp32 or bf16)."""
    D, n, args, workspace = _grad_args(ids, dy, pooled, workspace, stream)
    if grad is None:
        if accumulate:
            raise EngramError(ERR_INVALID_ARG, "accumulate needs a grad to add to")
        import torch
        grad = _made(stream, torch.empty, (rows, D), dtype=grad_dtype or torch.float32,
                     device=dy.device)
    gd = _dtype(grad, "grad")
    if grad.shape != (rows, D):
        raise EngramError(ERR_INVALID_ARG, f"grad must be {[rows, D]}")
    _check(lib.engram_embed_grad(*args, rows, D, scale, accumulate, grad.data_ptr(), gd,
                                 _row_stride(grad, "grad"), workspace.data_ptr(),
                                 workspace.numel(), _ptr(status), _stream(stream)),
           "engram_embed_grad")
    return grad


def engram_embed_grad_rows(ids, dy, rows: int, scale: float = 1.0, pooled: bool = False,
                           row_ids=None, grads=None, count=None, grad_dtype=None, workspace=None,
                           status=None, stream=None):
    """The same gradient as its distinct rows: (row_ids int32 [n], grads [n, D], count int32 [1])
    for n = ids.numel(): the ascending distinct ids and then -1, their gradients (the rows past
    count are not written), and their number."""
    import torch
    D, n, args, workspace = _grad_args(ids, dy, pooled, workspace, stream)
    if row_ids is None:
        row_ids = _made(stream, torch.empty, n, dtype=torch.int32, device=dy.device)
    if grads is None:
        grads = _made(stream, torch.empty, (n, D), dtype=grad_dtype or torch.float32,
                      device=dy.device)
    if count is None:
        count = _made(stream, torch.empty, 1, dtype=torch.int32, device=dy.device)
    _need(row_ids, (torch.int32,), "row_ids")
    _need(count, (torch.int32,), "count")
    gd = _dtype(grads, "grads")
    if row_ids.numel() != n or grads.shape != (n, D) or count.numel() != 1:
        raise EngramError(ERR_INVALID_ARG, "row_ids / grads / count sizes disagree with ids")
    _check(lib.engram_embed_grad_rows(*args, rows, D, scale, row_ids.data_ptr(), grads.data_ptr(),
                                      gd, _row_stride(grads, "grads"), count.data_ptr(),
                                      workspace.data_ptr(), workspace.numel(), _ptr(status),
                                      _stream(stream)), "engram_embed_grad_rows")
    return row_ids, grads, count


def fp8_empty(rows: int, cols: int, device):
    """An uninitialised uint8 [rows, cols] operand: rows a multiple of 16 bytes apart (of 128
    where they are long: the product reads them in 128-byte pieces)."""
    import torch
    step = 128 if cols > 512 else 16
    return torch.empty((rows, (cols + step - 1) // step * step), dtype=torch.uint8,
                       device=device)[:, :cols]


def _fp8_operand(t, name):
    """(rows, columns, stride) of a uint8 operand."""
    import torch
    if t.dtype != torch.uint8 or not t.is_cuda:
        _need(t, (torch.uint8,), name, contiguous=False)
    shape = t.shape
    if len(shape) != 2:
        raise EngramError(ERR_INVALID_ARG, f"{name} must be two-dimensional")
    return shape[0], shape[1], _strides(t, name)[0]


def _fp8_scales(t, rows, cols, block, name):
    import torch
    want = ((rows + block - 1) // block, (cols + FP8_BLOCK - 1) // FP8_BLOCK)
    if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
        _need(t, (torch.uint8,), name)
    if t.shape != want:
        raise EngramError(ERR_INVALID_ARG, f"{name} must be {list(want)}")
    return t.data_ptr()


def _fp8_copy(out, at, rows, cols, block):
    """The pointers and stride of one of the quantiser's copies, out[at] and out[at + 1]."""
    r, c, stride = _fp8_operand(out[at], "q")
    if r != rows or c != cols:
        raise EngramError(ERR_INVALID_ARG, f"q must be {[rows, cols]}")
    return out[at].data_ptr(), stride, _fp8_scales(out[at + 1], rows, cols, block, "scales")


def engram_fp8_quantise(x, block_rows: int = 1, rows: bool = True, cols: bool = False, out=None,
                        status=None, stream=None):
    """x bf16 or fp32 [M, K] as e4m3fn bytes with a power-of-two scale byte per block of 128.
    rows: (q [M, K], s [M, ceil(K/128)]), blocks along K.  cols: (qt [K, M], st [K,
    ceil(M/128)]), the transposed copy with blocks along M.  block_rows FP8_BLOCK: 128 x 128
    tiles share a scale.  Returns the copies asked for, in that order; out gives their
    buffers (rows a multiple of 16 bytes apart: fp8_empty)."""
    xd = _dtype(x, "x")
    if x.dim() != 2:
        raise EngramError(ERR_INVALID_ARG, "x must be [M, K]")
    if block_rows != 1 and block_rows != FP8_BLOCK:
        raise EngramError(ERR_INVALID_ARG, f"block_rows must be 1 or {FP8_BLOCK}")
    M, K = x.shape
    if out is None:
        import torch
        out = []
        for r, c in ([(M, K)] if rows else []) + ([(K, M)] if cols else []):
            out += [_made(stream, fp8_empty, r, c, x.device),
                    _made(stream, torch.empty, (-(-r // block_rows), -(-c // FP8_BLOCK)),
                          dtype=torch.uint8, device=x.device)]
    if len(out) != 2 * (bool(rows) + bool(cols)):
        raise EngramError(ERR_INVALID_ARG, "out must hold a value and a scale buffer per copy")
    q = _fp8_copy(out, 0, M, K, block_rows) if rows else (None, 0, None)
    qt = _fp8_copy(out, 2 if rows else 0, K, M, block_rows) if cols else (None, 0, None)
    _check(lib.engram_fp8_quantise(x.data_ptr(), xd, M, K, _row_stride(x, "x"), block_rows,
                                   *q, *qt, _ptr(status), _stream(stream)), "engram_fp8_quantise")
    return tuple(out)


def engram_fp8_matmul(a, a_scale, b, b_scale, a_block: int = 1, b_block: int = 1, out=None,
                      out_dtype=None, status=None, stream=None):
    """out[m, n] = sum_k a[m, k] b[n, k]: a uint8 [M, K] and b uint8 [N, K] with their scale
    bytes, as engram_fp8_quantise returns them (a_block / b_block: FP8_BLOCK where 128 x 128
    tiles share a scale).  out: fp32 (default) or bf16 [M, N]."""
    (M, K, sa), (N, kb, sb) = _fp8_operand(a, "a"), _fp8_operand(b, "b")
    if kb != K:
        raise EngramError(ERR_INVALID_ARG, "a and b disagree on K")
    if a_block not in (1, FP8_BLOCK) or b_block not in (1, FP8_BLOCK):
        raise EngramError(ERR_INVALID_ARG, f"a_block and b_block must be 1 or {FP8_BLOCK}")
    pa = _fp8_scales(a_scale, M, K, a_block, "a_scale")
    pb = _fp8_scales(b_scale, N, K, b_block, "b_scale")
    if out is None:
        import torch
        out = _made(stream, torch.empty, (M, N), dtype=out_dtype or torch.float32,
                    device=a.device)
    od = _dtype(out, "out")
    if out.shape != (M, N):
        raise EngramError(ERR_INVALID_ARG, f"out must be {[M, N]}")
    _check(lib.engram_fp8_matmul(a.data_ptr(), sa, pa, a_block, b.data_ptr(), sb, pb, b_block, M,
                                 N, K, out.data_ptr(), od, _row_stride(out, "out"), _ptr(status),
                                 _stream(stream)), "engram_fp8_matmul")
    return out


def engram_gate_add_grad_workspace_bytes() -> int:
    return int(lib.engram_gate_add_grad_workspace_bytes())


def engram_gate_add_grad(k, state, streams_in, alpha, dy, eps: float = 1e-6, dx=None, dk=None,
                         dalpha=None, dk_dtype=None, workspace=None, stream=None):
    """The backward pass of engram_gate_add: k fp32 [..., D], state uint8 [tokens] or None
    (every token live), streams_in and dy bf16 [..., 4, D].  Returns (dx, dk, dalpha); dx may
    be dy itself."""
    import torch
    bf = (torch.bfloat16, torch.int16)
    _need(k, (torch.float32,), "k")
    _need(state, (torch.uint8,), "state")
    _need(streams_in, bf, "streams_in")
    _need(dy, bf, "dy")
    _need(alpha, (torch.float32,), "alpha")
    D = streams_in.shape[-1]
    if streams_in.dim() < 2 or streams_in.shape[-2] != 4 or dy.shape != streams_in.shape:
        raise EngramError(ERR_INVALID_ARG, "streams_in and dy must be [..., 4, D]")
    T = streams_in.numel() // (4 * D) if D else 0
    if k.numel() != T * D or (state is not None and state.numel() != T) or alpha.numel() != 4:
        raise EngramError(ERR_INVALID_ARG, "k / state / alpha sizes disagree with the streams")
    if dx is None:
        dx = _made(stream, torch.empty_like, dy)
    if dk is None:
        dk = _made(stream, torch.empty, k.shape, dtype=dk_dtype or torch.float32,
                   device=k.device)
    if dalpha is None:
        dalpha = _made(stream, torch.empty, 4, dtype=torch.float32, device=k.device)
    _need(dx, bf, "dx")
    _need(dk, (torch.float32, *bf), "dk")
    _need(dalpha, (torch.float32,), "dalpha")
    if dx.numel() != dy.numel() or dk.numel() != k.numel() or dalpha.numel() != 4:
        raise EngramError(ERR_INVALID_ARG, "dx / dk / dalpha sizes")
    if workspace is None:
        workspace = _made(stream, torch.empty, engram_gate_add_grad_workspace_bytes(),
                          dtype=torch.uint8, device=k.device, scratch=True)
    _need(workspace, (workspace.dtype,), "workspace")
    _check(lib.engram_gate_add_grad(_ptr(k), _ptr(state), T, D, _ptr(streams_in), _ptr(alpha),
                                    float(eps), _ptr(dy), _ptr(dx), _ptr(dk), _dtype(dk, "dk"),
                                    _ptr(dalpha), _ptr(workspace), workspace.numel(),
                                    _stream(stream)), "engram_gate_add_grad")
    return dx, dk, dalpha
