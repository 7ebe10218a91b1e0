"""Python binding of libmr (argument marshalling only; every step of the path runs in libmr's kernels).

The names follow the C-ABI in ``include/mr.h``: ``compress`` -> ``mr_compress``, ``retrieve`` ->
``mr_retrieve``, ``dense_ref`` -> ``mr_dense_ref``.  PyTorch is used for device memory and streams;
``send_map`` / ``recv_map`` move a compressed map between ranks with torch.distributed.
Importing this module loads ``libmr.so`` and raises ``ImportError`` if it has not been built:
there is no fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading
from typing import Optional

import numpy as np
import torch

# MR_LIBRARY=checked selects the bounds-checked build (libmr_checked.so): same API and results,
# with every global store of the tensor-core kernels checked against its extent on the device.
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        "libmr_checked.so" if os.environ.get("MR_LIBRARY") == "checked" else "libmr.so")

MR_OK, MR_ERR_INVALID_ARG, MR_ERR_UNSUPPORTED, MR_ERR_CAPACITY = 0, 1, 2, 3
MR_ERR_CUDA, MR_ERR_TIMEOUT, MR_ERR_DEVICE_CHECK, MR_ERR_RANGE = 4, 5, 6, 7
MR_BF16, MR_F32, MR_FP8_E4M3 = 0, 1, 2

_c_i32, _c_i64, _c_f32, _c_p, _c_sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class LogitBias(ctypes.Structure):
    _fields_ = [("sink_len", _c_i32), ("sink_bias", _c_f32), ("window", _c_i32), ("window_bias", _c_f32),
                ("kb_bias", _c_p), ("kb_block", _c_i32), ("n_kb", _c_i32)]


class RetrieveOpts(ctypes.Structure):
    _fields_ = [("qb_begin", _c_i32), ("qb_end", _c_i32), ("v_group", _c_i32), ("v_pages", _c_p),
                ("page_rows", _c_i32), ("pages_per_req", _c_i32)]


class BSR(ctypes.Structure):
    _fields_ = [("H_s", _c_i32), ("L", _c_i32), ("block", _c_i32), ("val_dtype", ctypes.c_int),
                ("capacity_tiles", _c_i64), ("row_ptr", _c_p), ("col_idx", _c_p), ("vals", _c_p),
                ("kept_mass", _c_p), ("kept_bits", _c_p), ("mass", _c_p), ("lse", _c_p), ("nnz", _c_p),
                ("tile_scale", _c_p), ("renormalised", _c_i32)]


class Rows(ctypes.Structure):
    _fields_ = [("ptr", _c_p), ("head_stride", _c_i64), ("row_stride", _c_i64)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", _c_p), ("v", _c_p), ("dt", ctypes.c_int), ("H_kv", _c_i32), ("page_rows", _c_i32),
                ("d", _c_i32), ("n_pages", _c_i64)]


class KvSeqs(ctypes.Structure):
    _fields_ = [("table", _c_p), ("kv_len", _c_p), ("pages_per_seq", _c_i32), ("n_seq", _c_i32)]


class RopeTable(ctypes.Structure):
    _fields_ = [("d", _c_i32), ("rot_dim", _c_i32), ("interleaved", _c_i32), ("mscale", _c_f32),
                ("turn", ctypes.c_uint64 * 128)]


EXPORTS = {
    "mr_version": ([], ctypes.c_int),
    "mr_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "mr_device_supported": ([], ctypes.c_int),
    "mr_checked_build": ([], ctypes.c_int),
    "mr_compress_workspace_bytes": ([ctypes.c_int] * 4, _c_sz),
    "mr_bsr_max_tiles": ([ctypes.c_int] * 3, _c_i64),
    "mr_compress": ([_c_p, _c_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _c_f32, _c_f32,
                     ctypes.POINTER(LogitBias), ctypes.POINTER(BSR), _c_p, _c_sz, _c_p], ctypes.c_int),
    "mr_compress_blocks": ([_c_p, _c_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _c_f32, _c_f32,
                            ctypes.POINTER(LogitBias), ctypes.c_int, ctypes.c_int, ctypes.POINTER(BSR), _c_p, _c_sz,
                            _c_p], ctypes.c_int),
    "mr_compress_noalloc": ([_c_p, _c_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _c_f32, _c_f32,
                             ctypes.POINTER(LogitBias), ctypes.POINTER(BSR), _c_p], ctypes.c_int),
    "mr_compress_noalloc_status": ([_c_p], ctypes.c_int),
    "mr_retrieve_workspace_bytes": ([ctypes.POINTER(BSR), ctypes.c_int, ctypes.c_int, ctypes.c_int], _c_sz),
    "mr_retrieve": ([ctypes.POINTER(BSR), _c_p, ctypes.c_int, _c_p, _c_i64, _c_p, ctypes.c_int, ctypes.c_int,
                     ctypes.c_int, _c_p, _c_i64, _c_i64, ctypes.POINTER(RetrieveOpts), _c_p, _c_sz, _c_p],
                    ctypes.c_int),
    "mr_dense_ref_workspace_bytes": ([ctypes.c_int], _c_sz),
    "mr_dense_ref": ([_c_p, _c_p, _c_p, _c_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                      _c_p, _c_p, _c_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, _c_f32,
                      ctypes.POINTER(LogitBias), _c_p, _c_sz, _c_p], ctypes.c_int),
    "mr_sync_status": ([_c_p, _c_p], ctypes.c_int),
    "mr_bsr_nnz": ([ctypes.POINTER(BSR), ctypes.POINTER(_c_i64), _c_p], ctypes.c_int),
    "mr_bsr_export": ([ctypes.POINTER(BSR), _c_i64, _c_p, _c_p], ctypes.c_int),
    "mr_bm_create": ([ctypes.c_int, _c_i64], _c_p),
    "mr_bm_destroy": ([_c_p], None),
    "mr_bm_insert": ([_c_p, _c_p, ctypes.c_int, ctypes.POINTER(BSR), ctypes.c_int, _c_i64], _c_i64),
    "mr_bm_lookup": ([_c_p, _c_p, ctypes.c_int, ctypes.POINTER(_c_i64)], ctypes.c_int),
    "mr_bm_map": ([_c_p, _c_i64, ctypes.c_int, ctypes.POINTER(BSR)], ctypes.c_int),
    "mr_bm_release": ([_c_p, _c_i64], ctypes.c_int),
    "mr_bm_evicted": ([_c_p, ctypes.POINTER(_c_i64), ctypes.c_int], ctypes.c_int),
    "mr_bm_stats": ([_c_p, ctypes.POINTER(_c_i64)], ctypes.c_int),
    "mr_rope_init": ([ctypes.POINTER(RopeTable), ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_double, ctypes.c_int,
                      ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double, ctypes.c_double, _c_p],
                     ctypes.c_int),
    "mr_rope_apply": ([ctypes.POINTER(RopeTable), ctypes.POINTER(Rows), ctypes.POINTER(Rows), ctypes.c_int,
                       ctypes.c_int, ctypes.c_int, _c_p, ctypes.c_int, _c_p], ctypes.c_int),
    "mr_paged_workspace_bytes": ([ctypes.POINTER(KvCache), ctypes.c_int, ctypes.c_int], _c_sz),
    "mr_kv_append": ([ctypes.POINTER(KvCache), ctypes.POINTER(KvSeqs), ctypes.POINTER(RopeTable), ctypes.POINTER(Rows),
                      ctypes.POINTER(Rows), ctypes.c_int, ctypes.POINTER(Rows), ctypes.POINTER(Rows), _c_p, ctypes.c_int,
                      _c_p, _c_sz, _c_p], ctypes.c_int),
    "mr_paged_decode": ([ctypes.POINTER(KvCache), ctypes.POINTER(KvSeqs), ctypes.POINTER(Rows), ctypes.c_int, _c_f32,
                         ctypes.c_int, ctypes.c_int, ctypes.POINTER(Rows), _c_p, _c_p, _c_sz, _c_p], ctypes.c_int),
    "mr_paged_attn": ([ctypes.POINTER(KvCache), ctypes.POINTER(KvSeqs), ctypes.POINTER(Rows), ctypes.c_int, _c_p,
                       ctypes.c_int, _c_f32, ctypes.c_int, ctypes.c_int, ctypes.POINTER(Rows), _c_p, _c_p, _c_sz, _c_p],
                      ctypes.c_int),
    "mr_pages_copy_workspace_bytes": ([], _c_sz),
    "mr_pages_copy": ([ctypes.POINTER(_c_p), ctypes.c_int, _c_i64, _c_i64, _c_p, ctypes.c_int, _c_p, _c_sz, _c_p],
                      ctypes.c_int),
    "mr_pp_create": ([ctypes.c_int, ctypes.c_int], _c_p),
    "mr_pp_destroy": ([_c_p], None),
    "mr_pp_open": ([_c_p], _c_i64),
    "mr_pp_fork": ([_c_p, _c_i64, ctypes.c_int], _c_i64),
    "mr_pp_extend": ([_c_p, _c_i64, ctypes.c_int, _c_p], ctypes.c_int),
    "mr_pp_truncate": ([_c_p, _c_i64, ctypes.c_int], ctypes.c_int),
    "mr_pp_slide": ([_c_p, _c_i64, ctypes.c_int, ctypes.c_int], ctypes.c_int),
    "mr_pp_close": ([_c_p, _c_i64], ctypes.c_int),
    "mr_pp_compact": ([_c_p, _c_p, ctypes.c_int], ctypes.c_int),
    "mr_pp_table": ([_c_p, _c_i64, _c_p, ctypes.c_int, ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
    "mr_pp_stats": ([_c_p, ctypes.POINTER(_c_i64)], ctypes.c_int),
    "mr_gather_probe": ([ctypes.POINTER(BSR), ctypes.c_int, ctypes.c_int, _c_p, _c_sz, _c_p], ctypes.c_int),
    "mr_debug_set": ([ctypes.c_uint64, ctypes.c_int], ctypes.c_int),
    "mr_profile_enable": ([ctypes.c_int], ctypes.c_int),
    "mr_profile_read": ([_c_p, _c_p, ctypes.c_int], ctypes.c_int),
    "mr_kernel_name": ([ctypes.c_int], ctypes.c_char_p),
    "mr_kernel_launches": ([], _c_i64),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in EXPORTS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


LIB = _load()


class MRError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {LIB.mr_status_string(code).decode()} (status {code})")


def check(code: int, where: str) -> None:
    if code != MR_OK:
        raise MRError(code, where)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MR_BF16
    if t.dtype == torch.float32:
        return MR_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _torch_dtype(dt: int):
    return {MR_BF16: torch.bfloat16, MR_F32: torch.float32, MR_FP8_E4M3: torch.uint8}[dt]


def fp8_scales_per_tile(block: int) -> int:
    """Scales of an fp8 tile: one per 32-row x 64-key piece."""
    return (block // 32) * (block // 64)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:  # (an eighth of the time of building a Stream object)
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


class Workspace:
    """Device workspace (256-byte aligned torch allocation)."""

    def __init__(self, nbytes: int, device="cuda"):
        self.nbytes = max(256, int(nbytes))
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self.buf.data_ptr()) % 256
        self.ptr = self.buf.data_ptr() + off

    def sync_status(self, stream=None) -> int:
        """Status of the last call on this workspace, after all work on ``stream`` (default: the current stream of the
        workspace's device, whichever device is current)."""
        with _on(self.buf, stream):
            return LIB.mr_sync_status(self.ptr, _stream(None))


class Bias:
    """Device-side logit bias (holds the kb_bias tensor alive)."""

    def __init__(self, sink_len=0, sink_bias=0.0, window=0, window_bias=0.0, kb_bias=None,
                 kb_block=0, device="cuda"):
        self.kb = None
        if kb_bias is not None:
            kb = torch.as_tensor(np.ascontiguousarray(kb_bias, dtype=np.float32))
            self.kb = kb.to(device).contiguous()
        self.c = LogitBias(int(sink_len), float(sink_bias), int(window), float(window_bias),
                           self.kb.data_ptr() if self.kb is not None else None,
                           int(kb_block) if self.kb is not None else 0,
                           int(self.kb.shape[1]) if self.kb is not None else 0)

    @classmethod
    def from_spec(cls, b, device="cuda"):
        if b is None:
            return None
        return cls(b.sink_len, b.sink_bias, b.window, b.window_bias, b.kb_bias, b.kb_block, device)


def _bias_ptr(bias: Optional[Bias]):
    return ctypes.byref(bias.c) if bias is not None else None


class Map:
    """A compressed map: caller-owned device arrays described by an ``mr_bsr``."""

    def __init__(self, H_s: int, L: int, block: int, dtype: int, capacity: int, device="cuda",
                 store_mass: bool = False, store_lse: bool = False, renormalised: bool = False):
        self.H_s, self.L, self.block, self.dtype, self.capacity = H_s, L, block, dtype, int(capacity)
        self.nqb = L // block
        self.nkw = (self.nqb + 31) // 32
        n = H_s * self.nqb
        dev = device
        self.row_ptr = torch.zeros(n + 1, dtype=torch.int32, device=dev)
        self.col_idx = torch.zeros(max(1, self.capacity), dtype=torch.int32, device=dev)
        self.vals = torch.zeros((max(1, self.capacity), block, block), dtype=_torch_dtype(dtype), device=dev)
        self.kept_mass = torch.zeros(n, dtype=torch.float32, device=dev)
        self.kept_bits = torch.zeros((n, self.nkw), dtype=torch.int32, device=dev)
        self.mass = torch.zeros((n, self.nqb), dtype=torch.float32, device=dev) if store_mass else None
        self.lse = torch.zeros((H_s, L), dtype=torch.float32, device=dev) if store_lse else None
        self.nnz = torch.zeros(1, dtype=torch.int64, device=dev)
        self.tile_scale = (torch.zeros((max(1, self.capacity), fp8_scales_per_tile(block)), dtype=torch.float32,
                                       device=dev) if dtype == MR_FP8_E4M3 else None)
        self.c = BSR(H_s, L, block, dtype, self.capacity, self.row_ptr.data_ptr(), self.col_idx.data_ptr(),
                     self.vals.data_ptr(), self.kept_mass.data_ptr(), self.kept_bits.data_ptr(),
                     self.mass.data_ptr() if self.mass is not None else None,
                     self.lse.data_ptr() if self.lse is not None else None, self.nnz.data_ptr(),
                     self.tile_scale.data_ptr() if self.tile_scale is not None else None,
                     1 if renormalised else 0)

    def nnz_host(self, stream=None) -> int:
        v = _c_i64(0)
        check(LIB.mr_bsr_nnz(ctypes.byref(self.c), ctypes.byref(v), _stream(stream)), "mr_bsr_nnz")
        return int(v.value)

    def kept_bits_host(self) -> np.ndarray:
        """Kept flags [H_s][nqb][nkb] as uint8 (host copy)."""
        w = self.kept_bits.cpu().numpy().view(np.uint32).reshape(self.H_s, self.nqb, self.nkw)
        bits = ((w[..., :, None] >> np.arange(32, dtype=np.uint32)) & 1).astype(np.uint8)
        return bits.reshape(self.H_s, self.nqb, self.nkw * 32)[..., : self.nqb]

    def to(self, device) -> "Map":
        """A copy of this map on `device` (same capacity and flags), e.g. to move a received map
        from host memory onto the GPU that retrieves from it."""
        m = Map(self.H_s, self.L, self.block, self.dtype, max(1, self.capacity), device, self.mass is not None,
                self.lse is not None, bool(self.c.renormalised))
        m.capacity = self.capacity
        m.c.capacity_tiles = self.capacity
        pairs = [(m.row_ptr, self.row_ptr), (m.col_idx, self.col_idx), (m.vals, self.vals),
                 (m.kept_mass, self.kept_mass), (m.kept_bits, self.kept_bits), (m.nnz, self.nnz)]
        for opt in ("mass", "lse", "tile_scale"):
            if getattr(self, opt) is not None:
                pairs.append((getattr(m, opt), getattr(self, opt)))
        for dst, src in pairs:
            dst.copy_(src)
        return m

    def export(self, n_tiles: Optional[int] = None, stream=None) -> torch.Tensor:
        n = self.nnz_host(stream) if n_tiles is None else int(n_tiles)
        n = min(n, self.capacity)
        out = torch.empty((max(1, n), self.block, self.block), dtype=torch.float32, device=self.vals.device)
        check(LIB.mr_bsr_export(ctypes.byref(self.c), n, out.data_ptr(), _stream(stream)), "mr_bsr_export")
        return out[:n]


# ------------------------------------------------------------------------------------------------
# Moving a compressed map to another rank (MapFlow section 5.3: the sender's compressed maps are
# shipped to the receiver instance, which then runs the fused retrieval locally).
# torch.distributed point-to-point: NCCL between GPUs, gloo between CPU ranks.
# ------------------------------------------------------------------------------------------------
def _map_arrays(m: "Map", n_stored: int):
    arrays = [m.row_ptr, m.kept_bits, m.kept_mass]
    if n_stored > 0:
        # bf16 travels as its bit pattern, so every backend moves it unchanged
        vals = m.vals[:n_stored]
        arrays += [m.col_idx[:n_stored], vals.view(torch.int16) if vals.dtype == torch.bfloat16 else vals]
        if m.tile_scale is not None:
            arrays.append(m.tile_scale[:n_stored])
    return arrays


def send_map(m: "Map", dst: int, group=None) -> None:
    """Send the arrays the retrieval reads: row pointers, kept bits and masses, and the column
    indices and values of the stored tiles (min(kept tiles, capacity) of them)."""
    import torch.distributed as dist
    nnz = int(m.nnz.item())
    n = min(nnz, m.capacity)
    hdr = torch.tensor([m.H_s, m.L, m.block, m.dtype, nnz, n], dtype=torch.int64, device=m.row_ptr.device)
    dist.send(hdr, dst, group=group)
    for t in _map_arrays(m, n):
        dist.send(t.contiguous(), dst, group=group)


def recv_map(src: int, device="cuda", group=None) -> "Map":
    """Receive a map sent by send_map into a new Map on `device` whose capacity is the number of
    stored tiles; the kept-tile count is the sender's (tiles past the sender's capacity stay
    unstored, as they were)."""
    import torch.distributed as dist
    hdr = torch.empty(6, dtype=torch.int64, device=device)
    dist.recv(hdr, src, group=group)
    H_s, L, block, dtype, nnz, n = (int(x) for x in hdr.tolist())
    m = Map(H_s, L, block, dtype, max(1, n), device)
    m.capacity = n
    m.c.capacity_tiles = n
    for t in _map_arrays(m, n):
        dist.recv(t, src, group=group)
    m.nnz.fill_(nnz)
    return m


# ------------------------------------------------------------------------------------------------
# One sequence split across ranks by query-block range (MapFlow section 6: distributed settings).
# Compression units (head, query block) and retrieval rows are independent once every key and
# value row up to the range's end is present, so the only exchange is an all-gather of the
# ranks' K and V row shards; maps and outputs stay on their rank.
# ------------------------------------------------------------------------------------------------
def split_query_blocks(nqb: int, world: int, align: int = 1):
    """Contiguous ranges [(qb_begin, qb_end)] of the nqb query blocks, one per rank, balanced by
    causal work (query block I costs I + 1 key blocks).  Cuts fall on multiples of ``align``
    (2 for block 64, whose kernels work on pairs of query blocks); a rank may get an empty range
    when there are fewer aligned pieces than ranks."""
    if nqb < 1 or world < 1 or align < 1:
        raise ValueError("need nqb, world, align >= 1")
    cum = np.concatenate([[0.0], np.cumsum(np.arange(1, nqb + 1, dtype=np.float64))])  # work before cut c
    total = cum[-1]
    cands = sorted(set(list(range(0, nqb + 1, align)) + [nqb]))
    cuts = [0]
    for r in range(1, world):
        target = total * r / world
        # the aligned cut whose prefix work is closest to the target, never before the previous cut
        best = min((c for c in cands if c >= cuts[-1]), key=lambda c: abs(cum[c] - target))
        cuts.append(best)
    cuts.append(nqb)
    return [(cuts[r], cuts[r + 1]) for r in range(world)]


def row_shards(L: int, ranges, block: int):
    """Token rows [(row_begin, row_end)] of each rank's query-block range."""
    return [(q0 * block, q1 * block) for q0, q1 in ranges]


def gather_row_shards(local: torch.Tensor, shards, group=None) -> torch.Tensor:
    """All-gather of per-rank row shards [H][rows_r][d] into the full [H][L][d] on every rank
    (torch.distributed: NCCL between GPUs, gloo between CPU ranks).  Shards are padded to the
    longest one so every rank sends the same number of bytes."""
    import torch.distributed as dist
    H, _, d = local.shape
    longest = max(e - b for b, e in shards)
    L = shards[-1][1]
    pad = torch.zeros((H, longest, d), dtype=local.dtype, device=local.device)
    pad[:, : local.shape[1]] = local
    parts = [torch.empty_like(pad) for _ in shards]
    dist.all_gather(parts, pad.contiguous(), group=group)
    full = torch.empty((H, L, d), dtype=local.dtype, device=local.device)
    for (b, e), part in zip(shards, parts):
        full[:, b:e] = part[:, : e - b]
    return full


def max_tiles(H_s: int, L: int, block: int) -> int:
    return int(LIB.mr_bsr_max_tiles(H_s, L, block))


def compress_workspace_bytes(H_s, L, d, block) -> int:
    return int(LIB.mr_compress_workspace_bytes(H_s, L, d, block))


def compress(Q: torch.Tensor, K: torch.Tensor, p: float, block: int, bias: Optional[Bias] = None,
             scale: Optional[float] = None, capacity: Optional[int] = None, out: Optional[Map] = None,
             ws: Optional[Workspace] = None, store_mass=False, store_lse=False, stream=None,
             blocks: Optional[tuple] = None, map_dtype: Optional[int] = None,
             renormalised: bool = False) -> Map:
    """mr_compress: Q, K [H_s][L][d] (bf16 or fp32, CUDA) -> Map.  ``blocks=(qb_begin, qb_end)``
    calls mr_compress_blocks: only those query blocks, the other rows of the map left empty.
    ``map_dtype=MR_FP8_E4M3`` stores e4m3 values with per-piece scales (bf16 inputs);
    ``renormalised=True`` stores each row divided by its kept mass."""
    _need_cuda(Q, K)
    H, L, d = Q.shape
    dt = _dt(Q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        cap = max_tiles(H, L, block) if capacity is None else capacity
        out = Map(H, L, block, dt if map_dtype is None else map_dtype, cap, Q.device, store_mass, store_lse,
                  renormalised)
    if ws is None:
        ws = Workspace(compress_workspace_bytes(H, L, d, block), Q.device)
    out.ws = ws
    if blocks is None:
        check(LIB.mr_compress(Q.data_ptr(), K.data_ptr(), dt, H, L, d, float(scale), float(p), _bias_ptr(bias),
                              ctypes.byref(out.c), ws.ptr, ws.nbytes, _stream(stream)), "mr_compress")
    else:
        check(LIB.mr_compress_blocks(Q.data_ptr(), K.data_ptr(), dt, H, L, d, float(scale), float(p),
                                     _bias_ptr(bias), int(blocks[0]), int(blocks[1]), ctypes.byref(out.c), ws.ptr,
                                     ws.nbytes, _stream(stream)), "mr_compress_blocks")
    return out


def retrieve_workspace_bytes(m: Map, H_r: int, d_v: int, n_req: int) -> int:
    return int(LIB.mr_retrieve_workspace_bytes(ctypes.byref(m.c), H_r, d_v, n_req))


def retrieve(m: Map, W: torch.Tensor, V: torch.Tensor, out: Optional[torch.Tensor] = None,
             v_req_off: Optional[torch.Tensor] = None, v_req_stride: Optional[int] = None,
             v_head_stride: Optional[int] = None, n_req: Optional[int] = None,
             ws: Optional[Workspace] = None, stream=None, blocks: Optional[tuple] = None,
             v_group: int = 1, v_elems: Optional[int] = None, v_pages: Optional[torch.Tensor] = None,
             page_rows: int = 0) -> torch.Tensor:
    """mr_retrieve: W [H_r][H_s] fp32; V [H_v][L][d_v] or [n_req][H_v][L][d_v] (or a packed buffer
    with explicit strides/offsets), H_v = H_r / v_group -> O [n_req][H_r][L][d_v].
    ``blocks=(qb_begin, qb_end)`` writes only those query blocks' rows of O; ``v_elems`` defaults to
    the number of elements of V.  ``v_pages`` [n_req][pages_per_req] (int32, device) reads V as a
    pool of pages [page][H_v][page_rows][d_v]."""
    _need_cuda(W, V, v_req_off, v_pages)
    H_r = W.shape[0]
    dt = _dt(V)
    d_v = V.shape[-1]
    if v_head_stride is None:
        v_head_stride = V.shape[-2] * d_v
    if n_req is None:
        n_req = V.shape[0] if V.dim() == 4 else 1
    if v_req_stride is None:
        v_req_stride = (H_r // max(1, v_group)) * v_head_stride
    if v_elems is None:
        v_elems = V.numel()
    if out is None:
        out = torch.empty((n_req, H_r, m.L, d_v), dtype=V.dtype, device=V.device)
    _need_cuda(out)
    if ws is None:
        ws = Workspace(retrieve_workspace_bytes(m, H_r, d_v, n_req), V.device)
    opts = None
    if blocks is not None or v_group != 1 or v_pages is not None:
        b = blocks if blocks is not None else (0, 0)
        opts = ctypes.byref(RetrieveOpts(int(b[0]), int(b[1]), int(v_group),
                                         v_pages.data_ptr() if v_pages is not None else None, int(page_rows),
                                         int(v_pages.shape[1]) if v_pages is not None else 0))
    check(LIB.mr_retrieve(ctypes.byref(m.c), W.data_ptr(), H_r, V.data_ptr(), int(v_elems), out.data_ptr(), dt,
                          d_v, n_req, v_req_off.data_ptr() if v_req_off is not None else None, int(v_req_stride),
                          int(v_head_stride), opts, ws.ptr, ws.nbytes, _stream(stream)), "mr_retrieve")
    return out


def dense_ref(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
              q_offset: Optional[torch.Tensor], total_q: int, total_k: int, bias: Optional[Bias] = None,
              scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
              ws: Optional[Workspace] = None, stream=None) -> torch.Tensor:
    """mr_dense_ref: packed Q [H][total_q][d], K/V [H][total_k][d] -> O [H][total_q][d_v]."""
    _need_cuda(Q, K, V, cu_q, cu_k, q_offset)
    H, _, d = Q.shape
    d_v = V.shape[-1]
    n_seq = cu_q.shape[0] - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((H, total_q, d_v), dtype=V.dtype, device=V.device)
    if ws is None:
        ws = Workspace(int(LIB.mr_dense_ref_workspace_bytes(n_seq)), Q.device)
    check(LIB.mr_dense_ref(Q.data_ptr(), K.data_ptr(), V.data_ptr(), out.data_ptr(), _dt(Q), H, d, d_v,
                           cu_q.data_ptr(), cu_k.data_ptr(),
                           q_offset.data_ptr() if q_offset is not None else None, n_seq, int(total_q),
                           int(total_k), float(scale), _bias_ptr(bias), ws.ptr, ws.nbytes, _stream(stream)),
          "mr_dense_ref")
    return out


def gather_probe(m: "Map", readers: int, ws: Optional[Workspace] = None, stream=None, ring_slots: int = 8) -> None:
    """mr_gather_probe: the retrieval's map reads alone (measurement)."""
    if ws is None:
        ws = Workspace(256, m.vals.device)
    check(LIB.mr_gather_probe(ctypes.byref(m.c), int(readers), int(ring_slots), ws.ptr, ws.nbytes, _stream(stream)),
          "mr_gather_probe")


def profile_enable(on: bool = True) -> bool:
    return bool(LIB.mr_profile_enable(1 if on else 0))


def profile_read() -> dict:
    """{kernel name: (total ms, launches)} for kernels launched since profiling was enabled."""
    n = 64
    ms = (ctypes.c_double * n)()
    cnt = (_c_i64 * n)()
    k = LIB.mr_profile_read(ctypes.cast(ms, _c_p), ctypes.cast(cnt, _c_p), n)
    out = {}
    for i in range(min(k, n)):
        if cnt[i]:
            out[LIB.mr_kernel_name(i).decode()] = (float(ms[i]), int(cnt[i]))
    return out


def kernel_launches() -> int:
    return int(LIB.mr_kernel_launches())


def compress_noalloc(Q: torch.Tensor, K: torch.Tensor, p: float, out: Map, bias: Optional[Bias] = None,
                     scale: Optional[float] = None, stream=None) -> Map:
    """mr_compress_noalloc: as compress, with the library's fixed scratch instead of a workspace."""
    _need_cuda(Q, K)
    H, L, d = Q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    check(LIB.mr_compress_noalloc(Q.data_ptr(), K.data_ptr(), _dt(Q), H, L, d, float(scale), float(p),
                                  _bias_ptr(bias), ctypes.byref(out.c), _stream(stream)), "mr_compress_noalloc")
    return out


def compress_noalloc_status(stream=None) -> int:
    """mr_compress_noalloc_status: device status of the last allocation-free compression."""
    return int(LIB.mr_compress_noalloc_status(_stream(stream)))



class BlockManager:
    """mr_bm_*: prefix-hash index from token prefixes to stored maps (MapFlow section 5.3).

    ``insert(tokens, maps)`` registers the per-layer maps of one sequence (the Map objects are kept
    alive here until their entry is evicted and collected by ``collect_evicted``);
    ``lookup(tokens)`` returns (reusable query blocks, entry id); ``map(entry, layer)`` gives a Map
    view to pass to ``retrieve(..., blocks=(0, k))``."""

    def __init__(self, block: int, budget_bytes: int = 0):
        self.h = LIB.mr_bm_create(int(block), int(budget_bytes))
        if not self.h:
            raise MRError(MR_ERR_INVALID_ARG, "mr_bm_create")
        self.block = block
        self._maps = {}

    def __del__(self):
        if getattr(self, "h", None):
            LIB.mr_bm_destroy(self.h)
            self.h = None

    def insert(self, tokens, maps, map_bytes: Optional[int] = None) -> int:
        tok = np.ascontiguousarray(tokens, dtype=np.int32)
        arr = (BSR * len(maps))(*[m.c for m in maps])
        if map_bytes is None:
            map_bytes = sum(m.vals.numel() * m.vals.element_size() for m in maps)
        eid = int(LIB.mr_bm_insert(self.h, tok.ctypes.data_as(_c_p), int(tok.shape[0]), arr, len(maps),
                                   int(map_bytes)))
        if eid < 0:
            raise MRError(-eid, "mr_bm_insert")
        self._maps[eid] = list(maps)
        return eid

    def lookup(self, tokens):
        tok = np.ascontiguousarray(tokens, dtype=np.int32)
        e = _c_i64(-1)
        k = int(LIB.mr_bm_lookup(self.h, tok.ctypes.data_as(_c_p), int(tok.shape[0]), ctypes.byref(e)))
        if k < 0:
            raise MRError(-k, "mr_bm_lookup")
        return k, int(e.value)

    def map(self, entry: int, layer: int) -> "Map":
        d = BSR()
        check(LIB.mr_bm_map(self.h, int(entry), int(layer), ctypes.byref(d)), "mr_bm_map")
        m = self._maps[entry][layer]
        assert m.c.vals == d.vals  # the descriptor is the registered map's
        return m

    def release(self, entry: int) -> None:
        check(LIB.mr_bm_release(self.h, int(entry)), "mr_bm_release")

    def collect_evicted(self):
        """Ids evicted since the last call; their Map objects (device arrays) are dropped here."""
        ids = (_c_i64 * 64)()
        out = []
        while True:
            n = int(LIB.mr_bm_evicted(self.h, ids, 64))
            out += [int(ids[i]) for i in range(n)]
            if n < 64:
                break
        for i in out:
            self._maps.pop(i, None)
        return out

    def stats(self) -> dict:
        v = (_c_i64 * 5)()
        check(LIB.mr_bm_stats(self.h, v), "mr_bm_stats")
        return dict(zip(("entries", "bytes", "lookups", "hits", "hit_blocks"), [int(x) for x in v]))


# ------------------------------------------------------------------------------------------------
# The receiver's paged key-value cache (MapFlow section 6): rotary positions, appending rows,
# attention of new rows over the cache, copying pages, and the host-side page pool.
# These calls run on the device of their tensors, whichever device is current.  What they find wrong on the device (pages
# outside the pool, lengths beyond the table, conflicting pairs) is in the workspace's status: ``ws.sync_status()``, or
# ``last_status()`` for a call that was given no workspace.
# ------------------------------------------------------------------------------------------------
_NO_SWITCH = contextlib.nullcontext()


def _on(t: torch.Tensor, stream):
    """Context for a call on the tensors of t's device: that device is current (the library launches on the current
    one), and `stream`, where given, is the current stream, so that outputs and workspaces made here belong to it."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be CUDA tensors")
    if stream is None:
        return _NO_SWITCH if index == torch.cuda.current_device() else torch.cuda.device(index)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index) if stream else torch.cuda.default_stream(index)
    if stream.device.index != index:
        raise ValueError(f"the stream is not on {t.device}")
    return torch.cuda.stream(stream)


def _rows(t: torch.Tensor, like: torch.Tensor, what: str) -> Rows:
    """mr_rows of a [heads][rows][d] tensor with any strides over heads and rows."""
    stride = t.stride()
    if len(stride) != 3 or (stride[2] != 1 and t.shape[2] > 1):
        raise ValueError(f"{what} must be [heads][rows][d] with adjacent elements in a row")
    if t.dtype != like.dtype:
        raise TypeError(f"{what} must have dtype {like.dtype}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{what} must be on {like.device}")
    return Rows(t.data_ptr(), stride[0], stride[1])


def _new_like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _ints(t: torch.Tensor, like: torch.Tensor, what: str, dim: int = 1) -> int:
    """Address of a contiguous int32 tensor on the device of `like`."""
    if t.dtype is not torch.int32 or t.dim() != dim or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of {dim} dimension(s)")
    if t.get_device() != like.get_device():
        raise ValueError(f"{what} must be on {like.device}")
    return t.data_ptr()


class Rope:
    """Rotary positions of the first `rot_dim` of d elements (mr_rope_init).  ``scaling`` is "none",
    "linear", "base" or "ramp" with ``factor`` (and ``orig_len``, ``beta_slow``, ``beta_fast`` for the
    ramp); ``inv_freq`` gives the angles per position directly.  Host data only: keep and reuse it."""

    SCALING = {"none": 0, "linear": 1, "base": 2, "ramp": 3}

    def __init__(self, d: int, rot_dim: Optional[int] = None, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, orig_len: int = 0, beta_slow: float = 1.0,
                 beta_fast: float = 32.0, mscale: float = 1.0, inv_freq=None):
        self.d, self.rot_dim = int(d), int(d if rot_dim is None else rot_dim)
        if scaling not in self.SCALING:
            raise ValueError(f"scaling must be one of {sorted(self.SCALING)}")
        freq = None
        if inv_freq is not None:
            freq = np.ascontiguousarray(inv_freq, dtype=np.float64)
            if freq.shape != (self.rot_dim // 2,):
                raise ValueError("inv_freq must hold rot_dim / 2 angles")
        self.c = RopeTable()
        check(LIB.mr_rope_init(ctypes.byref(self.c), self.d, self.rot_dim, int(interleaved), float(base),
                               self.SCALING[scaling], float(factor), int(orig_len), float(beta_slow), float(beta_fast),
                               float(mscale), freq.ctypes.data if freq is not None else None), "mr_rope_init")


def rope(r: Rope, X: torch.Tensor, pos: torch.Tensor, out: Optional[torch.Tensor] = None, adjoint: bool = False,
         stream=None) -> torch.Tensor:
    """mr_rope_apply: X [H][rows][d] (any strides over heads and rows) rotated by each row's position
    (int32, device).  ``out=X`` rotates in place; ``adjoint=True`` gives the gradient with respect to X
    for a gradient with respect to the result."""
    with _on(X, stream):
        dt = _dt(X)
        x = _rows(X, X, "X")
        H, n, d = X.shape
        if d != r.d:
            raise ValueError(f"rows of {d} elements, rotation for {r.d}")
        if pos.shape[0] != n:
            raise ValueError("pos must give one position per row")
        if out is None:
            out = _new_like(X)
        elif out.shape != X.shape:
            raise ValueError("out must have the shape of X")
        check(LIB.mr_rope_apply(ctypes.byref(r.c), ctypes.byref(x), ctypes.byref(_rows(out, X, "out")), dt, H, n,
                                _ints(pos, X, "pos"), 1 if adjoint else 0, _stream(None)), "mr_rope_apply")
    return out


class KVCache:
    """A pool of pages: k and v, each [n_pages][H_kv][page_rows][d] (bf16 or fp32, contiguous, CUDA)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        _need_cuda(k, v)
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must both be [n_pages][H_kv][page_rows][d], of one dtype, on one device")
        self.k, self.v = k, v
        self.n_pages, self.H_kv, self.page_rows, self.d = k.shape
        self.c = KvCache(k.data_ptr(), v.data_ptr(), _dt(k), self.H_kv, self.page_rows, self.d, self.n_pages)

    @classmethod
    def empty(cls, n_pages: int, H_kv: int, page_rows: int, d: int, dtype=torch.bfloat16, device="cuda") -> "KVCache":
        """A new cache whose pages hold nothing yet."""
        shape = (n_pages, H_kv, page_rows, d)
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device))


def _ws_for(ws: Optional[Workspace], nbytes, t: torch.Tensor) -> Workspace:
    """The caller's workspace (it must be on the device of t), or a new one of nbytes() bytes."""
    if ws is None:
        return Workspace(nbytes(), t.device)
    if ws.buf.get_device() != t.get_device():
        raise ValueError(f"the workspace must be on {t.device}")
    return ws


_made = threading.local()  # workspace and stream of this thread's last call that made its own


def _keep(given: Optional[Workspace], ws: Workspace) -> None:
    if given is None:
        _made.last = ws, _stream(None)


def last_status(stream=None) -> int:
    """Device status of this thread's last kv_append, paged_decode, paged_attn or pages_copy that was given no
    workspace, after all work on ``stream`` (default: the call's own).  That workspace is kept until the next such call."""
    last = getattr(_made, "last", None)
    if last is None:
        raise ValueError("no call without a workspace was made")
    ws, own = last
    return ws.sync_status(own if stream is None else stream)


def _seqs(cache: KVCache, table: torch.Tensor, kv_len: torch.Tensor) -> KvSeqs:
    n = kv_len.shape[0]
    t, l = _ints(table, cache.k, "table", 2), _ints(kv_len, cache.k, "kv_len")
    if table.shape[0] != n:
        raise ValueError("table must have one row per sequence")
    return KvSeqs(t, l, table.shape[1], n)


def paged_workspace_bytes(cache: KVCache, H_q: int, n_seq: int) -> int:
    return int(LIB.mr_paged_workspace_bytes(ctypes.byref(cache.c), int(H_q), int(n_seq)))


def kv_append(cache: KVCache, table: torch.Tensor, kv_len: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
              cu_q: Optional[torch.Tensor] = None, rope: Optional[Rope] = None, Q: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, ws: Optional[Workspace] = None,
              stream=None) -> Optional[torch.Tensor]:
    """mr_kv_append: store the new rows K, V [H_kv][total_q][d] (K rotated) in the pages that table
    [n_seq][pages_per_seq] names, ending at kv_len [n_seq], and return Q [H_q][total_q][d] rotated (None
    without Q; ``q_out=Q`` rotates in place).  ``cu_q`` [n_seq + 1]: rows of each sequence (None: one each)."""
    with _on(cache.k, stream):
        k, v = _rows(K, cache.k, "K"), _rows(V, cache.k, "V")
        total = K.shape[1]
        if K.shape != V.shape or K.shape[0] != cache.H_kv or K.shape[2] != cache.d:
            raise ValueError("K and V must be [H_kv][total_q][d] of the cache")
        q = qo = None
        H_q = 0
        if Q is not None:
            H_q = Q.shape[0]
            if Q.shape[1:] != K.shape[1:]:
                raise ValueError("Q must be [H_q][total_q][d]")
            if q_out is None:
                q_out = _new_like(Q)
            elif q_out.shape != Q.shape:
                raise ValueError("q_out must have the shape of Q")
            q, qo = ctypes.byref(_rows(Q, cache.k, "Q")), ctypes.byref(_rows(q_out, cache.k, "q_out"))
        elif q_out is not None:
            raise ValueError("q_out without Q")
        seqs = _seqs(cache, table, kv_len)
        if cu_q is not None and cu_q.shape[0] != seqs.n_seq + 1:
            raise ValueError("cu_q must have n_seq + 1 entries")
        given, ws = ws, _ws_for(ws, lambda: 0, cache.k)  # (the status word is all this call needs)
        check(LIB.mr_kv_append(ctypes.byref(cache.c), ctypes.byref(seqs), ctypes.byref(rope.c) if rope else None, q, qo,
                               H_q, ctypes.byref(k), ctypes.byref(v),
                               _ints(cu_q, cache.k, "cu_q") if cu_q is not None else None, total, ws.ptr, ws.nbytes,
                               _stream(None)), "mr_kv_append")
        _keep(given, ws)
    return q_out


def _attn_out(Q: torch.Tensor, out, lse, return_lse: bool):
    """Output and log-normaliser tensors of an attention call on Q [H_q][rows][d]."""
    H, n, _ = Q.shape
    if out is None:
        out = _new_like(Q)
    elif out.shape != Q.shape:
        raise ValueError("out must have the shape of Q")
    if lse is not None:
        if lse.shape != (H, n) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != Q.device:
            raise ValueError("lse must be a contiguous fp32 tensor [H_q][rows]")
    elif return_lse:
        lse = torch.empty((H, n), dtype=torch.float32, device=Q.device)
    return out, lse


def paged_decode(cache: KVCache, table: torch.Tensor, kv_len: torch.Tensor, Q: torch.Tensor,
                 scale: Optional[float] = None, window: int = 0, sinks: int = 0, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, return_lse: bool = False, ws: Optional[Workspace] = None,
                 stream=None):
    """mr_paged_decode: attention of one new token per sequence, Q [H_q][n_seq][d], over the kv_len [n_seq]
    rows that table [n_seq][pages_per_seq] names -> O [H_q][n_seq][d], or (O, lse [H_q][n_seq]) with
    ``return_lse`` or an ``lse`` tensor.  ``window`` rows back and the first ``sinks`` rows are visible
    (window 0: all)."""
    with _on(cache.k, stream):
        q = _rows(Q, cache.k, "Q")
        seqs = _seqs(cache, table, kv_len)
        H = Q.shape[0]
        if Q.shape[1] != seqs.n_seq or Q.shape[2] != cache.d:
            raise ValueError("Q must be [H_q][n_seq][d]")
        out, lse = _attn_out(Q, out, lse, return_lse)
        given, ws = ws, _ws_for(ws, lambda: paged_workspace_bytes(cache, H, seqs.n_seq), cache.k)
        check(LIB.mr_paged_decode(ctypes.byref(cache.c), ctypes.byref(seqs), ctypes.byref(q), H,
                                  1.0 / math.sqrt(cache.d) if scale is None else float(scale), int(window), int(sinks),
                                  ctypes.byref(_rows(out, cache.k, "out")), lse.data_ptr() if lse is not None else None,
                                  ws.ptr, ws.nbytes, _stream(None)), "mr_paged_decode")
        _keep(given, ws)
    return out if lse is None else (out, lse)


def paged_attn(cache: KVCache, table: torch.Tensor, kv_len: torch.Tensor, Q: torch.Tensor, cu_q: torch.Tensor,
               scale: Optional[float] = None, window: int = 0, sinks: int = 0, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, return_lse: bool = False, ws: Optional[Workspace] = None, stream=None):
    """mr_paged_attn: causal attention of the new rows Q [H_q][total_q][d] (rows cu_q[s] .. cu_q[s + 1] - 1 are the
    last ones of sequence s) over the cache -> O [H_q][total_q][d], or (O, lse [H_q][total_q]).  The rows' own keys
    and values must be in the cache (kv_append).  Rows behind cu_q[n_seq] are left as they are."""
    with _on(cache.k, stream):
        q = _rows(Q, cache.k, "Q")
        seqs = _seqs(cache, table, kv_len)
        H, total = Q.shape[:2]
        if Q.shape[2] != cache.d:
            raise ValueError("Q must be [H_q][total_q][d] of the cache")
        if cu_q.shape[0] != seqs.n_seq + 1:
            raise ValueError("cu_q must have n_seq + 1 entries")
        out, lse = _attn_out(Q, out, lse, return_lse)
        given, ws = ws, _ws_for(ws, lambda: paged_workspace_bytes(cache, H, seqs.n_seq), cache.k)
        check(LIB.mr_paged_attn(ctypes.byref(cache.c), ctypes.byref(seqs), ctypes.byref(q), H,
                                _ints(cu_q, cache.k, "cu_q"), total,
                                1.0 / math.sqrt(cache.d) if scale is None else float(scale), int(window), int(sinks),
                                ctypes.byref(_rows(out, cache.k, "out")), lse.data_ptr() if lse is not None else None,
                                ws.ptr, ws.nbytes, _stream(None)), "mr_paged_attn")
        _keep(given, ws)
    return out if lse is None else (out, lse)


def pages_copy_workspace_bytes() -> int:
    return int(LIB.mr_pages_copy_workspace_bytes())


def pages_copy(pools, pairs: torch.Tensor, ws: Optional[Workspace] = None, stream=None) -> None:
    """mr_pages_copy: page pairs[t][1] <- page pairs[t][0] (int32, device) in every pool (tensors
    [n_pages][...], e.g. the k and v of every layer's cache)."""
    if not pools:
        raise ValueError("no pools")
    first = pools[0]
    with _on(first, stream):
        page_bytes = first.stride(0) * first.element_size()
        for t in pools:
            _need_cuda(t)
            if t.shape[0] != first.shape[0] or t.device != first.device or t.stride(0) * t.element_size() != page_bytes:
                raise ValueError("pools must have the same pages on the same device")
        p = _ints(pairs, first, "pairs", 2)
        if pairs.shape[1] != 2:
            raise ValueError("pairs must be [n][2]")
        given, ws = ws, _ws_for(ws, pages_copy_workspace_bytes, first)
        ptrs = (_c_p * len(pools))(*[t.data_ptr() for t in pools])
        check(LIB.mr_pages_copy(ptrs, len(pools), page_bytes, first.shape[0], p, pairs.shape[0], ws.ptr, ws.nbytes,
                                _stream(None)), "mr_pages_copy")
        _keep(given, ws)


class PagePool:
    """mr_pp_*: which pages of a pool each sequence holds (host only), with shared pages after a fork.

    ``extend`` and ``compact`` return (source, destination) pairs; copy them with ``pages_copy`` before the
    pages are used again."""

    def __init__(self, n_pages: int, page_rows: int):
        self.h = LIB.mr_pp_create(int(n_pages), int(page_rows))
        if not self.h:
            raise MRError(MR_ERR_INVALID_ARG, "mr_pp_create")
        self.n_pages, self.page_rows = int(n_pages), int(page_rows)

    def __del__(self):
        if getattr(self, "h", None) and LIB is not None:  # LIB is gone while the interpreter ends
            LIB.mr_pp_destroy(self.h)
        self.h = None

    @staticmethod
    def _count(n, where: str) -> int:
        if n < 0:
            raise MRError(-int(n), where)
        return int(n)

    def open(self) -> int:
        return self._count(LIB.mr_pp_open(self.h), "mr_pp_open")

    def fork(self, seq: int, rows: int) -> int:
        """New sequence that shares the first `rows` rows of `seq`."""
        return self._count(LIB.mr_pp_fork(self.h, int(seq), int(rows)), "mr_pp_fork")

    def extend(self, seq: int, rows: int) -> list:
        """Room for `rows` more rows; the list holds one pair when a shared page has to be copied first."""
        pair = (_c_i32 * 2)()
        n = self._count(LIB.mr_pp_extend(self.h, int(seq), int(rows), pair), "mr_pp_extend")
        return [(int(pair[0]), int(pair[1]))] if n else []

    def truncate(self, seq: int, rows: int) -> None:
        """Drop the last rows so that `rows` remain; refused, as a fork is, when `slide` gave up a page that the next
        query would see then."""
        check(LIB.mr_pp_truncate(self.h, int(seq), int(rows)), "mr_pp_truncate")

    def slide(self, seq: int, window: int, sinks: int = 0) -> int:
        """Release the pages that no later query sees; returns how many."""
        return self._count(LIB.mr_pp_slide(self.h, int(seq), int(window), int(sinks)), "mr_pp_slide")

    def close(self, seq: int) -> None:
        check(LIB.mr_pp_close(self.h, int(seq)), "mr_pp_close")

    def compact(self, max_pairs: Optional[int] = None) -> np.ndarray:
        """Move the pages in use to the front; returns the pairs [n][2] to copy."""
        most = self.n_pages if max_pairs is None else int(max_pairs)
        pairs = np.empty((max(0, most), 2), np.int32)
        n = self._count(LIB.mr_pp_compact(self.h, pairs.ctypes.data, most), "mr_pp_compact")
        return pairs[:n]

    def rows(self, seq: int) -> int:
        return self._table(seq, self.n_pages_of(seq))[1]

    def n_pages_of(self, seq: int) -> int:
        """Entries of the sequence's table."""
        most = 64
        while True:
            buf = (_c_i32 * most)()
            n = LIB.mr_pp_table(self.h, int(seq), buf, most, None)
            if n != -MR_ERR_CAPACITY:
                return self._count(n, "mr_pp_table")
            most *= 4

    def _table(self, seq: int, width: int):
        pages, rows = np.empty(width, np.int32), ctypes.c_int(0)
        self._count(LIB.mr_pp_table(self.h, int(seq), pages.ctypes.data, width, ctypes.byref(rows)), "mr_pp_table")
        return pages, int(rows.value)

    def tables(self, seqs, width: Optional[int] = None):
        """Host arrays (table [n][width] int32, rows [n] int32) of some sequences, to copy to the device as
        `table` and `kv_len`; entries without a page are -1."""
        if width is None:
            width = max([1] + [self.n_pages_of(s) for s in seqs])
        got = [self._table(s, width) for s in seqs]
        return np.stack([g[0] for g in got]), np.array([g[1] for g in got], np.int32)

    def stats(self) -> dict:
        v = (_c_i64 * 4)()
        check(LIB.mr_pp_stats(self.h, v), "mr_pp_stats")
        return dict(zip(("pages", "free", "sequences", "shared"), [int(x) for x in v]))
