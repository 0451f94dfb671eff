"""MI355X-native SplitZip BF16 KV-cache codec: Python binding.

A thin ctypes layer over ``libsplitzip.so`` (hand-written HIP for gfx950,
C ABI declared in ``include/splitzip.h``).  The functions named ``sz_*`` are
the C entry points with the same names and arguments; they only marshal
arguments (a torch tensor's data pointer, or a raw integer device pointer,
and the current torch stream by default) and turn a non-zero status into
``SplitZipError``.  Every step of the codec runs in the library's kernels;
PyTorch only provides device memory and streams.

``encode`` and ``decode`` are conveniences that allocate their outputs with
torch and call the entry points.

The method follows the SplitZip explainers (gist.science, arXiv 2605.01708):
top-16 exponent codebook with 4-bit codes two per byte, sign|mantissa bytes,
and (position, exponent) escapes for the remaining exponents (section
"3. La strategie SplitZip"), decoded by lookup, recombination and escape
overwrite (section "4. Pourquoi est-ce rapide ?").
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "SplitZipError", "lib_path", "sz_max_compressed_size", "sz_workspace_size", "sz_encode",
    "sz_decode", "sz_encode_noalloc", "sz_encode_histogram", "sz_encode_codebook", "sz_encode_pack",
    "sz_encode_pack_ranked", "sz_encode_single_read", "sz_encode_sample", "sz_encode_first_pass", "sz_encode_finish",
    "sz_decode_unpack", "sz_decode_scatter", "sz_decode_fused", "sz_decode_dense",
    "sz_decode_workspace_size", "sz_decode_index", "sz_decode_tiles",
    "sz_encode_pages", "sz_decode_pages", "sz_blocks_workspace_size", "sz_encode_blocks",
    "sz_decode_blocks", "sz_blocks_decode_workspace_size", "sz_ship_to_host", "sz_ship_from_host", "ShipContext",
    "sz_rope_frequencies", "sz_rope_phases", "sz_qk_norm_rope", "sz_kv_append",
    "sz_attend_workspace_size", "sz_attend_pages", "Heads", "KVCache", "Batch", "Rope",
    "rope_phases", "rope", "paged_cache", "qk_norm_rope", "kv_append", "attend_pages",
    "sz_latent_append", "sz_attend_latent_workspace_size", "sz_attend_latent", "LatentCache",
    "latent_cache", "latent_append", "attend_latent",
    "sz_attend_expanded_workspace_size", "sz_attend_expanded", "attend_expanded",
    "sz_weigh_workspace_size", "sz_weigh_pages", "sz_evict_pages",
    "sz_evict_pages_pitched", "weigh_pages", "evict_pages",
    "sz_status_string", "encode",
    "decode", "encode_blocks", "decode_blocks", "BlockContainers",
    "PREFIX_BYTES", "MAX_ELEMENTS", "NOALLOC_WORKSPACE_BYTES",
]

PREFIX_BYTES = 176
MAX_ELEMENTS = 1 << 36
NOALLOC_WORKSPACE_BYTES = 4608 * 1024

SZ_OK = 0
SZ_ERR_INVALID_ARGUMENT = 1
SZ_ERR_CAPACITY = 2
SZ_ERR_TOO_LARGE = 3
SZ_ERR_CORRUPT = 4
SZ_ERR_HIP = 5

SZ_TYPE_BF16 = 1
SZ_TYPE_F32 = 2

SZ_ROPE_PLAIN = 0
SZ_ROPE_LINEAR = 1
SZ_ROPE_BASE = 2
SZ_ROPE_RAMP = 3
SZ_ROPE_BANDS = 4

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libsplitzip.so")


class SplitZipError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call}: {sz_status_string(status)} (status {status})")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(lib_path):
        raise ImportError(
            f"{lib_path} is missing: build the HIP library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(lib_path)
    u64, p, i32 = ctypes.c_uint64, ctypes.c_void_p, ctypes.c_int
    L.sz_max_compressed_size.argtypes = [u64]
    L.sz_max_compressed_size.restype = u64
    L.sz_workspace_size.argtypes = [u64]
    L.sz_workspace_size.restype = u64
    L.sz_encode.argtypes = [p, u64, p, u64, p, p]
    L.sz_decode.argtypes = [p, u64, p, u64, p, p]
    L.sz_encode_noalloc.argtypes = [p, u64, p, u64, p, p]
    L.sz_encode_histogram.argtypes = [p, u64, p, u64, p]
    L.sz_encode_codebook.argtypes = [u64, p, u64, p, u64, p, p]
    L.sz_encode_pack.argtypes = [p, u64, p, u64, p, u64, p]
    L.sz_encode_pack_ranked.argtypes = [p, u64, p, u64, p, u64, p, p]
    L.sz_encode_single_read.argtypes = [u64]
    L.sz_encode_single_read.restype = i32
    L.sz_encode_sample.argtypes = [p, u64, p, u64, p]
    L.sz_encode_first_pass.argtypes = [p, u64, p, u64, p, u64, p]
    L.sz_encode_finish.argtypes = [p, u64, p, u64, p, u64, p, p]
    L.sz_decode_unpack.argtypes = [p, u64, p, u64, p, p]
    L.sz_decode_scatter.argtypes = [p, u64, p, u64, p, p]
    L.sz_decode_fused.argtypes = [p, u64, p, u64, p, p]
    L.sz_decode_dense.argtypes = [p, u64, p, u64, p, p]
    L.sz_decode_workspace_size.argtypes = [u64]
    L.sz_decode_workspace_size.restype = u64
    L.sz_decode_index.argtypes = [p, u64, u64, p, u64, p]
    L.sz_decode_tiles.argtypes = [p, u64, p, u64, p, u64, p, p]
    L.sz_encode_pages.argtypes = [p, u64, u64, u64, p, u64, p, p, p]
    L.sz_decode_pages.argtypes = [p, u64, p, u64, u64, u64, p, p]
    L.sz_blocks_workspace_size.argtypes = [u64, u64]
    L.sz_blocks_workspace_size.restype = u64
    L.sz_encode_blocks.argtypes = [p, u64, u64, p, u64, p, p, u64, p, p]
    L.sz_blocks_decode_workspace_size.argtypes = [u64, u64]
    L.sz_blocks_decode_workspace_size.restype = u64
    L.sz_decode_blocks.argtypes = [p, u64, p, u64, u64, p, p, u64, p, p]
    L.sz_ship_to_host.argtypes = [p, u64, u64, p, u64, p, p]
    L.sz_ship_from_host.argtypes = [p, p, u64, u64, p, p, p]
    L.sz_ship_context_create.argtypes = [u64, ctypes.POINTER(ctypes.c_void_p)]
    L.sz_ship_context_destroy.argtypes = [p]
    L.sz_ship_context_destroy.restype = None
    L.sz_ship_to_host_ctx.argtypes = [p, p, u64, p, u64, p, p]
    L.sz_ship_from_host_ctx.argtypes = [p, p, p, u64, p, p, p]
    f32, f64, pd = ctypes.c_float, ctypes.c_double, ctypes.POINTER(ctypes.c_double)
    L.sz_rope_frequencies.argtypes = [ctypes.c_uint32, f64, i32, f64, f64, f64, f64, pd,
                                      ctypes.POINTER(f32)]
    L.sz_rope_phases.argtypes = [pd, u64, p]
    # descriptors go as addresses (None = NULL)
    L.sz_qk_norm_rope.argtypes = [p, p, p, p, p, p, ctypes.c_uint32, u64, p, f32, p, p]
    L.sz_kv_append.argtypes = [p, p, p, p, p, p, f32, p, p, p, p, p, p]
    L.sz_attend_workspace_size.argtypes = [u64, p, p, u64]
    L.sz_attend_workspace_size.restype = u64
    L.sz_attend_pages.argtypes = [p, p, p, p, p, u64, f32, f32, i32, u64, p, u64, p, p]
    L.sz_latent_append.argtypes = [p, p, f32, p, p, p, p, p, p, p, p, p]
    L.sz_attend_latent_workspace_size.argtypes = [u64, p, p, u64]
    L.sz_attend_latent_workspace_size.restype = u64
    L.sz_attend_latent.argtypes = [p, p, p, p, p, u64, f32, i32, p, u64, p, p]
    L.sz_attend_expanded_workspace_size.argtypes = [u64, ctypes.c_uint32, p, u64]
    L.sz_attend_expanded_workspace_size.restype = u64
    u32 = ctypes.c_uint32
    L.sz_attend_expanded.argtypes = [p, p, p, p, p, p, u32, u32, u32, p, u64, p, u64, f32, i32, p,
                                     u64, p, p]
    L.sz_weigh_workspace_size.argtypes = [u64, p, p, u64]
    L.sz_weigh_workspace_size.restype = u64
    L.sz_weigh_pages.argtypes = [p, p, p, p, u64, f32, p, p, u64, f32, f32, i32, u64, p, u64, p, p]
    L.sz_evict_pages.argtypes = [p, u64, u64, p, p, u64, u64, u64, u64, u64, p, p, p, p, p, p]
    L.sz_evict_pages_pitched.argtypes = [p, u64, u64, p, p, u64, u64, u64, u64, u64, p, p, u64, p,
                                         p, p, p]
    for name in ("sz_latent_append", "sz_attend_latent", "sz_attend_expanded",
                 "sz_weigh_pages", "sz_evict_pages", "sz_evict_pages_pitched",
                 "sz_rope_frequencies", "sz_rope_phases", "sz_qk_norm_rope", "sz_kv_append",
                 "sz_attend_pages", "sz_encode", "sz_decode", "sz_encode_noalloc", "sz_encode_histogram", "sz_encode_codebook",
                 "sz_encode_pack", "sz_encode_pack_ranked", "sz_encode_sample",
                 "sz_encode_first_pass", "sz_encode_finish",
                 "sz_decode_unpack", "sz_decode_scatter", "sz_decode_fused",
                 "sz_decode_dense", "sz_decode_index", "sz_decode_tiles", "sz_encode_pages",
                 "sz_decode_pages", "sz_encode_blocks", "sz_decode_blocks", "sz_ship_to_host",
                 "sz_ship_from_host", "sz_ship_context_create", "sz_ship_to_host_ctx",
                 "sz_ship_from_host_ctx"):
        getattr(L, name).restype = i32
    L.sz_status_string.argtypes = [i32]
    L.sz_status_string.restype = ctypes.c_char_p
    return L


_lib = _load()


def _ptr(x) -> int | None:
    """Address of a tensor's data (device, or host for the ship calls' host
    buffers), of a NumPy array's data, or an integer pointer as given
    (None = NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return x.ctypes.data


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, call: str) -> None:
    if status != SZ_OK:
        raise SplitZipError(status, call)


def sz_status_string(status: int) -> str:
    return _lib.sz_status_string(status).decode()


def sz_max_compressed_size(n_elements: int) -> int:
    return int(_lib.sz_max_compressed_size(n_elements))


def sz_workspace_size(n_elements: int) -> int:
    return int(_lib.sz_workspace_size(n_elements))


def sz_encode(src, n_elements: int, dst, dst_capacity: int, d_compressed_size=None,
              stream=None) -> None:
    _check(_lib.sz_encode(_ptr(src), n_elements, _ptr(dst), dst_capacity,
                          _ptr(d_compressed_size), _stream(stream)), "sz_encode")


def sz_encode_noalloc(src, n_elements: int, dst, dst_capacity: int, d_compressed_size=None,
                      stream=None) -> None:
    _check(_lib.sz_encode_noalloc(_ptr(src), n_elements, _ptr(dst), dst_capacity,
                                  _ptr(d_compressed_size), _stream(stream)), "sz_encode_noalloc")


def sz_decode(src, src_bytes: int, dst, n_elements: int, d_status=None, stream=None) -> None:
    _check(_lib.sz_decode(_ptr(src), src_bytes, _ptr(dst), n_elements, _ptr(d_status),
                          _stream(stream)), "sz_decode")


def sz_encode_histogram(src, n_elements: int, workspace, workspace_bytes: int,
                        stream=None) -> None:
    _check(_lib.sz_encode_histogram(_ptr(src), n_elements, _ptr(workspace), workspace_bytes,
                                    _stream(stream)), "sz_encode_histogram")


def sz_encode_codebook(n_elements: int, workspace, workspace_bytes: int, dst,
                       dst_capacity: int, d_compressed_size=None, stream=None) -> None:
    _check(_lib.sz_encode_codebook(n_elements, _ptr(workspace), workspace_bytes, _ptr(dst),
                                   dst_capacity, _ptr(d_compressed_size), _stream(stream)),
           "sz_encode_codebook")


def sz_encode_pack(src, n_elements: int, workspace, workspace_bytes: int, dst,
                   dst_capacity: int, stream=None) -> None:
    _check(_lib.sz_encode_pack(_ptr(src), n_elements, _ptr(workspace), workspace_bytes,
                               _ptr(dst), dst_capacity, _stream(stream)), "sz_encode_pack")


def sz_encode_pack_ranked(src, n_elements: int, workspace, workspace_bytes: int, dst,
                          dst_capacity: int, d_compressed_size=None, stream=None) -> None:
    _check(_lib.sz_encode_pack_ranked(_ptr(src), n_elements, _ptr(workspace), workspace_bytes,
                                      _ptr(dst), dst_capacity, _ptr(d_compressed_size),
                                      _stream(stream)), "sz_encode_pack_ranked")


def sz_encode_single_read(n_elements: int) -> bool:
    return bool(_lib.sz_encode_single_read(n_elements))


def sz_encode_sample(src, n_elements: int, workspace, workspace_bytes: int, stream=None) -> None:
    _check(_lib.sz_encode_sample(_ptr(src), n_elements, _ptr(workspace), workspace_bytes,
                                 _stream(stream)), "sz_encode_sample")


def sz_encode_first_pass(src, n_elements: int, workspace, workspace_bytes: int, dst,
                         dst_capacity: int, stream=None) -> None:
    _check(_lib.sz_encode_first_pass(_ptr(src), n_elements, _ptr(workspace), workspace_bytes,
                                     _ptr(dst), dst_capacity, _stream(stream)),
           "sz_encode_first_pass")


def sz_encode_finish(src, n_elements: int, workspace, workspace_bytes: int, dst,
                     dst_capacity: int, d_compressed_size=None, stream=None) -> None:
    _check(_lib.sz_encode_finish(_ptr(src), n_elements, _ptr(workspace), workspace_bytes,
                                 _ptr(dst), dst_capacity, _ptr(d_compressed_size),
                                 _stream(stream)), "sz_encode_finish")


def sz_decode_unpack(src, src_bytes: int, dst, n_elements: int, d_status=None,
                     stream=None) -> None:
    _check(_lib.sz_decode_unpack(_ptr(src), src_bytes, _ptr(dst), n_elements, _ptr(d_status),
                                 _stream(stream)), "sz_decode_unpack")


def sz_decode_scatter(src, src_bytes: int, dst, n_elements: int, d_status=None,
                      stream=None) -> None:
    _check(_lib.sz_decode_scatter(_ptr(src), src_bytes, _ptr(dst), n_elements, _ptr(d_status),
                                  _stream(stream)), "sz_decode_scatter")


def sz_decode_fused(src, src_bytes: int, dst, n_elements: int, d_status=None,
                    stream=None) -> None:
    _check(_lib.sz_decode_fused(_ptr(src), src_bytes, _ptr(dst), n_elements, _ptr(d_status),
                                _stream(stream)), "sz_decode_fused")


def sz_decode_workspace_size(n_elements: int) -> int:
    return int(_lib.sz_decode_workspace_size(n_elements))


def sz_decode_index(src, src_bytes: int, n_elements: int, workspace, workspace_bytes: int,
                    stream=None) -> None:
    _check(_lib.sz_decode_index(_ptr(src), src_bytes, n_elements, _ptr(workspace),
                                workspace_bytes, _stream(stream)), "sz_decode_index")


def sz_decode_tiles(src, src_bytes: int, workspace, workspace_bytes: int, dst, n_elements: int,
                    d_status=None, stream=None) -> None:
    _check(_lib.sz_decode_tiles(_ptr(src), src_bytes, _ptr(workspace), workspace_bytes,
                                _ptr(dst), n_elements, _ptr(d_status), _stream(stream)),
           "sz_decode_tiles")


def sz_decode_dense(src, src_bytes: int, dst, n_elements: int, d_status=None,
                    stream=None) -> None:
    _check(_lib.sz_decode_dense(_ptr(src), src_bytes, _ptr(dst), n_elements, _ptr(d_status),
                                _stream(stream)), "sz_decode_dense")


def sz_encode_pages(d_pages, n_pages: int, page_elems: int, n_elements: int, dst,
                    dst_capacity: int, d_compressed_size=None, d_status=None, stream=None) -> None:
    """d_pages: device array of page addresses (e.g. an int64 CUDA tensor)."""
    _check(_lib.sz_encode_pages(_ptr(d_pages), n_pages, page_elems, n_elements, _ptr(dst),
                                dst_capacity, _ptr(d_compressed_size), _ptr(d_status),
                                _stream(stream)), "sz_encode_pages")


def sz_decode_pages(src, src_bytes: int, d_pages, n_pages: int, page_elems: int,
                    n_elements: int, d_status=None, stream=None) -> None:
    _check(_lib.sz_decode_pages(_ptr(src), src_bytes, _ptr(d_pages), n_pages, page_elems,
                                n_elements, _ptr(d_status), _stream(stream)), "sz_decode_pages")


def sz_blocks_workspace_size(block_elems: int, n_blocks: int) -> int:
    return int(_lib.sz_blocks_workspace_size(block_elems, n_blocks))


def sz_encode_blocks(d_blocks, n_blocks: int, block_elems: int, dst, dst_pitch: int, d_sizes,
                     workspace, workspace_bytes: int, d_status=None, stream=None) -> None:
    """d_blocks: device array of block addresses (e.g. an int64 CUDA tensor);
    d_sizes: device uint64 array of n_blocks entries (e.g. an int64 tensor)."""
    _check(_lib.sz_encode_blocks(_ptr(d_blocks), n_blocks, block_elems, _ptr(dst), dst_pitch,
                                 _ptr(d_sizes), _ptr(workspace), workspace_bytes, _ptr(d_status),
                                 _stream(stream)), "sz_encode_blocks")


def sz_blocks_decode_workspace_size(block_elems: int, n_blocks: int) -> int:
    return int(_lib.sz_blocks_decode_workspace_size(block_elems, n_blocks))


def sz_decode_blocks(src, src_pitch: int, d_sizes, n_blocks: int, block_elems: int, d_blocks,
                     d_status, workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    """d_status: device int32 array of n_blocks entries (required); with a
    workspace the tile form, without it the single-pass form."""
    _check(_lib.sz_decode_blocks(_ptr(src), src_pitch, _ptr(d_sizes), n_blocks, block_elems,
                                 _ptr(d_blocks), _ptr(workspace), workspace_bytes,
                                 _ptr(d_status), _stream(stream)), "sz_decode_blocks")


def sz_ship_to_host(src, n_elements: int, chunk_elems: int, h_dst, h_capacity: int, h_offsets,
                    stream=None) -> None:
    """h_dst: pinned host buffer; h_offsets: host uint64 array of
    ceil(n / chunk_elems) + 1 entries (a NumPy array or a CPU tensor)."""
    _check(_lib.sz_ship_to_host(_ptr(src), n_elements, chunk_elems, _ptr(h_dst), h_capacity,
                                _ptr(h_offsets), _stream(stream)), "sz_ship_to_host")


def sz_ship_from_host(h_src, h_offsets, n_elements: int, chunk_elems: int, dst, d_status=None,
                      stream=None) -> None:
    _check(_lib.sz_ship_from_host(_ptr(h_src), _ptr(h_offsets), n_elements, chunk_elems,
                                  _ptr(dst), _ptr(d_status), _stream(stream)),
           "sz_ship_from_host")


class ShipContext:
    """A transfer context (sz_ship_context_create) for one chunk size on the
    current device; released by close() or when collected."""

    def __init__(self, chunk_elems: int):
        self.handle = None
        h = ctypes.c_void_p()
        _check(_lib.sz_ship_context_create(chunk_elems, ctypes.byref(h)),
               "sz_ship_context_create")
        self.handle = h.value
        self.chunk_elems = chunk_elems

    def close(self) -> None:
        if getattr(self, "handle", None):
            _lib.sz_ship_context_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()

    def to_host(self, src, n_elements: int, h_dst, h_capacity: int, h_offsets,
                stream=None) -> None:
        _check(_lib.sz_ship_to_host_ctx(self.handle, _ptr(src), n_elements, _ptr(h_dst),
                                        h_capacity, _ptr(h_offsets), _stream(stream)),
               "sz_ship_to_host_ctx")

    def from_host(self, h_src, h_offsets, n_elements: int, dst, d_status=None,
                  stream=None) -> None:
        _check(_lib.sz_ship_from_host_ctx(self.handle, _ptr(h_src), _ptr(h_offsets), n_elements,
                                          _ptr(dst), _ptr(d_status), _stream(stream)),
               "sz_ship_from_host_ctx")


# ---- operators on a paged cache --------------------------------------------
# Descriptors of tensors, cache, batch and rotation: made once, kept as long
# as the buffers they describe (which they hold a reference to), and passed to
# any number of calls.

def _on_device(t, dtype, what: str, dim: int | None = None):
    if not hasattr(t, "is_cuda") or not t.is_cuda or t.dtype != dtype or \
            (dim is not None and t.dim() != dim) or (t.numel() > 0 and t.stride(-1) != 1):
        raise ValueError(f"{what} must be a CUDA tensor of {dtype}"
                         + (f" with {dim} dimensions" if dim else "")
                         + ", its last dimension contiguous")
    return t


_U32, _U64 = 1 << 32, 1 << 64


def _fits(limit: int, *sizes) -> None:
    """Sizes as their C type holds them (ctypes would cut them to it)."""
    for x in sizes:
        if not 0 <= x < limit:
            raise ValueError(f"a size of {x}")


class _Descriptor(ctypes.Structure):
    def _set(self, device, *keep):
        self._keep, self._at = keep, ctypes.addressof(self)
        self._index = device.index


class Heads(_Descriptor):
    """sz_heads of a CUDA tensor [tokens, heads, head_dim] of bfloat16 or
    float32 with a contiguous last dimension (any view of one whose strides
    and address are multiples of 8 elements and 16 bytes)."""
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_uint64),
                ("token_stride", ctypes.c_uint64), ("head_stride", ctypes.c_uint64),
                ("type", ctypes.c_uint32)]

    def __init__(self, t):
        import torch
        if not hasattr(t, "is_cuda") or not t.is_cuda or t.dim() != 3 or \
                t.dtype not in (torch.bfloat16, torch.float32) or \
                (t.shape[2] > 1 and t.stride(2) != 1):
            raise ValueError("head rows must be a CUDA tensor [tokens, heads, head_dim] of "
                             "bfloat16 or float32, its last dimension contiguous")
        strides = [t.stride(i) if t.shape[i] > 1 else 0 for i in (0, 1)]
        super().__init__(t.data_ptr(), t.shape[1], strides[0], strides[1],
                         SZ_TYPE_F32 if t.dtype == torch.float32 else SZ_TYPE_BF16)
        self.tokens, self.dim = t.shape[0], t.shape[2]
        self._set(t.device, t)


class KVCache(_Descriptor):
    """sz_kv_cache: k_pages and v_pages are int64 CUDA tensors [sequences,
    pages] of page addresses, of the same shape and row stride; strides in
    elements of a page (default: [token][head][dim])."""
    _fields_ = [("d_k_pages", ctypes.c_void_p), ("d_v_pages", ctypes.c_void_p),
                ("pages_per_seq", ctypes.c_uint64), ("table_pitch", ctypes.c_uint64),
                ("token_stride", ctypes.c_uint64), ("head_stride", ctypes.c_uint64),
                ("kv_heads", ctypes.c_uint32), ("head_dim", ctypes.c_uint32),
                ("page_tokens", ctypes.c_uint32)]

    def __init__(self, k_pages, v_pages, kv_heads: int, head_dim: int, page_tokens: int,
                 token_stride: int | None = None, head_stride: int | None = None, keep=None):
        import torch
        for t in (k_pages, v_pages):
            _on_device(t, torch.int64, "a page table", 2)
        pitch = [t.stride(0) if t.shape[0] > 1 else t.shape[1] for t in (k_pages, v_pages)]
        if k_pages.shape != v_pages.shape or k_pages.device != v_pages.device or \
                pitch[0] != pitch[1]:
            raise ValueError("the page tables must have the same shape, strides and device")
        token_stride = kv_heads * head_dim if token_stride is None else token_stride
        head_stride = head_dim if head_stride is None else head_stride
        _fits(_U32, kv_heads, head_dim, page_tokens)
        _fits(_U64, token_stride, head_stride)
        super().__init__(k_pages.data_ptr(), v_pages.data_ptr(), k_pages.shape[1], pitch[0],
                         token_stride, head_stride, kv_heads, head_dim, page_tokens)
        self.rows = k_pages.shape[0]
        self._set(k_pages.device, k_pages, v_pages, keep)


class LatentCache(_Descriptor):
    """sz_latent_cache: pages is an int64 CUDA tensor [sequences, pages] of
    page addresses; token_stride in elements of a page (default: rows side
    by side)."""
    _fields_ = [("d_pages", ctypes.c_void_p), ("pages_per_seq", ctypes.c_uint64),
                ("table_pitch", ctypes.c_uint64), ("token_stride", ctypes.c_uint64),
                ("latent_dim", ctypes.c_uint32), ("rotary_dim", ctypes.c_uint32),
                ("page_tokens", ctypes.c_uint32)]

    def __init__(self, pages, latent_dim: int, rotary_dim: int, page_tokens: int,
                 token_stride: int | None = None, keep=None):
        import torch
        _on_device(pages, torch.int64, "a page table", 2)
        token_stride = latent_dim + rotary_dim if token_stride is None else token_stride
        _fits(_U32, latent_dim, rotary_dim, page_tokens)
        _fits(_U64, token_stride)
        super().__init__(pages.data_ptr(), pages.shape[1],
                         pages.stride(0) if pages.shape[0] > 1 else pages.shape[1], token_stride,
                         latent_dim, rotary_dim, page_tokens)
        self.rows = pages.shape[0]
        self._set(pages.device, pages, keep)


class Batch(_Descriptor):
    """sz_batch: starts and lens are int32 CUDA tensors of n_seqs + 1 and
    n_seqs entries; n_tokens is the row count of the token-major tensors."""
    _fields_ = [("d_starts", ctypes.c_void_p), ("d_lens", ctypes.c_void_p),
                ("n_seqs", ctypes.c_uint64), ("n_tokens", ctypes.c_uint64)]

    def __init__(self, starts, lens, n_tokens: int):
        import torch
        for t in (starts, lens):
            _on_device(t, torch.int32, "starts and lens", 1)
        if starts.numel() != lens.numel() + 1 or starts.device != lens.device:
            raise ValueError("starts must have one entry more than lens, on the same device")
        _fits(_U64, n_tokens)
        super().__init__(starts.data_ptr(), lens.data_ptr(), lens.numel(), n_tokens)
        self._set(starts.device, starts, lens)


class Rope(_Descriptor):
    """sz_rope: phases is an int64 CUDA tensor of rotary_dim / 2 entries (the
    64-bit patterns of sz_rope_phases, see rope_phases and rope)."""
    _fields_ = [("d_phases", ctypes.c_void_p), ("rotary_dim", ctypes.c_uint32),
                ("interleaved", ctypes.c_uint32), ("magnitude", ctypes.c_float)]

    def __init__(self, phases, interleaved: bool = False, magnitude: float = 1.0):
        import torch
        _on_device(phases, torch.int64, "phases", 1)
        super().__init__(phases.data_ptr(), 2 * phases.numel(), int(bool(interleaved)), magnitude)
        self._set(phases.device, phases)


def _at(x) -> int | None:
    """Address of a descriptor."""
    return None if x is None else x._at


def _heads(x):
    """A descriptor as it is, or one of a tensor (to be kept until the call
    returns)."""
    return x if x is None or type(x) is Heads else Heads(x)


def _call_stream(stream, first, *rest):
    """The stream of a call whose descriptors and tensors are given (None and
    integer addresses skipped): all on the current device, as `stream` must
    be."""
    import torch
    index = first._index
    for x in rest:
        # (descriptors before tensors: one attribute)
        if x is not None and getattr(x, "_index", index) != index:
            raise ValueError("the call's tensors are on different devices")
    if torch.cuda.current_device() != index:
        raise ValueError(f"the tensors are on device {index}, the current device is "
                         f"{torch.cuda.current_device()}")
    if stream is None:
        # (a tenth of the time of torch.cuda.current_stream(), which counts
        # beside kernels of a few microseconds)
        return torch._C._cuda_getCurrentRawStream(index)
    return _stream(stream)


def _tokens(n: int, *xs) -> None:
    for x in xs:
        if x is not None and x.tokens != n:
            raise ValueError(f"{x.tokens} tokens where {n} are expected")


def _dims(dim: int, *xs) -> None:
    for x in xs:
        if x is not None and x.dim != dim:
            raise ValueError(f"rows of {x.dim} elements where {dim} are expected")


def _array(x, dtype: str, n: int, index: int, what: str) -> int | None:
    """Address of a device array of at least n elements (None and integer
    addresses as they are)."""
    if x is None or type(x) is int:
        return x
    import torch
    if x.dtype is not getattr(torch, dtype) or x.numel() < n or not x.is_contiguous() or \
            x.get_device() != index:
        raise ValueError(f"{what} must be a contiguous tensor of at least {n} {dtype}s on the "
                         "call's device")
    return x.data_ptr()


def sz_rope_frequencies(rotary_dim: int, base: float, stretch: int = SZ_ROPE_PLAIN,
                        factor: float = 1.0, original_len: float = 0.0, slow: float = 1.0,
                        fast: float = 32.0):
    """Angles per position (a list of rotary_dim / 2 floats) and magnitude."""
    if not 0 <= rotary_dim < 1 << 32:  # (ctypes would cut it to 32 bits)
        raise SplitZipError(SZ_ERR_INVALID_ARGUMENT, "sz_rope_frequencies")
    out = (ctypes.c_double * max(1, rotary_dim // 2))()
    magnitude = ctypes.c_float()
    _check(_lib.sz_rope_frequencies(rotary_dim, base, stretch, factor, original_len, slow, fast,
                                    out, ctypes.byref(magnitude)), "sz_rope_frequencies")
    return list(out), magnitude.value


def sz_rope_phases(inv_freq):
    """Phases of a sequence of angles per position, as a ctypes uint64 array."""
    n = len(inv_freq)
    out = (ctypes.c_uint64 * n)()
    _check(_lib.sz_rope_phases((ctypes.c_double * n)(*inv_freq), n, out), "sz_rope_phases")
    return out


def sz_qk_norm_rope(q, q_out, q_weight, k, k_out, k_weight, head_dim: int, n_tokens: int,
                    positions, eps: float, rope, stream=None) -> None:
    """q, q_out, k, k_out: Heads, or tensors [tokens, heads, head_dim]; rope: a
    Rope or None."""
    q, q_out, k, k_out = _heads(q), _heads(q_out), _heads(k), _heads(k_out)
    some = q if q is not None else k
    if some is None:
        raise ValueError("neither queries nor keys")
    stream = _call_stream(stream, some, q_out, k, k_out, rope)
    index = some._index
    _tokens(n_tokens, q, q_out, k, k_out)
    _dims(head_dim, q, q_out, k, k_out)
    _check(_lib.sz_qk_norm_rope(
        _at(q), _at(q_out), _array(q_weight, "float32", head_dim, index, "q_weight"),
        _at(k), _at(k_out), _array(k_weight, "float32", head_dim, index, "k_weight"),
        head_dim, n_tokens, _array(positions, "int32", n_tokens, index, "positions"), eps,
        _at(rope), stream), "sz_qk_norm_rope")


def _check_rows(cache, batch) -> None:
    if batch.n_seqs > cache.rows:
        raise ValueError(f"{batch.n_seqs} sequences, {cache.rows} rows in the page tables")


def sz_kv_append(k, v, k_weight, q, q_out, q_weight, eps: float, rope, positions, cache, batch,
                 d_status=None, stream=None) -> None:
    """k, v, q, q_out: Heads, or tensors [tokens, heads, head_dim]; cache: a
    KVCache; batch: a Batch; rope: a Rope or None."""
    k, v, q, q_out = _heads(k), _heads(v), _heads(q), _heads(q_out)
    stream = _call_stream(stream, cache, batch, k, v, q, q_out, rope)
    index, dim, n = cache._index, cache.head_dim, batch.n_tokens
    _tokens(n, k, v, q, q_out)
    _dims(dim, k, v, q, q_out)
    _check_rows(cache, batch)
    _check(_lib.sz_kv_append(
        _at(k), _at(v), _array(k_weight, "float32", dim, index, "k_weight"), _at(q), _at(q_out),
        _array(q_weight, "float32", dim, index, "q_weight"), eps, _at(rope),
        _array(positions, "int32", n, index, "positions"), cache._at, batch._at,
        _array(d_status, "int32", batch.n_seqs, index, "d_status"), stream), "sz_kv_append")


def sz_attend_workspace_size(q_heads: int, cache, batch, max_len: int = 0) -> int:
    _fits(_U64, q_heads, max_len)
    return int(_lib.sz_attend_workspace_size(q_heads, _at(cache), _at(batch), max_len))


def sz_attend_pages(q, out, lse, cache, batch, max_len: int, scale: float, softcap: float = 0.0,
                    causal: bool = True, window: int = 0, workspace=None,
                    workspace_bytes: int = 0, d_status=None, stream=None) -> None:
    """q, out: Heads, or tensors [tokens, heads, head_dim]; lse: a float32
    tensor [tokens, heads] or None; cache: a KVCache; batch: a Batch."""
    q, out = _heads(q), _heads(out)
    if not (0 <= max_len < _U64 and 0 <= window < _U64 and 0 <= workspace_bytes < _U64):
        _fits(_U64, max_len, window, workspace_bytes)
    stream = _call_stream(stream, cache, batch, q, out)
    index, n = cache._index, batch.n_tokens
    _tokens(n, q, out)
    _dims(cache.head_dim, q, out)
    _check_rows(cache, batch)
    _check(_lib.sz_attend_pages(
        q._at, out._at, _array(lse, "float32", n * q.heads, index, "lse"), cache._at, batch._at,
        max_len, scale, softcap, int(causal), window,
        _array(workspace, "uint8", workspace_bytes, index, "workspace"), workspace_bytes,
        _array(d_status, "int32", batch.n_seqs, index, "d_status"), stream), "sz_attend_pages")


def sz_latent_append(latent, weight, eps: float, k_rotary, q, q_out, rope, positions, cache,
                     batch, d_status=None, stream=None) -> None:
    """latent, k_rotary, q, q_out: Heads, or tensors [tokens, heads, elements]
    (one head in the first two); cache: a LatentCache; batch: a Batch; rope: a
    Rope or None."""
    latent, k_rotary, q, q_out = _heads(latent), _heads(k_rotary), _heads(q), _heads(q_out)
    stream = _call_stream(stream, cache, batch, latent, k_rotary, q, q_out, rope)
    index, n = cache._index, batch.n_tokens
    _tokens(n, latent, k_rotary, q, q_out)
    _dims(cache.latent_dim, latent)
    _dims(cache.rotary_dim, k_rotary, q, q_out)
    _check_rows(cache, batch)
    _check(_lib.sz_latent_append(
        _at(latent), _array(weight, "float32", cache.latent_dim, index, "weight"), eps,
        _at(k_rotary), _at(q), _at(q_out), _at(rope),
        _array(positions, "int32", n, index, "positions"), cache._at, batch._at,
        _array(d_status, "int32", batch.n_seqs, index, "d_status"), stream), "sz_latent_append")


def sz_attend_latent_workspace_size(heads: int, cache, batch, max_len: int = 0) -> int:
    _fits(_U64, heads, max_len)
    return int(_lib.sz_attend_latent_workspace_size(heads, _at(cache), _at(batch), max_len))


def sz_attend_latent(q, out, lse, cache, batch, max_len: int, scale: float, causal: bool = True,
                     workspace=None, workspace_bytes: int = 0, d_status=None,
                     stream=None) -> None:
    """q, out: Heads, or tensors [tokens, heads, elements]; lse: a float32
    tensor [tokens, heads] or None; cache: a LatentCache; batch: a Batch."""
    q, out = _heads(q), _heads(out)
    if not (0 <= max_len < _U64 and 0 <= workspace_bytes < _U64):
        _fits(_U64, max_len, workspace_bytes)
    stream = _call_stream(stream, cache, batch, q, out)
    index, n = cache._index, batch.n_tokens
    _tokens(n, q, out)
    _dims(cache.latent_dim + cache.rotary_dim, q)
    _dims(cache.latent_dim, out)
    _check_rows(cache, batch)
    _check(_lib.sz_attend_latent(
        q._at, out._at, _array(lse, "float32", n * q.heads, index, "lse"), cache._at, batch._at,
        max_len, scale, int(causal), _array(workspace, "uint8", workspace_bytes, index, "workspace"),
        workspace_bytes, _array(d_status, "int32", batch.n_seqs, index, "d_status"), stream),
        "sz_attend_latent")


def sz_attend_expanded_workspace_size(heads: int, value_dim: int, batch, max_len: int = 0) -> int:
    _fits(_U64, heads, max_len)
    _fits(_U32, value_dim)
    return int(_lib.sz_attend_expanded_workspace_size(heads, value_dim, _at(batch), max_len))


def sz_attend_expanded(q, out, lse, k, k_rotary, v, key_starts, batch, max_len: int, scale: float,
                       causal: bool = True, workspace=None, workspace_bytes: int = 0,
                       d_status=None, stream=None) -> None:
    """q, out, k, k_rotary (or None), v: Heads, or tensors [rows, heads,
    elements]; key_starts: an int32 tensor [sequences]; lse: a float32 tensor
    [tokens, heads] or None; batch: a Batch."""
    q, out, k, k_rotary, v = (_heads(x) for x in (q, out, k, k_rotary, v))
    if not (0 <= max_len < _U64 and 0 <= workspace_bytes < _U64):
        _fits(_U64, max_len, workspace_bytes)
    stream = _call_stream(stream, batch, q, out, k, k_rotary, v)
    index, n = batch._index, batch.n_tokens
    _tokens(n, q, out)
    _tokens(k.tokens, v, k_rotary)
    rotary = 0 if k_rotary is None else k_rotary.dim
    _dims(k.dim + rotary, q)
    _dims(v.dim, out)
    _check(_lib.sz_attend_expanded(
        q._at, out._at, _array(lse, "float32", n * q.heads, index, "lse"), k._at, _at(k_rotary),
        v._at, k.dim, rotary, v.dim, _array(key_starts, "int32", batch.n_seqs, index, "key_starts"),
        k.tokens, batch._at, max_len, scale, int(causal),
        _array(workspace, "uint8", workspace_bytes, index, "workspace"), workspace_bytes,
        _array(d_status, "int32", batch.n_seqs, index, "d_status"), stream), "sz_attend_expanded")


def sz_weigh_workspace_size(q_heads: int, cache, batch, max_len: int = 0) -> int:
    _fits(_U64, q_heads, max_len)
    return int(_lib.sz_weigh_workspace_size(q_heads, _at(cache), _at(batch), max_len))


def sz_weigh_pages(q, lse, before, weights, weights_pitch: int, keep: float, cache, batch,
                   max_len: int, scale: float, softcap: float = 0.0, causal: bool = True,
                   window: int = 0, workspace=None, workspace_bytes: int = 0, d_status=None,
                   stream=None) -> None:
    """q: Heads, or a tensor [tokens, heads, head_dim]; lse: a float32 tensor
    [tokens, heads]; before (or None) and weights: float32 tensors [sequences,
    KV heads, weights_pitch]; cache: a KVCache; batch: a Batch."""
    q = _heads(q)
    if not (0 <= max_len < _U64 and 0 <= window < _U64 and 0 <= workspace_bytes < _U64 and
            0 <= weights_pitch < _U64):
        _fits(_U64, max_len, window, workspace_bytes, weights_pitch)
    stream = _call_stream(stream, cache, batch, q)
    index, n = cache._index, batch.n_tokens
    _tokens(n, q)
    _dims(cache.head_dim, q)
    _check_rows(cache, batch)
    size = batch.n_seqs * cache.kv_heads * weights_pitch
    _check(_lib.sz_weigh_pages(
        q._at, _array(lse, "float32", n * q.heads, index, "lse"),
        _array(before, "float32", size, index, "before"),
        _array(weights, "float32", size, index, "weights"), weights_pitch, keep, cache._at,
        batch._at, max_len, scale, softcap, int(causal), window,
        _array(workspace, "uint8", workspace_bytes, index, "workspace"), workspace_bytes,
        _array(d_status, "int32", batch.n_seqs, index, "d_status"), stream), "sz_weigh_pages")


def sz_evict_pages(weights, weights_to, from_cache, to_cache, lens, lens_to, max_len: int,
                   budget: int, first: int, recent: int, kept, d_status=None,
                   stream=None) -> None:
    """weights: a float32 tensor [sequences, weight heads, pitch]; weights_to
    and kept: float32 and int32 tensors [sequences, weight heads, budget]; lens
    and lens_to: int32 tensors [sequences]; from_cache, to_cache: KVCaches."""
    _evict("sz_evict_pages", weights, weights_to, None, from_cache, to_cache, lens, lens_to,
           max_len, budget, first, recent, kept, d_status, stream)


def sz_evict_pages_pitched(weights, weights_to, weights_to_pitch: int, from_cache, to_cache, lens,
                           lens_to, max_len: int, budget: int, first: int, recent: int, kept,
                           d_status=None, stream=None) -> None:
    """As sz_evict_pages, weights_to a tensor [sequences, weight heads,
    weights_to_pitch]."""
    _evict("sz_evict_pages_pitched", weights, weights_to, weights_to_pitch, from_cache, to_cache,
           lens, lens_to, max_len, budget, first, recent, kept, d_status, stream)


def _evict(call, weights, weights_to, to_pitch, from_cache, to_cache, lens, lens_to, max_len,
           budget, first, recent, kept, d_status, stream) -> None:
    if weights.dim() != 3:
        raise ValueError("weights must have 3 dimensions")
    n, heads, pitch = weights.shape
    if not (0 <= max_len < _U64 and 0 <= budget < _U64 and 0 <= first < _U64 and
            0 <= recent < _U64):
        _fits(_U64, max_len, budget, first, recent)
    pitched = () if to_pitch is None else (to_pitch,)
    _fits(_U64, *pitched)
    stream = _call_stream(stream, from_cache, to_cache)
    index = from_cache._index
    if n > from_cache.rows or n > to_cache.rows:
        raise ValueError(f"{n} sequences, {from_cache.rows} and {to_cache.rows} rows in the page "
                         "tables")
    size = n * heads * budget
    to_size = size
    if to_pitch is not None and size > 0:
        to_size = (n * heads - 1) * to_pitch + budget
    _check(getattr(_lib, call)(
        _array(weights, "float32", n * heads * pitch, index, "weights"), heads, pitch,
        from_cache._at, _array(lens, "int32", n, index, "lens"), n, max_len, budget, first, recent,
        to_cache._at, _array(weights_to, "float32", to_size, index, "weights_to"), *pitched,
        _array(kept, "int32", size, index, "kept"), _array(lens_to, "int32", n, index, "lens_to"),
        _array(d_status, "int32", n, index, "d_status"), stream), call)


# ---- conveniences (torch allocates; the library computes) -----------------

def encode(x, stream=None):
    """Compress a CUDA tensor of BF16 (or 16-bit integer) words; returns the
    container as a uint8 CUDA tensor trimmed to its exact size (this reads
    the size back, so it synchronises the stream)."""
    import torch
    if x.element_size() != 2 or not x.is_cuda:
        raise ValueError("encode expects a CUDA tensor of 16-bit elements")
    x = x.contiguous()
    n = x.numel()
    cap = sz_max_compressed_size(n)
    dst = torch.empty(cap, dtype=torch.uint8, device=x.device)
    size = torch.zeros(1, dtype=torch.int64, device=x.device)
    sz_encode(x, n, dst, cap, size, stream)
    return dst[: int(size.item())]


def decode(container, n_elements: int, dtype=None, stream=None, check: bool = True):
    """Decompress a uint8 CUDA container into ``n_elements`` words (bfloat16
    unless ``dtype`` says otherwise).  With ``check`` the device status is
    read back (synchronising) and a corrupt container raises."""
    import torch
    out = torch.empty(n_elements, dtype=dtype or torch.bfloat16, device=container.device)
    status = torch.zeros(1, dtype=torch.int32, device=container.device)
    sz_decode(container, container.numel(), out, n_elements, status, stream)
    if check:
        st = int(status.item())
        if st != SZ_OK:
            raise SplitZipError(st, "sz_decode (device check)")
    return out


class BlockContainers:
    """Containers of equal-length blocks as sz_encode_blocks leaves them:
    block b's container is ``data[b * pitch : b * pitch + sizes[b]]``, and
    ``sizes`` stays on the device (a uint64 array held as an int64 tensor)."""

    def __init__(self, data, pitch: int, sizes, block_elems: int):
        self.data, self.pitch, self.sizes, self.block_elems = data, pitch, sizes, block_elems

    def __len__(self) -> int:
        return self.sizes.numel()

    def container(self, b: int):
        """Block b's container, trimmed (reads its size back: synchronises)."""
        return self.data[b * self.pitch: b * self.pitch + int(self.sizes[b].item())]


def _block_table(tensors):
    import torch
    if not tensors:
        raise ValueError("no blocks")
    n = tensors[0].numel()
    for t in tensors:
        if t.element_size() != 2 or not t.is_cuda or t.numel() != n or not t.is_contiguous():
            raise ValueError("blocks must be contiguous CUDA tensors of 16-bit elements, "
                             "all of the same length")
    return torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64,
                        device=tensors[0].device), n


def encode_blocks(tensors, stream=None) -> BlockContainers:
    """Compress equal-length CUDA tensors (one per layer, say), one container
    each, in one launch per pass (sz_encode_blocks); nothing is read back."""
    import torch
    table, n = _block_table(tensors)
    nb = len(tensors)
    dev = tensors[0].device
    pitch = (sz_max_compressed_size(n) + 15) // 16 * 16
    data = torch.empty(nb * pitch, dtype=torch.uint8, device=dev)
    sizes = torch.zeros(nb, dtype=torch.int64, device=dev)
    wb = sz_blocks_workspace_size(n, nb)
    ws = torch.empty(wb, dtype=torch.uint8, device=dev)
    sz_encode_blocks(table, nb, n, data, pitch, sizes, ws, wb, None, stream)
    return BlockContainers(data, pitch, sizes, n)


def decode_blocks(blocks: BlockContainers, outputs, stream=None, check: bool = True):
    """Decompress every container into the matching output tensor (same
    count and length as encoded), with the tile form's workspace; with
    ``check`` the per-block statuses are read back (synchronising) and any
    failure raises, naming the first block that failed."""
    import torch
    table, n = _block_table(outputs)
    nb = len(outputs)
    if nb != len(blocks) or n != blocks.block_elems:
        raise ValueError("outputs do not match the containers' block count and length")
    dev = outputs[0].device
    status = torch.zeros(nb, dtype=torch.int32, device=dev)
    wb = sz_blocks_decode_workspace_size(n, nb)
    ws = torch.empty(wb, dtype=torch.uint8, device=dev)
    sz_decode_blocks(blocks.data, blocks.pitch, blocks.sizes, nb, n, table, status, ws, wb,
                     stream)
    if check:
        st = status.cpu()
        bad = (st != SZ_OK).nonzero()
        if bad.numel():
            b = int(bad[0])
            raise SplitZipError(int(st[b]), f"sz_decode_blocks (block {b})")
    return outputs


def rope_phases(inv_freq):
    """sz_rope_phases as a CPU int64 tensor (the same 64 bits)."""
    import torch
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in sz_rope_phases(inv_freq)],
                        dtype=torch.int64)


def rope(rotary_dim: int, base: float = 10000.0, stretch: int = SZ_ROPE_PLAIN,
         factor: float = 1.0, original_len: float = 0.0, slow: float = 1.0, fast: float = 32.0,
         interleaved: bool = False, device="cuda") -> Rope:
    """The rotation of sz_rope_frequencies' frequencies, on a device."""
    freq, magnitude = sz_rope_frequencies(rotary_dim, base, stretch, factor, original_len, slow,
                                          fast)
    return Rope(rope_phases(freq).to(device), interleaved, magnitude)


def _bf16_pool(pool, dim: int) -> None:
    import torch
    _on_device(pool, torch.bfloat16, "a pool", dim)


def _page_addresses(pool, table):
    """The address table of a table of page numbers."""
    import torch
    if table.dim() != 2 or table.dtype not in (torch.int32, torch.int64) or \
            table.device != pool.device:
        raise ValueError("the table must be a 2-D integer tensor on the pools' device")
    ids = table.to(torch.int64)
    if ids.numel() > 0 and int(ids.max()) >= pool.shape[0]:
        raise ValueError("a page number past the pool")
    return torch.where(ids >= 0, pool.data_ptr() + ids * (pool.stride(0) * 2),
                       torch.zeros_like(ids))


def paged_cache(k_pool, v_pool, table) -> KVCache:
    """The cache of two pools [pages, page_tokens, kv_heads, head_dim] of
    bfloat16 (any strides that keep head_dim contiguous, so that a permuted
    [pages, kv_heads, page_tokens, head_dim] pool does too) and an integer
    table [sequences, pages] of page numbers, negative for none.  The address
    tables are made here (the largest page number is read back, which waits
    for the device); make the cache again when the table changes, or keep
    address tables of your own up to date and make a KVCache of them once."""
    for t in (k_pool, v_pool):
        _bf16_pool(t, 4)
    if k_pool.shape != v_pool.shape or k_pool.stride() != v_pool.stride():
        raise ValueError("the pools must have the same shape and strides")
    return KVCache(_page_addresses(k_pool, table), _page_addresses(v_pool, table),
                   k_pool.shape[2], k_pool.shape[3], k_pool.shape[1], k_pool.stride(1),
                   k_pool.stride(2), keep=(k_pool, v_pool))


def latent_cache(pool, table, latent_dim: int) -> LatentCache:
    """The latent cache of a pool [pages, page_tokens, latent_dim + rotary_dim]
    of bfloat16 and an integer table [sequences, pages] of page numbers,
    negative for none; as paged_cache."""
    _bf16_pool(pool, 3)
    return LatentCache(_page_addresses(pool, table), latent_dim, pool.shape[2] - latent_dim,
                       pool.shape[1], pool.stride(1), keep=pool)


def _raise_on(status, call: str) -> None:
    st = status.cpu()
    bad = (st != SZ_OK).nonzero()
    if bad.numel():
        s = int(bad[0])
        raise SplitZipError(int(st[s]), f"{call} (sequence {s})")


def qk_norm_rope(q, k, positions, rope=None, q_weight=None, k_weight=None, eps: float = 1e-6):
    """Norm and rotate queries and keys [tokens, heads, head_dim] (either may
    be None); returns new bfloat16 tensors (sz_qk_norm_rope)."""
    import torch
    some = q if q is not None else k
    if some is None:
        raise ValueError("neither queries nor keys")
    out = [None if x is None else torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
           for x in (q, k)]
    sz_qk_norm_rope(q, out[0], q_weight, k, out[1], k_weight, some.shape[2], some.shape[0],
                    positions, eps, rope)
    return out[0], out[1]


def kv_append(k, v, cache, batch, rope=None, q=None, k_weight=None, q_weight=None,
              eps: float = 1e-6, positions=None, check: bool = True):
    """Append new tokens to a paged cache (sz_kv_append); returns the turned
    queries as a new bfloat16 tensor where q is given (rows of no sequence
    are zero).  With ``check`` the statuses are read back (synchronising)
    and a failure raises, naming the first sequence that failed."""
    import torch
    out = None if q is None else torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
    status = torch.zeros(batch.n_seqs, dtype=torch.int32, device=k.device) if check else None
    sz_kv_append(k, v, k_weight, q, out, q_weight, eps, rope, positions, cache, batch, status)
    if check:
        _raise_on(status, "sz_kv_append")
    return out


def attend_pages(q, cache, batch, max_len: int = 0, scale: float | None = None,
                 softcap: float = 0.0, causal: bool = True, window: int = 0, out_dtype=None,
                 check: bool = True):
    """Attention of queries [tokens, heads, head_dim] over a paged cache
    (sz_attend_pages); returns the output (bfloat16 unless ``out_dtype`` is
    float32) and the log-sums [tokens, heads], zero for rows of no sequence.
    scale defaults to head_dim ** -0.5; ``check`` as in kv_append."""
    import torch
    out = torch.zeros(q.shape, dtype=out_dtype or torch.bfloat16, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=q.device)
    size = sz_attend_workspace_size(q.shape[1], cache, batch, max_len)
    ws = torch.empty(size, dtype=torch.uint8, device=q.device) if size else None
    status = torch.zeros(batch.n_seqs, dtype=torch.int32, device=q.device) if check else None
    sz_attend_pages(q, out, lse, cache, batch, max_len,
                    q.shape[2] ** -0.5 if scale is None else scale, softcap, causal, window, ws,
                    size, status)
    if check:
        _raise_on(status, "sz_attend_pages")
    return out, lse


def latent_append(latent, cache, batch, k_rotary=None, rope=None, q=None, weight=None,
                  eps: float = 1e-6, positions=None, check: bool = True):
    """Append new tokens' latents [tokens, 1, latent_dim] and rotary parts
    [tokens, 1, rotary_dim] to a cache of latents (sz_latent_append); returns
    the turned rotary parts of the queries as a new bfloat16 tensor where q
    is given (rows of no sequence are zero).  ``check`` as in kv_append."""
    import torch
    out = None if q is None else torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
    status = torch.zeros(batch.n_seqs, dtype=torch.int32, device=latent.device) if check else None
    sz_latent_append(latent, weight, eps, k_rotary, q, out, rope, positions, cache, batch, status)
    if check:
        _raise_on(status, "sz_latent_append")
    return out


def attend_latent(q, cache, batch, scale: float, max_len: int = 0, causal: bool = True,
                  out_dtype=None, check: bool = True):
    """Attention of absorbed queries [tokens, heads, latent_dim + rotary_dim]
    over a cache of latents (sz_attend_latent); returns the output [tokens,
    heads, latent_dim] (bfloat16 unless ``out_dtype`` is float32) and the
    log-sums [tokens, heads], zero for rows of no sequence.  scale is that of
    the heads before they were absorbed; ``check`` as in kv_append."""
    import torch
    out = torch.zeros((*q.shape[:2], cache.latent_dim), dtype=out_dtype or torch.bfloat16,
                      device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=q.device)
    size = sz_attend_latent_workspace_size(q.shape[1], cache, batch, max_len)
    ws = torch.empty(size, dtype=torch.uint8, device=q.device) if size else None
    status = torch.zeros(batch.n_seqs, dtype=torch.int32, device=q.device) if check else None
    sz_attend_latent(q, out, lse, cache, batch, max_len, scale, causal, ws, size, status)
    if check:
        _raise_on(status, "sz_attend_latent")
    return out, lse


def attend_expanded(q, k, v, key_starts, batch, scale: float, k_rotary=None, max_len: int = 0,
                    causal: bool = True, out_dtype=None, check: bool = True):
    """Attention of queries [tokens, heads, key_dim + rotary_dim] over keys and
    values [keys, heads, ..] expanded from latents, their rotary part [keys, 1
    or heads, rotary_dim] beside them (sz_attend_expanded); returns the output
    [tokens, heads, value_dim] (bfloat16 unless ``out_dtype`` is float32) and
    the log-sums, zero for rows of no sequence; ``check`` as in kv_append."""
    import torch
    out = torch.zeros((*q.shape[:2], v.shape[2]), dtype=out_dtype or torch.bfloat16,
                      device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=q.device)
    most = max_len if 0 < max_len < k.shape[0] else k.shape[0]
    size = sz_attend_expanded_workspace_size(q.shape[1], v.shape[2], batch, most) if most else 0
    ws = torch.empty(size, dtype=torch.uint8, device=q.device) if size else None
    status = torch.zeros(batch.n_seqs, dtype=torch.int32, device=q.device) if check else None
    sz_attend_expanded(q, out, lse, k, k_rotary, v, key_starts, batch, max_len, scale, causal, ws,
                       size, status)
    if check:
        _raise_on(status, "sz_attend_expanded")
    return out, lse


def weigh_pages(q, lse, cache, batch, weights=None, keep: float = 1.0, max_len: int = 0,
                scale: float | None = None, softcap: float = 0.0, causal: bool = True,
                window: int = 0, check: bool = True):
    """The attention weights that cached tokens receive from queries [tokens,
    heads, head_dim] whose log-sums attend_pages returned (sz_weigh_pages):
    added in place to keep * ``weights`` [sequences, KV heads, tokens], or to a
    new tensor, zero past the lengths.  Other arguments as in attend_pages."""
    import torch
    before = weights
    if weights is None:
        most = cache.pages_per_seq * cache.page_tokens
        most = max_len if 0 < max_len < most else most
        weights = torch.zeros((batch.n_seqs, cache.kv_heads, most), dtype=torch.float32,
                              device=q.device)
    elif weights.dim() != 3 or tuple(weights.shape[:2]) != (batch.n_seqs, cache.kv_heads):
        raise ValueError("weights must be a tensor [sequences, KV heads, tokens]")
    size = sz_weigh_workspace_size(q.shape[1], cache, batch, max_len)
    ws = torch.empty(size, dtype=torch.uint8, device=q.device) if size else None
    status = torch.zeros(batch.n_seqs, dtype=torch.int32, device=q.device) if check else None
    sz_weigh_pages(q, lse, before, weights, weights.shape[2], keep, cache, batch, max_len,
                   q.shape[2] ** -0.5 if scale is None else scale, softcap, causal, window, ws,
                   size, status)
    if check:
        _raise_on(status, "sz_weigh_pages")
    return weights


def evict_pages(weights, from_cache, to_cache, lens, budget: int, first: int = 0,
                recent: int = 0, max_len: int = 0, check: bool = True, room: int | None = None):
    """Keep at most ``budget`` tokens of each sequence, in the pages of
    to_cache (sz_evict_pages); returns the kept old positions (int32
    [sequences, weight heads, budget], -1 past those that stay), their weights
    (zero there) and the new lengths.  With ``room`` (at least budget) the
    weights are a tensor [sequences, KV heads, room] that weigh_pages goes on
    with in place, where there is room for the tokens that to_cache will hold
    (its pages' or max_len); one choice for all heads leaves what stays in the
    first head's row, for the heads' sum to go on.  ``check`` as in kv_append."""
    import torch
    shape = (*weights.shape[:2], budget)
    kept = torch.empty(shape, dtype=torch.int32, device=weights.device)
    pitch = budget if room is None else room
    if pitch < budget:
        raise ValueError(f"room for {room} weights, {budget} tokens stay")
    rows = shape[1] if room is None else from_cache.kv_heads
    weights_to = torch.zeros((shape[0], rows, pitch), dtype=torch.float32, device=weights.device)
    if rows > shape[1]:
        pitch *= rows
    lens_to = torch.empty_like(lens)
    status = torch.zeros(lens.shape, dtype=torch.int32, device=lens.device) if check else None
    sz_evict_pages_pitched(weights, weights_to, pitch, from_cache, to_cache, lens, lens_to,
                           max_len, budget, first, recent, kept, status)
    if check:
        _raise_on(status, "sz_evict_pages")
    return kept, weights_to, lens_to
