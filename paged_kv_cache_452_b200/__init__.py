"""Paged KV-cache decode attention for B200 (sm_100a): a thin Python binding
over the C ABI of libpa.so (include/pa.h).

Every function here only marshals arguments (torch tensors -> device
pointers, the current CUDA stream) and calls the library function of the
same name; all work runs in the library's CUDA kernels or its C++ block pool.
Importing fails loudly if libpa.so has not been built
(``python paged_kv_cache_452_b200/build.py``); there is no fallback.
"""
import ctypes
import math
import os

import torch

from ._lib import LIB_PATH, PaError, lib  # noqa: F401

PA_F32, PA_BF16, PA_FP8_E4M3 = 0, 1, 2
_CODES = {"f32": PA_F32, "bf16": PA_BF16, "e4m3": PA_FP8_E4M3}
_TORCH = {PA_F32: torch.float32, PA_BF16: torch.bfloat16, PA_FP8_E4M3: torch.uint8}
_NAMES = {v: k for k, v in _CODES.items()}
_SIZES = {PA_F32: 4, PA_BF16: 2, PA_FP8_E4M3: 1}


class CacheDesc(ctypes.Structure):
    """pa_cache_desc: shape and storage of one layer's paged cache."""
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("q_dtype", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("k_head_scales", ctypes.c_void_p),
                ("v_head_scales", ctypes.c_void_p)]

    @classmethod
    def make(cls, num_blocks, block_size, num_kv_heads, num_q_heads, head_dim, kv_dtype="bf16",
             q_dtype="bf16", k_scale=1.0, v_scale=1.0, k_head_scales=None, v_head_scales=None):
        """k_head_scales / v_head_scales: optional device fp32 tensors
        [num_kv_heads] (an e4m3 pool's per-kv-head scales); the desc keeps a
        reference so they stay alive as long as it does."""
        kv = _CODES.get(kv_dtype, kv_dtype)
        q = _CODES.get(q_dtype, q_dtype)
        d = cls(num_blocks, block_size, num_kv_heads, num_q_heads, head_dim, kv, q,
                float(k_scale), float(v_scale), _ptr(k_head_scales), _ptr(v_head_scales))
        d._keep = (k_head_scales, v_head_scales)
        return d

    @property
    def group(self):
        return self.num_q_heads // self.num_kv_heads

    @property
    def kv_torch_dtype(self):
        return _TORCH[self.kv_dtype]

    @property
    def q_torch_dtype(self):
        return _TORCH[self.q_dtype]


def _check(rc, what):
    if rc != 0:
        raise PaError(rc, f"{what}: {lib().pa_last_error().decode()}")


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def pa_block_bytes(desc: CacheDesc) -> int:
    return int(lib().pa_block_bytes(ctypes.byref(desc)))


def alloc_cache(desc: CacheDesc, device, fill=None):
    """Allocate (K pool, V pool) as torch tensors in the library's layout:
    K [NB][Hkv][bs][D]; V the same, or [NB][Hkv][D][bs] for an e4m3 pool.
    fill: optional element value (a raw byte for e4m3)."""
    nb, bs, h, d = desc.num_blocks, desc.block_size, desc.num_kv_heads, desc.head_dim
    dt = desc.kv_torch_dtype
    k = torch.empty((nb, h, bs, d), dtype=dt, device=device)
    v = torch.empty((nb, h, d, bs) if desc.kv_dtype == PA_FP8_E4M3 else (nb, h, bs, d), dtype=dt,
                    device=device)
    if fill is not None:
        k.fill_(fill)
        v.fill_(fill)
    return k, v


def pa_cache_write(desc, k_new, v_new, slot_mapping, k_cache, v_cache, stream=None):
    """Scatter new K/V rows [T][Hkv][D] into the pools through int64 slots."""
    n = int(slot_mapping.shape[0])
    _check(lib().pa_cache_write(ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), n,
                                _ptr(k_cache), _ptr(v_cache), _stream(stream)), "pa_cache_write")


def _rows(who, name, t, dtype, dev, n, heads, dim):
    """Checks a [n][heads][dim] tensor whose tokens' rows may lie apart; the elements between two of them."""
    if t.dtype != dtype or t.get_device() != dev or t.shape != (n, heads, dim):
        raise PaError(1, f"{who}: {name} must be {(n, heads, dim)} of {dtype} on cuda:{dev}, got {tuple(t.shape)} of "
                         f"{t.dtype} on {t.device}")
    step, head, one = t.stride()
    if one != 1 or (head != dim and heads > 1) or (n > 1 and step < heads * dim):
        raise PaError(1, f"{who}: {name} has strides {t.stride()}")
    return step if n > 1 else heads * dim


def _array(who, name, t, dtype, dev, shape):
    """Checks a contiguous tensor of a given type, place and shape."""
    if t.dtype != dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise PaError(1, f"{who}: {name} must be a contiguous {tuple(shape)} of {dtype} on cuda:{dev}, got "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device}")


def _pools(who, desc, k_cache, v_cache, dev):
    """Checks the pools against the desc (any view of the same bytes is taken)."""
    need = desc.num_blocks * desc.num_kv_heads * desc.block_size * desc.head_dim * _SIZES[desc.kv_dtype]
    for t in (k_cache, v_cache):
        if t.nbytes != need or t.get_device() != dev or not t.is_contiguous():
            name = "k_cache" if t is k_cache else "v_cache"
            raise PaError(1, f"{who}: {name} must hold {need} contiguous bytes on cuda:{dev}")
    if desc.k_head_scales or desc.v_head_scales:
        for name, t in zip(("k_head_scales", "v_head_scales"), getattr(desc, "_keep", ())):
            if isinstance(t, torch.Tensor):
                _array(who, name, t, torch.float32, dev, (desc.num_kv_heads,))


def _call(who, dev, stream, f, *args):
    """f(*args, stream) with the tensors' device current (the library launches on the current one), on that device's
    current stream if none is given."""
    if dev < 0:
        raise PaError(1, f"{who}: tensors must be on a CUDA device")
    # (a Stream object costs 3 us to make, a third of a small call)
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    if torch.cuda.current_device() == dev:
        rc = f(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, handle)
    if rc != 0:
        raise PaError(rc, f"{who}: {lib().pa_last_error().decode()}")


def _parameter(who, name, t, dtypes, dims):
    """Checks a tensor that a parameter block holds: contiguous, of one of the dtypes; its device's index."""
    if t.dtype not in dtypes or t.dim() != dims or not t.is_contiguous():
        raise PaError(1, f"{who}: {name} must be a contiguous {dims}-d tensor of {dtypes}, got {tuple(t.shape)} of {t.dtype}")
    return t.get_device()


class QkPrep(ctypes.Structure):
    """pa_qk_prep: norm weights and rotation table of one layer (kept alive by this object)."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("cos_sin", ctypes.c_void_p), ("num_positions", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]
    _dev = _weights = None

    @classmethod
    def make(cls, q_weight=None, k_weight=None, eps=1e-6, cos_sin=None, interleaved=False):
        """q_weight / k_weight: device [head_dim] in the query dtype, or None (no norm).  cos_sin: device fp32
        [num_positions][rot_dim], a position's cosines and then its sines, or None (no rotation)."""
        who = "QkPrep.make"
        held = [(t.dtype, t.shape[0], _parameter(who, name, t, (torch.float32, torch.bfloat16), 1))
                for name, t in (("q_weight", q_weight), ("k_weight", k_weight)) if t is not None]
        devs = {h[2] for h in held}
        n = rot = 0
        if cos_sin is not None:
            devs.add(_parameter(who, "cos_sin", cos_sin, (torch.float32,), 2))
            n, rot = (int(v) for v in cos_sin.shape)
        if len(devs) > 1 or len({h[:2] for h in held}) > 1:
            raise PaError(1, f"{who}: weights of one dtype and length, and all tensors on one device")
        p = cls(_ptr(q_weight), _ptr(k_weight), float(eps), _ptr(cos_sin), n, rot, int(bool(interleaved)))
        p._keep = (q_weight, k_weight, cos_sin)
        p._dev = devs.pop() if devs else None
        p._weights = held[0][:2] if held else None
        return p


def pa_norm_rope_write(desc, prep, q, k, v, positions, slot_mapping, q_out, k_cache, v_cache, stream=None):
    """Norm and rotation of q [T][Hq][D] and k [T][Hkv][D], queries to q_out, k and v to the pools through int64
    slots.  q, k, v may be slices of one projection's output (token stride above a row); positions: int32 [T]
    (None without a rotation table); q_out contiguous, or q itself."""
    who, dev, dt = "pa_norm_rope_write", q.get_device(), desc.q_torch_dtype
    n, hq, hkv, d = q.shape[0], desc.num_q_heads, desc.num_kv_heads, desc.head_dim
    qs = _rows(who, "q", q, dt, dev, n, hq, d)
    ks = _rows(who, "k", k, dt, dev, n, hkv, d)
    vs = _rows(who, "v", v, dt, dev, n, hkv, d)
    _array(who, "q_out", q_out, dt, dev, (n, hq, d))
    _array(who, "slot_mapping", slot_mapping, torch.int64, dev, (n,))
    if positions is not None:
        _array(who, "positions", positions, torch.int32, dev, (n,))
    elif prep.cos_sin:
        raise PaError(1, f"{who}: a rotation needs positions")
    if (prep._dev is not None and prep._dev != dev) or (prep._weights is not None and prep._weights != (dt, d)):
        raise PaError(1, f"{who}: prep holds q_weight, k_weight or cos_sin of another device, dtype or head_dim")
    _pools(who, desc, k_cache, v_cache, dev)
    _call(who, dev, stream, lib().pa_norm_rope_write, ctypes.byref(desc), ctypes.byref(prep), q.data_ptr(), qs,
          k.data_ptr(), ks, v.data_ptr(), vs, _ptr(positions), slot_mapping.data_ptr(), n, q_out.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr())


def pa_cache_read(desc, slot_mapping, k_cache, v_cache, k_out, v_out, stream=None):
    """Rows of int64 slots out of the pools into k_out, v_out [T][Hkv][D], dequantised."""
    who, dev, dt = "pa_cache_read", k_out.get_device(), desc.q_torch_dtype
    n = slot_mapping.shape[0]
    shape = (n, desc.num_kv_heads, desc.head_dim)
    _array(who, "slot_mapping", slot_mapping, torch.int64, dev, (n,))
    _array(who, "k_out", k_out, dt, dev, shape)
    _array(who, "v_out", v_out, dt, dev, shape)
    _pools(who, desc, k_cache, v_cache, dev)
    _call(who, dev, stream, lib().pa_cache_read, ctypes.byref(desc), slot_mapping.data_ptr(), n, k_cache.data_ptr(),
          v_cache.data_ptr(), k_out.data_ptr(), v_out.data_ptr())


def pa_copy_blocks(desc, src, dst, k_cache, v_cache, stream=None):
    """Copy-on-write's device half: K/V block dst[i] := block src[i] (int32 device tensors)."""
    n = int(src.shape[0])
    if int(dst.shape[0]) != n:
        raise PaError(1, "pa_copy_blocks: src and dst differ in length")
    _check(lib().pa_copy_blocks(ctypes.byref(desc), _ptr(src), _ptr(dst), n, _ptr(k_cache), _ptr(v_cache),
                                _stream(stream)), "pa_copy_blocks")


def pa_decode_workspace_size(desc, num_seqs) -> int:
    n = int(lib().pa_decode_workspace_size(ctypes.byref(desc), int(num_seqs)))
    if n == 0:
        raise PaError(1, "pa_decode_workspace_size: " + lib().pa_last_error().decode())
    return n


def pa_prefill_workspace_size(desc, num_seqs, num_tokens) -> int:
    n = int(lib().pa_prefill_workspace_size(ctypes.byref(desc), int(num_seqs), int(num_tokens)))
    if n == 0:
        raise PaError(1, "pa_prefill_workspace_size: " + lib().pa_last_error().decode())
    return n


def alloc_workspace(nbytes, device):
    """Caller-owned scratch; the error word in its first bytes starts at zero."""
    return torch.zeros(int(nbytes), dtype=torch.uint8, device=device)


def workspace_error(workspace) -> int:
    """The error word a kernel sets when a bounded wait times out (1) or a
    block table entry is outside the pool (2).  Synchronises."""
    return int(workspace[:4].view(torch.int32).item())


def pa_decode(desc, q, k_cache, v_cache, block_tables, seq_lens, scale, out, workspace, stream=None):
    """One decode step: q [S][Hq][D] attends seq_lens[s] keys via block_tables [S][max_blocks]."""
    s = int(seq_lens.shape[0])
    _check(lib().pa_decode(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                           int(block_tables.shape[1]), _ptr(seq_lens), s, float(scale), _ptr(out),
                           _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                           _stream(stream)), "pa_decode")


def pa_decode_fused(desc, q, k_new, v_new, k_cache, v_cache, block_tables, seq_lens, scale, out, workspace,
                    stream=None):
    """pa_cache_write of each sequence's new token (rows k_new[s], v_new[s],
    at position seq_lens[s] - 1 through its block table) and pa_decode, in
    one launch."""
    s = int(seq_lens.shape[0])
    _check(lib().pa_decode_fused(ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                 _ptr(v_cache), _ptr(block_tables), int(block_tables.shape[1]), _ptr(seq_lens), s,
                                 float(scale), _ptr(out), _ptr(workspace),
                                 int(workspace.numel() * workspace.element_size()), _stream(stream)),
           "pa_decode_fused")


def pa_decode_static(desc, q, k_cache, v_cache, block_tables, seq_lens, scale, out, stream=None):
    """pa_decode without a workspace: the scratch is a fixed 8 MiB area built
    into the library, for callers that cannot allocate device memory."""
    s = int(seq_lens.shape[0])
    _check(lib().pa_decode_static(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                  int(block_tables.shape[1]), _ptr(seq_lens), s, float(scale), _ptr(out),
                                  _stream(stream)), "pa_decode_static")


def pa_decode_chunked_prefill(desc, q, k_cache, v_cache, block_tables, query_start_loc, seq_lens,
                              max_q_len, scale, out, workspace, stream=None):
    """A mixed step: sequence s owns rows query_start_loc[s]..query_start_loc[s+1]-1 (causal)."""
    s = int(seq_lens.shape[0])
    _check(lib().pa_decode_chunked_prefill(
        ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        int(block_tables.shape[1]), _ptr(query_start_loc), _ptr(seq_lens), s, int(q.shape[0]),
        int(max_q_len), float(scale), _ptr(out), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _stream(stream)),
        "pa_decode_chunked_prefill")


class PrefixGroups:
    """Shared prefixes of a decode batch (pa_prefix_groups): CSR prefix_start
    / prefix_members, prefix_blocks, and per sequence seq_prefix / seq_slot
    (-1 outside any prefix), as int32 tensors on the host."""

    def __init__(self, block_tables, seq_lens, block_size):
        bt = block_tables.detach().cpu().contiguous().to(torch.int32)
        sl = seq_lens.detach().cpu().contiguous().to(torch.int32)
        n = int(sl.shape[0])
        self.prefix_start = torch.zeros(n + 1, dtype=torch.int32)
        self.prefix_members = torch.zeros(max(1, n), dtype=torch.int32)
        self.prefix_blocks = torch.zeros(max(1, n), dtype=torch.int32)
        self.seq_prefix = torch.zeros(max(1, n), dtype=torch.int32)
        self.seq_slot = torch.zeros(max(1, n), dtype=torch.int32)
        np_, nm = ctypes.c_int32(), ctypes.c_int32()
        _check(lib().pa_prefix_groups(_ptr(bt), int(bt.shape[1]), _ptr(sl), n, int(block_size),
                                      _ptr(self.prefix_start), _ptr(self.prefix_members), _ptr(self.prefix_blocks),
                                      _ptr(self.seq_prefix), _ptr(self.seq_slot), ctypes.byref(np_),
                                      ctypes.byref(nm)), "pa_prefix_groups")
        self.num_prefixes, self.num_members = np_.value, nm.value
        self.max_prefix_blocks = int(self.prefix_blocks[:self.num_prefixes].max()) if self.num_prefixes else 0

    def to(self, device):
        """The arrays pa_decode_prefix reads, on `device` (a dict)."""
        return {k: getattr(self, k).to(device) for k in
                ("prefix_start", "prefix_members", "prefix_blocks", "seq_prefix", "seq_slot")}


def pa_decode_prefix_workspace_size(desc, num_seqs, num_members, max_prefix_blocks) -> int:
    n = int(lib().pa_decode_prefix_workspace_size(ctypes.byref(desc), int(num_seqs), int(num_members),
                                                  int(max_prefix_blocks)))
    if n == 0:
        raise PaError(1, "pa_decode_prefix_workspace_size: " + lib().pa_last_error().decode())
    return n


def pa_decode_prefix(desc, q, k_cache, v_cache, block_tables, seq_lens, groups, dev_groups, scale, out,
                     workspace, stream=None):
    """pa_decode with each shared prefix attended once for all its sequences
    (groups: a PrefixGroups; dev_groups: its arrays on the device)."""
    s = int(seq_lens.shape[0])
    g = dev_groups
    _check(lib().pa_decode_prefix(
        ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), int(block_tables.shape[1]),
        _ptr(seq_lens), s, _ptr(g["prefix_start"]), _ptr(g["prefix_members"]), _ptr(g["prefix_blocks"]),
        _ptr(g["seq_prefix"]), _ptr(g["seq_slot"]), int(groups.num_prefixes), int(groups.num_members),
        int(groups.max_prefix_blocks), float(scale), _ptr(out), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _stream(stream)), "pa_decode_prefix")


class ScoreMod(ctypes.Structure):
    """pa_score_mod: what the biased attention does to the scores (keeps its tensors alive)."""
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32), ("slopes", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p)]
    _dev = _heads = _seqs = None

    @classmethod
    def make(cls, softcap=0.0, window=0, slopes=None, prefix_lens=None):
        """softcap: cap * tanh(score / cap), 0 for none; window: keys a row sees up to itself, 0 for all; slopes:
        device fp32 [num_q_heads], the score loses slope * distance; prefix_lens: device int32 [num_seqs], leading
        keys that every row sees."""
        who = "ScoreMod.make"
        if not 0 <= int(window) < 2**31:  # (the struct's field would wrap)
            raise PaError(1, f"{who}: window {window} (0, or keys up to 2^31 - 1)")
        devs = set()
        if slopes is not None:
            devs.add(_parameter(who, "slopes", slopes, (torch.float32,), 1))
        if prefix_lens is not None:
            devs.add(_parameter(who, "prefix_lens", prefix_lens, (torch.int32,), 1))
        if len(devs) > 1:
            raise PaError(1, f"{who}: slopes and prefix_lens on one device")
        m = cls(float(softcap), int(window), _ptr(slopes), _ptr(prefix_lens))
        m._keep = (slopes, prefix_lens)
        m._dev = devs.pop() if devs else None
        m._heads = slopes.shape[0] if slopes is not None else None
        m._seqs = prefix_lens.shape[0] if prefix_lens is not None else None
        return m


def pa_biased_workspace_size(desc, num_seqs, num_tokens) -> int:
    n = int(lib().pa_biased_workspace_size(ctypes.byref(desc), int(num_seqs), int(num_tokens)))
    if n == 0:
        raise PaError(1, "pa_biased_workspace_size: " + lib().pa_last_error().decode())
    return n


def _biased_args(who, desc, mod, q, k_cache, v_cache, block_tables, seq_lens, out, workspace):
    dev, dt, hq = q.get_device(), desc.q_torch_dtype, desc.num_q_heads
    shape = (q.shape[0], hq, desc.head_dim)
    _array(who, "q", q, dt, dev, shape)
    _array(who, "out", out, dt, dev, shape)
    n = seq_lens.shape[0]
    _array(who, "seq_lens", seq_lens, torch.int32, dev, (n,))
    if block_tables.dim() != 2:
        raise PaError(1, f"{who}: block_tables must be [num_seqs][max_blocks]")
    _array(who, "block_tables", block_tables, torch.int32, dev, (n, block_tables.shape[1]))
    if ((mod._dev is not None and mod._dev != dev) or (mod._heads is not None and mod._heads != hq) or
            (mod._seqs is not None and mod._seqs != n)):
        raise PaError(1, f"{who}: mod holds slopes or prefix_lens of another device, head or sequence count")
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise PaError(1, f"{who}: workspace must be contiguous on cuda:{dev}")
    _pools(who, desc, k_cache, v_cache, dev)
    return dev, n


def pa_decode_biased(desc, mod, q, k_cache, v_cache, block_tables, seq_lens, scale, out, workspace, stream=None):
    """pa_decode with capped, distance-biased or window- and prefix-masked scores (mod: a ScoreMod)."""
    who = "pa_decode_biased"
    dev, n = _biased_args(who, desc, mod, q, k_cache, v_cache, block_tables, seq_lens, out, workspace)
    if q.shape[0] != n:
        raise PaError(1, f"{who}: {q.shape[0]} query rows for {n} sequences")
    _call(who, dev, stream, lib().pa_decode_biased, ctypes.byref(desc), ctypes.byref(mod), q.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(), n,
          float(scale), out.data_ptr(), workspace.data_ptr(), workspace.nbytes)


def pa_decode_chunked_prefill_biased(desc, mod, q, k_cache, v_cache, block_tables, query_start_loc, seq_lens,
                                     max_q_len, scale, out, workspace, stream=None):
    """pa_decode_chunked_prefill with capped, distance-biased or window- and prefix-masked scores (mod: a ScoreMod)."""
    who = "pa_decode_chunked_prefill_biased"
    dev, n = _biased_args(who, desc, mod, q, k_cache, v_cache, block_tables, seq_lens, out, workspace)
    _array(who, "query_start_loc", query_start_loc, torch.int32, dev, (n + 1,))
    _call(who, dev, stream, lib().pa_decode_chunked_prefill_biased, ctypes.byref(desc), ctypes.byref(mod), q.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
          query_start_loc.data_ptr(), seq_lens.data_ptr(), n, q.shape[0], int(max_q_len), float(scale), out.data_ptr(),
          workspace.data_ptr(), workspace.nbytes)


def default_scale(head_dim):
    return 1.0 / math.sqrt(head_dim)


class BlockPool:
    """Host block pool (pa_pool_*): free_block_queue, ref_cnt, prefix sharing,
    fork with copy-on-write."""

    def __init__(self, num_blocks, block_size, initial_free_order=None):
        self._lib = lib()
        h = ctypes.c_void_p()
        arr = None
        if initial_free_order is not None:
            order = [int(b) for b in initial_free_order]
            if len(order) != num_blocks:
                raise PaError(1, "initial_free_order must have num_blocks entries")
            arr = (ctypes.c_int32 * num_blocks)(*order)
        _check(self._lib.pa_pool_create(int(num_blocks), int(block_size), arr, ctypes.byref(h)),
               "pa_pool_create")
        self._h = h
        self.num_blocks = num_blocks
        self.block_size = block_size

    def close(self):
        if self._h:
            self._lib.pa_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_seq(self, seq_id, num_tokens, token_ids=None) -> int:
        arr = None
        if token_ids is not None:
            ids = [int(t) for t in token_ids]
            arr = (ctypes.c_int32 * len(ids))(*ids)
        cached = ctypes.c_int32(0)
        _check(self._lib.pa_pool_add_seq(self._h, int(seq_id), arr, int(num_tokens), ctypes.byref(cached)),
               "pa_pool_add_seq")
        return cached.value

    def append(self, seq_id, n_new):
        out = (ctypes.c_int64 * max(1, n_new))()
        _check(self._lib.pa_pool_append(self._h, int(seq_id), int(n_new), out), "pa_pool_append")
        return list(out[:n_new])

    def fork(self, parent_id, child_id):
        """child_id shares every block of parent_id (copy on write)."""
        _check(self._lib.pa_pool_fork(self._h, int(parent_id), int(child_id)), "pa_pool_fork")

    def take_copies(self):
        """The (src, dst) block copies queued by copy-on-write, oldest first."""
        n = ctypes.c_int32()
        self._lib.pa_pool_take_copies(self._h, None, None, 0, ctypes.byref(n))
        src = (ctypes.c_int32 * max(1, n.value))()
        dst = (ctypes.c_int32 * max(1, n.value))()
        _check(self._lib.pa_pool_take_copies(self._h, src, dst, n.value, ctypes.byref(n)), "pa_pool_take_copies")
        return [(src[i], dst[i]) for i in range(n.value)]

    def slots(self, seq_id, start, n):
        out = (ctypes.c_int64 * max(1, n))()
        _check(self._lib.pa_pool_slots(self._h, int(seq_id), int(start), int(n), out), "pa_pool_slots")
        return list(out[:n])

    def free_seq(self, seq_id):
        _check(self._lib.pa_pool_free_seq(self._h, int(seq_id)), "pa_pool_free_seq")

    def num_tokens(self, seq_id):
        n = ctypes.c_int32()
        _check(self._lib.pa_pool_num_tokens(self._h, int(seq_id), ctypes.byref(n)), "pa_pool_num_tokens")
        return n.value

    def block_table(self, seq_id):
        n = ctypes.c_int32()
        self._lib.pa_pool_block_table(self._h, int(seq_id), None, 0, ctypes.byref(n))
        out = (ctypes.c_int32 * max(1, n.value))()
        _check(self._lib.pa_pool_block_table(self._h, int(seq_id), out, n.value, ctypes.byref(n)),
               "pa_pool_block_table")
        return list(out[:n.value])

    def block_tables(self, seq_ids, max_blocks):
        """Padded int32 table [len(seq_ids)][max_blocks] as a CPU torch tensor."""
        ids = (ctypes.c_int64 * max(1, len(seq_ids)))(*[int(s) for s in seq_ids])
        out = torch.empty((len(seq_ids), max_blocks), dtype=torch.int32)
        _check(self._lib.pa_pool_block_tables(self._h, ids, len(seq_ids), int(max_blocks),
                                              ctypes.c_void_p(out.data_ptr())), "pa_pool_block_tables")
        return out

    def ref_cnt(self, block):
        return int(self._lib.pa_pool_ref_cnt(self._h, int(block)))

    def num_free(self):
        return int(self._lib.pa_pool_num_free(self._h))

    def free_order(self):
        n = ctypes.c_int32()
        cap = self.num_blocks
        out = (ctypes.c_int32 * max(1, cap))()
        _check(self._lib.pa_pool_free_order(self._h, out, cap, ctypes.byref(n)), "pa_pool_free_order")
        return list(out[:n.value])
