"""GB300-native query-dependent prefix reads of a bit-plane K cache.

The compute path is libbpkv (CUDA kernels for sm_103a behind the C ABI in
``include/bpkv.h``).  This package is its thin Python binding: the functions
named ``bpkv_*`` marshal torch tensors to the C entry points of the same name;
``Cache`` holds one layer's cache buffers as torch tensors (torch is used only
to own device or pinned host memory and streams).
"""
from __future__ import annotations

import ctypes

from ._binding import (  # noqa: F401
    BpkvError, bpkv_alloc_depths, bpkv_cache, bpkv_calibrate_channels, bpkv_clear_status, bpkv_decode_step,
    bpkv_dense_attend, bpkv_encode_append, bpkv_fixed_depths, bpkv_read_status, bpkv_rotate, bpkv_row_cache_stats, bpkv_scan, bpkv_scan_topk, bpkv_scan_topk_noalloc, bpkv_selection_map, bpkv_selftest_wait, bpkv_sparse_attend, bpkv_sparse_attend_vdepth,
    bpkv_qkv_args, bpkv_qkv_rope, bpkv_rows8, bpkv_rows8_append, bpkv_rows8_read, bpkv_shared_attend,
    bpkv_shared_attend8, bpkv_shared_workspace_size, bpkv_status_string, bpkv_step_args, bpkv_topk, bpkv_union, bpkv_version, bpkv_workspace_size, header_symbols, load)

HEAD_DIM = 128
WS_SCAN_TOPK, WS_ATTEND, WS_DENSE, WS_STEP = 1, 2, 4, 8
DEPTH_WATERFILL, DEPTH_FIXED, DEPTH_DENSE, DEPTH_GIVEN = 0, 1, 2, 3
DEV_OVERFLOW, DEV_SELECT, DEV_TIMEOUT = 1, 2, 4
STEP_VDEPTH = 1
QKV_PAIRS, QKV_Q_BF16 = 1, 2


class Cache:
    """One layer's bit-plane K cache and bf16 K/V rows for N sequences x H KV heads.

    residency "hbm": all buffers in device memory.  "host": planes, scales and
    rows in pinned host memory, read by the kernels in place over the host link.
    """

    def __init__(self, n_seq: int, n_kv_heads: int, group: int, cap_tokens: int, device="cuda",
                 residency: str = "hbm", values: bool = False, rc_slots: int = 0):
        import torch
        if cap_tokens % 512:
            raise ValueError("cap_tokens must be a multiple of 512")
        D, nb = HEAD_DIM, cap_tokens // 64
        self.device = torch.device(device)
        host = residency == "host"

        def buf(shape, dtype):
            if host:
                # pinned host memory from a 256-byte boundary: the kernels' reads
                # of it are not cached, so a row segment that starts inside a
                # 32-byte sector moves one more sector over the link
                n = dtype.itemsize
                for e in shape:
                    n *= e
                raw = torch.empty(n + 256, dtype=torch.uint8, pin_memory=True)
                off = (-raw.data_ptr()) % 256
                return raw[off:off + n].view(dtype).view(shape)
            return torch.empty(shape, dtype=dtype, device=self.device)

        self.planes = buf((n_seq, n_kv_heads, D, 4, nb), torch.int64)
        self.scales = buf((n_seq, n_kv_heads, D, nb), torch.int16)
        self.k_rows = buf((n_seq, n_kv_heads, cap_tokens, D), torch.bfloat16)
        self.v_rows = buf((n_seq, n_kv_heads, cap_tokens, D), torch.bfloat16)
        self.seq_len = torch.zeros(n_seq, dtype=torch.int64, device=self.device)
        self.basis = None
        # the value rows' own code (value-side read depth), when asked for
        self.vplanes = buf((n_seq, n_kv_heads, cap_tokens, 4, D // 64), torch.int64) if values else None
        self.vscales = buf((n_seq, n_kv_heads, cap_tokens), torch.int16) if values else None
        self.c = bpkv_cache(n_seq, n_kv_heads, group, D, cap_tokens, 0, 1 if host else 0, 0,
                            self.planes.data_ptr(), self.scales.data_ptr(), self.k_rows.data_ptr(),
                            self.v_rows.data_ptr(), self.seq_len.data_ptr(), None,
                            self.vplanes.data_ptr() if values else None, self.vscales.data_ptr() if values else None)
        # device row cache of recently selected rows (host-resident caches)
        self.rc_rows = self.rc_tok = None
        if rc_slots:
            self.rc_rows = torch.empty((n_seq, n_kv_heads, rc_slots, 2, D), dtype=torch.bfloat16, device=self.device)
            self.rc_tok = torch.full((n_seq, n_kv_heads, rc_slots), -1, dtype=torch.int32, device=self.device)
            self.c.rc_rows = self.rc_rows.data_ptr()
            self.c.rc_tok = self.rc_tok.data_ptr()
            self.c.rc_slots = rc_slots

    def set_basis(self, basis):
        """Code the keys in an orthogonal basis R, float [H][D][D] on the device
        (None: the raw channels); set it before the first append."""
        self.basis = None if basis is None else basis.contiguous()
        self.c.basis = None if basis is None else self.basis.data_ptr()

    @property
    def n_max(self) -> int:
        return int(self.c.n_max)

    def append(self, k_new, v_new, stream=None):
        """Append k_new/v_new [N][H][t][D] bf16 (device) to every sequence."""
        bpkv_encode_append(self.c, k_new, v_new, k_new.shape[2], stream)

    def copy_from(self, other: "Cache"):
        """Take over another cache's contents (same shapes), e.g. a host-resident
        copy of a cache built in device memory; copies run on the current stream."""
        for name in ("planes", "scales", "k_rows", "v_rows", "seq_len", "vplanes", "vscales"):
            if getattr(self, name) is not None and getattr(other, name) is not None:
                getattr(self, name).copy_(getattr(other, name), non_blocking=True)
        self.c.n_max = other.c.n_max

    def workspace(self, k: int, what: int):
        import torch
        n = bpkv_workspace_size(self.c, k, what)
        if n == 0:
            raise BpkvError("bpkv_workspace_size", -1)
        return torch.empty(n, dtype=torch.uint8, device=self.device)


def _check_arg(fn, name, x, dtype, shape, device):
    """A tensor that a kernel reads or writes at its address alone: raises unless it is what the kernel takes it for.
    None and raw addresses pass."""
    if x is None or isinstance(x, int):
        return
    if x.shape != shape or x.dtype is not dtype or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{fn}: {name} must be {dtype} {shape}, contiguous, on {device}; "
                         f"got {x.dtype} {tuple(x.shape)} with strides {x.stride()} on {x.device}")


def _check_status(fn, status, device):
    """A status word: the first four bytes of a tensor (a workspace has one too)."""
    if status is not None and not isinstance(status, int) and (
            status.device != device or status.numel() * status.element_size() < 4):
        raise ValueError(f"{fn}: status must have four bytes on {device}")


class Rows8:
    """One layer's cache of 8-bit K and V rows (e4m3 codes, one power-of-two
    scale per row) for N sequences x H KV heads, in device memory."""

    def __init__(self, n_seq: int, n_kv_heads: int, group: int, cap_tokens: int, device="cuda"):
        import torch
        if cap_tokens % 512:
            raise ValueError("cap_tokens must be a multiple of 512")
        self.device = torch.device(device)
        rows = (n_seq, n_kv_heads, cap_tokens)
        self.k8 = torch.empty((*rows, HEAD_DIM), dtype=torch.uint8, device=self.device)
        self.v8 = torch.empty((*rows, HEAD_DIM), dtype=torch.uint8, device=self.device)
        self.kexp = torch.empty(rows, dtype=torch.uint8, device=self.device)
        self.vexp = torch.empty(rows, dtype=torch.uint8, device=self.device)
        self.seq_len = torch.zeros(n_seq, dtype=torch.int64, device=self.device)
        self.c = bpkv_rows8(n_seq, n_kv_heads, group, HEAD_DIM, cap_tokens, 0, self.k8.data_ptr(), self.v8.data_ptr(),
                            self.kexp.data_ptr(), self.vexp.data_ptr(), self.seq_len.data_ptr())

    @property
    def n_max(self) -> int:
        """What the host knows the sequences' lengths to be at most.  Every
        append adds its tokens, also one that overwrites rows (start given):
        set it when the lengths are known to be less, or more."""
        return int(self.c.n_max)

    @n_max.setter
    def n_max(self, tokens: int):
        if not 0 <= tokens <= self.c.cap_tokens:
            raise ValueError(f"n_max must be 0 .. {self.c.cap_tokens}")
        self.c.n_max = int(tokens)

    def append(self, k_new, v_new, start=None, status=None, stream=None):
        """Quantise k_new/v_new [N][H][t][D] bf16 (device) behind every
        sequence's rows, or at rows start[i] .. (int64 [N], device).  ValueError
        for tensors of another type, shape or device, or with other strides."""
        import torch
        device = self.k8.device
        t = k_new.shape[2] if k_new.dim() == 4 else 0
        shape = (self.c.n_seq, self.c.n_kv_heads, t, HEAD_DIM)
        _check_arg("Rows8.append", "k_new", k_new, torch.bfloat16, shape, device)
        _check_arg("Rows8.append", "v_new", v_new, torch.bfloat16, shape, device)
        _check_arg("Rows8.append", "start", start, torch.int64, shape[:1], device)
        _check_status("Rows8.append", status, device)
        bpkv_rows8_append(self.c, k_new, v_new, t, start, status, stream)

    def read(self, t0: int, n: int, stream=None):
        """(K, V) rows t0 .. t0 + n - 1 of every sequence, bf16 [N][H][n][D]; zeros past its length."""
        import torch
        shape = (self.c.n_seq, self.c.n_kv_heads, n, HEAD_DIM)
        k = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
        v = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
        bpkv_rows8_read(self.c, t0, n, k, v, stream)
        return k, v


def qkv_args(qkv, q_out, n_kv_heads: int, pos=None, inv_freq=None, q_weight=None, k_weight=None, eps: float = 1e-6,
             pairs: bool = False, k_out=None, v_out=None, rows8=None, status=None):
    """bpkv_qkv_args for qkv [N][t][>= (G + 2) H D] bf16 (its last dimension
    dense) and q_out [N][t][H][G][D] float32 or bf16; inv_freq [rot / 2]
    float32 says how many channels are rotated; rows8: a Rows8.  All on one
    device.  The struct keeps the tensors it points to alive."""
    import torch
    N, t = qkv.shape[0], qkv.shape[1]
    H, G = q_out.shape[2], q_out.shape[3]

    def need(ok, what):
        if not ok:
            raise ValueError(f"qkv_args: {what}")

    need(qkv.dtype == torch.bfloat16 and qkv.dim() == 3 and qkv.stride(2) == 1, "qkv must be bf16 [N][t][row]")
    need(N == 1 or t == 1 or qkv.stride(0) == t * qkv.stride(1), "qkv's tokens must lie one stride apart")
    need(H == n_kv_heads and q_out.shape == (N, t, H, G, HEAD_DIM) and q_out.is_contiguous(), "q_out's shape")
    need(q_out.dtype in (torch.float32, torch.bfloat16), "q_out must be float32 or bf16")
    need(qkv.shape[2] >= (G + 2) * H * HEAD_DIM, "qkv's rows hold (G + 2) H heads")
    device = qkv.device
    need(q_out.device == device and (rows8 is None or rows8.k8.device == device), "tensors on several devices")
    for name, x, dt, shape in (("pos", pos, torch.int64, (N,)), ("q_weight", q_weight, torch.float32, (HEAD_DIM,)),
                               ("k_weight", k_weight, torch.float32, (HEAD_DIM,)),
                               ("k_out", k_out, torch.bfloat16, (N, H, t, HEAD_DIM)),
                               ("v_out", v_out, torch.bfloat16, (N, H, t, HEAD_DIM))):
        _check_arg("qkv_args", name, x, dt, shape, device)
    if inv_freq is not None:
        need(inv_freq.dim() == 1, "inv_freq must be float32 [rot / 2]")
        _check_arg("qkv_args", "inv_freq", inv_freq, torch.float32, tuple(inv_freq.shape), device)
    _check_status("qkv_args", status, device)
    # one token of one sequence has no stride between tokens; of several sequences it is theirs
    ld = qkv.stride(1) if t > 1 else qkv.stride(0) if N > 1 else qkv.shape[2] // 8 * 8

    def p(x):
        return None if x is None else x.data_ptr()

    a = bpkv_qkv_args(N, H, G, HEAD_DIM, t, 0 if inv_freq is None else 2 * inv_freq.numel(),
                      (QKV_PAIRS if pairs else 0) | (QKV_Q_BF16 if q_out.dtype == torch.bfloat16 else 0), eps, p(qkv),
                      ld, p(pos), p(inv_freq), p(q_weight), p(k_weight), p(q_out), p(k_out), p(v_out),
                      ctypes.pointer(rows8.c) if rows8 is not None else None, p(status))
    a.keep = (qkv, q_out, pos, inv_freq, q_weight, k_weight, k_out, v_out, rows8, status)
    return a


def shared_workspace(cache, prefix=None):
    """Workspace (uint8, device) of bpkv_shared_attend / bpkv_shared_attend8 for a Cache or Rows8 and its
    prefixes; its status word is clear."""
    import torch
    c = cache.c
    n = bpkv_shared_workspace_size(c.n_seq, 0 if prefix is None else prefix.c.n_seq, c.n_kv_heads, c.group)
    if n == 0:
        raise BpkvError("bpkv_shared_workspace_size", -4)
    ws = torch.empty(n, dtype=torch.uint8, device=cache.device)
    ws[:256].zero_()
    return ws


def cache_array(caches):
    """ctypes array of the bpkv_cache structs of several layers (for bpkv_decode_step)."""
    arr = (bpkv_cache * len(caches))(*[c.c for c in caches])
    return arr


def sync_n_max(caches, arr):
    """Copy n_max back from a cache array after bpkv_decode_step raised it."""
    for c, s in zip(caches, arr):
        c.c.n_max = s.n_max


__all__ = [n for n in dir() if n.startswith("bpkv_")] + ["Cache", "Rows8", "cache_array", "qkv_args", "shared_workspace", "sync_n_max", "BpkvError"]
_ = ctypes
