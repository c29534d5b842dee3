"""ctypes binding of libnys (include/nys.h): same names, argument marshalling only.

Every operation runs in the CUDA kernels of libnys.so.  Importing this module
raises ImportError if the library has not been built, and every call raises
NysError on a non-zero status: there is no fallback.

``NystromStates`` is a convenience wrapper that keeps the state buffer in a
torch tensor and passes torch tensors' device pointers and the current torch
stream to the C calls.
"""
from __future__ import annotations

import ctypes
import math
import os

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnys.so")

NYS_OK = 0
NYS_E_INVAL = -1
NYS_E_RANGE = -2
NYS_E_NOT_SEALED = -3
NYS_E_EXACT_ONLY = -4
NYS_E_BUF = -5
NYS_E_ALIGN = -6
NYS_E_CUDA = -7
NYS_E_UNSUPPORTED = -8
NYS_E_SCRATCH = -9
NYS_E_CAPACITY = -10
NYS_RECT_AGGREGATE = 0
NYS_RECT_FM = 1
NYS_F32 = 0
NYS_BF16 = 1
NYS_F16 = 2
NYS_ATTN_GAVE_UP = 1
NYS_ATTN_BAD_OFFSETS = 2
NYS_ATTN_BAD_PAGE = 4
NYS_ATTN_BAD_LENGTH = 8
NYS_PLAN_BAD_LENGTH = 16
NYS_PLAN_NO_PAGES = 32
NYS_PLAN_TABLE_FULL = 64

# Every entry point include/nys.h declares.
EXPORTED = ("nys_memory_bytes", "nys_alloc_states", "nys_free_states",
            "nys_seal", "nys_step_batch", "nys_query", "nys_layout_of",
            "nys_mark_sealed", "nys_config_of", "nys_strerror",
            "nys_seal_static", "nys_seal_ragged", "nys_o1_begin", "nys_o1_push_q",
            "nys_o1_seal", "nys_o1_sealed", "nys_o1_step", "nys_o1_memory_bytes",
            "nys_o1_states", "nys_o1_free", "nys_debug_stall_once",
            "nys_debug_stall_replay_once", "nys_attn_workspace_bytes",
            "nys_attn_prompt", "nys_attn_shared", "nys_kv_plan", "nys_kv_write",
            "nys_debug_stall_attn_once", "nys_qk_rows", "nys_kv_append",
            "nys_kv4_page_bytes", "nys_kv4_write", "nys_kv4_append", "nys_kv4_read",
            "nys_attn4_workspace_bytes", "nys_attn4")


class NysConfig(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int32), ("w", ctypes.c_int32),
                ("sink", ctypes.c_int32), ("heads_per_kv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("rect", ctypes.c_int32), ("exact_cap", ctypes.c_int32)]


class NysLayout(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_size_t),
                ("off_win_k", ctypes.c_size_t), ("off_win_v", ctypes.c_size_t),
                ("off_sink_k", ctypes.c_size_t), ("off_sink_v", ctypes.c_size_t),
                ("off_k_tilde", ctypes.c_size_t), ("off_q_tilde", ctypes.c_size_t),
                ("off_mu", ctypes.c_size_t), ("off_t_hat", ctypes.c_size_t),
                ("off_z_hat", ctypes.c_size_t), ("off_m_max", ctypes.c_size_t),
                ("off_t_lo", ctypes.c_size_t), ("off_z_lo", ctypes.c_size_t),
                ("off_far_len", ctypes.c_size_t), ("off_ints", ctypes.c_size_t),
                ("off_exact_k", ctypes.c_size_t), ("off_exact_v", ctypes.c_size_t),
                ("n_groups", ctypes.c_int64), ("ints_per_group", ctypes.c_int32)]


class NysGroupInfo(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("m_eff", ctypes.c_int32),
                ("t", ctypes.c_int32), ("win_len", ctypes.c_int32),
                ("win_head", ctypes.c_int32), ("status", ctypes.c_int32)]


class NysAttnConfig(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class NysRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class NysPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("page", ctypes.c_int32)]


class NysPool4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page", ctypes.c_int32)]


class NysQkPrepare(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("turns", ctypes.c_void_p), ("rot", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("shift", ctypes.c_int32)]


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with "
            "`python -m streaming_nystr_landmark_gb300.build` (nvcc, sm_103a)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I64, I32, VP = ctypes.POINTER, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    sig = {
        "nys_memory_bytes": [P(NysConfig), I64, P(ctypes.c_size_t)],
        "nys_alloc_states": [P(NysConfig), I64, VP, ctypes.c_size_t, P(VP)],
        "nys_free_states": [VP],
        "nys_seal": [VP, I64, I64, I32, VP, VP, VP, VP],
        "nys_step_batch": [VP, I64, I64, VP, VP, VP, VP, VP],
        "nys_query": [VP, I64, P(NysGroupInfo), P(I32), VP],
        "nys_layout_of": [VP, P(VP), P(NysLayout)],
        "nys_mark_sealed": [VP, I64, I64],
        "nys_config_of": [VP, P(NysConfig), P(I64)],
        "nys_strerror": [ctypes.c_int],
        "nys_seal_static": [VP, I64, I64, I32, VP, VP, VP, VP],
        "nys_seal_ragged": [VP, I64, I64, P(I32), VP, VP, VP, VP],
        "nys_o1_begin": [P(NysConfig), I32, I32, I32, I32, P(VP)],
        "nys_o1_push_q": [VP, VP, VP],
        "nys_o1_seal": [VP, VP, VP, I32, I32, VP, P(I32)],
        "nys_o1_sealed": [VP, P(I32)],
        "nys_o1_step": [VP, VP, VP, VP, VP, VP],
        "nys_o1_memory_bytes": [VP, P(ctypes.c_size_t)],
        "nys_o1_states": [VP, P(VP)],
        "nys_o1_free": [VP],
        "nys_debug_stall_once": [VP, I32],
        "nys_debug_stall_replay_once": [VP],
        "nys_attn_workspace_bytes": [P(NysAttnConfig), I64, I64, I64, P(ctypes.c_size_t)],
        "nys_attn_prompt": [P(NysAttnConfig), I64, I64, I64, VP, VP, P(NysRows), P(NysRows),
                            P(NysRows), P(NysRows), VP, VP, ctypes.c_size_t, VP, VP],
        "nys_attn_shared": [P(NysAttnConfig), I64, P(NysPool), VP, I32, VP, VP, I32,
                            P(NysRows), P(NysRows), VP, VP, ctypes.c_size_t, VP, VP],
        "nys_kv_plan": [I64, I32, VP, VP, VP, I64, VP, I32, I64, VP, VP, VP, VP, VP, VP, VP],
        "nys_kv_write": [P(NysAttnConfig), P(NysPool), I64, P(NysRows), P(NysRows), VP, VP],
        "nys_debug_stall_attn_once": [I32],
        "nys_qk_rows": [P(NysAttnConfig), P(NysQkPrepare), I64, P(NysRows), P(NysRows), VP,
                        P(NysRows), P(NysRows), VP],
        "nys_kv_append": [P(NysAttnConfig), P(NysQkPrepare), P(NysPool), I64, P(NysRows),
                          P(NysRows), P(NysRows), VP, VP, P(NysRows), P(NysRows), VP],
        "nys_kv4_page_bytes": [P(NysAttnConfig), I32, P(ctypes.c_size_t)],
        "nys_kv4_write": [P(NysAttnConfig), P(NysPool4), I64, P(NysRows), P(NysRows), VP, VP],
        "nys_kv4_append": [P(NysAttnConfig), P(NysQkPrepare), P(NysPool4), I64, P(NysRows),
                           P(NysRows), P(NysRows), VP, VP, P(NysRows), P(NysRows), VP],
        "nys_kv4_read": [P(NysAttnConfig), P(NysPool4), I64, VP, P(NysRows), P(NysRows), VP],
        "nys_attn4_workspace_bytes": [P(NysAttnConfig), I64, I64, P(ctypes.c_size_t)],
        "nys_attn4": [P(NysAttnConfig), I64, P(NysPool4), VP, VP, I32, P(NysRows), P(NysRows),
                      VP, P(NysRows), VP, VP, ctypes.c_size_t, VP, VP],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name == "nys_strerror" else ctypes.c_int
    return lib


_lib = _load()


class NysError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {nys_strerror(code)} (status {code})")


def _check(code: int, where: str):
    if code != NYS_OK:
        raise NysError(code, where)


def nys_strerror(code: int) -> str:
    return _lib.nys_strerror(code).decode()


def make_config(m, w, sink, heads_per_kv, d, dv, rect=NYS_RECT_AGGREGATE,
                exact_cap=0) -> NysConfig:
    return NysConfig(m, w, sink, heads_per_kv, d, dv, rect, exact_cap)


def nys_memory_bytes(cfg: NysConfig, n_groups: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.nys_memory_bytes(ctypes.byref(cfg), n_groups, ctypes.byref(out)),
           "nys_memory_bytes")
    return out.value


def nys_alloc_states(cfg: NysConfig, n_groups: int, dev_buf: int = 0,
                     buf_bytes: int = 0) -> int:
    h = ctypes.c_void_p(0)
    _check(_lib.nys_alloc_states(ctypes.byref(cfg), n_groups, dev_buf or None,
                                 buf_bytes, ctypes.byref(h)), "nys_alloc_states")
    return h.value


def nys_free_states(handle: int):
    _check(_lib.nys_free_states(handle), "nys_free_states")


def nys_seal(handle, g0, n, t, q, k, v, stream=0):
    _check(_lib.nys_seal(handle, g0, n, t, q, k, v, stream or None), "nys_seal")


def nys_seal_static(handle, g0, n, t, q, k, v, stream=0):
    """nys_seal with the library's static workspace instead of an allocation
    (for callers that cannot allocate device memory while they run)."""
    _check(_lib.nys_seal_static(handle, g0, n, t, q, k, v, stream or None),
           "nys_seal_static")


def nys_seal_ragged(handle, g0, t_list, q, k, v, stream=0):
    """Seal len(t_list) groups from g0 on prompts of the given lengths,
    packed back to back (see include/nys.h)."""
    n = len(t_list)
    arr = (ctypes.c_int32 * max(n, 1))(*t_list)
    _check(_lib.nys_seal_ragged(handle, g0, n, arr, q, k, v, stream or None),
           "nys_seal_ragged")


def nys_step_batch(handle, g0, n, q, k, v, out, stream=0):
    _check(_lib.nys_step_batch(handle, g0, n, q, k, v, out, stream or None),
           "nys_step_batch")


def nys_query(handle, g, heads, stream=0):
    info = NysGroupInfo()
    far = (ctypes.c_int32 * heads)()
    _check(_lib.nys_query(handle, g, ctypes.byref(info), far, stream or None),
           "nys_query")
    return ({"mode": info.mode, "m_eff": info.m_eff, "t": info.t,
             "win_len": info.win_len, "win_head": info.win_head,
             "status": info.status}, list(far))


def nys_debug_stall_once(handle, stage):
    _check(_lib.nys_debug_stall_once(handle, stage), "nys_debug_stall_once")


def nys_debug_stall_replay_once(handle):
    _check(_lib.nys_debug_stall_replay_once(handle), "nys_debug_stall_replay_once")


def nys_layout_of(handle):
    base = ctypes.c_void_p(0)
    lay = NysLayout()
    _check(_lib.nys_layout_of(handle, ctypes.byref(base), ctypes.byref(lay)),
           "nys_layout_of")
    return base.value, lay


def nys_mark_sealed(handle, g0, n):
    _check(_lib.nys_mark_sealed(handle, g0, n), "nys_mark_sealed")


def nys_config_of(handle):
    cfg = NysConfig()
    n = ctypes.c_int64(0)
    _check(_lib.nys_config_of(handle, ctypes.byref(cfg), ctypes.byref(n)),
           "nys_config_of")
    return cfg, n.value


def nys_attn_workspace_bytes(cfg: NysAttnConfig, n: int, rows: int, keys: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.nys_attn_workspace_bytes(ctypes.byref(cfg), n, rows, keys, ctypes.byref(out)),
           "nys_attn_workspace_bytes")
    return out.value


def nys_attn_prompt(cfg, n, q_rows, k_rows, q_off, k_off, q, k, v, out, lse=None,
                    workspace=None, workspace_bytes=0, status=None, stream=0):
    """q, k, v, out: NysRows; the offsets and the rest: device addresses."""
    _check(_lib.nys_attn_prompt(cfg, n, q_rows, k_rows, q_off, k_off, q, k, v, out, lse,
                                workspace, workspace_bytes, status, stream or None),
           "nys_attn_prompt")


def nys_attn_shared(cfg, n, pool, prefix_pages, prefix_len, lens, table, width, q, out,
                    lse=None, workspace=None, workspace_bytes=0, status=None, stream=0):
    """q, out: NysRows; pool: NysPool; the rest: device addresses."""
    _check(_lib.nys_attn_shared(cfg, n, pool, prefix_pages, prefix_len, lens, table, width,
                                q, out, lse, workspace, workspace_bytes, status,
                                stream or None), "nys_attn_shared")


def nys_kv_plan(n, page, cached, fresh, free_pages, n_free, table, width, total, q_off,
                lens, slots, positions, taken, status=None, stream=0):
    _check(_lib.nys_kv_plan(n, page, cached, fresh, free_pages, n_free, table, width, total,
                            q_off, lens, slots, positions, taken, status, stream or None),
           "nys_kv_plan")


def nys_debug_stall_attn_once(role):
    _check(_lib.nys_debug_stall_attn_once(role), "nys_debug_stall_attn_once")


def nys_kv_write(cfg, pool, tokens, k, v, slots, stream=0):
    _check(_lib.nys_kv_write(cfg, pool, tokens, k, v, slots, stream or None), "nys_kv_write")


def nys_qk_rows(cfg, prep, tokens, q, k, positions, q_out, k_out, stream=0):
    """q, k, q_out, k_out: NysRows or None; positions: a device address."""
    _check(_lib.nys_qk_rows(cfg, prep, tokens, q, k, positions, q_out, k_out, stream or None),
           "nys_qk_rows")


def nys_kv_append(cfg, prep, pool, tokens, q, k, v, positions, slots, q_out=None, k_out=None,
                  stream=0):
    _check(_lib.nys_kv_append(cfg, prep, pool, tokens, q, k, v, positions, slots, q_out, k_out,
                              stream or None), "nys_kv_append")


def nys_kv4_page_bytes(cfg: NysAttnConfig, page: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.nys_kv4_page_bytes(ctypes.byref(cfg), page, ctypes.byref(out)),
           "nys_kv4_page_bytes")
    return out.value


def nys_kv4_write(cfg, pool, tokens, k, v, slots, stream=0):
    _check(_lib.nys_kv4_write(cfg, pool, tokens, k, v, slots, stream or None), "nys_kv4_write")


def nys_kv4_append(cfg, prep, pool, tokens, q, k, v, positions, slots, q_out=None, k_out=None,
                   stream=0):
    _check(_lib.nys_kv4_append(cfg, prep, pool, tokens, q, k, v, positions, slots, q_out, k_out,
                               stream or None), "nys_kv4_append")


def nys_kv4_read(cfg, pool, tokens, slots, k_out, v_out, stream=0):
    _check(_lib.nys_kv4_read(cfg, pool, tokens, slots, k_out, v_out, stream or None),
           "nys_kv4_read")


def nys_attn4_workspace_bytes(cfg: NysAttnConfig, n: int, keys: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.nys_attn4_workspace_bytes(ctypes.byref(cfg), n, keys, ctypes.byref(out)),
           "nys_attn4_workspace_bytes")
    return out.value


def nys_attn4(cfg, n, pool, lens, table, width, q, out, first=None, first_lse=None, lse=None,
              workspace=None, workspace_bytes=0, status=None, stream=0):
    """q, out, first: NysRows; pool: NysPool4; the rest: device addresses."""
    _check(_lib.nys_attn4(cfg, n, pool, lens, table, width, q, first, first_lse, out, lse,
                          workspace, workspace_bytes, status, stream or None), "nys_attn4")


# ---------------------------------------------------------------- torch wrapper
def _ptr(t, dtype, shape, where):
    import torch
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{where}: need a contiguous CUDA {dtype} tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{where}: shape {tuple(t.shape)} != {tuple(shape)}")
    return t.data_ptr()


class NystromStates:
    """A batch of group states in one torch-owned device buffer."""

    def __init__(self, m, w, sink, heads_per_kv, d, dv, n_groups,
                 rect=NYS_RECT_AGGREGATE, device="cuda", exact_cap=0):
        import torch
        self.torch = torch
        self.cfg = make_config(m, w, sink, heads_per_kv, d, dv, rect, exact_cap)
        self.n_groups = n_groups
        self.device = torch.device(device)
        nbytes = nys_memory_bytes(self.cfg, n_groups)
        self.buf = torch.empty(max(nbytes, 1) + 256, dtype=torch.uint8,
                               device=self.device)
        base = self.buf.data_ptr()
        self._off = (-base) % 256
        self.handle = nys_alloc_states(self.cfg, n_groups, base + self._off, nbytes)
        self.base, self.layout = nys_layout_of(self.handle)

    def close(self):
        if getattr(self, "handle", None):
            nys_free_states(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _stream(self):
        return self.torch.cuda.current_stream(self.device).cuda_stream

    def seal(self, q, k, v, g0=0, n=None):
        c = self.cfg
        n = k.shape[0] if n is None else n
        t = k.shape[1]
        torch = self.torch
        nys_seal(self.handle, g0, n, t,
                 _ptr(q, torch.float32, (n, c.heads_per_kv, t, c.d), "q"),
                 _ptr(k, torch.float32, (n, t, c.d), "k"),
                 _ptr(v, torch.float32, (n, t, c.dv), "v"), self._stream())

    def seal_ragged(self, t_list, q, k, v, g0=0):
        """Seal groups g0.. on prompts of lengths t_list packed back to back:
        k [sum t][d], v [sum t][dv], q [H * sum t][d] (per group [H][t][d])."""
        c = self.cfg
        torch = self.torch
        total = int(sum(t_list))
        nys_seal_ragged(self.handle, g0, list(t_list),
                        _ptr(q, torch.float32, (c.heads_per_kv * total, c.d), "q"),
                        _ptr(k, torch.float32, (total, c.d), "k"),
                        _ptr(v, torch.float32, (total, c.dv), "v"), self._stream())

    def step(self, q, k, v, out, g0=0, n=None):
        c = self.cfg
        n = k.shape[0] if n is None else n
        torch = self.torch
        nys_step_batch(self.handle, g0, n,
                       _ptr(q, torch.float32, (n, c.heads_per_kv, c.d), "q"),
                       _ptr(k, torch.float32, (n, c.d), "k"),
                       _ptr(v, torch.float32, (n, c.dv), "v"),
                       _ptr(out, torch.float32, (n, c.heads_per_kv, c.dv), "out"),
                       self._stream())
        return out

    def step_host(self, hq, hk, hv, hout, dq, dk, dv, dout):
        """One token from pinned host buffers: copy q/k/v to the device
        staging tensors, launch nys_step_batch, copy the outputs back to
        ``hout``; everything is enqueued on the current stream."""
        dq.copy_(hq, non_blocking=True)
        dk.copy_(hk, non_blocking=True)
        dv.copy_(hv, non_blocking=True)
        self.step(dq, dk, dv, dout)
        hout.copy_(dout, non_blocking=True)
        return hout

    def host_pipeline(self, n=None, depth=2):
        """A pipelined host-buffer driver for this handle (see HostPipeline)."""
        return HostPipeline(self, self.n_groups if n is None else n, depth)

    def query(self, g):
        return nys_query(self.handle, g, self.cfg.heads_per_kv, self._stream())

    def debug_stall_once(self, stage):
        """Test hook: the next step's first CTA withholds ring stage `stage`,
        so its bounded waits run out and its groups report status 1."""
        nys_debug_stall_once(self.handle, stage)

    def debug_stall_replay_once(self):
        """Test hook: the next seal's tensor-core replay withholds its first
        CTA's first MMAs; that group reports status 3."""
        nys_debug_stall_replay_once(self.handle)

    def region(self, name):
        """A torch view of one state region, shaped as nys_layout documents."""
        torch = self.torch
        c, G = self.cfg, self.n_groups
        H, m = c.heads_per_kv, c.m
        shapes = {
            "win_k": (torch.float32, (G, c.w, c.d)),
            "win_v": (torch.float32, (G, c.w, c.dv)),
            "sink_k": (torch.float32, (G, c.sink, c.d)),
            "sink_v": (torch.float32, (G, c.sink, c.dv)),
            "k_tilde": (torch.float32, (G, m, c.d)),
            "q_tilde": (torch.float32, (G, H, m, c.d)),
            "mu": (torch.float32, (G, H, m, m)),
            "t_hat": (torch.float32, (G, H, m, c.dv)),
            "z_hat": (torch.float32, (G, H, m)),
            "m_max": (torch.float32, (G, H, m)),
            "t_lo": (torch.bfloat16, (G, H, m, c.dv)),
            "z_lo": (torch.float32, (G, H, m)),
            "far_len": (torch.int32, (G, H)),
            "ints": (torch.int32, (G, self.layout.ints_per_group)),
            "exact_k": (torch.float32, (G, c.exact_cap, c.d)),
            "exact_v": (torch.float32, (G, c.exact_cap, c.dv)),
        }
        dtype, shape = shapes[name]
        off = getattr(self.layout, "off_" + name) + self._off
        count = 1
        for s in shape:
            count *= s
        size = 2 if dtype == torch.bfloat16 else 4
        raw = self.buf[off: off + size * count]
        return raw.view(dtype).view(shape)

    def far_numerator(self):
        """T^ = t_hat + t_lo as float64 on the host (test helper)."""
        return (self.region("t_hat").double() + self.region("t_lo").double()).cpu().numpy()

    def far_denominator(self):
        """Z^ = z_hat + z_lo as float64 on the host (test helper)."""
        return (self.region("z_hat").double() + self.region("z_lo").double()).cpu().numpy()

    def mark_sealed(self, g0=0, n=None):
        nys_mark_sealed(self.handle, g0, self.n_groups if n is None else n)


class HostPipeline:
    """Decode tokens from pinned host buffers with copies overlapped.

    Each ``submit`` enqueues, for one token: the host->device copy of q, k, v
    on an upload stream into one of ``depth`` device staging slots, the
    decode launch on the compute stream once that copy has landed, and the
    device->host copy of the outputs on a separate download stream once the
    launch is done.  Token n+1's inputs therefore travel while token n
    computes (uploads never queue behind downloads), and a staging slot is
    reused only after the launch that read it has finished.
    ``synchronize`` waits for everything submitted.  All ordering is by CUDA
    events; the decode itself is nys_step_batch.
    """

    def __init__(self, states, n, depth=2):
        import torch
        self.torch = torch
        self.st = states
        self.n = n
        c = states.cfg
        dev = states.device
        self.compute = torch.cuda.current_stream(dev)
        self.copy = torch.cuda.Stream(dev)      # uploads
        self.down = torch.cuda.Stream(dev)      # downloads
        mk = lambda *shape: torch.empty(shape, device=dev)
        self.slots = [dict(q=mk(n, c.heads_per_kv, c.d), k=mk(n, c.d), v=mk(n, c.dv),
                           out=mk(n, c.heads_per_kv, c.dv),
                           loaded=torch.cuda.Event(), done=torch.cuda.Event(),
                           drained=torch.cuda.Event())
                      for _ in range(depth)]
        for sl in self.slots:
            sl["done"].record(self.compute)
            sl["drained"].record(self.down)
        self.i = 0

    def submit(self, hq, hk, hv, hout):
        sl = self.slots[self.i % len(self.slots)]
        self.i += 1
        with self.torch.cuda.stream(self.copy):
            self.copy.wait_event(sl["done"])       # the last launch read this slot
            sl["q"].copy_(hq, non_blocking=True)
            sl["k"].copy_(hk, non_blocking=True)
            sl["v"].copy_(hv, non_blocking=True)
            sl["loaded"].record(self.copy)
        self.compute.wait_event(sl["loaded"])
        self.compute.wait_event(sl["drained"])      # its previous outputs left
        self.st.step(sl["q"], sl["k"], sl["v"], sl["out"])
        sl["done"].record(self.compute)
        with self.torch.cuda.stream(self.down):
            self.down.wait_event(sl["done"])
            hout.copy_(sl["out"], non_blocking=True)
            sl["drained"].record(self.down)

    def synchronize(self):
        self.torch.cuda.synchronize(self.st.device)


class O1Layer:
    """One attention layer's O(1) override for a batch of sequences (the
    LayerKvCache o1 lifecycle: begin -> push_q per prompt position -> seal ->
    step per decode token), over the nys_o1_* calls."""

    def __init__(self, m, w, sink, d, dv, batch, num_heads, num_kv_heads, max_prompt,
                 rect=NYS_RECT_AGGREGATE, exact_cap=0, device="cuda"):
        import torch
        self.torch = torch
        self.device = torch.device(device)
        self.cfg = make_config(m, w, sink, 1, d, dv, rect, exact_cap)
        self.batch, self.num_heads, self.num_kv = batch, num_heads, num_kv_heads
        h = ctypes.c_void_p(0)
        _check(_lib.nys_o1_begin(ctypes.byref(self.cfg), batch, num_heads, num_kv_heads,
                                 max_prompt, ctypes.byref(h)), "nys_o1_begin")
        self.handle = h.value

    def _stream(self):
        return self.torch.cuda.current_stream(self.device).cuda_stream

    def push_q(self, q_all):
        c = self.cfg
        _check(_lib.nys_o1_push_q(self.handle, _ptr(q_all, self.torch.float32,
                                                    (self.batch, self.num_heads, c.d), "q_all"),
                                  self._stream()), "nys_o1_push_q")

    def seal(self, k, v, kv_dense=True):
        """k [batch][num_kv][t][d], v [..][dv]; True when sealed."""
        c = self.cfg
        t = k.shape[2]
        flag = ctypes.c_int32(0)
        _check(_lib.nys_o1_seal(
            self.handle,
            _ptr(k, self.torch.float32, (self.batch, self.num_kv, t, c.d), "k"),
            _ptr(v, self.torch.float32, (self.batch, self.num_kv, t, c.dv), "v"),
            t, int(bool(kv_dense)), self._stream(), ctypes.byref(flag)), "nys_o1_seal")
        return bool(flag.value)

    def sealed(self):
        flag = ctypes.c_int32(0)
        _check(_lib.nys_o1_sealed(self.handle, ctypes.byref(flag)), "nys_o1_sealed")
        return bool(flag.value)

    def step(self, q_all, k_new, v_new, out):
        c, f = self.cfg, self.torch.float32
        _check(_lib.nys_o1_step(
            self.handle, _ptr(q_all, f, (self.batch, self.num_heads, c.d), "q_all"),
            _ptr(k_new, f, (self.batch, self.num_kv, c.d), "k_new"),
            _ptr(v_new, f, (self.batch, self.num_kv, c.dv), "v_new"),
            _ptr(out, f, (self.batch, self.num_heads, c.dv), "out"), self._stream()),
            "nys_o1_step")
        return out

    def memory_bytes(self):
        out = ctypes.c_size_t(0)
        _check(_lib.nys_o1_memory_bytes(self.handle, ctypes.byref(out)), "nys_o1_memory_bytes")
        return out.value

    def close(self):
        if getattr(self, "handle", None):
            _check(_lib.nys_o1_free(self.handle), "nys_o1_free")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------- exact attention, paged cache
def _dtype_code(dtype):
    import torch
    codes = {torch.float32: NYS_F32, torch.bfloat16: NYS_BF16, torch.float16: NYS_F16}
    if dtype not in codes:
        raise ValueError(f"dtype {dtype}: need float32, bfloat16 or float16")
    return codes[dtype]


def _wrong_place(t, dtype, where, index):
    if t.dtype is dtype and t.is_cuda:
        raise ValueError(f"{where}: on cuda:{t.get_device()}, need cuda:{index}")
    raise ValueError(f"{where}: need a CUDA {dtype} tensor")


def _rows(t, dtype, heads, dim, where, index=None):
    """A [rows][heads][dim] CUDA tensor as NysRows: any row and head strides,
    the last dimension contiguous; on device `index`, if given."""
    if t.dtype is not dtype or (not t.is_cuda if index is None else t.get_device() != index):
        _wrong_place(t, dtype, where, index)
    shape, st = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{where}: shape {tuple(shape)} != (rows, {heads}, {dim})")
    if st[2] != 1 and dim > 1:
        raise ValueError(f"{where}: the last dimension must be contiguous")
    return NysRows(t.data_ptr(), st[0], st[1])


def _ints(t, dtype, shape, where, index=None):
    """Address of a contiguous CUDA tensor of this type and shape, on device
    `index`, if given."""
    if t.dtype is not dtype or (not t.is_cuda if index is None else t.get_device() != index):
        _wrong_place(t, dtype, where, index)
    if t.shape != shape:
        raise ValueError(f"{where}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: need a contiguous CUDA {dtype} tensor")
    return t.data_ptr()


def _cuda_device(device):
    """A torch.device with its index: "cuda" is the device current now."""
    import torch
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


class _OnDevice:
    """Calls are made with the object's device current (a legacy default stream is
    the current device's, whatever the tensors are), on its current torch stream,
    whose address _stream() gives without making an object: 0.1 us against 3.5."""

    def _elsewhere(self):
        return self.torch._C._cuda_getDevice() != self.device.index

    def _stream(self):
        return self.torch._C._cuda_getCurrentRawStream(self.device.index)


class _Status(_OnDevice):
    """A device status word that kernels set bits of (NYS_ATTN_*, NYS_PLAN_*)."""

    def _init_status(self, torch, device):
        self._status = torch.zeros(1, dtype=torch.int32, device=device)
        self._status_ptr = self._status.data_ptr()

    def share_status(self, other):
        """Reports into other's status word from here on."""
        self._status, self._status_ptr = other._status, other._status_ptr

    def status(self):
        """The status bits since the last clear (synchronises)."""
        return int(self._status.item())

    def clear_status(self):
        self._status.zero_()


class PagedKV(_OnDevice):
    """A pool of KV pages of one layer: k [n_pages][page][kv_heads][d],
    v [..][dv], allocated here or given.  Page numbers come from a PagePlan."""

    def __init__(self, n_pages, page, kv_heads, d, dv, dtype=None, device="cuda", k=None, v=None):
        import torch
        self.torch = torch
        self.dtype = torch.float32 if dtype is None else dtype
        self.device = _cuda_device(device)
        self.n_pages, self.page = n_pages, page
        self.kv_heads, self.d, self.dv = kv_heads, d, dv
        make = lambda c: torch.empty((n_pages, page, kv_heads, c), dtype=self.dtype,
                                     device=self.device)
        self.k = make(d) if k is None else k
        self.v = make(dv) if v is None else v
        for name, t, c in (("k", self.k, d), ("v", self.v, dv)):
            if (t.dtype != self.dtype or not t.is_cuda or not t.is_contiguous()
                    or tuple(t.shape) != (n_pages, page, kv_heads, c)
                    or t.get_device() != self.device.index):
                raise ValueError(f"{name}: need a contiguous {self.dtype} tensor of shape "
                                 f"{(n_pages, page, kv_heads, c)} on {self.device}")
        self._cfg = NysAttnConfig(kv_heads, kv_heads, d, dv, _dtype_code(self.dtype), 0.0)
        self._pool = NysPool(self.k.data_ptr(), self.v.data_ptr(), n_pages, page)

    def write(self, k, v, slots):
        """Rows k [tokens][kv_heads][d], v [..][dv] into slots int64 [tokens];
        a slot of -1 is skipped."""
        torch, index = self.torch, self.device.index
        if self._elsewhere():
            with torch.cuda.device(index):
                return self.write(k, v, slots)
        n = k.shape[0]
        if v.shape[0] != n:
            raise ValueError(f"v: {v.shape[0]} rows, k has {n}")
        nys_kv_write(self._cfg, self._pool, n,
                     _rows(k, self.dtype, self.kv_heads, self.d, "k", index),
                     _rows(v, self.dtype, self.kv_heads, self.dv, "v", index),
                     _ints(slots, torch.int64, (n,), "slots", index), self._stream())


class PagedKV4(_OnDevice):
    """A pool of KV pages of one layer in 4 bits (4.5 with their scales; nys.h says what
    a row is held as): `page` a multiple of 16.  Rows come and go in `dtype`.  data,
    uint8 [n_pages][kv_heads][bytes], is allocated here or given; pages that were
    never written hold whatever was there."""

    def __init__(self, n_pages, page, kv_heads, d, dv, dtype=None, device="cuda", data=None):
        import torch
        self.torch = torch
        self.dtype = torch.float32 if dtype is None else dtype
        self.device = _cuda_device(device)
        self.n_pages, self.page = n_pages, page
        self.kv_heads, self.d, self.dv = kv_heads, d, dv
        self._cfg = NysAttnConfig(kv_heads, kv_heads, d, dv, _dtype_code(self.dtype), 0.0)
        if page < 16 or page % 16:
            raise ValueError(f"page {page}: need a multiple of 16 tokens")
        shape = (n_pages, kv_heads, nys_kv4_page_bytes(self._cfg, page) // kv_heads)
        self.data = (torch.empty(shape, dtype=torch.uint8, device=self.device) if data is None
                     else data)
        if (self.data.dtype != torch.uint8 or not self.data.is_cuda
                or not self.data.is_contiguous() or tuple(self.data.shape) != shape
                or self.data.get_device() != self.device.index):
            raise ValueError(f"data: need a contiguous uint8 tensor of shape {shape} on "
                             f"{self.device}")
        self._pool = NysPool4(self.data.data_ptr(), n_pages, page)

    def write(self, k, v, slots):
        """Rows k [tokens][kv_heads][d], v [..][dv] into slots int64 [tokens] (no slot
        twice); a slot of -1 is skipped."""
        torch, index = self.torch, self.device.index
        if self._elsewhere():
            with torch.cuda.device(index):
                return self.write(k, v, slots)
        n = k.shape[0]
        if v.shape[0] != n:
            raise ValueError(f"v: {v.shape[0]} rows, k has {n}")
        nys_kv4_write(self._cfg, self._pool, n,
                      _rows(k, self.dtype, self.kv_heads, self.d, "k", index),
                      _rows(v, self.dtype, self.kv_heads, self.dv, "v", index),
                      _ints(slots, torch.int64, (n,), "slots", index), self._stream())

    def read(self, slots, k, v):
        """The rows in slots int64 [tokens] as the values they stand for, into k
        [tokens][kv_heads][d] and v [..][dv] of the cache's type; zeros for a slot of -1."""
        torch, index = self.torch, self.device.index
        if self._elsewhere():
            with torch.cuda.device(index):
                return self.read(slots, k, v)
        n = slots.shape[0]
        if k.shape[0] != n or v.shape[0] != n:
            raise ValueError(f"k and v must have a row for each of the {n} slots")
        nys_kv4_read(self._cfg, self._pool, n, _ints(slots, torch.int64, (n,), "slots", index),
                     _rows(k, self.dtype, self.kv_heads, self.d, "k", index),
                     _rows(v, self.dtype, self.kv_heads, self.dv, "v", index), self._stream())


class Rotation:
    """The rotation of the first `rot` (all, if not given) of a head's d numbers by their
    position: pair i turns by base^(-2i / rot), or by freqs[i], radians a position.  Pairs
    are numbers i and i + rot/2, or 2i and 2i + 1 (interleaved)."""

    # 2 pi to 50 digits, times 10^49.
    _TURN = 62831853071795864769252867665590057683943387987502

    def __init__(self, d, base=10000.0, rot=None, interleaved=False, freqs=None, device="cuda"):
        import torch
        rot = d if rot is None else rot
        if rot < 0 or rot % 2 or rot > d:
            raise ValueError(f"rot {rot}: need an even number of at most {d}")
        if freqs is None:
            if rot and not 1e-300 <= base < float("inf"):
                raise ValueError(f"base {base}: need a positive finite number")
            freqs = [float(base) ** (-2.0 * i / rot) for i in range(rot // 2)]
        freqs = [float(f) for f in freqs]
        if len(freqs) != rot // 2 or not all(math.isfinite(f) for f in freqs):
            raise ValueError(f"freqs: need {rot // 2} finite numbers")
        self.d, self.rot, self.interleaved = d, rot, bool(interleaved)
        self.device = _cuda_device(device)
        # Fractions of a turn in 64 bits; torch holds them as int64.
        turns = []
        for f in freqs:
            a, b = f.as_integer_ratio()
            a, b = a * 10 ** 49 << 64, b * self._TURN
            t = (2 * a + b) // (2 * b) % 2 ** 64      # to the nearest
            turns.append(t - 2 ** 64 if t >= 2 ** 63 else t)
        self.turns = torch.tensor(turns, dtype=torch.int64, device=self.device)


class QKPrepare(_OnDevice):
    """What stands between a layer's projections and its attention: RMS norms of queries
    and keys for each head (weights [d] or None) and their rotation (a Rotation or None),
    in one pass (``rows``), or in one with the write into the cache's pages (``append``).
    Calls on any stream may follow the constructor, which waits for its copies of the
    weights; the object's memory stays until the calls that are queued are through.  One
    whose calls a CUDA graph has captured has to stay for the graph's replays."""

    _private = ()             # tensors of this object's own
    _streams = frozenset()    # that their allocator knows to be reading them

    def __init__(self, heads, kv_heads, d, dtype=None, q_weight=None, k_weight=None, eps=1e-6,
                 rotation=None, device="cuda"):
        import torch
        self.torch = torch
        self.dtype = torch.float32 if dtype is None else dtype
        self.device = _cuda_device(device)
        self.heads, self.kv_heads, self.d = heads, kv_heads, d
        if not 0 <= eps < float("inf"):
            raise ValueError(f"eps {eps}: need a finite number that is not negative")
        if rotation is not None and (rotation.d != d or rotation.device != self.device):
            raise ValueError(f"rotation: made for {rotation.d} numbers on {rotation.device}, "
                             f"need {d} on {self.device}")
        self.rotation = rotation
        # Copies in f32 of this object's own: a weight that changes later needs a new one.
        self._weights = []
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                if tuple(w.shape) != (d,):
                    raise ValueError(f"{name}: shape {tuple(w.shape)} != ({d},)")
                w = w.detach().to(device=self.device, dtype=torch.float32, copy=True).contiguous()
            self._weights.append(w)
        self._private = [w for w in self._weights if w is not None]
        if self.device.type == "cuda" and self._private and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.device).synchronize()
        if rotation is not None:
            self._private.append(rotation.turns)
        self._int32 = torch.int32
        self.cfg = NysAttnConfig(heads, kv_heads, d, d, _dtype_code(self.dtype), 0.0)
        at = [None if w is None else w.data_ptr() for w in self._weights]
        rot = 0 if rotation is None else rotation.rot
        self._prep = NysQkPrepare(*at, eps, rotation.turns.data_ptr() if rot else None, rot,
                                  int(rot > 0 and rotation.interleaved), 0)
        nys_qk_rows(self.cfg, self._prep, 0, NysRows(), None, None, NysRows(), None)

    def _stream(self):
        stream = super()._stream()
        if stream not in self._streams:
            # The memory of tensors that nobody else knows goes back only after what this stream reads.
            for t in self._private:
                t.record_stream(self.torch.cuda.current_stream(self.device))
            self._streams |= {stream}
        return stream

    def _shifted(self, shift):
        """The arguments of the C calls for this shift."""
        if not -2 ** 31 <= shift < 2 ** 31:
            raise ValueError(f"shift {shift}: past 32 bits")
        p = self._prep
        return NysQkPrepare(p.q_weight, p.k_weight, p.eps, p.turns, p.rot, p.interleaved, shift)

    def _at(self, positions, n):
        if positions is None:
            if self._prep.rot:
                raise ValueError("positions: needed for a rotation")
            return None
        return _ints(positions, self._int32, (n,), "positions", self.device.index)

    def _out(self, out, n, heads, where):
        if out.shape[0] != n:
            raise ValueError(f"{where}: {out.shape[0]} rows, need {n}")
        return _rows(out, self.dtype, heads, self.d, where, self.device.index)

    def rows(self, q, k, positions, q_out=None, k_out=None, shift=0):
        """q [tokens][heads][d] and k [tokens][kv_heads][d] (either may be None), normalised
        and rotated by positions (int32 [tokens], plus shift), into q_out and k_out, or in
        place where those are not given.  Returns them."""
        if self._elsewhere():
            with self.torch.cuda.device(self.device.index):
                return self.rows(q, k, positions, q_out, k_out, shift)
        index, dtype = self.device.index, self.dtype
        qs = qo = ks = ko = None
        if q is not None:
            n = q.shape[0]
            qs = qo = _rows(q, dtype, self.heads, self.d, "q", index)
            if q_out is None:
                q_out = q
            else:
                qo = self._out(q_out, n, self.heads, "q_out")
        elif k is None or q_out is not None:
            raise ValueError("q and k: need one of them, and none for an output without it")
        if k is not None:
            if q is None:
                n = k.shape[0]
            elif k.shape[0] != n:
                raise ValueError(f"k: {k.shape[0]} rows, q has {n}")
            ks = ko = _rows(k, dtype, self.kv_heads, self.d, "k", index)
            if k_out is None:
                k_out = k
            else:
                ko = self._out(k_out, n, self.kv_heads, "k_out")
        elif k_out is not None:
            raise ValueError("k_out: there is no k")
        nys_qk_rows(self.cfg, self._shifted(shift) if shift else self._prep, n, qs, ks,
                    self._at(positions, n), qo, ko, self._stream())
        return q_out, k_out

    def append(self, q, k, v, positions, slots, cache, q_out=None, k_out=None, shift=0):
        """The same with the prepared keys and the values v [tokens][kv_heads][dv] going into
        slots int64 [tokens] of cache (a PagedKV or PagedKV4 of this type; no slot twice, a
        slot of -1 is skipped).  q may be None; its rows go to q_out, or stay in place.  Keys
        go to k_out as well, if given.  Returns q_out."""
        torch, index = self.torch, self.device.index
        if self._elsewhere():
            with torch.cuda.device(index):
                return self.append(q, k, v, positions, slots, cache, q_out, k_out, shift)
        dtype, kv_heads, d = self.dtype, self.kv_heads, self.d
        if cache.dtype != dtype or cache.kv_heads != kv_heads or cache.d != d:
            raise ValueError("the cache's geometry is not this object's")
        if cache.device.index != index:
            raise ValueError(f"the cache is on {cache.device}, this object on {self.device}")
        n, dv, cfg = k.shape[0], cache.dv, self.cfg
        if v.shape[0] != n or (q is not None and q.shape[0] != n):
            raise ValueError("q, k and v must have as many rows as each other")
        if dv != d:
            cfg = NysAttnConfig(self.heads, kv_heads, d, dv, cfg.dtype, 0.0)
        qs = qo = None
        if q is not None:
            qs = qo = _rows(q, dtype, self.heads, d, "q", index)
            if q_out is None:
                q_out = q
            else:
                qo = self._out(q_out, n, self.heads, "q_out")
        elif q_out is not None:
            raise ValueError("q_out: there is no q")
        (nys_kv4_append if isinstance(cache, PagedKV4) else nys_kv_append)(
            cfg, self._shifted(shift) if shift else self._prep, cache._pool, n, qs,
            _rows(k, dtype, kv_heads, d, "k", index), _rows(v, dtype, kv_heads, dv, "v", index),
            self._at(positions, n), _ints(slots, torch.int64, (n,), "slots", index), qo,
            None if k_out is None else self._out(k_out, n, kv_heads, "k_out"), self._stream())
        return q_out


class PagePlan(_Status):
    """Block tables, slots and positions of a batch's next tokens, built on
    the GPU from its lengths (nys_kv_plan): up to n requests, `width` pages a
    request, `total` new tokens, `page` tokens a page.  The outputs are
    tensors of this object: q_off int32 [n+1], lens int32 [n], slots int64
    [total], positions int32 [total], taken int32 [1]."""

    def __init__(self, n, width, total, page, device="cuda"):
        import torch
        self.torch = torch
        self.device = _cuda_device(device)
        self.n, self.width, self.total, self.page = n, width, total, page
        make = lambda size, dt: torch.empty(size, dtype=dt, device=self.device)
        self.q_off = make(n + 1, torch.int32)
        self.lens = make(n, torch.int32)
        self.slots = make(total, torch.int64)
        self.positions = make(total, torch.int32)
        self.taken = make(1, torch.int32)
        self._init_status(torch, self.device)
        self._out = [t.data_ptr() for t in (self.q_off, self.lens, self.slots, self.positions,
                                            self.taken)]

    def update(self, cached, fresh, free_pages, table):
        """cached, fresh int32 [n]; free_pages int32 [any]; table int32
        [n][width], whose new columns are filled in place.  cached may be this
        plan's lens, which then grows in place."""
        i32, index = self.torch.int32, self.device.index
        if self._elsewhere():
            with self.torch.cuda.device(index):
                return self.update(cached, fresh, free_pages, table)
        nys_kv_plan(self.n, self.page, _ints(cached, i32, (self.n,), "cached", index),
                    _ints(fresh, i32, (self.n,), "fresh", index),
                    _ints(free_pages, i32, free_pages.shape[:1], "free_pages", index),
                    free_pages.shape[0], _ints(table, i32, (self.n, self.width), "table", index),
                    self.width, self.total, *self._out, self._status_ptr, self._stream())
        return self


class ExactAttention(_Status):
    """Exact grouped-query attention of one layer's geometry: packed causal
    prompts (``prompt``) and one token over a shared prefix and paged own keys
    (``shared``).  The workspace grows on demand and is kept, so calls on one
    object must be ordered (one stream, or events).  One that a CUDA graph has
    captured is kept for the graph's replays, which count as calls, even when a
    larger one takes its place."""

    def __init__(self, heads, kv_heads, d, dv, dtype=None, scale=None, device="cuda"):
        import torch
        if scale is not None and not 0 < ctypes.c_float(scale).value < float("inf"):
            raise ValueError(f"scale {scale}: need a positive number of f32, or None for 1/sqrt(d)")
        self.torch = torch
        self.dtype = torch.float32 if dtype is None else dtype
        self.device = _cuda_device(device)
        self.heads, self.kv_heads, self.d, self.dv = heads, kv_heads, d, dv
        self.cfg = NysAttnConfig(heads, kv_heads, d, dv, _dtype_code(self.dtype),
                                 0.0 if scale is None else scale)
        self._init_status(torch, self.device)
        self._work = None
        self._work_ptr = None
        self._work_bytes = 0
        self._sizes = None
        self._captured = False   # a graph may hold the workspace's address
        self._held = []          # workspaces that were outgrown and that one holds
        nys_attn_workspace_bytes(self.cfg, 0, 0)   # refuses a bad geometry here

    def _workspace(self, n, rows, keys):
        """Makes the workspace large enough for a call of these sizes."""
        capturing = self.torch.cuda.is_current_stream_capturing()
        if (n, rows, keys) == self._sizes:
            self._captured |= capturing
            return
        if keys is None:      # paged4: n requests of up to `rows` tokens
            need = nys_attn4_workspace_bytes(self.cfg, n, rows)
        else:
            need = nys_attn_workspace_bytes(self.cfg, n, rows, keys)
        if need > self._work_bytes:
            # May raise: nothing is noted before it is there.
            work = self.torch.empty(need, dtype=self.torch.uint8, device=self.device)
            if self._captured:
                self._held.append(self._work)
            elif self._work is not None:
                # Work that uses it may be queued on a stream other than its own.
                self._work.record_stream(self.torch.cuda.current_stream(self.device))
            self._captured = False
            self._work = work
            self._work_ptr, self._work_bytes = work.data_ptr(), need
        self._sizes = (n, rows, keys)
        self._captured |= capturing

    def prompt(self, q, k, v, q_off, out, k_off=None, lse=None):
        """Packed causal attention (nys_attn_prompt): q [rows][heads][d], k and
        v [keys][kv_heads][d|dv], q_off and k_off int32 [n+1]; writes out
        [rows][heads][dv] and, if given, lse fp32 [rows][heads]."""
        torch, index = self.torch, self.device.index
        if self._elsewhere():
            with torch.cuda.device(index):
                return self.prompt(q, k, v, q_off, out, k_off, lse)
        n, rows, keys = q_off.shape[0] - 1, q.shape[0], k.shape[0]
        if v.shape[0] != keys or out.shape[0] != rows:
            raise ValueError("k and v, and q and out, must have as many rows as each other")
        self._workspace(n, rows, keys)
        nys_attn_prompt(
            self.cfg, n, rows, keys, _ints(q_off, torch.int32, (n + 1,), "q_off", index),
            None if k_off is None else _ints(k_off, torch.int32, (n + 1,), "k_off", index),
            _rows(q, self.dtype, self.heads, self.d, "q", index),
            _rows(k, self.dtype, self.kv_heads, self.d, "k", index),
            _rows(v, self.dtype, self.kv_heads, self.dv, "v", index),
            _rows(out, self.dtype, self.heads, self.dv, "out", index),
            None if lse is None else _ints(lse, torch.float32, (rows, self.heads), "lse", index),
            self._work_ptr, self._work_bytes, self._status_ptr, self._stream())
        return out

    def shared(self, q, cache, lens, table, out, prefix_pages=None, prefix_len=0, lse=None):
        """One token for each of n requests (nys_attn_shared): q [n][heads][d]
        over the prefix's keys and lens[b] own keys in cache's pages table[b]
        (lens int32 [n], table int32 [n][width]); writes out [n][heads][dv]."""
        torch, index = self.torch, self.device.index
        if self._elsewhere():
            with torch.cuda.device(index):
                return self.shared(q, cache, lens, table, out, prefix_pages, prefix_len, lse)
        n = q.shape[0]
        if isinstance(cache, PagedKV4):
            raise ValueError("cache: need a PagedKV (paged4 takes one in 4 bits)")
        if (cache.dtype != self.dtype or cache.kv_heads != self.kv_heads or cache.d != self.d
                or cache.dv != self.dv):
            raise ValueError("the cache's geometry is not this attention's")
        if cache.device.index != index:
            raise ValueError(f"the cache is on {cache.device}, this attention on {self.device}")
        if out.shape[0] != n or len(table.shape) != 2:
            raise ValueError("out must have q's rows, and table be [n][width]")
        pages = None
        if prefix_len > 0:
            if prefix_pages is None:
                raise ValueError("prefix_pages: needed for a prefix")
            pages = _ints(prefix_pages, torch.int32, prefix_pages.shape[:1], "prefix_pages", index)
            if prefix_pages.shape[0] * cache.page < prefix_len:
                raise ValueError("prefix_pages: too few pages for prefix_len")
        self._workspace(n, n, prefix_len)
        nys_attn_shared(
            self.cfg, n, cache._pool, pages, prefix_len,
            _ints(lens, torch.int32, (n,), "lens", index),
            _ints(table, torch.int32, (n, table.shape[1]), "table", index), table.shape[1],
            _rows(q, self.dtype, self.heads, self.d, "q", index),
            _rows(out, self.dtype, self.heads, self.dv, "out", index),
            None if lse is None else _ints(lse, torch.float32, (n, self.heads), "lse", index),
            self._work_ptr, self._work_bytes, self._status_ptr, self._stream())
        return out

    def paged4(self, q, cache, lens, table, out, first=None, first_lse=None, lse=None):
        """One token for each of n requests over a 4-bit cache (nys_attn4): q [n][heads][d]
        over lens[b] keys in the pages table[b] of cache, a PagedKV4 (lens int32 [n], table
        int32 [n][width]); writes out [n][heads][dv] and, if given, lse fp32 [n][heads].
        first [n][heads][dv] and first_lse: the same queries' result over other keys, joined
        in (shared() over a prefix); they may be out and lse themselves."""
        torch, index = self.torch, self.device.index
        if self._elsewhere():
            with torch.cuda.device(index):
                return self.paged4(q, cache, lens, table, out, first, first_lse, lse)
        n = q.shape[0]
        if not isinstance(cache, PagedKV4):
            raise ValueError("cache: need a PagedKV4")
        if (cache.dtype != self.dtype or cache.kv_heads != self.kv_heads or cache.d != self.d
                or cache.dv != self.dv):
            raise ValueError("the cache's geometry is not this attention's")
        if cache.device.index != index:
            raise ValueError(f"the cache is on {cache.device}, this attention on {self.device}")
        if out.shape[0] != n or len(table.shape) != 2:
            raise ValueError("out must have q's rows, and table be [n][width]")
        if (first is None) != (first_lse is None) or (first is not None and first.shape[0] != n):
            raise ValueError("first and first_lse go together, and have q's rows")
        width = table.shape[1]
        self._workspace(n, width * cache.page, None)
        nys_attn4(
            self.cfg, n, cache._pool, _ints(lens, torch.int32, (n,), "lens", index),
            _ints(table, torch.int32, (n, width), "table", index), width,
            _rows(q, self.dtype, self.heads, self.d, "q", index),
            _rows(out, self.dtype, self.heads, self.dv, "out", index),
            None if first is None else _rows(first, self.dtype, self.heads, self.dv, "first",
                                             index),
            None if first is None else _ints(first_lse, torch.float32, (n, self.heads),
                                             "first_lse", index),
            None if lse is None else _ints(lse, torch.float32, (n, self.heads), "lse", index),
            self._work_ptr, self._work_bytes, self._status_ptr, self._stream())
        return out
