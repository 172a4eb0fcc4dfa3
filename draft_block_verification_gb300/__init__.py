"""draft_block_verification_gb300: draft-block verification on GB300 (sm_103a).

A thin ctypes binding over the C ABI of ``libsv.so`` (declared in
``include/sv.h``).  Each function has the C name, takes torch CUDA tensors,
marshals pointers, sizes and the current CUDA stream, and raises ``SVError``
on any status other than SV_OK.  With ``stream=`` a call runs on that stream, and
what it allocates comes from that stream's memory.  Every step of the computation
runs in the library's kernels; there is no other code path.  The library must have been
built (``draft_block_verification_gb300._build.build()``); importing the
functions when it is missing raises immediately.
"""
from __future__ import annotations

import atexit
import ctypes as C
import os
import sys
import threading

import torch

from ._build import LIBPATH, build  # noqa: F401  (build is part of the API)

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_CUDA, SV_ERR_OOM = 0, 1, 2, 3
SV_ERR_TIMEOUT, SV_ERR_UNSUPPORTED, SV_ERR_DEVICE_BOUNDS = 4, 5, 6
SV_F32, SV_BF16 = 0, 1
SV_LOSSLESS, SV_LENIENT_RATIO, SV_LENIENT_LINEAR, SV_LENIENT_CACTUS = 0, 1, 2, 3
SV_OPT_FORCE_RESCUE, SV_OPT_TIMING_EVENTS = 1, 2

_lib = None
_lock = threading.Lock()
_handles = {}


class SVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, status_string(status), status))


def lib():
    """The loaded libsv.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBPATH):
            raise RuntimeError("libsv.so is not built: run draft_block_verification_gb300."
                               "_build.build() (nvcc with sm_103a support)")
        L = C.CDLL(LIBPATH)
        vp, i32, i64, u64, f32 = C.c_void_p, C.c_int, C.c_int64, C.c_uint64, C.c_float
        L.sv_status_string.restype, L.sv_status_string.argtypes = C.c_char_p, [i32]
        L.sv_create.restype, L.sv_create.argtypes = i32, [C.POINTER(vp)]
        L.sv_destroy.restype, L.sv_destroy.argtypes = i32, [vp]
        L.sv_sync_status.restype, L.sv_sync_status.argtypes = i32, [vp, vp]
        L.sv_rescue_count.restype = i32
        L.sv_rescue_count.argtypes = [vp, vp, C.POINTER(C.c_int64)]
        L.sv_set_option.restype, L.sv_set_option.argtypes = i32, [vp, i32, i64]
        L.sv_selftest.restype = i32
        L.sv_selftest.argtypes = [vp, u64, i64, C.POINTER(C.c_double), vp]
        L.sv_wait_selftest.restype, L.sv_wait_selftest.argtypes = i32, [vp, i64, vp]
        L.sv_verify_greedy.restype = i32
        L.sv_verify_greedy.argtypes = [vp, vp, i32, i64, i32, i32, i32, vp, vp, vp, vp, vp]
        L.sv_verify_greedy_static.restype = i32
        L.sv_verify_greedy_static.argtypes = [vp, i32, i64, i32, i32, i32, vp, vp, vp, vp, vp,
                                              vp]
        L.sv_verify_sample.restype = i32
        L.sv_verify_sample.argtypes = [vp, vp, vp, i32, i64, i32, i32, i32, vp, vp, f32, f32,
                                       i32, f32, u64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.sv_verify_tree.restype = i32
        L.sv_verify_tree.argtypes = [vp, vp, i32, i64, i32, i32, i32, vp, vp, vp, f32, u64, vp,
                                     vp, vp, i32, vp, vp, vp, vp]
        L.sv_verify_spot.restype = i32
        L.sv_verify_spot.argtypes = [vp, vp, i32, i64, i32, i32, i32, i32, vp, vp, vp, vp, f32,
                                     u64, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.sv_packed_anyorder_step.restype = i32
        L.sv_packed_anyorder_step.argtypes = [vp, vp, i32, i64, i32, i32, i32, i32, vp, vp, vp,
                                              vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.sv_packed_step.restype = i32
        L.sv_packed_step.argtypes = [vp, vp, i32, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp,
                                     f32, u64, u64, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                     vp]
        L.sv_packed_topk_step.restype = i32
        L.sv_packed_topk_step.argtypes = [vp, vp, i32, i64, i32, i32, i32, i32, i32, i32, vp, vp,
                                          vp, vp, vp, f32, u64, u64, vp, i32, vp, vp, vp, vp, vp,
                                          vp, vp, vp, vp, vp, vp]
        L.sv_kv_plan.restype = i32
        L.sv_kv_plan.argtypes = [vp] + [i32] * 5 + [vp] * 13
        L.sv_kv_append.restype = i32
        L.sv_kv_append.argtypes = ([vp] * 3 + [i32] + [i64] * 4 + [i32] * 5 + [vp] * 6)
        L.sv_kv_attention.restype = i32
        L.sv_kv_attention.argtypes = ([vp] * 2 + [i64] * 2 + [i32] * 4 + [vp] * 4 + [i32] * 2 +
                                      [vp, i32] + [vp] * 2 + [i32, vp, i32, f32] + [vp] * 3)
        L.sv_kv_prefix_work_bytes.restype = C.c_size_t
        L.sv_kv_prefix_work_bytes.argtypes = [vp] + [i32] * 6
        L.sv_kv_prefix_attention.restype = i32
        L.sv_kv_prefix_attention.argtypes = (
            [vp] * 2 + [i64] * 2 + [i32] * 4 + [vp] * 4 + [i32] * 2 + [vp, i32] + [vp] * 2 +
            [i32] + [vp] * 2 + [i32, vp, i32, f32] + [vp] * 3 + [C.c_size_t, vp])
        L.sv_kv_read.restype = i32
        L.sv_kv_read.argtypes = ([vp] * 5 + [i32] * 4 + [vp, i32] + [vp] * 2 + [i32] * 2 +
                                 [vp] * 2 + [i32] + [i64] * 4 + [vp])
        L.sv_qk_norm_rope.restype = i32
        L.sv_qk_norm_rope.argtypes = ([vp] * 3 + [i32] + [i64] * 4 + [i32] * 4 + [vp] * 2 +
                                      [f32, vp] + [i32] * 2 + [vp] * 3 + [i32] + [i64] * 4 + [vp])
        L.sv_sample_rows.restype = i32
        L.sv_sample_rows.argtypes = [vp, vp, i32, i64, i32, i32] + [vp] * 9
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().sv_status_string(int(s)).decode()


def _check(s: int, where: str):
    if s != SV_OK:
        raise SVError(s, where)


class Handle:
    """An sv_handle bound to one CUDA device."""

    def __init__(self, device=None):
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None
                                   else torch.device(device).index or 0)
        with torch.cuda.device(self.device):
            h = C.c_void_p()
            _check(lib().sv_create(C.byref(h)), "sv_create")
        self.ptr = h

    def close(self):
        if self.ptr:
            lib().sv_destroy(self.ptr)
            self.ptr = None

    def __del__(self):
        # At interpreter shutdown the CUDA runtime may already be gone; the
        # process exit releases the device memory then.
        if sys.is_finalizing():
            return
        try:
            self.close()
        except Exception:
            pass

    def sync_status(self, stream=None):
        """Synchronise and raise the first device-side error latched."""
        _check(lib().sv_sync_status(self.ptr, _stream(stream, self.device)), "device")

    def rescue_count(self, stream=None) -> int:
        c = C.c_int64()
        _check(lib().sv_rescue_count(self.ptr, _stream(stream, self.device), C.byref(c)),
               "sv_rescue_count")
        return int(c.value)

    def selftest(self, seed: int = 1, n: int = 1 << 22, stream=None):
        """Ratios of the measured fp32 errors to the bounds the kernels assume,
        the count of skip gaps whose fast evaluation is not exact, and the
        count of ids outside their Gumbel bound table entries."""
        r = (C.c_double * 5)()
        _check(lib().sv_selftest(self.ptr, int(seed), int(n), r, _stream(stream, self.device)),
               "sv_selftest")
        return list(r)

    def wait_selftest(self, limit: int = 1000, stream=None):
        """Enqueue the self-test whose bounded waits run out: the next
        sync_status raises SVError with SV_ERR_TIMEOUT."""
        _check(lib().sv_wait_selftest(self.ptr, int(limit), _stream(stream, self.device)),
               "sv_wait_selftest")

    def set_option(self, opt: int, value: int):
        _check(lib().sv_set_option(self.ptr, int(opt), int(value)), "sv_set_option")


@atexit.register
def _close_default_handles():
    with _lock:
        for h in _handles.values():
            try:
                h.close()
            except Exception:
                pass
        _handles.clear()


def default_handle(device=None) -> Handle:
    dev = torch.cuda.current_device() if device is None else torch.device(device).index or 0
    with _lock:
        if dev not in _handles:
            _handles[dev] = Handle(dev)
        return _handles[dev]


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _rows(t, name):
    """(dtype code, row stride in elements) of a [..., rows, V] logit tensor."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype == torch.bfloat16:
        code = SV_BF16
    elif t.dtype == torch.float32:
        code = SV_F32
    else:
        raise ValueError("%s must be bfloat16 or float32" % name)
    if t.stride(-1) != 1:
        raise ValueError("%s: the vocabulary dimension must be contiguous" % name)
    rs = t.stride(-2) if t.dim() >= 2 else t.shape[-1]
    for d in range(t.dim() - 2):
        if t.stride(d) != t.shape[d + 1] * t.stride(d + 1):
            raise ValueError("%s: rows must be evenly strided" % name)
    return code, rs


def _i32(t, shape, name, dev):
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_cuda or t.device != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor on %s" % (name, dev))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    return t


def _out(t, shape, dtype, dev):
    return torch.empty(shape, dtype=dtype, device=dev) if t is None else t


def _tensors(x):
    """The tensors of a call's arguments or results."""
    if isinstance(x, torch.Tensor):
        yield x
    elif isinstance(x, (tuple, list, dict)):
        for y in x.values() if isinstance(x, dict) else x:
            yield from _tensors(y)


def _on_stream(stream, call, given):
    """A call with stream=, `given` its arguments: runs with that stream as torch's
    current one.  What it allocates comes from that stream's memory, not from blocks that
    work queued on the current stream may still use.  Results may be used and freed on the
    current stream as before."""
    given = dict(given, stream=None)
    dev = next((t.device for t in _tensors(given) if t.is_cuda), None)
    if dev is None:
        return call(**given)                      # (refused)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device=dev)
    now = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        out = call(**given)
    if now.cuda_stream != stream.cuda_stream:
        for t in _tensors(out):
            t.record_stream(now)
    return out


def sv_verify_greedy(target, draft_ids, draft_len=None, *, handle=None, stream=None,
                     accept_len=None, next_token=None):
    """Greedy verification; target [B, K+1, V]; returns (accept_len, next_token)."""
    if stream is not None:
        return _on_stream(stream, sv_verify_greedy, locals())
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    code, rs = _rows(target, "target")
    h = handle or default_handle(dev)
    ids = _i32(draft_ids, (B, K), "draft_ids", dev)
    dl = _i32(draft_len, (B,), "draft_len", dev)
    acc = _out(accept_len, (B,), torch.int32, dev)
    nxt = _out(next_token, (B,), torch.int32, dev)
    _check(lib().sv_verify_greedy(h.ptr, _p(target), code, rs, B, K, V, _p(ids), _p(dl),
                                  _p(acc), _p(nxt), _stream(stream, dev)), "sv_verify_greedy")
    return acc, nxt


def sv_verify_greedy_static(target, draft_ids, draft_len=None, *, stream=None, accept_len=None,
                            next_token=None, status=None):
    """Greedy verification with the library's fixed scratch (no device
    allocation by the library; see sv.h).  Returns (accept_len, next_token,
    status); status[0] holds the first device-side error of the call, 0 if
    none.  Pass preallocated outputs to keep the call free of allocations on
    the Python side as well."""
    if stream is not None:
        return _on_stream(stream, sv_verify_greedy_static, locals())
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    code, rs = _rows(target, "target")
    ids = _i32(draft_ids, (B, K), "draft_ids", dev)
    dl = _i32(draft_len, (B,), "draft_len", dev)
    acc = _out(accept_len, (B,), torch.int32, dev)
    nxt = _out(next_token, (B,), torch.int32, dev)
    st = _out(status, (1,), torch.int32, dev)
    _check(lib().sv_verify_greedy_static(_p(target), code, rs, B, K, V, _p(ids), _p(dl), _p(acc),
                                         _p(nxt), _p(st), _stream(stream, dev)),
           "sv_verify_greedy_static")
    return acc, nxt, st


def sv_verify_sample(target, draft, draft_ids, draft_len=None, *, T_p=1.0, T_q=1.0,
                     mode=SV_LOSSLESS, lam=1.0, seed=0, pos_base=None, want_rows=True,
                     want_tv=False, handle=None, stream=None):
    """Lossless / lenient speculative sampling; target [B, K+1, V], draft [B, K, V].
    Returns a dict of output tensors (see sv.h)."""
    if stream is not None:
        return _on_stream(stream, sv_verify_sample, locals())
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    code, rs = _rows(target, "target")
    if K > 0:
        code2, rs2 = _rows(draft, "draft")
        if code2 != code or rs2 != rs or tuple(draft.shape) != (B, K, V):
            raise ValueError("draft must be [B, K, V] with the target's dtype and row stride")
    h = handle or default_handle(dev)
    ids = _i32(draft_ids, (B, K), "draft_ids", dev)
    dl = _i32(draft_len, (B,), "draft_len", dev)
    if pos_base is not None and (pos_base.dtype != torch.int64 or not pos_base.is_cuda):
        raise ValueError("pos_base must be an int64 CUDA tensor")
    f = lambda *s: torch.empty(s, dtype=torch.float32, device=dev)
    out = {"accept_len": torch.empty(B, dtype=torch.int32, device=dev),
           "next_token": torch.empty(B, dtype=torch.int32, device=dev),
           "flags": torch.empty(B, dtype=torch.int32, device=dev)}
    if want_rows:
        out.update(p_at_draft=f(B, K), q_at_draft=f(B, K), lse_p=f(B, K + 1), lse_q=f(B, K))
    if want_tv:
        out["tv"] = f(B, K)
    g = out.get
    _check(lib().sv_verify_sample(
        h.ptr, _p(target), _p(draft) if K > 0 else None, code, rs, B, K, V, _p(ids), _p(dl),
        float(T_p), float(T_q), int(mode), float(lam), int(seed) & (2**64 - 1), _p(pos_base),
        _p(out["accept_len"]), _p(out["next_token"]), _p(g("p_at_draft")), _p(g("q_at_draft")),
        _p(g("lse_p")), _p(g("lse_q")), _p(g("tv")), _p(out["flags"]), _stream(stream, dev)),
        "sv_verify_sample")
    return out


def sv_verify_tree(node_logits, parent, node_pos, node_tok, *, T=0.0, seed=0, pos_base=None,
                   max_depth=None, handle=None, stream=None):
    """Coupled-noise tree verification; node_logits [B, N, V]."""
    if stream is not None:
        return _on_stream(stream, sv_verify_tree, locals())
    B, N, V = node_logits.shape
    dev = node_logits.device
    code, rs = _rows(node_logits, "node_logits")
    h = handle or default_handle(dev)
    par = _i32(parent, (B, N), "parent", dev)
    pos = _i32(node_pos, (B, N), "node_pos", dev)
    tok = _i32(node_tok, (B, N), "node_tok", dev)
    md = N if max_depth is None else int(max_depth)
    out = {"path_len": torch.empty(B, dtype=torch.int32, device=dev),
           "path_nodes": torch.empty((B, md), dtype=torch.int32, device=dev),
           "commit_count": torch.empty(B, dtype=torch.int32, device=dev),
           "match": torch.empty((B, N), dtype=torch.uint8, device=dev),
           "flags": torch.empty(B, dtype=torch.int32, device=dev)}
    _check(lib().sv_verify_tree(
        h.ptr, _p(node_logits), code, rs, B, N, V, _p(par), _p(pos), _p(tok), float(T),
        int(seed) & (2**64 - 1), _p(pos_base), _p(out["path_len"]), _p(out["path_nodes"]), md,
        _p(out["commit_count"]), _p(out["match"]), _p(out["flags"]), _stream(stream, dev)),
        "sv_verify_tree")
    return out


def sv_verify_spot(state_logits, parent, node_pos, node_tok, root_mask, *, T=0.0, seed=0,
                   pos_base=None, max_depth=None, handle=None, stream=None):
    """SPOT verification with the target's position selection (see sv.h):
    state_logits [B, 1+N, L, V]; parent/node_pos/node_tok [B, N] int32;
    root_mask [B] int64 (bit s: position s is masked in the root state)."""
    if stream is not None:
        return _on_stream(stream, sv_verify_spot, locals())
    B, S, L, V = state_logits.shape
    N = S - 1
    dev = state_logits.device
    code, rs = _rows(state_logits, "state_logits")
    h = handle or default_handle(dev)
    par = _i32(parent, (B, N), "parent", dev) if N > 0 else None
    pos = _i32(node_pos, (B, N), "node_pos", dev) if N > 0 else None
    tok = _i32(node_tok, (B, N), "node_tok", dev) if N > 0 else None
    if (root_mask.dtype != torch.int64 or not root_mask.is_cuda or root_mask.device != dev
            or not root_mask.is_contiguous() or tuple(root_mask.shape) != (B,)):
        raise ValueError("root_mask must be a contiguous int64 CUDA tensor of shape [B]")
    if pos_base is not None and (pos_base.dtype != torch.int64 or not pos_base.is_cuda):
        raise ValueError("pos_base must be an int64 CUDA tensor")
    md = max(N, 1) if max_depth is None else int(max_depth)
    i = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)
    out = {"path_len": i(B), "path_nodes": i(B, md), "commit_count": i(B), "commit_pos": i(B),
           "commit_tok": i(B), "match": torch.empty((B, N), dtype=torch.uint8, device=dev),
           "state_pos": i(B, S), "state_tok": i(B, S), "flags": i(B)}
    _check(lib().sv_verify_spot(
        h.ptr, _p(state_logits), code, rs, B, N, L, V, _p(par), _p(pos), _p(tok),
        _p(root_mask), float(T), int(seed) & (2**64 - 1), _p(pos_base), _p(out["path_len"]),
        _p(out["path_nodes"]), md, _p(out["commit_count"]), _p(out["commit_pos"]),
        _p(out["commit_tok"]), _p(out["match"]) if N > 0 else None, _p(out["state_pos"]),
        _p(out["state_tok"]), _p(out["flags"]), _stream(stream, dev)), "sv_verify_spot")
    return out


def sv_packed_anyorder_step(logits, Kv, W, u, win_pos, order, draft, end_pos, *, eos_id=-1,
                            handle=None, stream=None):
    """One any-order Packed-SS iteration (see sv.h); logits [B, Kv + W, V];
    u, end_pos [B]; win_pos, order, draft [B, W] (int32 CUDA tensors)."""
    if stream is not None:
        return _on_stream(stream, sv_packed_anyorder_step, locals())
    B, R, V = logits.shape
    if R != Kv + W:
        raise ValueError("logits must be [B, Kv + W, V]")
    dev = logits.device
    code, rs = _rows(logits, "logits")
    h = handle or default_handle(dev)
    uu, end = _i32(u, (B,), "u", dev), _i32(end_pos, (B,), "end_pos", dev)
    wp, od, dr = (_i32(a, (B, W), n, dev) for a, n in ((win_pos, "win_pos"), (order, "order"),
                                                        (draft, "draft")))
    i = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)
    out = {"accept_len": i(B), "commit_len": i(B), "commit_pos": i(B, W), "commit_tok": i(B, W),
           "end_pos": i(B), "next_draft": i(B, W),
           "score": torch.empty((B, W), dtype=torch.float32, device=dev)}
    _check(lib().sv_packed_anyorder_step(
        h.ptr, _p(logits), code, rs, B, Kv, W, V, _p(uu), _p(wp), _p(od), _p(dr), _p(end),
        int(eos_id), _p(out["accept_len"]), _p(out["commit_len"]), _p(out["commit_pos"]),
        _p(out["commit_tok"]), _p(out["end_pos"]), _p(out["next_draft"]), _p(out["score"]),
        _stream(stream, dev)), "sv_packed_anyorder_step")
    return out


def sv_packed_step(logits, K, W, prev_draft, prev_len, *, prev_q_at_draft=None,
                   prev_draft_logits=None, prev_q_offset=None, T=0.0, seed=0, it=0,
                   pos_base=None, eos_id=-1, remaining=None, handle=None, stream=None):
    """One Packed-SS iteration; logits [B, K+W, V]."""
    if stream is not None:
        return _on_stream(stream, sv_packed_step, locals())
    B, R, V = logits.shape
    if R != K + W:
        raise ValueError("logits must be [B, K+W, V]")
    dev = logits.device
    code, rs = _rows(logits, "logits")
    if T > 0:
        code2, rs2 = _rows(prev_draft_logits, "prev_draft_logits")
        if code2 != code or rs2 != rs:
            raise ValueError("prev_draft_logits must match the logits' dtype and row stride")
    h = handle or default_handle(dev)
    pd = _i32(prev_draft, (B, K - 1), "prev_draft", dev) if K > 1 else None
    pl = _i32(prev_len, (B,), "prev_len", dev)
    off = _i32(prev_q_offset, (B,), "prev_q_offset", dev)
    rem = _i32(remaining, (B,), "remaining", dev)
    pq = prev_q_at_draft
    if pq is not None and (pq.dtype != torch.float32 or not pq.is_contiguous()):
        raise ValueError("prev_q_at_draft must be a contiguous float32 tensor")
    out = {"accept_len": torch.empty(B, dtype=torch.int32, device=dev),
           "commit_len": torch.empty(B, dtype=torch.int32, device=dev),
           "committed": torch.empty((B, K), dtype=torch.int32, device=dev),
           "next_draft": torch.empty((B, W), dtype=torch.int32, device=dev),
           "next_len": torch.empty(B, dtype=torch.int32, device=dev),
           "next_q_at_draft": torch.empty((B, W), dtype=torch.float32, device=dev),
           "confidence": torch.empty((B, W), dtype=torch.float32, device=dev),
           "flags": torch.empty(B, dtype=torch.int32, device=dev)}
    _check(lib().sv_packed_step(
        h.ptr, _p(logits), code, rs, B, K, W, V, _p(pd), _p(pl), _p(pq),
        _p(prev_draft_logits) if T > 0 else None, _p(off), float(T), int(seed) & (2**64 - 1),
        int(it) & (2**64 - 1), _p(pos_base), int(eos_id), _p(rem), _p(out["accept_len"]),
        _p(out["commit_len"]), _p(out["committed"]), _p(out["next_draft"]),
        _p(out["next_len"]), _p(out["next_q_at_draft"]), _p(out["confidence"]),
        _p(out["flags"]), _stream(stream, dev)), "sv_packed_step")
    return out


def sv_packed_topk_step(logits, K, W, kp, kq, prev_draft, prev_len, prev_q_ids, prev_q_probs,
                        prev_q_offset, *, T=1.0, seed=0, it=0, pos_base=None, eos_id=-1,
                        remaining=None, handle=None, stream=None):
    """One Packed-SS iteration with top-k truncated target (kp) and drafter
    (kq) distributions; logits [B, K+W, V]; the previous call's drafter lists
    prev_q_ids / prev_q_probs [B, W, kq] (int32 / float32)."""
    if stream is not None:
        return _on_stream(stream, sv_packed_topk_step, locals())
    B, R, V = logits.shape
    if R != K + W:
        raise ValueError("logits must be [B, K+W, V]")
    dev = logits.device
    code, rs = _rows(logits, "logits")
    h = handle or default_handle(dev)
    pd = _i32(prev_draft, (B, K - 1), "prev_draft", dev) if K > 1 else None
    pl = _i32(prev_len, (B,), "prev_len", dev)
    qi = _i32(prev_q_ids, (B, W, kq), "prev_q_ids", dev)
    off = _i32(prev_q_offset, (B,), "prev_q_offset", dev)
    rem = _i32(remaining, (B,), "remaining", dev)
    qp = prev_q_probs
    if (qp is None or qp.dtype != torch.float32 or not qp.is_contiguous() or
            tuple(qp.shape) != (B, W, kq) or qp.device != dev):
        raise ValueError("prev_q_probs must be a contiguous float32 [B, W, kq] tensor on the "
                         "logits' device")
    out = {"accept_len": torch.empty(B, dtype=torch.int32, device=dev),
           "commit_len": torch.empty(B, dtype=torch.int32, device=dev),
           "committed": torch.empty((B, K), dtype=torch.int32, device=dev),
           "next_draft": torch.empty((B, W), dtype=torch.int32, device=dev),
           "next_len": torch.empty(B, dtype=torch.int32, device=dev),
           "next_q_at_draft": torch.empty((B, W), dtype=torch.float32, device=dev),
           "q_ids": torch.empty((B, W, kq), dtype=torch.int32, device=dev),
           "q_probs": torch.empty((B, W, kq), dtype=torch.float32, device=dev),
           "flags": torch.empty(B, dtype=torch.int32, device=dev)}
    _check(lib().sv_packed_topk_step(
        h.ptr, _p(logits), code, rs, B, K, W, V, int(kp), int(kq), _p(pd), _p(pl), _p(qi),
        _p(qp), _p(off), float(T), int(seed) & (2**64 - 1), int(it) & (2**64 - 1),
        _p(pos_base), int(eos_id), _p(rem), _p(out["accept_len"]), _p(out["commit_len"]),
        _p(out["committed"]), _p(out["next_draft"]), _p(out["next_len"]),
        _p(out["next_q_at_draft"]), _p(out["q_ids"]), _p(out["q_probs"]), _p(out["flags"]),
        _stream(stream, dev)), "sv_packed_topk_step")
    return out



def _dense(t, dtype, shape, name, dev):
    """Address of a contiguous tensor of this type and shape."""
    if t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor on %s" % (name, dtype, dev))
    if t.shape != shape:
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    return t.data_ptr()


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.device


def _call_on(handle, stream, dev):
    """(handle pointer, raw stream): the given ones, or the device's default
    handle and torch's current stream."""
    if handle is None:
        handle = _handles.get(dev.index) or default_handle(dev)
    if stream is None:
        return handle.ptr, torch._C._cuda_getCurrentRawStream(dev.index)
    return handle.ptr, stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def sv_kv_plan(cached_len, new_len, held, table, free_ids, free_pos, block, max_tokens, *,
               handle=None, stream=None):
    """Places of new tokens in the paged cache (see sv.h): cached_len, new_len,
    held [B] and table [B, cols], free_ids [ring] int32; free_pos [2] int64.
    Updates table and free_ids in place and returns a dict of new tensors
    (kv_len, cu_new, held, free_pos, slot, pos)."""
    if stream is not None:
        return _on_stream(stream, sv_kv_plan, locals())
    dev = _cuda(cached_len, "cached_len")
    i32, empty = torch.int32, torch.empty
    B, cap = cached_len.shape[0], int(max_tokens)
    if table.dim() != 2 or free_ids.dim() != 1:
        raise ValueError("table must be [B, cols] and free_ids [ring]")
    cols, ring = table.shape[1], free_ids.shape[0]
    row = (B,)
    ptr, raw = _call_on(handle, stream, dev)
    kv_len, held_out = torch.empty_like(cached_len), torch.empty_like(held)
    free_out = torch.empty_like(free_pos)
    cu_new = empty(B + 1, dtype=i32, device=dev)
    slot = empty(cap, dtype=i32, device=dev)
    pos = torch.empty_like(slot)
    _check(lib().sv_kv_plan(
        ptr, B, int(block), cols, ring, cap, _dense(cached_len, i32, row, "cached_len", dev),
        _dense(new_len, i32, row, "new_len", dev), _dense(held, i32, row, "held", dev),
        _dense(free_pos, torch.int64, (2,), "free_pos", dev),
        _dense(free_ids, i32, (ring,), "free_ids", dev),
        _dense(table, i32, (B, cols), "table", dev), kv_len.data_ptr(), cu_new.data_ptr(),
        held_out.data_ptr(), free_out.data_ptr(), slot.data_ptr(), pos.data_ptr(), raw),
        "sv_kv_plan")
    return {"kv_len": kv_len, "cu_new": cu_new, "held": held_out, "free_pos": free_out,
            "slot": slot, "pos": pos}


def _kv_cache(k_cache, v_cache, k_scale, v_scale, dev):
    """Shape (pages, Hkv, block, D) and addresses of a paged cache."""
    if k_cache.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise ValueError("k_cache must be float8_e4m3fn or uint8")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, Hkv, block, D]")
    shape = k_cache.shape
    return shape, (_dense(k_cache, k_cache.dtype, shape, "k_cache", dev),
                   _dense(v_cache, k_cache.dtype, shape, "v_cache", dev),
                   _dense(k_scale, torch.float32, shape[:2], "k_scale", dev),
                   _dense(v_scale, torch.float32, shape[:2], "v_scale", dev))


def sv_kv_append(k, v, slot, k_cache, v_cache, k_scale, v_scale, *, handle=None, stream=None):
    """Write k, v [T, Hkv, D] (float32 or bfloat16) to the cache's slots
    slot [T] int32 in place (see sv.h); caches [pages, Hkv, block, D]
    float8_e4m3fn, scales [pages, Hkv] float32."""
    if stream is not None:
        return _on_stream(stream, sv_kv_append, locals())
    dev = _cuda(k, "k")
    (pages, H, block, D), cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    T = k.shape[0]
    if k.shape != (T, H, D) or v.shape != k.shape:
        raise ValueError("k and v must be [T, Hkv, D] with the cache's Hkv and D")
    if k.dtype != v.dtype or v.device != dev or k.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("k and v must both be bfloat16 or float32, on one device")
    if k.stride(2) != 1 or v.stride(2) != 1:
        raise ValueError("k and v: the last dimension must be contiguous")
    ptr, raw = _call_on(handle, stream, dev)
    _check(lib().sv_kv_append(
        ptr, k.data_ptr(), v.data_ptr(), SV_BF16 if k.dtype == torch.bfloat16 else SV_F32,
        k.stride(0), k.stride(1), v.stride(0), v.stride(1), T, H, D, block, pages,
        _dense(slot, torch.int32, (T,), "slot", dev), *cache, raw),
        "sv_kv_append")


def sv_kv_attention(q, k_cache, v_cache, k_scale, v_scale, table, kv_len, cu_new, *, scale=None,
                    mask=None, want_lse=False, handle=None, stream=None):
    """Attention of the new tokens' queries q [T, Hq, D] (bfloat16) over the
    paged cache (see sv.h); table [B, cols], kv_len [B], cu_new [B + 1] int32;
    mask [T, words] int32 bits over the sequence's new tokens, or None for
    causal.  scale defaults to D ** -0.5.  Returns a dict (out, and lse)."""
    if stream is not None:
        return _on_stream(stream, sv_kv_attention, locals())
    dev = _cuda(q, "q")
    (pages, H, block, D), cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    if q.dim() != 3 or q.shape[2] != D or q.dtype != torch.bfloat16 or q.stride(2) != 1:
        raise ValueError("q must be a bfloat16 [T, Hq, D] tensor with the cache's D, contiguous "
                         "in its last dimension")
    if table.dim() != 2:
        raise ValueError("table must be [B, cols]")
    T, Hq, _ = q.shape
    B, cols = kv_len.shape[0], table.shape[1]
    i32 = torch.int32
    words = 0
    if mask is not None:
        if mask.dim() != 2:
            raise ValueError("mask must be [T, words]")
        words = mask.shape[1]
    ptr, raw = _call_on(handle, stream, dev)
    out = {"out": torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)}
    if want_lse:
        out["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    _check(lib().sv_kv_attention(
        ptr, q.data_ptr(), q.stride(0), q.stride(1), T, Hq, H, D, *cache, block, pages,
        _dense(table, i32, (B, cols), "table", dev), cols,
        _dense(kv_len, i32, (B,), "kv_len", dev), _dense(cu_new, i32, (B + 1,), "cu_new", dev), B,
        None if mask is None else _dense(mask, i32, (T, words), "mask", dev), words,
        float(D ** -0.5 if scale is None else scale), out["out"].data_ptr(),
        out["lse"].data_ptr() if want_lse else None, raw),
        "sv_kv_attention")
    return out


def sv_kv_prefix_attention(q, k_cache, v_cache, k_scale, v_scale, table, kv_len, cu_new,
                           prefix_len=None, *, cu_group=None, scale=None, mask=None,
                           want_lse=False, handle=None, stream=None):
    """sv_kv_attention for sequences that share a prefix, whose pages are read
    once for all (see sv.h): sequences cu_group[g] .. cu_group[g + 1] - 1
    ([groups + 1] int32; None: all) share at most their first prefix_len[g]
    tokens ([groups] int32; None: as far as their tables agree).  Returns a
    dict (out, and lse)."""
    if stream is not None:
        return _on_stream(stream, sv_kv_prefix_attention, locals())
    dev = _cuda(q, "q")
    (pages, H, block, D), cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    if q.dim() != 3 or q.shape[2] != D or q.dtype != torch.bfloat16 or q.stride(2) != 1:
        raise ValueError("q must be a bfloat16 [T, Hq, D] tensor with the cache's D, contiguous "
                         "in its last dimension")
    if table.dim() != 2:
        raise ValueError("table must be [B, cols]")
    T, Hq, _ = q.shape
    B, cols = kv_len.shape[0], table.shape[1]
    i32 = torch.int32
    if cu_group is not None and (cu_group.dim() != 1 or cu_group.shape[0] < 2):
        raise ValueError("cu_group must be [groups + 1]")
    groups = 1 if cu_group is None else cu_group.shape[0] - 1
    words = 0
    if mask is not None:
        if mask.dim() != 2:
            raise ValueError("mask must be [T, words]")
        words = mask.shape[1]
    ptr, raw = _call_on(handle, stream, dev)
    L = lib()
    size = L.sv_kv_prefix_work_bytes(ptr, T, Hq, H, D, B, groups)
    out = {"out": torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)}
    if want_lse:
        out["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    work = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(L.sv_kv_prefix_attention(
        ptr, q.data_ptr(), q.stride(0), q.stride(1), T, Hq, H, D, *cache, block, pages,
        _dense(table, i32, (B, cols), "table", dev), cols,
        _dense(kv_len, i32, (B,), "kv_len", dev), _dense(cu_new, i32, (B + 1,), "cu_new", dev), B,
        None if prefix_len is None else _dense(prefix_len, i32, (groups,), "prefix_len", dev),
        None if cu_group is None else _dense(cu_group, i32, (groups + 1,), "cu_group", dev),
        groups, None if mask is None else _dense(mask, i32, (T, words), "mask", dev), words,
        float(D ** -0.5 if scale is None else scale), out["out"].data_ptr(),
        out["lse"].data_ptr() if want_lse else None, work.data_ptr(), size, raw),
        "sv_kv_prefix_attention")
    return out


_CODE = {torch.bfloat16: SV_BF16, torch.float32: SV_F32}


def _rows_out(t, shape, dtype, dev, name):
    """Checks a given output: this shape, its last dimension contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.device != dev or t.stride(2) != 1:
        raise ValueError("%s must be a %s tensor of shape %s on %s, contiguous in its last "
                         "dimension" % (name, dtype, tuple(shape), dev))
    return t


def sv_kv_read(k_cache, v_cache, k_scale, v_scale, table, cu, rows, *, first=None,
               dtype=torch.bfloat16, out=None, handle=None, stream=None):
    """Tokens read back from the paged cache (see sv.h): rows cu[b] .. cu[b + 1]
    - 1 ([B + 1] int32) are positions first[b] on of sequence b (None: 0), in
    bfloat16 or float32.  rows: the outputs' rows; out: (k, v) [rows, Hkv, D] to
    write to.  Returns a dict (k, v); rows from cu[B] on are not written."""
    if stream is not None:
        return _on_stream(stream, sv_kv_read, locals())
    dev = _cuda(k_cache, "k_cache")
    (pages, H, block, D), cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    if table.dim() != 2:
        raise ValueError("table must be [B, cols]")
    if dtype not in _CODE:
        raise ValueError("dtype must be bfloat16 or float32")
    B, cols = table.shape
    T, i32 = int(rows), torch.int32
    if T < 0:
        raise ValueError("rows must not be negative")
    shape = (T, H, D)
    if out is None:
        k = torch.empty(shape, dtype=dtype, device=dev)
        v = torch.empty_like(k)
        strides = (H * D, D, H * D, D)
    else:
        k, v = (_rows_out(t, shape, dtype, dev, n) for t, n in zip(out, "kv"))
        strides = (*k.stride()[:2], *v.stride()[:2])
    ptr, raw = _call_on(handle, stream, dev)
    _check(lib().sv_kv_read(
        ptr, *cache, H, D, block, pages, _dense(table, i32, (B, cols), "table", dev), cols,
        None if first is None else _dense(first, i32, (B,), "first", dev),
        _dense(cu, i32, (B + 1,), "cu", dev), B, T, k.data_ptr(), v.data_ptr(), _CODE[dtype],
        *strides, raw), "sv_kv_read")
    return {"k": k, "v": v}


def sv_qk_norm_rope(q, k, pos, inv_freq, *, q_weight=None, k_weight=None, eps=1e-6,
                    interleaved=False, dtype=None, out=None, handle=None, stream=None):
    """Norms of queries and keys for each head, and the rotation by position, in
    one pass (see sv.h): q [T, Hq, D] and k [T, Hkv, D] (bfloat16 or float32, one
    of them may be None), pos [T] int32 (negative: the row is skipped), inv_freq
    [rot / 2] float32 (None: no rotation), weights [D] float32 (None: no norm).
    dtype: of the outputs (None: the inputs'); out: (q, k) to write to, which may
    be the inputs.  Returns a dict (q, k)."""
    if stream is not None:
        return _on_stream(stream, sv_qk_norm_rope, locals())
    x = k if q is None else q
    dev = _cuda(x, "k" if q is None else "q")
    given = x.dtype
    if x.dim() != 3 or given not in _CODE:
        raise ValueError("q and k must be bfloat16 or float32 tensors [T, heads, D]")
    T, Hq, D = x.shape
    H, qi, qo, ki, ko = 0, (0, 0, 1), (0, 0), (0, 0, 1), (0, 0)
    if dtype is None:
        dtype = given
    elif dtype not in _CODE:
        raise ValueError("dtype must be bfloat16 or float32")
    y = z = None
    if q is None:
        Hq = 0
    else:
        qi = q.stride()
        if out is None or out[0] is None:
            y, qo = torch.empty((T, Hq, D), dtype=dtype, device=dev), (Hq * D, D)
        else:
            y = _rows_out(out[0], q.shape, dtype, dev, "q of out")
            qo = y.stride()
    if k is not None:
        ki = k.stride()
        if k is not x and (k.dim() != 3 or k.shape[0] != T or k.shape[2] != D or
                           k.dtype is not given or k.device != dev):
            raise ValueError("q and k must have one T, D, type and device")
        H = k.shape[1]
        if out is None or out[1] is None:
            z, ko = torch.empty((T, H, D), dtype=dtype, device=dev), (H * D, D)
        else:
            z = _rows_out(out[1], k.shape, dtype, dev, "k of out")
            ko = z.stride()
    if qi[2] != 1 or ki[2] != 1:
        raise ValueError("q and k: the last dimension must be contiguous")
    f32, rot, row = torch.float32, 0, (D,)
    if inv_freq is not None:
        rot = inv_freq.shape[0]
        inv_freq, rot = _dense(inv_freq, f32, (rot,), "inv_freq", dev), 2 * rot
    ptr, raw = _call_on(handle, stream, dev)
    _check(lib().sv_qk_norm_rope(
        ptr, None if q is None else q.data_ptr(), None if k is None else k.data_ptr(),
        _CODE[given], qi[0], qi[1], ki[0], ki[1], T, Hq, H, D,
        None if q_weight is None else _dense(q_weight, f32, row, "q_weight", dev),
        None if k_weight is None else _dense(k_weight, f32, row, "k_weight", dev), eps,
        inv_freq, rot, 1 if interleaved else 0, _dense(pos, torch.int32, (T,), "pos", dev),
        None if y is None else y.data_ptr(), None if z is None else z.data_ptr(), _CODE[dtype],
        qo[0], qo[1], ko[0], ko[1], raw), "sv_qk_norm_rope")
    return {"q": y, "k": z}


def sv_sample_rows(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None,
                   handle=None, stream=None):
    """One draw from each row of logits [R, V] with the filters of sv.h; u,
    temperature, top_p, min_p [R] float32 and top_k [R] int32 (None: off; for
    the temperature 1).  Returns a dict (token, prob, kept)."""
    if stream is not None:
        return _on_stream(stream, sv_sample_rows, locals())
    dev = _cuda(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [R, V]")
    code, rs = _rows(logits, "logits")
    R, V = logits.shape
    f32, row = torch.float32, (R,)
    opt = lambda t, dt, n: None if t is None else _dense(t, dt, row, n, dev)
    ptr, raw = _call_on(handle, stream, dev)
    token, prob = torch.empty(R, dtype=torch.int32, device=dev), torch.empty_like(u)
    kept = torch.empty_like(token)
    _check(lib().sv_sample_rows(
        ptr, logits.data_ptr(), code, rs if R > 1 else max(rs, V), R, V,
        _dense(u, f32, row, "u", dev), opt(temperature, f32, "temperature"),
        opt(top_k, torch.int32, "top_k"), opt(top_p, f32, "top_p"), opt(min_p, f32, "min_p"),
        token.data_ptr(), prob.data_ptr(), kept.data_ptr(), raw), "sv_sample_rows")
    return {"token": token, "prob": prob, "kept": kept}
