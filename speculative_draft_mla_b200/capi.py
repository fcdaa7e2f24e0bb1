"""Python binding of the C ABI in include/dspark_attn.h and include/dspark_latent.h (argument
marshalling only).

Every step of the attention runs in the CUDA library ``libdspark_attn.so``
built in-tree by ``speculative_draft_mla_b200.build``. There is no fallback:
if the library is missing or the tensors are not CUDA tensors, the calls raise.
Function names follow the C entry points without the ``dspark_`` prefix.

A call runs on the current stream of its tensors' device, or on ``stream``. Tensors that it allocates
come from that stream's memory and stay safe to use and to drop on the current one; that the inputs are
ready there, and live until they have been read, is the caller's part, as is waiting for ``stream``.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdspark_attn.so")

F32, BF16 = 0, 1
FLAG_REUSE_DESCRIPTOR = 1
STATUS = {0: "OK", 1: "ERR_NULL", 2: "ERR_SHAPE", 3: "ERR_DTYPE", 4: "ERR_ANCHOR", 5: "ERR_WORKSPACE",
          6: "ERR_CUDA", 7: "ERR_DEVICE", 8: "ERR_ALIGN", 9: "ERR_UNSUPPORTED", 10: "ERR_PAGE"}
EXPORTS = ("dspark_workspace_size", "dspark_build_descriptor", "dspark_attn_fwd", "dspark_attn_bwd",
           "dspark_get_error", "dspark_status_string", "dspark_sample_anchors", "dspark_launch_counter",
           "dspark_set_wait_limit_ns", "dspark_sample_anchors_gpu", "dspark_build_draft_inputs",
           "dspark_loss_workspace_size", "dspark_loss_fwd_bwd", "dspark_latent_workspace_size",
           "dspark_latent_attn_fwd", "dspark_latent_attn_bwd", "dspark_latent_row_bytes",
           "dspark_latent_cache_write", "dspark_latent_cache_read", "dspark_latent_paged_workspace_size",
           "dspark_latent_attn_paged")
MASK_ID = 154821  # the page's MASK token id


class Problem(ctypes.Structure):
    """Mirror of dspark_problem."""
    _fields_ = [("B", ctypes.c_int32), ("n_h", ctypes.c_int32), ("S", ctypes.c_int32), ("N", ctypes.c_int32),
                ("W", ctypes.c_int32), ("d_c", ctypes.c_int32), ("d_r", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("rope_base", ctypes.c_double), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class LatentProblem(ctypes.Structure):
    """Mirror of dspark_latent_problem."""
    _fields_ = [("B", ctypes.c_int32), ("n_h", ctypes.c_int32), ("S", ctypes.c_int32), ("N", ctypes.c_int32),
                ("W", ctypes.c_int32), ("d_l", ctypes.c_int32), ("d_r", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("rope_base", ctypes.c_double), ("scale", ctypes.c_double), ("reserved", ctypes.c_int32 * 2)]


class LatentCache(ctypes.Structure):
    """Mirror of dspark_latent_cache."""
    _fields_ = [("T", ctypes.c_int32), ("d_l", ctypes.c_int32), ("d_r", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class LatentPaged(ctypes.Structure):
    """Mirror of dspark_latent_paged."""
    _fields_ = [(f, ctypes.c_int32) for f in ("n_seq", "T", "n_h", "d_l", "d_r", "page_size", "n_pages", "max_pages",
                                              "max_kv_len", "window", "causal", "dtype", "kind", "reserved")] + \
               [(f, ctypes.c_int64) for f in ("q_token_stride", "q_head_stride", "o_token_stride", "o_head_stride")] + \
               [("rope_base", ctypes.c_double), ("scale", ctypes.c_double)]


class DsparkError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, STATUS.get(status, status), status_string(status)))


_lib = None


def load():
    """Load the CUDA library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libdspark_attn.so is not built; run `python -m speculative_draft_mla_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, u32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32
    pp = ctypes.POINTER(Problem)
    lib.dspark_workspace_size.argtypes = [pp]
    lib.dspark_workspace_size.restype = sz
    lib.dspark_build_descriptor.argtypes = [pp, vp, vp, vp, sz, vp]
    lib.dspark_attn_fwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp]
    lib.dspark_attn_bwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp]
    lib.dspark_get_error.argtypes = [vp, vp]
    lib.dspark_status_string.argtypes = [ctypes.c_int]
    lib.dspark_status_string.restype = ctypes.c_char_p
    lib.dspark_sample_anchors.argtypes = [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64, vp, vp]
    lib.dspark_sample_anchors.restype = ctypes.c_int64
    lib.dspark_attn_fwd_noalloc.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.dspark_attn_fwd_noalloc.restype = ctypes.c_int
    lib.dspark_launch_counter.argtypes = []
    lib.dspark_launch_counter.restype = ctypes.c_uint64
    i32 = ctypes.c_int32
    lib.dspark_sample_anchors_gpu.argtypes = [vp, i32, i32, i32, ctypes.c_uint64, vp, vp, vp]
    lib.dspark_sample_anchors_gpu.restype = ctypes.c_int
    lib.dspark_build_draft_inputs.argtypes = [vp, vp, i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp]
    lib.dspark_build_draft_inputs.restype = ctypes.c_int
    lib.dspark_loss_workspace_size.argtypes = [i32]
    lib.dspark_loss_workspace_size.restype = sz
    f32 = ctypes.c_float
    lib.dspark_loss_fwd_bwd.argtypes = [i32, i32, vp, vp, vp, vp, vp, f32, f32, f32, vp, vp, vp, vp, sz, vp]
    lib.dspark_loss_fwd_bwd.restype = ctypes.c_int
    lib.dspark_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.dspark_set_wait_limit_ns.restype = ctypes.c_uint64
    lp, lc, lq = ctypes.POINTER(LatentProblem), ctypes.POINTER(LatentCache), ctypes.POINTER(LatentPaged)
    f64 = ctypes.c_double
    lib.dspark_latent_workspace_size.argtypes = [lp]
    lib.dspark_latent_workspace_size.restype = sz
    lib.dspark_latent_attn_fwd.argtypes = [lp, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp]
    lib.dspark_latent_attn_bwd.argtypes = [lp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp]
    lib.dspark_latent_row_bytes.argtypes = [i32, i32, i32]
    lib.dspark_latent_row_bytes.restype = sz
    lib.dspark_latent_cache_write.argtypes = [lc, vp, vp, vp, f64, f64, vp, vp, vp, vp]
    lib.dspark_latent_cache_read.argtypes = [lc, vp, vp, vp, vp, vp]
    lib.dspark_latent_paged_workspace_size.argtypes = [lq]
    lib.dspark_latent_paged_workspace_size.restype = sz
    lib.dspark_latent_attn_paged.argtypes = [lq, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for f in ("dspark_latent_attn_fwd", "dspark_latent_attn_bwd", "dspark_latent_cache_write",
              "dspark_latent_cache_read", "dspark_latent_attn_paged"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("dspark_build_descriptor", "dspark_attn_fwd", "dspark_attn_bwd", "dspark_get_error"):
        getattr(lib, f).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status):
    return load().dspark_status_string(int(status)).decode()


def problem(B, n_h, S, N, W, d_c, d_r, d_v, rope_base=10000.0, dtype=BF16):
    return Problem(B, n_h, S, N, W, d_c, d_r, d_v, float(rope_base), int(dtype), 0)


def dtype_code(t):
    if t == torch.float32:
        return F32
    if t == torch.bfloat16:
        return BF16
    raise TypeError("unsupported dtype %s" % t)


def _ptr(t):
    return None if t is None or t.numel() == 0 else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, device, stream):
    """A tensor for a call on stream (None: the current one). It comes from that stream's memory, so that no work of
    the current stream can still hold it when the call writes it, and its memory is given away only after what both
    streams have been given by the time it is dropped."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if here != stream:
        t.record_stream(here)
    return t


def _check(status, where):
    if status != 0:
        raise DsparkError(status, where)


def workspace_size(prob):
    return int(load().dspark_workspace_size(ctypes.byref(prob)))


def alloc_workspace(prob, device, stream=None):
    n = workspace_size(prob)
    if n == 0:
        raise DsparkError(2, "workspace_size")
    return _empty(n, torch.uint8, device, stream)


def _cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def problem_of(q, kc, kr, v, anchors, S, W, rope_base):
    B, n_h, R, dqk = q.shape
    return problem(B, n_h, S, R // 5, W, kc.shape[-1], kr.shape[-1], v.shape[-1], rope_base, dtype_code(q.dtype))


def build_descriptor(prob, anchors, keep, workspace, stream=None):
    _cuda(anchors, keep, workspace)
    st = _stream(stream, workspace.device)
    _check(load().dspark_build_descriptor(ctypes.byref(prob), _ptr(anchors), _ptr(keep), _ptr(workspace),
                                          workspace.numel(), st), "dspark_build_descriptor")


def attn_fwd(q, kc, kr, v, anchors, keep, S, W, rope_base=10000.0, workspace=None, flags=0, out=None, stream=None):
    """Returns (o, lse, workspace). ``out`` may pass preallocated (o, lse)."""
    _cuda(q, kc, kr, v, anchors, keep)
    prob = problem_of(q, kc, kr, v, anchors, S, W, rope_base)
    if workspace is None:
        workspace = alloc_workspace(prob, q.device, stream)
    if out is None:
        o = _empty(q.shape[:3] + (v.shape[-1],), q.dtype, q.device, stream)
        lse = _empty(q.shape[:3], torch.float32, q.device, stream)
    else:
        o, lse = out
    _cuda(o, lse, workspace)
    st = _stream(stream, q.device)
    _check(load().dspark_attn_fwd(ctypes.byref(prob), _ptr(q), _ptr(kc), _ptr(kr), _ptr(v), _ptr(anchors),
                                  _ptr(keep), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(), flags, st),
           "dspark_attn_fwd")
    return o, lse, workspace


def attn_bwd(q, kc, kr, v, anchors, keep, o, lse, dout, S, W, rope_base=10000.0, workspace=None, flags=0,
             out=None, stream=None):
    """Returns (dq, dkc, dkr, dv). ``out`` may pass preallocated gradients."""
    _cuda(q, kc, kr, v, anchors, keep, o, lse, dout)
    prob = problem_of(q, kc, kr, v, anchors, S, W, rope_base)
    if workspace is None:
        workspace = alloc_workspace(prob, q.device, stream)
    if out is None:
        dq, dkc, dkr, dv = (_empty(t.shape, t.dtype, t.device, stream) for t in (q, kc, kr, v))
    else:
        dq, dkc, dkr, dv = out
    _cuda(dq, dkc, dkr, dv, workspace)
    st = _stream(stream, q.device)
    _check(load().dspark_attn_bwd(ctypes.byref(prob), _ptr(q), _ptr(kc), _ptr(kr), _ptr(v), _ptr(anchors),
                                  _ptr(keep), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dkc), _ptr(dkr),
                                  _ptr(dv), _ptr(workspace), workspace.numel(), flags, st), "dspark_attn_bwd")
    return dq, dkc, dkr, dv


def attn_fwd_noalloc(q, kc, kr, v, anchors, keep, S, W, rope_base=10000.0, out=None, error_word=None,
                     stream=None):
    """Forward through dspark_attn_fwd_noalloc (no workspace argument: the
    library's built-in scratch array is used). Returns (o, lse)."""
    _cuda(q, kc, kr, v, anchors, keep, error_word)
    prob = problem_of(q, kc, kr, v, anchors, S, W, rope_base)
    if out is None:
        o = _empty(q.shape[:3] + (v.shape[-1],), q.dtype, q.device, stream)
        lse = _empty(q.shape[:3], torch.float32, q.device, stream)
    else:
        o, lse = out
    _cuda(o, lse)
    st = _stream(stream, q.device)
    _check(load().dspark_attn_fwd_noalloc(ctypes.byref(prob), _ptr(q), _ptr(kc), _ptr(kr), _ptr(v), _ptr(anchors),
                                          _ptr(keep), _ptr(o), _ptr(lse), _ptr(error_word), st),
           "dspark_attn_fwd_noalloc")
    return o, lse


def get_error(workspace, stream=None):
    """Synchronise and read (and clear) the device error word; raises on error."""
    st = _stream(stream, workspace.device)
    _check(load().dspark_get_error(_ptr(workspace), st), "dspark_get_error")


def launch_counter():
    """Kernels the library has launched in this process so far."""
    return int(load().dspark_launch_counter())


def set_wait_limit_ns(ns):
    """Limit (ns) of the kernels' pipeline waits for later calls; 0 restores
    the default (2 s). Returns the previous limit."""
    return int(load().dspark_set_wait_limit_ns(int(ns)))


def sample_anchors_gpu(loss_mask, N, seed, stream=None):
    """GPU anchor sampler: loss_mask uint8 [B, S] (CUDA) -> (anchors int32 [B, N], keep uint8 [B, N])."""
    _cuda(loss_mask)
    if loss_mask.dtype != torch.uint8:
        raise TypeError("loss_mask must be uint8")
    B, S = loss_mask.shape
    anchors = _empty((B, N), torch.int32, loss_mask.device, stream)
    keep = _empty((B, N), torch.uint8, loss_mask.device, stream)
    _check(load().dspark_sample_anchors_gpu(_ptr(loss_mask), B, S, N, ctypes.c_uint64(seed & (2 ** 64 - 1)),
                                            _ptr(anchors), _ptr(keep), _stream(stream, loss_mask.device)),
           "dspark_sample_anchors_gpu")
    return anchors, keep


def build_draft_inputs(input_ids, loss_mask, anchors, keep, mask_id=MASK_ID, stream=None):
    """Draft-block inputs: input_ids int32 [B, S], loss_mask uint8 [B, S], anchors int32 / keep uint8
    [B, N] (CUDA) -> dict of [B, 5N] tensors: draft_ids, position_ids, labels, prev_ids (int32) and
    eval_mask (uint8)."""
    _cuda(input_ids, loss_mask, anchors, keep)
    if input_ids.dtype != torch.int32 or anchors.dtype != torch.int32 or loss_mask.dtype != torch.uint8 or \
            keep.dtype != torch.uint8:
        raise TypeError("input_ids / anchors int32, loss_mask / keep uint8")
    B, S = input_ids.shape
    N = anchors.shape[1]
    dev = input_ids.device
    out = {k: _empty((B, 5 * N), torch.int32, dev, stream)
           for k in ("draft_ids", "position_ids", "labels", "prev_ids")}
    out["eval_mask"] = _empty((B, 5 * N), torch.uint8, dev, stream)
    _check(load().dspark_build_draft_inputs(_ptr(input_ids), _ptr(loss_mask), B, S, N, _ptr(anchors), _ptr(keep),
                                            int(mask_id), _ptr(out["draft_ids"]), _ptr(out["position_ids"]),
                                            _ptr(out["labels"]), _ptr(out["prev_ids"]), _ptr(out["eval_mask"]),
                                            _stream(stream, dev)), "dspark_build_draft_inputs")
    return out


CE_ALPHA, L1_ALPHA, CONF_ALPHA = 1.0, 0.9, 1.0  # the page's loss coefficients


def dspark_loss(student_logits, teacher_logits, labels, conf_logits, eval_mask, with_grad=True,
                alphas=(CE_ALPHA, L1_ALPHA, CONF_ALPHA), workspace=None, stream=None):
    """DSpark loss over R draft steps: bf16 [R, V] logits, int32 labels, float conf logits, uint8
    eval_mask (CUDA). Returns (loss [4] float: total, CE, L1, BCE means; grad_logits or None;
    grad_conf or None; workspace)."""
    _cuda(student_logits, teacher_logits, labels, conf_logits, eval_mask)
    if student_logits.dtype != torch.bfloat16 or teacher_logits.dtype != torch.bfloat16:
        raise TypeError("logits must be bf16")
    R, V = student_logits.shape
    dev = student_logits.device
    if workspace is None:
        workspace = _empty(int(load().dspark_loss_workspace_size(R)), torch.uint8, dev, stream)
    out = _empty(4, torch.float32, dev, stream)
    grad = _empty(student_logits.shape, student_logits.dtype, dev, stream) if with_grad else None
    gconf = _empty(R, torch.float32, dev, stream) if with_grad else None
    _check(load().dspark_loss_fwd_bwd(R, V, _ptr(student_logits), _ptr(teacher_logits), _ptr(labels),
                                      _ptr(conf_logits), _ptr(eval_mask), float(alphas[0]), float(alphas[1]),
                                      float(alphas[2]), _ptr(out), _ptr(grad), _ptr(gconf), _ptr(workspace),
                                      workspace.numel(), _stream(stream, dev)), "dspark_loss_fwd_bwd")
    return out, grad, gconf, workspace


def sample_anchors(loss_mask, N, seed):
    """Host anchor sampler: loss_mask uint8 [B, S] (CPU) -> (anchors int32, keep uint8), CPU."""
    lm = loss_mask.to(torch.uint8).contiguous().cpu()
    B, S = lm.shape
    anchors = torch.empty(B, N, dtype=torch.int32)
    keep = torch.empty(B, N, dtype=torch.uint8)
    rc = load().dspark_sample_anchors(_ptr(lm), B, S, N, ctypes.c_uint64(seed), _ptr(anchors), _ptr(keep))
    if rc < 0:
        raise DsparkError(2, "dspark_sample_anchors")
    return anchors, keep


# ---- latent space (include/dspark_latent.h) --------------------------------------------------
CACHE_F32, CACHE_BF16, CACHE_FP8 = 0, 1, 2
LATENT_SCALE = 256 ** -0.5  # of the page's expanded head, 192 + 64 wide


def latent_problem(B, n_h, S, N, W, d_l=512, d_r=64, scale=LATENT_SCALE, rope_base=10000.0, dtype=BF16):
    return LatentProblem(B, n_h, S, N, W, d_l, d_r, int(dtype), float(rope_base), float(scale), (0, 0))


def latent_workspace_size(prob):
    return int(load().dspark_latent_workspace_size(ctypes.byref(prob)))


def alloc_latent_workspace(prob, device, stream=None):
    n = latent_workspace_size(prob)
    if n == 0:
        raise DsparkError(2, "latent_workspace_size")
    return _empty(n, torch.uint8, device, stream)


def _same(name, t, shape, dtype, device):
    """t is a contiguous CUDA tensor of this shape, type and device."""
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous() and t.is_cuda:
        return
    if t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s is on %s, not %s" % (name, t.device, device))
    _cuda(t)


def _ws_ok(ws, device):
    if not (ws.is_cuda and ws.dtype is torch.uint8 and ws.device == device and ws.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % device)


def _call(name, device, stream, *args):
    """The entry point on the tensors' device and, unless one is given, its current stream (the last argument)."""
    f = getattr(_lib or load(), name)
    at = device.index
    if torch._C._cuda_getDevice() == at:
        status = f(*args, torch._C._cuda_getCurrentRawStream(at) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            status = f(*args, torch._C._cuda_getCurrentRawStream(at) if stream is None else stream.cuda_stream)
    if status:
        raise DsparkError(status, name)


def _at(t):
    return t.data_ptr() or None  # (an empty tensor has no address)


def _latent_args(q, c, kr, anchors, keep, S, W, scale, rope_base):
    if not q.is_cuda or not q.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    if q.dim() != 4 or c.dim() != 3 or kr.dim() != 3 or q.shape[2] % 5:
        raise ValueError("q [B, n_h, 5N, d_l + d_r], c [B, S + 5N, d_l], kr [B, S + 5N, d_r]")
    B, n_h, R, dk = q.shape
    d_l, d_r = c.shape[2], kr.shape[2]
    if dk != d_l + d_r:
        raise ValueError("q is %d wide, c and kr %d + %d" % (dk, d_l, d_r))
    dt, dev = q.dtype, q.device
    _same("c", c, (B, S + R, d_l), dt, dev)
    _same("kr", kr, (B, S + R, d_r), dt, dev)
    _same("anchors", anchors, (B, R // 5), torch.int32, dev)
    _same("keep", keep, (B, R // 5), torch.uint8, dev)
    return latent_problem(B, n_h, S, R // 5, W, d_l, d_r, scale, rope_base, dtype_code(dt))


def latent_attn_fwd(q, c, kr, anchors, keep, S, W, scale=LATENT_SCALE, rope_base=10000.0, workspace=None, flags=0,
                    out=None, stream=None):
    """Draft attention over latents: q [B, n_h, 5N, d_l + d_r], c [B, S + 5N, d_l], kr [B, S + 5N, d_r].
    Returns (o [B, n_h, 5N, d_l], lse, workspace). ``out`` may pass preallocated (o, lse)."""
    prob = _latent_args(q, c, kr, anchors, keep, S, W, scale, rope_base)
    dev, rows = q.device, tuple(q.shape[:3])
    if workspace is None:
        workspace = alloc_latent_workspace(prob, dev, stream)
    if out is None:
        o = _empty(rows + (prob.d_l,), q.dtype, dev, stream)
        lse = _empty(rows, torch.float32, dev, stream)
    else:
        o, lse = out
        _same("o", o, rows + (prob.d_l,), q.dtype, dev)
        _same("lse", lse, rows, torch.float32, dev)
    _ws_ok(workspace, dev)
    _call("dspark_latent_attn_fwd", dev, stream, ctypes.byref(prob), _at(q), _at(c), _at(kr), _at(anchors), _at(keep),
          _at(o), _at(lse), _at(workspace), workspace.numel(), flags)
    return o, lse, workspace


def latent_attn_bwd(q, c, kr, anchors, keep, lse, dout, S, W, scale=LATENT_SCALE, rope_base=10000.0, workspace=None,
                    flags=0, out=None, stream=None):
    """Returns (dq, dc, dkr) for dL/dO = dout and the forward's lse (its O is not needed). ``out`` may pass
    preallocated gradients."""
    prob = _latent_args(q, c, kr, anchors, keep, S, W, scale, rope_base)
    dev, rows = q.device, tuple(q.shape[:3])
    if workspace is None:
        workspace = alloc_latent_workspace(prob, dev, stream)
    _same("lse", lse, rows, torch.float32, dev)
    _same("dout", dout, rows + (prob.d_l,), q.dtype, dev)
    if out is None:
        dq, dc, dkr = (_empty(t.shape, t.dtype, dev, stream) for t in (q, c, kr))
    else:
        dq, dc, dkr = out
        for name, g, x in (("dq", dq, q), ("dc", dc, c), ("dkr", dkr, kr)):
            _same(name, g, x.shape, q.dtype, dev)
    _ws_ok(workspace, dev)
    _call("dspark_latent_attn_bwd", dev, stream, ctypes.byref(prob), _at(q), _at(c), _at(kr), _at(anchors), _at(keep),
          _at(lse), _at(dout), _at(dq), _at(dc), _at(dkr), _at(workspace), workspace.numel(), flags)
    return dq, dc, dkr


def latent_row_bytes(kind, d_l, d_r):
    return int(load().dspark_latent_row_bytes(int(kind), int(d_l), int(d_r)))


_KINDS = {torch.float32: CACHE_F32, torch.bfloat16: CACHE_BF16, torch.uint8: CACHE_FP8}


def _cache_kind(cache, d_l, d_r):
    """Kind of a cache tensor [n_pages, page_size, row]: float32 / bfloat16 rows of d_l + d_r values, or the
    bytes (uint8) of the 8-bit kind."""
    kind = _KINDS.get(cache.dtype)
    if kind is None or cache.dim() != 3:
        raise ValueError("cache must be [n_pages, page_size, row] of float32, bfloat16 or uint8 (the 8-bit kind)")
    if not cache.is_cuda or not cache.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    if cache.shape[2] * cache.itemsize != latent_row_bytes(kind, d_l, d_r):
        raise ValueError("cache rows of %d elements do not fit d_l = %d, d_r = %d" % (cache.shape[2], d_l, d_r))
    return kind


def latent_cache(n_pages, page_size, d_l=512, d_r=64, kind=CACHE_BF16, device="cuda"):
    """A zeroed paged cache of the given kind."""
    nb = latent_row_bytes(kind, d_l, d_r)
    if nb == 0:
        raise DsparkError(9, "latent_row_bytes")
    dt = {CACHE_F32: torch.float32, CACHE_BF16: torch.bfloat16, CACHE_FP8: torch.uint8}[kind]
    return torch.zeros(n_pages, page_size, nb // dt.itemsize, dtype=dt, device=device)


def latent_cache_write(cache, c, kr, positions, slots, norm_weight=None, eps=1e-5, rope_base=10000.0, stream=None):
    """Writes T tokens' latents c [T, d_l] (RMS-normed when norm_weight [d_l] is given) and rope keys kr [T, d_r]
    (turned to positions [T] int32) into rows slots [T] int64 of the cache; a slot out of range writes nothing."""
    if c.dim() != 2 or kr.dim() != 2:
        raise ValueError("c [T, d_l], kr [T, d_r]")
    T, d_l = c.shape
    d_r, dt, dev = kr.shape[1], c.dtype, cache.device
    kind = _cache_kind(cache, d_l, d_r)
    _same("c", c, (T, d_l), dt, dev)
    _same("kr", kr, (T, d_r), dt, dev)
    _same("positions", positions, (T,), torch.int32, dev)
    _same("slots", slots, (T,), torch.int64, dev)
    if norm_weight is not None:
        _same("norm_weight", norm_weight, (d_l,), dt, dev)
    prob = LatentCache(T, d_l, d_r, kind, cache.shape[0], cache.shape[1], dtype_code(dt), 0)
    _call("dspark_latent_cache_write", dev, stream, ctypes.byref(prob), _at(c), _at(kr),
          None if norm_weight is None else _at(norm_weight), float(eps), float(rope_base), _at(positions), _at(slots),
          _at(cache))


def latent_cache_read(cache, slots, d_l=512, d_r=64, dtype=torch.bfloat16, stream=None):
    """Rows slots [T] int64 as the values that they stand for: (c [T, d_l], rotated rope keys [T, d_r])."""
    kind = _cache_kind(cache, d_l, d_r)
    dev, T = cache.device, slots.numel()
    _same("slots", slots, (T,), torch.int64, dev)
    if stream is None:  # (quicker than torch.empty)
        c, kr = cache.new_empty((T, d_l), dtype=dtype), cache.new_empty((T, d_r), dtype=dtype)
    else:
        c, kr = _empty((T, d_l), dtype, dev, stream), _empty((T, d_r), dtype, dev, stream)
    prob = LatentCache(T, d_l, d_r, kind, cache.shape[0], cache.shape[1], dtype_code(dtype), 0)
    _call("dspark_latent_cache_read", dev, stream, ctypes.byref(prob), _at(cache), _at(slots), _at(c), _at(kr))
    return c, kr


def _paged(q, cache, block_table, max_kv_len, d_l, d_r, scale, causal, window, rope_base, o=None):
    kind = _cache_kind(cache, d_l, d_r)
    if not q.is_cuda or q.dim() != 3 or q.shape[2] != d_l + d_r:
        raise ValueError("q must be a CUDA tensor [T, n_h, d_l + d_r]")
    T, n_h = q.shape[:2]

    def strides(name, t):
        if t is None or t.numel() == 0:
            return 0, 0
        a, b, c = t.stride()
        if c != 1:
            raise ValueError("%s must be contiguous in its last dimension" % name)
        if (a == 0 and T > 1) or (b == 0 and n_h > 1):  # (two zeros stand for contiguous)
            raise ValueError("%s must not repeat tokens or heads" % name)
        return a, b

    n_seq, max_pages = block_table.shape
    return LatentPaged(n_seq, T, n_h, d_l, d_r, cache.shape[1], cache.shape[0], max_pages, int(max_kv_len), int(window),
                       int(bool(causal)), dtype_code(q.dtype), kind, 0, *strides("q", q), *strides("o", o),
                       float(rope_base), float(scale))


def latent_paged_workspace_size(prob):
    return int(load().dspark_latent_paged_workspace_size(ctypes.byref(prob)))


def alloc_latent_paged_workspace(q, cache, block_table, max_kv_len=0, d_l=512, d_r=64, window=0, stream=None):
    """Workspace of latent_attn_paged for these sizes (any mask)."""
    prob = _paged(q, cache, block_table, max_kv_len, d_l, d_r, LATENT_SCALE, True, window, 10000.0)
    n = latent_paged_workspace_size(prob)
    if n == 0:
        raise DsparkError(2, "latent_paged_workspace_size")
    return _empty(n, torch.uint8, q.device, stream)


def latent_attn_paged(q, cache, block_table, q_start, kv_len, max_kv_len=0, d_l=512, d_r=64, scale=LATENT_SCALE,
                      causal=True, window=0, rope_base=10000.0, workspace=None, out=None, stream=None):
    """New tokens q [T, n_h, d_l + d_r] (token and head strides free) over a paged latent cache. q_start
    [n_seq + 1], kv_len [n_seq] and block_table [n_seq, max_pages] int32. causal=False is a draft block whose
    tokens see one another. Returns (o [T, n_h, d_l], lse [T, n_h], workspace); rows behind the last sequence are
    left as they were in ``out`` and are unspecified otherwise."""
    dev, T, n_h = q.device, q.shape[0], q.shape[1]
    if out is None:
        o = _empty((T, n_h, d_l), q.dtype, dev, stream)
        lse = _empty((T, n_h), torch.float32, dev, stream)
    else:
        o, lse = out
        if o.shape != (T, n_h, d_l) or o.dtype != q.dtype or o.device != dev:
            raise ValueError("o must be [T, n_h, d_l] like q")
        _same("lse", lse, (T, n_h), torch.float32, dev)
    prob = _paged(q, cache, block_table, max_kv_len, d_l, d_r, scale, causal, window, rope_base, o)
    if cache.device != dev:
        raise ValueError("cache is on %s, not %s" % (cache.device, dev))
    n_seq = prob.n_seq
    _same("block_table", block_table, (n_seq, prob.max_pages), torch.int32, dev)
    _same("q_start", q_start, (n_seq + 1,), torch.int32, dev)
    _same("kv_len", kv_len, (n_seq,), torch.int32, dev)
    if workspace is None:
        workspace = _empty(max(latent_paged_workspace_size(prob), 256), torch.uint8, dev, stream)
    _ws_ok(workspace, dev)
    _call("dspark_latent_attn_paged", dev, stream, ctypes.byref(prob), _at(q), _at(cache), _at(block_table),
          _at(q_start), _at(kv_len), _at(o), _at(lse), _at(workspace), workspace.numel())
    return o, lse, workspace
