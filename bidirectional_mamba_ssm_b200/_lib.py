"""Thin ctypes binding of libbimamba.so (the C ABI in include/bimamba.h).

Argument marshalling only: tensors are passed as device pointers, the stream
is torch's current CUDA stream unless one is given, and a non-OK status is
raised as BimambaError.  All computation happens in the library's kernels;
there is no fallback of any kind -- if the shared library is missing or
cannot be loaded, importing this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbimamba.so")

BIMAMBA_OK = 0
BIMAMBA_ERR_INVALID = 1
BIMAMBA_ERR_UNSUPPORTED = 2
BIMAMBA_ERR_CUDA = 3
BIMAMBA_ERR_TIMEOUT = 4
BIMAMBA_ERR_WORKSPACE = 5
BIMAMBA_F32 = 0
BIMAMBA_BF16 = 1
BIMAMBA_FUSE_SUM = 0
BIMAMBA_FUSE_CONCAT = 1

# every symbol include/bimamba.h declares
EXPORTED = (
    "bimamba_version",
    "bimamba_launch_count",
    "bimamba_set_timing_events",
    "bimamba_strerror",
    "bimamba_get_error",
    "bimamba_conv_silu",
    "bimamba_workspace_bytes",
    "bimamba_launch_plan",
    "bimamba_ssd_fwd_rev",
    "bimamba_ssd_fwd_rev_untied",
    "bimamba_shard_states",
    "bimamba_ssd_fwd_rev_shard",
    "bimamba_block_decode",
    "bimamba_block_decode_pool",
    "bimamba_backward_workspace_bytes",
    "bimamba_ssd_fwd_rev_backward",
    "bimamba_in_proj",
    "bimamba_out_proj",
    "bimamba_prompt_workspace_bytes",
    "bimamba_prompt_scan",
    "bimamba_token_step_workspace_bytes",
    "bimamba_token_step",
    "bimamba_layer_norm",
    "bimamba_layer_norm_backward_workspace_bytes",
    "bimamba_layer_norm_backward",
    "bimamba_noalloc_scratch_bytes",
    "bimamba_block_decode_noalloc",
)


class BimambaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("len", ctypes.c_int), ("heads", ctypes.c_int),
                ("headdim", ctypes.c_int), ("d_state", ctypes.c_int), ("ngroups", ctypes.c_int),
                ("d_conv", ctypes.c_int), ("dtype", ctypes.c_int)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with "
                          "`python -m bidirectional_mamba_ssm_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    dp = ctypes.POINTER(Dims)
    lib.bimamba_version.restype = i
    lib.bimamba_version.argtypes = []
    lib.bimamba_launch_count.restype = ctypes.c_ulonglong
    lib.bimamba_launch_count.argtypes = []
    lib.bimamba_set_timing_events.restype = i
    lib.bimamba_set_timing_events.argtypes = [vp, vp]
    lib.bimamba_strerror.restype = ctypes.c_char_p
    lib.bimamba_strerror.argtypes = [i]
    lib.bimamba_get_error.restype = i
    lib.bimamba_get_error.argtypes = [vp]
    lib.bimamba_conv_silu.restype = i
    lib.bimamba_conv_silu.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
    lib.bimamba_workspace_bytes.restype = sz
    lib.bimamba_workspace_bytes.argtypes = [dp]
    lib.bimamba_launch_plan.restype = i
    lib.bimamba_launch_plan.argtypes = [dp, ctypes.POINTER(ctypes.c_int)]
    lib.bimamba_ssd_fwd_rev.restype = i
    lib.bimamba_ssd_fwd_rev.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.bimamba_ssd_fwd_rev_untied.restype = i
    lib.bimamba_ssd_fwd_rev_untied.argtypes = [dp] + [vp] * 15 + [i, vp, sz, vp]
    lib.bimamba_shard_states.restype = i
    lib.bimamba_shard_states.argtypes = [dp] + [vp] * 10 + [sz, vp]
    lib.bimamba_ssd_fwd_rev_shard.restype = i
    lib.bimamba_ssd_fwd_rev_shard.argtypes = [dp] + [vp] * 11 + [i, i, vp, vp, vp, sz, vp]
    lib.bimamba_block_decode.restype = i
    lib.bimamba_block_decode.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.bimamba_block_decode_pool.restype = i
    lib.bimamba_block_decode_pool.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, i, vp, vp, vp, vp,
                                              sz, vp]
    lib.bimamba_backward_workspace_bytes.restype = sz
    lib.bimamba_backward_workspace_bytes.argtypes = [dp]
    lib.bimamba_ssd_fwd_rev_backward.restype = i
    lib.bimamba_ssd_fwd_rev_backward.argtypes = [dp] + [vp] * 16 + [sz, vp]
    lib.bimamba_in_proj.restype = i
    lib.bimamba_in_proj.argtypes = [i, i, i, i, i, vp, vp, vp, vp, vp, vp]
    lib.bimamba_out_proj.restype = i
    lib.bimamba_out_proj.argtypes = [i, i, i, vp, vp, vp, vp]
    lib.bimamba_prompt_workspace_bytes.restype = sz
    lib.bimamba_prompt_workspace_bytes.argtypes = [dp]
    lib.bimamba_prompt_scan.restype = i
    lib.bimamba_prompt_scan.argtypes = [dp] + [vp] * 9 + [i] + [vp] * 4 + [sz, vp]
    lib.bimamba_token_step_workspace_bytes.restype = sz
    lib.bimamba_token_step_workspace_bytes.argtypes = [dp]
    lib.bimamba_token_step.restype = i
    lib.bimamba_token_step.argtypes = [dp] + [vp] * 8 + [i] + [vp] * 3 + [sz, vp]
    ll, f = ctypes.c_longlong, ctypes.c_float
    lib.bimamba_layer_norm.restype = i
    lib.bimamba_layer_norm.argtypes = [ll, i, vp, vp, vp, vp, f, vp, vp, vp, vp, i, vp]
    lib.bimamba_layer_norm_backward_workspace_bytes.restype = sz
    lib.bimamba_layer_norm_backward_workspace_bytes.argtypes = [ll, i]
    lib.bimamba_layer_norm_backward.restype = i
    lib.bimamba_layer_norm_backward.argtypes = [ll, i] + [vp] * 9 + [i, vp, sz, vp]
    lib.bimamba_noalloc_scratch_bytes.restype = sz
    lib.bimamba_noalloc_scratch_bytes.argtypes = []
    lib.bimamba_block_decode_noalloc.restype = i
    lib.bimamba_block_decode_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _code_of(dtype) -> int:
    if dtype == torch.float32:
        return BIMAMBA_F32
    if dtype == torch.bfloat16:
        return BIMAMBA_BF16
    raise BimambaError(BIMAMBA_ERR_UNSUPPORTED, f"dtype {dtype}")


def _dtype_code(t: torch.Tensor) -> int:
    return _code_of(t.dtype)


def _check(status: int, where: str):
    if status != BIMAMBA_OK:
        raise BimambaError(status, where)


def bimamba_version() -> int:
    return _lib.bimamba_version()


def bimamba_launch_count() -> int:
    """Kernels this library has launched in this process so far."""
    return int(_lib.bimamba_launch_count())


def bimamba_set_timing_events(start=None, stop=None):
    """Record torch.cuda.Event `start`/`stop` around the main scan kernel of
    every later call on this thread (None, None switches it off)."""
    st = _lib.bimamba_set_timing_events(None if start is None else start.cuda_event,
                                        None if stop is None else stop.cuda_event)
    _check(st, "bimamba_set_timing_events")


def strerror(status: int) -> str:
    return _lib.bimamba_strerror(status).decode()


bimamba_strerror = strerror


def bimamba_get_error(stream=None) -> int:
    """Synchronise `stream`, then read and clear the device status word."""
    return _lib.bimamba_get_error(_stream(stream))


def make_dims(batch, seqlen, heads, headdim, d_state, dtype, ngroups=1, d_conv=4) -> Dims:
    code = dtype if isinstance(dtype, int) else (
        BIMAMBA_F32 if dtype in (torch.float32, "f32") else BIMAMBA_BF16)
    return Dims(batch, seqlen, heads, headdim, d_state, ngroups, d_conv, code)


def bimamba_workspace_bytes(dims: Dims) -> int:
    return int(_lib.bimamba_workspace_bytes(ctypes.byref(dims)))


def bimamba_launch_plan(dims: Dims) -> dict:
    """How a call with these dims is launched (host only): tensor-core path
    or not, segments per direction, chunks per segment, state-only items."""
    out = (ctypes.c_int * 4)()
    _check(_lib.bimamba_launch_plan(ctypes.byref(dims), out), "bimamba_launch_plan")
    return {"tensor_core": bool(out[0]), "segments": out[1], "seg_chunks": out[2],
            "items": out[3]}


def new_workspace(dims: Dims, device=None) -> torch.Tensor:
    """Zero-filled workspace of the size the library asks for (>= 256 bytes)."""
    n = max(256, bimamba_workspace_bytes(dims))
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def bimamba_conv_silu(u, out, w, bias=None, tail=None, reverse=False, silu=True, stream=None):
    """out = SiLU(depthwise conv(u)) (or the pre-activation with silu=False)."""
    bsz, L, ch = u.shape
    st = _lib.bimamba_conv_silu(_ptr(u), _ptr(out), _ptr(w), _ptr(bias), _ptr(tail), bsz, L, ch,
                                w.shape[1], int(bool(reverse)), int(bool(silu)), _dtype_code(u),
                                _stream(stream))
    _check(st, "bimamba_conv_silu")
    return out


def bimamba_ssd_fwd_rev(xbc, dt, A, D, conv_w, conv_b, init_state, final_state, y, workspace,
                        *, heads, headdim, d_state, ngroups=1, stream=None, dims=None):
    """y = forward stream + reverse stream of the conv+SiLU'd selective scan."""
    if dims is None:
        bsz, L, _ = xbc.shape
        dims = make_dims(bsz, L, heads, headdim, d_state, _dtype_code(xbc), ngroups)
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.bimamba_ssd_fwd_rev(ctypes.byref(dims), _ptr(xbc), _ptr(dt), _ptr(A), _ptr(D),
                                  _ptr(conv_w), _ptr(conv_b), _ptr(init_state), _ptr(final_state),
                                  _ptr(y), _ptr(workspace), wsz, _stream(stream))
    _check(st, "bimamba_ssd_fwd_rev")
    return y


def bimamba_ssd_fwd_rev_untied(fwd, rev, init_state, final_state, y, workspace, *, heads,
                               headdim, d_state, concat=False, ngroups=1, stream=None):
    """Untied directions: `fwd` and `rev` are dicts with keys xbc, dt, A, D,
    conv_w, conv_b (conv_w/conv_b may be None) holding each stream's own
    inputs.  y = forward + reverse (concat=False, (batch, len, H*P)) or
    per token [forward | reverse] (concat=True, (batch, len, 2*H*P))."""
    bsz, L, _ = fwd["xbc"].shape
    dims = make_dims(bsz, L, heads, headdim, d_state, _dtype_code(fwd["xbc"]), ngroups)
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    g = lambda d, k: _ptr(d.get(k))
    st = _lib.bimamba_ssd_fwd_rev_untied(
        ctypes.byref(dims), g(fwd, "xbc"), g(rev, "xbc"), g(fwd, "dt"), g(rev, "dt"), g(fwd, "A"),
        g(rev, "A"), g(fwd, "D"), g(rev, "D"), g(fwd, "conv_w"), g(rev, "conv_w"), g(fwd, "conv_b"),
        g(rev, "conv_b"), _ptr(init_state), _ptr(final_state), _ptr(y),
        BIMAMBA_FUSE_CONCAT if concat else BIMAMBA_FUSE_SUM, _ptr(workspace), wsz, _stream(stream))
    _check(st, "bimamba_ssd_fwd_rev_untied")
    return y


def bimamba_shard_states(xbc, dt, A, conv_w, conv_b, tail, head, states, decays, workspace, *,
                         heads, headdim, d_state, ngroups=1, stream=None):
    """One sequence shard's end states from zero, (2, batch, H, P, N) [forward,
    reverse], and log2 decays (2, batch, H).  tail/head: (batch, 4, ch) raw
    tokens before/after the shard, or None (zeros)."""
    bsz, L, _ = xbc.shape
    dims = make_dims(bsz, L, heads, headdim, d_state, _dtype_code(xbc), ngroups)
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.bimamba_shard_states(ctypes.byref(dims), _ptr(xbc), _ptr(dt), _ptr(A), _ptr(conv_w),
                                   _ptr(conv_b), _ptr(tail), _ptr(head), _ptr(states),
                                   _ptr(decays), _ptr(workspace), wsz, _stream(stream))
    _check(st, "bimamba_shard_states")
    return states, decays


def bimamba_ssd_fwd_rev_shard(xbc, dt, A, D, conv_w, conv_b, tail, head, init_state, all_states,
                              all_decays, rank, nranks, final_state, y, workspace, *, heads,
                              headdim, d_state, ngroups=1, stream=None):
    """One sequence shard's outputs, entering with the states the other
    shards hand on (all_states / all_decays: every rank's shard states)."""
    bsz, L, _ = xbc.shape
    dims = make_dims(bsz, L, heads, headdim, d_state, _dtype_code(xbc), ngroups)
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.bimamba_ssd_fwd_rev_shard(
        ctypes.byref(dims), _ptr(xbc), _ptr(dt), _ptr(A), _ptr(D), _ptr(conv_w), _ptr(conv_b),
        _ptr(tail), _ptr(head), _ptr(init_state), _ptr(all_states), _ptr(all_decays), int(rank),
        int(nranks), _ptr(final_state), _ptr(y), _ptr(workspace), wsz, _stream(stream))
    _check(st, "bimamba_ssd_fwd_rev_shard")
    return y


def bimamba_block_decode(xbc_block, dt_block, A, D, conv_w, conv_b, state, tail, y, state_out,
                         tail_out, workspace, *, heads, headdim, d_state, ngroups=1, stream=None):
    """Cached block decode: forward resumes from (state, tail); reverse covers the block."""
    S, L, _ = xbc_block.shape
    dims = make_dims(S, L, heads, headdim, d_state, _dtype_code(xbc_block), ngroups)
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.bimamba_block_decode(ctypes.byref(dims), _ptr(xbc_block), _ptr(dt_block), _ptr(A),
                                   _ptr(D), _ptr(conv_w), _ptr(conv_b), _ptr(state), _ptr(tail),
                                   _ptr(y), _ptr(state_out), _ptr(tail_out), _ptr(workspace), wsz,
                                   _stream(stream))
    _check(st, "bimamba_block_decode")
    return y


def bimamba_block_decode_pool(xbc_block, dt_block, A, D, conv_w, conv_b, state_pool, tail_pool,
                              slots, commit, y, workspace, *, heads, headdim, d_state, ngroups=1,
                              stream=None):
    """Cached block decode of a batch of streams held in a pool: row s uses
    pool entry slots[s] (int32 device tensor) and, where commit[s] != 0 (all
    rows when commit is None), writes its new state and conv tail back there."""
    S, L, _ = xbc_block.shape
    dims = make_dims(S, L, heads, headdim, d_state, _dtype_code(xbc_block), ngroups)
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.bimamba_block_decode_pool(ctypes.byref(dims), _ptr(xbc_block), _ptr(dt_block), _ptr(A),
                                        _ptr(D), _ptr(conv_w), _ptr(conv_b), _ptr(state_pool),
                                        _ptr(tail_pool), int(state_pool.shape[0]), _ptr(slots),
                                        _ptr(commit), _ptr(y), _ptr(workspace), wsz, _stream(stream))
    _check(st, "bimamba_block_decode_pool")
    return y


def bimamba_backward_workspace_bytes(dims: Dims) -> int:
    return int(_lib.bimamba_backward_workspace_bytes(ctypes.byref(dims)))


def bimamba_ssd_fwd_rev_backward(xbc, dt, A, D, conv_w, conv_b, init_state, dy, *, heads, headdim,
                                 d_state, want_dinit=False, workspace=None, stream=None):
    """Gradients of sum(dy * y) for y = bimamba_ssd_fwd_rev(...): returns a dict
    of fp32 tensors xbc, dt, A, D, conv_w, conv_b (None without a bias) and
    init (None unless want_dinit)."""
    bsz, L, ch = xbc.shape
    dims = make_dims(bsz, L, heads, headdim, d_state, _dtype_code(xbc))
    dev = xbc.device
    f32 = torch.float32
    g = {"xbc": torch.empty((bsz, L, ch), dtype=f32, device=dev),
         "dt": torch.empty((bsz, L, heads), dtype=f32, device=dev),
         "A": torch.empty((heads,), dtype=f32, device=dev),
         "D": torch.empty((heads,), dtype=f32, device=dev),
         "conv_w": torch.empty((ch, 4), dtype=f32, device=dev),
         "conv_b": None if conv_b is None else torch.empty((ch,), dtype=f32, device=dev),
         "init": torch.empty((bsz, heads, headdim, d_state), dtype=f32, device=dev)
         if want_dinit else None}
    if workspace is None:
        workspace = torch.empty(max(256, bimamba_backward_workspace_bytes(dims)), dtype=torch.uint8,
                                device=dev)
    wsz = workspace.numel() * workspace.element_size()
    st = _lib.bimamba_ssd_fwd_rev_backward(
        ctypes.byref(dims), _ptr(xbc), _ptr(dt), _ptr(A), _ptr(D), _ptr(conv_w), _ptr(conv_b),
        _ptr(init_state), _ptr(dy), _ptr(g["xbc"]), _ptr(g["dt"]), _ptr(g["A"]), _ptr(g["D"]),
        _ptr(g["conv_w"]), _ptr(g["conv_b"]), _ptr(g["init"]), _ptr(workspace), wsz, _stream(stream))
    _check(st, "bimamba_ssd_fwd_rev_backward")
    return g


def bimamba_in_proj(u, w_in, dt_bias, xbc, dt, *, heads, headdim, d_state, stream=None):
    """[xbc | dt] = u . W_in^T with dt = softplus(. + dt_bias); u (tokens,
    d_model) bf16, w_in (ch + H, d_model) bf16, xbc (tokens, ch), dt (tokens, H)."""
    tokens, d_model = u.shape[-2] if u.dim() == 2 else u.shape[0] * u.shape[1], u.shape[-1]
    st = _lib.bimamba_in_proj(int(tokens), int(d_model), heads, headdim, d_state, _ptr(u), _ptr(w_in),
                              _ptr(dt_bias), _ptr(xbc), _ptr(dt), _stream(stream))
    _check(st, "bimamba_in_proj")
    return xbc, dt


def bimamba_out_proj(y, w_out, out, stream=None):
    """out = y . W_out^T; y (tokens, d_inner) bf16, w_out (d_model, d_inner) bf16."""
    d_inner = y.shape[-1]
    tokens = y.numel() // d_inner
    st = _lib.bimamba_out_proj(int(tokens), int(d_inner), int(w_out.shape[0]), _ptr(y), _ptr(w_out),
                               _ptr(out), _stream(stream))
    _check(st, "bimamba_out_proj")
    return out


def _call(where, fn, stream, before, specs, args, after):
    """fn(*before, args, *after, stream) with each tensor's pointer in its
    place.  A tensor's spec is (name, dtype, shape), dense on the first one's
    CUDA device (or None itself); where the spec is None the argument stands
    for itself.  That device is made current for the call: the kernels launch
    there, on its current stream unless one is given."""
    lead = args[0] if args[0] is not None else args[1]   # (a missing one is the library's to refuse)
    index = lead.get_device()
    if index < 0:
        raise BimambaError(BIMAMBA_ERR_INVALID, f"{where}: a CUDA tensor is wanted, got one on {lead.device}")
    out = []
    for spec, t in zip(specs, args):
        if t is None or spec is None:
            out.append(t)
            continue
        if t.dtype is not spec[1] or t.shape != spec[2] or t.get_device() != index or not t.is_contiguous():
            name, dtype, shape = spec
            raise BimambaError(BIMAMBA_ERR_INVALID, f"{where}: {name}: a dense {dtype} tensor of shape {tuple(shape)} "
                               f"on {lead.device} is wanted, got {t.dtype} {tuple(t.shape)} with strides "
                               f"{t.stride()} on {t.device}")
        out.append(t.data_ptr())
    # (the raw handle: a Stream object takes 3 us to make, a fifth of a call)
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if torch.cuda.current_device() == index:
        st = fn(*before, *out, *after, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*before, *out, *after, handle)
    if st != BIMAMBA_OK:
        raise BimambaError(st, where)


def _workspace(where, t, lead):
    """(pointer, bytes) of a call's workspace."""
    if t is None:
        return None, 0
    if t.device != lead.device or not t.is_contiguous():
        raise BimambaError(BIMAMBA_ERR_INVALID, f"{where}: workspace: a dense tensor on {lead.device} is wanted")
    return t.data_ptr(), t.numel() * t.element_size()


# What a call's sizes alone decide is made once for them (a few microseconds,
# where a short call takes some fifteen).
@functools.lru_cache(maxsize=1024)
def _causal_specs(td, rows, prompts, pool, heads, headdim, d_state):
    """(dims, specs) of the prompt scan, and with prompts None of the token step."""
    f32, i32, inner, ch = torch.float32, torch.int32, heads * headdim, heads * headdim + 2 * d_state
    step = prompts is None
    dims = make_dims(rows if step else prompts, 1 if step else rows, heads, headdim, d_state, _code_of(td))
    n = rows if step else prompts
    specs = [("xbc", td, (rows, ch)), ("dt", td, (rows, heads)), ("A", f32, (heads,)), ("D", f32, (heads,)),
             ("conv_w", f32, (ch, 4)), ("conv_b", f32, (ch,)), ("cu_seqlens", i32, (n + 1,)),
             ("state_pool", f32, (pool, heads, headdim, d_state)), ("tail_pool", td, (pool, 4, ch)), None,
             ("slots", i32, (n,)), ("resume", i32, (n,)), ("y", td, (rows, inner))]
    if step:
        specs = [v for v in specs if v is None or v[0] not in ("cu_seqlens", "resume")]
    return (ctypes.byref(dims),), tuple(specs)


@functools.lru_cache(maxsize=1024)
def _norm_specs(td, shape, backward):
    """(dtype code, (rows, cols), specs) of the layer norm or its backward pass."""
    if not shape:
        raise BimambaError(BIMAMBA_ERR_INVALID, "layer norm of a tensor without dimensions")
    f32, cols, each = torch.float32, shape[-1], shape[:-1]
    vec, rows = (cols,), shape.numel() // cols if cols else 0
    if backward:
        specs = (("dy", td, shape), ("h", td, shape), ("gamma", f32, vec), ("mean", f32, each), ("rstd", f32, each),
                 ("dsum", td, shape), ("dx", td, shape), ("dgamma", f32, vec), ("dbeta", f32, vec))
    else:
        specs = (("x", td, shape), ("residual", td, shape), ("gamma", f32, vec), ("beta", f32, vec), None,
                 ("y", td, shape), ("sum_out", td, shape), ("mean", f32, each), ("rstd", f32, each))
    return _code_of(td), (rows, cols), specs


def bimamba_prompt_workspace_bytes(dims: Dims) -> int:
    return int(_lib.bimamba_prompt_workspace_bytes(ctypes.byref(dims)))


def new_prompt_workspace(xbc, *, batch, heads, headdim, d_state) -> torch.Tensor:
    """Workspace for bimamba_prompt_scan on packed rows like xbc's or fewer,
    for up to `batch` prompts."""
    n = bimamba_prompt_workspace_bytes(make_dims(batch, xbc.shape[0], heads, headdim, d_state,
                                                 _dtype_code(xbc)))
    return torch.empty(max(256, n), dtype=torch.uint8, device=xbc.device)


def bimamba_prompt_scan(xbc, dt, A, D, conv_w, conv_b, cu_seqlens, state_pool, tail_pool, slots,
                        resume, y, workspace, *, heads, headdim, d_state, stream=None):
    """Causal conv + scan of packed prompts (prompt s: rows cu_seqlens[s] ..
    cu_seqlens[s+1]-1 of xbc (rows, ch) and dt (rows, H)) into y (rows, H*P);
    pool entry slots[s] gets the prompt's state and last raw tokens, and is
    what it continues from where resume[s] != 0 (resume None: nowhere).
    cu_seqlens, slots and resume are int32 device tensors."""
    pool = state_pool.shape[0]
    dims, specs = _causal_specs(xbc.dtype, xbc.shape[0], slots.shape[0], pool, heads, headdim, d_state)
    _call("bimamba_prompt_scan", _lib.bimamba_prompt_scan, stream, dims, specs,
          (xbc, dt, A, D, conv_w, conv_b, cu_seqlens, state_pool, tail_pool, pool, slots, resume, y),
          _workspace("bimamba_prompt_scan", workspace, xbc))
    return y


def bimamba_token_step_workspace_bytes(dims: Dims) -> int:
    return int(_lib.bimamba_token_step_workspace_bytes(ctypes.byref(dims)))


def new_step_workspace(rows, *, heads, headdim, d_state, dtype, device=None) -> torch.Tensor:
    """Zero-filled workspace for bimamba_token_step on up to `rows` rows."""
    n = bimamba_token_step_workspace_bytes(make_dims(rows, 1, heads, headdim, d_state, dtype))
    return torch.zeros(max(256, n), dtype=torch.uint8, device=device or "cuda")


def bimamba_token_step(xbc, dt, A, D, conv_w, conv_b, state_pool, tail_pool, slots, y, workspace, *,
                       heads, headdim, d_state, stream=None):
    """One new token of each of a batch of cached streams: row s of xbc
    (rows, ch) and dt (rows, H) continues from pool entry slots[s], which is
    updated in place, into row s of y (rows, H*P)."""
    pool = state_pool.shape[0]
    dims, specs = _causal_specs(xbc.dtype, xbc.shape[0], None, pool, heads, headdim, d_state)
    _call("bimamba_token_step", _lib.bimamba_token_step, stream, dims, specs,
          (xbc, dt, A, D, conv_w, conv_b, state_pool, tail_pool, pool, slots, y),
          _workspace("bimamba_token_step", workspace, xbc))
    return y


def bimamba_layer_norm(x, gamma, beta, y, mean, rstd, *, residual=None, sum_out=None, eps=1e-5,
                       stream=None):
    """y = layer norm of x (+ residual) over the last dimension, gamma/beta
    (beta may be None) fp32; mean and rstd (one fp32 value a row) and, with a
    residual, sum_out = x + residual are written for the backward pass."""
    code, sizes, specs = _norm_specs(x.dtype, x.shape, False)
    _call("bimamba_layer_norm", _lib.bimamba_layer_norm, stream, sizes, specs,
          (x, residual, gamma, beta, eps, y, sum_out, mean, rstd), (code,))
    return y


def bimamba_layer_norm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return int(_lib.bimamba_layer_norm_backward_workspace_bytes(rows, cols))


def new_layer_norm_workspace(x) -> torch.Tensor:
    """Workspace for bimamba_layer_norm_backward over rows like x's."""
    cols = x.shape[-1]
    n = bimamba_layer_norm_backward_workspace_bytes(x.numel() // cols if cols else 0, cols)
    return torch.empty(max(256, n), dtype=torch.uint8, device=x.device)


def bimamba_layer_norm_backward(dy, h, gamma, mean, rstd, dx, dgamma, dbeta, workspace, *, dsum=None,
                                stream=None):
    """Gradients of the layer norm from dy (and dsum, the gradient that
    reaches h past the norm): writes dx, dgamma and, unless None, dbeta.
    h is the forward call's x, or its sum_out where it had a residual."""
    code, sizes, specs = _norm_specs(h.dtype, h.shape, True)
    _call("bimamba_layer_norm_backward", _lib.bimamba_layer_norm_backward, stream, sizes, specs,
          (dy, h, gamma, mean, rstd, dsum, dx, dgamma, dbeta),
          (code, *_workspace("bimamba_layer_norm_backward", workspace, h)))
    return dx


def bimamba_noalloc_scratch_bytes() -> int:
    """Size of the fixed scratch array bimamba_block_decode_noalloc uses."""
    return int(_lib.bimamba_noalloc_scratch_bytes())


def bimamba_block_decode_noalloc(xbc_block, dt_block, A, D, conv_w, conv_b, state, tail, y,
                                 state_out, tail_out, *, heads, headdim, d_state, ngroups=1,
                                 stream=None):
    """Cached block decode for callers that cannot allocate device memory:
    same as bimamba_block_decode, but the scratch is the library's own fixed
    array (no workspace argument).  Calls sharing that array must not
    overlap on the GPU."""
    S, L, _ = xbc_block.shape
    dims = make_dims(S, L, heads, headdim, d_state, _dtype_code(xbc_block), ngroups)
    st = _lib.bimamba_block_decode_noalloc(ctypes.byref(dims), _ptr(xbc_block), _ptr(dt_block),
                                           _ptr(A), _ptr(D), _ptr(conv_w), _ptr(conv_b),
                                           _ptr(state), _ptr(tail), _ptr(y), _ptr(state_out),
                                           _ptr(tail_out), _stream(stream))
    _check(st, "bimamba_block_decode_noalloc")
    return y
