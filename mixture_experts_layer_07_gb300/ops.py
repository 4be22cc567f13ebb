"""Binding of ``libmoe_gb300.so`` -- argument marshalling only: ctypes, and for the operators
around the layer (norm, router losses, gradients) the C module ``_moe_binding``.

Each function has the name of the C entry point it calls (without the
``moe_`` prefix), passes tensor data pointers and the current CUDA stream, and
raises ``MoEError`` when the library returns a status other than MOE_OK.
Every step of the layer runs in the library's CUDA kernels; nothing here
computes.  If the library is not built the import of any function raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sysconfig

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gb300.so")
BINDING_PATH = os.path.join(_HERE, "_moe_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

MODE_SOFTMAX, MODE_SIGMOID_BIAS = 0, 1
W_BF16, W_FP8, W_MXFP4, W8A8_FP8 = 0, 1, 2, 3
DISPATCH_PER_BLOCK, DISPATCH_GLOBAL_AVG, DISPATCH_SIMT, DISPATCH_ONE_LAUNCH, DISPATCH_GEMV = \
    0, 1, 2, 3, 4
VARIANT_SKIP, VARIANT_SKINNY, VARIANT_TILE, VARIANT_SIMT, VARIANT_WIDE = 0, 1, 2, 3, 4
WIDE_MIN_ROWS = 129
DEV_OK, DEV_BAD_EXPERT_ID, DEV_WAIT_TIMEOUT = 0, 1, 2

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_MISALIGNED", 5: "MOE_ERR_CUDA",
          6: "MOE_ERR_DEVICE_STATUS"}

EXPORTS = ["moe_status_string", "moe_default_m_skinny", "moe_block_variant", "moe_router_gemm",
           "moe_topk_route", "moe_permute_scratch_bytes", "moe_permute",
           "moe_grouped_gemm_scratch_bytes", "moe_grouped_gemm_scratch_bytes_ex",
           "moe_grouped_gemm", "moe_unpermute",
           "moe_workspace_bytes", "moe_layer", "moe_workspace_layout", "moe_permute_static",
           "moe_router_tc_scratch_bytes", "moe_router_gemm_tc", "moe_bounded_wait_check",
           "moe_add_rmsnorm", "moe_add_rmsnorm_backward_scratch_bytes",
           "moe_add_rmsnorm_backward", "moe_balance_loss_scratch_bytes", "moe_balance_loss",
           "moe_route_backward", "moe_unpermute_backward", "moe_layer_q8"]

PERMUTE_STATIC_SCRATCH_BYTES = 1 << 20
DT_BF16, DT_F32 = 0, 1


class MoEError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({_lib().moe_status_string(code).decode()})")


class Config(ctypes.Structure):
    _fields_ = [("T_max", ctypes.c_int), ("H", ctypes.c_int), ("E", ctypes.c_int),
                ("K", ctypes.c_int), ("I", ctypes.c_int), ("has_shared", ctypes.c_int),
                ("I_shared", ctypes.c_int), ("mode", ctypes.c_int),
                ("routed_scale", ctypes.c_float), ("wdtype", ctypes.c_int),
                ("m_skinny", ctypes.c_int), ("dispatch", ctypes.c_int)]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("wg", "gate_bias", "sel_bias", "w1", "w3", "w2", "s1", "s3", "s2",
                 "sw1", "sw3", "sw2")]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("logits", "ids", "weights", "shared_gate", "offsets", "row_to_flat",
                 "flat_to_row", "xp", "hact", "y", "shared_hact", "shared_y", "block_variant",
                 "permute_scratch", "gemm_scratch", "shared_gemm_scratch", "sync", "splitk",
                 "router_split", "total")]


_L = None
_B = None  # _moe_binding, once an operator that goes through it is called
_P, _I, _F, _S, _I64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                        ctypes.c_int64)


def _built(path):
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run __graft_entry__.build() "
                           "(the MoE path has no fallback)")
    return path


def _lib():
    global _L
    if _L is None:
        lib = ctypes.CDLL(_built(LIB_PATH))
        lib.moe_status_string.restype = ctypes.c_char_p
        lib.moe_status_string.argtypes = [_I]
        lib.moe_default_m_skinny.restype = _I
        lib.moe_default_m_skinny.argtypes = []
        lib.moe_block_variant.restype = _I
        lib.moe_block_variant.argtypes = [_I64, _I64, _I, _I, _I, _I]
        sig = {
            "moe_router_gemm": [_P, _P, _P, _P, _I, _I, _I, _P],
            "moe_router_tc_scratch_bytes": [_I, _I, ctypes.POINTER(_S)],
            "moe_router_gemm_tc": [_P, _P, _P, _P, _I, _I, _I, _P, _S, _P, _P],
            "moe_topk_route": [_P, _I, _P, _I, _I, _I, _I, _F, _P, _P, _P, _P],
            "moe_permute_scratch_bytes": [_I, _I, _I, ctypes.POINTER(_S)],
            "moe_permute": [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _S, _P, _P],
            "moe_permute_static": [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P],
            "moe_grouped_gemm_scratch_bytes": [_I, _I, ctypes.POINTER(_S)],
            "moe_grouped_gemm_scratch_bytes_ex": [_I, _I, _I, _I, _I, ctypes.POINTER(_S)],
            "moe_grouped_gemm": [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I,
                                 _I, _P, _P, _S, _P, _P],
            "moe_unpermute": [_P, _P, _P, _I, _I, _I, _P, _P, _P, _P],
            "moe_workspace_bytes": [ctypes.POINTER(Config), ctypes.POINTER(_S)],
            "moe_workspace_layout": [ctypes.POINTER(Config), ctypes.POINTER(WorkspaceLayout)],
            "moe_layer": [ctypes.POINTER(Config), _I, _P, ctypes.POINTER(Weights), _P, _P, _S,
                          _P, _P],
            "moe_bounded_wait_check": [_P, _I, _I, _P, _P],
            "moe_layer_q8": [ctypes.POINTER(Config), _I, _P, _P, _P, ctypes.POINTER(Weights), _P,
                             _P, _S, _P, _P],
            "moe_add_rmsnorm": [_P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _P, _P, _I, _P],
            "moe_add_rmsnorm_backward_scratch_bytes": [_I, _I, ctypes.POINTER(_S)],
            "moe_add_rmsnorm_backward": [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _S, _P],
            "moe_balance_loss_scratch_bytes": [_I, _I, _I, ctypes.POINTER(_S)],
            "moe_balance_loss": [_P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _S, _P,
                                 _P],
            "moe_route_backward": [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P,
                                   _P, _I, _P, _P],
            "moe_unpermute_backward": [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.restype = _I
            fn.argtypes = args
        _L = lib
    return _L


def lib():
    return _lib()


def binding():
    """The C module of the operators around the layer; nothing else needs it."""
    global _B
    if _B is None:
        name = __package__ + "._moe_binding"
        spec = importlib.util.spec_from_file_location(name, _built(BINDING_PATH))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.connect(*[ctypes.cast(getattr(_lib(), "moe_" + n), _P).value for n in
                         ("add_rmsnorm", "add_rmsnorm_backward", "balance_loss",
                          "route_backward", "unpermute_backward")])
        _B = module
    return _B


def _p(t):
    """Device pointer of a tensor (or None / a raw int)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:  # torch.cuda.current_stream().cuda_stream without its Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _empty_like(x, stream):
    """A tensor like x that `stream` fills: of that stream's memory, as torch allocates inside
    torch.cuda.stream(stream) -- memory freed on another stream may still be in use there."""
    if stream is None or not x.is_cuda:
        return torch.empty_like(x)
    handle = _stream(stream)  # 0, the default stream's, would make ExternalStream a new stream
    s = torch.cuda.ExternalStream(handle, device=x.device) if handle else \
        torch.cuda.default_stream(x.device)
    with torch.cuda.stream(s):
        return torch.empty_like(x)


def _check(code, where):
    if code != 0:
        raise MoEError(code, where)


# ---------------------------------------------------------------- host-only
def status_string(code: int) -> str:
    return _lib().moe_status_string(code).decode()


def default_m_skinny() -> int:
    return _lib().moe_default_m_skinny()


def block_variant(m_size: int, R: int, E: int, m_skinny: int = -1,
                  dispatch: int = DISPATCH_PER_BLOCK, wdtype: int = W_BF16) -> int:
    return _lib().moe_block_variant(m_size, R, E, m_skinny, dispatch, wdtype)


def permute_scratch_bytes(T: int, E: int, K: int) -> int:
    n = _S()
    _check(_lib().moe_permute_scratch_bytes(T, E, K, ctypes.byref(n)), "moe_permute_scratch_bytes")
    return n.value


def grouped_gemm_scratch_bytes(R: int, E_blocks: int, H: int = 0, I: int = 0,
                               wdtype: int = W_BF16) -> int:
    n = _S()
    if wdtype == W8A8_FP8:
        _check(_lib().moe_grouped_gemm_scratch_bytes_ex(R, E_blocks, H, I, wdtype,
                                                        ctypes.byref(n)),
               "moe_grouped_gemm_scratch_bytes_ex")
    else:
        _check(_lib().moe_grouped_gemm_scratch_bytes(R, E_blocks, ctypes.byref(n)),
               "moe_grouped_gemm_scratch_bytes")
    return n.value


def make_config(T_max, H, E, K, I, *, has_shared=False, I_shared=0, mode=MODE_SOFTMAX,
                routed_scale=1.0, wdtype=W_BF16, m_skinny=-1, dispatch=DISPATCH_PER_BLOCK) -> Config:
    return Config(T_max, H, E, K, I, int(has_shared), I_shared, mode, routed_scale, wdtype,
                  m_skinny, dispatch)


def workspace_bytes(cfg: Config) -> int:
    n = _S()
    _check(_lib().moe_workspace_bytes(ctypes.byref(cfg), ctypes.byref(n)), "moe_workspace_bytes")
    return n.value


def workspace_layout(cfg: Config) -> WorkspaceLayout:
    L = WorkspaceLayout()
    _check(_lib().moe_workspace_layout(ctypes.byref(cfg), ctypes.byref(L)), "moe_workspace_layout")
    return L


# ---------------------------------------------------------------- stages
def router_gemm(x, wg, gate_bias, logits, stream=None):
    T, H = x.shape
    G = wg.shape[0]
    _check(_lib().moe_router_gemm(_p(x), _p(wg), _p(gate_bias), _p(logits), T, H, G,
                                  _stream(stream)), "moe_router_gemm")


def router_tc_scratch_bytes(H: int, G: int) -> int:
    n = _S()
    _check(_lib().moe_router_tc_scratch_bytes(H, G, ctypes.byref(n)), "moe_router_tc_scratch_bytes")
    return n.value


def router_gemm_tc(x, wg, gate_bias, logits, scratch, dev_status=None, stream=None):
    T, H = x.shape
    G = wg.shape[0]
    _check(_lib().moe_router_gemm_tc(_p(x), _p(wg), _p(gate_bias), _p(logits), T, H, G,
                                     _p(scratch), scratch.numel() * scratch.element_size(),
                                     _p(dev_status), _stream(stream)), "moe_router_gemm_tc")


def topk_route(logits, E, K, mode, scale, ids, weights, sel_bias=None, shared_gate=None,
               stream=None):
    T, ld = logits.shape
    _check(_lib().moe_topk_route(_p(logits), ld, _p(sel_bias), T, E, K, mode, float(scale),
                                 _p(ids), _p(weights), _p(shared_gate), _stream(stream)),
           "moe_topk_route")


def permute(x, ids, E, offsets, row_to_flat, flat_to_row, xp, scratch, dev_status=None,
            stream=None, H=None):
    T, K = ids.shape
    H = x.shape[1] if x is not None else H
    _check(_lib().moe_permute(_p(x), _p(ids), T, H, E, K, _p(offsets), _p(row_to_flat),
                              _p(flat_to_row), _p(xp), _p(scratch), scratch.numel(),
                              _p(dev_status), _stream(stream)), "moe_permute")


def permute_static(x, ids, E, offsets, row_to_flat, flat_to_row, xp, dev_status=None,
                   stream=None, H=None):
    """moe_permute_static: moe_permute with the library's built-in scratch, for
    callers that cannot allocate device memory (see the header)."""
    T, K = ids.shape
    H = x.shape[1] if x is not None else H
    _check(_lib().moe_permute_static(_p(x), _p(ids), T, H, E, K, _p(offsets), _p(row_to_flat),
                                     _p(flat_to_row), _p(xp), _p(dev_status), _stream(stream)),
           "moe_permute_static")


def grouped_gemm(xp, offsets, E_blocks, H, I, w1, w3, w2, hact, y, scratch, *, wdtype=W_BF16,
                 s1=None, s3=None, s2=None, m_skinny=-1, dispatch=DISPATCH_PER_BLOCK,
                 block_variant=None, dev_status=None, stream=None, R=None):
    R = xp.shape[0] if R is None else R
    _check(_lib().moe_grouped_gemm(_p(xp), _p(offsets), E_blocks, R, H, I, wdtype, _p(w1),
                                   _p(w3), _p(w2), _p(s1), _p(s3), _p(s2), _p(hact), _p(y),
                                   m_skinny, dispatch, _p(block_variant), _p(scratch),
                                   scratch.numel(), _p(dev_status), _stream(stream)),
           "moe_grouped_gemm")


def unpermute(y, flat_to_row, weights, T, K, H, out, shared_y=None, shared_gate=None,
              stream=None):
    _check(_lib().moe_unpermute(_p(y), _p(flat_to_row), _p(weights), T, K, H, _p(shared_y),
                                _p(shared_gate), _p(out), _stream(stream)), "moe_unpermute")


def add_rmsnorm(x, weight, eps, y, *, residual=None, h=None, rstd=None, yq=None, yq_scale=None,
                q_group=128, stream=None):
    """y = rmsnorm(x + residual) * weight, h = x + residual; yq / yq_scale: y as e4m3 codes with
    a scale per 128 columns (q_group 128) or per row (q_group 0)."""
    _check(binding().add_rmsnorm(x, weight, eps, y, residual, h, rstd, yq, yq_scale, q_group, stream),
           "moe_add_rmsnorm")


def add_rmsnorm_backward_scratch_bytes(T: int, H: int) -> int:
    n = _S()
    _check(_lib().moe_add_rmsnorm_backward_scratch_bytes(T, H, ctypes.byref(n)),
           "moe_add_rmsnorm_backward_scratch_bytes")
    return n.value


def add_rmsnorm_backward(dy, h, rstd, weight, dx, dweight, scratch, *, dh=None, stream=None):
    """dx (of x and the residual alike) and dweight [H] fp32; scratch: uint8."""
    _check(binding().add_rmsnorm_backward(dy, h, rstd, weight, dx, dweight, scratch, dh, stream),
           "moe_add_rmsnorm_backward")


def balance_loss_scratch_bytes(T: int, E: int, n_seq: int = 1) -> int:
    n = _S()
    _check(_lib().moe_balance_loss_scratch_bytes(T, E, n_seq, ctypes.byref(n)),
           "moe_balance_loss_scratch_bytes")
    return n.value


def balance_loss(logits, ids, E, counts, mean_prob, valid, losses, scratch, *, n_seq=1,
                 mode=MODE_SOFTMAX, token_mask=None, dev_status=None, stream=None):
    """counts, mean_prob [n_seq, E], valid [n_seq + 2] and losses [2] (load balance, router z) of
    a routed batch; scratch: uint8, zero before its first use; see the header."""
    _check(binding().balance_loss(logits, ids, E, counts, mean_prob, valid, losses, scratch, n_seq,
                                mode, token_mask, dev_status, stream), "moe_balance_loss")


def route_backward(logits, ids, E, dlogits, *, mode=MODE_SOFTMAX, scale=1.0, weights=None,
                   d_weights=None, d_shared_gate=None, token_mask=None, n_seq=1, counts=None,
                   valid=None, grad_losses=None, dev_status=None, stream=None):
    """dlogits from the gradients of the routing weights, the shared gate and balance_loss's two
    losses; see the header."""
    _check(binding().route_backward(logits, ids, E, dlogits, mode, scale, weights, d_weights,
                                  d_shared_gate, token_mask, n_seq, counts, valid, grad_losses,
                                  dev_status, stream), "moe_route_backward")


def unpermute_backward(dout, flat_to_row, weights, T, K, H, *, y=None, dy=None, d_weights=None,
                       shared_y=None, shared_gate=None, d_shared_y=None, d_shared_gate=None,
                       stream=None):
    """Gradients of unpermute: dy, d_weights, d_shared_y, d_shared_gate, each where given."""
    _check(binding().unpermute_backward(dout, flat_to_row, weights, T, K, H, y, dy, d_weights,
                                      shared_y, shared_gate, d_shared_y, d_shared_gate, stream),
           "moe_unpermute_backward")


def _check_tensors(*specs):
    """Number of values (None: any), types, contiguity and place of (tensor, types, values, name)
    each, as the C module checks them; None as a tensor is left to the library."""
    specs = [s for s in specs if s[0] is not None]
    for t, _, n, name in specs:
        if n is not None and t.numel() != n:
            raise ValueError(f"{name}: {n} values expected, got shape {tuple(t.shape)}")
    for t, types, _, name in specs:
        if t.dtype not in types:
            raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(map(str, types))}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous tensor expected, got strides {t.stride()}")
    for t, _, _, name in specs:
        if not t.is_cuda:
            raise ValueError(f"{name}: a tensor on the GPU expected")


def layer(cfg: Config, x, weights: Weights, out, workspace, dev_status=None, stream=None, T=None):
    T = x.shape[0] if T is None else T
    _check(_lib().moe_layer(ctypes.byref(cfg), T, _p(x), ctypes.byref(weights), _p(out),
                            _p(workspace), workspace.numel(), _p(dev_status), _stream(stream)),
           "moe_layer")


def layer_q8(cfg: Config, x, xq, xq_scale, weights: Weights, out, workspace, dev_status=None,
             stream=None):
    """moe_layer on activations that are e4m3 codes already (W8A8 experts; see the header)."""
    T = x.shape[0]
    bf16, f32 = (torch.bfloat16,), (torch.float32,)
    _check_tensors((x, bf16, T * cfg.H, "x"),
                   (xq, (torch.float8_e4m3fn, torch.uint8), T * cfg.H, "xq"),
                   (xq_scale, f32, T * -(-cfg.H // 128), "xq_scale"), (out, bf16, T * cfg.H, "out"),
                   (workspace, (torch.uint8,), None, "workspace"),
                   (dev_status, (torch.int32,), 1, "dev_status"))
    _check(_lib().moe_layer_q8(ctypes.byref(cfg), T, _p(x), _p(xq), _p(xq_scale),
                               ctypes.byref(weights), _p(out), _p(workspace), workspace.numel(),
                               _p(dev_status), _stream(stream)), "moe_layer_q8")


class MoELayer:
    """Owns the config, the device workspace and the weight pointers of one
    layer and calls ``moe_layer``.  Tensors are kept referenced so their
    pointers stay valid.  The workspace serves one call at a time: calls on
    different streams have to be ordered by the caller.  An output that a call
    allocates belongs to the stream that the call runs on."""

    def __init__(self, cfg: Config, tensors: dict, device="cuda"):
        self.cfg = cfg
        self.tensors = tensors
        g = tensors.get
        self.weights = Weights(*[_p(g(k)) for k in ("wg", "gate_bias", "sel_bias", "w1", "w3",
                                                     "w2", "s1", "s3", "s2", "sw1", "sw3", "sw2")])
        self.workspace = torch.empty(workspace_bytes(cfg), dtype=torch.uint8, device=device)
        self.layout = workspace_layout(cfg)
        # the sync region (up to the logits) starts at zero; see moe_layer
        self.workspace[self.layout.sync:self.layout.logits].zero_()
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=device)

    def __call__(self, x, out=None, stream=None):
        if out is None:
            out = _empty_like(x, stream)
        layer(self.cfg, x, self.weights, out, self.workspace, self.dev_status, stream)
        return out

    def view(self, name, dtype, shape):
        """A typed view of one intermediate inside the workspace."""
        off = getattr(self.layout, name)
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.workspace[off:off + nbytes].view(dtype).view(*shape)


class MoEBlock:
    """A pre-norm block: h = x + residual, y = rmsnorm(h) * weight, out = MoELayer(y).

    With W8A8 experts the norm also writes y's e4m3 codes and the layer reads those.  Calls with
    up to cfg.T_max tokens; returns (out, h), of which h is the residual stream's next value.
    As with MoELayer, the block's buffers serve one call at a time, and what a call allocates
    belongs to the stream that it runs on."""

    def __init__(self, cfg: Config, tensors: dict, norm_weight, eps=1e-6, device="cuda"):
        self.layer = MoELayer(cfg, tensors, device)
        self.norm_weight, self.eps = norm_weight, eps
        T, H = cfg.T_max, cfg.H
        self.y = torch.empty(T, H, dtype=torch.bfloat16, device=device)
        self.q8 = cfg.wdtype == W8A8_FP8
        if self.q8:
            self.yq = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=device)
            self.yq_scale = torch.empty(T, -(-H // 128), dtype=torch.float32, device=device)

    def __call__(self, x, residual=None, out=None, stream=None):
        T = x.shape[0]
        _check_tensors((out, (torch.bfloat16,), T * self.layer.cfg.H, "out"))
        h = _empty_like(x, stream) if residual is not None else None
        out = _empty_like(x, stream) if out is None else out
        y, L = self.y[:T], self.layer
        if self.q8:
            yq, ys = self.yq[:T], self.yq_scale[:T]
            add_rmsnorm(x, self.norm_weight, self.eps, y, residual=residual, h=h, yq=yq,
                        yq_scale=ys, stream=stream)
            layer_q8(L.cfg, y, yq, ys, L.weights, out, L.workspace, L.dev_status, stream)
        else:
            add_rmsnorm(x, self.norm_weight, self.eps, y, residual=residual, h=h, stream=stream)
            layer(L.cfg, y, L.weights, out, L.workspace, L.dev_status, stream)
        return out, (x if h is None else h)


def bounded_wait_check(counter, target, limit_us, dev_status, stream=None):
    _check(_lib().moe_bounded_wait_check(_p(counter), target, limit_us, _p(dev_status),
                                         _stream(stream)), "moe_bounded_wait_check")
