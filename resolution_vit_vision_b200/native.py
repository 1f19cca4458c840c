"""ctypes binding of ``libvit_b200.so`` (the C ABI in ``include/vit.h``, ``include/vit_ops.h`` and
``include/vit_decoder.h``).

Argument marshalling only: torch supplies device memory and streams; every step of the encoder
runs in the library's CUDA kernels. There is no fallback: if the library is missing or the
device is not an sm_100 GPU, the calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Dict, Optional, Sequence

import numpy as np
import torch

from . import synthetic as syn

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvit_b200.so")

VIT_OK, VIT_ERR_ARG, VIT_ERR_GRID, VIT_ERR_ALIGN, VIT_ERR_NOMEM, VIT_ERR_CUDA, VIT_ERR_TOKENS, \
    VIT_ERR_TIMEOUT, VIT_ERR_UNSUPPORTED, VIT_ERR_LIMIT = range(10)
EPI_STORE_F32, EPI_ADD_F32, EPI_STORE_BF16, EPI_GELU_BF16, EPI_QKV_ROPE = range(5)

c_void_p, c_int, c_int64, c_float = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
c_i32p = ctypes.POINTER(ctypes.c_int32)


class VitLayerW(ctypes.Structure):
    _fields_ = [(k, c_void_p) for k in syn.LAYER_KEYS]


FP8_LINEARS = ("qkv", "proj", "fc1", "fc2")


class VitLayerFp8(ctypes.Structure):
    _fields_ = [(f"{k}_{x}", c_void_p) for k in FP8_LINEARS for x in ("q", "s")]


class VitWeightsDesc(ctypes.Structure):
    _fields_ = [("depth", c_int), ("out_dim", c_int), ("ln_eps", c_float), ("patch_order", c_int),
                ("pe_w", c_void_p), ("pe_b", c_void_p), ("layers", ctypes.POINTER(VitLayerW)),
                ("lnq_w", c_void_p), ("lnq_b", c_void_p), ("m0_w", c_void_p), ("m0_b", c_void_p),
                ("m2_w", c_void_p), ("m2_b", c_void_p), ("window", c_int),
                ("full_attention", ctypes.POINTER(ctypes.c_uint8)),
                ("fp8_layers", ctypes.POINTER(VitLayerFp8))]



class PrefixAttentionDesc(ctypes.Structure):
    _fields_ = [("dtype", c_int), ("n_heads", c_int), ("n_kv_heads", c_int), ("head_dim", c_int), ("scale", c_float),
                ("causal", c_int), ("q", c_void_p), ("q_stride", c_int64), ("out", c_void_p), ("out_stride", c_int64),
                ("lse", c_void_p), ("total_q", c_int64), ("max_q", c_int64), ("cu_q", c_void_p), ("n_seq", c_int),
                ("prefix_k", c_void_p), ("prefix_v", c_void_p), ("prefix_len", c_int64),
                ("prefix_k_token", c_int64), ("prefix_k_head", c_int64), ("prefix_v_token", c_int64),
                ("prefix_v_head", c_int64), ("k", c_void_p), ("v", c_void_p), ("k_seq", c_int64), ("k_token", c_int64),
                ("k_head", c_int64), ("v_seq", c_int64), ("v_token", c_int64), ("v_head", c_int64),
                ("lens", c_void_p), ("max_len", c_int64)]


# The Qwen2.5-VL tower's full-attention blocks (0-based) when windows are on
QWEN25_FULL_BLOCKS = (7, 15, 23, 31)


_SIGS = {
    "vit_status_string": (ctypes.c_char_p, [c_int]),
    "vit_encode_sizes": (c_int, [c_i32p, c_int, ctypes.POINTER(c_int64), ctypes.POINTER(c_int64)]),
    "vit_weights_create": (c_int, [ctypes.POINTER(VitWeightsDesc), ctypes.POINTER(c_void_p)]),
    "vit_weights_destroy": (None, [c_void_p]),
    "vit_reserve": (c_int, [c_void_p, c_int64]),
    "vit_encode": (c_int, [c_void_p, c_i32p, c_int, c_void_p, c_void_p, c_void_p]),
    "vit_encode_host": (c_int, [c_void_p, c_i32p, c_int, c_void_p, c_void_p, c_void_p]),
    "vit_encode_noalloc": (c_int, [c_void_p, c_i32p, c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "mrope_index": (c_int, [c_void_p, c_int64, c_i32p, c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "vit_device_status": (c_int, [c_void_p, c_void_p, c_i32p]),
    "vit_launch_count": (c_int64, [c_void_p]),
    "vit_graph_enable": (c_int, [c_void_p, c_int]),
    "vit_profile_enable": (c_int, [c_void_p, c_int]),
    "vit_profile_read": (c_int, [c_void_p, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(c_int64), c_int]),
    "vit_profile_name": (ctypes.c_char_p, [c_int]),
    "vit_op_gemm": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int, c_int, c_int, c_void_p,
                            c_void_p, c_void_p, c_void_p]),
    "vit_op_rope_table": (c_int, [c_void_p, c_int, c_void_p]),
    "vit_op_positions": (c_int, [c_i32p, c_int, c_int, c_void_p, c_void_p, c_void_p]),
    "vit_op_layernorm": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_float, c_void_p, c_void_p]),
    "vit_op_attention": (c_int, [c_void_p, c_int64, c_i32p, c_int, c_void_p, c_void_p, c_void_p]),
    "vit_op_wait_selftest": (c_int, [c_void_p, c_int64, c_void_p]),
    "vit_op_exp2_fma": (c_int, [c_void_p, c_void_p, c_int64, c_void_p]),
    "vit_quantize_fp8": (c_int, [c_void_p, c_int64, c_int, c_void_p, c_void_p, c_void_p]),
    "vit_op_gemm_fp8": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int, c_int,
                                c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "vit_op_layernorm_fp8": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_float,
                                     c_void_p]),
    "mrope_apply": (c_int, [c_void_p, c_int, c_void_p, c_int, c_int, c_void_p, c_int64, ctypes.c_double, c_i32p,
                            c_void_p]),
    "scatter_vision_tokens": (c_int, [c_void_p, c_int64, c_void_p, c_int64, c_int, c_void_p, c_int64, c_void_p,
                                      c_void_p, c_void_p]),
    "mrope_norm_apply": (c_int, [c_void_p, c_int64, c_void_p, c_int64, c_int, c_void_p, c_int64, c_void_p, c_int64,
                                 c_int, c_int, c_int, c_void_p, c_void_p, c_float, c_void_p, c_int64, ctypes.c_double,
                                 c_i32p, c_void_p]),
    "mrope_norm_grad_workspace": (c_int64, [c_int]),
    "mrope_norm_grad": (c_int, [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int, c_void_p, c_int64,
                                c_void_p, c_int64, c_void_p, c_int64, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_float, c_void_p, c_int64, ctypes.c_double, c_i32p, c_void_p, c_int64,
                                c_void_p]),
    "embed_vision_tokens": (c_int, [c_void_p, c_int64, c_void_p, c_int, c_int64, c_int, c_float, c_void_p, c_int64,
                                    c_void_p, c_void_p, c_void_p]),
    "embed_vision_tokens_grad_workspace": (c_int64, [c_int64, c_int64, c_int]),
    "embed_vision_tokens_grad": (c_int, [c_void_p, c_int64, c_void_p, c_int, c_int64, c_int, c_float, c_void_p, c_int,
                                         c_int, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p]),
    "prefix_attention_workspace": (c_int64, [ctypes.POINTER(PrefixAttentionDesc)]),
    "prefix_attention": (c_int, [ctypes.POINTER(PrefixAttentionDesc), c_void_p, c_int64, c_void_p, c_void_p]),
    "vit_op_window_positions": (c_int, [c_i32p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                        ctypes.POINTER(c_int), c_void_p]),
    "vit_op_gather_rows": (c_int, [c_void_p, c_void_p, c_void_p, c_int64, c_int, c_void_p]),
    "vit_op_window_attention": (c_int, [c_void_p, c_int64, c_void_p, c_int, c_void_p, c_void_p, c_void_p]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Loads the library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m resolution_vit_vision_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


class VitError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {lib().vit_status_string(code).decode()} (status {code})")


def check(rc: int, what: str) -> None:
    if rc != VIT_OK:
        raise VitError(rc, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _grid_arg(grid_thw) -> np.ndarray:
    g = np.ascontiguousarray(np.asarray(grid_thw, dtype=np.int32).reshape(-1, 3))
    return g


def _gp(g: np.ndarray):
    return g.ctypes.data_as(c_i32p)


def encode_sizes(grid_thw):
    g = _grid_arg(grid_thw)
    P, M = c_int64(), c_int64()
    check(lib().vit_encode_sizes(_gp(g), g.shape[0], ctypes.byref(P), ctypes.byref(M)), "vit_encode_sizes")
    return P.value, M.value


# ------------------------------------------------------------------------------------------------
def weights_to_device(w_np: Dict, device="cuda") -> Dict:
    """bf16-bit numpy weights (synthetic.make_weights) -> dict of bf16 CUDA tensors."""
    def t(a):
        if a is None:
            return None
        return torch.from_numpy(np.ascontiguousarray(a)).view(torch.bfloat16).to(device)
    out = {k: t(v) for k, v in w_np.items() if k != "layers"}
    out["layers"] = [{k: t(v) for k, v in L.items()} for L in w_np["layers"]]
    return out


def random_weights_device(depth: int, out_dim: int, seed: int, device="cuda", std: float = 0.02) -> Dict:
    """Same shapes and distribution as synthetic.make_weights (N(0, 0.02) matrices, zero biases,
    unit gamma), drawn on the device with a seeded torch generator (fast, for benchmarking)."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def mat(shape):
        return (torch.randn(shape, generator=g, device=device, dtype=torch.float32) * std).to(torch.bfloat16)

    def zeros(n):
        return torch.zeros(n, device=device, dtype=torch.bfloat16)

    def ones(n):
        return torch.ones(n, device=device, dtype=torch.bfloat16)

    w = {"pe_w": mat((syn.WIDTH, syn.PATCH_K)), "pe_b": None}
    layers = []
    for _ in range(depth):
        L = {}
        for k in syn.LAYER_KEYS:
            shape = syn.LAYER_SHAPES[k]
            L[k] = ones(shape[0]) if k in ("ln1_w", "ln2_w") else (zeros(shape[0]) if len(shape) == 1 else mat(shape))
        layers.append(L)
    w["layers"] = layers
    w["lnq_w"], w["lnq_b"] = ones(syn.WIDTH), zeros(syn.WIDTH)
    w["m0_w"], w["m0_b"] = mat((syn.MERGE_K, syn.MERGE_K)), zeros(syn.MERGE_K)
    w["m2_w"], w["m2_b"] = mat((out_dim, syn.MERGE_K)), zeros(out_dim)
    return w


def quantize_fp8(x: torch.Tensor, stream=None):
    """E4M3 codes (uint8, same shape) and per-row power-of-two scales (fp32 [rows]) of a bf16
    [rows, cols] device tensor, by vit_quantize_fp8."""
    assert x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous() and x.dim() == 2
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty((x.shape[0],), dtype=torch.float32, device=x.device)
    check(lib().vit_quantize_fp8(_ptr(x), x.shape[0], x.shape[1], _ptr(codes), _ptr(scales), _stream(stream)),
          "vit_quantize_fp8")
    return codes, scales


def fp8_layers_device(weights: Dict, stream=None):
    """Per layer {"qkv": (codes, scales), "proj": ..., "fc1": ..., "fc2": ...} of the device bf16
    weights' four block linears, quantised on the device."""
    return [{k: quantize_fp8(L[f"{k}_w"], stream) for k in FP8_LINEARS} for L in weights["layers"]]


class VisionEncoder:
    """A validated weight view (vit_handle) and its workspace; ``encode`` runs vit_encode.
    window > 0 makes the windowed (Qwen2.5-VL) tower: blocks in ``full_blocks`` attend over the
    whole frame, the others inside window x window patches. fp8: per layer the E4M3 codes and
    scales of the four block linears (``fp8_layers_device``): the fp8 tower."""

    def __init__(self, weights: Dict, out_dim: int, eps: float = 1e-6, patch_order: int = 0, window: int = 0,
                 full_blocks: Sequence[int] = (), fp8=None):
        self.weights = weights          # keeps the device tensors alive
        self.out_dim = out_dim
        depth = len(weights["layers"])
        self._layers = (VitLayerW * depth)()
        for i, L in enumerate(weights["layers"]):
            for k in syn.LAYER_KEYS:
                setattr(self._layers[i], k, _ptr(L.get(k)))
        d = VitWeightsDesc()
        d.depth, d.out_dim, d.ln_eps, d.patch_order = depth, out_dim, eps, patch_order
        d.pe_w, d.pe_b = _ptr(weights["pe_w"]), _ptr(weights.get("pe_b"))
        d.layers = self._layers
        for k in ("lnq_w", "lnq_b", "m0_w", "m0_b", "m2_w", "m2_b"):
            setattr(d, k, _ptr(weights.get(k)))
        d.window = int(window)
        self._full = (ctypes.c_uint8 * depth)(*[1 if l in set(full_blocks) else 0 for l in range(depth)])
        d.full_attention = ctypes.cast(self._full, ctypes.POINTER(ctypes.c_uint8))
        self._fp8 = fp8                 # keeps the codes and scales alive
        if fp8 is not None:
            self._fp8_layers = (VitLayerFp8 * depth)()
            for i, Lq in enumerate(fp8):
                for k in FP8_LINEARS:
                    setattr(self._fp8_layers[i], f"{k}_q", _ptr(Lq[k][0]))
                    setattr(self._fp8_layers[i], f"{k}_s", _ptr(Lq[k][1]))
            d.fp8_layers = self._fp8_layers
        self._desc = d
        h = c_void_p()
        check(lib().vit_weights_create(ctypes.byref(d), ctypes.byref(h)), "vit_weights_create")
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().vit_weights_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def reserve(self, max_patches: int):
        check(lib().vit_reserve(self._h, int(max_patches)), "vit_reserve")

    def encode(self, patches: torch.Tensor, grid_thw, out: Optional[torch.Tensor] = None, stream=None):
        g = _grid_arg(grid_thw)
        P, M = encode_sizes(g)
        assert patches.dtype == torch.bfloat16 and patches.is_cuda and patches.is_contiguous()
        assert patches.shape == (P, syn.PATCH_K), (patches.shape, P)
        if out is None:
            out = torch.empty((M, self.out_dim), dtype=torch.bfloat16, device=patches.device)
        check(lib().vit_encode(_ptr(patches), _gp(g), g.shape[0], self._h, _ptr(out), _stream(stream)), "vit_encode")
        return out

    def encode_host(self, patches_host: torch.Tensor, grid_thw, out_host: torch.Tensor, stream=None):
        g = _grid_arg(grid_thw)
        check(lib().vit_encode_host(_ptr(patches_host), _gp(g), g.shape[0], self._h, _ptr(out_host),
                                    _stream(stream)), "vit_encode_host")
        return out_host

    def device_status(self, stream=None) -> int:
        v = ctypes.c_int32()
        check(lib().vit_device_status(self._h, _stream(stream), ctypes.byref(v)), "vit_device_status")
        return v.value

    def graph_enable(self, on: bool = True):
        check(lib().vit_graph_enable(self._h, 1 if on else 0), "vit_graph_enable")

    def launch_count(self) -> int:
        return int(lib().vit_launch_count(self._h))

    def profile_enable(self, on: bool = True):
        check(lib().vit_profile_enable(self._h, 1 if on else 0), "vit_profile_enable")

    def profile_read(self) -> Dict[str, Dict[str, float]]:
        n = 16
        ms = (ctypes.c_double * n)()
        cnt = (c_int64 * n)()
        k = lib().vit_profile_read(self._h, ms, cnt, n)
        return {lib().vit_profile_name(i).decode(): {"ms": ms[i], "launches": cnt[i]} for i in range(k)}


def mrope_index(input_ids: torch.Tensor, grid_thw, out=None, delta=None, status=None, stream=None):
    """3-D M-RoPE ids [3, L] int32 and delta [1] int32 (device tensors)."""
    assert input_ids.dtype == torch.int32 and input_ids.is_cuda
    g = _grid_arg(grid_thw) if grid_thw is not None else np.zeros((0, 3), np.int32)
    L = input_ids.numel()
    if out is None:
        out = torch.empty((3, L), dtype=torch.int32, device=input_ids.device)
    if delta is None:
        delta = torch.empty((1,), dtype=torch.int32, device=input_ids.device)
    check(lib().mrope_index(_ptr(input_ids), L, _gp(g), g.shape[0], _ptr(out), _ptr(delta), _ptr(status),
                            _stream(stream)), "mrope_index")
    return out, delta


# ------------------------------------------------------------------------------------------------
# kernel-level ops (include/vit_ops.h)
def op_gemm(A, B, bias, C, epilogue, pos=None, rope_cs=None, status=None, stream=None):
    M, K = A.shape
    N = B.shape[0]
    check(lib().vit_op_gemm(_ptr(A), _ptr(B), _ptr(bias), _ptr(C), M, N, K, epilogue, _ptr(pos), _ptr(rope_cs),
                            _ptr(status), _stream(stream)), "vit_op_gemm")
    return C


def op_rope_table(n_pos: int, device="cuda", stream=None):
    cs = torch.empty((n_pos, 20, 2), dtype=torch.float32, device=device)
    check(lib().vit_op_rope_table(_ptr(cs), n_pos, _stream(stream)), "vit_op_rope_table")
    return cs


def op_positions(grid_thw, patch_order: int, device="cuda", stream=None):
    g = _grid_arg(grid_thw)
    P, _ = encode_sizes(g)
    pos = torch.empty(P, dtype=torch.int32, device=device)
    mr = torch.empty(P, dtype=torch.int32, device=device)
    check(lib().vit_op_positions(_gp(g), g.shape[0], patch_order, _ptr(pos), _ptr(mr), _stream(stream)),
          "vit_op_positions")
    return pos, mr


def op_layernorm(X, gamma, beta, Y, eps=1e-6, out_row=None, stream=None):
    check(lib().vit_op_layernorm(_ptr(X), _ptr(gamma), _ptr(beta), _ptr(Y), X.shape[0], eps, _ptr(out_row),
                                 _stream(stream)), "vit_op_layernorm")
    return Y


def op_attention(qkv, cu_seqlens: Sequence[int], out, status=None, stream=None):
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    check(lib().vit_op_attention(_ptr(qkv), qkv.shape[0], cu.ctypes.data_as(c_i32p), cu.shape[0] - 1, _ptr(out),
                                 _ptr(status), _stream(stream)), "vit_op_attention")
    return out


def op_gemm_fp8(A, a_scale, B, b_scale, bias, C, epilogue, pos=None, rope_cs=None, status=None, stream=None):
    M, K = A.shape
    N = B.shape[0]
    check(lib().vit_op_gemm_fp8(_ptr(A), _ptr(a_scale), _ptr(B), _ptr(b_scale), _ptr(bias), _ptr(C), M, N, K,
                                epilogue, _ptr(pos), _ptr(rope_cs), _ptr(status), _stream(stream)), "vit_op_gemm_fp8")
    return C


def op_layernorm_fp8(X, gamma, beta, eps=1e-6, stream=None):
    rows = X.shape[0]
    codes = torch.empty((rows, syn.WIDTH), dtype=torch.uint8, device=X.device)
    scales = torch.empty((rows,), dtype=torch.float32, device=X.device)
    check(lib().vit_op_layernorm_fp8(_ptr(X), _ptr(gamma), _ptr(beta), _ptr(codes), _ptr(scales), rows, eps,
                                     _stream(stream)), "vit_op_layernorm_fp8")
    return codes, scales


def op_exp2_fma(x: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The attention softmax's FMA-pipe exponential 2^x, elementwise on fp32 device tensors."""
    assert x.dtype == torch.float32 and x.is_cuda and x.is_contiguous()
    y = torch.empty_like(x) if y is None else y
    check(lib().vit_op_exp2_fma(_ptr(x), _ptr(y), x.numel(), _stream(stream)), "vit_op_exp2_fma")
    return y


def op_window_positions(grid_thw, patch_order: int, window: int, device="cuda", stream=None):
    """(pos, merge_row, src_row) of the window-order rows, int32 [P] each, and the window table
    int32 [n_windows, 2] = (first row, rows)."""
    g = _grid_arg(grid_thw)
    P, _ = encode_sizes(g)
    pos, mr, src = (torch.empty(P, dtype=torch.int32, device=device) for _ in range(3))
    tab = torch.empty((P // 4 + 1, 2), dtype=torch.int32, device=device)
    n = c_int(0)
    check(lib().vit_op_window_positions(_gp(g), g.shape[0], patch_order, window, _ptr(pos), _ptr(mr), _ptr(src),
                                        _ptr(tab), ctypes.byref(n), _stream(stream)), "vit_op_window_positions")
    return pos, mr, src, tab[:n.value]


def op_gather_rows(src, src_row, dst, stream=None):
    row_bytes = src.shape[1] * src.element_size()
    check(lib().vit_op_gather_rows(_ptr(src), _ptr(src_row), _ptr(dst), dst.shape[0], row_bytes, _stream(stream)),
          "vit_op_gather_rows")
    return dst


def op_window_attention(qkv, win_table, out, status=None, stream=None):
    """win_table: int32 [n_windows, 2] device (first row, rows), as op_window_positions returns."""
    check(lib().vit_op_window_attention(_ptr(qkv), qkv.shape[0], _ptr(win_table), win_table.shape[0], _ptr(out),
                                        _ptr(status), _stream(stream)), "vit_op_window_attention")
    return out


MROPE_THETA = 1.0e6
MROPE_SECTIONS = (16, 24, 24)


def mrope_apply(q, k, pos, theta: float = MROPE_THETA, sections=MROPE_SECTIONS, stream=None):
    """3-D M-RoPE in place on q [L, heads, head_dim] and k [L, kv_heads, head_dim] (bf16, either may
    be None); pos int32 [3, L] from mrope_index."""
    x = q if q is not None else k
    L, D = x.shape[0], x.shape[2]
    sec = np.ascontiguousarray(np.asarray(sections, dtype=np.int32))
    check(lib().mrope_apply(_ptr(q), 0 if q is None else q.shape[1], _ptr(k), 0 if k is None else k.shape[1], D,
                            _ptr(pos), L, float(theta), sec.ctypes.data_as(c_i32p), _stream(stream)), "mrope_apply")
    return q, k


def scatter_vision_tokens(input_ids, embed_table, vision, out=None, status=None, stream=None):
    """The decoder's input rows: vision tokens at the image / video placeholders, embeddings elsewhere."""
    L, (V, D) = input_ids.shape[0], embed_table.shape
    if out is None:
        out = torch.empty((L, D), dtype=embed_table.dtype, device=embed_table.device)
    n_vis = 0 if vision is None else vision.shape[0]
    check(lib().scatter_vision_tokens(_ptr(input_ids), L, _ptr(embed_table), V, D, _ptr(vision), n_vis, _ptr(out),
                                      _ptr(status), _stream(stream)), "scatter_vision_tokens")
    return out


# ------------------------------------------------------------------------------------------------
# decoder-side steps with their gradients, and attention over a shared prefix (include/vit_decoder.h).
# Decoding calls them once per layer and token with kernels of a few microseconds, so the marshalling
# below reads each tensor property once and allocates with new_empty / empty_like.
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_HERE_AND_NOW = contextlib.nullcontext()


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _device_of(*tensors) -> int:
    """The index of the GPU that holds all the tensors (None is skipped)."""
    dev = None
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != dev:
                _need(dev is None, "tensors are on different devices")
                _need(i >= 0, "tensors must be on a GPU")
                dev = i
    return dev


def _place(dev: int, stream):
    """The context a call on GPU ``dev`` runs in: that GPU current and, where a stream is given, that
    stream current, so that outputs and workspaces made inside belong to it."""
    if stream is not None:
        _need(stream.device.index == dev, "the stream belongs to another device than the tensors")
        return torch.cuda.stream(stream)
    return _HERE_AND_NOW if torch.cuda.current_device() == dev else torch.cuda.device(dev)


# the current stream's handle without making a torch.cuda.Stream of it (3 us), where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: _stream(None))


def _rows_arg(t, L: int, H: int, D: int, what: str) -> int:
    """Token stride of t [L, H, D], whose heads must be contiguous."""
    s0, s1, s2 = t.stride()
    if (s1 == D or H == 1) and (s2 == 1 or D == 1):
        return s0 if L > 1 else H * D
    raise ValueError(f"{what}: the heads of a token must be contiguous")


def _out_rows(x, out, L: int, H: int, D: int, what: str):
    """``out``, or a new contiguous tensor like x [L, H, D], and its token stride."""
    if out is None:
        return x.new_empty((L, H, D)), H * D
    _need(out.shape == x.shape and out.dtype == x.dtype and out.get_device() == x.get_device(),
          f"{what} must have its input's shape, type and device")
    return out, _rows_arg(out, L, H, D, what)


def _key_strides(t):
    """Strides of [..., tokens, heads, head_dim] in elements; those of dimensions of one element, which
    torch leaves arbitrary, become head_dim."""
    st = t.stride()
    return tuple(t.shape[-1] if n == 1 else s for n, s in zip(t.shape, st)) if 1 in t.shape else st


def _status_arg(status):
    if status is None:
        return None
    _need(status.dtype == torch.int32 and status.numel() >= 1, "status must be int32 [1]")
    return status.data_ptr()


@functools.lru_cache(maxsize=64)
def _sections_arg(sections):
    return (ctypes.c_int32 * 3)(*sections)


_NORM_OPERANDS = ("q and k must be [L, heads, head_dim] of the same tokens, head_dim and type (bf16, fp16 or fp32), pos "
                  "contiguous int32 [3, L], weights contiguous [head_dim] of the type of q and k")


def _norm_args(q, k, pos, q_weight, k_weight):
    """(L, H, Hk, D, dtype code) of the operands of the norm calls; H or Hk is 0 for a missing q or k."""
    x = k if q is None else q
    _need(x is not None, "q or k must be given")
    _need(x.dim() == 3, _NORM_OPERANDS)
    L, H, D = x.shape
    t = x.dtype
    Hk = 0
    if q is None:
        H, Hk = 0, H
    elif k is not None:
        _need(k.dim() == 3 and k.dtype == t, _NORM_OPERANDS)
        Lk, Hk, Dk = k.shape
        _need(Lk == L and Dk == D, _NORM_OPERANDS)
    if not (t in DTYPES and pos.dtype == torch.int32 and pos.shape == (3, L) and pos.is_contiguous()
            and (q_weight is None or (q_weight.dtype == t and q_weight.shape == (D,) and q_weight.is_contiguous()))
            and (k_weight is None or (k_weight.dtype == t and k_weight.shape == (D,) and k_weight.is_contiguous()))):
        raise ValueError(_NORM_OPERANDS)
    return L, H, Hk, D, DTYPES[t]


def mrope_norm_apply(q, k, pos, q_weight=None, k_weight=None, eps: float = 1e-6, theta: float = MROPE_THETA,
                     sections=MROPE_SECTIONS, q_out=None, k_out=None, stream=None):
    """Per-head RMS norm and 3-D M-RoPE of q [L, heads, head_dim] and k [L, kv_heads, head_dim] in one
    pass (either may be None; token strides are free, so slices of a packed QKV product work); weights
    [head_dim] or None (ones); pos int32 [3, L]. Returns (q_out, k_out): new tensors, or the given
    ones, which may be q and k themselves."""
    L, H, Hk, D, dt = _norm_args(q, k, pos, q_weight, k_weight)
    _need((q is not None or q_out is None) and (k is not None or k_out is None), "an output is given without its input")
    dev = _device_of(q, k, pos, q_weight, k_weight)
    qp = kp = qo = ko = None
    qs = ks = qos = kos = 0
    with _place(dev, stream):
        if q is not None:
            qp, qs = q.data_ptr(), _rows_arg(q, L, H, D, "q")
            q_out, qos = _out_rows(q, q_out, L, H, D, "q_out")
            qo = q_out.data_ptr()
        if k is not None:
            kp, ks = k.data_ptr(), _rows_arg(k, L, Hk, D, "k")
            k_out, kos = _out_rows(k, k_out, L, Hk, D, "k_out")
            ko = k_out.data_ptr()
        rc = lib().mrope_norm_apply(qp, qs, qo, qos, H, kp, ks, ko, kos, Hk, D, dt, _ptr(q_weight), _ptr(k_weight), eps,
                                    pos.data_ptr(), L, theta, _sections_arg(tuple(sections)), _raw_stream(dev))
    check(rc, "mrope_norm_apply")
    return q_out, k_out


def mrope_norm_grad(dq_out, dk_out, q, k, pos, q_weight=None, k_weight=None, eps: float = 1e-6,
                    theta: float = MROPE_THETA, sections=MROPE_SECTIONS, dq=None, dk=None, weight_grads: bool = True,
                    stream=None):
    """Gradient of ``mrope_norm_apply`` at the same q, k, weights and positions: (dq, dk, dq_weight,
    dk_weight), the weights' in fp32 (None with weight_grads False, or for a missing q or k)."""
    L, H, Hk, D, dt = _norm_args(q, k, pos, q_weight, k_weight)
    _need((dq_out is None) == (q is None) and (dk_out is None) == (k is None) and (q is not None or dq is None)
          and (k is not None or dk is None), "gradients go with q and k")
    dev = _device_of(q, k, pos, q_weight, k_weight, dq_out, dk_out)
    qp = kp = qo = ko = gq = gk = dwq = dwk = wq = wk = ws = None
    qs = ks = qos = kos = gqs = gks = ws_bytes = 0
    L_ = lib()
    with _place(dev, stream):
        if q is not None:
            _need(dq_out.shape == q.shape and dq_out.dtype == q.dtype, "dq_out must have q's shape and type")
            qp, qs = q.data_ptr(), _rows_arg(q, L, H, D, "q")
            gq, gqs = dq_out.data_ptr(), _rows_arg(dq_out, L, H, D, "dq_out")
            dq, qos = _out_rows(q, dq, L, H, D, "dq")
            qo = dq.data_ptr()
        if k is not None:
            _need(dk_out.shape == k.shape and dk_out.dtype == k.dtype, "dk_out must have k's shape and type")
            kp, ks = k.data_ptr(), _rows_arg(k, L, Hk, D, "k")
            gk, gks = dk_out.data_ptr(), _rows_arg(dk_out, L, Hk, D, "dk_out")
            dk, kos = _out_rows(k, dk, L, Hk, D, "dk")
            ko = dk.data_ptr()
        if weight_grads:
            ws_bytes = L_.mrope_norm_grad_workspace(D)
            space = pos.new_empty(ws_bytes // 4)
            ws = space.data_ptr()
            if q is not None:
                dwq = q.new_empty(D, dtype=torch.float32)
                wq = dwq.data_ptr()
            if k is not None:
                dwk = k.new_empty(D, dtype=torch.float32)
                wk = dwk.data_ptr()
        rc = L_.mrope_norm_grad(gq, gqs, qp, qs, qo, qos, H, gk, gks, kp, ks, ko, kos, Hk, D, dt, _ptr(q_weight),
                                _ptr(k_weight), wq, wk, eps, pos.data_ptr(), L, theta, _sections_arg(tuple(sections)), ws,
                                ws_bytes, _raw_stream(dev))
    check(rc, "mrope_norm_grad")
    return dq, dk, dwq, dwk


def _ids_arg(input_ids) -> int:
    _need(input_ids.dtype == torch.int32 and input_ids.dim() == 1 and input_ids.is_contiguous(),
          "input_ids must be contiguous int32 [L]")
    return input_ids.shape[0]


def embed_vision_tokens(input_ids, embed_table, vision=None, scale: float = 1.0, out=None, status=None, stream=None):
    """The decoder's input rows: scale * embedding for text ids, vision tokens (unscaled) at the image /
    video placeholders. bf16, fp16 or fp32, all of one type."""
    L = _ids_arg(input_ids)
    V, D = embed_table.shape
    dtype = embed_table.dtype
    dt = DTYPES.get(dtype)
    _need(dt is not None and embed_table.is_contiguous(), "embed_table must be contiguous bf16, fp16 or fp32")
    n_vis = 0
    if vision is not None:
        n_vis = vision.shape[0]
        _need(vision.dtype == dtype and vision.shape == (n_vis, D) and vision.is_contiguous(),
              "vision must be contiguous [n_vision, dim] of the table's type")
    dev = _device_of(embed_table, input_ids, vision, out, status)
    with _place(dev, stream):
        if out is None:
            out = embed_table.new_empty((L, D))
        else:
            _need(out.shape == (L, D) and out.dtype == dtype and out.is_contiguous(),
                  "out must be contiguous [L, dim] of the table's type")
        check(lib().embed_vision_tokens(input_ids.data_ptr(), L, embed_table.data_ptr(), dt, V, D, scale,
                                        vision.data_ptr() if n_vis else None, n_vis, out.data_ptr(),
                                        _status_arg(status), _raw_stream(dev)), "embed_vision_tokens")
    return out


def embed_vision_tokens_grad(input_ids, d_out, vocab: int, n_vision: int = 0, scale: float = 1.0, table_dtype=None,
                             d_table=None, accumulate: bool = False, d_vision=None, status=None, stream=None):
    """Gradient of ``embed_vision_tokens``: (d_table [vocab, dim], d_vision [n_vision, dim] or None). d_table
    is of table_dtype (d_out's type, or fp32); a given d_table is overwritten, or added to with
    accumulate (then only the rows that input_ids names are touched)."""
    L = _ids_arg(input_ids)
    dtype = d_out.dtype
    dt = DTYPES.get(dtype)
    _need(dt is not None and d_out.dim() == 2 and d_out.shape[0] == L and d_out.is_contiguous(),
          "d_out must be contiguous [L, dim] in bf16, fp16 or fp32")
    D = d_out.shape[1]
    _need(d_table is not None or not accumulate, "accumulate needs a d_table to add to")
    if table_dtype is None:
        table_dtype = dtype if d_table is None else d_table.dtype
    _need(table_dtype in (dtype, torch.float32), "the table's gradient is of d_out's type or fp32")
    dev = _device_of(d_out, input_ids, d_table, d_vision, status)
    with _place(dev, stream):
        if d_table is None:
            d_table = d_out.new_empty((vocab, D), dtype=table_dtype)
        _need(d_table.shape == (vocab, D) and d_table.dtype == table_dtype and d_table.is_contiguous(),
              "d_table must be contiguous [vocab, dim] of table_dtype")
        if d_vision is None and n_vision:
            d_vision = d_out.new_empty((n_vision, D))
        _need(d_vision is None or (d_vision.shape == (n_vision, D) and d_vision.dtype == dtype
                                   and d_vision.is_contiguous()),
              "d_vision must be contiguous [n_vision, dim] of d_out's type")
        L_ = lib()
        ws_bytes = L_.embed_vision_tokens_grad_workspace(L, vocab, D)
        ws = d_out.new_empty((ws_bytes,), dtype=torch.uint8)
        check(L_.embed_vision_tokens_grad(input_ids.data_ptr(), L, d_out.data_ptr(), dt, vocab, D, scale,
                                          d_table.data_ptr(), DTYPES[table_dtype], 1 if accumulate else 0,
                                          _ptr(d_vision), n_vision, ws.data_ptr(), ws_bytes, _status_arg(status),
                                          _raw_stream(dev)), "embed_vision_tokens_grad")
    return d_table, d_vision


def prefix_attention(q, prefix_k=None, prefix_v=None, k=None, v=None, lens=None, cu_q=None, max_q: Optional[int] = None,
                     max_len: Optional[int] = None, scale: Optional[float] = None, causal: bool = True, out=None,
                     lse=None, status=None, stream=None):
    """Attention of a batch of sequences over a prefix they share and over keys of their own.

    q [total_q, heads, head_dim]: the sequences' queries one after another, cu_q int32 [n_seq + 1]
    their first rows (None: max_q each); prefix_k, prefix_v [prefix_len, kv_heads, head_dim] or None;
    k, v [n_seq, capacity, kv_heads, head_dim] with lens int32 [n_seq] keys in use, or None; any strides
    with contiguous head_dim (head-major caches as permuted views). cu_q and lens are read on the device.
    max_q defaults to 1 without cu_q, else to total_q; max_len to the capacity. With ``causal`` query j
    of n sees its sequence's keys s <= lens - n + j. Returns (out, lse): out like q, lse fp32 [total_q, heads]."""
    _need(q.dim() == 3, "q must be bf16 or fp16 [total_q, heads, head_dim]")
    T, H, D = q.shape
    dtype = q.dtype
    dt = DTYPES.get(dtype, 2)
    _need(dt != 2, "q must be bf16 or fp16 [total_q, heads, head_dim]")
    _need((prefix_k is None) == (prefix_v is None) and (k is None) == (v is None), "keys and values go together")
    _need((k is None) == (lens is None), "own keys need their lengths")
    Lp, B, Hk = 0, None, None
    pk_token = pk_head = pv_token = pv_head = k_seq = k_token = k_head = v_seq = v_token = v_head = 0
    pk = pv = kp = vp = lp = None
    if prefix_k is not None:
        Lp, Hk, Dk = prefix_k.shape
        pk_token, pk_head, i0 = _key_strides(prefix_k)
        pv_token, pv_head, i1 = _key_strides(prefix_v)
        _need(Dk == D and prefix_v.shape == prefix_k.shape and prefix_k.dtype == dtype and prefix_v.dtype == dtype
              and ((i0 == 1 and i1 == 1) or D == 1),
              "prefix keys and values must be [prefix_len, kv_heads, head_dim] of q's type, head_dim contiguous")
        if Lp:
            pk, pv = prefix_k.data_ptr(), prefix_v.data_ptr()
    if k is not None:
        B, cap, h, Dk = k.shape
        k_seq, k_token, k_head, i0 = _key_strides(k)
        v_seq, v_token, v_head, i1 = _key_strides(v)
        _need(Dk == D and (Hk is None or Hk == h) and v.shape == k.shape and k.dtype == dtype and v.dtype == dtype
              and ((i0 == 1 and i1 == 1) or D == 1),
              "own keys and values must be [n_seq, capacity, kv_heads, head_dim] of q's type, head_dim contiguous")
        Hk = h
        _need(lens.dtype == torch.int32 and lens.shape == (B,) and lens.is_contiguous(), "lens must be int32 [n_seq]")
        max_len = cap if max_len is None else max_len
        _need(0 <= max_len <= cap, "max_len must be within the capacity")
        if cap:
            kp, vp, lp = k.data_ptr(), v.data_ptr(), lens.data_ptr()
    _need(Hk is not None, "a prefix or own keys must be given")
    if cu_q is not None:
        _need(cu_q.dtype == torch.int32 and cu_q.dim() == 1 and cu_q.shape[0] >= 2 and cu_q.is_contiguous(),
              "cu_q must be int32 [n_seq + 1]")
        n_seq = cu_q.shape[0] - 1
        max_q = max(T, 1) if max_q is None else max_q
    else:
        max_q = 1 if max_q is None else max_q
        n_seq = B if B is not None else T // max(max_q, 1)
        _need(n_seq * max_q == T or T == 0, "without cu_q there must be max_q queries for each sequence")
    _need(B is None or B == n_seq, "k and cu_q disagree on the number of sequences")
    dev = _device_of(q, prefix_k, prefix_v, k, v, lens, cu_q, out, lse, status)
    with _place(dev, stream):
        if out is None:
            out = q.new_empty((T, H, D))
        else:
            _need(out.shape == q.shape and out.dtype == dtype, "out must have q's shape and type")
        if lse is None:
            lse = q.new_empty((T, H), dtype=torch.float32)
        else:
            _need(lse.shape == (T, H) and lse.dtype == torch.float32 and lse.is_contiguous(),
                  "lse must be fp32 [total_q, heads]")
        if T == 0:
            return out, lse
        d = PrefixAttentionDesc(dt, H, Hk, D, D ** -0.5 if scale is None else scale, 1 if causal else 0, q.data_ptr(),
                                _rows_arg(q, T, H, D, "q"), out.data_ptr(), _rows_arg(out, T, H, D, "out"), lse.data_ptr(),
                                T, max_q, _ptr(cu_q), n_seq, pk, pv, Lp, pk_token, pk_head, pv_token, pv_head, kp, vp,
                                k_seq, k_token, k_head, v_seq, v_token, v_head, lp, max_len if kp is not None else 0)
        L = lib()
        ref = ctypes.byref(d)
        ws_bytes = L.prefix_attention_workspace(ref)
        ws = q.new_empty(ws_bytes // 2) if ws_bytes else None
        rc = L.prefix_attention(ref, _ptr(ws), ws_bytes, _status_arg(status), _raw_stream(dev))
    check(rc, "prefix_attention")
    return out, lse


def op_wait_selftest(status, limit_cycles: int, stream=None):
    check(lib().vit_op_wait_selftest(_ptr(status), int(limit_cycles), _stream(stream)), "vit_op_wait_selftest")
