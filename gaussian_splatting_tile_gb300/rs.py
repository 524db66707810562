"""Thin Python binding of the C ABI in include/rs.h (librs.so), with the same names.

Argument marshalling only: torch tensors are checked (device, dtype, contiguity, shape) and
their device pointers and the current CUDA stream are handed to the library; every step of the
rasteriser runs in the library's kernels.  There is no fallback: if librs.so is missing or the
GPU is unavailable, the calls raise.
"""
from __future__ import annotations

import ctypes
import glob
import dataclasses
import os
import re
import struct

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librs.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "rs.h")

RS_OK, RS_ERR_INVALID_ARG, RS_ERR_CAPACITY, RS_ERR_WORKSPACE, RS_ERR_CUDA = 0, -1, -2, -3, -4
RS_ERR_DEVICE_TIMEOUT, RS_ERR_DEVICE_CHECK = -5, -6
RS_TILE, RS_RECORD_BYTES, RS_MAX_GAUSSIANS, RS_MAX_ENTRIES = 16, 48, 1 << 26, (1 << 30) - 1
RECORD_BYTES = 48
TILE = 16


class RsError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with {code}: {msg}")
        self.code = code


class rs_camera(ctypes.Structure):
    _fields_ = [("R", ctypes.c_float * 9), ("t", ctypes.c_float * 3),
                ("fx", ctypes.c_float), ("fy", ctypes.c_float),
                ("cx", ctypes.c_float), ("cy", ctypes.c_float),
                ("width", ctypes.c_int32), ("height", ctypes.c_int32)]


class rs_gaussians(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("d_means", ctypes.c_void_p), ("d_scales", ctypes.c_void_p),
                ("d_quats", ctypes.c_void_p), ("d_opacity", ctypes.c_void_p),
                ("d_sh", ctypes.c_void_p), ("sh_degree", ctypes.c_int32),
                ("d_colors", ctypes.c_void_p)]


class rs_projected(ctypes.Structure):
    _fields_ = [("d_means2d", ctypes.c_void_p), ("d_depth", ctypes.c_void_p),
                ("d_conic", ctypes.c_void_p), ("d_color", ctypes.c_void_p),
                ("d_radius", ctypes.c_void_p), ("d_tiles_touched", ctypes.c_void_p),
                ("d_records", ctypes.c_void_p), ("d_ellipse", ctypes.c_void_p),
                ("tile_test", ctypes.c_int32)]


RS_TILE_TEST_SQUARE, RS_TILE_TEST_ELLIPSE = 0, 1
RS_ELLIPSE_WORDS = 12  # rows of the ellipse tile test's per-Gaussian words
RS_RASTER_CHUNK = 256  # entries per backward task; spacing of the forward's recorded states


class rs_mlp(ctypes.Structure):
    _fields_ = [("latent_dim", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("d_W1", ctypes.c_void_p), ("d_b1", ctypes.c_void_p),
                ("d_W2", ctypes.c_void_p), ("d_b2", ctypes.c_void_p)]


class rs_mlp_grads(ctypes.Structure):
    _fields_ = [("d_dW1", ctypes.c_void_p), ("d_db1", ctypes.c_void_p),
                ("d_dW2", ctypes.c_void_p), ("d_db2", ctypes.c_void_p)]


class rs_adam_segment(ctypes.Structure):
    _fields_ = [("d_param", ctypes.c_void_p), ("d_grad", ctypes.c_void_p), ("d_m", ctypes.c_void_p),
                ("d_v", ctypes.c_void_p), ("d_activated", ctypes.c_void_p), ("count", ctypes.c_size_t),
                ("lr", ctypes.c_float), ("activation", ctypes.c_int32)]


class rs_fp8_matrix(ctypes.Structure):
    _fields_ = [("d_q", ctypes.c_void_p), ("stride", ctypes.c_size_t), ("d_scales", ctypes.c_void_p)]


class rs_sandwich(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate_cols", ctypes.c_int32),
                ("d_x", ctypes.c_void_p), ("x_stride", ctypes.c_size_t), ("d_x_scales", ctypes.c_void_p),
                ("d_r", ctypes.c_void_p), ("r_stride", ctypes.c_size_t), ("d_r_scales", ctypes.c_void_p),
                ("d_gate", ctypes.c_void_p), ("gate_stride", ctypes.c_size_t), ("d_gate_scales", ctypes.c_void_p),
                ("d_residual_scale", ctypes.c_void_p), ("d_post_weight", ctypes.c_void_p),
                ("d_pre_weight", ctypes.c_void_p)]


class rs_sandwich_out(ctypes.Structure):
    _fields_ = [("d_sum", ctypes.c_void_p), ("sum_stride", ctypes.c_size_t), ("d_y", ctypes.c_void_p),
                ("y_stride", ctypes.c_size_t), ("q", rs_fp8_matrix), ("kept_x", rs_fp8_matrix),
                ("kept_r", rs_fp8_matrix), ("kept_gate", rs_fp8_matrix), ("d_rstd_r", ctypes.c_void_p),
                ("d_rstd_s", ctypes.c_void_p)]


class rs_sandwich_grads(ctypes.Structure):
    _fields_ = [("d_rstd_r", ctypes.c_void_p), ("d_rstd_s", ctypes.c_void_p), ("d_dL_dy", ctypes.c_void_p),
                ("dy_stride", ctypes.c_size_t), ("d_dL_dsum", ctypes.c_void_p), ("dsum_stride", ctypes.c_size_t),
                ("d_dL_dx", ctypes.c_void_p), ("dx_stride", ctypes.c_size_t), ("d_dL_dr", ctypes.c_void_p),
                ("dr_stride", ctypes.c_size_t), ("d_dL_dgate", ctypes.c_void_p), ("dgate_stride", ctypes.c_size_t),
                ("d_dL_dresidual_scale", ctypes.c_void_p), ("d_dL_dpost_weight", ctypes.c_void_p),
                ("d_dL_dpre_weight", ctypes.c_void_p)]


RS_ACT_IDENTITY, RS_ACT_EXP, RS_ACT_SIGMOID = 0, 1, 2
RS_ADAM_MAX_SEGMENTS = 16

_lib = None
_VP = ctypes.c_void_p


def declared_signatures(header: str | None = None):
    """(return type, name) of the entry points the headers under include/ declare (or `header`)."""
    headers = [header] if header else sorted(glob.glob(os.path.join(os.path.dirname(HEADER), "*.h")))
    text = "".join(open(h).read() for h in headers)
    return sorted(set(re.findall(r"^\s*(int|const char\*|size_t)\s+(rs_\w+)\s*\(", text, re.M)))


def declared_symbols(header: str | None = None):
    """Names of the entry points the headers under include/ declare (or `header`)."""
    return sorted({name for _, name in declared_signatures(header)})


_RESTYPES = {"int": ctypes.c_int, "size_t": ctypes.c_size_t, "const char*": ctypes.c_char_p}


def lib():
    """Load librs.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m gaussian_splatting_tile_gb300.build_lib`")
        L = ctypes.CDLL(LIB_PATH)
        L.rs_error_string.restype = ctypes.c_char_p
        L.rs_error_string.argtypes = [ctypes.c_int]
        L.rs_project.argtypes = [ctypes.POINTER(rs_camera), ctypes.POINTER(rs_gaussians),
                                 ctypes.POINTER(rs_projected), _VP]
        L.rs_bin_workspace_size.argtypes = [ctypes.c_int32, ctypes.POINTER(rs_camera), ctypes.c_size_t,
                                            ctypes.POINTER(ctypes.c_size_t)]
        L.rs_bin.argtypes = [ctypes.POINTER(rs_camera), ctypes.POINTER(rs_projected), ctypes.c_int32,
                             _VP, ctypes.c_size_t, ctypes.c_size_t, _VP, _VP, _VP,
                             ctypes.POINTER(ctypes.c_size_t), _VP]
        L.rs_bin_async.argtypes = [ctypes.POINTER(rs_camera), ctypes.POINTER(rs_projected), ctypes.c_int32,
                                   _VP, ctypes.c_size_t, ctypes.c_size_t, _VP, _VP, _VP, _VP, _VP]
        L.rs_bin_noalloc.argtypes = [ctypes.POINTER(rs_camera), ctypes.POINTER(rs_projected), ctypes.c_int32,
                                     ctypes.c_size_t, _VP, _VP, _VP, ctypes.POINTER(ctypes.c_size_t), _VP]
        L.rs_raster_workspace_size.argtypes = [ctypes.POINTER(rs_camera), ctypes.c_size_t]
        L.rs_raster_workspace_size.restype = ctypes.c_size_t
        L.rs_rasterize_fwd.argtypes = [ctypes.POINTER(rs_camera), ctypes.POINTER(rs_projected),
                                       ctypes.c_int32, _VP, _VP, ctypes.c_size_t, ctypes.POINTER(ctypes.c_float),
                                       _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]
        L.rs_rasterize_bwd.argtypes = [ctypes.POINTER(rs_camera), ctypes.POINTER(rs_projected),
                                       ctypes.c_int32, _VP, _VP, ctypes.c_size_t, ctypes.POINTER(ctypes.c_float),
                                       _VP, _VP, _VP, ctypes.c_size_t, _VP, _VP, _VP, _VP, _VP, _VP]
        L.rs_project_bwd.argtypes = [ctypes.POINTER(rs_camera), ctypes.POINTER(rs_gaussians),
                                     ctypes.POINTER(rs_projected), _VP, _VP, _VP, _VP, _VP, _VP,
                                     _VP, _VP]
        L.rs_appearance_fwd.argtypes = [ctypes.POINTER(rs_camera), ctypes.c_int32, _VP, _VP,
                                        ctypes.POINTER(rs_mlp), _VP, _VP]
        L.rs_appearance_bwd.argtypes = [ctypes.POINTER(rs_camera), ctypes.c_int32, _VP, _VP,
                                        ctypes.POINTER(rs_mlp), _VP, _VP, ctypes.POINTER(rs_mlp_grads), _VP]
        L.rs_l1_loss_grad.argtypes = [ctypes.c_size_t, _VP, _VP, ctypes.c_float, _VP, _VP, _VP]
        L.rs_adam_step.argtypes = [ctypes.POINTER(rs_adam_segment), ctypes.c_int32, ctypes.c_double,
                                   ctypes.c_double, ctypes.c_double, ctypes.c_int32, _VP]
        L.rs_densify_stats.argtypes = [ctypes.c_int32, _VP, _VP, _VP, _VP, _VP]
        L.rs_densify_workspace_size.argtypes = [ctypes.c_int32]
        L.rs_densify_plan.argtypes = [ctypes.c_int32, _VP, _VP, _VP, _VP, ctypes.POINTER(rs_densify_rule), _VP,
                                      ctypes.c_size_t, _VP, ctypes.POINTER(ctypes.c_int32), _VP]
        L.rs_densify_apply.argtypes = [ctypes.c_int32, _VP, ctypes.c_size_t, _VP, _VP, _VP,
                                       ctypes.POINTER(rs_densify_group), ctypes.c_int32, ctypes.c_int32, _VP]
        L.rs_l1_dssim_workspace_size.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.POINTER(ctypes.c_size_t)]
        L.rs_l1_dssim_loss_grad.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _VP, _VP, ctypes.c_float,
                                            ctypes.c_float, _VP, _VP, _VP, ctypes.c_size_t, _VP]
        L.rs_device_error.argtypes = []
        i32, sz = ctypes.c_int32, ctypes.c_size_t
        L.rs_rms_norm_fwd.argtypes = [i32, i32, i32, _VP, sz, _VP, sz, _VP, ctypes.c_float, _VP, sz, _VP, sz, _VP, sz,
                                      _VP, _VP, _VP]
        L.rs_rms_norm_bwd_workspace_size.argtypes = [i32, i32]
        L.rs_rms_norm_bwd.argtypes = [i32, i32, i32, _VP, sz, _VP, _VP, _VP, sz, _VP, sz, _VP, sz, _VP, _VP, sz, _VP]
        L.rs_quantize_fp8.argtypes = [i32, i32, i32, _VP, sz, _VP, sz, _VP, sz, _VP, _VP, sz, _VP, _VP]
        L.rs_quantize_fp8_blocks.argtypes = [i32, i32, i32, _VP, sz, _VP, sz, _VP, _VP, sz, _VP, _VP]
        L.rs_matmul_fp8_workspace_size.argtypes = [i32, i32, i32]
        L.rs_matmul_fp8.argtypes = [i32, i32, i32, _VP, sz, _VP, _VP, sz, _VP, i32, i32, i32, _VP, sz, _VP, sz, _VP]
        L.rs_grad_norm_workspace_size.argtypes = [i32]
        L.rs_grad_norm.argtypes = [_VP, i32, _VP, _VP, sz, _VP]
        L.rs_grad_clip.argtypes = [_VP, i32, ctypes.c_float, _VP, _VP, sz, _VP]
        L.rs_adam_step_clipped.argtypes = [ctypes.POINTER(rs_adam_segment), i32, ctypes.c_double, ctypes.c_double,
                                           ctypes.c_double, i32, ctypes.c_float, _VP, _VP, sz, _VP]
        L.rs_adam_step_clipped_counted.argtypes = [ctypes.POINTER(rs_adam_segment), i32, ctypes.c_double, ctypes.c_double,
                                                   ctypes.c_double, _VP, ctypes.c_float, _VP, _VP, sz, _VP]
        # rs_sandwich and its companions come by reference or as their packed bytes
        L.rs_sandwich_norm_fwd.argtypes = [_VP, ctypes.c_float, _VP, _VP]
        L.rs_sandwich_norm_bwd_workspace_size.argtypes = [i32, i32]
        L.rs_sandwich_norm_bwd.argtypes = [_VP, _VP, _VP, sz, _VP]
        L.rs_quantize_fp8_relu8.argtypes = [i32, i32, i32, _VP, sz, _VP, sz, _VP, sz, _VP, _VP, sz, _VP, _VP]
        L.rs_transpose_fp8.argtypes = [i32, i32, _VP, sz, _VP, _VP, sz, _VP, _VP]
        L.rs_matmul_fp8_q_workspace_size.argtypes = [i32, i32, i32]
        L.rs_matmul_fp8_q.argtypes = [i32, i32, i32, _VP, sz, _VP, _VP, sz, _VP, i32, i32, _VP, sz, _VP, _VP, sz, _VP]
        for ret, name in declared_signatures():
            getattr(L, name).restype = _RESTYPES[ret]
        _lib = L
    return _lib


def error_string(code: int) -> str:
    return lib().rs_error_string(code).decode()


def _check(fn: str, code: int):
    if code != RS_OK:
        raise RsError(fn, code, error_string(code))


# the current stream's handle without building a Stream object (3 us of a small call's 13), where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


# the current device without a look at whether CUDA has been set up, which whoever has a CUDA tensor has seen to
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream):
    if stream is None:
        return _raw_stream(_device())
    return stream.cuda_stream


def _ptr(t, dtype=None, numel=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return ctypes.c_void_p(t.data_ptr())


def camera_struct(cam) -> rs_camera:
    c = rs_camera()
    R = np.asarray(cam.R, np.float32).reshape(9)
    t = np.asarray(cam.t, np.float32).reshape(3)
    for i in range(9):
        c.R[i] = float(R[i])
    for i in range(3):
        c.t[i] = float(t[i])
    c.fx, c.fy, c.cx, c.cy = float(cam.fx), float(cam.fy), float(cam.cx), float(cam.cy)
    c.width, c.height = int(cam.width), int(cam.height)
    return c


@dataclasses.dataclass
class DeviceGaussians:
    """Planar float32 CUDA tensors: means [3,N], scales [3,N], quats [4,N], opacity [N],
    sh [3K,N] (sh_degree 0..3) or colors [3,N] (sh_degree -1)."""
    means: torch.Tensor
    scales: torch.Tensor
    quats: torch.Tensor
    opacity: torch.Tensor
    sh: torch.Tensor | None
    sh_degree: int
    colors: torch.Tensor | None = None

    @property
    def n(self) -> int:
        return int(self.opacity.shape[0])

    @staticmethod
    def from_numpy(g, device="cuda"):
        f = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(device)
        return DeviceGaussians(f(g.means), f(g.scales), f(g.quats), f(g.opacity), f(g.sh),
                               int(g.sh_degree), f(g.colors))

    def struct(self) -> rs_gaussians:
        n = self.n
        s = rs_gaussians()
        s.n = n
        s.d_means = _ptr(self.means, torch.float32, 3 * n, "means")
        s.d_scales = _ptr(self.scales, torch.float32, 3 * n, "scales")
        s.d_quats = _ptr(self.quats, torch.float32, 4 * n, "quats")
        s.d_opacity = _ptr(self.opacity, torch.float32, n, "opacity")
        s.sh_degree = int(self.sh_degree)
        if self.sh_degree >= 0:
            s.d_sh = _ptr(self.sh, torch.float32, 3 * (self.sh_degree + 1) ** 2 * n, "sh")
        else:
            s.d_colors = _ptr(self.colors, torch.float32, 3 * n, "colors")
        return s


@dataclasses.dataclass
class DeviceProjected:
    means2d: torch.Tensor
    depth: torch.Tensor
    conic: torch.Tensor
    color: torch.Tensor
    radius: torch.Tensor
    tiles_touched: torch.Tensor
    records: torch.Tensor  # uint8 [N*48]
    ellipse: torch.Tensor | None = None  # [RS_ELLIPSE_WORDS, N], the ellipse tile test's words:
                                         # row 0 its k, the rest its setup for the binning
    tile_test: int = 0                   # RS_TILE_TEST_SQUARE or RS_TILE_TEST_ELLIPSE

    @staticmethod
    def empty(n: int, device="cuda", tile_test: int = 0):
        f = lambda *s: torch.empty(*s, dtype=torch.float32, device=device)
        return DeviceProjected(f(2, n), f(n), f(3, n), f(3, n),
                               torch.empty(n, dtype=torch.int32, device=device),
                               torch.empty(n, dtype=torch.int32, device=device),
                               torch.empty(max(n, 1) * RECORD_BYTES, dtype=torch.uint8, device=device),
                               f(RS_ELLIPSE_WORDS, max(n, 1)) if tile_test == RS_TILE_TEST_ELLIPSE else None,
                               int(tile_test))

    @property
    def alpha_k(self) -> torch.Tensor | None:
        """k of the alpha >= 1/255 ellipse, per Gaussian (0 when culled); ellipse test only."""
        return None if self.ellipse is None else self.ellipse[0, : self.depth.shape[0]]

    def struct(self) -> rs_projected:
        n = int(self.depth.shape[0])
        s = rs_projected()
        s.d_means2d = _ptr(self.means2d, torch.float32, 2 * n, "means2d")
        s.d_depth = _ptr(self.depth, torch.float32, n, "depth")
        s.d_conic = _ptr(self.conic, torch.float32, 3 * n, "conic")
        s.d_color = _ptr(self.color, torch.float32, 3 * n, "color")
        s.d_radius = _ptr(self.radius, torch.int32, n, "radius")
        s.d_tiles_touched = _ptr(self.tiles_touched, None, n, "tiles_touched")
        s.d_records = _ptr(self.records, torch.uint8, n * RECORD_BYTES, "records")
        s.tile_test = int(self.tile_test)
        if self.tile_test == RS_TILE_TEST_ELLIPSE:
            if self.ellipse is None or self.ellipse.dtype != torch.float32 or not self.ellipse.is_contiguous() \
                    or tuple(self.ellipse.shape) != (RS_ELLIPSE_WORDS, max(n, 1)):
                raise ValueError(f"ellipse: want a contiguous float32 [{RS_ELLIPSE_WORDS}, {max(n, 1)}] tensor")
            s.d_ellipse = ctypes.c_void_p(self.ellipse.data_ptr())
        return s


# ------------------------------------------------------------------ prepared calls
class PreparedCall:
    """One C-ABI call with its arguments marshalled once: the pointer arguments of a fixed set of
    buffers are built a single time and the camera struct is shared (and updated in place when the
    view changes), so a frame loop pays only the foreign call.  `run(stream_handle)` returns the
    library's return code after raising on errors."""

    def __init__(self, name: str, args):
        self.name = name
        self.fn = getattr(lib(), name)
        self.args = tuple(args)

    def run(self, stream_handle) -> int:
        rc = self.fn(*self.args, stream_handle)
        if rc != RS_OK:
            raise RsError(self.name, rc, error_string(rc))
        return rc


def set_camera_struct(c: rs_camera, cam) -> rs_camera:
    """Overwrite an existing rs_camera with `cam` (prepared calls keep pointing at it)."""
    R = np.asarray(cam.R, np.float32).reshape(9)
    t = np.asarray(cam.t, np.float32).reshape(3)
    c.R[:] = [float(x) for x in R]
    c.t[:] = [float(x) for x in t]
    c.fx, c.fy, c.cx, c.cy = float(cam.fx), float(cam.fy), float(cam.cx), float(cam.cy)
    c.width, c.height = int(cam.width), int(cam.height)
    return c


def stream_handle(stream=None):
    return ctypes.c_void_p(_stream(stream))


# ------------------------------------------------------------------ the five calls

def rs_project(camera, gaussians: DeviceGaussians, out: DeviceProjected, stream=None):
    c, g, o = camera_struct(camera), gaussians.struct(), out.struct()
    _check("rs_project", lib().rs_project(ctypes.byref(c), ctypes.byref(g), ctypes.byref(o), _stream(stream)))


def rs_bin_workspace_size(n: int, camera, capacity: int) -> int:
    c = camera_struct(camera)
    b = ctypes.c_size_t(0)
    _check("rs_bin_workspace_size", lib().rs_bin_workspace_size(int(n), ctypes.byref(c), int(capacity), ctypes.byref(b)))
    return int(b.value)


def rs_bin(camera, proj: DeviceProjected, n: int, workspace: torch.Tensor, capacity: int,
           keys_sorted, point_list: torch.Tensor, tile_ranges: torch.Tensor, stream=None) -> int:
    """Returns the entry count E; raises RsError (code RS_ERR_CAPACITY, .n_entries set) when
    E exceeds `capacity`."""
    c = camera_struct(camera)
    p = proj.struct()
    E = ctypes.c_size_t(0)
    rc = lib().rs_bin(ctypes.byref(c), ctypes.byref(p), int(n), _ptr(workspace, torch.uint8, None, "workspace"),
                      int(workspace.numel()), int(capacity), _ptr(keys_sorted, torch.int64, capacity, "keys_sorted"),
                      _ptr(point_list, torch.int32, capacity, "point_list"),
                      _ptr(tile_ranges, torch.int32, 2 * ((camera.width + 15) // 16) * ((camera.height + 15) // 16),
                           "tile_ranges"),
                      ctypes.byref(E), _stream(stream))
    if rc == RS_ERR_CAPACITY:
        err = RsError("rs_bin", rc, error_string(rc))
        err.n_entries = int(E.value)
        raise err
    _check("rs_bin", rc)
    return int(E.value)


def rs_bin_async(camera, proj: DeviceProjected, n: int, workspace: torch.Tensor, capacity: int,
                 keys_sorted, point_list: torch.Tensor, tile_ranges: torch.Tensor, result: torch.Tensor,
                 stream=None):
    """rs_bin without the host wait: enqueues the binning and a copy of (E, error flag) into
    `result` (int64 [2], pinned host memory); read it after synchronising the stream."""
    if result.is_cuda or result.dtype != torch.int64 or result.numel() < 2 or not result.is_contiguous():
        raise TypeError("result must be a contiguous int64 host tensor with 2 elements (pinned)")
    c = camera_struct(camera)
    p = proj.struct()
    _check("rs_bin_async", lib().rs_bin_async(
        ctypes.byref(c), ctypes.byref(p), int(n), _ptr(workspace, torch.uint8, None, "workspace"),
        int(workspace.numel()), int(capacity), _ptr(keys_sorted, torch.int64, capacity, "keys_sorted"),
        _ptr(point_list, torch.int32, capacity, "point_list"),
        _ptr(tile_ranges, torch.int32, 2 * ((camera.width + 15) // 16) * ((camera.height + 15) // 16), "tile_ranges"),
        ctypes.c_void_p(result.data_ptr()), _stream(stream)))


def rs_bin_noalloc(camera, proj: DeviceProjected, n: int, capacity: int, keys_sorted,
                   point_list: torch.Tensor, tile_ranges: torch.Tensor, stream=None) -> int:
    """rs_bin without a workspace (the library's fixed scratch array is used).  Returns E; raises
    RsError (RS_ERR_CAPACITY with .n_entries, or RS_ERR_WORKSPACE when the sizes exceed the
    fixed scratch)."""
    c = camera_struct(camera)
    p = proj.struct()
    E = ctypes.c_size_t(0)
    rc = lib().rs_bin_noalloc(ctypes.byref(c), ctypes.byref(p), int(n), int(capacity),
                              _ptr(keys_sorted, torch.int64, capacity, "keys_sorted"),
                              _ptr(point_list, torch.int32, capacity, "point_list"),
                              _ptr(tile_ranges, torch.int32,
                                   2 * ((camera.width + 15) // 16) * ((camera.height + 15) // 16), "tile_ranges"),
                              ctypes.byref(E), _stream(stream))
    if rc == RS_ERR_CAPACITY:
        err = RsError("rs_bin_noalloc", rc, error_string(rc))
        err.n_entries = int(E.value)
        raise err
    _check("rs_bin_noalloc", rc)
    return int(E.value)


def _bg(bg):
    arr = (ctypes.c_float * 3)(*[float(x) for x in bg])
    return arr


def rs_raster_workspace_size(camera, capacity: int) -> int:
    """Bytes of the compositing workspace for a point list of `capacity` entries."""
    c = camera_struct(camera)
    n = int(lib().rs_raster_workspace_size(ctypes.byref(c), int(capacity)))
    if n == 0:
        raise ValueError("invalid camera or capacity")
    return n


def rs_rasterize_fwd(camera, proj: DeviceProjected, n: int, tile_ranges, point_list, bg, image,
                     final_T, n_contrib, workspace, stream=None):
    c = camera_struct(camera)
    p = proj.struct()
    HW = camera.width * camera.height
    _check("rs_rasterize_fwd", lib().rs_rasterize_fwd(
        ctypes.byref(c), ctypes.byref(p), int(n), _ptr(tile_ranges, torch.int32, None, "tile_ranges"),
        _ptr(point_list, torch.int32, None, "point_list"), int(point_list.numel()), _bg(bg),
        _ptr(image, torch.float32, 3 * HW, "image"), _ptr(final_T, torch.float32, HW, "final_T"),
        _ptr(n_contrib, torch.int32, HW, "n_contrib"), _ptr(workspace, torch.uint8, None, "workspace"),
        int(workspace.numel()), _stream(stream)))


def rs_rasterize_bwd(camera, proj: DeviceProjected, n: int, tile_ranges, point_list, bg, final_T,
                     n_contrib, workspace, dL_dimage, dL_dmeans2d, dL_dconic, dL_dopacity, dL_dcolor,
                     stream=None):
    c = camera_struct(camera)
    p = proj.struct()
    HW = camera.width * camera.height
    _check("rs_rasterize_bwd", lib().rs_rasterize_bwd(
        ctypes.byref(c), ctypes.byref(p), int(n), _ptr(tile_ranges, torch.int32, None, "tile_ranges"),
        _ptr(point_list, torch.int32, None, "point_list"), int(point_list.numel()), _bg(bg),
        _ptr(final_T, torch.float32, HW, "final_T"),
        _ptr(n_contrib, torch.int32, HW, "n_contrib"), _ptr(workspace, torch.uint8, None, "workspace"),
        int(workspace.numel()), _ptr(dL_dimage, torch.float32, 3 * HW, "dL_dimage"),
        _ptr(dL_dmeans2d, torch.float32, 2 * n, "dL_dmeans2d"), _ptr(dL_dconic, torch.float32, 3 * n, "dL_dconic"),
        _ptr(dL_dopacity, torch.float32, n, "dL_dopacity"), _ptr(dL_dcolor, torch.float32, 3 * n, "dL_dcolor"),
        _stream(stream)))


def rs_project_bwd(camera, gaussians: DeviceGaussians, proj: DeviceProjected, dL_dmeans2d, dL_dconic,
                   dL_dcolor, dL_dmeans, dL_dscales, dL_dquats, dL_dsh, stream=None):
    c = camera_struct(camera)
    g = gaussians.struct()
    p = proj.struct()
    n = gaussians.n
    K = (gaussians.sh_degree + 1) ** 2 if gaussians.sh_degree >= 0 else 0
    _check("rs_project_bwd", lib().rs_project_bwd(
        ctypes.byref(c), ctypes.byref(g), ctypes.byref(p), _ptr(dL_dmeans2d, torch.float32, 2 * n, "dL_dmeans2d"),
        _ptr(dL_dconic, torch.float32, 3 * n, "dL_dconic"), _ptr(dL_dcolor, torch.float32, 3 * n, "dL_dcolor"),
        _ptr(dL_dmeans, torch.float32, 3 * n, "dL_dmeans"), _ptr(dL_dscales, torch.float32, 3 * n, "dL_dscales"),
        _ptr(dL_dquats, torch.float32, 4 * n, "dL_dquats"),
        _ptr(dL_dsh, torch.float32, 3 * K * n, "dL_dsh") if K else None, _stream(stream)))


# ------------------------------------------------------------------ appearance MLP and L1 loss

@dataclasses.dataclass
class DeviceMLP:
    """Appearance MLP weights as float32 CUDA tensors: W1 [hidden, latent_dim + 3], b1 [hidden],
    W2 [3, hidden], b2 [3]."""
    W1: torch.Tensor
    b1: torch.Tensor
    W2: torch.Tensor
    b2: torch.Tensor

    @property
    def hidden(self) -> int:
        return int(self.W1.shape[0])

    @property
    def latent_dim(self) -> int:
        return int(self.W1.shape[1]) - 3

    @staticmethod
    def from_numpy(p, device="cuda"):
        f = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(device)
        return DeviceMLP(f(p["W1"]), f(p["b1"]), f(p["W2"]), f(p["b2"]))

    def struct(self) -> rs_mlp:
        m = rs_mlp()
        H, L = self.hidden, self.latent_dim
        m.latent_dim, m.hidden = L, H
        m.d_W1 = _ptr(self.W1, torch.float32, H * (L + 3), "W1")
        m.d_b1 = _ptr(self.b1, torch.float32, H, "b1")
        m.d_W2 = _ptr(self.W2, torch.float32, 3 * H, "W2")
        m.d_b2 = _ptr(self.b2, torch.float32, 3, "b2")
        return m


@dataclasses.dataclass
class DeviceMLPGrads:
    dW1: torch.Tensor
    db1: torch.Tensor
    dW2: torch.Tensor
    db2: torch.Tensor

    @staticmethod
    def like(m: DeviceMLP):
        return DeviceMLPGrads(torch.empty_like(m.W1), torch.empty_like(m.b1), torch.empty_like(m.W2),
                              torch.empty_like(m.b2))

    def struct(self) -> rs_mlp_grads:
        g = rs_mlp_grads()
        g.d_dW1 = _ptr(self.dW1, torch.float32, None, "dW1")
        g.d_db1 = _ptr(self.db1, torch.float32, None, "db1")
        g.d_dW2 = _ptr(self.dW2, torch.float32, None, "dW2")
        g.d_db2 = _ptr(self.db2, torch.float32, None, "db2")
        return g


def rs_appearance_fwd(camera, means: torch.Tensor, latents: torch.Tensor, mlp: DeviceMLP,
                      colors: torch.Tensor, stream=None):
    n = int(latents.shape[1])
    c, m = camera_struct(camera), mlp.struct()
    _check("rs_appearance_fwd", lib().rs_appearance_fwd(
        ctypes.byref(c), n, _ptr(means, torch.float32, 3 * n, "means"),
        _ptr(latents, torch.float32, mlp.latent_dim * n, "latents"), ctypes.byref(m),
        _ptr(colors, torch.float32, 3 * n, "colors"), _stream(stream)))


def rs_device_error() -> int:
    """RS_ERR_DEVICE_CHECK if a compositing kernel skipped caller data out of range (a point-list
    entry >= n, a tile range past the capacity), RS_ERR_DEVICE_TIMEOUT if a bounded wait gave up,
    since the last call (the flags are cleared), else RS_OK; synchronises the device."""
    return int(lib().rs_device_error())


def rs_appearance_bwd(camera, means: torch.Tensor, latents: torch.Tensor, mlp: DeviceMLP,
                      dL_dcolors: torch.Tensor, dL_dlatents: torch.Tensor, grads: DeviceMLPGrads,
                      stream=None):
    n = int(latents.shape[1])
    c, m, g = camera_struct(camera), mlp.struct(), grads.struct()
    _check("rs_appearance_bwd", lib().rs_appearance_bwd(
        ctypes.byref(c), n, _ptr(means, torch.float32, 3 * n, "means"),
        _ptr(latents, torch.float32, mlp.latent_dim * n, "latents"), ctypes.byref(m),
        _ptr(dL_dcolors, torch.float32, 3 * n, "dL_dcolors"),
        _ptr(dL_dlatents, torch.float32, mlp.latent_dim * n, "dL_dlatents"), ctypes.byref(g), _stream(stream)))


def rs_l1_loss_grad(image: torch.Tensor, target: torch.Tensor, scale: float, dL_dimage: torch.Tensor,
                    loss: torch.Tensor | None = None, stream=None):
    count = int(image.numel())
    if int(target.numel()) != count:
        raise ValueError("image and target differ in size")
    _check("rs_l1_loss_grad", lib().rs_l1_loss_grad(
        count, _ptr(image, torch.float32, count, "image"), _ptr(target, torch.float32, count, "target"),
        ctypes.c_float(scale), _ptr(dL_dimage, torch.float32, count, "dL_dimage"),
        _ptr(loss, torch.float32, 1, "loss"), _stream(stream)))


# ------------------------------------------------------------------ optimiser

@dataclasses.dataclass
class AdamGroup:
    """One parameter group of rs_adam_step: float32 CUDA tensors of equal size."""
    param: torch.Tensor
    grad: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    lr: float
    activation: int = RS_ACT_IDENTITY
    activated: torch.Tensor | None = None


def _adam_segments(groups):
    if len(groups) > RS_ADAM_MAX_SEGMENTS:
        raise ValueError(f"at most {RS_ADAM_MAX_SEGMENTS} groups per call")
    f32, segs = torch.float32, []
    for gr in groups:
        k = gr.param.numel()
        segs.append((_vec(gr.param, f32, k, "param"), _vec(gr.grad, f32, k, "grad"), _vec(gr.m, f32, k, "m"),
                     _vec(gr.v, f32, k, "v"), _vec(gr.activated, f32, k, "activated"), k, float(gr.lr), int(gr.activation)))
    return (rs_adam_segment * max(1, len(segs)))(*segs)


def rs_adam_step(groups, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-15,
                 stream=None):
    arr = _adam_segments(groups)
    _check("rs_adam_step", lib().rs_adam_step(arr, len(groups), float(beta1), float(beta2), float(eps), int(step),
                                              _stream(stream)))


def rs_densify_stats(dL_dmeans2d: torch.Tensor, radius: torch.Tensor, accum: torch.Tensor, count: torch.Tensor,
                     stream=None):
    n = int(radius.numel())
    _check("rs_densify_stats", lib().rs_densify_stats(
        n, _ptr(dL_dmeans2d, torch.float32, 2 * n, "dL_dmeans2d"), _ptr(radius, torch.int32, n, "radius"),
        _ptr(accum, torch.float32, n, "accum"), _ptr(count, torch.float32, n, "count"), _stream(stream)))


RS_DENSIFY_COPY, RS_DENSIFY_MEANS, RS_DENSIFY_LOG_SCALES, RS_DENSIFY_MAX_GROUPS = 0, 1, 2, 8


class rs_densify_rule(ctypes.Structure):
    _fields_ = [("grad_threshold", ctypes.c_float), ("dense_scale", ctypes.c_float),
                ("min_opacity", ctypes.c_float), ("max_scale", ctypes.c_float)]


class rs_densify_group(ctypes.Structure):
    _fields_ = [("d_param", _VP), ("d_m", _VP), ("d_v", _VP), ("d_param_out", _VP), ("d_m_out", _VP),
                ("d_v_out", _VP), ("rows", ctypes.c_int32), ("kind", ctypes.c_int32)]


@dataclasses.dataclass
class DensifyGroup:
    """One parameter array [rows, n] of rs_densify_apply with its Adam moments (m, v may be None);
    the outputs [rows, n_out] (m_out, v_out may be None)."""
    param: torch.Tensor
    param_out: torch.Tensor
    m: torch.Tensor | None = None
    v: torch.Tensor | None = None
    m_out: torch.Tensor | None = None
    v_out: torch.Tensor | None = None
    kind: int = RS_DENSIFY_COPY


def rs_densify_workspace_size(n: int) -> int:
    return int(lib().rs_densify_workspace_size(int(n)))


def rs_densify_plan(accum, count, log_scales, opacity_logits, grad_threshold: float, dense_scale: float,
                    min_opacity: float, max_scale: float, workspace: torch.Tensor, action: torch.Tensor | None = None,
                    stream=None) -> dict:
    """Classification and counts of rs_densify_plan (float32 CUDA tensors; workspace uint8 CUDA of at
    least rs_densify_workspace_size(n) bytes; action: optional uint8 CUDA [n])."""
    n = int(accum.numel())
    rule = rs_densify_rule(float(grad_threshold), float(dense_scale), float(min_opacity), float(max_scale))
    counts = (ctypes.c_int32 * 5)()
    _check("rs_densify_plan", lib().rs_densify_plan(
        n, _ptr(accum, torch.float32, n, "accum"), _ptr(count, torch.float32, n, "count"),
        _ptr(log_scales, torch.float32, 3 * n, "log_scales"), _ptr(opacity_logits, torch.float32, n, "opacity_logits"),
        ctypes.byref(rule), _ptr(workspace, torch.uint8, rs_densify_workspace_size(n), "workspace"),
        ctypes.c_size_t(workspace.numel()), _ptr(action, torch.uint8, n, "action"), counts, _stream(stream)))
    return dict(zip(("n_out", "kept", "cloned", "split", "removed"), (int(x) for x in counts)))


def rs_densify_apply(n: int, workspace: torch.Tensor, quats, log_scales, noise, groups, n_out: int, stream=None):
    """Moves every group (list of DensifyGroup) to its densified outputs; noise: float32 CUDA [2, 3, n]."""
    if len(groups) > RS_DENSIFY_MAX_GROUPS:
        raise ValueError(f"at most {RS_DENSIFY_MAX_GROUPS} groups per call")
    arr = (rs_densify_group * max(1, len(groups)))()
    for k, gr in enumerate(groups):
        rows = int(gr.param.numel()) // max(n, 1)
        arr[k].d_param = _ptr(gr.param, torch.float32, rows * n, "param")
        arr[k].d_m = _ptr(gr.m, torch.float32, rows * n, "m")
        arr[k].d_v = _ptr(gr.v, torch.float32, rows * n, "v")
        arr[k].d_param_out = _ptr(gr.param_out, torch.float32, rows * n_out, "param_out")
        arr[k].d_m_out = _ptr(gr.m_out, torch.float32, rows * n_out, "m_out")
        arr[k].d_v_out = _ptr(gr.v_out, torch.float32, rows * n_out, "v_out")
        arr[k].rows = rows
        arr[k].kind = int(gr.kind)
    _check("rs_densify_apply", lib().rs_densify_apply(
        int(n), _ptr(workspace, torch.uint8, rs_densify_workspace_size(n), "workspace"),
        ctypes.c_size_t(workspace.numel()), _ptr(quats, torch.float32, 4 * n, "quats"),
        _ptr(log_scales, torch.float32, 3 * n, "log_scales"), _ptr(noise, torch.float32, 6 * n, "noise"),
        arr, len(groups), int(n_out), _stream(stream)))


def rs_l1_dssim_workspace_size(channels: int, height: int, width: int) -> int:
    b = ctypes.c_size_t(0)
    _check("rs_l1_dssim_workspace_size", lib().rs_l1_dssim_workspace_size(int(channels), int(height), int(width),
                                                                          ctypes.byref(b)))
    return int(b.value)


def rs_l1_dssim_loss_grad(image: torch.Tensor, target: torch.Tensor, lam: float, scale: float,
                          dL_dimage: torch.Tensor, loss: torch.Tensor | None, workspace: torch.Tensor, stream=None):
    """image, target, dL_dimage: float32 CUDA [C, H, W]; workspace: uint8 CUDA tensor of at least
    rs_l1_dssim_workspace_size bytes."""
    C, H, W = (int(x) for x in image.shape)
    n = C * H * W
    _check("rs_l1_dssim_loss_grad", lib().rs_l1_dssim_loss_grad(
        C, H, W, _ptr(image, torch.float32, n, "image"), _ptr(target, torch.float32, n, "target"),
        ctypes.c_float(lam), ctypes.c_float(scale), _ptr(dL_dimage, torch.float32, n, "dL_dimage"),
        _ptr(loss, torch.float32, 1, "loss"), _ptr(workspace, torch.uint8, None, "workspace"),
        int(workspace.numel()), _stream(stream)))


# ------------------------------------------------------------------ wide appearance networks

RS_F32, RS_F16, RS_BF16 = 0, 1, 2
RS_FP8_BLOCK, RS_NORM_MAX_COLS = 128, 16384
_DTYPES = {torch.float32: RS_F32, torch.float16: RS_F16, torch.bfloat16: RS_BF16}
_FP8 = torch.float8_e4m3fn  # or the bytes as uint8


def _dtype(t, name="tensor") -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return code


_Tensor, _F32 = torch.Tensor, torch.float32


def _mat(t, name, dtype, shape):
    """(pointer, row stride in elements) of a row-major CUDA matrix of `shape` (rows, columns); its rows may be apart."""
    if t is None:
        return None, 0
    # the common cases in a few lines: these checks are most of a small call's time
    if type(t) is _Tensor and t.is_cuda and t.dtype is dtype and t.shape == shape:
        rows, cols = shape
        if t.is_contiguous():
            # a single row's stride is never followed: give one that the alignment rules allow
            return t.data_ptr(), (cols if rows > 1 else (cols + 15) // 16 * 16)
        s0, s1 = t.stride()
        if s1 == 1 and rows > 1:
            return t.data_ptr(), s0
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype and not (dtype is _FP8 and t.dtype is torch.uint8):
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, needs {tuple(shape)}")
    s0, s1 = t.stride()
    rows, cols = shape
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must be contiguous along its rows")
    return t.data_ptr(), (s0 if rows > 1 else (cols + 15) // 16 * 16)


def _vec(t, dtype, numel: int, name: str):
    """Pointer of a contiguous CUDA tensor of at least `numel` elements."""
    if t is None:
        return None
    if type(t) is _Tensor and t.is_cuda and t.dtype is dtype and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    return _ptr(t, dtype, numel, name).value  # says what is wrong


def fp8_empty(rows: int, cols: int, device="cuda"):
    """An 8-bit matrix [rows, cols] with rows on 16-byte boundaries, and its scales [ceil(cols / 128), rows]."""
    q = torch.empty(rows, max(16, -(-cols // 16) * 16), dtype=torch.uint8, device=device)
    return (q.view(torch.float8_e4m3fn)[:, :cols],
            torch.empty(-(-cols // RS_FP8_BLOCK), rows, dtype=torch.float32, device=device))


def fp8_dequantize(q: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """The float32 values of an 8-bit matrix with scales per row or per 128 x 128 block (plain torch, for inspection)."""
    r, c = q.shape
    s = scales if scales.shape[1] == r else scales.repeat_interleave(RS_FP8_BLOCK, 1)[:, :r]
    return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(RS_FP8_BLOCK, 0)[:c].t()


def _scales(t, name, blocks: int, rows: int):
    if type(t) is _Tensor and t.is_cuda and t.dtype is _F32 and t.shape == (blocks, rows) and t.is_contiguous():
        return t.data_ptr()
    if t is not None and t.shape != (blocks, rows):
        raise ValueError(f"{name} is {tuple(t.shape)}, needs {(blocks, rows)}")
    return _vec(t, torch.float32, 0, name)


def _blocks(n: int) -> int:
    return -(-n // RS_FP8_BLOCK)


def rs_rms_norm_fwd(x, weight, q=None, scales=None, residual=None, sum=None, y=None, rstd=None, eps: float = 1e-6,
                    stream=None):
    """x, residual, sum, y: [rows, cols] float32 / float16 / bfloat16 CUDA; weight float32 [cols]; q, scales as
    fp8_empty(rows, cols) gives them; rstd float32 [rows].  sum, y and rstd are optional outputs."""
    shape = rows, cols = x.shape
    dt = x.dtype
    code = _dtype(x, "x")
    px, sx = _mat(x, "x", dt, shape)
    pr, sr = _mat(residual, "residual", dt, shape)
    ps, ss = _mat(sum, "sum", dt, shape)
    py, sy = _mat(y, "y", dt, shape)
    pq, sq = _mat(q, "q", _FP8, shape)
    _check("rs_rms_norm_fwd", lib().rs_rms_norm_fwd(
        rows, cols, code, px, sx, pr, sr, _vec(weight, torch.float32, cols, "weight"), eps, ps, ss, py, sy, pq, sq,
        _scales(scales, "scales", _blocks(cols), rows), _vec(rstd, torch.float32, rows, "rstd"), _stream(stream)))


def rs_rms_norm_bwd_workspace_size(rows: int, cols: int) -> int:
    return int(lib().rs_rms_norm_bwd_workspace_size(int(rows), int(cols)))


def rs_rms_norm_bwd(s, weight, rstd, dL_dy, dL_dx, dL_dweight, workspace, dL_dsum=None, stream=None):
    """s: the forward's sum (x without a residual); dL_dx also is the residual's gradient; dL_dweight may be None."""
    shape = rows, cols = s.shape
    dt = s.dtype
    code = _dtype(s, "s")
    ps, ss = _mat(s, "s", dt, shape)
    pg, sg = _mat(dL_dy, "dL_dy", dt, shape)
    pd, sd = _mat(dL_dsum, "dL_dsum", dt, shape)
    px, sx = _mat(dL_dx, "dL_dx", dt, shape)
    _check("rs_rms_norm_bwd", lib().rs_rms_norm_bwd(
        rows, cols, code, ps, ss, _vec(weight, torch.float32, cols, "weight"), _vec(rstd, torch.float32, rows, "rstd"),
        pg, sg, pd, sd, px, sx, _vec(dL_dweight, torch.float32, cols, "dL_dweight"),
        _vec(workspace, torch.uint8, 0, "workspace"), 0 if workspace is None else workspace.numel(), _stream(stream)))


def rs_quantize_fp8(x, q=None, scales=None, qt=None, scales_t=None, relu=None, stream=None):
    """8-bit forms of x [rows, cols]: q, scales as fp8_empty(rows, cols), and / or the transpose qt, scales_t as
    fp8_empty(cols, rows).  relu: a relu's output; x counts as zero where it is <= 0."""
    shape = rows, cols = x.shape
    code = _dtype(x, "x")
    px, sx = _mat(x, "x", x.dtype, shape)
    pr, sr = _mat(relu, "relu", x.dtype, shape)
    pq, sq = _mat(q, "q", _FP8, shape)
    pt, st = _mat(qt, "qt", _FP8, (cols, rows))
    _check("rs_quantize_fp8", lib().rs_quantize_fp8(
        rows, cols, code, px, sx, pr, sr, pq, sq, _scales(scales, "scales", _blocks(cols), rows), pt, st,
        _scales(scales_t, "scales_t", _blocks(rows), cols), _stream(stream)))


def rs_quantize_fp8_blocks(x, q=None, scales=None, qt=None, scales_t=None, stream=None):
    """As rs_quantize_fp8 with one scale per 128 x 128 block: scales [ceil(cols / 128), ceil(rows / 128)], scales_t its
    transpose."""
    shape = rows, cols = x.shape
    code = _dtype(x, "x")
    px, sx = _mat(x, "x", x.dtype, shape)
    pq, sq = _mat(q, "q", _FP8, shape)
    pt, st = _mat(qt, "qt", _FP8, (cols, rows))
    _check("rs_quantize_fp8_blocks", lib().rs_quantize_fp8_blocks(
        rows, cols, code, px, sx, pq, sq, _scales(scales, "scales", _blocks(cols), _blocks(rows)), pt, st,
        _scales(scales_t, "scales_t", _blocks(rows), _blocks(cols)), _stream(stream)))


def rs_matmul_fp8_workspace_size(m: int, n: int, k: int) -> int:
    return int(lib().rs_matmul_fp8_workspace_size(int(m), int(n), int(k)))


def rs_matmul_fp8(a, a_scales, b, b_scales, out, workspace=None, relu: bool = False, stream=None):
    """out [m, n] (float32, float16 or bfloat16) = a [m, k] b [n, k]^T.  a_scales [ceil(k / 128), m]; b_scales per row of b
    [ceil(k / 128), n] or per 128 x 128 block [ceil(k / 128), ceil(n / 128)]."""
    m, k = a.shape
    n = b.shape[0]
    kb = _blocks(k)
    pa, sa = _mat(a, "a", _FP8, (m, k))
    pb, sb = _mat(b, "b", _FP8, (n, k))
    po, so = _mat(out, "out", out.dtype, (m, n))
    per_row = b_scales.shape == (kb, n)
    _check("rs_matmul_fp8", lib().rs_matmul_fp8(
        m, n, k, pa, sa, _scales(a_scales, "a_scales", kb, m), pb, sb,
        _scales(b_scales, "b_scales", kb, n if per_row else _blocks(n)), 1 if per_row else RS_FP8_BLOCK, int(relu),
        _dtype(out, "out"), po, so, _vec(workspace, torch.uint8, 0, "workspace"),
        0 if workspace is None else workspace.numel(), _stream(stream)))


def _gate_cols(gate, shape) -> int:
    """Of a gate (a matrix or a kept (q, scales)): 0 none, 1 one a row, else one an element."""
    if gate is None:
        return 0
    m = (gate[0] if type(gate) is tuple else gate).shape
    if m == shape:
        return shape[1]
    if len(m) != 2 or m[0] != shape[0] or m[1] != 1:
        raise ValueError(f"the gate is {tuple(m)}, needs {tuple(shape)} or {(shape[0], 1)}")
    return 1


def _form(pair, name, shape):
    """(pointer, stride, scales) of an 8-bit matrix, (q, scales) as fp8_empty gives them."""
    q, scales = pair
    p, stride = _mat(q, name, _FP8, shape)
    return p or 0, stride, _scales(scales, name, -(-shape[1] // RS_FP8_BLOCK), shape[0]) or 0


_NO_FORM = (0, 0, 0)


def _kept(pair, name, shape):
    """The same of an operand, whose scales have to be there (without rows they lie nowhere)."""
    got = _form(pair, name, shape)
    if pair[1] is None:
        raise ValueError(f"{name} needs its scales")
    return got


# The structures' fields, packed at once: a ctypes structure filled field by field takes a small call 3 us of its 14.
_SANDWICH, _SANDWICH_OUT, _SANDWICH_GRADS = (struct.Struct(f).pack for f in ("4i12Q", "18Q", "15Q"))


def _sandwich(x, r, gate, gate_cols, dtype, shape, post_weight, pre_weight, residual_scale):
    """rs_sandwich's bytes."""
    rows, cols = shape
    f32 = torch.float32
    px, sx, qx = _kept(x, "x", shape) if type(x) is tuple else (*_mat(x, "x", dtype, shape), 0)
    pr, sr, qr = _kept(r, "r", shape) if type(r) is tuple else (*_mat(r, "r", dtype, shape), 0)
    pz, sz, qz = (_NO_FORM if gate_cols == 0 else _kept(gate, "gate", shape) if type(gate) is tuple else
                  (*_mat(gate, "gate", dtype, shape if gate_cols == cols else (rows, 1)), 0))
    return _SANDWICH(rows, cols, _DTYPES[dtype], gate_cols, px or 0, sx, qx, pr or 0, sr, qr, pz or 0, sz, qz,
                     0 if residual_scale is None else _vec(residual_scale, f32, cols, "residual_scale"),
                     _vec(post_weight, f32, cols, "post_weight") or 0, _vec(pre_weight, f32, cols, "pre_weight") or 0)


def rs_sandwich_norm_fwd(x, r, post_weight, pre_weight, q=None, scales=None, gate=None, residual_scale=None, sum=None,
                         y=None, rstd_r=None, rstd_s=None, kept_x=None, kept_r=None, kept_gate=None, eps: float = 1e-6,
                         stream=None):
    """The end of a residual block: sum = residual_scale x + sigmoid(gate) norm(r) post_weight, and q, scales = the 8-bit
    form of y = norm(sum) pre_weight.  x, r, sum, y [rows, cols] float32 / float16 / bfloat16 CUDA; gate [rows, cols] or
    [rows, 1] of the same type; weights and residual_scale float32 [cols]; rstd_r, rstd_s float32 [rows].  kept_x, kept_r
    and kept_gate, (q, scales) as fp8_empty(rows, cols) gives them, receive the operands in 8 bits for the backward (gates
    within 80 of zero)."""
    shape = x.shape
    rows = shape[0]
    dt, f32 = x.dtype, torch.float32
    _dtype(x, "x")
    block = _sandwich(x, r, gate, _gate_cols(gate, shape), dt, shape, post_weight, pre_weight, residual_scale)
    ps, ss = (0, 0) if sum is None else _mat(sum, "sum", dt, shape)
    py, sy = (0, 0) if y is None else _mat(y, "y", dt, shape)
    out = _SANDWICH_OUT(
        ps, ss, py, sy, *(_NO_FORM if q is None and scales is None else _form((q, scales), "q", shape)),
        *(_NO_FORM if kept_x is None else _form(kept_x, "kept_x", shape)),
        *(_NO_FORM if kept_r is None else _form(kept_r, "kept_r", shape)),
        *(_NO_FORM if kept_gate is None else _form(kept_gate, "kept_gate", shape)),
        0 if rstd_r is None else _vec(rstd_r, f32, rows, "rstd_r") or 0,
        0 if rstd_s is None else _vec(rstd_s, f32, rows, "rstd_s") or 0)
    code = lib().rs_sandwich_norm_fwd(block, eps, out, _stream(stream))
    if code:
        _check("rs_sandwich_norm_fwd", code)


def rs_sandwich_norm_bwd_workspace_size(rows: int, cols: int) -> int:
    return int(lib().rs_sandwich_norm_bwd_workspace_size(int(rows), int(cols)))


def rs_sandwich_norm_bwd(x, r, post_weight, pre_weight, rstd_r, rstd_s, dL_dy, dL_dx, dL_dr, workspace, gate=None,
                         dL_dgate=None, residual_scale=None, dL_dsum=None, dL_dpost_weight=None, dL_dpre_weight=None,
                         dL_dresidual_scale=None, stream=None):
    """Gradients of rs_sandwich_norm_fwd.  x, r and gate: the forward's matrices, or what it kept of them, (q, scales);
    a gate of one a row always is the matrix.  The vectors' gradients and dL_dgate may be None."""
    shape = rows, cols = dL_dy.shape
    dt, f32 = dL_dy.dtype, torch.float32
    _dtype(dL_dy, "dL_dy")
    gate_cols = _gate_cols(gate, shape)
    block = _sandwich(x, r, gate, gate_cols, dt, shape, post_weight, pre_weight, residual_scale)
    pg, sg = _mat(dL_dy, "dL_dy", dt, shape)
    pu, su = (0, 0) if dL_dsum is None else _mat(dL_dsum, "dL_dsum", dt, shape)
    px, sx = _mat(dL_dx, "dL_dx", dt, shape)
    pr, sr = _mat(dL_dr, "dL_dr", dt, shape)
    pz, sz = ((0, 0) if dL_dgate is None else
              _mat(dL_dgate, "dL_dgate", dt, shape if gate_cols == cols else (rows, gate_cols)))
    grads = _SANDWICH_GRADS(
        _vec(rstd_r, f32, rows, "rstd_r") or 0, _vec(rstd_s, f32, rows, "rstd_s") or 0, pg, sg, pu, su, px or 0, sx,
        pr or 0, sr, pz, sz,
        0 if dL_dresidual_scale is None else _vec(dL_dresidual_scale, f32, cols, "dL_dresidual_scale"),
        0 if dL_dpost_weight is None else _vec(dL_dpost_weight, f32, cols, "dL_dpost_weight"),
        0 if dL_dpre_weight is None else _vec(dL_dpre_weight, f32, cols, "dL_dpre_weight"))
    code = lib().rs_sandwich_norm_bwd(
        block, grads, _vec(workspace, torch.uint8, 0, "workspace"), 0 if workspace is None else workspace.numel(),
        _stream(stream))
    if code:
        _check("rs_sandwich_norm_bwd", code)


def rs_quantize_fp8_relu8(x, relu, q=None, scales=None, qt=None, scales_t=None, stream=None):
    """rs_quantize_fp8 through a relu whose output was kept in 8 bits: x counts as zero where relu [rows, cols] (e4m3) is
    <= 0."""
    shape = rows, cols = x.shape
    code = _dtype(x, "x")
    px, sx = _mat(x, "x", x.dtype, shape)
    pr, sr = _mat(relu, "relu", _FP8, shape)
    pq, sq = _mat(q, "q", _FP8, shape)
    pt, st = _mat(qt, "qt", _FP8, (cols, rows))
    _check("rs_quantize_fp8_relu8", lib().rs_quantize_fp8_relu8(
        rows, cols, code, px, sx, pr, sr, pq, sq, _scales(scales, "scales", _blocks(cols), rows), pt, st,
        _scales(scales_t, "scales_t", _blocks(rows), cols), _stream(stream)))


def rs_transpose_fp8(q, scales, qt, scales_t, stream=None):
    """A kept matrix q [rows, cols] with scales [ceil(cols / 128), rows] as the operand of a weight's gradient: qt, scales_t
    as fp8_empty(cols, rows), the 8-bit form of the transposed values."""
    shape = rows, cols = q.shape
    pq, sq = _mat(q, "q", _FP8, shape)
    pt, st = _mat(qt, "qt", _FP8, (cols, rows))
    _check("rs_transpose_fp8", lib().rs_transpose_fp8(
        rows, cols, pq, sq, _scales(scales, "scales", _blocks(cols), rows), pt, st,
        _scales(scales_t, "scales_t", _blocks(rows), cols), _stream(stream)))


def rs_matmul_fp8_q_workspace_size(m: int, n: int, k: int) -> int:
    return int(lib().rs_matmul_fp8_q_workspace_size(int(m), int(n), int(k)))


def rs_matmul_fp8_q(a, a_scales, b, b_scales, q, scales, workspace=None, relu: bool = False, stream=None):
    """rs_matmul_fp8 with its result in 8 bits: q [m, n], scales [ceil(n / 128), m] as fp8_empty(m, n) gives them."""
    m, k = a.shape
    n = b.shape[0]
    kb = _blocks(k)
    pa, sa = _mat(a, "a", _FP8, (m, k))
    pb, sb = _mat(b, "b", _FP8, (n, k))
    pq, sq = _mat(q, "q", _FP8, (m, n))
    per_row = b_scales.shape == (kb, n)
    _check("rs_matmul_fp8_q", lib().rs_matmul_fp8_q(
        m, n, k, pa, sa, _scales(a_scales, "a_scales", kb, m), pb, sb,
        _scales(b_scales, "b_scales", kb, n if per_row else _blocks(n)), 1 if per_row else RS_FP8_BLOCK, int(relu),
        pq, sq, _scales(scales, "scales", _blocks(n), m), _vec(workspace, torch.uint8, 0, "workspace"),
        0 if workspace is None else workspace.numel(), _stream(stream)))


class rs_grad_tensor(ctypes.Structure):
    _fields_ = [("d_grad", _VP), ("d_out", _VP), ("d_param", _VP), ("count", ctypes.c_size_t),
                ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


@dataclasses.dataclass
class GradTensor:
    """One gradient of rs_grad_norm / rs_grad_clip (float32, float16 or bfloat16 CUDA, contiguous).  out: where the
    clipped values go (may be grad itself; None: only the norm).  With an activation, param holds the stored float32
    parameters and the norm counts dL/dparam."""
    grad: torch.Tensor
    out: torch.Tensor | None = None
    param: torch.Tensor | None = None
    activation: int = RS_ACT_IDENTITY


class GradTable:
    """A list of GradTensor marshalled once, for a loop that clips the same buffers every step."""

    def __init__(self, tensors):
        self.tensors = list(tensors)  # keeps the buffers alive
        self.n = len(self.tensors)
        self.arr = (rs_grad_tensor * max(1, self.n))()
        for e, g in zip(self.arr, self.tensors):
            k = int(g.grad.numel())
            e.dtype = _dtype(g.grad, "grad")
            e.d_grad = _ptr(g.grad, None, k, "grad")
            e.d_out = _ptr(g.out, g.grad.dtype, k, "out")
            e.d_param = _ptr(g.param, torch.float32, k, "param")
            e.count, e.activation = k, int(g.activation)


def _table(tensors) -> GradTable:
    return tensors if isinstance(tensors, GradTable) else GradTable(tensors)


def rs_grad_norm_workspace_size(n_tensors: int = RS_ADAM_MAX_SEGMENTS) -> int:
    return int(lib().rs_grad_norm_workspace_size(int(n_tensors)))


def rs_grad_norm(tensors, norm: torch.Tensor, workspace: torch.Tensor, stream=None):
    """norm (float32 CUDA [1]) = the global norm of `tensors` (a GradTable or a list of GradTensor)."""
    t = _table(tensors)
    _check("rs_grad_norm", lib().rs_grad_norm(t.arr, t.n, _vec(norm, torch.float32, 1, "norm"),
                                              _vec(workspace, torch.uint8, 0, "workspace"), workspace.numel(),
                                              _stream(stream)))


def rs_grad_clip(tensors, max_norm: float, norm: torch.Tensor, workspace: torch.Tensor, stream=None):
    """rs_grad_norm, and every tensor's out = grad * min(1, max_norm / (norm + 1e-6))."""
    t = _table(tensors)
    _check("rs_grad_clip", lib().rs_grad_clip(t.arr, t.n, float(max_norm), _vec(norm, torch.float32, 1, "norm"),
                                              _vec(workspace, torch.uint8, 0, "workspace"), workspace.numel(),
                                              _stream(stream)))


def rs_adam_step_clipped(groups, step, max_norm: float, norm: torch.Tensor, workspace: torch.Tensor,
                         beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-15, stream=None):
    """rs_adam_step on the gradients clipped to the global norm max_norm (nothing waits on the host; a norm that is not
    finite skips the step).  step: the step's number, or an int32 CUDA tensor [1] that counts the steps taken, which the
    call raises by one unless it skips the step (needed in a captured call, whose number would stay the same)."""
    arr = _adam_segments(groups)
    counted = isinstance(step, torch.Tensor)
    name = "rs_adam_step_clipped_counted" if counted else "rs_adam_step_clipped"
    _check(name, getattr(lib(), name)(
        arr, len(groups), float(beta1), float(beta2), float(eps),
        _vec(step, torch.int32, 1, "step") if counted else int(step), float(max_norm),
        _vec(norm, torch.float32, 1, "norm"), _vec(workspace, torch.uint8, 0, "workspace"), workspace.numel(),
        _stream(stream)))
