"""Forward and backward of one view through the five C-ABI calls, with torch-owned buffers.

This layer only allocates (through torch's caching allocator) and sequences the calls of
`rs`; all arithmetic happens in librs.so.  Buffers are kept between frames and grown when
rs_bin reports that the entry count exceeded the capacity.
"""
from __future__ import annotations

import dataclasses

import torch

from . import rs


@dataclasses.dataclass
class Forward:
    proj: rs.DeviceProjected
    n_entries: int
    point_list: torch.Tensor   # int32 [capacity] (uint32 bits)
    keys_sorted: torch.Tensor  # int64 [capacity] (uint64 bits)
    tile_ranges: torch.Tensor  # int32 [n_tiles, 2] (uint32 bits)
    image: torch.Tensor        # [3, H, W]
    final_T: torch.Tensor      # [H, W]
    n_contrib: torch.Tensor    # int32 [H, W] (uint32 bits)
    bg: tuple


@dataclasses.dataclass
class Backward:
    dmeans2d: torch.Tensor
    dconic: torch.Tensor
    dopacity: torch.Tensor
    dcolor: torch.Tensor
    dmeans: torch.Tensor
    dscales: torch.Tensor
    dquats: torch.Tensor
    dsh: torch.Tensor | None


class Renderer:
    """Holds the buffers for one camera size and Gaussian count."""

    def __init__(self, camera, n: int, device="cuda", capacity: int | None = None,
                 keep_keys: bool = True, tile_test: int = rs.RS_TILE_TEST_SQUARE):
        self.camera = camera
        self.n = int(n)
        self.device = torch.device(device)
        self.n_tiles = ((camera.width + 15) // 16) * ((camera.height + 15) // 16)
        self.keep_keys = keep_keys
        self.cam_struct = rs.camera_struct(camera)
        self._bound = None
        self.proj = rs.DeviceProjected.empty(self.n, self.device, tile_test)
        H, W = camera.height, camera.width
        self.image = torch.empty(3, H, W, dtype=torch.float32, device=self.device)
        self.final_T = torch.empty(H, W, dtype=torch.float32, device=self.device)
        self.n_contrib = torch.empty(H, W, dtype=torch.int32, device=self.device)
        self.tile_ranges = torch.empty(self.n_tiles, 2, dtype=torch.int32, device=self.device)
        self._alloc(capacity if capacity is not None else max(4096, 16 * self.n))
        self.grads = None

    def _alloc(self, capacity: int):
        self._fwd_valid = False  # new entry buffers: a forward must run before any backward
        self.capacity = int(capacity)
        ws = rs.rs_bin_workspace_size(self.n, self.camera, self.capacity)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=self.device)
        self.point_list = torch.empty(max(self.capacity, 1), dtype=torch.int32, device=self.device)
        self.raster_ws = torch.empty(rs.rs_raster_workspace_size(self.camera, self.capacity), dtype=torch.uint8,
                                     device=self.device)
        self.keys_sorted = (torch.empty(max(self.capacity, 1), dtype=torch.int64, device=self.device)
                            if self.keep_keys else None)

    def set_camera(self, camera):
        assert camera.width == self.camera.width and camera.height == self.camera.height
        self.camera = camera
        rs.set_camera_struct(self.cam_struct, camera)

    # ---- prepared calls: the ctypes arguments of this renderer's buffers, built once
    def _prepare(self, g: rs.DeviceGaussians, bg):
        ptrs = tuple(0 if t is None else t.data_ptr() for t in (g.means, g.scales, g.quats, g.opacity, g.sh, g.colors))
        key = (ptrs, g.n, g.sh_degree, tuple(float(x) for x in bg), self.capacity, self.grads is not None)
        if self._bound is not None and self._bound[0] == key:
            return self._bound[1]
        import ctypes
        cam = ctypes.byref(self.cam_struct)
        gs = g.struct()
        ps = self.proj.struct()
        self._keep = (gs, ps)
        self._E = ctypes.c_size_t(0)
        bgv = (ctypes.c_float * 3)(*[float(x) for x in bg])
        self._bgv = bgv
        vp = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
        self._hres = ctypes.c_void_p(0)  # pinned (E, error) slot of the next rs_bin_async call
        calls = dict(
            project=rs.PreparedCall("rs_project", (cam, ctypes.byref(gs), ctypes.byref(ps))),
            bin_async=rs.PreparedCall("rs_bin_async", (cam, ctypes.byref(ps), self.n, vp(self.workspace),
                                                       self.workspace.numel(), self.capacity, vp(self.keys_sorted),
                                                       vp(self.point_list), vp(self.tile_ranges), self._hres)),
            bin=rs.PreparedCall("rs_bin", (cam, ctypes.byref(ps), self.n, vp(self.workspace),
                                           self.workspace.numel(), self.capacity, vp(self.keys_sorted),
                                           vp(self.point_list), vp(self.tile_ranges), ctypes.byref(self._E))),
            fwd=rs.PreparedCall("rs_rasterize_fwd", (cam, ctypes.byref(ps), self.n, vp(self.tile_ranges),
                                                     vp(self.point_list), self.capacity, bgv, vp(self.image),
                                                     vp(self.final_T), vp(self.n_contrib), vp(self.raster_ws),
                                                     self.raster_ws.numel())))
        if self.grads is not None:
            gr = self.grads
            calls["rbwd_args"] = (cam, ctypes.byref(ps), self.n, vp(self.tile_ranges), vp(self.point_list),
                                  self.capacity, bgv, vp(self.final_T), vp(self.n_contrib),
                                  vp(self.raster_ws), self.raster_ws.numel())
            calls["rbwd_out"] = (vp(gr.dmeans2d), vp(gr.dconic), vp(gr.dopacity), vp(gr.dcolor))
            calls["pbwd"] = rs.PreparedCall("rs_project_bwd", (
                cam, ctypes.byref(gs), ctypes.byref(ps), vp(gr.dmeans2d), vp(gr.dconic), vp(gr.dcolor),
                vp(gr.dmeans), vp(gr.dscales), vp(gr.dquats), vp(gr.dsh)))
        self._bound = (key, calls)
        return calls

    def project(self, g: rs.DeviceGaussians, stream=None):
        self._g = g
        self._prepare(g, getattr(self, "bg", (0.0, 0.0, 0.0)))["project"].run(rs.stream_handle(stream))

    def bin(self, stream=None) -> int:
        h = rs.stream_handle(stream)
        while True:
            try:
                self._prepare(self._g, getattr(self, "bg", (0.0, 0.0, 0.0)))["bin"].run(h)
                return int(self._E.value)
            except rs.RsError as e:
                if e.code != rs.RS_ERR_CAPACITY:
                    raise
                self._alloc(int(self._E.value * 1.25) + 1024)
                self._bound = None

    def bin_async(self, result: torch.Tensor, stream=None):
        """Enqueue the binning without waiting: (E, error flag) land in `result` (pinned int64
        [2]) once the stream gets there.  If E turns out above the capacity, the frame rendered
        the background: grow with `reserve(E)` and redo it."""
        if result.is_cuda or result.dtype != torch.int64 or result.numel() < 2:
            raise TypeError("result must be a pinned int64 host tensor with 2 elements")
        calls = self._prepare(self._g, getattr(self, "bg", (0.0, 0.0, 0.0)))
        self._hres.value = result.data_ptr()
        calls["bin_async"].run(rs.stream_handle(stream))

    def reserve(self, entries: int):
        """Grow the entry buffers to hold at least `entries` entries."""
        if entries > self.capacity:
            self._alloc(int(entries * 1.25) + 1024)
            self._bound = None

    def rasterize(self, bg=(0.0, 0.0, 0.0), stream=None):
        self.bg = tuple(bg)
        self._prepare(self._g, self.bg)["fwd"].run(rs.stream_handle(stream))
        self._fwd_valid = True

    def forward(self, g: rs.DeviceGaussians, bg=(0.0, 0.0, 0.0), stream=None) -> Forward:
        self.bg = tuple(bg)
        self.project(g, stream)
        E = self.bin(stream)
        self.rasterize(bg, stream)
        self.n_entries = E
        return Forward(self.proj, E, self.point_list, self.keys_sorted, self.tile_ranges,
                       self.image, self.final_T, self.n_contrib, self.bg)

    def forward_async(self, g: rs.DeviceGaussians, result: torch.Tensor, bg=(0.0, 0.0, 0.0), stream=None):
        """forward() with the sync-free binning: nothing waits for the entry count, which lands
        in `result` (pinned int64 [2]: E, error flag).  After synchronising, check it with
        `check_async(result)`; a frame whose E exceeded the capacity rendered the background."""
        self.bg = tuple(bg)
        self.project(g, stream)
        self.bin_async(result, stream)
        self.rasterize(bg, stream)

    def check_async(self, result: torch.Tensor) -> int:
        """E of a finished rs_bin_async; raises (after growing the buffers) on overflow or timeout."""
        E, err = int(result[0]), int(result[1])
        if err:
            raise rs.RsError("rs_bin_async", rs.RS_ERR_DEVICE_TIMEOUT, rs.error_string(rs.RS_ERR_DEVICE_TIMEOUT))
        if E > self.capacity:
            self.reserve(E)
            err = rs.RsError("rs_bin_async", rs.RS_ERR_CAPACITY, rs.error_string(rs.RS_ERR_CAPACITY))
            err.n_entries = E
            raise err
        self.n_entries = E
        return E

    def _grads(self, sh_degree: int):
        n, d = self.n, self.device
        K = (sh_degree + 1) ** 2 if sh_degree >= 0 else 0
        if self.grads is None or (self.grads.dsh is None) != (K == 0) or (K and self.grads.dsh.shape[0] != 3 * K):
            f = lambda *s: torch.empty(*s, dtype=torch.float32, device=d)
            self.grads = Backward(f(2, n), f(3, n), f(n), f(3, n), f(3, n), f(3, n), f(4, n),
                                  f(3 * K, n) if K else None)
            self._bound = None  # prepared calls must point at the new gradient buffers
            return True
        return False

    def rasterize_backward(self, dL_dimage, stream=None) -> Backward:
        import ctypes
        if not (dL_dimage.is_cuda and dL_dimage.dtype == torch.float32 and dL_dimage.is_contiguous()
                and dL_dimage.numel() >= 3 * self.camera.width * self.camera.height):
            raise ValueError("dL_dimage must be a contiguous float32 CUDA tensor [3, H, W]")
        if not self._fwd_valid:
            raise RuntimeError("the entry buffers changed since the last forward: run the forward again")
        calls = self._prepare(self._g, self.bg)
        fn = rs.PreparedCall("rs_rasterize_bwd", calls["rbwd_args"] + (ctypes.c_void_p(dL_dimage.data_ptr()),)
                             + calls["rbwd_out"])
        fn.run(rs.stream_handle(stream))
        return self.grads

    def project_backward(self, gs: rs.DeviceGaussians, stream=None) -> Backward:
        self._prepare(gs, self.bg)["pbwd"].run(rs.stream_handle(stream))
        return self.grads

    def backward(self, gs: rs.DeviceGaussians, dL_dimage, stream=None) -> Backward:
        self._grads(gs.sh_degree)
        self.rasterize_backward(dL_dimage, stream)
        return self.project_backward(gs, stream)


class AppearanceStep:
    """The training-shaped step of rigel's appearance-MLP model ("Appearance MLP" and its training
    loop): per view, the MLP gives every Gaussian its colour, the rasteriser renders it, the L1
    loss against the view's target gives dL/dimage, and the backward runs through compositing,
    projection and the MLP.  Every stage is a call of the C ABI; this class only owns buffers.

    `forward` and `backward` are separate so that a caller can inspect or change dL/dimage in
    between; `view` runs both."""

    def __init__(self, camera, g: rs.DeviceGaussians, mlp: rs.DeviceMLP, latents: torch.Tensor,
                 device="cuda", capacity: int | None = None):
        self.device = torch.device(device)
        self.g, self.mlp, self.latents = g, mlp, latents
        n = g.n
        self.R = Renderer(camera, n, self.device, capacity)
        self.colors = torch.empty(3, n, dtype=torch.float32, device=self.device)
        # geometry of g with the MLP's colours as the colour source
        self.gc = rs.DeviceGaussians(g.means, g.scales, g.quats, g.opacity, None, -1, self.colors)
        H, W = camera.height, camera.width
        self.dL_dimage = torch.empty(3, H, W, dtype=torch.float32, device=self.device)
        self.loss = torch.zeros(1, dtype=torch.float32, device=self.device)
        self.dL_dlatents = torch.empty_like(latents)
        self.mlp_grads = rs.DeviceMLPGrads.like(mlp)

    def forward(self, camera, target: torch.Tensor, scale: float, bg=(0.0, 0.0, 0.0), stream=None) -> Forward:
        """MLP colours, render, L1 loss and its gradient (into self.dL_dimage, self.loss)."""
        self.R.set_camera(camera)
        rs.rs_appearance_fwd(camera, self.g.means, self.latents, self.mlp, self.colors, stream)
        F = self.R.forward(self.gc, bg=bg, stream=stream)
        rs.rs_l1_loss_grad(F.image, target, scale, self.dL_dimage, self.loss, stream)
        return F

    def forward_async(self, camera, target: torch.Tensor, scale: float, result: torch.Tensor, bg=(0.0, 0.0, 0.0),
                      stream=None):
        """forward() with the sync-free binning (Renderer.forward_async): nothing waits on the
        host; check the entry count in `result` with self.R.check_async after the stream."""
        self.R.set_camera(camera)
        rs.rs_appearance_fwd(camera, self.g.means, self.latents, self.mlp, self.colors, stream)
        self.R.forward_async(self.gc, result, bg=bg, stream=stream)
        rs.rs_l1_loss_grad(self.R.image, target, scale, self.dL_dimage, self.loss, stream)

    def backward(self, dL_dimage: torch.Tensor | None = None, stream=None) -> Backward:
        """Compositing and projection backward from dL/dimage (default: the L1 gradient), then
        the MLP backward (into self.dL_dlatents and self.mlp_grads)."""
        B = self.R.backward(self.gc, self.dL_dimage if dL_dimage is None else dL_dimage, stream)
        self.mlp_backward(B.dcolor, stream)
        return B

    def mlp_backward(self, dL_dcolor: torch.Tensor, stream=None):
        rs.rs_appearance_bwd(self.R.camera, self.g.means, self.latents, self.mlp, dL_dcolor,
                             self.dL_dlatents, self.mlp_grads, stream)

    def view(self, camera, target, scale, bg=(0.0, 0.0, 0.0), stream=None):
        F = self.forward(camera, target, scale, bg, stream)
        return F, self.backward(stream=stream)


class _Linear:
    """A linear layer's float32 weights [out, in] with their 8-bit form per 128 x 128 block, both ways round."""

    def __init__(self, w: torch.Tensor):
        self.w, self.dw = w, torch.empty_like(w)
        o, i = w.shape
        ob, ib = -(-o // rs.RS_FP8_BLOCK), -(-i // rs.RS_FP8_BLOCK)
        self.q, self.qt = rs.fp8_empty(o, i, w.device)[0], rs.fp8_empty(i, o, w.device)[0]
        self.s = torch.empty(ib, ob, dtype=torch.float32, device=w.device)
        self.st = torch.empty(ob, ib, dtype=torch.float32, device=w.device)
        self.refresh()

    def refresh(self, stream=None):
        rs.rs_quantize_fp8_blocks(self.w, self.q, self.s, self.qt, self.st, stream=stream)


class WideAppearance:
    """A residual appearance network wider than rs_mlp allows: per Gaussian, features [width] -> colour [3],

        h_0 = features;  r_b = relu(norm_b(h_b) W1_b^T) W2_b^T,  h_{b+1} = h_b + r_b;  colour = sigmoid(norm(h_B) Wo^T)

    with root-mean-square norms, every product on 8-bit operands (float32 sums, `dtype` activations) and float32 master
    weights.  `forward` gives the planar colours that rs_project reads when sh_degree is -1, `backward` takes
    the colours' gradient that rs_rasterize_bwd returns, and `step` is one Adam step over all parameters (and the caller's own
    groups) with their gradients clipped to a global norm; nothing in the three waits on the host.

    sandwich: a norm after every block too, and a learned scale a_b [width] of the residual stream,

        h_{b+1} = a_b h_b + g_b norm'_b(r_b),

    with gates g_b = sigmoid(norm_b(h_b) Wg_b^T), one for each Gaussian (gate="row") or for each of its features
    (gate="element"), or 1 (None).

    checkpoints: what the forward keeps for the backward is kept in 8 bits: the norms' and relus' outputs, which the
    products read in that form anyway, and a sandwich block's operands, from which its backward then starts (a block of the
    plain kind keeps its residual stream in `dtype`).  The colours stay the same with float32 activations; in 16 bits the
    hidden layer's are no longer rounded to those before they are to 8."""

    def __init__(self, features: torch.Tensor, hidden: int, blocks: int = 2, dtype=torch.bfloat16, seed: int = 0,
                 sandwich: bool = False, gate: str | None = None, checkpoints: bool = False):
        n, c = features.shape
        if 3 * blocks + 3 > rs.RS_ADAM_MAX_SEGMENTS:
            raise ValueError(f"at most {(rs.RS_ADAM_MAX_SEGMENTS - 3) // 3} blocks")
        if gate not in (None, "row", "element") or (gate and not sandwich):
            raise ValueError("a gate is 'row', 'element' or None, and needs sandwich blocks")
        self.n, self.width, self.hidden, self.dtype = int(n), int(c), int(hidden), dtype
        self.sandwich, self.checkpoints = bool(sandwich), bool(checkpoints)
        self.device = dev = features.device
        g = torch.Generator(dev).manual_seed(seed)
        rand = lambda o, i: torch.randn(o, i, device=dev, generator=g) / i ** 0.5
        self.features, self.dfeatures = features, torch.empty_like(features)
        if sandwich:
            # every vector is a row of one parameter (rows on 16-byte boundaries: the columns past the width stay as they are)
            self.vectors = torch.ones(3 * blocks + 1, -(-c // 4) * 4, device=dev)
            self.dvectors = torch.zeros_like(self.vectors)
            split = lambda t: (lambda r: (r[:blocks + 1], r[blocks + 1:2 * blocks + 1], r[2 * blocks + 1:]))(
                [row[:c] for row in t])
            (self.norms, self.posts, self.scales), (self.dnorms, self.dposts, self.dscales) = map(
                split, (self.vectors, self.dvectors))
        else:
            self.norms = [torch.ones(c, device=dev) for _ in range(blocks + 1)]
            self.dnorms = [torch.empty(c, device=dev) for _ in range(blocks + 1)]
        self.up = [_Linear(rand(hidden, c)) for _ in range(blocks)]
        self.down = [_Linear(rand(c, hidden)) for _ in range(blocks)]
        self.head = _Linear(rand(3, c))
        gates = {None: 0, "row": 1, "element": c}[gate]
        elements = gates > 1  # one column is a gate a row
        self.gates = [_Linear(rand(gates, c)) for _ in range(blocks)] if gate else [None] * blocks
        e = lambda r, k, d=dtype: torch.empty(r, k, dtype=d, device=dev)
        q8 = lambda r, k: rs.fp8_empty(r, k, dev)
        # kept for the backward: each norm's input sum, output and statistic, each relu's output; of a sandwich block also
        # its result, its gate and their statistic
        fewer = checkpoints and sandwich
        self.h = [e(n, c)] * (blocks + 1) if fewer else [e(n, c) for _ in range(blocks + 1)]
        self.rstd = [torch.empty(n, dtype=torch.float32, device=dev) for _ in range(blocks + 1)]
        if checkpoints:
            self.yq, self.uq = [q8(n, c) for _ in range(blocks + 1)], [q8(n, hidden) for _ in range(blocks)]
        else:
            self.y, self.u = [e(n, c) for _ in range(blocks + 1)], [e(n, hidden) for _ in range(blocks)]
        if sandwich:
            self.rstd_r = [torch.empty(n, dtype=torch.float32, device=dev) for _ in range(blocks)]
            self.results = [e(n, c)] * blocks if fewer else [e(n, c) for _ in range(blocks)]
            self.zs = [None] * blocks
            if gate:
                self.zs = [e(n, gates)] * blocks if fewer and elements else [e(n, gates) for _ in range(blocks)]
            if fewer:
                kept = ("x", "r") + (("gate",) if elements else ())
                self.kept = [{k: q8(n, c) for k in kept} for _ in range(blocks)]
        # scratch: 8-bit operands by rows and by columns, gradients, results of products
        self.qc, self.qct = q8(n, c), q8(c, n)
        self.qh, self.qht = q8(n, hidden), q8(hidden, n)
        self.q3, self.q3t = q8(n, 3), q8(3, n)
        self.dh, self.dy, self.du = e(n, c), e(n, c), e(n, hidden)
        if not sandwich:
            self.r = e(n, c)
        else:
            self.dr = e(n, c)
            if gate:
                self.dgate, self.qg, self.qgt = e(n, gates), q8(n, gates), q8(gates, n)
        self.z = torch.empty(n, 3, dtype=torch.float32, device=dev)
        self.colors = torch.empty(3, n, dtype=torch.float32, device=dev)
        sizes = [(n, hidden, c), (n, c, hidden), (n, 3, c), (n, c, 3), (hidden, c, n), (c, hidden, n), (3, c, n)]
        if gate:
            sizes += [(n, gates, c), (n, c, gates), (gates, c, n), (c, gates, n)]
        need = max([rs.rs_matmul_fp8_workspace_size(*s) for s in sizes] +
                   [rs.rs_rms_norm_bwd_workspace_size(n, c), rs.rs_grad_norm_workspace_size(rs.RS_ADAM_MAX_SEGMENTS)])
        if checkpoints:
            need = max(need, rs.rs_matmul_fp8_q_workspace_size(n, hidden, c))
        if sandwich:
            need = max(need, rs.rs_sandwich_norm_bwd_workspace_size(n, c))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)
        self.moments = None
        self.steps = torch.zeros(1, dtype=torch.int32, device=dev)  # taken so far: skipped ones do not count

    def kept_bytes(self) -> int:
        """Bytes of the matrices that hold activations from the forward on (what blocks share counts once)."""
        blocks = len(self.up)
        rows = [*self.h[:blocks + 1], *self.rstd]
        rows += [t for pair in (*self.yq, *self.uq) for t in pair] if self.checkpoints else [*self.y, *self.u]
        if self.sandwich:
            rows += [*self.rstd_r, *self.results, *(z for z in self.zs if z is not None)]
            rows += [t for k in getattr(self, "kept", ()) for pair in k.values() for t in pair]
        return sum({t.data_ptr(): t.numel() * t.element_size() for t in rows}.values())

    def _product(self, a, b, b_scales, out, relu=False):
        rs.rs_matmul_fp8(*a, b, b_scales, out, self.workspace, relu=relu)

    def _hidden(self, b, y):
        """The relu of block b's first layer in 8 bits, the second layer's operand, from the norm's output."""
        up = self.up[b]
        if self.checkpoints:
            rs.rs_matmul_fp8_q(*y, up.q, up.s, *self.uq[b], self.workspace, relu=True)
            return self.uq[b]
        self._product(y, up.q, up.s, self.u[b], relu=True)
        rs.rs_quantize_fp8(self.u[b], *self.qh)
        return self.qh

    def forward(self, stream=None) -> torch.Tensor:
        """colours [3, n] (planar) of the features and weights as they are."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.device)):
            x, residual, last = self.h[0], None, len(self.up)
            x.copy_(self.features)
            y = lambda b: self.yq[b] if self.checkpoints else self.qc
            wide = lambda b: None if self.checkpoints else self.y[b]
            for b in range(last + 1):
                if b == 0 or not self.sandwich:
                    rs.rs_rms_norm_fwd(x, self.norms[b], *y(b), residual=residual, sum=self.h[b] if b else None,
                                       y=wide(b), rstd=self.rstd[b])
                if b == last:
                    break
                r = self.results[b] if self.sandwich else self.r
                self._product(self._hidden(b, y(b)), self.down[b].q, self.down[b].s, r)
                if self.sandwich:
                    if self.gates[b]:
                        self._product(y(b), self.gates[b].q, self.gates[b].s, self.zs[b])
                    kept = {f"kept_{k}": v for k, v in self.kept[b].items()} if self.checkpoints else {}
                    rs.rs_sandwich_norm_fwd(x, r, self.posts[b], self.norms[b + 1], *y(b + 1), gate=self.zs[b],
                                            residual_scale=self.scales[b], sum=self.h[b + 1], y=wide(b + 1),
                                            rstd_r=self.rstd_r[b], rstd_s=self.rstd[b + 1], **kept)
                    x = self.h[b + 1]
                else:
                    x, residual = self.h[b], self.r
            self._product(y(last), self.head.q, self.head.s, self.z)
            torch.sigmoid(self.z.t(), out=self.colors)
        return self.colors

    def _weight_grad(self, grad_t, x, scratch_t, layer):
        """layer.dw = grad^T x, both in 8 bits by columns; x a matrix, or one kept in 8 bits by rows."""
        if type(x) is tuple:
            rs.rs_transpose_fp8(*x, *scratch_t)
        else:
            rs.rs_quantize_fp8(x, qt=scratch_t[0], scales_t=scratch_t[1])
        self._product(grad_t, *scratch_t, layer.dw)

    @staticmethod
    def _powers(x):
        """The power of two that brings the largest |x| into [0.5, 1), and its inverse, float32 [1] on the device."""
        e = torch.frexp(x.abs().amax().view(1)).exponent.clamp(-125, 125)  # any in range will do where it is not finite
        return ((127 - e) << 23).view(torch.float32), ((127 + e) << 23).view(torch.float32)

    def backward(self, dL_dcolors: torch.Tensor, stream=None):
        """Gradients of every weight (dnorms, the layers' dw; of sandwich blocks dposts and dscales) and of the features from
        dL/dcolours [3, n].

        float16 activations hold nothing much below 6e-8, and a loss over an image has gradients of that size: between the
        layers they then carry a power of two, exact in every step, that is taken out of what leaves."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.device)):
            dz = (dL_dcolors * self.colors * (1 - self.colors)).t().contiguous()
            last = len(self.up)
            undo, down = lambda t: t, None
            if self.dtype is torch.float16 and self.n > 0:
                up, down = self._powers(dz)
                dz.mul_(up)
                undo = lambda t: t.mul_(down)
            y, u = (self.yq, self.uq) if self.checkpoints else (self.y, self.u)
            rs.rs_quantize_fp8(dz, *self.q3, *self.q3t)
            undo(self.q3t[1])  # a weight's gradient takes it out with the scales of the gradient's transposed form
            self._weight_grad(self.q3t, y[last], self.qct, self.head)
            self._product(self.q3, self.head.qt, self.head.st, self.dy)
            if not self.sandwich:
                self._norm_backward(last, self.h[last], None, undo)
            for b in reversed(range(last)):
                dr = self.dh
                if self.sandwich:
                    dr = self.dr
                    self._sandwich_backward(b, undo)
                # without one, dh is the gradient of h_{b+1} = h_b + r_b: of r_b as it is, of h_b with what comes through the
                # block
                rs.rs_quantize_fp8(dr, *self.qc, *self.qct)
                undo(self.qct[1])
                self._weight_grad(self.qct, u[b], self.qht, self.down[b])
                self._product(self.qc, self.down[b].qt, self.down[b].st, self.du)
                if self.checkpoints:
                    rs.rs_quantize_fp8_relu8(self.du, u[b][0], *self.qh, *self.qht)
                else:
                    rs.rs_quantize_fp8(self.du, *self.qh, *self.qht, relu=u[b])
                undo(self.qht[1])
                self._weight_grad(self.qht, y[b], self.qct, self.up[b])
                self._product(self.qh, self.up[b].qt, self.up[b].st, self.dy)
                if self.gates[b]:
                    # the block's norm feeds its gate too; dr has been read
                    rs.rs_quantize_fp8(self.dgate, *self.qg, *self.qgt)
                    undo(self.qgt[1])
                    self._product(self.qg, self.gates[b].qt, self.gates[b].st, self.dr)
                    self.dy.add_(self.dr)
                    dw = self.gates[b].dw  # qct still holds the norm's output by columns
                    if dw.shape[0] == 1:  # as a column of many rows: one row's long contraction would run on few SMs
                        self._product(self.qct, *self.qgt, dw.view(-1, 1))
                    else:
                        self._product(self.qgt, *self.qct, dw)
                if not self.sandwich:
                    self._norm_backward(b, self.h[b], self.dh, undo)
            if self.sandwich:
                x = self.h[0]
                if self.checkpoints:  # the stream has moved on, and is not read again: the features once more
                    x.copy_(self.features)
                self._norm_backward(0, x, self.dh if last else None, undo)
            if down is None:
                self.dfeatures.copy_(self.dh)
            else:
                torch.mul(self.dh, down, out=self.dfeatures)  # in float32: down is a tensor of one dimension

    def _norm_backward(self, b, x, dsum, undo):
        rs.rs_rms_norm_bwd(x, self.norms[b], self.rstd[b], self.dy, self.dh, self.dnorms[b], self.workspace, dL_dsum=dsum)
        undo(self.dnorms[b])

    def _sandwich_backward(self, b, undo):
        """From dy and dh (the gradient of h_{b+1} by its later uses) to dr, dh of h_b's direct use and the gate's gradient."""
        kept = self.kept[b] if self.checkpoints else {"x": self.h[b], "r": self.results[b]}
        rs.rs_sandwich_norm_bwd(
            kept["x"], kept["r"], self.posts[b], self.norms[b + 1], self.rstd_r[b], self.rstd[b + 1], self.dy, self.dh,
            self.dr, self.workspace, gate=kept.get("gate", self.zs[b]), dL_dgate=self.dgate if self.gates[b] else None,
            residual_scale=self.scales[b], dL_dsum=self.dh if b + 1 < len(self.up) else None,
            dL_dpost_weight=self.dposts[b], dL_dpre_weight=self.dnorms[b + 1], dL_dresidual_scale=self.dscales[b])
        for t in (self.dposts[b], self.dnorms[b + 1], self.dscales[b]):
            undo(t)

    def _layers(self):
        return [l for l in (*self.up, *self.down, *self.gates, self.head) if l is not None]

    def parameters(self):
        """(parameter, gradient) of every group: the features, the norms (of a sandwich network all vectors as one), the
        layers."""
        vectors = [(self.vectors, self.dvectors)] if self.sandwich else list(zip(self.norms, self.dnorms))
        return [(self.features, self.dfeatures)] + vectors + [(l.w, l.dw) for l in self._layers()]

    def step(self, max_norm: float, lr: float = 1e-3, groups=(), stream=None):
        """One clipped Adam step over the network and `groups` (rs.AdamGroup, e.g. the geometry's); the norm before
        clipping is in self.norm.  In a captured step `lr`, `max_norm` and the groups' rates are those of the capture; the
        step's number is counted on the device."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.device)):
            if self.moments is None:
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("the moments have to exist before a step is captured (each replay would begin with "
                                       "zeros): take one step first")
                self.moments = [(torch.zeros_like(p), torch.zeros_like(p)) for p, _ in self.parameters()]
            own = [rs.AdamGroup(p, g, m, v, lr) for (p, g), (m, v) in zip(self.parameters(), self.moments)]
            rs.rs_adam_step_clipped([*own, *groups], self.steps, max_norm, self.norm, self.workspace)
            for layer in self._layers():
                layer.refresh()


class AppearanceGraph:
    """One view of the training-shaped step (MLP colours, render, L1 loss, render backward, MLP
    backward) captured as a single CUDA graph, like FrameGraph: the camera is fixed, the
    latents, weights, Gaussians and target are read from their buffers at every replay, and
    `check()` (after the stream has passed the replay) returns the entry count."""

    def __init__(self, step: AppearanceStep, camera, target: torch.Tensor, scale: float, bg=(0.0, 0.0, 0.0)):
        self.step, self.camera = step, camera
        self.result = torch.zeros(2, dtype=torch.int64).pin_memory()
        R = step.R
        R._grads(-1)
        step.forward_async(camera, target, scale, self.result, bg)
        step.backward()
        torch.cuda.current_stream(R.device).synchronize()
        R.check_async(self.result)
        self.capacity = R.capacity
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            step.forward_async(camera, target, scale, self.result, bg)
            step.backward()

    def replay(self):
        if self.step.R.capacity != self.capacity:
            raise RuntimeError("the renderer's buffers changed since the capture")
        self.graph.replay()

    def check(self) -> int:
        return self.step.R.check_async(self.result)


class FrameGraph:
    """One view's forward and backward captured as a single CUDA graph and replayed.

    Every call of the frame is stream-ordered with no host wait (the binning's entry count is
    copied to pinned host memory in stream order, `rs_bin_async`), so projection, binning,
    compositing and both backward passes fit in one graph launch -- the sync-free, graph-captured
    pipeline that "3D Gaussian Splatting ビューワを作る" (4.2-4.3, indirect dispatch) and the rigel
    README ("Binning", the one device-to-host sync) point to.  The kernels take the camera by
    value, so a graph belongs to one view (`FrameGraphs` keeps one per view).  A replay reads the
    Gaussians and dL/dimage from the buffers given at capture and writes the renderer's buffers.
    `check()` (after the stream has passed the replay) returns the entry count and raises when
    it exceeded the capacity: that frame rendered the background, the renderer has grown and the
    graph must be captured again."""

    def __init__(self, R: Renderer, gs: rs.DeviceGaussians, dL_dimage: torch.Tensor, camera,
                 bg=(0.0, 0.0, 0.0)):
        self.R, self.camera, self.bg = R, camera, tuple(bg)
        self.result = torch.zeros(2, dtype=torch.int64).pin_memory()
        R.set_camera(camera)
        R._grads(gs.sh_degree)
        # one eager frame: builds the prepared calls and checks that the buffers are big enough
        R.forward_async(gs, self.result, bg)
        R.backward(gs, dL_dimage)
        torch.cuda.current_stream(R.device).synchronize()
        R.check_async(self.result)
        self.capacity = R.capacity
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            R.forward_async(gs, self.result, bg)
            R.backward(gs, dL_dimage)

    def replay(self):
        if self.R.capacity != self.capacity:
            raise RuntimeError("the renderer's buffers changed since the capture")
        self.graph.replay()

    def check(self) -> int:
        return self.R.check_async(self.result)


class FrameGraphs:
    """One `FrameGraph` per view of a fixed camera list, captured on first use."""

    def __init__(self, R: Renderer, gs: rs.DeviceGaussians, dL_dimage: torch.Tensor, cameras,
                 bg=(0.0, 0.0, 0.0)):
        self.R, self.gs, self.dL, self.cameras, self.bg = R, gs, dL_dimage, list(cameras), tuple(bg)
        self.graphs: dict[int, FrameGraph] = {}

    def get(self, view: int) -> FrameGraph:
        fg = self.graphs.get(view)
        if fg is None or fg.capacity != self.R.capacity:
            fg = FrameGraph(self.R, self.gs, self.dL, self.cameras[view], self.bg)
            self.graphs[view] = fg
        return fg


class StreamedFrames:
    """Forward + backward of a sequence of views whose Gaussian parameters and dL/dimage come
    from pinned host memory and whose per-Gaussian gradients go back to pinned host memory, with
    the copies of one frame overlapping the compute of its neighbours.

    `slots` slots (at least two), each a renderer with its own device inputs, gradients,
    per-view frame graphs and compute stream, take the frames in turn.  Frame k's host-to-device
    copies run on an input copy stream once frame k - slots (same slot) has finished reading its
    inputs; its graph replays on its slot's compute stream once those copies and frame
    k - slots' device-to-host copies are done; its gradients go back on an output copy stream
    once it has finished.  So the two copy directions and the compute of neighbouring frames
    proceed at once (one frame's latency-bound binning overlaps another's compositing), and a
    step costs about the longest of them.

    `host_in`: pinned float32 tensors means [3,N], scales [3,N], quats [4,N], opacity [N] and
    sh [3K,N] (or colors [3,N] with sh_degree -1); `host_dL`: pinned [3,H,W].  `host_out[slot]`
    receives dmeans, dscales, dquats, dopacity, dsh (or dcolor) of that slot's frames."""

    OUT = ("dmeans", "dscales", "dquats", "dopacity")

    def __init__(self, cameras, host_in: dict, sh_degree: int, host_dL: torch.Tensor, device="cuda",
                 capacity: int | None = None, bg=(0.0, 0.0, 0.0), slots: int = 2):
        self.device = torch.device(device)
        self.cameras = list(cameras)
        self.host_in, self.host_dL, self.sh_degree = host_in, host_dL, sh_degree
        n = int(host_in["opacity"].shape[0])
        self.out_names = self.OUT + (("dsh",) if sh_degree >= 0 else ("dcolor",))
        self.slots = []
        self.n_slots = max(2, int(slots))
        for _ in range(self.n_slots):
            R = Renderer(self.cameras[0], n, self.device, capacity=capacity, keep_keys=False)
            dev = {k: torch.empty_like(v, device=self.device) for k, v in host_in.items()}
            if sh_degree >= 0:
                dg = rs.DeviceGaussians(dev["means"], dev["scales"], dev["quats"], dev["opacity"], dev["sh"],
                                        sh_degree)
            else:
                dg = rs.DeviceGaussians(dev["means"], dev["scales"], dev["quats"], dev["opacity"], None, -1,
                                        dev["colors"])
            ddL = torch.empty_like(host_dL, device=self.device)
            R._grads(sh_degree)
            host_out = {k: torch.empty(tuple(getattr(R.grads, k).shape), dtype=torch.float32).pin_memory()
                        for k in self.out_names}
            ev = lambda: torch.cuda.Event()
            self.slots.append(dict(R=R, dev=dev, dg=dg, ddL=ddL, host_out=host_out,
                                   graphs=FrameGraphs(R, dg, ddL, self.cameras, bg), in_ready=ev(),
                                   comp_done=ev(), out_done=ev(), frames=[]))
        self.compute = [torch.cuda.Stream(self.device) for _ in self.slots]
        self.h2d = torch.cuda.Stream(self.device)
        self.d2h = torch.cuda.Stream(self.device)
        self.k = 0

    @property
    def host_out(self):
        return [s["host_out"] for s in self.slots]

    def prepare(self, views):
        """Captures the frame graphs of `views` in both slots (each capture runs one frame)."""
        cur = torch.cuda.current_stream(self.device)
        for s in self.slots:
            for v in sorted(set(views)):
                self._copy_in(s)
                cur.wait_event(s["in_ready"])
                s["graphs"].get(v)
        torch.cuda.synchronize(self.device)

    def _copy_in(self, s):
        with torch.cuda.stream(self.h2d):
            self.h2d.wait_event(s["comp_done"])  # the slot's previous frame has read its inputs
            for k, v in self.host_in.items():
                s["dev"][k].copy_(v, non_blocking=True)
            s["ddL"].copy_(self.host_dL, non_blocking=True)
            s["in_ready"].record(self.h2d)

    def frame(self, view: int):
        """Enqueues one frame of `view`; nothing waits on the host."""
        slot = self.k % self.n_slots
        s, cs = self.slots[slot], self.compute[slot]
        self.k += 1
        fg = s["graphs"].get(view)  # captured already after prepare(); else captured here
        self._copy_in(s)
        cs.wait_event(s["in_ready"])
        cs.wait_event(s["out_done"])  # the slot's previous gradients are on the host
        with torch.cuda.stream(cs):
            fg.replay()
        s["comp_done"].record(cs)
        with torch.cuda.stream(self.d2h):
            self.d2h.wait_event(s["comp_done"])
            for k in self.out_names:
                s["host_out"][k].copy_(getattr(s["R"].grads, k), non_blocking=True)
            s["out_done"].record(self.d2h)
        s["frames"].append(fg)

    def finish(self) -> list[int]:
        """Waits for every enqueued frame; returns their entry counts (raises on an overflow)."""
        torch.cuda.synchronize(self.device)
        counts = []
        for s in self.slots:
            counts += [fg.check() for fg in s["frames"]]
            s["frames"].clear()
        return counts
