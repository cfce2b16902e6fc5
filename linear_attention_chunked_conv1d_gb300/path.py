"""One prefill pass of a GDN/KDA layer's hot path through the C ABI.

Order of the steps as on "glm5next_kda/prefill.rs" (Glm5NextKdaLayer::prefill_with_pad_fill)
and "split_prefill.rs" (prefill_phase1_conv1d_one per request, prefill_phase1_l2_batched, then
prefill_gdn_full_batched when all streams have one length, else the varlen call):

    conv1d + SiLU (per stream, carried conv state)  ->  L2 over the q|k heads  ->  recurrence

With bf16 activations and head dim 128 the whole pass is one launch (`fused`, the library's
la_prefill_front): the tensor-core recurrence computes its q, k, v tiles from the pre-conv rows
itself. Otherwise (and in `run_unfused`) the packed front-end output
[tokens][q heads | k heads | v heads] is handed to the recurrence as three strided views
(q, k, v), which is all the pages' split_widen step amounts to here.
This module only sequences the library calls; it holds no arithmetic.
"""
from __future__ import annotations

import math

import torch

from . import (LA_W4_MAX_ROWS, conv1d_silu_backward, conv1d_silu_backward_workspace_bytes, conv1d_silu_l2_prefill,
               conv1d_silu_prefill, conv1d_silu_prefill_varlen, decode_step,
               decode_workspace_bytes, gate_activations, gated_scan, gated_scan_backward,
               gated_scan_saved_bytes, gated_scan_step, gated_scan_workspace_bytes,
               gdn_prefill_batched, gdn_prefill_varlen, gemm_bf16, kda_prefill, l2norm_heads,
               pointer_array, prefill_front, prefill_segmented, prefill_segmented_workspace_bytes,
               prefill_workspace_bytes, rmsnorm_rows, w4_matvec, _on_stream)


class PrefillPass:
    """Buffers and state pointers for repeated passes over one packed batch on one device.

    `inputs` holds device tensors: x [T][cd], conv_w [cd][K], conv_state [B][K-1][cd],
    h [B][Hv][d][d] (fp32), g, beta, cu_seqlens, plus `lengths` (host list)."""

    def __init__(self, wl, inputs: dict, *, eps: float = 1e-6, pad_fill: float = 0.0):
        self.wl = wl
        self.inp = inputs
        self.eps = eps
        self.pad_fill = pad_fill
        x = inputs["x"]
        self.T = x.shape[0]
        self.lengths = list(inputs["lengths"])
        self.max_seqlen = max(self.lengths)
        dev = x.device
        self.conv_out = torch.empty_like(x)
        self.out = torch.empty(self.T, wl.Hv, wl.d, dtype=x.dtype, device=dev)
        B = wl.B
        self.conv_state_ptrs = pointer_array([inputs["conv_state"][s] for s in range(B)])
        self.h_ptrs = pointer_array([inputs["h"][s] for s in range(B)])
        nbytes = prefill_workspace_bytes(B, self.T, wl.Hk, wl.Hv, wl.d, wl.d, x.dtype)
        self.workspace = (torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes
                          else None)
        hk = wl.Hk * wl.d
        self.q = self.conv_out[:, :hk]
        self.k = self.conv_out[:, hk:2 * hk]
        self.v = self.conv_out[:, 2 * hk:]
        self.scale = 1.0 / math.sqrt(wl.d)
        self.can_fuse = x.dtype == torch.bfloat16 and wl.d == 128

    def front_end(self, stream=None):
        """conv1d + SiLU and the q|k L2 norm in one fused launch (bitwise equal to the two)."""
        wl, inp = self.wl, self.inp
        conv1d_silu_l2_prefill(self.conv_state_ptrs, inp["x"], inp["conv_w"], self.conv_out,
                               None if wl.B == 1 else inp["cu_seqlens"], l2_heads=2 * wl.Hk,
                               head_dim=wl.d, eps=self.eps, stream=stream)

    def front_end_unfused(self, stream=None):
        """The pages' two launches: conv_prefill, then l2 in place over q|k."""
        wl, inp = self.wl, self.inp
        if wl.B == 1:
            conv1d_silu_prefill(inp["conv_state"][0], inp["x"], inp["conv_w"], self.conv_out,
                                stream=stream)
        else:
            conv1d_silu_prefill_varlen(self.conv_state_ptrs, inp["x"], inp["conv_w"],
                                       self.conv_out, inp["cu_seqlens"], stream=stream)
        l2norm_heads(self.conv_out, 2 * wl.Hk, wl.d, eps=self.eps, stream=stream)

    def recurrence(self, stream=None):
        wl, inp = self.wl, self.inp
        d = wl.d
        common = dict(Hk=wl.Hk, Hv=wl.Hv, dk=d, dv=d, scale=self.scale, workspace=self.workspace,
                      stream=stream)
        if wl.variant == "kda":
            kda_prefill(self.h_ptrs, self.q, self.k, self.v, inp["g"], inp["beta"], self.out,
                        None if wl.B == 1 else inp["cu_seqlens"], max_seqlen=self.max_seqlen,
                        pad_fill=self.pad_fill, **common)
        elif wl.batched:
            gdn_prefill_batched(self.h_ptrs, self.q, self.k, self.v, inp["g"], inp["beta"],
                                self.out, B=wl.B, T=self.lengths[0], **common)
        else:
            gdn_prefill_varlen(self.h_ptrs, self.q, self.k, self.v, inp["g"], inp["beta"],
                               self.out, inp["cu_seqlens"], max_seqlen=self.max_seqlen, **common)

    def recurrence_segmented(self, segments, stream=None):
        """The recurrence of a single stream as a chunk-parallel scan (la_prefill_segmented)."""
        wl, inp = self.wl, self.inp
        assert wl.B == 1, "the segmented scan covers one stream"
        nbytes = prefill_segmented_workspace_bytes(self.T, wl.Hv, segments)
        if getattr(self, "_seg_ws", None) is None or self._seg_ws.numel() < nbytes:
            self._seg_ws = torch.empty(nbytes, dtype=torch.uint8, device=self.out.device)
        prefill_segmented(self.h_ptrs, self.q, self.k, self.v, inp["g"], inp["beta"], self.out,
                          Hk=wl.Hk, Hv=wl.Hv, dk=wl.d, dv=wl.d, kda=wl.variant == "kda",
                          segments=segments, scale=self.scale, workspace=self._seg_ws,
                          stream=stream)

    def fused(self, stream=None):
        """conv1d + SiLU + L2 + recurrence in one launch (bf16, head dim 128)."""
        wl, inp = self.wl, self.inp
        prefill_front(self.conv_state_ptrs, self.h_ptrs, inp["x"], inp["conv_w"], inp["g"],
                      inp["beta"], self.out, None if wl.batched or wl.B == 1 else inp["cu_seqlens"],
                      B=wl.B, Hk=wl.Hk, Hv=wl.Hv, dk=wl.d, dv=wl.d, kda=wl.variant == "kda",
                      max_seqlen=self.max_seqlen, l2_eps=self.eps, scale=self.scale,
                      pad_fill=self.pad_fill, workspace=self.workspace, stream=stream)

    def run_unfused(self, stream=None):
        self.front_end(stream)
        self.recurrence(stream)
        return self.out

    def run(self, stream=None):
        if self.can_fuse:
            self.fused(stream)
            return self.out
        return self.run_unfused(stream)


class DecodeStep:
    """One decode step of a GDN/KDA layer for B streams (one new token each) on one device,
    through la_decode_step. `inputs` as for PrefillPass, with x [B][cd] (row s = stream s)."""

    def __init__(self, wl, inputs: dict, *, eps: float = 1e-6):
        self.wl = wl
        self.inp = inputs
        self.eps = eps
        x = inputs["x"]
        B = wl.B
        assert x.shape[0] == B, "a decode step takes one token per stream"
        dev = x.device
        self.out = torch.empty(B, wl.Hv, wl.d, dtype=x.dtype, device=dev)
        self.conv_state_ptrs = pointer_array([inputs["conv_state"][s] for s in range(B)])
        self.h_ptrs = pointer_array([inputs["h"][s] for s in range(B)])
        nbytes = decode_workspace_bytes(B, wl.Hk, wl.Hv, wl.d, wl.d, x.dtype)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.scale = 1.0 / math.sqrt(wl.d)

    def run(self, stream=None):
        wl, inp = self.wl, self.inp
        decode_step(self.conv_state_ptrs, self.h_ptrs, inp["x"], inp["conv_w"], inp["g"],
                    inp["beta"], self.out, Hk=wl.Hk, Hv=wl.Hv, dk=wl.d, dv=wl.d,
                    kda=wl.variant == "kda", l2_eps=self.eps, scale=self.scale,
                    workspace=self.workspace, stream=stream)
        return self.out


def project(y, w, out=None, stream=None):
    """y W^T for a linear layer's weight: bf16 [out][in], or the pair (q, scales) of w4_quantize (then
    at most LA_W4_MAX_ROWS rows)."""
    if isinstance(w, torch.Tensor):
        return gemm_bf16(y, w, out, stream=stream)
    q, scales = w
    return w4_matvec(y, q, scales, out, stream=stream)


def _outputs(w) -> int:
    return (w if isinstance(w, torch.Tensor) else w[0]).shape[0]


class Phase1:
    """Phase 1 of a layer over the stacked hidden rows ("split_prefill.rs",
    prefill_phase1_proj_batched: norm, QKVZ, gates), through the library:
    rmsnorm_rows -> three projection GEMMs (q|k|v, z, gate pre-activations a|b) -> gate
    activations. Weights are the caller's ([out][in] bf16, or the 4-bit (q, scales) of w4_quantize
    for the few rows of a decode step); outputs are device tensors: x [t][cd] (the conv input),
    z [t][Hv*dv], g (fp32 [t][Hv] or [t][Hv*dk]), beta [t][Hv]."""

    def __init__(self, wl, norm_w, w_qkv, w_z, w_ab, *, eps=1e-6):
        self.wl, self.norm_w, self.w_qkv, self.w_z, self.w_ab, self.eps = (
            wl, norm_w, w_qkv, w_z, w_ab, eps)
        self.na = wl.Hv * (wl.d if wl.variant == "kda" else 1)

    def run(self, hidden, stream=None):
        y = rmsnorm_rows(hidden, self.norm_w, eps=self.eps, stream=stream)
        x = project(y, self.w_qkv, stream=stream)
        z = project(y, self.w_z, stream=stream)
        n_ab = _outputs(self.w_ab)  # rows padded to 16 bytes (the GEMM's output stride rule)
        ab = torch.empty(y.shape[0], (n_ab + 7) // 8 * 8, dtype=y.dtype, device=y.device)[:, :n_ab]
        project(y, self.w_ab, ab, stream=stream)
        g, beta = gate_activations(ab, self.na, stream=stream)
        return dict(y=y, x=x, z=z, ab=ab, g=g, beta=beta)


class StreamedPrefill:
    """Prefill steps fed from pinned host memory and read back to it, pipelined over three
    streams: the host->device copy of step i+1 and the device->host copy of step i-1 overlap
    the compute of step i. Two sets of device inputs and outputs alternate; the carried conv and
    h states are shared and advance in step order on the compute stream.

    `mode`: "split" (fused conv+L2, then the recurrence), "fused" (la_prefill_front) or "seg"
    (fused conv+L2, then the segmented recurrence with `segments` pieces, one stream)."""

    def __init__(self, wl, inputs: dict, *, mode="split", segments=1, compute_stream=None):
        self.mode, self.segments = mode, segments
        dev = inputs["x"].device
        self.passes = []
        for _ in range(2):
            inp = dict(inputs)
            for name in ("x", "g", "beta"):
                inp[name] = torch.empty_like(inputs[name])
            self.passes.append(PrefillPass(wl, inp))
        self.compute = compute_stream or torch.cuda.current_stream(dev)
        self.copy_in = torch.cuda.Stream(dev)
        self.copy_out = torch.cuda.Stream(dev)
        self.copied = [torch.cuda.Event() for _ in range(2)]
        self.computed = [torch.cuda.Event() for _ in range(2)]
        self.drained = [torch.cuda.Event() for _ in range(2)]

    def _run(self, p):
        if self.mode == "fused":
            p.fused(self.compute)
        elif self.mode == "seg":
            p.front_end(self.compute)
            p.recurrence_segmented(self.segments, self.compute)
        else:
            p.run_unfused(self.compute)

    def step(self, i, x_h, g_h, beta_h, out_h):
        """Step i: inputs from the pinned host tensors, the output into out_h (all queued)."""
        b = i % 2
        p = self.passes[b]
        with torch.cuda.stream(self.copy_in):
            self.copy_in.wait_event(self.computed[b])  # step i-2 is done with these inputs
            p.inp["x"].copy_(x_h, non_blocking=True)
            p.inp["g"].copy_(g_h, non_blocking=True)
            p.inp["beta"].copy_(beta_h, non_blocking=True)
            self.copied[b].record(self.copy_in)
        self.compute.wait_event(self.copied[b])
        self.compute.wait_event(self.drained[b])  # step i-2's output has been read back
        self._run(p)
        self.computed[b].record(self.compute)
        with torch.cuda.stream(self.copy_out):
            self.copy_out.wait_event(self.computed[b])
            out_h.copy_(p.out, non_blocking=True)
            self.drained[b].record(self.copy_out)

    def start(self, event):
        """Make every stream of the pipeline start after `event` (recorded by the caller)."""
        for st in (self.compute, self.copy_in, self.copy_out):
            st.wait_event(event)

    def finish(self):
        """Make the compute stream wait for the last copies back (then record on it)."""
        self.compute.wait_event(self.drained[0])
        self.compute.wait_event(self.drained[1])


def _fits(name, t, shape, dtype, dev, *, rows=False):
    """Refuses a tensor that a gated layer's kernels would read or write past or misread. rows: the first
    dimension may have any stride of whole 16 bytes; the rest is dense."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != dev:
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected {tuple(shape)} {dtype} on {dev}")
    dense = t[0] if rows and t.shape[0] else t
    if not dense.is_contiguous() or t.data_ptr() % 16 or (dense is not t and t.shape[0] > 1
                                                          and t.stride(0) * t.element_size() % 16):
        raise ValueError(f"{name}: strides {t.stride()} at {t.data_ptr():#x}, expected dense "
                         f"{'rows' if rows else 'values'} on 16-byte boundaries")


class GatedPass:
    """Repeated passes of a gated recurrent layer (one state per channel) over one packed batch:
    conv1d + SiLU over the carried windows, then the gated scan from the carried states.

    `inputs` holds device tensors: x [T][C] (before the conv) and ab [T][2C] (gate rows a | b),
    conv_w [C][K], conv_bias [C] or None, conv_state [B][K-1][C], h [B][C] (fp32; each stream's state
    dense), cu_seqlens [B+1] (int32).
    forward() advances both states; with train=True it also keeps what backward() needs: the
    conv states as they were, and the scan's saved states. Outputs and gradients are the pass's own
    tensors, written again by the next call."""

    def __init__(self, inputs: dict, *, train: bool = False):
        self.inp, self.train = inputs, train
        x, h, conv_state = inputs["x"], inputs["h"], inputs["conv_state"]
        (T, C), B, dev = x.shape, h.shape[0], x.device
        K, dt = inputs["conv_w"].shape[1], x.dtype
        _fits("x", x, (T, C), dt, dev, rows=True)
        _fits("ab", inputs["ab"], (T, 2 * C), dt, dev, rows=True)
        _fits("conv_w", inputs["conv_w"], (C, K), dt, dev)
        if inputs["conv_bias"] is not None:
            _fits("conv_bias", inputs["conv_bias"], (C,), dt, dev)
        _fits("conv_state", conv_state, (B, K - 1, C), dt, dev, rows=True)
        _fits("h", h, (B, C), torch.float32, dev, rows=True)
        _fits("cu_seqlens", inputs["cu_seqlens"], (B + 1,), torch.int32, dev)
        self.u, self.y = torch.empty_like(x), torch.empty_like(x)
        self.h_ptrs = pointer_array(list(h))
        self.conv_ptrs = pointer_array(list(conv_state)) if K > 1 else None
        room = lambda n: torch.empty(n, dtype=torch.uint8, device=dev)  # noqa: E731
        self.workspace = room(gated_scan_workspace_bytes(B, T, C, x.dtype))
        self.forwarded = False
        if train:
            self.saved = room(gated_scan_saved_bytes(B, T, C, x.dtype))
            self.conv_workspace = room(conv1d_silu_backward_workspace_bytes(B, T, C, K, x.dtype))
            self.conv_start = torch.empty_like(conv_state)
            self.conv_start_ptrs = pointer_array(list(self.conv_start)) if K > 1 else None
            self.grads = dict(x=torch.empty_like(x), ab=torch.empty_like(inputs["ab"]),
                              conv_w=torch.empty(C, K, device=dev), conv_bias=None,
                              conv_state=torch.empty_like(conv_state), h=torch.empty_like(h))
            if inputs["conv_bias"] is not None:
                self.grads["conv_bias"] = torch.empty(C, device=dev)
            self.du = torch.empty_like(x)
            self.dh_ptrs = pointer_array(list(self.grads["h"]))
            self.dconv_ptrs = pointer_array(list(self.grads["conv_state"])) if K > 1 else None

    def forward(self, stream=None):
        inp = self.inp
        if self.train:
            with _on_stream(stream):
                self.conv_start.copy_(inp["conv_state"])
        conv1d_silu_prefill_varlen(self.conv_ptrs, inp["x"], inp["conv_w"], self.u, inp["cu_seqlens"],
                                   bias=inp["conv_bias"], stream=stream)
        gated_scan(self.h_ptrs, self.u, inp["ab"], self.y, inp["cu_seqlens"],
                   saved=self.saved if self.train else None, workspace=self.workspace, stream=stream)
        self.forwarded = True
        return self.y

    def backward(self, dy, *, dh_final_ptrs=None, dconv_final_ptrs=None, stream=None):
        """Gradients of the last forward(), by the names of `inputs` (conv_bias: None without one).
        dh_final_ptrs, dconv_final_ptrs: gradients of the states that it left (pointer arrays, as
        gated_scan_backward and conv1d_silu_backward take them)."""
        if not self.train:
            raise RuntimeError("backward() needs GatedPass(..., train=True)")
        if not self.forwarded:
            raise RuntimeError("backward() needs a forward() before it")
        inp, g = self.inp, self.grads
        gated_scan_backward(self.u, inp["ab"], self.saved, dy, self.du, g["ab"], inp["cu_seqlens"],
                            dh_final_ptrs=dh_final_ptrs, dh0_ptrs=self.dh_ptrs,
                            workspace=self.workspace, stream=stream)
        conv1d_silu_backward(self.conv_start_ptrs, inp["x"], inp["conv_w"], self.du, g["x"], g["conv_w"],
                             inp["cu_seqlens"], bias=inp["conv_bias"], dbias=g["conv_bias"],
                             dstate_final_ptrs=dconv_final_ptrs, dstate_ptrs=self.dconv_ptrs,
                             workspace=self.conv_workspace, stream=stream)
        return g


class GatedDecode:
    """Decode steps of a gated recurrent layer for B streams (one token each): row RMSNorm, one
    projection to x | a | b (3C outputs; bf16 weight or the 4-bit (q, scales) of w4_quantize),
    conv1d + SiLU and the gated recurrence on the carried states, the projection back (w_out). With a
    4-bit weight B is at most LA_W4_MAX_ROWS: more streams take several objects, or bf16 weights."""

    def __init__(self, norm_w, w_in, w_out, conv_w, conv_bias, conv_state, h, *, eps=1e-6):
        self.norm_w, self.w_in, self.w_out, self.eps = norm_w, w_in, w_out, eps
        self.conv_w, self.conv_bias = conv_w, conv_bias
        self.B, self.C = h.shape
        if self.B > LA_W4_MAX_ROWS and not all(isinstance(w, torch.Tensor) for w in (w_in, w_out)):
            raise ValueError(f"{self.B} streams: 4-bit weights take at most {LA_W4_MAX_ROWS} rows")
        dev, bf16 = h.device, torch.bfloat16
        D, K = norm_w.numel(), conv_w.shape[1]
        _fits("norm_w", norm_w, (D,), bf16, dev)
        _fits("conv_w", conv_w, (self.C, K), bf16, dev)
        if conv_bias is not None:
            _fits("conv_bias", conv_bias, (self.C,), bf16, dev)
        _fits("conv_state", conv_state, (self.B, K - 1, self.C), bf16, dev, rows=True)
        _fits("h", h, (self.B, self.C), torch.float32, dev, rows=True)
        for name, w, outputs, inputs in (("w_in", w_in, 3 * self.C, D), ("w_out", w_out, None, self.C)):
            if isinstance(w, torch.Tensor):
                _fits(name, w, (outputs or w.shape[0], inputs), bf16, dev, rows=True)
            elif (w[0].shape[0], 2 * w[0].shape[1]) != (outputs or w[0].shape[0], inputs):
                raise ValueError(f"{name}: 4-bit weight of {w[0].shape[0]} x {2 * w[0].shape[1]}, expected {outputs} x {inputs}")
        self.conv_ptrs = pointer_array(list(conv_state)) if conv_w.shape[1] > 1 else None
        self.h_ptrs = pointer_array(list(h))
        self.normed = torch.empty(self.B, norm_w.numel(), dtype=bf16, device=dev)
        self.rows = torch.empty(self.B, 3 * self.C, dtype=bf16, device=dev)
        self.y = torch.empty(self.B, self.C, dtype=bf16, device=dev)
        self.out = torch.empty(self.B, _outputs(w_out), dtype=bf16, device=dev)

    def run(self, hidden, stream=None):
        if (hidden.shape != self.normed.shape or hidden.dtype != self.normed.dtype
                or hidden.device != self.normed.device or hidden.stride(1) != 1):
            raise ValueError(f"hidden: {tuple(hidden.shape)} {hidden.dtype} on {hidden.device}, expected dense rows of "
                             f"{tuple(self.normed.shape)} {self.normed.dtype} on {self.normed.device}")
        rmsnorm_rows(hidden, self.norm_w, self.normed, eps=self.eps, stream=stream)
        project(self.normed, self.w_in, self.rows, stream=stream)
        gated_scan_step(self.h_ptrs, self.rows[:, :self.C], self.rows[:, self.C:], self.y,
                        conv_state_ptrs=self.conv_ptrs, conv_w=self.conv_w, conv_bias=self.conv_bias,
                        stream=stream)
        return project(self.y, self.w_out, self.out, stream=stream)
