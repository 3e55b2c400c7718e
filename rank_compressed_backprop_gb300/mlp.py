"""MLP block of a transformer, trained with its activations kept in 8 bits.

    h = x + residual, n = rms_norm(h) gamma, a = act(n w1^T + b1), y = a w2^T + b2 + h

Between forward and backward the block keeps one byte an element of the
normalised input u, of the activation's input z and of the activation a (with a
scale byte per 128 channels), and one fp32 factor a token; the bf16 tensors of
the forward are scratch.  The backward reads nothing else: the norm's gradient
and w1's take u (w1's input was u gamma, so its gradient is scaled by gamma per
column), w2's takes a, and z gives the activation's slope.

The block holds its buffers and gradients, and the checkpoints of one forward: the
next one overwrites them.  Several batches under way at once take a block each
(the weights may be shared).  Torch only owns memory, every arithmetic step runs
in the CUDA library.
"""

from __future__ import annotations

import torch

from . import api


class CheckpointedMLP:
    def __init__(self, gamma: torch.Tensor, w1: torch.Tensor, b1: torch.Tensor | None,
                 w2: torch.Tensor, b2: torch.Tensor | None, rows: int, *, act: str = "gelu",
                 eps: float = 1e-5):
        if w1.dim() != 2 or w2.dim() != 2 or not w1.is_cuda:
            raise ValueError("w1 [H, C] and w2 [C, H] must be CUDA matrices")
        H, C = w1.shape
        if w2.shape != (C, H) or gamma.shape != (C,):
            raise ValueError(f"w1 [{H}, {C}] goes with w2 [{C}, {H}] and gamma [{C}]")
        self.gamma, self.w1, self.b1, self.w2, self.b2 = gamma, w1, b1, w2, b2
        self.C, self.H, self.rows, self.act, self.eps = C, H, rows, act, eps
        dev, dt, f32 = w1.device, w1.dtype, torch.float32
        # kept between forward and backward
        self.u = api.ckpt_buffers(rows, C, dev)
        self.z = api.ckpt_buffers(rows, H, dev)
        self.a = api.ckpt_buffers(rows, H, dev)
        self.r = torch.empty(rows, dtype=f32, device=dev)
        # forwards since the backward before them, and whether their last one has been used
        self._forwards, self._used = 0, False
        # scratch of one pass
        self.h = torch.empty(rows, C, dtype=dt, device=dev)
        self.n = torch.empty(rows, C, dtype=dt, device=dev)
        self.wide = torch.empty(rows, H, dtype=dt, device=dev)
        self.ws_norm = api.rms_norm_backward_workspace(rows, C, dev)
        self.ws_w1 = api.ckpt_grad_w_workspace(rows, C, H, dev)
        self.ws_w2 = api.ckpt_grad_w_workspace(rows, H, C, dev)
        # gradients of the parameters
        self.ggamma = torch.zeros(C, dtype=f32, device=dev)
        self.gw1 = torch.zeros(H, C, dtype=f32, device=dev)
        self.gb1 = None if b1 is None else torch.zeros(H, dtype=f32, device=dev)
        self.gw2 = torch.zeros(C, H, dtype=f32, device=dev)
        self.gb2 = None if b2 is None else torch.zeros(C, dtype=f32, device=dev)

    def kept_bytes(self) -> int:
        """Bytes that live from the forward to the backward."""
        return sum(t.numel() * t.element_size() for t in (*self.u, *self.z, *self.a, self.r))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None,
                y: torch.Tensor | None = None) -> torch.Tensor:
        """The training forward of x ``[rows, C]``: y ``[rows, C]``; leaves the
        checkpoints for :meth:`backward`, over those of the forward before."""
        y = torch.empty_like(x) if y is None else y
        h = x if residual is None else self.h
        api.rms_norm(x, self.gamma, self.n, residual=residual, h=None if residual is None else h,
                     q=self.u[0], s=self.u[1], r=self.r, eps=self.eps)
        before = 0 if self._used else self._forwards
        self._forwards = 0   # until all of the checkpoints are there
        api.linear_act(self.n, self.w1, self.wide, bias=self.b1, act=self.act, zq=self.z[0],
                       zs=self.z[1], yq=self.a[0], ys=self.a[1])
        api.linear_act(self.wide, self.w2, y, bias=self.b2, residual=h)
        self._forwards, self._used = before + 1, False
        return y

    def generate(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        """The forward without checkpoints, for any number of tokens (one and up)."""
        n, y = torch.empty_like(x), torch.empty_like(x)
        wide = x.new_empty(x.shape[0], self.H)
        h = x if residual is None else torch.empty_like(x)
        api.rms_norm(x, self.gamma, n, residual=residual, h=None if residual is None else h,
                     eps=self.eps)
        api.linear_act(n, self.w1, wide, bias=self.b1, act=self.act)
        return api.linear_act(wide, self.w2, y, bias=self.b2, residual=h)

    def backward(self, g_y: torch.Tensor, gx: torch.Tensor | None = None,
                 accumulate: bool = False) -> torch.Tensor:
        """Gradient of the block's input (x and residual alike) at the last forward;
        the parameters' gradients go to (or are added to) ``ggamma``, ``gw1``, ``gb1``,
        ``gw2``, ``gb2``.

        Without a forward there is nothing to read, and two forwards followed by two
        backwards have lost the first one's checkpoints: both are refused."""
        if self._forwards == 0:
            raise RuntimeError("CheckpointedMLP.backward: no forward has left its checkpoints")
        if self._used and self._forwards > 1:
            raise RuntimeError(f"CheckpointedMLP.backward: {self._forwards} forwards in a row, and only the last "
                               "one's checkpoints are kept: use a block for each batch under way")
        gx = torch.empty_like(g_y) if gx is None else gx
        api.ckpt_grad_w(g_y, *self.a, self.gw2, self.ws_w2, gb=self.gb2, accumulate=accumulate)
        gz = api.linear_act_grad(g_y, self.w2, self.wide, act=self.act, zq=self.z[0], zs=self.z[1])
        api.ckpt_grad_w(gz, *self.u, self.gw1, self.ws_w1, gb=self.gb1, col_scale=self.gamma,
                        accumulate=accumulate)
        gn = api.linear_act_grad(gz, self.w1, self.n)
        api.rms_norm_backward(gn, *self.u, self.r, self.gamma, gx, self.ggamma, self.ws_norm,
                              residual=g_y, accumulate=accumulate)
        self._used = True
        return gx
