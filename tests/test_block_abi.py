"""Refusals of the MLP-block entry points, answered on the host before anything
touches a GPU."""

import ctypes

import pytest

OK, ARG, SHAPE, DTYPE, ALIGN, WORKSPACE = range(6)
F = ctypes.c_void_p(0x1000)     # never dereferenced: validation returns first
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def L():
    from rank_compressed_backprop_gb300.build import build

    build()
    from rank_compressed_backprop_gb300._lib import lib

    return lib()


def refused(fn, good, cases):
    """Every (position, value, status) of cases, put into the good call, is
    refused with that status and nothing is launched."""
    for pos, value, status in cases:
        args = list(good)
        args[pos] = value
        assert fn(*args) == status, (pos, value)


def test_checkpoint_refusals(L):
    n0 = L.instant_launch_count()
    for fn in (L.instant_ckpt_pack, L.instant_ckpt_unpack):
        # pack(x, q, s, rows, C, dt, stream), unpack(q, s, x, ...)
        refused(fn, [F, F, F, 4, 64, 1, None],
                [(0, None, ARG), (1, None, ARG), (2, None, ARG), (3, 0, SHAPE), (3, -1, SHAPE),
                 (4, 0, SHAPE), (4, 1 << 25, SHAPE), (4, 60, ALIGN), (5, 7, DTYPE), (0, ODD, ALIGN)])
    assert L.instant_ckpt_pack(F, ODD, F, 4, 64, 1, None) == ALIGN
    assert L.instant_launch_count() == n0


def test_norm_refusals(L):
    n0 = L.instant_launch_count()
    # x, residual, gamma, h, y, q, s, r, rows, C, eps, dt, stream
    refused(L.instant_rms_norm, [F, F, F, F, F, F, F, F, 4, 64, 1e-5, 1, None],
            [(0, None, ARG), (2, None, ARG), (5, None, ARG), (6, None, ARG), (8, 0, SHAPE),
             (9, 0, SHAPE), (9, 32776, SHAPE), (9, 68, ALIGN), (10, -1.0, ARG),
             (10, float("nan"), ARG), (11, 2, DTYPE)] + [(i, ODD, ALIGN) for i in range(6)])
    assert L.instant_rms_norm(F, None, F, None, None, None, None, F, 4, 64, 1e-5, 1, None) == ARG
    need = L.instant_rms_norm_backward_workspace_bytes(4, 64)
    assert need > 0
    assert L.instant_rms_norm_backward_workspace_bytes(0, 64) == 0
    assert L.instant_rms_norm_backward_workspace_bytes(4, 32769) == 0
    # gy, q, s, r, gamma, residual, gx, ggamma, accumulate, ws, ws_bytes, rows, C, dt, stream
    refused(L.instant_rms_norm_backward, [F, F, F, F, F, F, F, F, 0, F, 1 << 20, 4, 64, 1, None],
            [(i, None, ARG) for i in (0, 1, 2, 3, 4, 6, 7)]
            + [(9, None, WORKSPACE), (10, need - 1, WORKSPACE), (11, 0, SHAPE), (12, 0, SHAPE),
               (12, 68, ALIGN), (13, 9, DTYPE)] + [(i, ODD, ALIGN) for i in (0, 1, 4, 5, 6, 7, 9)])
    assert L.instant_launch_count() == n0


def test_linear_refusals(L):
    n0 = L.instant_launch_count()
    # x, w, bias, residual, y, zq, zs, yq, ys, rows, Cx, Cy, act, dt, stream
    refused(L.instant_linear_act, [F, F, F, F, F, F, F, F, F, 4, 64, 64, 2, 1, None],
            [(0, None, ARG), (1, None, ARG), (5, None, ARG), (6, None, ARG), (7, None, ARG),
             (8, None, ARG), (9, 0, SHAPE), (10, 0, SHAPE), (11, 0, SHAPE), (10, 60, ALIGN),
             (11, 60, ALIGN), (12, 4, ARG), (12, -1, ARG), (13, 3, DTYPE)]
            + [(i, ODD, ALIGN) for i in (0, 1, 2, 3, 4, 5, 7)])
    assert L.instant_linear_act(F, F, F, F, None, F, F, None, None, 4, 64, 64, 2, 1, None) == ARG
    # gy, w, zq, zs, residual, gx, rows, Cx, Cy, act, dt, stream
    refused(L.instant_linear_act_grad, [F, F, F, F, F, F, 4, 64, 64, 1, 1, None],
            [(0, None, ARG), (1, None, ARG), (2, None, ARG), (3, None, ARG), (5, None, ARG),
             (6, 0, SHAPE), (7, 0, SHAPE), (8, 0, SHAPE), (7, 60, ALIGN), (8, 60, ALIGN),
             (9, 4, ARG), (10, 3, DTYPE)] + [(i, ODD, ALIGN) for i in (0, 1, 2, 4, 5)])
    assert L.instant_linear_act_grad(F, F, None, None, F, F, 4, 64, 64, 3, 1, None) == ARG
    need = L.instant_ckpt_grad_w_workspace_bytes(4, 64, 64)
    assert need > 0 and L.instant_ckpt_grad_w_workspace_bytes(4, 0, 64) == 0
    # gy, q, s, col_scale, gw, gb, accumulate, ws, ws_bytes, rows, Cx, Cy, dt, stream
    refused(L.instant_ckpt_grad_w, [F, F, F, F, F, F, 0, F, 1 << 20, 4, 64, 64, 1, None],
            [(0, None, ARG), (1, None, ARG), (2, None, ARG), (4, None, ARG), (7, None, WORKSPACE),
             (8, need - 1, WORKSPACE), (9, 0, SHAPE), (10, 0, SHAPE), (11, 0, SHAPE),
             (10, 60, ALIGN), (11, 60, ALIGN), (12, 5, DTYPE)]
            + [(i, ODD, ALIGN) for i in (0, 1, 3, 4, 5, 7)])
    assert L.instant_launch_count() == n0


def test_python_binding_refusals():
    torch = pytest.importorskip("torch")
    from rank_compressed_backprop_gb300 import api

    bf = torch.bfloat16
    x, w = torch.zeros(3, 64, dtype=bf), torch.zeros(72, 64, dtype=bf)
    y = torch.zeros(3, 72, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        api.linear_act(x, w, y)
    with pytest.raises(ValueError, match=r"w must be \[72, 64\]"):
        api.linear_act(x, torch.zeros(72, 56, dtype=bf), y)
    with pytest.raises(TypeError):
        api.linear_act(x, w.float(), y)
    with pytest.raises(ValueError, match="come together"):
        api.linear_act(x, w, y, zq=torch.zeros(3, 80, dtype=torch.int8))
    with pytest.raises(ValueError, match="checkpoint of"):
        api.linear_act(x, w, y, zq=torch.zeros(3, 72, dtype=torch.int8),
                       zs=torch.zeros(1, 3, dtype=torch.uint8))
    with pytest.raises(TypeError):
        api.ckpt_pack(x, torch.zeros(3, 64, dtype=torch.uint8), torch.zeros(1, 3, dtype=torch.uint8))
    with pytest.raises(ValueError, match="r must be"):
        api.rms_norm(x, torch.zeros(64, dtype=bf), x, r=torch.zeros(4))
    with pytest.raises(ValueError, match="workspace"):
        api.ckpt_grad_w(x, torch.zeros(3, 64, dtype=torch.int8), torch.zeros(1, 3, dtype=torch.uint8),
                        torch.zeros(64, 64), gb=torch.zeros(64))
    q, s = api.ckpt_buffers(3, 200, "cpu")
    assert q.shape == (3, 208) and s.shape == (2, 3)
