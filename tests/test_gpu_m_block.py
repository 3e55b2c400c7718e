"""MLP-block operators against the fp64 oracle: 8-bit checkpoints, the norm,
linear layers with epilogues, and the gradients that read checkpoints.

Bounds, derived from the arithmetic:
* an output in bf16 is rounded once: half an ulp, at most 2^-8 of the value
  (2^-24 in fp32);
* a sum of n products accumulated in fp32 in any order is off by at most
  n 2^-23 sum|a_i b_i| (twice the unit roundoff a step: the tensor cores may cut
  instead of round);
* an activation carries its argument's error with a slope of at most 1.13 and
  adds at most 2^-16 |z| of its own; a slope function has a slope of at most 1
  and adds at most 2^-16;
* a checkpoint made from a computed value t' is within half a step of t', the
  step being right for a largest magnitude as far off as t' may be.
"""

import numpy as np
import pytest

from gpu_util import nan_like, rng, stored, to_dev, to_np, torch_or_skip
from oracle import block_oracle as O
from oracle import decode

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def torch():
    return torch_or_skip()


def _api():
    from rank_compressed_backprop_gb300 import api

    return api


def tdt(torch, dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


def ulp(dtype):
    return 2.0 ** -24 if dtype == "f32" else 2.0 ** -8


def acts(g, rows, C, dtype):
    """Normal activations with a few channels twenty times larger."""
    t = g.standard_normal((rows, C))
    t[:, g.integers(0, C, max(1, C // 100))] *= 20
    a = stored(t, dtype)
    return a, decode(a)


def near(got, ref, bound, what):
    got = to_np(got)
    assert got.shape == ref.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (what, "NaN in other places")
    bad = ~(np.abs(got - ref) <= bound) & ~np.isnan(ref)
    assert not bad.any(), (what, np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


def ckpt_np(q, s, C):
    return O.ckpt_decode(q.cpu().numpy(), s.cpu().numpy(), C)


def near_ckpt(q, s, t, err, what):
    """The checkpoint q, s stands for t, computed to within err."""
    C = t.shape[1]
    v = ckpt_np(q, s, C)
    step = 2.0 ** (s.cpu().numpy().astype(np.float64).T - 127)
    wide = np.repeat(step, 128, axis=1)[:, :C]
    assert (np.abs(v - t) <= 0.5 * wide + err).all(), what
    for g in range(step.shape[1]):
        top = np.abs(t[:, g * 128:(g + 1) * 128]).max(1)
        e = (err + 0 * t)[:, g * 128:(g + 1) * 128].max(1)
        assert (top - e <= 127 * step[:, g]).all(), (what, "step too small")
        low = step[:, g] <= 2.0 ** -120
        assert (low | (top + e > 63.5 * step[:, g])).all(), (what, "step too large")


def blank_ckpt(torch, rows, C):
    q, s = _api().ckpt_buffers(rows, C, "cuda")
    return q.fill_(77), s.fill_(3)


# ---------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(1, 8), (1, 128), (3, 136), (257, 448), (33, 11008), (4096, 64),
                                    (70001, 8)])
def test_pack_is_the_oracle_bit_for_bit(torch, dtype, rows, C):
    api = _api()
    a, x = acts(rng(rows + C), rows, C, dtype)
    q, s = blank_ckpt(torch, rows, C)
    api.ckpt_pack(to_dev(a), q, s)
    wq, ws = O.ckpt_encode(x) if rows < 5000 else (None, None)
    if wq is not None:
        assert np.array_equal(q.cpu().numpy()[:, :C], wq[:, :C])
        assert np.array_equal(s.cpu().numpy(), ws)
    want = ckpt_np(q, s, C)
    assert np.abs(want - x).max() <= 0.5 * 2.0 ** (int(s.max()) - 127)
    for out in ("bf16", "f32"):   # the codes' values are exact in both types
        v = nan_like(torch, (rows, C), tdt(torch, out))
        assert np.array_equal(to_np(api.ckpt_unpack(q, s, v)), want)


@pytest.mark.parametrize("C", [1, 3, 130, 1021])
def test_fp32_checkpoints_of_any_width(torch, C):
    api = _api()
    a, x = acts(rng(C), 37, C, "f32")
    q, s = blank_ckpt(torch, 37, C)
    api.ckpt_pack(to_dev(a), q, s)
    wq, ws = O.ckpt_encode(x)
    assert np.array_equal(q.cpu().numpy()[:, :C], wq[:, :C]) and np.array_equal(s.cpu().numpy(), ws)
    v = nan_like(torch, (37, C), torch.float32)
    assert np.array_equal(to_np(api.ckpt_unpack(q, s, v)), O.ckpt_round(x))


def test_extreme_values(torch):
    """Zeros, subnormals, the largest finite values, ties, infinities and NaN."""
    api = _api()
    big, tiny = 3.3895313892515355e38, 2.0 ** -133     # bf16's largest and smallest
    rows = [[0.0, -0.0], [tiny, -tiny], [2.0 ** -121, 2.0 ** -122], [big, -big], [big, 2.0 ** 120],
            [127.0, 0.5], [127.0, 1.5], [127.5, 1.0], [1.984375, 1.0], [2.0, 1.0], [np.inf, 1.0],
            [1.0, -np.inf], [np.nan, 1.0], [63.5, -63.5]]
    x = np.zeros((len(rows), 256))
    x[:, [3, 100]] = rows
    x[:, 200] = 1.0                                   # the other group is not disturbed
    for dtype in ("f32", "bf16"):
        a = stored(x, dtype)
        q, s = blank_ckpt(torch, *x.shape)
        api.ckpt_pack(to_dev(a), q, s)
        wq, ws = O.ckpt_encode(decode(a))
        assert np.array_equal(s.cpu().numpy(), ws)
        fin = (ws != 255).repeat(128, axis=0).T
        assert np.array_equal(q.cpu().numpy()[fin], wq[fin])
        v = nan_like(torch, x.shape, torch.float32)
        assert np.array_equal(to_np(api.ckpt_unpack(q, s, v)), O.ckpt_decode(wq, ws, 256), equal_nan=True)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def norm_bounds(x, gamma, res, dtype):
    """Reference outputs and error bounds: h is one fp32 addition, the mean of C
    squares is off by C 2^-23 of itself, the root by half of that."""
    h, r, u, y = O.rms_norm(x, gamma, res, EPS)
    rel = x.shape[1] * 2.0 ** -24 + 2.0 ** -21
    return h, r, u, y, rel


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C,res,keep", [
    (1, 8, True, True), (1, 4096, True, True), (5, 136, False, True), (19, 448, True, True),
    (9, 1024, True, False), (7, 1032, True, True), (33, 2048, False, False), (5, 4104, True, True),
    (3, 11008, True, True), (2, 16392, False, True), (2, 32768, True, True), (1000, 64, True, True)])
def test_norm(torch, dtype, rows, C, res, keep):
    api = _api()
    g = rng(100 + rows + C)
    ax, x = acts(g, rows, C, dtype)
    ar, rs = acts(g, rows, C, dtype) if res else (None, None)
    ag = stored(1 + 0.1 * g.standard_normal(C), dtype)
    dt = tdt(torch, dtype)
    y = nan_like(torch, (rows, C), dt)
    h = nan_like(torch, (rows, C), dt) if res else None
    r = nan_like(torch, (rows,), torch.float32)
    q, s = blank_ckpt(torch, rows, C) if keep else (None, None)
    api.rms_norm(to_dev(ax), to_dev(ag), y, residual=to_dev(ar) if res else None, h=h, q=q, s=s, r=r,
                 eps=EPS)
    wh, wr, wu, wy, rel = norm_bounds(x, decode(ag), rs, dtype)
    near(y, wy, np.abs(wy) * (ulp(dtype) + rel), "y")
    near(r, wr, np.abs(wr) * (rel + 2.0 ** -22), "r")
    if res:
        near(h, wh, np.abs(wh) * (ulp(dtype) + 2.0 ** -23), "h")
    if keep:
        near_ckpt(q, s, wu, np.abs(wu) * (rel + 2.0 ** -22), "u")


def test_norm_in_place_and_odd_fp32_width(torch):
    api = _api()
    g = rng(7)
    ax, x = acts(g, 5, 333, "f32")
    ar, rs = acts(g, 5, 333, "f32")
    gm = g.standard_normal(333)
    X, R = to_dev(ax), to_dev(ar)
    y = nan_like(torch, (5, 333), torch.float32)
    api.rms_norm(X, to_dev(stored(gm, "f32")), y, residual=R, h=R)   # the residual stream in place
    wh, _, _, wy, rel = norm_bounds(x, decode(stored(gm, "f32")), rs, "f32")
    near(R, wh, np.abs(wh) * 2.0 ** -22, "h")
    near(y, wy, np.abs(wy) * (rel + 2.0 ** -22), "y")


def test_norm_rows_of_zero_infinity_and_nan(torch):
    """A zero row stays zero (eps), a NaN or infinity spoils its own row only."""
    api = _api()
    x = np.ones((5, 256))
    x[0] = 0
    x[1, 3] = np.nan
    x[2, 200] = np.inf
    a = stored(x, "bf16")
    y = nan_like(torch, x.shape, torch.bfloat16)
    q, s = blank_ckpt(torch, *x.shape)
    api.rms_norm(to_dev(a), to_dev(stored(np.ones(256), "bf16")), y, q=q, s=s, eps=EPS)
    got = to_np(y)
    assert (got[0] == 0).all() and np.isnan(got[1]).all() and np.isnan(got[2, 200])
    assert (np.delete(got[2], 200) == 0).all() and np.abs(got[3:] - 1).max() < 1e-2
    v = ckpt_np(q, s, 256)
    assert (v[0] == 0).all() and np.isnan(v[1]).all() and np.isnan(v[2, 128:]).all()
    assert (v[2, :128] == 0).all() and np.isfinite(v[3:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C,res", [
    (1, 8, False), (1, 4096, True), (5, 136, True), (2600, 448, True), (9, 1032, False),
    (331, 2048, True), (5, 4104, True), (700, 4096, True), (3, 11008, True), (2, 32768, True), (3000, 64, True)])
def test_norm_backward(torch, dtype, rows, C, res):
    api = _api()
    g = rng(200 + rows + C)
    _, h = acts(g, rows, C, dtype)
    u0, r = O.rms_norm(h, np.ones(C))[2], O.rms_norm(h, np.ones(C))[1].astype(np.float32)
    wq, wsc = O.ckpt_encode(u0)
    u = O.ckpt_decode(wq, wsc, C)
    wq[:, C:] = 99                                    # padding codes are never used
    agy = stored(g.standard_normal((rows, C)) * 1e-2, dtype)
    ar = stored(g.standard_normal((rows, C)) * 1e-2, dtype) if res else None
    ag = stored(1 + 0.1 * g.standard_normal(C), dtype)
    gy, gm = decode(agy), decode(ag)
    rs = decode(ar) if res else None
    wgx, wgg = O.rms_norm_backward(gy, u, r.astype(np.float64), gm, rs)
    q, s = torch.from_numpy(wq).cuda(), torch.from_numpy(wsc).cuda()
    gx = nan_like(torch, (rows, C), tdt(torch, dtype))
    gg = nan_like(torch, (C,), torch.float32)
    ws = api.rms_norm_backward_workspace(rows, C, "cuda")
    args = (to_dev(agy), q, s, torch.from_numpy(r).cuda(), to_dev(ag), gx, gg, ws)
    api.rms_norm_backward(*args, residual=to_dev(ar) if res else None)
    d = np.abs(gy * gm)
    dot = (d * np.abs(u)).mean(1, keepdims=True) * (C * 2.0 ** -23)
    egx = r[:, None] * (2.0 ** -21 * (d + np.abs(u) * (d * np.abs(u)).mean(1, keepdims=True))
                        + np.abs(u) * dot)
    near(gx, wgx, np.abs(wgx) * (ulp(dtype) + 2.0 ** -22) + egx, "gx")
    egg = (np.abs(gy) * np.abs(u)).sum(0) * (rows + 8) * 2.0 ** -23
    near(gg, wgg, egg, "ggamma")
    first = gg.clone()
    api.rms_norm_backward(*args, residual=to_dev(ar) if res else None, accumulate=True)
    near(gg, 2 * wgg, 2 * egg, "ggamma accumulated")
    api.rms_norm_backward(*args, residual=to_dev(ar) if res else None)
    assert torch.equal(gg, first)                     # the same bits on every call


# ---------------------------------------------------------------------------
# linear layers
# ---------------------------------------------------------------------------
SHAPES = [  # rows, Cx, Cy: one token to several tiles, ragged in every direction
    (1, 64, 72), (1, 4096, 1000), (2, 128, 128), (7, 72, 136), (17, 520, 1160), (63, 264, 448),
    (65, 64, 64), (130, 448, 200), (255, 8, 8), (257, 328, 520), (300, 1032, 264), (700, 200, 776)]


def lin_inputs(rows, Cx, Cy, dtype, seed):
    g = rng(seed + rows + 3 * Cx + 7 * Cy)
    ax, x = acts(g, rows, Cx, dtype)
    aw = stored(g.standard_normal((Cy, Cx)) / np.sqrt(Cx), dtype)
    ab = stored(g.standard_normal(Cy), dtype)
    ar = stored(g.standard_normal((rows, Cy)), dtype)
    return ax, x, aw, ab, ar


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,Cx,Cy", SHAPES)
@pytest.mark.parametrize("act,bias,res,keep", [
    ("none", False, False, False), ("gelu", True, False, True), ("silu", True, True, True),
    ("relu", False, True, False)])
def test_linear(torch, dtype, rows, Cx, Cy, act, bias, res, keep):
    api = _api()
    ax, x, aw, ab, ar = lin_inputs(rows, Cx, Cy, dtype, 300)
    w, b, rs = decode(aw), decode(ab) if bias else None, decode(ar) if res else None
    y = nan_like(torch, (rows, Cy), tdt(torch, dtype))
    zq, zs = blank_ckpt(torch, rows, Cy) if keep else (None, None)
    yq, ys = blank_ckpt(torch, rows, Cy) if keep else (None, None)
    api.linear_act(to_dev(ax), to_dev(aw), y, bias=to_dev(ab) if bias else None, act=act,
                   residual=to_dev(ar) if res else None, zq=zq, zs=zs, yq=yq, ys=ys)
    wz, wy = O.linear_act(x, w, b, act, rs)
    ez = (np.abs(x) @ np.abs(w).T) * (Cx * 2.0 ** -23) + np.abs(wz) * 2.0 ** -22
    ey = 1.13 * ez + 2.0 ** -16 * np.abs(wz) * (act not in ("none", "relu")) + np.abs(wy) * 2.0 ** -22
    near(y, wy, np.abs(wy) * ulp(dtype) + ey, "y")
    if keep:
        near_ckpt(zq, zs, wz, ez, "z")
        near_ckpt(yq, ys, wy, ey, "y checkpoint")
    assert api.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,Cy,Cx", SHAPES)
@pytest.mark.parametrize("act,res", [("none", True), ("gelu", False), ("silu", True), ("relu", False)])
def test_linear_grad(torch, dtype, rows, Cy, Cx, act, res):
    api = _api()
    agy, gy, awt, _, ar = lin_inputs(rows, Cy, Cx, dtype, 400)
    g = rng(401 + rows + Cx)
    aw = np.ascontiguousarray(awt.T)                  # [Cy, Cx]
    w, rs = decode(aw), decode(ar) if res else None
    wq, wsc = O.ckpt_encode(g.standard_normal((rows, Cx)) * 2)
    z = O.ckpt_decode(wq, wsc, Cx)
    q, s = torch.from_numpy(wq).cuda(), torch.from_numpy(wsc).cuda()
    gx = nan_like(torch, (rows, Cx), tdt(torch, dtype))
    kept = dict(zq=q, zs=s) if act != "none" else {}
    api.linear_act_grad(to_dev(agy), to_dev(aw), gx, act=act, residual=to_dev(ar) if res else None, **kept)
    want = O.linear_act_grad(gy, w, z, act, rs)
    g0 = gy @ w
    e = (np.abs(gy) @ np.abs(w)) * (Cy * 2.0 ** -23) * 1.13 + 2.0 ** -16 * np.abs(g0) * (act not in ("none", "relu"))
    near(gx, want, np.abs(want) * (ulp(dtype) + 2.0 ** -22) + e, "gx")
    assert api.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,Cx,Cy", SHAPES + [(1571, 776, 768), (5000, 136, 264), (9001, 440, 1000), (12544, 448, 1792)])
@pytest.mark.parametrize("scale", [False, True])
def test_grad_w(torch, dtype, rows, Cx, Cy, scale):
    api = _api()
    g = rng(500 + rows + Cx + Cy)
    agy = stored(g.standard_normal((rows, Cy)) * 1e-2, dtype)
    gy = decode(agy)
    wq, wsc = O.ckpt_encode(acts(g, rows, Cx, dtype)[1])
    v = O.ckpt_decode(wq, wsc, Cx)
    wq[:, Cx:] = 55                                   # padding codes are never used
    asc = stored(1 + 0.1 * g.standard_normal(Cx), dtype) if scale else None
    sc = decode(asc) if scale else None
    gw = nan_like(torch, (Cy, Cx), torch.float32)
    gb = nan_like(torch, (Cy,), torch.float32)
    ws = api.ckpt_grad_w_workspace(rows, Cx, Cy, "cuda")
    args = (to_dev(agy), torch.from_numpy(wq).cuda(), torch.from_numpy(wsc).cuda(), gw, ws)
    kw = dict(gb=gb, col_scale=to_dev(asc) if scale else None)
    api.ckpt_grad_w(*args, **kw)
    wgw, wgb = O.grad_w(gy, v, sc)
    mag = np.abs(gy).T @ np.abs(v) * (1 if sc is None else np.abs(sc))
    # the operands are exact: only the fp32 sums round
    egw = mag * (rows + 4) * 2.0 ** -23
    egb = np.abs(gy).sum(0) * (rows + 4) * 2.0 ** -23
    near(gw, wgw, egw, "gw")
    near(gb, wgb, egb, "gb")
    first = gw.clone(), gb.clone()
    api.ckpt_grad_w(*args, accumulate=True, **kw)
    near(gw, 2 * wgw, 2 * egw + np.abs(wgw) * 2.0 ** -22, "gw accumulated")
    near(gb, 2 * wgb, 2 * egb + np.abs(wgb) * 2.0 ** -22, "gb accumulated")
    gw.fill_(float("nan"))
    api.ckpt_grad_w(*args, **kw)
    assert torch.equal(gw, first[0]) and torch.equal(gb, first[1])   # the same bits on every call
    assert api.device_status() == 0


@pytest.mark.parametrize("rows,Cx,Cy", [(5, 131, 77), (70, 33, 130)])
def test_fp32_products_of_any_width(torch, rows, Cx, Cy):
    api = _api()
    ax, x, aw, ab, ar = lin_inputs(rows, Cx, Cy, "f32", 600)
    w = decode(aw)
    y = nan_like(torch, (rows, Cy), torch.float32)
    zq, zs = blank_ckpt(torch, rows, Cy)
    api.linear_act(to_dev(ax), to_dev(aw), y, bias=to_dev(ab), act="gelu", residual=to_dev(ar), zq=zq, zs=zs)
    wz, wy = O.linear_act(x, w, decode(ab), "gelu", decode(ar))
    ez = (np.abs(x) @ np.abs(w).T) * (Cx * 2.0 ** -23) + np.abs(wz) * 2.0 ** -22
    near(y, wy, 1.13 * ez + 2.0 ** -16 * np.abs(wz) + np.abs(wy) * 2.0 ** -22, "y")
    near_ckpt(zq, zs, wz, ez, "z")
    q, s = blank_ckpt(torch, rows, Cx)
    api.ckpt_pack(to_dev(ax), q, s)
    gw = nan_like(torch, (Cy, Cx), torch.float32)
    api.ckpt_grad_w(y, q, s, gw)
    v, gy = ckpt_np(q, s, Cx), to_np(y)
    near(gw, gy.T @ v, (np.abs(gy).T @ np.abs(v)) * (rows + 4) * 2.0 ** -23, "gw")
    z = O.ckpt_decode(zq.cpu().numpy(), zs.cpu().numpy(), Cy)
    gz = nan_like(torch, (rows, Cy), torch.float32)
    awb = np.ascontiguousarray(aw.T)                  # a layer [Cx, Cy] after the activation
    api.linear_act_grad(to_dev(ax), to_dev(awb), gz, act="silu", zq=zq, zs=zs)
    want = O.linear_act_grad(x, decode(awb), z, "silu")
    e = (np.abs(x) @ np.abs(decode(awb))) * (Cx * 2.0 ** -23) * 1.13 + 2.0 ** -16 * np.abs(x @ decode(awb))
    near(gz, want, np.abs(want) * 2.0 ** -22 + e, "gz")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [3, 300])
def test_linear_special_values(torch, dtype, rows):
    """NaN and infinities stay in their rows; their checkpoint groups read NaN."""
    api = _api()
    x = np.ones((rows, 64))
    x[1, 5] = np.nan
    x[2, 5] = np.inf
    w = np.full((256, 64), 1 / 64)
    y = nan_like(torch, (rows, 256), tdt(torch, dtype))
    zq, zs = blank_ckpt(torch, rows, 256)
    api.linear_act(to_dev(stored(x, dtype)), to_dev(stored(w, dtype)), y, act="relu", zq=zq, zs=zs)
    got, v = to_np(y), ckpt_np(zq, zs, 256)
    assert np.isnan(got[1]).all() and np.isposinf(got[2]).all()
    assert np.isnan(v[1:3]).all()
    assert (np.delete(got, [1, 2], 0) == 1).all() and (np.delete(v, [1, 2], 0) == 1).all()


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activations_over_their_range(torch, act):
    """Activation and slope from one product with an identity weight: arguments
    of every size, the tails and zero among them."""
    api = _api()
    z = np.concatenate([np.linspace(-12, 12, 4096 - 5), [0.0, 30.0, -30.0, 87.0, -87.0]]).reshape(32, 128)
    az = stored(z, "bf16")
    eye = to_dev(stored(np.eye(128), "bf16"))
    for rows in (32, 320):
        a = np.tile(az, (rows // 32, 1))
        y = nan_like(torch, a.shape, torch.bfloat16)
        q, s = blank_ckpt(torch, *a.shape)
        api.linear_act(to_dev(a), eye, y, act=act, zq=q, zs=s)
        want = O.act(decode(a), act)
        # relative in the tails too: down to where the value itself underflows 2^-100
        near(y, want, np.abs(want) * (2.0 ** -8 + 2.0 ** -16) + 2.0 ** -100, "y")
        gx = nan_like(torch, a.shape, torch.bfloat16)
        one = to_dev(stored(np.ones_like(decode(a)), "bf16"))
        api.linear_act_grad(one, eye, gx, act=act, zq=q, zs=s)
        want = O.act_slope(ckpt_np(q, s, 128), act)
        near(gx, want, np.abs(want) * 2.0 ** -8 + 2.0 ** -16, "slope")


def test_y_may_be_the_residual(torch):
    api = _api()
    for rows in (3, 400):
        ax, x, aw, ab, ar = lin_inputs(rows, 264, 392, "bf16", 700)
        fresh = nan_like(torch, (rows, 392), torch.bfloat16)
        kw = dict(bias=to_dev(ab), act="silu")
        api.linear_act(to_dev(ax), to_dev(aw), fresh, residual=to_dev(ar), **kw)
        R = to_dev(ar)
        api.linear_act(to_dev(ax), to_dev(aw), R, residual=R, **kw)
        assert torch.equal(R, fresh)


def test_side_stream(torch):
    """Calls on a stream of their own, ordered by events only."""
    api = _api()
    ax, x, aw, ab, ar = lin_inputs(300, 264, 392, "bf16", 800)
    X, Wt = to_dev(ax), to_dev(aw)
    a, b = (nan_like(torch, (300, 392), torch.bfloat16) for _ in range(2))
    api.linear_act(X, Wt, a)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    api.linear_act(X, Wt, b, stream=st)
    st.synchronize()
    assert torch.equal(a, b)


def test_more_than_two_to_the_31_elements(torch):
    """Offsets past 32 bits: the last rows of tensors with over 2^31 elements."""
    api = _api()
    rows, C = 70001, 32768
    x = torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda")
    x[-2:] = torch.arange(C, device="cuda") % 7 - 3
    q, s = api.ckpt_buffers(rows, C, "cuda")
    api.ckpt_pack(x, q, s)
    y = torch.empty_like(x)
    api.ckpt_unpack(q, s, y)
    assert torch.equal(y[-2:], x[-2:]) and not y[:3].any()
    r = torch.empty(rows, device="cuda")
    api.rms_norm(x, torch.ones(C, dtype=torch.bfloat16, device="cuda"), y, q=q, s=s, r=r)
    want = O.rms_norm(to_np(x[-1:]), np.ones(C))[3]
    near(y[-1:], want, np.abs(want) * (2.0 ** -8 + C * 2.0 ** -24), "y")
    w = torch.zeros(8, C, dtype=torch.bfloat16, device="cuda")
    w[:, :3] = 1
    out = torch.empty(rows, 8, dtype=torch.bfloat16, device="cuda")
    api.linear_act(x, w, out)
    assert (out[-2:] == -6).all() and not out[:-2].any()
    gx = x.zero_()
    g = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    g[-1] = 1
    api.linear_act_grad(g, w, gx)
    assert (gx[-1, :3] == 8).all() and not gx[-1, 3:].any() and not gx[:-1].any()
    api.ckpt_pack(x, q, s)
    gw = nan_like(torch, (8, C), torch.float32)
    api.ckpt_grad_w(g, q, s, gw)
    assert (gw[:, :3] == 8).all() and not gw[:, 3:].any()


# ---------------------------------------------------------------------------
# the block
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,rows,C,H", [("f32", 50, 64, 72), ("bf16", 333, 448, 1792), ("bf16", 1, 264, 520)])
def test_mlp_block(torch, dtype, rows, C, H):
    """Forward and backward of the block, every stage's output recomputed by the
    oracle from what the stage before it left."""
    from rank_compressed_backprop_gb300 import CheckpointedMLP

    api = _api()
    g = rng(900 + rows)
    ax, x = acts(g, rows, C, dtype)
    ar, rs = acts(g, rows, C, dtype)
    gm = stored(1 + 0.1 * g.standard_normal(C), dtype)
    w1, w2 = (stored(g.standard_normal(s) / np.sqrt(s[1]), dtype) for s in ((H, C), (C, H)))
    b1, b2 = (stored(0.1 * g.standard_normal(n), dtype) for n in (H, C))
    mlp = CheckpointedMLP(to_dev(gm), to_dev(w1), to_dev(b1), to_dev(w2), to_dev(b2), rows)
    X, R = to_dev(ax), to_dev(ar)
    y = mlp.forward(X, R)
    n, wide, h = (to_np(t) for t in (mlp.n, mlp.wide, mlp.h))
    tol = 3 * ulp(dtype) + 1e-4
    rel = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)  # noqa: E731
    assert rel(n, O.rms_norm(x, decode(gm), rs)[3]) < tol
    z, a = O.linear_act(n, decode(w1), decode(b1), "gelu")
    assert rel(wide, a) < tol
    assert rel(to_np(y), O.linear_act(wide, decode(w2), decode(b2), "none", h)[1]) < tol
    assert torch.equal(mlp.generate(X, R), y)
    # kept: one byte an element of u, z and a, a scale byte per 128, r
    groups = lambda c: -(-c // 128)  # noqa: E731
    pad = lambda c: -(-c // 16) * 16  # noqa: E731
    assert mlp.kept_bytes() == rows * (pad(C) + 2 * pad(H) + groups(C) + 2 * groups(H) + 4)
    agy = stored(1e-2 * g.standard_normal((rows, C)), dtype)
    gy = decode(agy)
    u, zc, ac = (ckpt_np(*k, c) for k, c in ((mlp.u, C), (mlp.z, H), (mlp.a, H)))
    gx = mlp.backward(to_dev(agy))
    gz, gn = to_np(mlp.wide), to_np(mlp.n)
    for got, want in [(mlp.gw2, O.grad_w(gy, ac)[0]), (mlp.gb2, gy.sum(0)),
                      (gz, O.linear_act_grad(gy, decode(w2), zc, "gelu")),
                      (mlp.gw1, O.grad_w(gz, u, decode(gm))[0]), (mlp.gb1, gz.sum(0)),
                      (gn, O.linear_act_grad(gz, decode(w1)))]:
        assert rel(got if isinstance(got, np.ndarray) else to_np(got), want) < tol
    wgx, wgg = O.rms_norm_backward(gn, u, to_np(mlp.r), decode(gm), gy)
    assert rel(to_np(gx), wgx) < tol and rel(to_np(mlp.ggamma), wgg) < tol
    # against the unrounded block: the 8-bit checkpoints cost about a percent
    hx, r_, u_, y_ = O.rms_norm(x, decode(gm), rs)
    z_, a_ = O.linear_act(y_, decode(w1), decode(b1), "gelu")
    gz_ = O.linear_act_grad(gy, decode(w2), z_, "gelu")
    assert rel(to_np(mlp.gw2), gy.T @ a_) < 0.05
    assert rel(to_np(mlp.gw1), O.grad_w(gz_, u_, decode(gm))[0]) < 0.05
    first = {k: getattr(mlp, k).clone() for k in ("gw1", "gb1", "gw2", "gb2", "ggamma")}
    mlp.forward(X, R)
    mlp.backward(to_dev(agy), accumulate=True)
    for k, v in first.items():
        assert rel(to_np(getattr(mlp, k)), 2 * to_np(v)) < 1e-5, k
    assert api.device_status() == 0


# ---------------------------------------------------------------------------
# sizes at which every CTA has several tiles, segments or blocks of rows to do;
# the reference is the same formula in float64 on the GPU
# ---------------------------------------------------------------------------
def act64(torch, z, kind):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "gelu": lambda: z * torch.special.ndtr(z),
            "silu": lambda: z * torch.sigmoid(z)}[kind]()


def slope64(torch, z, kind):
    if kind == "relu":
        return (z > 0).double()
    if kind == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5
    s = torch.sigmoid(z)
    return s + z * s * (1 - s)


def far(torch, got, ref, bound):
    """The largest error in units of its bound (NaN where an element was not written)."""
    return float(((got.double() - ref).abs() / bound).max())


def values64(torch, q, s, C):
    step = torch.exp2(s.double() - 127).t().repeat_interleave(128, 1)[:, :C]
    return q[:, :C].double() * step, step


@pytest.mark.parametrize("rows,Cx,Cy", [(2600, 328, 2056), (3001, 4104, 1800), (20000, 64, 136)])
@pytest.mark.parametrize("act,res", [("gelu", True), ("silu", False), ("none", True)])
def test_products_of_many_tiles(torch, rows, Cx, Cy, act, res):
    api = _api()
    gen = torch.Generator("cuda").manual_seed(rows + Cx)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    x, w, b = rn(rows, Cx).to(bf), (rn(Cy, Cx) * Cx ** -0.5).to(bf), rn(Cy).to(bf)
    r = rn(rows, Cy).to(bf) if res else None
    X, Wt = x.double(), w.double()
    z = X @ Wt.t() + b.double()
    y = act64(torch, z, act) + (r.double() if res else 0)
    ez = (X.abs() @ Wt.abs().t()) * (Cx * 2.0 ** -23) + z.abs() * 2.0 ** -22
    ey = 1.13 * ez + 2.0 ** -16 * z.abs() * (act != "none") + y.abs() * 2.0 ** -22
    plain = nan_like(torch, (rows, Cy), bf)
    api.linear_act(x, w, plain, bias=b, act=act, residual=r)
    assert far(torch, plain, y, y.abs() * 2.0 ** -8 + ey) <= 1
    kept = nan_like(torch, (rows, Cy), bf)
    (zq, zs), (yq, ys) = blank_ckpt(torch, rows, Cy), blank_ckpt(torch, rows, Cy)
    api.linear_act(x, w, kept, bias=b, act=act, residual=r, zq=zq, zs=zs, yq=yq, ys=ys)
    assert far(torch, kept, y, y.abs() * 2.0 ** -8 + ey) <= 1
    for q, s, t, e in ((zq, zs, z, ez), (yq, ys, y, ey)):
        v, step = values64(torch, q, s, Cy)
        assert ((v - t).abs() <= 0.5 * step + e).all()
    # back, from z's checkpoint
    zv, _ = values64(torch, zq, zs, Cy)
    g, w2 = (rn(rows, Cx) * 1e-2).to(bf), w.t().contiguous()     # a layer [Cx, Cy] after the activation
    want = g.double() @ w2.double()
    eg = (g.double().abs() @ w2.double().abs()) * (Cx * 2.0 ** -23) * 1.13
    if act != "none":
        eg = eg + 2.0 ** -16 * want.abs()
        want = want * slope64(torch, zv, act)
    if res:
        want = want + r.double()
    gx = nan_like(torch, (rows, Cy), bf)
    api.linear_act_grad(g, w2, gx, act=act, zq=zq, zs=zs, residual=r)
    assert far(torch, gx, want, want.abs() * (2.0 ** -8 + 2.0 ** -22) + eg) <= 1
    # weight gradient, from y's checkpoint
    yv, _ = values64(torch, yq, ys, Cy)
    want, mag = g.double().t() @ yv, g.double().abs().t() @ yv.abs()
    gw = nan_like(torch, (Cx, Cy), torch.float32)
    gb = nan_like(torch, (Cx,), torch.float32)
    ws = api.ckpt_grad_w_workspace(rows, Cy, Cx, "cuda")
    api.ckpt_grad_w(g, yq, ys, gw, ws, gb=gb)
    assert far(torch, gw, want, mag * (rows + 4) * 2.0 ** -23) <= 1
    assert far(torch, gb, g.double().sum(0), g.double().abs().sum(0) * (rows + 4) * 2.0 ** -23) <= 1
    first = gw.clone()
    api.ckpt_grad_w(g, yq, ys, gw, ws, accumulate=True)
    assert far(torch, gw, 2 * want, 2 * mag * (rows + 4) * 2.0 ** -23 + want.abs() * 2.0 ** -22) <= 1
    api.ckpt_grad_w(g, yq, ys, gw, ws)
    assert torch.equal(gw, first)
    assert api.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C,res", [
    (1000000, 64, False), (9001, 448, True), (5003, 1024, False), (3001, 2048, True), (2003, 4096, True),
    (1501, 8192, False), (1001, 11008, True), (400, 11008, False)])
def test_norm_backward_of_many_rows(torch, dtype, rows, C, res):
    """Several blocks of rows a CTA, more rows than it holds factors and scales of."""
    api = _api()
    dt = tdt(torch, dtype)
    gen = torch.Generator("cuda").manual_seed(rows + C)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    h = rn(rows, C).to(dt)
    gamma = (1 + 0.1 * rn(C)).to(dt)
    y = torch.empty_like(h)
    q, s = blank_ckpt(torch, rows, C)
    r = torch.empty(rows, device="cuda")
    api.rms_norm(h, gamma, y, q=q, s=s, r=r)
    gy = (rn(rows, C) * 1e-2).to(dt)
    bypass = (rn(rows, C) * 1e-2).to(dt) if res else None
    gx, gg = nan_like(torch, (rows, C), dt), nan_like(torch, (C,), torch.float32)
    ws = api.rms_norm_backward_workspace(rows, C, "cuda")
    api.rms_norm_backward(gy, q, s, r, gamma, gx, gg, ws, residual=bypass)
    u, _ = values64(torch, q, s, C)
    d = gy.double() * gamma.double()
    c, ca = (d * u).mean(1, keepdim=True), (d * u).abs().mean(1, keepdim=True)
    want = r.double()[:, None] * (d - u * c) + (bypass.double() if res else 0)
    e = r.double()[:, None] * (2.0 ** -21 * (d.abs() + u.abs() * ca) + u.abs() * ca * C * 2.0 ** -23)
    assert far(torch, gx, want, want.abs() * (ulp(dtype) + 2.0 ** -22) + e) <= 1
    p = gy.double() * u
    assert far(torch, gg, p.sum(0), p.abs().sum(0) * (rows + 8) * 2.0 ** -23) <= 1
    first = gg.clone()
    api.rms_norm_backward(gy, q, s, r, gamma, gx, gg, ws, residual=bypass)
    assert torch.equal(gg, first)
    assert api.device_status() == 0
