"""MLP-block operators at the edges of what their header promises: outputs left
out, scratch on side streams, very many rows, tails and infinities of the
activations, long sums, and calls that are refused."""

import numpy as np
import pytest

from gpu_util import nan_like, rng, stored, to_dev, to_np, torch_or_skip
from oracle import block_oracle as O
from oracle import decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return torch_or_skip()


def _api():
    from rank_compressed_backprop_gb300 import api

    return api


def blank_ckpt(torch, rows, C):
    q, s = _api().ckpt_buffers(rows, C, "cuda")
    return q.fill_(77), s.fill_(3)


# ---------------------------------------------------------------------------
# outputs left out: the same bits in what is asked for
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,Cx,Cy", [(8192, 448, 1792), (4096, 1024, 1288), (20000, 64, 136), (33, 264, 448)])
@pytest.mark.parametrize("act,res", [("none", True), ("none", False), ("gelu", True), ("relu", False)])
def test_outputs_left_out(torch, rows, Cx, Cy, act, res):
    """y may be left out when its checkpoint is asked for, and each checkpoint too."""
    api = _api()
    gen = torch.Generator("cuda").manual_seed(rows + Cx)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    x, w, b = rn(rows, Cx), rn(Cy, Cx) * Cx ** -0.5, rn(Cy)
    kw = dict(bias=b, act=act, residual=rn(rows, Cy) if res else None)
    y = nan_like(torch, (rows, Cy), torch.bfloat16)
    z0, y0 = blank_ckpt(torch, rows, Cy), blank_ckpt(torch, rows, Cy)
    api.linear_act(x, w, y, zq=z0[0], zs=z0[1], yq=y0[0], ys=y0[1], **kw)
    for with_y, with_z, with_yk in [(False, True, True)] * 4 + [(False, False, True), (True, True, False),
                                                              (True, False, True)]:
        out = nan_like(torch, (rows, Cy), torch.bfloat16) if with_y else None
        z1, y1 = blank_ckpt(torch, rows, Cy), blank_ckpt(torch, rows, Cy)
        got = api.linear_act(x, w, out, zq=z1[0] if with_z else None, zs=z1[1] if with_z else None,
                             yq=y1[0] if with_yk else None, ys=y1[1] if with_yk else None, **kw)
        assert got is out and (out is None or torch.equal(out, y))
        for asked, a, k in ((with_z, z0, z1), (with_yk, y0, y1)):
            if asked:
                assert torch.equal(a[0][:, :Cy], k[0][:, :Cy]) and torch.equal(a[1], k[1])
    assert api.device_status() == 0


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("handle", [False, True])
def test_own_workspace_on_a_side_stream(torch, handle):
    """A call that allocates its workspace does so on the stream it runs on: a block
    that the current stream has freed but not yet finished with stays as it is."""
    api = _api()
    rows, Cx, Cy = 4096, 512, 256
    gen = torch.Generator("cuda").manual_seed(5)
    g = torch.randn(rows, Cy, generator=gen, device="cuda").bfloat16()
    x = torch.randn(rows, Cx, generator=gen, device="cuda").bfloat16()
    q, s = blank_ckpt(torch, rows, Cx)
    api.ckpt_pack(x, q, s)
    want = nan_like(torch, (Cy, Cx), torch.float32)
    api.ckpt_grad_w(g, q, s, want)
    n = api.ckpt_grad_w_workspace(rows, Cx, Cy, "cuda").numel()
    kept = torch.empty(n, dtype=torch.uint8, device="cuda")
    got = nan_like(torch, (Cy, Cx), torch.float32)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.full((n,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)          # some 50 ms
    kept.copy_(block)
    del block                               # free for the current stream, its copy still to come
    api.ckpt_grad_w(g, q, s, got, stream=st.cuda_stream if handle else st)
    torch.cuda.synchronize()
    assert bool((kept == 7).all())
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------
# narrow products of more row tiles than a grid has in y
# ---------------------------------------------------------------------------
def test_narrow_products_of_very_many_rows(torch):
    """8.4 million rows of 64 channels: over 65535 tiles of 128 rows."""
    api = _api()
    rows, C = 65535 * 128 + 8, 64
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randint(-3, 4, (rows, C), generator=gen, device="cuda").bfloat16()
    w = torch.randint(-2, 3, (C, C), generator=gen, device="cuda").bfloat16()
    some = torch.tensor([0, 1, rows // 2, 65535 * 128 - 1, 65535 * 128, rows - 2, rows - 1], device="cuda")
    y = nan_like(torch, (rows, C), torch.bfloat16)
    api.linear_act(x, w, y)                 # whole numbers of up to 384: exact in fp32, rounded once
    assert torch.equal(y[some].double(), (x[some].double() @ w.double().t()).bfloat16().double())
    assert not bool(y.isnan().any())
    y.fill_(float("nan"))
    api.linear_act_grad(x, w, y)
    assert torch.equal(y[some].double(), (x[some].double() @ w.double()).bfloat16().double())
    assert not bool(y.isnan().any())
    del y
    # a layer of that many outputs: its weight gradient over 64 rows
    g = x.view(C, rows)                     # [64, rows]
    t = torch.randint(-3, 4, (C, C), generator=gen, device="cuda").bfloat16()
    q, s = blank_ckpt(torch, C, C)
    api.ckpt_pack(t, q, s)
    gw, gb = nan_like(torch, (rows, C), torch.float32), nan_like(torch, (rows,), torch.float32)
    api.ckpt_grad_w(g, q, s, gw, api.ckpt_grad_w_workspace(C, C, rows, "cuda"), gb=gb)
    assert torch.equal(gw[some].double(), g[:, some].double().t() @ t.double())
    assert torch.equal(gb[some].double(), g[:, some].double().sum(0))
    assert not bool(gw.isnan().any()) and not bool(gb.isnan().any())
    assert api.device_status() == 0


# ---------------------------------------------------------------------------
# tails and infinities of the activations
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,Cy", [(32, 128), (320, 128), (32, 2048)])
def test_gelu_slope_in_its_negative_tail(torch, dtype, rows, Cy):
    """gelu'(z) = Phi(z) + z phi(z) keeps its relative accuracy down to z = -10.

    Bound: both terms hold exp(-z^2 / 2), whose argument has two roundings: up to
    2^-23 z^2 / 2, at most 6e-6 of the term, and 1e-6 for the functions themselves;
    the terms differ in sign and add up to at most 1.6 times the slope from -2 on."""
    api = _api()
    z = np.sort(-2 - 8 * np.linspace(0, 1, 32 * 128)).reshape(32, 128)
    wq, wsc = (np.ascontiguousarray(np.tile(a, t)) for a, t in
               zip(O.ckpt_encode(z), ((rows // 32, 1), (1, rows // 32))))
    q, s = torch.from_numpy(wq).cuda(), torch.from_numpy(wsc).cuda()
    eye, one = (to_dev(stored(a, dtype)) for a in (np.eye(Cy, 128), np.ones((rows, Cy))))
    gx = torch.full((rows, 128), float("nan"), dtype=one.dtype, device="cuda")
    api.linear_act_grad(one, eye, gx, act="gelu", zq=q, zs=s)
    want = O.act_slope(O.ckpt_decode(wq, wsc, 128), "gelu")
    err = np.abs(to_np(gx) - want) / np.abs(want)
    assert err.max() <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) + 2.0 ** -15


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,Cx", [(6, 64), (300, 64), (6, 2048)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_activations_of_infinities(torch, dtype, rows, Cx, act):
    """act(+-inf) and act(NaN) are what the formula says, whatever the type and size:
    relu(-inf) is 0, z Phi(z) and z / (1 + exp(-z)) have no value at -inf."""
    api = _api()
    x = np.ones((rows, Cx))
    x[[1, 2, 4], 5] = [np.inf, -np.inf, np.nan]
    w = np.full((256, Cx), 1 / Cx)
    y = nan_like(torch, (rows, 256), torch.float32 if dtype == "f32" else torch.bfloat16).fill_(3)
    yq, ys = blank_ckpt(torch, rows, 256)
    for kw in (dict(), dict(yq=yq, ys=ys)):
        api.linear_act(to_dev(stored(x, dtype)), to_dev(stored(w, dtype)), y, act=act, **kw)
        with np.errstate(invalid="ignore", over="ignore"):
            want = O.act(x @ w.T, act)
        assert np.array_equal(np.isnan(to_np(y)), np.isnan(want))
        assert np.array_equal(np.isinf(to_np(y)), np.isinf(want))
        assert np.abs(to_np(y)[0] - want[0]).max() <= 2.0 ** -8
    bad = ~np.isfinite(want[:, 0])
    assert np.array_equal(np.isnan(O.ckpt_decode(yq.cpu().numpy(), ys.cpu().numpy(), 256)).all(1), bad)


# ---------------------------------------------------------------------------
# long sums: what the tensor cores cut off must not add up
# ---------------------------------------------------------------------------
def in_order(torch, a, b):
    """a^T b over the first axis, one fp32 addition a term (products of bf16 are exact)."""
    out = torch.zeros(a.shape[1], b.shape[1], device="cuda")
    for k in range(a.shape[0]):
        out.addcmul_(a[k, :, None], b[k])
    return out


@pytest.mark.parametrize("rows,Cx,Cy", [(8192, 1152, 4096), (8192, 2432, 2048), (32768, 128, 11008),
                                        (16384, 256, 1024), (32768, 64, 64), (4096, 1024, 1024)])
def test_weight_gradient_over_many_rows(torch, rows, Cx, Cy):
    """An accumulator takes 16 chunks of 64 rows, in 64 steps that cut off at most 2^-23
    of the sum so far: 33 2^-23 of a segment of positive terms.  Up to 32 segments are
    added in fp32, at most 2^-24 each."""
    api = _api()
    gen = torch.Generator("cuda").manual_seed(rows + Cx)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    for positive in (False, True):
        g, x = rn(rows, Cy), rn(rows, Cx)
        if positive:
            g, x = g.abs() + 0.5, x.abs() + 0.5
        g = g.bfloat16()
        q, s = blank_ckpt(torch, rows, Cx)
        api.ckpt_pack(x, q, s)
        v = torch.empty(rows, Cx, device="cuda")
        api.ckpt_unpack(q, s, v)
        gw = nan_like(torch, (Cy, Cx), torch.float32)
        api.ckpt_grad_w(g, q, s, gw)
        want = g.double().t() @ v.double()
        if positive:
            assert float(((gw.double() - want).abs() / want).max()) <= (33 + 16) * 2.0 ** -23
        elif rows * Cx * Cy < 1e11:   # random signs: no farther than twice what sums in order are
            off = (in_order(torch, g.float(), v).double() - want).norm()
            assert float((gw.double() - want).norm()) <= 2 * float(off)


def rounded(torch, t):
    """What the checkpoint of t (float64) stands for."""
    rows, C = t.shape
    g = torch.nn.functional.pad(t, (0, -C % 128)).view(rows, -1, 128)
    m, e = torch.frexp(g.abs().amax(-1, keepdim=True))
    step = torch.exp2((e - 7 + (m > 127 / 128)).clamp(-120, 121).double())
    return ((g / step).round().clamp(-127, 127) * step).view(rows, -1)[:, :C]


@pytest.mark.parametrize("rows,Cx,Cy", [(128, 4096, 11008), (100, 11008, 4096), (4096, 576, 4096), (12544, 448, 1792),
                                        (2048, 1536, 4096)])
def test_checkpoint_of_a_product(torch, rows, Cx, Cy):
    """Codes that differ from those of exact sums: an error of the sums flips a code that
    lies within it of the middle of two, so their number goes with the error.  Twice
    what fp32 sums in order flip, and half as many again for chance."""
    api = _api()
    gen = torch.Generator("cuda").manual_seed(rows + Cx)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, w = rn(rows, Cx).bfloat16(), (rn(Cy, Cx) * Cx ** -0.5).bfloat16()
    y = nan_like(torch, (rows, Cy), torch.bfloat16)
    q, s = blank_ckpt(torch, rows, Cy)
    api.linear_act(x, w, y, zq=q, zs=s)
    v = nan_like(torch, (rows, Cy), torch.float32)
    api.ckpt_unpack(q, s, v)
    want = rounded(torch, x.double() @ w.double().t())
    ordered = rounded(torch, in_order(torch, x.float().t().contiguous(), w.float().t().contiguous()).double())
    assert int((v.double() != want).sum()) <= 3 * int((ordered != want).sum()) + 10


# ---------------------------------------------------------------------------
# the block
# ---------------------------------------------------------------------------
def small_mlp(torch, rows, C=64, H=136):
    from rank_compressed_backprop_gb300 import CheckpointedMLP

    gen = torch.Generator("cuda").manual_seed(11)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    mlp = CheckpointedMLP(1 + 0.1 * rn(C), rn(H, C) * C ** -0.5, rn(H), rn(C, H) * H ** -0.5, rn(C), rows)
    return mlp, rn


def test_block_keeps_one_forward(torch):
    """A backward whose checkpoints are not there, or are another batch's, is refused;
    everything else runs: a forward that nobody went back through, two gradients at
    one forward, any number of steps."""
    mlp, rn = small_mlp(torch, 33)
    a, b, g = rn(33, 64), rn(33, 64), rn(33, 64)
    with pytest.raises(RuntimeError, match="no forward"):
        mlp.backward(g)
    mlp.forward(a)
    first = mlp.backward(g).clone()
    assert torch.equal(mlp.backward(g), first)      # twice at one forward
    for _ in range(2):                              # steps, one forward of them left unused
        mlp.forward(b)
        mlp.forward(a)
        assert torch.equal(mlp.backward(g), first)
        mlp.forward(a)
        assert torch.equal(mlp.backward(g), first)
    mlp.forward(a)                                  # two batches under way in one block
    mlp.forward(b)
    mlp.backward(g)
    with pytest.raises(RuntimeError, match="2 forwards in a row"):
        mlp.backward(g)
    mlp.forward(a)
    assert torch.equal(mlp.backward(g), first)
    with pytest.raises(ValueError, match="x must be a matrix"):
        mlp.forward(a.view(3, 11, 64))
    with pytest.raises(ValueError):
        mlp.forward(a[:5])                          # another number of rows than the block's
    assert torch.equal(mlp.backward(g), first)      # a refused forward has left them alone
    with pytest.raises(ValueError, match="y must be"):
        mlp.forward(b, y=a[:5])                     # refused at its end, over what was kept
    with pytest.raises(RuntimeError, match="no forward"):
        mlp.backward(g)


# ---------------------------------------------------------------------------
# captured in a graph, and called from several threads
# ---------------------------------------------------------------------------
def test_block_in_a_graph(torch):
    """A captured step (forward and backward, a weight gradient with scratch of its own)
    replayed over other inputs gives what the calls by themselves give."""
    api = _api()
    mlp, rn = small_mlp(torch, 300, 264, 1032)
    x, r, g = rn(300, 264), rn(300, 264), rn(300, 264)
    y, gx, gw = torch.empty_like(x), torch.empty_like(x), torch.empty(1032, 264, device="cuda")

    def step():
        mlp.forward(x, r, y)
        mlp.backward(g, gx)
        api.ckpt_grad_w(mlp.wide, *mlp.u, gw)

    names = ("gw1", "gb1", "gw2", "gb2", "ggamma")
    results = lambda: [t.clone() for t in (y, gx, gw, *(getattr(mlp, n) for n in names))]  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (x, r, g):
            t.copy_(rn(300, 264))
        step()
        want = results()
        for t in (y, gx, gw, *(getattr(mlp, n) for n in names)):
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    assert api.device_status() == 0


def test_blocks_of_several_threads(torch):
    """Four host threads, a block and a stream each, at the same time."""
    import threading

    jobs = []
    for i, (rows, C, H) in enumerate([(1, 264, 520), (700, 448, 1792), (129, 1024, 2048), (2600, 64, 328)]):
        mlp, rn = small_mlp(torch, rows, C, H)
        x, g = rn(rows, C), rn(rows, C)
        y = mlp.forward(x)
        jobs.append((mlp, x, g, y.clone(), mlp.backward(g).clone(), mlp.gw1.clone(), mlp.ggamma.clone()))
    torch.cuda.synchronize()
    wrong = []

    def work(mlp, x, g, y, gx, gw1, gg):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(20):
                    a = mlp.forward(x)
                    b = mlp.backward(g)
                    if not (torch.equal(a, y) and torch.equal(b, gx) and torch.equal(mlp.gw1, gw1)
                            and torch.equal(mlp.ggamma, gg)):
                        wrong.append(x.shape)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert _api().device_status() == 0


# ---------------------------------------------------------------------------
# the norm's gradient over wide rows, more of them than CTAs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C,res", [(700, 12296, True), (1300, 16384, True), (650, 32768, False)])
def test_norm_backward_of_wide_rows(torch, dtype, rows, C, res):
    """Bounds as for the narrow ones: C products a row, rows products a column, each sum
    off by at most 2^-23 of its terms' magnitudes a step."""
    api = _api()
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = torch.Generator("cuda").manual_seed(rows + C)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    h, gamma = rn(rows, C).to(dt), (1 + 0.1 * rn(C)).to(dt)
    q, s = blank_ckpt(torch, rows, C)
    r = torch.empty(rows, device="cuda")
    api.rms_norm(h, gamma, None, q=q, s=s, r=r)
    gy = (rn(rows, C) * 1e-2).to(dt)
    bypass = (rn(rows, C) * 1e-2).to(dt) if res else None
    gx, gg = nan_like(torch, (rows, C), dt), nan_like(torch, (C,), torch.float32)
    ws = api.rms_norm_backward_workspace(rows, C, "cuda")
    api.rms_norm_backward(gy, q, s, r, gamma, gx, gg, ws, residual=bypass)
    u = torch.empty(rows, C, device="cuda")
    api.ckpt_unpack(q, s, u)
    u, d = u.double(), gy.double() * gamma.double()
    c, ca = (d * u).mean(1, keepdim=True), (d * u).abs().mean(1, keepdim=True)
    want = r.double()[:, None] * (d - u * c) + (bypass.double() if res else 0)
    e = r.double()[:, None] * (2.0 ** -21 * (d.abs() + u.abs() * ca) + u.abs() * ca * C * 2.0 ** -23)
    ulp = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    assert bool(((gx.double() - want).abs() <= want.abs() * (ulp + 2.0 ** -22) + e).all())
    p = gy.double() * u
    assert bool(((gg.double() - p.sum(0)).abs() <= p.abs().sum(0) * (rows + 8) * 2.0 ** -23).all())
    first = gg.clone()
    api.rms_norm_backward(gy, q, s, r, gamma, gx, gg, ws, residual=bypass, accumulate=True)
    assert bool(((gg.double() - 2 * p.sum(0)).abs() <= 2 * p.abs().sum(0) * (rows + 8) * 2.0 ** -23
                 + p.sum(0).abs() * 2.0 ** -22).all())
    api.rms_norm_backward(gy, q, s, r, gamma, gx, gg, ws, residual=bypass)
    assert torch.equal(gg, first)


@pytest.mark.parametrize("rows,Cx,Cy", [(16384, 576, 4096), (8192, 1536, 4096), (8192, 2048, 4096)])
def test_checkpoints_over_some_hundred_channels(torch, rows, Cx, Cy):
    """Over 30 million values and more, with a few channels twenty times larger, at most
    twice the codes that fp32 sums in order flip (some 200 to 600: chance is a tenth)."""
    api = _api()
    gen = torch.Generator("cuda").manual_seed(rows + Cx)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = rn(rows, Cx)
    x[:, ::256] *= 20
    x, w = x.bfloat16(), (rn(Cy, Cx) * Cx ** -0.5).bfloat16()
    q, s = blank_ckpt(torch, rows, Cy)
    api.linear_act(x, w, None, yq=q, ys=s)
    v = nan_like(torch, (rows, Cy), torch.float32)
    api.ckpt_unpack(q, s, v)
    want = rounded(torch, x.double() @ w.double().t())
    ordered = rounded(torch, in_order(torch, x.float().t().contiguous(), w.float().t().contiguous()).double())
    assert int((v.double() != want).sum()) <= 2 * int((ordered != want).sum())
