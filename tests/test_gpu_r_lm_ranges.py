"""The operators at the ends of a language model over the whole range of their values and
sizes: finite masks of any size, logits around the bound between the two forms of an
exponent, gradients around the bounds between the sums of their squares."""

import numpy as np
import pytest

from gpu_util import nan_like, rng, stored, torch_or_skip
from test_gpu_p_lm import H, U, check_clip, check_logprobs, check_logprobs_grad, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return torch_or_skip()


def _api():
    from rank_compressed_backprop_gb300 import api

    return api


# ---------------------------------------------------------------------------
# finite masks and large logits
# ---------------------------------------------------------------------------
FILLS = [1e4, 1e6, 1e9, 1e10, 1e12, 1e15, 1e20, 1e30, 1e36, 2e36, 1e38]
KINDS = ["whole", "few", "front", "back", "edge", "some", "large", "peak", "rising", "falling", "border", "minus_border"]


def masked_row(g, kind, fill, V, scale):
    """Ordinary logits of which some are -fill (kinds up to "some"), or logits as large as fill, or
    ones that lie around the 2^20 / (scale log2 e) beyond which an exponent is a difference's."""
    x = g.standard_normal(V) * 2.5
    if kind == "whole":
        x[:] = -fill
    elif kind == "few":            # constrained decoding: some tokens allowed
        keep = g.integers(0, V, 5)
        x, ordinary = np.full(V, -fill), x
        x[keep] = ordinary[keep]
    elif kind == "front":
        x[:V - V // 3] = -fill
    elif kind == "back":
        x[V // 3:] = -fill
    elif kind == "edge":           # outside the vectors, where the row is not aligned
        x[[0, -1]] = -fill
    elif kind == "some":
        x[g.random(V) < 0.2] = -fill
    elif kind == "large":
        x[:] = fill
    elif kind == "peak":
        x[g.integers(0, V, 3)] = fill
    elif kind in ("rising", "falling"):
        x = np.linspace(-fill, fill, V)[::1 if kind == "rising" else -1]
    else:
        x = x + 2 ** 20 / (scale * np.log2(np.e))
        x = x if kind == "border" else -x
    return x


def masked_rows(rows, V, scale, dtype):
    g = rng(rows + V)
    each = [(k, f) for f in FILLS for k in KINDS]
    # 59 has no factor with the 132 combinations: any number of rows takes fills and kinds of all sorts
    return stored(np.array([masked_row(g, *each[59 * i % len(each)], V, scale) for i in range(rows)]), dtype)


MASKED = [(132, 9001), (70, 30523), (16, 70001), (330, 4203), (660, 4203), (1320, 4201)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", MASKED)
@pytest.mark.parametrize("scale", [0.7, 1.0, 1.5])
def test_finite_masks_and_large_logits(torch, dtype, rows, V, scale):
    """Clusters of several sizes and every size of a CTA; rows of odd length that start anywhere."""
    x = masked_rows(rows, V, scale, dtype)
    tok = rng(V).integers(0, V, rows)
    k = (1, 5, 20)[V % 3]
    check_logprobs(torch, x, V, tok, scale, k, dtype)
    check_logprobs(torch, x, V, tok, scale, 0, dtype)
    check_logprobs_grad(torch, x, V, tok, scale, dtype, "both")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_finite_masks_in_one_row_over_a_cluster(torch, dtype, kind):
    """A generated token's row, a call for each size of the mask."""
    g, V = rng(17), 128000
    for fill in FILLS:
        x = stored(masked_row(g, kind, fill, V, 1.25)[None], dtype)
        check_logprobs(torch, x, V, np.array([g.integers(0, V)]), 1.25, 20, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 9, 255])
def test_finite_masks_in_short_rows(torch, dtype, V):
    """Rows of no or few vectors: most of their elements are edges."""
    g = rng(V)
    x = stored(np.array([masked_row(g, k, f, V, 1.0) for f in FILLS for k in KINDS]), dtype)
    tok = g.integers(0, V, len(x))
    check_logprobs(torch, x, V, tok, 1.0, 1, dtype)
    check_logprobs_grad(torch, x, V, tok, 1.0, dtype, "logp")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -119.5, 2.0 ** -60, 0.25, 1.0, 2.0 ** 60, 2.0 ** 120])
def test_logits_over_the_whole_range_at_the_smallest_and_largest_scales(torch, dtype, scale):
    """Differences of logits beyond the type's range, whose product with the scale is within it."""
    g = rng(3)
    for rows, V in ((6, 7), (6, 2600), (330, 300)):
        x = g.standard_normal((rows, V)) * 2.5
        x[:, ::3] = g.choice([-3.38e38, -1e38, 1e38], (rows, len(x[0, ::3])))
        x[::2, 1] = 3e38
        x[1::3] = g.standard_normal((len(x[1::3]), V))
        x = stored(x, dtype)
        tok = np.zeros(rows, int)
        check_logprobs(torch, x, V, tok, scale, 2, dtype)
        if scale <= 1:             # beyond, the gradient itself passes the range
            check_logprobs_grad(torch, x, V, tok, scale, dtype, "both")


# ---------------------------------------------------------------------------
# the norm's range
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("size", [1.1 * 2.0 ** 39, 1.9 * 2.0 ** 39, 1.1 * 2.0 ** 40, 1.9 * 2.0 ** 49, 1.1 * 2.0 ** 50, 2.0 ** 63])
def test_the_norm_of_many_large_gradients(torch, size):
    """2^29 bf16 values whose squares add up to more than 2^128, or 2^30 below it: the norm is finite
    in fp32, and clips."""
    api = _api()
    n = 1 << 29
    g = torch.full((n,), size, device="cuda", dtype=torch.bfloat16)
    v = float(g[0])
    norm = nan_like(torch, (2,), torch.float32)
    api.grad_clip([g], 2.0 ** 40, norm)
    want = v * n ** 0.5
    f = min(1.0, 2.0 ** 40 / want)
    # as for other lists: 65 squares of a chunk in fp32, then the root, the quotient and the product
    close(norm, [want, f], np.array([want, f]) * 36 * U, "norm")
    lo, hi = torch.aminmax(g)
    assert float(lo) == float(hi) and abs(float(hi) - v * f) <= v * f * (36 * U + 1.01 * H["bf16"])


@pytest.mark.parametrize("size", [2.0 ** -50, 2.0 ** -49, 2.0 ** 39, 2.0 ** 40, 2.0 ** 49, 2.0 ** 50])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_about_the_bounds_of_plain_squares(torch, size, dtype):
    """Values on both sides of the bounds between sums in fp32 and in 64 bits."""
    g = rng(6)
    a = stored(size * np.exp2(g.uniform(-2, 2, 70001)) * g.choice([-1, 1], 70001), dtype)
    check_clip(torch, [a, stored(size * g.standard_normal(333), dtype)], [dtype] * 2, size)


@pytest.mark.parametrize("count", [32, 33, 120, 121, 128, 129, 400, 401, 512, 513, 940, 941, 1880, 1881])
@pytest.mark.parametrize("in_place", [False, True])
def test_as_many_gradients_as_a_launch_takes_and_one_more(torch, count, in_place):
    g = rng(count)
    dtypes = ["bf16" if i % 4 == 0 else "f32" for i in range(count)]
    check_clip(torch, [stored(g.standard_normal(1 + (i * 37) % 300), d) for i, d in enumerate(dtypes)], dtypes, 1.0,
               in_place=in_place)


@pytest.mark.parametrize("count", [20, 100, 500, 900, 1000])
@pytest.mark.parametrize("in_place,scale", [(False, 1.0), (True, 0.5)])
def test_long_lists_of_many_tensors(torch, count, in_place, scale):
    """More than 64 MB in lists of every size, of two launches too: a CTA a chunk where they are written."""
    api = _api()
    gen = torch.Generator("cuda").manual_seed(count)
    sizes = [40_000_000 // count + (i * 977) % 5000 for i in range(count)]
    g = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
    for i in range(0, count, 3):
        g[i] = g[i].bfloat16()
    keep = [t.clone() for t in g]
    outs = g if in_place else [nan_like(torch, t.shape, t.dtype) for t in g]
    norm = nan_like(torch, (2,), torch.float32)
    api.GradClip(g, None if in_place else outs)(1.0, norm, scale=scale)
    n = scale * float(torch.sqrt(sum(t.double().square().sum() for t in keep)))
    close(norm, [n, 1 / n], np.array([n, 1 / n]) * 36 * U, "norm")
    for o, k in zip(outs, keep):
        want = k.double() * (scale / n)
        h = H["bf16" if o.dtype == torch.bfloat16 else "f32"]
        assert bool(((o.double() - want).abs() <= want.abs() * (36 * U + 1.01 * h)).all())
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(g, keep))


# ---------------------------------------------------------------------------
# more positions than the tiles of a few launches
# ---------------------------------------------------------------------------
def call_ms(torch, f, calls):
    """Time of a call among `calls`, the best of three runs."""
    f()
    best = float("inf")
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(calls):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / calls)
    return best


def test_a_table_gradient_takes_time_in_proportion_to_its_positions(torch):
    """2^29 positions in 32768 tiles against 2^23 in 512."""
    api = _api()
    V, C = 1000, 8
    gen = torch.Generator("cuda").manual_seed(1)
    per = []
    for rows in (1 << 23, 1 << 29):
        tok = torch.randint(0, V, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        gy = torch.ones(rows, C, device="cuda", dtype=torch.bfloat16)
        gt, ws = nan_like(torch, (V, C), torch.float32), api.embed_grad_workspace(rows, V, C, "cuda")
        per.append(call_ms(torch, lambda: api.embed_grad(gy, tok, gt, ws), 2) / rows)
        assert torch.equal(gt, torch.bincount(tok, minlength=V).float()[:, None].expand(V, C))
    assert per[1] <= 1.5 * per[0]


@pytest.mark.parametrize("rows", [199 * 1024, 199 * 1024 + 1, 304 * 1024, 199 * 2048 + 1, 304 * 16384 + 5])
def test_table_gradients_of_as_many_tiles_as_are_scanned(torch, rows):
    """199 and 200 tiles of 1024 positions, 304 of them, 200 of 2048, and more than 304 of 16384."""
    api, V, C = _api(), 70001, 4
    gen = torch.Generator("cuda").manual_seed(rows)
    tok = torch.randint(-3, V, (rows,), generator=gen, device="cuda")
    gy = torch.randint(-8, 9, (rows, C), generator=gen, device="cuda").float()
    ws = api.embed_grad_workspace(rows, V, C, "cuda").fill_(0xff)
    gt = nan_like(torch, (V, C), torch.float32)
    api.embed_grad(gy, tok, gt, ws)
    # small whole numbers: their sums are exact in any order
    want = torch.zeros(V + 1, C, device="cuda", dtype=torch.float64)
    want.index_add_(0, torch.where(tok < 0, V, tok), gy.double())
    assert torch.equal(gt, want[:V].float())
    again = nan_like(torch, (V, C), torch.float32)
    g2 = torch.randn(rows, C, generator=gen, device="cuda")
    api.embed_grad(g2, tok, gt, ws)
    api.embed_grad(g2, tok, again, ws.fill_(0xff))
    assert torch.equal(gt, again)
    assert api.device_status() == 0


# ---------------------------------------------------------------------------
# the largest tables and widths
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,rows,V,C", [("bf16", 300, 1 << 24, 8), ("f32", 5000, 1 << 24, 3), ("f32", 40000, 1 << 24, 4),
                                            ("bf16", 300, 9, 65536), ("bf16", 3000, 9, 65536), ("f32", 300, 9, 65535),
                                            ("f32", 2100, 9, 65535), ("f32", 33000, 5, 4097)])
def test_the_largest_tables_and_widths(torch, dtype, rows, V, C):
    """A table of 2^24 rows takes a fourth pass of the sort; its last rows, its first and none."""
    api = _api()
    gen = torch.Generator("cuda").manual_seed(rows + C)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    tok = torch.randint(0, V, (rows,), generator=gen, device="cuda")
    tok[::3] = V - 1 - torch.arange(len(tok[::3]), device="cuda") % min(V, 11)
    tok[::7] = 0
    tok[::13] = -1
    gy = torch.randint(-8, 9, (rows, C), generator=gen, device="cuda").to(dt)
    ws = api.embed_grad_workspace(rows, V, C, "cuda").fill_(0xff)
    gt = nan_like(torch, (V, C), torch.float32)
    api.embed_grad(gy, tok, gt, ws)
    # whole numbers below 2^24: their sums are exact in any order
    want = torch.zeros(V, C, device="cuda").index_add_(0, tok.clamp(min=0), gy.float() * (tok >= 0)[:, None])
    assert torch.equal(gt, want)
    api.embed_grad(gy, tok, gt, ws, scale=-1.0, accumulate=True)
    assert int(gt.count_nonzero()) == 0
    y = nan_like(torch, (rows, C), dt)
    table = torch.zeros(V, C, device="cuda", dtype=dt)
    table[tok.clamp(min=0)] = gy                       # some position's row for each token
    api.embed(tok, table, y)
    assert torch.equal(y, torch.where((tok >= 0)[:, None], table[tok.clamp(min=0)], 0))
    assert api.device_status() == 0
