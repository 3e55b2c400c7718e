"""Refusals of the operators at the ends of a language model, answered on the host
before anything touches a GPU."""

import ctypes

import pytest

OK, ARG, SHAPE, DTYPE, ALIGN, WORKSPACE = range(6)
F = ctypes.c_void_p(0x1000)     # never dereferenced: validation returns first
ODD = ctypes.c_void_p(0x1008)
ODDER = ctypes.c_void_p(0x1002)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from rank_compressed_backprop_gb300.build import build

    build()
    from rank_compressed_backprop_gb300._lib import lib

    return lib()


def refused(fn, good, cases):
    for pos, value, status in cases:
        args = list(good)
        args[pos] = value
        assert fn(*args) == status, (pos, value)


def test_embed_refusals(L):
    n0 = L.instant_launch_count()
    # tokens, token_bytes, table, y, rows, V, C, scale, dt, stream
    refused(L.instant_embed, [F, 8, F, F, 4, 100, 64, 1.0, 1, None],
            [(0, None, ARG), (2, None, ARG), (3, None, ARG), (1, 2, DTYPE), (1, 0, DTYPE), (4, 0, SHAPE),
             (4, (1 << 30) + 1, SHAPE), (5, 0, SHAPE), (5, (1 << 24) + 1, SHAPE), (6, 0, SHAPE), (6, 65544, SHAPE),
             (6, 60, ALIGN), (7, NAN, ARG), (7, INF, ARG), (8, 2, DTYPE), (0, ODDER, ALIGN), (2, ODD, ALIGN),
             (3, ODD, ALIGN)])
    need = L.instant_embed_grad_workspace_bytes(4, 100, 64)
    assert need > 0
    for bad in ((0, 100, 64), (4, 0, 64), (4, 100, 0), (4, 100, 65537), (-1, 100, 64)):
        assert L.instant_embed_grad_workspace_bytes(*bad) == 0
    # gy, tokens, token_bytes, gtable, accumulate, ws, ws_bytes, rows, V, C, scale, dt, stream
    refused(L.instant_embed_grad, [F, F, 4, F, 0, F, 1 << 20, 4, 100, 64, 1.0, 1, None],
            [(0, None, ARG), (1, None, ARG), (3, None, ARG), (2, 3, DTYPE), (5, None, WORKSPACE),
             (6, need - 1, WORKSPACE), (7, 0, SHAPE), (8, 0, SHAPE), (9, 0, SHAPE), (9, 60, ALIGN), (10, NAN, ARG),
             (11, 5, DTYPE), (0, ODD, ALIGN), (1, ODDER, ALIGN), (3, ODD, ALIGN), (5, ODD, ALIGN)])
    assert L.instant_launch_count() == n0


def test_token_logprobs_refusals(L):
    n0 = L.instant_launch_count()
    # x, tokens, token_bytes, logp, stats, entropy, top_ids, top_logp, rows, V, ld, top, scale, dt, stream
    good = [F, F, 8, F, F, F, F, F, 4, 100, 104, 5, 1.0, 1, None]
    refused(L.instant_token_logprobs, good,
            [(0, None, ARG), (1, None, ARG), (2, 1, DTYPE), (8, 0, SHAPE), (9, 0, SHAPE), (9, 105, SHAPE),
             (10, 99, SHAPE), (10, (1 << 24) + 1, SHAPE), (11, -1, SHAPE), (11, 33, SHAPE), (11, 0, ARG),
             (12, 0.0, ARG), (12, -1.0, ARG), (12, NAN, ARG), (12, INF, ARG), (13, 7, DTYPE), (0, ODD, ALIGN),
             (1, ODDER, ALIGN), (3, ODDER, ALIGN), (4, ctypes.c_void_p(0x1004), ALIGN), (5, ODDER, ALIGN),
             (6, ctypes.c_void_p(0x1004), ALIGN), (7, ODDER, ALIGN)])
    assert L.instant_token_logprobs(F, F, 8, F, F, F, F, F, 4, 3, 104, 5, 1.0, 1, None) == SHAPE  # top > V
    assert L.instant_token_logprobs(F, F, 8, F, F, F, None, None, 4, 100, 104, 5, 1.0, 1, None) == ARG
    assert L.instant_token_logprobs(F, F, 8, None, None, None, None, None, 4, 100, 104, 0, 1.0, 1, None) == ARG
    # x, tokens, token_bytes, stats, g_logp, g_entropy, entropy, gx, rows, V, ld, scale, dt, stream
    good = [F, F, 4, F, F, F, F, F, 4, 100, 104, 1.0, 1, None]
    refused(L.instant_token_logprobs_grad, good,
            [(0, None, ARG), (1, None, ARG), (2, 5, DTYPE), (3, None, ARG), (5, None, ARG), (6, None, ARG),
             (7, None, ARG), (8, 0, SHAPE), (9, 0, SHAPE), (10, 99, SHAPE), (11, 0.0, ARG), (11, NAN, ARG),
             (12, 2, DTYPE), (0, ODD, ALIGN), (3, ctypes.c_void_p(0x1004), ALIGN), (7, ODD, ALIGN),
             (4, ODDER, ALIGN)])
    assert L.instant_token_logprobs_grad(F, F, 4, F, None, None, None, F, 4, 100, 104, 1.0, 1, None) == ARG
    assert L.instant_launch_count() == n0


def test_scales_that_no_logits_are_multiplied_by(L):
    for scale in (2.0 ** -121, 2.0 ** 121, 3e38, 1e-45, -2.0):
        assert L.instant_token_logprobs(F, F, 8, F, F, F, F, F, 4, 100, 104, 5, scale, 1, None) == ARG
        assert L.instant_token_logprobs_grad(F, F, 4, F, F, F, F, F, 4, 100, 104, scale, 1, None) == ARG


def test_grad_clip_refusals(L):
    from rank_compressed_backprop_gb300._lib import GradItem

    n0 = L.instant_launch_count()
    assert L.instant_grad_clip_workspace_bytes(0) == 0 and L.instant_grad_clip_workspace_bytes(-3) == 0
    need = L.instant_grad_clip_workspace_bytes(2)
    assert 0 < need < L.instant_grad_clip_workspace_bytes(1001)

    def call(items, max_norm=1.0, scale=1.0, norm=F, ws=F, ws_bytes=1 << 20, count=None):
        arr = (GradItem * max(1, len(items)))(*[GradItem(*i) for i in items])
        return L.instant_grad_clip(arr, len(items) if count is None else count, max_norm, scale, norm, ws, ws_bytes,
                                   None)

    a = (0x1000, 0x2000, 8, 0)
    assert L.instant_grad_clip(None, 1, 1.0, 1.0, F, F, 1 << 20, None) == ARG
    for kw, status in [(dict(max_norm=0.0), ARG), (dict(max_norm=-1.0), ARG), (dict(max_norm=NAN), ARG),
                       (dict(scale=0.0), ARG), (dict(scale=INF), ARG), (dict(scale=NAN), ARG), (dict(norm=None), ARG),
                       (dict(ws=None), WORKSPACE), (dict(ws_bytes=need - 1), WORKSPACE), (dict(ws=ODD), ALIGN),
                       (dict(norm=ctypes.c_void_p(0x1004)), ALIGN), (dict(count=0), ARG)]:
        assert call([a, a], **kw) == status, kw
    for item, status in [((0, 0x2000, 8, 0), ARG), ((0x1000, 0, 8, 0), ARG), ((0x1000, 0x2000, -1, 0), SHAPE),
                         ((0x1000, 0x2000, (1 << 45) + 1, 0), SHAPE), ((0x1000, 0x2000, 8, 2), DTYPE),
                         ((0x1002, 0x2000, 8, 0), ALIGN), ((0x1000, 0x2001, 8, 1), ALIGN)]:
        assert call([a, item]) == status, item
    assert L.instant_launch_count() == n0


def test_python_binding_refusals(L):
    torch = pytest.importorskip("torch")
    from rank_compressed_backprop_gb300 import api

    bf = torch.bfloat16
    tok, table, y = torch.zeros(3, dtype=torch.int64), torch.zeros(10, 8, dtype=bf), torch.zeros(3, 8, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        api.embed(tok, table, y)
    with pytest.raises(ValueError, match="tokens must be a vector"):
        api.embed(tok[None], table, y)
    with pytest.raises(TypeError, match="int32 or int64"):
        api.embed(tok.float(), table, y)
    with pytest.raises(ValueError, match=r"y must be \[3, 8\]"):
        api.embed(tok, table, y[:2])
    with pytest.raises(TypeError):
        api.embed(tok, table, y.float())
    with pytest.raises(TypeError):
        api.embed(tok, table, [1])
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        api.embed_grad(y, tok, torch.zeros(10, 8), ws)
    with pytest.raises(TypeError):
        api.embed_grad(y, tok, torch.zeros(10, 8, dtype=bf), ws)
    with pytest.raises(ValueError, match=r"tokens must be \[3\]"):
        api.embed_grad(y, tok[:2], torch.zeros(10, 8), ws)
    x, p = torch.zeros(3, 16, dtype=bf), torch.zeros(3)
    with pytest.raises(ValueError, match="CUDA"):
        api.token_logprobs(x, tok, p)
    with pytest.raises(ValueError, match="a vocabulary of 17"):
        api.token_logprobs(x, tok, p, vocab=17)
    with pytest.raises(ValueError, match="needs tokens"):
        api.token_logprobs(x, None, p)
    with pytest.raises(ValueError, match="1 to 16 alternatives"):
        api.token_logprobs(x, tok, p, top_ids=torch.zeros(3, 17, dtype=torch.int64))
    with pytest.raises(ValueError, match="as many as the other"):
        api.token_logprobs(x, tok, p, top_ids=torch.zeros(3, 2, dtype=torch.int64), top_logp=torch.zeros(3, 3))
    with pytest.raises(TypeError):
        api.token_logprobs(x, tok, p, top_ids=torch.zeros(3, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match=r"stats must be \[3, 2\]"):
        api.token_logprobs(x, tok, p, stats=torch.zeros(3))
    st = torch.zeros(3, 2)
    with pytest.raises(ValueError, match="come together"):
        api.token_logprobs_grad(x, tok, st, x, g_logp=p, g_entropy=p)
    with pytest.raises(ValueError, match="give g_logp"):
        api.token_logprobs_grad(x, tok, st, x)
    with pytest.raises(ValueError, match=r"g_logits must be \[3, 16\]"):
        api.token_logprobs_grad(x, tok, st, x[:, :8], g_logp=p)
    with pytest.raises(ValueError, match="CUDA"):
        api.token_logprobs_grad(x, tok, st, x, g_logp=p)
    with pytest.raises(ValueError, match="a list of gradients"):
        api.GradClip([])
    with pytest.raises(ValueError, match="CUDA"):
        api.GradClip([p])


def test_the_alternatives_limit_is_the_headers(L):
    import os
    import re

    from rank_compressed_backprop_gb300._lib import TOP_MAX

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "instant.h")).read()
    assert int(re.search(r"#define INSTANT_TOP_MAX (\d+)", text).group(1)) == TOP_MAX
