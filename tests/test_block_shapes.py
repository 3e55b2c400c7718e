"""Tensors that are no matrices are refused by name, before anything touches a GPU."""

import pytest

torch = pytest.importorskip("torch")
bf = torch.bfloat16


@pytest.fixture(scope="module")
def api():
    from rank_compressed_backprop_gb300.build import build

    build()
    from rank_compressed_backprop_gb300 import api

    return api


X, W, Y = (torch.zeros(*s, dtype=bf) for s in ((3, 64), (72, 64), (3, 72)))
Q, S = torch.zeros(3, 64, dtype=torch.int8), torch.zeros(1, 3, dtype=torch.uint8)
GW, G, WS = torch.zeros(72, 64), torch.zeros(64), torch.zeros(1 << 16, dtype=torch.uint8)
R = torch.zeros(3)
CALLS = {
    "ckpt_pack": ([X, Q, S], {"x": 0}),
    "ckpt_unpack": ([Q, S, X], {"x": 2}),
    "rms_norm": ([X, G.to(bf), X], {"x": 0}),
    "rms_norm_backward": ([X, Q, S, R, G.to(bf), X, G, WS], {"g_y": 0}),
    "linear_act": ([X, W, Y], {"x": 0, "w": 1}),
    "linear_act_grad": ([Y, W, X], {"g_y": 0, "w": 1}),
    "ckpt_grad_w": ([Y, Q, S, GW], {"g_y": 0, "gw": 3}),
}


@pytest.mark.parametrize("name,arg", [(n, a) for n, (_, args) in CALLS.items() for a in args])
@pytest.mark.parametrize("shape", [(), (64,), (1, 3, 64)])
def test_a_matrix_is_asked_for(api, name, arg, shape):
    good, at = CALLS[name]
    args = list(good)
    args[at[arg]] = torch.zeros(shape, dtype=good[at[arg]].dtype)
    with pytest.raises(ValueError, match=f"{name}: {arg} must be a matrix"):
        getattr(api, name)(*args)


@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_is_asked_for(api, name):
    good, at = CALLS[name]
    for arg, i in at.items():
        args = list(good)
        args[i] = [[1.0, 2.0]]
        with pytest.raises(TypeError, match=f"{arg} must be a torch.Tensor"):
            getattr(api, name)(*args)


@pytest.mark.parametrize("name", CALLS)
def test_the_good_calls_fail_for_their_device_only(api, name):
    with pytest.raises(ValueError, match="CUDA"):
        getattr(api, name)(*CALLS[name][0])
