"""The fp64 oracle of the MLP-block operators against differences, hand-made
checkpoints and identities (CPU)."""

import numpy as np
import pytest

from oracle import block_oracle as O


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def test_checkpoint_of_hand_made_groups():
    t = np.zeros((6, 130))
    t[0, 0] = 127.0          # exactly 127 steps of 1
    t[1, 0] = 127.25         # just above: steps of 2
    t[2, 5] = -1e-300        # below the smallest step
    t[3, 7] = np.inf
    t[4, 129] = 0.75         # the short last group has its own scale
    t[5, :3] = [64.0, 0.5, 1.5]   # steps of 1: ties go to even
    s = O.ckpt_scales(t)
    assert s[0, 0] == 1.0 and s[1, 0] == 2.0 and s[2, 0] == 2.0 ** -120 and np.isnan(s[3, 0])
    assert s[4, 0] == 2.0 ** -120 and s[4, 1] == 2.0 ** -7
    v = O.ckpt_round(t)
    assert v[0, 0] == 127 and v[1, 0] == 128 and v[2, 5] == 0 and np.isnan(v[3]).sum() == 128
    assert v[4, 129] == 0.75 and list(v[5, :3]) == [64, 0, 2]
    q, c = O.ckpt_encode(t)
    assert q.shape == (6, 144) and c.shape == (2, 6) and c[0, 3] == 255
    assert np.array_equal(O.ckpt_decode(q, c, 130), v, equal_nan=True)


def test_checkpoint_error_is_half_a_step():
    t = rng(1).standard_normal((40, 300)) * np.exp(rng(2).standard_normal((40, 1)) * 8)
    s = np.repeat(O.ckpt_scales(t), 128, axis=1)[:, :300]
    assert (np.abs(O.ckpt_round(t) - t) <= 0.5 * s).all()
    top = np.abs(t[:, :128]).max(1)
    assert (top <= 127 * s[:, 0]).all() and (top > 63.5 * s[:, 0]).all()


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
def test_slopes_are_differences(kind):
    z = np.linspace(-6, 6, 241) + 0.013
    e = 1e-5
    d = (O.act(z + e, kind) - O.act(z - e, kind)) / (2 * e)
    assert np.abs(d - O.act_slope(z, kind)).max() < 1e-8


def test_gradients_are_differences():
    """Norm, two linears with an activation between and the residual around
    them, all unrounded: the oracle's gradients against central differences."""
    g = rng(3)
    n, C, H = 3, 5, 7
    x, gamma = g.standard_normal((n, C)), 1 + 0.1 * g.standard_normal(C)
    w1, b1 = g.standard_normal((H, C)), g.standard_normal(H)
    w2, b2 = g.standard_normal((C, H)), g.standard_normal(C)
    gy = g.standard_normal((n, C))

    def loss(x, gamma, w1, b1, w2, b2):
        h, _, _, y = O.rms_norm(x, gamma)
        _, a = O.linear_act(y, w1, b1, "gelu")
        return (O.linear_act(a, w2, b2, residual=h)[1] * gy).sum()

    h, r, u, y = O.rms_norm(x, gamma)
    z, a = O.linear_act(y, w1, b1, "gelu")
    gw2, gb2 = O.grad_w(gy, a)
    gz = O.linear_act_grad(gy, w2, z, "gelu")
    gw1, gb1 = O.grad_w(gz, u, gamma)
    gx, ggamma = O.rms_norm_backward(O.linear_act_grad(gz, w1), u, r, gamma, gy)
    p = [x, gamma, w1, b1, w2, b2]
    for i, want in enumerate([gx, ggamma, gw1, gb1, gw2, gb2]):
        for j in np.ndindex(p[i].shape):
            e = 1e-6
            hi, lo = [q.copy() for q in p], [q.copy() for q in p]
            hi[i][j] += e
            lo[i][j] -= e
            assert abs((loss(*hi) - loss(*lo)) / (2 * e) - want[j]) < 1e-7 * (1 + abs(want[j]))
