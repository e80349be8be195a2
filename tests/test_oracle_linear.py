"""The oracle's linear layer (CPU only): the generator against its published
known answers, the mask's definition element by element, and every gradient
against central differences of the forward formula in float64."""

import numpy as np
import pytest
import torch

from oracle import linear as OL

# Philox-4x32-10's published known answers: counter, key, output
KNOWN = [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
]


@pytest.mark.parametrize("counter,key,out", KNOWN)
def test_philox_known_answers(counter, key, out):
    got = OL.philox([np.array([c], dtype=np.uint64) for c in counter], key)
    assert tuple(int(w[0]) for w in got) == out


def test_mask_element_by_element():
    rows, cols, p, seed, offset = 3, 19, 0.3, 0x0123456789ABCDEF, (5 << 40) + 7
    f = OL.keep_factor(rows, cols, p, seed, offset)
    t = round(p * 65536)
    for i in range(rows):
        for j in range(cols):
            b = i * 3 + j // 8
            w = OL.philox([np.array([v], dtype=np.uint64) for v in
                           (b, 0, offset & OL.M32, offset >> 32)], (seed & OL.M32, seed >> 32))
            bits = (int(w[(j % 8) // 2][0]) >> (16 * (j % 2))) & 0xFFFF
            assert f[i, j] == (65536 / (65536 - t) if bits >= t else 0.0)


def test_mask_of_later_rows():
    whole = OL.keep_factor(20, 33, 0.4, 8, 9)
    assert np.array_equal(whole[7:], OL.keep_factor(13, 33, 0.4, 8, 9, first=7))


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 2.0 ** -16, 0.1, 0.5, 1.0 - 2.0 ** -16, 1.0])
def test_mask_rate(p):
    f = OL.keep_factor(256, 256, p, 1, 2)
    t = round(p * 65536)
    share = t / 65536
    # the number dropped is binomial: within 6 standard deviations
    assert abs((f == 0).mean() - share) <= 6 * np.sqrt(share * (1 - share) / f.size)
    assert np.all((f == 0) | (f == (65536 / (65536 - t) if t < 65536 else 0)))


def test_masks_of_other_offsets_seeds_and_widths_differ():
    base = OL.keep_factor(64, 64, 0.5, 1, 2)
    for other in (OL.keep_factor(64, 64, 0.5, 1, 3), OL.keep_factor(64, 64, 0.5, 2, 2),
                  OL.keep_factor(64, 64, 0.5, 1, 2 + (1 << 32)), OL.keep_factor(64, 64, 0.5, 1 + (1 << 32), 2)):
        same = ((base == 0) == (other == 0)).mean()
        assert abs(same - 0.5) < 6 * 0.5 / 64


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
def test_activation_against_torch_and_differences(name):
    z = np.concatenate([np.linspace(-9, 9, 1801), [1e-3, -1e-3]])
    z = z[np.abs(z) > 1e-5]  # relu has no slope at 0
    t = torch.from_numpy(z)
    ref = {"none": t, "relu": torch.relu(t), "gelu": torch.nn.functional.gelu(t),
           "silu": torch.nn.functional.silu(t)}[name].numpy()
    assert np.allclose(OL.act(z, name), ref, rtol=1e-12, atol=1e-15)
    h = 1e-5
    diff = (OL.act(z + h, name) - OL.act(z - h, name)) / (2 * h)
    # central differences: h^2 / 6 times a third derivative below 2, and 2^-53 |z| / h
    assert np.allclose(OL.act_grad(z, name), diff, rtol=0, atol=2e-10)
    assert np.all(OL.act_grad_slack(z, name) >= np.abs(OL.act_grad(z, name)) - 1e-15)


@pytest.mark.parametrize("name", ["relu", "gelu", "silu"])
def test_slope_at_nan_is_nan(name):
    z = np.array([np.nan, -1.0, 1.0])
    assert np.array_equal(np.isnan(OL.act_grad(z, name)), [True, False, False])
    assert np.array_equal(np.isnan(OL.act(z, name)), [True, False, False])


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
def test_layer_gradients_against_differences(name):
    rng = np.random.default_rng(3)
    m, n, k = 4, 5, 3
    x, w, b, dy = (rng.standard_normal(s) for s in ((m, k), (n, k), (n,), (m, n)))
    d = OL.keep_factor(m, n, 0.4, 11, 12)

    def loss(x, w, b):
        return float(np.sum(dy * OL.act(OL.product(x, w)[0] + b, name) * d))

    z = OL.product(x, w)[0] + b
    assert np.abs(z).min() > 1e-3
    dz = dy * d * OL.act_grad(z, name)
    grads = {"x": OL.product(dz, w.T)[0], "w": OL.product(dz.T, x.T)[0], "b": dz.sum(0)}
    h = 1e-5
    for which, g in grads.items():
        args = {"x": x, "w": w, "b": b}
        for at in np.ndindex(g.shape):
            up, down = ({**args, which: args[which].copy()} for _ in range(2))
            up[which][at] += h
            down[which][at] -= h
            diff = (loss(**up) - loss(**down)) / (2 * h)
            assert abs(diff - g[at]) < 1e-8, (which, at)
