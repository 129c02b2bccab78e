"""The epilogue's reference against published and independent values (CPU)."""
import numpy as np
import torch

from tests import epilogue_reference as E


def words(s):
    return np.array([int(v, 16) for v in s.split()], dtype=np.uint64)


def test_philox_known_answers():
    """The generator's published known-answer vectors (Philox 4x32, 10 rounds)."""
    for ctr, key, out in (
            ("0 0 0 0", "0 0", "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
            ("ffffffff ffffffff ffffffff ffffffff", "ffffffff ffffffff", "408f276d 41c83b0e a20bc7c6 6d5451fd"),
            ("243f6a88 85a308d3 13198a2e 03707344", "a4093822 299f31d0", "d16cfe09 94fdcceb 5001e420 24126ea1")):
        assert np.array_equal(E.philox(words(ctr), words(key)), words(out))


def test_keep_share_and_scale():
    for p in (0.1, 0.5, 0.9):
        k = E.keep((123, 456), 400, 1003, p)
        n, share = k.size, (k > 0).mean()
        assert abs(share - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5 + 2.0 ** -16
        t = int(65536 * float(np.float32(p)) + 0.5)
        assert set(np.unique(k)) == {0.0, 65536 / (65536 - t)}
    assert (E.keep((1, 2), 4, 9, 0.0) == 1).all() and (E.keep((1, 2), 4, 9, 1.0) == 0).all()
    assert (E.keep((1, 2), 4, 9, 2.0 ** -18) == 1).all()


def test_masks_differ_by_key_offset_and_row():
    a = E.keep((1, 2), 64, 64, 0.5)
    for other in (E.keep((2, 2), 64, 64, 0.5), E.keep((1, 3), 64, 64, 0.5), E.keep((1 + 2 ** 32, 2), 64, 64, 0.5),
                  E.keep((1, 2 + 2 ** 32), 64, 64, 0.5), np.roll(a, 1, axis=0), np.roll(a, 8, axis=1)):
        assert 0.4 < (a == other).mean() < 0.6


def test_activations_against_torch_and_slopes_against_differences():
    h = np.linspace(-12, 12, 4801)
    t = torch.tensor(h, requires_grad=True)
    F = torch.nn.functional
    fns = {E.RELU: F.relu, E.SILU: F.silu, E.GELU: F.gelu, E.GELU_TANH: lambda v: F.gelu(v, approximate="tanh")}
    for a, f in fns.items():
        y = f(t)
        assert np.allclose(E.act(h, a), y.detach().numpy(), rtol=1e-12, atol=1e-14)
        g, = torch.autograd.grad(y.sum(), t)
        assert np.allclose(E.slope(h, a), g.numpy(), rtol=1e-10, atol=1e-13)
        d = 1e-5
        away = np.abs(h) > 1e-3  # relu's corner
        diff = (E.act(h + d, a) - E.act(h - d, a)) / (2 * d)
        assert np.allclose(E.slope(h, a)[away], diff[away], rtol=1e-6, atol=1e-9)
    assert all(E.act(np.array([-np.inf]), a)[0] == 0 for a in fns)
