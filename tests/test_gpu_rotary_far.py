"""GPU rotation by far positions against the fp64 oracle.

Bound, with U = 2^-24.  The angle: frequencies are turns within 2^-65, so that a position p adds |p| 2^-65 turns;
its rest of at most pi/4 is rounded three times (to fp32 and by the product, U each, and by 2 pi 2^-32 in fp32, 0.47
U): 1.95 U. Of a cosine (at most 0.71 of the angle's error, and 0.5 + 0.25 + 0.15 U of its last sums and z) or a sine
(0.5 U of its last sum beside the angle's) that and the product with the scale, U, leave at most 4 U of scale;
the two products and their sum add 2 U of their magnitudes: |y - y'| <= (6 U + 2 pi |p| 2^-65) scale (|u| + |v|)."""
import numpy as np
import pytest

from oracle import orthogonal as oo

torch = pytest.importorskip("torch")
import dense_tensor_decomposition_gb300 as mk  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("width", [24, 25])
def test_far_positions(interleaved, width):
    """Both signs of both, frequencies of all sizes; rows at odd offsets too."""
    f = torch.tensor([1.0, -0.37, 1e-5, -1e-5, 2 * np.pi, 7.5, 1e-12, -1e-12, 0.999, 1e-9, 3.0, 0.01], dtype=torch.float64)
    p = torch.tensor([0, 1, -1, 1 << 20, -(1 << 26) - 1, (1 << 31) - 1, -(1 << 31), (1 << 36) + 777, (1 << 40) + 12345,
                      -(1 << 40) - 1], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(len(p), 5, width, generator=gen, device="cuda")
    got = mk.rotary(x, p, f, interleaved)
    want = oo.rotary(x.double().cpu(), p.cpu().numpy(), f.numpy(), interleaved)
    mag = x[..., :24].abs().double().cpu().numpy()
    both = np.repeat(mag[..., 0::2] + mag[..., 1::2], 2, -1) if interleaved else np.tile(mag[..., :12] + mag[..., 12:], 2)
    # the oracle's angles have 64 bits: p f 2^-64 radians (of at most 7.5 p)
    far = np.abs(p.cpu().numpy().astype(float))[:, None, None]
    bound = (6 * U + far * (2 * np.pi * 2.0 ** -65 + 7.5 * 2.0 ** -64)) * both + 2.0 ** -149
    err = np.abs(got.double().cpu().numpy()[..., :24] - want[..., :24])
    assert np.all(err <= bound), (err / bound).max(axis=(1, 2))
    assert torch.equal(got[..., 24:], x[..., 24:])
    back = mk.rotary_grad(got, p, f, interleaved)
    assert np.all(np.abs((back - x)[..., :24].double().cpu().numpy()) <= 16 * U * both * 2)
