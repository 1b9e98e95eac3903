"""GPU rotation by far positions against the fp64 oracle.

Bound, with U = 2^-24.  The angle: frequencies are turns within 2^-65, so that a position p adds |p| 2^-65 turns;
its rest of at most pi/4 is rounded three times (to fp32 and by the product, U each, and by 2 pi 2^-32 in fp32, 0.47
U): 1.95 U. Of a cosine (at most 0.71 of the angle's error, and 0.5 + 0.25 + 0.15 U of its last sums and z) or a sine
(0.5 U of its last sum beside the angle's) that and the product with the scale, U, leave at most 4 U of scale;
the two products and their sum add 2 U of their magnitudes: |y - y'| <= (6 U + 2 pi |p| 2^-65) scale (|u| + |v|)."""
import ctypes
import threading

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


class Tensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("x_strides", ctypes.c_int64 * 3), ("out_strides", ctypes.c_int64 * 3)]


def test_two_threads_at_once():
    """The C entry point called by two threads on streams of their own (the interpreter lets go during a call):
    tokens of dense rows at odd offsets that need 98 and 51 KB of shared memory, by the same kernel."""
    lib, w = mk.load_library(), 257
    f = mk.rotary_frequencies(256)
    freqs = (ctypes.c_double * 128)(*f.tolist())
    made = []
    for heads in (95, 50):
        gen = torch.Generator(device="cuda").manual_seed(heads)
        x = torch.randn(3, heads, w, generator=gen, device="cuda")
        p = torch.randint(0, 1 << 20, (3,), generator=gen, device="cuda")
        made.append((heads, x, p, mk.rotary(x, p, f, True), torch.zeros_like(x), torch.cuda.Stream()))
    torch.cuda.synchronize()
    codes = [[], []]

    def call(k):
        heads, x, p, _, out, stream = made[k]
        strides = (ctypes.c_int64 * 3)(3 * heads * w, heads * w, w)
        t = Tensor(x.data_ptr(), out.data_ptr(), heads, strides, strides)
        for _ in range(2000):
            codes[k].append(lib.mttkrp_rotary(1, ctypes.byref(t), 0, 1, 3, w, p.data_ptr(), 8, 0, 1, freqs, 256, 1, 1.0, 0,
                                              stream.cuda_stream))

    threads = [threading.Thread(target=call, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert set(codes[0] + codes[1]) == {0}
    for _, _, _, want, out, _ in made:
        assert torch.equal(out, want)
