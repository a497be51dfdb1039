"""Pins of the numpy oracle of the 4-bit cache and of the rotary append."""
import numpy as np
import torch

from oracle import q4


def test_e4m3_table_and_rounding():
    bits = torch.arange(127, dtype=torch.uint8)
    np.testing.assert_array_equal(bits.view(torch.float8_e4m3fn).double().numpy(), q4.E4M3)
    x = torch.rand(5000, generator=torch.Generator().manual_seed(1)) * \
        torch.exp(4 * torch.randn(5000, generator=torch.Generator().manual_seed(2)))
    want = x.clamp_max(448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(q4.nearest(x.numpy(), q4.E4M3), want)


def test_bf16_is_torch_s():
    x = torch.randn(5000, generator=torch.Generator().manual_seed(3), dtype=torch.float64) * 7
    np.testing.assert_array_equal(q4.bf16(x.numpy()), x.float().bfloat16().double().numpy())


def test_ties_go_to_the_even_code():
    x = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0,
                   -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0]])
    code, s = q4.quantise(x, np.ones((1, 1), np.float32))
    assert s[0, 0] == 0x38                                  # 1.0
    np.testing.assert_array_equal(code[0] & 7, [0, 2, 2, 4, 4, 6, 6, 7] * 2)
    np.testing.assert_array_equal(code[0] >> 3, [0] * 8 + [1] * 8)


def test_quantise_is_nearest_and_packs():
    rng = np.random.default_rng(4)
    x = q4.bf16(rng.standard_normal((50, 64)))
    code, s = q4.quantise(x, np.ones((50, 1), np.float32))
    v = q4.values(code, s)
    t = np.repeat(q4.E4M3[s], 16, axis=1)
    for c in range(16):                                     # no other code is nearer
        other = (-q4.E2M1[c & 7] if c >= 8 else q4.E2M1[c & 7]) * t
        assert (np.abs(v - x) <= np.abs(other - x)).all()
    np.testing.assert_array_equal(q4.unpack(q4.pack(code)), code)
    amax = np.abs(x).reshape(50, 4, 16).max(-1)
    assert (np.abs(q4.E4M3[s] - amax / 6) <= amax / 6 * 2.0 ** -4 * (1 + 1e-12)).all()


def test_rotation_turns_pairs():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 2, 32))
    inv = 1e4 ** (-np.arange(0, 16, 2) / 16)
    pos = np.array([0, 7, 123456])
    half = q4.rotate(x, pos, inv, 16, False)
    adjacent = q4.rotate(x, pos, inv, 16, True)
    np.testing.assert_array_equal(half[0], x[0])            # position 0
    np.testing.assert_array_equal(half[..., 16:], x[..., 16:])
    z = (x[..., :8] + 1j * x[..., 8:16]) * np.exp(1j * pos[:, None, None] * inv)
    np.testing.assert_allclose(half[..., :8] + 1j * half[..., 8:16], z, rtol=0, atol=1e-9)
    z = (x[..., 0:16:2] + 1j * x[..., 1:16:2]) * np.exp(1j * pos[:, None, None] * inv)
    np.testing.assert_allclose(adjacent[..., 0:16:2] + 1j * adjacent[..., 1:16:2], z, rtol=0, atol=1e-9)


def test_attention_is_torch_s():
    rng = np.random.default_rng(6)
    q, k, v = rng.standard_normal((4, 8)), rng.standard_normal((11, 8)), rng.standard_normal((11, 8))
    limit = np.array([1, 5, 11, 0])
    o, lse, a, mag, vsum = q4.attention(q, k, v, limit, 0.3)
    for i, n in enumerate(limit):
        if n == 0:
            assert (o[i] == 0).all() and lse[i] == -np.inf
            continue
        x = torch.tensor(q[i] @ k[:n].T * 0.3)
        np.testing.assert_allclose(o[i], torch.softmax(x, 0).numpy() @ v[:n], atol=1e-12)
        np.testing.assert_allclose(lse[i], torch.logsumexp(x, 0).item(), atol=1e-12)
    assert (a >= np.abs(o) - 1e-12).all() and np.allclose(vsum, np.abs(v).sum(0))
