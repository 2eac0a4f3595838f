"""The float64 restatements of the norms and of the 8-bit SwiGLU backward,
against differences and hand-derived values (CPU)."""
import numpy as np
import pytest

import block_ref as ref


def grad(f, x, dy, eps=1e-6):
    """Gradient of sum(dy f(x)) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + eps
        up = (dy * f()).sum()
        x[i] = old - eps
        g[i] = (up - (dy * f()).sum()) / (2 * eps)
        x[i] = old
    return g


def test_norm_by_hand():
    y, r = ref.pre_norm([[3.0, 4.0, 0.0, 0.0]], [1.0, 2.0, 1.0, 1.0], 0.0 + 1e-300)
    assert np.allclose(r, 0.4) and np.allclose(y, [[1.2, 3.2, 0, 0]])  # mean of squares 25/4
    o = ref.post_norm([[2.0, -2.0]], [[1.0, 1.0]], [1.0, 3.0], 1, 1e-300, [0.0], 2.0, 4.0)
    assert np.allclose(o["out"], [[2 + 4 * 0.5 * 1, 2 - 4 * 0.5 * 3]])


def test_pre_norm_gradients():
    rng = np.random.default_rng(0)
    x, gain, dy, dres = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    f = lambda: ref.pre_norm(x, gain, 0.1)[0]  # noqa: E731
    b = ref.pre_norm_bwd(dy, x, gain, ref.rstd(x, 0.1), dres, 0.7)
    assert np.allclose(b["dx"], grad(f, x, dy) + 0.7 * dres, atol=1e-7)
    assert np.allclose(b["dgain"], grad(f, gain, dy), atol=1e-7)


@pytest.mark.parametrize("gate", ["none", "token", "element"])
@pytest.mark.parametrize("norm", [0, 1])
def test_post_norm_gradients(norm, gate):
    rng = np.random.default_rng(1)
    z, gain, dout, res = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    g = {"none": None, "token": rng.normal(size=3), "element": rng.normal(size=(3, 8))}[gate]
    f = lambda: ref.post_norm(z, res, gain, norm, 0.1, g, 0.9, 0.6)["out"]  # noqa: E731
    b = ref.post_norm_bwd(dout, z, gain, norm, ref.rstd(z, 0.1), g, 0.6)
    assert np.allclose(b["dz"], grad(f, z, dout), atol=1e-7)
    assert np.allclose(b["dgain"], grad(f, gain, dout), atol=1e-7)
    assert np.allclose(0.9 * dout, grad(f, res, dout), atol=1e-7)
    if g is not None:
        assert np.allclose(b["dgate"], grad(f, g, dout), atol=1e-7)


def test_pack_by_hand():
    a = np.zeros((1, 64), np.float32)
    a[0, :3] = [127.0, -127.0, 0.5]  # scale 1; ties to even
    a[0, 3:6] = [1.5, 2.5, -1.5]
    q, s = ref.pack(a)
    assert s.tolist() == [[1.0, np.float32(2.0 ** -126)]]
    assert q[0, :7].tolist() == [127, -127, 0, 2, 2, -2, 0] and not q[0, 7:].any()
    a[0, 0] = 128.0  # 128/127 is no bf16 number: the next one is 1 + 2^-6... of 2^-7 steps
    q, s = ref.pack(a)
    assert s[0, 0] == 1 + 2.0 ** -7 * np.ceil((128 / 127 - 1) * 128) and q[0, 0] == np.rint(128 / s[0, 0])
    rng = np.random.default_rng(2)
    a = (rng.normal(size=(50, 96)) * np.exp(4 * rng.normal(size=(50, 1)))).astype(np.float32)
    q, s = ref.pack(a)
    err = np.abs(ref.unpack(q, s) - a).reshape(50, 3, 32).max(2)
    assert (err <= s * (0.5 + 2.0 ** -16)).all() and (s >= np.abs(a).reshape(50, 3, 32).max(2) / 127 * (1 - 2.0 ** -23)).all()


def test_pack_of_the_largest_values():
    """Codes and scales of amax from 252 * 2^120 to fp32's largest number: no value of a bf16 group
    comes back as more than bf16's largest, 255 * 2^120, and each is off by half a scale at most."""
    top = np.array([252, 253, 253.99, 254, 254.01, 255, 255.49, 256 * (1 - 2.0 ** -24)], np.float64) * 2.0 ** 120
    a = np.repeat(top.astype(np.float32)[:, None], 32, 1) * np.linspace(-1, 1, 32, dtype=np.float32)
    q, s = ref.pack(a)
    v = ref.unpack(q, s)
    assert (np.abs(v) <= 255 * 2.0 ** 120).all()
    assert (np.abs(v - a) <= s * (0.5 + 2.0 ** -16)).all()


def test_down_bwd_is_the_weighted_backward():
    """dgu, dWd and d_w of y = sum_rows w_r h_r Wd^T . dy, by differences."""
    rng = np.random.default_rng(3)
    R, H, I = 5, 6, 4
    g, u, w = rng.normal(size=(R, I)), rng.normal(size=(R, I)), rng.normal(size=R)
    Wd, dy = rng.normal(size=(2, H, I)), rng.normal(size=(R, H))
    segs = ref.experts([0, 3, 5])

    def y():
        h = g / (1 + np.exp(-g)) * u
        return np.concatenate([w[a:b, None] * (h[a:b] @ Wd[e].T) for e, a, b in segs])
    o = ref.down_bwd(dy, w, g, u, Wd, segs)
    assert np.allclose(o["dgu"], np.concatenate([grad(y, g, dy), grad(y, u, dy)], 1), atol=1e-7)
    assert np.allclose(o["d_w"], grad(y, w, dy), atol=1e-7)
    dWd = np.stack([dy[a:b].T @ o["h_w"][a:b] for _, a, b in segs])
    assert np.allclose(dWd, grad(y, Wd, dy), atol=1e-7)
