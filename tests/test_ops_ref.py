"""The float64 restatements the GPU tests compare with, checked on their own:
Philox4x32-10 against its published vectors, the balance loss at its closed
forms, the adapters against differences."""
import numpy as np

import ops_ref


def test_philox_published_vectors():
    z = ops_ref.philox4x32(np.zeros((1, 4)), (0, 0))[0]
    assert [hex(v) for v in z] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    o = ops_ref.philox4x32(np.full((1, 4), 0xFFFFFFFF), (0xFFFFFFFF, 0xFFFFFFFF))[0]
    assert [hex(v) for v in o] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]


def test_balance_closed_forms():
    # uniform probabilities, any counts: the loss is 1 and z is log(E)^2
    T, E, k = 12, 4, 2
    idx = np.stack([np.arange(T) % E, (np.arange(T) + 1) % E], 1)
    r = ops_ref.balance(np.zeros((T, E)), idx, None, [0, 5, T], k, 1.0, 0.0)
    assert abs(r["loss"][0] - 1) < 1e-12 and abs(r["loss"][1] - np.log(E) ** 2) < 1e-12
    # all tokens to one expert with all the probability: E / k
    l = np.full((T, E), -1e9)
    l[:, 1] = 0
    r = ops_ref.balance(l, np.ones((T, 1), int), None, [0, T], 1, 1.0, 0.0)
    assert abs(r["loss"][0] - E) < 1e-12


def test_adapter_differences():
    g = np.random.RandomState(0)
    T, K, N, r, nA = 7, 6, 5, 2, 3
    x, W, A, B = g.randn(T, K), g.randn(N, K), g.randn(nA, r, K), g.randn(nA, N, r)
    off, which, sc, dy = [0, 2, 2, 5, 7], [1, 0, -1, 1], np.array([1.0, 0.5, 2.0]), g.randn(T, N)
    o = ops_ref.adapter(x, W, A, B, sc, off, which, dy)
    f = lambda **kw: (ops_ref.adapter(**{**dict(x=x, W=W, A=A, B=B, scale=sc, offsets=off, which=which), **kw})["y"] * dy).sum()  # noqa: E731
    for name, v, got in (("x", x, o["dx"]), ("A", A, o["dA"]), ("B", B, o["dB"])):
        for _ in range(20):
            i = tuple(g.randint(s) for s in v.shape)
            up, dn = v.copy(), v.copy()
            up[i] += 1e-5
            dn[i] -= 1e-5
            assert abs((f(**{name: up}) - f(**{name: dn})) / 2e-5 - got[i]) < 1e-6
    assert not o["dA"][2].any() and not o["dB"][2].any() and not o["dA"][0].any()
