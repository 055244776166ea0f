"""The fp64 attention reference against differences and against hand-made cases (CPU only)."""
import numpy as np
import pytest

import attn_ref


def _inputs(N, Hq, Hkv, d, seed):
    r = np.random.default_rng(seed)
    return r.standard_normal((N, Hq, d)), r.standard_normal((N, Hkv, d)), r.standard_normal((N, Hkv, d)), \
        r.standard_normal((N, Hq, d))


@pytest.mark.parametrize("Hq,Hkv,cu", [(2, 2, None), (4, 2, [0, 3, 3, 4, 9]), (3, 1, [0, 1, 9])])
def test_gradients_against_central_differences(Hq, Hkv, cu):
    q, k, v, g = _inputs(9, Hq, Hkv, 4, 5)
    segs = attn_ref.segments(1, 9, cu)
    got = attn_ref.full(q, k, v, g, 0.7, segs, "fp32")
    loss = lambda: float(np.sum(g * attn_ref.forward(q, k, v, 0.7, segs)[0]))
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        num = np.zeros_like(x)
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + 1e-5
            up = loss()
            x[i] = keep - 1e-5
            num[i] = (up - loss()) / 2e-5
            x[i] = keep
        # central differences: truncation h^2 and cancellation 2^-52 / h, both near 1e-10
        assert np.max(np.abs(num - got[name][0])) < 1e-8, name


def test_first_token_and_uniform_scores():
    q, k, v, _ = _inputs(6, 2, 1, 4, 7)
    o, lse = attn_ref.forward(q * 0, k, v, 1.0, [(0, 4), (4, 6)])
    assert np.allclose(o[0, 0], v[0, 0]) and np.allclose(o[4, 1], v[4, 0])
    assert np.allclose(o[3, 1], v[:4, 0].mean(0)) and np.allclose(lse[:, 3], np.log(4.0))


def test_decode_is_the_last_row_of_the_prompt():
    q, k, v, _ = _inputs(7, 4, 2, 8, 9)
    o, _ = attn_ref.forward(q, k, v, 0.3, [(0, 7)])
    d, _ = attn_ref.decode(q[-1:], [k], [v], 0.3, "fp32")
    assert np.allclose(d[0], o[-1])


def test_rotation_depends_on_the_distance_only():
    q, k, _, _ = _inputs(1, 1, 1, 8, 11)
    dots = [float(np.sum(attn_ref.rope(q, np.array([m]), 100.0) * attn_ref.rope(k, np.array([m - 3]), 100.0)))
            for m in (3, 10, 77)]
    assert np.allclose(dots, dots[0])
