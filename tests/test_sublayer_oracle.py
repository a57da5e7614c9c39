"""Pins of the float64 sublayer oracle (CPU only)."""
import numpy as np
import pytest

from oracle import sublayer_oracle as S


def test_bf16_rounds_half_to_even():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=2000) * 10.0 ** rng.integers(-30, 30, 2000), [0.0, 1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    np.testing.assert_array_equal(S.bf16(x), want)


def test_codes_cover_the_group_and_constants_are_exact():
    rng = np.random.default_rng(1)
    x = S.bf16(rng.normal(size=(7, 3, 128)))
    code, scale, bias = S.kv4_quantise(x)
    assert code.min() == 0 and code.max() == 15
    err = np.abs(S.kv4_values(x) - x).reshape(7, 3, 2, 64)
    # half a step, plus what the scale's own rounding moves the largest code by
    assert np.all(err <= scale[..., None] * (0.5 + 15 * 2.0 ** -8))
    flat = np.full((1, 64), 0.75)
    np.testing.assert_array_equal(S.kv4_values(flat), flat)


def test_what_rows_see():
    assert S.seen(3, 2, 3, False, 0).all()
    np.testing.assert_array_equal(S.seen(2, 3, 2, True, 0), [[1, 1, 1, 1, 0], [1, 1, 1, 1, 1]])
    np.testing.assert_array_equal(S.seen(2, 3, 0, True, 2), [[1, 1, 0], [0, 1, 1]])
    assert not S.seen(4, 1, 0, True, 0)[:3].any()  # rows before the first key see nothing


def test_attention_of_equal_scores_is_the_mean():
    K = np.ones((5, 1, 64))
    V = np.arange(5.0)[:, None, None] * np.ones((5, 1, 64))
    out, _ = S.attention(np.ones((1, 2, 64)), K, V, np.array([[1, 0, 1, 1, 0]], bool), 0.125)
    np.testing.assert_allclose(out, 5.0 / 3.0)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gradients_against_differences(kind):
    rng = np.random.default_rng(2)
    x, wg, wu, dh = (rng.normal(size=s) for s in ((3, 5), (4, 5), (4, 5), (3, 4)))
    f = lambda: (S.gated_ffn(x, wg, wu, kind)[0] * dh).sum()
    _, g, u = S.gated_ffn(x, wg, wu, kind)
    grads = S.gated_ffn_backward(dh, g, u, x, wg, wu, kind)
    for arr, grad in zip((x, wg, wu), grads):
        for at in np.ndindex(arr.shape):
            keep, e = arr[at], 1e-5
            arr[at] = keep + e
            hi = f()
            arr[at] = keep - e
            lo = f()
            arr[at] = keep
            assert abs((hi - lo) / (2 * e) - grad[at]) < 1e-7  # differences: e^2 f''' / 6 and 1e-16 f / e
