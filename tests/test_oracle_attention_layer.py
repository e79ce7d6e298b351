"""Pins for the attention layer's oracle (CPU only): closed forms, agreement with the causal
attention oracle, and the invariants the definitions fix."""
import numpy as np
import pytest

from oracle import attention_layer as al
from oracle.attention import causal_attention


def test_norm_rope_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 16))
    pos = np.array([0, 1, 7, 1000, 3])
    y, _ = al.norm_rope(x, None, pos, 8, base=100.0, eps=0.0)
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True))
    assert np.allclose(y[0], n[0], atol=1e-15)                    # position 0 turns nothing
    assert np.array_equal(y[..., 8:], n[..., 8:])                 # the rest is not turned
    assert np.allclose((y ** 2).mean(-1), 1.0, atol=1e-14)        # a rotation keeps the norm
    # the pair (1, 5) turns by pos * 100^(-1/4)
    a = 7 * 100.0 ** -0.25
    assert np.allclose(y[2, 0, 1], n[2, 0, 1] * np.cos(a) - n[2, 0, 5] * np.sin(a), atol=1e-14)
    assert np.allclose(y[2, 0, 5], n[2, 0, 5] * np.cos(a) + n[2, 0, 1] * np.sin(a), atol=1e-14)
    # scores depend on the distance of positions only
    u, w = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    dot = lambda p, q: float((al.norm_rope(u, None, [p], 16)[0] * al.norm_rope(w, None, [q], 16)[0]).sum())  # noqa: E731
    assert abs(dot(3, 10) - dot(103, 110)) < 1e-11
    assert abs(dot(3, 10) - dot(3, 11)) > 1e-3


def test_prompt_attention_matches_the_causal_oracle_per_group():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((9, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    o, a = al.prompt_attention(q, k, v, [4, 0, 5])
    ref = causal_attention(q, np.repeat(k, 2, 1), np.repeat(v, 2, 1), cu_seqlens=[0, 4, 4, 9])
    assert np.allclose(o, ref, atol=1e-13)
    assert (a >= np.abs(o) - 1e-13).all()


def test_decode_attention_is_the_last_row_of_the_prompt():
    rng = np.random.default_rng(2)
    d, page, pre, n = 8, 4, 6, 5
    k, v, q = rng.standard_normal((pre + n, 2, d)), rng.standard_normal((pre + n, 2, d)), rng.standard_normal((1, 4, d))
    kc, vc = np.full((5, 2, page, d), np.nan), np.full((5, 2, page, d), np.nan)
    prefix, own = [3, 0], [4, 1]
    for c, x in ((kc, k), (vc, v)):
        for t in range(pre):
            c[prefix[t // page], :, t % page] = x[t]
        for t in range(n):
            c[own[t // page], :, t % page] = x[pre + t]
    o, _ = al.decode_attention(q, kc, vc, [own], [n], prefix, pre)
    ref, _ = al.prompt_attention(np.repeat(q, pre + n, 0), k, v, [pre + n])
    assert np.allclose(o[0], ref[-1], atol=1e-13)
    # nothing to see: zeros
    assert np.array_equal(al.decode_attention(q, kc, vc, [own], [0])[0], np.zeros((1, 4, d)))


@pytest.mark.parametrize("mistake", ["mask", "group", "scale"])
def test_planted_mistakes_are_seen(mistake):
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((9, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    right, _ = al.prompt_attention(q, k, v, [9])
    if mistake == "mask":
        wrong, _ = al.prompt_attention(q, np.concatenate([k[1:], k[-1:]]), np.concatenate([v[1:], v[-1:]]), [9])
    elif mistake == "group":
        wrong, _ = al.prompt_attention(q, k[:, ::-1], v[:, ::-1], [9])
    else:
        wrong, _ = al.prompt_attention(q, k, v, [9], scale=1.0)
    assert np.abs(right - wrong).max() > 1e-2
