"""The long rows' bounds (tests/attention_bounds.py) see what they are there to see: keys left out and weights rounded
once too often, planted in the fp64 oracle, on the CPU."""
import numpy as np
import pytest
import torch

from tests import attention_bounds as ab


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def inputs(n, d, seed):
    rng = np.random.default_rng(seed)
    return tuple(bf(rng.standard_normal(s)) for s in ((d,), (n, d), (n, d)))


def weights(q, k):
    s = (k @ q) * q.shape[0] ** -0.5
    return np.exp(s - s.max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 40, 3000, 40000])
def test_the_right_row_is_within(n, d):
    """With the weights as two bf16 values, and as one."""
    for seed in range(4):
        q, k, v = inputs(n, d, seed)
        p = weights(q, k)
        o, e, _ = ab.row(q, k, v, 200)
        hi = bf(p)
        assert ab.rounded_within(bf((hi + bf(p - hi)) @ v / p.sum()), o, e)
        o, e, r = ab.row(q, k, v, 200, rounded=n)
        assert ab.norm_within(bf(bf(p) @ v / p.sum()), o, e, r)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,lost", [(40000, 1000), (40000, 64), (10240, 64), (3000, 16), (3000, 1)])
def test_keys_left_out_are_seen(n, lost, d):
    for seed in range(8):
        q, k, v = inputs(n, d, seed)
        o, e, _ = ab.row(q, k, v, 200)
        p = weights(q, k)[lost:]
        assert not ab.rounded_within(bf(p @ v[lost:] / p.sum()), o, e)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,lost,chain", [(4096, 64, 4096), (10240, 64, 400), (10240, 1000, 400)])
def test_key_tiles_left_out_are_seen_in_the_norm(n, lost, chain, d):
    for seed in range(8):
        q, k, v = inputs(n, d, seed)
        o, e, r = ab.row(q, k, v, chain, rounded=n)
        p = weights(q, k)[lost:]
        assert not ab.norm_within(bf(p @ v[lost:] / p.sum()), o, e, r)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [16, 64])
def test_weights_as_one_bf16_value_are_seen(n, d):
    for seed in range(8):
        q, k, v = inputs(n, d, seed)
        o, e, _ = ab.row(q, k, v, 200)
        p = weights(q, k)
        assert not ab.rounded_within(bf(bf(p) @ v / p.sum()), o, e)
