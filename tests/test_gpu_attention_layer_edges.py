"""Edges of the attention layer's operators, against the fp64 oracle with the bounds that
tests/test_gpu_attention_layer.py derives."""
import pytest
import torch

from linear_attention_recurrent_chunked_b200 import gdn
from tests.test_gpu_attention_layer import cached, check_decode, on_gpu

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load_library()


# ------------------------------------------------------------------ scores of minus infinity

def lowered(w, b, keys):
    """Gives some of sequence b's keys the score minus infinity: their first element infinite, every query's negative."""
    page = w["k_cache"].shape[2]
    w["q"][..., 0] = -w["q"][..., 0].abs() - 0.5
    for t in keys:
        w["k_cache"][int(w["page_table"][b, t // page]), :, t % page, 0] = INF
    return w


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (9, 1)])
@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("n,keys", [(17, [16]), (16, range(3, 16)), (40, range(16)), (3000, range(1000)), (2, [0]), (33, [0, 31, 32])])
def test_decode_keys_at_minus_infinity_weigh_nothing(n, keys, prefix, Hq, Hkv, d):
    """Keys whose score is minus infinity have weight zero wherever they stand: alone in a step of keys, filling
    a warp's first steps, or here and there."""
    gen = torch.Generator().manual_seed(n + prefix + Hq)
    check_decode(lowered(cached(gen, [5, n, 0, 20], Hq, Hkv, d, 16, prefix), 1, keys))


@pytest.mark.parametrize("prefix", [0, 70])
def test_decode_sequence_with_no_finite_score(prefix):
    """Every own key at minus infinity: the prefix alone counts; without one the softmax is 0 / 0, and the other
    sequences do not notice."""
    gen = torch.Generator().manual_seed(40 + prefix)
    w = lowered(cached(gen, [30, 21, 50], 4, 2, 64, 16, prefix), 1, range(21))
    if prefix:
        check_decode(w)
        return
    o = gdn.attn_decode(**on_gpu(w), check=True)
    assert torch.isnan(o[1]).all()
    check_decode(dict(w, q=w["q"][::2], page_table=w["page_table"][::2], lens=w["lens"][::2]), got=o[::2])
