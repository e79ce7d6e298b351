"""Edges of the attention layer's operators, against the fp64 oracle with the bounds that
tests/test_gpu_attention_layer.py derives."""
import pytest
import torch

from oracle import attention_layer as al
from linear_attention_recurrent_chunked_b200 import gdn
from tests.test_gpu_attention_layer import attn_tol, cached, check_decode, close, on_gpu, prompt

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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("low", [64, 70, 200])
def test_prefill_first_keys_at_minus_infinity_weigh_nothing(low, Hq, Hkv, d):
    """A prompt whose first keys all have the score minus infinity: later rows see the other keys alone, the rows
    that see none but those are 0 / 0."""
    T = 330
    gen = torch.Generator().manual_seed(low + d)
    q, k, v, _ = prompt(gen, [T], Hq, Hkv, d)
    v = v[:, Hq + Hkv:].contiguous()
    q[..., 0] = -q[..., 0].abs() - 0.5
    k[:low, :, 0] = INF
    o = gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), check=True)
    assert torch.isnan(o[:low]).all()
    ref, a = al.prompt_attention(q, k, v, [T])
    close(o[low:], ref[low:], attn_tol(ref, a, q, torch.nan_to_num(k, 0.0, 0.0, 0.0), d, T)[low:])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low", [64, 200, 500])
def test_decode_prefix_keys_at_minus_infinity_weigh_nothing(low, d):
    """The shared prefix starts with keys at minus infinity, down to all of it: then the own keys alone count, and a
    sequence without any is 0 / 0."""
    prefix, page = 500, 16
    gen = torch.Generator().manual_seed(low + d)
    w = cached(gen, [5, 40, 0, 200], 8, 2, d, page, prefix)
    w["q"][..., 0] = -w["q"][..., 0].abs() - 0.5
    for t in range(low):
        w["k_cache"][int(w["prefix_pages"][t // page]), :, t % page, 0] = INF
    if low < prefix:
        check_decode(w)
        return
    o = gdn.attn_decode(**on_gpu(w), check=True)
    assert torch.isnan(o[2]).all()
    rows = [0, 1, 3]
    check_decode(dict(w, q=w["q"][rows], page_table=w["page_table"][rows], lens=w["lens"][rows]), got=o[rows])
