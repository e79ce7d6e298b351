"""Long rows of the attention layer's operators, held to bounds that a lost tile of keys, or weights rounded once too
often, would break (tests/attention_bounds.py; what they see is shown in tests/test_attention_bounds.py)."""
import pytest
import torch

from linear_attention_recurrent_chunked_b200 import gdn
from tests import attention_bounds as ab
from tests.test_gpu_attention_layer import cached, f64, on_gpu, prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load_library()


def decode_rows(w):
    """(sequence, query head, q, k, v) of every row in 64 bits, the prefix's keys first."""
    q, table = f64(w["q"]), w["page_table"].tolist()
    caches = [f64(w[c]) for c in ("k_cache", "v_cache")]
    page, G = caches[0].shape[2], q.shape[1] // caches[0].shape[1]
    for b, n in enumerate(w["lens"].tolist()):
        slots = [int(w["prefix_pages"][t // page]) * page + t % page for t in range(w["prefix_len"])]
        slots = torch.tensor(slots + [table[b][t // page] * page + t % page for t in range(n)]).numpy()
        for h in range(q.shape[1]):
            yield (b, h, q[b, h], *(c[slots // page, h // G, slots % page] for c in caches))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv,page", [([40000, 1], 4, 2, 64), ([3000], 9, 1, 16), ([10240, 300, 64, 16, 40], 8, 2, 32),
                                              ([16, 33, 64, 1, 20] * 30, 4, 4, 16)])
def test_decode_long_rows(lens, Hq, Hkv, page, d):
    w = cached(torch.Generator().manual_seed(80 + d), lens, Hq, Hkv, d, page)
    o = f64(gdn.attn_decode(**on_gpu(w), check=True))
    # additions one after another: 16 in each of the two products of a step, the steps of a warp's run, the pieces
    steps = sum(-(-n // 16) for n in lens) * Hkv
    chain = 32 * (-(-steps // (148 * 8)) + 1) + 8 + 148
    for b, h, q, k, v in decode_rows(w):
        assert ab.rounded_within(o[b, h], *ab.row(q, k, v, chain)[:2]), (b, h)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,page,prefix", [(8, 2, 16, 10230), (16, 1, 64, 5000), (4, 4, 128, 3001)])
def test_decode_behind_a_long_prefix(Hq, Hkv, page, prefix, d):
    lens = [0, 1, 500, 37, 0, 64, 9, 130]
    w = cached(torch.Generator().manual_seed(82 + d), lens, Hq, Hkv, d, page, prefix)
    o = f64(gdn.attn_decode(**on_gpu(w), check=True))
    # the prefix in splits: 64 additions in each step of one; 148 pieces of the own keys and 296 splits at most
    splits = min(-(-prefix // 64), 296 // Hkv)  # (the 8 sequences' query heads of a key head are one tile of rows)
    chain = 64 * (-(-(-(-prefix // 64)) // splits)) + 64 + 148 + 296
    for b, h, q, k, v in decode_rows(w):
        assert ab.norm_within(o[b, h], *ab.row(q, k, v, chain, rounded=prefix)), (b, h)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv", [([4096], 8, 2), ([300, 4001, 77], 3, 1), ([2048, 2049], 4, 4)])
def test_prefill_long_rows(lens, Hq, Hkv, d):
    q, k, v, cu = prompt(torch.Generator().manual_seed(84 + d), lens, Hq, Hkv, d)
    v = v[:, Hq + Hkv:].contiguous()
    o = f64(gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), max_len=max(lens), check=True))
    q, k, v, cu = f64(q), f64(k), f64(v), cu.tolist()
    for t0, t1 in zip(cu, cu[1:]):
        n = t1 - t0
        for t in {t for t in (0, 63, 64, n // 4, n // 2, n - 64, n - 2, n - 1) if 0 <= t < n}:
            for h in range(Hq):
                r = slice(t0, t0 + t + 1)
                bound = ab.row(q[t0 + t, h], k[r, h * Hkv // Hq], v[r, h * Hkv // Hq], t + 64, rounded=t + 1)
                assert ab.norm_within(o[t0 + t, h], *bound), (t, h)
