"""The attention layer's operators (gdn_qk_norm_rope, gdn_attn_prefill, gdn_attn_decode) against the fp64 oracle
(oracle.attention_layer), element by element.

Bounds, per element (u = 2^-8 the half step of bf16, e = 2^-24 that of fp32):
* qk_norm_rope: with b the sum of the magnitudes of the element's terms, b (d / 2 + 32) e for the
  fp32 arithmetic (d roundings in the mean, halved by the root; a few ulp each for the reciprocal
  root, weight, angle, sine, cosine and the two products), and u |y| when y is bf16.
* attention: the output's rounding u |o|; the weights' rounding u a with a = sum_j p_j |v_j|; the
  scores' fp32 sums, 2 d e |scale| max|q| max|k| each (the tensor core may truncate: 2 e a step),
  which moves a weight against the others by twice that; the sums over the n keys, 2 n e a.
"""
import threading

import numpy as np
import pytest
import torch

from oracle import attention_layer as al
from linear_attention_recurrent_chunked_b200 import gdn

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load_library()


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(gen, *shape, dtype=BF):
    return torch.randn(shape, generator=gen).to(dtype)


def close(got, ref, tol):
    got = f64(got)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), ("%d of %d off, worst by %.3g times its bound" %
                           (bad.sum(), bad.size, (np.abs(got - ref) / np.maximum(tol, 1e-300)).max()))


def rope_tol(y, bound, d, dtype):
    return bound * (d / 2 + 32) * E + (U * np.abs(y) if dtype == BF else 0) + 1e-30


def attn_tol(o, a, q, k, d, n, scale=None):
    scale = d ** -0.5 if scale is None else scale
    big = scale * np.linalg.norm(f64(q), axis=-1).max() * np.linalg.norm(f64(k), axis=-1).max() if q.numel() else 0.0
    return U * (np.abs(o) + a) * (1 + U) + a * (4 * d * E * big + 2 * n * E) + 1e-30


# ------------------------------------------------------------------ qk_norm_rope

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot", [(1, 1, 1, 64, 64), (3, 5, 1, 128, 32), (33, 16, 4, 128, 128), (2, 3, 3, 64, 16),
                                            (7, 4, 2, 128, 0), (1500, 2, 1, 64, 32)])
def test_norm_rope_matches(T, Hq, Hkv, d, rot, dtype):
    gen = torch.Generator().manual_seed(T)
    qkv = randn(gen, T, Hq + 2 * Hkv, d, dtype=dtype)
    wq, wk = randn(gen, d, dtype=F32), randn(gen, d, dtype=F32)
    pos = torch.randint(-5, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    pos[-1] = 2 ** 31 - 1
    page = 16
    pages = T // page + 2
    slots = torch.randperm(pages * page, generator=gen)[:T].to(torch.int32)
    slots[T // 2] = -1 if T > 2 else slots[T // 2]
    dev = qkv.cuda()
    kc = torch.full((pages, Hkv, page, d), 7.0, dtype=dtype, device="cuda")
    vc = torch.full((pages, Hkv, page, d), 9.0, dtype=dtype, device="cuda")
    q, k = gdn.qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], wq.cuda(), wk.cuda(), pos.cuda(), v=dev[:, Hq + Hkv:], rot=rot,
                            k_cache=kc, v_cache=vc, slots=slots.cuda(), check=True)
    qr, qb = al.norm_rope(qkv[:, :Hq], wq, pos, rot)
    kr, kb = al.norm_rope(qkv[:, Hq:Hq + Hkv], wk, pos, rot)
    close(q, qr, rope_tol(qr, qb, d, dtype))
    close(k, kr, rope_tol(kr, kb, d, dtype))
    # the cache: exactly the keys that came back and the values that went in; other slots untouched
    want_k, want_v = torch.full_like(kc, 7.0), torch.full_like(vc, 9.0)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // page, :, s % page], want_v[s // page, :, s % page] = k[t], dev[t, Hq + Hkv:]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    # without the cache, without k, in place: the same bits
    q2, k2 = gdn.qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], wq.cuda(), wk.cuda(), pos.cuda(), rot=rot)
    assert torch.equal(q2, q) and torch.equal(k2, k)
    qi, ki = dev[:, :Hq].contiguous(), dev[:, Hq:Hq + Hkv].contiguous()
    gdn.qk_norm_rope(qi, ki, wq.cuda(), wk.cuda(), pos.cuda(), rot=rot, q_out=qi, k_out=ki)
    assert torch.equal(qi, q) and torch.equal(ki, k)
    assert gdn.qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], wq.cuda(), wk.cuda(), pos.cuda(), v=dev[:, Hq + Hkv:], rot=rot,
                            k_cache=kc, v_cache=vc, slots=slots.cuda(), want_k=False)[1] is None


def test_norm_rope_options_and_extremes():
    """No weights; base and eps; rows of zeros (eps decides), tiny and huge rows in fp32."""
    gen = torch.Generator().manual_seed(9)
    x = randn(gen, 6, 2, 64, dtype=F32)
    x[1], x[2], x[3] = 0.0, x[2] * 1e-12, x[3] * 1e15
    pos = torch.arange(6, dtype=torch.int32) * 1000
    q, _ = gdn.qk_norm_rope(x.cuda(), x[:, :1].contiguous().cuda(), None, None, pos.cuda(), base=1e6, eps=1e-5, check=True)
    y, b = al.norm_rope(x, None, pos, 64, base=1e6, eps=float(np.float32(1e-5)))
    close(q, y, rope_tol(y, b, 64, F32))
    assert (f64(q)[1] == 0).all()


def test_norm_rope_bad_slots_are_reported_and_skipped():
    gen = torch.Generator().manual_seed(3)
    x = randn(gen, 5, 2, 64).cuda()
    pos = torch.arange(5, dtype=torch.int32).cuda()
    for bad in (32, -2, 2 ** 31 - 1, -2 ** 31):
        kc, vc = torch.zeros((2, 2, 16, 64), dtype=BF, device="cuda"), torch.zeros((2, 2, 16, 64), dtype=BF, device="cuda")
        slots = torch.tensor([0, 31, bad, -1, 5], dtype=torch.int32).cuda()
        with pytest.raises(gdn.GdnError) as e:
            gdn.qk_norm_rope(x, x, None, None, pos, v=x, k_cache=kc, v_cache=vc, slots=slots, check=True)
        assert e.value.status == 10
        assert torch.equal(vc[0, :, 0], x[0]) and torch.equal(vc[1, :, 15], x[1]) and torch.equal(vc[0, :, 5], x[4])
        vc[0, :, 0] = vc[1, :, 15] = vc[0, :, 5] = 0
        assert not vc.any()
    # the next good call clears the report
    gdn.qk_norm_rope(x, x, None, None, pos, check=True)


def test_norm_rope_no_tokens():
    x = torch.zeros((0, 4, 64), dtype=BF, device="cuda")
    q, k = gdn.qk_norm_rope(x, x, None, None, torch.zeros(0, dtype=torch.int32, device="cuda"), check=True)
    assert q.shape == (0, 4, 64) and k.shape == (0, 4, 64)


# ------------------------------------------------------------------ attn_prefill

def prompt(gen, lens, Hq, Hkv, d, std=1.0):
    T = sum(lens)
    q, k = randn(gen, T, Hq, d) * std, randn(gen, T, Hkv, d)
    v = randn(gen, T, Hq + 2 * Hkv, d)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    return q.to(BF), k, v, cu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (6, 2), (8, 2), (5, 1), (7, 1), (16, 2), (16, 1), (3, 3), (13, 1)])
def test_prefill_groups_and_ragged_lengths(Hq, Hkv, d):
    lens = [1, 0, 130, 7, 257, 64]
    gen = torch.Generator().manual_seed(Hq * 100 + d)
    q, k, v, cu = prompt(gen, lens, Hq, Hkv, d)
    v = v.cuda()[:, Hq + Hkv:]
    o = gdn.attn_prefill(q.cuda(), k.cuda(), v, cu.cuda(), max_len=max(lens), check=True)
    ref, a = al.prompt_attention(q, k, v, lens)
    close(o, ref, attn_tol(ref, a, q, k, d, max(lens)))


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255], [256], [513], [700, 1, 1, 1], [0, 0, 3]])
def test_prefill_tile_edges(lens):
    gen = torch.Generator().manual_seed(sum(lens))
    q, k, v, cu = prompt(gen, lens, 4, 2, 128)
    v = v[:, 6:].contiguous()
    o = gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), max_len=max(lens), check=True)
    ref, a = al.prompt_attention(q, k, v, lens)
    close(o, ref, attn_tol(ref, a, q, k, 128, max(lens)))


@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (16, 4)])
def test_prefill_many_short_prompts(Hq, Hkv):
    """Thousands of blocks whose first query tile has only a few steps of keys: no wait gives up, and
    equal prompts give equal outputs whichever block computes them."""
    gen = torch.Generator().manual_seed(13)
    lens = [256, 140, 200, 256] * 40
    q, k, v, _ = prompt(gen, lens[:4], Hq, Hkv, 128)
    q, k, v = (x.repeat(40, 1, 1).cuda() for x in (q, k, v[:, Hq + Hkv:]))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    o = gdn.attn_prefill(q, k, v, cu, max_len=256, check=True)
    assert torch.isfinite(o).all()
    assert torch.equal(o.view(40, -1), o[:sum(lens[:4])].reshape(1, -1).expand(40, -1))


@pytest.mark.parametrize("G", [1, 4])
def test_prefill_long_sequences_that_leave_a_query_tile_empty(G):
    """Lengths whose last block has rows in its first query tile only (or few steps less in it), over
    many key tiles and sequences: key tiles that one query tile alone uses are freed in their turn."""
    gen = torch.Generator().manual_seed(14)
    lens = [4032 + 15, 3968 + 21, 832 + 27, 1984 + 6, 3904 + 30, 130, 4096 - 127]
    q, k, v, cu = prompt(gen, lens, 4 * G, 4, 128)
    q, k, v, cu = q.cuda(), k.cuda(), v[:, 4 * G + 4:].contiguous().cuda(), cu.cuda()
    want = gdn.attn_prefill(q, k, v, cu, max_len=max(lens), check=True)
    for _ in range(20):
        assert torch.equal(gdn.attn_prefill(q, k, v, cu, max_len=max(lens), check=True), want)
    b = sum(lens[:2]) + lens[2]
    ref, a = al.prompt_attention(q[b - lens[2]:b], k[b - lens[2]:b], v[b - lens[2]:b], [lens[2]])
    close(want[b - lens[2]:b], ref, attn_tol(ref, a, q, k, 128, lens[2]))


@pytest.mark.parametrize("N", [33, 128, 129, 300])
def test_prefill_many_sequences(N):
    """Sequence counts around those up to which blocks are placed by looking through the lengths."""
    gen = torch.Generator().manual_seed(N)
    lens = torch.randint(0, 90, (N,), generator=gen).tolist()
    lens[N // 2] = 400
    q, k, v, cu = prompt(gen, lens, 6, 2, 64)
    v = v[:, 8:].contiguous()
    o = gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), max_len=500, check=True)
    ref, a = al.prompt_attention(q, k, v, lens)
    close(o, ref, attn_tol(ref, a, q, k, 64, 400))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", [0, 150, 299])
def test_prefill_one_long_prompt_among_many_short(where, d):
    """One prompt that is far longer than the others, first, among or last of them, empty ones on both sides:
    every prompt has the bits of a call of its own, and a malformed pack of this kind is not written."""
    gen = torch.Generator().manual_seed(15 + where)
    lens = torch.randint(0, 20, (300,), generator=gen).tolist()
    lens[1] = lens[298] = 0
    lens[where] = 2500
    q, k, v, cu = (x.cuda() for x in prompt(gen, lens, 8, 2, d))
    v = v[:, 8 + 2:]
    o = gdn.attn_prefill(q, k, v, cu, max_len=2500, check=True)
    ends = np.cumsum(lens)
    for n in (0, 2, where, 149, 151, 297, 299):
        i, j = ends[n] - lens[n], ends[n]
        if i < j:
            assert torch.equal(o[i:j], gdn.attn_prefill(q[i:j], k[i:j], v[i:j], check=True))
    i = ends[where] - 40
    ref, a = al.prompt_attention(q[ends[where] - 2500:ends[where]], k[ends[where] - 2500:ends[where]],
                                 v[ends[where] - 2500:ends[where]], [2500])
    close(o[i:i + 40], ref[-40:], attn_tol(ref, a, q, k, d, 2500)[-40:])
    for at, value in ((0, 1), (300, int(ends[-1]) - 1), (where + 1, int(ends[where]) + 1), (77, -5)):
        bad = cu.clone()
        bad[at] = value
        kept = torch.full_like(o, 3.0)
        with pytest.raises(gdn.GdnError) as e:
            gdn.attn_prefill(q, k, v, bad, max_len=2500, o=kept, check=True)
        assert e.value.status == 5 and (kept == 3.0).all()


def test_prefill_one_token_with_any_stride():
    """Of a single token the distance to the next one is not looked at."""
    gen = torch.Generator().manual_seed(16)
    q, k, v, _ = (x.cuda() for x in prompt(gen, [1], 4, 2, 64))
    o, ws = torch.zeros_like(q), torch.zeros(256, dtype=torch.uint8, device="cuda")
    v = v[:, 6:].contiguous()
    for stride in (0, 8, 1 << 30):
        o.zero_()
        gdn._check(gdn.load_library().gdn_attn_prefill(
            q.data_ptr(), stride, k.data_ptr(), stride, v.data_ptr(), stride, None, 1, 1, 4, 2, 64, 1, 0.0, gdn.GDN_BF16,
            o.data_ptr(), ws.data_ptr(), 256, torch.cuda.current_stream().cuda_stream))
        assert torch.equal(o, v.repeat_interleave(2, 1))


@pytest.mark.parametrize("trend", ["rising", "falling", "spikes"])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_moving_maximum(trend, d):
    """Scores up to about 30 that rise along the keys move the running maximum tile after tile, falling
    ones never do, spikes do at single rows."""
    T, Hq, Hkv = 600, 4, 1
    gen = torch.Generator().manual_seed(5)
    q, k, v, cu = prompt(gen, [T], Hq, Hkv, d)
    u = torch.nn.functional.normalize(torch.randn(d, generator=gen), dim=0)
    if trend == "spikes":
        k[::97] = (12 * u).to(BF)
        q[:] = (2.5 * d ** 0.5 * u).to(BF) * torch.rand((T, Hq, 1), generator=gen).to(BF)
    else:
        ramp = torch.linspace(0, 12, T) if trend == "rising" else torch.linspace(12, 0, T)
        q[:] = (2.5 * d ** 0.5 * u).to(BF)
        k = (ramp[:, None, None] * u + 0.1 * k.float()).to(BF)
    v = v[:, Hq + Hkv:].contiguous()
    o = gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), check=True)
    ref, a = al.prompt_attention(q, k, v, [T])
    close(o, ref, attn_tol(ref, a, q, k, d, T))


def test_prefill_equal_split_and_scale():
    gen = torch.Generator().manual_seed(6)
    q, k, v, _ = prompt(gen, [300, 300], 4, 4, 64)
    v = v[:, 8:].contiguous()
    o = gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), N=2, scale=0.3, check=True)
    ref, a = al.prompt_attention(q, k, v, [300, 300], scale=0.3)
    close(o, ref, attn_tol(ref, a, q, k, 64, 300, 0.3))


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_neighbours_do_not_leak(d):
    """NaN and infinity in a packed neighbour's rows leave a sequence's outputs as they were, bit for
    bit; rows beyond the last sequence's end stay untouched."""
    lens = [70, 90, 200]
    gen = torch.Generator().manual_seed(7)
    q, k, v, cu = prompt(gen, lens, 4, 2, d)
    v = v[:, 6:].contiguous()
    want = gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), max_len=200, check=True)
    for n in range(3):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        a, b = int(cu[n]), int(cu[n + 1])
        for x in (q2, k2, v2):
            x[:a], x[b:] = float("nan"), float("inf")
        got = gdn.attn_prefill(q2.cuda(), k2.cuda(), v2.cuda(), cu.cuda(), max_len=200, check=True)
        assert torch.equal(got[a:b], want[a:b])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [1, 63, 64, 130, 299])
def test_prefill_later_queries_and_keys_do_not_reach_back(at, d):
    """NaN and infinity in later tokens' queries and keys leave the earlier ones as they were, bit for bit."""
    gen = torch.Generator().manual_seed(17)
    q, k, v, _ = (x.cuda() for x in prompt(gen, [300], 4, 2, d))
    v = v[:, 6:]
    want = gdn.attn_prefill(q, k, v, check=True)
    for value in (float("nan"), float("inf"), -float("inf")):
        q2, k2 = q.clone(), k.clone()
        q2[at:], k2[at:] = value, value
        assert torch.equal(gdn.attn_prefill(q2, k2, v, check=True)[:at], want[:at])


def test_prefill_malformed_seqlens_reported_not_written():
    gen = torch.Generator().manual_seed(8)
    q, k, v, _ = prompt(gen, [256], 4, 2, 128)
    v = v[:, 6:].contiguous()
    for cu, most in (([0, 150, 100, 256], 150), ([0, 100, 200, 255], 128), ([1, 100, 200, 256], 128), ([0, 90, 220, 256], 128),
                     ([0, -5, 200, 256], 256), ([0, 300, 200, 256], 256)):
        o = torch.full_like(q, 7.0).cuda()
        with pytest.raises(gdn.GdnError) as e:
            gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), max_len=most, o=o, check=True)
        assert e.value.status == 5
        assert bool((o == 7.0).all())


def test_prefill_long_rows_sampled():
    """2500 tokens, 16 query heads on 4 key heads; all heads of sampled rows against the oracle."""
    T, Hq, Hkv, d = 2500, 16, 4, 128
    gen = torch.Generator().manual_seed(11)
    q, k, v, _ = prompt(gen, [T], Hq, Hkv, d)
    v = v[:, Hq + Hkv:].contiguous()
    o = gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), check=True)
    assert torch.isfinite(o).all()
    qf, kf, vf = f64(q), f64(k), f64(v)
    for t in [0, 31, 32, 63, 64, 127, 128, 1024, 2303, 2304, 2498, 2499]:
        for h in range(Hq):
            ref, a = al._attend(qf[t, h][None], kf[:t + 1, h // 4], vf[:t + 1, h // 4], d ** -0.5, np.ones((1, t + 1), bool))
            close(o[t, h][None], ref, attn_tol(ref, a, q[t], k, d, t + 1))


def test_prefill_same_inputs_same_bits_and_graph_replay():
    gen = torch.Generator().manual_seed(12)
    lens = [300, 41]
    q, k, v, cu = prompt(gen, lens, 4, 2, 128)
    q, k, v, cu = q.cuda(), k.cuda(), v[:, 6:].contiguous().cuda(), cu.cuda()
    want = gdn.attn_prefill(q, k, v, cu, max_len=300)
    assert torch.equal(gdn.attn_prefill(q, k, v, cu, max_len=300), want)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        o = torch.zeros_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gdn.attn_prefill(q, k, v, cu, max_len=300, o=o)
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)


# ------------------------------------------------------------------ attn_decode

def cached(gen, lens, Hq, Hkv, d, page, prefix=0, stale=float("nan")):
    """A cache whose pages lie in a random order, stale slots and unused pages holding `stale`."""
    counts = [-(-n // page) for n in lens]
    shared = -(-prefix // page)
    total = sum(counts) + shared + 2
    order = torch.randperm(total, generator=gen).tolist()
    kc, vc = (torch.full((total, Hkv, page, d), stale, dtype=BF) for _ in range(2))
    table = torch.full((len(lens), max(1, max(counts))), -77, dtype=torch.int32)

    def fill(pages, n):
        for c in (kc, vc):
            for i, p in enumerate(pages):
                m = min(page, n - i * page)
                c[p, :, :m] = randn(gen, Hkv, m, d)

    for b, n in enumerate(lens):
        mine = [order.pop() for _ in range(counts[b])]
        table[b, :counts[b]] = torch.tensor(mine, dtype=torch.int32)
        fill(mine, n)
    pp = [order.pop() for _ in range(shared)]
    fill(pp, prefix)
    q = randn(gen, len(lens), Hq, d)
    return dict(q=q, k_cache=kc, v_cache=vc, page_table=table, lens=torch.tensor(lens, dtype=torch.int32),
                prefix_pages=torch.tensor(pp, dtype=torch.int32) if prefix else None, prefix_len=prefix)


def on_gpu(w):
    return {k: (x.cuda() if hasattr(x, "cuda") else x) for k, x in w.items()}


def check_decode(w, scale=None, got=None):
    if got is None:
        got = gdn.attn_decode(**on_gpu(w), scale=scale or 0.0, check=True)
    ref, a = al.decode_attention(w["q"], w["k_cache"], w["v_cache"], w["page_table"].tolist(), w["lens"].tolist(),
                                 w["prefix_pages"], w["prefix_len"], scale)
    d = w["q"].shape[2]
    n = int(w["lens"].max()) + w["prefix_len"]
    close(got, ref, attn_tol(ref, a, w["q"], torch.nan_to_num(w["k_cache"], 0.0, 0.0, 0.0), d, n, scale))
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,page", [(1, 1, 16), (2, 2, 32), (6, 2, 16), (16, 4, 64), (7, 1, 128), (8, 1, 16), (9, 1, 32),
                                         (16, 1, 64), (32, 2, 16)])
def test_decode_groups_pages_and_ragged_lengths(Hq, Hkv, page, d):
    gen = torch.Generator().manual_seed(Hq * 10 + page)
    check_decode(cached(gen, [1, 0, 15, 16, 17, 127, 128, 129, 400, 3], Hq, Hkv, d, page))


@pytest.mark.parametrize("lens", [[0], [1], [16], [128], [129], [3000], [0, 0, 5], [1] * 300, [40000, 1]])
def test_decode_lengths(lens):
    gen = torch.Generator().manual_seed(sum(lens))
    check_decode(cached(gen, lens, 4, 2, 128, 64))


def test_decode_many_sequences_split_anywhere():
    """More sequences than threads in the scan, with runs that end inside, at and across borders."""
    gen = torch.Generator().manual_seed(21)
    lens = torch.randint(0, 700, (333,), generator=gen).tolist()
    check_decode(cached(gen, lens, 2, 1, 64, 32))


@pytest.mark.parametrize("Hq,Hkv,B,prefix", [(14, 2, 700, 0), (13, 1, 350, 40), (13, 13, 350, 0), (16, 1, 500, 100), (6, 2, 500, 0)])
def test_decode_more_rows_than_run_at_once(Hq, Hkv, B, prefix):
    """Several query heads for each CTA that joins pieces, in numbers that do not divide the heads, whole and cut
    sequences, some without keys."""
    gen = torch.Generator().manual_seed(23 + B + Hq)
    lens = torch.randint(0, 70, (B,), generator=gen).tolist()
    lens[B // 3], lens[-1] = 900, 0
    check_decode(cached(gen, lens, Hq, Hkv, 64, 16, prefix))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,page,prefix", [(4, 4, 16, 1), (16, 4, 16, 1000), (16, 4, 64, 2048), (5, 1, 32, 129), (16, 1, 128, 700),
                                                (6, 2, 16, 128), (2, 1, 128, 5000)])
def test_decode_shared_prefix(Hq, Hkv, page, prefix, d):
    gen = torch.Generator().manual_seed(prefix + d)
    check_decode(cached(gen, [0, 1, 200, 17, 0, 129, 64, 3, 5], Hq, Hkv, d, page, prefix))


def test_decode_shared_prefix_many_sequences():
    """Several row tiles of the prefix product, the last one partly filled; and no own keys at all."""
    gen = torch.Generator().manual_seed(22)
    check_decode(cached(gen, torch.randint(0, 60, (150,), generator=gen).tolist(), 4, 2, 128, 16, 500))
    check_decode(cached(gen, [0] * 70, 8, 2, 64, 16, 300))


@pytest.mark.parametrize("prefix", [0, 300])
def test_decode_moving_maximum_and_scale(prefix):
    """Scores between -40 and 40: pieces whose maxima are far apart join exactly enough."""
    gen = torch.Generator().manual_seed(23)
    w = cached(gen, [2000, 500, 3], 8, 2, 64, 16, prefix)
    u = torch.nn.functional.normalize(torch.randn(64, generator=gen), dim=0)
    w["q"] = (4 * u + 0.1 * w["q"].float()).to(BF)
    ramp = torch.randn(w["k_cache"].shape[0], 1, 1, 1, generator=gen) * 4
    w["k_cache"] = (w["k_cache"].float() * 0.3 + ramp * u).to(BF)
    check_decode(w, scale=0.7)


def test_decode_prefix_equals_the_same_keys_copied():
    """A shared prefix gives what the same keys give when they stand in every sequence's own table."""
    gen = torch.Generator().manual_seed(24)
    w = cached(gen, [10, 0, 33, 128], 8, 2, 128, 16, 64)  # the prefix ends on a page's end
    got = check_decode(w)
    w2 = dict(w, page_table=torch.cat([w["prefix_pages"].expand(4, 4), w["page_table"]], 1).contiguous(), lens=w["lens"] + 64,
              prefix_pages=None, prefix_len=0)
    # the two orders of summation differ by rounding only: each within its bound of the same oracle
    check_decode(w2)
    ref, _ = al.decode_attention(w["q"], w["k_cache"], w["v_cache"], w["page_table"].tolist(), w["lens"].tolist(), w["prefix_pages"], 64)
    ref2, _ = al.decode_attention(w2["q"], w2["k_cache"], w2["v_cache"], w2["page_table"].tolist(), w2["lens"].tolist())
    assert np.allclose(ref, ref2, atol=1e-12) and got.shape == w["q"].shape


def test_decode_bad_pages_and_lengths_are_reported():
    """No access leaves the cache and the other sequences' rows stay right."""
    gen = torch.Generator().manual_seed(25)
    for prefix in (0, 40):
        w = cached(gen, [40, 100, 7], 4, 2, 64, 16, prefix)
        for name, place, bad in (("page_table", (1, 3), 10 ** 6), ("page_table", (1, 0), -1), ("lens", (1,), -5), ("lens", (1,), 10 ** 6)):
            w2 = dict(w, **{name: w[name].clone()})
            w2[name][place] = bad
            if name == "lens" and bad > 0:
                w2["page_table"][1] = w2["page_table"][1].clamp(min=0)
            o = torch.zeros_like(w["q"]).cuda()
            with pytest.raises(gdn.GdnError) as e:
                gdn.attn_decode(**on_gpu(w2), o=o, check=True)
            assert e.value.status == 10
            ok = dict(w, q=w["q"][::2], page_table=w["page_table"][::2], lens=w["lens"][::2])
            check_decode(ok, got=o[::2])
        if prefix:
            w2 = dict(w, prefix_pages=torch.tensor([10 ** 6, -1, 0], dtype=torch.int32))
            with pytest.raises(gdn.GdnError) as e:
                gdn.attn_decode(**on_gpu(w2), check=True)
            assert e.value.status == 10
        check_decode(w)  # and the next good call reports nothing


def test_decode_same_bits_other_stream_and_graphs():
    """Equal calls give equal bits; two graphs captured one after the other keep workspaces of their own
    and may be replayed in any order and on two streams at once."""
    gen = torch.Generator().manual_seed(26)
    ws = [on_gpu(cached(gen, [700, 30, 1500], 8, 2, 128, 16, 200)), on_gpu(cached(gen, [90, 2500], 8, 2, 128, 32))]
    want = [gdn.attn_decode(**w) for w in ws]
    assert torch.equal(gdn.attn_decode(**ws[0]), want[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert torch.equal(gdn.attn_decode(**ws[1]), want[1])
    graphs, outs = [], []
    for w in ws:
        o = torch.zeros_like(w["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gdn.attn_decode(**w, o=o)
        graphs.append(g)
        outs.append(o)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for o, x in zip(outs, want):
        assert torch.equal(o, x)


# ------------------------------------------------------------------ the layer

@pytest.mark.parametrize("d,rot", [(128, 32), (64, 64)])
def test_layer_prompt_then_steps(d, rot):
    """A layer in use: three prompts are normed, rotated, cached and attended; then each sequence
    decodes four tokens from the cache. Each operator's result is held to the oracle of its formula on the
    inputs it was given, and the cached keys of all steps to a second path: one long prompt."""
    Hq, Hkv, page, steps = 8, 2, 16, 4
    lens = [37, 130, 64]
    gen = torch.Generator().manual_seed(d)
    T, N = sum(lens), len(lens)
    wq, wk = (1 + 0.1 * randn(gen, d, dtype=F32) for _ in range(2))
    qkv = randn(gen, T + steps * N, Hq + 2 * Hkv, d)
    dev = qkv.cuda()
    per = -(-(max(lens) + steps) // page)
    table = torch.randperm(N * per, generator=gen).reshape(N, per).to(torch.int32)
    kc, vc = (torch.full((N * per, Hkv, page, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    slot = lambda b, t: int(table[b, t // page]) * page + t % page  # noqa: E731
    pos = torch.tensor([t for n in lens for t in range(n)], dtype=torch.int32)
    slots = torch.tensor([slot(b, t) for b, n in enumerate(lens) for t in range(n)], dtype=torch.int32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    args = dict(rot=rot, k_cache=kc, v_cache=vc)
    x = dev[:T]
    q, k = gdn.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], wq.cuda(), wk.cuda(), pos.cuda(), v=x[:, Hq + Hkv:], slots=slots.cuda(), check=True, **args)
    o = gdn.attn_prefill(q, k, x[:, Hq + Hkv:], cu.cuda(), max_len=max(lens), check=True)
    ref, a = al.prompt_attention(q, k, x[:, Hq + Hkv:], lens)
    close(o, ref, attn_tol(ref, a, q, k, d, max(lens)))
    have = list(lens)
    seen = [[(qkv[int(cu[b]) + t], t) for t in range(n)] for b, n in enumerate(lens)]
    for i in range(steps):
        x = dev[T + i * N:T + (i + 1) * N]
        pos = torch.tensor(have, dtype=torch.int32)
        slots = torch.tensor([slot(b, have[b]) for b in range(N)], dtype=torch.int32)
        q, _ = gdn.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], wq.cuda(), wk.cuda(), pos.cuda(), v=x[:, Hq + Hkv:], slots=slots.cuda(),
                                want_k=False, check=True, **args)
        for b in range(N):
            seen[b].append((qkv[T + i * N + b], have[b]))
        have = [n + 1 for n in have]
        o = gdn.attn_decode(q, kc, vc, table.cuda(), torch.tensor(have, dtype=torch.int32).cuda(), check=True)
        ref, a = al.decode_attention(q, kc, vc, table.tolist(), have)
        close(o, ref, attn_tol(ref, a, q, torch.nan_to_num(kc, 0.0), d, max(have)))
    # the last step's rows are the last rows of prompts of everything seen so far
    rows = torch.stack([x for s in seen for x, _ in s]).cuda()
    pos = torch.tensor([t for s in seen for _, t in s], dtype=torch.int32).cuda()
    q, k = gdn.qk_norm_rope(rows[:, :Hq], rows[:, Hq:Hq + Hkv], wq.cuda(), wk.cuda(), pos, rot=rot)
    ends = np.cumsum(have)
    cu = torch.tensor(np.concatenate([[0], ends]), dtype=torch.int32).cuda()
    full = gdn.attn_prefill(q, k, rows[:, Hq + Hkv:], cu, max_len=max(have), check=True)
    ref, a = al.prompt_attention(q, k, rows[:, Hq + Hkv:], have)
    tol = attn_tol(ref, a, q, k, d, max(have))
    close(full[ends - 1], ref[ends - 1], tol[ends - 1])
    close(o, ref[ends - 1], tol[ends - 1])


def test_layer_chain_without_gaps_and_in_a_graph():
    """The operators back to back on one stream, each reading what the one before has just written and
    starting while that one drains; eagerly many times over and in one captured graph with other work
    between them: the same bits as with the device idle in between."""
    gen = torch.Generator().manual_seed(31)
    Hq, Hkv, d, page, B = 8, 2, 128, 16, 40
    x = randn(gen, B, Hq + 2 * Hkv, d).cuda()
    pos = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    w = on_gpu(cached(gen, [100] * B, Hq, Hkv, d, page, 200, stale=0.0))
    slots = (w["page_table"][:, 6] * page + 3).to(torch.int32)  # key 99 of each
    k0, v0 = w["k_cache"].clone(), w["v_cache"].clone()

    def chain(sync, o):
        w["k_cache"].copy_(k0)
        w["v_cache"].copy_(v0)
        for i in range(3):
            sync()
            q, _ = gdn.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], None, None, pos, v=x[:, Hq + Hkv:], k_cache=w["k_cache"],
                                    v_cache=w["v_cache"], slots=slots, want_k=False)
            sync()
            y = gdn.attn_decode(q, w["k_cache"], w["v_cache"], w["page_table"], w["lens"], w["prefix_pages"] if i else None, 200 if i else 0)
            sync()
            z = gdn.attn_prefill(y, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])
            sync()
            o[i].copy_(z)
            x[:, :Hq].copy_(z)
        x[:, :Hq].copy_(x0)

    x0 = x[:, :Hq].clone()
    want, got = (torch.zeros((3, B, Hq, d), dtype=BF, device="cuda") for _ in range(2))
    chain(torch.cuda.synchronize, want)
    torch.cuda.synchronize()
    for _ in range(10):
        chain(lambda: None, got)
        assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(lambda: None, got)
    for _ in range(5):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("T,H", [(2048, 4), (700, 2)])
def test_layer_after_a_recurrent_layer(T, H):
    """A recurrent layer's pack, whose last kernel lets the next one start early, then an attention layer on its output
    with the same workspace: the same bits as with the device idle in between; and after a malformed pack, which
    that layer reports and does not write, the attention layer's own error word."""
    gen = torch.Generator().manual_seed(32)
    q, k = (torch.nn.functional.normalize(torch.randn(T, H, 128, generator=gen), dim=-1).to(BF).cuda() for _ in range(2))
    v = randn(gen, T, H, 128).cuda()
    g, beta = (-torch.rand(T, H, generator=gen)).cuda(), torch.rand(T, H, generator=gen).cuda()
    good = torch.tensor([0, T // 3, T], dtype=torch.int32).cuda()
    bad = torch.tensor([0, T, T // 3], dtype=torch.int32).cuda()
    pos = torch.arange(T, dtype=torch.int32).cuda()
    ws = torch.zeros(gdn.chunk_fwd_workspace_size(2, T, H, 128, 128, BF), dtype=torch.uint8, device="cuda")

    def run(sync, cu, check):
        o = torch.full_like(v, 3.0)
        gdn.chunk_fwd(q, k, v, g, beta, cu_seqlens=cu, o=o, workspace=ws)
        sync()
        x, y = gdn.qk_norm_rope(o, k, None, None, pos, workspace=ws)
        sync()
        return o, gdn.attn_prefill(x, y, o, good, max_len=T, workspace=ws, check=check)

    for cu in (good, bad):
        want = run(torch.cuda.synchronize, cu, True)
        assert torch.isfinite(want[1]).all() and bool((want[0] == 3.0).all()) == (cu is bad)
        for _ in range(20):
            got = run(lambda: None, cu, True)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_threads_on_one_stream():
    """Two threads call the operators on the same stream at once, with kernels of one call between those of another:
    each gets the bits of calls made alone."""
    gen = torch.Generator().manual_seed(33)
    works = [on_gpu(cached(gen, [200, 33, 0, 600, 5], 8, 2, 128, 16, 300)), on_gpu(cached(gen, [90] * 60, 16, 4, 64, 32, 1000))]
    want = [gdn.attn_decode(**w) for w in works]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), []

    def serve(w, y):
        start.wait()
        got = [gdn.attn_decode(**w) for _ in range(200)]
        torch.cuda.current_stream().synchronize()
        wrong.append(sum(not torch.equal(x, y) for x in got))

    threads = [threading.Thread(target=serve, args=(w, y)) for w, y in zip(works, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]
