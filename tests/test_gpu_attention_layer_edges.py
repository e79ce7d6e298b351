"""Edges of the attention layer's operators, against the fp64 oracle with the bounds that
tests/test_gpu_attention_layer.py derives."""
import time

import pytest
import torch

from oracle import attention_layer as al
from linear_attention_recurrent_chunked_b200 import gdn
from tests.test_gpu_attention_layer import BF, attn_tol, cached, check_decode, close, on_gpu, prompt, randn, rope_tol

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


# ------------------------------------------------------------------ waits that run out

def given_up(kind, call):
    """Runs a call of which one load is withheld: it must report the time-out, soon."""
    gdn.debug_inject(kind, 20000)
    try:
        t0 = time.perf_counter()
        with pytest.raises(gdn.GdnError) as e:
            call()
        assert e.value.status == 8 and time.perf_counter() - t0 < 5.0
    finally:
        gdn.debug_inject(0, 0)


@pytest.mark.parametrize("kind", [2, 3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[100], [700], [640, 130, 20], [2500] + [9] * 80])
def test_prefill_wait_that_runs_out(lens, d, kind):
    """Keys, or values, of the first block that never come: its outputs are not written, the time-out is reported,
    every other block's outputs are those of an undisturbed call, and so are the next call's. (The last pack numbers
    its tiles sequence by sequence; the first one's withheld values are a sequence's last.)"""
    gen = torch.Generator().manual_seed(50 + d)
    Hq, Hkv, T = 8, 2, sum(lens)
    q, k, v, cu = (x.cuda() for x in prompt(gen, lens, Hq, Hkv, d))
    v = v[:, Hq + Hkv:]
    want = gdn.attn_prefill(q, k, v, cu, max_len=max(lens), check=True)
    o = torch.full_like(want, 3.0)
    given_up(kind, lambda: gdn.attn_prefill(q, k, v, cu, max_len=max(lens), o=o, check=True))
    first = (lens[0] - 1) // 32 * 32  # a tile has 32 positions of 4 heads; the longest one's block comes first
    assert (o[first:lens[0], :4] == 3.0).all()
    rest = torch.ones((T, Hq), dtype=torch.bool, device="cuda")
    rest[first:lens[0], :4] = False
    assert torch.equal(o[rest], want[rest])
    assert torch.equal(gdn.attn_prefill(q, k, v, cu, max_len=max(lens), check=True), want)


@pytest.mark.parametrize("kind", [2, 3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,prefix", [(16, 4, 0), (9, 1, 0), (16, 4, 6000), (16, 1, 3000)])
def test_decode_wait_that_runs_out(Hq, Hkv, prefix, d, kind):
    """The same for one token per sequence: the first block of the own keys' kernel, and of the prefix's."""
    gen = torch.Generator().manual_seed(60 + d)
    w = on_gpu(cached(gen, [2000] * (160 // Hkv), Hq, Hkv, d, 16, prefix))
    want = gdn.attn_decode(**w, check=True)
    o = torch.full_like(want, 3.0)
    given_up(kind, lambda: gdn.attn_decode(**w, o=o, check=True))
    # the first block's run of 1/148 of the keys lies within the first two sequences; the prefix's first block has rows
    # of the first key head and of the sequences that fill 128 rows
    n = 128 // (Hq // Hkv) if prefix else 2
    assert torch.equal(o[n:], want[n:]) and torch.equal(o[2:, Hq // Hkv:], want[2:, Hq // Hkv:])
    assert torch.equal(gdn.attn_decode(**w, check=True), want)


# ------------------------------------------------------------------ nothing of its own

@pytest.mark.parametrize("prefix", [0, 100])
def test_decode_page_table_without_columns(prefix):
    """A batch none of whose sequences has a page yet: the prefix alone, or zeros; a length that says otherwise is
    reported. And a batch of no sequences at all."""
    gen = torch.Generator().manual_seed(70)
    w = cached(gen, [0] * 5, 8, 2, 64, 16, prefix)
    w["page_table"] = w["page_table"][:, :0].contiguous()
    check_decode(w)
    with pytest.raises(gdn.GdnError) as e:
        gdn.attn_decode(**on_gpu(dict(w, lens=w["lens"] + 3)), check=True)
    assert e.value.status == 10
    none = dict(w, q=w["q"][:0], page_table=w["page_table"][:0], lens=w["lens"][:0])
    assert gdn.attn_decode(**on_gpu(none), check=True).shape == (0, 8, 64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("at", [[0], [2999], [0, 2999], [5, 6, 37, 38, 70, 1500], [31, 32, 63, 64, 96]])
def test_decode_few_sequences_with_keys_among_many_without(at, prefix, d):
    """Runs of a warp that cross stretches of empty sequences, of less and more than 32, up to the batch's end."""
    lens = [0] * 3000
    for i, b in enumerate(at):
        lens[b] = 1200 + 17 * i
    w = cached(torch.Generator().manual_seed(71 + len(at)), lens, 2, 1, d, 16, prefix)
    o = gdn.attn_decode(**on_gpu(w), check=True)
    some = sorted({0, 1, 33, 2998, 2999, *at})
    check_decode(dict(w, q=w["q"][some], page_table=w["page_table"][some], lens=w["lens"][some]), got=o[some])
    if not prefix:
        empty = torch.tensor([n == 0 for n in lens])
        assert (o[empty.cuda()] == 0).all()


# ------------------------------------------------------------------ packs

@pytest.mark.parametrize("lens,Hq,Hkv", [([70, 90, 200], 4, 2), ([33], 3, 1), ([900] + [3] * 40, 8, 2), ([0, 0], 4, 2)])
def test_prefill_rows_around_the_output_stay(lens, Hq, Hkv):
    """An output inside a larger buffer: the rows before it and those behind the last sequence stay as they were."""
    gen = torch.Generator().manual_seed(90)
    T, d = sum(lens), 64
    q, k, v, cu = (x.cuda() for x in prompt(gen, lens, Hq, Hkv, d))
    v = v[:, Hq + Hkv:]
    buffer = torch.full((T + 300, Hq, d), 3.0, dtype=BF, device="cuda")
    o = gdn.attn_prefill(q, k, v, cu, max_len=max(lens), o=buffer[150:150 + T], check=True)
    assert (buffer[:150] == 3.0).all() and (buffer[150 + T:] == 3.0).all()
    ref, a = al.prompt_attention(q.cpu(), k.cpu(), v.cpu(), lens)
    close(o, ref, attn_tol(ref, a, q, k, d, max(lens)))


@pytest.mark.parametrize("N", [223, 224, 225, 448, 449])
def test_prefill_sequence_counts_around_the_threads(N):
    """Packs numbered sequence by sequence, with one sequence for each thread that counts the tiles, one less and one
    more; and the same with two."""
    gen = torch.Generator().manual_seed(N)
    lens = torch.randint(0, 40, (N,), generator=gen).tolist()
    lens[0], lens[N // 2], lens[-1] = 0, 700, 1
    q, k, v, cu = prompt(gen, lens, 4, 2, 64)
    v = v[:, 6:].contiguous()
    o = gdn.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), max_len=700, check=True)
    ref, a = al.prompt_attention(q, k, v, lens)
    close(o, ref, attn_tol(ref, a, q, k, 64, 700))


@pytest.mark.parametrize("lens,Hkv,most", [([100] + [5] * 28 + [64], 2, m) for m in (100, 128, 129, 160, 304)] +
                         [([64] * 10, 8, m) for m in (64, 96, 128, 129, 640)])
def test_prefill_both_numberings_of_a_pack(lens, Hkv, most):
    """The bound on the lengths decides how blocks are numbered, between 128 and 129 in both packs (tiles of 32 positions: in
    the first the blocks then outnumber those that run at once, in the second they exceed the tiles by more than half).
    The outputs do not depend on it, bit for bit, and are those of each sequence alone."""
    gen = torch.Generator().manual_seed(91)
    q, k, v, cu = (x.cuda() for x in prompt(gen, lens, 4 * Hkv, Hkv, 128))
    v = v[:, 5 * Hkv:]
    want = torch.cat([gdn.attn_prefill(x, y, z, check=True) for x, y, z in zip(*(t.split(lens) for t in (q, k, v)))])
    assert torch.equal(gdn.attn_prefill(q, k, v, cu, max_len=most, check=True), want)


# ------------------------------------------------------------------ angles

@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("base", [1.01, 500.0, 1e12])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (128, 16)])
def test_norm_rope_ends_of_the_positions(d, rot, base, dtype):
    """The first and last int32 positions and others far out, where the frequencies of a base near 1 all count. (The kernel's
    angle is within 2e-7 of the formula's, the fp64 oracle's within 2^31 2^-51 = 1e-6: 3 and 16 fp32 half steps of the 32 that
    rope_tol allows for angle, sine, cosine and products.)"""
    gen = torch.Generator().manual_seed(92)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, -1, 10 ** 9 + 7, 2 ** 30, 1], dtype=torch.int32)
    x = randn(gen, len(pos), 3, d, dtype=dtype)
    y, b = al.norm_rope(x, None, pos, rot, base=base)
    q, k = gdn.qk_norm_rope(x.cuda(), x[:, :1].contiguous().cuda(), None, None, pos.cuda(), rot=rot, base=base, check=True)
    close(q, y, rope_tol(y, b, d, dtype))
    close(k, y[:, :1], rope_tol(y, b, d, dtype)[:, :1])


# ------------------------------------------------------------------ a cache of more than 2^32 elements

def test_cache_beyond_32_bits():
    """Pages on both sides of element 2^31 and 2^32 of the cache (9 GB each for keys and values), written by the norms'
    kernel and read as own keys and as a shared prefix; what stands in the other slots of these pages stays."""
    Hq, Hkv, d, page = 8, 4, 128, 64
    size = Hkv * page * d
    pages = 2 ** 32 // size + 40
    at = [3, 2 ** 31 // size - 1, 2 ** 31 // size, 2 ** 32 // size - 1, 2 ** 32 // size, pages - 1]
    gen = torch.Generator().manual_seed(93)
    kc, vc = (torch.empty((pages, Hkv, page, d), dtype=BF, device="cuda") for _ in range(2))
    for c in (kc, vc):
        for p in at:
            c[p] = 5.0
    # every page but two gets 50 tokens of its own sequence; those two 64 and 6 of a prefix
    own, prefix = [at[0], at[1], at[2], at[5]], [at[4], at[3]]
    slots = torch.tensor([p * page + t for p in own for t in range(50)] + [prefix[0] * page + t for t in range(64)] +
                         [prefix[1] * page + t for t in range(6)], dtype=torch.int32).cuda()
    T = len(slots)
    x = randn(gen, T, Hq + 2 * Hkv, d).cuda()
    pos = torch.arange(T, dtype=torch.int32).cuda()
    q, k = gdn.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], None, None, pos, v=x[:, Hq + Hkv:], k_cache=kc, v_cache=vc, slots=slots,
                            check=True)
    small = {p: i for i, p in enumerate(at)}  # the same pages in a cache of their own
    for c, want in ((kc, k), (vc, x[:, Hq + Hkv:])):
        got = torch.stack([c[p] for p in at])
        expect = torch.full_like(got, 5.0)
        for t, s in enumerate(slots.tolist()):
            expect[small[s // page], :, s % page] = want[t]
        assert torch.equal(got, expect)
    lens, i32 = [50, 33, 1, 50], torch.int32
    args = dict(q=q[:4].contiguous(), lens=torch.tensor(lens, dtype=i32).cuda(), prefix_len=70)
    big = dict(k_cache=kc, v_cache=vc, page_table=torch.tensor(own, dtype=i32).view(4, 1).cuda(),
               prefix_pages=torch.tensor(prefix, dtype=i32).cuda())
    near = dict(k_cache=torch.stack([kc[p] for p in at]), v_cache=torch.stack([vc[p] for p in at]),
                page_table=torch.tensor([small[p] for p in own], dtype=i32).view(4, 1).cuda(),
                prefix_pages=torch.tensor([small[p] for p in prefix], dtype=i32).cuda())
    o = gdn.attn_decode(**args, **big, check=True)
    assert torch.equal(o, gdn.attn_decode(**args, **near, check=True))
    check_decode({n: (y.cpu() if hasattr(y, "cpu") else y) for n, y in {**args, **near}.items()}, got=o)
