"""Host-side tests of the attention layer's entry points (no GPU needed): bad arguments come back as
the documented status before anything touches the device, from the C ABI and from the binding."""
import ctypes
import math

import pytest
import torch

VP = ctypes.c_void_p
FAKE = VP(1 << 20)  # aligned, never dereferenced: validation fails before any device work
MIS = VP((1 << 20) + 4)
ODD = VP((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    from linear_attention_recurrent_chunked_b200 import build, gdn
    build.build()
    return gdn.load_library()


def apart(args):
    """The fake pointers of a call, each with 16 GB of its own."""
    return {n: (VP((1 << 40) + i * (1 << 34)) if v is FAKE else v) for i, (n, v) in enumerate(args.items())}


ROPE = dict(q=FAKE, qs=16 * 128, k=FAKE, ks=4 * 128, v=FAKE, vs=4 * 128, wq=FAKE, wk=FAKE, eps=1e-6, positions=FAKE, T=8,
            Hq=16, Hkv=4, d=128, rot=128, base=1e4, dt=1, q_out=FAKE, k_out=FAKE, k_cache=FAKE, v_cache=FAKE, slots=FAKE,
            pages=8, page=16, ws=FAKE, ws_bytes=256, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(dt=2), 3), (dict(d=96), 2), (dict(T=-1), 2), (dict(Hq=0), 2), (dict(Hkv=0), 2),
    (dict(rot=8), 2), (dict(rot=48), 2), (dict(rot=256), 2), (dict(base=1.0), 2), (dict(base=math.nan), 2),
    (dict(base=math.inf), 2), (dict(eps=-1.0), 2), (dict(eps=math.nan), 2),
    (dict(qs=15 * 128), 2), (dict(qs=16 * 128 + 4), 2), (dict(ks=-512), 2), (dict(vs=0), 2),
    (dict(q=None), 1), (dict(k=None), 1), (dict(q_out=None), 1), (dict(positions=None), 1), (dict(v=None), 1),
    (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(slots=None), 1),
    (dict(k_out=None, slots=None, k_cache=None, v_cache=None), 1),
    (dict(page=24), 2), (dict(page=256), 2), (dict(pages=0), 2), (dict(pages=1 << 27), 2),
    (dict(q=MIS), 4), (dict(v_cache=MIS), 4), (dict(wk=MIS), 4), (dict(positions=ODD), 4), (dict(slots=ODD), 4),
    (dict(ws=None), 6), (dict(ws_bytes=255), 6), (dict(ws=ODD), 4),
])
def test_qk_norm_rope_refuses(lib, over, status):
    assert lib.gdn_qk_norm_rope(*{**apart(ROPE), **over}.values()) == status
    assert lib.gdn_last_error()


PREFILL = dict(q=FAKE, qs=16 * 128, k=FAKE, ks=4 * 128, v=FAKE, vs=4 * 128, cu=FAKE, N=2, T=256, Hq=16, Hkv=4, d=128,
               max_len=200, scale=0.0, dt=1, o=FAKE, ws=FAKE, ws_bytes=256, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(dt=0), 3), (dict(d=96), 2), (dict(N=0), 2), (dict(T=-2), 2), (dict(Hq=0), 2), (dict(Hkv=0), 2),
    (dict(Hkv=5), 2), (dict(Hq=17 * 4), 2), (dict(cu=None, N=3), 5), (dict(max_len=-1), 2), (dict(max_len=257), 2),
    (dict(max_len=127), 2), (dict(qs=8), 2), (dict(ks=4 * 128 + 2), 2), (dict(vs=1 << 40), 2),
    (dict(N=2000000, T=2000000000, max_len=2000000000), 2),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(o=MIS), 4), (dict(v=MIS), 4),
    (dict(cu=ODD), 4), (dict(ws=None), 6), (dict(ws_bytes=100), 6), (dict(ws=ODD), 4),
])
def test_attn_prefill_refuses(lib, over, status):
    assert lib.gdn_attn_prefill(*{**apart(PREFILL), **over}.values()) == status
    assert lib.gdn_last_error()


def at(offset):
    return VP((1 << 30) + offset)


@pytest.mark.parametrize("call,base,over", [
    # decode: o on q, and next to it
    ("gdn_attn_decode", "DECODE", dict(q=at(0), o=at(0))),
    ("gdn_attn_decode", "DECODE", dict(q=at(0), o=at(4 * 16 * 128 * 2 - 16))),
    # prefill: o on a key slice of a fused buffer that q shares
    ("gdn_attn_prefill", "PREFILL", dict(q=at(0), qs=2560, k=at(4096), ks=2560, o=at(8192))),
    # rope: in place is fine for whole tensors only
    ("gdn_qk_norm_rope", "ROPE", dict(q=at(0), q_out=at(256))),
    ("gdn_qk_norm_rope", "ROPE", dict(q=at(0), qs=25 * 128, q_out=at(0))),
    ("gdn_qk_norm_rope", "ROPE", dict(k=at(0), q_out=at(0))),
    ("gdn_qk_norm_rope", "ROPE", dict(q_out=at(0), k_out=at(16))),
])
def test_overlapping_outputs_are_refused(lib, call, base, over):
    assert getattr(lib, call)(*{**apart(globals()[base]), **over}.values()) == 2
    assert b"overlap" in lib.gdn_last_error()


def test_binding_refuses(lib):
    """CPU tensors, wrong types and shapes raise from the binding, with the status the ABI would give."""
    from linear_attention_recurrent_chunked_b200 import gdn
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    pos = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: gdn.qk_norm_rope(bf(4, 8, 64), bf(4, 2, 64), None, None, pos),
                 lambda: gdn.attn_prefill(bf(4, 8, 64), bf(4, 2, 64), bf(4, 2, 64))):
        with pytest.raises(gdn.GdnError) as e:
            call()
        assert e.value.status == 1  # no CPU path
    with pytest.raises(gdn.GdnError) as e:
        gdn.qk_norm_rope(bf(4, 8, 64).half(), bf(4, 2, 64), None, None, pos)
    assert e.value.status == 3
    with pytest.raises(gdn.GdnError) as e:
        gdn.attn_prefill(bf(4, 8, 64).float(), bf(4, 2, 64), bf(4, 2, 64))
    assert e.value.status == 3
    with pytest.raises(gdn.GdnError) as e:
        gdn.attn_prefill(bf(4, 512), bf(4, 2, 64), bf(4, 2, 64))
    assert e.value.status == 2


DECODE = dict(q=FAKE, kc=FAKE, vc=FAKE, pages=64, page=16, table=FAKE, max_pages=8, lens=FAKE, prefix_pages=FAKE, prefix_len=100,
              B=4, Hq=16, Hkv=4, d=128, scale=0.0, dt=1, o=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(dt=0), 3), (dict(d=96), 2), (dict(B=0), 2), (dict(Hq=0), 2), (dict(Hkv=0), 2), (dict(Hkv=3), 2), (dict(Hkv=0x7fffffff), 2),
    (dict(Hq=68), 2), (dict(prefix_len=-1), 2), (dict(prefix_len=(1 << 30) + 1), 2), (dict(B=1 << 29), 2),
    (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(pages=0), 2), (dict(pages=1 << 27), 2),
    (dict(max_pages=0), 2), (dict(max_pages=(1 << 26) + 1), 2), (dict(max_pages=1 << 26, B=1 << 10), 2), (dict(pages=1 << 26, Hkv=32, Hq=32), 2),
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(o=None), 1),
    (dict(prefix_pages=None), 1), (dict(q=MIS), 4), (dict(kc=MIS), 4), (dict(o=MIS), 4), (dict(table=ODD), 4), (dict(lens=ODD), 4),
    (dict(prefix_pages=ODD), 4), (dict(ws=None), 6), (dict(ws_bytes=256), 6), (dict(ws=VP((1 << 20) + 16)), 4),
])
def test_attn_decode_refuses(lib, over, status):
    assert lib.gdn_attn_decode(*{**apart(DECODE), **over}.values()) == status
    assert lib.gdn_last_error()


def test_attn_decode_workspace_size(lib):
    """At least the error word; the prefix adds a piece per sequence and per split."""
    size = lib.gdn_attn_decode_workspace_size
    plain = size(64, 16, 4, 128, 0)
    assert plain >= 256 + 2 * 148 * 4 * 130 * 4
    assert size(64, 16, 4, 128, 8192) >= plain + 64 * 16 * 130 * 4 * 2
    assert size(0, 16, 4, 128, 0) == 256  # refused by the call
    # a byte less than it says is refused
    assert lib.gdn_attn_decode(*{**apart(DECODE), "ws_bytes": size(4, 16, 4, 128, 100) - 1}.values()) == 6


def test_binding_refuses_decode(lib):
    from linear_attention_recurrent_chunked_b200 import gdn
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(q=bf(2, 4, 64), k_cache=bf(3, 2, 16, 64), v_cache=bf(3, 2, 16, 64), page_table=i32(2, 1), lens=i32(2))
    for over, status in ((dict(), 1), (dict(q=bf(2, 4, 64).float()), 3), (dict(v_cache=bf(3, 2, 16, 32)), 2), (dict(lens=i32(3)), 2),
                         (dict(page_table=i32(2, 1).long()), 3), (dict(prefix_len=5), 1),
                         (dict(prefix_len=33, prefix_pages=i32(2)), 2), (dict(q=bf(2, 4, 128)[..., :64]), 2)):
        with pytest.raises(gdn.GdnError) as e:
            gdn.attn_decode(**{**good, **over})
        assert e.value.status == status, over
