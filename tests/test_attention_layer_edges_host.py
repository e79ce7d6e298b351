"""Host-side edges of the attention layer's entry points and of the binding's workspaces (no GPU needed)."""
import contextlib
import gc
import threading
import types
import weakref

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from linear_attention_recurrent_chunked_b200 import build, gdn
    build.build()
    return gdn.load_library()


def test_injection_kinds_of_the_attention_layer(lib):
    """The kinds that withhold a load, their bounds, and nothing beyond them."""
    try:
        for kind in (2, 3):
            assert lib.gdn_debug_inject(kind, 20000) == 0
            assert lib.gdn_debug_inject(kind, 0) == 2
            assert lib.gdn_debug_inject(kind, 1000001) == 2
        for kind in (4, -1):
            assert lib.gdn_debug_inject(kind, 20000) == 2
    finally:
        assert lib.gdn_debug_inject(0, 0) == 0


# ------------------------------------------------------------------ the binding's workspaces

class Library:
    """Takes every call and notes the address of its workspace."""

    def __init__(self):
        self.seen = []

    def gdn_chunk_fwd_workspace_size(self, *args):
        return 1024 * args[1]

    def gdn_attn_decode_workspace_size(self, *args):
        return 4096

    def __getattr__(self, name):
        def call(*args):
            # the workspace stands before its size and the stream
            self.seen.append((name, getattr(args[-3], "value", args[-3])))
            return 0
        return call


@pytest.fixture
def binding(monkeypatch):
    """The binding on CPU tensors over a library that computes nothing, with a fake stream that may be capturing."""
    from linear_attention_recurrent_chunked_b200 import gdn
    lib, state = Library(), {"capturing": False}
    monkeypatch.setattr(gdn, "load_library", lambda: lib)
    monkeypatch.setattr(gdn, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(gdn, "_on", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(gdn, "_index", lambda name, t: -1)
    monkeypatch.setattr(gdn, "_bytes", lambda n, index: torch.empty(n, dtype=torch.uint8), raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0x7001))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x7001)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: state["capturing"])
    return gdn, lib, state


def calls(gdn):
    """Every entry point that takes a workspace, by name, for T tokens."""
    def bf(*s):
        return torch.zeros(s, dtype=torch.bfloat16)

    def f32(*s):
        return torch.zeros(s)

    def i32(*s):
        return torch.zeros(s, dtype=torch.int32)

    return {
        "chunk_fwd": lambda T: gdn.chunk_fwd(bf(T, 2, 128), bf(T, 2, 128), bf(T, 2, 128), f32(T, 2), f32(T, 2)),
        "chunk_fwd_raw": lambda T: gdn.chunk_fwd_raw(bf(T, 2, 128), bf(T, 2, 128), bf(T, 2, 128), f32(T, 2), f32(T, 2)),
        "proj_w8": lambda T: gdn.proj_w8(bf(T, 64), torch.zeros((26, 64), dtype=torch.int8), f32(26), 1, 8, 8),
        "attn_fwd": lambda T: gdn.attn_fwd(bf(T, 2, 128), bf(T, 2, 128), bf(T, 2, 128)),
        "qk_norm_rope": lambda T: gdn.qk_norm_rope(bf(T, 2, 64), bf(T, 2, 64), None, None, i32(T)),
        "attn_prefill": lambda T: gdn.attn_prefill(bf(T, 2, 64), bf(T, 2, 64), bf(T, 2, 64)),
        "attn_decode": lambda T: gdn.attn_decode(bf(T, 2, 64), bf(3, 2, 16, 64), bf(3, 2, 16, 64), i32(T, 1), i32(T)),
    }


NAMES = ["chunk_fwd", "chunk_fwd_raw", "proj_w8", "attn_fwd", "qk_norm_rope", "attn_prefill", "attn_decode"]


@pytest.mark.parametrize("name", NAMES)
def test_a_captured_call_keeps_a_workspace_of_its_own(binding, name):
    """A graph's workspace is not the cached one, which a later, larger call replaces and frees."""
    gdn, lib, state = binding
    call = calls(gdn)[name]
    call(64)
    call(64)
    cached = lib.seen[0][1]
    assert cached and lib.seen[1][1] == cached  # eager calls of one thread and stream share theirs
    state["capturing"] = True
    call(64)
    assert lib.seen[2][1] != cached
    state["capturing"] = False
    call(64)
    assert lib.seen[3][1] == cached


@pytest.mark.parametrize("name", NAMES)
def test_two_threads_on_one_stream_have_workspaces_of_their_own(binding, name):
    """Their calls' kernels may take turns on the stream."""
    gdn, lib, _ = binding
    call = calls(gdn)[name]
    call(64)
    t = threading.Thread(target=call, args=(64,))
    t.start()
    t.join()
    assert len(lib.seen) == 2 and lib.seen[0][1] != lib.seen[1][1]


@pytest.mark.parametrize("name", NAMES)
def test_workspaces_of_a_thread_end_with_it(binding, name, monkeypatch):
    """A server that starts threads does not gather their workspaces; its own stays."""
    gdn, lib, _ = binding
    made = []

    def make(n, index):
        t = torch.empty(n, dtype=torch.uint8)
        made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(gdn, "_bytes", make)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x7100 + NAMES.index(name))  # unused so far
    call, together = calls(gdn)[name], threading.Barrier(5)

    def serve():
        together.wait()
        call(64)
        together.wait()

    call(64)
    threads = [threading.Thread(target=serve) for _ in range(5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    gc.collect()
    assert [r() is not None for r in made] == [True] + [False] * 5
    call(64)
    assert lib.seen[-1][1] == lib.seen[0][1]


# ------------------------------------------------------------------ arguments

@pytest.mark.parametrize("which", [("k_cache",), ("v_cache",), ("k_cache", "v_cache")])
def test_caches_without_slots_are_refused(binding, which):
    """As the C entry point does: the cache would stay as it was, without a word."""
    gdn, lib, _ = binding
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(gdn.GdnError) as e:
        gdn.qk_norm_rope(x, x, None, None, torch.zeros(4, dtype=torch.int32), v=x, **dict.fromkeys(which, cache))
    assert e.value.status == 1 and not lib.seen


def test_decode_of_no_sequences(binding):
    """An empty batch, as the other operators take no tokens: an empty output, nothing launched; its arguments are
    still checked."""
    gdn, lib, _ = binding
    bf, i32 = torch.bfloat16, torch.int32
    cache = torch.zeros((3, 2, 16, 64), dtype=bf)
    args = dict(q=torch.zeros((0, 4, 64), dtype=bf), k_cache=cache, v_cache=cache, page_table=torch.zeros((0, 5), dtype=i32),
                lens=torch.zeros(0, dtype=i32))
    assert gdn.attn_decode(**args, check=True).shape == (0, 4, 64) and not lib.seen
    o = torch.zeros((0, 4, 64), dtype=bf)
    assert gdn.attn_decode(**args, o=o) is o and not lib.seen
    with pytest.raises(gdn.GdnError) as e:
        gdn.attn_decode(**dict(args, lens=torch.zeros(1, dtype=i32)))
    assert e.value.status == 2
