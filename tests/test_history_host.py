"""Host-side checks of the history-cache and sampling entry points (CPU only: no kernel is launched): bad sizes,
null and misaligned pointers and small workspaces are refused, and empty calls do nothing."""
import ctypes

import pytest

import hashed_lookup_row_amd as hlr

OK, INVALID, DIM, MISALIGNED, WS_SMALL = 0, 1, 2, 3, 4
P = ctypes.c_void_p(1 << 20)        # stand-in addresses (never dereferenced)
ODD = ctypes.c_void_p((1 << 20) + 2)
P4 = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    return hlr.load_library()


def plan(lib, requests=0, cols=4, num_free=3, block=16, max_tokens=5, cached=P, table=P, slots=P, counts=P):
    return lib.hist_plan(cached, P, requests, table, cols, P, num_free, block, max_tokens, slots, P, P, counts, None)


def test_plan(lib):
    assert plan(lib, requests=-1) == INVALID
    assert plan(lib, requests=65536) == INVALID
    assert plan(lib, requests=2, block=24) == INVALID
    assert plan(lib, requests=2, block=512) == INVALID
    assert plan(lib, requests=2, max_tokens=1 << 31) == INVALID
    assert plan(lib, requests=2, cached=None) == INVALID
    assert plan(lib, requests=2, table=None) == INVALID
    assert plan(lib, requests=2, slots=None) == INVALID
    assert plan(lib, requests=2, counts=None) == INVALID
    assert plan(lib, requests=2, slots=P4) == MISALIGNED
    assert plan(lib, requests=2, cached=ODD) == MISALIGNED


def test_plan_refuses_outputs_that_overlap(lib):
    at = [ctypes.c_void_p((1 << 20) + (i << 12)) for i in range(8)]
    names = ("cached", "fresh", "table", "free", "slots", "cu", "lengths", "counts")
    size = {"cached": 28, "fresh": 28, "table": 7 * 3 * 4, "free": 20, "slots": 72, "cu": 32, "lengths": 28, "counts": 16}

    def call(**other):
        a = dict(zip(names, at), **other)
        return lib.hist_plan(a["cached"], a["fresh"], 7, a["table"], 3, a["free"], 5, 16, 9, a["slots"], a["cu"], a["lengths"],
                             a["counts"], None)

    for x in ("table", "slots", "cu", "lengths", "counts"):
        for y in names:
            if x == y or (x == "lengths" and y in ("cached", "fresh")):
                continue
            assert call(**{x: at[names.index(y)]}) == INVALID, (x, y)
            last = at[names.index(y)].value + (size[y] - 1) // 8 * 8  # one element shared
            assert call(**{x: ctypes.c_void_p(last)}) == INVALID, (x, y)
    for y in ("cached", "fresh"):  # the lengths in place are right, but not moved by an element
        assert call(lengths=ctypes.c_void_p(at[names.index(y)].value + 4)) == INVALID


def append(lib, blocks=4, heads=2, block=16, dim=64, k=P, type_=1, kt=128, kh=64, slots=P, tokens=3, codes=P):
    return lib.hist_append(codes, P, P, P, blocks, heads, block, dim, k, P, type_, kt, kh, 128, 64, slots, tokens, None)


def test_append_and_read(lib):
    assert append(lib, tokens=0) == OK
    assert append(lib, dim=48) == DIM
    assert append(lib, heads=0) == INVALID
    assert append(lib, block=8) == INVALID
    assert append(lib, blocks=-1) == INVALID
    assert append(lib, codes=None) == INVALID
    assert append(lib, k=None) == INVALID
    assert append(lib, type_=3) == INVALID
    assert append(lib, tokens=-1) == INVALID
    assert append(lib, k=P4) == MISALIGNED
    assert append(lib, codes=P4) == MISALIGNED
    assert append(lib, kt=129) == MISALIGNED
    assert append(lib, slots=P4) == MISALIGNED
    read = lambda slots=P, out=P, n=3, type_=0: lib.hist_read(P, P, P, P, 4, 2, 16, 64, slots, n, out, P, type_, None)  # noqa: E731
    assert read(n=0) == OK
    assert read(slots=None) == INVALID
    assert read(type_=-1) == INVALID
    assert read(out=P4) == MISALIGNED


def attention(lib, q=P, type_=1, tokens=2, q_heads=4, qt=256, qh=64, codes=P, blocks=4, kv=2, block=16, dim=64, table=P,
              cols=2, lengths=P, requests=2, max_q=1, max_len=32, scale=0.125, causal=1, window=0, out=P, ws=None, wsb=0):
    return lib.hist_attention(q, type_, tokens, q_heads, qt, qh, codes, P, P, P, blocks, kv, block, dim, table, cols,
                              lengths, P, requests, max_q, max_len, scale, causal, window, out, None, ws, wsb, None)


def test_attention(lib):
    assert attention(lib, tokens=0) == OK
    assert attention(lib, requests=0) == OK
    assert attention(lib, max_q=0) == OK
    assert attention(lib, dim=80) == DIM
    assert attention(lib, q_heads=3) == INVALID
    assert attention(lib, q_heads=0) == INVALID
    assert attention(lib, kv=0) == INVALID
    assert attention(lib, type_=7) == INVALID
    assert attention(lib, causal=2) == INVALID
    assert attention(lib, causal=0, window=4) == INVALID
    assert attention(lib, window=-4) == INVALID
    assert attention(lib, requests=70_000) == INVALID
    assert attention(lib, max_len=-1) == INVALID
    assert attention(lib, block=48) == INVALID
    assert attention(lib, scale=float("nan")) == INVALID
    assert attention(lib, q=None) == INVALID
    assert attention(lib, out=None) == INVALID
    assert attention(lib, codes=None) == INVALID
    assert attention(lib, table=None) == INVALID
    assert attention(lib, lengths=None) == INVALID
    assert attention(lib, q=P4) == MISALIGNED
    assert attention(lib, qt=260) == MISALIGNED
    assert attention(lib, codes=P4) == MISALIGNED
    need = lib.hist_attention_workspace_size(2, 2, 4, 2, 64, 1, 100_000)
    assert need > 0 and need % 256 == 0
    assert attention(lib, max_len=100_000) == WS_SMALL
    assert attention(lib, max_len=100_000, ws=P, wsb=need - 1) == WS_SMALL
    assert attention(lib, max_len=100_000, ws=P4, wsb=need) == MISALIGNED


def test_attention_workspace(lib):
    size = lambda *a: lib.hist_attention_workspace_size(*a)  # noqa: E731
    assert size(2, 2, 3, 2, 64, 1, 100) == 0      # sizes that the call refuses
    assert size(2, 2, 4, 2, 80, 1, 100) == 0
    assert size(4096, 4096, 8, 8, 64, 1, 2048) == 0  # enough requests to fill the GPU without splitting
    assert size(1, 1, 8, 8, 64, 1, 1 << 20) >= size(1, 1, 8, 8, 64, 1, 1 << 14) > 0


def sample(lib, scores=P, type_=0, rows=3, items=10, noise=P, stride=10, index=P, top_k=None):
    return lib.sample_scores(scores, type_, rows, items, stride, noise, 10, None, top_k, None, None, index, P, None)


def test_sample(lib):
    assert sample(lib, rows=0) == OK
    assert sample(lib, rows=-1) == INVALID
    assert sample(lib, items=-1) == INVALID
    assert sample(lib, items=(1 << 27) + 1) == INVALID
    assert sample(lib, type_=3) == INVALID
    assert sample(lib, stride=-1) == INVALID
    assert sample(lib, scores=None) == INVALID
    assert sample(lib, noise=None) == INVALID
    assert sample(lib, index=None) == INVALID
    assert sample(lib, scores=ODD) == MISALIGNED
    assert sample(lib, scores=ODD, type_=1, noise=ODD) == MISALIGNED
    assert sample(lib, index=P4) == MISALIGNED
    assert sample(lib, top_k=ODD) == MISALIGNED
