"""HistoryCache against the entry points it is made of and 64-bit attention, and the serving example end to end."""
import importlib.util
import os

import pytest
import torch

import hashed_lookup_row_amd as hlr
from hashed_lookup_row_amd.history import HistoryCache

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hlr.load_library()
    return torch.device("cuda:0")


def attention64(q, k, v, hidden):
    """q [n, H, D], k, v [m, heads, D], hidden [n, m] or None; 64 bits."""
    group = q.shape[1] // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    for h in range(q.shape[1]):
        s = q[:, h].double().cpu() @ k[:, h // group].double().cpu().T * q.shape[2] ** -0.5
        if hidden is not None:
            s = s.masked_fill(hidden, float("-inf"))
        out[:, h] = torch.softmax(s, 1) @ v[:, h // group].double().cpu()
    return out


@pytest.mark.parametrize("side_stream", [False, True])
def test_histories_grow_are_attended_and_released(dev, side_stream):
    stream = torch.cuda.Stream(dev) if side_stream else None
    users, heads, D, B = 5, 2, 64, 16
    cache = HistoryCache(users, 40, heads, D, 150, dev, block=B, stream=stream)
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    on = torch.cuda.stream(stream) if side_stream else torch.cuda.stream(torch.cuda.current_stream(dev))
    with on:
        for step, new in enumerate([[30, 1, 0, 17, 64], [1, 1, 1, 1, 1], [0, 40, 3, 0, 2], [1, 0, 0, 0, 0]]):
            if step == 2:
                cache.release(4)
                assert cache.held == [31, 2, 1, 18, 0]
            n = sum(new)
            qkv = torch.randn((n, 3, 4, D), generator=g, device=dev)
            cache.append(qkv[:, 1, :heads], qkv[:, 2, :heads], new)
            out = cache.attend(qkv[:, 0])
            torch.cuda.synchronize()
            assert cache.lengths.tolist() == cache.held
            for u in range(users):
                assert cache.table[u, :len(cache.blocks[u])].tolist() == cache.blocks[u]
            assert sorted(cache._free + sum(cache.blocks, [])) == list(range(40))  # no block is lost or held twice
            at = 0
            for u, m in enumerate(new):
                if m:
                    k, v = cache.read(u)
                    pos = torch.arange(len(k))
                    hidden = pos[None] > (len(k) - m + torch.arange(m))[:, None]
                    want = attention64(qkv[at:at + m, 0], k, v, hidden)
                    # fp32: values of about 1, scores below 16 in log2: (8 + 4 * 16) 2^-23 of sums of |v| < 8
                    assert float((out[at:at + m].double().cpu() - want).abs().max()) < 72 * 2.0 ** -23 * 8
                at += m
        q = torch.randn((10, 4, D), generator=g, device=dev)
        out = cache.attend(q, counts=[4, 0, 5, 1, 0])
        torch.cuda.synchronize()
        for u, lo, hi in ((0, 0, 4), (2, 4, 9), (3, 9, 10)):
            k, v = cache.read(u)
            want = attention64(q[lo:hi], k, v, None)
            assert float((out[lo:hi].double().cpu() - want).abs().max()) < 72 * 2.0 ** -23 * 8


def test_refusals(dev):
    with pytest.raises(hlr.HLRError):
        HistoryCache(2, 4, 1, 64, 100, dev, block=20)
    with pytest.raises(hlr.HLRError):
        HistoryCache(2, 4, 1, 48, 100, dev)
    with pytest.raises(TypeError):
        HistoryCache(2, 4, 1, 64, 100, dev, stream=0)
    cache = HistoryCache(2, 4, 1, 64, 100, dev, block=16)
    kv = torch.zeros((70, 1, 64), device=dev)
    with pytest.raises(hlr.HLRError):
        cache.append(kv, kv, [70])          # a count per user
    with pytest.raises(hlr.HLRError):
        cache.append(kv, kv, [70, 1])       # 71 events
    with pytest.raises(hlr.HLRError):
        cache.append(kv, kv, [70, 0])       # five blocks of four
    with pytest.raises(hlr.HLRError):
        cache.append(torch.zeros((101, 1, 64), device=dev), torch.zeros((101, 1, 64), device=dev), [101, 0])
    odd = torch.zeros(64 * 64 + 1, device=dev)[1:].view(64, 1, 64)
    with pytest.raises(hlr.HLRError):
        cache.append(odd, odd, [64, 0])     # not 16-byte aligned: nothing is held afterwards
    assert cache.held == [0, 0] and cache.free_blocks == 4 and cache.lengths.tolist() == [0, 0]
    cache.append(kv[:64], kv[:64], [64, 0])
    assert cache.free_blocks == 0
    with pytest.raises(hlr.HLRError):
        cache.attend(kv[:3])


def test_serving_example(dev, capsys):
    spec = importlib.util.spec_from_file_location("history_serving", os.path.join(ROOT, "examples", "history_serving.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    last, logprob = example.main(["--users", "7", "--items", "3000", "--candidates", "50", "--history", "90", "--steps", "4"])
    assert "us a step" in capsys.readouterr().out
    assert last.shape == (7,) and bool((last > 0).all())
    assert bool((logprob <= 0).all()) and bool(torch.isfinite(logprob).all())


@pytest.mark.parametrize("gone", [[0], [1], [4], [3, 0], [0, 1, 2, 3, 4]])
def test_released_users_have_no_queries_left(dev, gone):
    """The newest events, once some of their users are released: the others' queries, users in order."""
    users, heads, D, new = 5, 2, 64, [2, 3, 0, 1, 70]
    cache = HistoryCache(users, 40, heads, D, 150, dev, block=16)
    g = torch.Generator(device=dev)
    g.manual_seed(7)
    kv = torch.randn((2, 50, heads, D), generator=g, device=dev)
    cache.append(kv[0], kv[1], [10, 20, 5, 15, 0])
    kv = torch.randn((2, sum(new), heads, D), generator=g, device=dev)
    cache.append(kv[0], kv[1], new)
    for u in gone:
        cache.release(u)
    left = [0 if u in gone else n for u, n in enumerate(new)]
    q = torch.randn((sum(left), 4, D), generator=g, device=dev)
    out = cache.attend(q)
    at = 0
    for u, m in enumerate(left):
        if m:
            k, v = cache.read(u)
            hidden = torch.arange(len(k))[None] > (len(k) - m + torch.arange(m))[:, None]
            want = attention64(q[at:at + m], k, v, hidden)
            # the bound of the growing histories above
            assert float((out[at:at + m].double().cpu() - want).abs().max()) < 72 * 2.0 ** -23 * 8
        at += m
    with pytest.raises(hlr.HLRError):
        cache.attend(torch.zeros((sum(new), 4, D), device=dev))  # rows of users that are gone


@pytest.mark.parametrize("return_lse", [False, True])
def test_a_stream_of_its_own_is_ordered_with_the_callers(dev, return_lse):
    """Inputs that the current stream has yet to make, overwritten and dropped right after the call, and results used
    at once, while the cache runs on another stream: the same as on one stream."""
    users, heads, D, steps = 6, 2, 64, 4
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    new = [[40, 3, 0, 17, 64, 1], [1, 1, 1, 1, 1, 1], [0, 9, 33, 2, 0, 5], [2, 0, 1, 1, 30, 1]]
    data = [torch.randn((sum(n), 3, 4, D), generator=g, device=dev) for n in new]
    busy = torch.randn((8192, 8192), generator=g, device=dev).to(torch.bfloat16)

    def run(stream):
        cache = HistoryCache(users, 60, heads, D, 200, dev, block=16, stream=stream)
        got = []
        for n, x in zip(new, data):
            qkv = torch.full_like(x, 1e4)
            for _ in range(20):  # about 15 ms that the inputs come after
                busy @ busy
            qkv.copy_(x)
            q, k, v = qkv[:, 0].clone(), qkv[:, 1, :heads].clone(), qkv[:, 2, :heads].clone()
            got.append(cache.append(k, v, n).clone())
            k.fill_(-1e4)
            v.fill_(-1e4)
            del k, v
            for c in (None, [2, 0, 1, 0, 3, 1]):
                part = q if c is None else q[:7] if len(q) >= 7 else q.repeat(2, 1, 1)[:7]
                part = part.clone()
                out = cache.attend(part, counts=c, return_lse=return_lse)
                part.fill_(1e4)
                got += [t.clone() for t in (out if return_lse else (out,))]
                del part, out
                torch.full((64, 4, D), 1e4, device=dev)  # takes freed memory
            got += [t.clone() for t in cache.read(4)]
        cache.release(1)
        got.append(cache.lengths.clone())
        return got

    want, got = run(None), run(torch.cuda.Stream(dev))
    torch.cuda.synchronize()
    assert len(want) == len(got)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_calls_do_not_wait_for_the_gpu(dev):
    """A pool of more than a million blocks and a history of 600,000 events, with a third of a second of work queued."""
    cache = HistoryCache(3, 1_200_000, 1, 32, 700_000, dev, block=16)
    kv = torch.randn((600_000, 1, 32), device=dev)
    cache.append(kv, kv, [5, 0, 599_995])
    k, _ = cache.read(2)
    cache.attend(kv[:2], counts=[1, 0, 1])
    busy = torch.randn((8192, 8192), device=dev).to(torch.bfloat16)
    busy @ busy
    torch.cuda.synchronize()
    for _ in range(400):
        busy @ busy
    done = torch.cuda.Event()
    done.record()
    again, _ = cache.read(2)
    cache.release(2)
    cache.append(kv[:70], kv[:70], [0, 30, 40])
    cache.attend(kv[:2], counts=[1, 0, 1])
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(k, again) and cache.held == [5, 30, 40]
    # a step is at most 1/127 of a block's largest value, a code half a step off
    assert float((k - kv[5:]).abs().max()) <= 0.5001 / 127 * float(kv.abs().max())


def test_the_free_list_outlasts_many_releases(dev):
    """Blocks handed out and given back for longer than the list's room on the GPU: table and host agree."""
    users, B = 4, 16
    cache = HistoryCache(users, 9, 1, 32, 120, dev, block=B)
    kv = torch.randn((300, 1, 32), device=dev)
    g = torch.Generator()
    g.manual_seed(3)
    for step in range(60):
        u = int(torch.randint(0, users, (1,), generator=g))
        cache.release(u)
        new = [0] * users
        new[u] = min(int(torch.randint(0, 61, (1,), generator=g)), cache.free_blocks * B)
        cache.append(kv[:sum(new)], kv[:sum(new)], new)
        assert sorted(cache._free + sum(cache.blocks, [])) == list(range(9))
        for v in range(users):
            assert cache.table[v, :len(cache.blocks[v])].tolist() == cache.blocks[v]
            assert not (cache.table[v, len(cache.blocks[v]):] != -1).any()
        assert torch.equal(cache.read(u)[0], hlr.hist_read(*cache.tensors(), torch.tensor(
            [b * B + i for b in cache.blocks[u] for i in range(B)][:new[u]], dtype=torch.int64, device=dev))[0])
