"""The 8-bit history cache (plan, append, read, attention) against plain implementations: whole numbers and codes
bit for bit, attention against its definition in 64 bits.

Attention's tolerance: with A = sum p|v| for the row and output element, an output may be off by
  its own rounding (2^-9 |o| for bf16, 2^-12 |o| for fp16, 2^-24 |o| for fp32; doubled here),
  the rounding of the weights, 2^-12 A (bf16: 11 bits, half a unit) or 2^-23 A (two parts), and
  fp32's: a score s (in log2) is a product of three roundings and a fused multiply-add, so it is off by at most
  4 * 2^-24 (|s| + sum |q k| / |..|), bounded by 4 * 2^-23 (1 + max |s|); 2^ and the sums add a few 2^-24:
  (8 + 4 max |s|) 2^-23 A,
  weights below 2^-126 of the largest, which fp32 does not hold: 2^-126 sum |v| over what the row sees, and
  the f16 grid's end: a weight times its value scale is held to 2^-35 of the row's largest such product (f16's
  steps are 2^-24 at the least, and the largest product lies at 2^10 or above): 2^-35 max(p vs) sum |code|.
The lse is off by the scores' error and its own rounding: (8 + 4 max |s|) 2^-23 + 2^-22 |lse|."""
import math

import numpy as np
import pytest
import torch

import hashed_lookup_row_amd as hlr

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hlr.load_library()
    return torch.device("cuda:0")


# ------------------------------------------------------------------ plan
def plan_oracle(cached, new, table, free, B, max_tokens):
    table = [list(r) for r in table]
    slots, cu, at = [], [0], 0
    lost = 0
    for r, (c, n) in enumerate(zip(cached, new)):
        c, n = max(c, 0), max(n, 0)
        cols = len(table[r])
        first = -(-c // B)
        got = {}
        for j in range(-(-(c + n) // B) - first):
            got[first + j] = free[at] if at < len(free) else -1
            at += 1
        for p in range(c, c + n):
            col = p // B
            b = got[col] if col in got else (table[r][col] if col < cols else -1)
            ok = col < cols and b >= 0
            if col in got and col < cols:
                table[r][col] = got[col]
            lost += not ok
            slots.append(b * B + p % B if ok else -1)
        cu.append(cu[-1] + n)
    slots += [-1] * (max_tokens - len(slots))
    return slots, cu, [max(c, 0) + max(n, 0) for c, n in zip(cached, new)], [min(at, len(free)), lost], table


@pytest.mark.parametrize("requests,B,cols,spare,seed", [
    (0, 16, 4, 3, 0), (1, 16, 8, 50, 1), (1, 256, 1, 1, 2), (7, 32, 6, 100, 3), (64, 64, 33, 400, 4),
    (300, 16, 9, 40, 5),      # the free list runs out
    (50, 16, 2, 500, 6),      # requests longer than their table rows
    (4097, 16, 4, 20000, 7),  # more requests than prefix groups
    (9001, 128, 3, 30000, 8),
])
def test_plan(dev, requests, B, cols, spare, seed):
    g = np.random.default_rng(seed)
    cached = g.integers(0, cols * B, size=requests)
    new = np.where(g.random(requests) < 0.3, 0, g.integers(0, 3 * B if requests < 1000 else 6, size=requests))
    if requests > 5:
        cached[3], new[4] = -2, -7  # negative lengths count as none
        cached[1], new[1] = 0, 0
    ids = g.permutation(requests * cols + spare + 1)
    table = np.full((requests, cols), -1)
    k = 0
    for r in range(requests):
        held = -(-max(cached[r], 0) // B)
        table[r, :held] = ids[k:k + held]
        k += held
    free = ids[k:k + spare]
    total = int(np.maximum(new, 0).sum())
    max_tokens = total + 37
    want = plan_oracle(cached.tolist(), new.tolist(), table.tolist(), free.tolist(), B, max_tokens)
    on = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    t = on(table)
    for again in range(2):  # the second call finds its own entries and writes the same ones
        slots, cu, lengths, counts = hlr.hist_plan(on(cached), on(new), t, on(free), B, max_tokens)
        assert slots.tolist() == want[0]
        assert cu.tolist() == want[1]
        assert lengths.tolist() == want[2]
        assert counts.tolist() == want[3]
        assert t.tolist() == want[4]


def test_plan_drops_tokens_past_the_given_number(dev):
    on = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.full((2, 4), -1, dtype=torch.int32, device=dev)
    slots, cu, _, _ = hlr.hist_plan(on([0, 0]), on([20, 20]), table, on([5, 6, 7, 8]), 16, 24)
    assert slots.tolist() == list(range(80, 96)) + list(range(96, 100)) + list(range(112, 116))
    assert cu.tolist() == [0, 20, 40]
    assert table.tolist() == [[5, 6, -1, -1], [7, -1, -1, -1]]  # request 1's second block holds dropped tokens only


@pytest.mark.parametrize("requests,new_hi,B", [(3, 5, 16), (64, 400, 64), (4096, 60, 32), (9001, 12, 16)])
@pytest.mark.parametrize("which", ["cached", "new"])
def test_plan_with_the_lengths_in_place(dev, requests, new_hi, B, which):
    """lengths written over cached or new: the same as apart, step by step."""
    g = torch.Generator(device=dev)
    g.manual_seed(requests)
    free = torch.randperm(requests * 30, generator=g, device=dev).to(torch.int32)
    tables = [torch.full((requests, 9 * new_hi // B + 2), -1, dtype=torch.int32, device=dev) for _ in range(2)]
    cached, taken, B8 = torch.zeros(requests, dtype=torch.int32, device=dev), 0, requests * new_hi
    for step in range(8):
        new = torch.randint(-1, new_hi + 1, (requests,), generator=g, device=dev).to(torch.int32)
        a = hlr.hist_plan(cached, new, tables[0], free[taken:], B, B8)
        c, n = cached.clone(), new.clone()
        out = tuple(torch.empty_like(t) for t in a[:2]) + (c if which == "cached" else n, torch.empty_like(a[3]))
        b = hlr.hist_plan(c, n, tables[1], free[taken:], B, B8, out=out)
        for x, y in zip(a, b):
            assert torch.equal(x, y)
        assert torch.equal(*tables)
        cached, taken = a[2], taken + int(a[3][0])


# ---------------------------------------------------------------- append
class Pool:
    """A cache with garbage in it, and a host copy that follows the definition in fp32."""

    def __init__(self, dev, blocks, heads, B, D, seed):
        g = np.random.default_rng(seed)
        self.k = g.integers(-127, 128, size=(blocks, heads, B, D)).astype(np.int8)
        self.v = g.integers(-127, 128, size=(blocks, heads, B, D)).astype(np.int8)
        self.ks = np.exp(g.standard_normal((blocks, heads))).astype(np.float32) * np.float32(0.02)
        self.vs = np.exp(g.standard_normal((blocks, heads))).astype(np.float32) * np.float32(0.02)
        self.B, self.D, self.heads, self.blocks = B, D, heads, blocks
        self.dev = [torch.from_numpy(self.k).to(dev), torch.from_numpy(self.transposed()).to(dev),
                    torch.from_numpy(self.ks.copy()).to(dev), torch.from_numpy(self.vs.copy()).to(dev)]

    def transposed(self):
        b, h, B, D = self.v.shape
        return np.ascontiguousarray(self.v.reshape(b, h, B // 16, 16, D).swapaxes(-1, -2))

    def append(self, which, x, slots):
        """x float32 [tokens, heads, D]; one run of a block at a time."""
        codes, scale = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        x = np.nan_to_num(x, nan=0.0, posinf=np.finfo(np.float32).max, neginf=-np.finfo(np.float32).max)
        f = np.float32
        i = 0
        while i < len(slots):
            if slots[i] < 0 or slots[i] >= self.blocks * self.B:
                i += 1
                continue
            j = i + 1
            while j < len(slots) and slots[j] == slots[j - 1] + 1 and slots[j] // self.B == slots[i] // self.B:
                j += 1
            b, p = slots[i] // self.B, slots[i] % self.B
            for h in range(self.heads):
                y = x[i:j, h]
                s = f(np.abs(y).max() * (f(1) / f(127)))
                if s < f(2.0 ** -126):
                    s = f(0)
                old = scale[b, h] if p else f(0)
                s = max(s, old)
                inv = f(1) / s if s > 0 else f(0)
                if p and s > old:
                    codes[b, h, :p] = np.rint(codes[b, h, :p].astype(f) * f(old * inv)).astype(np.int8)
                codes[b, h, p:p + j - i] = np.clip(np.rint(y * inv), -127, 127).astype(np.int8)
                scale[b, h] = s
            i = j

    def same(self):
        k, v, ks, vs = (t.cpu().numpy() for t in self.dev)
        for name, got, want in (("k", k, self.k), ("v", v, self.transposed()), ("ks", ks, self.ks), ("vs", vs, self.vs)):
            off = np.argwhere(got != want)
            assert not len(off), f"{name}: {len(off)} differ, the first at {off[0].tolist()}"


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("D,B,heads", [(32, 16, 3), (64, 64, 2), (128, 32, 1), (256, 128, 2), (64, 256, 1)])
def test_append_and_read(dev, dtype, D, B, heads):
    g = np.random.default_rng(D + B)
    pool = Pool(dev, 40, heads, B, D, 1)
    order = g.permutation(40)
    ends = {r: 0 for r in range(5)}
    tables = {r: order[8 * r:8 * r + 8] for r in range(5)}
    for step, sizes in enumerate([(1, 16, 17, 0, B), (1, 1, 1, 1, 1), (B + 3, 15, 1, 40, 2), (1, 2, 0, 5, 31), (3, 1, 1, 1, 1)]):
        slots = []
        for r, n in enumerate(sizes):
            for p in range(ends[r], min(ends[r] + n, 8 * B)):
                slots.append(int(tables[r][p // B]) * B + p % B)
            ends[r] = min(ends[r] + n, 8 * B)
        n = len(slots)
        cut = next(i for i in range(n // 2, n + 1) if i == n or i == 0 or slots[i] // B != slots[i - 1] // B)
        slots[cut:cut] = [-1, 40 * B + 5]  # tokens with no slot in the pool (a block's own tokens stand together)
        n += 2
        x = g.standard_normal((n, 3, heads, D)).astype(np.float32) * (4.0 ** (step - 1))  # scales grow step by step
        x[0, 1, 0, :5] = [np.nan, 0.0, -0.0, 1e-30, 7.5]
        if step == 2 and dtype != "fp16":
            x[-1, 2, heads - 1, 3] = -np.inf
        if step == 3:
            x[:, :, 0] = 0.0
        qkv = torch.from_numpy(x).to(dev).to(TYPES[dtype])
        host = qkv.float().cpu().numpy()
        hlr.hist_append(*pool.dev, qkv[:, 1], qkv[:, 2], torch.tensor(slots, device=dev))
        pool.append("k", host[:, 1], slots)
        pool.append("v", host[:, 2], slots)
        pool.same()
        k, v = hlr.hist_read(*pool.dev, torch.tensor(slots, device=dev), dtype=TYPES[dtype])
        for out, codes, scale in ((k, pool.k, pool.ks), (v, pool.v, pool.vs)):
            want = np.zeros((n, heads, D), np.float32)
            for i, s in enumerate(slots):
                if 0 <= s < 40 * B:
                    want[i] = codes[s // B, :, s % B].astype(np.float32) * scale[s // B][:, None]
            assert torch.equal(out.cpu(), torch.from_numpy(want).to(TYPES[dtype]))


def test_append_many_tokens_at_once(dev):
    """Enough tokens that a thread block looks after several runs; heads and tokens in either order in memory."""
    g = np.random.default_rng(3)
    B, D, heads, n = 16, 32, 4, 30011
    pool = Pool(dev, n // B + 60, heads, B, D, 2)
    slots, at = [], 0
    blocks = g.permutation(n // B + 60).tolist()
    while len(slots) < n:
        first = int(g.integers(0, B)) if g.random() < 0.2 else 0
        size = min(int(g.integers(1, B - first + 1)) if g.random() < 0.2 else B - first, n - len(slots))
        if at == len(blocks):
            break
        slots += [blocks[at] * B + first + i for i in range(size)]
        at += 1
    n = len(slots)
    x = g.standard_normal((2, heads, n, D)).astype(np.float32)
    d = torch.from_numpy(x).to(dev).transpose(1, 2)  # [2][tokens][heads][D], head-major in memory
    hlr.hist_append(*pool.dev, d[0], d[1], torch.tensor(slots, device=dev))
    pool.append("k", x[0].swapaxes(0, 1), slots)
    pool.append("v", x[1].swapaxes(0, 1), slots)
    pool.same()


def test_append_in_steps_stays_near_the_values(dev):
    """Token by token with growing magnitudes, a code is rounded once per growth: at most half a step each time."""
    B, D = 16, 32
    pool = Pool(dev, 1, 1, B, D, 4)
    g = np.random.default_rng(5)
    x = (g.standard_normal((B, 1, D)) * 1.2 ** np.arange(B)[:, None, None]).astype(np.float32)
    for t in range(B):
        d = torch.from_numpy(x[t:t + 1]).to(dev)
        hlr.hist_append(*pool.dev, d, d, torch.tensor([t], device=dev))
    k, v = hlr.hist_read(*pool.dev, torch.arange(B, device=dev))
    # scales grow, so half a step each time sums to at most half the number of growths of the last step
    s = float(pool.dev[2][0, 0])
    assert torch.equal(k, v)
    assert float((k.cpu() - torch.from_numpy(x)).abs().max()) <= 0.5 * B * s


# ------------------------------------------------------------- attention
class Cache:
    def __init__(self, dev, held, heads, B, D, seed, v_spread=0.3, extra=5):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.dev, self.B, self.D, self.heads = dev, B, D, heads
        blocks = sum(-(-n // B) for n in held) + extra
        self.k = torch.randint(-127, 128, (blocks, heads, B, D), generator=g, device=dev, dtype=torch.int8)
        self.v = torch.randint(-127, 128, (blocks, heads, B // 16, D, 16), generator=g, device=dev, dtype=torch.int8)
        self.ks = torch.randn((blocks, heads), generator=g, device=dev).mul_(0.3).exp_().mul_(0.02)
        self.vs = torch.randn((blocks, heads), generator=g, device=dev).mul_(v_spread).exp_().mul_(0.02)
        ids = torch.randperm(blocks, generator=g, device=dev).to(torch.int32).tolist()
        cols = max([-(-n // B) for n in held] + [1])
        table, at = [], 0
        for n in held:
            m = -(-n // B)
            table.append(ids[at:at + m] + [-1] * (cols - m))
            at += m
        self.unused = ids[at:]
        self.table = torch.tensor(table, dtype=torch.int32, device=dev)
        self.lengths = torch.tensor(held, dtype=torch.int32, device=dev)

    def tensors(self):
        return self.k, self.v, self.ks, self.vs

    def rows(self, r, length):
        """K, V [heads, length, D] in 64 bits and which positions have a block, on the host."""
        pos = torch.arange(length, device=self.dev)
        b = self.table[r].long()[pos // self.B]
        ok = (b >= 0) & (b < self.k.shape[0])
        b = torch.where(ok, b, 0)
        i = pos % self.B
        k = self.k[b, :, i].double() * self.ks[b].double()[..., None]
        code = self.v[b, :, i // 16, :, i % 16].double()
        vs = self.vs[b].double()
        return k.transpose(0, 1).cpu(), code.transpose(0, 1).cpu(), vs.T.cpu(), ok.cpu()


def attend(cache, q, cu, scale, causal, window):
    """(out, lse, A, largest |score| in log2, what underflow may cost) in 64 bits."""
    T, H, D = q.shape
    out = torch.zeros((T, H, D), dtype=torch.float64)
    A = torch.zeros_like(out)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    big = torch.zeros((T, H), dtype=torch.float64)
    lost = torch.zeros_like(out)
    group = H // cache.heads
    for r, length in enumerate(cache.lengths.tolist()):
        lo, hi = cu[r], cu[r + 1]
        if hi == lo or length == 0:
            continue
        k, code, vs, ok = cache.rows(r, length)
        v = code * vs[..., None]
        pos = torch.arange(length)
        at = length - (hi - lo) + torch.arange(hi - lo)
        seen = ok[None].expand(hi - lo, -1)
        if causal:
            seen = seen & (pos[None] <= at[:, None])
            if window:
                seen = seen & (pos[None] > at[:, None] - window)
        for h in range(H):
            s = q[lo:hi, h].double().cpu() @ k[h // group].T * scale
            s = torch.where(seen, s, torch.tensor(-math.inf, dtype=torch.float64))
            any_ = seen.any(1)
            p = torch.where(any_[:, None], torch.softmax(s, 1), torch.zeros((), dtype=torch.float64))
            p = torch.nan_to_num(p) if not any_.all() else p
            out[lo:hi, h] = p @ v[h // group]
            A[lo:hi, h] = p @ v[h // group].abs()
            c = h // group
            lost[lo:hi, h] = seen.double() @ v[c].abs() * 2.0 ** -126
            lost[lo:hi, h] += (p * vs[c]).amax(1, keepdim=True) * (seen.double() @ code[c].abs()) * 2.0 ** -35
            lse[lo:hi, h] = torch.where(any_, torch.logsumexp(s, 1), torch.tensor(-math.inf, dtype=torch.float64))
            big[lo:hi, h] = torch.where(seen, s.abs(), torch.zeros((), dtype=torch.float64)).amax(1) * 1.4427
    return out, lse, A, big, lost


ROUND = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
WEIGHT = {torch.float32: 2.0 ** -22, torch.bfloat16: 2.0 ** -11, torch.float16: 2.0 ** -22}


def check(cache, q, cu, max_q=None, max_len=None, scale=None, causal=True, window=0, **kw):
    T, H, D = q.shape
    n = [b - a for a, b in zip(cu, cu[1:])]
    max_q = max(n + [1]) if max_q is None else max_q
    max_len = max(cache.lengths.tolist() + [1]) if max_len is None else max_len
    dcu = torch.tensor(cu, dtype=torch.int32, device=q.device)
    out, lse = hlr.hist_attention(q, *cache.tensors(), cache.table, cache.lengths, dcu, max_q, max_len, scale=scale,
                                  causal=causal, window=window, return_lse=True, **kw)
    want, wlse, A, big, lost = attend(cache, q, cu, D ** -0.5 if scale is None else scale, causal, window)
    fp = (8 + 4 * big) * 2.0 ** -23
    tol = ROUND[q.dtype] * want.abs() + (WEIGHT[q.dtype] + fp)[..., None] * A + lost + 1e-37
    assert not torch.isnan(out).any()
    got = out.double().cpu()
    if q.dtype == torch.float16:  # its range: infinities past 65504, steps of 2^-24 near zero
        tol = tol + 2.0 ** -24
        got, want = got.clamp(-65504, 65504), want.clamp(-65504, 65504)
    off = (got - want).abs()
    assert bool((off <= tol).all()), f"out off by {float((off / tol).max())} of its tolerance"
    l_off = torch.where(torch.isinf(wlse), (lse.cpu() != wlse).double(), (lse.double().cpu() - wlse).abs())
    l_tol = fp + 2.0 ** -22 * torch.where(torch.isinf(wlse), 0.0, wlse.abs())
    assert bool((l_off <= l_tol).all()), f"lse off by {float((l_off / l_tol).max())} of its tolerance"
    return out, lse


def queries(dev, n, H, D, dtype, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn((n, H, D), generator=g, device=dev).to(TYPES[dtype])


LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 255, 257, 700, 1025]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("D,B,kv,group", [(32, 16, 2, 1), (64, 64, 3, 2), (128, 32, 1, 16), (256, 128, 2, 3), (64, 256, 1, 5)])
def test_single_tokens(dev, dtype, D, B, kv, group):
    cache = Cache(dev, LENGTHS, kv, B, D, 1)
    q = queries(dev, len(LENGTHS), kv * group, D, dtype, 2)
    check(cache, q, list(range(len(LENGTHS) + 1)))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 70), (False, 0)])
@pytest.mark.parametrize("D,B,kv,group", [(32, 32, 1, 4), (64, 16, 2, 1), (128, 64, 1, 3), (256, 16, 1, 2)])
def test_many_queries(dev, dtype, causal, window, D, B, kv, group):
    new = [1, 40, 0, 17, 130, 64, 3]
    held = [300, 40, 50, 20, 600, 64, 1000]
    cache = Cache(dev, held, kv, B, D, 3)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    check(cache, queries(dev, cu[-1], kv * group, D, dtype, 4), cu, causal=causal, window=window)


@pytest.mark.parametrize("group,new", [(1, 16), (1, 17), (16, 1), (17, 1), (24, 2), (5, 3), (2, 65)])
def test_row_counts_around_the_tiles(dev, group, new):
    cache = Cache(dev, [new, new + 100, 513], 2, 64, 64, 5)
    check(cache, queries(dev, 3 * new, 2 * group, 64, "bf16", 6), [0, new, 2 * new, 3 * new])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("D,kv,group,new,window", [(32, 1, 17, 1, 0), (64, 2, 8, 3, 0), (128, 1, 16, 2, 700), (128, 2, 11, 5, 0),
                                                   (64, 1, 16, 4, 0), (256, 1, 9, 3, 0)])
def test_few_queries_of_long_histories(dev, dtype, D, kv, group, new, window):
    """17 to 64 rows per key head: the waves of a block share keys, in one or two tiles of 32 rows."""
    held = [1500, new, 300, 2049, 1]
    cache = Cache(dev, held, kv, 32, D, 31)
    cu = [0, new, 2 * new, 2 * new, 3 * new, 3 * new + 1]
    check(cache, queries(dev, cu[-1], kv * group, D, dtype, 32), cu, window=window)
    check(cache, queries(dev, cu[-1], kv * group, D, dtype, 33), cu, causal=False)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(dev, causal):
    """No history, queries before its first event, no blocks at all, lost blocks."""
    held = [0, 3, 70, 200, 64]
    cache = Cache(dev, held, 2, 16, 64, 7)
    cache.table[2] = -1                       # every block lost
    cache.table[3, 2] = -1                    # one block lost
    cache.table[3, 5] = cache.k.shape[0] + 3  # and one id outside the pool
    new = [4, 9, 2, 5, 1]                     # request 1 has more queries than events
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    for dtype in ("bf16", "fp32"):
        out, lse = check(cache, queries(dev, cu[-1], 4, 64, dtype, 8), cu, causal=causal)
        assert not out[:4].any() and bool((lse[:4] == -math.inf).all())
        if causal:
            assert not out[4:10].any() and bool(out[10].any())
        assert not out[13:15].any()


def test_one_request_and_a_long_history(dev):
    """The length is split over many thread blocks and joined."""
    for dtype, length in (("fp32", 40_001), ("bf16", 100_003)):
        cache = Cache(dev, [length], 1, 16, 64, 9)
        check(cache, queries(dev, 1, 4, 64, dtype, 10), [0, 1])
    cache = Cache(dev, [30_000, 5], 1, 64, 32, 11)
    check(cache, queries(dev, 33, 2, 32, "fp16", 12), [0, 30, 33])
    check(cache, queries(dev, 33, 2, 32, "fp16", 12), [0, 30, 33], window=100)


def test_bounds_larger_than_needed(dev):
    cache = Cache(dev, [100, 7], 2, 32, 64, 13)
    q = queries(dev, 3, 4, 64, "bf16", 14)
    a, _ = check(cache, q, [0, 2, 3])
    b, _ = check(cache, q, [0, 2, 3], max_q=50, max_len=5000)
    assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(a.float().abs().max())


def test_scales_of_every_size(dev):
    """Value scales over 60 binary orders, key scales of zero, queries of zero and of the types' extremes."""
    cache = Cache(dev, [500, 90, 64], 2, 16, 64, 15, v_spread=6.0)
    cache.ks[:, 0].masked_fill_(torch.rand(cache.ks.shape[0], device=dev) < 0.3, 0.0)
    cache.vs.masked_fill_(torch.rand(cache.vs.shape, device=dev) < 0.1, 0.0)
    q = queries(dev, 3, 4, 64, "fp32", 16)
    q[1] = 0
    check(cache, q, [0, 1, 2, 3])
    check(cache, (q * 1e-30), [0, 1, 2, 3])
    check(cache, q * 1e30, [0, 1, 2, 3], scale=1e-30)
    check(cache, (q * 1e-4).to(torch.bfloat16), [0, 1, 2, 3])
    check(cache, (q * 1e37).to(torch.bfloat16), [0, 1, 2, 3], scale=1e-37)
    check(cache, (q * 1e-6).to(torch.float16), [0, 1, 2, 3], scale=1e4)
    check(cache, (q * 9000).to(torch.float16), [0, 1, 2, 3], scale=1e-5)
    check(cache, q, [0, 1, 2, 3], scale=20.0)  # nearly all the weight on one event
    check(cache, q, [0, 1, 2, 3], scale=-0.3)
    check(cache, q, [0, 1, 2, 3], scale=0.0)


def test_values_and_scales_that_are_not_seen_do_not_matter(dev):
    held = [37, 200]
    cache = Cache(dev, held, 2, 64, 64, 17)
    q = queries(dev, 4, 4, 64, "bf16", 18)
    a, la = check(cache, q, [0, 2, 4])
    cache.ks[cache.unused] = math.nan
    cache.vs[cache.unused] = math.inf
    t = int(cache.table[0, 0])
    cache.k[t, :, 37:] = 127       # places past the end of the block's tokens
    cache.v[t, :, 2, :, 5:] = -128
    cache.v[t, :, 3] = -128
    b, lb = check(cache, q, [0, 2, 4])
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_a_row_that_is_not_finite_stays_alone(dev):
    cache = Cache(dev, [90, 300], 1, 16, 64, 19)
    q = queries(dev, 24, 2, 64, "fp32", 20)
    want, wl = check(cache, q, [0, 4, 24])
    q[2, 1, 7] = math.nan
    q[9, 0, 3] = math.inf
    cu = torch.tensor([0, 4, 24], dtype=torch.int32, device=dev)
    out, lse = hlr.hist_attention(q, *cache.tensors(), cache.table, cache.lengths, cu, 20, 300, return_lse=True)
    bad = torch.zeros((24, 2), dtype=torch.bool, device=dev)
    bad[2, 1] = bad[9, 0] = True
    assert torch.isnan(out[2, 1]).all() and torch.isnan(lse[2, 1])
    assert torch.isnan(out[9, 0]).all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], wl[~bad])


def test_strided_queries_streams_and_repeats(dev):
    cache = Cache(dev, [400, 100, 33], 2, 32, 128, 21)
    g = torch.Generator(device=dev)
    g.manual_seed(22)
    qkv = torch.randn((9, 3, 8, 128), generator=g, device=dev).to(torch.bfloat16)
    q = qkv[:, 0]  # rows of a fused projection
    a, la = check(cache, q, [0, 3, 6, 9])
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    b, lb = check(cache, heads_first, [0, 3, 6, 9])
    assert torch.equal(a, b) and torch.equal(la, lb)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    cu = torch.tensor([0, 3, 6, 9], dtype=torch.int32, device=dev)
    need = hlr.hist_attention_workspace_size(9, 3, 8, 2, 128, 3, 400)
    ws = hlr.new_workspace(dev, need)
    torch.cuda.synchronize()
    c = hlr.hist_attention(q, *cache.tensors(), cache.table, cache.lengths, cu, 3, 400, ws=ws, stream=side)
    d = hlr.hist_attention(q, *cache.tensors(), cache.table, cache.lengths, cu, 3, 400)
    torch.cuda.synchronize()
    assert torch.equal(c, a) and torch.equal(d, a)


def test_a_pool_past_32_bits(dev):
    """Block ids whose bytes lie past 4 GiB (only the blocks used are filled)."""
    heads, B, D = 2, 256, 256
    blocks = (5 << 30) // (heads * B * D)
    k = torch.empty((blocks, heads, B, D), dtype=torch.int8, device=dev)
    v = torch.empty((blocks, heads, B // 16, D, 16), dtype=torch.int8, device=dev)
    scale = torch.zeros((2, blocks, heads), device=dev)
    use = [blocks - 1, 3, blocks - 7]
    cache = Cache(dev, [600], heads, B, D, 23, extra=0)
    table = torch.tensor([use], dtype=torch.int32, device=dev)
    for j, b in enumerate(use):
        src = int(cache.table[0, j])
        k[b], v[b], scale[0, b], scale[1, b] = cache.k[src], cache.v[src], cache.ks[src], cache.vs[src]
    q = queries(dev, 2, 4, D, "bf16", 24)
    cu = torch.tensor([0, 2], dtype=torch.int32, device=dev)
    want = hlr.hist_attention(q, *cache.tensors(), cache.table, cache.lengths, cu, 2, 600)
    got = hlr.hist_attention(q, k, v, scale[0].contiguous(), scale[1].contiguous(), table, cache.lengths, cu, 2, 600)
    assert torch.equal(want, got)
    x = torch.randn((3, heads, D), device=dev)
    slots = torch.tensor([use[0] * B, use[0] * B + 1, use[2] * B], device=dev)
    hlr.hist_append(k, v, scale[0], scale[1], x, x, slots)
    a, b = hlr.hist_read(k, v, scale[0], scale[1], slots)
    assert torch.equal(a, b)
    # a code is at most half a step off; a step is at most 1/127 of the largest value
    assert float((a - x).abs().max()) <= 0.5001 / 127 * float(x.abs().max())


def test_replayed_as_a_graph(dev):
    """Plan, append and attention captured once: each replay equals the eager calls, lengths changing in between."""
    B, D, kv, R = 16, 64, 2, 3
    cache = Cache(dev, [40, 7, 90], kv, B, D, 25, extra=40)
    table = torch.full((R, 12), -1, dtype=torch.int32, device=dev)
    table[:, :cache.table.shape[1]] = cache.table
    free = torch.tensor(cache.unused, dtype=torch.int32, device=dev)
    cached, new = cache.lengths.clone(), torch.ones(R, dtype=torch.int32, device=dev)
    qkv = torch.randn((R, 3, kv, D), device=dev).to(torch.bfloat16)
    need = hlr.hist_attention_workspace_size(R, R, kv, kv, D, 1, 12 * B)
    ws = hlr.new_workspace(dev, need)
    out = torch.empty((R, kv, D), dtype=torch.bfloat16, device=dev)
    plan = (torch.empty(R, dtype=torch.int64, device=dev), torch.empty(R + 1, dtype=torch.int32, device=dev),
            torch.empty(R, dtype=torch.int32, device=dev), torch.empty(2, dtype=torch.int64, device=dev))

    def step(tensors, table, plan, out):
        hlr.hist_plan(cached, new, table, free, B, R, out=plan)
        hlr.hist_append(*tensors, qkv[:, 1], qkv[:, 2], plan[0])
        hlr.hist_attention(qkv[:, 0], *tensors, table, plan[2], plan[1], 1, 12 * B, out=out, ws=ws)

    mine = [t.clone() for t in cache.tensors()]
    theirs = [t.clone() for t in cache.tensors()]
    t1, t2 = table.clone(), table.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(mine, t1, plan, out)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        other = tuple(torch.empty_like(t) for t in plan)
        want = torch.empty_like(out)
        step(theirs, t2, other, want)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(t1, t2)
        for a, b in zip(mine, theirs):
            assert torch.equal(a, b)
        cached += 1
        qkv.copy_(torch.randn((R, 3, kv, D), device=dev) * (1.5 ** i))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D,group,new", [(64, 2, 3), (64, 2, 60), (32, 2, 70), (128, 1, 130), (256, 3, 40)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 90), (False, 0)])
def test_histories_longer_than_their_table_rows(dev, dtype, D, group, new, causal, window):
    """Positions past the table row are positions without a block: the queries stay at the history's end."""
    held, cu = [300, 70, 1500], [0, new, 2 * new, 3 * new]
    cache = Cache(dev, held, 2, 16, D, 41)
    whole = cache.table
    q = queries(dev, 3 * new, 2 * group, D, dtype, 42)
    for cols in (1, 6, 40):
        cache.table = whole.clone()
        cache.table[:, cols:] = -1
        want, wl = check(cache, q, cu, causal=causal, window=window)
        got, gl = hlr.hist_attention(q, *cache.tensors(), whole[:, :cols].contiguous(), cache.lengths,
                                     torch.tensor(cu, dtype=torch.int32, device=dev), new, max(held), causal=causal,
                                     window=window, return_lse=True)
        assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("D,group", [(32, 1), (64, 3), (128, 2), (256, 1), (64, 1)])
def test_the_widest_windows(dev, D, group):
    """A window of up to 2^31 - 1 hides nothing, also from requests with more queries than events."""
    held, new = [1, 20, 400], [20, 300, 90]
    cache = Cache(dev, held, 1, 32, D, 43)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = queries(dev, cu[-1], group, D, "bf16", 44)
    want, wl = check(cache, q, cu)
    for window in (400, 401, 2 ** 31 - 400, 2 ** 31 - 2, 2 ** 31 - 1):
        got, gl = check(cache, q, cu, window=window)
        assert torch.equal(got, want) and torch.equal(gl, wl), window


@pytest.mark.parametrize("D,group,new", [(64, 2, 1), (32, 2, 90), (64, 1, 70), (128, 4, 20), (256, 2, 40)])
def test_scales_of_blocks_that_nobody_sees_may_be_anything(dev, D, group, new):
    """Blocks of a table row behind the length, or before the window, in a tile with blocks that are seen."""
    cache = Cache(dev, [112, 160, 192], 2, 16, D, 45)
    cache.lengths = torch.tensor([100, 98, 130], dtype=torch.int32, device=dev)
    cu = [0, new, 2 * new, 3 * new]
    q = queries(dev, 3 * new, 2 * group, D, "bf16", 46)
    for window in (0, 5):
        first_seen = [max(0, n - new - window) // 16 if window else 0 for n in (100, 98, 130)]
        want, wl = check(cache, q, cu, window=window)
        for bad in (math.nan, math.inf, -math.inf, -3e38):
            dirty = Cache(dev, [112, 160, 192], 2, 16, D, 45)
            dirty.lengths = cache.lengths
            for r, n in enumerate((100, 98, 130)):
                blocks = dirty.table[r].tolist()
                for col, b in enumerate(blocks):
                    if b >= 0 and (col * 16 >= n or col < first_seen[r]):
                        dirty.ks[b] = dirty.vs[b] = bad
            got, gl = hlr.hist_attention(q, *dirty.tensors(), dirty.table, dirty.lengths,
                                         torch.tensor(cu, dtype=torch.int32, device=dev), new, 130, window=window,
                                         return_lse=True)
            assert torch.equal(got, want) and torch.equal(gl, wl), bad


def test_append_and_read_beyond_one_launch(dev):
    """More blocks than the 2^32 threads of a launch hold: 130 spans of 64 tokens, keys and values of 65,535 heads."""
    heads, B, D, n = 65535, 16, 32, 64 * 129 + 10
    g = torch.Generator(device=dev)
    g.manual_seed(51)
    x = torch.randn((2, n, 1, D), generator=g, device=dev).to(torch.bfloat16)
    slots = torch.full((n,), -1, dtype=torch.int64, device=dev)
    real = [10, 8190, 8191, 8192, 8193, 8260, n - 1]  # spans 0, 127, 128 and 129; a run over the border of the launches
    slots[real] = torch.tensor([17, 32, 33, 34, 35, 0, 50], device=dev)
    pools = []
    for h in (heads, 2):
        pool = [torch.zeros((4, h, B, D), dtype=torch.int8, device=dev), torch.zeros((4, h, 1, D, 16), dtype=torch.int8, device=dev),
                torch.zeros((4, h), device=dev), torch.zeros((4, h), device=dev)]
        hlr.hist_append(*pool, x[0].expand(n, h, D), x[1].expand(n, h, D), slots)
        pools.append(pool)
    for big, small in zip(*pools):
        assert bool((big == small[:, :1]).all()) and bool(small.any())
    want = hlr.hist_read(*pools[1], slots, dtype=torch.bfloat16)
    got = hlr.hist_read(*pools[0], slots, dtype=torch.bfloat16)
    for a, b in zip(got, want):
        for t in real + [0, 11, 8189, 8194, n - 2]:
            assert bool((a[t] == b[t, :1]).all()) and bool(b[t].any()) == (t in real)
    del got, a
    torch.cuda.empty_cache()


def test_attention_beyond_one_launch(dev):
    """More blocks than the 2^32 threads of a launch hold, over requests and over the joined rows."""
    R, D = 65535, 32
    cache = Cache(dev, [16] * 9, 1, 16, D, 53)
    g = torch.Generator(device=dev)
    g.manual_seed(54)
    q = torch.randn((R, 1, D), generator=g, device=dev).to(torch.bfloat16)
    table = torch.randint(0, 9, (R, 1), generator=g, device=dev).to(torch.int32)
    lengths = torch.randint(0, 17, (R,), generator=g, device=dev).to(torch.int32)
    cu = torch.arange(R + 1, dtype=torch.int32, device=dev)
    max_q = 128 * 256 + 1  # 257 blocks of rows for each request
    out, lse = hlr.hist_attention(q, *cache.tensors(), table, lengths, cu, max_q, 16, return_lse=True)
    for a, b in ((0, 30_000), (30_000, R)):
        want, wl = hlr.hist_attention(q[a:b], *cache.tensors(), table[a:b], lengths[a:b], cu[:b - a + 1], max_q, 16,
                                      return_lse=True)
        assert torch.equal(out[a:b], want) and torch.equal(lse[a:b], wl)
    cache = Cache(dev, [1100, 1], 1, 16, D, 55)
    n = (1 << 22) + 10
    q = torch.zeros((n, 4, D), dtype=torch.bfloat16, device=dev)  # all but the last two tokens belong to no request
    q[-2:] = queries(dev, 2, 4, D, "bf16", 56)
    want, wl = check(cache, q[-2:], [0, 1, 2])
    ws = hlr.new_workspace(dev, hlr.hist_attention_workspace_size(n, 2, 4, 1, D, 1, 1100))
    got, gl = hlr.hist_attention(q, *cache.tensors(), cache.table, cache.lengths,
                                 torch.tensor([n - 2, n - 1, n], dtype=torch.int32, device=dev), 1, 1100, return_lse=True,
                                 ws=ws)
    assert torch.equal(got[-2:], want) and torch.equal(gl[-2:], wl)


# --------------------------------------------------------------- refusals
def test_refusals(dev):
    cache = Cache(dev, [20, 20], 2, 16, 64, 27)
    q = queries(dev, 2, 4, 64, "bf16", 28)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)
    good = dict(table=cache.table, lengths=cache.lengths, cu=cu)

    def call(q=q, t=cache.tensors(), table=cache.table, lengths=cache.lengths, cu=cu, max_q=1, max_len=20, **kw):
        return hlr.hist_attention(q, *t, table, lengths, cu, max_q, max_len, **kw)

    call(**good)
    with pytest.raises(hlr.HLRError):
        call(q=q.cpu())
    with pytest.raises(TypeError):
        call(q=q.double())
    with pytest.raises(hlr.HLRError):
        call(q=q[:, :3])  # 3 heads over 2
    with pytest.raises(hlr.HLRError):
        call(q=q[..., :32])
    with pytest.raises(hlr.HLRError):
        call(cu=cu[:2])
    with pytest.raises(TypeError):
        call(lengths=cache.lengths.long())
    with pytest.raises(hlr.HLRError):
        call(causal=False, window=3)
    with pytest.raises(hlr.HLRError):
        call(window=-1)
    with pytest.raises(hlr.HLRError):
        call(scale=math.nan)
    with pytest.raises(hlr.HLRError):
        call(max_q=-1)
    odd = torch.zeros(2 * 4 * 64 + 1, dtype=torch.bfloat16, device=dev)[1:].view(2, 4, 64)
    with pytest.raises(hlr.HLRError):
        call(q=odd)  # not 16-byte aligned
    with pytest.raises(hlr.HLRError):
        call(max_len=100_000, ws=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(hlr.HLRError):
        hlr.hist_append(*cache.tensors(), q[:, :2], q[:, :2], torch.zeros(1, dtype=torch.int64, device=dev))
    with pytest.raises(hlr.HLRError):
        hlr.hist_append(*cache.tensors(), q[:, :2], q[:, :2].float(), torch.zeros(2, dtype=torch.int64, device=dev))
    with pytest.raises(hlr.HLRError):
        hlr.hist_plan(cu[:2], cu[:2], cache.table[:1], cu, 16, 4)
    with pytest.raises(hlr.HLRError):
        hlr.hist_plan(cu[:2], cu[:2], cache.table, cu, 24, 4)  # not a power of two
    bad = torch.zeros((3, 2, 16, 48), dtype=torch.int8, device=dev)
    with pytest.raises(hlr.HLRError):  # 48 elements
        hlr.hist_read(bad, bad.view(3, 2, 1, 48, 16), cache.ks[:3], cache.vs[:3], torch.zeros(1, dtype=torch.int64, device=dev))
