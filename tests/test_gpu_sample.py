"""sample_scores against its definition in 64 bits.

A row's item has to be the definition's wherever that does not hang on roundings: the drawn item's margin over the
next in the race, and the distance of each filter's edge, are larger than what fp32 can move them by.  z carries
|z| 2^-24 and log(noise) as much again, so the race needs a margin of 1e-5 (|z| + |log noise| stay below 100
here); masses are relative to 1 and carry at most 1e-6 of their sum; min_p compares exp(z - max z), off by at most
(2 + |z - max z|) 2^-23 of itself.  logprob: 2^-22 (4 + |z| + |logprob|)."""
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


def draw_row(x, e, t, k, p, mp):
    """(index, logprob, safe) of one row: x, e float64 arrays."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    left = np.flatnonzero(x > -np.inf)
    if not len(left):
        return -1, -np.inf, True
    z = x[left] / t if t > 0 else x[left]
    by = np.argsort(-z, kind="stable")
    left, z = left[by], z[by]
    with np.errstate(under="ignore"):
        w = np.exp(z - z[0])
    logprob = lambda i: z[i] - z[0] - math.log(w.sum())  # noqa: E731
    if not t > 0:
        return left[0], logprob(0), True
    n = len(z) if k <= 0 else min(k, len(z))
    safe = True
    if p < 1:
        before = np.cumsum(w[:n]) - w[:n]
        edge = p * w[:n].sum()
        # an edge near the border of an item matters only as far as that item is likely to be drawn
        safe &= bool((np.abs(before - edge) > 1e-6 * w[:n].sum())[1:].all())
        n = max(1, int((before < edge).sum()))
    if mp > 0:
        safe &= bool((np.abs(w[:n] - mp) > 1e-5 * mp).all() or mp >= 1)
        n = max(1, int((w[:n] >= mp).sum()))
    race = z[:n] - np.log(e[left[:n]])
    i = int(np.argmax(race))
    top = np.sort(race)[::-1]
    safe &= n == 1 or top[0] - top[1] > 1e-5
    return left[i], logprob(i), safe


def check(dev, x, e, t=None, k=None, p=None, mp=None, few=0.05):
    """x: scores on the GPU; e: noise; filters as lists or None."""
    R = x.shape[0]
    on = lambda v, dt: None if v is None else torch.tensor(v, dtype=dt, device=dev)  # noqa: E731
    f = torch.float32
    index, logprob = hlr.sample_scores(x, e, on(t, f), on(k, torch.int32), on(p, f), on(mp, f))
    again = hlr.sample_scores(x, e, on(t, f), on(k, torch.int32), on(p, f), on(mp, f))
    assert torch.equal(index, again[0]) and torch.equal(logprob, again[1])
    xs, es = x.double().cpu().numpy(), e.double().cpu().numpy()
    unsafe = 0
    f32 = lambda v, d: d if v is None else float(np.float32(v))  # noqa: E731
    for r in range(R):
        i, lp, safe = draw_row(xs[r], es[r], f32(t and t[r], 1.0), 0 if k is None else k[r], f32(p and p[r], 1.0),
                               f32(mp and mp[r], 0.0))
        if not safe:
            unsafe += 1
            continue
        assert int(index[r]) == i, f"row {r}: {int(index[r])}, not {i}"
        if i < 0:
            assert float(logprob[r]) == -math.inf
        else:
            by = f32(t and t[r], 1.0)
            tol = 2.0 ** -22 * (4 + abs(xs[r][i]) / (by if by > 0 else 1.0) + abs(lp))
            assert abs(float(logprob[r]) - lp) <= tol
    assert unsafe <= few * R + 1


def inputs(dev, R, V, dtype, seed, spread=2.5):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.randn((R, V), generator=g, device=dev) * spread
    e = torch.empty((R, V), device=dev).exponential_(generator=g).clamp_(min=1e-30)
    return x.to(TYPES[dtype]), e


def filters(R, seed):
    g = np.random.default_rng(seed)
    t = np.where(g.random(R) < 0.1, 0.0, g.uniform(0.3, 2.0, R)).tolist()
    k = np.where(g.random(R) < 0.2, 0, np.exp(g.uniform(0, 7, R))).astype(int).tolist()
    return t, k, g.uniform(0.05, 0.999, R).tolist(), (0.3 * g.random(R) ** 3).tolist()


SIZES = [1, 2, 3, 63, 64, 65, 255, 257, 1024, 2047, 2049, 2500, 8191, 32768, 32769, 50_003, 131_072]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", SIZES)
def test_sizes(dev, dtype, V):
    R = 40 if V < 10_000 else 6
    x, e = inputs(dev, R, V, dtype, V)
    check(dev, x, e, *filters(R, V + 1))


@pytest.mark.parametrize("which", ["none", "t", "k", "p", "m", "kp", "km", "pm"])
@pytest.mark.parametrize("V", [700, 5000, 40_000])
def test_filters_apart(dev, which, V):
    R = 12
    x, e = inputs(dev, R, V, "fp32", 5)
    t, k, p, m = filters(R, 6)
    check(dev, x, e, t if "t" in which else None, k if "k" in which else None, p if "p" in which else None,
          m if "m" in which else None, few=0.1)


@pytest.mark.parametrize("V", [90, 3000, 70_000])
def test_equal_scores_go_by_index(dev, V):
    """Few distinct values: the filters' edges fall among equal items, of which the first by index stay."""
    g = np.random.default_rng(V)
    x = torch.from_numpy(g.integers(-3, 4, size=(30, V)).astype(np.float32)).to(dev)
    x[5] = 0.0
    x[6, ::2] = -0.0  # equal to +0
    x[6, 1::2] = 0.0
    _, e = inputs(dev, 30, V, "fp32", 1)
    k = [int(v) for v in g.integers(1, V, size=30)]
    check(dev, x, e, k=k, few=0.1)
    # the noise makes the last kept item win: one past it must not be drawn
    e2 = torch.full_like(e, 1.0)
    x[:] = 1.0
    for r in range(30):
        e2[r, k[r] - 1] = 0.5
        e2[r, k[r]:] = 0.25
    index, _ = hlr.sample_scores(x, e2, top_k=torch.tensor(k, dtype=torch.int32, device=dev))
    assert index.tolist() == [v - 1 for v in k]
    # top-p among equal items: the first ceil(p V) of them
    p = [0.25, 0.5, 0.75] * 10
    n = [math.ceil(v * V) for v in p]
    e2.fill_(1.0)
    for r in range(30):
        e2[r, n[r] - 1] = 0.5
        e2[r, n[r]:] = 0.25
    index, _ = hlr.sample_scores(x, e2, top_p=torch.tensor(p, device=dev))
    assert index.tolist() == [v - 1 for v in n]
    # and in the race: equal everywhere, the lowest index
    e2.fill_(1.0)
    assert hlr.sample_scores(x, e2)[0].tolist() == [0] * 30


def test_masked_and_odd_values(dev):
    V = 300
    x, e = inputs(dev, 12, V, "fp32", 9)
    x[0] = -math.inf                       # nothing left
    x[1] = math.nan
    x[2] = -math.inf
    x[2, 77] = -50.0                       # one left
    x[3, ::3] = math.nan
    x[4, 11] = math.inf                    # counts as the largest number
    x[5] = torch.finfo(torch.float32).min  # a mask of the type's lowest value everywhere
    x[6, 1:] = torch.finfo(torch.float32).min
    x[7] = 3e38
    x[8] *= 1e-38
    t = [1.0] * 12
    t[9], t[10], t[11] = 0.0, -1.0, 1e-3
    check(dev, x, e, t=t, few=0.2)  # in rows 5 and 7 the noise is below a step of the scores: no margin
    index, logprob = hlr.sample_scores(x, e, torch.tensor(t, device=dev), torch.full((12,), 5, dtype=torch.int32, device=dev),
                                       torch.zeros(12, device=dev), torch.full((12,), 2.0, device=dev))
    # a top_p of 0 and a min_p above 1 leave the first item
    for r in range(12):
        row = np.where(np.isnan(x[r].cpu().numpy()), -np.inf, x[r].cpu().numpy())
        assert int(index[r]) == (-1 if row.max() == -np.inf else int(row.argmax()))
    assert float(logprob[0]) == -math.inf and float(logprob[2]) == 0.0
    assert abs(float(logprob[5]) + math.log(V)) < 1e-5


@pytest.mark.parametrize("V", [90, 700, 3000, 20_000, 70_000])
def test_infinite_temperature(dev, V):
    """Every item that can be drawn weighs the same; rank still goes by score."""
    R = 8
    x, e = inputs(dev, R, V, "fp32", V)
    x[:, ::3] = -math.inf
    x[:, 1::7] = math.nan
    x[5, :] = -math.inf
    x[5, V // 2] = 3.0
    xs, es = x.cpu().numpy(), e.cpu().numpy()
    for t in (math.inf, 3e38):
        for k, p, m in ((0, 1.0, 0.0), (7, 1.0, 0.0), (0, 0.37, 0.0), (0, 1.0, 0.5), (V // 2, 0.61, 0.2), (V // 5, 1.0, 0.0)):
            on = lambda v, dt=torch.float32: torch.full((R,), v, dtype=dt, device=dev)  # noqa: E731
            index, logprob = hlr.sample_scores(x, e, on(t), on(k, torch.int32), on(p), on(m))
            for r in range(R):
                left = np.flatnonzero(xs[r] > -np.inf)
                by = left[np.argsort(-xs[r][left], kind="stable")]
                n = min(k, len(by)) if k else len(by)
                if p < 1 and n > 1:
                    # equal weights: item i is kept while i < p n, where p n is no whole number's neighbour
                    edge = float(np.float32(p)) * n
                    if abs(edge - round(edge)) < 1e-3:
                        continue
                    n = int(edge) + 1
                kept = by[:n]
                assert int(index[r]) == kept[np.argmin(es[r][kept])], (t, k, p, m, r)
                assert abs(float(logprob[r]) + math.log(len(left))) <= 2.0 ** -22 * (4 + math.log(len(left)))


def test_no_rows_no_items(dev):
    x = torch.zeros((0, 7), device=dev)
    assert hlr.sample_scores(x, x)[0].numel() == 0
    x = torch.zeros((3, 0), device=dev)
    index, logprob = hlr.sample_scores(x, x)
    assert index.tolist() == [-1] * 3 and logprob.tolist() == [-math.inf] * 3


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strided_rows_and_streams(dev, dtype):
    x, e = inputs(dev, 9, 4001, dtype, 11)
    t, k, p, m = filters(9, 12)
    check(dev, x[:, 3:3700], e[:, 7:3704], t, k, p, m, few=0.2)  # rows that start anywhere
    check(dev, x[::2], e[::2], t[::2], k[::2], p[::2], m[::2], few=0.2)
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    a = hlr.sample_scores(x, e, stream=side)
    b = hlr.sample_scores(x, e)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_frequencies(dev):
    """60,000 draws of one row, kept to its first 4 items: their shares are those of exp(z)."""
    n = 60_000
    x = torch.tensor([0.5, 2.0, 1.0, -1.0, 1.5, 0.0], device=dev).repeat(n, 1)
    _, e = inputs(dev, n, 6, "fp32", 13)
    index, _ = hlr.sample_scores(x, e, torch.full((n,), 0.8, device=dev), torch.full((n,), 4, dtype=torch.int32, device=dev))
    got = torch.bincount(index, minlength=6).double().cpu().numpy()
    w = np.exp(np.array([0.5, 2.0, 1.0, -1.0, 1.5, 0.0]) / 0.8)
    w[[3, 5]] = 0
    want = n * w / w.sum()
    assert got[3] == 0 and got[5] == 0
    kept = want > 0
    assert float(((got - want)[kept] ** 2 / want[kept]).sum()) < 27.9  # chi-square, 3 degrees, 4e-6


def test_more_rows_than_a_launch_has_blocks(dev):
    """2^22 blocks of 1,024 threads pass the 2^32 threads of one launch."""
    rows, items = (1 << 22) + 5, 600
    x = torch.zeros((1, items), device=dev).expand(rows, items)
    e = (1.0 / torch.arange(1, items + 1, device=dev))[None].expand(rows, items)  # of equal scores the last one kept wins
    k = 1 + torch.arange(rows, device=dev, dtype=torch.int32) % 577
    index, logprob = hlr.sample_scores(x, e, top_k=k)
    assert torch.equal(index, k.long() - 1)
    assert float((logprob + math.log(items)).abs().max()) <= 2.0 ** -22 * (4 + math.log(items))


def test_refusals(dev):
    x, e = inputs(dev, 4, 100, "fp32", 15)
    with pytest.raises(hlr.HLRError):
        hlr.sample_scores(x.cpu(), e)
    with pytest.raises(TypeError):
        hlr.sample_scores(x.double(), e)
    with pytest.raises(hlr.HLRError):
        hlr.sample_scores(x, e[:, :99])
    with pytest.raises(hlr.HLRError):
        hlr.sample_scores(x, e.to(torch.bfloat16))
    with pytest.raises(hlr.HLRError):
        hlr.sample_scores(x.t(), e.t())
    with pytest.raises(hlr.HLRError):
        hlr.sample_scores(x, e, torch.ones(3, device=dev))
    with pytest.raises(TypeError):
        hlr.sample_scores(x, e, top_k=torch.ones(4, device=dev))
