"""The 4-bit KV cache (append, read, attention, eviction) against its plain 64-bit form, through the public
interface.  Pools start as garbage (NaN scales), so anything read from a row that does not exist shows.

Tolerances.  fp32 attention: a score is a sum of d products; its operands carry 22 bits (2^-22) and its
fp32 sums at most 2^-23 a step, errors that add like independent ones, so a score of size S (at most
scale |q| |k|, plus the bias where it matters, below 32) is off by about S (2^-22 + sqrt(d) 2^-23) and a weight
by that share of itself; the weights' own pairs, exp2 and the sums add less than 2^-19.  The output is a mean
with these weights, so its 2-norm error relative to its 2-norm is held to that sum.  bf16: the output's
rounding, 2^-8 at most, and the weights' rounding to fp16, 2^-11, come on top.
"""
import numpy as np
import pytest
import torch

import kv4_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_decode_megakernel_gb300 import build
    build.build()


class Setup:
    """A plain pool and the same bytes on the GPU, with shuffled pages and ragged sequences."""

    def __init__(self, rows, counts, heads=4, kv=2, d=64, page=32, track=False, layers=2, layer=1, seed=0, spare=2, fill=True, gap=1):
        from persistent_decode_megakernel_gb300.kv4 import Kv4Cache
        rng = np.random.default_rng(seed)
        self.rng, self.layer, self.heads, self.kv, self.d = rng, layer, heads, kv, d
        self.rows, self.counts = list(rows), list(counts)
        self.offsets = [0] + np.cumsum(counts).tolist()
        need = [-(-max(r, 1) // page) for r in rows]
        # a table that may reach far makes prompts of few tokens worth the prompt kernel
        self.max_pages = 2 ** 17 // page if max(counts) * heads >= 64 * kv else max(need) + 1
        perm = rng.permutation(sum(need) + spare)
        self.tables = np.full((len(rows), self.max_pages), -7, np.int32)  # entries behind the last page are never read
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = perm[at:at + n]
            at += n
        self.spare = perm[at:]
        self.pool = plain.PlainPool(layers, kv, d, len(perm), page, track)
        # positions with gaps: old row i at gap * i, the new tokens one after the other
        self.positions = [gap * (r - c) for r, c in zip(rows, counts)] if track else None
        self.shift = rng.normal(size=(2, kv, d)) * np.array([1.0, 0.1]).reshape(2, 1, 1)
        if fill:
            for s, (r, c) in enumerate(zip(rows, counts)):
                for i in range(r):
                    pos = gap * i if i < r - c else gap * (r - c) + i - (r - c)
                    for h in range(kv):
                        x = (rng.normal(size=(2, d)) + self.shift[:, h]).astype(np.float32)
                        self.pool.put(layer, self.tables[s], i, h, x[0], x[1], pos, float(rng.random()))
        self.cache = Kv4Cache(layers, heads, kv, d, len(perm), page, self.max_pages, track,
                              pool=torch.from_numpy(self.pool.bytes.reshape(-1).copy()).cuda())
        self.dev = {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in
                    dict(offsets=self.offsets, rows=self.rows, tables=self.tables.tolist()).items()}
        self.dev["positions"] = torch.tensor(self.positions, dtype=torch.int32, device="cuda") if track else None
        self.batch = self.cache.batch(self.dev["offsets"], self.dev["rows"], self.dev["tables"], self.dev["positions"])

    def q(self, dtype):
        x = torch.from_numpy(self.rng.normal(size=(self.offsets[-1], self.heads, self.d)) * 1.5).to(dtype)
        return x

    def bytes(self):
        return self.cache.pool.cpu().numpy().reshape(self.pool.bytes.shape)

    def expect(self, q, **kw):
        return plain.attention(self.pool, self.layer, q.double().numpy(), self.offsets, self.rows, self.tables, self.positions, self.heads,
                               self.d ** -0.5, **kw)

    def tolerance(self, q, dtype):
        k = max(np.linalg.norm(self.pool.get(self.layer, self.tables[s], i, h)[0])
                for s, r in enumerate(self.rows) for i in range(0, r, 7) for h in range(self.kv)) * 1.2 if max(self.rows) else 0.0
        size = float(q.double().norm(dim=-1).max()) * k * self.d ** -0.5 + 32
        tol = size * (2.0 ** -22 + self.d ** 0.5 * 2.0 ** -23) + 2.0 ** -19
        return tol + (2.0 ** -8 + 2.0 ** -11 if dtype == torch.bfloat16 else 0.0)


def check(got, want, tol, what):
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert np.isfinite(got).all(), what
    off = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
    assert off <= tol, f"{what}: {off:.3g} off, {tol:.3g} allowed"
    assert (got[want == 0] == 0).all(), what


HEADS = [(4, 2, 64), (9, 3, 64), (16, 1, 64), (3, 3, 128), (8, 1, 128), (14, 2, 64), (16, 1, 128)]
BATCHES = {
    "one": ([1], [1]),
    "edges": ([31, 32, 33, 64, 1, 7], [1] * 6),
    "empty": ([0, 5, 0, 40], [1, 0, 0, 1]),        # no rows; idle slots with and without rows
    "few": ([3, 40, 10, 129], [3, 1, 0, 5]),
    "prompt": ([70, 300, 95], [70, 1, 33]),
}
FEATURES = {"plain": {}, "cap": dict(cap=5.0), "bias": dict(slopes=True), "window": dict(window=17), "own": dict(window=1),
            "all": dict(cap=20.0, slopes=True, window=40)}


def _kw(s, name):
    kw = dict(FEATURES[name])
    if "slopes" in kw:
        kw["slopes"] = np.array([2.0 ** (-8.0 * (h + 1) / s.heads) for h in range(s.heads)], np.float32)
    return kw


def _run(s, q, kw, **more):
    dev = dict(kw)
    if "slopes" in dev:
        dev["slopes"] = torch.from_numpy(dev["slopes"]).cuda()
    return s.cache.attention(s.layer, s.batch, q.cuda(), **dev, **more)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_attention_shapes(heads, batch, dtype):
    s = Setup(*BATCHES[batch], *heads)
    q = s.q(dtype)
    want, _ = s.expect(q)
    check(_run(s, q, {}), want, s.tolerance(q, dtype), "out")
    assert s.cache.status() == 0


@pytest.mark.parametrize("track", [False, True], ids=["untracked", "tracked"])
@pytest.mark.parametrize("feature", list(FEATURES))
@pytest.mark.parametrize("heads,dtype", [((9, 3, 64), torch.float32), ((8, 2, 128), torch.bfloat16), ((4, 2, 128), torch.float32)], ids=str)
@pytest.mark.parametrize("batch", ["edges", "few", "prompt"])
def test_attention_features(heads, dtype, feature, track, batch):
    s = Setup(*BATCHES[batch], *heads, track=track, gap=2, seed=3)
    q = s.q(dtype)
    kw = _kw(s, feature)
    want, _ = s.expect(q, **kw)
    check(_run(s, q, kw), want, s.tolerance(q, dtype), feature)


@pytest.mark.parametrize("feature", ["plain", "all"])
@pytest.mark.parametrize("heads,dtype", [((9, 3, 64), torch.float32), ((8, 2, 128), torch.bfloat16), ((16, 1, 64), torch.bfloat16)], ids=str)
@pytest.mark.parametrize("batch", ["edges", "empty", "few", "prompt"])
def test_attention_adds_up_the_weights(heads, dtype, feature, batch):
    s = Setup(*BATCHES[batch], *heads, track=True, gap=2, seed=4)
    q = s.q(dtype)
    kw = _kw(s, feature)
    want, w = s.expect(q, **kw)
    before = s.bytes().copy()
    check(_run(s, q, kw, accumulate=True), want, s.tolerance(q, dtype), "out")
    tol = s.tolerance(q, torch.float32)
    after = plain.PlainPool.__new__(plain.PlainPool)
    after.__dict__.update(s.pool.__dict__)
    after.bytes = s.bytes()
    for (q_, i, h), x in w.items():
        old = s.pool.weight(s.layer, s.tables[q_], i, h)
        # the share of x that the scores' errors make, and the rounding of the sum
        assert abs(after.weight(s.layer, s.tables[q_], i, h) - old - x) <= 4 * tol * x + 2.0 ** -23 * (old + x), (q_, i, h)
    # nothing else of the pool changed
    at = 2 * (s.pool.code + s.pool.pair) + 128
    same = after.bytes == before
    assert same[..., :at].all() and same[:, 0].all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("rows,counts,heads", [([5000, 3, 900], [1, 1, 1], (6, 2, 64)), ([4097], [2], (8, 1, 128)), ([2500], [200], (2, 1, 64))],
                         ids=["decode", "two", "prompt"])
def test_attention_split_over_many_ctas(rows, counts, heads, dtype):
    s = Setup(rows, counts, *heads, page=128)
    q = s.q(dtype)
    want, _ = s.expect(q)
    check(_run(s, q, {}), want, s.tolerance(q, dtype), "out")


def test_attention_large_and_small_values():
    """Scales of V from 1e-4 to 1e3 in one sequence, K near fp16's end, queries of 1e-6 and 1e4."""
    s = Setup([200], [1], 4, 2, 64, fill=False)
    for i in range(200):
        for h in range(2):
            k = s.rng.normal(size=64) * 10.0 ** s.rng.uniform(-4, 2)
            v = s.rng.normal(size=64) * 10.0 ** s.rng.uniform(-4, 3)
            s.pool.put(s.layer, s.tables[0], i, h, k.astype(np.float32), v.astype(np.float32))
    s.cache.pool.copy_(torch.from_numpy(s.pool.bytes.reshape(-1)))
    for size in (1e-6, 0.02):
        q = s.q(torch.float32) * size
        want, _ = s.expect(q)
        check(_run(s, q, {}), want, s.tolerance(q, torch.float32), str(size))


def test_nan_in_a_masked_row_stays_there():
    """Row 5 is NaN: the tokens before it do not see it, the others become NaN."""
    s = Setup([8], [8], 4, 2, 64)
    bad = np.full(64, np.nan, np.float32)
    for h in range(2):
        s.pool.put(s.layer, s.tables[0], 5, h, bad, bad)
    s.cache.pool.copy_(torch.from_numpy(s.pool.bytes.reshape(-1)))
    q = s.q(torch.float32)
    out = _run(s, q, {}).cpu()
    s.rows, s.offsets = [5], [0, 5]
    want, _ = s.expect(q[:5])
    check(out[:5], want, 1e-4, "rows before the NaN")
    assert out[5:].isnan().all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("heads", [(3, 3, 64), (8, 2, 128)], ids=str)
@pytest.mark.parametrize("track", [False, True], ids=["untracked", "tracked"])
def test_append_writes_the_format_and_nothing_else(heads, dtype, track):
    s = Setup([3, 70, 10, 33, 2], [3, 41, 0, 1, 2], *heads, track=track, gap=3, seed=5)
    n, kv, d = s.offsets[-1], s.kv, s.d
    x = torch.from_numpy(s.rng.normal(size=(n, 3 * kv, d)) * 2).to(dtype)  # k and v inside a wider row, as a projection leaves them
    x[0, 0] = 1.25                                 # a constant row
    x[1, kv, :64] = torch.linspace(0, 15, 64).to(dtype)
    x[2, 1, 3] = float("inf")
    x[2, 2, 7] = -1e30
    x[3, 0] = 1e-7
    y = x.cuda()
    s.cache.append(s.layer, s.batch, y[:, :kv], y[:, kv:2 * kv])
    xs = x.float().numpy()
    for q in range(len(s.rows)):
        for i in range(s.counts[q]):
            t = s.offsets[q] + i
            for h in range(kv):
                s.pool.put(s.layer, s.tables[q], s.rows[q] - s.counts[q] + i, h, xs[t, h], xs[t, kv + h],
                           s.positions[q] + i if track else None, 0.0)
    assert (s.bytes() == s.pool.bytes).all()
    # read gives the rows back
    for out in (torch.float32, torch.bfloat16):
        k, v = s.cache.read(s.layer, s.batch, out)
        step = 2.0 ** -23 if out == torch.float32 else 2.0 ** -8
        for q in range(len(s.rows)):
            for i in range(s.counts[q]):
                for h in range(kv):
                    want = s.pool.get(s.layer, s.tables[q], s.rows[q] - s.counts[q] + i, h)
                    for a, b in zip((k, v), want):
                        got = a[s.offsets[q] + i, h].double().cpu().numpy()
                        assert np.all(np.abs(got - b) <= step * np.abs(b) + 2.0 ** -23 * np.abs(b).max()), (q, i, h)
    assert s.cache.status() == 0


def test_append_of_nan_makes_the_group_nan():
    s = Setup([4], [4], 2, 1, 128)
    x = torch.from_numpy(s.rng.normal(size=(4, 1, 128))).float()
    x[1, 0, 70] = float("nan")
    s.cache.append(s.layer, s.batch, x.cuda(), x.cuda())
    k, v = s.cache.read(s.layer, s.batch)
    for t in (k, v):
        assert t[1, 0, 64:].isnan().all() and t[1, 0, :64].isfinite().all() and t[[0, 2, 3]].isfinite().all()


@pytest.mark.parametrize("inputs", ["random", "ties", "nan"])
@pytest.mark.parametrize("place", ["in place", "elsewhere"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (3, 3, 128)], ids=str)
@pytest.mark.parametrize("rows,keep,recent", [([100, 40, 0, 64, 65], 64, 16), ([33, 1, 3000], 1, 1), ([2200, 1100], 1000, 0), ([70], 37, 37)], ids=str)
def test_evict(rows, keep, recent, heads, place, inputs):
    s = Setup(rows, [min(r, 1) for r in rows], *heads, track=True, gap=2, seed=6, spare=2 + len(rows) * -(-keep // 32))
    pool, layer = s.pool, s.layer
    at = 2 * (pool.code + pool.pair) + 128
    w = pool.bytes[..., at:at + 128].copy().view(np.float32)
    if inputs != "random":
        w[...] = np.round(np.abs(s.rng.normal(size=w.shape)) * 3) / 4
    if inputs == "nan":
        w[s.rng.random(w.shape) < 0.2] = np.nan
        w[s.rng.random(w.shape) < 0.1] = -0.0
    pool.bytes[..., at:at + 128] = w.view(np.uint8)
    s.cache.pool.copy_(torch.from_numpy(pool.bytes.reshape(-1)))
    before = pool.bytes.copy()
    nxt = [2 * (r - min(r, 1)) + 1 for r in rows]
    out = None
    if place == "elsewhere":
        out = s.spare[:len(rows) * -(-keep // 32)].reshape(len(rows), -1).astype(np.int32)
    got = s.cache.evict(s.dev["rows"], s.dev["tables"], torch.tensor(nxt, dtype=torch.int32, device="cuda"), keep, recent,
                        out_tables=None if out is None else torch.from_numpy(out).cuda(), layer=layer, n_layers=1)
    assert got.tolist() == [min(r, keep) for r in rows]
    old = plain.PlainPool.__new__(plain.PlainPool)
    old.__dict__.update(pool.__dict__)
    old.bytes = before
    new = plain.PlainPool.__new__(plain.PlainPool)
    new.__dict__.update(pool.__dict__)
    new.bytes = s.bytes()
    touched = np.zeros(before.shape[:4], bool)
    for q, r in enumerate(rows):
        to = s.tables[q] if out is None else out[q]
        for h in range(s.kv):
            src = plain.evict_map([old.weight(layer, s.tables[q], i, h) for i in range(r)], [old.pos(layer, s.tables[q], i, h) for i in range(r)],
                                  keep, nxt[q] - recent)
            for j, i in enumerate(src):
                assert (new.row_bytes(layer, to, j, h) == old.row_bytes(layer, s.tables[q], i, h)).all(), (q, h, j, i)
            for j in range(0, len(src), 32):
                touched[int(to[j // 32]), layer, h, 0] = True
    assert (new.bytes == before)[~touched].all()
    assert s.cache.status() == 0


def test_bad_pages_and_batches_are_reported_and_left_alone():
    from persistent_decode_megakernel_gb300 import mbk
    s = Setup([70, 64, 40], [1, 1, 1], track=True)
    q = s.q(torch.float32)
    good = _run(s, q, {}).cpu()
    assert s.cache.status() == 0
    for bad in (-1, s.pool.bytes.shape[0], 2 ** 31 - 1):
        s.cache.clear_status()
        s.dev["tables"][0, 1] = bad
        out = _run(s, q, {}, accumulate=True).cpu()
        assert s.cache.status() == mbk.MBK_KV4_BAD_PAGE
        assert torch.equal(out[1:], good[1:]) and out.isfinite().all()
        k = torch.zeros(3, 2, 64, device="cuda")
        before = s.bytes().copy()
        s.dev["tables"][0, 2] = bad  # the page of the new row
        s.cache.append(s.layer, s.batch, k, k)
        s.cache.evict(s.dev["rows"], s.dev["tables"], s.dev["rows"], 32, layer=s.layer)
        k, v = s.cache.read(s.layer, s.batch)
        assert (k[0] == 0).all() and (v[0] == 0).all()
        assert s.bytes().shape == before.shape
        s.cache.pool.copy_(torch.from_numpy(s.pool.bytes.reshape(-1)))
        s.dev["tables"].copy_(torch.from_numpy(s.tables))
    for name, at, value in (("rows", 0, 10 ** 6), ("rows", 0, -1), ("offsets", 1, 77), ("offsets", 1, -3)):
        s.cache.clear_status()
        keep = s.dev[name].clone()
        s.dev[name][at] = value
        out = _run(s, q, {}).cpu()
        s.cache.append(s.layer, s.batch, torch.zeros(3, 2, 64, device="cuda"), torch.zeros(3, 2, 64, device="cuda"))
        assert s.cache.status() & mbk.MBK_KV4_BAD_BATCH
        assert torch.equal(out[2:], good[2:])
        s.dev[name].copy_(keep)
        s.cache.pool.copy_(torch.from_numpy(s.pool.bytes.reshape(-1)))
    torch.cuda.synchronize()


def test_graph_replays_read_lengths_and_pages_again():
    """A captured step (append, attention, weights) replayed after rows, offsets, positions and tables changed."""
    s = Setup([40, 70], [1, 1], 4, 2, 64, track=True, layers=1, layer=0, spare=8)
    q, k, v = s.q(torch.float32).cuda(), torch.randn(2, 2, 64, device="cuda"), torch.randn(2, 2, 64, device="cuda")
    out = torch.zeros(2, 4, 64, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.cache.append(0, s.batch, k, v)
        s.cache.attention(0, s.batch, q, accumulate=True, out=out)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.cache.append(0, s.batch, k, v)
        s.cache.attention(0, s.batch, q, accumulate=True, out=out)
    s.cache.pool.copy_(torch.from_numpy(s.pool.bytes.reshape(-1)))
    eager = Setup([40, 70], [1, 1], 4, 2, 64, track=True, layers=1, layer=0, spare=8)
    for rows in ([40, 70], [41, 71], [42, 72], [1, 95]):
        k.copy_(torch.randn_like(k))
        q.copy_(torch.randn_like(q))
        for t in (s, eager):
            t.dev["rows"].copy_(torch.tensor(rows, dtype=torch.int32))
            t.dev["positions"].copy_(torch.tensor([r + 5 for r in rows], dtype=torch.int32))
        g.replay()
        eager.cache.append(0, eager.batch, k, v)
        want = eager.cache.attention(0, eager.batch, q, accumulate=True)
        assert torch.equal(out.view(torch.int32), want.view(torch.int32))  # rows 72 .. 94 of the last step are NaN
        assert torch.equal(s.cache.pool, eager.cache.pool)


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, give what they give one after the other."""
    s = Setup([3000, 500], [1, 1], 6, 2, 64)
    q = [s.q(torch.float32).cuda() for _ in range(2)]
    want = [s.cache.attention(s.layer, s.batch, x) for x in q]
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(st[i]):
                got[i].append(s.cache.attention(s.layer, s.batch, q[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_rows_behind_the_last_token_are_left_alone():
    s = Setup([40, 70], [1, 2], 4, 2, 64)
    batch = s.cache.batch(s.dev["offsets"], s.dev["rows"], s.dev["tables"], n_tokens=8, max_count=2)
    q = torch.randn(8, 4, 64, device="cuda")
    out = torch.full((8, 6, 64), 7.0, device="cuda")[:, 1:5]
    s.cache.attention(s.layer, batch, q, out=out)
    assert (out[3:] == 7).all() and not (out[:3] == 7).all(-1).any()
    assert torch.equal(out[:3], s.cache.attention(s.layer, s.batch, q[:3]))


def test_decode_with_eviction_step_by_step():
    """The operators as they are used together: a prompt, then decode steps that add up weights, and an
    eviction whenever the cache is over its budget, against the plain form fed the same tokens."""
    heads, kv, d, keep, recent = 6, 2, 64, 40, 8
    s = Setup([30, 50], [30, 50], heads, kv, d, page=32, track=True, layers=1, layer=0, fill=False, spare=6)
    ref, rows, nxt = s.pool, [0, 0], [0, 0]
    s.tables[:, :3] = np.arange(6).reshape(2, -1)
    s.dev["tables"].copy_(torch.from_numpy(s.tables))
    counts = [30, 50]
    for step in range(14):
        off = [0, counts[0], sum(counts)]
        n = off[-1]
        x = s.rng.normal(size=(n, 2 * kv, d)).astype(np.float32)
        q = torch.from_numpy(s.rng.normal(size=(n, heads, d)) * 2).float()
        for b in range(2):
            for i in range(counts[b]):
                for h in range(kv):
                    ref.put(0, s.tables[b], rows[b] + i, h, x[off[b] + i, h], x[off[b] + i, kv + h], nxt[b] + i, 0.0)
            rows[b] += counts[b]
        dev = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (off, rows, nxt)]
        batch = s.cache.batch(dev[0], dev[1], s.dev["tables"], dev[2])
        y = torch.from_numpy(x).cuda()
        s.cache.append(0, batch, y[:, :kv], y[:, kv:])
        out = s.cache.attention(0, batch, q.cuda(), accumulate=True)
        want, w = plain.attention(ref, 0, q.numpy(), off, rows, s.tables, nxt, heads, d ** -0.5)
        check(out, want, 1e-4, f"step {step}")
        # the weights go on from the library's own, so that rows that are nearly equal are evicted alike
        ref.bytes = s.bytes().copy()
        nxt = [a + c for a, c in zip(nxt, counts)]
        if max(rows) > keep:
            dev[1] = s.cache.evict(dev[1], s.dev["tables"], torch.tensor(nxt, dtype=torch.int32, device="cuda"), keep, recent, rows_out=dev[1])
            old = ref.bytes.copy()
            view = plain.PlainPool.__new__(plain.PlainPool)
            view.__dict__.update(ref.__dict__)
            view.bytes = old
            ref.bytes = s.bytes().copy()
            for b in range(2):
                for h in range(kv):
                    src = plain.evict_map([view.weight(0, s.tables[b], i, h) for i in range(rows[b])],
                                          [view.pos(0, s.tables[b], i, h) for i in range(rows[b])], keep, nxt[b] - recent)
                    assert all((ref.row_bytes(0, s.tables[b], j, h) == view.row_bytes(0, s.tables[b], i, h)).all() for j, i in enumerate(src))
            rows = dev[1].tolist()
            assert rows == [min(keep, r) for r in rows]
        counts = [1, 1]
    assert s.cache.status() == 0


def test_many_sequences_take_the_block_wide_scan():
    """More than 32 sequences (the split's scan over warps) and more than a block of threads, with idle slots among them."""
    rng = np.random.default_rng(7)
    for n in (33, 300):
        rows = rng.integers(0, 5, n).tolist()
        counts = [int(r > 0 and rng.random() < 0.8) for r in rows]
        counts[0], rows[0] = 1, 3
        s = Setup(rows, counts, 4, 2, 64, seed=n)
        q = s.q(torch.float32)
        want, _ = s.expect(q)
        check(_run(s, q, {}), want, s.tolerance(q, torch.float32), str(n))


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
@pytest.mark.parametrize("heads,dtype", [((4, 2, 64), torch.float32), ((8, 2, 128), torch.bfloat16)], ids=str)
def test_scales(heads, dtype, scale):
    s = Setup([60, 10, 150], [60, 1, 2], *heads)
    q = s.q(dtype)
    want, _ = plain.attention(s.pool, s.layer, q.double().numpy(), s.offsets, s.rows, s.tables, s.positions, s.heads, scale)
    got = s.cache.attention(s.layer, s.batch, q.cuda(), scale=scale)
    check(got, want, s.tolerance(q, dtype) * max(1.0, abs(scale) * s.d ** 0.5), str(scale))


@pytest.mark.parametrize("heads,dtype", [((9, 3, 64), torch.float32), ((4, 2, 128), torch.bfloat16), ((4, 2, 128), torch.float32)], ids=str)
@pytest.mark.parametrize("counts", [[10, 11, 12], [32, 33, 1], [17], [16], [8], [34, 35, 36], [48, 56, 64], [56], [40]], ids=str)
def test_around_the_border_between_the_kernels(heads, dtype, counts):
    """Query rows per KV head just below and above the prompt kernel's least, one sequence and several."""
    s = Setup([c + 45 for c in counts], counts, *heads, track=True, gap=1)
    q = s.q(dtype)
    want, w = s.expect(q)
    check(_run(s, q, {}, accumulate=True), want, s.tolerance(q, dtype), str(counts))
    got = s.cache.weights.cpu()
    for (b, i, h), x in list(w.items())[::5]:
        page, blk, lane = int(s.tables[b][i // 32]), i % 32 // 32, i % 32
        old = s.pool.weight(s.layer, s.tables[b], i, h)
        assert abs(float(got[page, s.layer, h, blk, lane]) - old - x) <= 4 * s.tolerance(q, torch.float32) * x + 2.0 ** -23 * (old + x)


def test_bounds_above_what_the_batch_holds():
    """max_count, n_tokens and max_rows are bounds: a batch of prompts whose sequences turn out to be short."""
    s = Setup([40, 70, 5], [1, 2, 0], 4, 2, 64)
    q = s.q(torch.float32)
    want, _ = s.expect(q)
    for max_count in (3, 100, 200):
        big = torch.zeros(200, 4, 64)
        big[:3] = q
        b = s.cache.batch(s.dev["offsets"], s.dev["rows"], s.dev["tables"], n_tokens=200, max_count=max_count, max_rows=96)
        check(s.cache.attention(s.layer, b, big.cuda())[:3], want, s.tolerance(q, torch.float32), str(max_count))
    one = Setup([70], [2], 4, 2, 64)
    q = one.q(torch.float32)
    want, _ = one.expect(q)
    b = one.cache.batch(one.dev["offsets"], one.dev["rows"], one.dev["tables"], n_tokens=64, max_count=64)
    big = torch.zeros(64, 4, 64)
    big[:2] = q
    check(one.cache.attention(one.layer, b, big.cuda())[:2], want, one.tolerance(q, torch.float32), "one")


def test_graphs_of_split_calls_and_evictions_at_once():
    """Two captured graphs (a long decode, a prompt; each with its own workspaces) replayed together on two streams, and an
    eviction captured with them, give what eager calls give."""
    a = Setup([3000, 900], [1, 1], 6, 2, 64, track=True, layers=1, layer=0, page=64)
    b = Setup([600, 130], [100, 90], 4, 1, 128, page=64)
    qa, qb = a.q(torch.float32).cuda(), b.q(torch.bfloat16).cuda()
    nxt = torch.tensor([4000, 4000], dtype=torch.int32, device="cuda")
    start = a.cache.pool.clone()
    def step_a():
        out = a.cache.attention(0, a.batch, qa, accumulate=True)
        return out, a.cache.evict(a.dev["rows"], a.dev["tables"], nxt, 500, 10)
    def step_b():
        return b.cache.attention(b.layer, b.batch, qb)
    want_a, want_rows = step_a()
    want_pool, want_b = a.cache.pool.clone(), step_b()
    graphs, outs, st = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for f in (step_a, step_b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for _ in range(5):
        a.cache.pool.copy_(start)
        torch.cuda.synchronize()
        for g, stream in zip(graphs, st):
            with torch.cuda.stream(stream):
                g.replay()
                if g is graphs[1]:
                    g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], want_a) and torch.equal(outs[0][1], want_rows) and torch.equal(outs[1], want_b)
        assert torch.equal(a.cache.pool, want_pool)
    assert a.cache.status() == 0 and b.cache.status() == 0


def test_a_pool_of_more_than_four_gigabytes():
    """Pages whose bytes lie beyond 2^32: append, read, attention, eviction there, and nothing written below."""
    from persistent_decode_megakernel_gb300.kv4 import Kv4Cache
    page, layers, kv, d = 1024, 8, 8, 128
    per_page = layers * kv * page * 152
    pages = 5 * 2 ** 30 // per_page + 3
    cache = Kv4Cache(layers, 16, kv, d, pages, page, 2, True)
    assert cache.bytes > 2 ** 32 + 2 * per_page
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tables, n = dev([[pages - 1, pages - 2]]), 1100
    b = cache.batch(dev([0, n]), dev([n]), tables, n_tokens=n, max_count=n)
    k, v = torch.randn(n, kv, d, device="cuda"), torch.randn(n, kv, d, device="cuda")
    cache.append(layers - 1, b, k, v)
    k4, v4 = cache.read(layers - 1, b)
    assert (k4 - k).abs().max() < 0.4 and (v4 - v).abs().max() < 0.4
    q = torch.randn(n, 16, d, device="cuda", dtype=torch.bfloat16)
    out = cache.attention(layers - 1, b, q, accumulate=True)
    p = torch.einsum("qhd,khd->hqk", q.double(), k4.double().repeat_interleave(2, 1)) * d ** -0.5
    p = p.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -np.inf).softmax(-1)
    want = torch.einsum("hqk,khd->qhd", p, v4.double().repeat_interleave(2, 1))
    assert (out.double() - want).norm() / want.norm() < 2.0 ** -8 + 2.0 ** -9
    rows = cache.evict(dev([n]), tables, dev([n]), 1000, 100, layer=layers - 1)
    assert rows.tolist() == [1000] and cache.status() == 0
    assert not cache.pool[:2 ** 32].any()


def test_evict_of_more_rows_than_keys_fit_in_shared_memory():
    """40,000 rows: the selection reads the weights again instead of keeping the keys."""
    from persistent_decode_megakernel_gb300.kv4 import Kv4Cache
    n, keep = 40000, 15000
    cache = Kv4Cache(1, 1, 1, 64, 320, 128, 320, True)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    order = torch.randperm(320, generator=torch.Generator().manual_seed(1))
    w = (torch.rand(n, generator=torch.Generator().manual_seed(2)) * 1000).round() / 8
    w = torch.cat([w, torch.full((320 * 128 - n,), 1e9)])
    cache.weights[order.cuda()] = w.view(320, 1, 1, 4, 32).cuda()
    cache.positions[order.cuda()] = torch.arange(320 * 128, dtype=torch.int32).view(320, 1, 1, 4, 32).cuda()
    rows = cache.evict(dev([n]), order.to(torch.int32).view(1, -1).cuda(), dev([n]), keep, 100)
    src = plain.evict_map(w[:n].tolist(), list(range(n)), keep, n - 100)
    assert rows.tolist() == [keep]
    assert torch.equal(cache.positions.cpu()[order].flatten()[:keep], torch.tensor(src, dtype=torch.int32))


def test_evict_leaves_a_sequence_with_a_bad_row_count_alone():
    from persistent_decode_megakernel_gb300 import mbk
    s = Setup([100, 90], [1, 1], 4, 2, 64, track=True)
    before = s.bytes().copy()
    rows = torch.tensor([10 ** 6, 90], dtype=torch.int32, device="cuda")
    got = s.cache.evict(rows, s.dev["tables"], rows, 32, layer=s.layer, max_rows=128)
    assert got.tolist() == [10 ** 6, 32] and s.cache.status() == mbk.MBK_KV4_BAD_BATCH
    for page in s.tables[0][:4]:
        assert (s.bytes()[page] == before[page]).all()


def test_tensors_refused():
    s = Setup([40], [1], 4, 2, 64)
    q = s.q(torch.float32).cuda()
    wide = torch.zeros(2, 4, 130, device="cuda")
    for bad in (q.cpu(), q.half(), q[0], q.expand(2, 4, 64), wide[:1, :, 1:65], wide[:1, :, :64], q.transpose(0, 1)):
        with pytest.raises(ValueError):
            s.cache.attention(s.layer, s.batch, bad)
    with pytest.raises(ValueError):
        s.cache.attention(s.layer, s.batch, q, out=torch.empty(1, 4, 64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        s.cache.attention(s.layer, s.batch, q, slopes=torch.zeros(3, device="cuda"))
    from persistent_decode_megakernel_gb300 import mbk
    for kw in (dict(out=q), dict(accumulate=True), dict(window=-1), dict(cap=-1.0), dict(scale=float("nan"))):
        with pytest.raises(mbk.MbkError):
            s.cache.attention(s.layer, s.batch, q, **kw)
    for layer in (-1, 2):
        with pytest.raises(mbk.MbkError):
            s.cache.attention(layer, s.batch, q)
    k = torch.zeros(1, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        s.cache.append(0, s.batch, k, k.bfloat16())
    with pytest.raises(ValueError):
        s.cache.batch(s.dev["offsets"].long(), s.dev["rows"], s.dev["tables"])
    with pytest.raises(ValueError):
        s.cache.batch(s.dev["offsets"], s.dev["rows"], s.dev["tables"][:, :1])


def test_a_batch_of_another_cache_is_refused():
    a, b = Setup([40], [1], 4, 2, 64), Setup([400], [1], 4, 2, 64)
    q, k = torch.zeros(1, 4, 64, device="cuda"), torch.zeros(1, 2, 64, device="cuda")
    for call in (lambda: b.cache.attention(0, a.batch, q), lambda: b.cache.append(0, a.batch, k, k), lambda: b.cache.read(0, a.batch)):
        with pytest.raises(ValueError):
            call()


PROMPTS = [((4, 2, 64), torch.float32), ((4, 2, 128), torch.bfloat16), ((4, 2, 128), torch.float32)]


@pytest.mark.parametrize("window", [0, 10])
@pytest.mark.parametrize("heads,dtype", PROMPTS, ids=str)
def test_nan_rows_under_a_prompt(heads, dtype, window):
    """The last group of V is NaN in row 70, K in row 93: each query's dims are NaN exactly where it sees them."""
    s = Setup([100], [60], *heads)
    for row, k_bad in ((70, False), (93, True)):
        for h in range(s.kv):
            k, v = (x.astype(np.float32) for x in s.pool.get(s.layer, s.tables[0], row, h))
            (k if k_bad else v)[-64:] = np.nan
            s.pool.put(s.layer, s.tables[0], row, h, k, v)
    s.cache.pool.copy_(torch.from_numpy(s.pool.bytes.reshape(-1)))
    q = s.q(dtype)
    want, _ = s.expect(q, window=window)
    got = s.cache.attention(s.layer, s.batch, q.cuda(), window=window).double().cpu().numpy()
    assert (np.isnan(got) == np.isnan(want)).all()
    good = Setup([70], [30], *heads)  # the tolerance of the rows before them, whose values are of the same size
    check(torch.from_numpy(np.nan_to_num(got)), np.nan_to_num(want), good.tolerance(q, dtype), "others")


@pytest.mark.parametrize("window", [0, 30, 2 ** 31 - 1])
@pytest.mark.parametrize("counts", [[60, 40, 50], [10, 1, 2]], ids=["prompts", "few"])
@pytest.mark.parametrize("heads,dtype", PROMPTS, ids=str)
def test_more_new_tokens_than_rows(heads, dtype, counts, window):
    """The first tokens see no row: zero; a sequence without rows and one that sees all; the largest window."""
    s = Setup([counts[0] // 3, 0, 70], counts, *heads)
    q = s.q(dtype)
    want, _ = s.expect(q, window=window)
    assert (want[:counts[0] - counts[0] // 3] == 0).all() and (want[counts[0]:counts[0] + counts[1]] == 0).all()
    check(_run(s, q, dict(window=window)), want, s.tolerance(q, dtype), "out")


@pytest.mark.parametrize("heads,dtype", PROMPTS, ids=str)
def test_prompts_inside_wider_rows(heads, dtype):
    s = Setup([90, 40], [60, 33], *heads)
    n, nq, d = s.offsets[-1], s.heads, s.d
    wide = torch.randn(n, nq + 3, d, device="cuda").to(dtype)
    out = torch.full((n, nq + 2, d), 7.0, device="cuda", dtype=dtype)
    s.cache.attention(s.layer, s.batch, wide[:, 1:1 + nq], out=out[:, 2:])
    assert (out[:, :2] == 7).all()
    assert torch.equal(out[:, 2:], s.cache.attention(s.layer, s.batch, wide[:, 1:1 + nq].contiguous()))


@pytest.mark.parametrize("count", [1, 50])
@pytest.mark.parametrize("heads,dtype", PROMPTS, ids=str)
def test_values_at_the_end_of_fp16(heads, dtype, count):
    """K and V up to +-65504 (a scale that is rounded up may lead lo + 15 scale beyond it)."""
    s = Setup([80], [count], *heads, fill=False)
    for i in range(80):
        for h in range(s.kv):
            k, v = s.rng.uniform(-65504, 65504, size=(2, s.d)).astype(np.float32)
            k[0], k[1], v[0], v[1] = 65504, -65504, 65504, -65504
            s.pool.put(s.layer, s.tables[0], i, h, k, v)
    s.cache.pool.copy_(torch.from_numpy(s.pool.bytes.reshape(-1)))
    q, scale = s.q(dtype), 1e-6
    want, _ = plain.attention(s.pool, s.layer, q.double().numpy(), s.offsets, s.rows, s.tables, None, s.heads, scale)
    size = float(q.double().norm(dim=-1).max()) * 65504 * s.d ** 0.5 * scale
    tol = size * (2.0 ** -22 + s.d ** 0.5 * 2.0 ** -23) + 2.0 ** -19
    if dtype == torch.bfloat16:  # prompts: K and V are rounded to fp16 too, off by 2^-11 of themselves (independent from row to row)
        tol += 2.0 ** -8 + 2 * 2.0 ** -11 + size * 2.0 ** -11
    check(s.cache.attention(s.layer, s.batch, q.cuda(), scale=scale), want, tol, str(count))


def test_evict_when_everything_is_recent():
    """next_pos - recent below the least int: every row counts as recent, and the lowest rows are kept."""
    s = Setup([100], [1], 4, 2, 64, track=True)
    nxt = torch.tensor([-2 ** 31 + 3], dtype=torch.int32, device="cuda")
    before = s.bytes().copy()
    assert s.cache.evict(s.dev["rows"], s.dev["tables"], nxt, 50, 20, layer=s.layer).tolist() == [50]
    assert (s.bytes() == before).all()


def _random_cache(heads, kv, d, seqs, rows, counts, dtype, layers=1):
    """A cache of normal rows (pages in order), a batch of the last `counts` tokens of each sequence, and queries."""
    from persistent_decode_megakernel_gb300.kv4 import Kv4Cache
    per = -(-rows // 64)
    cache = Kv4Cache(layers, heads, kv, d, seqs * per, 64, per)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tables, held = dev(list(range(seqs * per))).view(seqs, per), dev([rows] * seqs)
    g = torch.Generator(device="cuda").manual_seed(5)
    every = cache.batch(dev([i * rows for i in range(seqs + 1)]), held, tables, n_tokens=seqs * rows, max_count=rows)
    k, v = (torch.randn(seqs * rows, kv, d, device="cuda", generator=g) for _ in range(2))
    cache.append(0, every, k, v)
    n = sum(counts)
    off = dev([0] + np.cumsum(counts).tolist())
    batch = cache.batch(off, held, tables, n_tokens=n, max_count=max(counts), max_rows=rows)
    q = torch.randn(n, heads, d, device="cuda", generator=g).to(dtype)
    return cache, every, batch, q


@pytest.mark.parametrize("counts", [[30] * 16, [32] * 15 + [50], [64, 33] * 8], ids=["half", "mixed", "uneven"])
@pytest.mark.parametrize("heads,dtype", [((32, 8, 64), torch.bfloat16), ((32, 8, 128), torch.bfloat16), ((32, 8, 64), torch.float32)], ids=str)
def test_query_tiles_that_run_ahead_of_each_other(heads, dtype, counts):
    """Prompts whose second query tile is empty or short get through its keys much faster than the first: many calls
    end without a wait that gives up, and all give the same."""
    nq, kv, d = heads
    rows = 4096
    cache, every, batch, q = _random_cache(nq, kv, d, len(counts), rows, counts, dtype)
    first = cache.attention(0, batch, q)
    assert cache.status() == 0
    for _ in range(60):
        out = cache.attention(0, batch, q)
    assert cache.status() == 0 and torch.equal(out, first)
    k, v = (x.view(len(counts), rows, kv, d).double() for x in cache.read(0, every))
    at = 0
    for s, c in list(enumerate(counts))[::5]:
        at = sum(counts[:s])
        x = torch.einsum("qhgd,khd->hgqk", q[at:at + c].double().view(c, kv, nq // kv, d), k[s]) * d ** -0.5
        x = x.masked_fill(torch.ones(c, rows, dtype=torch.bool, device="cuda").triu(rows - c + 1), -np.inf).softmax(-1)
        want = torch.einsum("hgqk,khd->qhgd", x, v[s]).reshape(c, nq, d)
        # scores below 8 in size: weights off by 8 (2^-22 + 11 2^-23); bf16: out 2^-8, weights and V 2^-11 each, K 2^-11 of a score's terms
        tol = 2.0 ** -16 if dtype == torch.float32 else 2.0 ** -8 + 3 * 2.0 ** -11
        assert (first[at:at + c].double() - want).norm() <= tol * want.norm()


@pytest.mark.parametrize("size", [0.3, 1.0, 2.0])
@pytest.mark.parametrize("count", [1, 1024], ids=["decode", "prompt"])
def test_fp32_is_as_exact_as_fp32_arithmetic(count, size):
    """Over 30,000 rows, whose average is small against them: at most twice as far off as the same formula in fp32."""
    nq, kv, d, rows = 6, 2, 64, 30000
    cache, every, batch, q = _random_cache(nq, kv, d, 1, rows, [count], torch.float32)
    q *= size
    got = cache.attention(0, batch, q).double()
    k, v = cache.read(0, every)
    sums = [0.0, 0.0, 0.0]
    for h in range(nq):
        out = []
        for t in (torch.float64, torch.float32):
            x = (q[:, h].to(t) @ k[:, h * kv // nq].to(t).T) * d ** -0.5
            x = x.masked_fill(torch.ones(count, rows, dtype=torch.bool, device="cuda").triu(rows - count + 1), -np.inf)
            out.append((x.softmax(-1) @ v[:, h * kv // nq].to(t)).double())
        for i, x in enumerate((got[:, h] - out[0], out[1] - out[0], out[0])):
            sums[i] += float(x.square().sum())
    assert sums[0] ** 0.5 <= 2 * sums[1] ** 0.5, [(x / sums[2]) ** 0.5 for x in sums]
