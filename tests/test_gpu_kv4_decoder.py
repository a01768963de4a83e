"""A decoder on a 4-bit pool (mbk_create_kv4): prompts, batches and steps after an eviction, each against a plain
decoder in 64 bits that starts from the pool's bytes before the step.

Tolerance.  The step's own K and V rows are quantised on both sides from values that differ by the projections'
rounding (bf16 pairs: 2^-16 of a value); where that crosses the middle between two codes a row's element moves by one
step of its group, about a fifteenth of six standard deviations.  That is about 2^-16 * 3 / 0.4 of the elements (1e-4), or
a row's relative error of 0.4 sqrt(1e-4) = 4e-3 at most, in the new rows only; the logits stay within 1e-2 (2-norm).
"""
import numpy as np
import pytest
import torch

import kv4_plain as plain
from persistent_decode_megakernel_gb300 import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_decode_megakernel_gb300 import build
    build.build()


def _f64(t):
    return t.to(torch.float32).numpy().astype(np.float64)


def plain_step(wl, pool, tokens, start, held, table):
    """Logits [n, vocab] of tokens at positions start .. that become rows held .. of the sequence; `pool` gets the rows."""
    s = wl.shape
    d, g, half = s.head_dim, s.group, s.head_dim // 2
    norm = lambda x, w: x / np.sqrt((x * x).mean(-1, keepdims=True) + s.rms_eps) * _f64(w)  # noqa: E731
    x = _f64(wl.embed)[tokens]
    n = len(tokens)
    ang = (start + np.arange(n))[:, None, None] * s.rope_theta ** (-2.0 * np.arange(half) / d)
    rot = lambda v: np.concatenate([v[..., :half] * np.cos(ang) - v[..., half:] * np.sin(ang),  # noqa: E731
                                    v[..., half:] * np.cos(ang) + v[..., :half] * np.sin(ang)], -1)
    for layer, w in enumerate(wl.layers):
        h = norm(x, w["attn_norm"])
        proj = lambda m, b, k: (h @ _f64(w[m]).T + (_f64(w[b]) if s.qkv_bias else 0.0)).reshape(n, k, d)  # noqa: E731
        q, k, v = rot(proj("wq", "bq", s.n_heads)), rot(proj("wk", "bk", s.n_kv_heads)), proj("wv", "bv", s.n_kv_heads)
        for i in range(n):
            for j in range(s.n_kv_heads):
                pool.put(layer, table, held + i, j, k[i, j].astype(np.float32), v[i, j].astype(np.float32), start + i, 0.0)
        out, _ = plain.attention(pool, layer, q, [0, n], [held + n], [table], [start], s.n_heads, d ** -0.5)
        x = x + out.reshape(n, -1) @ _f64(w["wo"]).T
        h = norm(x, w["mlp_norm"])
        a = h @ _f64(w["w_gate"]).T
        x = x + (a / (1 + np.exp(-a)) * (h @ _f64(w["w_up"]).T)) @ _f64(w["w_down"]).T
    return norm(x, wl.final_norm) @ _f64(wl.embed).T


class Pool:
    """The plain pool, refreshed from a decoder's bytes."""

    def __init__(self, dec, track):
        c = dec.cache.cfg
        self.dec, self.plain = dec, plain.PlainPool(c.n_layers, c.n_kv_heads, c.head_dim, c.num_pages, c.page_size, track)

    def now(self):
        self.plain.bytes = self.dec.cache.pool.cpu().numpy().reshape(self.plain.bytes.shape).copy()
        return self.plain


def _close(got, want):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.linalg.norm(got - want, axis=-1) / np.linalg.norm(want, axis=-1)
    assert off.max() <= 1e-2, off


SHAPES = {
    "tiny": "tiny",
    "bias, 7 heads a group": workloads.DecoderShape("kv4-qwen", 2, 448, 512, 14, 2, 64, 1024, 256, 1e-6, 1e6, True, steps=8),
    "head dim 128": workloads.DecoderShape("kv4-128", 2, 512, 512, 8, 4, 128, 1024, 256, 1e-5, 1e4, False, steps=8),
}


def _decoder(shape, track, page=32, spare=0, n_seq=1):
    from persistent_decode_megakernel_gb300.mbk import Decoder
    wl = workloads.generate(SHAPES[shape], seed=2)
    per = -(-wl.shape.kv_capacity // page)
    tables = np.random.default_rng(5).permutation(per * n_seq + spare)[:per * n_seq].reshape(n_seq, per)
    dec = Decoder(wl, paged=(per * n_seq + spare, page, tables[0].tolist()), kv4=True, track=track)
    return wl, dec, tables


@pytest.mark.parametrize("track", [False, True], ids=["untracked", "tracked"])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_prefill_and_next_chunk(shape, track):
    wl, dec, tables = _decoder(shape, track, spare=3)
    pool = Pool(dec, track)
    toks = np.random.default_rng(0).integers(0, wl.shape.vocab, 60)
    for a, b in ((0, 37), (37, 38), (38, 60)):
        want = plain_step(wl, pool.now(), toks[a:b], a, a, tables[0])
        _close(dec.prefill(toks[a:b].tolist(), a, logits="all"), want)
    assert dec.status() == 0
    dec.close()


@pytest.mark.parametrize("shape", ["tiny", "head dim 128"])
def test_batches_with_eviction_between(shape):
    """Prompts of three sequences in one step, decode steps, an eviction, and steps on what is left."""
    keep, recent = 24, 4
    wl, dec, tables = _decoder(shape, True, n_seq=3)
    pool, rng, V = Pool(dec, True), np.random.default_rng(1), wl.shape.vocab
    pos, rows = [0, 0, 0], [0, 0, 0]
    dev = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")  # noqa: E731
    for step in range(7):
        counts = [33, 5, 20] if step == 0 else [1, 1, 1] if step != 4 else [1, 9, 3]
        toks = [rng.integers(0, V, c).tolist() for c in counts]
        plain_pool = pool.now()
        want = np.concatenate([plain_step(wl, plain_pool, t, p, r, tab) for t, p, r, tab in zip(toks, pos, rows, tables)])
        got = dec.batch_step(list(zip(pos, toks)), tables, logits="all", held=rows)
        _close(got, want)
        pos, rows = [p + c for p, c in zip(pos, counts)], [r + c for r, c in zip(rows, counts)]
        # every row has got the weights of the queries that saw it: they add up to the queries, per head of the group
        total = sum(pool.now().weight(0, tables[0], i, 0) for i in range(rows[0]))
        if step == 0:
            assert abs(total - counts[0] * wl.shape.group) <= 1e-3 * total
        if step in (1, 4):
            rows = dec.cache.evict(dev(rows), dev(tables), dev(pos), keep, recent).tolist()
            assert rows == [min(keep, r) for r in rows] and rows[0] == keep
    assert dec.status() == 0 and dec.cache.status() == 0
    dec.close()


def test_what_a_4_bit_handle_refuses():
    from persistent_decode_megakernel_gb300 import mbk
    wl, dec, tables = _decoder("tiny", False)
    stream, out = torch.cuda.current_stream().cuda_stream, torch.empty(8 * wl.shape.vocab, device="cuda")
    p = out.data_ptr()
    assert mbk.mbk_decode_step(dec.handle, 1, 0, p, stream) == mbk.MBK_ERR_UNSUPPORTED
    assert mbk.mbk_decode_steps(dec.handle, [1, 2], 0, p, stream) == mbk.MBK_ERR_UNSUPPORTED
    assert mbk.mbk_decode_greedy(dec.handle, 1, 2, 0, p, 0, stream) == mbk.MBK_ERR_UNSUPPORTED
    assert mbk.mbk_kv_fill(dec.handle, 0, p, p, 0, 1, stream) == mbk.MBK_ERR_UNSUPPORTED
    t = tables.tolist()
    assert mbk.mbk_batch_step_kv4(dec.handle, [1], [5], [3], [1], t, p, 1, stream) == mbk.MBK_ERR_INVALID_ARG  # not tracked
    dec.close()
    wl, dec, tables = _decoder("tiny", True)
    t = tables.tolist()
    for held in (-1, 6):
        assert mbk.mbk_batch_step_kv4(dec.handle, [1], [5], [held], [1], t, p, 1, stream) == mbk.MBK_ERR_INVALID_ARG
    assert mbk.mbk_batch_step_kv4(dec.handle, [1], [5], [3], [wl.shape.vocab], t, p, 1, stream) == mbk.MBK_ERR_INVALID_ARG
    dec.close()
    plain_dec = mbk.Decoder(wl, paged=(4, 32, [0, 1, 2, 3]))
    assert mbk.mbk_batch_step_kv4(plain_dec.handle, [1], [5], [3], [1], [[0, 1, 2, 3]], p, 1, stream) == mbk.MBK_ERR_INVALID_ARG
    plain_dec.close()
    for kw in (dict(fp8=True), dict(paged=(4, 48, [0]))):
        with pytest.raises(mbk.MbkError) as e:
            mbk.Decoder(wl, **dict(dict(paged=(4, 32, [0]), kv4=True), **kw))
        assert e.value.code == mbk.MBK_ERR_INVALID_ARG
