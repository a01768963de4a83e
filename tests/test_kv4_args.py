"""Refusals of the 4-bit KV cache's entry points, and the plain form's own pins: no GPU needed, as the host checks
run before any CUDA call that could fail."""
import ctypes

import numpy as np
import pytest

import kv4_plain as plain
from persistent_decode_megakernel_gb300 import build as mbk_build
from persistent_decode_megakernel_gb300 import mbk


@pytest.fixture(scope="module")
def lib():
    mbk_build.build()
    return mbk.load_library()


GOOD = dict(device=0, n_layers=2, n_heads=8, n_kv_heads=2, head_dim=64, num_pages=10, page_size=64, max_pages=4, track=1)
P = 0x10000000  # an address that is never read: every call here is refused on the host


def config(**kw):
    return mbk.MbkKv4Config(*[dict(GOOD, **kw)[k] for k, _ in mbk.MbkKv4Config._fields_])


def batch(**kw):
    b = dict(n_seq=2, n_tokens=3, max_count=2, max_rows=256, offsets=P, rows=P, positions=None, tables=P, status=None)
    b.update(kw)
    return mbk.MbkKv4Batch(*[b[k] for k, _ in mbk.MbkKv4Batch._fields_])


def test_pool_bytes(lib):
    size = lambda **kw: lib.mbk_kv4_pool_bytes(ctypes.byref(config(**kw)))  # noqa: E731
    for d, track, row in ((64, 0, 72), (64, 1, 80), (128, 0, 144), (128, 1, 152)):
        assert size(head_dim=d, track=track) == 10 * 2 * 2 * 64 * row
        pool = plain.PlainPool(2, 2, d, 10, 64, track)
        assert pool.bytes.size == size(head_dim=d, track=track)
    # a pool of more than 2^32 bytes
    assert size(num_pages=1 << 20, n_layers=32, n_kv_heads=8) == (1 << 20) * 32 * 8 * 64 * 80


@pytest.mark.parametrize("bad", [dict(device=-1), dict(n_layers=0), dict(n_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=3), dict(n_heads=34),
                                 dict(head_dim=32), dict(head_dim=96), dict(num_pages=0), dict(page_size=16), dict(page_size=48),
                                 dict(max_pages=0), dict(max_pages=1 << 30), dict(track=2), dict(n_heads=-8, n_kv_heads=-2)], ids=str)
def test_configurations_refused(lib, bad):
    c = config(**bad)
    assert lib.mbk_kv4_pool_bytes(ctypes.byref(c)) == mbk.MBK_ERR_INVALID_ARG
    b = batch()
    assert lib.mbk_kv4_append(ctypes.byref(c), P, 0, ctypes.byref(b), P, P, 128, 0, None) == mbk.MBK_ERR_INVALID_ARG
    assert lib.mbk_kv4_evict_workspace(ctypes.byref(c), 1, 1, 1) == mbk.MBK_ERR_INVALID_ARG


def _append(lib, c=None, pool=P, layer=0, b=None, k=P, v=P, ld=128, dtype=0, fn="mbk_kv4_append"):
    c, b = c or config(), b or batch()
    return getattr(lib, fn)(ctypes.byref(c), pool, layer, ctypes.byref(b), k, v, ld, dtype, None)


def _attention(lib, c=None, pool=P, layer=0, b=None, q=P, ldq=512, out=P, ldo=512, dtype=0, scale=1.0, cap=0.0, slopes=None, window=0,
               accumulate=0, ws=P, size=1 << 40, same=False):
    c, b = c or config(), b or batch()
    out = out + 0x1000000 if out == q and not same else out
    return lib.mbk_kv4_attention(ctypes.byref(c), pool, layer, ctypes.byref(b), q, ldq, out, ldo, dtype, scale, cap, slopes, window, accumulate,
                                 ws, size, None)


BATCHES = [dict(n_seq=0), dict(n_seq=1025), dict(n_tokens=0), dict(max_count=0), dict(max_count=4), dict(max_rows=-1), dict(max_rows=257),
           dict(offsets=None), dict(rows=None), dict(tables=None), dict(offsets=P + 2), dict(status=P + 1), dict(positions=P + 3)]


@pytest.mark.parametrize("bad", BATCHES, ids=str)
def test_batches_refused(lib, bad):
    for fn in ("mbk_kv4_append", "mbk_kv4_read"):
        assert _append(lib, b=batch(**bad), fn=fn) == mbk.MBK_ERR_INVALID_ARG
    assert _attention(lib, b=batch(**bad)) == mbk.MBK_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(pool=None), dict(pool=P + 8), dict(layer=-1), dict(layer=2), dict(k=None), dict(v=None), dict(k=P + 4),
                                 dict(v=P + 8), dict(ld=127), dict(ld=130), dict(ld=132, dtype=1), dict(dtype=2), dict(dtype=-1)], ids=str)
def test_rows_refused(lib, bad):
    for fn in ("mbk_kv4_append", "mbk_kv4_read"):
        assert _append(lib, fn=fn, **bad) == mbk.MBK_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(pool=None), dict(layer=2), dict(q=None), dict(out=None), dict(q=P + 4), dict(ldq=508), dict(ldo=514),
                                 dict(dtype=3), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("nan")),
                                 dict(cap=float("inf")), dict(slopes=P + 1), dict(window=-1), dict(accumulate=2),
                                 dict(accumulate=1, c=config(track=0)), dict(same=True),
                                 dict(b=batch(n_seq=1024, n_tokens=1 << 30, max_count=1 << 30))], ids=lambda b: "-".join(b))
def test_attention_refused(lib, bad):
    assert _attention(lib, **bad) == mbk.MBK_ERR_INVALID_ARG


def _evict(lib, c=None, pool=P, layer=0, n_layers=2, n_seq=2, max_rows=256, rows=P, tables=P, nxt=P, keep=64, recent=8, out=None, pages=0,
           rows_out=P, status=None, ws=P, size=1 << 40):
    c = c or config()
    return lib.mbk_kv4_evict(ctypes.byref(c), pool, layer, n_layers, n_seq, max_rows, rows, tables, nxt, keep, recent, out, pages, rows_out,
                             status, ws, size, None)


@pytest.mark.parametrize("bad", [dict(c=config(track=0)), dict(pool=None), dict(layer=2), dict(layer=1), dict(n_layers=0), dict(n_seq=0),
                                 dict(n_seq=1025), dict(max_rows=0), dict(max_rows=257), dict(rows=None), dict(tables=None), dict(nxt=None),
                                 dict(keep=0), dict(keep=257), dict(recent=-1), dict(recent=65), dict(out=P), dict(out=P, pages=0),
                                 dict(out=P + 2, pages=4), dict(rows_out=None), dict(rows_out=P + 1), dict(ws=None), dict(ws=P + 8),
                                 dict(size=16)], ids=lambda b: "-".join(f"{k}={v}" if k != "c" else k for k, v in b.items()))
def test_evict_refused(lib, bad):
    assert _evict(lib, **bad) == mbk.MBK_ERR_INVALID_ARG


def test_plain_format_pins():
    """The plain form against values worked out by hand."""
    x = np.zeros(64, np.float32)
    x[:4] = (-3.0, 12.0, 0.5, -0.5)     # lo -3, scale 1: codes 0, 15, 3.5 -> 4 (even), 2.5 -> 2
    code, scale, lo = plain.quantize(x)
    assert scale.tolist() == [1.0] and lo.tolist() == [-3.0]
    assert code[:5].tolist() == [0, 15, 4, 2, 3]
    assert plain.values(code, scale, lo)[:5].tolist() == [-3.0, 12.0, 1.0, -1.0, 0.0]
    code, scale, lo = plain.quantize(np.full(64, 2.5, np.float32))
    assert not code.any() and scale[0] == 0 and lo[0] == 2.5
    _, scale, lo = plain.quantize(np.array([np.inf, -np.inf] + [0.0] * 62, np.float32))
    assert lo[0] == -65504 and scale[0] == np.float16(131008 / 15)
    assert plain.evict_map([5.0, 1.0, 3.0, 3.0, 0.0, 9.0], [0, 1, 2, 3, 4, 5], 3, 4) == [0, 4, 5]
    assert plain.evict_map([5.0, 1.0, 3.0, 3.0, 0.0], [0, 1, 2, 3, 9], 3, 9) == [0, 4, 2]


def test_positions_need_a_tracked_pool(lib):
    assert _append(lib, c=config(track=0), b=batch(positions=P)) == mbk.MBK_ERR_INVALID_ARG
    assert _attention(lib, c=config(track=0), b=batch(positions=P)) == mbk.MBK_ERR_INVALID_ARG


def test_4_bit_handles_are_refused_before_any_device_is_touched(lib):
    from persistent_decode_megakernel_gb300 import workloads
    h = ctypes.c_void_p()
    cfg, w = mbk.config_from_shape(workloads.SHAPES["tiny"]), mbk.MbkWeights()
    fp8 = mbk.config_from_shape(workloads.SHAPES["tiny"], mbk.MBK_WEIGHTS_FP8)
    make = lambda c, pages, size, track: lib.mbk_create_kv4(ctypes.byref(c), ctypes.byref(w), P, pages, size, track, 0, ctypes.byref(h))  # noqa: E731
    for c, pages, size, track in ((fp8, 4, 32, 0), (cfg, 0, 32, 0), (cfg, 4, 48, 0), (cfg, 4, 16, 0), (cfg, 4, 256, 0), (cfg, 4, 32, 2)):
        assert make(c, pages, size, track) == mbk.MBK_ERR_INVALID_ARG and not h.value
    assert lib.mbk_create_kv4(ctypes.byref(cfg), ctypes.byref(w), P, 4, 32, 0, 0, None) == mbk.MBK_ERR_INVALID_ARG
    one = (ctypes.c_int32 * 1)(1)
    assert lib.mbk_batch_step_kv4(None, 1, one, one, one, one, one, None, 0, None) == mbk.MBK_ERR_INVALID_ARG
