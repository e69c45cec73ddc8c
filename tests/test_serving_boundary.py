"""Host-side checks of the chunk, copy and rotary calls: no GPU is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def kvq():
    import bit_asymmetric_kv_kvq_gb300 as kvq
    from bit_asymmetric_kv_kvq_gb300 import _build
    try:
        _build.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    return kvq


def test_null_handles(kvq):
    L = kvq.lib()
    n = ctypes.c_int64()
    assert L.kvq_append_chunk(None, 256, 256, 1, 1, None) == -1
    assert L.kvq_chunk_attention(None, 256, 256, 256, 1, 256, 256, 1 << 30, None) == -1
    assert L.kvq_chunk_step(None, 256, 256, 256, 1, 256, 256, 1 << 30, None) == -1
    assert L.kvq_chunk_workspace(None, 1, ctypes.byref(n)) == -1
    assert L.kvq_copy_sequences(None, None, 256, None) == -1
    assert L.kvq_buffers(None, ctypes.byref(kvq.kvq.kvq_device_view())) == -1


def _rope(kvq, parts=1, x_type=0, out_type=0, batch=1, n=1, positions=None, part=None, **over):
    cfg = kvq.make_rope_config(128, original_context=4096)
    for k, v in over.items():
        setattr(cfg, k, v)
    p = kvq.kvq.kvq_rope_part(256, 256, 128, 128, 128, 128, 128, 128, 1, 1)
    for k, v in (part or {}).items():
        setattr(p, k, v)
    arr = (kvq.kvq.kvq_rope_part * max(parts, 1))(*[p] * max(parts, 1))
    return kvq.lib().kvq_rope(ctypes.byref(cfg), arr, parts, x_type, out_type, batch, n, positions, 0, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(head_dim=0), -1), (dict(head_dim=127), -1), (dict(rot_dim=0), -1), (dict(rot_dim=5), -1),
    (dict(rot_dim=130), -1), (dict(interleaved=2), -1), (dict(base=1.0), -1), (dict(base=float("inf")), -1),
    (dict(base=float("nan")), -1), (dict(scaling=-1), -1), (dict(scaling=4), -1), (dict(scaling=1, factor=0.0), -1),
    (dict(scaling=2, original_context=0), -1), (dict(scaling=2, low=4.0, high=4.0), -1),
    (dict(scaling=3, low=0.0), -1), (dict(attention_factor=0.0), -1), (dict(attention_factor=float("nan")), -1),
    (dict(x_type=3), -1), (dict(out_type=-1), -1), (dict(parts=0), -1), (dict(parts=5), -2), (dict(batch=0), -1),
    (dict(n=0), -1), (dict(n=1 << 41), -2), (dict(positions=260), -1), (dict(part=dict(x=None)), -1),
    (dict(part=dict(out=None)), -1), (dict(part=dict(num_heads=0)), -1), (dict(part=dict(rotate=2)), -1),
    (dict(part=dict(x=257)), -1), (dict(x_type=2, part=dict(x=258)), -1), (dict(part=dict(num_heads=70000)), -2),
    (dict(head_dim=258, rot_dim=2), -2),
])
def test_rope_checks_arguments_on_the_host(kvq, kw, expect):
    assert _rope(kvq, **kw) == expect


@pytest.mark.parametrize("kw", [dict(x_type=1), dict(out_type=2), dict(batch=2, part=dict(out_batch_stride=256)),
                                dict(n=2, part=dict(out_token_stride=256)),
                                dict(part=dict(num_heads=2, out_head_stride=256))])
def test_rope_in_place_needs_the_same_layout(kvq, kw):
    assert _rope(kvq, **kw) == -1


def test_rope_nulls(kvq):
    L = kvq.lib()
    cfg = kvq.make_rope_config(128)
    p = kvq.kvq.kvq_rope_part(256, 256, 128, 128, 128, 128, 128, 128, 1, 1)
    assert L.kvq_rope(None, ctypes.byref(p), 1, 0, 0, 1, 1, None, 0, None) == -1
    assert L.kvq_rope(ctypes.byref(cfg), None, 1, 0, 0, 1, 1, None, 0, None) == -1


def test_rope_config_defaults(kvq):
    c = kvq.make_rope_config(128, scaling="yarn", factor=16.0, original_context=4096)
    assert (c.rot_dim, c.low, c.high) == (128, 1.0, 32.0) and abs(c.attention_factor - 1.2772588722) < 1e-9
    c = kvq.make_rope_config(128, 64, scaling="wavelength", factor=8.0, original_context=8192)
    assert (c.rot_dim, c.low, c.high, c.attention_factor) == (64, 1.0, 4.0, 1.0)
