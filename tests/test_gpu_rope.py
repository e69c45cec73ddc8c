"""Rotary positions of new queries and keys against fp64.

The bound per element with pair (x_a, x_b): half a step of the output type (2^-11, 2^-8 or 2^-24 of the value; fp16's
smallest step 2^-25 near zero) for the one rounding, plus the fp32 arithmetic before it: cosine and sine are off by at
most 2 ulp (2^-23 below 1, 2^-22 together with the angle's 2^-26 of a turn = 2^-23.3 rad), products and sum by 2^-23 of
their size: 2^-21 m (|x_a| + |x_b|) covers them.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _kvq():
    import bit_asymmetric_kv_kvq_gb300 as kvq
    return kvq


def _freq(rot, base, scaling, factor, context):
    i = np.arange(rot // 2, dtype=np.float64)
    w = base ** (-2.0 * i / rot)
    gain = 1.0
    if scaling == "linear":
        w = w / factor
    elif scaling == "wavelength":
        turns = context * w / (2 * math.pi)
        keep = np.clip((turns - 1.0) / 3.0, 0, 1)
        w = w / factor * (1 - keep) + w * keep
    elif scaling == "yarn":
        index = [rot * math.log(context / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(index[0]), 0), min(math.ceil(index[1]), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        w = w / factor * ramp + w * (1 - ramp)
        gain = 0.1 * math.log(factor) + 1.0
    return w, gain


def _check(x, out, pos, rot, interleaved, w, gain, turned):
    """x [B, n, H, D] and out [B, H, n, D] as stored, pos [B, n] python ints as fp64-exact integers."""
    xd = x.double().cpu().numpy()
    got = out.double().cpu().numpy().transpose(0, 2, 1, 3)
    want, slack = xd.copy(), np.zeros_like(xd)
    if turned:
        # whole turns go before the product loses them: pos = hi * 2^20 + lo
        hi, lo = pos // (1 << 20), pos % (1 << 20)
        turn = np.mod(np.mod(w / (2 * math.pi) * (1 << 20), 1.0) * hi[..., None] + w / (2 * math.pi) * lo[..., None], 1.0)
        c, s = np.cos(2 * math.pi * turn) * gain, np.sin(2 * math.pi * turn) * gain
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        xa, xb = xd[..., a], xd[..., b]
        c, s = c[:, :, None], s[:, :, None]
        want[..., a], want[..., b] = xa * c - xb * s, xa * s + xb * c
        slack[..., a] = slack[..., b] = gain * (np.abs(xa) + np.abs(xb))
    tiny = 2.0 ** -25 if out.dtype == torch.float16 else 0.0
    bound = HALF_STEP[out.dtype] * np.abs(want) * 1.001 + tiny + 2.0 ** -21 * slack
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) - bound).max())


def _positions(B, n, positions):
    if isinstance(positions, int):
        return np.broadcast_to(positions + np.arange(n, dtype=np.int64), (B, n))
    return positions.cpu().numpy()


@pytest.mark.parametrize("x_type", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out_type", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,n,heads", [(1, 1, (4, 4, 4)), (3, 37, (8, 2, 2)), (2, 700, (5, 1))])
def test_types_and_sizes(x_type, out_type, B, n, heads):
    """Views of one projection, queries and keys turned, values moved along."""
    kvq = _kvq()
    D = 128
    qkv = torch.randn(B, n, sum(heads) * D, device="cuda").to(x_type)
    parts = list(qkv.view(B, n, sum(heads), D).split(list(heads), dim=2))
    rotate = [True, True, False][:len(parts)]
    cfg = kvq.make_rope_config(D)
    outs = kvq.rope(cfg, parts, 123, rotate=rotate, out_dtype=out_type)
    w, gain = _freq(D, 10000.0, "none", 1.0, 0)
    for x, o, r in zip(parts, outs, rotate):
        assert o.dtype == out_type and o.is_contiguous()
        _check(x, o, _positions(B, n, 123), D, False, w, gain, r)


@pytest.mark.parametrize("scaling,factor,base,context", [("none", 1.0, 500000.0, 0), ("linear", 4.0, 10000.0, 0),
                                                         ("wavelength", 8.0, 500000.0, 8192), ("yarn", 16.0, 10000.0, 4096)])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 96), (64, 32), (256, 256), (80, 20), (10, 6), (128, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts_and_scalings(scaling, factor, base, context, D, rot, interleaved):
    kvq = _kvq()
    B, n = 2, 19
    x = torch.randn(B, n, 3, D, device="cuda").half()
    pos = torch.randint(0, 1 << 20, (B, n), device="cuda", dtype=torch.int64)
    cfg = kvq.make_rope_config(D, rot, base, interleaved, scaling, factor, original_context=context)
    (out,) = kvq.rope(cfg, [x], pos)
    w, gain = _freq(rot, base, scaling, factor, context)
    _check(x, out, _positions(B, n, pos), rot, interleaved, w, gain, True)


def test_far_and_negative_positions():
    """Positions beyond 2^31 and below zero; a turn forth and back is the identity within the roundings."""
    kvq = _kvq()
    x = torch.randn(1, 5, 2, 128, device="cuda")
    pos = torch.tensor([[0, (1 << 31) + 12345, (1 << 33) + 7, -1, -(1 << 31) - 99]], device="cuda")
    cfg = kvq.make_rope_config(128)
    (out,) = kvq.rope(cfg, [x], pos, out_dtype=torch.float32)
    (back,) = kvq.rope(cfg, [out.transpose(1, 2)], -pos, out_dtype=torch.float32)
    assert (back.transpose(1, 2) - x).abs().max() <= 4 * 2.0 ** -21 * 2 * x.abs().max()
    # |pos| < 2^21 so that fp64 angles are exact enough to compare with
    w, gain = _freq(128, 10000.0, "none", 1.0, 0)
    pos = torch.tensor([[-5, 0, 1, -1048576, 1999999]], device="cuda")
    (out,) = kvq.rope(cfg, [x], pos, out_dtype=torch.float32)
    _check(x, out, pos.cpu().numpy(), 128, False, w, gain, True)


@pytest.mark.parametrize("x_type", [torch.float16, torch.float32])
@pytest.mark.parametrize("offset", [0, 1])
def test_strides_alignment_and_in_place(x_type, offset):
    """Rows that start off a 16-byte boundary, padded rows, strided outputs, expanded inputs and in-place turns."""
    kvq = _kvq()
    B, n, H, D = 2, 9, 3, 64
    cfg = kvq.make_rope_config(D)
    w, gain = _freq(D, 10000.0, "none", 1.0, 0)
    pos = _positions(B, n, 40)
    buf = torch.randn(B * n * H * (D + 8 + offset) + 1, device="cuda").to(x_type)
    x = buf[offset:].as_strided((B, n, H, D), (n * H * (D + 8 + offset), H * (D + 8 + offset), D + 8 + offset, 1))
    o = torch.full((B, H, n, 2 * D), 5.0, device="cuda", dtype=torch.float16)
    kvq.rope(cfg, [x], 40, outs=[o[..., :D]])
    _check(x, o[..., :D], pos, D, False, w, gain, True)
    assert (o[..., D:] == 5.0).all()
    one = torch.randn(B, n, 1, D, device="cuda").to(x_type).expand(B, n, H, D)  # one head for all (stride 0)
    (out,) = kvq.rope(cfg, [one], 40)
    _check(one, out, pos, D, False, w, gain, True)
    before = x.clone()
    kvq.rope(cfg, [x], 40, outs=[x.transpose(1, 2)])
    _check(before, x.transpose(1, 2), pos, D, False, w, gain, True)


def test_rows_behind_stay_and_other_stream():
    kvq = _kvq()
    cfg = kvq.make_rope_config(128)
    x = torch.randn(1, 33, 4, 128, device="cuda").half()
    big = torch.full((1, 4, 40, 128), 3.0, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kvq.rope(cfg, [x], 0, outs=[big[:, :, :33]], stream=s)
    s.synchronize()
    (want,) = kvq.rope(cfg, [x], 0)
    assert torch.equal(big[:, :, :33], want) and (big[:, :, 33:] == 3.0).all()
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    pos = torch.arange(33, device="cuda")[None].contiguous()
    with torch.cuda.graph(graph):
        kvq.rope(cfg, [x], pos, outs=[out])
    pos += 100
    graph.replay()
    assert torch.equal(out, kvq.rope(cfg, [x], 100)[0])


def test_binding_refusals():
    kvq = _kvq()
    cfg = kvq.make_rope_config(128)
    x = torch.zeros(1, 4, 2, 128, device="cuda", dtype=torch.float16)
    for bad in (lambda: kvq.rope(cfg, []), lambda: kvq.rope(cfg, [x[0]]), lambda: kvq.rope(cfg, [x.cpu()]),
                lambda: kvq.rope(cfg, [x, x.float()]), lambda: kvq.rope(cfg, [x[..., :64]]),
                lambda: kvq.rope(cfg, [x], torch.zeros(1, 4, device="cuda")),
                lambda: kvq.rope(cfg, [x], torch.zeros(1, 3, dtype=torch.int64, device="cuda")),
                lambda: kvq.rope(cfg, [x], rotate=[True, False]), lambda: kvq.rope(cfg, [x], outs=[x]),
                lambda: kvq.rope(cfg, [x.transpose(2, 3).contiguous().transpose(2, 3)]),
                lambda: kvq.rope(cfg, [x], outs=[torch.zeros(1, 1, 4, 128, device="cuda").half().expand(1, 2, 4, 128)]),
                lambda: kvq.rope(cfg, [x], out_dtype=torch.float64),
                lambda: kvq.make_rope_config(scaling="other")):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kvq.KVQError):
        kvq.rope(cfg, [x] * 5)


def test_from_projection_to_decode():
    """The operators together, as a server runs them: turn, step a prompt, fork it, verify drafted tokens on the forks,
    reorder them and decode -- against the same steps with the whole history attended at once."""
    kvq = _kvq()
    D, H, Hq, n, m = 128, 2, 8, 300, 6
    cfg = kvq.make_rope_config(D, base=10000.0)
    one = kvq.KVCache(1, H, Hq, D, 400, 4, 4, 32, 128)
    many = kvq.KVCache(3, H, Hq, D, 400, 4, 4, 32, 128)
    qkv = torch.randn(1, n, (Hq + 2 * H) * D, device="cuda").to(torch.bfloat16)
    q, k, v = kvq.rope(cfg, list(qkv.view(1, n, Hq + 2 * H, D).split([Hq, H, H], dim=2)), 0, rotate=[True, True, False])
    one.chunk_step(k, v, q)
    many.copy_sequences(one, torch.zeros(3, dtype=torch.int32, device="cuda"))
    draft = torch.randn(3, m, (Hq + 2 * H) * D, device="cuda").to(torch.bfloat16)
    q2, k2, v2 = kvq.rope(cfg, list(draft.view(3, m, Hq + 2 * H, D).split([Hq, H, H], dim=2)), n, rotate=[True, True, False])
    out = many.chunk_attention(k2, v2, q2)
    many.append_chunk(k2, v2, n_tokens=4)  # two drafted tokens are turned down
    order = torch.tensor([2, 0, 2], dtype=torch.int32, device="cuda")
    many.copy_sequences(many, order)
    last = many.decode_attention(q2[order.long(), :, 4].contiguous())
    assert many.state()[0] == n + 4 and many.sync_status() == 0
    # plain attention over exported values
    for b in range(3):
        src = int(order[b])
        for h in range(H):
            u = many.export_unit(b, h)
            assert np.array_equal(u["wk"][-4:].view(np.float16), k2[src, h, :4].cpu().numpy())
    ref = kvq.KVCache(3, H, Hq, D, 400, 4, 4, 32, 128)
    ref.prefill_quantize(k.expand(3, -1, -1, -1).contiguous(), v.expand(3, -1, -1, -1).contiguous())
    for i in range(4):
        ref.append(k2[:, :, i].contiguous(), v2[:, :, i].contiguous())
        if i < 3:
            step = ref.decode_attention(q2[:, :, i].contiguous())
            err = (step.float() - out[:, :, i].float()).abs().amax(-1) / step.float().abs().amax(-1)
            assert err.max() <= 4.2e-3  # two results, each within 2e-3 of the exact one
    want = ref.decode_attention(q2[:, :, 4].contiguous())[order.long()]
    err = (last.float() - want.float()).abs().amax(-1) / want.float().abs().amax(-1)
    assert err.max() <= 4.2e-3
    for c in (one, many, ref):
        c.close()
