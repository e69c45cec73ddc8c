"""Copies of sequences between caches and within one: every store of every unit bit for bit, and decode after it."""
import numpy as np
import pytest

import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

D = 128


def _kvq():
    import bit_asymmetric_kv_kvq_gb300 as kvq
    return kvq


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _filled(w, max_tokens=None):
    kvq = _kvq()
    T = w.prefill_tokens
    c = kvq.KVCache.for_workload(w, max_tokens=max_tokens)
    c.prefill_quantize(_dev(synth.keys(w)[:, :, :T]), _dev(synth.values(w)[:, :, :T]))
    return c


def _units(c):
    return [[c.export_unit(b, h) for h in range(c.cfg.num_kv_heads)] for b in range(c.cfg.batch)]


def _same(got, want):
    for a, b in zip(got, want):
        for key in b:
            assert np.array_equal(a[key], b[key]), key


def _idx(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("widx,kw", [
    (0, dict(batch=3, kv_heads=2, q_heads=2, prefill_tokens=1)),
    (0, dict(batch=3, kv_heads=2, q_heads=2, prefill_tokens=128)),
    (1, dict(batch=3, kv_heads=4, q_heads=4, prefill_tokens=700)),
    (2, dict(batch=3, kv_heads=2, q_heads=2, prefill_tokens=391, sink=5)),
    (3, dict(batch=3, kv_heads=2, q_heads=8, prefill_tokens=385, sink=3, residual=64)),
    (4, dict(batch=3, kv_heads=2, q_heads=8, prefill_tokens=300)),
    (4, dict(batch=3, kv_heads=1, q_heads=4, prefill_tokens=2, sink=7)),
])
@pytest.mark.parametrize("index", [[0], [2, 0, 0, 1, 2], [1] * 40])
def test_into_another_cache(widx, kw, index):
    """Forks, repeats and compactions into a cache of another batch and capacity, which then decodes like its source."""
    kvq = _kvq()
    w = synth.WORKLOADS[widx].scaled(**kw)
    src = _filled(w)
    want = _units(src)
    dst = kvq.KVCache.for_workload(w.scaled(batch=len(index)), max_tokens=w.prefill_tokens + 50)
    # dst holds something else before
    one = torch.ones(len(index), w.kv_heads, 9, D, dtype=torch.float16, device="cuda")
    dst.prefill_quantize(one, one)
    dst.copy_sequences(src, _idx(index))
    assert dst.state() == src.state() and dst.sync_status() == 0
    for b, i in enumerate(index[:6]):
        _same([dst.export_unit(b, h) for h in range(w.kv_heads)], want[i])
    _same(sum(_units(src), []), sum(want, []))
    # the copies go on by themselves: the same token everywhere gives the same state as in the source
    k1 = torch.randn(3, w.kv_heads, D, device="cuda").half()
    src.append(k1, k1)
    at = _idx(index).long()
    dst.append(k1[at].contiguous(), k1[at].contiguous())
    assert dst.state() == src.state()
    after = _units(src)
    for b, i in enumerate(index[:6]):
        _same([dst.export_unit(b, h) for h in range(w.kv_heads)], after[i])
    src.close()
    dst.close()


@pytest.mark.parametrize("index", [[0, 1, 2, 3, 4], [1, 0, 3, 4, 2], [4, 4, 4, 4, 4], [0, 0, 2, 2, 1], [3, 2, 0, 0, 3]])
@pytest.mark.parametrize("widx", [1, 4])
def test_in_place(widx, index):
    """Reordering within a cache under any map, cycles and repeats among them."""
    w = synth.WORKLOADS[widx].scaled(batch=5, kv_heads=2, q_heads=8 if widx == 4 else 2, prefill_tokens=333, sink=2)
    c = _filled(w)
    want = _units(c)
    state = c.state()
    c.copy_sequences(c, _idx(index))
    assert c.state() == state and c.sync_status() == 0
    got = _units(c)
    for b, i in enumerate(index):
        _same(got[b], want[i])
    c.close()


@pytest.mark.parametrize("B", [130, 1000])
def test_in_place_large_batches(B):
    kvq = _kvq()
    c = kvq.KVCache(B, 1, 1, D, 140, 2, 2, 32, 128)
    k = torch.randn(B, 1, 140, D, device="cuda").half()
    c.prefill_quantize(k, k)
    before = {n: t.clone() for n, t in c.buffers().items()}
    perm = torch.randperm(B, device="cuda").to(torch.int32)
    c.copy_sequences(c, perm)
    assert c.sync_status() == 0
    for n, t in c.buffers().items():
        used = t if n == "pages" else t[:, :12]
        want = before[n] if n == "pages" else before[n][:, :12]
        assert torch.equal(used, want[perm.long()]), n
    c.close()


def test_rows_behind_the_last_token_stay():
    """Only pages and rows in use are written."""
    kvq = _kvq()
    src = kvq.KVCache(1, 2, 2, D, 600, 2, 2, 32, 128)
    k = torch.randn(1, 2, 300, D, device="cuda").half()
    src.prefill_quantize(k, k)
    dst = kvq.KVCache(2, 2, 2, D, 900, 2, 2, 32, 128)
    view = dst.buffers()
    view["pages"].fill_(0xA5)
    view["wk"].fill_(7.0)
    view["wv"].fill_(7.0)
    dst.copy_sequences(src, _idx([0, 0]))
    torch.cuda.synchronize()
    used = 2 * src.buffers()["pages"].shape[1] // 4  # two of the source's four pages
    assert torch.equal(view["pages"].view(2, 2, -1)[1, :, :used], src.buffers()["pages"][:, :used])
    assert (view["pages"][:, used:] == 0xA5).all()
    assert (view["wk"][:, 300 - 256:] == 7.0).all() and (view["wv"][:, 300 - 256:] == 7.0).all()
    src.close()
    dst.close()


def test_index_out_of_range_is_reported_and_leaves_the_sequence():
    kvq = _kvq()
    w = synth.WORKLOADS[1].scaled(batch=3, kv_heads=2, q_heads=2, prefill_tokens=300)
    src, dst = _filled(w), _filled(w.scaled(seed=99))
    before = {n: t.clone() for n, t in dst.buffers().items()}
    want = {n: t.clone() for n, t in src.buffers().items()}
    dst.copy_sequences(src, _idx([1, 3, -1]))
    assert dst.sync_status() == kvq.kvq.KVQ_ERR_CUDA
    for n, t in dst.buffers().items():
        rows = t.shape[1] if n == "pages" else 300 - 256
        assert torch.equal(t[:2, :rows], want[n][2:4, :rows]) and torch.equal(t[2:], before[n][2:]), n
    src.close()
    dst.close()


def test_captured_copy_reads_the_index_of_the_moment():
    kvq = _kvq()
    c = kvq.KVCache(4, 2, 2, D, 300, 4, 2, 32, 128)
    k = torch.randn(4, 2, 300, D, device="cuda").half()
    c.prefill_quantize(k, k)
    idx = _idx([0, 1, 2, 3])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.copy_sequences(c, idx)
    now = torch.arange(4, device="cuda")
    base = c.buffers()["pages"].clone().view(4, 2, -1)
    for m in ([3, 0, 1, 2], [1, 1, 0, 3], [2, 3, 2, 0]):
        idx.copy_(_idx(m))
        graph.replay()
        now = now[torch.tensor(m, device="cuda")]
        torch.cuda.synchronize()
        assert torch.equal(c.buffers()["pages"].view(4, 2, -1), base[now])
    c.close()


def test_empty_source_and_refusals():
    kvq = _kvq()
    E = kvq.kvq
    a = kvq.KVCache(2, 2, 2, D, 300, 2, 2, 32, 128)
    b = kvq.KVCache(2, 2, 2, D, 200, 2, 2, 32, 128)
    k = torch.randn(2, 2, 250, D, device="cuda").half()
    a.prefill_quantize(k, k)
    idx = _idx([0, 1])

    def status(f):
        with pytest.raises(kvq.KVQError) as e:
            f()
        return e.value.status
    assert status(lambda: b.copy_sequences(a, idx)) == E.KVQ_ERR_CAPACITY
    assert b.state() == (0, 0, 0)
    for other in (dict(k_bits=4), dict(residual=64), dict(group_size=64), dict(sink_tokens=1), dict(k_sparse=1),
                  dict(softmax_scale=1.0)):
        c = kvq.KVCache(2, 2, 2, D, 300, **{**dict(k_bits=2, v_bits=2, group_size=32, residual=128), **other})
        assert status(lambda: c.copy_sequences(a, idx)) == E.KVQ_ERR_INVALID_ARG, other
        c.close()
    L = kvq.lib()
    assert L.kvq_copy_sequences(a.handle, None, idx.data_ptr(), None) == -1
    assert L.kvq_copy_sequences(a.handle, a.handle, None, None) == -1
    assert L.kvq_copy_sequences(a.handle, a.handle, idx.data_ptr() + 2, None) == -1
    for bad in (idx.long(), idx[:1], idx.cpu(), torch.stack([idx, idx], 1)[:, 0]):
        with pytest.raises(ValueError):
            a.copy_sequences(a, bad)
    with pytest.raises(TypeError):
        a.copy_sequences(a.handle, idx)
    launches = a.launch_count()
    a.copy_sequences(b, idx)  # an empty source empties
    assert a.state() == (0, 0, 0) and a.launch_count() == launches
    a.append(k[:, :, 0].contiguous(), k[:, :, 0].contiguous())
    assert a.state() == (1, 0, 1) and a.sync_status() == 0
    lv = [0.0, 1.2, 1.9, 3.0]
    x = kvq.KVCache(2, 2, 2, D, 300, 2, 2, 32, 128, k_levels=lv, v_levels=lv)
    y = kvq.KVCache(2, 2, 2, D, 300, 2, 2, 32, 128, k_levels=[0.0, 1.0, 2.0, 3.0], v_levels=lv)
    assert status(lambda: x.copy_sequences(y, idx)) == E.KVQ_ERR_INVALID_ARG
    for c in (a, b, x, y):
        c.close()
