"""Attention of a chunk of new tokens over the cache, the append of a chunk, and the two as one step.

The attention is compared with fp64 attention over the CPU oracle's dequantized cache followed by the
chunk's fp16 tokens (causal), for every unit and query row, with the metric of the decode tests: per row
||o - o*||_inf / ||o*||_inf <= 2e-3.  What the bound has to hold: the output's rounding (2^-11 of an
element), one fp16 rounding of every weight and value (2^-11 each, independent over tokens, so they shrink
like the output itself does when many tokens share the weight) and of every shifted key (2^-11 of |k - mu|;
for the outlier channels here |k - mu| <= 25, |q| ~ 1 and scale 1/sqrt(128), so a weight moves by at most
4 * 25 * 2^-11 / 11.3 = 4.3e-3 and by 1e-3 in the mean square, again independent over tokens).  The
appended state must equal the oracle's bit for bit.
"""
import numpy as np
import pytest

import oracle
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 2e-3
D = 128


def _kvq():
    import bit_asymmetric_kv_kvq_gb300 as kvq
    return kvq


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _workload(method, B, Hkv, hg, T, n, sink=0, queries="normal"):
    base = {"k2v2": (2, 2, 32, 128, 0, 0), "k4v2": (4, 2, 32, 128, 0, 0), "k4v4g64": (4, 4, 64, 64, 0, 0),
            "k2v2r32sp": (2, 2, 32, 32, 2, 0), "k2v2r96": (2, 2, 32, 96, 0, 0), "k4v4r128g64": (4, 4, 64, 128, 3, 0),
            "k3v3": (3, 3, 32, 96, 1, 0), "k3v3r128": (3, 3, 64, 128, 0, 0), "k3v3rope": (3, 3, 64, 128, 2, 1),
            "k2v2rope": (2, 2, 32, 64, 0, 1), "k4v2rope": (4, 2, 32, 128, 4, 1), "k4v4rope": (4, 4, 32, 32, 0, 1),
            "lut22": (2, 2, 32, 128, 0, 0), "lut33": (3, 3, 32, 64, 2, 0), "lut42": (4, 2, 64, 128, 0, 0),
            "lut33rope": (3, 3, 32, 128, 1, 1)}[method]
    kb, vb, G, R, nsp, rope = base
    levels = {}
    if method.startswith("lut"):
        def lev(bits):
            x = np.linspace(0.0, 1.0, 1 << bits) ** 1.3 * ((1 << bits) - 1)
            x[0], x[-1] = 0.0, (1 << bits) - 1
            return tuple(np.float32(x).tolist())
        levels = dict(k_levels=lev(kb), v_levels=lev(vb))
    return synth.WORKLOADS[0].scaled(batch=B, kv_heads=Hkv, q_heads=Hkv * hg, prefill_tokens=max(T, 1), decode_steps=n,
                                     k_bits=kb, v_bits=vb, group=G, residual=R, k_sparse=nsp, rope=rope, sink=sink,
                                     queries=queries, seed=17, **levels)


def _inputs(w, T, n):
    K = synth.keys(w)[:, :, :T + n]
    V = synth.values(w)[:, :, :T + n]
    rng = np.random.default_rng(5)
    q = rng.standard_normal((w.batch, w.q_heads, n, D)).astype(np.float16)
    return np.ascontiguousarray(K), np.ascontiguousarray(V), q


def _dequant(u):
    k, v = np.zeros((u.T, D)), np.zeros((u.T, D))
    for t in range(u.T):
        k[t], v[t] = u.dequant(t)
    return k, v


def _reference(w, u, k_new, v_new, q):
    """fp64 attention [hg][n][D] of one unit: the oracle's cache, then the chunk, causal."""
    kc, vc = _dequant(u)
    T, n = u.T, k_new.shape[0]
    kn = k_new.astype(np.float64)
    if w.rope:
        kn = np.stack([oracle.rope(kn[i], T + i, w.rope_base) for i in range(n)])
    K, V = np.concatenate([kc, kn]), np.concatenate([vc, v_new.astype(np.float64)])
    out = np.zeros(q.shape)
    for h in range(q.shape[0]):
        for i in range(n):
            m = T + i + 1
            s = K[:m] @ q[h, i].astype(np.float64) * w.softmax_scale
            p = np.exp(s - s.max())
            out[h, i] = (p / p.sum()) @ V[:m]
    return out


def _unit(w, K, V):
    u = oracle.OracleUnit.for_workload(w)
    if K.shape[0]:
        u.prefill(K, V)
    return u


def _check(w, units, K, V, q, out, T, t1, where=""):
    out = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(out).all(), where
    hg, worst = w.group_q, 0.0
    for (b, h), u in units.items():
        hs = slice(h * hg, (h + 1) * hg)
        ref = _reference(w, u, K[b, h, T:t1], V[b, h, T:t1], q[b, hs])
        worst = max(worst, oracle.max_rel_err(out[b, hs].reshape(-1, D), ref.reshape(-1, D)))
    assert worst <= TOL, (where, worst)
    return worst


CASES = [
    # method, B, Hkv, query heads per kv head, T, n, sink
    ("k2v2", 1, 1, 1, 0, 1, 0),         # a single token on an empty cache
    ("k2v2", 1, 2, 4, 0, 130, 0),       # a prompt on an empty cache, rows past one job
    ("k2v2", 2, 2, 4, 1, 1, 0),
    ("k2v2", 1, 2, 1, 128, 129, 0),     # a full window, a chunk past one tile
    ("k2v2", 1, 2, 4, 129, 5, 0),       # the first page
    ("k2v2", 2, 3, 2, 1000, 33, 0),
    ("k2v2", 3, 4, 4, 700, 150, 4),     # many jobs, sink rows
    ("k4v2", 2, 2, 1, 900, 17, 0),
    ("k4v2", 1, 2, 4, 515, 64, 128),    # as many sink tokens as window tokens
    ("k4v4g64", 1, 2, 4, 333, 40, 3),   # two pages a tile, an odd number of pages
    ("k2v2r32sp", 1, 2, 1, 357, 19, 0),  # four pages a tile, sparse entries in fragment-order pages
    ("k2v2r96", 1, 2, 2, 500, 70, 0),   # pages of 96 tokens: tiles of 96 keys
    ("k4v4r128g64", 1, 1, 4, 400, 31, 0),
    ("k3v3", 2, 2, 2, 611, 43, 3),
    ("k3v3r128", 1, 2, 4, 520, 9, 0),
    ("k3v3rope", 1, 2, 4, 700, 37, 0),
    ("k3v3rope", 1, 1, 1, 0, 140, 7),
    ("k2v2rope", 1, 2, 4, 333, 12, 1),
    ("k4v2rope", 1, 2, 1, 300, 130, 0),
    ("k4v4rope", 1, 1, 4, 100, 3, 0),
    ("lut22", 1, 2, 4, 400, 20, 0),
    ("lut33", 1, 1, 1, 300, 21, 2),
    ("lut42", 1, 2, 1, 300, 5, 0),
    ("lut33rope", 1, 1, 4, 400, 11, 0),
]


@pytest.mark.parametrize("method,B,Hkv,hg,T,n,sink", CASES)
def test_chunk_attention_and_step(method, B, Hkv, hg, T, n, sink):
    kvq = _kvq()
    w = _workload(method, B, Hkv, hg, T, n, sink)
    K, V, q = _inputs(w, T, n)
    cache = kvq.KVCache.for_workload(w, max_tokens=T + n)
    if T:
        cache.prefill_quantize(_dev(K[:, :, :T]), _dev(V[:, :, :T]))
    units = {(b, h): _unit(w, K[b, h, :T], V[b, h, :T]) for b in range(B) for h in range(Hkv)}
    before = cache.state()
    kn, vn, qd = _dev(K[:, :, T:]), _dev(V[:, :, T:]), _dev(q)
    out = cache.chunk_attention(kn, vn, qd)
    assert cache.sync_status() == 0
    worst = _check(w, units, K, V, q, out, T, T + n, "attention")
    print(f"worst {worst:.2e}")
    assert cache.state() == before  # the cache is as it was
    again = cache.chunk_attention(kn, vn, qd)
    assert torch.equal(out, again)  # sums in a fixed order
    stepped = cache.chunk_step(kn, vn, qd)
    assert torch.equal(out, stepped)
    assert cache.sync_status() == 0
    for (b, h), u in units.items():
        for i in range(T, T + n):
            u.append(K[b, h, i], V[b, h, i])
        got, ref = cache.export_unit(b, h), u.stores()
        for key in ref:
            assert np.array_equal(got[key], ref[key]), (b, h, key)
    u0 = units[(0, 0)]
    assert cache.state() == (u0.T, u0.Tq, u0.n_r)
    cache.close()


@pytest.mark.parametrize("method", ["k3v3", "k3v3rope", "k4v2rope", "lut33", "k2v2r32sp"])
def test_sparse_entries_in_both_channels_of_a_pair(method):
    """Entries c and c + 64 of one token are the two halves of a rotated pair, and their places change from token to
    token, so the scores themselves are rounded coarsely.  The bound per row: a key's channel is rounded to fp16 once (half
    a step: 2^-11 of it) after a rotation whose sine and cosine are off by 2^-20, so score j is off by at most e_j =
    scale sum_c |q_c| (2^-11 |k_c| + 2^-19 |k_pair|); mu is 0 here (the ranges hold 0 well inside).  With e the largest,
    weights p_j move by factors within exp(+-2e) that keep their sum, so the output by at most expm1(2e) sum_j p_j |v_j - o|;
    weights and values are rounded once each (2^-11, 2^-11 of |v_j|) and so is the output."""
    kvq = _kvq()
    B, Hkv, hg, T, n = 1, 2, 4, 420, 6
    w = _workload(method, B, Hkv, hg, T, n)
    K, V, q = _inputs(w, T, n)
    rng = np.random.default_rng(11)
    K = np.clip(K, -1, 1)
    for t in range(T):
        c = int(rng.integers(0, 64)) if t % 3 else 5
        K[:, :, t, c] = 25.0 * rng.choice([-1.0, 1.0], K[:, :, t, c].shape)
        if t % 2:
            K[:, :, t, c + 64] = 24.0 * rng.choice([-1.0, 1.0], K[:, :, t, c].shape)
    K = np.ascontiguousarray(K.astype(np.float16))
    cache = kvq.KVCache.for_workload(w, max_tokens=T + n)
    cache.prefill_quantize(_dev(K[:, :, :T]), _dev(V[:, :, :T]))
    units = {(b, h): _unit(w, K[b, h, :T], V[b, h, :T]) for b in range(B) for h in range(Hkv)}
    out = cache.chunk_attention(_dev(K[:, :, T:]), _dev(V[:, :, T:]), _dev(q)).float().cpu().numpy().astype(np.float64)
    assert cache.sync_status() == 0
    worst = 0.0
    for (b, h), u in units.items():
        kc, vc = _dequant(u)
        kn = K[b, h, T:].astype(np.float64)
        if w.rope:
            kn = np.stack([oracle.rope(kn[i], T + i, w.rope_base) for i in range(n)])
        keys, vals = np.concatenate([kc, kn]), np.concatenate([vc, V[b, h, T:].astype(np.float64)])
        step = 2.0 ** -11 * np.abs(keys) + 2.0 ** -19 * np.tile(np.hypot(keys[:, :64], keys[:, 64:]), 2)
        for g in range(hg):
            for i in range(n):
                m, x = T + i + 1, q[b, h * hg + g, i].astype(np.float64)
                s = keys[:m] @ x * w.softmax_scale
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ vals[:m]
                e = (step[:m] @ np.abs(x)).max() * w.softmax_scale
                bound = np.expm1(2 * e) * (p @ np.abs(vals[:m] - o)) + 2.0 ** -10 * (p @ np.abs(vals[:m])) + 2.0 ** -11 * np.abs(o) + 1e-6
                err = np.abs(out[b, h * hg + g, i] - o)
                worst = max(worst, (err / bound).max())
    print(f"worst {worst:.3f} of the bound")
    assert worst <= 1.0
    cache.close()


@pytest.mark.parametrize("method,sink,pieces", [
    ("k2v2", 0, [1, 127, 1, 128, 257, 3, 130]),
    ("k2v2", 5, [3, 2, 128, 128, 1, 300]),
    ("k4v4g64", 9, [700, 1, 64, 63]),
    ("k3v3", 1, [95, 2, 96, 200]),
    ("k3v3rope", 0, [129, 129, 129]),
])
def test_append_chunk_equals_the_oracle(method, sink, pieces):
    """Pieces appended one after the other leave what single appends leave, bit for bit; a piece may be
    the head of a longer buffer."""
    kvq = _kvq()
    total = sum(pieces)
    w = _workload(method, 2, 2, 1 if method != "k3v3rope" else 4, total, 1, sink)
    K, V, _ = _inputs(w, total, 0)
    cache = kvq.KVCache.for_workload(w, max_tokens=total)
    units = {(b, h): oracle.OracleUnit.for_workload(w) for b in range(2) for h in range(2)}
    at = 0
    for i, n in enumerate(pieces):
        end = min(total, at + n + (7 if i % 2 else 0))  # more tokens in the buffer than are taken
        cache.append_chunk(_dev(K[:, :, at:end]), _dev(V[:, :, at:end]), n_tokens=n)
        for (b, h), u in units.items():
            for t in range(at, at + n):
                u.append(K[b, h, t], V[b, h, t])
        at += n
        u0 = units[(0, 0)]
        assert cache.state() == (u0.T, u0.Tq, u0.n_r), i
        for (b, h), u in units.items():
            got, ref = cache.export_unit(b, h), u.stores()
            for key in ref:
                assert np.array_equal(got[key], ref[key]), (i, b, h, key)
    with pytest.raises(kvq.KVQError) as e:
        cache.append_chunk(_dev(K[:, :, :1]), _dev(V[:, :, :1]))
    assert e.value.status == kvq.kvq.KVQ_ERR_CAPACITY
    assert cache.state()[0] == total
    cache.close()


@pytest.mark.parametrize("method,hg,sink,pieces", [
    ("k2v2", 4, 0, [200, 130, 1, 77]), ("k4v2", 1, 4, [150, 150]), ("k3v3rope", 4, 0, [140, 139, 2]),
    ("k3v3", 2, 3, [43, 43, 43, 43]),
])
def test_prompt_in_pieces(method, hg, sink, pieces):
    """Every piece attends the quantized cache the pieces before it left, and itself in fp16."""
    kvq = _kvq()
    total = sum(pieces)
    w = _workload(method, 1, 2, hg, total, 1, sink)
    K, V, q = _inputs(w, 0, total)
    cache = kvq.KVCache.for_workload(w, max_tokens=total)
    units = {(0, h): oracle.OracleUnit.for_workload(w) for h in range(2)}
    ws = cache.chunk_workspace(max(pieces))
    at = 0
    for n in pieces:
        sl = slice(at, at + n)
        out = cache.chunk_step(_dev(K[:, :, sl]), _dev(V[:, :, sl]), _dev(q[:, :, sl]), workspace=ws)
        _check(w, units, K, V, q[:, :, sl], out, at, at + n, at)
        for (b, h), u in units.items():
            for t in range(at, at + n):
                u.append(K[b, h, t], V[b, h, t])
        at += n
    assert cache.sync_status() == 0
    # the cache goes on with single tokens
    qd = _dev(q[:, :, 0])
    got = cache.decode_attention(qd).cpu().numpy().astype(np.float64)
    for (b, h), u in units.items():
        hs = slice(h * hg, (h + 1) * hg)
        assert oracle.max_rel_err(got[b, hs], u.attention(q[b, hs, 0], w.softmax_scale)) <= TOL
    cache.close()


def test_one_token_chunk_agrees_with_decode():
    """A chunk of one token attends what decode_step attends."""
    kvq = _kvq()
    w = _workload("k2v2", 2, 2, 4, 1500, 1)
    K, V, q = _inputs(w, 1500, 1)
    a, b = kvq.KVCache.for_workload(w), kvq.KVCache.for_workload(w)
    for c in (a, b):
        c.prefill_quantize(_dev(K[:, :, :1500]), _dev(V[:, :, :1500]))
    x = a.chunk_step(_dev(K[:, :, 1500:]), _dev(V[:, :, 1500:]), _dev(q))[:, :, 0]
    y = b.decode_step(_dev(K[:, :, 1500]), _dev(V[:, :, 1500]), _dev(q[:, :, 0]))
    assert a.state() == b.state()
    # each is within 2e-3 of the exact result
    assert oracle.max_rel_err(x.cpu().numpy().reshape(-1, D), y.cpu().numpy().astype(np.float64).reshape(-1, D)) <= 2.1 * TOL
    a.close()
    b.close()


@pytest.mark.parametrize("method", ["k2v2", "k3v3rope"])
@pytest.mark.parametrize("what", ["nan", "inf", "lowest"])
def test_hidden_tokens_cannot_reach_a_row(method, what):
    """What a later token holds does not change the rows before it: bit for bit the same outputs; the rows that
    do see it show it."""
    kvq = _kvq()
    T, n, bad = 200, 150, 70
    w = _workload(method, 1, 2, 4, T, n)
    K, V, q = _inputs(w, T, n)
    cache = kvq.KVCache.for_workload(w, max_tokens=T + n)
    cache.prefill_quantize(_dev(K[:, :, :T]), _dev(V[:, :, :T]))
    clean = cache.chunk_attention(_dev(K[:, :, T:]), _dev(V[:, :, T:]), _dev(q))
    x = {"nan": np.float16(np.nan), "inf": np.float16(np.inf), "lowest": np.float16(-65504)}[what]
    K2, V2 = K.copy(), V.copy()
    V2[:, 0, T + bad, 3] = x      # one value of one channel
    K2[:, 1, T + bad] = x         # a whole key
    out = cache.chunk_attention(_dev(K2[:, :, T:]), _dev(V2[:, :, T:]), _dev(q))
    assert torch.equal(out[:, :, :bad], clean[:, :, :bad])
    seen = out[:, :, bad:].float()
    if what == "nan":
        assert torch.isnan(seen[:, :4, :, 3]).all()
        assert torch.isfinite(seen[:, :4, :, :3]).all() and torch.isfinite(seen[:, :4, :, 4:]).all()
        assert torch.isnan(seen[:, 4:]).all()
    elif what == "inf":
        assert (~torch.isfinite(seen[:, :4, :, 3])).all()
        assert torch.isfinite(seen[:, :4, :, 4:]).all()
    cache.close()


def test_keys_far_from_zero_and_equal_keys():
    """A channel with a large common part: its rounding must not reach the weights (keys enter as differences)."""
    kvq = _kvq()
    T, n = 400, 24
    w = _workload("k4v2", 1, 2, 1, T, n)
    K, V, q = _inputs(w, T, n)
    K = K.astype(np.float32)
    K[..., 7] = 500.0 + K[..., 7] % 4.0
    K[..., 90] = -300.0
    K = K.astype(np.float16)
    cache = kvq.KVCache.for_workload(w, max_tokens=T + n)
    cache.prefill_quantize(_dev(K[:, :, :T]), _dev(V[:, :, :T]))
    out = cache.chunk_attention(_dev(K[:, :, T:]), _dev(V[:, :, T:]), _dev(q))
    units = {(0, h): _unit(w, K[0, h, :T], V[0, h, :T]) for h in range(2)}
    _check(w, units, K, V, q, out, T, T + n)
    cache.close()


def test_other_stream_and_captured_graph():
    """On a stream of the caller's, and captured once and replayed with other inputs in the same buffers."""
    kvq = _kvq()
    T, n = 700, 20
    w = _workload("k2v2", 2, 2, 4, T, n)
    K, V, q = _inputs(w, T, n)
    cache = kvq.KVCache.for_workload(w, max_tokens=T + n)
    cache.prefill_quantize(_dev(K[:, :, :T]), _dev(V[:, :, :T]))
    kn, vn, qd = _dev(K[:, :, T:]), _dev(V[:, :, T:]), _dev(q)
    want = cache.chunk_attention(kn, vn, qd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = cache.chunk_attention(kn, vn, qd, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    got = cache.chunk_attention(kn, vn, qd, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)
    # two caches, each with a workspace of its own, at the same time on two streams
    other = kvq.KVCache.for_workload(w, max_tokens=T + n)
    other.prefill_quantize(_dev(K[:, :, :T]), _dev(V[:, :, :T]))
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [c.chunk_attention(kn, vn, qd, stream=x) for _ in range(8) for c, x in ((cache, a), (other, b))]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)
    other.close()
    out, ws = torch.empty_like(qd), cache.chunk_workspace(n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.chunk_attention(kn, vn, qd, out=out, workspace=ws)
    for scale in (1.0, 0.5):
        q2 = (q.astype(np.float32) * scale).astype(np.float16)
        qd.copy_(_dev(q2))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cache.chunk_attention(kn, vn, _dev(q2)))
    cache.close()


@pytest.mark.parametrize("method", ["k2v2", "k3v3rope"])
def test_wait_runs_out_and_is_reported(method):
    """A key tile that is never reported ready: every wait gives up after 1 ms, the call comes back, the error is
    reported, and the context goes on working."""
    import time
    kvq = _kvq()
    T, n = 900, 20
    w = _workload(method, 1, 2, 4, T, n)
    K, V, q = _inputs(w, T, n)
    kn, vn, qd = _dev(K[:, :, T:]), _dev(V[:, :, T:]), _dev(q)
    caches = [kvq.KVCache.for_workload(w, max_tokens=T + n) for _ in range(2)]
    for c in caches:
        c.prefill_quantize(_dev(K[:, :, :T]), _dev(V[:, :, :T]))
        assert c.sync_status() == 0
    kvq.kvq.kvq_test_inject(caches[0].handle, 0, 1_000_000)
    t0 = time.perf_counter()
    caches[0].chunk_attention(kn, vn, qd)
    assert caches[0].sync_status() == kvq.kvq.KVQ_ERR_CUDA
    assert time.perf_counter() - t0 < 1.0
    with pytest.raises(kvq.KVQError):
        caches[0].chunk_step(kn, vn, qd)
    out = caches[1].chunk_attention(kn, vn, qd)
    assert caches[1].sync_status() == 0
    units = {(0, h): _unit(w, K[0, h, :T], V[0, h, :T]) for h in range(2)}
    _check(w, units, K, V, q, out, T, T + n)
    for c in caches:
        c.close()


def test_refusals():
    kvq = _kvq()
    w = _workload("k2v2", 1, 2, 4, 64, 8)
    cache = kvq.KVCache.for_workload(w, max_tokens=72)
    k = torch.zeros(1, 2, 8, D, dtype=torch.float16, device="cuda")
    q = torch.zeros(1, 8, 8, D, dtype=torch.float16, device="cuda")
    ws = cache.chunk_workspace(8)
    L, h = kvq.lib(), cache.handle
    nb = ws.numel()
    st = torch.cuda.current_stream().cuda_stream
    call = lambda *a: L.kvq_chunk_attention(h, *a)  # noqa: E731
    ok = (k.data_ptr(), k.data_ptr(), q.data_ptr(), 8, q.data_ptr(), ws.data_ptr(), nb, st)
    for i, bad in ((0, None), (1, None), (2, None), (3, 0), (3, -1), (3, 1 << 31), (4, None), (5, None), (6, nb - 1),
                   (0, k.data_ptr() + 2), (5, ws.data_ptr() + 8)):
        args = list(ok)
        args[i] = bad
        assert call(*args) == kvq.kvq.KVQ_ERR_INVALID_ARG, (i, bad)
    for bad in ((8, 7), (0, 8), (-1, 8)):
        assert L.kvq_append_chunk(h, k.data_ptr(), k.data_ptr(), bad[0], bad[1], st) == kvq.kvq.KVQ_ERR_INVALID_ARG
    with pytest.raises(kvq.KVQError):
        kvq.kvq_chunk_workspace(h, 0)
    with pytest.raises(ValueError):
        cache.chunk_attention(k.float(), k, q)
    with pytest.raises(ValueError):
        cache.chunk_attention(k, k, q[:, :, :4])
    with pytest.raises(ValueError):
        cache.chunk_attention(k, k, q, workspace=torch.zeros(nb, dtype=torch.uint8))
    with pytest.raises(kvq.KVQError) as e:
        cache.append_chunk(torch.zeros(1, 2, 73, D, dtype=torch.float16, device="cuda"),
                           torch.zeros(1, 2, 73, D, dtype=torch.float16, device="cuda"))
    assert e.value.status == kvq.kvq.KVQ_ERR_CAPACITY
    assert cache.state() == (0, 0, 0) and cache.sync_status() == 0
    # a codebook cache without levels
    cfg = kvq.make_config(1, 2, 8, D, 72, 2, 2, 32, 128, codebook=1)
    hc = kvq.kvq_create(cfg)
    assert L.kvq_chunk_attention(hc, *ok) == kvq.kvq.KVQ_ERR_STATE
    assert L.kvq_append_chunk(hc, k.data_ptr(), k.data_ptr(), 8, 8, st) == kvq.kvq.KVQ_ERR_STATE
    kvq.kvq_destroy(hc)
    cache.close()
