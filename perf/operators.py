"""Cases for the operators that serve a chunk of tokens over the quantized cache.

Four operators, as a server around the cache calls them:

  rope   rotary positions of the projections' queries and keys (values moved along), into the cache's layout
  chunk  attention of n new tokens over the cached tokens and, causally, over each other (drafted tokens to verify)
  step   a prompt in pieces on an empty cache: each piece attends, then is appended
  copy   sequences of one cache copied into another or within one (fork a prompt, reorder beams, compact a batch)

Where `own` is false, `run` computes them with elementary torch operations in fp32 (angles in fp64); where it is true it
calls the framework.  The cache's quantizer is part of the definitions: keys in groups of G tokens of a channel, values in
groups of G channels of a token, zero point z = min, step s = fp16((max - min) / (2^B - 1)), code = rint((x - z) / s)
clamped, all in IEEE fp32; an element stands for z + s * code.  The newest 1..R tokens stay fp16, as do the first `sink`.
"""
import math

import torch

own = False

D = 128  # the cache's head dimension
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}

# cache configurations: bits of keys and values, G, R, sparse entries, keys rotated at decode, outlier channels (count, mean)
METHODS = {
    "k2v2": dict(kb=2, vb=2, G=32, R=128, nsp=0, rope=0, outl=(4, 40.0)),
    "k4v2": dict(kb=4, vb=2, G=32, R=128, nsp=0, rope=0, outl=(1, 50.0)),
    "k4v4": dict(kb=4, vb=4, G=64, R=64, nsp=0, rope=0, outl=(4, 40.0)),
    "k3v3": dict(kb=3, vb=3, G=32, R=96, nsp=1, rope=0, outl=(4, 40.0)),
    "k3v3r": dict(kb=3, vb=3, G=64, R=128, nsp=2, rope=1, outl=(4, 40.0)),
}


def _chunk(name, method, B, Hkv, Hq, T, n, sink=0, queries="normal"):
    return dict(name=name, op="chunk", method=method, B=B, Hkv=Hkv, Hq=Hq, T=T, n=n, sink=sink, queries=queries)


def _step(name, method, B, Hkv, Hq, n, piece, sink=0):
    return dict(name=name, op="step", method=method, B=B, Hkv=Hkv, Hq=Hq, n=n, piece=piece, sink=sink)


def _copy(name, method, Bs, Bd, Hkv, T, inplace):
    return dict(name=name, op="copy", method=method, Bs=Bs, Bd=Bd, Hkv=Hkv, T=T, inplace=inplace)


def _rope(name, B, n, Hq, Hkv, dtype, pos, per_token=False, interleaved=False, rot=128, scaling="none", factor=1.0,
          base=10000.0, context=0):
    return dict(name=name, op="rope", B=B, n=n, Hq=Hq, Hkv=Hkv, dtype=dtype, pos=pos, per_token=per_token,
                interleaved=interleaved, rot=rot, scaling=scaling, factor=factor, base=base, context=context)


def listed():
    return [
        # one token of eight sequences of a Llama-2-7B-shaped layer: latency of a single small launch
        _rope("rope-step-7b", 8, 1, 32, 32, "f16", 4096),
        # a long prompt of a bf16 model, GQA heads, positions scaled by wavelength for a long context
        _rope("rope-prompt-gqa", 1, 32768, 32, 8, "bf16", 0, scaling="wavelength", factor=8.0, base=500000.0, context=8192),
        # ragged positions far out, interleaved pairs over half of the head, odd sizes, fp32 activations
        _rope("rope-far-odd", 3, 1021, 12, 4, "f32", 1040000, per_token=True, interleaved=True, rot=64, scaling="yarn",
              factor=16.0, context=4096),
        # four drafted tokens over the tiny cache: latency of the smallest chunk
        _chunk("chunk-tiny", "k2v2", 1, 4, 4, 1024, 4),
        # eight drafted tokens of 32 sequences over 32768 cached tokens: the Llama-3-8B-shaped verification step
        _chunk("chunk-verify-gqa", "k2v2", 32, 8, 32, 32768, 8),
        # a piece of 512 prompt tokens over a Llama-2-13B-shaped cache, peaked queries
        _chunk("chunk-piece-13b", "k4v2", 4, 40, 40, 8192, 512, queries="peaked"),
        # 33 tokens over a million cached ones, keys rotated at decode, sparse outliers
        _chunk("chunk-1m-rope", "k3v3r", 1, 8, 32, 1048576, 33),
        # a whole prompt on an empty cache, odd length: causal attention of new tokens alone
        _step("step-prompt", "k2v2", 2, 8, 32, 4099, 4099),
        # the same prompt arriving in pieces that end inside pages, with sink tokens
        _step("step-pieces", "k4v4", 2, 8, 32, 4099, 1000, sink=4),
        # a short prompt in tiny pieces, 3-bit codes: many small steps
        _step("step-short", "k3v3", 1, 2, 4, 301, 43, sink=3),
        # one prompt becomes eight samples (Llama-2-7B-shaped cache)
        _copy("copy-fork", "k2v2", 1, 8, 32, 4096, False),
        # half of 32 beams replaced by the survivors, in place (Llama-3-8B-shaped cache)
        _copy("copy-beams", "k2v2", 32, 32, 8, 32768, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "chunk", "step", "copy"])
    if op == "rope":
        Hq, Hkv = rng.choice([(32, 32), (32, 8), (12, 4), (40, 40), (4, 1)])
        n = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(32, 32768 // n)))
        scaling = rng.choice(["none", "linear", "wavelength", "yarn"])
        return dict(op="rope", B=B, n=n, Hq=Hq, Hkv=Hkv, dtype=rng.choice(["f16", "bf16", "f32"]),
                    pos=_log(rng, 1, 1000000), per_token=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                    rot=rng.choice([128, 128, 64, 32, 96]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 16.0]),
                    base=rng.choice([10000.0, 500000.0]), context=0 if scaling in ("none", "linear") else 8192)
    method = rng.choice(sorted(METHODS))
    heads = [(1, 4), (8, 32), (2, 8), (4, 4), (32, 32)]
    if METHODS[method]["kb"] == 3 and not METHODS[method]["rope"]:
        heads.append((4, 8))
    Hkv, Hq = rng.choice(heads)
    sink = rng.choice([0, 0, 1, 4, 31])
    if op == "chunk":
        n = _log(rng, 1, 1024)
        T = _log(rng, 1, min(131072, (1 << 25) // n))
        B = _log(rng, 1, max(1, min(32, (1 << 29) // (Hq * T * max(n, 16)))))
        return dict(op="chunk", method=method, B=B, Hkv=Hkv, Hq=Hq, T=T, n=n, sink=sink,
                    queries=rng.choice(["normal", "peaked"]))
    if op == "step":
        n = _log(rng, 1, 4096)
        piece = max(1, n // rng.choice([1, 1, 2, 3, 7]) + rng.choice([0, 1]))
        B = _log(rng, 1, max(1, min(8, 256 * 4096 // (Hq * n))))
        return dict(op="step", method=method, B=B, Hkv=Hkv, Hq=Hq, n=n, piece=piece, sink=sink)
    T = _log(rng, 150, 16384)
    Bs = _log(rng, 1, 32)
    inplace = rng.random() < 0.5
    return dict(op="copy", method=method, Bs=Bs, Bd=Bs if inplace else _log(rng, 1, 32), Hkv=Hkv, T=T, inplace=inplace)


# ---------------------------------------------------------------- what the definitions fix

def _quantized(T, R, sink):
    """(sink tokens, quantized tokens) of a cache that holds T tokens."""
    ns = min(T, sink)
    rest = T - ns
    return ns, 0 if rest <= 0 else R * ((rest - 1) // R)


def _page_bytes(m):
    def up(x):
        return (x + 15) // 16 * 16
    R, G = m["R"], m["G"]
    return (up(R * D * m["kb"] // 8) + up(R // G * D * 4) + up(R * D * m["vb"] // 8) + up(R * (D // G) * 4)
            + up(R * m["nsp"]) + up(R * m["nsp"] * 2))


def _seq_bytes(m, T, sink, Hkv):
    """Bytes of one sequence's cache: pages in use and fp16 rows."""
    ns, tq = _quantized(T, m["R"], sink)
    return Hkv * (tq // m["R"] * _page_bytes(m) + (T - tq) * D * 4)


def work(case):
    op = case["op"]
    if op == "rope":
        x = case["B"] * case["n"] * (case["Hq"] + 2 * case["Hkv"]) * D
        per = {"f16": 2, "bf16": 2, "f32": 4}[case["dtype"]]
        pos = case["B"] * case["n"] * 8 if case["per_token"] else 0
        rot = case["B"] * case["n"] * (case["Hq"] + case["Hkv"]) * case["rot"]
        return {"bytes": x * (per + 2) + pos, "flops": 3 * rot}
    m = METHODS[case["method"]]
    if op == "copy":
        row = _seq_bytes(m, case["T"], 0, case["Hkv"])
        if case["inplace"]:
            kept = (case["Bs"] + 1) // 2
            gone = case["Bs"] - kept
            return {"bytes": row * (gone + min(gone, kept)) + 4 * case["Bd"], "flops": 0}
        return {"bytes": row * (case["Bd"] + min(case["Bs"], case["Bd"])) + 4 * case["Bd"], "flops": 0}
    B, Hkv, Hq = case["B"], case["Hkv"], case["Hq"]

    def attend(T, n):
        return (B * (_seq_bytes(m, T, case["sink"], Hkv) + n * D * 4 * Hkv + n * D * 4 * Hq),
                4 * B * Hq * D * (n * T + n * (n + 1) // 2))
    if op == "chunk":
        b, f = attend(case["T"], case["n"])
        return {"bytes": b, "flops": f}
    b = f = 0
    for t0, t1 in _pieces(case):
        bi, fi = attend(t0, t1 - t0)
        # what the append stores: the pages that became full and the fp16 rows that are new
        _, q0 = _quantized(t0, m["R"], case["sink"])
        _, q1 = _quantized(t1, m["R"], case["sink"])
        rows = min(t1 - t0, t1 - q1)
        b += bi + B * Hkv * ((q1 - q0) // m["R"] * _page_bytes(m) + rows * D * 4)
        f += fi
    return {"bytes": b, "flops": f}


def _pieces(case):
    n, p = case["n"], case["piece"]
    return [(t, min(t + p, n)) for t in range(0, n, p)]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _keys_values(case, n_tokens, g):
    """fp16 keys with a few channels per head of large values of a fixed sign, and N(0,1) values."""
    m = METHODS[case["method"]]
    B, H = case["B"], case["Hkv"]
    count, mean = m["outl"]
    where = torch.rand(H, D, generator=g, device="cuda").argsort(dim=1)[:, :count]
    sign = torch.randint(0, 2, (H, count), generator=g, device="cuda").float() * 2 - 1
    mu = torch.zeros(H, D, device="cuda").scatter_(1, where, sign * mean)
    sd = torch.ones(H, D, device="cuda").scatter_(1, where, 5.0)
    K = torch.empty(B, H, n_tokens, D, dtype=torch.float16, device="cuda")
    V = torch.empty_like(K)
    for b in range(B):
        K[b] = torch.randn(H, n_tokens, D, generator=g, device="cuda").mul_(sd[:, None]).add_(mu[:, None]).half()
        V[b] = torch.randn(H, n_tokens, D, generator=g, device="cuda").half()
    return K, V


def _queries(case, K, n, g):
    """N(0,1) queries; peaked ones lean toward eight cached keys, so a few tokens hold most of the weight."""
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    q = torch.randn(B, Hq, n, D, generator=g, device="cuda")
    if case.get("queries") == "peaked":
        at = torch.randint(0, K.shape[2], (8,), generator=g, device="cuda")
        u = K[:, :, at].float().sum(2)
        u = u / u.norm(dim=-1, keepdim=True)
        q = q + 1.5 * u.repeat_interleave(Hq // Hkv, 1)[:, :, None]
    return q.half()


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "rope":
        B, n, Hq, Hkv = case["B"], case["n"], case["Hq"], case["Hkv"]
        qkv = torch.randn(B, n, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(DTYPES[case["dtype"]])
        pos = case["pos"]
        if case["per_token"]:  # every sequence at a place of its own
            first = torch.randint(0, 4096, (B, 1), generator=g, device="cuda", dtype=torch.int64) + case["pos"]
            pos = first + torch.arange(n, device="cuda", dtype=torch.int64)
        return qkv, pos
    if op == "copy":
        Bs, Bd, Hkv, m = case["Bs"], case["Bd"], case["Hkv"], METHODS[case["method"]]
        _, tq = _quantized(case["T"], m["R"], 0)
        used = tq // m["R"] * _page_bytes(m)
        pages = torch.randint(0, 256, (Bs, Hkv, used), generator=g, device="cuda", dtype=torch.uint8)
        wk = torch.randn(Bs, Hkv, case["T"] - tq, D, generator=g, device="cuda").half()
        wv = torch.randn(Bs, Hkv, case["T"] - tq, D, generator=g, device="cuda").half()
        if case["inplace"]:  # the ended half takes over the survivors, which stay where they are
            kept = (Bs + 1) // 2
            perm = torch.rand(Bs, generator=g, device="cuda").argsort()
            idx = torch.arange(Bs, device="cuda")
            idx[perm[kept:]] = perm[:Bs - kept]
        else:
            idx = torch.arange(Bd, device="cuda") % Bs
            idx = idx[torch.rand(Bd, generator=g, device="cuda").argsort()]
        return pages, wk, wv, idx.to(torch.int32)
    n_cached = case["T"] if op == "chunk" else 0
    K, V = _keys_values(case, n_cached + case["n"], g)
    return K, V, _queries(case, K, case["n"], g)


def prepare(case, seed):
    st = _prepare_own(case, seed) if own else _prepare_plain(case, seed)
    st["case"] = case
    return st


# ---------------------------------------------------------------- the framework

def _cache(case, batch, max_tokens, Hq, sink):
    import bit_asymmetric_kv_kvq_gb300 as kvq
    m = METHODS[case["method"]]
    return kvq.KVCache(batch, case["Hkv"], Hq, D, max_tokens, m["kb"], m["vb"], m["G"], m["R"], k_sparse=m["nsp"],
                       rope=m["rope"], sink_tokens=sink)


def _prepare_own(case, seed):
    import bit_asymmetric_kv_kvq_gb300 as kvq
    x = _inputs(case, seed)
    op = case["op"]
    if op == "rope":
        cfg = kvq.make_rope_config(head_dim=D, rot_dim=case["rot"], base=case["base"], interleaved=case["interleaved"],
                                   scaling=case["scaling"], factor=case["factor"], original_context=case["context"])
        return dict(qkv=x[0], pos=x[1], cfg=cfg)
    if op == "copy":
        pages, wk, wv, idx = x
        Bs, Bd, Hkv, T = case["Bs"], case["Bd"], case["Hkv"], case["T"]
        src = _cache(case, Bs, T, Hkv, 0)
        fill = torch.zeros(Bs, Hkv, T, D, dtype=torch.float16, device="cuda")
        src.prefill_quantize(fill, fill)
        view = src.buffers()
        view["pages"].view(Bs, Hkv, -1)[:, :, :pages.shape[2]] = pages
        view["wk"].view(Bs, Hkv, -1, D)[:, :, :wk.shape[2]] = wk
        view["wv"].view(Bs, Hkv, -1, D)[:, :, :wv.shape[2]] = wv
        dst = src if case["inplace"] else _cache(case, Bd, T, Hkv, 0)
        view = dst.buffers()
        outs = [view["pages"].view(Bd, Hkv, -1)[:, :, :pages.shape[2]],
                view["wk"].view(Bd, Hkv, -1, D)[:, :, :wk.shape[2]],
                view["wv"].view(Bd, Hkv, -1, D)[:, :, :wv.shape[2]]]
        return dict(src=src, dst=dst, idx=idx, outs=outs)
    K, V, q = x
    if op == "chunk":
        T, n = case["T"], case["n"]
        cache = _cache(case, case["B"], T + n, case["Hq"], case["sink"])
        cache.prefill_quantize(K[:, :, :T].contiguous(), V[:, :, :T].contiguous())
        return dict(cache=cache, k=K[:, :, T:].contiguous(), v=V[:, :, T:].contiguous(), q=q,
                    ws=cache.chunk_workspace(n))
    cache = _cache(case, case["B"], case["n"], case["Hq"], case["sink"])
    parts = [(K[:, :, a:b].contiguous(), V[:, :, a:b].contiguous(), q[:, :, a:b].contiguous()) for a, b in _pieces(case)]
    view = cache.buffers()
    return dict(cache=cache, parts=parts, ws=cache.chunk_workspace(max(b - a for a, b in _pieces(case))),
                rows=[view["wk"].view(case["B"], case["Hkv"], -1, D), view["wv"].view(case["B"], case["Hkv"], -1, D)])


def _run_own(st):
    import bit_asymmetric_kv_kvq_gb300 as kvq
    case = st["case"]
    op = case["op"]
    if op == "rope":
        B, n, Hq, Hkv = case["B"], case["n"], case["Hq"], case["Hkv"]
        q, k, v = st["qkv"].view(B, n, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=2)
        return kvq.rope(st["cfg"], [q, k, v], st["pos"], rotate=[True, True, False])
    if op == "copy":
        st["dst"].copy_sequences(st["src"], st["idx"])
        return st["outs"]
    cache = st["cache"]
    if op == "chunk":
        return cache.chunk_attention(st["k"], st["v"], st["q"], workspace=st["ws"])
    cache.reset()
    outs = [cache.chunk_step(k, v, q, workspace=st["ws"]) for k, v, q in st["parts"]]
    _, tq, nr = cache.state()
    ns = case["n"] - tq - nr
    at = [slice(case["sink"], case["sink"] + nr)] + ([slice(0, ns)] if ns else [])
    return outs + [buf[:, :, a] for buf in st["rows"] for a in at]  # and the rows that stay fp16, window first


# ---------------------------------------------------------------- the plain forms (fp32)

def _codes(x, dim, bits, hole=None):
    """Codes, zero points and steps of groups along `dim` of fp32 values; `hole` marks entries left out of the range."""
    L = 2 ** bits - 1
    if hole is None:
        mn, mx = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    else:
        mn = x.masked_fill(hole, math.inf).amin(dim, keepdim=True)
        mx = x.masked_fill(hole, -math.inf).amax(dim, keepdim=True)
        none = hole.all(dim, keepdim=True)
        mn, mx = mn.masked_fill(none, 0.0), mx.masked_fill(none, 0.0)
    mn = mn + 0.0
    s = ((mx - mn) / float(L)).half().float()
    c = torch.where(s > 0, ((x - mn) / s).round().clamp(0, L), torch.zeros((), device=x.device))
    if hole is not None:
        c = c.masked_fill(hole, 0.0)
    return c.to(torch.uint8), mn.half(), s.half()


def _sparse_mask(K16, nsp):
    """Marks the nsp largest |x| of each key vector, ties to the lower channel."""
    key = (K16.view(torch.int16).int() & 0x7FFF) * D + (D - 1 - torch.arange(D, device=K16.device, dtype=torch.int32))
    mask = torch.zeros(K16.shape, dtype=torch.bool, device=K16.device)
    for _ in range(nsp):
        at = key.argmax(-1, keepdim=True)
        mask.scatter_(-1, at, True)
        key.scatter_(-1, at, -1)
    return mask


def _quantize(case, K, V):
    """Codes and parameters of whole pages of keys and values [B][H][Tq][D], one sequence at a time."""
    m = METHODS[case["method"]]
    G, parts = m["G"], []
    for b in range(K.shape[0]):
        H, Tq, _ = K[b].shape
        hole = _sparse_mask(K[b], m["nsp"]) if m["nsp"] else None
        kc, kz, ks = _codes(K[b].float().view(H, Tq // G, G, D), 2, m["kb"],
                            None if hole is None else hole.view(H, Tq // G, G, D))
        vc, vz, vs = _codes(V[b].float().view(H, Tq, D // G, G), 3, m["vb"])
        parts.append((kc, kz, ks, vc, vz, vs, hole, torch.where(hole, K[b], K[b].new_zeros(())) if m["nsp"] else None))
    return parts


def _rotate_half(x, pos, base):
    """Rotate-half rotation of x [..., t, D] fp32 at integer positions, angles in fp64."""
    f = base ** (-2.0 * torch.arange(D // 2, device=x.device, dtype=torch.float64) / D)
    a = pos.double()[:, None] * f
    c, s = a.cos().float(), a.sin().float()
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([lo * c - hi * s, lo * s + hi * c], -1)


def _prepare_plain(case, seed):
    x = _inputs(case, seed)
    op = case["op"]
    if op == "rope":
        return dict(qkv=x[0], pos=x[1])
    if op == "copy":
        return dict(x=x)
    K, V, q = x
    m = METHODS[case["method"]]
    if op == "chunk":
        T = case["T"]
        ns, tq = _quantized(T, m["R"], case["sink"])
        quant = _quantize(case, K[:, :, ns:ns + tq], V[:, :, ns:ns + tq]) if tq else None
        keep = torch.cat([torch.arange(ns, device="cuda"), torch.arange(ns + tq, T, device="cuda")])
        return dict(quant=quant, rk=K[:, :, keep], rv=V[:, :, keep], k=K[:, :, T:].contiguous(), v=V[:, :, T:].contiguous(),
                    q=q, ns=ns, tq=tq)
    return dict(K=K, V=V, q=q)


def _attend_plain(case, quant, rk, rv, k, v, q, ns, tq):
    """softmax(q.K^T / sqrt(D)).V over sink rows, pages, window rows and, causally, the new tokens; one sequence at a time."""
    m = METHODS[case["method"]]
    B, Hkv, n = k.shape[0], k.shape[1], k.shape[2]
    hg = q.shape[1] // Hkv
    T = rk.shape[2] + tq
    pos = torch.arange(T + n, device=q.device)
    # row j of the new tokens sees the T cached ones and the new ones up to itself
    hidden = torch.arange(T + n, device=q.device)[None, :] > (T + torch.arange(n, device=q.device))[:, None]
    outs = []
    for b in range(B):
        ks, vs = [rk[b, :, :ns].float()], [rv[b, :, :ns].float()]
        if tq:
            kc, kz, kst, vc, vz, vst, hole, val = quant[b]
            kd = (kc.float() * kst.float() + kz.float()).view(Hkv, tq, D)
            ks.append(torch.where(hole, val.float(), kd) if hole is not None else kd)
            vs.append((vc.float() * vst.float() + vz.float()).view(Hkv, tq, D))
        K = torch.cat(ks + [rk[b, :, ns:].float(), k[b].float()], 1)
        V = torch.cat(vs + [rv[b, :, ns:].float(), v[b].float()], 1)
        if m["rope"]:
            K = _rotate_half(K, pos, 10000.0)
        Q = q[b].float().view(Hkv, hg, n, D)
        s = torch.matmul(Q.reshape(Hkv, hg * n, D), K.transpose(1, 2)).view(Hkv, hg, n, T + n) / math.sqrt(D)
        s = s.masked_fill(hidden, -math.inf)
        p = (s - s.amax(-1, keepdim=True)).exp()
        o = torch.matmul(p.view(Hkv, hg * n, T + n), V).view(Hkv, hg, n, D) / p.sum(-1, keepdim=True)
        outs.append(o.reshape(Hkv * hg, n, D).half())
    return torch.stack(outs)


def _frequencies(case):
    """Angle per position of every pair of the rotated part, and the factor on cosine and sine."""
    rot, base, f = case["rot"], case["base"], case["factor"]
    out, gain = [], 1.0
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if case["scaling"] == "linear":
            w /= f
        elif case["scaling"] == "wavelength":  # long waves divided by the factor, short ones kept, a blend between
            turns = case["context"] * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
            w = w / f * (1 - keep) + w * keep
        elif case["scaling"] == "yarn":  # as above, with the blend linear in the pair's index
            def index(beta):
                return rot * math.log(case["context"] / (beta * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), rot - 1)
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w / f * ramp + w * (1 - ramp)
            gain = 0.1 * math.log(f) + 1.0
        out.append(w)
    return torch.tensor(out, dtype=torch.float64, device="cuda"), gain


def _positions(case, pos):
    if isinstance(pos, int):
        return (pos + torch.arange(case["n"], device="cuda", dtype=torch.int64)).expand(case["B"], -1)
    return pos


def _rope_plain(st):
    case = st["case"]
    B, n, Hq, Hkv, rot = case["B"], case["n"], case["Hq"], case["Hkv"], case["rot"]
    w, gain = _frequencies(case)
    a = _positions(case, st["pos"]).double()[..., None] * w
    c, s = (a.cos() * gain).float()[:, :, None], (a.sin() * gain).float()[:, :, None]
    q, k, v = st["qkv"].view(B, n, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=2)
    outs = []
    for x in (q, k):
        y = x.float().clone()
        if case["interleaved"]:
            u, t = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
            y[..., 0:rot:2], y[..., 1:rot:2] = u * c - t * s, u * s + t * c
        else:
            u, t = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
            y[..., :rot // 2], y[..., rot // 2:rot] = u * c - t * s, u * s + t * c
        outs.append(y.half().transpose(1, 2).contiguous())
    outs.append(v.half().transpose(1, 2).contiguous())
    return outs


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "rope":
        return _rope_plain(st)
    if op == "copy":
        pages, wk, wv, idx = st["x"]
        at = idx.long()
        return [pages[at], wk[at], wv[at]]
    if op == "chunk":
        return _attend_plain(case, *(st[x] for x in ("quant", "rk", "rv", "k", "v", "q", "ns", "tq")))
    m = METHODS[case["method"]]
    K, V, q = st["K"], st["V"], st["q"]
    outs = []
    for a, b in _pieces(case):
        ns, tq = _quantized(a, m["R"], case["sink"])
        quant = _quantize(case, K[:, :, ns:ns + tq], V[:, :, ns:ns + tq]) if tq else None
        rk = torch.cat([K[:, :, :ns], K[:, :, ns + tq:a]], 2)
        rv = torch.cat([V[:, :, :ns], V[:, :, ns + tq:a]], 2)
        outs.append(_attend_plain(case, quant, rk, rv, K[:, :, a:b], V[:, :, a:b], q[:, :, a:b], ns, tq))
    n = case["n"]
    ns, tq = _quantized(n, m["R"], case["sink"])
    at = [slice(ns + tq, n)] + ([slice(0, ns)] if ns else [])
    return outs + [x[:, :, a].clone() for x in (K, V) for a in at]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- 64 bits

def _grid64(x16, groups, bits, out_of_range=None):
    """The values that quantized fp16 numbers stand for; `groups` [N][group length] indexes them, result in fp64."""
    top = float(2 ** bits - 1)
    g = x16.reshape(-1)[groups].float()
    skip = None if out_of_range is None else out_of_range.reshape(-1)[groups]
    low = g if skip is None else torch.where(skip, torch.full_like(g, math.inf), g)
    high = g if skip is None else torch.where(skip, torch.full_like(g, -math.inf), g)
    z = low.min(1).values
    span = torch.clamp(high.max(1).values - z, min=0.0)
    z = torch.where(torch.isinf(z), torch.zeros_like(z), z)
    step = torch.nan_to_num(span / top, posinf=0.0).half().float()
    code = torch.round((g - z[:, None]) / torch.where(step > 0, step, torch.ones_like(step))[:, None])
    code = torch.where(step[:, None] > 0, torch.clamp(code, 0.0, top), torch.zeros_like(code))
    val = z.double()[:, None] + step.double()[:, None] * code.double()
    if skip is not None:
        val = torch.where(skip, g.double(), val)
    out = torch.empty(x16.numel(), dtype=torch.float64, device=x16.device)
    out[groups.reshape(-1)] = val.reshape(-1)
    return out.view(x16.shape)


def _stored64(m, Kt, Vt, sink):
    """Keys and values of one (sequence, head) as a cache of these tokens holds them, fp64."""
    T = Kt.shape[0]
    ns, tq = _quantized(T, m["R"], sink)
    K, V = Kt.double(), Vt.double()
    if tq:
        G, dev = m["G"], Kt.device
        big = None
        k16, v16 = Kt[ns:ns + tq].contiguous(), Vt[ns:ns + tq].contiguous()
        if m["nsp"]:
            big = torch.zeros(tq, D, dtype=torch.bool, device=dev)
            left = k16.float().abs()
            for _ in range(m["nsp"]):
                hit = left == left.max(1, keepdim=True).values
                hit &= hit.cumsum(1) == 1
                big |= hit
                left = left.masked_fill(hit, -1.0)
        t = torch.arange(tq, device=dev).view(-1, G)
        per_channel = (t[:, None, :] * D + torch.arange(D, device=dev)[None, :, None]).reshape(-1, G)
        K[ns:ns + tq] = _grid64(k16, per_channel, m["kb"], big)
        V[ns:ns + tq] = _grid64(v16, torch.arange(tq * D, device=dev).view(-1, G), m["vb"])
    return K, V


def _attend64(case, K16, V16, q16, t0, t1):
    """Attention of tokens t0..t1 over a cache of the first t0 and over themselves, fp64, one head group at a time."""
    m = METHODS[case["method"]]
    B, Hkv = K16.shape[:2]
    hg = q16.shape[1] // Hkv
    out = torch.empty(B, q16.shape[1], t1 - t0, D, dtype=torch.float64, device=K16.device)
    limit = torch.arange(t0 + 1, t1 + 1, device=K16.device)
    for b in range(B):
        for h in range(Hkv):
            K, V = _stored64(m, K16[b, h, :t0], V16[b, h, :t0], case["sink"])
            K = torch.cat([K, K16[b, h, t0:t1].double()])
            V = torch.cat([V, V16[b, h, t0:t1].double()])
            if m["rope"]:
                ang = torch.arange(t1, device=K.device, dtype=torch.float64)[:, None] * torch.exp(
                    torch.arange(D // 2, device=K.device, dtype=torch.float64) * (-2.0 * math.log(10000.0) / D))
                z = torch.polar(torch.ones_like(ang), ang) * torch.complex(K[:, :D // 2], K[:, D // 2:])
                K = torch.cat([z.real, z.imag], 1)
            for j in range(hg):
                s = q16[b, h * hg + j].double() @ K.T * D ** -0.5
                s = torch.where(torch.arange(t1, device=K.device)[None] < limit[:, None], s,
                                torch.full((), -math.inf, dtype=torch.float64, device=K.device))
                out[b, h * hg + j] = torch.softmax(s, 1) @ V
    return out


def exact(case, seed):
    op = case["op"]
    x = _inputs(case, seed)
    if op == "copy":
        return [None] + [torch.stack([rows[i] for i in x[3].tolist()]).double() for rows in x[1:3]]
    if op == "chunk":
        K, V, q = x
        return _attend64(case, K, V, q, case["T"], case["T"] + case["n"])
    if op == "step":
        K, V, q = x
        m = METHODS[case["method"]]
        outs = [_attend64(case, K[:, :, :b], V[:, :, :b], q[:, :, a:b], a, b) for a, b in _pieces(case)]
        ns, tq = _quantized(case["n"], m["R"], case["sink"])
        first = [0] if ns else []
        return outs + [t[:, :, a:ns if a < ns else None].double() for t in (K, V) for a in [ns + tq] + first]
    qkv, pos = x
    B, n, Hq, Hkv, rot = case["B"], case["n"], case["Hq"], case["Hkv"], case["rot"]
    w, gain = _frequencies(case)
    turn = _positions(case, pos).double()[:, None, :, None] * w
    turn = torch.polar(torch.full_like(turn, gain), turn)
    outs = []
    for i, x in enumerate(qkv.view(B, n, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=2)):
        y = x.double().permute(0, 2, 1, 3).contiguous()
        if i < 2:
            head = y[..., :rot]
            pair = head.unflatten(-1, (-1, 2)) if case["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_real(turn * torch.view_as_complex(pair.contiguous()))
            z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
            y = torch.cat([z, y[..., rot:]], -1)
        outs.append(y)
    return outs
