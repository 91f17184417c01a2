"""Measured cases of the operators around a quantized KV cache kept in pages.

Three operators, as a serving loop uses them one after another:

  prompt  causal attention of whole prompts (packed sequences, grouped heads)
          on the raw 16-bit queries, keys and values: tq_attend_prompt;
  store   the encoded keys and values of new tokens put into the pages of the
          cache, by slot: tq_paged_store;
  paged   causal attention of a chunk of new tokens (one token when decoding)
          over the pages of quantized keys and values: tq_attend_paged.

Every case is a dict with "op" and the sizes; `run` computes the operator in
elementary torch operations, or, where `own` is true, through the package.
The quantizer's tables (rotation, codebook, QJL matrix) follow from
(d, bits, seed) by the definitions in include/tq.h; the plain form builds
them here from those definitions.
"""
import functools
import math

import numpy as np
import torch

own = False

SEED_K, SEED_V = 0, 1  # the quantizers' seeds: part of the set-up, like weights

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a few chat turns' prompts arriving together: latency counts
        dict(name="prompt short", op="prompt", d=128, heads=32, kv_heads=8, seqs=5, lo=1, hi=90, dtype="bf16"),
        # a prefill batch of requests of very different lengths
        dict(name="prompt ragged", op="prompt", d=128, heads=32, kv_heads=8, seqs=16, lo=90, hi=2011, dtype="bf16"),
        # a small model: head dimension 64, 7 query heads to a KV head, fp16
        dict(name="prompt d64 f16", op="prompt", d=64, heads=14, kv_heads=2, seqs=3, lo=701, hi=4100, dtype="f16"),
        # two long documents
        dict(name="prompt long", op="prompt", d=128, heads=32, kv_heads=8, seqs=2, lo=8192, hi=8192, dtype="bf16"),
        # the new token of each sequence of a decode batch; the batch is padded
        dict(name="store decode", op="store", d=128, kbits=3, kip=True, vbits=4, kv_heads=8, tokens=40, padded=8,
             page=16),
        # the tokens of a prefill batch
        dict(name="store prompt", op="store", d=128, kbits=4, kip=True, vbits=4, kv_heads=8, tokens=16384, padded=0,
             page=64),
        # a small decode batch with short contexts: latency counts
        dict(name="decode small", op="paged", d=128, kbits=4, kip=False, vbits=4, heads=32, kv_heads=8, seqs=4,
             lo=300, hi=1100, new_lo=1, new_hi=1, page=16, dtype="bf16"),
        # one sequence of 131072 keys (the KV-layer workload's shape), decoding
        dict(name="decode one long", op="paged", d=128, kbits=4, kip=True, vbits=4, heads=32, kv_heads=8, seqs=1,
             lo=131072, hi=131072, new_lo=1, new_hi=1, page=64, dtype="bf16"),
        # the decode workload's shape: 32 sequences of up to 32768 keys
        dict(name="decode batch", op="paged", d=128, kbits=4, kip=False, vbits=4, heads=32, kv_heads=8, seqs=32,
             lo=16001, hi=32768, new_lo=1, new_hi=1, page=32, dtype="bf16"),
        # drafted tokens verified together: 5 new tokens a sequence, a small model
        dict(name="verify d64 f16", op="paged", d=64, kbits=3, kip=False, vbits=3, heads=16, kv_heads=4, seqs=16,
             lo=2000, hi=9000, new_lo=5, new_hi=5, page=16, dtype="f16"),
        # a long prompt's next chunk against what is already in the cache
        dict(name="chunk 512", op="paged", d=128, kbits=4, kip=False, vbits=4, heads=32, kv_heads=8, seqs=1,
             lo=16384, hi=16384, new_lo=512, new_hi=512, page=64, dtype="bf16"),
        # a mixed batch: some sequences decode, others bring chunks
        dict(name="chunk mixed", op="paged", d=128, kbits=3, kip=True, vbits=2, heads=32, kv_heads=8, seqs=7,
             lo=333, hi=6000, new_lo=1, new_hi=300, page=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    """What a case costs the plain form, which pads every sequence to the longest."""
    if c["op"] == "store":
        return c["tokens"] * c["kv_heads"] * c["d"]
    if c["op"] == "prompt":
        return c["seqs"] * c["hi"] ** 2 * c["heads"] * c["d"]
    pages = -(-max(c["hi"], c["new_hi"]) // c["page"]) * c["page"]
    return c["seqs"] * pages * c["d"] * (20 * c["kv_heads"] + c["new_hi"] * c["heads"])


def draw(rng):
    op = rng.choice(("prompt", "store", "paged", "paged"))
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        d, kv_heads, group = rng.choice((64, 128)), rng.choice((1, 2, 4, 5, 8)), rng.choice((1, 2, 3, 4, 6, 7, 8, 16))
        kbits, kip, vbits = rng.randint(2, 4), rng.random() < 0.5, rng.randint(2, 4)
        page = 16 * rng.choice((1, 2, 3, 4, 8))
        dtype = rng.choice(("bf16", "bf16", "f16"))
        if op == "prompt":
            hi = _log_int(rng, 16, 8192)
            c = dict(op=op, d=d, heads=kv_heads * group, kv_heads=kv_heads, seqs=_log_int(rng, 1, 24),
                     lo=_log_int(rng, 1, hi), hi=hi, dtype=dtype)
        elif op == "store":
            tokens = _log_int(rng, 1, 16384)
            c = dict(op=op, d=d, kbits=kbits, kip=kip, vbits=vbits, kv_heads=kv_heads, tokens=tokens,
                     padded=rng.randint(0, tokens // 4), page=page)
        else:
            hi = _log_int(rng, 20, 65536)
            new_hi = rng.choice((1, 1, 1, _log_int(rng, 2, 16), _log_int(rng, 16, 600)))
            new_hi = min(new_hi, hi)
            c = dict(op=op, d=d, kbits=kbits, kip=kip, vbits=vbits, heads=kv_heads * group, kv_heads=kv_heads,
                     seqs=_log_int(rng, 1, 40), lo=max(new_hi, _log_int(rng, 1, hi)), hi=hi,
                     new_lo=rng.choice((1, new_hi)), new_hi=new_hi, page=page, dtype=dtype)
        if _cost(c) <= most:
            return c


def _spread(lo, hi, n, step):
    """n whole numbers over [lo, hi], the last of them hi, in an irregular order that the case alone fixes."""
    return [lo + int((hi - lo) * ((i * step) % 1.0) + 0.5) for i in range(1, n)] + [hi]


def _lens(c):
    return _spread(c["lo"], c["hi"], c["seqs"], 0.6180339887)


def _news(c):
    return [min(n, k) for n, k in zip(_spread(c["new_lo"], c["new_hi"], c["seqs"], 0.7548776662), _lens(c))]


# ---------------------------------------------------------------- the quantizers' tables

def _mix64(z):
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


def _splitmix(state, k):
    """Outputs k (an array of counters) of SplitMix64 started from `state`."""
    with np.errstate(over="ignore"):
        return _mix64(np.uint64(state) + (k.astype(np.uint64) + np.uint64(1)) * np.uint64(0x9E3779B97F4A7C15))


def _stream_key(seed, stream):
    return int(_splitmix(seed, np.array([stream]))[0])


def _signs(seed, stream, d):
    """The +-1 diagonal number `stream` of the rotation, by bit 0 of each draw."""
    return np.where(_splitmix(_stream_key(seed, stream), np.arange(d)) & np.uint64(1), -1.0, 1.0)


def _rotation(seed, d):
    """R = H D3 H D2 H D1 with the orthonormal Walsh-Hadamard matrix H."""
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    h = h / math.sqrt(d)
    r = np.eye(d)
    for stream in range(3):
        r = h @ (_signs(seed, stream, d)[:, None] * r)
    return r


def _centroids(d, w):
    """Lloyd-Max levels of the density ~ (1 - x^2)^((d-3)/2): the fixed point of bin means and midpoints."""
    t, g = np.polynomial.legendre.leggauss(400)
    top = min(1.0, 9.0 / math.sqrt(d))  # the density beyond is below 1e-17 of its peak
    cen = np.linspace(-1, 1, 2 ** w + 2)[1:-1] * 2.5 / math.sqrt(d)
    for _ in range(20000):
        edge = np.concatenate([[-top], (cen[1:] + cen[:-1]) / 2, [top]])
        half, mid = (edge[1:] - edge[:-1]) / 2, (edge[1:] + edge[:-1]) / 2
        x = mid[:, None] + half[:, None] * t[None]
        f = g[None] * np.exp(0.5 * (d - 3) * np.log1p(-np.minimum(x * x, 1 - 1e-12)))
        new = (f * x).sum(1) / f.sum(1)
        new = (new - new[::-1]) / 2
        if np.abs(new - cen).max() < 1e-15:
            break
        cen = new
    return new


def _qjl(seed, d):
    """S: N(0,1) by Box-Muller (cosine branch) from stream 3, rounded to fp16."""
    w = _splitmix(_stream_key(seed, 3), np.arange(2 * d * d)) >> np.uint64(11)
    u1, u2 = (w[0::2].astype(np.float64) + 1) * 2.0 ** -53, w[1::2].astype(np.float64) * 2.0 ** -53
    return (np.sqrt(-2 * np.log(u1)) * np.cos(2 * np.pi * u2)).astype(np.float16).astype(np.float64).reshape(d, d)


@functools.lru_cache(maxsize=None)
def _tables(d, bits, ip, seed):
    """The quantizer as a program without the package would hold it, in 64 bits."""
    w = bits - 1 if ip else bits
    pos = np.zeros((32, w), dtype=np.int64)  # word * 32 + bit of each bit of the code of coordinate i of 32
    for i in range(32):
        for b in range(w):
            pos[i, b] = (i if w == 1 else (i // 16) * 32 + 4 * (i % 8) + 2 * ((i // 8) % 2) + b if w == 2
                         else ((i // 8) * 32 + 4 * (i % 8) + b if i < 24 else (2 - b) * 32 + 4 * (i - 24) + 3)
                         if w == 3 else (i // 8) * 32 + 4 * (i % 8) + b)
    return dict(d=d, w=w, ip=ip, pos=pos, R=torch.from_numpy(_rotation(seed, d)).cuda(),
                c=torch.from_numpy(_centroids(d, w)).cuda(),
                S=torch.from_numpy(_qjl(seed, d)).cuda() if ip else None, kappa=math.sqrt(math.pi / 2) / d)


@functools.lru_cache(maxsize=None)
def _handle(d, bits, ip, seed):
    """The package's quantizer, kept by a user's program for as long as its cache lives."""
    import online_vector_quantization_tq_b200 as tq
    return tq.tq_codebook(d, bits, seed=seed) if ip else tq.tq_codebook_mse(d, bits, seed=seed)


def _encode(t, x):
    """Packed codes, sign bits and norms of the rows of x (fp32), as include/tq.h defines them."""
    d, w = t["d"], t["w"]
    n = x.shape[0]
    norm = x.norm(dim=1)
    u = (x / norm.clamp_min(1e-30)[:, None]) @ t["R"].float().T
    c = t["c"].float()
    code = torch.bucketize(u, (c[1:] + c[:-1]) / 2)
    r = u - c[code]
    code = code.view(n, d // 32, 32)
    words = torch.zeros(n, d // 32, w, dtype=torch.int64, device=x.device)
    for b in range(w):
        for k in range(w):
            here = [i for i in range(32) if t["pos"][i, b] // 32 == k]
            if here:
                shift = torch.tensor([int(t["pos"][i, b]) % 32 for i in here], device=x.device)
                words[:, :, k] += (((code[:, :, here] >> b) & 1) << shift).sum(2)
    codes = (words & 0xFFFFFFFF).to(torch.uint32).view(torch.uint8).view(n, w * d // 8)
    signs = torch.empty(n, 0, dtype=torch.uint8, device=x.device)
    if t["ip"]:
        bit = (r @ t["S"].float().T >= 0).view(n, d // 8, 8).to(torch.uint8)
        signs = (bit << torch.arange(8, device=x.device, dtype=torch.uint8)).sum(2, dtype=torch.uint8)
    return codes, signs, torch.stack([norm, r.norm(dim=1)], 1)


def _encode_rows(t, rows, gen, values):
    """`rows` encoded keys (four channels x10, the KV-layer workload's law) or values (rows scaled by 1/4 to 4)."""
    got = []
    for at in range(0, rows, 1 << 19):
        x = torch.randn(min(1 << 19, rows - at), t["d"], device="cuda", generator=gen)
        if values:
            x *= torch.exp((torch.rand(x.shape[0], 1, device="cuda", generator=gen) * 2 - 1) * math.log(4.0))
        else:
            x[:, 3::t["d"] // 4] *= 10.0
        got.append(_encode(t, x))
    return [torch.cat(p) for p in zip(*got)]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    d = case["d"]
    s = dict(op=case["op"], d=d, kv_heads=case["kv_heads"], scale=1.0 / math.sqrt(d))
    if case["op"] == "prompt":
        lens, dt = _lens(case), DTYPES[case["dtype"]]
        total, hq, hk = sum(lens), case["heads"], case["kv_heads"]
        # queries, keys and values side by side, as one projection leaves them
        qkv = torch.randn(total, (hq + 2 * hk) * d, device="cuda", generator=gen)
        # heads attend more or less sharply
        sharp = torch.exp2(torch.rand(hq, device="cuda", generator=gen) * 3 - 1).repeat_interleave(d)
        qkv[:, : hq * d] *= sharp
        qkv = qkv.to(dt)
        s.update(heads=hq, y=qkv[:, : hq * d], k=qkv[:, hq * d: (hq + hk) * d], v=qkv[:, (hq + hk) * d:],
                 cu=torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda"),
                 seqs=len(lens), longest=max(lens), q=_handle(d, 4, False, SEED_K) if own else None)
        return s
    s.update(tk=_tables(d, case["kbits"], case["kip"], SEED_K), tv=_tables(d, case["vbits"], False, SEED_V),
             qk=_handle(d, case["kbits"], case["kip"], SEED_K) if own else None,
             qv=_handle(d, case["vbits"], False, SEED_V) if own else None, page=case["page"])
    hk, ps = case["kv_heads"], case["page"]
    if case["op"] == "store":
        tokens = case["tokens"]
        npages = -(-tokens // ps) + 3
        s["rows"] = [_encode_rows(s[t], tokens * hk, gen, t == "tv") for t in ("tk", "tv")]
        slots = torch.randperm(npages * ps, device="cuda", generator=gen)[:tokens]
        if case["padded"]:  # a padded batch's rows have no slot
            slots[torch.randperm(tokens, device="cuda", generator=gen)[: case["padded"]]] = -1
        s["slots"] = slots
        s["pages"] = [[torch.randint(0, 256, (npages, hk, ps, p.shape[1]), device="cuda", generator=gen,
                                     dtype=torch.uint8) if p.dtype == torch.uint8 else
                       torch.randn(npages, hk, ps, 2, device="cuda", generator=gen) for p in rows]
                      for rows in s["rows"]]
    else:
        lens, news, hq = _lens(case), _news(case), case["heads"]
        need = [-(-n // ps) for n in lens]
        npages = sum(need) + 5
        order = torch.randperm(npages, device="cuda", generator=gen)
        table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at: at + n].to(torch.int32)
            at += n
        used = torch.zeros(npages, ps, dtype=torch.bool, device="cuda")
        for i, n in enumerate(lens):
            used[table[i, : need[i]].long()] = True
            if n % ps:
                used[int(table[i, need[i] - 1]), n % ps:] = False
        s["pages"] = []
        for t in ("tk", "tv"):
            p = [x.view(npages, hk, ps, x.shape[1]) for x in _encode_rows(s[t], npages * hk * ps, gen, t == "tv")]
            # what no token has been written to holds what the memory held before
            p[2].masked_fill_(~used[:, None, :, None], float("nan"))
            s["pages"].append(p)
        y = torch.randn(sum(news), hq, d, device="cuda", generator=gen)
        y *= torch.exp2(torch.rand(hq, 1, device="cuda", generator=gen) * 3 - 2)
        s.update(heads=hq, y=y.view(sum(news), hq * d).to(DTYPES[case["dtype"]]), table=table, longest=max(lens),
                 most_new=max(news), seqs=len(lens),
                 q_start=torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device="cuda"),
                 kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if own:
        import online_vector_quantization_tq_b200 as tq
        s["caches"] = [tq.PagedCache(*p) for p in s["pages"]]
        if case["op"] == "store":
            s["encs"] = [tq.Encoded(*p) for p in s["rows"]]
        else:
            s["ws"] = tq.attend_paged_workspace(s["qk"], s["qv"], s["y"].shape[0], s["seqs"], s["heads"],
                                                s["kv_heads"], s["most_new"], s["table"].shape[1], s["page"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        import online_vector_quantization_tq_b200 as tq
        if s["op"] == "prompt":
            return tq.tq_attend_prompt(s["q"], s["y"], s["k"], s["v"], s["cu"], s["scale"])
        if s["op"] == "store":
            tq.tq_paged_store(s["qk"], s["qv"], s["encs"][0], s["encs"][1], s["slots"], s["caches"][0],
                              s["caches"][1])
            return s["pages"]
        return tq.tq_attend_paged(s["qk"], s["qv"], s["y"], s["q_start"], s["caches"][0], s["caches"][1],
                                  s["table"], s["kv_len"], s["most_new"], s["scale"], workspace=s["ws"])
    return {"prompt": _prompt, "store": _store, "paged": _paged}[s["op"]](s)


def _softmax_(x):
    """exp(x - max) over the last axis and its sums, in place; rows of -inf alone give zeros."""
    top = x.amax(-1, keepdim=True).nan_to_num_(neginf=0.0)
    x.sub_(top).exp_()
    return x, x.sum(-1, keepdim=True)


def _prompt(s):
    d, hq, hk, b, n = s["d"], s["heads"], s["kv_heads"], s["seqs"], s["longest"]
    cu = s["cu"].long()
    lens, at = cu[1:] - cu[:-1], torch.arange(n, device="cuda")
    row = (cu[:-1, None] + at).clamp_(max=s["y"].shape[0] - 1)  # [b, n]
    real = at < lens[:, None]
    q = s["y"][row].float().view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    k, v = (s[x][row].float().view(b, n, hk, d).transpose(1, 2) for x in "kv")
    v = v.masked_fill(~real[:, None, :, None], 0.0)
    x = (q * s["scale"] @ k.transpose(2, 3)).view(b, hk, hq // hk, n, n)
    x.masked_fill_((at > at[:, None]) | ~real[:, None, None, None], -math.inf)
    x, total = _softmax_(x)
    o = (x.view(b, hk, -1, n) @ v).view(b, hk, hq // hk, n, d) / total
    return o.permute(0, 3, 1, 2, 4).reshape(b * n, hq * d)[real.view(-1)].to(s["y"].dtype)


def _store(s):
    there = s["slots"] >= 0
    page, at = s["slots"][there] // s["page"], s["slots"][there] % s["page"]
    for i in (0, 1):
        for j in (0, 1, 2):
            p, rows = s["pages"][i][j], s["rows"][i][j]
            p[page, :, at] = rows.view(len(there), s["kv_heads"], p.shape[3])[there]
    return s["pages"]


def _decode(t, pages, table):
    """Levels [b, heads, keys, d], norms and sign bits of the keys of each sequence, in their order."""
    d, w = t["d"], t["w"]
    at = table.long().clamp_min(0)
    codes, signs, norms = (p[at].transpose(1, 2).flatten(2, 3) for p in pages)
    words = codes.view(torch.int32).view(*codes.shape[:3], d // 32, w)
    code = None
    for b in range(w):
        word = words[..., torch.from_numpy(t["pos"][:, b] // 32).cuda()]
        bit = ((word >> torch.from_numpy(t["pos"][:, b] % 32).int().cuda()) & 1) << b
        code = bit if code is None else code.add_(bit)
    c = t["c"].float().index_select(0, code.view(-1)).view(*codes.shape[:3], d)
    if not t["ip"]:
        return c, norms, None
    bit = (signs[..., None] >> torch.arange(8, dtype=torch.uint8, device="cuda")) & 1
    return c, norms, bit.view(*signs.shape[:3], d).float().mul_(2).sub_(1)


def _paged(s):
    d, hq, hk, b, n = s["d"], s["heads"], s["kv_heads"], s["seqs"], s["most_new"]
    start = s["q_start"].long()
    new, at = start[1:] - start[:-1], torch.arange(n, device="cuda")
    row = (start[:-1, None] + at).clamp_(max=s["y"].shape[0] - 1)
    real = at < new[:, None]
    q = s["y"][row].float().view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    q = q @ s["tk"]["R"].float().T * s["scale"]
    c, norm, sign = _decode(s["tk"], s["pages"][0], s["table"])
    x = q @ c.transpose(2, 3)
    if sign is not None:
        p = q @ s["tk"]["S"].float().T * s["tk"]["kappa"]
        x += p @ sign.transpose(2, 3) * norm[..., None, :, 1]
    x *= norm[..., None, :, 0]
    m = x.shape[3]
    last = (s["kv_len"].long() - new)[:, None] + at  # the last key that each new token sees
    hidden = torch.arange(m, device="cuda") > last[..., None]
    x = x.view(b, hk, hq // hk, n, m).masked_fill_(hidden[:, None, None], -math.inf)
    del c, norm, sign
    x, total = _softmax_(x)
    c, norm, _ = _decode(s["tv"], s["pages"][1], s["table"])
    norm = norm[..., :1].masked_fill(torch.arange(m, device="cuda")[:, None] >= s["kv_len"][:, None, None, None], 0.0)
    o = (x.view(b, hk, -1, m) @ c.mul_(norm)).view(b, hk, hq // hk, n, d)
    o = torch.where(total > 0, o / total, 0.0) @ s["tv"]["R"].float()
    return o.permute(0, 3, 1, 2, 4).reshape(b * n, hq * d)[real.view(-1)].to(s["y"].dtype)


# ---------------------------------------------------------------- work

def work(case):
    d, hk = case["d"], case["kv_heads"]
    if case["op"] == "prompt":
        lens, hq = _lens(case), case["heads"]
        return {"bytes": sum(lens) * 2 * d * (2 * hq + 2 * hk) + 4 * (len(lens) + 1),
                "flops": sum(2 * 2 * d * hq * (n * (n + 1) // 2) for n in lens)}
    kw = case["kbits"] - 1 if case["kip"] else case["kbits"]
    kbytes, vbytes = kw * d // 8 + (d // 8 if case["kip"] else 0) + 8, case["vbits"] * d // 8 + 8
    if case["op"] == "store":
        return {"bytes": 8 * case["tokens"] + 2 * (case["tokens"] - case["padded"]) * hk * (kbytes + vbytes),
                "flops": 0}
    lens, news, hq = _lens(case), _news(case), case["heads"]
    pairs = sum(n * k - n * (n - 1) // 2 for n, k in zip(news, lens))  # (new token, key) pairs that attend
    return {"bytes": sum(lens) * hk * (kbytes + vbytes) + sum(news) * hq * d * 2 * 2 +
            4 * (sum(-(-k // case["page"]) for k in lens) + 2 * len(lens) + 1),
            "flops": 2 * d * hq * pairs * (3 if case["kip"] else 2)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        return None
    d, hq, hk = case["d"], case["heads"], case["kv_heads"]
    group = hq // hk
    out = torch.empty(s["y"].shape[0], hq, d, dtype=torch.float64, device="cuda")
    y = s["y"].double().view(-1, hq, d)
    if case["op"] == "prompt":
        at = 0
        for n in _lens(case):
            for h in range(hq):
                k, v = (s[x][at: at + n, h // group * d: (h // group + 1) * d].double() for x in "kv")
                for i in range(0, n, 2048):
                    x = y[at + i: at + min(n, i + 2048), h] @ k.T * s["scale"]
                    x = x.masked_fill(torch.ones_like(x, dtype=torch.bool).triu(i + 1), -math.inf)
                    out[at + i: at + min(n, i + 2048), h] = torch.softmax(x, 1) @ v
            at += n
        return out.view(-1, hq * d)
    at = 0
    for b, (n, m) in enumerate(zip(_news(case), _lens(case))):
        seen = s["table"][b, : -(-m // case["page"])].tolist()
        for h in range(hk):
            k = _rebuilt(s["tk"], s["pages"][0], seen, h, m)
            v = _rebuilt(s["tv"], s["pages"][1], seen, h, m)
            for i in range(0, n, 128):
                j = min(n, i + 128)
                x = torch.einsum("tgd,kd->tgk", y[at + i: at + j, h * group: (h + 1) * group], k) * s["scale"]
                hide = torch.ones(j - i, m, dtype=torch.bool, device="cuda").triu(m - n + i + 1)
                x = x.masked_fill(hide[:, None], -math.inf)
                out[at + i: at + j, h * group: (h + 1) * group] = torch.einsum("tgk,kd->tgd", torch.softmax(x, 2), v)
        at += n
    return out.view(-1, hq * d)


def _rebuilt(t, pages, seen, head, count):
    """The vectors that a sequence's encoded rows of one head stand for: norm R^T (c + gamma kappa S^T sign)."""
    codes, signs, norms = (p[seen, head].flatten(0, 1)[:count] for p in pages)
    u = torch.zeros(count, t["d"], dtype=torch.int64, device="cuda")
    size = 4 * t["w"]  # bytes of 32 coordinates
    for i in range(32):
        for b in range(t["w"]):
            p = int(t["pos"][i, b])
            u[:, i::32] += ((codes[:, p // 8:: size] >> (p % 8)) & 1).long() << b
    u = t["c"][u]
    if t["ip"]:
        sign = torch.stack([((signs >> i) & 1).double() * 2 - 1 for i in range(8)], 2).view(count, t["d"])
        u = u + norms[:, 1:].double() * t["kappa"] * (sign @ t["S"])
    return norms[:, :1].double() * (u @ t["R"])
