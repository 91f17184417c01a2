"""Causal attention of packed prompts on the GPU against plain fp64, with
bounds that follow from the roundings: 16-bit inputs are exact, logits and
sums are fp32, each weight is rounded once to 16 bits and the output once."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
F = 2.0 ** -23  # an fp32 add that may truncate


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from online_vector_quantization_tq_b200 import build
    build.build()
    import online_vector_quantization_tq_b200 as pkg
    pkg.lib()
    return pkg


_MADE = {}


def handle(tq, d):
    if d not in _MADE:
        _MADE[d] = tq.tq_codebook_mse(d, 4)
    return _MADE[d]


def reference(y, k, v, scale, dtype):
    """One sequence and head in fp64: the output and, per coordinate, the most
    that the kernel's roundings can move it."""
    n, d = y.shape
    u = torch.finfo(DT[dtype]).eps / 2
    y, k, v = y.double(), k.double(), v.double()
    x = scale * (y @ k.T)
    # fp32 sums of d exact products; the exponent's factor, its difference from the reference (both rounded)
    err = abs(scale) * (y.abs() @ k.abs().T) * (d / 8 + 2) * F
    hide = torch.ones(n, n, dtype=torch.bool, device=y.device).triu(1)
    x = x.masked_fill(hide, -math.inf)
    top = x.amax(1, keepdim=True)
    err = err + (x.abs().masked_fill(hide, 0.0) + top.abs() + 10) * 4 * F
    w = torch.exp(x - top)
    total = w.sum(1, keepdim=True)
    w = w / total
    # 2^x: the approximate instruction 2^-22, the polynomial 2^-13.2 (bf16) or 2^-18.4
    eps = torch.expm1(err) + 2.0 ** -22 + (2.0 ** -13.2 if dtype == "bf16" else 2.0 ** -18.4)
    eps = eps.masked_fill(hide, 0.0)
    mean = (w * eps).sum(1, keepdim=True)
    rel = (1 + eps) / (1 - mean).clamp_min(0.1) * (1 + u) - 1 + (n / 8 + 40) * F
    # an fp16 weight below 2^-14 is rounded absolutely (the largest weight is at least 1 before the division);
    # weights below 2^-126 may be lost
    small = (2.0 ** -25 if dtype == "f16" else 2.0 ** -126) / total
    out = w @ v
    bound = (w * rel) @ v.abs() + small * (v.abs().cumsum(0))
    tiny = 2.0 ** -25 if dtype == "f16" else 2.0 ** -133
    return out, bound + (out.abs() + bound) * u + tiny


def make(total, heads, kv_heads, d, dtype, seed, sharp=1.0):
    """One projection's output: queries, keys and values as views of it."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(total, (heads + 2 * kv_heads) * d + 8, generator=g)
    x[:, : heads * d] *= sharp
    x = x.to(DT[dtype]).cuda()
    return x[:, : heads * d], x[:, heads * d: (heads + kv_heads) * d], x[:, (heads + kv_heads) * d: -8]


def check(out, y, k, v, starts, lens, heads, kv_heads, d, scale, dtype):
    worst, group = 0.0, heads // kv_heads
    for s, n in zip(starts, lens):
        if n == 0:
            continue
        for h in range(heads):
            kh = slice(h // group * d, (h // group + 1) * d)
            ref, bound = reference(y[s:s + n, h * d:(h + 1) * d], k[s:s + n, kh], v[s:s + n, kh], scale, dtype)
            got = out[s:s + n, h * d:(h + 1) * d].double()
            assert bool(torch.isfinite(got).all()), f"sequence at {s}, head {h}"
            ratio = float(((got - ref).abs() / bound).max())
            assert ratio <= 1.0, f"sequence of {n} at {s}, head {h}: {ratio:.2f} of the bound"
            worst = max(worst, ratio)
    return worst


def run_case(tq, d, kv_heads, group, lens, dtype, seed, scale=None, sharp=1.0, gap=3):
    """`gap` tokens that belong to no sequence stand before the first and
    behind the last; out is a wider tensor's view."""
    heads = kv_heads * group
    starts = [gap + sum(lens[:i]) for i in range(len(lens) + 1)]
    total = starts[-1] + gap
    y, k, v = make(total, heads, kv_heads, d, dtype, seed, sharp)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    wide = torch.full((total, heads * d + 8), -7.0, dtype=DT[dtype], device="cuda")
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    q = handle(tq, d)
    tq.tq_attend_prompt(q, y, k, v, cu, scale, out=wide[:, : heads * d])
    tq.tq_sync_check(q)
    assert bool((wide[:, heads * d:] == -7.0).all())
    assert bool((wide[:gap] == -7.0).all()) and bool((wide[starts[-1]:] == -7.0).all())
    worst = check(wide, y, k, v, starts, lens, heads, kv_heads, d, scale, dtype)
    print(f"d={d} heads={heads}/{kv_heads} {dtype}: worst {worst:.3f} of the bound")


LENS = [1, 0, 2, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1, 513]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kv_heads,group", [(2, 1), (1, 4)])
def test_lengths_about_a_tile(tq, d, dtype, kv_heads, group):
    run_case(tq, d, kv_heads, group, LENS, dtype, seed=d + group)


@pytest.mark.parametrize("kv_heads,group,dtype", [(1, 3, "f16"), (3, 2, "bf16"), (2, 7, "bf16"), (1, 16, "f16"),
                                                  (1, 65, "bf16"), (1, 128, "bf16")])
def test_head_layouts(tq, kv_heads, group, dtype):
    """Groups that do and do not divide a tile's rows, up to one token a tile."""
    run_case(tq, 128, kv_heads, group, [5, 130, 33], dtype, seed=group)
    run_case(tq, 64, kv_heads, group, [140, 3], dtype, seed=group + 1)


def test_long_prompts_and_sharp_heads(tq):
    run_case(tq, 128, 1, 4, [3000, 1111], "bf16", seed=1)
    run_case(tq, 128, 1, 2, [2500], "bf16", seed=2, sharp=6.0)  # one key has most of the weight
    run_case(tq, 64, 1, 7, [2049], "f16", seed=3, sharp=4.0)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-3, 0.7])
def test_scales(tq, scale):
    run_case(tq, 128, 1, 2, [200, 64], "bf16", seed=9, scale=scale)
    run_case(tq, 64, 1, 2, [200, 64], "f16", seed=9, scale=scale)


def test_rising_maximum(tq):
    """Logits that grow with the key's position by more than the reference's
    slack from tile to tile: the output is rescaled again and again."""
    d, n = 128, 1500
    y, k, v = make(n, 1, 1, d, "bf16", 5)
    k = k.clone()
    y = (y * 0.1 + 1.0).to(torch.bfloat16)
    k += torch.linspace(0, 12, n, device="cuda")[:, None].to(torch.bfloat16)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = tq.tq_attend_prompt(handle(tq, d), y, k, v, cu, 0.1)
    check(out, y, k, v, [0], [n], 1, 1, d, 0.1, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_what_a_token_does_not_see(tq, dtype, what):
    """NaN and infinities in the keys and values of another sequence, and of a
    later token of the same one, leave a token's output as it was, bit for bit;
    the tokens that see them are not finite."""
    d, lens, group = 128, [70, 200, 40], 4
    y, k, v = make(sum(lens), group, 1, d, dtype, 11)
    cu = torch.tensor([0, 70, 270, 310], dtype=torch.int32, device="cuda")
    q = handle(tq, d)
    clean = tq.tq_attend_prompt(q, y, k, v, cu, 0.1)
    for at in (70 + 0, 70 + 63, 70 + 64, 70 + 130, 70 + 199):
        for both in (False, True):
            k2, v2 = k.clone(), v.clone()
            v2[at, 5] = what
            if both:
                k2[at] = what
            out = tq.tq_attend_prompt(q, y, k2, v2, cu, 0.1)
            same = torch.ones(310, dtype=torch.bool, device="cuda")
            same[at:270] = False
            assert torch.equal(out[same], clean[same])
            assert not bool(torch.isfinite(out[at:270].view(-1, group, d)[:, :, 5]).any())
            if not both:
                rest = [c for c in range(d) if c != 5]
                assert torch.equal(out.view(310, group, d)[:, :, rest], clean.view(310, group, d)[:, :, rest])
                if not math.isnan(what):
                    assert bool((out[at:270].view(-1, group, d)[:, :, 5] == what).all())


def test_replayed_graph_reads_new_lengths(tq):
    """Captured once, replayed with other lengths: as a fresh call, bit for bit,
    also on another stream; two captured calls share nothing."""
    d, total = 128, 700
    y, k, v = make(total, 8, 2, d, "bf16", 12)
    q = handle(tq, d)
    cu = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    outs, graphs = [torch.zeros_like(y) for _ in range(2)], []
    tq.tq_attend_prompt(q, y, k, v, cu, 0.09)
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.tq_attend_prompt(q, y, k, v, cu, 0.09, out=outs[i])
        graphs.append(g)
    for cut, end in ((300, 700), (0, 700), (699, 700), (128, 500)):
        cu.copy_(torch.tensor([0, cut, end], dtype=torch.int32))
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        ref = tq.tq_attend_prompt(q, y, k, v, cu, 0.09, out=torch.zeros_like(y))
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
        assert bool((ref[end:] == 0).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = tq.tq_attend_prompt(q, y, k, v, cu, 0.09, out=torch.zeros_like(y), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, ref)


def test_bad_lengths_stay_in_bounds(tq):
    """Lengths that break the rules read and write nothing outside the arrays."""
    d, total = 128, 300
    y, k, v = make(total, 4, 1, d, "bf16", 13)
    q = handle(tq, d)
    wide = torch.full((total + 8, 4 * d), -7.0, dtype=torch.bfloat16, device="cuda")
    for cu in ([-5, 100], [0, 10 ** 9], [200, 100], [-2 ** 31, 2 ** 31 - 1], [299, 301]):
        tq.tq_attend_prompt(q, y, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), 0.1, out=wide[:total])
        tq.tq_sync_check(q)
        assert bool((wide[total:] == -7.0).all())


def test_many_sequences(tq):
    """More sequences than a warp has lanes, most of them empty."""
    lens = [(7 * i) % 5 * ((i * 13) % 11) for i in range(150)]
    run_case(tq, 64, 1, 2, lens, "bf16", seed=14)


def test_argument_checks(tq):
    d = 128
    y, k, v = make(10, 4, 2, d, "bf16", 15)
    q = handle(tq, d)
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    out = torch.full((10, 4 * d), 3.0, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(scale=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(tq.TQError):
            tq.tq_attend_prompt(q, y, k, v, cu, out=out, **bad)
    x = torch.zeros(10, 4 * d + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tq.TQError):  # rows that are not 16-byte aligned
        tq.tq_attend_prompt(q, x[:, : 4 * d], k, v, cu, 0.1, out=out)
    with pytest.raises(TypeError):
        tq.tq_attend_prompt(q, y.float(), k.float(), v.float(), cu, 0.1)
    with pytest.raises(TypeError):
        tq.tq_attend_prompt(q, y, k.half(), v, cu, 0.1, out=out)
    with pytest.raises(TypeError):
        tq.tq_attend_prompt(q, y, k, v, cu.long(), 0.1, out=out)
    with pytest.raises(ValueError):
        tq.tq_attend_prompt(q, y[:, : 3 * d], k, v, cu, 0.1)
    with pytest.raises(ValueError):
        tq.tq_attend_prompt(q, y, k[:9], v, cu, 0.1, out=out)
    with pytest.raises(ValueError):
        tq.tq_attend_prompt(q, y, k, v, cu.cpu(), 0.1, out=out)
    with pytest.raises(ValueError):
        tq.tq_attend_prompt(q, y, k, v, cu, 0.1, out=out[:5])
    assert bool((out == 3.0).all())
    none = torch.empty(0, 4 * d, dtype=torch.bfloat16, device="cuda")
    assert tq.tq_attend_prompt(q, none, none[:, : 2 * d], none[:, : 2 * d], cu[:1], 0.1).shape == (0, 4 * d)


@pytest.mark.parametrize("d,kv_heads,group", [(64, 8, 1), (128, 8, 2), (64, 5, 7)])
def test_more_items_than_blocks(tq, d, kv_heads, group):
    """Several rounds of work items to a block, of one and of two tiles."""
    run_case(tq, d, kv_heads, group, [1 + (97 * i) % 640 for i in range(24)], "bf16", seed=41 + d)


def test_bad_values_among_many_items(tq):
    """Infinities and NaN in some sequences of a batch that takes several rounds:
    every other sequence, and every earlier token, keeps its result, bit for bit."""
    d, heads = 64, 8
    lens = [(53 * i) % 400 + 1 for i in range(30)]
    starts = [sum(lens[:i]) for i in range(len(lens) + 1)]
    y, k, v = make(starts[-1], heads, heads, d, "bf16", 43)
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    q = handle(tq, d)
    clean = tq.tq_attend_prompt(q, y, k, v, cu, 0.125)
    same = torch.ones(starts[-1], dtype=torch.bool, device="cuda")
    v2 = v.clone()
    for i in range(0, 30, 4):
        at = starts[i] + lens[i] // 2
        v2[at] = math.nan if i % 8 else math.inf
        same[at: starts[i + 1]] = False
    for _ in range(3):
        out = tq.tq_attend_prompt(q, y, k, v2, cu, 0.125)
        assert torch.equal(out[same], clean[same])
        assert not bool(torch.isfinite(out[~same]).any())
