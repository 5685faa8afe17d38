"""Token sampling against the float64 definition: the token is equal in every
row, whatever the sizes, strides, cut-offs and masks; logp within float32."""
import ctypes
import math

import numpy as np
import pytest
import torch

from grpo_loss_gb300 import _lib as L
from tests.operator_reference import f64, sample_row

# float32 weights at worst: 2^-22 of a weight for its exponential, 2^-23 |y| for
# its argument, |y| <= 40 binary orders; and the rounding of logp itself
LOGP_ABS = 2.0 ** -22 + 40 * 2.0 ** -23


def check(logits, u, T=None, k=None, p=None, q=None, **kw):
    import grpo_loss_gb300 as G
    rows = logits.shape[0]
    dev = logits.device
    dt = {"temperature": torch.float32, "top_k": torch.int32, "top_p": torch.float32, "min_p": torch.float32}
    par = {n: None if v is None else torch.as_tensor(v, dtype=dt[n], device=dev).expand(rows).contiguous()
           for n, v in zip(dt, (T, k, p, q))}
    tokens, logp = G.sample(logits, u, **par, **kw)
    torch.cuda.synchronize()
    z, un = f64(logits), f64(u)
    cpu = {n: None if v is None else f64(v) for n, v in par.items()}
    off = [1.0, 0, 1.0, 0.0]
    got = tokens.cpu().numpy(), f64(logp)
    for r in range(rows):
        a = [off[i] if cpu[n] is None else cpu[n][r] for i, n in enumerate(dt)]
        tok, lp = sample_row(z[r], un[r], a[0], int(a[1]), a[2], a[3])
        assert got[0][r] == tok, (r, got[0][r], tok, a, un[r])
        if math.isinf(lp):
            assert got[1][r] == lp
        else:
            assert abs(got[1][r] - lp) <= LOGP_ABS + 2.0 ** -24 * abs(lp), (r, got[1][r], lp)
    return tokens, logp


def logits_of(rows, V, dtype, seed, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(rows, V, generator=g, device="cuda") * spread
    return z.to(dtype), torch.rand(rows, generator=g, device="cuda")


PARAMS = {"plain": {}, "temperature": dict(T=0.7), "top_k": dict(k=5), "top_p": dict(p=0.9),
          "min_p": dict(q=0.05), "all": dict(T=1.3, k=40, p=0.8, q=0.01), "greedy": dict(T=0.0),
          "one": dict(k=1, p=0.5), "hot": dict(T=30.0, p=0.99), "cold": dict(T=0.01)}


@pytest.mark.gpu
@pytest.mark.parametrize("par", list(PARAMS), ids=list(PARAMS))
@pytest.mark.parametrize("V", [1, 2, 31, 33, 257, 1000, 4097, 20011, 128256])
def test_sizes_and_cutoffs(V, par):
    for dtype in (torch.float32, torch.bfloat16):
        z, u = logits_of(3 if V > 10000 else 9, V, dtype, V + len(par))
        check(z, u, **PARAMS[par])


@pytest.mark.gpu
@pytest.mark.parametrize("V,rows", [(151936, 2), (201088, 2), (262144, 1), (700001, 2)])
def test_long_rows(V, rows):
    for dtype in (torch.float32, torch.bfloat16):
        z, u = logits_of(rows, V, dtype, 5)
        check(z, u)
        check(z, u, p=0.95, k=1000)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0.0, 0.01, 1.0, 40.0])
def test_flat_and_peaked_rows(spread):
    """Flat rows: every token is a border, and all tie (equal bf16 logits too)."""
    for dtype in (torch.float32, torch.bfloat16):
        z, u = logits_of(24, 5003, dtype, 3, spread)
        check(z, u)
        check(z, u, p=0.5)
        check(z, u, k=700, p=0.75)
        check(z, u, q=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("V,row_of", [(1048572, 1), (524284, 4), (262140, 2)])
def test_flat_rows_that_fill_a_slice(V, row_of):
    """Slices of 131072 equal logits: the most that a bin's 32-bit sum may meet in
    its finer units. (Clusters of 8, 4 and 2 CTAs a row, as few rows as take those.)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 1 if row_of == 1 else sms // row_of
    z = torch.full((rows, V), 1.5, device="cuda")
    u = torch.rand(rows, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    import grpo_loss_gb300 as G
    p = torch.full((rows,), 0.9, device="cuda")
    tokens, logp = G.sample(z, u, top_p=p)
    torch.cuda.synchronize()
    # of n = ceil(0.9 V) equal weights the first whose running sum exceeds u n
    n = math.ceil(float(np.float32(0.9)) * V)
    assert tokens.tolist() == [math.floor(float(x) * n) for x in u.tolist()]
    assert np.all(np.abs(f64(logp) + math.log(V)) <= LOGP_ABS)


@pytest.mark.gpu
@pytest.mark.parametrize("par", [dict(p=0.9), dict(p=0.5, q=1e-4), dict(k=5000), dict(k=900, p=0.97), dict(k=20000, p=0.6, T=1.5),
                                 dict(p=0.99999), dict(p=1e-3), dict(k=1024), dict(k=1025)], ids=str)
@pytest.mark.parametrize("V", [30011, 128256])
def test_cuts_that_keep_many_tokens(V, par):
    """Cuts among thousands of tokens: of one value each (float32) and of many
    ties (bf16); spread-out rows and almost flat ones."""
    for dtype, spread in ((torch.float32, 1.0), (torch.bfloat16, 1.0), (torch.float32, 0.05), (torch.bfloat16, 0.05),
                          (torch.bfloat16, 4.0)):
        z, u = logits_of(2, V, dtype, 31, spread)
        check(z, u, **par)


@pytest.mark.gpu
@pytest.mark.parametrize("par", [{}, dict(p=0.9), dict(k=40, p=0.8, q=0.01, T=0.7), dict(T=0.0), dict(k=3000), dict(q=0.02)],
                         ids=str)
def test_bf16_values_of_every_magnitude(par):
    """Logits far from 1 in either direction, orders apart within a row, zeros of
    both signs, subnormals, masked ones, and rows of one value."""
    V = 30011
    z, u = logits_of(20, V, torch.float32, 41)
    z[0] *= 1e-6
    z[1] *= 100.0                                   # beyond 2^7
    z[2] = z[2] * 100.0 - 2000.0
    z[3] = z[3].abs() * -1e-3
    z[4] *= 1e-36
    z[5, ::2] *= 1e-30                              # too far below the others, and not 0
    z[6, ::2] = 0.0
    z[7, ::2], z[7, 1::4] = 0.0, -0.0
    z[8] = 0.0
    z[9] = -1e-39
    z[10, 1:] = torch.finfo(torch.bfloat16).min
    z[11] = torch.where(z[11] > 0, z[11], -math.inf)
    z[12, :29000] = -math.inf
    z[13] = math.nan
    z[13, ::3] = -math.inf
    z[14, 5::3] = math.nan
    z[15, ::2] = math.inf
    z[16] = -math.inf
    z[16, 30010] = 3e38
    z[17] += 1000.0
    z[18] = 150.0
    z[18, 7] = 1e-30
    check(z.to(torch.bfloat16), u, **par)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spread", [1.0, 4.0])
def test_many_rows_with_parameters_of_their_own(dtype, spread):
    """More rows than SMs, each with other cut-offs, masks among them: rows that
    need one CTA's passes and rows that need more."""
    rows, V = 200, 20011
    z, u = logits_of(rows, V, dtype, 43, spread)
    g = torch.Generator().manual_seed(5)
    pick = lambda *v: torch.tensor(v)[torch.randint(len(v), (rows,), generator=g)]
    z[::9, ::2] = -math.inf
    z[5] = -math.inf
    z[6] = math.nan
    z[7, 11] = math.inf
    z[8] = 0.0
    z[9] *= 1e-8
    check(z, u, T=pick(0.0, 0.3, 0.7, 1.0, 1.0, 1.5), k=pick(0, 0, 0, 1, 20, 256, 257, 3000), p=pick(1.0, 1.0, 0.3, 0.9, 0.95),
          q=pick(0.0, 0.0, 0.05, 1e-4))


@pytest.mark.gpu
@pytest.mark.parametrize("par", [{}, dict(p=0.9), dict(p=0.9, k=200), dict(q=0.004)], ids=str)
def test_many_rows_whose_weights_err_alike(par):
    """One likely token and a floor of equal ones, whose float32 weights are all off in
    the same direction, as far as a product and its factor can be."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows, V = sms + 8, 131072
    for dtype in (torch.bfloat16, torch.float32):
        z = torch.full((rows, V), -7.96875, device="cuda", dtype=dtype)
        z[:, 777] = 0.0
        u = (torch.arange(rows, device="cuda") + 0.5) / rows
        check(z, u, T=1.4333123, **par)


def wanted(z, u, T=1.0, k=0, p=1.0, q=0.0):
    """The definition for all rows at once, in float64 on the GPU (parameters of the
    whole call; no masked rows)."""
    z = z.double()
    w = ((z - z.max(1, keepdim=True).values) / float(np.float32(T))).exp()
    w[w < 2.0 ** -40] = 0.0
    ws, order = torch.sort(z, dim=1, descending=True, stable=True)
    ws = w.gather(1, order)
    ws[ws < float(np.float32(q))] = 0.0
    if k:
        ws[:, k:] = 0.0
    upto = ws.cumsum(1)
    ws[:, 1:][(upto - ws)[:, 1:] >= float(np.float32(p)) * upto[:, -1:]] = 0.0
    upto = torch.zeros_like(w).scatter_(1, order, ws).cumsum(1)
    tokens = (upto <= u.double()[:, None] * upto[:, -1:]).sum(1)
    return tokens.int(), w.gather(1, tokens[:, None])[:, 0].log() - w.sum(1).log()


@pytest.mark.gpu
@pytest.mark.parametrize("par", [{}, dict(p=0.9), dict(p=0.95, q=1e-3), dict(k=50, p=0.9), dict(k=3000, p=0.9, T=0.7)], ids=str)
@pytest.mark.parametrize("V", [40001, 128256])
@pytest.mark.parametrize("rows", [(1, 20), (1, 6), (2, 5), (4, 5), (21, 20)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_number_of_ctas_a_row(dtype, rows, V, par):
    """From rows that take a cluster each to rows for every SM, in shares of the SMs:
    clusters of 8, 4 and 2 CTAs, large ones and small, slices kept and read again."""
    import grpo_loss_gb300 as G
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms * rows[0] // rows[1]
    z, u = logits_of(n, V, dtype, n + V, 1.0)
    names = dict(T="temperature", k="top_k", p="top_p", q="min_p")
    tokens, logp = G.sample(z, u, **{names[a]: torch.full((n,), v, device="cuda", dtype=torch.int32 if a == "k" else torch.float32)
                                     for a, v in par.items()})
    want, lp = wanted(z, u, **par)
    assert torch.equal(tokens, want)
    assert bool(((logp.double() - lp).abs() <= LOGP_ABS + 2.0 ** -24 * lp.abs()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("V", [500009, 1000009])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_rows_too_long_for_one_cta_each(dtype, V):
    """Float32 slices of up to, and of more than, the 500000 that are weighed fast."""
    import grpo_loss_gb300 as G
    n = torch.cuda.get_device_properties(0).multi_processor_count + 3
    z, u = logits_of(n, V, dtype, V, 1.0)
    for par in ({}, dict(p=0.9)):
        kw = {"top_p": torch.full((n,), v, device="cuda") for v in par.values()}
        tokens, logp = G.sample(z, u, **kw)
        want, lp = wanted(z, u, **par)
        assert torch.equal(tokens, want)
        assert bool(((logp.double() - lp).abs() <= LOGP_ABS + 2.0 ** -24 * lp.abs()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1.0, 4.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logp_of_few_rows_loses_no_more_than_float32(dtype, spread):
    """In units of 2^-24, with S = sum w, d = (z - zmax) / T: the sum S itself (bf16
    rows: integers of exact weights; float32 rows 5.5 + 0.8 log2(V / S)); its logarithm
    2 ln S and their sum 1; d's difference and quotient 2 |d|; the result |logp|."""
    import grpo_loss_gb300 as G
    rows, V = 5, 128256
    z, u = logits_of(rows, V, dtype, 77, spread)
    temp = torch.full((rows,), 0.7, device="cuda")
    tokens, logp = G.sample(z, u, temperature=temp)
    y = z.double() / float(np.float32(0.7))
    top = y.max(1).values
    ln_s = (y - top[:, None]).exp().sum(1).log()
    d = y.gather(1, tokens.long()[:, None])[:, 0] - top
    mass = 0.01 if dtype == torch.bfloat16 else 5.5 + 0.8 * (math.log2(V) - ln_s / math.log(2))
    units = mass + 3 * ln_s + 2 * d.abs() + (d - ln_s).abs()
    assert bool(((logp.double() - (d - ln_s)).abs() <= 1.001 * units * 2.0 ** -24).all())


@pytest.mark.gpu
def test_borders_of_u():
    z = torch.zeros(8, 4096, device="cuda")
    u = torch.tensor([0.0, 2.0 ** -12, 0.5, 0.5 - 2.0 ** -25, 1 - 2.0 ** -24, 1.0, 2.0, float("nan")], device="cuda")
    tokens, _ = check(z, u)
    assert tokens.tolist() == [0, 1, 2048, 2047, 4095, 4095, 4095, 0]
    check(z, u, p=0.5)          # exactly half of the tokens
    check(z, u, k=1000, p=0.25)
    z[:, :100] = -math.inf      # the first token that can be drawn
    assert check(z, torch.zeros(8, device="cuda"))[0].tolist() == [100] * 8


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_rows(dtype):
    """-inf, the type's lowest value, NaN and +inf among the logits, rows with
    one token and with none."""
    z, u = logits_of(12, 3001, dtype, 9)
    inf, low = math.inf, torch.finfo(dtype).min
    z[0] = -inf
    z[1] = math.nan
    z[2] = -inf
    z[2, 2999] = -7.0
    z[3, :3000] = low
    z[4] = low
    z[5, ::2] = math.nan
    z[6, 17] = inf
    z[7, 5::1000] = inf
    z[8, 1:] = -inf
    z[9, :2990] = -inf
    z[10, ::3] = low
    z[11] = torch.where(torch.arange(3001, device="cuda") % 2 == 0, 0.0, -0.0).to(dtype)
    tokens, logp = check(z, u)
    assert tokens[:2].tolist() == [-1, -1] and tokens[2].item() == 2999 and tokens[8].item() == 0
    for par in (dict(p=0.6), dict(k=3), dict(q=0.3), dict(T=0.0), dict(T=2.0, k=50, p=0.7, q=0.001)):
        check(z, u, **par)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest_index(dtype):
    z = torch.full((16, 2000), -5.0, device="cuda", dtype=dtype)
    z[:, 1000:1200] = 1.0
    z[:, 300] = 2.0
    u = torch.arange(16, device="cuda") / 16.0
    check(z, u, k=11)           # 300 and the first ten of the ties
    check(z, u, p=0.2)
    check(z, u, k=150, p=0.5, q=0.1)
    tokens, _ = check(z, u, k=11)
    assert set(tokens.tolist()) <= {300} | set(range(1000, 1010))
    z[:, 300] = 1.0
    assert check(z, u, T=0.0)[0].tolist() == [300] * 16


@pytest.mark.gpu
def test_parameter_edges():
    """Values that switch a cut-off off, and out-of-range ones."""
    z, u = logits_of(8, 1003, torch.float32, 21)
    nan, inf = math.nan, math.inf
    check(z, u, k=[0, -1, 1003, 2000, 1002, 1, 2, 3])
    check(z, u, p=[1.0, 1.5, inf, 0.0, -1.0, 1e-9, 0.999999, 0.5])
    check(z, u, q=[0.0, -1.0, 1.0, 2.0, 1e-9, 1e-30, 0.5, inf])
    check(z, u, T=[1.0, 0.0, -1.0, nan, inf, 1e-30, 1e30, 1e-3])
    import grpo_loss_gb300 as G
    ones = torch.full((8,), nan, device="cuda")
    assert torch.equal(G.sample(z, u, top_p=ones, min_p=ones)[0], G.sample(z, u)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_strided_and_unaligned_rows(dtype, offset):
    big, u = logits_of(7, 5000, dtype, 2)
    for V in (4096, 4001):
        check(big[:, offset:offset + V], u, p=0.9)
        check(big[1:2, offset:offset + V], u[1:2].clone())
    check(big[::2, :1001], u[::2].clone(), k=20)


@pytest.mark.gpu
def test_draws_follow_the_distribution():
    """Over an even grid of u, each token is drawn as often as its share."""
    n = 4096
    z, _ = logits_of(1, 50, torch.float32, 4, 1.5)
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tokens, logp = check(z.expand(n, 50).contiguous(), u)
    share = torch.bincount(tokens.long(), minlength=50).double() / n
    assert (share - z[0].double().softmax(0)).abs().max().item() <= 1.0 / n + 1e-6


@pytest.mark.gpu
def test_rows_past_two_to_the_31_elements():
    V, rows = 128256, 17000                         # 2.18e9 elements
    z = torch.empty(rows, V, device="cuda", dtype=torch.bfloat16)
    z.fill_(-math.inf)
    want = torch.randint(0, V, (rows,), device="cuda")
    z.scatter_(1, want[:, None], 1.0)
    import grpo_loss_gb300 as G
    tokens, logp = G.sample(z, torch.rand(rows, device="cuda"))
    assert torch.equal(tokens.long(), want) and not logp.any()


@pytest.mark.gpu
def test_other_streams_and_graphs():
    import grpo_loss_gb300 as G
    z, u = logits_of(4, 9001, torch.bfloat16, 8)
    p = torch.full((4,), 0.9, device="cuda")
    want = G.sample(z, u, top_p=p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = G.sample(z, u, top_p=p)
    b = G.sample(z, u, top_p=p, stream=side)
    side.synchronize()
    out = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        G.sample(z, u, top_p=p, tokens=out[0], logp=out[1])
    g.replay()
    torch.cuda.synchronize()
    for got in (a, b, out):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    z2, u2 = logits_of(4, 9001, torch.bfloat16, 80)
    z.copy_(z2)
    u.copy_(u2)
    g.replay()
    again = G.sample(z2, u2, top_p=p)
    torch.cuda.synchronize()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("library not built (python -m grpo_loss_gb300.build)")
    return L.lib()


@pytest.mark.parametrize("field,value,status", [
    ("rows", -1, 1), ("V", 0, 1), ("ld", 99, 1), ("dtype", 2, 1), ("dtype", 9, 1),
    ("rows", 1 << 31, 2), ("V", 1 << 31, 2)])
def test_refuses_bad_problems_on_the_host(lib, field, value, status):
    pr = L.SampleProblem(4, 100, 0, L.GRPO_F32)
    setattr(pr, field, value)
    at = ctypes.c_void_p(256)
    assert lib.grpo_sample(ctypes.byref(pr), at, at, None, None, None, None, at, at, None) == status


def test_refuses_bad_pointers_on_the_host(lib):
    pr, at, odd = L.SampleProblem(4, 100, 0, L.GRPO_BF16), ctypes.c_void_p(256), ctypes.c_void_p(257)
    good = [at, at, at, at, at, at, at, at]
    assert lib.grpo_sample(None, *good, None) == 1
    for i in (0, 1, 6, 7):
        assert lib.grpo_sample(ctypes.byref(pr), *[None if j == i else g for j, g in enumerate(good)], None) == 1
    for i in range(8):
        assert lib.grpo_sample(ctypes.byref(pr), *[odd if j == i else g for j, g in enumerate(good)], None) == 2
    pr.rows = 0
    assert lib.grpo_sample(ctypes.byref(pr), *[None] * 8, None) == 0


def test_binding_refuses_wrong_tensors():
    import grpo_loss_gb300 as G
    with pytest.raises(ValueError, match="2-D"):
        G.sample(torch.zeros(5), torch.zeros(1))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        G.sample(torch.zeros(1, 5, dtype=torch.float16), torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA"):
        G.sample(torch.zeros(1, 5), torch.zeros(1))


@pytest.mark.gpu
def test_binding_refuses_wrong_gpu_tensors():
    import grpo_loss_gb300 as G
    z, u = torch.zeros(4, 8, device="cuda"), torch.zeros(4, device="cuda")
    for bad, word in ((dict(u=u[:3]), "elements"), (dict(u=u.double()), "float32"), (dict(u=u.cpu()), "on cuda"),
                      (dict(top_k=u), "int32"), (dict(top_p=u[:1]), "elements"), (dict(tokens=u), "int32"),
                      (dict(logits=z.t()), "contiguous"), (dict(logits=z[:1].expand(4, 8)), "row stride")):
        with pytest.raises(ValueError, match=word):
            G.sample(**{"logits": z, "u": u, **bad})
    tokens, logp = G.sample(z[:0], u[:0])
    assert tokens.numel() == 0 and logp.numel() == 0
