"""Values that the products of unquantized tokens with 4-bit weights have to
keep: infinities and NaN, single codes, single values over the exponent range,
blocks of a few large values among small ones.  Every form of the kernel is
reached: it has one for up to 2, 4 and 8 tokens of a pass, each dense and per
expert, with float and with integer scales, and takes K whole, split over a
cluster or in panels.

Tolerance (units of 2^-24, u).  A token's block of 128 values is held as
integers, off by at most 2^-30 of the block's largest magnitude a value; sums
over a block are exact.  Each pair of digits is converted to fp32 (1 u of the
high pair's sum, which the products' magnitudes bound; the low pair is at most
2^-14 of the largest value a product) and joined (1 u); scales and factors enter
by one FMA a block (1 u of a partial sum), and the sums of up to 16 warps, 8
CTAs and the panels of K are added (1 u each).  The blocks that are multiplied in
fp32 instead take chains of 32 FMAs, 4 adds and one FMA a block.
"""
import numpy as np
import pytest
import torch

import bit_gemm_quantize_b200 as bgq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
TOKENS = (1, 2, 3, 4, 8, 11)


def _pack(q):
    """Packed bytes [N, K/2] of int codes [N, K]: code j of each word of eight in byte j mod 4, low nibble first."""
    b = (q & 15).astype(np.uint8).reshape(q.shape[0], -1, 2, 4)
    return torch.from_numpy((b[:, :, 0] | b[:, :, 1] << 4).reshape(q.shape[0], -1))


def _call(form, x, q, scale, kind, alpha=1024, out="f32"):
    """y of tokens x (a CUDA tensor) with codes q [N, K] and scales [K/128, N] (float, or integers over alpha), dense or
    as the only expert with rows."""
    dev = x.device
    packed = _pack(q).to(dev)
    s = torch.from_numpy(scale.astype(np.float32 if kind == "float" else np.int16)).to(dev)
    kw = dict(s_g=s) if kind == "float" else dict(S=s, alpha=alpha)
    if form == "dense":
        return bgq.w4a16_gemv(x, packed, out=out, **kw)
    off = torch.tensor([0, x.shape[0]], dtype=torch.int64, device=dev)
    kw = {k: [v] if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    return bgq.w4a16_gemv_grouped(x, None, off, [packed], out=out, **kw)


def _scales(rng, K, N, kind):
    return rng.uniform(0.001, 0.02, (K // 128, N)).astype(np.float32) if kind == "float" else rng.integers(
        1, 30, (K // 128, N))


def _definition(x, q, scale, kind, alpha=1024):
    """sum_k x q s in 64 bits, product by product (so that infinities and NaN meet as the formula has them), and
    sum |x q s| of the finite ones."""
    s = scale.astype(np.float64) / (1 if kind == "float" else alpha)
    w = q * np.repeat(s.T, 128, axis=1)
    xh = x.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        y = np.stack([(row[None] * w).sum(1) for row in xh])
    mag = np.abs(np.where(np.isfinite(xh), xh, 0.0)) @ np.abs(w).T
    return y, mag


def _same(got, ref, mag, slack_of_mag, absolute=0.0):
    """Infinities and NaN where the definition has them, the finite ones within slack."""
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]) and not np.isinf(got[~inf]).any()
    fin = np.isfinite(ref)
    slack = np.broadcast_to(slack_of_mag * mag + absolute, ref.shape)
    err = np.abs(got[fin] - ref[fin])
    assert np.all(err <= slack[fin]), float((err / slack[fin]).max())


def _block_slack(x, q, scale, kind, alpha=1024):
    """The integers' part of the tolerance: 2^-30 of each block's largest value for every product, and the low pair's
    conversions (at most 2^-14 of the largest value a product, 1 u a block in a chain of them)."""
    s = scale.astype(np.float64) / (1 if kind == "float" else alpha)
    w = np.abs(q * np.repeat(s.T, 128, axis=1)).reshape(q.shape[0], -1, 128).sum(2)
    xh = np.abs(x.double().cpu().numpy())
    top = np.where(np.isfinite(xh), xh, 0.0).reshape(xh.shape[0], -1, 128).max(2)
    n = w.shape[1]
    return (2.0 ** -30 + (n + 2) * U * 2.0 ** -14) * (top @ w.T)


def _chain(K):
    return (K // 128 + 2 + 16 + 8 + 8 + 1 + 37) * U  # 37: a block multiplied in fp32


@pytest.mark.parametrize("form", ["dense", "experts"])
@pytest.mark.parametrize("kind", ["float", "int"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("codes,values,want", [
    ((2, -1), (1, 1), "nan"), ((3, -1), (1, -1), "+"), ((3, 0), (1, 1), "nan"), ((3, 2), (1, 1), "+"),
    ((-3, -2), (1, 1), "-"), ((1, 1), (1, -1), "nan"), ((0, 0), (1, 1), "nan"), ((-8, 7), (-1, 1), "+")])
def test_two_infinities_of_a_block(cuda_device, form, kind, dt, codes, values, want):
    K, N = 256, 16
    for M in TOKENS:
        x = torch.zeros(M, K)
        x[:, ::3] = 0.25
        x[M - 1, 130], x[M - 1, 201] = values[0] * float("inf"), values[1] * float("inf")
        q = np.ones((N, K), np.int64)
        q[:, 130], q[:, 201] = codes
        y = _call(form, x.to(DT[dt]).to(cuda_device), q, np.ones((2, N)), kind)
        last = y[M - 1].cpu()
        assert torch.isnan(last).all() if want == "nan" else torch.isinf(last).all() and (last > 0).all() == (want == "+")
        assert torch.isfinite(y[:M - 1]).all()


@pytest.mark.parametrize("form", ["dense", "experts"])
@pytest.mark.parametrize("kind", ["float", "int"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(1, 256, 24), (2, 4096, 1048), (3, 512, 40), (4, 11008, 72), (8, 1024, 136),
                                   (8, 16384, 40), (11, 384, 520)])
def test_infinities_and_nan(cuda_device, form, kind, dt, M, K, N):
    """Tokens with none, one or several infinities in a block, with NaN beside them, and blocks full of them."""
    rng = np.random.default_rng(M + K)
    x = rng.standard_normal((M, K)).astype(np.float32)
    for m in range(0, M, 2):
        at = 128 * rng.integers(K // 128) + rng.permutation(128)[:rng.integers(1, 5)]
        x[m, at] = rng.choice([-np.inf, np.inf], at.size)
    if M > 2:
        x[2, :128] = np.inf
        x[M - 2, rng.integers(K, size=2)] = np.nan, np.inf
    q = rng.integers(-8, 8, (N, K))
    scale = _scales(rng, K, N, kind)
    x = torch.from_numpy(x).to(DT[dt]).to(cuda_device)
    y = _call(form, x, q, scale, kind)
    ref, mag = _definition(x, q, scale, kind)
    _same(y, ref, mag, _chain(K), _block_slack(x, q, scale, kind))
    assert bgq.device_status() == 0


@pytest.mark.parametrize("form", ["dense", "experts"])
@pytest.mark.parametrize("kind", ["float", "int"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("ratio", [30.0, 1e3, 1e4, 3e6])
@pytest.mark.parametrize("outliers", [1, 5, 20])
def test_large_values_over_zero_codes(cuda_device, form, kind, dt, ratio, outliers):
    """A few values far above the rest of their block, where the codes are 0: they are in no product, and what is left is
    as exact as the products that there are.  Beside them an exact zero or two, eight values without a large one, and
    blocks without any."""
    K, N = 384, 40
    for M in TOKENS:
        rng = np.random.default_rng(M + outliers)
        x = rng.standard_normal((M, K)) * (30000.0 / ratio / 3)
        q = rng.integers(-8, 8, (N, K))
        for m in range(M):
            at = rng.permutation(120)
            block = 128 * (m % 3)
            x[m, block + at[:outliers]] = rng.uniform(0.5, 1, outliers) * 30000.0
            x[m, block + at[60:62]] = 0.0
            q[:, block + at[:outliers]] = 0
        scale = _scales(rng, K, N, kind)
        x = torch.from_numpy(x.astype(np.float32)).to(DT[dt]).to(cuda_device)
        y = _call(form, x, q, scale, kind)
        ref = x.double().cpu().numpy() @ (q * np.repeat(scale.astype(np.float64).T / (1 if kind == "float" else 1024), 128,
                                                        axis=1)).T
        mag = _definition(x, q, scale, kind)[1]
        _same(y, ref, mag, _chain(K))
    assert bgq.device_status() == 0


def _in_groups(x, M):
    return [x[i:i + M] for i in range(0, x.shape[0], M)]


@pytest.mark.parametrize("form", ["dense", "experts"])
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("kind,alpha", [("float", 1), ("int", 1), ("int", 256), ("int", 1024), ("int", 1 << 14),
                                        ("int", 1 << 22)])
def test_single_values_over_the_exponent_range(cuda_device, form, M, kind, alpha):
    """One value at a time over codes of 1 and a scale that is a power of two: the value times the scale, to the last
    bit, from the largest fp32 value down to 2^-100 (or as far as the integers reach)."""
    K, N = 256, 16
    rng = np.random.default_rng(M)
    S = min(alpha, 1 << 14)
    low = max(-100, -115 + int(np.log2(alpha)))
    vals = np.ldexp(rng.uniform(1, 2, 24).astype(np.float32), rng.integers(low, 127, 24)).astype(np.float32)
    vals = np.concatenate([vals, -vals, np.float32([np.finfo(np.float32).max, -np.finfo(np.float32).max, 2.0 ** low, 0.0])])
    x = np.zeros((vals.size, K), np.float32)
    x[np.arange(vals.size), np.arange(vals.size) * 5 % K] = vals
    scale = np.full((2, N), 1.0 if kind == "float" else S)
    want = vals * np.float32(S / alpha)
    y = torch.cat([_call(form, part, np.ones((N, K), np.int64), scale, kind, alpha=alpha)
                   for part in _in_groups(torch.from_numpy(x).to(cuda_device), M)])
    assert np.array_equal(y.cpu().numpy(), np.repeat(want[:, None], N, axis=1))


@pytest.mark.parametrize("form", ["dense", "experts"])
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("kind", ["float", "int"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_every_place_and_code(cuda_device, form, M, kind, dt):
    """Unit tokens read the weights back exactly: every code, every place of the packed word, every token of a pass."""
    K, N = 256, 40
    rng = np.random.default_rng(M)
    q = rng.integers(-8, 8, (N, K))
    scale = rng.integers(1, 9, (K // 128, N))
    eye = torch.eye(K)[rng.permutation(K)[:66]]
    y = torch.cat([_call(form, part, q, scale, kind, alpha=1) for part in _in_groups(eye.to(DT[dt]).to(cuda_device), M)])
    w = q * np.repeat(scale.T, 128, axis=1)
    assert np.array_equal(y.cpu().numpy(), eye.numpy().astype(np.float64) @ w.T)


@pytest.mark.parametrize("form", ["dense", "experts"])
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("kind", ["float", "int"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_every_value_keeps_its_bits(cuda_device, form, M, kind, dt):
    """Columns with a single code: each value of a token comes back on its own, off by at most 2^-30 of the largest of
    its block (in no unit of sums, so that the lowest digit counts), in a pass of every number of tokens."""
    K, N = 384, 384
    rng = np.random.default_rng(M)
    x = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-8, 9, (M, 3)).repeat(128, axis=1)
    x[:, 5::61] *= 30.0
    x = torch.from_numpy(x.astype(np.float32)).to(DT[dt]).to(cuda_device)
    code = rng.permutation([1, 2, 4, -1, -2, -4, -8] * 55)[:N]
    y = _call(form, x, np.diag(code), np.ones((3, N)), kind, alpha=1).double().cpu().numpy()
    xh = x.double().cpu().numpy()
    top = np.abs(xh).reshape(M, 3, 128).max(2).repeat(128, axis=1)
    assert np.all(np.abs(y - xh * code) <= 2.0 ** -30 * top * np.abs(code))


@pytest.mark.parametrize("M,K,N", [(1301, 256, 24), (700, 2048, 40), (333, 4096, 16)])
@pytest.mark.parametrize("kind", ["float", "int"])
def test_infinities_among_many_tokens(cuda_device, M, K, N, kind):
    """More passes than clusters, so that each takes several: some with tokens that are multiplied in fp32, some not."""
    rng = np.random.default_rng(M)
    x = rng.standard_normal((M, K)).astype(np.float32)
    for m in rng.permutation(M)[:M // 7]:
        x[m, rng.integers(K, size=2)] = rng.choice([-np.inf, np.inf], 2)
    q = rng.integers(-8, 8, (N, K))
    scale = _scales(rng, K, N, kind)
    x = torch.from_numpy(x).to(cuda_device)
    y = _call("dense", x, q, scale, kind)
    ref, mag = _definition(x, q, scale, kind)
    _same(y, ref, mag, _chain(K), _block_slack(x, q, scale, kind))
    clean = torch.isfinite(x).all(1)
    other = torch.where(clean[:, None], x, torch.zeros_like(x))  # the tokens beside them are as without them
    assert torch.equal(y[clean], _call("dense", other, q, scale, kind)[clean])


@pytest.mark.parametrize("T,k,E,K,N", [(400, 2, 200, 256, 24), (16, 2, 8, 4096, 264), (90, 3, 5, 1408, 40)])
@pytest.mark.parametrize("kind", ["float", "int"])
def test_infinities_among_experts(cuda_device, T, k, E, K, N, kind):
    """Every expert its own weights, dropped slots, outputs in slot order: infinities in some tokens, and blocks of a few
    large values over zero codes in others."""
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, K)).astype(np.float32)
    x[::5, 7], x[::5, 100] = np.inf, -np.inf
    x[1::5, 128:256] *= 1e-4
    x[1::5, 131] = 2e4
    x = torch.from_numpy(x).to(cuda_device)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    ids[rng.random((T, k)) < 0.1] = -1
    r = bgq.moe_route_sort(torch.from_numpy(ids).to(cuda_device), E)
    qs = [rng.integers(-8, 8, (N, K)) for _ in range(E)]
    for q in qs:
        q[:, 131] = 0
    scales = [_scales(rng, K, N, kind) for _ in range(E)]
    packed = [_pack(q).to(cuda_device) for q in qs]
    s = [torch.from_numpy(v.astype(np.float32 if kind == "float" else np.int16)).to(cuda_device) for v in scales]
    kw = dict(s_g=s) if kind == "float" else dict(S=s, alpha=1024)
    y = torch.full((T * k, N), 5.0, device=cuda_device)
    bgq.w4a16_gemv_grouped(x, r["row_index"], r["expert_offsets"], packed, out="f32", y=y, out_row=r["out_row"], **kw)
    y = y.reshape(T, k, N)
    for e in range(E):
        t, slot = np.nonzero(ids == e)
        if t.size:
            xe = x[torch.from_numpy(t).to(cuda_device)]
            ref, mag = _definition(xe, qs[e], scales[e], kind)
            slack = _block_slack(xe, qs[e], scales[e], kind)
            slack[t % 5 == 1] = 0.0  # multiplied in fp32
            _same(y[torch.from_numpy(t).to(cuda_device), torch.from_numpy(slot).to(cuda_device)], ref, mag, _chain(K), slack)
    assert torch.all(y[torch.from_numpy(ids < 0).to(cuda_device)] == 5.0)
    assert bgq.device_status() == 0


def test_graph_and_streams_with_tokens_in_fp32(cuda_device):
    """A captured call whose tokens hold infinities in some replays and not in others, beside calls on another stream."""
    rng = np.random.default_rng(0)
    K, N, M = 2048, 520, 5
    q, scale = rng.integers(-8, 8, (N, K)), _scales(rng, K, N, "float")
    clean = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(cuda_device)
    bad = clean.clone()
    bad[3, 11], bad[0, 2000] = float("inf"), float("-inf")
    want = [_call("dense", v, q, scale, "float") for v in (clean, bad)]
    assert torch.equal(torch.isnan(want[1][3]), torch.from_numpy(q[:, 11] == 0).to(cuda_device))
    packed, s = _pack(q).to(cuda_device), torch.from_numpy(scale).to(cuda_device)
    x = clean.clone()
    call = lambda v: bgq.w4a16_gemv(v, packed, s_g=s, out="f32")
    call(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(x)
    other = torch.cuda.Stream()
    for i in (1, 0, 1, 1, 0):
        x.copy_((clean, bad)[i])
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            beside = call((clean, bad)[1 - i])
        torch.cuda.synchronize()
        for got, ref in ((y, want[i]), (beside, want[1 - i])):
            assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(ref, nan=7.0))
            assert torch.equal(torch.isnan(got), torch.isnan(ref))


@pytest.mark.parametrize("form", ["dense", "experts"])
@pytest.mark.parametrize("M,K", [(2, 128), (3, 384), (4, 128), (8, 128), (7, 640)])
def test_a_token_in_fp32_leaves_its_neighbours(cuda_device, form, M, K):
    """Beside a token that is multiplied in fp32, one at the border (every eight values hold a large one, nearly all others
    are tiny) gives the same bits as beside ordinary tokens."""
    rng = np.random.default_rng(M)
    N = 40
    x = rng.standard_normal((M, K)) * 2.0 ** -13
    x[:, ::8] = rng.uniform(1.0, 1.9, (M, K // 8)) * 2.0 ** -9
    x[:, ::128] = 1.5
    q, scale = rng.integers(-8, 8, (N, K)), _scales(rng, K, N, "float")
    for bad in range(M):
        other = x.copy()
        other[bad] = rng.standard_normal(K) * 1e-6
        other[bad, 5::128] = 3e4
        a, b = (torch.from_numpy(v.astype(np.float32)).to(cuda_device) for v in (x, other))
        keep = [m for m in range(M) if m != bad]
        assert torch.equal(_call(form, a, q, scale, "float")[keep], _call(form, b, q, scale, "float")[keep]), bad
