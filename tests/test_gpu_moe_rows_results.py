"""The row calls' results as the binding allocates them, and the forms that
prompts take, against plain 64-bit evaluations.

Tolerances: a sum of k products in fp32, in order, is off by at most
k * 2^-24 * sum |terms|; an output's rounding by half a step of its type.
"""
import numpy as np
import pytest
import torch

import bit_gemm_quantize_b200 as bgq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INVALID_ARG = 1


def _poison(nbytes):
    """Leaves freed memory full of NaN for the next results of that size (the allocator hands out freed blocks again)."""
    for n in (nbytes, nbytes + 512):
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")


def _rows(T, k, seed, none, drop=0.0):
    """slot_row [T, k] of distinct rows of [0, T * k): a random order, with plain -1 in `none` of the slots and -2 - row
    in `drop` of them."""
    rng = np.random.default_rng(seed)
    sr = rng.permutation(T * k).astype(np.int32)
    u = rng.random(T * k)
    return np.where(u < none, -1, np.where(u < none + drop, -2 - sr, sr)).reshape(T, k).astype(np.int32)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (3, 2, 64), (40, 3, 77), (500, 4, 256), (700, 2, 2048), (1500, 3, 33),
                                   (9, 2, 14336)])
@pytest.mark.parametrize("none,drop", [(0.0, 0.0), (0.1, 0.0), (0.2, 0.3), (1.0, 0.0)])
def test_rows_that_no_slot_names_are_zero(cuda_device, dt, T, k, H, none, drop):
    """A slot of -1 names no row: a result allocated by the call has zeros there, not what the memory held."""
    sr = _rows(T, k, T + H, none, drop)
    if none in (0.1, 0.2):
        sr[T // 2, 0] = -1
    g = torch.Generator().manual_seed(T)
    x, d = torch.randn(T, H, generator=g).to(DT[dt]).to(cuda_device), torch.randn(T, H, generator=g).to(cuda_device)
    y = torch.randn(T * k, H, generator=g).to(DT[dt]).to(cuda_device)
    w = torch.rand(T, k, generator=g).to(cuda_device)
    slot_row = torch.from_numpy(sr).to(cuda_device)
    size = T * k * H * x.element_size()
    kept = sr >= 0

    _poison(size)
    x_r = bgq.moe_dispatch(x, slot_row)
    ref = torch.zeros(T * k, H, dtype=DT[dt])
    ref[sr[kept].astype(np.int64)] = x.cpu()[np.nonzero(kept)[0]]
    assert torch.equal(x_r.cpu(), ref)

    _poison(size)
    d_y, d_w = bgq.moe_combine_backward(d, y, w, slot_row)
    ref = np.zeros((T * k, H))
    t, s = np.nonzero(kept)
    ref[sr[kept]] = w.double().cpu().numpy()[t, s, None] * d.double().cpu().numpy()[t]
    err = np.abs(d_y.double().cpu().numpy() - ref)
    half = torch.finfo(DT[dt]).eps / 2
    assert np.all(err <= np.abs(ref) * (2.0 ** -24 + half * (1 + 2.0 ** -24)) + (2.0 ** -25 if dt == "f16" else 0.0))
    assert np.all(d_w.cpu().numpy()[~kept] == 0.0) and torch.isfinite(d_w).all()
    assert bgq.device_status() == 0


def test_rows_outside_leave_zeros(cuda_device):
    """A row beyond the result is reported, and the row that its slot should have named is zero."""
    sr = _rows(30, 2, 1, 0.0)
    lost = sr[7, 1]
    sr[7, 1] = 60
    slot_row = torch.from_numpy(sr).to(cuda_device)
    x, w = torch.randn(30, 72, device=cuda_device), torch.rand(30, 2, device=cuda_device)
    for call in (lambda: bgq.moe_dispatch(x, slot_row),
                 lambda: bgq.moe_combine_backward(x, torch.ones(60, 72, device=cuda_device), w, slot_row)[0]):
        bgq.device_status(clear=True)
        _poison(60 * 72 * 4)
        got = call()
        torch.cuda.synchronize()
        assert bgq.device_status(clear=True) == INVALID_ARG
        assert torch.all(got[lost] == 0.0) and torch.isfinite(got).all()


def test_given_results_keep_the_rows_that_no_slot_names(cuda_device):
    sr = _rows(600, 2, 5, 0.2)
    slot_row = torch.from_numpy(sr).to(cuda_device)
    x, w = torch.randn(600, 136, device=cuda_device), torch.rand(600, 2, device=cuda_device)
    unnamed = np.setdiff1d(np.arange(1200), sr)
    assert unnamed.size > 100
    mine = torch.full((1200, 136), 3.0, device=cuda_device)
    assert torch.all(bgq.moe_dispatch(x, slot_row, x_r=mine)[unnamed] == 3.0)
    mine.fill_(3.0)
    y = torch.ones(1200, 136, device=cuda_device)
    assert torch.all(bgq.moe_combine_backward(x, y, w, slot_row, d_y=mine)[0][unnamed] == 3.0)
    # rows beyond the slots', and fewer rows than slots
    assert torch.all(bgq.moe_combine_backward(x, torch.ones(1300, 136, device=cuda_device), w, slot_row)[0][1200:] == 0.0)


def test_unnamed_rows_in_a_replayed_graph_and_beside_another_stream(cuda_device):
    T, k, H = 300, 2, 264
    x, w = torch.randn(T, H, device=cuda_device), torch.rand(T, k, device=cuda_device)
    y = torch.randn(T * k, H, device=cuda_device)
    slot_row = torch.from_numpy(_rows(T, k, 0, 0.0)).to(cuda_device)

    def both():
        return bgq.moe_dispatch(x, slot_row), bgq.moe_combine_backward(x, y, w, slot_row)[0]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    other = torch.cuda.Stream()
    for seed in range(4):
        sr = _rows(T, k, seed, 0.15 * seed)
        slot_row.copy_(torch.from_numpy(sr))
        for t in got:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            beside = both()
        torch.cuda.synchronize()
        for a, b in zip(got, beside):
            assert torch.equal(a, b) and torch.isfinite(a).all()
            assert torch.all(a[np.setdiff1d(np.arange(T * k), sr)] == 0.0)


# ------------------------------------------------------------------ prompts

# Enough tokens that every CTA of combine and of its gradient takes several: two slots of long 16-bit rows (128 threads a
# token), three and eight slots, fp32, a row length that is not a multiple of 8, and one below 1024
PROMPTS = [(2000, 2, 2048, "f16", "bf16"), (2500, 2, 4096, "bf16", "bf16"), (2000, 3, 1024, "bf16", "f32"),
           (1300, 8, 512, "f16", "f16"), (3001, 2, 2048, "f32", "f32"), (3000, 2, 2051, "bf16", "f16"),
           (2600, 3, 1027, "f32", "bf16"), (20011, 2, 136, "f16", "f16"), (21001, 5, 67, "bf16", "bf16")]


def _half_step(ref, dt, slack):
    mag = np.abs(ref) + slack
    return slack + mag * (torch.finfo(DT[dt]).eps / 2) + (2.0 ** -25 if dt == "f16" else 2.0 ** -126)


@pytest.mark.parametrize("T,k,H,dt,out", PROMPTS)
@pytest.mark.parametrize("none,drop", [(0.0, 0.0), (0.05, 0.1)])
def test_prompts(cuda_device, T, k, H, dt, out, none, drop):
    v = _rows(T, k, H, none, drop).astype(np.int64)
    slot_row = torch.from_numpy(v.astype(np.int32)).to(cuda_device)
    g = torch.Generator().manual_seed(T)
    y = torch.randn(T * k, H, generator=g).to(DT[dt])
    w = torch.rand(T, k, generator=g)
    d = torch.randn(T, H, generator=g).to(DT[out])
    yd, wd, dd = y.to(cuda_device), w.to(cuda_device), d.to(cuda_device)
    got = bgq.moe_combine(yd, wd, slot_row, out=out).cpu().double().numpy()
    back = bgq.moe_dispatch_backward(yd, slot_row).cpu().double().numpy()
    d_y, d_w = (t.cpu().double().numpy() for t in bgq.moe_combine_backward(dd, yd, wd, slot_row))
    x_r = bgq.moe_dispatch(dd, slot_row).cpu()
    yh, wh, dh = y.double().numpy(), w.double().numpy(), d.double().numpy()
    kept = v >= 0
    ref_y, ref_x = np.zeros((T * k, H)), torch.zeros(T * k, H, dtype=DT[out])
    t, s = np.nonzero(kept)
    ref_y[v[kept]] = wh[t, s, None] * dh[t]
    ref_x[v[kept]] = d[t]
    assert torch.equal(x_r, ref_x)
    assert np.all(np.abs(d_y - ref_y) <= _half_step(ref_y, dt, 2.0 ** -24 * np.abs(ref_y)))
    comb, comb_mag, plain, plain_mag = np.zeros((4, T, H))
    for i in range(k):
        rows = np.where(kept[:, i, None], yh[np.maximum(v[:, i], 0)], 0.0)
        comb += wh[:, i, None] * rows
        comb_mag += np.abs(wh[:, i, None] * rows)
        plain += rows
        plain_mag += np.abs(rows)
        prod = rows * dh
        # chains of at least H / 32 products (and 8 more of a vector), then 13 tree steps
        assert np.all(np.abs(d_w[:, i] - prod.sum(1)) <= (H / 32 + 8 + 13 + 1) * 2.0 ** -24 * np.abs(prod).sum(1))
    assert np.all(d_w[~kept] == 0.0)
    assert np.all(np.abs(got - comb) <= _half_step(comb, out, k * 2.0 ** -24 * comb_mag))
    assert np.all(np.abs(back - plain) <= _half_step(plain, dt, k * 2.0 ** -24 * plain_mag))
    assert bgq.device_status() == 0


@pytest.mark.parametrize("T,k,H", [(20000, 2, 24), (9000, 4, 17), (70000, 1, 8), (600000, 2, 8)])
@pytest.mark.parametrize("missing", ["one", "last", "few", "most", "all"])
def test_unnamed_rows_among_many(cuda_device, T, k, H, missing):
    """More rows than are marked at a time, more than the CTAs that look for missing slots; one slot without a row, in
    one share of the slots or in all."""
    n = T * k
    rng = np.random.default_rng(T)
    sr = rng.permutation(n).astype(np.int32)
    if missing == "one":
        sr[n // 3] = -1
    elif missing == "last":
        sr[-1] = n + 5  # outside: reported, and none
    else:
        sr[rng.random(n) < dict(few=0.001, most=0.9, all=2.0)[missing]] = -1
    named = (sr >= 0) & (sr < n)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    ref = torch.zeros(n, H, dtype=torch.bfloat16)
    ref[sr[named].astype(np.int64)] = x[np.nonzero(named)[0] // k]
    slot_row, xd = torch.from_numpy(sr.reshape(T, k)).to(cuda_device), x.to(cuda_device)
    bgq.device_status(clear=True)
    _poison(n * H * 2)
    x_r = bgq.moe_dispatch(xd, slot_row)
    assert torch.equal(x_r.cpu(), ref)
    _poison(n * H * 2)
    d_y, _ = bgq.moe_combine_backward(xd, x_r, torch.ones(T, k, device=cuda_device), slot_row)
    assert torch.equal(d_y.cpu(), ref)
    torch.cuda.synchronize()
    assert bgq.device_status(clear=True) == (INVALID_ARG if missing == "last" else 0)


def test_kept_rows_only(cuda_device):
    """A result of fewer rows than slots (those of the kept slots): what is not named there is zero too."""
    T, k, H, R = 3000, 2, 40, 4100
    rng = np.random.default_rng(2)
    order = rng.permutation(T * k).astype(np.int32)
    sr = np.where(order < R, order, -2 - order).reshape(T, k)  # rows behind the kept ones: to be cleared, but outside
    sr[7, 1] = -1
    sr[1234, 0] = -1
    y = torch.randn(R, H, generator=torch.Generator().manual_seed(1)).to(cuda_device)
    d, w = torch.randn(T, H, device=cuda_device), torch.rand(T, k, device=cuda_device)
    _poison(R * H * 4)
    d_y, d_w = bgq.moe_combine_backward(d, y, w, torch.from_numpy(sr).to(cuda_device))
    ref = torch.zeros(R, H, device=cuda_device)
    t, s = np.nonzero(sr >= 0)
    ref[torch.from_numpy(sr[sr >= 0].astype(np.int64)).to(cuda_device)] = w[t, s][:, None] * d[t]
    assert torch.equal(d_y, ref) and torch.isfinite(d_w).all()
    assert bgq.device_status() == 0


def test_no_rows_at_all(cuda_device):
    """Every slot dropped and the experts' outputs empty: zeros, and no row to write."""
    sr = torch.from_numpy(np.array([[-2, -1], [-3, -4]], np.int32)).to(cuda_device)
    y, w, d = (torch.ones(s, device=cuda_device) for s in ((0, 40), (2, 2), (2, 40)))
    assert torch.all(bgq.moe_combine(y, w, sr) == 0.0)
    d_y, d_w = bgq.moe_combine_backward(d, y, w, sr)
    assert d_y.shape == (0, 40) and torch.all(d_w == 0.0)
    assert torch.all(bgq.moe_dispatch(d, sr) == 0.0)
    assert bgq.device_status() == 0
