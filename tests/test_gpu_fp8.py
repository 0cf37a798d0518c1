"""The FP8 quantizer and the block-scaled FP8 GEMM against the oracle, on a GPU.

Quantizer: bit-exact codes and scales.

GEMM tolerance: the products of E4M3 values are exact in fp32.  A K-long sum of
terms t with fp32 additions is off by at most one unit in the last place (2^-23:
the tensor core may chop instead of round) of a partial sum, itself at most
sum |t|, per addition; the scales' product, its product with a block's sum and
the addition across blocks are three more roundings per block.  So
|err| <= (K + 4 ceil(K/128)) 2^-23 sum |t|, and half a step of the output type
(bf16: 2^-8 relative) on top.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import fp8
from parity import bf16_torch_to_bits, bits_to_torch_cuda, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    from fp4_micro_block_b200 import build
    build.build()
    import fp4_micro_block_b200 as m
    assert m.fp4q_device_error() == 0
    yield m
    assert m.fp4q_device_error() == 0


def host(t):
    """float32 values of a bf16 CUDA tensor."""
    return fp8.bf16_values(bf16_torch_to_bits(t))


def activations(M, K, seed):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((M, K)) * np.exp(rng.standard_normal(K))
    return torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).cuda()


SHAPES = [(1, 1), (1, 64), (3, 127), (128, 128), (129, 130), (5, 1000), (130, 385), (300, 257), (1, 4096), (257, 1024)]


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_codes_and_scales(fq, shape, block):
    M, K = shape
    tile = block == "tile"
    x = activations(M, -(-K // 8) * 8, M + K)[:, :K]
    want, want_s = fp8.quantize(host(x), tile)
    want_t, want_ts = fp8.quantize(np.ascontiguousarray(host(x).T), tile)
    b = fq.FP4Q_FP8_TILE if tile else fq.FP4Q_FP8_ROW
    for transpose in (False, True):
        got = fq.quantize_fp8(x, b, transpose)
        assert np.array_equal(to_np(got[0]), want) and np.array_equal(to_np(got[1]), want_s)
    assert np.array_equal(to_np(got[2]), want_t) and np.array_equal(to_np(got[3]), want_ts)
    alone = fq.alloc_fp8(K, M, b)
    fq.fp4q_quantize_fp8(x, b, codes_t=alone[0], scales_t=alone[1])
    assert np.array_equal(to_np(alone[0]), want_t) and np.array_equal(to_np(alone[1]), want_ts)


@pytest.mark.parametrize("block", ["row", "tile"])
def test_quantize_extreme_values(fq, block):
    """Zeros of both signs, subnormals, the largest values, NaN and infinities, block by block."""
    rng = np.random.default_rng(7)
    M, K = 140, 700
    x = (rng.standard_normal((M, K)) * np.exp2(rng.integers(-130, 120, (M, 1)))).astype(np.float32)
    x[:5, :128] = 0.0
    x[2, 3] = -0.0
    x[6, 128:256] = 2.0 ** -133  # the smallest bf16 subnormal
    x[7, :] = 3.3895e38
    x[8, 140] = np.nan
    x[9, 300] = np.inf
    x[10, 301] = -np.inf
    x[130:, 512:] = 0.0
    t = torch.zeros((M, 704), dtype=torch.bfloat16, device="cuda")[:, :K]  # rows 16 bytes apart in step
    t.copy_(torch.from_numpy(x))
    tile = block == "tile"
    got = fq.quantize_fp8(t, fq.FP4Q_FP8_TILE if tile else fq.FP4Q_FP8_ROW, True)
    for (c, s), v in (((got[0], got[1]), host(t)), ((got[2], got[3]), np.ascontiguousarray(host(t).T))):
        want, want_s = fp8.quantize(v, tile)
        assert np.array_equal(to_np(s), want_s)
        same = to_np(c) == want
        nan = (want & 0x7F) == 0x7F  # a NaN code has no sign to keep
        assert same[~nan].all() and ((to_np(c)[nan] & 0x7F) == 0x7F).all()


def test_quantize_leaves_padding_alone_and_reads_views(fq):
    M, K = 37, 130
    wide = activations(M, 400, 3)
    x = wide[:, 8:8 + K]
    for b in (fq.FP4Q_FP8_ROW, fq.FP4Q_FP8_TILE):
        tile = b == fq.FP4Q_FP8_TILE
        bufs = [torch.full((M, 160), 0xA5, dtype=torch.uint8, device="cuda"), torch.full((2, 48), -7.0, device="cuda"),
                torch.full((K, 64), 0xA5, dtype=torch.uint8, device="cuda"), torch.full((1, 144), -7.0, device="cuda")]
        n, k = (1, 2) if tile else (M, K)
        fq.fp4q_quantize_fp8(x, b, bufs[0][:, :K], bufs[1][:, :n], bufs[2][:, :M], bufs[3][:, :k])
        want, want_s = fp8.quantize(host(x), tile)
        assert np.array_equal(to_np(bufs[0])[:, :K], want) and np.array_equal(to_np(bufs[1])[:, :n], want_s)
        assert (to_np(bufs[0])[:, K:] == 0xA5).all() and (to_np(bufs[1])[:, n:] == -7).all()
        assert (to_np(bufs[2])[:, M:] == 0xA5).all() and (to_np(bufs[3])[:, k:] == -7).all()


# ------------------------------------------------------------------ GEMM

def operands(fq, M, N, K, b_tile, seed, gain=1.0):
    pad = lambda n: -(-n // 8) * 8  # noqa: E731
    a = fq.quantize_fp8(activations(M, pad(K), seed)[:, :K])
    rng = np.random.default_rng(seed + 1)
    w = torch.from_numpy((rng.standard_normal((N, pad(K))) * gain).astype(np.float32)).to(torch.bfloat16).cuda()[:, :K]
    return a, fq.quantize_fp8(w, fq.FP4Q_FP8_TILE if b_tile else fq.FP4Q_FP8_ROW)


def reference(a, b, b_tile):
    return fp8.gemm(fp8.values(to_np(a[0]), to_np(a[1]), False), fp8.values(to_np(b[0]), to_np(b[1]), b_tile))


def check(D, want, total, K, what):
    tol = (K + 4 * -(-K // 128)) * 2.0 ** -23 * total + 1e-37
    if D.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    else:
        tol = tol + 2.0 ** -24 * np.abs(want)
    off = np.abs(to_np(D.double()) - want)
    assert np.isfinite(to_np(D.float())).all() and (off <= tol).all(), \
        f"{what}: {int((off > tol).sum())} of {off.size} outputs off, worst {np.max(off / tol)} of the tolerance"


GEMMS = [(1, 1, 1), (1, 256, 4096), (1, 8, 130), (2, 1000, 128), (7, 100, 129), (16, 136, 384), (17, 513, 300),
         (33, 257, 1024), (64, 128, 512), (65, 72, 1100), (100, 1000, 2100), (128, 256, 256), (129, 384, 640),
         (200, 300, 1000), (257, 520, 777), (300, 1030, 513), (1000, 264, 400), (37, 4096, 4352)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b_tile", [True, False])
@pytest.mark.parametrize("shape", GEMMS)
def test_gemm(fq, shape, b_tile, out):
    M, N, K = shape
    a, b = operands(fq, M, N, K, b_tile, M + N + K)
    D = fq.gemm_fp8(*a, *b, fq.FP4Q_FP8_TILE if b_tile else fq.FP4Q_FP8_ROW, out)
    check(D, *reference(a, b, b_tile), K, f"{shape}")


@pytest.mark.parametrize("M", [3, 40, 300])
def test_gemm_scales_differ_by_block(fq, M):
    """Scales of very different size in neighbouring rows and blocks, so that a misplaced one shows."""
    N, K = 300, 900
    a, b = operands(fq, M, N, K, False, 5)
    rng = np.random.default_rng(9)
    a[1].copy_(torch.from_numpy(np.exp2(rng.integers(-20, 20, a[1].shape)).astype(np.float32)))
    b[1].copy_(torch.from_numpy(np.exp2(rng.integers(-20, 20, b[1].shape)).astype(np.float32)))
    check(fq.gemm_fp8(*a, *b, fq.FP4Q_FP8_ROW, torch.float32), *reference(a, b, False), K, "scales")


@pytest.mark.parametrize("M,N", [(1, 130), (20, 130), (200, 130), (200, 128), (200, 132), (300, 129)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_gemm_writes_only_its_output(fq, M, N, out):
    K = 200
    a, b = operands(fq, M, N, K, True, 11)
    for ldd in (144, 137):  # rows 16 bytes apart in step, and not
        buf = torch.full((M + 2, ldd), 123.0, dtype=out, device="cuda").contiguous()
        flat = buf.view(-1)
        # the block starts one row into the buffer where that keeps it 16-byte aligned
        start = ldd if ldd % 8 == 0 else 8 * ldd if M >= 8 else 0
        d = flat.as_strided((M, N), (ldd, 1), start if start + (M - 1) * ldd + N <= flat.numel() else 0)
        at = d.storage_offset()
        fq.fp4q_gemm_fp8(*a, *b, fq.FP4Q_FP8_TILE, d)
        check(d, *reference(a, b, True), K, f"ldd {ldd}")
        rest = to_np(flat.float()).copy()
        for r in range(M):
            rest[at + r * ldd:at + r * ldd + N] = 123.0
        assert (rest == 123.0).all()


def test_gemm_ignores_bytes_past_the_operands(fq):
    """NaN codes and scales right behind the rows, columns and K that are used."""
    M, N, K = 21, 70, 200
    a, b = operands(fq, M, N, K, False, 13)
    big = []
    for (c, s), n in ((a, M), (b, N)):
        c2 = torch.full((n + 3, 240), 0x7F, dtype=torch.uint8, device="cuda")
        s2 = torch.full((5, n + 8 - n % 4), float("nan"), device="cuda")
        c2[:n, :K] = c
        s2[:2, :n] = s
        big.append((c2[:n, :K], s2[:2, :n]))
    D = fq.gemm_fp8(*big[0], *big[1], fq.FP4Q_FP8_ROW, torch.float32)
    check(D, *reference(a, b, False), K, "padding")


def test_gemm_keeps_a_nan_in_its_row(fq):
    for M in (5, 200):
        a, b = operands(fq, M, 256, 256, True, 17)
        a[0][2, 130] = 0x7F
        D = to_np(fq.gemm_fp8(*a, *b).float())
        assert np.isnan(D[2]).all() and np.isfinite(np.delete(D, 2, 0)).all()


def test_gemm_twice_is_the_same_and_follows_its_stream(fq):
    a, b = operands(fq, 48, 512, 2048, True, 19)
    first = fq.gemm_fp8(*a, *b, out_dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = fq.gemm_fp8(*a, *b, out_dtype=torch.float32)
    side.synchronize()
    assert torch.equal(first, again)


# ------------------------------------------------------------------ a linear layer and its gradients

def test_linear_layer_and_gradients(fq):
    """y = x W^T, dx = dy W, dW = dy^T x from one quantization of each of x, W and dy (both directions), against the
    formulas on the dequantized values, and against differences of L = <y, dy> (linear in x and in W)."""
    M, N, K = 203, 264, 392
    x, dy = activations(M, K, 23), activations(M, N, 24)
    w = activations(N, K, 25)
    xq = fq.quantize_fp8(x, fq.FP4Q_FP8_ROW, True)
    wq = fq.quantize_fp8(w, fq.FP4Q_FP8_TILE, True)
    gq = fq.quantize_fp8(dy, fq.FP4Q_FP8_ROW, True)
    y = fq.gemm_fp8(*xq[:2], *wq[:2], fq.FP4Q_FP8_TILE, torch.float32)
    dx = fq.gemm_fp8(*gq[:2], *wq[2:], fq.FP4Q_FP8_TILE, torch.float32)
    dw = fq.gemm_fp8(*gq[2:], *xq[2:], fq.FP4Q_FP8_ROW, torch.float32)
    check(y, *reference(xq[:2], wq[:2], True), K, "y")
    check(dx, *reference(gq[:2], wq[2:], True), N, "dx")
    check(dw, *reference(gq[2:], xq[2:], False), M, "dw")
    # differences of the loss along random directions: L(x + e) - L(x) = <dx, e>, up to the operands' quantization,
    # half an E4M3 step (2^-4 relative) in each factor
    rng = np.random.default_rng(26)
    X, W, G = (host(t).astype(np.float64) for t in (x, w, dy))
    for grad, part, loss in ((dx, X, lambda t: ((t @ W.T) * G).sum()), (dw, W, lambda t: ((X @ t.T) * G).sum())):
        for _ in range(3):
            e = rng.standard_normal(part.shape)
            diff = loss(part + 0.5 * e) - loss(part - 0.5 * e)
            got = (to_np(grad).astype(np.float64) * e).sum()
            scale = (np.abs(G).T @ np.abs(X) if grad is dw else np.abs(G) @ np.abs(W))
            assert abs(got - diff) <= (2 * 2.0 ** -4 + 2.0 ** -8 + 1e-4) * (scale * np.abs(e)).sum()


def test_graph_capture_and_replay(fq):
    """Quantize and multiply inside a graph, replayed on new inputs in the same buffers."""
    M, N, K = 24, 256, 640
    w = fq.quantize_fp8(activations(N, K, 31), fq.FP4Q_FP8_TILE)
    x = activations(M, K, 32)
    a = fq.alloc_fp8(M, K)
    d = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    fq.fp4q_quantize_fp8(x, fq.FP4Q_FP8_ROW, *a)
    fq.fp4q_gemm_fp8(*a, *w, fq.FP4Q_FP8_TILE, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.fp4q_quantize_fp8(x, fq.FP4Q_FP8_ROW, *a)
        fq.fp4q_gemm_fp8(*a, *w, fq.FP4Q_FP8_TILE, d)
    for seed in (33, 34):
        x.copy_(activations(M, K, seed))
        graph.replay()
        torch.cuda.synchronize()
        fresh = fq.quantize_fp8(x)
        assert torch.equal(fresh[0], a[0]) and torch.equal(fresh[1], a[1])
        assert torch.equal(d, fq.gemm_fp8(*fresh, *w))
        check(d, *reference(fresh, w, True), K, "replay")


def test_quantized_nvfp4_workload_values(fq):
    """The library's own synthetic activations, at one of its widths."""
    x = bits_to_torch_cuda(workloads.nvfp4_outliers(64, 4096, seed=41))
    got = fq.quantize_fp8(x)
    want = fp8.quantize(host(x), False)
    assert np.array_equal(to_np(got[0]), want[0]) and np.array_equal(to_np(got[1]), want[1])


def test_offsets_past_32_bits(fq):
    """More than 2^31 elements of x, codes and D: the last rows are those of a call on them alone."""
    M, K, N, last = 1_050_112, 2056, 2056, 4096  # whole blocks of 128 rows
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    x[:-last].fill_(1.0)
    x[-last:] = activations(last, K, 51)
    assert x.numel() > 2 ** 31
    for block, rows in ((fq.FP4Q_FP8_ROW, last), (fq.FP4Q_FP8_TILE, last // 128)):
        whole, part = fq.quantize_fp8(x, block, True), fq.quantize_fp8(x[-last:], block, True)
        assert torch.equal(whole[0][-last:], part[0]) and torch.equal(whole[1][:, -rows:], part[1])
        assert torch.equal(whole[2][:, -last:], part[2]) and torch.equal(whole[3][-last // 128:], part[3])
        if block == fq.FP4Q_FP8_ROW:
            a, alone = whole[:2], part[:2]
    alone_rows = fq.quantize_fp8(x)
    assert torch.equal(alone_rows[0], a[0]) and torch.equal(alone_rows[1], a[1])
    del whole, alone_rows, x
    w = fq.quantize_fp8(activations(N, K, 52), fq.FP4Q_FP8_TILE)
    D = fq.gemm_fp8(*a, *w)
    assert D.numel() > 2 ** 31 and torch.equal(D[-last:], fq.gemm_fp8(*alone, *w))


# ------------------------------------------------------------------ NaN in blocks without numbers

@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("shape", [(1, 128), (3, 200), (130, 300)])
def test_quantize_keeps_nans_of_blocks_without_numbers(fq, shape, block):
    """A row, a tile and a column that are NaN throughout, and NaN among zeros: the NaN code wherever x is NaN."""
    M, K = shape
    x = activations(M, -(-K // 8) * 8, 61)[:, :K]
    x[0] = float("nan")
    if M > 2:
        x[:, 128:] = 0.0
        x[1, 130] = float("nan")
        x[2] = -0.0
        x[2, K - 1] = float("nan")
        x[:, 7] = float("nan")
    if M > 128:
        x[:128, :128] = float("nan")
    tile = block == "tile"
    got = fq.quantize_fp8(x, fq.FP4Q_FP8_TILE if tile else fq.FP4Q_FP8_ROW, True)
    alone = fq.quantize_fp8(x, fq.FP4Q_FP8_TILE if tile else fq.FP4Q_FP8_ROW)
    assert torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1])
    for (c, s), v in ((got[:2], host(x)), (got[2:], np.ascontiguousarray(host(x).T))):
        want, want_s = fp8.quantize(v, tile)
        assert np.array_equal(to_np(s), want_s) and np.array_equal(to_np(c) == 0x7F, np.isnan(v))
        assert np.array_equal(to_np(c), want)


@pytest.mark.parametrize("M", [1, 5, 200])
def test_gemm_of_a_row_that_is_all_nan(fq, M):
    """The row's products are NaN, not zeros, and the others' are as without it."""
    N, K = 300, 392
    x = activations(M, K, 63)
    w = fq.quantize_fp8(activations(N, K, 64), fq.FP4Q_FP8_TILE)
    clean = fq.gemm_fp8(*fq.quantize_fp8(x), *w)
    x[M // 2] = float("nan")
    D = fq.gemm_fp8(*fq.quantize_fp8(x), *w)
    rest = [i for i in range(M) if i != M // 2]
    assert torch.isnan(D[M // 2]).all() and torch.equal(D[rest], clean[rest])


# ------------------------------------------------------------------ bytes around an output; gradients against differences

@pytest.mark.parametrize("M,N", [(1, 130), (20, 130), (200, 130), (200, 128), (200, 132), (300, 129)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ldd", [137, 139, 144])
def test_gemm_writes_nothing_around_its_output(fq, M, N, out, ldd):
    """The output begins eight rows into a buffer (16-byte aligned whatever the row's length) and ends before it does."""
    K = 200
    a, b = operands(fq, M, N, K, True, 11)
    flat = torch.full(((M + 16) * ldd,), 123.0, dtype=out, device="cuda")
    at = 8 * ldd
    d = flat.as_strided((M, N), (ldd, 1), at)
    assert d.data_ptr() % 16 == 0 and 0 < at and at + (M - 1) * ldd + N < flat.numel()
    fq.fp4q_gemm_fp8(*a, *b, fq.FP4Q_FP8_TILE, d)
    check(d, *reference(a, b, True), K, f"ldd {ldd}")
    rest = to_np(flat.float()).copy()
    for r in range(M):
        rest[at + r * ldd:at + r * ldd + N] = 123.0
    assert (rest == 123.0).all()


def test_gradients_against_differences_along_the_gradient(fq):
    """L(x + e/2) - L(x - e/2) = <dL/dx, e> for L = <x W^T, dy>, which is linear in x and in W, with e the signs of the
    true gradient: the sum of its magnitudes, which a wrong gradient misses.

    Tolerance.  With dx' = G' W' (G' = G + dG, W' = W + dW: the quantized operands),
      <dx' - dx, e> = sum dG_in (e W^T)_in + sum dW_nk (G^T e)_nk + sum e dG dW.
    A rounding to E4M3 is off by at most r = 2^-4 |v| + 2^-10 s (s the block's scale, at most max |v| / 448).  As sums
    of independent bounded terms (e depends on neither rounding) the first two leave 6 sqrt(sum (bound of a term)^2)
    with probability below 2 exp(-18) (Hoeffding); the products of two roundings are such a sum too.  The fp32 sums of
    the GEMM add their worst case, (N + 4 ceil(N/128)) 2^-23 sum |G'| |W'|."""
    M, N, K = 203, 264, 392
    x, dy, w = activations(M, K, 23), activations(M, N, 24), activations(N, K, 25)
    xq = fq.quantize_fp8(x, fq.FP4Q_FP8_ROW, True)
    wq = fq.quantize_fp8(w, fq.FP4Q_FP8_TILE, True)
    gq = fq.quantize_fp8(dy, fq.FP4Q_FP8_ROW, True)
    dx = fq.gemm_fp8(*gq[:2], *wq[2:], fq.FP4Q_FP8_TILE, torch.float32)
    dw = fq.gemm_fp8(*gq[2:], *xq[2:], fq.FP4Q_FP8_ROW, torch.float32)
    X, W, G = (host(t).astype(np.float64) for t in (x, w, dy))
    off = lambda v: 2.0 ** -4 * np.abs(v) + 2.0 ** -10 * np.abs(v).max() / 448  # noqa: E731
    rss = lambda *terms: np.sqrt(sum((t ** 2).sum() for t in terms))  # noqa: E731
    for got, part, left, right, loss in ((dx, X, G, W, lambda t: ((t @ W.T) * G).sum()), (dw, W, G.T, X, lambda t: ((X @ t.T) * G).sum())):
        e = np.sign(left @ right)  # of the true gradient
        diff = loss(part + 0.5 * e) - loss(part - 0.5 * e)
        got = to_np(got.double())
        n = left.shape[1]
        both = np.sqrt(((off(left) ** 2).sum(0) * (off(right) ** 2).sum(1)).sum())
        tol = 6 * (rss(off(left) * (e @ right.T), off(right) * (left.T @ e)) + both) + \
            (n + 4 * -(-n // 128)) * 2.0 ** -23 * 1.2 * (np.abs(left) @ np.abs(right)).sum()
        assert abs((got * e).sum() - diff) <= tol
        # what this test is there to reject: no gradient, the negated one, one of another size or a row off
        for wrong in (np.zeros_like(got), -got, 10 * got, 0.5 * got, np.roll(got, 1, 0)):
            assert abs((wrong * e).sum() - diff) > tol
