"""Host-side refusals of the 8-bit entry points (no GPU, no launch)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def fq():
    from fp4_micro_block_b200 import build
    build.build()
    import fp4_micro_block_b200 as m
    return m


# Fake, aligned, never dereferenced addresses.
X, A, SA, B, SB, D, CU, LENS, TAB = (0x10000 * i for i in range(1, 10))


def test_quantize_refusals(fq):
    q = fq.lib().fp4q_quantize_fp8
    ok = [X, 4, 200, 200, 0, A, 208, SA, 4, B, 16, SB, 200, None]
    bad = lambda i, v: q(*[v if j == i else a for j, a in enumerate(ok)])  # noqa: E731
    assert bad(1, -1) == bad(2, 0) == bad(3, 199) == bad(4, 2) == bad(0, None) == fq.FP4Q_ERR_INVALID_ARG
    assert bad(7, None) == bad(11, None) == bad(6, 192) == bad(10, 0) == bad(8, 0) == fq.FP4Q_ERR_INVALID_ARG
    assert bad(12, 196) == fq.FP4Q_ERR_INVALID_ARG
    assert bad(1, 1 << 31) == bad(3, 1 << 31) == fq.FP4Q_ERR_UNSUPPORTED
    assert bad(3, 201) == bad(0, X + 8) == bad(6, 201) == bad(5, A + 8) == bad(7, SA + 4) == fq.FP4Q_ERR_ALIGNMENT
    assert bad(8, 5) == bad(10, 17) == bad(12, 202) == fq.FP4Q_ERR_ALIGNMENT
    assert q(X, 4, 200, 200, 0, None, 0, None, 0, None, 0, None, 0, None) == fq.FP4Q_ERR_INVALID_ARG
    assert q(None, 0, 200, 200, 1, None, 0, None, 0, None, 0, None, 0, None) == fq.FP4Q_OK


def test_gemm_refusals(fq):
    g = fq.lib().fp4q_gemm_fp8
    ok = [A, 208, SA, 8, B, 208, SB, 4, 1, 5, 300, 200, D, 300, 1, None]
    bad = lambda i, v: g(*[v if j == i else a for j, a in enumerate(ok)])  # noqa: E731
    for i, v in ((0, None), (2, None), (4, None), (6, None), (12, None), (1, 192), (3, 4), (5, 192), (8, 2), (9, -1),
                 (10, 0), (11, 0), (13, 299), (14, 2), (7, 0), (7, 2)):
        assert bad(i, v) == fq.FP4Q_ERR_INVALID_ARG, (i, v)
    # per-row scales of B need a column for every row
    assert bad(8, 0) == fq.FP4Q_ERR_INVALID_ARG
    for i, v in ((1, 201), (3, 9), (5, 210), (7, 5), (0, A + 8), (2, SA + 4), (4, B + 1), (6, SB + 8), (12, D + 2)):
        assert bad(i, v) == fq.FP4Q_ERR_ALIGNMENT, (i, v)
    for i in (9, 10, 11):
        assert bad(i, 1 << 31) in (fq.FP4Q_ERR_UNSUPPORTED, fq.FP4Q_ERR_INVALID_ARG)
    assert bad(9, 0) == fq.FP4Q_OK


def cache(fq, **over):
    c = dict(k=A, v=B, k_scale=SA, v_scale=SB, num_pages=10, num_kv_heads=2, page_size=64, head_dim=128,
             block_table=TAB, table_stride=3)
    c.update(over)
    return fq.Fp4qKvCache(**c)


BAD_CACHES = [(dict(num_pages=-1), 1), (dict(num_kv_heads=0), 1), (dict(page_size=0), 1), (dict(head_dim=-64), 1),
              (dict(table_stride=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1),
              (dict(v_scale=None), 1), (dict(block_table=None), 1), (dict(num_pages=0), 1), (dict(table_stride=0), 1),
              (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(head_dim=96), 2),
              (dict(num_pages=1 << 30), 2), (dict(k=A + 8), 3), (dict(v=B + 4), 3), (dict(k_scale=SA + 2), 3),
              (dict(block_table=TAB + 2), 3)]


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_cache_refusals(fq, over, status):
    c = cache(fq, **over)
    L = fq.lib()
    assert L.fp4q_kv_append_fp8(X, 256, X, 256, 5, C.addressof(c), CU, LENS, 2, 5, None) == status
    assert L.fp4q_attention_fp8(X, 512, 5, 4, C.addressof(c), CU, LENS, 2, 5, 100, 1, 0.1, D, 512, None, None, 0,
                                None) == status


def test_append_refusals(fq):
    c = cache(fq)
    ok = [X, 256, X, 256, 5, C.addressof(c), CU, LENS, 2, 5, None]
    bad = lambda i, v: fq.lib().fp4q_kv_append_fp8(*[v if j == i else a for j, a in enumerate(ok)])  # noqa: E731
    for i, v in ((0, None), (2, None), (5, None), (6, None), (7, None), (1, 128), (3, 255), (4, -1), (8, -1), (9, -1)):
        assert bad(i, v) == fq.FP4Q_ERR_INVALID_ARG, (i, v)
    for i, v in ((0, X + 8), (1, 257), (3, 260), (6, CU + 2), (7, LENS + 1)):
        assert bad(i, v) == fq.FP4Q_ERR_ALIGNMENT, (i, v)
    for i in (1, 4, 8, 9):
        assert bad(i, 1 << 31) == fq.FP4Q_ERR_UNSUPPORTED, i
    for i in (4, 8, 9):
        assert bad(i, 0) == fq.FP4Q_OK


def test_attention_refusals(fq):
    c = cache(fq)
    ok = [X, 512, 5, 4, C.addressof(c), CU, LENS, 2, 5, 100, 1, 0.1, D, 512, None, None, 0, None]
    bad = lambda i, v: fq.lib().fp4q_attention_fp8(*[v if j == i else a for j, a in enumerate(ok)])  # noqa: E731
    for i, v in ((0, None), (4, None), (5, None), (6, None), (12, None), (1, 511), (13, 504), (2, -1), (3, 0), (3, 3),
                 (7, -1), (8, -1), (9, -1), (10, 2), (11, float("nan")), (11, float("inf"))):
        assert bad(i, v) == fq.FP4Q_ERR_INVALID_ARG, (i, v)
    for i, v in ((0, X + 8), (1, 514), (13, 515), (5, CU + 2), (6, LENS + 1), (12, D + 4), (14, D + 2)):
        assert bad(i, v) == fq.FP4Q_ERR_ALIGNMENT, (i, v)
    for i in (1, 2, 7, 8, 9, 13):
        assert bad(i, 1 << 31) == fq.FP4Q_ERR_UNSUPPORTED, i
    for i in (2, 7, 8):
        assert bad(i, 0) == fq.FP4Q_OK
    w = fq.lib().fp4q_attention_fp8_workspace_bytes
    none = C.c_size_t(-1).value
    assert w(-1, 1, 1, 4, 2, 64) == w(1, -1, 1, 4, 2, 64) == w(1, 1, -1, 4, 2, 64) == w(1, 1, 1, 3, 2, 64) == none
    assert w(1, 1, 1, 4, 0, 64) == w(1, 1, 1, 4, 2, 0) == none
    assert w(0, 1, 1, 4, 2, 64) == w(1, 0, 1, 4, 2, 64) == 0


def test_binding_refuses_host_tensors_wrong_types_and_shapes(fq):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fq.fp4q_quantize_fp8(x, fq.FP4Q_FP8_ROW, *fq.alloc_fp8(4, 64, device="cpu"))
    with pytest.raises(ValueError):
        fq._want(x, "x", (torch.uint8,), 4, 64)
    with pytest.raises(ValueError):
        fq._want(x, "x", (torch.bfloat16,), 4, 65)
    codes, scales = fq.alloc_fp8(4, 70, device="cpu")
    assert codes.shape == (4, 70) and codes.stride(0) == 80 and scales.shape == (1, 4)
    assert fq._fp8_side(codes, scales, 4, 70, fq.FP4Q_FP8_ROW, "x") == (80, 4)
    codes, scales = fq.alloc_fp8(300, 300, fq.FP4Q_FP8_TILE, device="cpu")
    assert fq._fp8_side(codes, scales, 300, 300, fq.FP4Q_FP8_TILE, "x") == (304, 4) and scales.shape == (3, 3)
    with pytest.raises(ValueError):
        fq._fp8_side(codes, scales, 300, 300, fq.FP4Q_FP8_ROW, "x")
    with pytest.raises(ValueError):
        fq._fp8_side(codes.t(), scales, 300, 300, fq.FP4Q_FP8_TILE, "x")
    cache = fq.alloc_kv_cache(3, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        fq._kv_cache(*cache, torch.zeros((1, 2), dtype=torch.int64))
    with pytest.raises(ValueError):
        fq._tokens(torch.zeros((2, 4, 64), dtype=torch.bfloat16).transpose(0, 1), "q", 4, 2, 64)
    with pytest.raises(ValueError):
        fq._tokens(torch.zeros((2, 4, 64)), "q", 2, 4, 64)
    assert fq._tokens(torch.zeros((5, 8, 64), dtype=torch.bfloat16)[:, 2:4], "q", 5, 2, 64) == 512
    c = fq.Fp4qKvCache(1, 2, 3, 4, 5, 6, 7, 8, 9, 10)
    assert bytes(c) == fq._KV.pack(1, 2, 3, 4, 5, 6, 7, 8, 9, 10)


def test_workspace_query_refuses_the_head_dims_that_the_call_refuses(fq):
    w = fq.lib().fp4q_attention_fp8_workspace_bytes
    for dim in (1, 32, 96, 512):
        assert w(1, 1, 1, 4, 2, dim) == C.c_size_t(-1).value


def test_binding_refuses_codes_without_scales(fq):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    codes, scales = fq.alloc_fp8(4, 64, device="cpu")
    for out in ((codes, None), (None, scales), (codes, scales, codes, None), (codes, scales, None, scales)):
        with pytest.raises(ValueError, match="together"):
            fq.fp4q_quantize_fp8(x, fq.FP4Q_FP8_ROW, *out)


def test_attention_refuses_work_that_31_bits_do_not_count(fq):
    """Before anything of the device is asked: the products of batch, heads and row tiles themselves may pass 64 bits."""
    c = cache(fq, num_kv_heads=65536)
    row = 65536 * 128
    call = lambda batch, max_q, max_len, heads: fq.lib().fp4q_attention_fp8(  # noqa: E731
        X, row * heads // 65536, 5, heads, C.addressof(c), CU, LENS, batch, max_q, max_len, 1, 0.1, D,
        row * heads // 65536, None, None, 0, None)
    assert call(1 << 30, 1 << 25, 64, 65536) == fq.FP4Q_ERR_UNSUPPORTED
    assert call(1 << 30, 1, 64, 65536) == fq.FP4Q_ERR_UNSUPPORTED
    assert call(1, (1 << 30) + 1, 64, 65536) == fq.FP4Q_ERR_UNSUPPORTED
    assert call(1, (1 << 29) + 1, 64, 131072) == fq.FP4Q_ERR_UNSUPPORTED
    assert call(1, 1, (1 << 30) + 1, 65536) == fq.FP4Q_ERR_UNSUPPORTED
    assert call(4, 1 << 23, 64, 65536) == fq.FP4Q_ERR_UNSUPPORTED


def test_every_workspace_is_contiguous(fq):
    """A view with gaps, or one that repeats its elements, has fewer bytes behind its pointer than it counts or bytes
    between them that are not its own."""
    x = torch.zeros((16, 64), dtype=torch.bfloat16)
    buf = torch.zeros(64, dtype=torch.uint8)
    f = torch.zeros(1)
    perm = torch.zeros(64, dtype=torch.int32)
    kv = fq.alloc_kv_cache(3, 2, 16, 64, device="cpu")
    table = torch.zeros((1, 2), dtype=torch.int32)
    cu, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    for ws in (buf[::2], buf[:1].expand(32768), buf.view(8, 8).t(), buf.view(8, 8)[:, :4]):
        for call in (lambda: fq.fp4q_attention_fp8(q, *kv, table, cu, lens, 1, 16, q, workspace=ws),
                     lambda: fq.attention_fp8(q, *kv, table, cu, lens, 1, 16, ws=ws),
                     lambda: fq.fp4q_quantize_nvfp4(x, buf, buf, f, workspace=ws),
                     lambda: fq.fp4q_hadamard_quantize(x, 64, fq.FP4Q_NVFP4, buf, buf, f, workspace=ws),
                     lambda: fq.fp4q_hadamard_quantize_signed(x, 64, [1, 2], fq.FP4Q_NVFP4, buf, buf, f, workspace=ws),
                     lambda: fq.fp4q_arc_quantize(x, perm, 1e-6, perm, None, fq.FP4Q_NVFP4, buf, buf, f, workspace=ws)):
            with pytest.raises(ValueError, match="contiguous"):
                call()
