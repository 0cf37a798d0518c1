"""Bounded device waits of the 8-bit kernels that run out, on a GPU, without a fault.

The test build of the library (compiled with FP4Q_TEST_HOOKS: the poll limit cut
to 2^14, and a hook that withholds one group of copies) arms a barrier of CTA 0
for copies that it never issues.  Every role that waits for them, or for what
would be made of them, gives up by its limit; copies and products that are on
their way land first; the CTA frees its tensor memory and leaves, and the CTAs of
its cluster with it.  The call must complete, fp4q_device_error() must report
bit 0, and the next calls, through the test build and through the production
library, must give the results of a call that nothing was withheld from.
"""
import ctypes as C

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    from fp4_micro_block_b200 import build
    import fp4_micro_block_b200 as fq
    build.build()
    T = fq.declare(C.CDLL(build.build(test_hooks=True)))
    T.fp4q_test_skip_copy.restype = None
    T.fp4q_test_skip_copy.argtypes = [C.c_int64]
    assert T.fp4q_device_error() == 0 and fq.fp4q_device_error() == 0
    return fq, T


def runs_out(libs, monkeypatch, call, which):
    """The call with copies number `which` of CTA 0 withheld, and afterwards without."""
    fq, T = libs
    want = call()
    with monkeypatch.context() as m:
        m.setattr(fq, "_lib", T)
        for i in which:
            T.fp4q_test_skip_copy(i)
            call()  # the launch itself is fine; the waits run out on the device
            torch.cuda.synchronize()  # returns: every wait ended by its limit
            assert T.fp4q_device_error() == 1, i
            assert T.fp4q_device_error() == 0  # read and cleared
            again = call()
            torch.cuda.synchronize()
            assert T.fp4q_device_error() == 0
            assert all(torch.equal(a, b) for a, b in zip(again, want)), i
    again = call()
    torch.cuda.synchronize()
    assert fq.fp4q_device_error() == 0 and all(torch.equal(a, b) for a, b in zip(again, want))


def activations(M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("tile", [False, True])
def test_quantizer(libs, monkeypatch, tile):
    """The first, a middle and the last of the four tiles of CTA 0."""
    fq = libs[0]
    x = activations(4096, 4096, 1)
    block = fq.FP4Q_FP8_TILE if tile else fq.FP4Q_FP8_ROW
    runs_out(libs, monkeypatch, lambda: fq.quantize_fp8(x, block, True), (0, 1, 2, 3))


# (M, N, K, tile scales of B, withheld K blocks): K split over a cluster (its first block, and one behind the ring's
# first turn), not split; 128 x 256 tiles, one for a CTA and several (within the third)
GEMMS = [(1, 4096, 4096, True, (0, 5)), (40, 256, 2048, True, (0, 1)), (40, 16384, 4096, False, (2, 9, 31)),
         (100, 1024, 1024, True, (1,)), (512, 4096, 2048, True, (0, 7, 15)), (512, 4096, 2048, False, (3,)),
         (8192, 4096, 512, True, (9,)), (8192, 4096, 512, False, (0, 27))]


@pytest.mark.parametrize("M,N,K,tile,which", GEMMS)
def test_gemm(libs, monkeypatch, M, N, K, tile, which):
    fq = libs[0]
    block = fq.FP4Q_FP8_TILE if tile else fq.FP4Q_FP8_ROW
    a, b = fq.quantize_fp8(activations(M, K, 2)), fq.quantize_fp8(activations(N, K, 3), block)
    runs_out(libs, monkeypatch, lambda: (fq.gemm_fp8(*a, *b, block),), which)


# (sequences, queries, keys, K/V heads, group, withheld turns or tiles): 16 rows a CTA in a cluster, with the splits
# joined by a second kernel, in several turns of the ring; 128 rows a CTA, of two and of many tiles, and keys split
ATTENTIONS = [(1, 1, 500, 8, 4, (0, 3)), (1, 1, 9000, 1, 4, (1,)), (32, 1, 1000, 8, 4, (0, 6, 13)),
              (24, 40, 200, 1, 2, (0, 1)), (2, 1000, 3000, 4, 4, (0, 1, 2, 9)), (2, 64, 1537, 8, 2, (0, 2))]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,new,L,heads,G,which", ATTENTIONS)
def test_attention(libs, monkeypatch, B, new, L, heads, G, which, D):
    fq = libs[0]
    page, width = 64, -(-L // 64)
    rng = np.random.default_rng(4)
    cache = fq.alloc_kv_cache(B * width, heads, page, D)
    table = torch.from_numpy(rng.permutation(B * width).reshape(B, width).astype(np.int32)).cuda()
    k, v = (activations(B * L, heads * D, s).view(B * L, heads, D) for s in (5, 6))
    cu = lambda n: torch.arange(0, (B + 1) * n, n, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    fq.kv_append_fp8(k, v, *cache, table, cu(L), lens, L)
    q = activations(B * new, heads * G * D, 7).view(B * new, heads * G, D)
    runs_out(libs, monkeypatch, lambda: fq.attention_fp8(q, *cache, table, cu(new), lens, new, L), which)
