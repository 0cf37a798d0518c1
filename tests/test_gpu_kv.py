"""The paged 8-bit K/V cache, its writer and the attention over it, against the oracle, on a GPU.

Append: bit-exact codes and scales.

Attention tolerance, per query, head and column (p = the exact probabilities):
 - the output's rounding, half a bf16 step: 2^-8 |o|;
 - the logits: a D-long fp32 sum of products that are exact (bf16 x E4M3) but
   for chopping, at most (D + 8) 2^-23 of R = max_j scale * sum |q| |k_j|, which
   moves a probability by twice that, relative (numerator and denominator);
 - each probability's rounding to fp16 (2^-11 relative) and its exponential
   (2 units in the last place, and those of its argument: 2^-22 + R 2^-22);
 - the fp32 sums over the keys: len 2^-23;
all of sum_j p_j |v_j|.  Probabilities below fp16's normals are off by at most
2^-25 of the largest weight: len 2^-25 max |v|.
lse: the logits' part, the exponentials' and the sum's, and its own rounding.
"""
import numpy as np
import pytest
import torch

from oracle import fp8
from parity import bf16_torch_to_bits, to_np

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
    return fp8.bf16_values(bf16_torch_to_bits(t))


def bf16(rng, *shape, gain=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * gain).astype(np.float32)).to(torch.bfloat16).cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cum(ns):
    return [0] + list(np.cumsum(ns))


def table_for(rng, lens, page, pool, width=None):
    """Distinct random pages for each sequence; unused entries hold an id that must not be read."""
    need = [-(-n // page) for n in lens]
    ids = rng.permutation(pool)[:sum(need)]
    t = np.full((len(lens), width or max(need + [1])), 2 ** 30, np.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = ids[at:at + n]
        at += n
    return t


def random_cache(rng, pool, heads, page, D, spread=2.0):
    """Codes of every value but NaN, page scales over a few octaves, powers of two and not."""
    out = []
    for _ in range(2):
        c = rng.integers(0, 256, (pool, heads, page, D)).astype(np.uint8)
        c[(c & 0x7F) > 0x70] &= 0x8F  # mostly moderate magnitudes, none of them NaN
        out.append(c)
    for _ in range(2):
        out.append((np.exp2(rng.uniform(-spread, spread, (pool, heads))) / 64).astype(np.float32))
    return out


def up(arrays):
    return [torch.from_numpy(np.array(a)).cuda() for a in arrays]


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D,heads", [(64, 1), (128, 2), (256, 3)])
def test_append(fq, page, D, heads):
    """Sequences that begin, end and go on inside pages, at page borders, with nothing new, of one token and many."""
    rng = np.random.default_rng(page + D)
    new = [1, 0, page, page + 1, 3 * page - 5, 7, 2, 1]
    old = [0, 40, page, page - 1, 5, 2 * page - 3, page, page - 1]
    lens = [n + o for n, o in zip(new, old)]
    pool = sum(-(-n // page) for n in lens) + 2
    cache = random_cache(rng, pool, heads, page, D)
    for s in cache[2:]:
        s[:] = np.exp2(rng.integers(-9, -5, s.shape))
        s[::5] = 0.0  # pages of zeros so far
    cache[0][cache[2] == 0] = 0
    cache[1][cache[3] == 0] = 0
    table = table_for(rng, lens, page, pool)
    k, v = bf16(rng, sum(new) + 3, heads, D), bf16(rng, sum(new) + 3, heads, D, gain=0.01)
    dev = up(cache)
    fq.kv_append_fp8(k, v, *dev, i32(table.tolist()), i32(cum(new)), i32(lens), max(new))
    want = fp8.kv_append(host(k), host(v), cache, table, cum(new), lens)
    for got, w, name in zip(dev, want, ("k", "v", "k_scale", "v_scale")):
        assert np.array_equal(to_np(got), w), name


def test_append_token_by_token(fq):
    """A growing sequence: every step equals the oracle's, and rows past the end keep what they held."""
    rng = np.random.default_rng(3)
    page, D, heads = 16, 64, 2
    cache = random_cache(rng, 4, heads, page, D)
    dev = up(cache)
    table = np.array([[2, 0, 3]], np.int32)
    for t in range(36):
        k, v = bf16(rng, 1, heads, D, gain=1.1 ** t), bf16(rng, 1, heads, D, gain=1.0 / (1 + t))
        fq.kv_append_fp8(k, v, *dev, i32(table.tolist()), i32([0, 1]), i32([t + 1]), 1)
        cache = fp8.kv_append(host(k), host(v), cache, table, [0, 1], [t + 1])
    for got, w in zip(dev, cache):
        assert np.array_equal(to_np(got), w)


def test_append_strided_and_extreme_values(fq):
    """K and V as slices of one projection; zeros, subnormals, the largest values, NaN and infinities."""
    rng = np.random.default_rng(5)
    page, D, heads, n = 32, 128, 2, 70
    qkv = bf16(rng, n, 4 * heads, D)
    qkv[:32, :, :] = 0
    qkv[40, heads, 3] = float("nan")
    qkv[64:, heads:, :] *= 1e-38
    qkv[33, 2 * heads, 5] = 3.0e38
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:3 * heads]
    cache = [np.zeros((5, heads, page, D), np.uint8) for _ in range(2)] + [np.ones((5, heads), np.float32) for _ in range(2)]
    table = np.array([[4, 1, 2]], np.int32)
    dev = up(cache)
    fq.kv_append_fp8(k, v, *dev, i32(table.tolist()), i32([0, n]), i32([n]), n)
    want = fp8.kv_append(host(k.contiguous()), host(v.contiguous()), cache, table, [0, n], [n])
    for got, w in zip(dev, want):
        assert np.array_equal(to_np(got), w)
    inf = qkv[:1, :heads].clone()
    inf[0, 0, 0] = float("inf")
    dev = up(cache)
    fq.kv_append_fp8(inf, inf, *dev, i32(table.tolist()), i32([0, 1]), i32([1]), 1)
    assert float(dev[2][4, 0]) == 2.0 ** 120 and int(dev[0][4, 0, 0, 0]) == 0x7E


def test_append_to_pages_with_scales_that_are_no_powers_of_two(fq):
    """A page that carries a calibrated scale keeps it while it suffices, and moves to a power of two where it does not."""
    rng = np.random.default_rng(8)
    page, D, heads = 32, 64, 2
    cache = random_cache(rng, 4, heads, page, D)
    for s in cache[2:]:
        s[:] = np.float32(0.013) * np.float32([[1], [3], [0.1], [1]])
    table = np.array([[0], [1], [2]], np.int32)
    k, v = bf16(rng, 30, heads, D), bf16(rng, 30, heads, D, gain=0.5)
    dev = up(cache)
    fq.kv_append_fp8(k, v, *dev, i32(table.tolist()), i32([0, 10, 20, 30]), i32([12, 31, 20]), 10)
    want = fp8.kv_append(host(k), host(v), cache, table, [0, 10, 20, 30], [12, 31, 20])
    for got, w in zip(dev, want):
        assert np.array_equal(to_np(got), w)


def test_append_reports_entries_out_of_range(fq):
    """Bad page ids, positions past the table and offsets past the tokens write nothing and are reported."""
    rng = np.random.default_rng(6)
    page, D, heads = 16, 64, 1
    cache = random_cache(rng, 3, heads, page, D)
    k = bf16(rng, 4, heads, D)
    assert fq.fp4q_device_error() == 0
    for table, cu, lens, most in (([[3]], [0, 1], [1], 1), ([[-1]], [0, 1], [1], 1), ([[0]], [0, 1], [17], 1),
                                  ([[0]], [0, 5], [5], 8), ([[0]], [0, 3], [3], 2), ([[0]], [0, 2], [1], 2),
                                  ([[0]], [2, 1], [1], 2), ([[0]], [-1, 1], [2], 2)):
        dev = up(cache)
        fq.kv_append_fp8(k, k, *dev, i32(table), i32(cu), i32(lens), most)
        assert fq.fp4q_device_error() == 2, (table, cu, lens)
        for got, w in zip(dev, cache):
            assert np.array_equal(to_np(got), w)


# ------------------------------------------------------------------ attention

def run(fq, rng, new, lens, page, D, heads, G, causal=True, cache=None, pool=None, q=None, **kw):
    pool = pool or sum(-(-n // page) for n in lens) + 1
    cache = random_cache(rng, pool, heads, page, D) if cache is None else cache
    table = table_for(rng, lens, page, pool)
    cu = cum(new)
    q = bf16(rng, cu[-1], heads * G, D) if q is None else q
    # codes past the sequences' ends are NaN: they must not be seen
    for b, n in enumerate(lens):
        if n % page:
            cache[0][table[b, n // page], :, n % page:] = 0x7F
            cache[1][table[b, n // page], :, n % page:] = 0xFF
    dev = up(cache)
    o, lse = fq.attention_fp8(q, *dev, i32(table.tolist()), i32(cu), i32(lens), max(new), max(lens), causal, **kw)
    compare(o, lse, q, cache, table, cu, lens, causal, kw.get("softmax_scale") or D ** -0.5)
    return o, lse, q, dev, table, cu


def compare(o, lse, q, cache, table, cu, lens, causal, scale):
    D = q.shape[2]
    want, want_lse, pv, reach, vmax = fp8.attention(host(q), cache, table, cu, lens, causal, scale)
    most = max(list(lens) + [1])
    logits = (D + 8) * 2.0 ** -23 * reach
    rel = 2 * logits + 2.0 ** -11 + 2.0 ** -22 + reach * 2.0 ** -22 + most * 2.0 ** -23
    tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * (rel[..., None] * pv + most * 2.0 ** -25 * vmax[..., None]) + 1e-38
    off = np.abs(to_np(o.double()) - want)
    assert np.isfinite(to_np(o.float())).all() and (off <= tol).all(), \
        f"{int((off > tol).sum())} of {off.size} off, worst {np.nanmax(off / tol)} of the tolerance"
    got, none = to_np(lse.double()), np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got), none)
    ltol = logits + 2.0 ** -21 + reach * 2.0 ** -22 + most * 2.0 ** -23 + 2.0 ** -22 * np.abs(want_lse)
    assert (np.abs(got[~none] - want_lse[~none]) <= ltol[~none]).all()
    assert (to_np(o.float())[none] == 0).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_single_tokens(fq, D, page):
    rng = np.random.default_rng(D + page)
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 300, 511, 900]
    run(fq, rng, [1] * len(lens), lens, page, D, 2, 4)


@pytest.mark.parametrize("heads,G", [(1, 1), (1, 8), (3, 5), (2, 16), (1, 20), (8, 1)])
def test_head_layouts(fq, heads, G):
    rng = np.random.default_rng(heads * 100 + G)
    run(fq, rng, [1, 1, 3], [70, 333, 12], 32, 128, heads, G)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,page,G", [(64, 16, 1), (128, 64, 4), (128, 128, 3), (256, 32, 2)])
def test_several_queries(fq, D, page, G, causal):
    """From the few tokens of a speculative step to chunks of a prompt, alone and over a cached prefix; sequences
    without queries, without keys, and with more queries than keys (rows that see nothing)."""
    rng = np.random.default_rng(D + page + G)
    run(fq, rng, [2, 5, 0, 17, 40, 130, 3, 9, 1], [2, 64, 50, 17, 200, 131, 0, 4, 77], page, D, 2, G, causal)


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_lengths_around_tiles(fq, D):
    rng = np.random.default_rng(D)
    run(fq, rng, [127, 128, 129, 64, 63, 65, 256, 255], [127, 128, 129, 200, 300, 65, 256, 400], 64, D, 1, 2)


@pytest.mark.parametrize("B", [1, 3])
def test_long_sequences(fq, B):
    rng = np.random.default_rng(11)
    run(fq, rng, [1] * B, [20000, 9000, 13][:B], 64, 128, 1, 4)


def test_softmax_scale_and_peaked_rows(fq):
    """A scale far from 1/sqrt(D): one key holds nearly all the weight, and a negative one."""
    rng = np.random.default_rng(12)
    for scale in (1.0, -0.3, 1e-6):
        run(fq, rng, [1, 4], [500, 100], 32, 64, 2, 2, softmax_scale=scale)


def test_page_scales_far_apart(fq):
    """Pages whose V scales differ by many octaves, zero scales among them, with the weight on the small ones."""
    rng = np.random.default_rng(13)
    page, D, heads, pool = 32, 64, 1, 12
    cache = random_cache(rng, pool, heads, page, D)
    cache[3][:, 0] = np.exp2(-6.0 * np.arange(pool)).astype(np.float32)
    cache[2][:, 0] = np.linspace(0.02, 0.2, pool).astype(np.float32)
    cache[3][5] = 0.0
    cache[2][7] = 0.0
    run(fq, rng, [1, 3], [300, 40], page, D, heads, 2, cache=cache, pool=pool)


def test_values_of_one_page_only_small(fq):
    """Every visible V scale far below one: the result is as exact as with ordinary ones."""
    rng = np.random.default_rng(14)
    cache = random_cache(rng, 8, 1, 32, 128)
    cache[3][:] = 2.0 ** -90
    run(fq, rng, [1, 20], [100, 60], 32, 128, 1, 2, cache=cache, pool=8)


@pytest.mark.parametrize("new", [1, 4, 40, 150])
def test_masked_nan_does_not_leak(fq, new):
    """A NaN in the last token's K and V reaches only the last query, which sees it."""
    rng = np.random.default_rng(15 + new)
    page, D, heads, G, L = 32, 128, 1, 2, 200
    pool = 8
    cache = random_cache(rng, pool, heads, page, D)
    table = table_for(rng, [L], page, pool)
    q = bf16(rng, new, heads * G, D)
    clean = fq.attention_fp8(q, *up(cache), i32(table.tolist()), i32([0, new]), i32([L]), new, L)
    for side in (0, 1):
        broken = [c.copy() for c in cache]
        broken[side][table[0, (L - 1) // page], 0, (L - 1) % page, 3] = 0x7F
        o, _ = fq.attention_fp8(q, *up(broken), i32(table.tolist()), i32([0, new]), i32([L]), new, L)
        assert torch.equal(o[:-1], clean[0][:-1])
        last = to_np(o[-1].float())
        if side == 0:
            assert np.isnan(last).all()
        else:
            assert np.isnan(last[:, 3]).all() and np.isfinite(np.delete(last, 3, 1)).all()


def test_rows_outside_the_sequences_are_left(fq):
    rng = np.random.default_rng(16)
    page, D, heads, G = 16, 64, 2, 2
    cache = random_cache(rng, 6, heads, page, D)
    table = table_for(rng, [20, 30], page, 6)
    q = bf16(rng, 12, heads * G, D)
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    cu = [2, 5, 9]
    dev = up(cache)
    ws = fq.attention_fp8_workspace(q, dev[0], 2, 4, 30)
    fq.fp4q_attention_fp8(q, *dev, i32(table.tolist()), i32(cu), i32([20, 30]), 4, 30, o, lse, workspace=ws)
    assert (o[:2] == 7).all() and (o[9:] == 7).all() and (lse[:2] == 7).all() and (lse[9:] == 7).all()
    part, part_lse = fq.attention_fp8(q[2:9].contiguous(), *dev, i32(table.tolist()), i32([0, 3, 7]), i32([20, 30]), 4, 30)
    assert torch.equal(o[2:9], part) and torch.equal(lse[2:9], part_lse)


def test_views_and_no_lse(fq):
    """Queries as a slice of a fused projection, outputs into a slice of a wider buffer."""
    rng = np.random.default_rng(17)
    page, D, heads, G = 64, 128, 2, 4
    for new, lens in (([1, 1], [100, 900]), ([30, 1], [100, 40])):
        o, lse, q, dev, table, cu = run(fq, rng, new, lens, page, D, heads, G)
        wide = torch.zeros((cu[-1], heads * G + 2 * heads, D), dtype=torch.bfloat16, device="cuda")
        wide[:, :heads * G] = q
        out = torch.full((cu[-1], heads * G + 3, D), 5.0, dtype=torch.bfloat16, device="cuda")
        ws = fq.attention_fp8_workspace(q, dev[0], 2, max(new), max(lens))
        fq.fp4q_attention_fp8(wide[:, :heads * G], *dev, i32(table.tolist()), i32(cu), i32(lens), max(new), max(lens),
                              out[:, :heads * G], workspace=ws)
        assert torch.equal(out[:, :heads * G], o) and (out[:, heads * G:] == 5).all()


def test_bounds_given_larger_than_the_lengths(fq):
    """max_q and max_len may exceed what the sequences have (a graph captured for the largest batch)."""
    rng = np.random.default_rng(18)
    lens, new = [5, 700, 64], [1, 2, 1]
    _, _, q, dev, table, cu = run(fq, rng, new, lens, 32, 64, 2, 2)
    for most_q, most in ((7, 64 * 32), (40, 5000)):
        wide = np.zeros((3, 160), np.int32)
        wide[:, :table.shape[1]] = table
        o, lse = fq.attention_fp8(q, *dev, i32(wide.tolist()), i32(cu), i32(lens), most_q, most)
        compare(o, lse, q, [to_np(t) for t in dev], table, cu, lens, True, 64 ** -0.5)


def test_entries_out_of_range_are_reported(fq):
    rng = np.random.default_rng(19)
    page, D, heads = 16, 64, 1
    cache = random_cache(rng, 3, heads, page, D)
    dev = up(cache)
    assert fq.fp4q_device_error() == 0
    for n in (1, 20):
        q = bf16(rng, n, 2, D)
        for table, cu, lens, most_q, most in (([[1, 3]], [0, n], [20], n, 32), ([[1, -5]], [0, n], [20], n, 32),
                                              ([[1, 2]], [0, n], [40], n, 64), ([[1, 2]], [0, n], [32], n, 20),
                                              ([[1, 2]], [0, n + 1], [20], n + 1, 32), ([[1, 2]], [0, n], [-1], n, 32),
                                              ([[1, 2]], [-1, n], [20], n + 1, 32)):
            fq.attention_fp8(q, *dev, i32(table), i32(cu), i32(lens), most_q, most)
            assert fq.fp4q_device_error() == 2, (table, cu, lens)


def test_workspace_refusals(fq):
    rng = np.random.default_rng(20)
    cache = up(random_cache(rng, 80, 1, 64, 128))
    q = bf16(rng, 1, 4, 128)
    n = fq.fp4q_attention_fp8_workspace_bytes(1, 1, 5000, 4, 1, 128)
    args = (q, *cache, i32([list(range(79))]), i32([0, 1]), i32([5000]), 1, 5000, torch.empty_like(q))
    if n:
        with pytest.raises(fq.Fp4qError):
            fq.fp4q_attention_fp8(*args)
        with pytest.raises(fq.Fp4qError):
            fq.fp4q_attention_fp8(*args, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
        with pytest.raises(fq.Fp4qError):
            fq.fp4q_attention_fp8(*args, workspace=torch.empty(n + 8, dtype=torch.uint8, device="cuda")[8:])
    fq.fp4q_attention_fp8(*args, workspace=torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"))


def test_streams_and_repeats(fq):
    """Two calls at once on two streams with a workspace each; the same call twice gives the same bits."""
    rng = np.random.default_rng(21)
    o, lse, q, dev, table, cu = run(fq, rng, [1, 1, 1], [5000, 700, 64], 64, 128, 1, 4)
    args = (*dev, i32(table.tolist()), i32(cu), i32([5000, 700, 64]), 1, 5000)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            outs += [fq.attention_fp8(q, *args) for _ in range(4)]
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)


@pytest.mark.parametrize("new", [1, 33])
def test_decoding_steps_in_a_graph(fq, new):
    """Append and attend inside a graph captured once for the largest lengths, replayed as the sequences grow; two
    graphs that share one workspace, replayed in turn on one stream."""
    rng = np.random.default_rng(22)
    page, D, heads, G, B, pool = 32, 128, 2, 2, 2, 40
    cache = [np.zeros((pool, heads, page, D), np.uint8) for _ in range(2)] + [np.zeros((pool, heads), np.float32) for _ in range(2)]
    dev = up(cache)
    table = rng.permutation(pool)[:36].reshape(2, 18).astype(np.int32)
    T = B * new
    q, k, v = bf16(rng, T, heads * G, D), bf16(rng, T, heads, D), bf16(rng, T, heads, D)
    tab, cu, lens = i32(table.tolist()), i32([0, new, T]), i32([new, new])
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    most = 18 * page
    ws = fq.attention_fp8_workspace(q, dev[0], B, new, most)

    def step():
        fq.fp4q_kv_append_fp8(k, v, *dev, tab, cu, lens, new)
        fq.fp4q_attention_fp8(q, *dev, tab, cu, lens, new, most, o, lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step()
    for t in dev:
        t.zero_()
    length = np.array([0, 0])
    for turn in range(6):
        for x, n in ((q, heads * G), (k, heads), (v, heads)):
            x.copy_(bf16(rng, T, n, D))
        length = length + new
        lens.copy_(i32(length.tolist()))
        graphs[turn % 2].replay()
        torch.cuda.synchronize()
        cache = fp8.kv_append(host(k), host(v), cache, table, [0, new, T], length)
        for got, w in zip(dev, cache):
            assert np.array_equal(to_np(got), w)
        compare(o, lse, q, cache, table, [0, new, T], length, True, D ** -0.5)


def test_a_layer_of_all_of_them(fq):
    """The run that a served layer makes: an 8-bit projection to q, k, v, the cache's append, attention over it, and
    the 8-bit output projection; each link against the oracle of that link's own inputs."""
    rng = np.random.default_rng(23)
    heads, G, D, page, hidden = 2, 4, 64, 16, 512
    Hq = heads * G
    qkv_w = fq.quantize_fp8(bf16(rng, (Hq + 2 * heads) * D, hidden, gain=hidden ** -0.5), fq.FP4Q_FP8_TILE)
    out_w = fq.quantize_fp8(bf16(rng, hidden, Hq * D, gain=(Hq * D) ** -0.5), fq.FP4Q_FP8_TILE)
    cache = [np.zeros((9, heads, page, D), np.uint8) for _ in range(2)] + [np.zeros((9, heads), np.float32) for _ in range(2)]
    dev = up(cache)
    table = np.array([[3, 1, 8, 5], [0, 2, 7, 6]], np.int32)
    length = np.array([0, 0])
    for new in ([20, 33], [1, 1], [1, 1], [5, 3]):
        length = length + np.array(new)
        T = sum(new)
        x = bf16(rng, T, hidden)
        xq = fq.quantize_fp8(x)
        qkv = fq.gemm_fp8(*xq, *qkv_w).view(T, Hq + 2 * heads, D)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + heads], qkv[:, Hq + heads:]
        args = (i32(table.tolist()), i32(cum(new)), i32(length.tolist()))
        fq.kv_append_fp8(k, v, *dev, *args, max(new))
        o, lse = fq.attention_fp8(q, *dev, *args, max(new), int(length.max()))
        oq = fq.quantize_fp8(o.reshape(T, Hq * D))
        y = fq.gemm_fp8(*oq, *out_w, out_dtype=torch.float32)
        cache = fp8.kv_append(host(k.contiguous()), host(v.contiguous()), cache, table, cum(new), length)
        for got, w in zip(dev, cache):
            assert np.array_equal(to_np(got), w)
        compare(o, lse, q.contiguous(), cache, table, cum(new), length, True, D ** -0.5)
        codes, scales = fp8.quantize(host(o).reshape(T, Hq * D), False)
        assert np.array_equal(to_np(oq[0]), codes) and np.array_equal(to_np(oq[1]), scales)
        want, total = fp8.gemm(fp8.values(codes, scales, False), fp8.values(to_np(out_w[0]), to_np(out_w[1]), True))
        assert (np.abs(to_np(y.double()) - want) <= (Hq * D + 16) * 2.0 ** -23 * total + 1e-30).all()


# ------------------------------------------------------------------ batches of many rows: the kernel of 128 rows a CTA

def batch_of(fq, rng, B, new, L, page, D, heads, G, cache=None):
    """B sequences of the same lengths: enough rows that 128 of them a CTA is the faster kernel (head dims 64 and 128)."""
    pool = B * -(-L // page) + 1
    cache = random_cache(rng, pool, heads, page, D) if cache is None else cache
    table = table_for(rng, [L] * B, page, pool)
    cu = cum([new] * B)
    return cache, table, cu, bf16(rng, cu[-1], heads * G, D)


@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 32), (64, 128), (128, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_batches_of_chunks(fq, D, page, causal):
    rng = np.random.default_rng(D + page)
    new = [40, 1, 33, 0, 64, 70, 2, 129] * 4
    lens = [40, 1, 200, 60, 130, 64, 1, 400] * 4  # some with more queries than keys
    run(fq, rng, new, lens, page, D, 2, 3, causal)


@pytest.mark.parametrize("scale", [1.0, -0.3, 1e-6])
def test_batches_with_other_softmax_scales(fq, scale):
    rng = np.random.default_rng(31)
    run(fq, rng, [30] * 24, [150] * 24, 32, 64, 2, 2, softmax_scale=scale)


def test_batches_with_page_scales_far_apart(fq):
    rng = np.random.default_rng(32)
    page, D, B, L = 32, 128, 24, 300
    pool = B * 10 + 1
    cache = random_cache(rng, pool, 1, page, D)
    cache[3][:, 0] = np.exp2(-6.0 * (np.arange(pool) % 12)).astype(np.float32)
    cache[2][:, 0] = np.linspace(0.02, 0.2, pool).astype(np.float32)
    cache[3][5::17] = 0.0
    cache[2][7::19] = 0.0
    run(fq, rng, [40] * B, [L] * B, page, D, 1, 2, cache=cache, pool=pool)


@pytest.mark.parametrize("D", [64, 128])
def test_batches_masked_nan_does_not_leak(fq, D):
    """A NaN in one sequence's last token, and in a token that all of its queries see."""
    rng = np.random.default_rng(33)
    B, new, L, page, G = 24, 40, 200, 32, 2
    cache, table, cu, q = batch_of(fq, rng, B, new, L, page, D, 1, G)
    args = (i32(table.tolist()), i32(cu), i32([L] * B), new, L)
    clean = to_np(fq.attention_fp8(q, *up(cache), *args)[0].float()).reshape(B, new, G, D)
    for pos, first in ((L - 1, new - 1), (L - 7, new - 7), (100, 0)):
        for side in (0, 1):
            broken = [c.copy() for c in cache]
            broken[side][table[5, pos // page], 0, pos % page, 3] = 0xFF
            o = to_np(fq.attention_fp8(q, *up(broken), *args)[0].float()).reshape(B, new, G, D)
            bad = np.zeros(o.shape, bool)
            bad[5, first:, :, 3 if side else slice(None)] = True
            assert np.isnan(o[bad]).all() and np.array_equal(o[~bad], clean[~bad]), (pos, side)


def test_batches_in_views_without_lse_and_rows_outside(fq):
    rng = np.random.default_rng(34)
    B, new, L, page, D, G = 24, 40, 130, 64, 128, 2
    cache, table, cu, q = batch_of(fq, rng, B, new, L, page, D, 2, G)
    dev = up(cache)
    o, lse = fq.attention_fp8(q, *dev, i32(table.tolist()), i32(cu), i32([L] * B), new, L)
    compare(o, lse, q, cache, table, cu, [L] * B, True, D ** -0.5)
    T = cu[-1]
    wide = torch.zeros((T + 9, 8, D), dtype=torch.bfloat16, device="cuda")
    wide[4:4 + T, :4] = q
    out = torch.full((T + 9, 7, D), 5.0, dtype=torch.bfloat16, device="cuda")
    shifted = i32([c + 4 for c in cu])
    # bounds above the lengths, as a captured graph has them
    width = np.zeros((B, table.shape[1] + 3), np.int32)
    width[:, :table.shape[1]] = table
    fq.fp4q_attention_fp8(wide[:, :4], *dev, i32(width.tolist()), shifted, i32([L] * B), new + 5, L + 90, out[:, :4])
    assert torch.equal(out[4:4 + T, :4], o)
    assert (out[:4] == 5).all() and (out[4 + T:] == 5).all() and (out[:, 4:] == 5).all()


def test_batches_report_entries_out_of_range(fq):
    rng = np.random.default_rng(35)
    B, new, L, page, D = 24, 40, 200, 32, 64
    cache, table, cu, q = batch_of(fq, rng, B, new, L, page, D, 1, 2)
    dev = up(cache)
    good = (table, cu, [L] * B, new, L)
    assert fq.fp4q_device_error() == 0
    for which, change in ((0, lambda t: t.__setitem__((3, 2), 2 ** 20)), (0, lambda t: t.__setitem__((3, 6), -1)),
                          (1, lambda c: c.__setitem__(B, cu[-1] + 1)), (2, lambda n: n.__setitem__(2, 7 * page + 1)),
                          (2, lambda n: n.__setitem__(4, -3))):
        bad = [good[0].copy(), list(cu), [L] * B]
        change(bad[which])
        fq.attention_fp8(q, *dev, i32(bad[0].tolist()), i32(bad[1]), i32(bad[2]), new, L)
        assert fq.fp4q_device_error() == 2, which


def test_batches_of_chunks_in_a_graph_and_on_two_streams(fq):
    """Chunks appended and attended to inside a captured graph, replayed as the sequences grow, and the same calls on
    two streams at once."""
    rng = np.random.default_rng(36)
    B, new, page, D, heads, G, width = 16, 48, 32, 128, 2, 2, 6
    pool = B * width
    cache = [np.zeros((pool, heads, page, D), np.uint8) for _ in range(2)] + [np.zeros((pool, heads), np.float32) for _ in range(2)]
    dev = up(cache)
    table = rng.permutation(pool).reshape(B, width).astype(np.int32)
    cu = cum([new] * B)
    T = cu[-1]
    q, k, v = bf16(rng, T, heads * G, D), bf16(rng, T, heads, D), bf16(rng, T, heads, D)
    tab, dcu, lens = i32(table.tolist()), i32(cu), i32([new] * B)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    most = width * page
    ws = fq.attention_fp8_workspace(q, dev[0], B, new, most)

    def step():
        fq.fp4q_kv_append_fp8(k, v, *dev, tab, dcu, lens, new)
        fq.fp4q_attention_fp8(q, *dev, tab, dcu, lens, new, most, o, lse, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in dev:
        t.zero_()
    for turn in range(1, 4):
        for x, n in ((q, heads * G), (k, heads), (v, heads)):
            x.copy_(bf16(rng, T, n, D))
        lens.fill_(turn * new)
        graph.replay()
        torch.cuda.synchronize()
        cache = fp8.kv_append(host(k), host(v), cache, table, cu, [turn * new] * B)
        for got, w in zip(dev, cache):
            assert np.array_equal(to_np(got), w)
        compare(o, lse, q, cache, table, cu, [turn * new] * B, True, D ** -0.5)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            outs += [fq.attention_fp8(q, *dev, tab, dcu, lens, new, most) for _ in range(3)]
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)


@pytest.mark.parametrize("new,B", [(1, 3), (48, 16)])
def test_offsets_past_32_bits(fq, new, B):
    """Pages whose codes lie more than 2^31 bytes into the cache: the same bits as from a small cache."""
    rng = np.random.default_rng(41)
    heads, page, D, G, L = 8, 128, 128, 2, 300
    small_pool, big_pool = 3 * B, 17000
    shift = big_pool - small_pool
    cu = cum([new] * B)
    q, k, v = bf16(rng, cu[-1], heads * G, D), bf16(rng, cu[-1], heads, D), bf16(rng, cu[-1], heads, D)
    start = up(random_cache(rng, small_pool, heads, page, D))
    for s in start[2:]:
        s.copy_(torch.exp2(torch.floor(torch.log2(s))))
    table = rng.permutation(small_pool).reshape(B, 3).astype(np.int32)
    small = [t.clone() for t in start]
    big = [torch.empty((big_pool, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in start]
    for t, b in zip(start, big):
        b[shift:] = t
    outs = []
    for cache, tab in ((small, table), (big, table + shift)):
        args = (i32(tab.tolist()), i32(cu), i32([L] * B))
        fq.kv_append_fp8(k, v, *cache, *args, new)
        outs.append(fq.attention_fp8(q, *cache, *args, new, L))
    assert big[0].numel() > 2 ** 31
    for a, b in zip(small, big):
        assert torch.equal(a, b[shift:])
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_over_long_sequences(fq, D, page, causal):
    """Few tiles of 128 rows over many keys: the keys are split and joined through the workspace."""
    rng = np.random.default_rng(D + page + causal)
    # splits that a sequence does not reach; more queries than keys
    for heads, new, lens in ((3, [100, 3, 0, 130, 70], [2500, 700, 60, 130, 30]), (2, [100, 3, 0, 70], [2500, 700, 60, 30])):
        n = fq.fp4q_attention_fp8_workspace_bytes(len(new), max(new), max(lens), 4 * heads, heads, D)
        ws = torch.full((n + 16,), 255, dtype=torch.uint8, device="cuda")  # every word of it a NaN
        run(fq, rng, new, lens, page, D, heads, 4, causal, ws=ws)
    assert n > 0


@pytest.mark.parametrize("L", [511, 512, 513, 640, 1024, 1025, 1537])
def test_chunks_around_the_splits_ends(fq, L):
    rng = np.random.default_rng(L)
    run(fq, rng, [128], [L], 32, 128, 1, 8)
    run(fq, rng, [128, 60], [L, 513], 64, 64, 2, 4, causal=False)


def test_chunks_over_long_sequences_with_a_nan(fq):
    """A NaN code of V reaches the rows that see its key, whichever split it is in."""
    rng = np.random.default_rng(41)
    page, D, L, new, heads, G = 64, 128, 2000, 128, 2, 4
    cache, table, cu, q = batch_of(fq, rng, 1, new, L, page, D, heads, G)
    at = [700, L - 30]  # seen by all, and by the last queries only
    for d, pos in enumerate(at):
        cache[1][table[0, pos // page], 0, pos % page, 5 + d] = 0x7F
    o, _ = fq.attention_fp8(q, *up(cache), i32(table.tolist()), i32(cu), i32([L]), new, L)
    bad = np.isnan(to_np(o.float()))
    want = np.zeros_like(bad)
    want[:, :G, 5] = True
    want[new - 30:, :G, 6] = True  # key L - 30 is query new - 30's own
    assert np.array_equal(bad, want)


def test_chunks_over_long_sequences_in_a_graph(fq):
    """Lengths that change between replays, below the bound that the splits were made for."""
    rng = np.random.default_rng(42)
    page, D, L, new, heads, G = 64, 128, 3000, 100, 2, 4
    cache, table, cu, q = batch_of(fq, rng, 2, new, L, page, D, heads, G)
    dev, tab, dcu, lens = up(cache), i32(table.tolist()), i32(cu), i32([L, L])
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = fq.attention_fp8_workspace(q, dev[0], 2, new, L)
    call = lambda: fq.fp4q_attention_fp8(q, *dev, tab, dcu, lens, new, L, o, lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for ns in ([3000, 40], [600, 2999], [0, 513]):
        lens.copy_(i32(ns))
        graph.replay()
        torch.cuda.synchronize()
        compare(o, lse, q, cache, table, cu, ns, True, D ** -0.5)


def test_the_largest_bounds(fq):
    """max_q * G and max_len up to 2^30 are taken, whatever the heads; more is refused."""
    most = 1 << 30
    assert fq.fp4q_attention_fp8_workspace_bytes(2, most, 64, 8, 8, 128) == 0
    assert fq.fp4q_attention_fp8_workspace_bytes(2, most // 4, 64, 32, 8, 64) == 0
    for sizes in ((1, most + 1, 64, 8, 8, 128), (1, most // 4 + 1, 64, 32, 8, 128), (1, 1, most + 1, 8, 8, 128)):
        with pytest.raises(fq.Fp4qError):
            fq.fp4q_attention_fp8_workspace_bytes(*sizes)


# ------------------------------------------------------------------ NaN, infinities and scales at the ends of the range

@pytest.mark.parametrize("page,D", [(16, 64), (64, 128), (32, 256)])
def test_append_keeps_the_nan_of_pages_without_numbers(fq, page, D):
    """NaN throughout a token, among zeros, and zeros alone, then numbers: the NaN codes stay what they are."""
    rng = np.random.default_rng(page + D)
    heads = 3
    cache = random_cache(rng, 3, heads, page, D)
    dev = up(cache)
    table = np.array([[1]], np.int32)
    for t in range(5):
        k, v = bf16(rng, 1, heads, D), bf16(rng, 1, heads, D, gain=100.0)
        if t < 3:  # head 0: NaN; head 1: NaN among zeros of both signs; head 2: numbers
            for x in (k, v):
                x[:, 0] = float("nan") if t != 1 else 0.0
                x[:, 1] = -0.0
                x[:, 1, t::5] = float("nan")
        fq.kv_append_fp8(k, v, *dev, i32(table.tolist()), i32([0, 1]), i32([t + 1]), 1)
        cache = fp8.kv_append(host(k), host(v), cache, table, [0, 1], [t + 1])
        for got, w, name in zip(dev, cache, ("k", "v", "k_scale", "v_scale")):
            assert np.array_equal(to_np(got), w), (t, name)
        for codes in dev[:2]:
            kept = to_np(codes)[1, :, :t + 1]
            assert (kept[0, 0] == 0x7F).all() and (kept[1, 0, ::5] == 0x7F).all()
            assert not np.delete(kept[1, 0], np.s_[::5]).any() and not (t and kept[0, 1].any())
        assert t >= 3 or not (to_np(dev[2])[1, :2].any() or to_np(dev[3])[1, :2].any())
    q = bf16(rng, 1, heads, D)
    o, _ = fq.attention_fp8(q, *dev, i32(table.tolist()), i32([0, 1]), i32([5]), 1, 5)
    o = to_np(o.float())[0]
    assert np.isnan(o[:2]).all() and np.isfinite(o[2]).all()


# (sequences, queries, keys, heads, group): 16 rows a CTA, alone, in a cluster and joined by a second kernel (one row tile
# and many); 128 rows a CTA (head dims 64 and 128), alone and with the keys split.  The last page of 32 holds the last key
# alone, which only the last query sees.
LAST_ALONE = [(1, 1, 33, 1, 1), (2, 4, 97, 1, 2), (1, 4, 513, 1, 2), (1, 4, 9985, 1, 2), (1, 128, 2017, 2, 4), (24, 40, 193, 1, 2),
              (2, 64, 1537, 8, 2)]


def moderate(cache):
    """V codes of magnitudes up to 1, so that values stay in range under the largest scales."""
    cache[1] = (cache[1] & 0x80) | np.minimum(cache[1] & 0x7F, 0x38)
    return cache


@pytest.mark.parametrize("scale", [2.0 ** 114, 2.0 ** 120, 2.0 ** 127])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,new,L,heads,G", LAST_ALONE)
def test_a_large_page_scale_of_v_reaches_only_those_who_see_it(fq, B, new, L, heads, G, D, scale):
    """The other queries' results keep their bits; the last one's is the formula's."""
    rng = np.random.default_rng(L + D)
    page = 32
    cache, table, cu, q = batch_of(fq, rng, B, new, L, page, D, heads, G)
    moderate(cache)
    args = (i32(table.tolist()), i32(cu), i32([L] * B), new, L)
    clean = fq.attention_fp8(q, *up(cache), *args)
    cache[3][table[:, (L - 1) // page]] = scale
    o, lse = fq.attention_fp8(q, *up(cache), *args)
    first = np.delete(np.arange(cu[-1]), np.array(cu[1:]) - 1)
    assert torch.equal(o[first], clean[0][first]) and torch.equal(lse[first], clean[1][first])
    compare(o, lse, q, cache, table, cu, [L] * B, True, D ** -0.5)


@pytest.mark.parametrize("B,new,L,heads,G", LAST_ALONE)
@pytest.mark.parametrize("D", [64, 128])
def test_page_scales_of_v_up_to_the_largest(fq, B, new, L, heads, G, D):
    """Every page large, and large pages among ordinary and tiny ones, all of them seen: o and lse are the formula's."""
    rng = np.random.default_rng(L + D)
    cache, table, cu, q = batch_of(fq, rng, B, new, L, 32, D, heads, G)
    moderate(cache)
    for exponents in ([114, 117, 120, 127], [120], [0, 120, -3, -100], [60, -60, 90, 0], [0, -90, -100]):
        cache[3][:] = np.exp2(rng.choice(exponents, cache[3].shape)).astype(np.float32)
        o, lse = fq.attention_fp8(q, *up(cache), i32(table.tolist()), i32(cu), i32([L] * B), new, L)
        compare(o, lse, q, cache, table, cu, [L] * B, True, D ** -0.5)


@pytest.mark.parametrize("B,new,L,heads,G", LAST_ALONE[1:])
@pytest.mark.parametrize("side", [0, 1])
def test_an_infinity_in_the_last_token_reaches_only_its_query(fq, B, new, L, heads, G, side):
    """Through the append, which gives its page the scale 2^120."""
    rng = np.random.default_rng(L + side)
    page, D = 32, 128
    cache, table, cu, q = batch_of(fq, rng, B, new, L, page, D, heads, G)
    k, v = bf16(rng, cu[-1], heads, D), bf16(rng, cu[-1], heads, D)
    args = (i32(table.tolist()), i32(cu), i32([L] * B))
    outs = []
    for broken in (False, True):
        if broken:
            (k, v)[side][np.array(cu[1:]) - 1, :, 5] = float("inf")
        dev = up(cache)
        fq.kv_append_fp8(k, v, *dev, *args, new)
        assert not broken or (to_np(dev[2 + side])[table[:, (L - 1) // page]] == 2.0 ** 120).all()
        outs.append(fq.attention_fp8(q, *dev, *args, new, L))
    first = np.delete(np.arange(cu[-1]), np.array(cu[1:]) - 1)
    assert torch.equal(outs[0][0][first], outs[1][0][first]) and torch.equal(outs[0][1][first], outs[1][1][first])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,new,L,heads,G", LAST_ALONE)
def test_a_page_scale_that_is_no_number_reaches_only_those_who_see_it(fq, B, new, L, heads, G, D, bad):
    rng = np.random.default_rng(L + D)
    page = 32
    cache, table, cu, q = batch_of(fq, rng, B, new, L, page, D, heads, G)
    args = (i32(table.tolist()), i32(cu), i32([L] * B), new, L)
    clean = fq.attention_fp8(q, *up(cache), *args)
    last = np.array(cu[1:]) - 1
    first = np.delete(np.arange(cu[-1]), last)
    for side in (2, 3):
        broken = [c.copy() for c in cache]
        broken[side][table[:, (L - 1) // page]] = bad
        o, lse = fq.attention_fp8(q, *up(broken), *args)
        assert torch.equal(o[first], clean[0][first]) and torch.equal(lse[first], clean[1][first])
        # (an infinite scale of K leaves scores of -inf, which are no NaN)
        assert torch.isnan(o[last]).all() or (side == 2 and bad == float("inf"))


def test_the_largest_batches_and_head_counts(fq):
    """Work that 31 bits do not count is refused, however the sizes make it up."""
    big = 1 << 30
    for sizes in ((big, 2048, 64, big, big, 128), (big, 1, 64, 4, 4, 128), (big, 1 << 25, 64, 65536, 65536, 64),
                  (65536, 1, 64, 65536, 65536, 256), (4, big, 4096, 512, 512, 128)):
        with pytest.raises(fq.Fp4qError):
            fq.fp4q_attention_fp8_workspace_bytes(*sizes)


@pytest.mark.parametrize("B,new,L,heads,G", LAST_ALONE)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_code_of_the_last_token_reaches_only_its_query(fq, B, new, L, heads, G, D):
    rng = np.random.default_rng(L + D)
    page = 32
    cache, table, cu, q = batch_of(fq, rng, B, new, L, page, D, heads, G)
    args = (i32(table.tolist()), i32(cu), i32([L] * B), new, L)
    clean = fq.attention_fp8(q, *up(cache), *args)[0]
    last = np.array(cu[1:]) - 1
    for side in (0, 1):
        broken = [c.copy() for c in cache]
        broken[side][table[:, (L - 1) // page], :, 0, 3] = 0x7F
        o = fq.attention_fp8(q, *up(broken), *args)[0]
        bad = torch.zeros_like(o, dtype=torch.bool)
        bad[last, :, slice(3, 4) if side else slice(None)] = True
        assert torch.isnan(o[bad]).all() and torch.equal(o[~bad], clean[~bad]), side
