"""The paged-cache operators where their work is divided: many splits and key
tiles, tables wider than their sequences, row counts around the tiles' limits;
and the quantisation at its ties and at the ends of the range."""
import numpy as np
import pytest
import torch

import clustered_multipole_approximation_b200 as muse
from clustered_multipole_approximation_b200 import build
from cache_ref import CACHE, IN, Paged, attend, quantise
from test_gpu_cache import err_word, i32, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return muse.load_library()


@pytest.mark.parametrize("cache", list(CACHE))
@pytest.mark.parametrize("n,Hq,Hkv", [(1, 8, 1), (2, 8, 1), (3, 16, 2), (4, 8, 1), (1, 17, 1), (11, 3, 1),
                                      (33, 1, 1), (16, 8, 1), (43, 3, 1)])
def test_row_counts_around_the_tiles(n, Hq, Hkv, cache):
    """8, 16, 24, 32, 17, 33, 33, 128 and 129 packed rows of a kv-head."""
    run_attend(Paged(2, Hkv, 64, [300, n + 100], 16, cache), n, [n, max(0, n - 1)], Hq)
    if n < 12:
        run_attend(Paged(1, Hkv, 128, [300], 16, cache), n, [n], Hq, window=70)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cache", list(CACHE))
@pytest.mark.parametrize("kv,wide", [(700, None), (900, 2000), (2900, 400), (1, 3000), (130, 60000)])
def test_single_tokens_over_many_splits(kv, wide, cache, D):
    """Splits that join in a cluster and through the workspace, tables far wider
    than their sequences, splits without keys."""
    for dtype in ("bf16", "f32") if cache in ("f32", "i8") else ("bf16",):
        run_attend(Paged(2, 2, D, [kv, max(1, kv // 3)], 16, cache, wide=wide), 1, [1, 1], 6, dtype)
    run_attend(Paged(1, 1, D, [max(kv, 5)], 16, cache, wide=wide), 5, [5], 4, window=600)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("n,Hq,wide", [(140, 2, None), (70, 1, None), (40, 2, 900), (300, 1, 700)])
def test_chunks_over_many_tiles(n, Hq, wide, cache, D):
    """More key tiles than shared memory has stages, both forms of the streams,
    one split and several, odd and even numbers of tiles."""
    for kv in (2700, 1100):
        run_attend(Paged(1, 1, D, [kv], 16, cache, wide=wide), n, [n], Hq)
    run_attend(Paged(1, 1, D, [1900], 16, cache, wide=wide), n, [n], Hq, causal=False)
    run_attend(Paged(1, 1, D, [1900], 16, cache, wide=wide), n, [n], Hq, window=777)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,wide", [(3, 30), (3, 3000), (40, 400), (150, 30), (150, 400)])
def test_values_that_are_not_numbers_in_split_calls(n, wide, cache):
    """As in the unsplit calls: only the rows that see the value are not numbers."""
    kv, at = 2200 if wide == 400 else 400, None
    at = kv - n // 2 - 1
    P = Paged(1, 1, 64, [kv], 16, cache, wide=wide)
    pg, r = P.where(0, at)
    if cache == "e4m3":
        P.t["v"].view(torch.uint8)[pg, :, r, 5] = 0x7F
    else:
        P.t["v"][pg, :, r, 5] = float("nan")
    q = torch.randn(1, 3, n, 64, generator=torch.Generator().manual_seed(5)).bfloat16()
    e = err_word()
    o = muse.muse_attn_cache(q.cuda(), **P.gpu(), scale=0.125, device_error=e).double().cpu().numpy()
    assert int(e) == 0
    with np.errstate(all="ignore"):
        ro, _, to, _ = attend(P, q, [n], 0.125)
    first = at - (kv - n)
    assert (np.abs(o - ro) <= to)[:, :, :first].all()
    assert np.isnan(o[:, :, first:, 5]).all()
    rest = np.arange(64) != 5
    assert (np.abs(o - ro) <= to)[:, :, first:][..., rest].all()


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
@pytest.mark.parametrize("n", [1, 5, 150])
def test_magnitudes_of_queries(n, cache):
    """Queries and scale changed by opposite powers of two: the same bits, as far
    as fp16's range is from theirs."""
    c = Paged(1, 2, 64, [400], 16, cache).gpu()
    q = torch.randn(1, 8, n, 64, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    want = muse.muse_attn_cache(q, **c, scale=0.125)
    for k in (-80, -40, -17, 17, 40, 100):
        got = muse.muse_attn_cache(q * 2.0 ** k, **c, scale=0.125 * 2.0 ** -k)
        assert torch.equal(got, want), k
    # rows of very different magnitude do not touch one another
    z = q.clone()
    z[:, 1::2] *= 2.0 ** 60
    assert torch.equal(muse.muse_attn_cache(z, **c, scale=0.125)[:, ::2], want[:, ::2])
    z[:, 1::2] = 0
    assert torch.equal(muse.muse_attn_cache(z, **c, scale=0.125)[:, ::2], want[:, ::2])


def written(x, cache):
    """(values, scales) of rows x [n, D] after a write, from the cache itself."""
    n, D = x.shape
    c = muse.make_cache(1, 1, n, D, CACHE[cache])
    x = x.cuda()[None, None]
    muse.muse_cache_write(x, x, **c, table=i32([[0]]), kv_len=i32([n]))
    assert torch.equal(c["k_scale"], c["v_scale"])
    assert torch.equal(c["k_cache"].view(torch.uint8), c["v_cache"].view(torch.uint8))
    return c["k_cache"][0, 0].double().cpu().numpy(), c["k_scale"][0, 0].cpu().numpy()


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
@pytest.mark.parametrize("shift", [0, -118, 110])
def test_every_pair_of_bf16_significands(cache, shift):
    """Every value of every binade down to 2^-8 of every maximum: all ties."""
    rows = []
    for m2 in range(128, 256):
        for k in range(9):
            x = np.arange(128, 256) * 2.0 ** -k
            x = np.where(x <= m2, x, x / 2)
            x[0::2] *= -1
            x = x.reshape(2, 64)
            x[:, 7] = m2
            rows.append(x)
    x = np.concatenate(rows) * 2.0 ** shift
    q, s = written(torch.from_numpy(x).bfloat16(), cache)
    wq, ws = quantise(x, cache)
    assert (s == ws.astype(np.float32)).all()
    assert (q == wq).all(), np.argwhere(q != wq)[:4]


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
def test_fp32_values_next_to_ties_and_ends_of_the_range(cache):
    g = np.random.Generator(np.random.PCG64(11))
    top = np.exp2(g.uniform(-148, 127.9, 600)).astype(np.float32)
    top[:4] = [np.float32(2.0 ** -149), np.float32(2.0 ** -126), np.finfo(np.float32).max, 1.0]
    h = g.integers(0, 127, (600, 128)) + 0.5
    x = (h * top[:, None].astype(np.float64) / 127).astype(np.float32)
    step = g.integers(-2, 3, x.shape)
    for _ in range(2):
        x = np.where(step > 0, np.nextafter(x, np.float32(np.inf)), np.where(step < 0, np.nextafter(x, np.float32(0)), x))
        step -= np.sign(step)
    x = np.minimum(x, top[:, None]) * g.choice([-1, 1], x.shape).astype(np.float32)
    x[:, 3] = top
    q, s = written(torch.from_numpy(x), cache)
    wq, ws = quantise(x, cache)
    assert (s == ws.astype(np.float32)).all()
    assert (q == wq).all(), np.argwhere(q != wq)[:4]


def test_one_cache_written_and_read_by_two_streams_in_turn():
    c = muse.make_cache(8, 2, 16, 64, torch.int8)
    args = dict(c, table=i32([[5, 1, 7]]), kv_len=i32([40]))
    k = torch.randn(1, 2, 40, 64, device="cuda").bfloat16()
    want = None
    side = torch.cuda.Stream()
    for _ in range(20):
        muse.muse_cache_write(k, k, **args)
        got = muse.muse_cache_read(**args, N=40, stream=side)  # behind the write: the side stream waits
        torch.cuda.current_stream().wait_stream(side)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_arguments_that_are_refused():
    c = muse.make_cache(3, 2, 4, 64)
    q = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    args = dict(c, table=i32([[0, 1], [2, 1]]), kv_len=i32([1, 1]))
    for bad in (dict(window=1 << 31), dict(window=-1), dict(out=q), dict(k_cache=None), dict(table=None),
                dict(k_cache=c["k_cache"][0]), dict(stream=torch.cuda.Stream), dict(lse=3), dict(scale="a")):
        with pytest.raises((ValueError, TypeError, AttributeError, OverflowError, muse.MuseError)):
            muse.muse_attn_cache(q, **{**args, **bad})
    for bad in (dict(N=0), dict(N=-1), dict(N=1 << 40), dict(N=2, dtype=torch.float16), dict(N=2, out=(q, q))):
        with pytest.raises((ValueError, TypeError, muse.MuseError)):
            muse.muse_cache_read(**{**args, **bad})
    for x in (q[:, :, :0], q[:0], q[..., :0]):
        with pytest.raises((ValueError, TypeError, muse.MuseError)):
            muse.muse_cache_write(x, x, **args)
        with pytest.raises((ValueError, TypeError, muse.MuseError)):
            muse.muse_attn_cache(x, **args)
    muse.muse_attn_cache(q, **args)
    torch.cuda.synchronize()
