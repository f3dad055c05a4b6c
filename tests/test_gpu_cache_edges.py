"""The paged-cache operators at the edges of their tiles: values that are not
numbers in every place of a tile, and scales and rows at the ends of the range."""
import numpy as np
import pytest
import torch

import clustered_multipole_approximation_b200 as muse
from clustered_multipole_approximation_b200 import build
from cache_ref import IN, Paged, attend
from test_gpu_cache import err_word, i32, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return muse.load_library()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("n,Hq", [(33, 1), (70, 1), (20, 2), (130, 1), (50, 3), (5, 2)])
def test_a_value_that_is_not_a_number_in_every_place(n, Hq, window, D, cache):
    """Row counts that leave softmax warps without a row, the value at each of 16
    neighbouring positions: rows that do not see it are as if it were not there."""
    kv = n + 90
    P = Paged(1, 1, D, [kv], 16, cache)
    q = torch.randn(1, Hq, n, D, generator=torch.Generator().manual_seed(4)).bfloat16()
    scale = D ** -0.5
    ro, _, to, _ = attend(P, q, [n], scale, window=window)
    c = P.gpu()
    pos = kv - n + np.arange(n)
    for at in range(kv - 17, kv):
        pg, r = P.where(0, at)
        keep = c["v_cache"].clone()
        c["v_cache"].view(torch.uint8 if cache == "e4m3" else torch.int16)[pg, :, r, 5] = \
            0x7F if cache == "e4m3" else 0x7FC0
        o = muse.muse_attn_cache(q.cuda(), **c, scale=scale, window=window).double().cpu().numpy()
        c["v_cache"] = keep
        sees = (at <= pos) & ((at > pos - window) if window else True)
        assert np.isnan(o[:, :, sees, 5]).all(), at
        fine = np.ones(o.shape, bool)
        fine[:, :, sees, 5] = False
        bad = fine & ~(np.abs(o - ro) <= to)
        bad[:, :, sees] = False  # (their other columns: the split-call tests)
        assert not bad.any(), (at, np.argwhere(bad)[:4])


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("n", [1, 9, 40, 150])
@pytest.mark.parametrize("scale", [2.0 ** -148, 1e-20])
def test_scales_and_rows_next_to_zero(n, scale, cache):
    """The factor that undoes a row's power of two, times the scale, is zero in
    fp32: the weights are equal, and masked keys stay out."""
    q = torch.randn(1, 2, n, 64, generator=torch.Generator().manual_seed(6))
    q[:, :, 0::3] = 0.0
    q[:, :, 1::3] *= 1e-30
    run_attend(Paged(1, 1, 64, [n + 200], 16, cache), n, [n], 2, scale=scale, q=q.bfloat16())


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "i8", "f32"])
@pytest.mark.parametrize("B,Hkv", [(1, 1), (1, 2), (2, 1)])
@pytest.mark.parametrize("wide", [64, 1024])
@pytest.mark.parametrize("n", [1, 3])
def test_row_tiles_that_see_nothing_in_divided_calls(n, wide, B, Hkv, cache):
    """Tables of 1024 (splits that join in a cluster) and 16384 positions (through
    the workspace), no token cached, alone and beside a long sequence."""
    for kv in ([0] * B, [700] * (B - 1) + [0], [n - 1] * B):
        P = Paged(B, Hkv, 64, kv, 16, cache, wide=wide)
        for causal in (True, False):
            run_attend(P, n, [n] * B, 4 * Hkv, causal=causal)


@pytest.mark.parametrize("cache,D", [("bf16", 64), ("bf16", 128), ("e4m3", 64), ("i8", 128)])
@pytest.mark.parametrize("n,wide,load", [(40, None, 0), (40, None, 15), (150, None, 6), (150, 400, 0), (40, 400, 3)])
def test_a_load_that_never_arrives(n, wide, load, cache, D):
    """Failure path of the chunk kernel: the waits for a load that is not reported
    run out, the call says so and leaves NaN, unsplit and in splits; the next call
    is as before."""
    lib = muse.load_library()
    P = Paged(1, 1, D, [900], 16, cache, wide=wide)
    c, e = P.gpu(), err_word()
    q = torch.randn(1, 1, n, D, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    want, _ = muse.muse_attn_cache(q, **c, lse=True)
    lib.muse_debug_inject_cache_fault(load)
    try:
        o, lse = muse.muse_attn_cache(q, **c, lse=True, device_error=e)
        with pytest.raises(muse.MuseError) as err:
            muse.device_status(e)
    finally:
        lib.muse_debug_inject_cache_fault(-1)
    assert err.value.status == 5 and int(e) == 1
    assert o.isnan().all() and lse.isnan().all()
    assert torch.equal(muse.muse_attn_cache(q, **c, device_error=e), want)
    muse.device_status(e)


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("i8", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n", [1, 4, 150])
@pytest.mark.parametrize("other", [False, True])
def test_rows_that_are_not_there_of_outputs_made_by_the_call(other, n, cache, dtype):
    """o = 0 and lse = -inf behind new_len, whatever the memory held before."""
    P = Paged(3, 1, 64, [300, n, 40], 16, cache)
    c, new = P.gpu(), i32([n, n // 2, 0])
    q = torch.randn(3, 2, n, 64, generator=torch.Generator().manual_seed(2)).to(IN[dtype]).cuda()
    stream = torch.cuda.Stream() if other else None
    seen = []
    for _ in range(3):
        junk = [torch.full((3, 2, n, 64), float("nan"), dtype=IN[dtype], device="cuda") for _ in range(4)]
        junk += [torch.full((3, 2, n), float("nan"), device="cuda") for _ in range(4)]
        del junk
        o, lse = muse.muse_attn_cache(q, **c, new_len=new, lse=True, stream=stream)
        torch.cuda.synchronize()
        for b, m in enumerate([n, n // 2, 0]):
            assert (o[b, :, m:] == 0).all() and (lse[b, :, m:] == -float("inf")).all()
            assert o[b, :, :m].isfinite().all() and lse[b, :, :m].isfinite().all()
        seen.append((o.clone(), lse.clone()))
    assert all(torch.equal(a, b) for x in seen[1:] for a, b in zip(x, seen[0]))
