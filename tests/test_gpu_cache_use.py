"""The paged-cache operators as programs use them: workspaces of the exact size,
several threads, and stored values that are not numbers in the 8-bit caches."""
import threading

import numpy as np
import pytest
import torch

import clustered_multipole_approximation_b200 as muse
from clustered_multipole_approximation_b200 import build
from cache_ref import IN, Paged, attend
from test_gpu_cache import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return muse.load_library()


@pytest.mark.parametrize("n,cache,dtype,wide", [(1, "bf16", "bf16", 1024), (1, "i8", "bf16", 2048), (5, "e4m3", "bf16", 1024),
                                                (150, "bf16", "bf16", 256), (150, "e4m3", "bf16", 256),
                                                (40, "f32", "f32", 128), (1, "i8", "f32", 128)])
@pytest.mark.parametrize("window", [0, 100, 3000])
def test_a_workspace_of_the_exact_size(n, cache, dtype, wide, window):
    """Calls whose splits join through the workspace: whatever it holds before, the
    same bits, and not a byte behind it."""
    kv = 3900 if wide >= 256 else 1900
    P = Paged(1, 1, 64, [kv], 16, cache, wide=wide)
    c = P.gpu()
    q = torch.randn(1, 4, n, 64, generator=torch.Generator().manual_seed(1)).to(IN[dtype])
    size = muse.attn_cache_workspace_size(q.cuda(), **c)
    assert size > 256
    got = []
    for fill in (0, 255, 0x7F):
        mem = torch.full((size + 4096,), fill, dtype=torch.uint8, device="cuda")
        got.append(muse.muse_attn_cache(q.cuda(), **c, scale=0.125, window=window, workspace=mem[:size]))
        assert (mem[size:] == fill).all()
        if not window:
            assert (mem[:size] != fill).any()  # it is used
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    ro, _, to, _ = attend(P, q, [n], 0.125, window=window, q_type=dtype)
    assert (np.abs(got[0].double().cpu().numpy() - ro) <= to).all()
    with pytest.raises(muse.MuseError, match="workspace"):
        muse.muse_attn_cache(q.cuda(), **c, workspace=torch.empty(size - 256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("n,wide", [(1, 1024), (150, 256)])
def test_two_streams_with_workspaces_of_their_own(n, wide):
    P = Paged(1, 1, 64, [3900], 16, "bf16", wide=wide)
    c = P.gpu()
    qs = [torch.randn(1, 4, n, 64, device="cuda").bfloat16() for _ in range(2)]
    want = [muse.muse_attn_cache(q, **c) for q in qs]
    size = muse.attn_cache_workspace_size(qs[0], **c)
    streams = [torch.cuda.Stream() for _ in qs]
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(muse.muse_attn_cache(qs[i], **c, workspace=ws[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_calls_from_several_threads():
    """Each thread its own cache, on the default stream or one of its own; what each
    reads, answers and raises is its own."""
    def work(seed, out):
        try:
            torch.cuda.set_device(0)
            g = torch.Generator().manual_seed(seed)
            stream = torch.cuda.Stream() if seed % 2 else torch.cuda.current_stream()
            with torch.cuda.stream(stream):
                for i in range(20):
                    n = (1, 5, 60)[i % 3]
                    kv = 80 + n
                    c = dict(muse.make_cache(12, 2, 16, 64, (torch.bfloat16, torch.int8)[i % 2]),
                             table=i32([list(range(12))[::-1]]), kv_len=i32([kv]))
                    k, v = (torch.randn(1, 2, kv, 64, generator=g).bfloat16().cuda() for _ in range(2))
                    q = torch.randn(1, 4, n, 64, generator=g).bfloat16().cuda()
                    muse.muse_cache_write(k, v, **c)
                    o = muse.muse_attn_cache(q, **c, scale=0.125)
                    rk, rv = muse.muse_cache_read(**c, N=kv, dtype=torch.float32)
                    x = (q.double() @ rk.double().repeat_interleave(2, 1).transpose(2, 3)) * 0.125
                    mask = torch.ones(n, kv, dtype=torch.bool, device="cuda").tril(kv - n)
                    p = x.masked_fill(~mask, -torch.inf).softmax(-1)
                    rv = rv.double().repeat_interleave(2, 1)
                    # weights and output rounded to bf16 once each; the rest is far below half a step
                    tol = 1.1 * 2.0 ** -8 * (p @ rv.abs() + (p @ rv).abs()) + 1e-5
                    assert ((o.double() - p @ rv).abs() <= tol).all()
                    with pytest.raises(muse.MuseError, match="multiple of Hkv" if seed % 2 else "scale"):
                        if seed % 2:
                            muse.muse_attn_cache(q[:, :3], **c)
                        else:
                            muse.muse_attn_cache(q, **c, scale=float("inf"))
            out.append(None)
        except BaseException as e:  # noqa: BLE001  (raised in the test's own thread)
            out.append(e)

    out = []
    threads = [threading.Thread(target=work, args=(i, out)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(out) == 4
    for e in out:
        if e is not None:
            raise e


@pytest.mark.parametrize("cache,dtype", [("i8", "bf16"), ("i8", "f32"), ("e4m3", "f32")])
@pytest.mark.parametrize("n,Hq,window", [(2, 3, 0), (5, 3, 0), (9, 3, 2), (40, 1, 0), (60, 3, 2), (150, 1, 0)])
def test_rows_of_nan_in_8_bit_caches(n, Hq, window, cache, dtype):
    """A stored row whose scales are NaN (what a row with an infinity is written as)
    inside the chunk: rows that do not see it are as without it, the others NaN."""
    kv, D = 90 + n, 64
    P = Paged(1, 1, D, [kv], 16, cache)
    q = torch.randn(1, Hq, n, D, generator=torch.Generator().manual_seed(5)).to(IN[dtype])
    ro, rl, to, tl = attend(P, q, [n], D ** -0.5, window=window, q_type=dtype)
    pos = kv - n + np.arange(n)
    for at in (kv - n, kv - n // 2 - 1, kv - 1):
        pg, r = P.where(0, at)
        c = P.gpu()
        c["k_scale"][pg, :, r] = float("nan")
        c["v_scale"][pg, :, r] = float("nan")
        o, lse = muse.muse_attn_cache(q.cuda(), **c, scale=D ** -0.5, window=window, lse=True)
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        sees = (at <= pos) & ((at > pos - window) if window else True)
        assert np.isnan(o[:, :, sees]).all() and np.isnan(lse[:, :, sees]).all()
        assert (np.abs(o - ro) <= to)[:, :, ~sees].all() and (np.abs(lse - rl) <= tl)[:, :, ~sees].all()


@pytest.mark.parametrize("n", [1, 20, 150])
def test_e4m3_values_of_nan_under_fp32_queries(n):
    """Stored NaN values (0x7F) in a key and in a value."""
    kv, D = 90 + n, 64
    P = Paged(1, 1, D, [kv], 16, "e4m3")
    q = torch.randn(1, 2, n, D, generator=torch.Generator().manual_seed(5))
    ro, _, to, _ = attend(P, q, [n], D ** -0.5, q_type="f32")
    at = kv - n // 2 - 1
    sees = at <= kv - n + np.arange(n)
    pg, r = P.where(0, at)
    for which in ("k_cache", "v_cache"):
        c = P.gpu()
        c[which].view(torch.uint8)[pg, :, r, 5] = 0x7F
        o = muse.muse_attn_cache(q.cuda(), **c, scale=D ** -0.5).double().cpu().numpy()
        assert (np.abs(o - ro) <= to)[:, :, ~sees].all()
        assert np.isnan(o[:, :, sees] if which == "k_cache" else o[:, :, sees, 5]).all()


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.int8])
def test_one_cache_for_keys_that_are_values(cache):
    """K and V of the same rows may live in one cache; read back into two tensors
    beside one another."""
    c = muse.make_cache(6, 2, 16, 64, cache)
    for x in ("_cache", "_scale"):
        if "k" + x in c:
            c["v" + x] = c["k" + x]
    args = dict(c, table=i32([[4, 0, 5]]), kv_len=i32([40]))
    k = torch.randn(1, 2, 40, 64, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    muse.muse_cache_write(k, k, **args)
    with pytest.raises(muse.MuseError, match="share"):
        muse.muse_cache_write(k, k.clone(), **args)
    out = torch.empty(2, 1, 2, 40, 64, dtype=torch.bfloat16, device="cuda")
    rk, rv = muse.muse_cache_read(**args, N=40, out=(out[0], out[1]))
    assert torch.equal(rk, rv) and rk.data_ptr() == out.data_ptr()
    assert ((rk.float() - k.float()).abs() <= k.float().abs().amax(-1, keepdim=True) / 127 + 1e-2).all()
    one = muse.muse_cache_read(**args, N=40, out=(out[1], out[1]))[0]
    assert torch.equal(one, rk)
    args["v_cache"] = args["v_cache"].clone()
    with pytest.raises(muse.MuseError, match="share"):
        muse.muse_cache_read(**args, N=40, out=(out[0], out[0]))
    with pytest.raises(muse.MuseError, match="share"):
        flat = out.flatten()
        half = flat[:flat.numel() // 2].view_as(out[0]), flat[64:64 + flat.numel() // 2].view_as(out[0])
        muse.muse_cache_read(**args, N=40, out=half)
