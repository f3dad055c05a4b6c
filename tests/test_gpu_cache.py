"""The paged-cache operators on the GPU against their plain 64-bit forms."""
import itertools

import numpy as np
import pytest
import torch

import clustered_multipole_approximation_b200 as muse
from clustered_multipole_approximation_b200 import build
from cache_ref import CACHE, HALF, IN, Paged, attend, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return muse.load_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def err_word():
    return torch.full((1,), -1, dtype=torch.int32, device="cuda")


def run_attend(P, n, new, Hq, dtype="bf16", scale=None, causal=True, window=0, seed=1, layout="bhnd",
               q=None, errbits=0):
    """The call on P with random queries, every row checked."""
    B, D = P.B, P.D
    scale = D ** -0.5 if scale is None else scale
    g = torch.Generator().manual_seed(seed)
    if q is None:
        q = torch.randn(B, Hq, n, D, generator=g).to(IN[dtype])
    qd, out = q.cuda(), torch.full((B, Hq, n, D), 7.0, dtype=IN[dtype], device="cuda")
    if layout == "bnhd":  # a slice of a wider projection, and an output laid out for the next one
        wide = torch.full((B, n, Hq + 2, D), float("nan"), dtype=IN[dtype], device="cuda")
        wide[:, :, 1:Hq + 1] = q.transpose(1, 2).cuda()
        qd = wide[:, :, 1:Hq + 1].transpose(1, 2)
        out = torch.full((B, n, Hq, D), 7.0, dtype=IN[dtype], device="cuda").transpose(1, 2)
    lse = torch.full((B, Hq, n), 7.0, device="cuda")
    e = err_word()
    o, l2 = muse.muse_attn_cache(qd, **P.gpu(), new_len=i32(new), scale=scale, causal=causal,
                                 window=window, out=out, lse=lse, device_error=e)
    torch.cuda.synchronize()
    assert o is out and l2 is lse and int(e) == errbits
    ro, rl, to, tl = attend(P, q, new, scale, causal, window, dtype)
    o, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        assert (o[b, :, new[b]:] == 7).all() and (lse[b, :, new[b]:] == 7).all(), "rows past new_len"
        if not new[b]:
            continue
        x, y = o[b, :, :new[b]], ro[b, :, :new[b]]
        bad = ~(np.abs(x - y) <= to[b, :, :new[b]])
        assert not bad.any(), (b, np.argwhere(bad)[:4], x[bad][:4], y[bad][:4])
        x, y = lse[b, :, :new[b]], rl[b, :, :new[b]]
        empty = np.isneginf(y)
        assert (np.isneginf(x) == empty).all()
        assert (np.abs(x[~empty] - y[~empty]) <= tl[b, :, :new[b]][~empty]).all()
    return o, lse


ATTEND = [  # B, n, Hq, Hkv, D, kv, new, page
    (1, 1, 1, 1, 64, [1], [1], 16),
    (1, 1, 8, 2, 128, [17], [1], 16),
    (3, 1, 8, 8, 64, [1, 300, 64], [1, 1, 1], 16),
    (2, 1, 6, 2, 128, [129, 1000], [1, 0], 24),
    (2, 1, 32, 1, 64, [513, 5], [1, 1], 64),
    (2, 5, 8, 2, 128, [200, 5], [5, 3], 16),
    (2, 3, 7, 1, 64, [77, 3], [3, 2], 5),
    (2, 9, 4, 4, 64, [130, 9], [9, 0], 128),
    (1, 40, 4, 2, 128, [40], [40], 8),
    (2, 70, 6, 2, 64, [333, 70], [70, 31], 32),
    (1, 130, 4, 1, 128, [700], [130], 256),
    (2, 257, 2, 2, 64, [257, 400], [257, 100], 16),
    (1, 300, 3, 1, 64, [301], [300], 1),
]


@pytest.mark.parametrize("cache", list(CACHE))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "B%dn%dh%d.%dD%dp%d" % (c[:5] + (c[7],)))
def test_attend(case, dtype, cache):
    B, n, Hq, Hkv, D, kv, new, page = case
    run_attend(Paged(B, Hkv, D, kv, page, cache), n, new, Hq, dtype,
               layout="bnhd" if n % 2 else "bhnd")


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("n", [1, 3, 50, 140])
@pytest.mark.parametrize("window", [1, 2, 17, 64, 1000])
def test_window(n, window, cache):
    run_attend(Paged(2, 2, 64, [n + 210, n], 16, cache), n, [n, n], 4, window=window)


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "i8", "f32"])
@pytest.mark.parametrize("n", [1, 4, 100])
def test_cross_attention_sees_every_cached_state(n, cache):
    for dtype in ("bf16", "f32"):
        run_attend(Paged(3, 2, 64, [75, 1, 300], 16, cache), n, [n, n // 2, n], 4, dtype, causal=False)


@pytest.mark.parametrize("cache", ["bf16", "i8", "f32"])
@pytest.mark.parametrize("n", [2, 20, 150])
def test_rows_that_see_nothing(n, cache):
    """No cached token at all, and more new tokens than cached ones: the first
    rows' positions are negative."""
    for dtype in ("bf16", "f32"):
        run_attend(Paged(3, 1, 64, [0, 1, n - 1], 16, cache), n, [n, n, n], 2, dtype)
        run_attend(Paged(2, 1, 64, [0, 5], 16, cache), n, [n, n], 2, dtype, causal=False)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(scale):
    for n, cache in ((1, "bf16"), (4, "i8"), (140, "bf16"), (140, "e4m3"), (140, "i8")):
        run_attend(Paged(2, 2, 64, [n + 90, n], 16, cache), n, [n, n], 4, scale=scale)
    run_attend(Paged(2, 2, 64, [100, 20], 16, "f32"), 20, [20, 20], 4, "f32", scale=scale)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32"),
                                         ("f32", "bf16")])
@pytest.mark.parametrize("n", [2, 5, 60, 150])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_outside_a_rows_range_do_not_reach_it(n, dtype, cache, bad):
    """A key and a value that are NaN or infinite, inside the chunk: the rows
    before it are finite and right, the rows that see it are not numbers."""
    kv, D, at = 90 + n, 64, 90 + n // 2
    P = Paged(1, 1, D, [kv], 16, cache)
    pg, r = P.where(0, at)
    for x in ("k", "v"):
        if cache == "e4m3":
            P.t[x + "_s"][pg, :, r] = float("nan")
        else:
            P.t[x][pg, :, r] = bad
    g = torch.Generator().manual_seed(5)
    q = torch.randn(1, 3, n, D, generator=g).abs().to(IN[dtype])
    o = muse.muse_attn_cache(q.cuda(), **P.gpu(), scale=D ** -0.5).double().cpu().numpy()
    with np.errstate(all="ignore"):
        ro, _, to, _ = attend(P, q, [n], D ** -0.5, q_type=dtype)
    first = at - (kv - n)
    assert (np.abs(o - ro) <= to)[:, :, :first].all()
    assert np.isnan(o[:, :, first:]).all()
    # outside the window of the last rows, inside that of earlier ones
    if n >= 5:
        w = 2
        o = muse.muse_attn_cache(q.cuda(), **P.gpu(), scale=D ** -0.5, window=w).double().cpu().numpy()
        with np.errstate(all="ignore"):
            ro, _, to, _ = attend(P, q, [n], D ** -0.5, window=w, q_type=dtype)
        sees = np.zeros(n, bool)
        sees[first:first + w] = True
        assert (np.abs(o - ro) <= to)[:, :, ~sees].all()
        assert np.isnan(o[:, :, sees]).all()


@pytest.mark.parametrize("n", [1, 6, 140])
def test_lengths_and_pages_out_of_range(n):
    """Lengths past the table and table entries that name no page: the flag, no
    fault; a position without a page is a zero row."""
    P = Paged(2, 2, 64, [200, 160], 16, "bf16")
    P.table[0, 3] = -5
    P.table[1, 1] = P.pages
    run_attend(P, n, [n, n], 4, errbits=8)
    P = Paged(2, 2, 64, [200, 160], 16, "bf16")
    c = P.gpu()
    q = torch.randn(2, 4, n, 64, device="cuda", dtype=torch.bfloat16)
    for kv, new in (([1 << 30, 160], [n, n]), ([-3, 160], [n, n]), ([200, 160], [n + 1, n]),
                    ([200, 160], [-1, n])):
        e = err_word()
        c["kv_len"] = i32(kv)
        o = muse.muse_attn_cache(q, **c, new_len=i32(new), device_error=e)
        torch.cuda.synchronize()
        assert int(e) == 8 and o.shape == q.shape
        with pytest.raises(muse.MuseError, match="page-table"):
            muse.device_status(e)


def test_needed_device_errors_only():
    P = Paged(1, 1, 64, [20], 16, "bf16", wide=9)  # table entries past the need are -1
    run_attend(P, 1, [1], 1)


WRITE = [  # B, n, Hkv, D, kv, new, page
    (1, 1, 1, 64, [1], [1], 16),
    (3, 1, 8, 128, [17, 1, 32], [1, 1, 0], 16),
    (2, 5, 3, 64, [40, 5], [5, 2], 24),
    (2, 100, 2, 128, [100, 131], [100, 77], 16),
    (2, 33, 1, 64, [20, 33], [33, 33], 1),  # sequence 0 has more new tokens than positions
]


@pytest.mark.parametrize("cache", list(CACHE))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", WRITE, ids=lambda c: "B%dn%dh%dD%dp%d" % (c[:4] + (c[6],)))
def test_write_and_read_back(case, dtype, cache):
    B, n, Hkv, D, kv, new, page = case
    P = Paged(B, Hkv, D, kv, page, cache, garbage=False)
    g = torch.Generator().manual_seed(3)
    x = {}
    for t in ("k", "v"):
        x[t] = torch.randn(B, n, Hkv, D, generator=g) * torch.exp(3 * torch.randn(B, n, Hkv, 1, generator=g))
        x[t][0, 0, 0] = 0.0                                   # a row of zeros
        x[t][0, -1, 0, :] = torch.arange(D) - 40.0            # ties of every kind
        x[t][-1, 0, -1] *= 1e-37 if dtype == "f32" else 1e-30  # next to the smallest scales
        x[t] = x[t].to(IN[dtype])
    c, e = P.gpu(), err_word()
    muse.muse_cache_write(x["k"].cuda().transpose(1, 2), x["v"].cuda().transpose(1, 2), **c,
                          new_len=i32(new), device_error=e)
    assert int(e) == 0
    want = {}
    for t in ("k", "v"):
        want[t] = (P.t[t].double().clone(), None if P.t[t + "_s"] is None else P.t[t + "_s"].clone())
        q, s = quantise(x[t].double().numpy(), cache)
        for b, i in itertools.product(range(B), range(n)):
            p = kv[b] - new[b] + i
            if i < new[b] and p >= 0:
                pg, r = P.where(b, p)
                want[t][0][pg, :, r] = torch.from_numpy(q[b, i])
                if s is not None:
                    want[t][1][pg, :, r] = torch.from_numpy(s[b, i]).float()
        got = c[t + "_cache"].double().cpu()
        assert torch.equal(got, want[t][0]), t
        if s is not None:
            assert torch.equal(c[t + "_scale"].cpu(), want[t][1]), t
    # read back every position, past the end too, from a start of its own
    P.t["k"], P.t["v"] = c["k_cache"].cpu(), c["v_cache"].cpu()
    if "k_scale" in c:
        P.t["k_s"], P.t["v_s"] = c["k_scale"].cpu(), c["v_scale"].cpu()
    for start in (None, [max(0, a - 3) for a in kv]):
        N = 7 if start else max(kv) + 2
        for out_type in ("bf16", "f32"):
            got = muse.muse_cache_read(**c, N=N, start=None if start is None else i32(start),
                                       dtype=IN[out_type])
            for t, y in zip(("k", "v"), got):
                y = y.double().cpu().numpy()
                for b in range(B):
                    s0 = start[b] if start else 0
                    hi = min(kv[b], s0 + N)
                    ref = np.zeros((Hkv, N, D))
                    ref[:, :hi - s0] = P.rows(t, b, s0, hi)
                    # one rounding of value times scale, one to the output (2^-126: the fp32 and
                    # bf16 steps below which they are absolute)
                    tol = np.abs(ref) * (HALF["f32"] + HALF[out_type]) * 1.01 + 2.0 ** -133
                    assert (np.abs(y[b] - ref) <= tol).all(), (t, b)


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_write_of_rows_that_are_not_numbers(cache, bad):
    c = muse.make_cache(3, 2, 4, 64, CACHE[cache])
    k = torch.ones(1, 2, 5, 64, device="cuda", dtype=torch.bfloat16)
    k[0, 1, 2, 63] = bad
    v = torch.ones_like(k)
    args = dict(c, table=i32([[2, 0]]), kv_len=i32([5]))
    muse.muse_cache_write(k, v, **args)
    rk, rv = muse.muse_cache_read(**args, N=5)
    lost = torch.zeros(2, 5, dtype=torch.bool)
    lost[1, 2] = True
    assert torch.equal(rk[0].isnan().all(-1).cpu(), lost) and torch.equal(rk[0].isnan().any(-1).cpu(), lost)
    assert torch.isfinite(rv).all()


def test_write_and_read_flag_indices_out_of_range():
    c = muse.make_cache(3, 1, 4, 64)
    k = torch.randn(2, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
    for table, kv, bits in (([[0, 3], [1, 2]], [8, 4], 8), ([[0, -1], [1, 2]], [8, 4], 8),
                            ([[0, -1], [1, 2]], [4, 4], 0), ([[0, 1], [1, 2]], [9, 4], 8),
                            ([[0, 1], [1, 2]], [4, -1], 8)):
        args = dict(c, table=i32(table), kv_len=i32(kv))
        e = err_word()
        muse.muse_cache_write(k, k, **args, device_error=e)
        assert int(e) == bits
        rk, _ = muse.muse_cache_read(**args, N=8, device_error=e)
        assert int(e) == bits
        if table[0][1] in (3, -1):
            assert (rk[0, 0, 4:] == 0).all()
    e = err_word()
    muse.muse_cache_read(**dict(c, table=i32([[0, 1]]), kv_len=i32([8])), N=3, start=i32([-1]), device_error=e)
    assert int(e) == 8


@pytest.mark.parametrize("cache", list(CACHE))
def test_a_conversation(cache):
    """A prompt in chunks, then single tokens, for two sequences of other
    lengths: every answer equals the attention over all rows so far."""
    B, Hq, Hkv, D, page = 2, 4, 2, 64, 16
    c = muse.make_cache(30, Hkv, page, D, CACHE[cache])
    P = Paged(B, Hkv, D, [0, 0], page, cache, garbage=False, wide=12)
    P.table = np.arange(24, dtype=np.int32).reshape(2, 12)[:, ::-1].copy()
    P.pages = 30
    table = torch.from_numpy(P.table).cuda()
    g = torch.Generator().manual_seed(9)
    kv = np.zeros(B, int)
    for n, new in ((100, [100, 37]), (60, [20, 60]), (1, [1, 1]), (1, [1, 0]), (3, [3, 2])):
        q, k, v = (torch.randn(B, h, n, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
        kv = kv + new
        args = dict(c, table=table, kv_len=i32(kv.tolist()), new_len=i32(new))
        muse.muse_cache_write(k.cuda(), v.cuda(), **args)
        o = muse.muse_attn_cache(q.cuda(), **args, scale=0.125).double().cpu().numpy()
        P.kv = kv.tolist()
        P.t["k"], P.t["v"] = c["k_cache"].cpu(), c["v_cache"].cpu()
        if "k_scale" in c:
            P.t["k_s"], P.t["v_s"] = c["k_scale"].cpu(), c["v_scale"].cpu()
        ro, _, to, _ = attend(P, q, new, 0.125)
        for b in range(B):
            assert (np.abs(o[b] - ro[b]) <= to[b])[:, :new[b]].all()


def test_read_back_feeds_the_whole_sequence_operator():
    """A prompt through the causal operator with its keys cached, read back and
    attended by the same operator: the same output, bit for bit."""
    B, H, N, D = 1, 4, 512, 64
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(B, H, N, D, generator=g).mul(D ** -0.25).bfloat16().cuda() for _ in range(3))
    p = dict(C=8, block=128, iters=4, seed=7, topk=1)
    o = muse.muse_attn_fwd_causal(q, k, v, **p)
    c = dict(muse.make_cache(N // 32, H, 32, D), table=i32([list(range(N // 32))[::-1]]), kv_len=i32([N]))
    muse.muse_cache_write(k, v, **c)
    rk, rv = muse.muse_cache_read(**c, N=N)
    assert torch.equal(rk, k) and torch.equal(rv, v)
    assert torch.equal(muse.muse_attn_fwd_causal(q, rk, rv, **p), o)
    # with every key cluster retrieved the acausal operator is exact attention: what the cache answers
    full = muse.muse_attn_fwd(q, k, v, Cq=4, Ck=4, iters=2, seed=1, topk=4, out_dtype=torch.float32)
    got = muse.muse_attn_cache(q, **c, causal=False)
    # the operator's own bound on fp32 outputs of bf16 inputs, weights in bf16, the output's rounding
    tol = 2e-3 + 2.0 ** -8 * float(v.float().abs().max()) + 2.0 ** -8 * full.abs()
    assert ((got.float() - full).abs() <= tol).all()


@pytest.mark.parametrize("n,cache", [(1, "bf16"), (5, "i8"), (200, "e4m3"), (200, "bf16")])
def test_same_bits_and_captured_replays(n, cache):
    """The same call gives the same bits; captured once, replayed with other
    inputs and lengths in place, next to another graph with a workspace of its own."""
    P = Paged(3, 2, 128, [900, 700, n], 16, cache, wide=80)
    c = P.gpu()
    q = torch.randn(3, 8, n, 128, device="cuda").bfloat16()
    new = i32([n, n, n])
    o1 = muse.muse_attn_cache(q, **c, new_len=new, scale=0.1)
    o2 = muse.muse_attn_cache(q, **c, new_len=new, scale=0.1)
    assert torch.equal(o1, o2)
    outs, graphs = [], []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        muse.muse_attn_cache(q, **c, new_len=new, scale=0.1)
    torch.cuda.current_stream().wait_stream(s)
    for scale in (0.1, 0.2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(muse.muse_attn_cache(q, **c, new_len=new, scale=scale))
        graphs.append(g)
    for g in graphs:
        g.replay()
    assert torch.equal(outs[0], o1)
    q.copy_(torch.randn_like(q))
    c["kv_len"].copy_(i32([300, 699, n]))
    eager = [muse.muse_attn_cache(q, **c, new_len=new, scale=s) for s in (0.1, 0.2)]
    graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager[0]) and torch.equal(outs[1], eager[1])


@pytest.mark.parametrize("n", [1, 150])
def test_workspace_contents_and_other_streams(n):
    P = Paged(2, 2, 64, [500, 300 + n], 16, "bf16")
    c = P.gpu()
    q = torch.randn(2, 8, n, 64, device="cuda").bfloat16()
    want = muse.muse_attn_cache(q, **c)
    size = muse.attn_cache_workspace_size(q, **{k: v for k, v in c.items()})
    for fill in (0, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(muse.muse_attn_cache(q, **c, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [muse.muse_attn_cache(q, **c, stream=side) for _ in range(4)]
    both = [muse.muse_attn_cache(q, **c) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got + both)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements, its last pages in use."""
    Hkv, page, D = 8, 256, 128
    pages = (1 << 31) // (Hkv * page * D) + 9
    c = muse.make_cache(pages, Hkv, page, D, torch.float8_e4m3fn)
    table = i32([[pages - 1, 0, pages - 2]])
    kv = 2 * page + 100
    k, v = (torch.randn(1, Hkv, kv, D, device="cuda").bfloat16() for _ in range(2))
    args = dict(c, table=table, kv_len=i32([kv]))
    muse.muse_cache_write(k, v, **args)
    rk, rv = muse.muse_cache_read(**args, N=kv)
    small = dict(muse.make_cache(3, Hkv, page, D, torch.float8_e4m3fn), table=i32([[0, 1, 2]]),
                 kv_len=i32([kv]))
    muse.muse_cache_write(k, v, **small)
    assert all(torch.equal(a, b) for a, b in zip((rk, rv), muse.muse_cache_read(**small, N=kv)))
    for n in (1, 140):
        q = torch.randn(1, 16, n, D, device="cuda").bfloat16()
        assert torch.equal(muse.muse_attn_cache(q, **args, scale=0.1),
                           muse.muse_attn_cache(q, **small, scale=0.1))
