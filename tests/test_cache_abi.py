"""Host-side checks of the paged-cache calls, no GPU needed: refusals of the C
entry points and of the Python calls, and the plain forms that the GPU tests
compare with, against torch's own conversions and attention."""
import ctypes

import numpy as np
import pytest
import torch

import clustered_multipole_approximation_b200 as muse
from clustered_multipole_approximation_b200 import build
from clustered_multipole_approximation_b200.kv_cache import muse_cache, muse_cache_index, muse_strides
from cache_ref import Paged, attend, quantise, round_e4m3

FAKE = 0x1000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return muse.load_library()


def shape(B=2, Hq=4, Hkv=2, N=3, D=64, dt=0, out=0):
    return muse.muse_shape(B, Hq, Hkv, N, D, dt, out)


def cache(k=FAKE, v=FAKE, ks=None, vs=None, pages=4, page=16, dt=0):
    return muse_cache(k, v, ks, vs, pages, page, dt)


def index(table=FAKE, kv=FAKE, new=None, wide=2):
    return muse_cache_index(table, kv, new, wide)


def strides(H=4, N=3, D=64):
    return muse_strides(H * N * D, N * D, D)


BAD = [  # (status, what)
    (1, dict(sh=shape(B=0))), (1, dict(sh=shape(N=0))), (1, dict(sh=shape(Hq=3))),
    (2, dict(sh=shape(D=96))), (1, dict(sh=shape(dt=2))), (2, dict(sh=shape(out=1))),
    (2, dict(sh=shape(N=(1 << 28) + 1))), (2, dict(sh=shape(B=1 << 20, N=1 << 20))),
    (1, dict(ca=cache(k=None))), (1, dict(ca=cache(dt=4))), (1, dict(ca=cache(dt=-1))),
    (1, dict(ca=cache(pages=0))), (1, dict(ca=cache(page=0))), (1, dict(ca=cache(dt=2))),
    (1, dict(ca=cache(dt=3, ks=FAKE))), (1, dict(ca=cache(ks=FAKE, vs=FAKE))),
    (1, dict(ca=cache(k=FAKE + 8))), (1, dict(ca=cache(dt=2, ks=FAKE + 2, vs=FAKE))),
    (1, dict(ix=index(table=None))), (1, dict(ix=index(kv=None))), (1, dict(ix=index(wide=0))),
    (1, dict(ix=index(table=FAKE + 1))), (1, dict(ix=index(new=FAKE + 1))),
    (2, dict(ca=cache(page=1 << 20), ix=index(wide=(1 << 10) + 1))),
]
BAD_CALL = [
    (1, dict(x=None)), (1, dict(x=FAKE + 2)), (1, dict(err=FAKE + 1)),
    (1, dict(st=muse_strides(768, 192, 60))), (1, dict(st=muse_strides(768, -64, 64))),
    (1, dict(st=None)),
]


@pytest.mark.parametrize("call", ["write", "read", "attend"])
@pytest.mark.parametrize("want,bad", BAD + BAD_CALL)
def test_refusals(lib, call, want, bad):
    a = dict(sh=shape(), ca=cache(), ix=index(), x=FAKE, err=None, st=strides())
    a.update(bad)
    if call == "read" and "st" in bad:
        pytest.skip("read has no strides")
    if call == "write":
        st = lib.muse_cache_write(a["x"], a["st"], FAKE, strides(), a["sh"], a["ca"], a["ix"], a["err"], None)
    elif call == "read":
        st = lib.muse_cache_read(a["x"], FAKE, a["sh"], a["ca"], a["ix"], None, a["err"], None)
    else:
        st = lib.muse_attn_cache(a["x"], a["st"], FAKE, strides(), None, a["sh"], a["ca"], a["ix"], 1.0, 1, 0,
                                 a["err"], FAKE, 1 << 40, None)
        if "sh" in bad or "ca" in bad or "ix" in bad:
            assert lib.muse_attn_cache_workspace_size(a["sh"], a["ca"], a["ix"]) == 0
    assert st == want and lib.muse_last_error()


def test_refusals_of_the_attention(lib):
    def call(scale=1.0, causal=1, window=0, os=None, lse=None, ws=FAKE, size=1 << 40, sh=None):
        sh = sh or shape()
        return lib.muse_attn_cache(FAKE, strides(), FAKE, os or strides(), lse, sh, cache(), index(), scale,
                                   causal, window, None, ws, size, None)

    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(causal=2) == 1 and call(window=-1) == 1 and call(causal=0, window=4) == 1
    assert call(lse=FAKE + 2) == 1 and call(ws=FAKE + 16) == 1
    assert call(ws=None) == 3 and call(size=1) == 3
    for s in ((0, 192, 64), (768, 0, 64), (768, 192, 0), (768, 128, 64), (192, 192, 64)):
        assert call(os=muse_strides(*s)) == 1 and b"overlap" in lib.muse_last_error()
    assert lib.muse_attn_cache_workspace_size(shape(), cache(), index()) > 0
    assert lib.muse_cache_read(FAKE, FAKE, shape(), cache(), index(), FAKE + 2, None, None) == 1


def test_refusals_in_python():
    B, Hkv, D, page = 2, 2, 64, 4
    c = muse.make_cache(3, Hkv, page, D, device="cpu")
    k = torch.zeros(B, Hkv, 1, D, dtype=torch.bfloat16)
    t, n = torch.zeros(B, 2, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        muse.muse_cache_write(k, k, **c, table=t, kv_len=n)
    with pytest.raises(ValueError, match="CUDA"):
        muse.muse_attn_cache(k, **c, table=t, kv_len=n)
    with pytest.raises(ValueError, match="CUDA"):
        muse.muse_cache_read(**c, table=t, kv_len=n, N=4)
    with pytest.raises(ValueError, match="shape"):
        muse.muse_cache_write(k, k[:, :1], **c, table=t, kv_len=n)
    with pytest.raises(TypeError, match="cache dtype"):
        muse.make_cache(3, Hkv, page, D, torch.float16, device="cpu")


@pytest.mark.gpu
def test_refusals_in_python_on_the_device():
    B, Hkv, D, page = 2, 2, 64, 4
    c = muse.make_cache(3, Hkv, page, D)
    c8 = muse.make_cache(3, Hkv, page, D, torch.int8)
    q = torch.zeros(B, Hkv, 1, D, dtype=torch.bfloat16, device="cuda")
    t, n = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, 2), (B,)))
    ok = dict(c, table=t, kv_len=n)
    for bad in (dict(table=t.long()), dict(table=t[:1]), dict(kv_len=n.cpu()), dict(kv_len=n[:1]),
                dict(new_len=n.long()), dict(v_cache=c["v_cache"][:2]), dict(k_scale=c8["k_scale"]),
                dict(k_cache=c8["k_cache"], v_cache=c8["v_cache"]),
                dict(out=q.float()), dict(lse=torch.zeros(B, Hkv, 2, device="cuda")),
                dict(out=q[:1].expand(B, Hkv, 1, D)), dict(scale=float("inf")), dict(window=-1),
                dict(causal=False, window=3), dict(workspace=torch.zeros(0, dtype=torch.uint8, device="cuda")),
                dict(device_error=n)):
        with pytest.raises((ValueError, TypeError, muse.MuseError)):
            muse.muse_attn_cache(q, **{**ok, **bad})
    for x in (q.half(), q[:, :1], q[..., :32], q.transpose(2, 3), q.cpu()):
        with pytest.raises((ValueError, TypeError, muse.MuseError)):
            muse.muse_attn_cache(x, **ok)
        with pytest.raises((ValueError, TypeError, muse.MuseError)):
            muse.muse_cache_write(x, x, **ok)
    with pytest.raises(ValueError):
        muse.muse_cache_read(**ok, N=4, out=(q, q))
    with pytest.raises(ValueError):
        muse.muse_cache_read(**ok, N=4, start=n[:1])


def test_plain_e4m3_rounding_is_the_type_s():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    every = np.unique(every[np.isfinite(every)])
    mid = (every[1:] + every[:-1]) / 2
    x = np.concatenate([every, mid, mid * (1 + 1e-6), mid * (1 - 1e-6)])
    x = x.astype(np.float32).astype(np.float64)  # torch's conversion starts from fp32
    assert (round_e4m3(x) == torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()).all()


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
def test_plain_quantisation_is_within_half_a_step(cache):
    g = np.random.Generator(np.random.PCG64(1))
    x = g.standard_normal((50, 64)) * np.exp2(g.integers(-100, 100, (50, 1)))
    q, s = quantise(x.astype(np.float32), cache)
    err = np.abs(q * s[:, None] - x.astype(np.float32))
    top = np.abs(x).max(-1, keepdims=True)
    if cache == "i8":
        assert (err <= top / 127 * 0.5 * (1 + 1e-6) + 127 * s[:, None] * 2.0 ** -24).all() and np.abs(q).max() == 127
    else:
        assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, s[:, None] * 2.0 ** -10) * (1 + 1e-6)).all()
        assert (np.abs(q).max(-1) > 224 - 8).all() and np.abs(q).max() <= 448


def test_plain_attention_is_softmax_attention():
    P = Paged(2, 2, 64, [40, 23], 8, "f32")
    q = torch.randn(2, 4, 5, 64, generator=torch.Generator().manual_seed(0))
    o, lse, _, _ = attend(P, q, [5, 5], 0.2, q_type="f32")
    for b in range(2):
        K = torch.from_numpy(P.rows("k", b, 0, P.kv[b])).repeat_interleave(2, 0)
        V = torch.from_numpy(P.rows("v", b, 0, P.kv[b])).repeat_interleave(2, 0)
        mask = torch.ones(5, P.kv[b], dtype=torch.bool).tril(P.kv[b] - 5)
        want = torch.nn.functional.scaled_dot_product_attention(q[b].double(), K, V, attn_mask=mask, scale=0.2)
        assert np.allclose(o[b], want.numpy(), atol=1e-12)
        x = (0.2 * q[b].double() @ K.transpose(1, 2)).masked_fill(~mask, -torch.inf)
        assert np.allclose(lse[b], torch.logsumexp(x, -1).numpy(), atol=1e-12)


@pytest.mark.parametrize("call", ["write", "read", "attend"])
def test_more_rows_than_an_index_holds(lib, call):
    """2^31 page rows of a head dimension of 64 are more than 256 GB of K and V."""
    ca, ix, sh = cache(pages=1 << 26, page=16), index(), shape()
    args = dict(write=(FAKE, strides(), FAKE, strides(), sh, ca, ix, None, None),
                read=(FAKE, FAKE, sh, ca, ix, None, None, None),
                attend=(FAKE, strides(), FAKE, strides(), None, sh, ca, ix, 1.0, 1, 0, None, FAKE, 1, None))
    f = getattr(lib, "muse_attn_cache" if call == "attend" else "muse_cache_" + call)
    assert f(*args[call]) == 2 and b"2^31" in lib.muse_last_error()
    assert lib.muse_attn_cache_workspace_size(sh, ca, ix) == 0
