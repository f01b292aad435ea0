"""The target's operators (include/lookup_target.h): what needs no GPU.

Refusals of the C entry points (made before any CUDA call), the binding's checks,
and the rotary table's angles.
"""
from __future__ import annotations

import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import prompt_lookup_speculative_gb300 as pkg  # noqa: E402

FAKE = 0x10000        # a non-null, aligned address; never dereferenced by the host checks
S3 = (ctypes.c_int64 * 3)(4096, 512, 128)
S2 = (ctypes.c_int64 * 2)(4096, 512)


@pytest.fixture(scope="module")
def lib():
    return pkg.load_library()


def append(lib, **kw):
    a = dict(q=FAKE, qs=S3, k=FAKE, ks=S3, v=FAKE, vs=S3, kv_len=FAKE, q_len=FAKE, table=FAKE, B=2, N=3, Hq=4, Hkv=2,
             D=128, max_pages=4, pages=8, page=16, rotary=FAKE, rot=128, max_pos=64, inter=0, type=2, kc=FAKE, vc=FAKE,
             out_q=FAKE, status=FAKE, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.lookup_kv_append(*a.values())


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(N=-1), dict(Hq=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(D=1025), dict(max_pages=0),
    dict(pages=0), dict(page=0), dict(page=24), dict(rot=0), dict(rot=7), dict(rot=130), dict(max_pos=0), dict(type=0),
    dict(type=3), dict(kv_len=None), dict(table=None), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None),
    dict(out_q=None), dict(qs=None), dict(ks=None), dict(vs=None), dict(q=FAKE + 1), dict(k=FAKE + 1),
    dict(v=FAKE + 1), dict(kc=FAKE + 1), dict(vc=FAKE + 1), dict(out_q=FAKE + 1), dict(rotary=FAKE + 2),
    dict(kv_len=FAKE + 2), dict(q_len=FAKE + 2), dict(table=FAKE + 2), dict(status=FAKE + 2),
    dict(B=1 << 30, N=1 << 12, Hq=64),
])
def test_append_refuses(lib, bad):
    assert append(lib, **bad) == -1


def test_append_of_nothing(lib):
    assert append(lib, B=0, q=None, k=None, v=None, kv_len=None) == 0
    assert append(lib, N=0) == 0


def attend(lib, **kw):
    a = dict(q=FAKE, qs=S3, kc=FAKE, vc=FAKE, table=FAKE, kv_len=FAKE, q_len=FAKE, B=2, N=3, Hq=4, Hkv=2, D=128,
             max_pages=4, pages=8, page=16, scale=0.1, window=0, type=2, out=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 40,
             stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.lookup_paged_attention(*a.values())


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(N=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(D=96), dict(D=0), dict(D=512), dict(max_pages=0),
    dict(pages=0), dict(page=4), dict(page=48), dict(page=2048), dict(scale=math.inf), dict(scale=math.nan),
    dict(window=-1), dict(type=0), dict(type=5), dict(pages=1 << 27, page=16), dict(q=None), dict(qs=None),
    dict(kc=None), dict(vc=None), dict(table=None), dict(kv_len=None), dict(out=None), dict(ws=None), dict(nbytes=0),
    dict(q=FAKE + 8), dict(kc=FAKE + 8), dict(vc=FAKE + 2), dict(ws=FAKE + 4), dict(out=FAKE + 2), dict(lse=FAKE + 2),
    dict(qs=(ctypes.c_int64 * 3)(4096, 516, 128)), dict(table=FAKE + 1), dict(kv_len=FAKE + 2), dict(q_len=FAKE + 2),
    dict(B=1 << 20, N=1 << 10, Hq=64, Hkv=64),
])
def test_attention_refuses(lib, bad):
    assert attend(lib, **bad) == -1


def test_attention_of_nothing(lib):
    assert attend(lib, B=0, q=None, out=None) == 0
    assert attend(lib, N=0, q=None, out=None) == 0
    assert lib.lookup_paged_attention_workspace_bytes(2, 3, 4, 3, 128) == 0
    assert lib.lookup_paged_attention_workspace_bytes(2, 3, 4, 2, 100) == 0


def verify(lib, **kw):
    a = dict(block=FAKE, len=FAKE, logits=FAKE, ls=S2, type=2, V=1000, noise=FAKE, temperature=FAKE, u=FAKE,
             qprobs=FAKE, qs=S2, point=FAKE, B=2, P=7, acc=FAKE, commit=FAKE, nc=FAKE, lps=FAKE, ws=FAKE,
             nbytes=1 << 40, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.lookup_verify_logits(*a.values())


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(P=-1), dict(P=65537), dict(V=0), dict(V=1 << 30), dict(type=3), dict(type=-1), dict(block=None),
    dict(len=None), dict(logits=None), dict(ls=None), dict(u=None), dict(qs=None), dict(acc=None), dict(commit=None),
    dict(nc=None), dict(ws=None), dict(nbytes=16), dict(logits=FAKE + 1), dict(logits=FAKE + 2, type=0),
    dict(noise=FAKE + 2), dict(temperature=FAKE + 2), dict(u=FAKE + 2), dict(qprobs=FAKE + 2), dict(point=FAKE + 1),
    dict(block=FAKE + 2), dict(len=FAKE + 2), dict(acc=FAKE + 2), dict(commit=FAKE + 2), dict(nc=FAKE + 2),
    dict(lps=FAKE + 2), dict(ws=FAKE + 8),
])
def test_verify_refuses(lib, bad):
    assert verify(lib, **bad) == -1


def test_verify_of_nothing(lib):
    assert verify(lib, B=0, block=None, logits=None) == 0
    assert lib.lookup_verify_logits_workspace_bytes(2, -1, 10) == 0
    assert lib.lookup_verify_logits_workspace_bytes(2, 3, 0) == 0


def test_binding_refuses_host_tensors_and_bad_shapes():
    x = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkg.lookup_paged_attention(x, x, x, n[None], n)
    with pytest.raises(ValueError):
        pkg.lookup_kv_append(x, x, x, n, n[None], x, x)
    with pytest.raises(ValueError):
        pkg.lookup_verify_logits(n[None], n, torch.zeros((1, 2, 8)))


@pytest.mark.parametrize("rot", [2, 32, 128])
def test_rotary_table_angles(rot):
    t = pkg.rotary_table(300001, rot, base=10000.0, device="cpu").double()
    for p in (0, 1, 777, 300000):
        for i in {0, rot // 4, rot // 2 - 1}:
            a = p * 10000.0 ** (-2.0 * i / rot)
            assert abs(float(t[p, i]) - math.cos(a)) < 2 ** -24
            assert abs(float(t[p, rot // 2 + i]) - math.sin(a)) < 2 ** -24


def test_rotary_table_scaling():
    rot, half = 64, 32
    plain = [10000.0 ** (-i / half) for i in range(half)]

    def angle(t, i):          # at position 1
        return math.atan2(float(t[1, half + i]), float(t[1, i]))

    lin = pkg.rotary_table(2, rot, scaling=("linear", 4.0), device="cpu")
    grown = pkg.rotary_table(2, rot, scaling=("base", 4.0), device="cpu")
    bands = pkg.rotary_table(2, rot, scaling=("bands", 8.0, 4096, 32, 1), device="cpu")
    for i in range(half):
        assert angle(lin, i) == pytest.approx(plain[i] / 4, rel=1e-5)
    assert angle(grown, 0) == pytest.approx(plain[0], rel=1e-5)
    assert angle(grown, half - 1) == pytest.approx(plain[-1] / 4, rel=1e-4)
    size = 0.1 * math.log(8.0) + 1.0
    got = [angle(bands, i) / plain[i] for i in range(half)]
    turns = [4096 * f / (2 * math.pi) for f in plain]
    assert all(abs(g - 1) < 1e-4 for g, t in zip(got, turns) if t > 32)
    assert all(abs(g - 1 / 8) < 1e-4 for g, t in zip(got, turns) if t < 1)
    assert all(x >= y - 1e-4 for x, y in zip(got, got[1:]))
    assert float((bands[1, :half] ** 2 + bands[1, half:] ** 2).sqrt().mean()) == pytest.approx(size, rel=1e-5)
    with pytest.raises(ValueError):
        pkg.rotary_table(4, 64, scaling=("other", 2.0), device="cpu")
    with pytest.raises(ValueError):
        pkg.rotary_table(4, 7, device="cpu")
