"""The entry points of the passes around attention refuse bad arguments on the host.  Runs without a GPU."""
import ctypes

import pytest
import torch

import exact_attention_128_b200 as fa
from exact_attention_128_b200 import build as fabuild

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: every call below is rejected on the host
I64 = ctypes.c_int64 * 3
I3 = ctypes.c_int * 3
BAD, UNS, WS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    fabuild.build()
    return fa.lib()


def call(fn, base, kw):
    assert set(kw) <= set(base), kw
    return fn(*{**base, **kw}.values())


ST = dict(q_strides=I64(2048, 64, 512), k_strides=I64(2048, 64, 512))
ROPE_TAIL = dict(rotary_dim=64, sections=I3(32, 0, 0), n_axes=1, interleaved=0, eps=1e-6, dtype=fa.FA_DTYPE_BF16)
FWD = dict(q=FAKE, k=FAKE, **ST, wq=FAKE, wk=FAKE, pos=FAKE, pos_sa=0, pos_sb=0, freq=FAKE, qo=FAKE, ko=FAKE, B=1, Hq=4,
           Hkv=2, N=4, d=64, **ROPE_TAIL, stream=None)
APPEND = dict(q=FAKE, k=FAKE, v=FAKE, **ST, v_strides=I64(2048, 64, 512), wq=FAKE, wk=FAKE, pos=FAKE, pos_sa=0, pos_sb=0,
              freq=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, ctx=FAKE, ql=FAKE, qo=FAKE, R=1, Hq=4, Hkv=2, N=4, d=64, bs=16,
              maxb=4, nblocks=10, **ROPE_TAIL, stream=None)
BWD = dict(dqo=FAKE, dko=FAKE, gin=fa.FA_DTYPE_F32, q=FAKE, k=FAKE, **ST, wq=FAKE, wk=FAKE, pos=FAKE, pos_sa=0, pos_sb=0,
           freq=FAKE, dq=FAKE, dk=FAKE, dq_strides=I64(2048, 64, 512), dk_strides=I64(2048, 64, 512),
           gout=fa.FA_DTYPE_BF16, dwq=FAKE, dwk=FAKE, B=2, Hq=4, Hkv=2, N=4, d=64, **ROPE_TAIL, ws=FAKE, ws_bytes=1 << 30,
           stream=None)
SHARED = dict(q=FAKE, kc=FAKE, vc=FAKE, pt=FAKE, pl=FAKE, bt=FAKE, ctx=FAKE, o=FAKE, lse=None, R=4, Hq=12, Hkv=2, d=128,
              bs=16, pb=8, maxb=4, nblocks=100, scale=0.088, dtype=fa.FA_DTYPE_BF16, ws=FAKE, ws_bytes=1 << 40, stream=None)
SCORED = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, ctx=FAKE, w=FAKE, o=FAKE, lse=None, R=4, Hq=12, Hkv=2, d=128, bs=16,
              maxb=4, nblocks=100, scale=0.088, dtype=fa.FA_DTYPE_BF16, ws=FAKE, ws_bytes=1 << 40, stream=None)
EVICT = dict(kc=FAKE, vc=FAKE, bt=FAKE, ctx=FAKE, seq=FAKE, w=FAKE, sp=FAKE, wo=2 * FAKE, so=2 * FAKE, nc=2 * FAKE, R=4,
             Hkv=2, d=128, bs=16, maxb=4, nblocks=100, keep=8, recent=4, dtype=fa.FA_DTYPE_BF16, ws=FAKE,
             ws_bytes=1 << 40, stream=None)

ROTARY = [
    (dict(pos=None), BAD), (dict(freq=None), BAD), (dict(freq=FAKE + 4), BAD), (dict(sections=None), BAD),
    (dict(sections=I3(31, 0, 0)), BAD), (dict(n_axes=0), BAD), (dict(n_axes=4), BAD), (dict(n_axes=2, sections=I3(33, -1, 0)), BAD),
    (dict(eps=0.0), BAD), (dict(eps=float("nan")), BAD), (dict(interleaved=2), BAD), (dict(rotary_dim=128), BAD),
    (dict(rotary_dim=0), BAD), (dict(wq=None), BAD), (dict(q_strides=I64(2048, 68, 512)), BAD), (dict(q_strides=None), BAD),
    (dict(k=FAKE + 2), BAD), (dict(Hq=0), BAD), (dict(d=80), UNS), (dict(dtype=3), UNS),
    (dict(rotary_dim=24, sections=I3(12, 0, 0)), UNS),
]


@pytest.mark.parametrize("kw,code", ROTARY + [(dict(q=None), BAD), (dict(qo=None), BAD), (dict(ko=FAKE + 4), BAD)])
def test_rope_rejects_on_host(L, kw, code):
    assert call(L.fa_qk_norm_rope, FWD, kw) == code


@pytest.mark.parametrize(
    "kw,code",
    ROTARY + [(dict(v=None), BAD), (dict(v_strides=I64(2048, 4, 512)), BAD), (dict(bt=None), BAD), (dict(ql=FAKE + 1), BAD),
              (dict(qo=None), BAD), (dict(maxb=0), BAD), (dict(nblocks=-1), BAD), (dict(bs=32), UNS), (dict(d=256), UNS),
              (dict(dtype=fa.FA_DTYPE_F32), UNS)])
def test_append_rejects_on_host(L, kw, code):
    assert call(L.fa_qk_norm_rope_append, APPEND, kw) == code


@pytest.mark.parametrize(
    "kw,code",
    ROTARY + [(dict(dqo=None), BAD), (dict(dk=None), BAD), (dict(dwq=None), BAD), (dict(dq_strides=I64(0, 64, 512)), BAD),
              (dict(dk_strides=I64(2048, 32, 512)), BAD), (dict(gin=5), UNS), (dict(gout=5), UNS),
              (dict(dtype=fa.FA_DTYPE_F32), UNS), (dict(ws=None), WS), (dict(ws_bytes=16), WS), (dict(ws=FAKE + 16), WS)])
def test_rope_bwd_rejects_on_host(L, kw, code):
    assert call(L.fa_qk_norm_rope_bwd, BWD, kw) == code


DECODE = [
    (dict(q=None), BAD), (dict(kc=FAKE + 8), BAD), (dict(ctx=None), BAD), (dict(o=FAKE + 4), BAD), (dict(lse=FAKE + 2), BAD),
    (dict(Hq=13), BAD), (dict(R=0), BAD), (dict(maxb=0), BAD), (dict(nblocks=0), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("inf")), BAD), (dict(d=96), UNS), (dict(bs=32), UNS), (dict(dtype=fa.FA_DTYPE_F32), UNS),
    (dict(Hq=34), UNS), (dict(R=70000), UNS), (dict(nblocks=1 << 30), UNS), (dict(maxb=1 << 28), UNS), (dict(ws=None), WS),
    (dict(ws_bytes=16), WS), (dict(ws=FAKE + 16), WS),
]


@pytest.mark.parametrize("kw,code", DECODE + [(dict(pt=None), BAD), (dict(pl=FAKE + 2), BAD), (dict(pb=0), BAD)])
def test_shared_rejects_on_host(L, kw, code):
    assert call(L.fa_paged_decode_shared, SHARED, kw) == code


@pytest.mark.parametrize("kw,code", DECODE + [(dict(w=None), BAD), (dict(w=FAKE + 2), BAD)])
def test_scored_rejects_on_host(L, kw, code):
    assert call(L.fa_paged_decode_scored, SCORED, kw) == code


@pytest.mark.parametrize(
    "kw,code",
    [(dict(kc=None), BAD), (dict(sp=None), BAD), (dict(nc=None), BAD), (dict(keep=0), BAD), (dict(recent=-1), BAD),
     (dict(recent=9), BAD), (dict(R=0), BAD), (dict(w=FAKE + 2), BAD), (dict(vc=FAKE + 8), BAD), (dict(wo=FAKE), BAD),
     (dict(so=FAKE), BAD), (dict(nc=FAKE), BAD), (dict(d=80), UNS), (dict(bs=8), UNS), (dict(dtype=fa.FA_DTYPE_F32), UNS),
     (dict(R=70000), UNS), (dict(maxb=1 << 28), UNS), (dict(ws=None), WS), (dict(ws_bytes=16), WS)])
def test_evict_rejects_on_host(L, kw, code):
    assert call(L.fa_paged_evict, EVICT, kw) == code


def test_workspace_sizes(L):
    assert L.fa_qk_norm_rope_bwd_workspace_size(128) % 256 == 0 and L.fa_qk_norm_rope_bwd_workspace_size(0) == 0
    a = L.fa_paged_decode_shared_workspace_size(8, 12, 2, 128, 100, 20, 16)
    assert a >= 8 * 12 * 2 * 129 * 4 and a % 256 == 0
    assert L.fa_paged_decode_shared_workspace_size(8, 12, 2, 128, 0, 20, 16) == 0
    assert L.fa_paged_decode_shared_workspace_size(8, 13, 2, 128, 1, 20, 16) == 0
    b = L.fa_paged_decode_scored_workspace_size(8, 12, 2, 128, 20, 16)
    assert b >= 8 * 12 * 20 * 16 * 4 and b % 256 == 0
    assert L.fa_paged_evict_workspace_size(8, 2, 20, 100) > 0 and L.fa_paged_evict_workspace_size(8, 2, 20, 0) == 0


def test_binding_rejects_cpu_tensors():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    w, pos, freq = torch.zeros(64), torch.zeros(4, dtype=torch.int32), fa.rope_frequencies(64, device="cpu")
    assert freq.dtype == torch.float64 and freq[0] == 1 and abs(freq[16] - 0.01) < 1e-15
    for f in (lambda: fa.qk_norm_rope(q, q, w, w, pos, freq), lambda: fa.qk_norm_rope_bwd(q, q, q, q, w, w, pos, freq),
              lambda: fa.paged_decode_scored(q[0], q, q, pos, pos, w),
              lambda: fa.paged_evict(q, q, pos[None], pos, pos, w, w, 1, 0)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    for bad in (0, 7, -2):
        with pytest.raises(ValueError):
            fa.rope_frequencies(bad, device="cpu")
