"""The entry points of the passes around attention refuse bad arguments on the host.  Runs without a GPU."""
import struct

import pytest
import torch

import exact_attention_128_b200 as fa
from exact_attention_128_b200 import build as fabuild

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: every call below is rejected on the host
BAD, UNS, WS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE

# the argument structs of fa.h: pointers and sizes, int64 strides, ints, eps or scale, ints
PACKED = {
    "fa_qk_norm_rope": struct.Struct("8P8q11ifi"),
    "fa_qk_norm_rope_append": struct.Struct("13P11q14ifi"),
    "fa_qk_norm_rope_bwd": struct.Struct("14P14q11if3i"),
    "fa_paged_decode_shared": struct.Struct("11P8ifi"),
    "fa_paged_decode_scored": struct.Struct("10P7ifi"),
    "fa_paged_evict": struct.Struct("12P9i"),
}


@pytest.fixture(scope="module")
def L():
    fabuild.build()
    return fa.lib()


def call(L, name, base, kw):
    """Pack base, with the changes kw, as the entry point's struct."""
    assert set(kw) <= set(base), kw
    flat = []
    for v in {**base, **kw}.values():
        flat += v if isinstance(v, (list, tuple)) else [0 if v is None else v]
    return getattr(L, name)(PACKED[name].pack(*flat), None)


SX, ROW = (32, 0, 0), (2048, 64, 512)  # sections; strides of [1, 4, 4, 64] in a projection
X = dict(q=FAKE, k=FAKE)
W = dict(wq=FAKE, wk=FAKE, pos=FAKE, freq=FAKE)
TAIL = dict(rotary_dim=64, sections=SX, n_axes=1, interleaved=0, eps=1e-6, dtype=fa.FA_DTYPE_BF16)
FWD = dict(**X, **W, qo=FAKE, ko=FAKE, q_strides=ROW, k_strides=ROW, pos_sa=0, pos_sb=0, B=1, Hq=4, Hkv=2, N=4, d=64, **TAIL)
APPEND = dict(**X, v=FAKE, **W, kc=FAKE, vc=FAKE, bt=FAKE, ctx=FAKE, ql=FAKE, qo=FAKE, q_strides=ROW, k_strides=ROW,
              v_strides=ROW, pos_sa=0, pos_sb=0, R=1, Hq=4, Hkv=2, N=4, d=64, bs=16, maxb=4, nblocks=10, **TAIL)
BWD = dict(dqo=FAKE, dko=FAKE, **X, **W, dq=FAKE, dk=FAKE, dwq=FAKE, dwk=FAKE, ws=FAKE, ws_bytes=1 << 30, q_strides=ROW,
           k_strides=ROW, dq_strides=ROW, dk_strides=ROW, pos_sa=0, pos_sb=0, B=2, Hq=4, Hkv=2, N=4, d=64, **TAIL,
           gin=fa.FA_DTYPE_F32, gout=fa.FA_DTYPE_BF16)
SPACE = dict(ws=FAKE, ws_bytes=1 << 40)
SHARED = dict(q=FAKE, kc=FAKE, vc=FAKE, pt=FAKE, pl=FAKE, bt=FAKE, ctx=FAKE, o=FAKE, lse=None, **SPACE, R=4, Hq=12, Hkv=2,
              d=128, bs=16, pb=8, maxb=4, nblocks=100, scale=0.088, dtype=fa.FA_DTYPE_BF16)
SCORED = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, ctx=FAKE, w=FAKE, o=FAKE, lse=None, **SPACE, R=4, Hq=12, Hkv=2, d=128,
              bs=16, maxb=4, nblocks=100, scale=0.088, dtype=fa.FA_DTYPE_BF16)
EVICT = dict(kc=FAKE, vc=FAKE, bt=FAKE, ctx=FAKE, seq=FAKE, w=FAKE, sp=FAKE, wo=2 * FAKE, so=2 * FAKE, nc=2 * FAKE, **SPACE,
             R=4, Hkv=2, d=128, bs=16, maxb=4, nblocks=100, keep=8, recent=4, dtype=fa.FA_DTYPE_BF16)

ROTARY = [
    (dict(pos=None), BAD), (dict(freq=None), BAD), (dict(freq=FAKE + 4), BAD),
    (dict(sections=(31, 0, 0)), BAD), (dict(n_axes=0), BAD), (dict(n_axes=4), BAD), (dict(n_axes=2, sections=(33, -1, 0)), BAD),
    (dict(eps=0.0), BAD), (dict(eps=float("nan")), BAD), (dict(interleaved=2), BAD), (dict(rotary_dim=128), BAD),
    (dict(rotary_dim=0), BAD), (dict(wq=None), BAD), (dict(wk=FAKE + 1), BAD),
    (dict(q_strides=(2048, 68, 512)), BAD),
    (dict(k=FAKE + 2), BAD), (dict(Hq=0), BAD), (dict(d=80), UNS), (dict(dtype=3), UNS),
    (dict(rotary_dim=24, sections=(12, 0, 0)), UNS),
]


@pytest.mark.parametrize("kw,code", ROTARY + [(dict(q=None), BAD), (dict(qo=None), BAD), (dict(ko=FAKE + 4), BAD),
                                              (dict(wk=FAKE + 2, dtype=fa.FA_DTYPE_F32), BAD)])
def test_rope_rejects_on_host(L, kw, code):
    assert call(L, "fa_qk_norm_rope", FWD, kw) == code


@pytest.mark.parametrize(
    "kw,code",
    ROTARY + [(dict(v=None), BAD), (dict(v_strides=(2048, 4, 512)), BAD), (dict(bt=None), BAD), (dict(ql=FAKE + 1), BAD),
              (dict(qo=None), BAD), (dict(maxb=0), BAD), (dict(nblocks=-1), BAD), (dict(bs=32), UNS), (dict(d=256), UNS),
              (dict(dtype=fa.FA_DTYPE_F32), UNS)])
def test_append_rejects_on_host(L, kw, code):
    assert call(L, "fa_qk_norm_rope_append", APPEND, kw) == code


@pytest.mark.parametrize(
    "kw,code",
    ROTARY + [(dict(dqo=None), BAD), (dict(dk=None), BAD), (dict(dwq=None), BAD), (dict(dq_strides=(0, 64, 512)), BAD),
              (dict(dk_strides=(2048, 32, 512)), BAD), (dict(gin=5), UNS), (dict(gout=5), UNS),
              (dict(dtype=fa.FA_DTYPE_F32), UNS), (dict(ws=None), WS), (dict(ws_bytes=16), WS), (dict(ws=FAKE + 16), WS)])
def test_rope_bwd_rejects_on_host(L, kw, code):
    assert call(L, "fa_qk_norm_rope_bwd", BWD, kw) == code


DECODE = [
    (dict(q=None), BAD), (dict(kc=FAKE + 8), BAD), (dict(ctx=None), BAD), (dict(o=FAKE + 4), BAD), (dict(lse=FAKE + 2), BAD),
    (dict(Hq=13), BAD), (dict(R=0), BAD), (dict(maxb=0), BAD), (dict(nblocks=0), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("inf")), BAD), (dict(d=96), UNS), (dict(bs=32), UNS), (dict(dtype=fa.FA_DTYPE_F32), UNS),
    (dict(Hq=34), UNS), (dict(R=70000), UNS), (dict(nblocks=1 << 30), UNS), (dict(maxb=1 << 28), UNS), (dict(ws=None), WS),
    (dict(ws_bytes=16), WS), (dict(ws=FAKE + 16), WS),
]


@pytest.mark.parametrize("kw,code", DECODE + [(dict(pt=None), BAD), (dict(pl=FAKE + 2), BAD), (dict(pb=0), BAD)])
def test_shared_rejects_on_host(L, kw, code):
    assert call(L, "fa_paged_decode_shared", SHARED, kw) == code


@pytest.mark.parametrize("kw,code", DECODE + [(dict(w=None), BAD), (dict(w=FAKE + 2), BAD)])
def test_scored_rejects_on_host(L, kw, code):
    assert call(L, "fa_paged_decode_scored", SCORED, kw) == code


@pytest.mark.parametrize(
    "kw,code",
    [(dict(kc=None), BAD), (dict(sp=None), BAD), (dict(nc=None), BAD), (dict(keep=0), BAD), (dict(recent=-1), BAD),
     (dict(recent=9), BAD), (dict(R=0), BAD), (dict(w=FAKE + 2), BAD), (dict(vc=FAKE + 8), BAD), (dict(wo=FAKE), BAD),
     (dict(so=FAKE), BAD), (dict(nc=FAKE), BAD), (dict(d=80), UNS), (dict(bs=8), UNS), (dict(dtype=fa.FA_DTYPE_F32), UNS),
     (dict(R=70000), UNS), (dict(maxb=1 << 28), UNS), (dict(maxb=200, keep=1000, ws=None), WS),
     (dict(maxb=200, keep=1000, ws_bytes=16), WS)])
def test_evict_rejects_on_host(L, kw, code):
    assert call(L, "fa_paged_evict", EVICT, kw) == code


def test_null_struct_is_refused(L):
    for name in PACKED:
        assert getattr(L, name)(None, None) == BAD


def test_structs_match_the_header(L, tmp_path):
    """PACKED fills exactly the C structs: their sizes, and one field near each end."""
    import os
    import subprocess

    names = list(PACKED)
    body = "".join(f'printf("%zu %zu\\n", sizeof({n}_args), offsetof({n}_args, dtype));' for n in names)
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "fa.h"\nint main(void){' + body + "return 0;}")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-I", inc, "-o", str(tmp_path / "s"), str(src)], check=True)
    out = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split()
    for i, n in enumerate(names):
        size, at = int(out[2 * i]), int(out[2 * i + 1])
        packed = PACKED[n]
        last = 2 if n == "fa_qk_norm_rope_bwd" else 0  # ints behind dtype
        assert packed.size + (-packed.size) % 8 == size and at == packed.size - 4 * (1 + last), n


def test_workspace_sizes(L):
    assert L.fa_qk_norm_rope_bwd_workspace_size(128) % 256 == 0 and L.fa_qk_norm_rope_bwd_workspace_size(0) == 0
    a = L.fa_paged_decode_shared_workspace_size(8, 12, 2, 128, 100, 20, 16)
    assert a >= 8 * 12 * 2 * 129 * 4 and a % 256 == 0
    assert L.fa_paged_decode_shared_workspace_size(8, 12, 2, 128, 0, 20, 16) == 0
    assert L.fa_paged_decode_shared_workspace_size(8, 13, 2, 128, 1, 20, 16) == 0
    b = L.fa_paged_decode_scored_workspace_size(8, 12, 2, 128, 20, 16)
    assert b >= 8 * 12 * 20 * 16 * 4 and b % 256 == 0
    assert L.fa_paged_evict_workspace_size(8, 2, 200, 1000) > 8 * 2 * 1000 * 8  # two lists of up to 1000 rows
    assert L.fa_paged_evict_workspace_size(8, 2, 20, 100) == 0  # few rows: none
    assert L.fa_paged_evict_workspace_size(8, 2, 200, 0) == 0


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


@pytest.mark.parametrize("name,base,kw", [
    ("fa_qk_norm_rope_append", APPEND, dict(maxb=(1 << 26) + 1)), ("fa_paged_decode_shared", SHARED, dict(pb=(1 << 26) + 1)),
    ("fa_paged_decode_shared", SHARED, dict(maxb=(1 << 26) + 1)), ("fa_paged_decode_scored", SCORED, dict(maxb=(1 << 26) + 1)),
    ("fa_paged_evict", EVICT, dict(maxb=(1 << 26) + 1))])
def test_tables_of_more_than_2_30_tokens_are_refused(L, name, base, kw):
    """A kernel's token index plus its grid's stride stays inside 32 bits."""
    assert call(L, name, base, kw) == UNS


def on_tensor_cores(L, R, Hq, Hkv, d, blocks):
    """Which way a prefix goes, by the workspace: the tensor-core kernel leaves partial results of 256 rows a CTA."""
    G = Hq // Hkv
    items = -(-R // (2 * (128 // G))) * Hkv
    tiles = items * (-(-148 // items) + 1) * 256 * (d + 1) * 4
    pieces = R * Hq * (64 + 1) * (d + 1) * 4  # (a request's own 4 blocks are one piece)
    assert tiles > 2 * pieces, "sizes at which the two cannot be told apart"
    return L.fa_paged_decode_shared_workspace_size(R, Hq, Hkv, d, blocks, 4, 16) >= tiles


@pytest.mark.parametrize("R,Hq,Hkv,d,blocks,want", [
    (1, 4, 1, 128, 1024, False), (4, 4, 1, 128, 44, True), (1, 32, 8, 128, 125, False), (2, 16, 2, 128, 125, True), (4, 8, 2, 128, 500, False),
    (10, 6, 2, 128, 250, False), (8, 12, 2, 128, 125, True), (8, 32, 8, 128, 1024, True), (4, 4, 1, 128, 2048, False),
    (4, 32, 8, 64, 2048, False), (16, 8, 2, 64, 500, False), (8, 32, 8, 64, 1024, True)])
def test_prefix_goes_the_faster_way(L, R, Hq, Hkv, d, blocks, want):
    """Calls of few rows of which both ways were measured."""
    assert on_tensor_cores(L, R, Hq, Hkv, d, blocks) == want


def test_the_timeout_self_test_takes_sizes_of_the_tensor_core_kernel(L):
    pack = lambda **kw: PACKED["fa_paged_decode_shared"].pack(*(0 if v is None else v for v in {**SHARED, **kw}.values()))
    assert L.fa_selftest_shared_timeout(None, 1, None) == BAD
    assert L.fa_selftest_shared_timeout(pack(R=64, pb=128), -1, None) == BAD
    assert L.fa_selftest_shared_timeout(pack(R=64, pb=128, o=None), 1, None) == BAD
    assert L.fa_selftest_shared_timeout(pack(R=1, pb=8), 1, None) == UNS


def test_dynamic_shared_memory_is_aligned():
    """16-byte accesses need it: every dynamic array says so, or its kernel rounds (or checks) the address itself."""
    import glob
    import os
    import re

    csrc = os.path.join(os.path.dirname(os.path.abspath(fa.__file__)), "csrc")
    seen = 0
    for path in sorted(glob.glob(os.path.join(csrc, "*.cu*"))):
        lines = open(path).read().splitlines()
        for i, line in enumerate(lines):
            if "extern __shared__" not in line:
                continue
            seen += 1
            aligned = re.search(r"__align__\((16|128|1024)\)", line) or "1023" in "".join(lines[i + 1 : i + 3])
            assert aligned, f"{os.path.basename(path)}:{i + 1}: {line.strip()}"
    assert seen >= 10


@pytest.mark.parametrize("which", ["dq", "dk"])
def test_gradient_rows_that_overlap_are_refused(L, which):
    """dq [2, 4, 4, 64], dk [2, 2, 4, 64]: a projection's layout and permuted slices pass (to the next check)."""
    H = 4 if which == "dq" else 2
    for strides in ((64 * H, 64, 64 * H), (1024, 64, 64), (64, 96, 2048), (2048, 64, 64 * H - 8), (64 * 4 * H - 64, 256, 64)):
        assert call(L, "fa_qk_norm_rope_bwd", BWD, {which + "_strides": strides, "ws": None}) == BAD, strides
    for strides in ((64 * 4 * H, 256, 64), (4096, 64, 512), (64, 128, 128 * H), (72, 4096, 1024), (256 * H, 64, 64 * H),
                    (2**62, 64, 512)):
        assert call(L, "fa_qk_norm_rope_bwd", BWD, {which + "_strides": strides, "ws": None}) == WS, strides
