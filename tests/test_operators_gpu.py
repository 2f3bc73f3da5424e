"""The passes around attention against their fp64 oracle.

Tolerances, from the arithmetic.  A result stored in a type is off by half a step of it
(relative eps / 2); in front of that stand fp32 operations:
  norm + rotation   a few roundings (2^-24 each) of the row's largest value: 2^-20 of it.
  scores            a dot product of d terms in fp32: (d + 8) 2^-24 sum_c |q_c k_c| scale =: delta, so a
                    probability is off by 2 delta relative, the log-sum by delta (+ 2^-20 of its size);
  P V               P as two bf16 parts keeps 2^-16 of it, the exponential 2^-22: 2^-15 max|v| with the sums.
Weight gradients: n products summed in fp32, in runs of at most n / 64: 2^-24 (n / 64 + 80) sum |g n| at most.  A
turned value g = a cos t - b sin t may cancel: cos and sin are off by 2^-22.3 (the angle, reduced to half a turn and
rounded to 2^-25 turns, times 2 pi) + 2^-23 (the function), the two products and the difference by 2^-24 each, so g is
off by at most 2^-21 (|a| + |b|) however small it is, and the sum by 2^-21 sum (|a| + |b|) |n| more.
"""
import math

import numpy as np
import pytest
import torch

import exact_attention_128_b200 as fa
from exact_attention_128_b200.workloads import randn
from oracle import attention_fp64 as ora
from oracle import operators_fp64 as ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0**-8, F32: 2.0**-24}


def near(got, ref, slack, what=""):
    """|got - ref| <= half a step of ref + slack, elementwise."""
    g = got.detach().double().cpu().numpy()
    with np.errstate(invalid="ignore"):  # -inf against -inf
        off = np.abs(g - ref) - (HALF.get(got.dtype, 0) * np.abs(ref) * (1 + 2.0**-6) + slack)
    same_inf = np.isinf(ref) & (g == ref)
    off = np.where(same_inf, 0.0, off)
    worst = off.max(initial=-1.0)
    assert worst <= 0, f"{what}: {worst:.3e} over its bound"


def clean():
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK


# ------------------------------------------------------------------------------------------ norm + rotation
def rope_inputs(B, Hq, Hkv, N, d, rd, sections, dtype, norm, seed, far=False):
    proj = randn((B, N, Hq + 2 * Hkv, d), seed, dtype).cuda()
    q, k, v = (t.transpose(1, 2) for t in proj.split([Hq, Hkv, Hkv], 2))
    w = [(1 + 0.2 * randn((d,), seed + i, F32)).to(dtype).cuda() if norm else None for i in (1, 2)]
    g = torch.Generator().manual_seed(seed)
    top = 2**31 - 1 if far else 9000
    pos = torch.randint(-top if far else 0, top, (len(sections), B, N), generator=g, dtype=torch.int64).to(torch.int32)
    return q, k, v, w, pos.cuda(), fa.rope_frequencies(rd)


ROPE = [
    # B, Hq, Hkv, N, d, rd, sections, interleaved, dtype, norm
    (1, 1, 1, 1, 64, 64, (32,), False, BF, True),
    (2, 12, 2, 1, 128, 128, (64,), False, BF, True),
    (2, 5, 5, 37, 96, 96, (48,), True, BF, True),
    (1, 8, 2, 301, 128, 128, (16, 24, 24), False, BF, True),
    (3, 6, 1, 67, 128, 64, (8, 12, 12), True, BF, True),
    (1, 4, 4, 130, 256, 128, (32, 32), False, BF, True),
    (2, 3, 1, 19, 256, 256, (128,), True, F32, True),
    (2, 12, 12, 49, 64, 64, (16, 16), True, F32, True),
    (1, 3, 3, 33, 96, 48, (24,), False, F32, False),
    (5, 2, 1, 7, 64, 32, (0, 16), False, BF, False),
    (1, 7, 7, 2050, 64, 16, (8,), False, BF, True),
]


def check_rope(x, got, w, pos, freq, sec, inter, what):
    ref = ops.norm_rope(x, w, pos.cpu(), freq, sec, inter, 1e-6)
    near(got, ref, 2.0**-20 * np.abs(ref).max(-1, keepdims=True), what)


@pytest.mark.parametrize("B,Hq,Hkv,N,d,rd,sec,inter,dtype,norm", ROPE)
def test_qk_norm_rope(B, Hq, Hkv, N, d, rd, sec, inter, dtype, norm):
    q, k, _, (wq, wk), pos, freq = rope_inputs(B, Hq, Hkv, N, d, rd, sec, dtype, norm, 100 + d)
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, pos, freq, sections=sec, interleaved=inter)
    clean()
    assert qo.is_contiguous() and ko.is_contiguous() and qo.dtype == dtype
    check_rope(q, qo, wq, pos, freq, sec, inter, "q")
    check_rope(k, ko, wk, pos, freq, sec, inter, "k")
    # contiguous inputs and shared positions give the same bits as views and repeated positions
    one = pos[:, :1]
    a = fa.qk_norm_rope(q.contiguous(), k.contiguous(), wq, wk, one.expand(-1, B, -1), freq, sections=sec, interleaved=inter)
    b = fa.qk_norm_rope(q, k, wq, wk, one.expand(-1, B, -1).contiguous(), freq, sections=sec, interleaved=inter)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def pair_size(dy, rd, inter):
    """|a| + |b| of each value's pair; |value| where it does not turn."""
    y = np.abs(ora.to_f64(dy))
    out = y.copy()
    i = np.arange(rd // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
    out[..., a] = out[..., b] = y[..., a] + y[..., b]
    return out


def test_far_and_negative_positions():
    q, k, _, (wq, wk), pos, freq = rope_inputs(2, 3, 1, 65, 128, 128, (64,), F32, True, 7, far=True)
    pos[0, 0, :2] = torch.tensor([2**31 - 1, -(2**31)])
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, pos, freq)
    clean()
    # a position of 2^31 radians in 64 bits is off by 2^31 2^-53 (the oracle's too), in turns by 2^-24 pi
    ref = ops.norm_rope(q, wq, pos.cpu(), freq, (64,), False, 1e-6)
    near(qo, ref, (2.0**-20 + 4 * 2.0**-22) * np.abs(ref).max(-1, keepdims=True))
    ref = ops.norm_rope(k, wk, pos.cpu(), freq, (64,), False, 1e-6)
    near(ko, ref, (2.0**-20 + 4 * 2.0**-22) * np.abs(ref).max(-1, keepdims=True))


def test_rows_of_zeros_and_huge_values():
    q, k, _, (wq, wk), pos, freq = rope_inputs(1, 2, 2, 8, 64, 64, (32,), BF, True, 8)
    q, k = q.clone(), k.clone()
    q[0, 0, 3] = 0
    k[0, 1] = 2.0**60  # squares near the top of fp32
    q[0, 1, 2, 5] = float("inf")
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, pos, freq)
    clean()
    assert (qo[0, 0, 3] == 0).all() and not torch.isfinite(qo[0, 1, 2]).all()
    keep = [t for t in range(8) if t != 2]
    assert torch.isfinite(qo[0, 1, keep]).all() and torch.isfinite(qo[0, 0]).all()
    check_rope(k, ko, wk, pos, freq, (32,), False, "k")


@pytest.mark.parametrize("gin,gout", [(F32, BF), (BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("B,Hq,Hkv,N,d,rd,sec,inter,dtype,norm", ROPE)
def test_qk_norm_rope_bwd(B, Hq, Hkv, N, d, rd, sec, inter, dtype, norm, gin, gout):
    if dtype == F32 and (gin, gout) != (F32, F32):
        pytest.skip("fp32 inputs have fp32 gradients")
    q, k, _, (wq, wk), pos, freq = rope_inputs(B, Hq, Hkv, N, d, rd, sec, dtype, norm, 200 + d)
    dqo, dko = (randn(t.shape, 300 + i, gin).cuda() for i, t in enumerate((q, k)))
    args = (dqo, dko, q, k, wq, wk, pos, freq)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(*args, sections=sec, interleaved=inter, grad_dtype=gout)
    clean()
    for x, dy, w, dx, dw in ((q, dqo, wq, dq, dwq), (k, dko, wk, dk, dwk)):
        assert dx.dtype == gout and dx.transpose(1, 2).is_contiguous()  # the projection's order
        ref, rw = ops.norm_rope_bwd(dy, x, w, pos.cpu(), freq, sec, inter, 1e-6)
        g = np.abs(ops.norm_rope_bwd(dy, x, None, pos.cpu(), freq, sec, inter, 1e-6)[0])
        scale = np.abs(ref).max(-1, keepdims=True)
        if norm:
            xx = ora.to_f64(x)
            n = np.abs(xx) / np.sqrt((xx * xx).mean(-1, keepdims=True) + 1e-6)
            r = 1 / np.sqrt((xx * xx).mean(-1, keepdims=True) + 1e-6)
            size = pair_size(dy, rd, inter)
            scale = (size * np.abs(ora.to_f64(w)) * r).max(-1, keepdims=True) * (1 + n.max(-1, keepdims=True))
            rows = x.shape[0] * x.shape[1] * x.shape[2]
            slack = 2.0**-24 * (rows / 64 + 80) * g * n + 2.0**-21 * size * n
            near(dw, rw, slack.reshape(-1, d).sum(0), "dw")
        else:
            assert dw is None
        near(dx, ref, 2.0**-20 * scale, "dx")
    again = fa.qk_norm_rope_bwd(*args, sections=sec, interleaved=inter, grad_dtype=gout)
    assert all(a is b or torch.equal(a, b) for a, b in zip((dq, dk, dwq, dwk), again))


def test_bwd_into_a_fused_projection_gradient():
    B, Hq, Hkv, N, d = 2, 4, 2, 21, 64
    q, k, _, (wq, wk), pos, freq = rope_inputs(B, Hq, Hkv, N, d, d, (32,), BF, True, 11)
    dqo, dko = (randn(t.shape, 310 + i, BF).cuda() for i, t in enumerate((q, k)))
    dproj = torch.full((B, N, Hq + 2 * Hkv, d), 7.0, device="cuda", dtype=BF)
    dq, dk = dproj[:, :, :Hq].transpose(1, 2), dproj[:, :, Hq : Hq + Hkv].transpose(1, 2)
    fa.qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, pos, freq, dq=dq, dk=dk)
    a, b, _, _ = fa.qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, pos, freq)
    clean()
    assert torch.equal(dq, a) and torch.equal(dk, b) and (dproj[:, :, Hq + Hkv :] == 7).all()
    with pytest.raises(fa.FAError):  # rows that share memory
        fa.qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, pos, freq, dq=dproj[:1, :, :Hq].transpose(1, 2).expand(B, -1, -1, -1))


def test_gradients_by_differences():
    """Central differences of the forward call itself, in fp32."""
    q, k, _, (wq, wk), pos, freq = rope_inputs(1, 2, 1, 3, 64, 64, (32,), F32, True, 12)
    dqo, dko = randn(q.shape, 320, F32).cuda(), randn(k.shape, 321, F32).cuda()
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, pos, freq)

    def f(x, kk, w):
        a, b = fa.qk_norm_rope(x, kk, w, wk, pos, freq)
        return ((a * dqo).double().sum() + (b * dko).double().sum()).item()

    h = 2.0**-7  # truncation h^2 f'''/6 ~ 1e-5 |dy||w|r, rounding 2^-22 sqrt(384) 2 / (2 h) ~ 6e-4
    for at in [(0, 0, 0, 0), (0, 1, 2, 63), (0, 0, 1, 31)]:
        e = torch.zeros_like(q)
        e[at] = h
        assert abs((f(q + e, k, wq) - f(q - e, k, wq)) / (2 * h) - dq[at].item()) < 2e-3
    for j in (0, 40):
        e = torch.zeros_like(wq)
        e[j] = h
        assert abs((f(q, k, wq + e) - f(q, k, wq - e)) / (2 * h) - dwq[j].item()) < 2e-3


# ----------------------------------------------------------------------------------------------- append
def pool(R, Hkv, d, maxb, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    blocks = R * maxb + extra + 3
    ids = torch.randperm(blocks, generator=g).to(torch.int32)
    kc, vc = (randn((blocks, Hkv, 16, d), seed + i, BF) for i in (1, 2))
    return ids[: R * maxb].reshape(R, maxb).contiguous(), ids[R * maxb : R * maxb + extra].contiguous(), kc, vc


@pytest.mark.parametrize(
    "Hq,Hkv,N,d,rd,sec,inter,norm,lens,past",
    [
        (12, 2, 1, 128, 128, (64,), False, True, (1, 1, 1, 0), (0, 15, 16, 40)),
        (8, 2, 37, 128, 128, (16, 24, 24), False, True, (37, 0, 1, 20), (3, 5, 63, 0)),
        (3, 3, 20, 64, 32, (16,), True, True, (20, 19, 1), (0, 0, 0)),
        (4, 1, 33, 96, 96, (24, 24), False, False, (33, 17), (90, 16)),
    ],
)
def test_append(Hq, Hkv, N, d, rd, sec, inter, norm, lens, past):
    R, maxb = len(lens), 8
    q, k, v, (wq, wk), pos, freq = rope_inputs(R, Hq, Hkv, N, d, rd, sec, BF, norm, 400 + d)
    q, k, v = q.clone(), k.clone(), v.clone()
    for r, m in enumerate(lens):  # padding rows may hold anything
        for t in (q, k, v):
            t[r, :, m:] = float("nan")
    table, _, kc, vc = pool(R, Hkv, d, maxb, 500 + d)
    ctx = torch.tensor([a + b for a, b in zip(lens, past)], dtype=torch.int32)
    for r in range(R):
        table[r, -(-int(ctx[r]) // 16) :] = -1
    ql = torch.tensor(lens, dtype=torch.int32)
    out = torch.full((R, Hq, N, d), 3.0, dtype=BF)
    kd, vd, od = kc.cuda(), vc.cuda(), out.cuda()
    got = fa.qk_norm_rope_append(q, k, v, wq, wk, pos, freq, kd, vd, table.cuda(), ctx.cuda(), ql.cuda(), sections=sec,
                                 interleaved=inter, q_out=od)
    clean()
    assert got.data_ptr() == od.data_ptr()
    Q, K, V = ops.norm_rope_append(q, k, v, wq, wk, pos.cpu(), freq, sec, inter, 1e-6, kc, vc, table, ctx, ql, out, 16)
    assert np.array_equal(ora.to_f64(vd), V)
    near(kd, K, 2.0**-20 * np.abs(K).max(-1, keepdims=True), "K")
    near(od, Q, 2.0**-20 * np.abs(Q).max(-1, keepdims=True), "q")
    for r, m in enumerate(lens):
        assert (od[r, :, m:] == 3).all()
    # every slot that no token went to is untouched
    untouched = (K == ora.to_f64(kc)).all(-1)
    assert torch.equal(kd.cpu()[torch.from_numpy(untouched)], kc[torch.from_numpy(untouched)])


def test_append_flags_bad_lengths_and_blocks():
    q, k, v, (wq, wk), pos, freq = rope_inputs(5, 4, 2, 2, 128, 128, (64,), BF, True, 21)
    table, _, kc, vc = pool(5, 2, 128, 2, 22)
    table[1, 0] = kc.shape[0]  # past the pool
    ctx = torch.tensor([2, 2, 33, 1, 2], dtype=torch.int32)  # request 2: past its table
    ql = torch.tensor([2, 2, 2, 2, 3], dtype=torch.int32)  # request 3: more rows than tokens, 4: than Nq_max
    out = torch.full((5, 4, 2, 128), 3.0, dtype=BF, device="cuda")
    kd, vd = kc.cuda(), vc.cuda()
    fa.device_status(reset=True)
    fa.qk_norm_rope_append(q, k, v, wq, wk, pos, freq, kd, vd, table.cuda(), ctx.cuda(), ql.cuda(), q_out=out)
    assert fa.device_status(reset=True) == fa.FA_ERR_INVALID_ARG
    assert (out[2:] == 3).all() and not (out[:2] == 3).any(-1).all()
    Q, K, V = ops.norm_rope_append(q[:1], k[:1], v[:1], wq, wk, pos[:, :1].cpu(), freq, (64,), False, 1e-6, kc, vc,
                                   table, ctx[:1], ql[:1], out[:1], 16)
    assert np.array_equal(ora.to_f64(vd), V)


# ------------------------------------------------------------------------------------- decode over pieces
def bounds(q, kc, vc, scale):
    """(delta, o slack) from the stored values."""
    d = q.shape[-1]
    k = kc.double().nan_to_num().abs().amax((0, 1, 2))
    delta = (d + 8) * 2.0**-24 * scale * float((q.double().abs() * k).sum(-1).max())
    return delta, (2 * delta + 2.0**-15) * float(vc.double().nan_to_num().abs().max())


def decode_case(lens, Hq, Hkv, d, maxb, seed, prefix=0):
    R = len(lens)
    pb = max(1, -(-prefix // 16)) + 1
    table, ptable, kc, vc = pool(R, Hkv, d, maxb, seed, pb)
    for c in (kc, vc):  # nothing behind a length may be read into a result
        for row, n in [(table[r], n) for r, n in enumerate(lens)] + [(ptable, prefix)]:
            for b in range(n // 16, len(row)):
                c[row[b].long(), :, max(0, n - 16 * b) :] = float("nan")
    for r, n in enumerate(lens):
        table[r, -(-n // 16) :] = -1
    ptable[-(-prefix // 16) :] = -1
    q = 2 * randn((R, Hq, d), seed + 5, BF)
    return q, kc, vc, table, ptable, torch.tensor(lens, dtype=torch.int32)


@pytest.mark.parametrize("wide", [0, 800])  # a much wider prefix table sends the prefix to the tensor cores
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize(
    "Hq,Hkv,prefix,lens",
    [
        (12, 2, 2000, (1, 15, 16, 17, 0, 200, 33)),
        (8, 8, 1, (0, 1)),
        (16, 1, 129, (5,)),
        (4, 4, 0, (3, 0, 40)),
        (32, 2, 300, (1, 2, 3)),
        (6, 2, 47, tuple(range(50))),
        (8, 1, 1040, tuple(i % 3 for i in range(70))),
        (3, 1, 5000, (600, 1)),
        (5, 1, 65, tuple(i % 20 for i in range(40))),  # 25 requests of 5 heads fill 125 of a tile's 128 rows
        (16, 16, 190, tuple(i % 2 for i in range(70))),
        (16, 1, 1, (0,) * 9),
        (8, 4, 64, (1,) * 150),
        (14, 2, 3333, (0, 5) * 30),
        (4, 1, 16, (2,) * 16),
    ],
)
def test_decode_shared(d, Hq, Hkv, prefix, lens, wide):
    q, kc, vc, table, ptable, ctx = decode_case(lens, Hq, Hkv, d, 40, 600 + d + prefix, prefix)
    ptable = torch.cat([ptable, torch.full((wide,), -1, dtype=torch.int32)])
    dev = [t.cuda() for t in (q, kc, vc, ptable, torch.tensor([prefix], dtype=torch.int32), table, ctx)]
    o, lse = fa.paged_decode_shared(*dev)
    clean()
    O, L = ops.decode_shared(q, kc, vc, ptable, prefix, table, ctx, 16, d**-0.5)
    delta, slack = bounds(q, kc, vc, d**-0.5)
    # with many rows P is rounded to bf16: sum p 2^-8 |v| at most, an attention over |v|
    V, _ = ops.decode_shared(q, kc, vc.abs(), ptable, prefix, table, ctx, 16, d**-0.5)
    near(o, O, slack + 2.0**-8 * V, "o")
    near(lse, L, delta + 2.0**-20 * np.abs(np.where(np.isinf(L), 0, L)), "lse")
    for _ in range(8):  # (a race between the roles of the prefix kernel once showed as runs that differ)
        again, _ = fa.paged_decode_shared(*dev, with_lse=False)
        assert torch.equal(o, again)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize(
    "Hq,Hkv,lens",
    [
        (12, 2, (1, 15, 16, 17, 0, 640, 333)),
        (8, 8, (1,)),
        (16, 1, (100, 0, 7)),
        (4, 4, (31, 32)),
        (3, 1, tuple(range(1, 41))),
        (8, 2, (9000,)),
    ],
)
def test_decode_scored(d, Hq, Hkv, lens):
    maxb = max(40, -(-max(lens) // 16))
    q, kc, vc, table, _, ctx = decode_case(lens, Hq, Hkv, d, maxb, 700 + d)
    w0 = randn((len(lens), Hkv, maxb * 16), 9, F32).abs()
    w = w0.cuda()
    dev = [t.cuda() for t in (q, kc, vc, table, ctx)]
    o, lse = fa.paged_decode_scored(*dev, w)
    clean()
    O, L, W = ops.decode_scored(q, kc, vc, table, ctx, w0, 16, d**-0.5)
    delta, slack = bounds(q, kc, vc, d**-0.5)
    near(o, O, slack, "o")
    near(lse, L, delta + 2.0**-20 * np.abs(np.where(np.isinf(L), 0, L)), "lse")
    added = W - ora.to_f64(w0)
    near(w, W, (2 * delta + 2.0**-19) * added, "weights")
    for r, n in enumerate(lens):
        assert torch.equal(w[r, :, n:].cpu(), w0[r, :, n:])
    w2 = w0.cuda()
    o2, lse2 = fa.paged_decode_scored(*dev, w2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(w, w2)


def minus_infinity(q, kc, rows):
    """Scores of -inf for the tokens of these (block, slots), by keys of -inf where q is positive."""
    q[..., 0] = q[..., 0].abs() + 1
    for block, slots in rows:
        kc[block, :, slots, 0] = -math.inf
    return kc.nan_to_num(0.0, 0.0, 0.0)  # for the bounds: every other key


@pytest.mark.parametrize("wide", [0, 800])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dead,prefix", [(128, 300), (64, 64), (1, 40), (299, 300)])
def test_shared_scores_of_minus_infinity(d, dead, prefix, wide):
    """Keys without weight: a tile's, a piece's and a whole prefix's, and every own one of a request."""
    lens = (40, 16, 3) + (5,) * 22
    q, kc, vc, table, ptable, ctx = decode_case(lens, 12, 4, d, 40, 640 + d + prefix, prefix)
    rows = [(ptable[b], slice(0, min(16, dead - 16 * b))) for b in range(-(-dead // 16))]
    rows += [(table[0, 0], slice(0, 16))]
    if dead < prefix:
        rows += [(table[1, 0], slice(0, 16))]
    finite = minus_infinity(q, kc, rows)
    ptable = torch.cat([ptable, torch.full((wide,), -1, dtype=torch.int32)])
    o, lse = fa.paged_decode_shared(*(t.cuda() for t in (q, kc, vc, ptable, torch.tensor([prefix], dtype=torch.int32),
                                                         table, ctx)))
    clean()
    O, L = ops.decode_shared(q, kc, vc, ptable, prefix, table, ctx, 16, d**-0.5)
    assert np.isfinite(O).all() and np.isfinite(L).all()
    delta, slack = bounds(q, finite, vc, d**-0.5)
    V, _ = ops.decode_shared(q, kc, vc.abs(), ptable, prefix, table, ctx, 16, d**-0.5)
    near(o, O, slack + 2.0**-8 * V, "o")
    near(lse, L, delta + 2.0**-20 * np.abs(L), "lse")


@pytest.mark.parametrize("d", [64, 128])
def test_scored_scores_of_minus_infinity(d):
    lens = (300, 17, 640)
    q, kc, vc, table, _, ctx = decode_case(lens, 8, 2, d, 40, 740 + d)
    rows = [(table[0, b], slice(0, 16)) for b in range(8)] + [(table[1, 0], slice(0, 16))]
    rows += [(table[2, b], slice(3, 12)) for b in range(40)]
    finite = minus_infinity(q, kc, rows)
    w0 = randn((3, 2, 640), 10, F32).abs()
    w = w0.cuda()
    o, lse = fa.paged_decode_scored(*(t.cuda() for t in (q, kc, vc, table, ctx)), w)
    clean()
    O, L, W = ops.decode_scored(q, kc, vc, table, ctx, w0, 16, d**-0.5)
    assert np.isfinite(O).all() and np.isfinite(L).all()
    delta, slack = bounds(q, finite, vc, d**-0.5)
    near(o, O, slack, "o")
    near(lse, L, delta + 2.0**-20 * np.abs(L), "lse")
    near(w, W, (2 * delta + 2.0**-19) * (W - ora.to_f64(w0)), "weights")


def test_decode_flags_bad_lengths_and_blocks():
    q, kc, vc, table, ptable, ctx = decode_case((20, 20, 20), 4, 2, 128, 4, 31, 40)
    table[1, 0] = kc.shape[0]
    ctx[2] = 65
    w0 = torch.zeros(3, 2, 64)
    w = w0.cuda()
    fa.device_status(reset=True)
    dev = [t.cuda() for t in (q, kc, vc, table, ctx)]
    o, lse = fa.paged_decode_scored(*dev, w)
    assert fa.device_status(reset=True) == fa.FA_ERR_INVALID_ARG
    assert (w[2] == 0).all()
    O, L, W = ops.decode_scored(q[:1], kc, vc, table[:1], ctx[:1], w0[:1], 16, 128**-0.5)
    _, slack = bounds(q, kc, vc, 128**-0.5)
    near(o[:1], O, slack)
    pl = torch.tensor([-1], dtype=torch.int32).cuda()
    fa.paged_decode_shared(*dev[:3], ptable.cuda(), pl, *dev[3:])
    assert fa.device_status(reset=True) == fa.FA_ERR_INVALID_ARG


# ---------------------------------------------------------------------------------------------- eviction
def evict_case(lens, Hkv, d, maxb, keep, seed, kind="random"):
    R, M = len(lens), maxb * 16
    table, _, kc, vc = pool(R, Hkv, d, maxb, seed)
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(R, Hkv, M, generator=g)
    if kind == "ties":
        w = (w * 4).floor()
    if kind == "odd":
        w[:, :, ::7] = 0.0
        w[:, :, 3::7] = -0.0
        w[:, :, 5::11] = float("nan")
        w[:, :, 4::13] = float("inf")
        w[:, :, 6::13] = -1.0
    ctx = torch.tensor(lens, dtype=torch.int32)
    sp = torch.full((R, Hkv, M), -1, dtype=torch.int32)
    for r, n in enumerate(lens):
        table[r, -(-n // 16) :] = -1
        kept = min(n, keep)
        for h in range(Hkv):
            sp[r, h, :kept] = torch.randperm(kept + 50, generator=g)[:kept].to(torch.int32)
    return kc, vc, table, ctx, ctx + 50, w, sp


@pytest.mark.parametrize(
    "lens,Hkv,d,keep,recent,kind",
    [
        ((1, 16, 17, 100, 0), 2, 128, 16, 4, "random"),
        ((300, 299, 512), 1, 64, 100, 100, "random"),
        ((512, 33), 3, 96, 1, 0, "random"),
        ((512, 511, 1), 2, 128, 500, 1, "ties"),
        ((700, 90), 2, 256, 33, 0, "ties"),
        ((640, 129), 2, 64, 77, 20, "odd"),
        ((5000,), 1, 64, 1024, 128, "random"),
        ((4096, 4097), 2, 64, 4096, 512, "ties"),
        ((2100, 1000, 2048) * 13, 2, 64, 1000, 100, "random"),  # enough CTAs to move their own rows
        ((3000, 2999), 1, 128, 1500, 0, "ties"),  # too few: a second kernel moves them
        ((50000,), 1, 64, 20000, 5000, "ties"),  # keys past shared memory
    ],
)
def test_evict(lens, Hkv, d, keep, recent, kind):
    maxb = max(45, -(-max(lens) // 16) + 1)
    case = evict_case(lens, Hkv, d, maxb, keep, 800 + d + keep, kind)
    dev = [t.cuda() for t in case]
    n, w, sp = fa.paged_evict(*dev, keep, recent)
    clean()
    kc, vc, N, W, P = ops.evict(*case, keep, recent, 16)
    assert np.array_equal(n.cpu().numpy(), N)
    assert np.array_equal(sp.cpu().numpy(), P)
    assert np.array_equal(ora.to_f64(w), W, equal_nan=True)
    assert np.array_equal(ora.to_f64(dev[0]), kc) and np.array_equal(ora.to_f64(dev[1]), vc)
    assert torch.equal(dev[5].cpu().nan_to_num(), case[5].nan_to_num()) and torch.equal(dev[6].cpu(), case[6])


def test_evict_flags_bad_lengths_and_blocks():
    case = evict_case((40, 40, 40), 2, 64, 4, 16, 41)
    case[3][1] = 65  # past its table
    case[2][2, 0] = case[0].shape[0]  # a freed slot's block past the pool
    dev = [t.cuda() for t in case]
    fa.device_status(reset=True)
    n, w, sp = fa.paged_evict(*dev, 16, 4)
    assert fa.device_status(reset=True) == fa.FA_ERR_INVALID_ARG
    assert n.tolist() == [16, 65, 16]
    assert torch.equal(w[1], dev[5][1]) and torch.equal(sp[1], dev[6][1])
    kc, vc, N, W, P = ops.evict(case[0], case[1], case[2][:1], case[3][:1], case[4][:1], case[5][:1], case[6][:1], 16, 4, 16)
    mine = case[2][:1].flatten().long()
    mine = mine[mine >= 0]
    assert np.array_equal(ora.to_f64(dev[0][mine.cuda()]), kc[mine.numpy()])
    other = torch.tensor([b for b in range(case[0].shape[0]) if b not in mine.tolist()])
    assert torch.equal(dev[0].cpu()[other], case[0][other])


def test_refusals_of_the_binding():
    q, k, v, (wq, wk), pos, freq = rope_inputs(2, 4, 2, 3, 64, 64, (32,), BF, True, 51)
    bad = [
        dict(q=q.cpu()), dict(k=k[..., :32]), dict(q_weight=None), dict(q_weight=wq.float()), dict(positions=pos.long()),
        dict(positions=pos[:, :, :2]), dict(inv_freq=freq.float()), dict(sections=(16, 16)), dict(sections=(31,)),
        dict(q_out=torch.empty(2, 4, 3, 64, device="cuda")), dict(q=q.transpose(2, 3)),
    ]
    base = dict(q=q, k=k, q_weight=wq, k_weight=wk, positions=pos, inv_freq=freq)
    for change in bad:
        with pytest.raises(ValueError):
            fa.qk_norm_rope(**{**base, **change})
    with pytest.raises(fa.FAError):  # rows that start off a 16-byte boundary
        wide = torch.zeros(2, 3, 4, 68, device="cuda", dtype=BF)[..., 1:65].transpose(1, 2)
        fa.qk_norm_rope(**{**base, "q": wide})
    qd, kc, vc, table, ptable, ctx = (t.cuda() for t in decode_case((20, 3), 4, 2, 128, 4, 52, 40))
    w = torch.zeros(2, 2, 64, device="cuda")
    for change in (dict(weights=w[:, :1]), dict(ctx_lens=ctx.long()), dict(q=qd.float()), dict(v_cache=vc[:-1]),
                   dict(block_table=table[:1])):
        with pytest.raises(ValueError):
            fa.paged_decode_scored(**{**dict(q=qd, k_cache=kc, v_cache=vc, block_table=table, ctx_lens=ctx, weights=w), **change})
    with pytest.raises(fa.FAError):
        fa.paged_decode_scored(qd, kc, vc, table, ctx, w, workspace=torch.empty(16, device="cuda", dtype=torch.uint8))
    sp = torch.full((2, 2, 64), -1, device="cuda", dtype=torch.int32)
    for keep, recent in ((0, 0), (4, 5), (4, -1)):
        with pytest.raises(fa.FAError):
            fa.paged_evict(kc, vc, table, ctx, ctx, w, sp, keep, recent)
    with pytest.raises(fa.FAError):  # in place
        fa.paged_evict(kc, vc, table, ctx, ctx, w, sp, 4, 2, weights_out=w)
    torch.cuda.synchronize()


def test_refusals_of_numbers():
    """Sizes that are no integers, or that do not fit the C type they are passed in."""
    _, kc, vc, table, _, ctx = (t.cuda() for t in decode_case((20, 3), 4, 2, 128, 4, 53))
    w, sp = torch.zeros(2, 2, 64, device="cuda"), torch.full((2, 2, 64), -1, device="cuda", dtype=torch.int32)
    for keep, recent in ((4.5, 2), (2**32 + 4, 2), (4, 2**40)):
        with pytest.raises(ValueError):
            fa.paged_evict(kc, vc, table, ctx, ctx, w, sp, keep, recent)
    torch.cuda.synchronize()


def test_gradients_of_broadcast_inputs():
    """q, k shared by heads and batches through strides of 0: one gradient row for each, dense."""
    _, _, _, (wq, wk), pos, freq = rope_inputs(2, 4, 2, 5, 64, 64, (32,), BF, True, 54)
    q, k = randn((2, 1, 5, 64), 55, BF).cuda(), randn((1, 1, 1, 64), 56, BF).cuda()
    dq, dk = randn((2, 4, 5, 64), 57, BF).cuda(), randn((2, 2, 5, 64), 58, BF).cuda()
    args = (wq, wk, pos, freq)
    wide = [t.expand(2, h, 5, 64) for t, h in ((q, 4), (k, 2))]
    got = fa.qk_norm_rope_bwd(dq, dk, *wide, *args)
    ref = fa.qk_norm_rope_bwd(dq, dk, *(t.contiguous() for t in wide), *args)
    clean()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    for a, b in zip(fa.qk_norm_rope(*wide, *args), fa.qk_norm_rope(*(t.contiguous() for t in wide), *args)):
        assert torch.equal(a, b)


def own_and_prefix_bound(q, kc, vc, V, keys, d):
    """Slack of o where P is carried as two bf16 parts everywhere: P off by 2 delta (scores) + 2^-22 (exponential) +
    2^-16 (its second part rounded), relative; each 16 keys are added to a running sum of at most V = sum p |v| in
    two products, which a tensor core may cut off below 2^-23 of it; the join adds 2^-20."""
    delta, _ = bounds(q, kc, vc, d**-0.5)
    return (2 * delta + 2.0**-22 + 2.0**-16 + keys / 16 * 2 * 2.0**-23 + 2.0**-20) * V


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,prefix,lens", [(12, 2, 40, (1,) * 8), (32, 8, 17, (0, 3) * 20), (4, 1, 300, (2,)),
                                                (16, 2, 2000, (5,) * 70)])
def test_shared_weights_are_not_rounded_to_bf16(d, Hq, Hkv, prefix, lens):
    """The same bound on every way: 16-row pieces (a table of the prefix's width) and tensor cores (a wide one)."""
    q, kc, vc, table, ptable, ctx = decode_case(lens, Hq, Hkv, d, 8, 660 + d + prefix, prefix)
    O, L = ops.decode_shared(q, kc, vc, ptable, prefix, table, ctx, 16, d**-0.5)
    V, _ = ops.decode_shared(q, kc, vc.abs(), ptable, prefix, table, ctx, 16, d**-0.5)
    slack = own_and_prefix_bound(q, kc, vc, V, prefix + max(lens), d)
    for wide in (0, 6000):
        pt = torch.cat([ptable, torch.full((wide,), -1, dtype=torch.int32)])
        o, _ = fa.paged_decode_shared(*(t.cuda() for t in (q, kc, vc, pt, torch.tensor([prefix], dtype=torch.int32),
                                                           table, ctx)))
        clean()
        near(o, O, slack, f"o, {wide} blocks wider")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,R,prefix,tiles", [(12, 2, 90, 900, 0), (16, 4, 70, 2500, 1), (32, 8, 300, 4000, 2)])
def test_a_prefix_wait_that_ran_out_leaves_nan(d, Hq, Hkv, R, prefix, tiles):
    """Key tiles that never come: no row shows what the workspace held before, and the next call is unharmed."""
    import struct

    blocks, maxb = 4096, 2  # (a wide table, so that the prefix goes to the kernel whose waits are meant)
    g = torch.Generator().manual_seed(R)
    used = -(-prefix // 16)
    ids = torch.randperm(used + R * maxb, generator=g).int()
    pt = torch.full((blocks,), -1, dtype=torch.int32)
    pt[:used] = ids[:used]
    kc, vc = (randn((used + R * maxb, Hkv, 16, d), 670 + i, BF).cuda() for i in (0, 1))
    q, table = randn((R, Hq, d), 672, BF).cuda(), ids[used:].view(R, maxb).cuda()
    ctx = torch.randint(0, 33, (R,), generator=g).int().cuda()
    pt, pl = pt.cuda(), torch.tensor([prefix], dtype=torch.int32).cuda()
    need = fa.paged_decode_shared_workspace_size(R, Hq, Hkv, d, blocks, maxb, 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    args = (q, kc, vc, pt, pl, table, ctx)
    o, lse = fa.paged_decode_shared(*args, workspace=ws)
    clean()
    assert torch.isfinite(lse).all()
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    at = [t.data_ptr() for t in (q, kc, vc, pt, pl, table, ctx, o2, lse2, ws)]
    packed = struct.pack("11P8ifi", *at, need, R, Hq, Hkv, d, 16, blocks, maxb, kc.shape[0], d**-0.5, fa.FA_DTYPE_BF16)
    fa.device_status(reset=True)
    assert fa.lib().fa_selftest_shared_timeout(packed, tiles, torch.cuda.current_stream().cuda_stream) == fa.FA_OK
    assert fa.device_status(reset=True) == fa.FA_ERR_DEVICE_TIMEOUT
    assert torch.isnan(lse2).all() and torch.isnan(o2).all()
    o3, lse3 = fa.paged_decode_shared(*args, workspace=ws)
    clean()
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


@pytest.mark.parametrize("dead", [1, 16, 64, 700, 2048, 2100])
def test_paged_decode_scores_of_minus_infinity(dead):
    """The decode step without weights, too: keys without mass in a block, in each warp's first, in a whole split."""
    lens = (2200, 2101, 4200)
    q, kc, vc, table, _, ctx = decode_case(lens, 8, 2, 128, 270, 760 + dead)
    rows = [(table[r, b], slice(0, min(16, dead - 16 * b))) for r in range(3) for b in range(-(-dead // 16))]
    finite = minus_infinity(q, kc, rows)
    o, lse = fa.paged_decode(*(t.cuda() for t in (q, kc, vc, table, ctx)))
    clean()
    O, L = ora.paged_decode(q, kc, vc, table, ctx, 16, 128**-0.5)
    assert np.isfinite(O).all() and np.isfinite(L).all()
    delta, slack = bounds(q, finite, vc, 128**-0.5)
    V, _ = ora.paged_decode(q, kc, vc.abs(), table, ctx, 16, 128**-0.5)
    near(o, O, slack + 2.0**-8 * V, "o")  # (this call rounds P to bf16 once)
    # the log-sum goes from base 2 to e and through the splits' merge: a rounding and a function's 2^-21 each
    near(lse, L, delta + 2.0**-20 * (np.abs(L) + 1), "lse")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_fp32_rotation_rounds_no_more_than_the_plain_form(norm, inter):
    """fp32 rows against 64 bits: the mean square error is at most that of the plain form, whose angles, cosines and
    roots are right to the last bit (it rounds three products and a sum to a value, the kernel two and a sum)."""
    q, k, _, (wq, wk), pos, freq = rope_inputs(4, 6, 2, 700, 128, 128, (64,), F32, norm, 60)
    dqo, dko = (randn(t.shape, 61 + i, F32).cuda() for i, t in enumerate((q, k)))
    got = fa.qk_norm_rope(q, k, wq, wk, pos, freq, interleaved=inter)
    grads = fa.qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, pos, freq, interleaved=inter)[:2]
    clean()

    def plain(x, dy, w, dtype):
        t = (pos[0].double()[:, None, :, None] * freq)
        c, s = t.cos().to(dtype), t.sin().to(dtype)
        i = torch.arange(64, device="cuda")
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + 64)

        def turn(y, s):
            out = torch.empty_like(y)
            out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
            return out

        x, dy = x.to(dtype), dy.to(dtype)
        g = turn(dy, -s)
        if w is None:
            return turn(x, s), g
        r = 1 / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        h = g * w.to(dtype)
        return turn(x * r * w.to(dtype), s), r * (h - x * r * (h * (x * r)).mean(-1, keepdim=True))

    for j, (x, dy, w) in enumerate(((q, dqo, wq), (k, dko, wk))):
        for mine, p32, p64 in zip((got[j], grads[j]), plain(x, dy, w, F32), plain(x, dy, w, torch.float64)):
            mine, p32 = ((v.double() - p64).square().mean().sqrt().item() for v in (mine, p32))
            assert mine <= p32, (mine, p32)
