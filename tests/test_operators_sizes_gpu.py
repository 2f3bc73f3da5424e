"""The passes around attention at sizes where their loops wrap: token groups that share a CTA, rows and cache blocks
past a ring's slots, a warp's second unit, a CTA's second span, the kernels that a wider table or batch chooses.

Large calls are held against calls on slices, which must give the same bits, and sums against 64 bits; tolerances as
in test_operators_gpu.py."""
import numpy as np
import pytest
import torch

import exact_attention_128_b200 as fa
from exact_attention_128_b200.workloads import randn
from operator_cases import (evict_moves_itself, piece_blocks, rope_shape, shared_workspace, tensor_core_prefix)
from oracle import attention_fp64 as ora
from oracle import operators_fp64 as ops
from test_operators_gpu import BF, F32, bounds, clean, decode_case, evict_case, near, own_and_prefix_bound, rope_inputs

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ norm + rotation
@pytest.mark.parametrize(
    "B,Hq,Hkv,N,d,sec,inter,dtype,norm,groups,rows",
    [
        (1, 32, 8, 5100, 128, (64,), False, BF, True, 2, 10),
        (3, 8, 2, 3334, 128, (16, 24, 24), True, BF, True, 4, 5),
        (1, 2, 1, 19103, 128, (64,), False, BF, False, 8, 3),
        (2, 32, 8, 3001, 96, (24, 24), False, BF, True, 2, 10),
        (64, 12, 12, 196, 64, (16, 16), True, F32, True, 2, 6),
        (7, 4, 4, 1373, 256, (64,), False, F32, True, 8, 8),
        (2, 56, 14, 67, 64, (32,), False, F32, True, 1, 9),
        (1, 40, 8, 130, 128, (64,), True, BF, True, 1, 6),
    ],
)
def test_large_rotation_equals_its_slices(B, Hq, Hkv, N, d, sec, inter, dtype, norm, groups, rows):
    assert rope_shape(B * N, Hq + Hkv, d) == (groups, rows)
    q, k, _, (wq, wk), pos, freq = rope_inputs(B, Hq, Hkv, N, d, 2 * sum(sec), sec, dtype, norm, 900 + d)
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, pos, freq, sections=sec, interleaved=inter)
    step = max(1, 250 // B)
    for a in range(0, N, step):
        b = min(N, a + step)
        x, y = fa.qk_norm_rope(q[:, :, a:b], k[:, :, a:b], wq, wk, pos[:, :, a:b], freq, sections=sec, interleaved=inter)
        assert torch.equal(x, qo[:, :, a:b]) and torch.equal(y, ko[:, :, a:b]), a
    clean()
    for at in (0, N // 2, N - 1):  # and the definition, at a few tokens
        for x, w, got in ((q, wq, qo), (k, wk, ko)):
            s = slice(at, at + 1)
            ref = ops.norm_rope(x[:, :, s], w, pos[:, :, s].cpu(), freq, sec, inter, 1e-6)
            near(got[:, :, s], ref, 2.0**-20 * np.abs(ref).max(-1, keepdims=True))


def turned_back(dy, pos, freq, sec, inter):
    """The gradient in front of the rotation, in 64 bits, and |a| + |b| of each value's pair."""
    rd = 2 * sum(sec)
    axis = torch.repeat_interleave(torch.arange(len(sec)), torch.tensor(sec)).cuda()
    t = (pos.double()[axis] * freq[:, None, None]).permute(1, 2, 0)[:, None]
    c, s = t.cos(), t.sin()
    i = torch.arange(rd // 2, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
    y = dy.double()
    a, b = y[..., ia], y[..., ib]
    g, size = y.clone(), y.abs()
    g[..., ia], g[..., ib] = a * c + b * s, b * c - a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return g, size


@pytest.mark.parametrize(
    "B,Hq,Hkv,N,d,sec,inter,dtype,gin,gout",
    [
        (1, 12, 3, 8192, 128, (64,), False, BF, F32, BF),  # chunks of 6 and 3 heads, 3 and 4 units a warp
        (4, 16, 16, 4000, 64, (32,), False, BF, BF, F32),  # 16 heads, 2 units
        (2, 16, 4, 2048, 256, (32, 32), True, BF, BF, BF),  # 8 and 4 heads, 3 and 4 units
        (1, 24, 2, 7001, 96, (48,), False, BF, F32, F32),  # 4 and 2 heads, 4 and 6 units
        (2, 32, 8, 2550, 128, (16, 24, 24), False, F32, F32, F32),  # 8 heads, 3 units
        (1, 40, 1, 9001, 128, (64,), True, BF, F32, BF),  # 8 heads and 1, 6 and 13 units
    ],
)
@pytest.mark.parametrize("norm", [True, False])
def test_large_rotation_gradient_equals_its_slices(B, Hq, Hkv, N, d, sec, inter, dtype, gin, gout, norm):
    q, k, _, (wq, wk), pos, freq = rope_inputs(B, Hq, Hkv, N, d, 2 * sum(sec), sec, dtype, norm, 930 + d)
    dqo, dko = (randn(t.shape, 940 + i, gin).cuda() for i, t in enumerate((q, k)))
    kw = dict(sections=sec, interleaved=inter, grad_dtype=gout)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, pos, freq, **kw)
    step = max(1, 250 // B)
    for a in range(0, N, step):
        s = slice(a, min(N, a + step))
        x, y, _, _ = fa.qk_norm_rope_bwd(dqo[:, :, s].contiguous(), dko[:, :, s].contiguous(), q[:, :, s], k[:, :, s], wq,
                                         wk, pos[:, :, s], freq, **kw)
        assert torch.equal(x, dq[:, :, s]) and torch.equal(y, dk[:, :, s]), a
    clean()
    if not norm:
        return
    for x, dy, dw in ((q, dqo, dwq), (k, dko, dwk)):
        g, size = turned_back(dy, pos, freq, sec, inter)
        n = x.double() * (x.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        rows = x.shape[0] * x.shape[1] * x.shape[2]
        slack = (2.0**-24 * (rows / 64 + 80) * (g * n).abs() + 2.0**-21 * size * n.abs()).sum((0, 1, 2))
        near(dw, (g * n).sum((0, 1, 2)).cpu().numpy(), slack.cpu().numpy(), "dw")


@pytest.mark.parametrize("Hq,Hkv,d,groups", [(32, 8, 128, 2), (8, 1, 64, 4), (2, 1, 96, 8)])
def test_large_append_equals_single_requests(Hq, Hkv, d, groups):
    R, N = 5, {2: 1100, 4: 4000, 8: 6000}[groups]
    assert rope_shape(R * N, Hq + 2 * Hkv, d)[0] == groups
    q, k, v, (wq, wk), pos, freq = rope_inputs(R, Hq, Hkv, N, d, d, (d // 2,), BF, True, 950 + d)
    lens = torch.tensor([N, 1, N // 2 + 3, 0, N - 1], dtype=torch.int32)
    ctx = lens + torch.tensor([0, 700, 13, 5, 0], dtype=torch.int32)
    maxb = -(-int(ctx.max()) // 16) + 1
    table = torch.randperm(R * maxb, generator=torch.Generator().manual_seed(d)).view(R, maxb).int().cuda()
    out = []
    for one in (False, True):
        kc, vc = (torch.full((R * maxb, Hkv, 16, d), 2.0 + i, dtype=BF, device="cuda") for i in (0, 1))
        qo = torch.full((R, Hq, N, d), 5.0, dtype=BF, device="cuda")
        for s in [slice(r, r + 1) for r in range(R)] if one else [slice(0, R)]:
            fa.qk_norm_rope_append(q[s], k[s], v[s], wq, wk, pos[:, s], freq, kc, vc, table[s], ctx[s].cuda(),
                                   lens[s].cuda(), q_out=qo[s])
        out.append((qo, kc, vc))
    clean()
    assert all(torch.equal(a, b) for a, b in zip(*out))
    qo, kc, vc = out[0]
    for r, m in enumerate(lens.tolist()):
        assert (qo[r, :, m:] == 5).all()
        if m:  # the last token's rows
            at = int(ctx[r]) - 1
            b = table[r, at // 16]
            assert torch.equal(vc[b, :, at % 16], v[r, :, m - 1])
            ref = ops.norm_rope(k[r : r + 1, :, m - 1 : m], wk, pos[:, r : r + 1, m - 1 : m].cpu(), freq, (d // 2,), False, 1e-6)
            near(kc[b, :, at % 16], ref[0, :, 0], 2.0**-20 * np.abs(ref[0, :, 0]).max(-1, keepdims=True))


# ------------------------------------------------------------------------------------- decode over pieces
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,lens", [(12, (4700, 2176, 2177, 8209) + (0, 1, 16, 33) * 15), (2, (5000,) + (7,) * 63)])
def test_scored_warps_and_spans_go_round(d, Hq, lens):
    """A warp's blocks past the 32 that it looks up at a time; a CTA's second span of weights."""
    R, Hkv, maxb = len(lens), 2, 1920
    assert piece_blocks(R * Hkv, maxb) // 4 > 32 and max(lens) > 1024 * (148 * 4 // (R * Hkv))
    need = [-(-n // 16) for n in lens]
    g = torch.Generator().manual_seed(d)
    ids = torch.randperm(sum(need) + 5, generator=g).int()
    table, at = torch.full((R, maxb), -1, dtype=torch.int32), 0
    for r, b in enumerate(need):
        table[r, :b], at = ids[at : at + b], at + b
    kc, vc = (randn((len(ids), Hkv, 16, d), 960 + i, BF) for i in (0, 1))
    for c in (kc, vc):
        for r, n in enumerate(lens):
            if n % 16:
                c[table[r, n // 16].long(), :, n % 16 :] = float("nan")
    q, ctx = 2 * randn((R, Hq, d), 962, BF), torch.tensor(lens, dtype=torch.int32)
    w0 = randn((R, Hkv, maxb * 16), 963, F32).abs()
    w = w0.cuda()
    o, lse = fa.paged_decode_scored(*(t.cuda() for t in (q, kc, vc, table, ctx)), w)
    clean()
    O, L, W = ops.decode_scored(q, kc, vc, table, ctx, w0, 16, d**-0.5)
    delta, slack = bounds(q, kc, vc, d**-0.5)
    near(o, O, slack, "o")
    near(lse, L, delta + 2.0**-20 * np.abs(np.where(np.isinf(L), 0, L)), "lse")
    near(w, W, (2 * delta + 2.0**-19) * (W - ora.to_f64(w0)), "weights")
    for r, n in enumerate(lens):
        assert torch.equal(w[r, :, n:].cpu(), w0[r, :, n:])


SHARED = [
    # Hq, Hkv, prefix, lens
    (12, 2, 2000, (1, 15, 16, 17, 0, 100, 33) * 7),
    (8, 8, 1, (0, 1) * 9),
    (16, 1, 129, (5,) * 17),
    (4, 4, 0, (3, 0, 40) * 30),
    (6, 2, 47, tuple(range(50))),
    (8, 1, 1040, tuple(i % 3 for i in range(70))),
    (3, 1, 3000, (60, 1) * 45),
    (5, 1, 65, tuple(i % 20 for i in range(60))),
    (16, 16, 190, tuple(i % 2 for i in range(70))),
    (8, 4, 64, (1,) * 150),
    (14, 2, 3333, (0, 5) * 30),
    (7, 1, 4111, (2,) * 40),
]


@pytest.mark.parametrize("tensor_cores", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,prefix,lens", SHARED)
def test_shared_on_either_way(Hq, Hkv, prefix, lens, d, tensor_cores):
    """The tables' widths choose the way; the bound is the same on both."""
    R, maxb = len(lens), 8
    used = max(1, -(-prefix // 16))
    want = [b for b in (used, used + 300, 2000, 9000) if tensor_core_prefix(R, Hq, Hkv, d, b) == tensor_cores]
    if not want:
        pytest.skip("no table of such a prefix goes this way")
    q, kc, vc, table, ptable, ctx = decode_case(lens, Hq, Hkv, d, maxb, 970 + d + prefix, prefix)
    wide = torch.full((want[0],), -1, dtype=torch.int32)
    wide[: min(want[0], len(ptable))] = ptable[: want[0]]
    size = fa.paged_decode_shared_workspace_size(R, Hq, Hkv, d, want[0], maxb, 16)
    assert size == shared_workspace(R, Hq, Hkv, d, want[0], maxb, tensor_cores)
    assert size != shared_workspace(R, Hq, Hkv, d, want[0], maxb, not tensor_cores)
    dev = [t.cuda() for t in (q, kc, vc, wide, torch.tensor([prefix], dtype=torch.int32), table, ctx)]
    o, lse = fa.paged_decode_shared(*dev)
    clean()
    O, L = ops.decode_shared(q, kc, vc, ptable, prefix, table, ctx, 16, d**-0.5)
    V, _ = ops.decode_shared(q, kc, vc.abs(), ptable, prefix, table, ctx, 16, d**-0.5)
    delta, _ = bounds(q, kc, vc, d**-0.5)
    near(o, O, own_and_prefix_bound(q, kc, vc, V, prefix + max(lens), d), "o")
    near(lse, L, delta + 2.0**-20 * np.abs(np.where(np.isinf(L), 0, L)), "lse")
    for _ in range(8):
        again, _ = fa.paged_decode_shared(*dev, with_lse=False)
        assert torch.equal(o, again)


@pytest.mark.parametrize("d,rows", [(128, 90), (64, 256)])
def test_tensor_core_prefix_past_32_bit_offsets(d, rows):
    """The prefix kernel on the last blocks of a pool of more than 2^31 values: the bits of a small pool."""
    Hkv, maxb, P = 8, 2, 330
    blocks = {128: 64, 64: 64}[d]
    assert tensor_core_prefix(rows, Hkv, Hkv, d, blocks)
    big, small = 2**31 // (Hkv * 16 * d) + 200, blocks + 4 * maxb
    ids = torch.randperm(small, generator=torch.Generator().manual_seed(d)).int()
    pre = ids[:blocks].clone()
    pre[-(-P // 16) :] = -1
    table = ids[blocks:].view(4, maxb).repeat(rows // 4 + 1, 1)[:rows].contiguous()
    far = big - small
    q = randn((rows, Hkv, d), 980, BF).cuda()
    ks, vs = (randn((small, Hkv, 16, d), 981 + i, BF).cuda() for i in (0, 1))
    kb, vb = (torch.empty((big, Hkv, 16, d), device="cuda", dtype=BF) for _ in range(2))
    kb[far:], vb[far:] = ks, vs
    ctx = (torch.arange(rows, dtype=torch.int32) % 33).cuda()
    pl = torch.tensor([P], dtype=torch.int32).cuda()
    a = fa.paged_decode_shared(q, ks, vs, pre.cuda(), pl, table.cuda(), ctx)
    b = fa.paged_decode_shared(q, kb, vb, torch.where(pre >= 0, pre + far, pre).cuda(), pl, (table + far).cuda(), ctx)
    clean()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[1]).all()


# ---------------------------------------------------------------------------------------------- eviction
@pytest.mark.parametrize("lens,Hkv,d,maxb,keep,recent,itself", [
    ((1024, 1023, 600, 513), 2, 64, 64, 512, 100, True),  # up to 512 rows move
    ((1040, 1026, 514), 2, 128, 65, 513, 0, False),  # up to 513
    ((2560, 2300, 2049), 1, 96, 160, 2048, 64, True),
    ((2561, 2300, 2049), 3, 64, 161, 2048, 2048, False),
    ((700, 40) * 20, 2, 64, 400, 300, 30, True),  # a table much wider than the contexts
    ((2176, 2049) * 10, 2, 128, 512, 2048, 512, False),  # a steady budget in such a table
])
def test_evict_with_either_mover(lens, Hkv, d, maxb, keep, recent, itself):
    assert evict_moves_itself(maxb, keep) == itself
    case = evict_case(lens, Hkv, d, maxb, keep, 990 + d + keep, "ties")
    dev = [t.cuda() for t in case]
    n, w, sp = fa.paged_evict(*dev, keep, recent)
    clean()
    kc, vc, N, W, P = ops.evict(*case, keep, recent, 16)
    assert np.array_equal(n.cpu().numpy(), N) and np.array_equal(sp.cpu().numpy(), P)
    assert np.array_equal(ora.to_f64(w), W)
    assert np.array_equal(ora.to_f64(dev[0]), kc) and np.array_equal(ora.to_f64(dev[1]), vc)
