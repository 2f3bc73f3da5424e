"""The passes around attention as they are used together: a training step's rotation, attention and gradients; a
serving loop that appends, decodes with weights and evicts; the same step captured and replayed; a shared prefix."""
import numpy as np
import pytest
import torch

import exact_attention_128_b200 as fa
from exact_attention_128_b200.workloads import randn
from oracle import attention_fp64 as ora
from oracle import operators_fp64 as ops
from parity import check_bf16_stored

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def weights(d, seed):
    return [(1 + 0.2 * randn((d,), seed + i, torch.float32)).to(BF).cuda() for i in (0, 1)]


def test_training_step():
    B, Hq, Hkv, N, d = 2, 4, 2, 130, 64
    proj = randn((B, N, Hq + 2 * Hkv, d), 1, BF).cuda()
    q, k, v = (t.transpose(1, 2) for t in proj.split([Hq, Hkv, Hkv], 2))
    wq, wk = weights(d, 2)
    pos, freq = torch.arange(N, device="cuda", dtype=torch.int32), fa.rope_frequencies(d)
    do = randn((B, Hq, N, d), 4, BF).cuda()
    q2, k2 = fa.qk_norm_rope(q, k, wq, wk, pos, freq)
    vc = v.contiguous()
    o, lse = fa.fwd(q2, k2, vc, causal=True)
    dq2, dk2, dv = fa.bwd(q2, k2, vc, o, lse, do, causal=True)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(dq2, dk2, q, k, wq, wk, pos, freq)
    torch.cuda.synchronize()
    P = np.broadcast_to(pos.cpu().numpy(), (1, B, N))
    O, _ = ora.attention_fwd(q2, k2, vc, d**-0.5, True)
    check_bf16_stored(o, O, "o")
    rq, rk, _ = ora.attention_bwd(q2, k2, vc, do, d**-0.5, True)
    for got, ref, x, w, dw in ((dq, rq, q, wq, dwq), (dk, rk, k, wk, dwk)):
        dx, rw = ops.norm_rope_bwd(ref, x, w, P, freq, (32,), False, 1e-6)
        check_bf16_stored(got, dx, "gradient")
        assert np.linalg.norm(dw.cpu().numpy() - rw) <= 5e-3 * np.linalg.norm(rw)


class Server:
    """One layer's state: caches, lengths, weights, positions."""

    def __init__(self, R=3, Hq=6, Hkv=2, d=128, maxb=5):
        self.R, self.Hq, self.Hkv, self.d, self.maxb = R, Hq, Hkv, d, maxb
        dev = dict(device="cuda")
        self.table = torch.randperm(R * maxb, generator=torch.Generator().manual_seed(3)).view(R, maxb).int().cuda()
        self.kc, self.vc = (torch.full((R * maxb, Hkv, 16, d), float("nan"), dtype=BF, **dev) for _ in range(2))
        self.w = torch.zeros(R, Hkv, maxb * 16, **dev)
        self.sp = torch.full((R, Hkv, maxb * 16), -1, dtype=torch.int32, **dev)
        self.ctx = torch.zeros(R, dtype=torch.int32, **dev)
        self.seq = torch.zeros(R, dtype=torch.int32, **dev)
        self.wq, self.wk = weights(d, 20)
        self.freq = fa.rope_frequencies(d)

    def token(self, proj, lens):
        """proj [R,N,heads,d]; lens [R]: append, and rotate q."""
        q, k, v = (t.transpose(1, 2) for t in proj.split([self.Hq, self.Hkv, self.Hkv], 2))
        N = proj.shape[1]
        pos = (self.seq[:, None] + torch.arange(N, device="cuda", dtype=torch.int32)).int()
        self.ctx += lens
        self.seq += lens
        return fa.qk_norm_rope_append(q, k, v, self.wq, self.wk, pos, self.freq, self.kc, self.vc, self.table, self.ctx,
                                      lens)

    def step(self, proj, lens):
        q = self.token(proj, lens)
        return fa.paged_decode_scored(q[:, :, 0], self.kc, self.vc, self.table, self.ctx, self.w)

    def evict(self, keep, recent):
        self.ctx, self.w, self.sp = fa.paged_evict(self.kc, self.vc, self.table, self.ctx, self.seq, self.w, self.sp,
                                                   keep, recent)


def test_serving_loop_with_eviction():
    """Prompts, then steps with an eviction every 8: each step's output is attention over exactly the tokens kept."""
    s = Server()
    R, Hkv, d, keep, recent = s.R, s.Hkv, s.d, 32, 12
    lens = torch.tensor([40, 7, 25], device="cuda", dtype=torch.int32)
    prompt = randn((R, 40, 10, d), 30, BF).cuda()
    q = s.token(prompt, lens)
    o, _ = fa.paged_prefill(q, s.kc, s.vc, s.table, s.ctx, lens, causal=True)
    torch.cuda.synchronize()
    # every token's key and value by its sequence position
    keys = [[{} for _ in range(Hkv)] for _ in range(R)]

    def note(r, h, p, slot):
        b, i = int(s.table[r, slot // 16]), slot % 16
        keys[r][h][p] = (s.kc[b, h, i].clone(), s.vc[b, h, i].clone())

    for r in range(R):
        for h in range(Hkv):
            for p in range(int(lens[r])):
                note(r, h, p, p)
    one = torch.ones(R, device="cuda", dtype=torch.int32)
    for t in range(20):
        s.step(randn((R, 1, 10, d), 40 + t, BF).cuda(), one)
        for r in range(R):
            for h in range(Hkv):
                note(r, h, int(s.seq[r]) - 1, int(s.ctx[r]) - 1)
        if t % 8 == 7:
            s.evict(keep, recent)
            n = s.ctx.tolist()
            assert n == [min(a, keep) for a in (s.seq - (s.seq - torch.tensor(n, device="cuda"))).tolist()]
            for r in range(R):
                for h in range(Hkv):
                    kept = s.sp[r, h, : n[r]].tolist()
                    if int(s.seq[r]) > n[r]:
                        assert set(range(int(s.seq[r]) - recent, int(s.seq[r]))) <= set(kept)
                    if min(kept) >= 0:
                        for slot, p in enumerate(kept):
                            b, i = int(s.table[r, slot // 16]), slot % 16
                            assert torch.equal(s.kc[b, h, i], keys[r][h][p][0])
                            assert torch.equal(s.vc[b, h, i], keys[r][h][p][1])
                    assert (s.w[r, h, n[r] :] == 0).all()
    # the heads' weights of one more step sum to the group size, over live slots only
    w0 = s.w.clone()
    o, lse = s.step(randn((R, 1, 10, d), 99, BF).cuda(), one)
    got = (s.w - w0).sum(-1).cpu()
    assert torch.allclose(got, torch.full_like(got, 3.0), atol=1e-3)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert fa.device_status() == 0


def test_step_replays_in_graphs():
    """Append + scored decode + eviction captured in two graphs that share a memory pool, replayed in turn."""
    a, b = Server(), Server()
    R, d = a.R, a.d
    proj = torch.empty(R, 1, 10, d, device="cuda", dtype=BF)
    one = torch.ones(R, device="cuda", dtype=torch.int32)

    def fill(s):
        s.token(randn((R, 30, 10, d), 60, BF).cuda(), torch.tensor([30, 18, 24], device="cuda", dtype=torch.int32))

    fill(a)
    fill(b)
    dev = dict(device="cuda")
    w2, sp2, n2 = torch.empty_like(a.w), torch.empty_like(a.sp), torch.empty_like(a.ctx)
    out = [torch.empty(R, a.Hq, d, dtype=BF, **dev) for _ in range(2)]

    def body(s, o):
        q, k, v = (t.transpose(1, 2) for t in proj.split([s.Hq, s.Hkv, s.Hkv], 2))
        s.ctx += one
        s.seq += one
        q2 = fa.qk_norm_rope_append(q, k, v, s.wq, s.wk, (s.seq - 1)[:, None], s.freq, s.kc, s.vc, s.table, s.ctx, one)
        fa.paged_decode_scored(q2[:, :, 0], s.kc, s.vc, s.table, s.ctx, s.w, out=o)
        fa.paged_evict(s.kc, s.vc, s.table, s.ctx, s.seq, s.w, s.sp, 22, 6, weights_out=w2, slot_pos_out=sp2, new_ctx=n2)
        s.w.copy_(w2)
        s.sp.copy_(sp2)
        s.ctx.copy_(n2)

    proj.copy_(randn((R, 1, 10, d), 70, BF))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm-up on another stream than the current one
        scratch = Server()
        fill(scratch)
        body(scratch, out[0])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        body(a, out[0])
    with torch.cuda.graph(graphs[1], pool=graphs[0].pool()):
        body(a, out[1])
    for t in range(6):
        proj.copy_(randn((R, 1, 10, d), 71 + t, BF))
        graphs[t % 2].replay()
        got = out[t % 2].clone()
        ref = torch.empty_like(got)
        body(b, ref)
        torch.cuda.synchronize()
        assert torch.equal(got, ref), t
        for x, y in ((a.kc, b.kc), (a.vc, b.vc)):
            assert torch.equal(x.nan_to_num(), y.nan_to_num())
        assert torch.equal(a.w, b.w) and torch.equal(a.sp, b.sp) and torch.equal(a.ctx, b.ctx)
    assert fa.device_status() == 0


def test_shared_prefix_step_equals_the_copied_prefix():
    """Requests behind one prompt: the shared call equals a decode whose table repeats the prompt's blocks."""
    R, Hq, Hkv, d, P = 9, 12, 2, 128, 208
    g = torch.Generator().manual_seed(4)
    ids = torch.randperm(200, generator=g).int()
    pre, table = ids[: P // 16], ids[20 : 20 + R * 4].view(R, 4).contiguous()
    kc, vc = (randn((200, Hkv, 16, d), 5 + i, BF).cuda() for i in (0, 1))
    wq, wk = weights(d, 7)
    ctx = torch.randint(0, 60, (R,), generator=g).int().cuda()
    proj = randn((R, 1, Hq + 2 * Hkv, d), 8, BF).cuda()
    q, k, v = (t.transpose(1, 2) for t in proj.split([Hq, Hkv, Hkv], 2))
    ctx += 1
    q = fa.qk_norm_rope_append(q, k, v, wq, wk, (P + ctx - 1)[:, None], fa.rope_frequencies(d), kc, vc, table.cuda(),
                               ctx, torch.ones_like(ctx))[:, :, 0]
    o, lse = fa.paged_decode_shared(q, kc, vc, pre.cuda(), torch.tensor([P], device="cuda", dtype=torch.int32),
                                    table.cuda(), ctx)
    joined = torch.cat([pre[None].expand(R, -1), table], 1).contiguous().cuda()
    o2, lse2 = fa.paged_decode(q, kc, vc, joined, ctx + P)
    torch.cuda.synchronize()
    assert (o.float() - o2.float()).abs().max() <= 2e-2 and (lse - lse2).abs().max() <= 1e-4
    assert fa.device_status() == 0


def shared_case(R=70, P=700, seed=90):
    Hq, Hkv, d = 8, 2, 128
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(60 + R * 3, generator=g).int()
    kc, vc = (randn((60 + R * 3, Hkv, 16, d), seed + i, BF).cuda() for i in (0, 1))
    q = randn((R, Hq, d), seed + 2, BF).cuda()
    ctx = torch.randint(0, 49, (R,), generator=g).int().cuda()
    return q, kc, vc, ids[:50].cuda(), torch.tensor([P]).int().cuda(), ids[60:].view(R, 3).contiguous().cuda(), ctx


def test_shared_prefix_step_replays_with_other_lengths():
    """Captured once (prefix on the tensor cores, the requests' own part beside it), replayed as lengths grow."""
    case = shared_case()
    q, kc, vc, pt, pl, table, ctx = case
    o = torch.empty_like(q)
    fa.paged_decode_shared(*case, out=o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse = fa.paged_decode_shared(*case, out=o)
    for t, P in enumerate((0, 1, 63, 64, 65, 640, 800)):
        pl.fill_(P)
        ctx.copy_((ctx + 7 * t) % 49)
        q.copy_(randn(q.shape, 95 + t, BF))
        graph.replay()
        got, got_lse = o.clone(), lse.clone()
        ref, ref_lse = fa.paged_decode_shared(*case)
        torch.cuda.synchronize()
        assert torch.equal(got, ref) and torch.equal(got_lse, ref_lse), P
    assert fa.device_status() == 0


def test_calls_on_several_streams_at_once():
    """The same calls, each with its own workspace, on four streams without any order between them."""
    cases = [shared_case(R, P, 200 + R) for R, P in ((70, 700), (3, 333), (128, 64), (1, 800))]
    ref = [fa.paged_decode_shared(*c) for c in cases]
    weights = [torch.zeros(c[0].shape[0], 2, 48, device="cuda") for c in cases]
    for c, w in zip(cases, weights):
        fa.paged_decode_scored(c[0], c[1], c[2], c[5], c[6], w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    mine = [torch.zeros_like(w) for w in weights]
    torch.cuda.synchronize()
    for i in range(10):
        for k, (s, c) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                got[k].append(fa.paged_decode_shared(*c))
                if i == 5:
                    fa.paged_decode_scored(c[0], c[1], c[2], c[5], c[6], mine[k])
    torch.cuda.synchronize()
    for k in range(len(cases)):
        for o, lse in got[k]:
            assert torch.equal(o, ref[k][0]) and torch.equal(lse, ref[k][1])
        assert torch.equal(mine[k], weights[k])
    assert fa.device_status() == 0


def test_blocks_past_32_bit_offsets():
    """A pool of more than 2^31 values: the same calls on its last blocks and on a small pool give the same bits."""
    Hkv, d, maxb, R, keep = 8, 128, 12, 3, 60
    big = 2**31 // (Hkv * 16 * d) + 200
    small = R * maxb + 4
    ids = torch.randperm(small, generator=torch.Generator().manual_seed(1)).int()
    table, pre = ids[: R * maxb].view(R, maxb).contiguous().cuda(), ids[R * maxb :].cuda()
    far = big - small
    ks, vs = (randn((small, Hkv, 16, d), 2 + i, BF).cuda() for i in (0, 1))
    kb, vb = (torch.empty((big, Hkv, 16, d), device="cuda", dtype=BF) for _ in range(2))
    kb[far:], vb[far:] = ks, vs
    ctx, seq = (torch.tensor(x, device="cuda", dtype=torch.int32) for x in ((190, 100, 61), (200, 100, 61)))
    wq, wk = weights(d, 5)
    proj = randn((R, 4, 3 * Hkv, d), 6, BF).cuda()
    q, k, v = (t.transpose(1, 2) for t in proj.split([Hkv, Hkv, Hkv], 2))
    pos, freq = torch.arange(4, device="cuda", dtype=torch.int32), fa.rope_frequencies(d)
    lens = torch.tensor([4, 0, 2], device="cuda", dtype=torch.int32)
    out = []
    for kc, vc, add in ((ks, vs, 0), (kb, vb, far)):
        tb, pt = table + add, pre + add
        q2 = torch.zeros(R, Hkv, 4, d, device="cuda", dtype=BF)
        fa.qk_norm_rope_append(q, k, v, wq, wk, pos, freq, kc, vc, tb, ctx, lens, q_out=q2)
        w = torch.rand(R, Hkv, maxb * 16, generator=torch.Generator().manual_seed(3)).cuda()
        qd = q2[:, :, 0].contiguous()
        o, lse = fa.paged_decode_scored(qd, kc, vc, tb, ctx, w)
        o2, lse2 = fa.paged_decode_shared(qd, kc, vc, pt, torch.tensor([50], device="cuda", dtype=torch.int32), tb, ctx)
        many = qd.repeat(30, 1, 1)  # enough rows for the tensor-core prefix
        o3, _ = fa.paged_decode_shared(many, kc, vc, pt, torch.tensor([50], device="cuda", dtype=torch.int32),
                                       tb.repeat(30, 1), ctx.repeat(30))
        n, w2, sp = fa.paged_evict(kc, vc, tb, ctx, seq, w, torch.full_like(w, -1, dtype=torch.int32), keep, 10)
        out.append((q2, o, lse, o2, lse2, o3, w, n, w2, sp, kc[add : add + small].clone(), vc[add : add + small].clone()))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert fa.device_status() == 0


def test_workspace_given_and_reused():
    """One workspace for many calls in a row, of the size that is asked for and larger."""
    case = shared_case(40, 300)
    q, kc, vc, pt, pl, table, ctx = case
    R, Hq, d = q.shape
    need = fa.paged_decode_shared_workspace_size(R, Hq, 2, d, pt.shape[0], table.shape[1], 16)
    ref = fa.paged_decode_shared(*case)
    for size in (need, need + 4096):
        ws = torch.full((size,), 255, device="cuda", dtype=torch.uint8)  # NaN everywhere
        for _ in range(3):
            o, lse = fa.paged_decode_shared(*case, workspace=ws)
            assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    with pytest.raises(fa.FAError):
        fa.paged_decode_shared(*case, workspace=torch.empty(need - 1, device="cuda", dtype=torch.uint8))
    assert fa.device_status() == 0


def test_threads_call_at_once():
    """Calls from several threads, each on its own stream, sizes of shared memory growing and shrinking between them."""
    import threading

    cases = [shared_case(R, P) for R, P in ((6, 200), (70, 800), (3, 40))]
    ref = [fa.paged_decode_shared(*c) for c in cases]
    sp = [torch.full((c[0].shape[0], 2, c[5].shape[1] * 16), -1, dtype=torch.int32, device="cuda") for c in cases]
    caches = [(c[1].clone(), c[2].clone()) for c in cases]
    w = [torch.rand(s.shape, generator=torch.Generator().manual_seed(i)).cuda() for i, s in enumerate(sp)]
    kept = [fa.paged_evict(*(x.clone() for x in caches[i]), c[5], c[6], c[6], w[i], sp[i], 16 + i, 4)
            for i, c in enumerate(cases)]
    torch.cuda.synchronize()
    got, failed = [[] for _ in cases], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(40):
                    o = fa.paged_decode_shared(*cases[i])
                    e = fa.paged_evict(*(x.clone() for x in caches[i]), *(cases[i][j] for j in (5, 6, 6)), w[i], sp[i],
                                       16 + i, 4)
                got[i] = [*o, *e]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # (a thread's exception does not reach the test)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for i in range(len(cases)):
        assert all(torch.equal(a, b) for a, b in zip(got[i], (*ref[i], *kept[i])))
    assert fa.device_status() == 0


@pytest.mark.parametrize("keep,recent", [(32, 12), (17, 0), (48, 48)])
def test_evictions_in_a_loop_keep_whole_tokens(keep, recent):
    """After each eviction: the lengths are min(before, keep), every live slot names its token, once, and holds that
    token's key, value and weight, whatever was evicted before."""
    s = Server(maxb=6)
    R, Hkv, d = s.R, s.Hkv, s.d
    lens = torch.tensor([50, 7, 31], device="cuda", dtype=torch.int32)
    s.token(randn((R, 50, 10, d), 130, BF).cuda(), lens)
    one = torch.ones(R, device="cuda", dtype=torch.int32)

    def rows():
        """{position: (key, value, weight)} of every (request, head)."""
        kc, vc, w, sp, table = (t.cpu() for t in (s.kc, s.vc, s.w, s.sp, s.table))
        out = {}
        for r, (n, seq) in enumerate(zip(s.ctx.tolist(), s.seq.tolist())):
            for h in range(Hkv):
                out[r, h] = {}
                for slot in range(n):
                    p = int(sp[r, h, slot]) if sp[r, h, slot] >= 0 else seq - n + slot
                    b, i = table[r, slot // 16], slot % 16
                    out[r, h][p] = (kc[b, h, i], vc[b, h, i], w[r, h, slot])
                assert len(out[r, h]) == n
        return out

    for t in range(24):
        s.step(randn((R, 1, 10, d), 140 + t, BF).cuda(), one)
        if t % 8 != 7:
            continue
        before, was = rows(), s.ctx.tolist()
        s.evict(keep, recent)
        assert s.ctx.tolist() == [min(n, keep) for n in was]
        after = rows()
        for (r, h), now in after.items():
            n, seq = int(s.ctx[r]), int(s.seq[r])
            assert (s.sp[r, h, :n] >= 0).all() and (s.sp[r, h, n:] == -1).all() and (s.w[r, h, n:] == 0).all()
            for p, (k, v, w) in now.items():
                assert torch.equal(k, before[r, h][p][0]) and torch.equal(v, before[r, h][p][1]) and w == before[r, h][p][2]
            newest = {p for p in before[r, h] if p >= seq - recent}
            assert newest <= set(now)
            dropped = [float(x[2]) for p, x in before[r, h].items() if p not in now]
            heavy = [float(x[2]) for p, x in now.items() if p < seq - recent]
            assert not dropped or not heavy or max(dropped) <= min(heavy)
    assert fa.device_status() == 0
