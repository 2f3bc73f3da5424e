"""The operators around attention that are measured: what each case is, its inputs, its plain form and its exact values.

Five calls: the per-head norm with the position rotation (forward, backward, and the serving form that fills a paged
cache), the decode step of a batch with a shared prefix, the decode step that accumulates attention weights, and the
eviction by those weights.  ``run`` takes the plain torch form, or the library's call where ``own`` is true.
"""
import math

import torch

own = False

BS = 16  # tokens of a cache block
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of 64 requests: the decode configuration's heads, all latency
        dict(name="append_decode_r64", op="append", R=64, N=1, lo=1, hi=1, past=4096, Hq=12, Hkv=2, d=128, rd=128,
             axes=1, inter=False, norm=True),
        # ragged prompt chunks behind 1000 cached tokens, image/video positions (time, height, width)
        dict(name="append_chunks_video", op="append", R=8, N=2047, lo=300, hi=2047, past=1000, Hq=32, Hkv=8, d=128,
             rd=128, axes=3, inter=False, norm=True),
        # the long causal prefill's q and k, straight from a fused projection
        dict(name="rope_prefill_n8192", op="rope", B=4, N=8192, Hq=32, Hkv=8, d=128, rd=128, axes=1, inter=False,
             norm=True, dtype="bf16"),
        # a batch of image layers in fp32: 196 patches, row and column positions, adjacent pairs
        dict(name="rope_vit_f32", op="rope", B=64, N=196, Hq=12, Hkv=12, d=64, rd=64, axes=2, inter=True, norm=True,
             dtype="f32"),
        # the training step's q and k: fp32 gradients from attention, bf16 ones for the projection
        dict(name="rope_bwd_train_n4096", op="rope_bwd", B=8, N=4096, Hq=16, Hkv=16, d=64, rd=64, axes=1, inter=False,
             norm=True, dtype="bf16", grad="f32"),
        # grouped heads, an odd length, half of the head rotated
        dict(name="rope_bwd_gqa_odd", op="rope_bwd", B=3, N=1021, Hq=16, Hkv=4, d=256, rd=128, axes=1, inter=False,
             norm=True, dtype="bf16", grad="bf16"),
        # a few samples from one prompt
        dict(name="shared_r8_p2000", op="shared", R=8, Hq=12, Hkv=2, d=128, P=2000, lo=1, hi=200),
        # a full batch behind a long system prompt
        dict(name="shared_r256_p16384", op="shared", R=256, Hq=32, Hkv=8, d=128, P=16384, lo=16, hi=512),
        # the decode configuration: 64 requests of 512 to 8192 tokens
        dict(name="scored_r64", op="scored", R=64, Hq=12, Hkv=2, d=128, lo=512, hi=8192),
        # two long documents
        dict(name="scored_r2_long", op="scored", R=2, Hq=32, Hkv=8, d=128, lo=40001, hi=65536),
        # a budget of 2048 tokens kept every 128 steps
        dict(name="evict_steady", op="evict", R=64, Hkv=2, d=128, lo=2049, hi=2176, keep=2048, recent=512),
        # long prompts cut down to the budget
        dict(name="evict_prompt", op="evict", R=32, Hkv=8, d=128, lo=4097, hi=8192, keep=2048, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rope", "rope_bwd", "shared", "scored", "evict"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8])
    Hq = Hkv * G
    if op in ("append", "rope", "rope_bwd"):
        d = rng.choice([64, 96, 128] if op == "append" else [64, 96, 128, 256])
        c = dict(op=op, Hq=Hq, Hkv=Hkv, d=d, rd=rng.choice([d, d, d // 2 // 16 * 16]), axes=rng.choice([1, 1, 2, 3]),
                 inter=rng.random() < 0.4, norm=rng.random() < 0.8)
        if op == "append":
            N = rng.choice([1, _log(rng, 2, 2048)])
            R = _log(rng, 1, max(1, min(128, 16384 // N)))
            c.update(R=R, N=N, lo=min(N, rng.choice([0, 1, (N + 1) // 2])), hi=N, past=_log(rng, 1, 4096))
        else:
            c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
            if op == "rope_bwd":
                c["grad"] = "f32" if c["dtype"] == "f32" else rng.choice(["f32", "bf16"])
            tokens = _log(rng, 1, min(32768, 64000000 // ((Hq + Hkv) * d)))
            c["B"] = min(tokens, _log(rng, 1, 64))
            c["N"] = tokens // c["B"]
        return c
    d = rng.choice([64, 128])
    if op == "shared":
        R = _log(rng, 1, 256)
        return dict(op=op, R=R, Hq=min(Hq, 32) // Hkv * Hkv, Hkv=Hkv, d=d, P=_log(rng, 1, 16384), lo=rng.choice([0, 1, 16]),
                    hi=_log(rng, 16, 512))
    if op == "scored":
        R = _log(rng, 1, 64)
        hi = _log(rng, 1, min(65536, 1048576 // (R * Hkv)))
        return dict(op=op, R=R, Hq=Hq, Hkv=Hkv, d=d, lo=rng.randint(1, hi), hi=hi)
    R = _log(rng, 1, 64)
    hi = _log(rng, 2, min(16384, 2097152 // (R * Hkv)))
    keep = rng.randint(1, hi)
    return dict(op=op, R=R, Hkv=Hkv, d=d, lo=rng.randint(1, hi), hi=hi, keep=keep, recent=rng.randint(0, keep))


def _lens(c):
    """R lengths from lo to hi, evenly spread (their order comes from the seed)."""
    R, lo, hi = c["R"], c["lo"], c["hi"]
    return [hi if R == 1 else lo + (hi - lo) * i // (R - 1) for i in range(R)]


def _sections(c):
    """Frequencies of each axis: one axis has all; two halves; or 1/4, 3/8, 3/8."""
    h = c["rd"] // 2
    if c["axes"] == 1:
        return (h,)
    if c["axes"] == 2:
        return (h // 2, h - h // 2)
    return (h // 4, (h - h // 4) // 2, h - h // 4 - (h - h // 4) // 2)


# --------------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def _table(g, lens, width, blocks, first=0):
    """A [R, width] block table over `blocks` physical blocks in a random order, -1 behind each request's last."""
    R = lens.numel()
    t = _perm(g, blocks)[first : first + R * width].view(R, width).to(torch.int32)
    used = torch.arange(width, device="cuda")[None] * BS < lens[:, None]
    return torch.where(used, t, torch.full_like(t, -1)).contiguous()


def _blocks(n):
    return max(1, -(-n // BS))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op, d = case["op"], case["d"]
    if op in ("append", "rope", "rope_bwd"):
        Hq, Hkv, N, A = case["Hq"], case["Hkv"], case["N"], case["axes"]
        B = case["R"] if op == "append" else case["B"]
        dt = DT[case.get("dtype", "bf16")]
        proj = _randn(g, B, N, Hq + 2 * Hkv, d, dtype=dt)  # one fused projection's output, as its views are used
        s["q"] = proj[:, :, :Hq].transpose(1, 2)
        s["k"] = proj[:, :, Hq : Hq + Hkv].transpose(1, 2)
        s["v"] = proj[:, :, Hq + Hkv :].transpose(1, 2)
        s["wq"] = (1 + 0.2 * _randn(g, d, dtype=torch.float32)).to(dt) if case["norm"] else None
        s["wk"] = (1 + 0.2 * _randn(g, d, dtype=torch.float32)).to(dt) if case["norm"] else None
        i = torch.arange(case["rd"] // 2, device="cuda", dtype=torch.float64)
        s["freq"] = torch.pow(torch.tensor(10000.0, device="cuda", dtype=torch.float64), -2 * i / case["rd"])
        s["sections"] = _sections(case)
        start = torch.randint(0, 100000, (A, B, 1), generator=g, device="cuda")
        step = torch.arange(N, device="cuda").view(1, 1, N)
        if A > 1:  # a grid walked row by row, frame by frame
            w = max(1, int(math.isqrt(N)))
            step = torch.cat([step // (w * w), step // w % w, step % w])[3 - A :]
        s["pos"] = (start + step).to(torch.int32).contiguous()
        if op == "append":
            lens = torch.tensor(_lens(case), device="cuda")[_perm(g, B)]
            past = torch.randint(0, case["past"] + 1, (B,), generator=g, device="cuda")
            ctx = lens + past
            width = _blocks(N + case["past"])
            s["kc"] = _randn(g, B * width, Hkv, BS, d)
            s["vc"] = _randn(g, B * width, Hkv, BS, d)
            s["table"] = _table(g, ctx, width, B * width)
            s["ctx"], s["lens"] = ctx.to(torch.int32), lens.to(torch.int32)
            s["q_out"] = torch.zeros(B, Hq, N, d, device="cuda", dtype=dt)  # the attention call's padded input
        if op == "rope_bwd":
            gd = DT[case["grad"]]
            s["dqo"] = _randn(g, B, Hq, N, d, dtype=gd)
            s["dko"] = _randn(g, B, Hkv, N, d, dtype=gd)
        return s
    R, Hkv, hi = case["R"], case["Hkv"], case["hi"]
    lens = torch.tensor(_lens(case), device="cuda")[_perm(g, R)]
    width = _blocks(hi)
    pw = _blocks(case["P"]) if op == "shared" else 0
    blocks = R * width + pw
    s["kc"] = _randn(g, blocks, Hkv, BS, d)
    s["vc"] = _randn(g, blocks, Hkv, BS, d)
    s["ctx"] = lens.to(torch.int32)
    if op != "evict":
        s["q"] = 2 * _randn(g, R, case["Hq"], d)
    if op == "shared":
        at = _perm(g, blocks).to(torch.int32)
        s["ptable"] = at[:pw].contiguous()
        s["plen"] = torch.tensor([case["P"]], device="cuda", dtype=torch.int32)
        t = at[pw:].view(R, width)
        used = torch.arange(width, device="cuda")[None] * BS < lens[:, None]
        s["table"] = torch.where(used, t, torch.full_like(t, -1)).contiguous()
        return s
    s["table"] = _table(g, lens, width, blocks)
    M = width * BS
    slot = torch.arange(M, device="cuda")
    live = slot < lens[:, None, None]
    # weights summed over the steps a token has seen: a few heavy tokens, many light ones, some that no head read
    w = torch.randn(R, Hkv, M, generator=g, device="cuda").mul(1.5).exp()
    w = torch.where(torch.rand(R, Hkv, M, generator=g, device="cuda") < 0.05, torch.zeros_like(w), w)
    s["weights"] = torch.where(live, w, torch.zeros_like(w))
    if op == "evict":
        # an earlier eviction dropped 100 tokens and left the first `kept` slots in no order of age; the rest came since
        kept = torch.minimum(lens, torch.tensor(case["keep"], device="cuda"))[:, None, None]
        u = torch.rand(R, Hkv, M + 100, generator=g, device="cuda")
        u = torch.where(torch.arange(M + 100, device="cuda") < kept + 100, u, torch.full_like(u, 2.0))
        age = u.argsort(-1)[..., :M]
        s["slot_pos"] = torch.where(slot < kept, age, torch.full_like(age, -1)).to(torch.int32).contiguous()
        s["seq"] = (lens + 100).to(torch.int32)
    return s


# ----------------------------------------------------------------------------------------------------- plain forms
def _angles(s):
    """cos and sin [B, 1, N, rd/2] of each pair's angle, in 64 bits until they are rounded."""
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=s["rd"] // 2)
    p = s["pos"].double()[axis]  # [rd/2, B, N]
    t = (p * s["freq"][:, None, None]).permute(1, 2, 0)[:, None]
    return t.cos().float(), t.sin().float()


def _rotate(x, cos, sin, rd, inter):
    if inter:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., : rd // 2], x[..., rd // 2 : rd]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rd:]], -1)


def _norm_rope(x, w, s, cos, sin):
    y = x.float()
    if w is not None:
        y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float()
    return _rotate(y, cos, sin, s["rd"], s["inter"]).to(x.dtype)


def _norm_rope_bwd(dy, x, w, s, cos, sin):
    g = _rotate(dy.float(), cos, -sin, s["rd"], s["inter"])
    if w is None:
        return g.to(x.dtype), None
    r = (x.float().square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = x.float() * r
    h = g * w.float()
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * n).sum((0, 1, 2))


def _gathered(cache, table, n):
    """[R, Hkv, n, d] in 32 bits: the first n slots of each table row."""
    R, (_, Hkv, _, d) = table.shape[0], cache.shape
    x = cache[table.clamp(min=0).long()]  # [R, width, Hkv, BS, d]
    return x.permute(0, 2, 1, 3, 4).reshape(R, Hkv, -1, d)[:, :, :n].float()


def _attend(s, with_prefix):
    """Weights, output and lse of each request's heads over its own slots (and the prefix before them)."""
    R, Hq, d = s["q"].shape
    Hkv = s["kc"].shape[1]
    q = s["q"].float().view(R, Hkv, Hq // Hkv, d) / math.sqrt(d)
    M = s["table"].shape[1] * BS
    k, v = _gathered(s["kc"], s["table"], M), _gathered(s["vc"], s["table"], M)
    dead = torch.arange(M, device="cuda") >= s["ctx"][:, None, None, None]
    sc = torch.matmul(q, k.transpose(-1, -2)).masked_fill(dead, -math.inf)
    if with_prefix:
        pk, pv = (_gathered(s[c], s["ptable"][None], s["P"])[0] for c in ("kc", "vc"))  # [Hkv, P, d]
        sp = torch.matmul(q.transpose(0, 1).reshape(Hkv, -1, d), pk.transpose(-1, -2))
        sp = sp.view(Hkv, R, Hq // Hkv, -1).transpose(0, 1)
        top = torch.maximum(sc.amax(-1, keepdim=True), sp.amax(-1, keepdim=True))
    else:
        top = sc.amax(-1, keepdim=True)
    p = (sc - top).exp()
    l = p.sum(-1, keepdim=True)
    u = torch.matmul(p, v)
    if with_prefix:
        pp = (sp - top).exp()
        l = l + pp.sum(-1, keepdim=True)
        up = torch.matmul(pp.transpose(0, 1).reshape(Hkv, R * (Hq // Hkv), -1), pv)
        u = u + up.view(Hkv, R, Hq // Hkv, d).transpose(0, 1)
    o = (u / l).reshape(R, Hq, d).to(s["q"].dtype)
    return p / l, o, (top + l.log()).reshape(R, Hq)


def _evict(s):
    n = s["ctx"].long()[:, None, None]
    M, keep = s["weights"].shape[-1], s["keep"]
    slot = torch.arange(M, device="cuda").expand_as(s["weights"])
    live = slot < n
    seq = s["seq"].long()[:, None, None]
    pos = torch.where(s["slot_pos"] >= 0, s["slot_pos"].long(), seq - n + slot)
    key = torch.where(pos >= seq - s["recent"], torch.full_like(s["weights"], math.inf), s["weights"])
    key = torch.where(live, key, torch.full_like(key, -1.0))
    order = key.argsort(dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(-1, order, slot)
    kept = live & (rank < keep)
    hole, mover = live & (slot < keep) & ~kept, kept & (slot >= keep)
    moves = min(keep, M)
    dst = (~hole).int().argsort(dim=-1, stable=True)[..., :moves]
    src = (~mover).int().argsort(dim=-1, stable=True)[..., :moves]
    moved = torch.arange(moves, device="cuda") < mover.sum(-1, keepdim=True)
    stays = kept & (slot < keep)
    w = torch.where(stays, s["weights"], torch.zeros_like(s["weights"]))
    p = torch.where(stays, pos, torch.full_like(pos, -1))
    to, at = dst[moved], src[moved]
    r, h, _ = moved.nonzero(as_tuple=True)
    w[r, h, to], p[r, h, to] = s["weights"][r, h, at], pos[r, h, at]
    pd, ps = s["table"][r, to // BS].long(), s["table"][r, at // BS].long()
    s["kc"][pd, h, to % BS] = s["kc"][ps, h, at % BS]
    s["vc"][pd, h, to % BS] = s["vc"][ps, h, at % BS]
    return {"ctx": s["ctx"].clamp(max=keep), "weights": w, "slot_pos": p.int(), "k": s["kc"], "v": s["vc"]}


def run(state):
    s = state
    op = s["op"]
    if own:
        import exact_attention_128_b200 as fa

        rope = dict(sections=s.get("sections"), interleaved=s.get("inter"), eps=EPS)
        if op == "rope":
            q, k = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], **rope)
            return {"q": q, "k": k}
        if op == "rope_bwd":
            dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(s["dqo"], s["dko"], s["q"], s["k"], s["wq"], s["wk"], s["pos"],
                                                   s["freq"], **rope)
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        if op == "append":
            q = fa.qk_norm_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["pos"], s["freq"], s["kc"], s["vc"],
                                       s["table"], s["ctx"], s["lens"], q_out=s["q_out"], **rope)
            return {"q": q, "k": s["kc"], "v": s["vc"]}
        if op == "shared":
            o, lse = fa.paged_decode_shared(s["q"], s["kc"], s["vc"], s["ptable"], s["plen"], s["table"], s["ctx"])
            return {"o": o, "lse": lse}
        if op == "scored":
            o, lse = fa.paged_decode_scored(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["weights"])
            return {"o": o, "lse": lse, "weights": s["weights"]}
        n, w, p = fa.paged_evict(s["kc"], s["vc"], s["table"], s["ctx"], s["seq"], s["weights"], s["slot_pos"],
                                 s["keep"], s["recent"])
        return {"ctx": n, "weights": w, "slot_pos": p, "k": s["kc"], "v": s["vc"]}
    if op == "rope":
        cos, sin = _angles(s)
        return {"q": _norm_rope(s["q"], s["wq"], s, cos, sin), "k": _norm_rope(s["k"], s["wk"], s, cos, sin)}
    if op == "rope_bwd":
        cos, sin = _angles(s)
        dq, dwq = _norm_rope_bwd(s["dqo"], s["q"], s["wq"], s, cos, sin)
        dk, dwk = _norm_rope_bwd(s["dko"], s["k"], s["wk"], s, cos, sin)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if op == "append":
        cos, sin = _angles(s)
        q, k = _norm_rope(s["q"], s["wq"], s, cos, sin), _norm_rope(s["k"], s["wk"], s, cos, sin)
        i = torch.arange(s["N"], device="cuda")
        real = i < s["lens"][:, None]
        s["q_out"].copy_(torch.where(real[:, None, :, None], q, s["q_out"]))
        r, t = real.nonzero(as_tuple=True)
        at = (s["ctx"] - s["lens"])[r].long() + t
        block = s["table"][r, at // BS].long()
        s["kc"][block, :, at % BS] = k[r, :, t]
        s["vc"][block, :, at % BS] = s["v"][r, :, t]
        return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}
    if op == "shared":
        _, o, lse = _attend(s, True)
        return {"o": o, "lse": lse}
    if op == "scored":
        p, o, lse = _attend(s, False)
        s["weights"] += p.sum(2)
        return {"o": o, "lse": lse, "weights": s["weights"]}
    return _evict(s)


# ------------------------------------------------------------------------------------------------------------ work
def work(case):
    op, d = case["op"], case["d"]
    if op in ("append", "rope", "rope_bwd"):
        H, e = case["Hq"] + case["Hkv"], 4 if case.get("dtype") == "f32" else 2
        rows = sum(_lens(case)) if op == "append" else case["B"] * case["N"]
        values = rows * H * d
        small = 4 * case["axes"] * rows + 4 * case["rd"]
        if op == "append":
            return {"bytes": 2 * e * (values + rows * case["Hkv"] * d) + small, "flops": 10 * values}
        if op == "rope":
            return {"bytes": 2 * e * values + small, "flops": 10 * values}
        ge = 4 if case["grad"] == "f32" else 2
        return {"bytes": (ge + (2 * e if case["norm"] else e)) * values + small, "flops": 16 * values}
    R, Hkv, n = case["R"], case["Hkv"], sum(_lens(case))
    if op == "evict":
        keep, recent, moved = case["keep"], case["recent"], 0.0
        for c in _lens(case):
            tail = max(0, c - keep)
            new = min(tail, recent)
            moved += new + (tail - new) * (keep - recent) / max(1, c - recent)
        slots = Hkv * (2 * 4 * n + 2 * 4 * R * _blocks(case["hi"]) * BS)
        return {"bytes": slots + moved * Hkv * d * 2 * 2 * 2, "flops": Hkv * n}
    io = R * case["Hq"] * (4 * d + 4)
    if op == "shared":
        return {"bytes": (case["P"] + n) * Hkv * d * 4 + io, "flops": 4 * case["Hq"] * d * (R * case["P"] + n)}
    return {"bytes": n * Hkv * (d * 4 + 8) + io, "flops": 4 * case["Hq"] * d * n}


# ----------------------------------------------------------------------------------------------------------- exact
def _exact_rope(x, w, s, forward=True):
    """The norm and the rotation in 64 bits, the pairs as complex numbers turned by a unit one."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    rd = s["rd"]
    t = torch.cat([s["pos"][a][..., None].double() * f for a, f in enumerate(s["freq"].split(s["sections"]))], -1)
    turn = torch.polar(torch.ones_like(t), t)[:, None]
    if s["inter"]:
        z = torch.view_as_complex(x[..., :rd].unflatten(-1, (-1, 2)).contiguous()) * turn
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., : rd // 2], x[..., rd // 2 : rd]) * turn
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., rd:]], -1)


def _exact_attend(s, r, prefix):
    """One request: its keys in order, softmax in 64 bits. Returns weights [Hkv, G, n], o, lse."""
    n = int(s["ctx"][r])
    at = torch.arange(n, device="cuda")
    k, v = (s[c][s["table"][r].long()[at // BS], :, at % BS].double().transpose(0, 1) for c in ("kc", "vc"))
    if prefix is not None:
        k, v = torch.cat([prefix["kc"], k], 1), torch.cat([prefix["vc"], v], 1)
    Hkv, _, d = k.shape
    q = s["q"][r].double().view(Hkv, -1, d)
    sc = q @ k.mT / d**0.5
    lse = torch.logsumexp(sc, -1)
    p = torch.exp(sc - lse[..., None])
    return p, (p @ v).reshape(-1, d), lse.reshape(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "rope":
        return {"q": _exact_rope(s["q"], s["wq"], s), "k": _exact_rope(s["k"], s["wk"], s)}
    if op == "rope_bwd":
        out = {}
        for n in ("q", "k"):
            x = s[n].double().detach().requires_grad_()
            w = None if s["w" + n] is None else s["w" + n].double().requires_grad_()
            got = torch.autograd.grad(_exact_rope(x, w, s), [x] if w is None else [x, w], s["d%so" % n].double())
            out["d" + n], out["dw" + n] = got[0], None if w is None else got[1]
        return out
    if op == "append":
        q, k = _exact_rope(s["q"], s["wq"], s), _exact_rope(s["k"], s["wk"], s)
        qo, kc, vc = s["q_out"].double(), s["kc"].double(), s["vc"].double()
        for r, m in enumerate(s["lens"].tolist()):
            at = int(s["ctx"][r]) - m + torch.arange(m, device="cuda")
            block = s["table"][r].long()[at // BS]
            qo[r, :, :m] = q[r, :, :m]
            kc[block, :, at % BS] = k[r, :, :m].transpose(0, 1)
            vc[block, :, at % BS] = s["v"][r, :, :m].transpose(0, 1).double()
        return {"q": qo, "k": kc, "v": vc}
    if op in ("shared", "scored"):
        prefix = None
        if op == "shared":
            at = torch.arange(s["P"], device="cuda")
            prefix = {c: s[c][s["ptable"].long()[at // BS], :, at % BS].double().transpose(0, 1) for c in ("kc", "vc")}
        o, lse, w = [], [], s["weights"].double() if op == "scored" else None
        for r in range(s["R"]):
            p, a, b = _exact_attend(s, r, prefix)
            o.append(a)
            lse.append(b)
            if w is not None:
                w[r, :, : p.shape[-1]] += p.sum(1)
        out = {"o": torch.stack(o), "lse": torch.stack(lse)}
        return out if w is None else {**out, "weights": w}
    # eviction: one request and head at a time, the tokens sorted by (protected, weight, slot) on the host
    kc, vc, keep = s["kc"].double(), s["vc"].double(), s["keep"]
    W, P = s["weights"].double().cpu(), s["slot_pos"].cpu()
    w_out = torch.zeros_like(W)
    for r in range(s["R"]):
        n, seq = int(s["ctx"][r]), int(s["seq"][r])
        slots = torch.arange(n)
        blocks = s["table"][r].cpu().long()
        for h in range(s["Hkv"]):
            pos = torch.where(P[r, h, :n] >= 0, P[r, h, :n].long(), seq - n + slots)
            w = W[r, h, :n].clone()
            heavy = torch.where(pos >= seq - s["recent"], torch.full_like(w, math.inf), w)
            kept = torch.sort(heavy, descending=True, stable=True)[1][:keep].sort()[0]
            at = torch.arange(n)[torch.isin(slots, kept)]
            src = at[at >= keep]
            dst = slots[:keep][~torch.isin(slots[:keep], at)]
            w_out[r, h, at[at < keep]] = w[at[at < keep]]
            w_out[r, h, dst] = w[src]
            for c in (kc, vc):
                c[blocks[dst // BS].cuda(), h, (dst % BS).cuda()] = c[blocks[src // BS].cuda(), h, (src % BS).cuda()]
    return {"ctx": None, "weights": w_out, "slot_pos": None, "k": kc, "v": vc}
