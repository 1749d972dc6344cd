"""Workloads of the gated delta rule (prefill, decode) and the block plan.

Three operators of a server whose layers keep a fixed-size fp32 state per
(sequence, head) in blocks of a shared pool:

* ``prefill``: the gated delta rule over packed sequences of new tokens, from
  the pool row each sequence resumes from to the row its last block owns, with
  a snapshot in the pool after every completed block;
* ``decode``: the same recurrence for one to a few tokens of many sequences;
* ``plan``: block tables, slot maps and packed offsets from request lengths.

The recurrence, per value head h that reads key head h // (H // Hk), with the
state S [dk, dv]:  Sb = e^{g} S;  S <- Sb + beta k (v - Sb^T k)^T;
o = scale S^T q.
"""
import math

import torch

own = False   # False: elementary torch operations; True: this package's kernels

BF16, F32 = "bf16", "f32"


# ------------------------------------------------------------------ cases --

def _prefill(name, lens, Hk, H, dk, dv, dtype, resume, block, ctx=""):
    """resume: sequences start from a pool row (else from zeros); block: tokens per
    snapshot block (0 = none); ctx: tokens each sequence already has ("" = none)."""
    return {"name": name, "op": "prefill", "lens": lens, "Hk": Hk, "H": H, "dk": dk, "dv": dv,
            "dtype": dtype, "resume": resume, "block": block, "ctx": ctx}


def _decode(name, B, Tq, Hk, H, dk, dv, dtype, update, ragged):
    """update: the states advance (else a verify pass that leaves them); ragged: each
    sequence applies its own number of the Tq tokens."""
    return {"name": name, "op": "decode", "B": B, "Tq": Tq, "Hk": Hk, "H": H, "dk": dk, "dv": dv,
            "dtype": dtype, "update": update, "ragged": ragged}


def _plan(name, N, new_lo, new_hi, ctx_hi, block, lens_seed):
    """N requests with new_lo .. new_hi new tokens and up to ctx_hi cached ones
    (log-uniform, fixed by lens_seed)."""
    return {"name": name, "op": "plan", "N": N, "new_lo": new_lo, "new_hi": new_hi,
            "ctx_hi": ctx_hi, "block": block, "lens_seed": lens_seed}


def listed():
    return [
        # One long prompt at the library's headline shape, every value head with its own keys.
        _prefill("prefill_32k", "32768", 96, 96, 128, 128, BF16, False, 0),
        # A single medium prompt on a smaller layer whose key heads serve two value heads:
        # few (sequence, head) chains for a whole GPU.
        _prefill("prefill_4k", "4096", 16, 32, 128, 128, BF16, False, 0),
        # A batch of ragged prompts, some resumed from prefix-cache snapshots, that leaves a
        # snapshot in the pool after every 512-token block.
        _prefill("prefill_ragged_resume",
                 "1531,8192,2777,4160,1024,6001,3329,1999,5120,1280,7013,2048", 32, 96, 128, 128,
                 BF16, True, 512, "512,0,1024,0,4096,512,0,1536,0,2560,0,512"),
        # A scheduler's mixed step: short chunks beside requests that are decoding.
        _prefill("prefill_short_mix", "1,1,1,1,17,1,64,1,130,1,1,33,1,257,1,5", 32, 32, 128, 128,
                 BF16, True, 0),
        # The fp32 check mode with narrow heads.
        _prefill("prefill_f32", "300,1,211", 2, 4, 64, 64, F32, True, 128, "0,0,77"),
        # The full decode batch of the library's benchmark.
        _decode("decode_256", 256, 1, 48, 96, 128, 128, BF16, True, False),
        # One request on a small layer: latency.
        _decode("decode_1", 1, 1, 16, 32, 128, 128, BF16, True, False),
        # Draft tokens: the verify pass, and the replay of what was accepted.
        _decode("verify_4", 64, 4, 96, 96, 128, 128, BF16, False, False),
        _decode("replay_ragged", 100, 6, 32, 96, 128, 128, BF16, True, True),
        # The plan of a decode batch: one new token each.
        _plan("plan_decode", 256, 1, 1, 32768, 512, 1),
        # The plan of a prefill batch, small blocks.
        _plan("plan_prefill", 64, 4096, 32768, 16384, 64, 2),
        # Thousands of short requests.
        _plan("plan_many", 4000, 1, 96, 2000, 16, 3),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "plan"])
    if op == "plan":
        N = _logint(rng, 1, 4096)
        hi = _logint(rng, 1, max(1, min(32768, 1000000 // N)))
        return {k: v for k, v in _plan("", N, rng.randint(0, min(2, hi)), hi,
                                       _logint(rng, 1, 40000), rng.choice([16, 32, 64, 128, 512]),
                                       rng.randint(0, 1 << 30)).items() if k != "name"}
    group = rng.choice([1, 2, 3, 4])
    Hk = _logint(rng, 1, 96 // group)
    H = Hk * group
    dtype = rng.choice([BF16, BF16, BF16, F32])
    dk = dv = 128
    if dtype == F32 or rng.random() < 0.25:
        dk, dv = rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
    if op == "decode":
        c = _decode("", _logint(rng, 1, 256), rng.choice([1, 1, 1, 2, 3, 4, 8]), Hk, H, dk, dv,
                    dtype, rng.random() < 0.7, rng.random() < 0.5)
        if c["Tq"] > 1:
            c["B"] = min(c["B"], 128)
    else:
        # The general path (fp32, narrow heads) serves checks and small models.
        general = dtype == F32 or dk != 128 or dv != 128
        total = _logint(rng, 1, min(4096 if general else 40000, 32768 * 96 // H))
        n = min(total, _logint(rng, 1, 64))
        cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        resume = rng.random() < 0.6
        ctx = [rng.choice([0, 64, 512, rng.randint(1, 5000)]) for _ in lens] if resume else []
        c = _prefill("", ",".join(map(str, lens)), Hk, H, dk, dv, dtype, resume,
                     rng.choice([0, 0, 128, 512]), ",".join(map(str, ctx)))
    return {k: v for k, v in c.items() if k != "name"}


# ----------------------------------------------------------------- inputs --

def _ints(text, n):
    return [int(x) for x in text.split(",")] if text else [0] * n


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _tokens(case, g, lead):
    """Post-projection inputs of ``lead`` tokens: unit q and k rows, v ~ N(0, 1), beta in
    (0, 1), and log-decays whose rate differs by head from slow to fast forgetting."""
    Hk, H, dk, dv = case["Hk"], case["H"], case["dk"], case["dv"]
    dt = torch.bfloat16 if case["dtype"] == BF16 else torch.float32
    f = dict(device="cuda", generator=g)
    q = _unit(torch.randn(*lead, Hk, dk, **f)).to(dt)
    k = _unit(torch.randn(*lead, Hk, dk, **f)).to(dt)
    v = torch.randn(*lead, H, dv, **f).to(dt)
    rate = torch.exp(torch.rand(H, **f) * 6.0 - 5.0)          # e^-5 .. e
    gl = -rate * torch.nn.functional.softplus(torch.randn(*lead, H, **f))
    beta = torch.sigmoid(torch.randn(*lead, H, **f))
    return q, k, v, gl, beta


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _plan_lens(case):
    g = torch.Generator().manual_seed(case["lens_seed"])
    u = torch.rand(2, case["N"], generator=g, dtype=torch.float64)
    lo, hi = case["new_lo"], case["new_hi"]
    # Log-uniform over lo .. hi (both reached); zero-length requests appear when lo is 0.
    new = (torch.exp(u[0] * math.log(hi + 2 - lo)) - 1 + lo).to(torch.int64).clamp(lo, hi)
    ctx = (torch.exp(u[1] * math.log(case["ctx_hi"] + 1)) - 1).to(torch.int64)
    return new, ctx


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "plan":
        new, ctx = _plan_lens(case)
        bs, N = case["block"], case["N"]
        have = (ctx + bs - 1) // bs
        want = (ctx + new + bs - 1) // bs
        M = max(1, int(want.max()))
        need, old = int((want - have).sum()), int(have.sum())
        rows = torch.randperm(need + old + 16, device="cuda", generator=g).to(torch.int32)
        table = torch.full((N, M), -1, dtype=torch.int32, device="cuda")
        cols = torch.arange(M, device="cuda")
        table[cols[None, :] < have.cuda()[:, None]] = rows[:old]
        return {"case": case, "new": new.to(torch.int32).cuda(), "ctx": ctx.to(torch.int32).cuda(),
                "table": table, "free": rows[old:].contiguous(),
                "head": _i32([3]), "T": int(new.sum()), "bs": bs}
    if case["op"] == "decode":
        B, Tq, H = case["B"], case["Tq"], case["H"]
        q, k, v, gl, beta = _tokens(case, g, (B, Tq))
        # Rows read and rows written differ: every sequence crosses into a new block.
        P = 2 * B if case["update"] else B
        perm = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
        state = torch.randn(P, H, case["dk"], case["dv"], device="cuda", generator=g) * 0.1
        nt = None
        if case["ragged"]:
            nt = torch.randint(0, Tq + 1, (B,), device="cuda", generator=g).to(torch.int32)
        return {"case": case, "q": q, "k": k, "v": v, "g": gl, "beta": beta, "state": state,
                "src": perm[:B].contiguous(), "dst": perm[B:].contiguous() if case["update"] else None,
                "nt": nt, "scale": case["dk"] ** -0.5, "o": torch.zeros_like(v)}
    lens = _ints(case["lens"], 0)
    N, T = len(lens), sum(lens)
    ctx = _ints(case["ctx"], N)
    q, k, v, gl, beta = _tokens(case, g, (T,))
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    st = {"case": case, "q": q, "k": k, "v": v, "g": gl, "beta": beta, "cu": _i32(cu),
          "cu_host": torch.tensor(cu, dtype=torch.int32), "lens": lens, "ctx_host": ctx,
          "ctx": _i32(ctx) if any(ctx) else None, "scale": case["dk"] ** -0.5,
          "table": None, "src": None, "ws": None, "o": torch.empty_like(v)}
    # Pool rows: one per sequence to resume from, one per sequence for its last block, one
    # per completed block.
    bs = case["block"]
    M = max((c + n) // bs for c, n in zip(ctx, lens)) if bs else 0
    done = sum((c + n) // bs - c // bs for c, n in zip(ctx, lens)) if bs else 0
    P = 2 * N + done
    perm = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
    st["state"] = torch.randn(P, case["H"], case["dk"], case["dv"], device="cuda",
                              generator=g) * 0.1
    if case["resume"]:
        # Fresh requests (no cached token) carry no row.
        fresh = torch.tensor([c == 0 and i % 2 == 1 for i, c in enumerate(ctx)], device="cuda")
        st["src"] = torch.where(fresh, -1, perm[:N]).to(torch.int32)
    st["dst"] = perm[N:2 * N].contiguous()
    if bs:
        table = torch.full((N, max(M, 1)), -1, dtype=torch.int32)
        rows, at = perm[2 * N:].cpu(), 0
        for n in range(N):
            a, b = ctx[n] // bs, (ctx[n] + lens[n]) // bs
            table[n, a:b] = rows[at:at + b - a]
            at += b - a
        st["table"] = table.cuda()
    if own:
        import linear_attention_serving_prefill_b200 as pkg
        need = pkg.kda_gdr_prefill_workspace_size(T, N, case["Hk"], case["H"], case["dk"],
                                                  case["dv"], q.dtype)
        st["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    return st


# -------------------------------------------------------------------- run --

def run(st):
    op = st["case"]["op"]
    if own:
        import linear_attention_serving_prefill_b200 as pkg
        if op == "plan":
            p = pkg.kda_block_plan(st["new"], st["ctx"], st["free"], st["head"], st["table"],
                                   st["bs"], st["T"])
            return (p.cu_seqlens, p.positions, p.token_slots, p.src_slots, p.dst_slots,
                    p.free_head, st["table"])
        if op == "decode":
            c = st["case"]
            o = pkg.kda_gdr_decode(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"],
                                   src_slots=st["src"], dst_slots=st["dst"], num_tokens=st["nt"],
                                   update_state=c["update"], scale=st["scale"], o=st["o"])
            return (o, st["state"]) if c["update"] else (o,)
        o = pkg.kda_gdr_prefill(st["q"], st["k"], st["v"], st["g"], st["beta"], st["cu"],
                                st["cu_host"], state=st["state"], src_slots=st["src"],
                                dst_slots=st["dst"], ctx_lens=st["ctx"], block_table=st["table"],
                                block_size=st["case"]["block"], scale=st["scale"], o=st["o"],
                                workspace=st["ws"])
        return o, st["state"]
    if op == "plan":
        return _plain_plan(st)
    return _plain_decode(st) if op == "decode" else _plain_prefill(st)


def _plain_plan(st):
    bs, T = st["bs"], st["T"]
    new, ctx, table = st["new"].long(), st["ctx"].long(), st["table"]
    N, M = table.shape
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    cu = torch.cat([zero, torch.cumsum(new, 0)])
    have, want = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    first = torch.cumsum(want - have, 0) - (want - have) + st["head"].long()
    col = torch.arange(M, device="cuda")[None, :]
    idx = first[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    F = st["free"].numel()
    got = torch.where(idx < F, st["free"][idx.clamp(0, F - 1)], -1)
    table.copy_(torch.where(fresh, got, table))
    row = torch.arange(N, device="cuda")

    def slot_of(tokens):
        return torch.where(tokens > 0, table[row, ((tokens - 1) // bs).clamp_min(0)], -1).int()

    seq = torch.repeat_interleave(row, new, output_size=T)
    pos = torch.arange(T, device="cuda") - cu[seq] + ctx[seq]
    blk = table[seq, pos // bs].long()
    slots = torch.where(blk >= 0, blk * bs + pos % bs, -1)
    head = st["head"] + (want - have).sum().int()
    return cu.int(), pos.int(), slots, slot_of(ctx), slot_of(ctx + new), head, table


def _step(S, q, k, v, a, beta, scale):
    """One token on states S [..., dk, dv]; returns the new states and the output."""
    S = S * a[..., None, None]
    seen = (S * k[..., :, None]).sum(-2)
    S = S + k[..., :, None] * (beta[..., None] * (v - seen))[..., None, :]
    return S, scale * (S * q[..., :, None]).sum(-2)


def _plain_decode(st):
    c = st["case"]
    rep = c["H"] // c["Hk"]
    q = st["q"].float().repeat_interleave(rep, -2)
    k = st["k"].float().repeat_interleave(rep, -2)
    v, a, beta = st["v"].float(), torch.exp(st["g"]), st["beta"]
    S = st["state"][st["src"].long()]
    o = torch.zeros_like(v)
    for t in range(c["Tq"]):
        S2, ot = _step(S, q[:, t], k[:, t], v[:, t], a[:, t], beta[:, t], st["scale"])
        if st["nt"] is not None:
            live = (t < st["nt"]).view(-1, 1, 1)
            S2 = torch.where(live[..., None], S2, S)
            ot = torch.where(live, ot, torch.zeros_like(ot))
        S, o[:, t] = S2, ot
    o = o.to(st["v"].dtype)
    if not c["update"]:
        return (o,)
    st["state"][st["dst"].long()] = S
    return o, st["state"]


def _plain_prefill(st):
    """Chunks of 64 tokens, aligned to multiples of 64 of the absolute position: inside a
    chunk with G the running log-decay, A = tril(beta K K^T e^{Gr-Gs}, -1), the edits
    D = (I + A)^-1 beta (V - e^G K S), o = scale (e^G Q S + tril(Q K^T e^{Gr-Gs}) D) and
    S <- e^{GC} S + (e^{GC-G} K)^T D."""
    c, C = st["case"], 64
    H, rep, bs = c["H"], c["H"] // c["Hk"], c["block"]
    lens, ctx = st["lens"], st["ctx_host"]
    N = len(lens)
    off = [x % C for x in ctx]
    nch = [(off[n] + lens[n] + C - 1) // C for n in range(N)]
    order = sorted(range(N), key=lambda n: -nch[n])
    state, table = st["state"], st["table"]
    # Rows of the chunk grid: chunk j of every sequence that has one, longest first.
    live_at = []
    for j in range(max(nch)):
        live = [n for n in order if nch[n] > j]
        live_at.append(live)
    starts = torch.tensor([[int(st["cu_host"][n]) + j * C - off[n], int(st["cu_host"][n]),
                            int(st["cu_host"][n + 1])]
                           for j, live in enumerate(live_at) for n in live], device="cuda")
    idx = starts[:, :1] + torch.arange(C, device="cuda")[None, :]
    ok = (idx >= starts[:, 1:2]) & (idx < starts[:, 2:])
    idx = idx.clamp(0, st["q"].shape[0] - 1)
    lower = torch.ones(C, C, device="cuda", dtype=torch.bool).tril()
    eye = torch.eye(C, device="cuda")
    out = torch.empty_like(st["v"], dtype=torch.float32)
    # Heads in groups, so that the intermediates of a long prompt stay a few GB.
    per = max(rep, int(2e9 // (idx.numel() * 128 * 4)) // rep * rep)
    for h0 in range(0, H, per):
        hs, ks = slice(h0, min(H, h0 + per)), slice(h0 // rep, min(H, h0 + per) // rep)

        def chunked(x, m=ok[..., None]):
            return torch.where(m if x.dim() == 2 else m[..., None], x[idx].float(), 0.0)

        q = chunked(st["q"][:, ks]).repeat_interleave(rep, 2).transpose(1, 2)
        k = chunked(st["k"][:, ks]).repeat_interleave(rep, 2).transpose(1, 2)
        v = chunked(st["v"][:, hs]).transpose(1, 2)
        G = torch.cumsum(chunked(st["g"][:, hs]), 1).transpose(1, 2)
        beta = chunked(st["beta"][:, hs]).transpose(1, 2)
        D = torch.exp(torch.where(lower, G[..., :, None] - G[..., None, :], -1e30))
        A = (k @ k.transpose(-1, -2)) * D * beta[..., None] * (1.0 - eye)
        P = (q @ k.transpose(-1, -2)) * D
        del D
        X = eye.expand_as(A).clone()       # (I + A)^-1 by forward substitution
        for r in range(1, C):
            X[..., r, :r] = -(A[..., r:r + 1, :r] @ X[..., :r, :r])[..., 0, :]
        W = X @ (k * (beta * torch.exp(G))[..., None])
        U = X @ (v * beta[..., None])
        q = q * torch.exp(G)[..., None]
        GC = G[..., -1]
        k = k * torch.exp(GC[..., None] - G)[..., None]
        S = torch.zeros(N, H if per >= H else hs.stop - hs.start, c["dk"], c["dv"], device="cuda")
        if st["src"] is not None:
            src = st["src"][order].long()
            S = torch.where((src >= 0).view(-1, 1, 1, 1), state[src.clamp_min(0), hs], S)
        o = torch.empty_like(v)
        at, decay = 0, torch.exp(GC)[..., None, None]
        for j, live in enumerate(live_at):
            m = len(live)
            r = slice(at, at + m)
            Sj = S[:m]
            d = U[r] - W[r] @ Sj
            o[r] = q[r] @ Sj + P[r] @ d
            Sj.mul_(decay[r]).add_(k[r].transpose(-1, -2) @ d)
            at += m
            if bs:
                for i, n in enumerate(live):
                    end = ctx[n] - off[n] + (j + 1) * C
                    if end % bs == 0 and end <= ctx[n] + lens[n]:
                        state[table[n, end // bs - 1].long(), hs] = Sj[i]
        state[:, hs].index_copy_(0, st["dst"][order].long(), S)
        flat = out[:, hs]
        flat[idx[ok]] = st["scale"] * o.transpose(1, 2)[ok]
    return out.to(st["v"].dtype), state


# ------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "plan":
        new, ctx = _plan_lens(case)
        bs, T, N = case["block"], int(new.sum()), case["N"]
        fresh = int(((ctx + new + bs - 1) // bs - (ctx + bs - 1) // bs).sum())
        return {"bytes": 8 * N + 8 * fresh + 4 * (N + 1) + 16 * N + 12 * T + 8, "flops": 4 * T + N}
    Hk, H, dk, dv = case["Hk"], case["H"], case["dk"], case["dv"]
    es = 2 if case["dtype"] == BF16 else 4
    per_token = es * (2 * Hk * dk + 2 * H * dv) + 8 * H
    row = 4 * H * dk * dv
    if case["op"] == "decode":
        tokens = case["B"] * case["Tq"]
        return {"bytes": tokens * per_token + case["B"] * row * (2 if case["update"] else 1),
                "flops": 7 * tokens * H * dk * dv}
    lens = _ints(case["lens"], 0)
    ctx, bs = _ints(case["ctx"], len(lens)), case["block"]
    rows = len(lens) * (2 if case["resume"] else 1)
    if bs:
        rows += sum((c + n) // bs - c // bs for c, n in zip(ctx, lens))
    return {"bytes": sum(lens) * per_token + rows * row, "flops": 7 * sum(lens) * H * dk * dv}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """The recurrence token by token in 64 bits (the plan: plain loops on the host)."""
    st = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(st)
    H, group, dbl = case["H"], case["H"] // case["Hk"], torch.float64
    pool = st["state"].to(dbl)
    head = torch.arange(H, device="cuda") // group
    if case["op"] == "decode":
        B, Tq = case["B"], case["Tq"]
        seqs = [(b * Tq, Tq if st["nt"] is None else int(st["nt"][b])) for b in range(B)]
        src = st["src"].tolist()
    else:
        seqs = [(int(st["cu_host"][n]), st["lens"][n]) for n in range(len(st["lens"]))]
        src = st["src"].tolist() if st["src"] is not None else [-1] * len(seqs)
    flat = {x: st[x].reshape(-1, *st[x].shape[-(1 if x in ("g", "beta") else 2):])
            for x in ("q", "k", "v", "g", "beta")}
    o = torch.zeros(flat["v"].shape, dtype=dbl, device="cuda")
    by_len = sorted(range(len(seqs)), key=lambda i: -seqs[i][1])
    M = torch.stack([pool[src[i]] if src[i] >= 0 else torch.zeros_like(pool[0]) for i in by_len])
    begin = torch.tensor([seqs[i][0] for i in by_len], device="cuda")
    length = [seqs[i][1] for i in by_len]
    marks = {}
    if case["op"] == "prefill" and case["block"]:
        bs = case["block"]
        rows = st["table"].tolist()
        for place, i in enumerate(by_len):
            c0 = st["ctx_host"][i]
            for j in range(c0 // bs, (c0 + length[place]) // bs):
                marks.setdefault((j + 1) * bs - c0 - 1, []).append((place, rows[i][j]))
    n = len(length)
    for t in range(length[0] if length else 0):
        while n and length[n - 1] <= t:
            n -= 1
        i = begin[:n] + t
        kt = flat["k"][i].to(dbl)[:, head].unsqueeze(-1)
        m = M[:n]
        m *= flat["g"][i].to(dbl).exp()[..., None, None]
        err = flat["v"][i].to(dbl) - (m * kt).sum(2)
        m += kt * (err * flat["beta"][i].to(dbl).unsqueeze(-1)).unsqueeze(2)
        o[i] = (m * flat["q"][i].to(dbl)[:, head].unsqueeze(-1)).sum(2) * st["scale"]
        for place, r in marks.get(t, ()):
            pool[r] = M[place]
    o = o.view(st["v"].shape)
    if case["op"] == "decode" and not case["update"]:
        return (o,)
    dst = st["dst"].tolist()
    for place, i in enumerate(by_len):
        pool[dst[i]] = M[place]
    return o, pool


def _exact_plan(st):
    bs = st["bs"]
    new, ctx = st["new"].tolist(), st["ctx"].tolist()
    table, free, head = st["table"].tolist(), st["free"].tolist(), int(st["head"])
    cu, pos, slots, src, dst = [0], [], [], [], []
    for n, (a, b) in enumerate(zip(ctx, new)):
        for j in range(-(-a // bs), -(-(a + b) // bs)):
            table[n][j] = free[head] if head < len(free) else -1
            head += 1
        cu.append(cu[-1] + b)
        src.append(table[n][(a - 1) // bs] if a else -1)
        dst.append(table[n][(a + b - 1) // bs] if a + b else -1)
        row = table[n]
        pos.extend(range(a, a + b))
        slots.extend(row[p // bs] * bs + p % bs if row[p // bs] >= 0 else -1
                     for p in range(a, a + b))
    return (_i32(cu), _i32(pos), torch.tensor(slots, device="cuda"), _i32(src), _i32(dst),
            _i32([head]), torch.tensor(table, dtype=torch.int32, device="cuda"))
