"""Gated delta rule on the GPU against the plain 64-bit form.

Tolerances, relative to the largest reference magnitude of a tensor.  The fp32 recurrence
gets 1e-4, the library's fp32 parity bar; storing an output in bf16 is off by at most 2^-8 of
its value, so o gets 2^-8 more.  On tensor cores the state passes five operands (S, R, T, R F
and the update's F) that are two bf16 numbers each, off by at most 2^-16 of the value, in each
of the few chunks that it survives undiminished: 5 * 2^-16 * 3 = 2.3e-4.  The outputs' own
products take S and P as one bf16 number: with the rounding of o itself 3 * 2^-8 more."""
import pytest
import torch

from tests import gdr_testutil as U

pytestmark = pytest.mark.gpu

TOL_F32, TOL_TC_S = 1e-4, 15 * 2.0 ** -16
TOL_TC = 3 * 2.0 ** -8 + TOL_TC_S
TOL_O = {"f32": TOL_F32, "bf16": 2.0 ** -8 + TOL_F32}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ALGOS = ["cuda_core", "tensor_core"]


@pytest.fixture(scope="module")
def K():
    from linear_attention_serving_prefill_b200 import binding
    return binding


def i32(x):
    return None if x is None else torch.as_tensor(x, dtype=torch.int32).cuda()


def dev(x):
    return {n: t.cuda() for n, t in x.items()}


def algos_for(dtype, dk, dv):
    return [a for a in ALGOS if a == "cuda_core" or (dtype == "bf16" and dk == 128 and dv == 128)]


def run_prefill(K, x, lens, state, src, dst, algo, scale, ctx=None, table=None, block=0,
                host=True, pad=0):
    """Returns (o, pool); o starts as a pattern so that untouched rows show."""
    cu = U.cu_of(lens)
    d = dev(x)
    o = torch.full(x["v"].shape, 7.0, dtype=x["v"].dtype, device="cuda")
    st = None if state is None else state.cuda()
    K.kda_gdr_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], cu.cuda(),
                      cu if host and not pad else None, state=st, src_slots=i32(src),
                      dst_slots=i32(dst), ctx_lens=i32(ctx),
                      block_table=None if table is None else i32(table), block_size=block,
                      scale=scale, o=o, algo=algo)
    torch.cuda.synchronize()
    assert K.kda_device_status() == 0
    return o, st


def spans_of(lens):
    cu = U.cu_of(lens).tolist()
    return [(cu[n], lens[n]) for n in range(len(lens))]


def check_prefill(K, x, lens, H, state, src, dst, scale, dtype, algo, ctx=None, table=None,
                  block=0, host=True, pad=0):
    ref_o, ref_S = U.reference(x, spans_of(lens), H, scale, state, src, dst, ctx, table, block)
    o, S = run_prefill(K, x, lens, state, src, dst, algo, scale, ctx, table, block, host, pad)
    T = sum(lens)
    tc = algo == "tensor_core"
    assert U.max_err(o[:T], ref_o[:T]) <= (TOL_TC if tc else TOL_O[dtype])
    if pad:
        assert bool((o[T:] == 7.0).all())
    if state is not None:
        touched = set() if table is None else {r for row in table.tolist() for r in row}
        touched |= set(dst or [])
        for r in range(state.shape[0]):
            if r in touched and not torch.equal(ref_S[r], state[r].double()):
                assert U.max_err(S[r], ref_S[r]) <= (TOL_TC_S if tc else TOL_F32), f"row {r}"
            else:
                assert torch.equal(S[r].cpu(), state[r]), f"row {r} was written"
    return o, S


LENS = [[1], [2, 1, 3], [63], [64], [65], [16, 17, 0, 130, 1], [128, 129], [127, 0, 0, 64], [300]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("f32", 128, 128), ("f32", 64, 32),
                                         ("bf16", 32, 128), ("f32", 32, 64), ("bf16", 64, 64)])
def test_prefill_lengths(K, lens, dtype, dk, dv):
    Hk, H = 2, 4
    x = U.tokens((sum(lens),), Hk, H, dk, dv, DT[dtype], seed=len(lens))
    N = len(lens)
    state = U.pool(2 * N + 1, H, dk, dv, seed=3)
    src = [i if i % 3 != 1 else -1 for i in range(N)]
    dst = [N + i for i in range(N)]
    for algo in algos_for(dtype, dk, dv):
        check_prefill(K, x, lens, H, state, src, dst, dk ** -0.5, dtype, algo)


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 3), (3, 3), (2, 10), (5, 5)])
def test_prefill_head_groups(K, Hk, H):
    lens = [70, 5]
    for dtype in ("f32", "bf16"):
        x = U.tokens((75,), Hk, H, 128, 128, DT[dtype], seed=Hk)
        state = U.pool(2, H, 128, 128, seed=5)
        for algo in algos_for(dtype, 128, 128):
            check_prefill(K, x, lens, H, state, [0, 1], [0, 1], 1.0, dtype, algo, host=False)


def test_prefill_without_pool(K):
    lens = [40, 100]
    for dtype in ("f32", "bf16"):
        x = U.tokens((140,), 2, 2, 128, 128, DT[dtype], seed=8)
        for algo in algos_for(dtype, 128, 128):
            check_prefill(K, x, lens, 2, None, None, None, 0.5, dtype, algo)


@pytest.mark.parametrize("ctx", [[0, 0, 0], [64, 5, 127], [1000, 1, 63], [128, 192, -3]], ids=str)
@pytest.mark.parametrize("block", [64, 128])
def test_prefill_block_rows(K, ctx, block):
    """A block's row gets the state at its boundary of the absolute position."""
    lens = [200, 130, 64]
    N, H = 3, 2
    pos = [max(c, 0) for c in ctx]
    cols = max((c + n) // block for c, n in zip(pos, lens)) + 1
    for dtype in ("f32", "bf16"):
        x = U.tokens((sum(lens),), 1, H, 128, 128, DT[dtype], seed=11)
        state = U.pool(2 * N + N * cols, H, 128, 128, seed=12)
        table = torch.arange(2 * N, 2 * N + N * cols, dtype=torch.int32).view(N, cols)
        table[1, -2:] = -1                       # blocks without a row
        table[2, 0] = state.shape[0] + 5         # a row outside the pool
        for algo in algos_for(dtype, 128, 128):
            check_prefill(K, x, lens, H, state, [0, -1, 2], [3, 4, 5], 0.3, dtype, algo, ctx=pos,
                          table=table, block=block)
            if min(ctx) < 0:                     # a negative context counts as none
                a = run_prefill(K, x, lens, state, [0, -1, 2], [3, 4, 5], algo, 0.3, ctx, table, block)
                b = run_prefill(K, x, lens, state, [0, -1, 2], [3, 4, 5], algo, 0.3, pos, table, block)
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prefill_fewer_table_columns_than_blocks(K):
    lens = [300]
    for dtype in ("f32", "bf16"):
        x = U.tokens((300,), 1, 1, 128, 128, DT[dtype], seed=13)
        state = U.pool(4, 1, 128, 128, seed=14)
        table = torch.tensor([[1, 2]], dtype=torch.int32)
        for algo in algos_for(dtype, 128, 128):
            check_prefill(K, x, lens, 1, state, [0], [3], 1.0, dtype, algo, table=table, block=64)


def test_prefill_rows_in_place_shared_and_missing(K):
    """In-place rows, one row read by several sequences, rows outside the pool."""
    lens = [70, 64, 3, 0, 0]
    for dtype in ("f32", "bf16"):
        x = U.tokens((sum(lens),), 2, 2, 128, 128, DT[dtype], seed=15)
        state = U.pool(6, 2, 128, 128, seed=16)
        for algo in algos_for(dtype, 128, 128):
            check_prefill(K, x, lens, 2, state, [0, 1, 1, 1, 99], [0, 2, -7, 3, 4], 1.0, dtype, algo)


@pytest.mark.parametrize("what", ["alpha1", "fast", "neg_inf", "beta0", "same_key", "mixed"])
def test_prefill_decays(K, what):
    """No decay, decays that wipe the state, g = -inf, beta = 0, one repeated key."""
    lens = [150]
    for dtype in ("f32", "bf16"):
        x = U.tokens((150,), 1, 3, 128, 128, DT[dtype], seed=17)
        if what == "alpha1":
            x["g"] = torch.zeros_like(x["g"])
        elif what == "fast":
            x["g"] = x["g"] * 100 - 20
        elif what == "neg_inf":
            x["g"][::7] = -float("inf")
        elif what == "beta0":
            x["beta"] = torch.zeros_like(x["beta"])
        elif what == "same_key":
            x["k"] = x["k"][:1].expand_as(x["k"]).contiguous()
            x["beta"] = torch.ones_like(x["beta"])
            x["g"] = x["g"] * 0.01
        else:
            x["g"][:, 0] = -200.0
            x["g"][:, 1] = 0.0
        state = U.pool(2, 3, 128, 128, seed=18, std=1.0)
        for algo in algos_for(dtype, 128, 128):
            check_prefill(K, x, lens, 3, state, [0], [1], 1.0, dtype, algo)


def test_prefill_padded_batch_and_foreign_values(K):
    """Device offsets that end before the buffers do: rows behind stay as they were, and
    infinities and NaN there, or in another sequence, reach no result."""
    lens = [37, 90, 1]
    T, pad = sum(lens), 50
    for dtype in ("f32", "bf16"):
        x = U.tokens((T + pad,), 2, 2, 128, 128, DT[dtype], seed=19)
        for n in ("q", "k", "v", "g", "beta"):
            x[n][T:] = float("nan")
            x[n][T + 3:T + 9] = float("inf")
        state = U.pool(6, 2, 128, 128, seed=20)
        for algo in algos_for(dtype, 128, 128):
            check_prefill(K, x, lens, 2, state, [0, 1, 2], [3, 4, 5], 1.0, dtype, algo, pad=pad)
        # A poisoned middle sequence: its neighbours are bit-equal to a clean run.
        for algo in algos_for(dtype, 128, 128):
            a, Sa = run_prefill(K, x, lens, state, [0, 1, 2], [3, 4, 5], algo, 1.0, pad=pad)
            y = {n: t.clone() for n, t in x.items()}
            for n in ("q", "k", "v"):
                y[n][37:127] = float("nan")
                y[n][40:50] = float("inf")
            b, Sb = run_prefill(K, y, lens, state, [0, 1, 2], [3, 4, 5], algo, 1.0, pad=pad)
            assert torch.equal(a[:37], b[:37]) and torch.equal(a[127:], b[127:])
            assert torch.equal(Sa[3], Sb[3]) and torch.equal(Sa[5], Sb[5])
            assert bool(torch.isnan(b[37:127]).any())


def test_prefill_split_in_two_calls_continues(K):
    """Two calls with the state carried in the pool equal one call (block rows too)."""
    for dtype in ("f32", "bf16"):
        x = U.tokens((333,), 1, 2, 128, 128, DT[dtype], seed=21)
        state = U.pool(8, 2, 128, 128, seed=22)
        table = torch.tensor([[3, 4, 5, 6]], dtype=torch.int32)
        for algo in algos_for(dtype, 128, 128):
            ref_o, ref_S = U.reference(x, [(0, 333)], 2, 1.0, state, [0], [1], None, table, 64)
            tol = (TOL_TC, TOL_TC_S) if algo == "tensor_core" else (TOL_O[dtype], TOL_F32)
            for cut in (1, 64, 100, 320):
                first = {n: t[:cut].contiguous() for n, t in x.items()}
                rest = {n: t[cut:].contiguous() for n, t in x.items()}
                oa, S = run_prefill(K, first, [cut], state, [0], [2], algo, 1.0, [0], table, 64)
                ob, S = run_prefill(K, rest, [333 - cut], S.cpu(), [2], [1], algo, 1.0, [cut], table, 64)
                assert U.max_err(torch.cat([oa, ob]), ref_o) <= tol[0]
                for r in (1, 3, 4, 5, 6):
                    assert U.max_err(S[r], ref_S[r]) <= tol[1], (cut, r)


@pytest.mark.parametrize("Tq", [1, 2, 3, 8, 9, 64])
@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("f32", 128, 64), ("f32", 32, 32),
                                         ("bf16", 64, 128)])
def test_decode(K, Tq, dtype, dk, dv):
    B, Hk, H = 5, 2, 6
    x = U.tokens((B * Tq,), Hk, H, dk, dv, DT[dtype], seed=Tq)
    state = U.pool(12, H, dk, dv, seed=23)
    nt = [Tq, 0, (Tq + 1) // 2, Tq + 3, -2]
    applied = [min(max(n, 0), Tq) for n in nt]
    src, dst = [3, 0, -1, 7, 2], [8, 1, 9, 7, 40]
    d = {n: t.cuda().view(B, Tq, *t.shape[1:]) for n, t in x.items()}
    spans = [(b * Tq, applied[b]) for b in range(B)]
    ref_o, ref_S = U.reference(x, spans, H, 0.7, state, src, dst)
    live = torch.isfinite(ref_o)
    ref_o = torch.where(live, ref_o, torch.full_like(ref_o, 7.0))
    for update in (True, False):
        st = state.cuda()
        o = torch.full_like(d["v"], 7.0)
        K.kda_gdr_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], st, src_slots=i32(src),
                         dst_slots=i32(dst) if update else None, num_tokens=i32(nt),
                         update_state=update, scale=0.7, o=o)
        flat = o.view(B * Tq, H, dv).cpu()
        assert bool((flat[~live] == 7.0).all())
        assert U.max_err(flat, ref_o) <= TOL_O[dtype]
        if update:
            for r in range(12):
                if r in dst:
                    assert U.max_err(st[r], ref_S[r]) <= TOL_F32
                else:
                    assert torch.equal(st[r].cpu(), state[r])
        else:
            assert torch.equal(st.cpu(), state)


def test_decode_defaults(K):
    """No slots: row b in place; three-dimensional tokens; no outputs wanted."""
    B, H = 4, 2
    x = U.tokens((B,), 1, H, 128, 128, torch.bfloat16, seed=30)
    state = U.pool(B + 1, H, 128, 128, seed=31)
    d = dev(x)
    st = state.cuda()
    o = K.kda_gdr_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], st)
    rows = list(range(B))
    ref_o, ref_S = U.reference(x, [(b, 1) for b in rows], H, 1.0, state, rows, rows)
    assert U.max_err(o, ref_o) <= TOL_O["bf16"] and U.max_err(st, ref_S) <= TOL_F32
    again = state.cuda()
    assert K.kda_gdr_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], again, want_outputs=False) is None
    assert torch.equal(st, again)


def test_decode_far_rows(K):
    """Pool rows whose element offsets pass 32 bits."""
    H, P = 96, 1500
    state = torch.zeros(P, H, 128, 128, device="cuda")
    x = U.tokens((2,), 1, H, 128, 128, torch.bfloat16, seed=32)
    row = U.pool(1, H, 128, 128, seed=33)
    state[P - 1].copy_(row[0])
    d = dev(x)
    o = K.kda_gdr_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], state,
                         src_slots=i32([P - 1, 0]), dst_slots=i32([P - 2, 1]))
    big = torch.cat([row, torch.zeros(3, H, 128, 128)])
    ref_o, ref_S = U.reference(x, [(0, 1), (1, 1)], H, 1.0, big, [0, 1], [2, 3])
    assert U.max_err(o, ref_o) <= TOL_O["bf16"]
    assert U.max_err(state[P - 2], ref_S[2]) <= TOL_F32
    assert U.max_err(state[1], ref_S[3]) <= TOL_F32
    for algo in algos_for("bf16", 128, 128):
        cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
        K.kda_gdr_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, state=state,
                          src_slots=i32([P - 1]), dst_slots=i32([P - 3]), algo=algo)
        _, S = U.reference(x, [(0, 2)], H, 1.0, big, [0], [2])
        assert U.max_err(state[P - 3], S[2]) <= (TOL_TC_S if algo == "tensor_core" else TOL_F32)
    del state


def plan_tensors(new, ctx, free, head, table):
    return (i32(new), i32(ctx), i32(free), i32([head]), i32(table))


@pytest.mark.parametrize("case", [
    dict(new=[1, 1, 1], ctx=[0, 5, 64], bs=64, F=20),
    dict(new=[0, 7, 0, 200, 1], ctx=[0, 0, 3, 60, 127], bs=16, F=40),
    dict(new=[5, 5, 5], ctx=None, bs=4, F=4),                    # the free list runs out
    dict(new=[100, 30], ctx=[0, 50], bs=16, F=40, cols=4),       # blocks past the table
    dict(new=[-3, 4], ctx=[2, -9], bs=3, F=9),                   # negative lengths count as 0
    dict(new=[9], ctx=[7], bs=1, F=30),
], ids=str)
@pytest.mark.parametrize("head,extra", [(0, 0), (2, 5), (-4, 0)])
def test_plan(K, case, head, extra):
    new, ctx, bs = case["new"], case["ctx"], case["bs"]
    c = [0] * len(new) if ctx is None else ctx
    cols = case.get("cols") or max(-(-(max(a, 0) + max(b, 0)) // bs) for a, b in zip(c, new)) + 1
    free = torch.randperm(case["F"], generator=torch.Generator().manual_seed(1)).tolist()
    table = [[1000 + 10 * n + j if j < -(-max(c[n], 0) // bs) else -7 for j in range(cols)]
             for n in range(len(new))]
    T = sum(max(x, 0) for x in new) + extra
    ref = U.plan_reference(new, ctx, free, head, table, bs, T)
    t = plan_tensors(new, ctx, free, head, table)
    p = K.kda_block_plan(t[0], t[1], t[2], t[3], t[4], bs, T)
    got = [p.cu_seqlens, p.positions, p.token_slots, p.src_slots, p.dst_slots, p.free_head, t[4]]
    for g, r in zip(got, [*ref[:5], [ref[5]], ref[6]]):
        assert g.tolist() == r


@pytest.mark.parametrize("N,hi,bs,seed", [(1, 9000, 64, 0), (1024, 9, 16, 1), (1025, 40, 64, 2),
                                          (3000, 3, 512, 3), (70, 500, 16, 4), (5, 20000, 128, 5)])
def test_plan_large(K, N, hi, bs, seed):
    gen = torch.Generator().manual_seed(seed)
    new = torch.randint(0, hi + 1, (N,), generator=gen).tolist()
    ctx = torch.randint(0, 300, (N,), generator=gen).tolist()
    cols = max(-(-(a + b) // bs) for a, b in zip(ctx, new)) + 1
    need = sum(-(-(a + b) // bs) - -(-a // bs) for a, b in zip(ctx, new))
    free = torch.randperm(need + 5, generator=gen).tolist()
    table = torch.randint(0, 1000, (N, cols), generator=gen).tolist()
    T = sum(new)
    ref = U.plan_reference(new, ctx, free, 3, table, bs, T)
    t = plan_tensors(new, ctx, free, 3, table)
    p = K.kda_block_plan(t[0], t[1], t[2], t[3], t[4], bs, T)
    got = [p.cu_seqlens, p.positions, p.token_slots, p.src_slots, p.dst_slots, p.free_head, t[4]]
    for g, r in zip(got, [*ref[:5], [ref[5]], ref[6]]):
        assert g.tolist() == r


def test_plan_fewer_token_entries_than_tokens(K):
    """A token buffer shorter than the batch is filled to its end, no further."""
    t = plan_tensors([10, 10], [0, 0], list(range(8)), 0, [[-1] * 4] * 2)
    p = K.kda_block_plan(*t, 4, 13)
    ref = U.plan_reference([10, 10], [0, 0], list(range(8)), 0, [[-1] * 4] * 2, 4, 20)
    assert p.positions.tolist() == ref[1][:13] and p.token_slots.tolist() == ref[2][:13]
    assert p.cu_seqlens.tolist() == [0, 10, 20]


def serve(K, x, prompt, steps, H, block, algo, rows, graph=False):
    """Plan -> prefill -> (plan -> decode) x steps over one pool; returns the outputs per
    request and the pool with its table."""
    N = len(prompt)
    total = [p + steps for p in prompt]
    d = dev(x)
    start = U.cu_of(total).tolist()
    idx = torch.cat([torch.arange(start[n], start[n] + prompt[n]) for n in range(N)]).cuda()
    cols = max(-(-t // block) for t in total)
    table = torch.full((N, cols), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(rows, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    head = i32([0])
    pool = torch.full((rows, H, 128, 128), float("nan"), device="cuda")
    new, ctx = i32(prompt), i32([0] * N)
    p = K.kda_block_plan(new, ctx, free, head, table, block, sum(prompt))
    sel = {n: t[idx].contiguous() for n, t in d.items()}
    o = torch.zeros_like(d["v"])
    o[idx] = K.kda_gdr_prefill(sel["q"], sel["k"], sel["v"], sel["g"], sel["beta"], p.cu_seqlens,
                               state=pool, src_slots=p.src_slots, dst_slots=p.dst_slots,
                               ctx_lens=ctx, block_table=table, block_size=block, scale=0.5,
                               algo=algo)
    head.copy_(p.free_head)
    one = i32([1] * N)
    ctx.copy_(new)
    at = torch.tensor(start[:N]).cuda() + ctx
    tok = {n: t[at].contiguous() for n, t in d.items()}
    out = torch.empty_like(tok["v"])
    pl = K.kda_block_plan(one, ctx, free, head, table.clone(), block, N)   # its buffers
    plan = K.BlockPlan(pl.cu_seqlens, pl.positions, pl.token_slots, pl.src_slots, pl.dst_slots, head)

    def decode():
        K.kda_block_plan(one, ctx, free, head, table, block, N, out=plan)
        K.kda_gdr_decode(tok["q"], tok["k"], tok["v"], tok["g"], tok["beta"], pool,
                         src_slots=plan.src_slots, dst_slots=plan.dst_slots, scale=0.5, o=out)
        ctx.add_(one)

    run = decode
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            decode()
        run = g.replay
    for _ in range(steps):
        for n, t in d.items():
            tok[n].copy_(t[at])
        run()
        o[at] = out
        at += 1
    torch.cuda.synchronize()
    return o, pool, table, int(head)


@pytest.mark.parametrize("graph", [False, True])
def test_serving_run(K, graph):
    """A run of them together: every output, every completed block's row and the last
    rows equal the plain form, eagerly and with the step captured in a graph."""
    prompt, steps, H, block = [60, 128, 1, 190], 70, 2, 64
    total = [p + steps for p in prompt]
    x = U.tokens((sum(total),), 1, H, 128, 128, torch.bfloat16, seed=40)
    need = sum(-(-t // block) for t in total)
    ids = torch.arange(need, dtype=torch.int32)
    cols = max(-(-t // block) for t in total)
    ref_table = torch.full((4, cols), -1, dtype=torch.int32)
    at = 0
    for n, t in enumerate(total):
        ref_table[n, :-(-t // block)] = ids[at:at - (-t // block)]
        at += -(-t // block)
    dst = [int(ref_table[n, (t - 1) // block]) for n, t in enumerate(total)]
    ref_o, ref_S = U.reference(x, spans_of(total), H, 0.5, torch.zeros(need, H, 128, 128), None,
                               dst, None, ref_table, block)
    for algo in algos_for("bf16", 128, 128):
        o, pool, table, head = serve(K, x, prompt, steps, H, block, algo, need + 3, graph)
        assert head == need
        tol = (TOL_TC, TOL_TC_S) if algo == "tensor_core" else (TOL_O["bf16"], TOL_F32)
        assert U.max_err(o, ref_o) <= tol[0]
        for n, t in enumerate(total):
            for j in range(-(-t // block)):
                assert U.max_err(pool[int(table[n, j])], ref_S[int(ref_table[n, j])]) <= tol[1]
        used = table[table >= 0].tolist()
        assert len(set(used)) == need
        rest = [r for r in range(need + 3) if r not in used]
        assert bool(torch.isnan(pool[rest]).all())


def test_streams_and_repeats(K):
    """Two calls at once on two streams, and repeated calls, give the same bits."""
    lens = [100, 260, 64]
    x = U.tokens((sum(lens),), 2, 4, 128, 128, torch.bfloat16, seed=50)
    state = U.pool(6, 4, 128, 128, seed=51)
    for algo in algos_for("bf16", 128, 128):
        o0, S0 = run_prefill(K, x, lens, state, [0, 1, 2], [3, 4, 5], algo, 1.0)
        d, cu = dev(x), U.cu_of(lens).cuda()
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs, pools = [torch.empty_like(d["v"]) for _ in streams], [state.cuda() for _ in streams]
        src, dst = i32([0, 1, 2]), i32([3, 4, 5])
        torch.cuda.synchronize()
        for _ in range(3):
            for s, o, st in zip(streams, outs, pools):
                K.kda_gdr_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, state=st,
                                  src_slots=src, dst_slots=dst, o=o, algo=algo, stream=s)
        torch.cuda.synchronize()
        for o, st in zip(outs, pools):
            assert torch.equal(o, o0) and torch.equal(st, S0)


def test_prefill_decays_head_by_head(K):
    """Constant decays of 4 to 256 bits per 64 tokens, one per head, and single steep tokens in
    slow heads: every output row is within the operands' roundings of the state it reads
    (|q| = 1: 2^-8 of S's 2-norm for each of S and P F), every head's state within its own."""
    T, H = 200, 32
    x = U.tokens((T,), H, H, 128, 128, torch.bfloat16, seed=60)
    bits = torch.linspace(4.0, 256.0, H) / 64
    for steep in (False, True):
        x["g"] = (-bits * 0.6931472).expand(T, H).contiguous()
        if steep:
            x["g"] = torch.full((T, H), -0.01)
            x["g"][9::37] = -torch.linspace(1.0, 140.0, H)
        f = {n: t.double() for n, t in x.items()}
        S = torch.zeros(H, 128, 128, dtype=torch.float64)
        ref, size = torch.empty(T, H, 128, dtype=torch.float64), torch.empty(T, H, dtype=torch.float64)
        for t in range(T):
            S, ref[t] = U.step(S, f["q"][t], f["k"][t], f["v"][t], f["g"][t], f["beta"][t], 1.0)
            size[t] = S.flatten(1).norm(dim=1)
        for algo in algos_for("bf16", 128, 128):
            o, st = run_prefill(K, x, [T], torch.zeros(1, H, 128, 128), None, [0], algo, 1.0)
            off = (o.double().cpu() - ref).norm(dim=-1)
            assert bool((off <= 2.0 ** -8 * (ref.norm(dim=-1) + 2 * size) + TOL_F32 * size).all())
            off = (st[0].double().cpu() - S).flatten(1).norm(dim=1)
            assert bool((off <= TOL_TC_S * size[-1]).all())


def test_prefill_growing_states(K):
    """Log-decays of either sign (the sum over a chunk stays small)."""
    x = U.tokens((150,), 1, 2, 128, 128, torch.bfloat16, seed=61)
    x["g"] = torch.sin(torch.arange(150.0))[:, None] * torch.tensor([0.5, 3.0])
    state = U.pool(2, 2, 128, 128, seed=62)
    for algo in algos_for("bf16", 128, 128):
        check_prefill(K, x, [150], 2, state, [0], [1], 1.0, "bf16", algo)


def test_prefill_nan_decay_reaches_what_follows(K):
    """A NaN among one head's log-decays: its outputs and state from there on are NaN, the
    chunks before it and the other head are bit-equal to a clean run."""
    x = U.tokens((200,), 1, 2, 128, 128, torch.bfloat16, seed=63)
    y = {n: t.clone() for n, t in x.items()}
    y["g"][70, 1] = float("nan")
    state = U.pool(2, 2, 128, 128, seed=64)
    for algo in algos_for("bf16", 128, 128):
        a, Sa = run_prefill(K, x, [200], state, [0], [1], algo, 1.0)
        b, Sb = run_prefill(K, y, [200], state, [0], [1], algo, 1.0)
        assert torch.equal(a[:, 0], b[:, 0]) and torch.equal(Sa[1, 0], Sb[1, 0])
        assert torch.equal(a[:64, 1], b[:64, 1])
        assert bool(torch.isnan(b[70:, 1]).all()) and bool(torch.isnan(Sb[1, 1]).all())


@pytest.mark.parametrize("N", [511, 513, 700])
def test_prefill_many_sequences(K, N):
    """More sequences than the launch orders by length."""
    lens = [(7 * n) % 4 for n in range(N)]
    lens[N // 2] = 70
    x = U.tokens((sum(lens),), 1, 1, 128, 128, torch.bfloat16, seed=N)
    state = U.pool(N, 1, 128, 128, seed=65)
    rows = list(range(N))
    for algo in algos_for("bf16", 128, 128):
        check_prefill(K, x, lens, 1, state, rows, rows, 1.0, "bf16", algo)


def test_prefill_no_tokens_passes_states_through(K):
    for dtype, d in (("bf16", 128), ("f32", 32)):
        x = U.tokens((0,), 1, 2, d, d, DT[dtype], seed=66)
        state = U.pool(6, 2, d, d, seed=67)
        for algo in algos_for(dtype, d, d):
            _, S = run_prefill(K, x, [0, 0, 0], state, [0, 5, -1], [3, 5, 2], algo, 1.0)
            want = state.clone()
            want[3], want[2] = state[0], 0.0
            assert torch.equal(S.cpu(), want)


def test_prefill_captured_and_replayed(K):
    """A captured call over a padded batch serves other lengths and inputs on replay; -1 in
    the unused entries."""
    cap, N = 300, 5
    state = U.pool(8, 2, 128, 128, seed=68)
    for algo in algos_for("bf16", 128, 128):
        d = {n: t.cuda() for n, t in U.tokens((cap,), 1, 2, 128, 128, torch.bfloat16, seed=69).items()}
        cu, src, dst = i32([0] * (N + 1)), i32([-1] * N), i32([-1] * N)
        st, o = state.cuda(), torch.empty_like(d["v"])

        def call():
            K.kda_gdr_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, state=st, src_slots=src,
                              dst_slots=dst, o=o, algo=algo)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for seed, lens in ((70, [100, 30, 1]), (71, [64, 64, 65, 0, 80])):
            x = U.tokens((cap,), 1, 2, 128, 128, torch.bfloat16, seed=seed)
            for n in d:
                d[n].copy_(x[n])
            m = len(lens)
            rows, to = [0, 1, -1, 3, 4][:m], [0, 7, 2, 5, 6][:m]
            cu.copy_(U.cu_of(lens + [0] * (N - m)))
            src.copy_(torch.tensor(rows + [-1] * (N - m)))
            dst.copy_(torch.tensor(to + [-1] * (N - m)))
            st.copy_(state)
            o.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            ref_o, ref_S = U.reference(x, spans_of(lens), 2, 1.0, state, rows, to)
            T = sum(lens)
            tc = algo == "tensor_core"
            assert U.max_err(o[:T], ref_o[:T]) <= (TOL_TC if tc else TOL_O["bf16"])
            assert bool((o[T:] == 7.0).all())
            assert U.max_err(st, ref_S) <= (TOL_TC_S if tc else TOL_F32)


@pytest.mark.parametrize("B,H", [(1, 1), (13, 17), (37, 6), (1, 222), (64, 5)])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_decode_batch_sizes(K, B, H, dv):
    """Both divisions of a step over the device, at the sizes where they change."""
    x = U.tokens((B,), 1, H, 64, dv, torch.float32, seed=B)
    state = U.pool(2 * B, H, 64, dv, seed=72)
    src, dst = list(range(B)), list(range(B, 2 * B))
    st, d = state.cuda(), dev(x)
    o = K.kda_gdr_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], st, src_slots=i32(src), dst_slots=i32(dst))
    ref_o, ref_S = U.reference(x, [(b, 1) for b in src], H, 1.0, state, src, dst)
    assert U.max_err(o, ref_o) <= TOL_F32 and U.max_err(st, ref_S) <= TOL_F32


def test_decode_graphs_share_nothing(K):
    """Two captured steps over one pool, replayed on two streams: no scratch in common."""
    H = 4
    pools = [U.pool(3, H, 128, 128, seed=s) for s in (73, 74)]
    runs = []
    for i, p in enumerate(pools):
        x = U.tokens((3 * 4,), 2, H, 128, 128, torch.bfloat16, seed=75 + i)
        d = {n: t.cuda().view(3, 4, *t.shape[1:]) for n, t in x.items()}
        st, o, s = p.cuda(), torch.empty_like(d["v"]), torch.cuda.Stream()

        def call(d=d, st=st, o=o):
            K.kda_gdr_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], st, o=o)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            call()
        runs.append((x, p, st, o, s, graph))
    for x, p, st, o, s, graph in runs:
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for x, p, st, o, s, graph in runs:
        rows = [0, 1, 2]
        ref_o, ref_S = U.reference(x, [(4 * b, 4) for b in rows], H, 1.0, p, rows, rows)
        assert U.max_err(o.view(12, H, 128), ref_o) <= TOL_O["bf16"] and U.max_err(st, ref_S) <= TOL_F32


@pytest.mark.parametrize("T", [23, 9000])
def test_plan_in_place_head_and_odd_addresses(K, T):
    """free_head advanced in place; token outputs that are not 16-byte aligned."""
    new, ctx, bs = [20, 3, T - 23], [0, 14, 5], 16
    cols, free = -(-(T + 30) // bs), list(range(T))
    table = [[500 + n if j < -(-ctx[n] // bs) else -7 for j in range(cols)] for n in range(3)]
    ref = U.plan_reference(new, ctx, free, 1, table, bs, T)
    t = plan_tensors(new, ctx, free, 1, table)
    pos = torch.empty(T + 1, dtype=torch.int32, device="cuda")[1:]
    slots = torch.empty(T + 1, dtype=torch.int64, device="cuda")[1:]
    out = K.BlockPlan(i32([0] * 4), pos, slots, i32([0] * 3), i32([0] * 3), t[3])
    p = K.kda_block_plan(t[0], t[1], t[2], t[3], t[4], bs, T, out=out)
    got = [p.cu_seqlens, p.positions, p.token_slots, p.src_slots, p.dst_slots, t[3], t[4]]
    for g, r in zip(got, [*ref[:5], [ref[5]], ref[6]]):
        assert g.tolist() == r


def test_plan_far_positions(K):
    """Contexts whose ends pass 31 bits: no block there, nothing is read out of range."""
    new, ctx = [2 ** 31 - 1, 5], [2 ** 31 - 1, 2 ** 31 - 3]
    t = plan_tensors(new, ctx, [4, 5], 0, [[1, 2], [3, 4]])
    p = K.kda_block_plan(*t, 64, 8)
    assert p.cu_seqlens.tolist() == [0, 2 ** 31 - 1, 2 ** 31 - 1]
    assert t[4].tolist() == [[1, 2], [3, 4]]
    assert p.token_slots.tolist() == [-1] * 8
    assert p.src_slots.tolist() == [-1, -1] and p.dst_slots.tolist() == [-1, -1]


def test_binding_checks_shapes(K):
    """Wrong shapes, types and layouts are refused before a launch."""
    d = dev(U.tokens((6,), 2, 4, 64, 64, torch.float32, seed=80))
    cu, st = i32([0, 6]), torch.zeros(2, 4, 64, 64, device="cuda")
    args = dict(q=d["q"], k=d["k"], v=d["v"], g=d["g"], beta=d["beta"], cu_seqlens=cu, state=st,
                src_slots=i32([0]), dst_slots=i32([1]))
    K.kda_gdr_prefill(**args)
    bad = [dict(k=d["k"][:5]), dict(v=d["v"][:5]), dict(v=d["v"].bfloat16()), dict(g=d["g"][:, :3]),
           dict(g=d["g"].double()), dict(beta=d["beta"].t()), dict(cu_seqlens=cu.long()),
           dict(cu_seqlens=cu.view(1, 2)), dict(state=st[:, :2]), dict(state=st.transpose(2, 3)),
           dict(src_slots=i32([0, 1])), dict(dst_slots=i32([0]).long()), dict(ctx_lens=i32([0, 1])),
           dict(q=d["q"].half(), k=d["k"].half()), dict(o=torch.empty_like(d["q"])),
           dict(block_table=i32([[0], [1]]), block_size=64),
           dict(cu_seqlens_host=torch.tensor([0, 3, 6], dtype=torch.int32)), dict(cu_seqlens_host=cu)]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            K.kda_gdr_prefill(**{**args, **kw})
    with pytest.raises(K.KdaError):
        K.kda_gdr_prefill(**{**args, "block_table": i32([[0]]), "block_size": 32})
    args.pop("cu_seqlens")
    st6 = torch.zeros(6, 4, 64, 64, device="cuda")
    args.update(state=st6, src_slots=None, dst_slots=None)
    K.kda_gdr_decode(**args)
    for kw in [dict(v=d["v"][:5]), dict(g=d["g"][:5]), dict(num_tokens=i32([1])), dict(state=st6[:, :2]),
               dict(src_slots=i32([0])), dict(o=torch.empty_like(d["q"]))]:
        with pytest.raises((ValueError, TypeError)):
            K.kda_gdr_decode(**{**args, **kw})
    with pytest.raises(K.KdaError):       # fewer rows than sequences, none named
        K.kda_gdr_decode(**{**args, "state": st})


SPLITS = [([1100], 2), ([2000], 16), ([1030, 1, 0, 700], 3), ([1500, 1400], 8), ([3300], 1)]


@pytest.mark.parametrize("lens,H", SPLITS, ids=str)
@pytest.mark.parametrize("block", [0, 128])
def test_prefill_few_chains(K, lens, H, block):
    """Long sequences of few heads, divided along their length: outputs, last rows and block
    rows as ever, with and without the host's offsets, in place, with heads of every decay."""
    N, T = len(lens), sum(lens)
    ctx = [37 * n for n in range(N)]
    x = U.tokens((T + 9,), 1, H, 128, 128, torch.bfloat16, seed=T, rate=(1e-4, 2.0))
    cols = max((c + n) // 128 for c, n in zip(ctx, lens)) + 1
    state = U.pool(2 * N + N * cols, H, 128, 128, seed=90)
    table = torch.arange(2 * N, 2 * N + N * cols, dtype=torch.int32).view(N, cols) if block else None
    src = [n if n != 1 else -1 for n in range(N)]
    for dst in ([N + n for n in range(N)], list(range(N))):      # other rows; in place
        if dst[0] == 0 and block:                                # and a block's row is the one read
            table[0, (ctx[0] + lens[0]) // 128 - 1] = 0
            dst[0] = -1
        for host, pad in ((True, 0), (False, 9)):
            y = x if pad else {n: t[:T].contiguous() for n, t in x.items()}
            check_prefill(K, y, lens, H, state, src, dst, 0.5, "bf16", "tensor_core", ctx=ctx, table=table,
                          block=block, host=host, pad=pad)


def test_prefill_few_chains_shorter_on_the_device(K):
    """Segments are planned from the host's lengths; the device's decide."""
    cap, H = 4000, 2
    x = U.tokens((cap,), 1, H, 128, 128, torch.bfloat16, seed=91)
    d, state = dev(x), U.pool(2, H, 128, 128, seed=92)
    for L in (0, 1, 64, 65, 700, 2049, 4000):
        o, st = torch.full_like(d["v"], 7.0), state.cuda()
        K.kda_gdr_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], i32([0, L]), state=st,
                          src_slots=i32([0]), dst_slots=i32([1]), o=o)
        ref_o, ref_S = U.reference(x, [(0, L)], H, 1.0, state, [0], [1])
        assert U.max_err(o[:L], ref_o[:L]) <= TOL_TC and bool((o[L:] == 7.0).all())
        assert U.max_err(st, ref_S) <= TOL_TC_S
    assert K.kda_device_status() == 0


def test_prefill_few_chains_nan_and_infinity_stay_in_their_columns(K):
    """An infinity in v spoils its column from its token on, across segments, and no other."""
    x = U.tokens((2500,), 1, 2, 128, 128, torch.bfloat16, seed=93)
    y = {n: t.clone() for n, t in x.items()}
    y["v"][300, 1, 5], y["v"][1700, 0, 9] = float("inf"), float("nan")
    state = U.pool(2, 2, 128, 128, seed=94)
    a, Sa = run_prefill(K, x, [2500], state, [0], [1], "tensor_core", 1.0)
    b, Sb = run_prefill(K, y, [2500], state, [0], [1], "tensor_core", 1.0)
    bad = torch.zeros_like(a, dtype=torch.bool)
    bad[256:, 1, 5], bad[1600:, 0, 9] = True, True
    assert torch.equal(a[~bad], b[~bad])
    assert not bool(torch.isfinite(b[1900:, 1, 5]).any()) and not bool(torch.isfinite(b[1900:, 0, 9]).any())
    ok = torch.ones(2, 128, 128, dtype=torch.bool)
    ok[1, :, 5], ok[0, :, 9] = False, False
    assert torch.equal(Sa[1].cpu()[ok], Sb[1].cpu()[ok])


def test_prefill_workspace_is_checked(K):
    x = dev(U.tokens((2000,), 1, 1, 128, 128, torch.bfloat16, seed=95))
    cu = i32([0, 2000])
    need = K.kda_gdr_prefill_workspace_size(2000, 1, 1, 1, 128, 128)
    assert need > 0 and K.kda_gdr_prefill_workspace_size(2000, 1, 1, 1, 128, 128, algo="cuda_core") == 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a = K.kda_gdr_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, workspace=ws)
    ws.fill_(0xFF)             # (NaN) nothing is kept there between calls
    b = K.kda_gdr_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, workspace=ws)
    assert torch.equal(a, b)
    small, other = torch.empty(64, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    c = K.kda_gdr_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, workspace=small)   # replaced
    assert torch.equal(a, c)
    c.zero_()
    torch.cuda.synchronize()
    K.kda_gdr_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, o=c, stream=other)
    other.synchronize()
    assert torch.equal(a, c)


@pytest.mark.parametrize("block", [0, 64])
def test_prefill_a_few_tokens_each(K, block):
    """Sequences of no, one and a few tokens beside longer ones, at and across block ends."""
    lens, ctx = [1, 3, 2, 0, 4, 5, 70, 1, 3, 2], [63, 62, 64, 10, 60, 0, 3, 0, 127, 126]
    N, H = len(lens), 3
    x = U.tokens((sum(lens),), 1, H, 128, 128, torch.bfloat16, seed=96)
    state = U.pool(2 * N + 3 * N, H, 128, 128, seed=97)
    table = torch.arange(2 * N, 5 * N, dtype=torch.int32).view(N, 3) if block else None
    src = [n if n != 2 else -1 for n in range(N)]
    for dst in ([N + n for n in range(N)], list(range(N))):
        for algo in algos_for("bf16", 128, 128):
            check_prefill(K, x, lens, H, state, src, dst, 0.5, "bf16", algo, ctx=ctx, table=table, block=block)


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("bf16", 64, 32), ("f32", 32, 64)])
def test_decode_more_states_than_fit_at_once(K, dtype, dk, dv):
    """Several tokens each of more states than the device holds at once, of 0 .. Tq tokens, with
    rows missing and states passed through."""
    B, Tq, Hk, H = 60, 5, 6, 24
    x = U.tokens((B * Tq,), Hk, H, dk, dv, DT[dtype], seed=98)
    state = U.pool(2 * B, H, dk, dv, seed=99)
    nt = [(3 * b) % (Tq + 1) for b in range(B)]
    src = [b if b % 7 else -1 for b in range(B)]
    dst = [B + b if b % 5 else (-1 if b % 2 else b) for b in range(B)]
    d = {n: t.cuda().view(B, Tq, *t.shape[1:]) for n, t in x.items()}
    ref_o, ref_S = U.reference(x, [(b * Tq, nt[b]) for b in range(B)], H, 0.7, state, src, dst)
    live = torch.isfinite(ref_o)
    ref_o = torch.where(live, ref_o, torch.full_like(ref_o, 7.0))
    st, o = state.cuda(), torch.full_like(d["v"], 7.0)
    K.kda_gdr_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], st, src_slots=i32(src), dst_slots=i32(dst),
                     num_tokens=i32(nt), scale=0.7, o=o)
    flat = o.view(B * Tq, H, dv).cpu()
    assert bool((flat[~live] == 7.0).all()) and U.max_err(flat, ref_o) <= TOL_O[dtype]
    assert U.max_err(st, ref_S) <= TOL_F32
    kept = [r for r in range(2 * B) if r not in dst]
    assert torch.equal(st[kept].cpu(), state[kept])


def test_prefill_fills_the_device(K):
    """As many (sequence, head) pairs as SMs, with ends inside every 16-token tile."""
    lens, H = [77, 121, 150], 49
    x = U.tokens((sum(lens),), 7, H, 128, 128, torch.bfloat16, seed=100)
    state = U.pool(6, H, 128, 128, seed=101)
    for algo in algos_for("bf16", 128, 128):
        check_prefill(K, x, lens, H, state, [0, 1, 2], [3, 4, 5], 0.5, "bf16", algo)


def test_empty_batches(K):
    """No requests, no sequences, no tokens: nothing is read or written past the fixed outputs."""
    none, head = torch.zeros(0, dtype=torch.int32, device="cuda"), i32([3])
    p = K.kda_block_plan(none, none, i32([5, 6]), head, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 16, 5)
    assert p.cu_seqlens.tolist() == [0] and p.free_head.tolist() == [3]
    assert p.positions.tolist() == [-1] * 5 and p.token_slots.tolist() == [-1] * 5
    p = K.kda_block_plan(i32([0, 0]), None, none, i32([0]), i32([[7], [8]]), 16, 0)
    assert p.cu_seqlens.tolist() == [0, 0, 0] and p.dst_slots.tolist() == [-1, -1]
    for dt, d in ((torch.bfloat16, 128), (torch.float32, 64)):
        e, st = dev(U.tokens((0,), 1, 2, d, d, dt, seed=1)), torch.ones(2, 2, d, d, device="cuda")
        o = K.kda_gdr_decode(e["q"], e["k"], e["v"], e["g"], e["beta"], st)
        assert o.shape == (0, 2, d)
        o = K.kda_gdr_prefill(e["q"], e["k"], e["v"], e["g"], e["beta"], i32([0]), state=st)
        assert o.shape == (0, 2, d) and bool((st == 1.0).all())


@pytest.mark.parametrize("L,H", [(1100, 2), (4500, 1), (3000, 16)])
@pytest.mark.parametrize("what", ["one row", "last row", "two in turn"])
def test_prefill_few_chains_rows_written_again(K, L, H, what):
    """A sequence whose blocks share rows, or whose last state goes to an earlier block's row: the
    latest token's state stays, although the segments run at once."""
    block, ctx = 128, 70
    cols = (ctx + L) // block + 1
    x = U.tokens((L,), 1, H, 128, 128, torch.bfloat16, seed=L, rate=(1e-3, 0.5))
    state = U.pool(6, H, 128, 128, seed=102)
    table, dst = torch.full((1, cols), 2, dtype=torch.int32), 3
    if what == "last row":
        table[0, 1::2], dst = 4, 2
    elif what == "two in turn":
        table[0, 1::2] = 4
        table[0, -1] = 5             # (the block that this call leaves unfinished)
    for host in (True, False):
        for _ in range(3):
            check_prefill(K, x, [L], H, state, [0], [dst], 1.0, "bf16", "tensor_core", ctx=[ctx],
                          table=table, block=block, host=host)


def stream_calls(K):
    """Every call that makes its own outputs, with the bytes of each output."""
    x = dev(U.tokens((2000,), 1, 1, 128, 128, torch.bfloat16, seed=103))
    one = {n: t[:512].view(64, 8, *t.shape[1:]) for n, t in x.items()}
    pool = torch.zeros(64, 1, 128, 128, device="cuda")
    cu, lens, A = i32([0, 2000]), i32([1000] * 2), torch.zeros(1, 128, device="cuda")
    free, head, table = i32(range(100)), i32([0]), i32([[-1] * 40] * 2)
    z = x["k"]
    return {
        "gdr_prefill": lambda s: [K.kda_gdr_prefill(*x.values(), cu, stream=s)],
        "gdr_decode": lambda s: [K.kda_gdr_decode(*one.values(), pool, stream=s)],
        "block_plan": lambda s: [t for n, t in K.kda_block_plan(
            lens, None, free, head, table, 64, 2000, stream=s)._asdict().items() if n in ("positions", "token_slots")],
        "prefill": lambda s: K.kda_prefill(x["q"], z, x["v"], z, A, x["beta"], cu, stream=s),
        "prefill_noalloc": lambda s: K.kda_prefill_noalloc(x["q"], z, x["v"], z, A, x["beta"], cu, stream=s),
        "prefill_checkpointed": lambda s: K.kda_prefill_checkpointed(
            x["q"], z, x["v"], z, A, x["beta"], cu, torch.tensor([0, 2000]), 512, stream=s),
        "decode_multi": lambda s: [K.kda_decode_multi(one["q"], one["k"], one["v"], one["k"], A, one["beta"], pool,
                                                      stream=s)],
        "decode_step": lambda s: [K.kda_decode_step(x["q"][:64], z[:64], x["v"][:64], z[:64], A, x["beta"][:64], pool,
                                                    stream=s)],
    }


@pytest.mark.parametrize("name", ["gdr_prefill", "gdr_decode", "block_plan", "prefill", "prefill_noalloc",
                                  "prefill_checkpointed", "decode_multi", "decode_step"])
def test_outputs_belong_to_the_stream_that_writes_them(K, name):
    """A call on another stream whose results are dropped at once: tensors that the current stream
    makes and fills meanwhile keep their values."""
    call, s = stream_calls(K)[name], torch.cuda.Stream()
    want = [t.clone() for t in call(None)]           # (and buffers of these sizes in the current stream's cache)
    sizes = [t.numel() * t.element_size() for t in want]
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                # about 10 ms, in front of the call's kernels
    outs = call(s)
    where = {t.untyped_storage().data_ptr() for t in outs}
    del outs
    mine = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    assert not where & {t.untyped_storage().data_ptr() for t in mine}
    torch.cuda.synchronize()
    assert all(bool((t == 77).all()) for t in mine)
    with torch.cuda.stream(s):                       # and the call itself is the same there
        got = [t.clone() for t in call(s)]
    torch.cuda.synchronize()
    if name in ("gdr_prefill", "prefill", "prefill_noalloc", "prefill_checkpointed"):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert K.kda_device_status() == 0


def test_plan_largest_table(K):
    """All 2^31 - 1 entries of a table newly reached in one call: every one is written, and
    nothing in front of the table or behind it."""
    cols, guard = 2 ** 31 - 1, 4096
    buf = torch.full((cols + 2 * guard,), 7, dtype=torch.int32, device="cuda")
    table = buf[guard:guard + cols].view(1, cols)
    p = K.kda_block_plan(i32([cols]), None, i32([5, 6, 4]), i32([0]), table, 1, 4)
    torch.cuda.synchronize()
    assert p.cu_seqlens.tolist() == [0, cols] and p.free_head.tolist() == [cols]
    assert p.src_slots.tolist() == [-1] and p.dst_slots.tolist() == [-1]
    assert p.positions.tolist() == [0, 1, 2, 3] and p.token_slots.tolist() == [5, 6, 4, -1]
    assert buf[:guard + 3].tolist() == [7] * guard + [5, 6, 4] and bool((buf[guard + cols:] == 7).all())
    rest = buf[guard + 3:guard + cols]
    assert int(rest.min()) == -1 and int(rest.max()) == -1


@pytest.mark.parametrize("Tq,block", [(1, 1), (1, 64), (2, 64), (4, 3), (5, 5), (9, 1), (64, 16), (64, 1000)])
@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("f32", 128, 64), ("f32", 32, 32), ("bf16", 64, 128)])
def test_decode_block_rows(K, Tq, block, dtype, dk, dv):
    """A few tokens at and across block ends: every completed block's row keeps the state at its
    end; rows outside the pool, columns past the table and unfinished blocks get none."""
    B, Hk, H = 7, 2, 4
    x = U.tokens((B * Tq,), Hk, H, dk, dv, DT[dtype], seed=104 + Tq)
    nt = [Tq, 0, (Tq + 1) // 2, Tq, Tq, 1, Tq]
    ctx = [0, 2 * block - 1, block - 1, -5, max(2 * block - 2, 0), 3 * block - 1, 5]
    pos = [max(c, 0) for c in ctx]
    cols = max((c + n) // block for c, n in zip(pos, nt)) + 1
    state = U.pool(2 * B + B * cols + 1, H, dk, dv, seed=105)
    table = torch.arange(2 * B, 2 * B + B * cols, dtype=torch.int32).view(B, cols)
    table[3, 0], table[4, -1] = -1, state.shape[0]
    if cols > 1:
        table[6] = table[6, 0]                     # every block under one row: the latest state stays
    src = [0, 1, -1, 3, 4, 5, 6]
    d = {n: t.cuda().view(B, Tq, *t.shape[1:]) for n, t in x.items()}
    spans = [(b * Tq, nt[b]) for b in range(B)]
    in_place = [0, 1, -1, 3, int(table[4, pos[4] // block]), 5, 6]
    for dst in ([B + b for b in range(B)], in_place, None):
        for short in (0, 1):
            tab = table[:, :cols - short].contiguous()
            if tab.shape[1] == 0:
                continue
            ref_o, ref_S = U.reference(x, spans, H, 0.7, state, src, src if dst is None else dst, pos, tab, block)
            live = torch.isfinite(ref_o)
            st, o = state.cuda(), torch.full_like(d["v"], 7.0)
            K.kda_gdr_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], st, src_slots=i32(src), dst_slots=i32(dst),
                             num_tokens=i32(nt), scale=0.7, o=o, ctx_lens=i32(ctx), block_table=i32(tab),
                             block_size=block)
            flat = o.view(B * Tq, H, dv).cpu()
            assert bool((flat[~live] == 7.0).all())
            assert U.max_err(flat[live], ref_o[live]) <= TOL_O[dtype]
            for r in range(state.shape[0]):
                if torch.equal(ref_S[r], state[r].double()):
                    assert torch.equal(st[r].cpu(), state[r]), r
                else:
                    assert U.max_err(st[r], ref_S[r]) <= TOL_F32, r


def test_decode_block_rows_leave_results_alone(K):
    """The same outputs and last rows, bit by bit, with and without blocks; no context is position 0."""
    B, Tq, H = 40, 6, 24
    x = U.tokens((B * Tq,), 6, H, 128, 128, torch.bfloat16, seed=106)
    d = {n: t.cuda().view(B, Tq, *t.shape[1:]) for n, t in x.items()}
    state = U.pool(3 * B, H, 128, 128, seed=107)
    table = torch.arange(B, 3 * B, dtype=torch.int32).view(B, 2)
    for tq in (1, Tq):
        y = {n: t[:, :tq].contiguous() for n, t in d.items()}
        a, b, c = state.cuda(), state.cuda(), state.cuda()
        oa = K.kda_gdr_decode(*y.values(), a)
        ob = K.kda_gdr_decode(*y.values(), b, block_table=i32(table), block_size=3)
        oc = K.kda_gdr_decode(*y.values(), c, ctx_lens=i32([0] * B), block_table=i32(table), block_size=3)
        assert torch.equal(oa, ob) and torch.equal(a[:B], b[:B]) and torch.equal(b, c)
        if tq == 1:
            assert torch.equal(b[B:].cpu(), state[B:])
        else:                                       # the second block ends with the call
            assert torch.equal(b[B + 1::2], a[:B]) and not torch.equal(b[B::2].cpu(), state[B::2])


@pytest.mark.parametrize("graph", [False, True])
def test_verify_and_replay_run_across_block_ends(K, graph):
    """Plan -> prefill -> (verify of the drafts -> plan of the accepted ones -> replay) ...: every
    completed block's row and the last rows equal the plain form."""
    prompt, steps, Tq, H, block = [62, 128, 1, 191], 20, 4, 2, 64
    N = len(prompt)
    gen = torch.Generator().manual_seed(108)
    acc = torch.randint(0, Tq + 1, (steps, N), generator=gen)
    acc[0], acc[1] = torch.tensor([4, 1, 4, 0]), torch.tensor([0, 4, 4, 3])
    total = [prompt[n] + int(acc[:, n].sum()) for n in range(N)]
    room = [t + Tq for t in total]                   # drafts behind the last accepted token
    x = U.tokens((sum(room),), 1, H, 128, 128, torch.bfloat16, seed=109)
    start = U.cu_of(room).tolist()[:N]
    need = sum(-(-t // block) for t in total)
    cols = max(-(-t // block) for t in total) + 1
    ref_table, at = torch.full((N, cols), -1, dtype=torch.int32), 0
    for n, t in enumerate(total):
        ref_table[n, :-(-t // block)] = torch.arange(at, at - (-t // block))
        at += -(-t // block)
    last = [int(ref_table[n, (t - 1) // block]) for n, t in enumerate(total)]
    ref_o, ref_S = U.reference(x, list(zip(start, total)), H, 0.5, torch.zeros(need, H, 128, 128), None, last, None,
                               ref_table, block)
    d = dev(x)
    table = torch.full((N, cols), -1, dtype=torch.int32, device="cuda")
    free, head = torch.randperm(need, generator=gen).to(torch.int32).cuda(), i32([0])
    pool = torch.full((need, H, 128, 128), float("nan"), device="cuda")
    new, ctx = i32(prompt), i32([0] * N)
    p = K.kda_block_plan(new, ctx, free, head, table, block, sum(prompt))
    idx = torch.cat([torch.arange(start[n], start[n] + prompt[n]) for n in range(N)]).cuda()
    K.kda_gdr_prefill(*(t[idx].contiguous() for t in d.values()), p.cu_seqlens, state=pool, src_slots=p.src_slots,
                      dst_slots=p.dst_slots, ctx_lens=ctx, block_table=table, block_size=block, scale=0.5)
    head.copy_(p.free_head)
    ctx.copy_(new)
    tok = {n: torch.empty(N, Tq, *t.shape[1:], dtype=t.dtype, device="cuda") for n, t in d.items()}
    drafts, plan = torch.empty_like(tok["v"]), p._replace(
        positions=torch.empty(N * Tq, dtype=torch.int32, device="cuda"),
        token_slots=torch.empty(N * Tq, dtype=torch.int64, device="cuda"), free_head=head)

    def step():
        K.kda_gdr_decode(*tok.values(), pool, src_slots=plan.dst_slots, update_state=False, scale=0.5, o=drafts)
        K.kda_block_plan(new, ctx, free, head, table, block, N * Tq, out=plan)
        K.kda_gdr_decode(*tok.values(), pool, src_slots=plan.src_slots, dst_slots=plan.dst_slots, num_tokens=new,
                         want_outputs=False, ctx_lens=ctx, block_table=table, block_size=block)
        ctx.add_(new)

    run = step
    if graph:
        keep = [t.clone() for t in (ctx, head, table, pool)]
        new.zero_()                                  # (the warm-up adds nothing)
        for t in tok.values():
            t.zero_()
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
        for t, k in zip((ctx, head, table, pool), keep):
            assert torch.equal(t.nan_to_num(9.0), k.nan_to_num(9.0))
    for i in range(steps):
        at = torch.tensor(start).cuda()[:, None] + ctx[:, None] + torch.arange(Tq).cuda()
        for n, t in d.items():
            tok[n].copy_(t[at])
        new.copy_(acc[i])
        run()
        for n in range(N):
            a, b = int(at[n, 0]), int(acc[i, n])
            if b:
                assert U.max_err(drafts[n, :b], ref_o[a:a + b]) <= TOL_TC
    torch.cuda.synchronize()
    assert ctx.tolist() == total and int(head) == need
    for n, t in enumerate(total):
        for j in range(-(-t // block)):
            assert U.max_err(pool[int(table[n, j])], ref_S[int(ref_table[n, j])]) <= TOL_TC_S, (n, j)


def test_decode_blocks_checks(K):
    d = dev(U.tokens((3,), 1, 2, 64, 64, torch.float32, seed=110))
    st, args = torch.zeros(3, 2, 64, 64, device="cuda"), list(d.values())
    ok = dict(block_table=i32([[0]] * 3), block_size=2, ctx_lens=i32([0, 1, 1]))
    K.kda_gdr_decode(*args, st, **ok)
    for kw in [dict(update_state=False), dict(block_table=i32([[0]])), dict(block_table=i32([[0]] * 3).long()),
               dict(ctx_lens=i32([0])), dict(ctx_lens=torch.zeros(3, device="cuda"))]:
        with pytest.raises(ValueError):
            K.kda_gdr_decode(*args, st, **{**ok, **kw})
    for kw in [dict(block_table=None), dict(block_size=-2)]:
        with pytest.raises(K.KdaError):
            K.kda_gdr_decode(*args, st, **{**ok, **kw})


def test_empty_verify(K):
    for dt, d in ((torch.bfloat16, 128), (torch.float32, 64)):
        st = torch.ones(2, 2, d, d, device="cuda")
        for lead in ((0,), (0, 4)):
            e = dev(U.tokens(lead, 1, 2, d, d, dt, seed=1))
            assert K.kda_gdr_decode(*e.values(), st, update_state=False).shape == (*lead, 2, d)
            table = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
            assert K.kda_gdr_decode(*e.values(), st, block_table=table, block_size=4).shape == (*lead, 2, d)
        assert bool((st == 1.0).all())


def test_empty_prefill(K):
    for dt, d in ((torch.bfloat16, 128), (torch.float32, 64)):
        st, table = torch.ones(2, 2, d, d, device="cuda"), torch.zeros(0, 3, dtype=torch.int32, device="cuda")
        for T in (0, 2000):
            e = dev(U.tokens((T,), 1, 2, d, d, dt, seed=1))
            o = torch.full_like(e["v"], 7.0)
            K.kda_gdr_prefill(*e.values(), i32([0]), state=st, block_table=table, block_size=64, o=o)
            assert bool((o == 7.0).all()) and bool((st == 1.0).all())


@pytest.mark.parametrize("e", [-20, -16, 0, 20])
@pytest.mark.parametrize("what", ["few bits", "many bits", "single steep tokens", "rates", "rates, small betas"])
def test_prefill_small_and_large_values(K, e, what):
    """The rule is linear in v and S: with both scaled by 2^e every output row and every head's
    state stay within the same roundings, relative to their own size, in heads of every decay."""
    T, H = 200, 32
    x = U.tokens((T,), H, H, 128, 128, torch.bfloat16, seed=111)
    lo, hi = (4.0, 256.0) if what == "few bits" else (90.0, 400.0)
    x["g"] = (-torch.linspace(lo, hi, H) / 64 * 0.6931472).expand(T, H).contiguous()
    if what == "single steep tokens":
        x["g"] = torch.full((T, H), -0.01)
        x["g"][9::37] = -torch.linspace(1.0, 140.0, H)
    elif what.startswith("rates"):
        gen = torch.Generator().manual_seed(113)
        rate = torch.exp(torch.rand(H, generator=gen) * 3 - 0.5)
        x["g"] = -rate * torch.nn.functional.softplus(torch.randn(T, H, generator=gen))
        if "betas" in what:
            x["beta"] = torch.sigmoid(3 * torch.randn(T, H, generator=gen) - 2)
    x["v"] = (x["v"].float() * 2.0 ** e).bfloat16()
    state = U.pool(1, H, 128, 128, seed=112, std=1.0) * 2.0 ** e
    f = {n: t.double() for n, t in x.items()}
    S = state[0].double()
    ref, size = torch.empty(T, H, 128, dtype=torch.float64), torch.empty(T, H, dtype=torch.float64)
    for t in range(T):
        S, ref[t] = U.step(S, f["q"][t], f["k"][t], f["v"][t], f["g"][t], f["beta"][t], 1.0)
        size[t] = S.flatten(1).norm(dim=1)
    for algo in algos_for("bf16", 128, 128):
        o, st = run_prefill(K, x, [T], state, [0], [0], algo, 1.0)
        off = (o.double().cpu() - ref).norm(dim=-1)
        assert bool((off <= 2.0 ** -8 * (ref.norm(dim=-1) + 2 * size) + TOL_F32 * size).all())
        off = (st[0].double().cpu() - S).flatten(1).norm(dim=1)
        assert bool((off <= TOL_TC_S * size[-1]).all())


def keys_around(T, H, cosine, gen):
    """Unit keys of pairwise cosine ``cosine``: a common direction per head and independent rest."""
    m = U.unit(torch.randn(1, H, 128, generator=gen))
    r = torch.randn(T, H, 128, generator=gen)
    r = U.unit(r - (r * m).sum(-1, keepdim=True) * m)
    return cosine ** 0.5 * m + (1 - cosine) ** 0.5 * r


# (cosine, bound of beta |k|^2, log2 of the span of the norms, log2 of v's size, q along the keys,
#  state and output errors that the header states)
STATED = [(0.0, 1.0, 0, 0, False, 2e-5, 3e-3), (0.0, 2.0, 0, 0, False, 2e-5, 3e-3),
          (0.5, 1.0, 0, 0, False, 2e-5, 3e-3), (0.5, 2.0, 0, 0, False, 2e-5, 3e-3),
          (0.5, 1.0, 0, 0, True, 2e-5, 1e-2), (0.5, 2.0, 0, 0, True, 2e-5, 1e-2),
          (0.9, 1.0, 0, 0, False, 5e-5, 1e-2), (0.9, 1.0, 0, 0, True, 5e-5, 1e-2),
          (0.99, 1.0, 0, 0, True, 5e-5, 1e-2), (1.0, 1.0, 0, 0, False, 5e-5, 1e-2),
          (0.0, 1.0, 8, 0, False, 2e-5, 3e-3), (0.0, 2.0, 8, 0, False, 2e-5, 3e-3),
          (0.0, 2.0, 14, 0, False, 1e-3, 3e-3), (0.0, 1.0, 0, 20, False, 2e-5, 3e-3),
          (0.0, 2.0, 8, -20, False, 2e-5, 3e-3), (1.0, 2.0, 0, 0, False, 5e-3, 5e-2),
          (1.0, 2.0, 8, 20, False, 5e-3, 5e-2)]


@pytest.mark.parametrize("cosine,bound,span,size,along,state_tol,o_tol", STATED)
@pytest.mark.parametrize("rate", [(1e-4, 1e-3), (1e-3, 0.5), (0.5, 3.0)], ids=["none", "slow", "fast"])
def test_prefill_stated_accuracy(K, cosine, bound, span, size, along, state_tol, o_tol, rate):
    """What the header says of the tensor-core path's errors, in 2-norm by head, at the edges of the
    ranges that it names; and every output row within 2^-8 of what it reads for cosines up to 0.9."""
    T, H = 400, 4
    gen = torch.Generator().manual_seed(114)
    x = U.tokens((T,), H, H, 128, 128, torch.bfloat16, seed=115, rate=rate)
    k = keys_around(T, H, cosine, gen)
    x["k"] = (k * 2.0 ** (span * (torch.rand(T, H, 1, generator=gen) - 0.5))).bfloat16()
    if along:
        x["q"] = k.bfloat16()
    u = torch.full((T, H), 0.99) if cosine == 1.0 and bound == 2.0 else torch.rand(T, H, generator=gen)
    x["beta"] = bound * u / x["k"].float().square().sum(-1)
    x["v"] = (x["v"].float() * 2.0 ** size).bfloat16()
    if size == 20:
        x["v"] = x["v"].clamp(-2.0 ** 20, 2.0 ** 20)
    state = U.pool(1, H, 128, 128, seed=116, std=1.0) * 2.0 ** size
    f = {n: t.double() for n, t in x.items()}
    S = state[0].double()
    ref, norm = torch.empty(T, H, 128, dtype=torch.float64), torch.empty(T, H, dtype=torch.float64)
    for t in range(T):
        S, ref[t] = U.step(S, f["q"][t], f["k"][t], f["v"][t], f["g"][t], f["beta"][t], 1.0)
        norm[t] = S.flatten(1).norm(dim=1)
    o, st = run_prefill(K, x, [T], state, [0], [0], "tensor_core", 1.0)
    off = o.double().cpu() - ref
    assert bool(((st[0].double().cpu() - S).flatten(1).norm(dim=1) <= state_tol * S.flatten(1).norm(dim=1)).all())
    assert bool((off.norm(dim=(0, 2)) <= o_tol * ref.norm(dim=(0, 2))).all())
    if cosine <= 0.9:
        assert bool((off.norm(dim=-1) <= 2.0 ** -8 * (ref.norm(dim=-1) + 2 * norm)).all())
