"""The paged decode cache on the GPU where it can go wrong: precision behind a prefix, layouts that
only large batches take, error paths, padded prefills. Plain 64-bit arithmetic is the reference;
each tolerance is derived where it stands."""
import math

import pytest
import torch

import oracle
from test_gpu_paged import BF, F32, Cache, P, ints, run_steps  # noqa: F401 (P: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,gate", [(7, True), (20, False), (40, True), (64, False)])
def test_queries_and_weights_meet_the_prefix_in_fp32(P, B, gate, dtype, d):
    """The turned-back query and the softmax weights are fp32 numbers, whatever the type of the
    cache. Values of three keys of a prefix are chosen so that their weighted sum all but vanishes
    in dim b of row b: what is left is the error of the weights, not the rounding of the output.

    w = 0 leaves the state as it is, and one-hot queries and keys make a logit one product
    z = scale G[r, i] c without a sum, G[r, i] being any fp32 number. In log2 units that
    logit is off by 6 steps of 2^-24 relative (two accumulations of parts of G, each cut or rounded
    to 24 bits: 2^-23 each; log2 e, the product and the sum with the gate: 2^-24 each, and 2^-24 in
    reserve), its gate bias by 4 (two products, two sums) and the maxima it is taken against by 4
    (a difference in the tile, one in the join, twice rounded); the exponentials of
    the weight and of the join, with their products, are off by 2^-20 in all."""
    H, page, n, J = 3, 16, 200, (5, 130, 199)
    c = Cache([0] * B, H, d, page, dtype, gate, seed=B + d, prefix=n)
    rng = torch.Generator(device="cuda").manual_seed(B)
    c.state = torch.randn(c.state.shape, device="cuda", generator=rng)
    x = c.step_inputs()
    for name in ("w", "v_new", "k_new", "q"):
        x[name].zero_()
    r = torch.randint(d, (B, H), device="cuda", generator=rng)
    x["q"].scatter_(2, r.unsqueeze(2), 1.0)
    i, size = [3, 17, 50], [1.75, -2.0, 1.5]
    pre, g = c.pages(None), torch.zeros((H, n), dtype=torch.float64, device="cuda")
    for p in pre:
        c.k[p] = 0
        c.v[p] = 0
    for j, key in enumerate(J):
        c.k[pre[key // page], :, key % page, i[j]] = size[j]
    if gate:
        g = c.rows(c.g, None, n)
    S = c.state[c.slot].double().gather(2, r[:, :, None, None].expand(B, H, 1, d)).squeeze(2)  # row r
    z = g.unsqueeze(0).repeat(B, 1, 1)
    for j, key in enumerate(J):
        z[:, :, key] += S[:, :, i[j]] * size[j]
    a, at = z[:, :, list(J)].exp().sort(-1, descending=True)  # weights, and which key each is of
    bf = lambda t: t.to(BF).double()
    v = torch.ones_like(a)
    v[..., 0] = -bf(a[..., 1] / a[..., 0])
    v[..., 2] = -bf((a * v)[..., :2].sum(-1) / a[..., 2])
    v = torch.empty_like(v).scatter_(-1, at, v)
    for j, key in enumerate(J):
        for b in range(B):
            c.v[pre[key // page], :, key % page, b] = v[b, :, j].to(dtype)
    out = c.call(P, x, scale=1.0)
    gs = c.gs[c.slot].double().unsqueeze(-1) if gate else 0.0  # after the step
    weights = (z + gs).exp()
    total = weights.sum(-1) + 1.0  # and the new token's
    parts = weights[:, :, list(J)] * v
    ref = parts.sum(-1) / total
    l2e = math.log2(math.e)
    zl, gl = (z - g).abs().amax(-1) * l2e, (g.abs().amax(-1) + (gs.abs().squeeze(-1) if gate else 0.0)) * l2e
    eps = math.log(2) * 2.0 ** -23 * (6 * zl + 4 * gl + 4 * (zl + gl)) + 2.0 ** -20
    tol = parts.abs().sum(-1) / total * eps + 2.0 ** -8 * ref.abs()
    dim = torch.arange(B, device="cuda")
    err = (out.double()[dim, :, dim] - ref).abs()
    worst = (err / tol).max().item()
    assert worst <= 1, f"off by {worst} of what fp32 weights and queries may be"


@pytest.mark.parametrize("B,d", [(5, 64), (40, 64), (3, 128)])
def test_long_sums_over_a_prefix_do_not_drift(P, B, d):
    """Weighted values of one sign over a long prefix (832 steps of 16 keys a block), cancelled by two
    rows of the sequence's own. The tensor cores cut each step's sum to fp32, up to 2^-23 of what
    has been added up, all in one direction; parts of a sum are therefore joined by rounded
    additions, and 64 steps lie between. What is added up since rises from nothing, so they cut
    33 times 2^-23 of the whole at most; additions of up to 14 parts and of the pieces are
    rounded (16 times 2^-24), the weights are off by 2^-20 (as above)."""
    H, n, page = 30, 65536, 1024
    c = Cache([1] * B, H, d, page, BF, True, seed=d, prefix=n)
    pre = c.prefix_table.long()
    c.v[pre] = (1 + torch.rand(c.v[pre].shape, device="cuda", generator=c.rng)).to(BF)
    c.gs.zero_()
    x = c.step_inputs()
    x["q"].zero_()
    x["log_f"].zero_()
    own = torch.tensor([c.pages(r)[0] for r in c.slot], device="cuda")
    c.g[own, :, 0] = 0.0
    w = c.rows(c.g, None, n).exp()  # of the prefix; an own row weighs 1
    total = w.sum(-1, keepdim=True) + 2
    s = torch.stack([w[h] @ c.v[pre, h].reshape(-1, d)[:n].double() for h in range(H)])
    bf = lambda t: t.to(BF).double()
    v1 = -bf(s)
    v0 = -bf(s + v1)
    x["v_new"][:] = v1.to(BF)
    c.v[own, :, 0] = v0.to(BF)
    out = c.call(P, x, scale=1.0)
    ref = (s + v1 + v0) / total
    eps = 33 * 2.0 ** -23 + 16 * 2.0 ** -24 + 2.0 ** -20
    tol = 2 * s / total * eps + 2.0 ** -8 * ref.abs()
    worst = ((out.double() - ref).abs() / tol).max().item()
    assert worst <= 1, f"off by {worst} of the bound"


TIMEOUT = 5


def same(a, b):
    return torch.equal(torch.nan_to_num(a.float(), nan=1e9), torch.nan_to_num(b.float(), nan=1e9))


def restore(c, snap):
    for name, t in zip(("k", "v", "g", "state", "gs"), snap):
        if t is not None:
            getattr(c, name).copy_(t)


def withheld_step(P, c, x, prefix=0):
    """The step three times from one state: undisturbed, with a load withheld, undisturbed again.
    The last is the first bit for bit; returns the two outputs and the pools after the second."""
    ws = torch.empty(P.path_decode_paged_workspace_bytes(len(c.slot), c.H, c.M, c.page, c.d, c.dtype, prefix),
                     dtype=torch.uint8, device="cuda")
    start = c.snap()
    want = c.call(P, x, workspace=ws)
    after = c.snap()
    assert P.path_attn_wait_status(ws) == 0
    restore(c, start)
    P.path_test_withhold_kv_load(True)
    try:
        out = c.call(P, x, workspace=ws)
        torch.cuda.synchronize()
        status = P.path_attn_wait_status(ws)
    finally:
        P.path_test_withhold_kv_load(False)
    assert status == TIMEOUT
    given_up = c.snap()
    restore(c, start)
    again = c.call(P, x, workspace=ws)
    assert P.path_attn_wait_status(ws) == 0
    assert same(again, want)
    for a, b in zip(after, c.snap()):
        assert a is None or same(a, b)
    return want, out, after, given_up


@pytest.mark.parametrize("d,dtype,gate,prefix,n", [
    (64, BF, True, 0, 2000),   # shares of about 22 granules, rings of 4
    (128, BF, False, 0, 1300),
    (64, F32, True, 0, 1300),
    (128, F32, False, 65, 300),
])
def test_an_own_part_that_gives_up(P, d, dtype, gate, prefix, n):
    """The first warp never gets its second granule: its unit is NaN, the others and the calls after it
    are as ever, and the report says so."""
    c = Cache([n] * 40, 8, d, 64, dtype, gate, seed=1, prefix=prefix)
    want, out, after, given_up = withheld_step(P, c, c.step_inputs(), prefix)
    assert torch.isnan(out[0, 0]).all()
    assert same(out[0, 1:], want[0, 1:]) and same(out[1:], want[1:])
    p0 = c.pages(c.slot[0])[0]
    a, b = after[0], given_up[0]
    assert same(a[p0, 0, :8], b[p0, 0, :8]), "the granule before it"
    assert not same(a[p0, 0, 16:], b[p0, 0, 16:]), "keys that were never there"
    assert same(a[:, 1:], b[:, 1:]) and all(x is None or same(x, y) for x, y in zip(after[3:], given_up[3:]))


@pytest.mark.parametrize("B,d,gate", [(5, 64, True), (40, 64, False), (64, 64, True), (20, 128, True), (40, 128, False),
                                      (9, 128, True)])
def test_a_prefix_that_gives_up(P, B, d, gate):
    """The first block never gets its second tile of keys: head 0 is NaN, all else is as ever, in this call
    and the next. (The own parts are one granule each, which the hook passes over.)"""
    c = Cache([0] * B, 8, d, 64, BF, gate, seed=B, prefix=40000)
    want, out, after, given_up = withheld_step(P, c, c.step_inputs(), 40000)
    assert torch.isnan(out[:, 0]).all()
    assert same(out[:, 1:], want[:, 1:])
    for a, b in zip(after, given_up):
        assert a is None or same(a, b)


@pytest.mark.parametrize("d,dtype,gate", [(64, BF, True), (64, F32, False), (128, BF, False), (128, F32, True)])
def test_a_padded_prefill_in_pages(P, d, dtype, gate):
    """Prompts of different lengths in one prefill, padded with beta = 0 and log f = 0, stored into
    pages and continued. Every output is the oracle's row of that sequence alone. The bars are the
    decode tests': 1e-4 at fp32, 2e-2 at bf16."""
    H, page, lens, steps = 2, 32, [150, 1, 77, 128], 3
    B, L = len(lens), max(lens)
    g = torch.Generator().manual_seed(d)
    n = L + steps
    x = {a: torch.randn((B, H, n, d), generator=g) for a in "qkvw"}
    x["w"] /= x["w"].norm(dim=-1, keepdim=True)
    x = {a: t.to(dtype) for a, t in x.items()}
    x["beta"] = 1.9 * torch.sigmoid(torch.randn((B, H, n), generator=g))
    x["log_f"] = torch.nn.functional.logsigmoid(torch.randn((B, H, n), generator=g) + 2)
    # the prompts are the sequences' first rows; what stands behind them in the prefill is padding
    pad = {a: t[:, :, :L].clone() for a, t in x.items()}
    for b, m in enumerate(lens):
        pad["beta"][b, :, m:] = 0
        pad["log_f"][b, :, m:] = 0
        for a in "qkvw":
            pad[a][b, :, m:] = torch.randn((H, L - m, d), generator=g).to(dtype)
    pad = {a: t.contiguous().cuda() for a, t in pad.items()}
    out, _, kc, vc, gc = P.path_attn_prefill(*(pad[a] for a in ("q", "k", "v", "w", "beta")), L + 4,
                                             log_f=pad["log_f"] if gate else None)
    M = n // page + 1
    N = B * M
    table = torch.randperm(N, generator=g).view(B, M).int().cuda()
    kp, vp = (torch.full((N, H, page, d), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    gp = torch.full((N, H, page), math.nan, device="cuda") if gate else None
    info, slot_len = ints([0] * 4), ints(lens)
    P.path_pages_store(kc, vc, kp, vp, table, None, slot_len, g_cache=gc, g_pages=gp, info=info)
    assert info.tolist()[0] == 0
    bar = 1e-4 if dtype == F32 else 2e-2
    refs = []
    for b, m in enumerate(lens):
        seq = {a: t[b:b + 1, :, :m + steps] for a, t in x.items()}
        ref, _ = oracle.fwd(seq["q"], seq["k"], seq["v"], seq["w"], seq["beta"], seq["log_f"] if gate else None)
        refs.append(torch.as_tensor(ref[0]))
        err = (out[b, :, :m].double().cpu() - refs[b][:, :m]).abs().max().item()
        assert err <= bar, f"prefill, row {b}: {err}"
    for t in range(steps):
        col = lambda a: torch.stack([x[a][b, :, m + t] for b, m in enumerate(lens)]).cuda()
        o = P.path_decode_step_paged(col("q"), col("k"), col("v"), col("w"), col("beta"), kp, vp, table, slot_len,
                                     log_f=col("log_f") if gate else None, g_pages=gp)
        slot_len += 1
        for b, m in enumerate(lens):
            err = (o[b].double().cpu() - refs[b][:, m + t]).abs().max().item()
            assert err <= bar, f"step {t}, row {b}: {err}"


# ------------------------------------------------------------------ layouts that only large batches take
@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("rows,few", [(12, False), (13, True), (24, True)])
def test_both_layouts_of_rows_of_128_bytes(P, rows, few, gate, prefix):
    """bf16, head dim 64: from 40 granules for each of eight warps an SM, eight warps work with longer
    rings, below it twelve (a granule is 16 rows, and a unit counts one more)."""
    H, lens = 24, [1500 + 997 * i % 1000 for i in range(rows)]
    total = H * sum(n // 16 + 2 for n in lens)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (total >= sms * 8 * 40) == few
    run_steps(P, Cache(lens, H, 64, 64, BF, gate, seed=rows, prefix=prefix), steps=1)


@pytest.mark.parametrize("prefix,lens,dtype,d", [
    (20000, [5, 0, 70], F32, 64),              # 296 blocks hold a piece of each row
    (20000, [5, 0, 70], F32, 128),
    (0, [100000] + [0] * 299, BF, 64),         # many units, so 64 or 128 threads join; over 128 pieces of one
    (0, [100000] + [0] * 299, BF, 128),
    (0, [60000] + [0] * 299, F32, 128),
])
def test_units_of_more_pieces_than_threads(P, prefix, lens, dtype, d):
    run_steps(P, Cache(lens, 1, d, 64, dtype, False, seed=d, prefix=prefix), steps=1)


@pytest.mark.parametrize("dtype,N", [(BF, 9000), (F32, 8400)])
def test_a_prefix_beyond_32_bit_offsets(P, dtype, N):
    """Pages of a sequence and of its prefix at the end of a pool of more than 2^31 elements."""
    H, page, d = 32, 64, 128
    assert N * H * page * d > 2 ** 31
    k = torch.empty((N, H, page, d), dtype=dtype, device="cuda")
    v = torch.empty_like(k)
    g = torch.empty((N, H, page), device="cuda")
    c = Cache([100, 3], H, d, page, dtype, True, seed=8, prefix=1000)
    used = sorted({p for r in c.slot for p in c.pages(r) if p >= 0} | set(c.pages(None)))
    table, pre = c.table.clone(), c.prefix_table.clone()
    for i, p in enumerate(used):
        k[N - 1 - i], v[N - 1 - i], g[N - 1 - i] = c.k[p], c.v[p], c.g[p]
        table[c.table == p] = N - 1 - i
        pre[c.prefix_table == p] = N - 1 - i
    x, state, gs = c.step_inputs(), c.state.clone(), c.gs.clone()
    out = P.path_decode_step_shared(x["q"], x["k_new"], x["v_new"], x["w"], x["beta"], k, v, table, c.lens, pre,
                                    1000, state, rows=ints(c.slot), log_f=x["log_f"], g_pages=g, g_state=gs)
    want = c.call(P, x)
    assert torch.equal(out, want) and torch.equal(state, c.state) and torch.equal(gs, c.gs)
    for i, p in enumerate(used):
        assert same(k[N - 1 - i], c.k[p]) and same(v[N - 1 - i], c.v[p]) and same(g[N - 1 - i], c.g[p])


# ------------------------------------------------------------------ bad pages, infinities, equal logits
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, BF), (64, F32), (128, F32)])
@pytest.mark.parametrize("prefix", [0, 500])
def test_bad_pages_in_every_form(P, prefix, d, dtype, gate):
    """A page out of range in the table or in the prefix's, first, in the middle or last: NaN where it
    belongs, the report, and all else bit for bit as without it."""
    lens, H, page = [40, 170, 33], 3, 32
    fresh = lambda: Cache(lens, H, d, page, dtype, gate, prefix=prefix, seed=5)
    c = fresh()
    x, N = c.step_inputs(), c.k.shape[0]
    want, good = c.call(P, x), c.snap()
    places = [("table", (c.slot[1], j), [1], p) for j, p in ((0, -1), (2, N), (5, 2 ** 31 - 1))]
    if prefix:
        places += [("prefix_table", (j,), [0, 1, 2], p) for j, p in ((0, N), (7, -(2 ** 31)), (15, 2 ** 31 - 1))]
    ws = torch.empty(P.path_decode_paged_workspace_bytes(3, H, c.M, page, d, dtype, prefix), dtype=torch.uint8,
                     device="cuda")
    for name, at, bad, p in places:
        c = fresh()
        getattr(c, name)[at] = p
        out = c.call(P, x, workspace=ws)
        assert P.path_attn_wait_status(ws) == 6
        keep = torch.ones(N, dtype=torch.bool, device="cuda")
        if name == "table":
            keep[[q for q in fresh().pages(c.slot[1]) if q >= 0]] = False
        for b in range(3):
            if b in bad:
                assert torch.isnan(out[b]).all()
            else:
                assert torch.equal(out[b], want[b])
        for a, b in zip(c.snap()[:3], good[:3]):
            assert a is None or same(a[keep], b[keep]), (name, at)


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_logits(P, prefix, dtype):
    """q = 0: the mean of all values."""
    c = Cache([40, 70, 0], 3, 64, 32, dtype, False, prefix=prefix, seed=3)
    before, x = c.snap(), c.step_inputs()
    x["q"].zero_()
    c.check(before, x, c.call(P, x))


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_stay_in_their_head(P, prefix, dtype):
    """An infinite query, key or value in head 0 of a row, or of the prefix, changes no other head and no
    other row; an infinite new value comes out as it is."""
    inf = math.inf
    fresh = lambda: Cache([40, 70], 3, 64, 32, dtype, True, prefix=prefix, seed=4)
    c = fresh()
    x0 = c.step_inputs()
    want = c.call(P, x0)

    def go(change):
        c = fresh()
        x = {a: t.clone() for a, t in x0.items()}
        change(c, x)
        return c.call(P, x)

    row0 = c.pages(c.slot[0])[0]
    pool = [("k", row0), ("v", row0)]
    for name, p in pool:
        def change(c, x):
            getattr(c, name)[p, 0, 5, 7] = -inf
        out = go(change)
        assert torch.equal(out[1], want[1]) and torch.equal(out[0, 1:], want[0, 1:])
        assert not torch.isfinite(out[0, 0]).all()
    for name in ("q", "v_new"):
        def change(c, x):
            x[name][0, 0, 7] = inf
        out = go(change)
        assert torch.equal(out[1], want[1]) and torch.equal(out[0, 1:], want[0, 1:])
        if name == "q":
            assert torch.isnan(out[0, 0]).all()
        else:
            assert out[0, 0, 7] == inf and torch.equal(out[0, 0, 8:], want[0, 0, 8:])
    if prefix:
        for name in ("k", "v"):
            def change(c, x):
                getattr(c, name)[c.pages(None)[3], 0, 9, 7] = inf
            out = go(change)
            assert torch.equal(out[:, 1:], want[:, 1:])
            if name == "v":
                assert not torch.isfinite(out[:, 0, 7]).any() and torch.equal(out[:, 0, 8:], want[:, 0, 8:])


def test_an_infinite_key_of_an_fp32_prefix(P):
    """A logit of -inf leaves the other keys' weights as they are; one of +inf is NaN. With w = 0 and
    the identity as state the queries meet the prefix as they are. Tolerances as for a step."""
    n, d, B = 200, 64, 6
    c = Cache([0] * B, 2, d, 32, F32, False, prefix=n, seed=7)
    c.state.copy_(torch.eye(d, device="cuda").expand_as(c.state))
    x = c.step_inputs()
    x["w"].zero_()
    c.k[c.pages(None)[3], 0, 9] = 0
    c.k[c.pages(None)[3], 0, 9, 7] = math.inf
    x["q"][:, 0, 7] = torch.tensor([1.0, -1, 0.5, -2, -0.25, 3], device="cuda")
    out = c.call(P, x)
    scale = d ** -0.5
    for b in range(B):
        q = x["q"][b, 0].double()
        keys, vals = c.rows(c.k, None, n)[0], c.rows(c.v, None, n)[0]
        there = torch.ones(n, dtype=torch.bool, device="cuda")
        there[3 * 32 + 9] = False
        if q[7] > 0:
            assert torch.isnan(out[b, 0]).all()
            continue
        k = torch.cat([keys[there], x["k_new"][b, :1].double()])
        v = torch.cat([vals[there], x["v_new"][b, :1].double()])
        ref = torch.softmax(scale * (k @ q), 0) @ v
        ez = scale * q.norm() * k.norm(dim=-1).max() * 8 * math.sqrt(d) * 2.0 ** -24
        tol = 2.0 ** -24 * ref.abs() + 2 * v.abs().max() * (ez + 2.0 ** -20)
        assert ((out[b, 0].double() - ref).abs() <= tol).all()


def test_tables_of_a_large_pool(P):
    """300003 pages: reserve gives the lowest free pages in the order of its list, compaction fills the
    lowest gaps with the used pages behind them."""
    N, R, M, page = 300003, 200, 1700, 16
    rng = torch.Generator().manual_seed(0)
    used = torch.randperm(N, generator=rng)[: R * 1200].view(R, 1200).int()
    table = torch.full((R, M), -1, dtype=torch.int32)
    table[:, :1200] = used
    owner = torch.full((N,), -1, dtype=torch.int32)
    owner[used.long()] = (torch.arange(R)[:, None] * M + torch.arange(1200)).int()
    held = torch.full((R,), 1200, dtype=torch.int32)
    rows, more = torch.randperm(R, generator=rng)[:150], torch.randint(0, 300, (150,), generator=rng)
    dev = [t.cuda() for t in (table, held, owner)]
    tokens = (1200 + more) * page - torch.randint(0, page, (150,), generator=rng) * (more > 0)
    info = P.path_pages_reserve(*dev, page, rows.int().cuda(), tokens.int().cuda())
    free = (owner < 0).nonzero().flatten()
    total = int(more.sum())
    assert info.tolist() == [0, 0, R * 1200 + total, total]
    at = 0
    for r, m in zip(rows.tolist(), more.tolist()):
        table[r, 1200:1200 + m] = free[at:at + m].int()
        owner[free[at:at + m]] = (r * M + 1200 + torch.arange(m)).int()
        held[r] += m
        at += m
    for a, b in zip(dev, (table, held, owner)):
        assert torch.equal(a.cpu(), b)
    moves, info = P.path_pages_compact(dev[0], dev[1], dev[2])
    n = int((owner >= 0).sum())
    src, dst = n + (owner[n:] >= 0).nonzero().flatten(), (owner[:n] < 0).nonzero().flatten()
    assert info.tolist() == [0, len(src), n, 0]
    assert torch.equal(moves[: len(src)].cpu(), torch.stack([src, dst], 1).int())
    table.view(-1)[owner[src].long()] = dst.int()
    owner[dst] = owner[src]
    owner[src] = -1
    assert torch.equal(dev[0].cpu(), table) and torch.equal(dev[2].cpu(), owner)


def test_the_current_stream_by_either_way(P, monkeypatch):
    """The handle that the calls get is the current stream's, with torch's short way to it and without."""
    s = torch.cuda.Stream()
    for stream in (torch.cuda.default_stream(), s):
        with torch.cuda.stream(stream):
            assert P._stream() == stream.cuda_stream
            with monkeypatch.context() as m:
                m.setattr(P, "_raw_stream", None)
                assert P._stream() == stream.cuda_stream
                c = Cache([20], 2, 64, 16, BF, False)
                before, x = c.snap(), c.step_inputs()
                c.check(before, x, c.call(P, x))
