"""The paged decode cache on the GPU, against plain 64-bit arithmetic.

Tolerances, fixed from the number formats before the first run:
- stored keys and values: exact, or half a step of the type (bf16 2^-8, fp32 2^-24 relative)
  around the 64-bit update of the stored rows, plus the fp32 error of the update itself;
- out: half a step of the type around the 64-bit attention over the rows as stored, plus the
  fp32 error of the logits carried through the softmax. A dot product of d terms in fp32
  is off by about sqrt(d) 2^-24 |a| |b| (signs of the roundings vary; a factor 8 on top), a
  logit that is off by e moves out by at most 2 e max|v|, and the exponentials and their sums
  are off by 2^-20. Where bf16 queries meet a shared prefix they are held as a sum of two
  bf16 numbers, off by 2^-17, and so are the softmax weights.
"""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32
PAGE_ERR = 6


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import softmax_attention_block_b200 as P

    P.lib()
    return P


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Cache:
    """A pool with its tables; sequences of the given lengths on scattered pages. Rows that hold
    nothing are NaN, and so are the pages of nobody."""

    def __init__(self, lens, H, d, page, dtype, gate, seed=0, spare=6, slots=None, prefix=0):
        g = self.rng = torch.Generator(device="cuda").manual_seed(seed)
        perm = torch.Generator().manual_seed(seed)
        self.H, self.d, self.page, self.dtype, self.gate = H, d, page, dtype, gate
        self.R = slots or len(lens) + 2
        self.M = max(n // page + 2 for n in lens + [prefix])
        need = [n // page + 1 for n in lens]
        npre = -(-prefix // page)
        N = sum(need) + npre + spare
        ids = torch.randperm(N, generator=perm).tolist()
        self.slot = torch.randperm(self.R, generator=perm).tolist()[: len(lens)]
        table = [[-1] * self.M for _ in range(self.R)]
        owner, held, slot_len = [-1] * N, [0] * self.R, [0] * self.R
        at = npre
        for b, r in enumerate(self.slot):
            for j in range(need[b]):
                table[r][j] = ids[at]
                owner[ids[at]] = r * self.M + j
                at += 1
            held[r], slot_len[r] = need[b], lens[b]
        self.table, self.held, self.lens, self.owner = ints(table), ints(held), ints(slot_len), ints(owner)
        self.prefix, self.prefix_table = prefix, ints(ids[:npre])
        nan = float("nan")
        self.k = torch.full((N, H, page, d), nan, device="cuda", dtype=dtype)
        self.v = torch.full((N, H, page, d), nan, device="cuda", dtype=dtype)
        self.g = torch.full((N, H, page), nan, device="cuda") if gate else None
        for r, n in list(zip(self.slot, lens)) + ([(None, prefix)] if prefix else []):
            pages = self.pages(r)
            for j in range(-(-n // page)):
                m = min(page, n - j * page)
                self.k[pages[j], :, :m] = self.randn(H, m, d).to(dtype)
                self.v[pages[j], :, :m] = self.randn(H, m, d).to(dtype)
                if gate:
                    self.g[pages[j], :, :m] = -2 * torch.rand((H, m), device="cuda", generator=g)
        if prefix:
            S = torch.eye(d, device="cuda").expand(self.R, H, d, d).contiguous()
            for _ in range(3):
                w = self.unit(self.R, H, d)
                S = S - 1.7 * w.unsqueeze(-1) * (w.unsqueeze(-2) @ S)
            self.state = S.contiguous()
            self.gs = -torch.rand((self.R, H), device="cuda", generator=g) if gate else None

    def randn(self, *s):
        return torch.randn(s, device="cuda", generator=self.rng)

    def unit(self, *s):
        w = self.randn(*s)
        return w / w.norm(dim=-1, keepdim=True)

    def pages(self, r):
        return (self.prefix_table if r is None else self.table[r]).tolist()

    def rows(self, pool, r, n):
        """Rows 0..n-1 of slot r (None: the prefix) in a pool, [H, n, ...] in 64 bits."""
        p = [x for x in self.pages(r)[: -(-n // self.page)]]
        if not p:
            return pool[:0, :, :].transpose(0, 1).reshape(self.H, 0, *pool.shape[3:]).double()
        return torch.cat([pool[x] for x in p], 1)[:, :n].double()

    def step_inputs(self, idle=0, w_unit=True):
        B, H, d = len(self.slot) + idle, self.H, self.d
        x = dict(q=self.randn(B, H, d), k_new=self.randn(B, H, d), v_new=self.randn(B, H, d),
                 w=self.unit(B, H, d))
        x = {n: t.to(self.dtype) for n, t in x.items()}
        x["beta"] = 2 * torch.rand((B, H), device="cuda", generator=self.rng)
        x["log_f"] = -torch.rand((B, H), device="cuda", generator=self.rng) if self.gate else None
        return x

    def call(self, P, x, idle=0, **kw):
        if "rows" not in kw:
            kw["rows"] = ints(self.slot + [-1] * idle)
        args = (x["q"], x["k_new"], x["v_new"], x["w"], x["beta"], self.k, self.v, self.table, self.lens)
        kw = dict(dict(log_f=x["log_f"], g_pages=self.g), **kw)
        if self.prefix:
            return P.path_decode_step_shared(*args, self.prefix_table, self.prefix, self.state,
                                             g_state=self.gs, **kw)
        return P.path_decode_step_paged(*args, **kw)

    def check(self, before, x, out, skip=(), scale=None):
        """One step from the pool as it was (`before`: clones of k, v, g, state, gs) to the pool
        and out as they are now."""
        H, d, page, half = self.H, self.d, self.page, HALF[self.dtype]
        k0, v0, g0, s0, gs0 = before
        scale = d ** -0.5 if scale is None else scale
        ek, ev = k0.clone(), v0.clone()  # what nothing may change is as it was
        eg = g0.clone() if g0 is not None else None
        lens = self.lens.tolist()
        for b, r in enumerate(self.slot):
            n = lens[r]
            pages = self.pages(r)
            for j in range(n // page + 1):
                m = min(page, n + 1 - j * page)
                ek[pages[j], :, :m] = self.k[pages[j], :, :m]
                if eg is not None:
                    eg[pages[j], :, :m] = self.g[pages[j], :, :m]
            ev[pages[n // page], :, n % page] = x["v_new"][b]
            if b in skip:
                ev[pages[n // page], :, n % page] = self.v[pages[n // page], :, n % page]
                continue
            q, w, beta = (x[i][b].double() for i in ("q", "w", "beta"))
            old, now = self.rows(k0, r, n), self.rows(self.k, r, n + 1)
            want = old - (beta[:, None] * (old @ w.unsqueeze(-1)).squeeze(-1)).unsqueeze(-1) * w.unsqueeze(1)
            wk = 2 * old.norm(dim=-1, keepdim=True) * w.abs().unsqueeze(1)
            tol = half * want.abs() * 1.01 + 2.0 ** -24 * (old.abs() + (8 * math.sqrt(d) + 3) * wk)
            assert ((now[:, :n] - want).abs() <= tol).all(), f"row {b}: keys"
            assert torch.equal(now[:, n], x["k_new"][b].double()), f"row {b}: new key"
            bias = torch.zeros((H, n + 1), dtype=torch.float64, device="cuda")
            if g0 is not None:
                gw = self.rows(g0, r, n) + x["log_f"][b].double().unsqueeze(1)
                bias = self.rows(self.g, r, n + 1)
                fin = torch.isfinite(gw)
                assert torch.equal(fin, torch.isfinite(bias[:, :n]))
                assert ((bias[:, :n] - gw)[fin].abs() <= 2.0 ** -24 * gw[fin].abs() + 1e-30).all()
                assert (bias[:, n] == 0).all()
            keys, vals = now, self.rows(self.v, r, n + 1)
            qk = q.norm(dim=-1) * keys.norm(dim=-1).amax(-1)
            z = scale * (keys @ q.unsqueeze(-1)).squeeze(-1) + bias
            two = 0.0
            if self.prefix:
                S = s0[r].double()
                S = S - beta[:, None, None] * w.unsqueeze(-1) * (w.unsqueeze(-2) @ S)
                assert (self.state[r].double() - S).abs().max() <= (8 * math.sqrt(d) + 4) * 2.0 ** -23, f"row {b}: state"
                qt = (q.unsqueeze(-2) @ S).squeeze(-2)
                pk, pv = self.rows(self.k, None, self.prefix), self.rows(self.v, None, self.prefix)
                zp = scale * (pk @ qt.unsqueeze(-1)).squeeze(-1)
                if g0 is not None:
                    gs = gs0[r].double() + x["log_f"][b].double()
                    fin = torch.isfinite(gs)
                    assert ((self.gs[r].double() - gs)[fin].abs() <= 2.0 ** -24 * gs[fin].abs()).all()
                    zp = zp + self.rows(self.g, None, self.prefix) + gs.unsqueeze(-1)
                z, vals = torch.cat([zp, z], 1), torch.cat([pv, vals], 1)
                qk = torch.maximum(qk, 2 * q.norm(dim=-1) * pk.norm(dim=-1).amax(-1))
                if self.dtype == BF:
                    two = 2.0 ** -17
            a = torch.softmax(z, -1)
            ref = (a.unsqueeze(1) @ vals).squeeze(1)
            zmax = z[torch.isfinite(z)].abs().max()
            ez = abs(scale) * qk * (8 * math.sqrt(d) * 2.0 ** -24 + 2 * two) + 4 * zmax * 2.0 ** -24
            vmax = vals.abs().amax((1, 2))
            tol = half * ref.abs() + (2 * vmax * (ez + two + 2.0 ** -20)).unsqueeze(-1)
            err = (out[b].double() - ref).abs()
            assert (err <= tol).all(), f"row {b}: out off by {err.max().item()}, may be {tol.max().item()}"
        same = lambda a, b: torch.equal(torch.nan_to_num(a.float(), nan=1e9), torch.nan_to_num(b.float(), nan=1e9))
        assert same(self.k, ek) and same(self.v, ev), "rows outside the step were written"
        if eg is not None:
            assert same(self.g, eg), "gate biases outside the step were written"

    def snap(self):
        c = lambda t: None if t is None else t.clone()
        return (c(self.k), c(self.v), c(self.g), c(getattr(self, "state", None)), c(getattr(self, "gs", None)))


def run_steps(P, c, steps=2, idle=0):
    ws = torch.full((P.path_decode_paged_workspace_bytes(len(c.slot) + idle, c.H, c.M, c.page, c.d, c.dtype,
                                                         c.prefix),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(steps):
        before, x = c.snap(), c.step_inputs(idle)
        out = torch.full((len(c.slot) + idle, c.H, c.d), 77.0, device="cuda", dtype=c.dtype)
        c.call(P, x, idle, out=out, workspace=ws)
        assert P.path_attn_wait_status(ws) == 0
        c.check(before, x, out)
        assert (out[len(c.slot):] == 77.0).all(), "an idle row was written"
        for r in c.slot:  # the caller advances; a sequence at its last row stops there
            if (int(c.lens[r]) + 1) // c.page < int(c.held[r]):
                c.lens[r] += 1


EDGES = [0, 1, 15, 16, 17, 62, 63, 64, 65, 127, 128, 129]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,H,page,gate,idle", [
    ([0], 1, 16, False, 0),
    ([1], 1, 1024, True, 0),
    (EDGES, 3, 16, True, 2),
    (EDGES, 2, 64, False, 1),
    ([700, 0, 3000, 5, 2047], 5, 32, True, 0),
    ([5000], 2, 256, False, 3),
])
def test_paged_step(P, lens, H, page, gate, idle, d, dtype):
    run_steps(P, Cache(lens, H, d, page, dtype, gate, seed=len(lens) + H), idle=idle)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows_and_one_long(P, dtype):
    """More units than blocks, and one sequence that most blocks share."""
    run_steps(P, Cache([i % 40 for i in range(300)], 2, 64, 16, dtype, False, seed=3), steps=1)
    run_steps(P, Cache([20000, 3, 0], 1, 128, 64, dtype, True, seed=4), steps=1)


PREFIX = [
    # prefix, lens, H, page, gate
    (1, [0], 1, 16, False),
    (64, [0, 1], 2, 16, True),
    (65, [17, 0, 3], 3, 32, False),
    (127, [0] * 33, 2, 128, True),
    (1000, [5, 70, 0, 64, 200], 5, 64, True),
    (5003, [i % 9 for i in range(70)], 3, 64, False),
    (300, [2] * 130, 1, 256, True),
    (2500, [3, 0], 1, 1024, False),
    (77, [i % 5 for i in range(600)], 1, 16, False),
    (6000, [1] * 20, 30, 16, True),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("prefix,lens,H,page,gate", PREFIX)
def test_shared_step(P, prefix, lens, H, page, gate, d, dtype):
    run_steps(P, Cache(lens, H, d, page, dtype, gate, seed=prefix, prefix=prefix), idle=1)


@pytest.mark.parametrize("prefix", [0, 100])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_gate_that_forgets_everything(P, prefix, dtype):
    """log f = -inf leaves the new token alone, in this step and the next."""
    c = Cache([30, 0, 100], 2, 64, 32, dtype, True, prefix=prefix)
    for _ in range(2):
        before, x = c.snap(), c.step_inputs()
        x["log_f"][:, 0] = -math.inf
        out = c.call(P, x)
        assert torch.equal(out[:, 0], x["v_new"][:, 0])
        c.check(before, x, out)


@pytest.mark.parametrize("prefix", [0, 90])
def test_lowest_values_infinities_and_nan(P, prefix):
    """Biases of the lowest fp32 value mask a key; NaN in one head stays there; equal logits."""
    c = Cache([40, 70], 3, 64, 32, BF, True, prefix=prefix)
    low = torch.finfo(torch.float32).min
    for r, n in ((c.slot[0], 40), (c.slot[1], 70)):
        for j in range(-(-n // 32)):
            c.g[c.pages(r)[j], 0] = low
    if prefix:
        for p in c.pages(None):
            c.g[p, 0] = low
    x = c.step_inputs()
    x["q"][:, 1] = 0
    x["q"][0, 2, 5] = float("nan")
    out = c.call(P, x)
    assert torch.equal(out[:, 0], x["v_new"][:, 0])
    assert torch.isnan(out[0, 2]).all() and torch.isfinite(out[1]).all() and torch.isfinite(out[0, :2]).all()


@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_batch_of_idle_rows(P, prefix, dtype):
    """Nothing is written, and the call after it is as ever."""
    c = Cache([20, 33], 2, 64, 16, dtype, True, prefix=prefix)
    before, x = c.snap(), c.step_inputs()
    out = torch.full_like(x["q"], 5.0)
    ws = torch.full((P.path_decode_paged_workspace_bytes(2, 2, c.M, 16, 64, dtype, prefix),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    c.call(P, x, out=out, workspace=ws, rows=ints([-1, -7]))
    assert (out == 5.0).all() and P.path_attn_wait_status(ws) == 0
    for a, b in zip(before, c.snap()):
        assert a is None or torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
    c.call(P, x, out=out, workspace=ws)
    c.check(before, x, out)


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
def test_scales(P, scale, dtype, prefix):
    c = Cache([30, 0, 100], 2, 64, 32, dtype, prefix > 0, prefix=prefix, seed=6)
    before, x = c.snap(), c.step_inputs()
    out = c.call(P, x, scale=scale)
    c.check(before, x, out, scale=scale)


@pytest.mark.parametrize("B", [5, 20, 40, 64])
@pytest.mark.parametrize("d,dtype,gate", [(64, BF, True), (128, BF, False), (64, F32, False), (128, F32, True)])
def test_a_maximum_that_keeps_rising(P, B, d, dtype, gate):
    """Keys that grow along the prefix: the running maximum moves many times, over many tiles of a
    block and from one head to the next."""
    H, n, page = 24, 9000, 64
    c = Cache([i % 3 for i in range(B)], H, d, page, dtype, gate, seed=B, prefix=n)
    for j, p in enumerate(c.pages(None)):
        c.k[p] *= 0.05 + 3.0 * j * page / n
    before, x = c.snap(), c.step_inputs()
    out = c.call(P, x, scale=0.7)
    c.check(before, x, out, scale=0.7)


@pytest.mark.parametrize("prefix", [0, 130])
def test_a_captured_step_serves_growing_sequences(P, prefix):
    """Lengths are read on the device: one graph is every step, until a page is missing."""
    kw = dict(gate=True, seed=12, prefix=prefix)
    c, e = (Cache([14, 40], 2, 64, 16, BF, **kw) for _ in range(2))
    x = c.step_inputs()
    ws = torch.empty(P.path_decode_paged_workspace_bytes(2, 2, c.M, 16, 64, BF, prefix), dtype=torch.uint8,
                     device="cuda")
    out = torch.zeros_like(x["q"])
    rows, ones = ints(c.slot), torch.ones_like(c.lens)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        c.call(P, x, out=out, workspace=ws, rows=rows)
        c.lens += ones
    for step in range(4):  # row 0 fills its page at 16 and has no other
        gr.replay()
        want = e.call(P, x, rows=rows)
        e.lens += ones
        assert torch.equal(out[1], want[1])
        if step < 2:
            assert torch.equal(out, want)
            assert P.path_attn_wait_status(ws) == 0
        else:
            assert torch.isnan(out[0]).all() and P.path_attn_wait_status(ws) == PAGE_ERR


@pytest.mark.parametrize("prefix", [0, 50])
def test_bad_tables_are_reported_and_harmless(P, prefix):
    def fresh():
        return Cache([40, 70, 33], 2, 64, 32, BF, False, prefix=prefix, seed=5)

    def go(c, bad, status=PAGE_ERR):
        ws = torch.empty(P.path_decode_paged_workspace_bytes(3, 2, c.M, 32, 64, BF, prefix),
                         dtype=torch.uint8, device="cuda")
        before, x = c.snap(), c.step_inputs()
        out = c.call(P, x, workspace=ws)
        assert P.path_attn_wait_status(ws) == status
        for b in range(3):
            assert torch.isnan(out[b]).all() == (b in bad)
        return before, x, out

    c = fresh()
    c.table[c.slot[1], 1] = -1
    go(c, [1])
    c = fresh()
    c.table[c.slot[2], 0] = c.k.shape[0]
    go(c, [2])
    for n in (-1, c.M * 32, 2 ** 31 - 1):
        c = fresh()
        c.lens[c.slot[0]] = n
        go(c, [0])
    c = fresh()
    c.slot[1] = c.R  # a slot that does not exist
    go(c, [1])
    c = fresh()
    c.slot[1] = c.slot[2]  # the same slot twice
    go(c, [1, 2])
    if prefix:
        c = fresh()
        c.prefix_table[0] = -3
        go(c, [0, 1, 2])
    # the next good call clears the report
    go(fresh(), [], status=0)


def test_pool_beyond_32_bit_offsets(P):
    """Pages at the end of a pool of 2.4e9 elements."""
    H, page, d, N = 32, 64, 128, 9000
    k = torch.empty((N, H, page, d), dtype=BF, device="cuda")
    v = torch.empty_like(k)
    c = Cache([100], H, d, page, BF, False, seed=8)
    used = [p for p in c.pages(c.slot[0]) if p >= 0]
    move = {p: N - 1 - i for i, p in enumerate(used)}
    for p, to in move.items():
        k[to], v[to] = c.k[p], c.v[p]
    x = c.step_inputs()
    table = c.table.clone()
    for i, p in enumerate(used):
        table[c.slot[0], i] = move[p]
    out = P.path_decode_step_paged(x["q"], x["k_new"], x["v_new"], x["w"], x["beta"], k, v, table, c.lens,
                                   rows=ints(c.slot))
    want = c.call(P, x)
    assert torch.equal(out, want)
    for p, to in move.items():
        assert torch.equal(torch.nan_to_num(k[to].float()), torch.nan_to_num(c.k[p].float()))


@pytest.mark.parametrize("prefix", [0, 700])
def test_repeats_exactly_on_another_stream_and_in_graphs(P, prefix):
    """Eager, on a side stream, and two captured graphs that share the workspace."""
    c = Cache([300, 1200, 0, 77], 6, 64, 64, BF, True, prefix=prefix, seed=9)
    start, x = c.snap(), c.step_inputs()

    def restore():
        for t, s in zip((c.k, c.v, c.g, getattr(c, "state", None), getattr(c, "gs", None)), start):
            if s is not None:
                t.copy_(s)

    ws = torch.empty(P.path_decode_paged_workspace_bytes(4, 6, c.M, 64, 64, BF, prefix), dtype=torch.uint8,
                     device="cuda")
    out = torch.zeros_like(x["q"])
    rows = ints(c.slot)
    c.call(P, x, out=out, workspace=ws, rows=rows)
    want = [out.clone(), *c.snap()]
    other = torch.cuda.Stream()
    restore()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        out.zero_()
        c.call(P, x, out=out, workspace=ws, rows=rows)
    torch.cuda.current_stream().wait_stream(other)
    got = [out.clone(), *c.snap()]
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.call(P, x, out=out, workspace=ws, rows=rows)
        graphs.append(gr)
    for gr in graphs:
        restore()
        out.zero_()
        gr.replay()
        for other_run in (got, [out, *c.snap()]):
            for a, b in zip(want, other_run):
                assert (a is None) == (b is None)
                if a is not None:
                    assert torch.equal(torch.nan_to_num(a.float(), nan=1e9), torch.nan_to_num(b.float(), nan=1e9))


def test_paged_agrees_with_contiguous_decode(P):
    """Equal lengths: path_decode_step's keys and outputs. Both steps add up w.k in an order of
    their own and round once, so a key may land on the neighbouring bf16 number (one step,
    2^-7 relative, plus the fp32 error of two updates); values and the new row are copies."""
    B, H, d, page, n = 3, 4, 128, 32, 333
    g = torch.Generator(device="cuda").manual_seed(1)
    kc = torch.randn((B, H, n + 1, d), device="cuda", generator=g).to(BF)
    vc = torch.randn((B, H, n + 1, d), device="cuda", generator=g).to(BF)
    M = n // page + 1
    table = ints(np.random.default_rng(0).permutation(B * M).reshape(B, M).tolist())
    k = torch.zeros((B * M, H, page, d), device="cuda", dtype=BF)
    v = torch.zeros_like(k)
    P.path_pages_store(kc, vc, k, v, table, None, ints([n] * B))
    x = Cache([n] * B, H, d, page, BF, False, seed=2).step_inputs()
    want = P.path_decode_step(x["q"], x["k_new"], x["v_new"], x["w"], x["beta"], kc, vc, n)
    out = P.path_decode_step_paged(x["q"], x["k_new"], x["v_new"], x["w"], x["beta"], k, v, table, ints([n] * B))
    rows = lambda t, b: torch.cat([t[p] for p in table[b].tolist()], 1)[:, : n + 1]
    for b in range(B):
        a, b_ = rows(k, b).float(), kc[b].float()
        assert ((a - b_).abs() <= 2.0 ** -7 * b_.abs() + 2 * 2.0 ** -24 * 8 * math.sqrt(d) * 2 * b_.norm(dim=-1, keepdim=True)).all()
        assert torch.equal(rows(k, b)[:, n], kc[b][:, n]) and torch.equal(rows(v, b), vc[b])
    assert (out.float() - want.float()).abs().max() <= 2 * 2.0 ** -8 * want.float().abs().max()


# ------------------------------------------------------------------------ tables and copies
class Tables:
    """The tables in plain Python, beside the device's."""

    def __init__(self, R, M, N, page):
        self.R, self.M, self.N, self.page = R, M, N, page
        self.table, self.held = [[-1] * M for _ in range(R)], [0] * R
        self.lens, self.owner = [0] * R, [-1] * N
        self.dev = [ints(self.table), ints(self.held), ints(self.lens), ints(self.owner)]

    def same(self):
        t, h, n, o = self.dev
        assert t.tolist() == self.table and h.tolist() == self.held
        assert n.tolist() == self.lens and o.tolist() == self.owner

    def give(self, wants):
        """[(slot, pages to add)] in order, or False and nothing given."""
        free = [p for p in range(self.N) if self.owner[p] < 0]
        if sum(max(0, w) for _, w in wants) > len(free):
            return False
        for r, w in wants:
            for _ in range(max(0, w)):
                p, j = free.pop(0), self.held[r]
                self.table[r][j], self.owner[p], self.held[r] = p, r * self.M + j, j + 1
        return True

    def used(self):
        return sum(o >= 0 for o in self.owner)


@pytest.mark.parametrize("R,M,N,page,seed", [(3, 4, 7, 16, 0), (40, 9, 200, 32, 1), (300, 40, 9000, 16, 2),
                                             (2, 1, 1, 1024, 3)])
def test_tables_follow_a_plain_model(P, R, M, N, page, seed):
    """Reserve, fork, free and compact in random order, refused calls among them."""
    rng = np.random.default_rng(seed)
    T = Tables(R, M, N, page)
    t, h, n, o = T.dev
    refused = 0
    for step in range(60):
        op = rng.choice(["reserve", "fork", "free", "compact"], p=[0.4, 0.25, 0.25, 0.1])
        cnt = int(rng.integers(1, min(R, 24) + 1))
        rows = rng.permutation(R)[:cnt].tolist()
        if op == "reserve":
            tokens = [int(rng.integers(0, M * page + 1)) for _ in rows]
            info = P.path_pages_reserve(t, h, o, page, ints(rows), ints(tokens)).tolist()
            before = T.used()
            if T.give([(r, -(-x // page) - T.held[r]) for r, x in zip(rows, tokens)]):
                assert info == [0, 0, T.used(), T.used() - before]
                for r in rows:
                    T.lens[r] = int(rng.integers(0, T.held[r] * page + 1))
                n.copy_(ints(T.lens))
            else:
                refused += 1
                assert info == [PAGE_ERR, 0, before, 0]
        elif op == "fork":
            kids = [r if T.held[r] == 0 else -1 for r in rows]
            par = [int(rng.integers(-1, R)) for _ in rows]
            moves, info = P.path_pages_fork(t, h, n, o, page, ints(par), ints(kids))
            info, before = info.tolist(), T.used()
            wants = [(c, -(-T.lens[p] // page) if p >= 0 else 0) for p, c in zip(par, kids) if c >= 0]
            if T.give(wants):
                mv = [[T.table[p][j], T.table[c][j]] for p, c in zip(par, kids) if c >= 0 and p >= 0
                      for j in range(-(-T.lens[p] // page))]
                new = {c: T.lens[p] if p >= 0 else 0 for p, c in zip(par, kids) if c >= 0}
                for c, x in new.items():
                    T.lens[c] = x
                assert info == [0, len(mv), T.used(), len(mv)]
                assert moves[: len(mv)].tolist() == mv
            else:
                refused += 1
                assert info == [PAGE_ERR, 0, before, 0]
        elif op == "free":
            P.path_pages_free(t, h, n, o, ints(rows + rows[:1] + [-1, R]))
            for r in rows:
                for j in range(T.held[r]):
                    T.owner[T.table[r][j]] = -1
                    T.table[r][j] = -1
                T.held[r] = T.lens[r] = 0
        else:
            moves, info = P.path_pages_compact(t, h, o)
            used = T.used()
            gaps = [p for p in range(used) if T.owner[p] < 0]
            mv = [[p, gaps.pop(0)] for p in range(used, N) if T.owner[p] >= 0]
            for a, b in mv:
                e = T.owner[a]
                T.table[e // M][e % M], T.owner[b], T.owner[a] = b, e, -1
            assert info.tolist() == [0, len(mv), used, 0]
            assert moves[: len(mv)].tolist() == mv
        T.same()


def test_refused_table_calls_change_nothing(P):
    T = Tables(4, 3, 8, 16)
    t, h, n, o = T.dev
    P.path_pages_reserve(t, h, o, 16, ints([0, 1]), ints([40, 16]))
    n.copy_(ints([40, 10, 0, 0]))
    state = lambda: [x.tolist() for x in (t, h, n, o)]
    was = state()
    for rows, tokens in (([0, 0], [48, 48]), ([4], [1]), ([2], [-1]), ([2], [49]), ([2, 3], [48, 32])):
        assert P.path_pages_reserve(t, h, o, 16, ints(rows), ints(tokens)).tolist() == [PAGE_ERR, 0, 4, 0]
        assert state() == was
    for par, kids in (([0], [1]), ([0, 0], [2, 2]), ([4], [2]), ([0], [7]), ([0, 0], [2, 3])):
        assert P.path_pages_fork(t, h, n, o, 16, ints(par), ints(kids))[1].tolist() == [PAGE_ERR, 0, 4, 0]
        assert state() == was
    o[7] = 0  # a page whose owner has another page there
    assert P.path_pages_compact(t, h, o)[1].tolist()[0] == PAGE_ERR
    assert t.tolist() == was[0]


@pytest.mark.parametrize("H,d,page,dtype,gate", [(1, 64, 16, BF, False), (5, 128, 32, F32, True),
                                                 (3, 64, 1024, BF, True)])
def test_copy_moves_whole_pages(P, H, d, page, dtype, gate):
    N, g = 11, torch.Generator(device="cuda").manual_seed(0)
    k = torch.randn((N, H, page, d), device="cuda", generator=g).to(dtype)
    v = torch.randn((N, H, page, d), device="cuda", generator=g).to(dtype)
    gp = torch.randn((N, H, page), device="cuda", generator=g) if gate else None
    pairs = [[3, 0], [3, 10], [7, 5], [-1, 2], [4, N], [6, 1]]
    info = ints([0, len(pairs), 0, 0])
    want = [x.clone() if x is not None else None for x in (k, v, gp)]
    for a, b in ((3, 0), (3, 10), (7, 5), (6, 1)):
        for x in want:
            if x is not None:
                x[b] = x[a]
    P.path_pages_copy(ints(pairs + [[8, 9]]), info, k, v, g_pages=gp)
    assert info.tolist()[0] == PAGE_ERR  # the two moves out of range
    for a, b in zip((k, v, gp), want):
        assert a is None or torch.equal(a, b)
    P.path_pages_copy(ints([[8, 9]]), ints([0, 0, 0, 0]), k, v, g_pages=gp)  # nothing listed
    assert torch.equal(k, want[0])


@pytest.mark.parametrize("d,page,dtype,gate", [(64, 16, BF, True), (128, 64, F32, False), (128, 512, BF, True)])
def test_store_writes_the_filled_rows_only(P, d, page, dtype, gate):
    H, cap, tokens = 3, 150, [0, 1, 16, 17, 150, 64, 99, 151, -1]
    B, M = len(tokens), 150 // page + 1
    g = torch.Generator(device="cuda").manual_seed(0)
    kc, vc = (torch.randn((B, H, cap, d), device="cuda", generator=g).to(dtype) for _ in range(2))
    gc = torch.randn((B, H, cap), device="cuda", generator=g) if gate else None
    N = (B + 2) * M
    table = ints(np.random.default_rng(1).permutation(N).reshape(B + 2, M).tolist())
    k, v = (torch.full((N, H, page, d), 3.0, device="cuda", dtype=dtype) for _ in range(2))
    gp = torch.full((N, H, page), 3.0, device="cuda") if gate else None
    rows = [5, 2, 0, 7, 3, -1, 10, 8, 9]
    table[10, 1 if M > 1 else 0] = -1
    info = ints([0] * 4)
    want = [x.clone() if x is not None else None for x in (k, v, gp)]
    for b, (r, n) in enumerate(zip(rows, tokens)):
        if r < 0 or n < 0 or n > cap:
            continue
        for i in range(n):
            p = int(table[r, i // page])
            if p >= 0:
                for x, y in zip(want, (kc, vc, gc)):
                    if x is not None:
                        x[p, :, i % page] = y[b, :, i]
    P.path_pages_store(kc, vc, k, v, table, ints(rows), ints(tokens), g_cache=gc, g_pages=gp, info=info)
    assert info.tolist() == [PAGE_ERR, 0, 0, 0]
    for a, b in zip((k, v, gp), want):
        assert a is None or torch.equal(a, b)


def test_state_copy(P):
    for d in (64, 128):
        s = torch.randn((6, 2, d, d), device="cuda")
        gs = torch.randn((6, 2), device="cuda")
        ws, wg = s.clone(), gs.clone()
        for a, b in ((0, 1), (0, 2), (-1, 3)):
            ws[b] = ws[a] if a >= 0 else torch.eye(d, device="cuda")
            wg[b] = wg[a] if a >= 0 else 0
        P.path_state_copy(s, ints([0, 0, -1, 4, 9]), ints([1, 2, 3, -1, 5]), g_state=gs)
        assert torch.equal(s, ws) and torch.equal(gs, wg)


# ------------------------------------------------------------------------ together
@pytest.mark.parametrize("d,dtype,gate", [(64, F32, True), (64, BF, False), (128, BF, True)])
def test_a_server_run_against_the_oracle(P, d, dtype, gate):
    """A prefix is prefilled and stored; three sequences continue it, decode, fork in the middle,
    one ends, the pool is compacted, and decoding goes on. Every output is the oracle's row of the
    whole sequence. The bars are the decode tests': 1e-4 at fp32; at bf16 2e-2, for own keys that
    are rounded to bf16 once a step (30 roundings of 2^-9 at most, sqrt(30) 2^-9 = 1.1e-2 on logits
    of order 1, averaged by the softmax)."""
    H, page, L0, steps = 2, 16, 45, 30
    g = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(s, generator=g)

    def tokens(n):
        w = rnd(n, H, d)
        x = dict(q=rnd(n, H, d), k=rnd(n, H, d), v=rnd(n, H, d), w=w / w.norm(dim=-1, keepdim=True))
        x = {a: t.to(dtype) for a, t in x.items()}
        x["beta"] = 1.9 * torch.sigmoid(rnd(n, H))
        x["log_f"] = torch.nn.functional.logsigmoid(rnd(n, H) + 2)
        return x

    prefix = tokens(L0)
    batch = lambda x, a: x[a].transpose(0, 1).unsqueeze(0).contiguous().cuda()  # [1, H, n, d]
    lf = batch(prefix, "log_f") if gate else None
    _, _, kc, vc, gc = P.path_attn_prefill(*(batch(prefix, a) for a in ("q", "k", "v", "w", "beta")), L0,
                                           log_f=lf)
    R, M, N = 8, 4, 24
    table, held = torch.full((R, M), -1, dtype=torch.int32, device="cuda"), ints([0] * R)
    lens, owner = ints([0] * R), ints([-1] * N)
    kp, vp = (torch.zeros((N, H, page, d), dtype=dtype, device="cuda") for _ in range(2))
    gp = torch.zeros((N, H, page), device="cuda") if gate else None
    state = torch.zeros((R, H, d, d), device="cuda")
    gs = torch.zeros((R, H), device="cuda") if gate else None
    PRE = 5
    assert P.path_pages_reserve(table, held, owner, page, ints([PRE]), ints([L0])).tolist()[0] == 0
    P.path_pages_store(kc, vc, kp, vp, table, ints([PRE]), ints([L0]), g_cache=gc, g_pages=gp)
    live = {0: [], 1: [], 6: []}
    kids = ints(list(live))
    P.path_pages_fork(table, held, lens, owner, page, ints([-1] * 3), kids)
    P.path_state_copy(state, ints([-1] * 3), kids, g_state=gs)
    for step in range(steps):
        if step == 6:  # a beam step: 1 goes on in 3 and 4; 6 ends
            moves, info = P.path_pages_fork(table, held, lens, owner, page, ints([1, 1]), ints([3, 4]))
            P.path_pages_copy(moves, info, kp, vp, g_pages=gp)
            P.path_state_copy(state, ints([1, 1]), ints([3, 4]), g_state=gs)
            P.path_pages_free(table, held, lens, owner, ints([6]))
            assert info.tolist()[0] == 0
            live[3], live[4] = list(live[1]), list(live[1])
            del live[6]
        if step == 9:
            P.path_pages_free(table, held, lens, owner, ints([0]))
            del live[0]
            moves, info = P.path_pages_compact(table, held, owner)
            P.path_pages_copy(moves, info, kp, vp, g_pages=gp)
            assert info.tolist()[0] == 0 and info.tolist()[1] > 0
        rows = list(live) + [-1]
        new = [tokens(1) for _ in live]
        x = {a: torch.cat([t[a] for t in new] + [torch.zeros_like(new[0][a])]).cuda() for a in new[0]}
        rr = ints(rows)
        want = ints([len(live[r]) + 1 for r in live] + [0])
        assert P.path_pages_reserve(table, held, owner, page, rr, want).tolist()[0] == 0
        out = P.path_decode_step_shared(x["q"], x["k"], x["v"], x["w"], x["beta"], kp, vp, table, lens,
                                        table[PRE], L0, state, rows=rr, log_f=x["log_f"] if gate else None,
                                        g_pages=gp, g_state=gs)
        lens[torch.tensor(list(live), device="cuda")] += 1
        for i, r in enumerate(live):
            live[r].append(new[i])
            if step not in (0, 1, 5, 6, 7, 9, 10, 17, steps - 1):
                continue
            full = {a: torch.cat([prefix[a]] + [t[a] for t in live[r]]).transpose(0, 1).unsqueeze(0)
                    for a in prefix}
            ref, _ = oracle.fwd(full["q"], full["k"], full["v"], full["w"], full["beta"],
                                full["log_f"] if gate else None)
            err = np.abs(out[i].double().cpu().numpy() - ref[0, :, -1]).max()
            assert err <= (1e-4 if dtype == F32 else 2e-2), f"step {step}, slot {r}: {err}"
        assert (out[len(live):] == 0).all()
