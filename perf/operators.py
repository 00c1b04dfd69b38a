"""Cases of the paged PaTH decode cache: the decode steps that read it and the moves of its pages.

Three groups, each with a plain form in elementary torch operations and, where ``own`` is true,
the calls that a serving program makes of the library:

- ``paged``: one decode step of a batch of sequences of different lengths whose keys and values
  lie in pages of one pool (in-place key update, then one-query softmax attention);
- ``shared``: the same for a batch whose sequences continue one long prefix. The prefix is kept
  once, as it was when it ended; each sequence carries the product of its Householder factors
  since then (``state``) and turns its query back by it;
- ``fork``, ``compact``, ``store``: copies of sequences for a beam step, the pool's pages moved
  to its front, a prefill's contiguous cache written into pages.

``own`` is set from outside.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one short conversation on a small model: latency is all there is
        dict(name="paged_one", op="paged", B=1, H=4, d=64, page=16, lmin=70, lmax=70, idle=0,
             dtype="bf16", gate=False),
        # fp32 with the forget gate: odd counts, an empty sequence, a padded batch
        dict(name="paged_fp32_gate", op="paged", B=5, H=7, d=64, page=16, lmin=0, lmax=1500,
             idle=3, dtype="f32", gate=True),
        # a training-sized model (24 heads of 64) with the forget gate, serving a mixed batch
        dict(name="paged_gate", op="paged", B=48, H=24, d=64, page=64, lmin=500, lmax=6000, idle=0,
             dtype="bf16", gate=True),
        # the decode workload's batch and heads (32 of 128), lengths from one token to 8K
        dict(name="paged_batch", op="paged", B=32, H=32, d=128, page=64, lmin=1, lmax=8192, idle=0,
             dtype="bf16", gate=False),
        # two samples of one short prompt
        dict(name="shared_one", op="shared", B=2, H=4, d=64, page=16, prefix=300, lmin=0, lmax=20,
             dtype="bf16", gate=False),
        # fp32 with the gate, a prefix that ends inside a page
        dict(name="shared_fp32_gate", op="shared", B=9, H=6, d=128, page=32, prefix=2047, lmin=0,
             lmax=300, dtype="f32", gate=True),
        # many samples of one long document, gated, 24 heads of 64
        dict(name="shared_gate", op="shared", B=96, H=24, d=64, page=64, prefix=16384, lmin=0,
             lmax=512, dtype="bf16", gate=True),
        # the decode workload's batch behind one 16K system prompt
        dict(name="shared_prompt", op="shared", B=32, H=32, d=128, page=64, prefix=16384, lmin=0,
             lmax=1024, dtype="bf16", gate=False),
        # a beam step of a small model: free the losers, fork the winners in their place
        dict(name="fork_small", op="fork", n=4, H=4, d=64, page=16, lmin=40, lmax=150,
             dtype="bf16", gate=False),
        # a beam step of the decode workload's model, own parts of 200 to 1500 tokens
        dict(name="fork_beams", op="fork", n=32, H=32, d=128, page=64, lmin=200, lmax=1500,
             dtype="bf16", gate=False),
        # after many sequences ended: the pool's pages in use move to its front
        dict(name="compact_pool", op="compact", pages=4096, slots=96, H=24, d=64, page=64,
             dtype="bf16", gate=True),
        # a prefill of B=8, L=4096 (24 heads of 64) goes into pages, ragged lengths
        dict(name="store_prefill", op="store", B=8, H=24, d=64, page=64, lmin=1, lmax=4096,
             dtype="bf16", gate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged", "paged", "shared", "shared", "shared", "fork", "compact", "store"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, H=_log(rng, 1, 32), d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             dtype=dtype, gate=rng.random() < 0.4)
    row = c["H"] * c["d"] * SIZE[dtype]  # bytes of one token's keys
    if op == "paged":
        c["B"] = _log(rng, 1, 64)
        c["lmax"] = min(_log(rng, 1, 16384), max(1, (900 << 20) // (row * c["B"])))
        c["lmin"] = rng.randint(0, c["lmax"])
        c["idle"] = rng.choice([0, 0, 1, 4])
    elif op == "shared":
        c["B"] = _log(rng, 2, 96 if dtype == "bf16" else 24)
        c["prefix"] = min(_log(rng, 64, 16384), (128 << 20) // row)
        c["lmax"] = _log(rng, 1, 1024)
        c["lmin"] = rng.randint(0, c["lmax"])
    elif op == "fork":
        c["n"] = _log(rng, 1, 32)
        c["lmax"] = min(_log(rng, 1, 4096), max(1, (400 << 20) // (row * c["n"])))
        c["lmin"] = rng.randint(0, c["lmax"])
    elif op == "compact":
        c["pages"] = max(16, min(_log(rng, 64, 8192), (600 << 20) // (row * c["page"])))
        c["slots"] = _log(rng, 2, 128)
    else:
        c["B"] = _log(rng, 1, 16)
        c["lmax"] = min(_log(rng, 1, 8192), max(1, (200 << 20) // (row * c["B"])))
        c["lmin"] = rng.randint(0, c["lmax"])
    return c


def _lens(c, n):
    """n lengths spread over lmin..lmax (the same for every seed; the last is lmax)."""
    span = c["lmax"] - c["lmin"]
    return [c["lmin"] + int(span * (((i + 1) * 0.6180339887) % 1.0)) for i in range(n - 1)] + [c["lmax"]]


def _compact_fill(c):
    """Which pages of the pool are in use before it is compacted: about two of three."""
    return [(p * 0.7548776662) % 1.0 < 0.66 for p in range(c["pages"])]


def work(case):
    c = case
    s, H, d = SIZE[c["dtype"]], c["H"], c["d"]
    gate = 4 if c["gate"] else 0
    if c["op"] in ("paged", "shared"):
        lens = _lens(c, c["B"])
        toks = sum(lens)
        # own keys read and written, values read, gate biases read and written
        b = toks * H * (3 * d * s + 2 * gate)
        # q, k_new, v_new, w, out and the new row's stores; beta and log f
        b += c["B"] * H * (7 * d * s + 4 + 2 * gate)
        f = toks * H * 8 * d + c["B"] * H * 4 * d
        if c["op"] == "shared":
            b += c["prefix"] * H * (2 * d * s + gate)      # the prefix, once for the batch
            b += c["B"] * H * (2 * d * d * 4 + 2 * gate)   # each sequence's state, read and written
            f += c["B"] * H * (c["prefix"] * 4 * d + 6 * d * d)
        return {"bytes": b, "flops": f}
    if c["op"] == "fork":
        lens = _lens(c, c["n"])
        # whole pages travel, and each child's state
        pages = sum(-(-n // c["page"]) for n in lens)
        b = 2 * pages * c["page"] * H * (2 * d * s + gate) + 2 * c["n"] * H * (d * d * 4 + gate)
        return {"bytes": b, "flops": 0}
    if c["op"] == "compact":
        fill = _compact_fill(c)
        used = sum(fill)
        moved = sum(fill[used:])
        return {"bytes": 2 * moved * c["page"] * H * (2 * d * s + gate) + 8 * c["pages"], "flops": 0}
    return {"bytes": 2 * sum(_lens(c, c["B"])) * H * (2 * d * s + gate), "flops": 0}


# ------------------------------------------------------------------------------- the inputs
class _Make:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.c = torch.Generator().manual_seed(seed)

    def randn(self, *shape, dtype=torch.float32):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=dtype)

    def rand(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda")

    def unit(self, *shape):
        w = self.randn(*shape)
        return w / w.norm(dim=-1, keepdim=True)

    def beta(self, *shape):
        return (2 * torch.sigmoid(self.randn(*shape))).clamp(0, 1.99)

    def log_f(self, *shape):
        return torch.nn.functional.logsigmoid(self.randn(*shape) + 3)

    def perm(self, n):
        return torch.randperm(n, generator=self.c).tolist()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(mk, c, pages):
    shape = (pages, c["H"], c["page"], c["d"])
    dt = DT[c["dtype"]]
    k, v = mk.randn(*shape, dtype=dt), mk.randn(*shape, dtype=dt)
    g = -0.07 * c["page"] * 4 * mk.rand(*shape[:3]) if c["gate"] else None
    return k, v, g


def _states(mk, slots, H, d):
    """Products of a few Householder factors, as decoding leaves them (fp32)."""
    S = torch.eye(d, device="cuda").expand(slots, H, d, d).contiguous()
    for _ in range(6):
        w, b = mk.unit(slots, H, d), mk.beta(slots, H)
        S -= w.unsqueeze(-1) * (b.unsqueeze(-1) * (S * w.unsqueeze(-1)).sum(-2)).unsqueeze(-2)
    return S


def prepare(case, seed):
    c = case
    mk = _Make(seed)
    if c["op"] in ("paged", "shared"):
        return _prepare_decode(c, mk)
    if c["op"] == "fork":
        return _prepare_fork(c, mk)
    if c["op"] == "compact":
        return _prepare_compact(c, mk)
    return _prepare_store(c, mk)


def _prepare_decode(c, mk):
    B, H, d, page = c["B"], c["H"], c["d"], c["page"]
    idle = c.get("idle", 0)
    prefix = c.get("prefix", 0)
    lens = _lens(c, B)
    M = -(-(c["lmax"] + 1) // page) + 1
    R = B + idle + 1
    need = [n // page + 1 for n in lens]
    npre = -(-prefix // page)
    N = sum(need) + npre + 5
    ids = mk.perm(N)
    slots = mk.perm(R)[:B]
    table = [[-1] * M for _ in range(R)]
    slot_len = [0] * R
    at = npre
    for b in range(B):
        table[slots[b]][: need[b]] = ids[at:at + need[b]]
        slot_len[slots[b]] = lens[b]
        at += need[b]
    k, v, g = _pool(mk, c, N)
    dt, nb = DT[c["dtype"]], B + idle
    if g is not None:  # biases as the gate leaves them: lower the older the key
        for b in range(B):
            if lens[b]:
                age = torch.arange(need[b] * page, device="cuda").sub(lens[b] - 1).clamp(max=0).float()
                idx = torch.tensor(table[slots[b]][: need[b]], device="cuda")
                g[idx] = (0.07 * age).view(need[b], 1, page) * (0.5 + mk.rand(need[b], H, 1))
        if prefix:
            age = torch.arange(npre * page, device="cuda").sub(prefix - 1).clamp(max=0).float()
            g[torch.tensor(ids[:npre], device="cuda")] = (0.002 * age).view(npre, 1, page) * (0.5 + mk.rand(1, H, 1))
    s = dict(c=c, k_pages=k, v_pages=v, g_pages=g, table=_ints(table), lens=_ints(slot_len),
             rows=_ints(slots + [-1] * idle), q=mk.randn(nb, H, d).to(dt),
             k_new=mk.randn(nb, H, d).to(dt), v_new=mk.randn(nb, H, d).to(dt),
             w=mk.unit(nb, H, d).to(dt), beta=mk.beta(nb, H),
             log_f=mk.log_f(nb, H) if c["gate"] else None,
             out=torch.zeros(nb, H, d, dtype=dt, device="cuda"), scale=d ** -0.5)
    # the scheduler's own view of the batch (host numbers it has anyway): which table entries
    # hold live rows, and the longest length
    live = [(b, j) for b in range(B) for j in range(need[b])]
    s["plan"] = dict(slots=torch.tensor(slots, device="cuda"), width=max(need),
                     lens=torch.tensor(lens, device="cuda"),
                     bj=torch.tensor(live, device="cuda").t().contiguous(),
                     last=torch.tensor([n // page for n in lens], device="cuda"),
                     off=torch.tensor([n % page for n in lens], device="cuda"))
    if prefix:
        s["prefix_table"] = _ints(ids[:npre])
        s["state"] = _states(mk, R, H, d)
        s["g_state"] = -0.3 * mk.rand(R, H) if c["gate"] else None
    return s


def _prepare_fork(c, mk):
    n, H, d, page = c["n"], c["H"], c["d"], c["page"]
    lens = _lens(c, n)
    need = [-(-x // page) for x in lens]
    R = 2 * n + 2
    M = max(need) + 2
    N = 2 * sum(need) + 2 * max(need) + 7
    ids = mk.perm(N)
    slots = mk.perm(R)
    parents, children = slots[:n], slots[n:2 * n]
    table, held, slot_len, owner = [[-1] * M for _ in range(R)], [0] * R, [0] * R, [-1] * N
    at = 0
    for i in range(n):
        # the children hold the parents' former copies, which this step frees first
        for r, cnt, ln in ((parents[i], need[i], lens[i]), (children[i], need[n - 1 - i], lens[n - 1 - i])):
            for j in range(cnt):
                table[r][j] = ids[at]
                owner[ids[at]] = r * M + j
                at += 1
            held[r], slot_len[r] = cnt, ln
    k, v, g = _pool(mk, c, N)
    total = sum(need)
    return dict(c=c, k_pages=k, v_pages=v, g_pages=g, table=_ints(table), held=_ints(held),
                lens=_ints(slot_len), owner=_ints(owner), parents=_ints(parents),
                children=_ints(children), state=_states(mk, R, H, d),
                g_state=-0.3 * mk.rand(R, H) if c["gate"] else None,
                moves=torch.zeros(max(n * M, 1), 2, dtype=torch.int32, device="cuda"),
                info=torch.zeros(4, dtype=torch.int32, device="cuda"), total=total)


def _prepare_compact(c, mk):
    N, R, page = c["pages"], c["slots"], c["page"]
    fill = _compact_fill(c)
    used = [p for p in range(N) if fill[p]]
    order = mk.perm(len(used))
    M = -(-len(used) // R) + 1
    table, held, owner = [[-1] * M for _ in range(R)], [0] * R, [-1] * N
    for i, o in enumerate(order):
        r = i % R
        table[r][held[r]] = used[o]
        owner[used[o]] = r * M + held[r]
        held[r] += 1
    k, v, g = _pool(mk, c, N)
    total = sum(fill[len(used):])
    t, o = _ints(table), _ints(owner)
    return dict(c=c, k_pages=k, v_pages=v, g_pages=g, table0=t, owner0=o, table=t.clone(),
                owner=o.clone(), held=_ints(held),
                moves=torch.zeros(N, 2, dtype=torch.int32, device="cuda"),
                info=torch.zeros(4, dtype=torch.int32, device="cuda"), total=total)


def _prepare_store(c, mk):
    B, H, d, page = c["B"], c["H"], c["d"], c["page"]
    lens = _lens(c, B)
    M = -(-c["lmax"] // page) + 1
    need = [-(-n // page) for n in lens]
    N = sum(need) + 3
    ids = mk.perm(N)
    R = B + 2
    slots = mk.perm(R)[:B]
    table = [[-1] * M for _ in range(R)]
    at = 0
    for b in range(B):
        table[slots[b]][: need[b]] = ids[at:at + need[b]]
        at += need[b]
    k, v, g = _pool(mk, c, N)
    cap, dt = c["lmax"] + 9, DT[c["dtype"]]
    live = [(b, j) for b in range(B) for j in range(need[b])]
    return dict(c=c, k_pages=k, v_pages=v, g_pages=g, table=_ints(table), rows=_ints(slots),
                tokens=_ints(lens), k_cache=mk.randn(B, H, cap, d, dtype=dt),
                v_cache=mk.randn(B, H, cap, d, dtype=dt),
                g_cache=-mk.rand(B, H, cap) if c["gate"] else None,
                plan=dict(bj=torch.tensor(live, device="cuda").reshape(-1, 2).t().contiguous()))


# ------------------------------------------------------------------------------- one pass
def run(state):
    op = state["c"]["op"]
    if own:
        return _own(state, op)
    return _PLAIN[op](state)


def _result(s, *names):
    return {n: s[n] for n in names if s.get(n) is not None}


def _own(s, op):
    import softmax_attention_block_b200 as P

    c = s["c"]
    if op in ("paged", "shared"):
        if "ws" not in s:  # a serving program keeps one workspace
            n = P.path_decode_paged_workspace_bytes(
                s["q"].shape[0], c["H"], s["table"].shape[1], c["page"], c["d"],
                s["q"].dtype, prefix_len=c.get("prefix", 0))
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        args = (s["q"], s["k_new"], s["v_new"], s["w"], s["beta"], s["k_pages"], s["v_pages"],
                s["table"], s["lens"])
        kw = dict(rows=s["rows"], scale=s["scale"], log_f=s["log_f"], g_pages=s["g_pages"],
                  out=s["out"], workspace=s["ws"])
        if op == "paged":
            P.path_decode_step_paged(*args, **kw)
            return _result(s, "out", "k_pages", "v_pages", "g_pages")
        P.path_decode_step_shared(*args, s["prefix_table"], c["prefix"], s["state"],
                                  g_state=s["g_state"], **kw)
        return _result(s, "out", "k_pages", "v_pages", "g_pages", "state", "g_state")
    if op == "fork":
        P.path_pages_free(s["table"], s["held"], s["lens"], s["owner"], s["children"])
        P.path_pages_fork(s["table"], s["held"], s["lens"], s["owner"], c["page"], s["parents"],
                          s["children"], moves=s["moves"], info=s["info"])
        P.path_pages_copy(s["moves"], s["info"], s["k_pages"], s["v_pages"], g_pages=s["g_pages"])
        P.path_state_copy(s["state"], s["parents"], s["children"], g_state=s["g_state"])
        return _result(s, "table", "held", "lens", "owner", "moves", "info", "k_pages", "v_pages",
                       "g_pages", "state", "g_state")
    if op == "compact":
        # the pass starts from the tables as they were, so that it can be made again
        s["table"].copy_(s["table0"])
        s["owner"].copy_(s["owner0"])
        P.path_pages_compact(s["table"], s["held"], s["owner"], moves=s["moves"], info=s["info"])
        P.path_pages_copy(s["moves"], s["info"], s["k_pages"], s["v_pages"], g_pages=s["g_pages"])
        return _result(s, "table", "owner", "moves", "info", "k_pages", "v_pages", "g_pages")
    P.path_pages_store(s["k_cache"], s["v_cache"], s["k_pages"], s["v_pages"], s["table"],
                       s["rows"], s["tokens"], g_cache=s["g_cache"], g_pages=s["g_pages"])
    return _result(s, "k_pages", "v_pages", "g_pages")


# ------------------------------------------------------------------------------- plain forms
def _plain_own_part(s):
    """The sequences' own pages: update them in place, and return logits [B,H,n+1] (masked) and
    values [B,H,n+1,d] of the live keys with the new one last."""
    c, p = s["c"], s["plan"]
    B, H, d, page = c["B"], c["H"], c["d"], c["page"]
    dt = s["k_pages"].dtype
    q, w = s["q"][:B].float(), s["w"][:B].float()
    ids = s["table"][p["slots"], : p["width"]].long().clamp(min=0)          # [B, P]
    n = ids.shape[1] * page
    pos = torch.arange(n, device=q.device)
    live = (pos < p["lens"].unsqueeze(1)).unsqueeze(1)                        # [B, 1, n]
    old = s["k_pages"][ids].transpose(2, 3).reshape(B, n, H, d).transpose(1, 2)  # [B, H, n, d]
    k = old.float()
    wk = (k * w.unsqueeze(2)).sum(-1)
    k = k - (s["beta"][:B].unsqueeze(-1) * wk).unsqueeze(-1) * w.unsqueeze(2)
    k = k.to(dt)
    k = torch.where(live.unsqueeze(-1), k, old)
    new_pages = k.view(B, H, -1, page, d).permute(0, 2, 1, 3, 4)
    bj = p["bj"]
    at = ids[bj[0], bj[1]]
    s["k_pages"][at] = new_pages[bj[0], bj[1]]
    z = (k.float() * q.unsqueeze(2)).sum(-1) * s["scale"]
    if s["g_pages"] is not None:
        g = s["g_pages"][ids].transpose(2, 3).reshape(B, n, H).transpose(1, 2)
        g = torch.where(live, g + s["log_f"][:B].unsqueeze(-1), g)
        s["g_pages"][at] = g.view(B, H, -1, page).permute(0, 2, 1, 3)[bj[0], bj[1]]
        z = z + g
    z = z.masked_fill(~live, -math.inf)
    v = s["v_pages"][ids].transpose(2, 3).reshape(B, n, H, d).transpose(1, 2).float()
    v = torch.where(live.unsqueeze(-1), v, torch.zeros((), device=v.device))
    # the new token's row
    last = ids.gather(1, p["last"].unsqueeze(1)).squeeze(1)
    s["k_pages"][last, :, p["off"]] = s["k_new"][:B]
    s["v_pages"][last, :, p["off"]] = s["v_new"][:B]
    if s["g_pages"] is not None:
        s["g_pages"][last, :, p["off"]] = 0.0
    zn = (s["k_new"][:B].float() * q).sum(-1, keepdim=True) * s["scale"]
    return torch.cat([z, zn], -1), torch.cat([v, s["v_new"][:B].float().unsqueeze(2)], 2)


def _weights(z):
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_paged(s):
    B = s["c"]["B"]
    z, v = _plain_own_part(s)
    s["out"][:B] = (_weights(z).unsqueeze(2) @ v).squeeze(2).to(s["out"].dtype)
    return _result(s, "out", "k_pages", "v_pages", "g_pages")


def _plain_shared(s):
    c, p = s["c"], s["plan"]
    B, H, d, n = c["B"], c["H"], c["d"], c["prefix"]
    q, w, beta = s["q"].float(), s["w"].float(), s["beta"]
    # the product of the factors since the prefix ended, and the query turned back by it
    S = s["state"][p["slots"]]
    S = S - w.unsqueeze(-1) * (beta.unsqueeze(-1) * (w.unsqueeze(2) @ S).squeeze(2)).unsqueeze(2)
    s["state"][p["slots"]] = S
    qt = (q.unsqueeze(2) @ S).squeeze(2)                                      # S^T q
    ids = s["prefix_table"].long()
    kp = s["k_pages"][ids].transpose(1, 2).reshape(-1, H, d)[:n].transpose(0, 1).float()  # [H, n, d]
    vp = s["v_pages"][ids].transpose(1, 2).reshape(-1, H, d)[:n].transpose(0, 1).float()
    zp = (qt.transpose(0, 1) @ kp.transpose(1, 2)).transpose(0, 1) * s["scale"]          # [B, H, n]
    if s["g_state"] is not None:
        gs = s["g_state"][p["slots"]] + s["log_f"]
        s["g_state"][p["slots"]] = gs
        gp = s["g_pages"][ids].transpose(1, 2).reshape(-1, H)[:n].t()
        zp = zp + gp.unsqueeze(0) + gs.unsqueeze(-1)
    z, v = _plain_own_part(s)
    a = _weights(torch.cat([zp, z], -1))
    o = (a[..., :n].transpose(0, 1) @ vp).transpose(0, 1)
    o = o + (a[..., n:].unsqueeze(2) @ v).squeeze(2)
    s["out"].copy_(o.to(s["out"].dtype))
    return _result(s, "out", "k_pages", "v_pages", "g_pages", "state", "g_state")


def _plain_copy(s, total):
    src, dst = s["moves"][:total, 0].long(), s["moves"][:total, 1].long()
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]
    if s["g_pages"] is not None:
        s["g_pages"][dst] = s["g_pages"][src]


def _scatter(dst, idx, val):
    """dst[idx] = val, where an index equal to len(dst) writes nothing."""
    pad = torch.cat([dst, dst[:1]])
    pad[idx] = val
    dst.copy_(pad[:-1])


def _plain_fork(s):
    page, N, M = s["c"]["page"], s["owner"].numel(), s["table"].shape[1]
    par, chi = s["parents"].long(), s["children"].long()
    minus = torch.full((), -1, dtype=torch.int32, device=par.device)
    old = s["table"][chi].long()
    _scatter(s["owner"], torch.where(old >= 0, old, N).reshape(-1), minus)
    # the lowest free pages, in order, for the children's rows in order
    need = (s["lens"][par].long() + page - 1) // page
    off = need.cumsum(0) - need
    free = torch.argsort((s["owner"] >= 0).to(torch.int8), stable=True)
    j = torch.arange(M, device=par.device)
    take = j < need.unsqueeze(1)
    at = torch.where(take, off.unsqueeze(1) + j, 0)
    new = torch.where(take, free[at], -1)
    src = s["table"][par].long()
    s["table"][chi] = new.int()
    _scatter(s["owner"], torch.where(take, new, N).reshape(-1),
             (chi.unsqueeze(1) * M + j).int().reshape(-1))
    s["held"][chi] = need.int()
    s["lens"][chi] = s["lens"][par]
    _scatter(s["moves"], torch.where(take, at, s["moves"].shape[0]).reshape(-1),
             torch.stack([src, new], -1).int().reshape(-1, 2))
    total = need.sum()
    s["info"].copy_(torch.stack([torch.zeros_like(total), total, (s["owner"] >= 0).sum(), total]).int())
    _plain_copy(s, s["total"])
    s["state"][chi] = s["state"][par]
    if s["g_state"] is not None:
        s["g_state"][chi] = s["g_state"][par]
    return _result(s, "table", "held", "lens", "owner", "moves", "info", "k_pages", "v_pages",
                   "g_pages", "state", "g_state")


def _plain_compact(s):
    s["table"].copy_(s["table0"])
    s["owner"].copy_(s["owner0"])
    total, N = s["total"], s["owner"].numel()
    used = s["owner"] >= 0
    count = used.sum()
    low = torch.arange(N, device=used.device) < count
    src = torch.argsort((~(used & ~low)).to(torch.int8), stable=True)[:total]
    dst = torch.argsort((~(~used & low)).to(torch.int8), stable=True)[:total]
    who = s["owner"][src]
    s["table"].view(-1)[who.long()] = dst.int()
    s["owner"][dst] = who
    s["owner"][src] = -1
    s["moves"][:total] = torch.stack([src, dst], -1).int()
    zero = torch.zeros_like(count)
    s["info"].copy_(torch.stack([zero, (used & ~low).sum(), count, zero]).int())
    _plain_copy(s, total)
    return _result(s, "table", "owner", "moves", "info", "k_pages", "v_pages", "g_pages")


def _plain_store(s):
    page, bj = s["c"]["page"], s["plan"]["bj"]
    ids = s["table"][s["rows"].long()[bj[0]], bj[1]].long()
    t = bj[1].unsqueeze(1) * page + torch.arange(page, device=ids.device)      # [live pages, page]
    keep = (t < s["tokens"].long()[bj[0]].unsqueeze(1)).unsqueeze(1)           # [., 1, page]
    t = t.clamp(max=s["k_cache"].shape[2] - 1)
    b = bj[0].unsqueeze(1)
    rows = s["k_cache"].transpose(1, 2)[b, t].transpose(1, 2)                  # [., H, page, d]
    s["k_pages"][ids] = torch.where(keep.unsqueeze(-1), rows, s["k_pages"][ids])
    rows = s["v_cache"].transpose(1, 2)[b, t].transpose(1, 2)
    s["v_pages"][ids] = torch.where(keep.unsqueeze(-1), rows, s["v_pages"][ids])
    if s["g_pages"] is not None:
        rows = s["g_cache"].transpose(1, 2)[b, t].transpose(1, 2)
        s["g_pages"][ids] = torch.where(keep, rows, s["g_pages"][ids])
    return _result(s, "k_pages", "v_pages", "g_pages")


_PLAIN = dict(paged=_plain_paged, shared=_plain_shared, fork=_plain_fork, compact=_plain_compact,
              store=_plain_store)


# ------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The definition, sequence by sequence: every Householder factor is applied to the keys,
    the prefix's too; pages move one by one."""
    s = prepare(case, seed)
    if case["op"] in ("paged", "shared"):
        return _exact_decode(case, s)
    if case["op"] == "store":
        return _exact_store(case, s)
    return _exact_moves(case, s)


def _exact_decode(c, s):
    page, d, B = c["page"], c["d"], c["B"]
    dt = s["k_pages"].dtype
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    gp = s["g_pages"].double() if s["g_pages"] is not None else None
    out = s["out"].double()
    table, lens, rows = s["table"].tolist(), s["lens"].tolist(), s["rows"].tolist()
    state = s["state"].double() if "state" in s else None
    gstate = s["g_state"].double() if s.get("g_state") is not None else None
    if state is not None:
        n = c["prefix"]
        ids = s["prefix_table"].long()
        pk = torch.cat(list(s["k_pages"][ids]), 1)[:, :n].double()            # [H, n, d]
        pv = torch.cat(list(s["v_pages"][ids]), 1)[:, :n].double()
        pg = torch.cat(list(s["g_pages"][ids]), 1)[:, :n].double() if gp is not None else None
    for b in range(B):
        r = rows[b]
        n_own = lens[r]
        q, w = s["q"][b].double(), s["w"][b].double()
        beta = s["beta"][b].double()
        Hm = torch.eye(d, dtype=torch.float64, device=q.device) - beta[:, None, None] * w[:, :, None] * w[:, None, :]
        ids = torch.tensor(table[r][: n_own // page + 1], device=q.device)
        k = torch.cat(list(s["k_pages"][ids]), 1)[:, :n_own].double() @ Hm      # H is symmetric
        v = torch.cat(list(s["v_pages"][ids]), 1)[:, :n_own].double()
        keys = torch.cat([k.to(dt).double(), s["k_new"][b].double().unsqueeze(1)], 1)
        vals = torch.cat([v, s["v_new"][b].double().unsqueeze(1)], 1)
        z = s["scale"] * (keys @ q.unsqueeze(-1)).squeeze(-1)
        g = None
        if gp is not None:
            g = torch.cat(list(s["g_pages"][ids]), 1)[:, :n_own].double() + s["log_f"][b].double().unsqueeze(-1)
            g = torch.cat([g, torch.zeros_like(g[:, :1]) if n_own else torch.zeros(c["H"], 1, dtype=torch.float64, device=q.device)], 1)
            z = z + g
        if state is not None:
            state[r] = Hm @ state[r]
            zp = s["scale"] * ((pk @ state[r].transpose(-1, -2)) @ q.unsqueeze(-1)).squeeze(-1)
            if gp is not None:
                gstate[r] = gstate[r] + s["log_f"][b].double()
                zp = zp + pg + gstate[r].unsqueeze(-1)
            z, vals = torch.cat([zp, z], 1), torch.cat([pv, vals], 1)
        a = torch.softmax(z, -1)
        out[b] = (a.unsqueeze(1) @ vals).squeeze(1)
        own_rows = torch.cat([k, s["k_new"][b].double().unsqueeze(1)], 1)
        for j, pid in enumerate(ids.tolist()):
            m = min(page, n_own + 1 - j * page)
            kp[pid, :, :m] = own_rows[:, j * page: j * page + m]
            if gp is not None:
                gp[pid, :, :m] = g[:, j * page: j * page + m]
        vp[int(ids[n_own // page]), :, n_own % page] = s["v_new"][b].double()
    r = dict(out=out, k_pages=kp, v_pages=vp, g_pages=gp, state=state, g_state=gstate)
    return {n: t for n, t in r.items() if t is not None}


def _exact_moves(c, s):
    M = s["table"].shape[1]
    names = ("k_pages", "v_pages", "g_pages")
    pools = {n: s[n].double() for n in names if s[n] is not None}
    owner, moves = s["owner"].tolist(), []
    if c["op"] == "fork":
        par, chi, lens = s["parents"].tolist(), s["children"].tolist(), s["lens"].tolist()
        table = s["table"].tolist()
        for x in chi:
            for p in table[x]:
                if p >= 0:
                    owner[p] = -1
        taken = iter([p for p, o in enumerate(owner) if o < 0])
        for a, x in zip(par, chi):
            for j in range(-(-lens[a] // c["page"])):
                moves.append((table[a][j], next(taken)))
    else:
        used = sum(o >= 0 for o in owner)
        gaps = iter([p for p in range(used) if owner[p] < 0])
        moves = [(p, next(gaps)) for p in range(used, len(owner)) if owner[p] >= 0]
    for a, x in moves:
        for t in pools.values():
            t[x] = t[a]
    out = dict(table=None, owner=None, moves=None, info=None, **pools)
    if c["op"] == "fork":
        st = s["state"].double()
        gs = s["g_state"].double() if s["g_state"] is not None else None
        for a, x in zip(par, chi):
            st[x] = st[a]
            if gs is not None:
                gs[x] = gs[a]
        out.update(held=None, lens=None, state=st, g_state=gs)
    return out


def _exact_store(c, s):
    names = (("k_pages", "k_cache"), ("v_pages", "v_cache"), ("g_pages", "g_cache"))
    out = {}
    table, page = s["table"].tolist(), c["page"]
    for pool, cache in names:
        if s[pool] is None:
            continue
        t = s[pool].double()
        for b, (r, n) in enumerate(zip(s["rows"].tolist(), s["tokens"].tolist())):
            for j in range(-(-n // page)):
                m = min(page, n - j * page)
                t[table[r][j], :, :m] = s[cache][b, :, j * page: j * page + m].double()
        out[pool] = t
    return out
