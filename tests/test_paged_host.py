"""Host-side checks of the paged decode cache (no GPU): sizes and refusals of the C ABI, which
validates before it launches anything, and the binding's checks of shapes and dtypes."""
import pytest
import torch

import softmax_attention_block_b200 as P

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16, MIXED = 0, 1, 2
FAKE = 0x1000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(P.LIB_PATH):
        from softmax_attention_block_b200 import build

        build.build()
    return P.lib()


def test_workspace_sizes(lib):
    f = lib.path_decode_paged_workspace_bytes
    base = f(8, 24, 100, 64, 64, BF16, 0)
    assert base > 0 and base % 256 == 0
    for more in ((9, 24, 100, 64, 64, BF16, 0), (8, 25, 100, 64, 64, BF16, 0), (8, 24, 300, 64, 64, BF16, 0),
                 (8, 24, 100, 128, 64, BF16, 0), (8, 24, 100, 64, 64, BF16, 1), (8, 24, 100, 64, 64, F32, 0)):
        assert f(*more) >= base
    assert f(8, 24, 100, 64, 64, BF16, 9000) >= f(8, 24, 100, 64, 64, BF16, 100) > base
    for dt in (BF16, F32):
        sizes = [f(b, 24, 100, 64, 128, dt, 5000) for b in range(1, 300)]
        assert sizes == sorted(sizes)
    for bad in ((0, 1, 1, 16, 64, BF16, 0), (1, 1, 0, 16, 64, BF16, 0), (1, 1, 1, 8, 64, BF16, 0),
                (1, 1, 1, 48, 64, BF16, 0), (1, 1, 1, 2048, 64, BF16, 0), (1, 1, 1, 16, 96, BF16, 0),
                (1, 1, 1, 16, 64, MIXED, 0), (1, 1, 1, 16, 64, BF16, -1), (65536, 1, 1, 16, 64, BF16, 0),
                (1, 1, 1 << 27, 16, 64, BF16, 0)):
        assert f(*bad) == 0, bad


def step(lib, shared=False, **kw):
    a = dict(q=FAKE, k_new=FAKE, v_new=FAKE, w=FAKE, beta=FAKE, log_f=None, scale=0.1, B=2, H=3, d=64, dt=BF16,
             k=FAKE, v=FAKE, g=None, N=10, page=16, table=FAKE, R=4, M=5, lens=FAKE, rows=FAKE, pt=FAKE, plen=20,
             state=FAKE, gs=None, out=FAKE, ws=None, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    args = [a[n] for n in ("q", "k_new", "v_new", "w", "beta", "log_f", "scale", "B", "H", "d", "dt", "k", "v", "g",
                           "N", "page", "table", "R", "M", "lens", "rows")]
    if shared:
        args += [a[n] for n in ("pt", "plen", "state", "gs")]
    f = lib.path_decode_step_shared if shared else lib.path_decode_step_paged
    return f(*args, a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("shared", [False, True])
def test_step_refusals(lib, shared):
    assert step(lib, shared) == WORKSPACE  # everything else is in order
    for n in ("q", "k_new", "v_new", "w", "beta", "k", "v", "table", "lens", "out"):
        assert step(lib, shared, **{n: None}) == INVALID, n
    for n in ("q", "k_new", "v_new", "w", "k", "v"):
        assert step(lib, shared, **{n: FAKE + 8}) == INVALID, n
    for n in ("B", "H", "N", "R", "M"):
        assert step(lib, shared, **{n: 0}) == INVALID, n
    gate = dict(log_f=FAKE, gs=FAKE)
    assert step(lib, shared, g=FAKE, **gate) == WORKSPACE
    assert step(lib, shared, g=FAKE + 8, **gate) == INVALID
    assert step(lib, shared, scale=float("inf")) == INVALID
    assert step(lib, shared, log_f=FAKE) == INVALID
    assert step(lib, shared, g=FAKE) == INVALID
    assert step(lib, shared, rows=None, B=5) == INVALID  # more rows than slots
    assert step(lib, shared, rows=None, B=4) == WORKSPACE
    assert step(lib, shared, ws=FAKE, wsb=100) == WORKSPACE
    assert step(lib, shared, ws=FAKE + 16) == INVALID
    for bad in (dict(page=24), dict(page=8), dict(page=2048), dict(d=32), dict(dt=MIXED), dict(B=70000),
                dict(N=1 << 30), dict(R=1 << 30, M=4), dict(M=(1 << 26) + 1)):
        assert step(lib, shared, **bad) == UNSUPPORTED, bad
    if shared:
        for bad in (dict(pt=None), dict(plen=0), dict(plen=-1), dict(state=None), dict(state=FAKE + 4),
                    dict(gs=FAKE), dict(log_f=FAKE, g=FAKE)):
            assert step(lib, shared, **bad) == INVALID, bad
        assert step(lib, shared, plen=(1 << 30) + 1) == UNSUPPORTED


def test_table_refusals(lib):
    def reserve(table=FAKE, held=FAKE, owner=FAKE, R=4, M=5, N=10, page=16, rows=FAKE, tokens=FAKE, n=0, info=FAKE):
        return lib.path_pages_reserve(table, held, owner, R, M, N, page, rows, tokens, n, info, None)

    def fork(table=FAKE, held=FAKE, lens=FAKE, owner=FAKE, R=4, M=5, N=10, page=16, par=FAKE, kids=FAKE, n=2,
             moves=FAKE, most=9, info=FAKE):
        return lib.path_pages_fork(table, held, lens, owner, R, M, N, page, par, kids, n, moves, most, info, None)

    assert reserve() == INVALID  # n = 0
    for n in ("table", "held", "owner", "rows", "tokens", "info"):
        assert reserve(n=1, **{n: None}) == INVALID
    for n in ("R", "M", "N"):
        assert reserve(n=1, **{n: 0}) == INVALID
    assert reserve(n=1, page=17) == UNSUPPORTED
    assert reserve(n=4097) == UNSUPPORTED
    assert reserve(n=1, R=1 << 16, M=1 << 15) == UNSUPPORTED
    assert fork() == INVALID  # 9 moves where 10 pages may move
    assert fork(n=1, most=4) == INVALID
    for n in ("table", "held", "lens", "owner", "par", "kids", "moves", "info"):
        assert fork(most=10, **{n: None}) == INVALID
    assert fork(most=1 << 20, n=4097) == UNSUPPORTED
    assert lib.path_pages_free(None, FAKE, FAKE, FAKE, 4, 5, 10, FAKE, 1, None) == INVALID
    assert lib.path_pages_free(FAKE, FAKE, FAKE, FAKE, 4, 5, 10, FAKE, 0, None) == INVALID
    assert lib.path_pages_compact(FAKE, FAKE, FAKE, 4, 5, 10, FAKE, 4, FAKE, None) == INVALID
    assert lib.path_pages_compact(FAKE, FAKE, FAKE, 4, 5, 10, FAKE, 5, None, None) == INVALID


def test_copy_and_store_refusals(lib):
    def copy(moves=FAKE, most=3, info=FAKE, k=FAKE, v=FAKE, g=None, N=10, H=2, page=16, d=64, dt=BF16):
        return lib.path_pages_copy(moves, most, info, k, v, g, N, H, page, d, dt, None)

    def store(kc=FAKE, vc=FAKE, gc=None, B=2, H=3, d=64, cap=40, dt=BF16, k=FAKE, v=FAKE, g=None, N=10, page=16,
              table=FAKE, R=4, M=5, rows=FAKE, tokens=FAKE):
        return lib.path_pages_store(kc, vc, gc, B, H, d, cap, dt, k, v, g, N, page, table, R, M, rows, tokens, None,
                                    None)

    for bad in (dict(moves=None), dict(info=None), dict(k=None), dict(v=None), dict(most=-1), dict(N=0), dict(H=0),
                dict(k=FAKE + 8), dict(g=FAKE + 4)):
        assert copy(**bad) == INVALID, bad
    for bad in (dict(page=20), dict(d=16), dict(dt=MIXED), dict(N=1 << 27, H=1)):
        assert copy(**bad) == UNSUPPORTED, bad
    for bad in (dict(kc=None), dict(vc=None), dict(k=None), dict(v=None), dict(table=None), dict(tokens=None),
                dict(gc=FAKE), dict(g=FAKE), dict(B=0), dict(cap=0), dict(rows=None, B=5), dict(kc=FAKE + 2)):
        assert store(**bad) == INVALID, bad
    for bad in (dict(page=20), dict(d=16), dict(dt=MIXED), dict(B=70000)):
        assert store(**bad) == UNSUPPORTED, bad
    assert lib.path_state_copy(None, None, 4, 2, 64, FAKE, FAKE, 1, None) == INVALID
    assert lib.path_state_copy(FAKE, None, 4, 2, 64, FAKE, FAKE, 0, None) == INVALID
    assert lib.path_state_copy(FAKE + 4, None, 4, 2, 64, FAKE, FAKE, 1, None) == INVALID
    assert lib.path_state_copy(FAKE, None, 4, 2, 32, FAKE, FAKE, 1, None) == UNSUPPORTED
    assert b"page" in lib.path_status_string(P.PATH_ERR_PAGE)


# ------------------------------------------------------------------------ the binding
B, H, D, PAGE, N, R, M = 2, 3, 64, 16, 7, 4, 2
I32 = torch.int32


def z(*s, dt=torch.bfloat16):
    return torch.zeros(*s, dtype=dt)


def bind(shared=False, **over):
    a = dict(q=z(B, H, D), k_new=z(B, H, D), v_new=z(B, H, D), w=z(B, H, D), beta=z(B, H, dt=torch.float32),
             k_pages=z(N, H, PAGE, D), v_pages=z(N, H, PAGE, D), table=z(R, M, dt=I32), lens=z(R, dt=I32),
             rows=None, log_f=None, g_pages=None, out=None)
    if shared:
        a.update(prefix_table=z(2, dt=I32), prefix_len=20, state=z(R, H, D, D, dt=torch.float32), g_state=None)
    a.update(over)
    return (P.path_decode_step_shared if shared else P.path_decode_step_paged)(**a)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("over,msg", [
    (dict(q=z(B, H, D + 8)), "q: shape"),
    (dict(q=z(H, D)), "q must be"),
    (dict(v_new=z(B, H, D, dt=torch.float32)), "v_new: dtype"),
    (dict(beta=z(B, H + 1, dt=torch.float32)), "beta: shape"),
    (dict(k_pages=z(N, H, PAGE, D, dt=torch.float16)), "k_pages must be"),
    (dict(v_pages=z(N, H, PAGE + 1, D)), "v_pages: shape"),
    (dict(table=z(R, M, dt=torch.int64)), "table: dtype"),
    (dict(table=z(R, dt=I32)), "table must be"),
    (dict(lens=z(R + 1, dt=I32)), "lens: shape"),
    (dict(rows=z(B, dt=torch.int64)), "rows: dtype"),
    (dict(rows=z(B + 1, dt=I32)), "rows: shape"),
    (dict(log_f=z(B, H, dt=torch.float32)), "go together"),
    (dict(g_pages=z(N, H, PAGE + 1, dt=torch.float32)), "g_pages: shape"),
    (dict(out=z(B, H, D, dt=torch.float32)), "out: dtype"),
    (dict(), "CUDA tensors"),
])
def test_step_checks(shared, over, msg):
    with pytest.raises(ValueError, match=msg):
        bind(shared, **over)


@pytest.mark.parametrize("over,msg", [
    (dict(prefix_table=z(2, dt=torch.int64)), "prefix_table: dtype"),
    (dict(prefix_len=33), "do not hold"),
    (dict(state=z(R, H, D, D)), "state: dtype"),
    (dict(state=z(B, H, D, D, dt=torch.float32)), "state: shape"),
    (dict(g_state=z(R, H, dt=torch.float32)), "go together"),
])
def test_shared_checks(over, msg):
    with pytest.raises(ValueError, match=msg):
        bind(True, **over)


def test_table_checks():
    table, held, lens, owner = z(R, M, dt=I32), z(R, dt=I32), z(R, dt=I32), z(N, dt=I32)
    a = z(2, dt=I32)
    with pytest.raises(ValueError, match="tokens: shape"):
        P.path_pages_reserve(table, held, owner, 16, a, z(3, dt=I32))
    with pytest.raises(ValueError, match="held: shape"):
        P.path_pages_reserve(table, z(R + 1, dt=I32), owner, 16, a, a)
    with pytest.raises(ValueError, match="owner: dtype"):
        P.path_pages_reserve(table, held, z(N, dt=torch.int64), 16, a, a)
    with pytest.raises(ValueError, match="info: shape"):
        P.path_pages_reserve(table, held, owner, 16, a, a, info=z(3, dt=I32))
    with pytest.raises(ValueError, match="moves: shape"):
        P.path_pages_fork(table, held, lens, owner, 16, a, a, moves=z(8, 3, dt=I32))
    with pytest.raises(ValueError, match="children: shape"):
        P.path_pages_fork(table, held, lens, owner, 16, a, z(3, dt=I32))
    with pytest.raises(ValueError, match="one dimension"):
        P.path_pages_free(table, held, lens, owner, z(2, 1, dt=I32))
    with pytest.raises(ValueError, match="CUDA tensors"):
        P.path_pages_compact(table, held, owner)
    k = z(N, H, PAGE, D)
    with pytest.raises(ValueError, match="moves must be"):
        P.path_pages_copy(a, z(4, dt=I32), k, k.clone())
    with pytest.raises(ValueError, match="v_pages: shape"):
        P.path_pages_copy(z(4, 2, dt=I32), z(4, dt=I32), k, z(N + 1, H, PAGE, D))
    kc = z(B, H, 30, D)
    with pytest.raises(ValueError, match="v_cache: shape"):
        P.path_pages_store(kc, z(B, H, 31, D), k, k.clone(), table, a, a)
    with pytest.raises(ValueError, match="go together"):
        P.path_pages_store(kc, kc.clone(), k, k.clone(), table, a, a, g_cache=z(B, H, 30, dt=torch.float32))
    with pytest.raises(ValueError, match="tokens: shape"):
        P.path_pages_store(kc, kc.clone(), k, k.clone(), table, a, z(3, dt=I32))
    with pytest.raises(ValueError, match="state: shape"):
        P.path_state_copy(z(R, H, D, D + 1, dt=torch.float32), a, a)
    with pytest.raises(ValueError, match="CUDA tensors"):
        P.path_state_copy(z(R, H, D, D, dt=torch.float32), a, a)


def test_the_readme_step_advances_the_rows_it_names():
    """README's step as it stands there, its calls replaced: with idle rows in the batch it asks for one
    token more for each slot in it and advances these slots' lengths, no other's."""
    import os
    import types

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    block = text.split("## A server's step")[1].split("\n\n    ")[1].split("\n\n")[0]
    asked = []
    names = dict(torch=torch, q=0, k=0, v=0, w=0, beta=0, k_pages=0, v_pages=0, ws=0, page=16, state=0, held=0,
                 owner=0, prefix_len=20, prefix_slot=3, table=z(5, 2, dt=I32))
    names["lens"] = torch.tensor([7, 8, 9, 10, 11], dtype=I32)
    names["rows"] = torch.tensor([2, -1, 0, -7], dtype=I32)
    names["path_pages_reserve"] = lambda t, h, o, p, rows, tokens: asked.append((rows, tokens))
    names["path_decode_step_shared"] = lambda *a, **kw: types.SimpleNamespace()
    exec("import torch\n" + "\n".join(line.removeprefix("    ") for line in block.split("\n")), names)
    rows, tokens = asked[0]
    assert tokens.dtype == I32 and [int(n) for r, n in zip(rows, tokens) if r >= 0] == [10, 8]
    assert names["lens"].tolist() == [8, 8, 10, 10, 11]
