"""The training operators against their definitions in 64 bits: types, odd
sizes, strides and offsets, one token to many, masked and empty rows, in
place, on streams and in CUDA graphs, gradients against differences.

Bounds: an output is rounded once to its type (half a unit in its last
place); before that every binary32 operation adds at most 2^-24 of the
magnitudes that it works on, so a sum of n terms is off by at most n 2^-24 of
the sum of their magnitudes, and the short chains around it by a small
multiple.  The multiples are stated where each check is made.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import collective_communication_algorithms_gb300 as hc  # noqa: E402
from training_util import (D, assert_close, distill, embedding, embedding_grad, block_norm, guarded,  # noqa: E402
                           strided)

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from collective_communication_algorithms_gb300 import build
    build.build()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def some_ids(g, tokens, vocab, kind, dtype=torch.int64):
    if kind == "uniform":
        ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    elif kind == "skewed":  # a few rows hold most tokens; some padding
        u = torch.rand(tokens, generator=g, device="cuda")
        ids = (torch.exp(u * math.log(vocab + 1)).long() - 1).clamp(0, vocab - 1)
        ids[torch.rand(tokens, generator=g, device="cuda") < 0.05] = -1
    elif kind == "one":
        ids = torch.full((tokens,), vocab // 2, device="cuda")
    elif kind == "none":
        ids = torch.full((tokens,), -1, device="cuda")
    else:  # every row once or twice, descending
        ids = (vocab - 1 - torch.arange(tokens, device="cuda") // 2) % vocab
    return ids.to(dtype)


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("table_dtype,out_dtype", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("tokens,rows,dim", [(1, 5, 1), (3, 7, 8), (65, 50, 33), (257, 1000, 1000), (4099, 300, 264),
                                             (2, 3, 20001), (9000, 64, 2056)])
def test_embedding(table_dtype, out_dtype, tokens, rows, dim):
    g = gen(tokens + dim)
    table = normal(g, rows, dim, dtype=table_dtype)
    first = 10
    ids = some_ids(g, tokens, rows + 20, "uniform", torch.int32 if dim % 2 else torch.int64)
    out, intact = guarded(tokens, dim, out_dtype)
    hc.embedding(table, ids, out=out, scale=1.7, first_id=first)
    ref = embedding(table, ids, torch.tensor(1.7, dtype=F32).double().item(), first)
    assert_close(out, ref, ref.abs(), 1, "out")
    assert intact()


@pytest.mark.parametrize("stride,offset", [(40, 0), (41, 0), (48, 3), (33, 8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_embedding_strided(dtype, stride, offset):
    g = gen(stride)
    table = strided(normal(g, 11, 33, dtype=dtype), stride, offset)
    ids = some_ids(g, 100, 11, "uniform")[1:]  # an offset of 8 bytes
    out, intact = guarded(99, 33, dtype, stride + 2, offset)
    hc.embedding(table, ids, out=out)
    assert torch.equal(out, table[ids])
    assert intact()


def test_embedding_far_ids():
    """Ids whose distance to first_id does not fit 64 bits are elsewhere."""
    table = normal(gen(1), 4, 16)
    big = 2 ** 63 - 1
    ids = torch.tensor([-big - 1, big, 2, -5, 0, 2 ** 40], device="cuda")
    out = hc.embedding(table, ids, first_id=2)["out"]
    assert torch.equal(out, embedding(table, ids.clamp(-1000, 1000), 1.0, 2).float())
    out = hc.embedding(table, ids, first_id=-big - 1)["out"]
    assert torch.equal(out[0], table[0]) and not bool(out[1:].any())


def test_vocabulary_split_over_ranks_and_allreduced_is_the_whole_lookup():
    P, vocab, dim, tokens = 4, 1003, 64, 500
    g = gen(5)
    table = normal(g, vocab, dim)
    ids = some_ids(g, tokens, vocab, "skewed")
    per = (vocab + P - 1) // P
    parts = [hc.embedding(table[r * per:(r + 1) * per], ids, scale=8.0, first_id=r * per)["out"] for r in range(P)]
    hc.allreduce(parts)
    whole = hc.embedding(table, ids, scale=8.0)["out"]
    for p in parts:
        assert torch.equal(p, whole)


# ------------------------------------------------------------------ embedding gradient
def run_embedding_grad(g, tokens, rows, dim, kind, grad_dtype, table_dtype, accumulate, first=0, padding=-1,
                       id_dtype=torch.int64, stride=None, offset=0):
    scale = 0.5  # a power of two: scaling adds no error
    ids = some_ids(g, tokens, rows + 2 * first, kind, id_dtype)
    go = strided(normal(g, tokens, dim, dtype=grad_dtype), stride, offset)
    old = normal(g, rows, dim, dtype=table_dtype)
    table, intact = guarded(rows, dim, table_dtype, stride, offset)
    table.copy_(old)
    hc.embedding_grad(go, ids, table, scale=scale, first_id=first, padding_id=padding, accumulate=accumulate)
    ref, mag, n = embedding_grad(go, ids, rows, scale, first, padding, old if accumulate else None)
    assert_close(table, ref, mag * (n[:, None] + 1), 1, "grad_table")  # n - 1 sums, the old value, one product
    if accumulate:
        assert torch.equal(table[n == 0], old[n == 0])  # rows without tokens are untouched
    else:
        assert not bool(table[n == 0].any())
    assert intact()
    again = old.clone()
    hc.embedding_grad(go, ids, again, scale=scale, first_id=first, padding_id=padding, accumulate=accumulate)
    assert torch.equal(table, again)  # the same order of sums, whatever the strides


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "none", "twice"])
@pytest.mark.parametrize("tokens", [1, 31, 256, 257, 2048, 5000])
def test_embedding_grad(tokens, kind, accumulate):
    run_embedding_grad(gen(tokens), tokens, 700, 72, kind, BF16, F32, accumulate, padding=2)


@pytest.mark.parametrize("grad_dtype,table_dtype", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("tokens,rows,dim,stride,offset", [(100, 37, 1, None, 0), (3001, 513, 257, None, 0),
                                                           (700, 50, 1000, 1008, 0), (999, 64, 40, 43, 1),
                                                           (200, 1, 2056, None, 0), (1000, 1, 300, None, 0)])
def test_embedding_grad_types_and_strides(grad_dtype, table_dtype, tokens, rows, dim, stride, offset):
    for accumulate in (False, True):
        run_embedding_grad(gen(dim), tokens, rows, dim, "skewed", grad_dtype, table_dtype, accumulate, first=5,
                           id_dtype=torch.int32, stride=stride, offset=offset)


@pytest.mark.parametrize("tokens,rows", [(300000, 1000), (5000, 300000), (3000, (1 << 18) + 7)])
def test_embedding_grad_many(tokens, rows):
    """Many sorting blocks of the larger size; three radix passes."""
    run_embedding_grad(gen(rows), tokens, rows, 16, "skewed", BF16, F32, True)
    run_embedding_grad(gen(rows), tokens, rows, 16, "uniform", F32, F32, False)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,rows", [(2049, 700), (16411, 8001), (32768, 700), (32769, 700), (40000, (1 << 18) + 7),
                                         (262144, 5000), (262145, (1 << 18) + 7)])
def test_embedding_grad_sorts(tokens, rows, accumulate):
    """The largest sorts of one cluster and the smallest over global memory, both
    sizes of its blocks, with two and three radix passes."""
    run_embedding_grad(gen(rows), tokens, rows, 9, "skewed", BF16, F32, accumulate)
    run_embedding_grad(gen(rows), tokens, rows, 16, "uniform", F32, F32, accumulate)


def test_embedding_grad_ignores_rows_of_tokens_elsewhere():
    g = gen(9)
    for tokens in (100, 3000):
        ids = some_ids(g, tokens, 50, "uniform")
        go = normal(g, tokens, 24)
        go[(ids < 10) | (ids >= 40) | (ids == 20)] = math.nan
        t = torch.empty(30, 24, device="cuda")
        hc.embedding_grad(go, ids, t, first_id=10, padding_id=20)
        assert torch.isfinite(t).all() and not bool(t[10].any())


def test_embedding_grad_without_tokens():
    t = torch.ones(9, 5, device="cuda")
    empty, ids = torch.empty(0, 5, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    hc.embedding_grad(empty, ids, t, accumulate=True)
    assert bool((t == 1).all())
    hc.embedding_grad(empty, ids, t)
    assert not bool(t.any())
    assert hc.embedding(t, ids)["out"].shape == (0, 5)


def test_embedding_grad_is_the_lookups_transpose():
    """<out(W), G> = <W, grad(G)> for the linear lookup: both sides in 64 bits
    from the kernels' binary32 outputs."""
    g = gen(3)
    W, ids, G = normal(g, 90, 70), some_ids(g, 1500, 95, "skewed"), normal(g, 1500, 70)
    out = hc.embedding(W, ids, scale=3.0, first_id=2)["out"]
    t = torch.empty_like(W)
    hc.embedding_grad(G, ids, t, scale=3.0, first_id=2)
    a, b = (out.double() * G).sum(), (W.double() * t).sum()
    size = (out.double() * G).abs().sum()
    assert abs(float(a - b)) <= 2.0 ** -24 * 1500 * float(size)


# ------------------------------------------------------------------ block norm
def norm_inputs(g, tokens, dim, dtype, wdtype, gates, weights=True):
    y, x = normal(g, tokens, dim, dtype=dtype, std=3.0), normal(g, tokens, dim, dtype=dtype, std=2.0)
    post = (1 + normal(g, dim, std=0.3)).to(wdtype) if weights else None
    pre = (1 + normal(g, dim, std=0.3)).to(wdtype) if weights else None
    gate = normal(g, gates, dim, dtype=wdtype) if gates else None
    return y, x, post, gate, pre


def wide(w):
    return w.to(D) if w is not None else torch.ones((), dtype=D, device="cuda")


def rows_of(gate, tokens):
    return gate.to(D).repeat_interleave(tokens // gate.shape[0], dim=0) if gate is not None else wide(None)


NORM_SHAPES = [(1, 1, 1), (1, 4096, 1), (3, 7, 3), (5, 64, 0), (37, 257, 1), (64, 1000, 8), (33, 1001, 11),
               (1021, 96, 1021), (640, 40, 320), (12, 5128, 4), (4, 20008, 2), (3, 32768, 1), (1216, 136, 304), (5, 16400, 1),
               (6, 8200, 2), (9, 300, 3), (1300, 515, 2), (330, 4097, 1), (400, 33, 1), (50, 8190, 1), (2500, 249, 5),
               (24, 500, 1), (2, 4000, 2), (90, 63, 90), (6, 1001, 2)]


def check_norm(tokens, dim, gates, dtype, wdtype, stride=None, offset=0, weights=True):
    a, eps = 0.75, 1e-5
    g = gen(tokens + dim)
    y, x, post, gate, pre = norm_inputs(g, tokens, dim, dtype, wdtype, gates, weights)
    y, x = strided(y, stride, offset), strided(x, stride, offset)
    (r, ok_r), (z, ok_z) = guarded(tokens, dim, dtype, stride, offset), guarded(tokens, dim, dtype, stride, offset)
    o = hc.block_norm(y, x, post, gate, pre, r=r, z=z, residual_scale=a, eps=eps)
    eps32 = torch.tensor(eps, dtype=F32).double().item()
    R, Z, S, Q, mag = block_norm(y, x, wide(post), rows_of(gate, tokens), wide(pre), a, eps32)
    # a row's sum of squares: at most 8 + 2 * 5 + 32 + 8 additions one after
    # another, halved by the root; its inverse and the products around it: 64
    assert_close(o["post_rstd"], S[:, 0], S[:, 0], 64, "post_rstd")
    assert_close(r, R, mag, 64, "r")
    # r's error reaches its norm relative to the row's mean magnitude
    err_q = Q * (mag * R.abs()).mean(dim=1, keepdim=True) * Q * Q + Q
    assert_close(o["pre_rstd"], Q[:, 0], err_q[:, 0], 128, "pre_rstd")
    assert_close(z, Z, (wide(pre) * (mag * Q + R * err_q)).abs() + (mag * Q * wide(pre)).abs(), 128, "z")
    assert ok_r() and ok_z()
    alone = hc.block_norm(y, x, post, gate, pre, residual_scale=a, eps=eps, next_norm=False)
    assert torch.equal(alone["r"], r) and set(alone) == {"r", "post_rstd"}


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("tokens,dim,gates", NORM_SHAPES)
def test_block_norm(tokens, dim, gates, dtype, wdtype):
    check_norm(tokens, dim, gates, dtype, wdtype)


@pytest.mark.parametrize("stride,offset", [(104, 0), (101, 0), (112, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_block_norm_strided(dtype, stride, offset):
    check_norm(40, 100, 4, dtype, dtype, stride, offset)
    check_norm(40, 100, 0, dtype, dtype, stride, offset, weights=False)


@pytest.mark.parametrize("dim", [64, 1000, 9000])
def test_block_norm_in_place(dim):
    y, x, post, gate, pre = norm_inputs(gen(2), 21, dim, BF16, F32, 7)
    ref = hc.block_norm(y, x, post, gate, pre)
    y2, x2 = y.clone(), x.clone()
    hc.block_norm(y2, x2, post, gate, pre, r=x2, z=y2)
    assert torch.equal(x2, ref["r"]) and torch.equal(y2, ref["z"])
    y2, x2 = y.clone(), x.clone()
    hc.block_norm(y2, x2, post, gate, pre, r=y2, z=x2)
    assert torch.equal(y2, ref["r"]) and torch.equal(x2, ref["z"])


def test_block_norm_rows_are_independent():
    """Zeros, infinities and NaN in one row leave the others as they are."""
    y, x, post, gate, pre = norm_inputs(gen(4), 6, 520, F32, F32, 1)
    ref = hc.block_norm(y, x, post, gate, pre)
    y[1], x[1] = 0.0, 0.0
    y[3, 5], x[4, 7] = math.inf, math.nan
    o = hc.block_norm(y, x, post, gate, pre)
    for k in (0, 2, 5):
        assert torch.equal(o["r"][k], ref["r"][k]) and torch.equal(o["z"][k], ref["z"][k])
    assert not bool(o["r"][1].any()) and not bool(o["z"][1].any())


# ------------------------------------------------------------------ block norm gradient
def check_norm_grad(tokens, dim, gates, dtype, wdtype, stride=None, offset=0, weights=True, gr=True, gz=True):
    a, eps = 0.75, 1e-5
    g = gen(tokens * 3 + dim)
    y, x, post, gate, pre = norm_inputs(g, tokens, dim, dtype, wdtype, gates, weights)
    y, x = strided(y, stride, offset), strided(x, stride, offset)
    dr = strided(normal(g, tokens, dim, dtype=dtype), stride, offset) if gr else None
    dz = strided(normal(g, tokens, dim, dtype=dtype), stride, offset) if gz else None
    f = hc.block_norm(y, x, post, gate, pre, residual_scale=a, eps=eps)
    (gy, ok_y), (gx, ok_x) = guarded(tokens, dim, dtype, stride, offset), guarded(tokens, dim, dtype, stride, offset)
    o = hc.block_norm_grad(dr, dz, y, x, f["post_rstd"], f["pre_rstd"], post, gate, pre, grad_y=gy, grad_x=gx,
                           residual_scale=a)
    # the formulas in 64 bits, from the kept (binary32) root mean squares
    S, Q = f["post_rstd"].to(D)[:, None], f["pre_rstd"].to(D)[:, None]
    G, P, W = rows_of(gate, tokens), wide(post), wide(pre)
    yh = y.to(D) * S
    rh = (a * x.to(D) + G * (yh * P)) * Q
    rm = ((a * x.to(D)).abs() + (G * (yh * P)).abs()) * Q  # magnitudes of rh's terms
    z = torch.zeros(tokens, dim, dtype=D, device="cuda")
    h = dz.to(D) * W if gz else z
    q = Q if gz else 0.0 * Q
    m1 = (h * rh).mean(dim=1, keepdim=True)
    m1m = (h.abs() * rm).mean(dim=1, keepdim=True)
    T = (dr.to(D) if gr else z) + q * (h - rh * m1)
    Tm = (dr.to(D).abs() if gr else z) + q * (h.abs() + rm * m1m * 2)
    k = T * G * P
    km = Tm * (G * P).abs()
    m2 = (k * yh).mean(dim=1, keepdim=True)
    m2m = (km * yh.abs()).mean(dim=1, keepdim=True)
    # chains: a row sum (8 + 10 + 16 + 8 additions) of products of up to six
    # factors, twice one after the other
    assert_close(gx, a * T, a * Tm, 128, "grad_x")
    assert_close(gy, S * (k - yh * m2), S * (km + yh.abs() * m2m), 256, "grad_y")
    # sums over the tokens, each term with the errors above
    n = max(1, tokens // max(gates, 1))
    A, Am = T * yh, Tm * yh.abs()
    shape = (max(gates, 1), n, dim)
    if weights:
        assert_close(o["grad_post_weight"], (A * G).sum(dim=0), (Am * G.abs()).sum(dim=0), 160 + tokens, "grad_post_weight")
        if gz:
            assert_close(o["grad_pre_weight"], (dz.to(D) * rh).sum(dim=0), (dz.to(D).abs() * rm).sum(dim=0),
                         64 + tokens, "grad_pre_weight")
        else:
            assert not bool(o["grad_pre_weight"].any())
    if gates:
        assert_close(o["grad_gate"], (A * P).view(shape).sum(dim=1), (Am * P.abs()).view(shape).sum(dim=1), 160 + n,
                     "grad_gate")
    assert ok_y() and ok_x()
    b = hc.block_norm_grad(dr, dz, y, x, f["post_rstd"], f["pre_rstd"], post, gate, pre, residual_scale=a)
    for name, t in o.items():
        assert torch.equal(t, b[name]), name


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("tokens,dim,gates", NORM_SHAPES + [(700, 128, 1), (2000, 72, 5), (912, 40, 456), (915, 33, 305)])
def test_block_norm_grad(tokens, dim, gates, dtype, wdtype):
    check_norm_grad(tokens, dim, gates, dtype, wdtype)


@pytest.mark.parametrize("stride,offset", [(104, 0), (101, 0), (112, 3)])
def test_block_norm_grad_strided_and_partial(stride, offset):
    for dtype in (F32, BF16):
        check_norm_grad(40, 100, 4, dtype, dtype, stride, offset)
        check_norm_grad(40, 100, 0, dtype, dtype, stride, offset, weights=False)
        check_norm_grad(40, 100, 2, dtype, F32, gr=False)
        check_norm_grad(40, 100, 2, dtype, F32, gz=False)
        check_norm_grad(620, 100, 310, dtype, F32, gz=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,dim", [(152, 257), (509, 1001), (200, 1024), (331, 3001), (160, 4512), (153, 5000),
                                        (152, 6656), (155, 6664), (154, 8192), (152, 20001), (170, 32768), (2500, 264)])
def test_block_norm_grad_with_a_gate_for_every_token(tokens, dim, dtype):
    check_norm_grad(tokens, dim, tokens, dtype, dtype)


@pytest.mark.parametrize("stride,offset", [(304, 0), (301, 0), (312, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_block_norm_grad_with_a_gate_for_every_token_strided_and_partial(dtype, stride, offset):
    check_norm_grad(160, 300, 160, dtype, dtype, stride, offset)
    check_norm_grad(160, 300, 160, dtype, dtype, stride, offset, weights=False)
    check_norm_grad(161, 299, 161, dtype, dtype, gr=False)
    check_norm_grad(161, 304, 161, dtype, dtype, gz=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [32761, 32762, 32765, 32766, 32767])
def test_block_norm_grad_of_the_longest_odd_rows(dim, dtype):
    """Rows whose 16-byte windows would begin before a cluster's columns."""
    check_norm(40, dim, 1, dtype, dtype)
    check_norm_grad(40, dim, 1, dtype, dtype)
    check_norm_grad(160, dim, 160, dtype, dtype)


@pytest.mark.parametrize("stride,offset", [(32768, 1), (32769, 0), (32771, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_block_norm_grad_of_the_longest_rows_strided(dtype, stride, offset):
    check_norm_grad(40, 32768, 1, dtype, dtype, stride, offset)
    check_norm_grad(153, 32768, 153, dtype, dtype, stride, offset)


@pytest.mark.parametrize("dim", [301, 1024, 5000])
def test_block_norm_grad_with_a_gate_for_every_token_in_place(dim):
    g = gen(8)
    y, x, post, gate, pre = norm_inputs(g, 200, dim, BF16, BF16, 200)
    dr, dz = normal(g, 200, dim, dtype=BF16), normal(g, 200, dim, dtype=BF16)
    f = hc.block_norm(y, x, post, gate, pre)
    args = (f["post_rstd"], f["pre_rstd"], post, gate, pre)
    ref = hc.block_norm_grad(dr, dz, y, x, *args)
    y2, x2 = y.clone(), x.clone()
    o = hc.block_norm_grad(dr, dz, y2, x2, *args, grad_x=y2, grad_y=x2)
    for name in ref:
        assert torch.equal(o[name], ref[name]), name


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("tokens,dim,gates", [(3, 40, 1), (40, 100, 2), (620, 100, 310), (37, 301, 1), (90, 1000, 3),
                                              (620, 520, 310), (200, 301, 200), (200, 1024, 200), (20, 9000, 1)])
def test_block_norm_grad_without_a_next_norm(tokens, dim, gates, dtype, wdtype):
    """Without grad_z neither x nor the next norm's weight has a part in any
    gradient, whatever they hold, and grad_x = a grad_r."""
    a = 0.75
    g = gen(dim)
    y, x, post, gate, pre = norm_inputs(g, tokens, dim, dtype, wdtype, gates)
    dr = normal(g, tokens, dim, dtype=dtype)
    s = hc.block_norm(y, x, post, gate, residual_scale=a, next_norm=False)["post_rstd"]
    ref = hc.block_norm_grad(dr, None, y, x, s, None, post, gate, pre, residual_scale=a)
    assert all(bool(torch.isfinite(t).all()) for t in ref.values())
    x[0], x[-1, 3], pre[1], pre[2] = math.inf, math.nan, math.nan, -math.inf
    pre_grad = torch.full_like(pre, 9.0)
    o = hc.block_norm_grad(dr, None, y, x, s, None, post, gate, pre, residual_scale=a, grad_pre_weight=pre_grad)
    assert not bool(pre_grad.any())
    for name in ref:
        assert torch.equal(o[name], ref[name]), name
    assert torch.equal(o["grad_x"], (dr.double() * a).to(dtype))


@pytest.mark.parametrize("dim", [64, 5000])
def test_block_norm_grad_in_place(dim):
    g = gen(8)
    y, x, post, gate, pre = norm_inputs(g, 30, dim, BF16, F32, 3)
    dr, dz = normal(g, 30, dim, dtype=BF16), normal(g, 30, dim, dtype=BF16)
    f = hc.block_norm(y, x, post, gate, pre)
    args = (f["post_rstd"], f["pre_rstd"], post, gate, pre)
    ref = hc.block_norm_grad(dr, dz, y, x, *args)
    r2, z2 = dr.clone(), dz.clone()
    o = hc.block_norm_grad(r2, z2, y, x, *args, grad_x=r2, grad_y=z2)
    for name in ref:
        assert torch.equal(o[name], ref[name]), name
    y2, x2 = y.clone(), x.clone()
    o = hc.block_norm_grad(dr, dz, y2, x2, *args, grad_x=y2, grad_y=x2)
    for name in ref:
        assert torch.equal(o[name], ref[name]), name


def test_block_norm_grad_without_tokens():
    for gates in (1, 400):
        y = torch.empty(0, 24, device="cuda")
        s = torch.empty(0, device="cuda")
        w, gate = torch.ones(24, device="cuda"), torch.ones(gates, 24, device="cuda")
        outs = [torch.full_like(t, 9.0) for t in (w, gate, w)]
        hc.block_norm(y, y.clone(), w, gate, w)
        hc.block_norm_grad(y, None, y, y, s, s, w, gate, w, grad_post_weight=outs[0], grad_gate=outs[1],
                           grad_pre_weight=outs[2])
        assert not any(bool(t.any()) for t in outs)


def test_block_norm_grad_without_tokens_is_zeros_whatever_the_weights():
    y, s = torch.empty(0, 24, device="cuda"), torch.empty(0, device="cuda")
    w = torch.full((24,), math.inf, device="cuda")
    w[3] = math.nan
    for gates in (1, 400):
        gate = w.repeat(gates, 1)
        o = hc.block_norm_grad(y, y, y, y, s, s, w, gate, w)
        assert not any(bool(o[k].any()) for k in ("grad_post_weight", "grad_gate", "grad_pre_weight"))


def test_block_norm_grad_against_differences():
    """Directional derivatives of the 64-bit forward pass by central
    differences: truncation of order h^2, the kernels' binary32 gradients."""
    g = gen(6)
    T, d, G, a, eps = 12, 48, 4, 0.75, 1e-3
    y, x, post, gate, pre = norm_inputs(g, T, d, F32, F32, G)
    dr, dz = normal(g, T, d), normal(g, T, d)
    f = hc.block_norm(y, x, post, gate, pre, residual_scale=a, eps=eps)
    o = hc.block_norm_grad(dr, dz, y, x, f["post_rstd"], f["pre_rstd"], post, gate, pre, residual_scale=a)
    at = {"y": y.to(D), "x": x.to(D), "post_weight": post.to(D), "gate": gate.to(D), "pre_weight": pre.to(D)}

    def value(v):
        R, Z, _, _, _ = block_norm(v["y"], v["x"], v["post_weight"], v["gate"].repeat_interleave(T // G, dim=0),
                                   v["pre_weight"], a, torch.tensor(eps, dtype=F32).double().item())
        return float((R * dr).sum() + (Z * dz).sum())
    h = 1e-5
    for name in at:
        v = torch.randn(at[name].shape, generator=g, device="cuda", dtype=D)
        up, down = dict(at), dict(at)
        up[name], down[name] = at[name] + h * v, at[name] - h * v
        diff = (value(up) - value(down)) / (2 * h)
        got = float((o["grad_" + name].to(D) * v).sum())
        size = float((o["grad_" + name].to(D) * v).abs().sum())
        assert abs(got - diff) <= 1e-5 * size, name  # 256 * 2^-24 of rounding; h^2 and 1e-16 / h are smaller


# ------------------------------------------------------------------ distillation
def distill_inputs(g, tokens, vocab, top, dtype, tdtype=F32, idtype=torch.int64):
    x = normal(g, tokens, vocab, dtype=dtype, std=3.0)
    t = normal(g, tokens, top, dtype=tdtype, std=3.0)
    ids = torch.randint(0, vocab, (tokens, top), generator=g, device="cuda").to(idtype)
    return x, t, ids


def check_distill(x, t, ids, weight=None, tau=2.0, scale=0.25, stride=None, offset=0):
    T, V = x.shape
    ref = distill(x, t, ids, weight, tau, scale)
    xs = strided(x, stride, offset)
    grad, intact = guarded(T, V, x.dtype, stride, offset)
    o = hc.distill(xs, t, ids, weight, grad=grad, temperature=tau, scale=scale)
    # exponents and logarithms: 4 units each; an exponent's argument is off by
    # 2 of its own units; the row's sum: at most V / 512 + 64 additions
    k = 64 + V / 256

    def check(out, name):
        assert_close(out["loss"], ref["loss"], ref["loss_mag"], 2 * k, name + " loss")
        assert_close(out["stats"], ref["stats"], ref["stats_mag"], k, name + " stats")
    check(o, "both")
    assert_close(grad, ref["grad"], ref["grad_mag"], k, "grad")
    assert intact()
    alone = hc.distill(xs, t, ids, weight, grad=False, temperature=tau, scale=scale)
    assert torch.equal(alone["loss"], o["loss"]) and torch.equal(alone["stats"], o["stats"])
    g2, intact2 = guarded(T, V, x.dtype, stride, offset)
    hc.distill_grad(xs, t, ids, alone["stats"], weight, grad=g2, temperature=tau, scale=scale)
    assert_close(g2, ref["grad"], ref["grad_mag"], k, "grad alone")
    assert intact2()
    for in_place in ("both", "grad"):
        xc = strided(x, stride, offset)
        if in_place == "both":
            hc.distill(xc, t, ids, weight, grad=xc, temperature=tau, scale=scale)
            assert torch.equal(xc, grad)
        else:
            hc.distill_grad(xc, t, ids, alone["stats"], weight, grad=xc, temperature=tau, scale=scale)
            assert torch.equal(xc, g2)


DISTILL_SHAPES = [(1, 1, 1), (1, 7, 3), (2, 8, 16), (3, 1001, 33), (5, 4096, 64), (1, 50021, 7), (9, 32768, 16),
                  (170, 600, 5), (3, 131072, 64), (2, 200003, 100), (4, 2000, 1024)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,vocab,top", DISTILL_SHAPES)
def test_distill(tokens, vocab, top, dtype):
    g = gen(vocab)
    x, t, ids = distill_inputs(g, tokens, vocab, top, dtype, BF16 if top % 2 else F32,
                               torch.int32 if tokens % 2 else torch.int64)
    check_distill(x, t, ids)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_distill_largest_rows(dtype):
    x, t, ids = distill_inputs(gen(1), 2, (3 << 19) // x_size(dtype), 4, dtype)
    check_distill(x, t, ids)


def x_size(dtype):
    return 2 if dtype == BF16 else 4


@pytest.mark.parametrize("stride,offset", [(1008, 0), (1001, 0), (1013, 3), (1004, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_distill_strided(dtype, stride, offset):
    x, t, ids = distill_inputs(gen(stride), 23, 1001, 8, dtype)
    check_distill(x, t, ids, stride=stride, offset=offset)


def test_distill_gradient_of_another_alignment():
    for dtype in (F32, BF16):
        x, t, ids = distill_inputs(gen(3), 5, 3000, 8, dtype)
        ref = hc.distill(x, t, ids)
        grad, intact = guarded(5, 3000, dtype, 3001, 1)
        o = hc.distill(x, t, ids, grad=grad)
        assert torch.equal(grad, ref["grad"]) and intact()
        hc.distill_grad(x, t, ids, o["stats"], grad=grad)
        assert intact()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [37, 5003, 70000])
def test_distill_masks(dtype, vocab):
    """Masked columns, short and empty teacher rows, the same id twice, rows
    without weight whose logits are NaN."""
    g = gen(vocab)
    T, K = 12, 9
    x, t, ids = distill_inputs(g, T, vocab, K, dtype)
    x[:, -5:] = -torch.inf
    ids = ids.clamp(max=vocab - 6)
    x[1, :vocab // 2] = torch.finfo(dtype).min
    ids[2, 3:] = -1
    ids[3, :] = -1
    t[4, :] = -torch.inf
    t[5, 2:] = -torch.inf
    ids[6, :] = 11
    ids[7, 1::2] = ids[7, 0]
    ids[8, 0] = vocab
    ids[8, 1] = 2 ** 40
    weight = torch.ones(T, device="cuda")
    weight[9] = 0.0
    weight[10] = -2.5
    x[9] = math.nan
    x[3] = math.nan
    check_distill(x, t, ids, weight)
    o = hc.distill(x, t, ids, weight)
    for row in (3, 4, 9):
        assert float(o["loss"][row]) == 0.0 and not bool(o["grad"][row].any()) and not bool(o["stats"][row].any())


def test_distill_teacher_mass_on_a_masked_column():
    """The loss of a row whose teacher likes a column of logit -inf is
    infinite, its gradient is not."""
    x, t, ids = distill_inputs(gen(1), 2, 100, 3, F32)
    x[0, int(ids[0, 1])] = -torch.inf
    o = hc.distill(x, t, ids)
    assert float(o["loss"][0]) == math.inf and torch.isfinite(o["grad"]).all() and torch.isfinite(o["loss"][1])


@pytest.mark.parametrize("tau", [0.25, 1.0, 20.0])
def test_distill_temperatures(tau):
    x, t, ids = distill_inputs(gen(2), 6, 3000, 12, F32)
    check_distill(x, t, ids, tau=tau, scale=1.0)


def test_distill_wide_range():
    """Logits of +-1e30 (a sharp row) and of all one value (a flat one)."""
    x, t, ids = distill_inputs(gen(2), 3, 2000, 4, F32)
    x[0] = 5.0
    x[1] = -1e30
    x[1, 77] = 1e30
    ids[1] = torch.tensor([77, 77, 77, 77], device="cuda")
    o = hc.distill(x, t, ids)
    ref = distill(x, t, ids, None, 1.0, 1.0)
    assert_close(o["grad"], ref["grad"], ref["grad_mag"], 100, "grad")
    assert_close(o["loss"], ref["loss"], ref["loss_mag"], 200, "loss")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [40, 5003, 70000])
@pytest.mark.parametrize("tau", [0.5, 1.0])
def test_distill_large_logits(dtype, vocab, tau):
    """Rows whose mask leaves nothing (every logit the type's lowest value, but
    for -inf), and rows of large logits, whose exponents need the difference
    from the row's largest before anything is rounded."""
    g = gen(vocab)
    x, t, ids = distill_inputs(g, 8, vocab, 6, dtype)
    low = torch.finfo(dtype).min
    x[0] = low
    x[1] = -torch.inf
    x[1, ids[1]] = low
    x[2] += 3e4
    x[3] = -1e6
    x[4] = torch.where(torch.rand(vocab, generator=g, device="cuda") < 0.5, 2.0 ** 20, low).to(dtype)
    x[4, ids[4]] = 2.0 ** 20
    x[5] = -1e30
    x[5, 7] = 1e30
    ids[5] = 7
    x[6] *= 40
    check_distill(x, t, ids, tau=tau)


def test_distill_grad_against_differences():
    g = gen(12)
    x, t, ids = distill_inputs(g, 4, 300, 10, F32)
    w = torch.tensor([1.0, 0.5, 0.0, 2.0], device="cuda")
    o = hc.distill(x, t, ids, w, temperature=1.5)
    v = torch.randn(x.shape, generator=g, device="cuda", dtype=D)
    h = 1e-4
    up = distill(x.to(D) + h * v, t, ids, w, 1.5, 1.0)["loss"].sum()
    down = distill(x.to(D) - h * v, t, ids, w, 1.5, 1.0)["loss"].sum()
    got = float((o["grad"].to(D) * v).sum())
    assert abs(got - float(up - down) / (2 * h)) <= 1e-5 * float((o["grad"].to(D) * v).abs().sum())


def test_distill_without_tokens():
    x = torch.empty(0, 40, device="cuda")
    o = hc.distill(x, torch.empty(0, 3, device="cuda"), torch.empty(0, 3, dtype=torch.int64, device="cuda"))
    assert o["loss"].shape == (0,) and o["grad"].shape == (0, 40)


def test_distill_wait_expiry():
    """In the wait-expiry test mode the first wait on the copies gives up: the
    status is reported, nothing hangs, later calls are unaffected."""
    from collective_communication_algorithms_gb300 import _binding as B
    x, t, ids = distill_inputs(gen(7), 3, 40000, 8, BF16)
    ref = hc.distill(x, t, ids)
    torch.cuda.synchronize()
    assert B.hc_device_status() == 0
    B.hc_test_expire_waits(True)
    try:
        hc.distill(x, t, ids)
        torch.cuda.synchronize()
    finally:
        B.hc_test_expire_waits(False)
    assert B.hc_device_status(clear=True) == 6  # HC_ERR_TIMEOUT
    assert B.hc_device_status() == 0
    o = hc.distill(x, t, ids)
    assert torch.equal(o["grad"], ref["grad"]) and torch.equal(o["loss"], ref["loss"])


def test_block_norm_wait_expiry():
    """The same for the block norm and its gradient on rows of a ring."""
    from collective_communication_algorithms_gb300 import _binding as B
    for dim in (1000, 1001, 9000):
        g = gen(dim)
        y, x, post, gate, pre = norm_inputs(g, 3, dim, BF16, F32, 1)
        dr, dz = normal(g, 3, dim, dtype=BF16), normal(g, 3, dim, dtype=BF16)
        ref = hc.block_norm(y, x, post, gate, pre)
        grads = hc.block_norm_grad(dr, dz, y, x, ref["post_rstd"], ref["pre_rstd"], post, gate, pre)
        torch.cuda.synchronize()
        for run in (lambda: hc.block_norm(y, x, post, gate, pre),
                    lambda: hc.block_norm_grad(dr, dz, y, x, ref["post_rstd"], ref["pre_rstd"], post, gate, pre)):
            assert B.hc_device_status() == 0
            B.hc_test_expire_waits(True)
            try:
                run()
                torch.cuda.synchronize()
            finally:
                B.hc_test_expire_waits(False)
            assert B.hc_device_status(clear=True) == 6
        o = hc.block_norm(y, x, post, gate, pre)
        assert torch.equal(o["r"], ref["r"]) and torch.equal(o["z"], ref["z"])
        o = hc.block_norm_grad(dr, dz, y, x, ref["post_rstd"], ref["pre_rstd"], post, gate, pre)
        for name in grads:
            assert torch.equal(o[name], grads[name]), name


# ------------------------------------------------------------------ streams, graphs, binding
def step_calls(stream=None):
    g = gen(77)
    T, V, d = 600, 500, 64
    s = {"ids": some_ids(g, T, V, "skewed"), "table": normal(g, V, d), "y": normal(g, T, d),
         "post": normal(g, d), "pre": normal(g, d), "gate": normal(g, 3, d), "logits": normal(g, T, V),
         "t": normal(g, T, 5), "tid": torch.randint(0, V, (T, 5), generator=g, device="cuda")}
    torch.cuda.synchronize()
    e = hc.bind_embedding(s["table"], s["ids"], stream=stream)
    x = e.outputs["out"]
    n = hc.bind_block_norm(s["y"], x, s["post"], s["gate"], s["pre"], stream=stream)
    l_ = hc.bind_distill(s["logits"], s["t"], s["tid"], stream=stream)
    f = n.outputs
    b = hc.bind_block_norm_grad(f["r"], f["z"], s["y"], x, f["post_rstd"], f["pre_rstd"], s["post"], s["gate"],
                                s["pre"], stream=stream)
    dt = torch.empty(V, d, device="cuda")
    eg = hc.bind_embedding_grad(b.outputs["grad_x"], s["ids"], dt, stream=stream)
    calls = [e, n, l_, b, eg]
    return calls, [t for c in calls for t in c.outputs.values()], s


def test_bound_calls_repeat_on_a_side_stream_and_in_a_graph():
    calls, outs, _ = step_calls()
    for c in calls:
        c()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    stream = torch.cuda.Stream()
    calls, outs, keep = step_calls(stream)
    for _ in range(3):
        for c in calls:
            c()
    stream.synchronize()
    for a, b in zip(ref, outs):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for c in calls:
            c()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(ref, outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_a_call_on_another_stream_is_not_handed_out_early(handle):
    """A call on a busy side stream, its inputs dropped at once: what the
    allocator hands out meanwhile is neither the call's inputs nor its scratch."""
    g = gen(5)
    T, V, d = 4000, 300, 64
    ids, dout = some_ids(g, T, V, "skewed"), normal(g, T, d)
    want = hc.embedding_grad(dout, ids, torch.empty(V, d, device="cuda"))["grad_table"]
    side = torch.cuda.Stream()

    def call():
        i2, d2 = ids.clone(), dout.clone()
        torch.cuda.current_stream().synchronize()
        return hc.embedding_grad(d2, i2, torch.empty(V, d, device="cuda"),
                                 stream=side.cuda_stream if handle else side)["grad_table"]

    def more():
        return [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                for n in (T * 8, T * d * 4, T * 8 + 512, 1 << 16, 1 << 18, 1 << 20) for _ in range(8)]
    call(), more()  # the kernels are loaded and the allocator has its memory
    torch.cuda._sleep(1 << 10)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1 << 27)
    got = call()
    other = more()
    torch.cuda.current_stream().synchronize()
    assert not side.query()  # the call has not run yet
    side.synchronize()
    assert torch.equal(got, want)
    assert all(bool((t == 255).all()) for t in other)


def test_offsets_past_32_bits():
    """Rows that begin more than 2^31 elements after the first."""
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    rows, dim = 1 << 20, 4096  # 2^32 elements, 8 GB in bf16
    table = torch.zeros(rows, dim, dtype=BF16, device="cuda")
    far = torch.tensor([rows - 1, 3, rows - 2], device="cuda")
    vals = normal(gen(1), 3, dim, dtype=BF16)
    table[far] = vals
    assert torch.equal(hc.embedding(table, far)["out"], vals)
    for reps in (1, 200):  # few tokens, and sorted
        ids = far.repeat(reps)
        hc.embedding_grad(vals.float().repeat(reps, 1), ids, table, accumulate=True)
        ref, mag, _ = embedding_grad(vals.float().repeat(reps, 1), torch.tensor([0, 1, 2], device="cuda").repeat(reps), 3,
                                     1.0, 0, -1, vals)
        assert_close(table[far], ref, mag * (reps + 1), 1, "far rows")
        table[far] = vals
    # the same matrix as logits of 2^20 columns: 4096 rows
    x = table.view(4096, 1 << 20)[:, :700000]
    x = x[4000:]  # offsets near 2^32
    t, tid = normal(gen(2), 96, 3), torch.randint(0, 700000, (96, 3), device="cuda")
    ref = distill(x[90:], t[90:], tid[90:], None, 1.0, 1.0)
    o = hc.distill(x, t, tid, grad=x)
    assert_close(o["grad"][90:], ref["grad"], ref["grad_mag"], 64 + 700000 / 256, "far logits")
