"""The decoder-block operators on the GPU against the fp64 oracle: residual addition with RMSNorm, routing,
experts, and the three in a row behind the ShortConv."""
import numpy as np
import pytest
import torch

from encoder_free_audio_b200 import build, dmel

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}  # a rounding, relative to the value


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    dmel.library()
    dmel.dmel_get_device_error(clear=True)
    yield


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------------------ add + RMSNorm

def norm_inputs(seed, n, d, dt, residual=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, d), generator=g, device=DEV)
    r = torch.randn((n, d), generator=g, device=DEV) * torch.exp(torch.randn((n, 1), generator=g, device=DEV))
    w = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
    return x.to(dt), r.to(dt) if residual else None, w.to(dt)


def norm_bound(d):
    """Relative error of fp32 y: the fp32 sum s (1), a chain of at most d / 8 / 32 * 8 squares in a thread
    and ten additions across threads, halved by the square root; its division, addition, square root and
    reciprocal (4, of which the square root halves two); two products (2). In units of 2^-24."""
    return ((d / 32 + 16 + 10) / 2 + 1 + 4 + 2) * 2.0 ** -24


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("odt", [F32, BF16])
@pytest.mark.parametrize("n,d", [(1, 8), (3, 40), (5, 256), (2, 264), (7, 1000), (4, 6144), (3, 8192), (2, 8200), (2, 16384)])
def test_add_rmsnorm(dt, odt, n, d, oracle_mod):
    for residual in (True, False):
        x, r, w = norm_inputs(d + n, n, d, dt, residual)
        out, rout = torch.empty((n, d), dtype=odt, device=DEV), torch.empty((n, d), dtype=dt, device=DEV)
        dmel.dmel_add_rmsnorm(x, w, out, residual=r, residual_out=rout, eps=1e-5)
        assert dmel.dmel_last_launch_count() == 1
        s, y = oracle_mod.add_rmsnorm(f64(x), None if r is None else f64(r), f64(w), 1e-5)
        assert (np.abs(f64(rout) - s) <= (HALF_STEP[dt] * 1.001 + 2.0 ** -24) * np.abs(s)).all()
        assert (np.abs(f64(out) - y) <= (HALF_STEP[odt] * 1.001 + norm_bound(d)) * np.abs(y) + 1e-37).all()
        alone = torch.empty_like(out)
        dmel.dmel_add_rmsnorm(x, w, alone, residual=r, eps=1e-5)  # without the stream out
        assert torch.equal(alone, out)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("block", [0, 32, 64, 128])
@pytest.mark.parametrize("n,d", [(1, 8), (3, 40), (5, 256), (2, 1000), (3, 5992), (4, 6144), (2, 16384)])
def test_add_rmsnorm_e4m3(dt, block, n, d, oracle_mod):
    x, r, w = norm_inputs(7 * d + n, n, d, dt)
    x[:, :8] *= 30.0       # blocks of very different size
    if d > 200:
        x[n - 1, 128:192] = 0.0
        r[n - 1, 128:192] = 0.0  # and whole blocks of zeros
    blocks = -(-d // block) if block else 1
    out = torch.empty((n, d), dtype=E4M3, device=DEV)
    scales, rout = torch.empty((n, blocks), device=DEV), torch.empty_like(x)
    dmel.dmel_add_rmsnorm(x, w, out, residual=r, residual_out=rout, eps=1e-6, scales=scales, scale_block=block)
    s, y, sc = oracle_mod.add_rmsnorm(f64(x), f64(r), f64(w), 1e-6, block)
    b = norm_bound(d)
    assert (np.abs(f64(scales) - sc) <= (b + 2 * 2.0 ** -24) * sc).all()
    each = np.repeat(sc, block or d, axis=1)[:, :d]
    # half a step of e4m3: 2^-4 of the value, 2^-10 below its smallest normal value 2^-6
    q = f64(out.float())
    assert np.isfinite(q).all() and (np.abs(q) <= 448).all()
    assert (np.abs(q - y / each) <= (2.0 ** -4 + 2 * b + 4 * 2.0 ** -24) * np.abs(y / each) + 2.0 ** -10).all()
    top = np.array([[np.abs(q[i, c:c + (block or d)]).max() for c in range(0, d, block or d)] for i in range(n)])
    assert ((top == 448) | (sc <= 1e-30)).all()  # each block's largest value fills the range
    assert (np.abs(f64(rout) - s) <= (HALF_STEP[dt] * 1.001 + 2.0 ** -24) * np.abs(s)).all()


def test_add_rmsnorm_zero_rows_nan_and_infinity():
    d = 520
    x, r, w = norm_inputs(3, 6, d, F32)
    x[1] = 0.0; r[1] = 0.0          # a row of zeros: zeros, whatever eps is
    x[2, 17] = float("nan")         # NaN spreads over its row
    x[3, 5] = float("inf")          # an infinity: the others are scaled to zero, itself is inf * 0
    x[4] = 1e-30; r[4] = 0.0        # squares that underflow: eps decides
    out, y8 = torch.empty_like(x), torch.empty((6, d), dtype=E4M3, device=DEV)
    sc = torch.empty((6, 5), device=DEV)
    dmel.dmel_add_rmsnorm(x, w, out, residual=r, eps=1e-6)
    dmel.dmel_add_rmsnorm(x, w, y8, residual=r, eps=1e-6, scales=sc, scale_block=128)
    clean, clean8, sc_clean = torch.empty_like(x), torch.empty_like(y8), torch.empty_like(sc)
    for i in (0, 5):  # the rows around them are as they are alone
        dmel.dmel_add_rmsnorm(x[i:i + 1], w, clean[i:i + 1], residual=r[i:i + 1], eps=1e-6)
        dmel.dmel_add_rmsnorm(x[i:i + 1], w, clean8[i:i + 1], residual=r[i:i + 1], eps=1e-6, scales=sc_clean[i:i + 1],
                              scale_block=128)
        assert torch.equal(out[i], clean[i]) and torch.equal(y8[i].view(torch.uint8), clean8[i].view(torch.uint8))
    assert (out[1] == 0).all() and (y8[1].float() == 0).all() and (sc[1] > 0).all()
    assert out[2].isnan().all() and y8[2].float().isnan().all() and sc[2].isfinite().all()
    assert out[3, 5].isnan() and (out[3, :5] == 0).all() and (out[3, 6:] == 0).all()
    torch.testing.assert_close(out[4], 1e-30 / 1e-3 * w, rtol=1e-5, atol=0)


@pytest.mark.parametrize("eps", [1e-12, 1e-30])
@pytest.mark.parametrize("block", [0, 32, 128])
def test_add_rmsnorm_e4m3_rows_next_to_zero(block, eps, oracle_mod):
    """Padding rows and rows of 1e-36 with a small eps: 1 / sqrt(eps) / scale is above fp32's range."""
    d = 264
    x, _, w = norm_inputs(4, 4, d, F32, residual=False)
    x[1] = 0.0
    x[2] *= 1e-36
    blocks = -(-d // block) if block else 1
    out, sc = torch.empty((4, d), dtype=E4M3, device=DEV), torch.empty((4, blocks), device=DEV)
    dmel.dmel_add_rmsnorm(x, w, out, eps=eps, scales=sc, scale_block=block)
    _, y, ref = oracle_mod.add_rmsnorm(f64(x), None, f64(w), float(np.float32(eps)), block)
    b = norm_bound(d) + 4 * 2.0 ** -24
    assert (np.abs(f64(sc) - ref) <= b * ref).all()
    q, each = f64(out.float()), np.repeat(ref, block or d, axis=1)[:, :d]
    # w s itself (1e-36) is rounded to fp32's normal numbers
    assert (np.abs(q - y / each) <= (2.0 ** -4 + 2 * b) * np.abs(y / each) + 2.0 ** -10).all()
    assert (q[1] == 0).all()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_add_rmsnorm_in_place(dt):
    """The stream updated in its own buffer and the normed rows over x: the same bits; rows behind the
    call's stay as they were."""
    n, d = 9, 6144
    x, r, w = norm_inputs(11, n, d, dt)
    out, rout = torch.empty_like(x), torch.empty_like(r)
    dmel.dmel_add_rmsnorm(x, w, out, residual=r, residual_out=rout)
    for a, b in (("x", "r"), ("r", "x")):
        bufs = {"x": x.clone(), "r": r.clone()}
        dmel.dmel_add_rmsnorm(bufs["x"], w, bufs[a], residual=bufs["r"], residual_out=bufs[b])
        assert torch.equal(bufs[a], out) and torch.equal(bufs[b], rout)
    big = torch.full((n + 3, d), 7.0, dtype=dt, device=DEV)
    dmel.dmel_add_rmsnorm(x, w, big[:n], residual=r)
    assert torch.equal(big[:n], out) and (big[n:] == 7.0).all()


def test_add_rmsnorm_more_rows_than_blocks(oracle_mod):
    """Rows past the largest grid: every row is its own (narrow rows keep it small)."""
    n, d = 148 * 64 * 8 + 77, 16
    x, r, w = norm_inputs(12, n, d, F32)
    out, scales = torch.empty((n, d), dtype=E4M3, device=DEV), torch.empty(n, device=DEV)
    dmel.dmel_add_rmsnorm(x, w, out, residual=r, scales=scales)
    s = x.double() + r.double()
    y = s * w.double() / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6)
    sc = y.abs().amax(1) / 448
    assert ((scales.double() - sc).abs() <= (norm_bound(d) + 2.0 ** -23) * sc).all()
    q = y / sc[:, None]
    assert ((out.double() - q).abs() <= (2.0 ** -4 + 2 * norm_bound(d) + 2.0 ** -22) * q.abs() + 2.0 ** -10).all()


# more rows than a block each, three to a block and more (the blocks' largest grids at 148 SMs, by width and types)
@pytest.mark.parametrize("dt,odt,block,n,d", [
    (BF16, E4M3, 128, 3 * 1480 + 7, 5992), (BF16, E4M3, 0, 2 * 1480 + 1, 6144), (BF16, E4M3, 32, 2 * 9472 + 5, 1000),
    (BF16, BF16, 0, 2 * 5920 + 77, 5992), (BF16, F32, 0, 2 * 5920 + 3, 6144), (BF16, BF16, 0, 2 * 37888 + 9, 1000),
    (F32, E4M3, 128, 2 * 592 + 417, 5992), (F32, E4M3, 0, 2 * 592 + 1, 6144), (F32, E4M3, 64, 2 * 9472 + 3, 264),
    (F32, F32, 0, 2 * 9472 + 3, 1000), (F32, BF16, 0, 2 * 9472 + 1, 264), (F32, F32, 0, 9472 + 99, 8200),
    (BF16, E4M3, 0, 2 * 592 + 5, 16384), (BF16, BF16, 0, 5000, 264), (BF16, BF16, 0, 5000, 512), (BF16, E4M3, 64, 5000, 256),
    # as many rows as SMs, and one more: another number of pieces per thread
    (BF16, BF16, 0, 148, 6144), (BF16, BF16, 0, 149, 6144), (BF16, E4M3, 128, 148, 1000), (BF16, E4M3, 128, 149, 1000),
    (BF16, E4M3, 0, 149, 264), (BF16, BF16, 0, 149, 8)])
def test_add_rmsnorm_rows_of_a_prompt(dt, odt, block, n, d):
    """Wide rows past the grid: a block walks its rows with barriers between. The stream in its own buffer, the rows
    behind the call's as they were; against fp64 on the device."""
    x, r, w = norm_inputs(n + d, n, d, dt)
    if odt is E4M3:
        x[::3, :8] *= 30.0
    blocks, b = -(-d // (block or d)), norm_bound(d)
    out = torch.full((n + 2, d), 7.0, device=DEV).to(odt)
    rout, scales = torch.cat([r, r[:2]]), torch.full((n + 2, blocks), 9.0, device=DEV)
    kw = dict(scales=scales[:n], scale_block=block) if odt is E4M3 else {}
    dmel.dmel_add_rmsnorm(x, w, out[:n], residual=rout[:n], residual_out=rout[:n], eps=1e-5, **kw)
    assert (out[n:].float() == 7.0).all() and torch.equal(rout[n:], r[:2]) and (scales[n:] == 9.0).all()
    for i in range(0, n, 4096):  # (rows in parts: fp64 copies)
        at = slice(i, min(i + 4096, n))
        s = x[at].double() + r[at].double()
        y = s * w.double() / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-5)
        assert ((rout[at].double() - s).abs() <= (HALF_STEP[dt] * 1.001 + 2.0 ** -24) * s.abs()).all()
        if odt is not E4M3:
            assert ((out[at].double() - y).abs() <= (HALF_STEP[odt] * 1.001 + b) * y.abs() + 1e-37).all()
            continue
        wide = torch.nn.functional.pad(y.abs(), (0, blocks * (block or d) - d)).view(-1, blocks, block or d)
        sc = wide.amax(2).clamp(min=1e-30) / 448
        assert ((scales[at].double() - sc).abs() <= (b + 2 * 2.0 ** -24) * sc).all()
        q = y / sc.repeat_interleave(block or d, 1)[:, :d]
        assert ((out[at].double() - q).abs() <= (2.0 ** -4 + 2 * b + 4 * 2.0 ** -24) * q.abs() + 2.0 ** -10).all()
    if odt is dt:  # the normed rows over x
        dmel.dmel_add_rmsnorm(x, w, x, residual=r, residual_out=r, eps=1e-5)
        assert torch.equal(x, out[:n]) and torch.equal(r, rout[:n])


# ------------------------------------------------------------------------------ routing

def run_route(logits, k, bias=None, shared=0, **kw):
    n = logits.shape[0]
    ids = torch.full((n, k + shared), -7, dtype=torch.int32, device=DEV)
    wts = torch.full((n, k + shared), 9.0, device=DEV)
    dmel.dmel_route(logits, ids, wts, n_shared=shared, bias=bias, **kw)
    return ids.cpu().numpy(), wts.double().cpu().numpy()


def check_route(logits, k, oracle_mod, bias=None, shared=0, sigmoid=True, groups=1, topk_groups=1, renorm=True, scale=1.0):
    ids, w = run_route(logits, k, bias, shared, scoring=int(sigmoid), n_groups=groups, topk_groups=topk_groups,
                       renormalise=renorm, scale=scale)
    rid, rw = oracle_mod.route(f64(logits), shared, k, sigmoid, None if bias is None else f64(bias), groups, topk_groups,
                               renorm, scale)
    np.testing.assert_array_equal(ids, rid)
    # two exponentials of rounded differences (their size, at most `spread`, and 4 units each), a sum of up
    # to 32 (5; 1024 logits in a softmax's denominator: 10), divisions and products, in units of 2^-24
    l = f64(logits)
    l = l[np.isfinite(l)]
    spread = (l.max() - l.min()) if l.size else 0.0
    assert (np.abs(w - rw) <= (2 * spread + 28) * 2.0 ** -24 * np.abs(rw) + 1e-37).all()
    return ids, w


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("n,e,shared,k", [(1, 1, 0, 1), (1, 256, 2, 6), (5, 7, 0, 7), (33, 60, 1, 4), (130, 256, 0, 8),
                                          (64, 31, 3, 5), (64, 33, 0, 2), (17, 1024, 0, 32), (9, 513, 4, 12), (20, 128, 1, 8), (20, 65, 0, 5),
                                          (20, 384, 0, 6), (7, 512, 2, 8)])
def test_route(dt, sigmoid, n, e, shared, k, oracle_mod):
    g = torch.Generator(device=DEV).manual_seed(e + n)
    logits = (2.0 * torch.randn((n, e + shared), generator=g, device=DEV)).to(dt)
    bias = 0.1 * torch.randn(e, generator=g, device=DEV)
    for b in (bias, torch.zeros(e, device=DEV), None):
        check_route(logits, k, oracle_mod, b, shared, sigmoid)
    check_route(logits, k, oracle_mod, bias, shared, sigmoid, renorm=False, scale=-2.5)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("e,groups,topk_groups,k", [(256, 8, 4, 8), (64, 32, 5, 9), (60, 4, 3, 7), (12, 12, 5, 5), (96, 3, 1, 20),
                                                    (6, 2, 2, 6), (1024, 16, 2, 16), (50, 5, 1, 10)])
def test_route_groups(dt, e, groups, topk_groups, k, oracle_mod):
    g = torch.Generator(device=DEV).manual_seed(e)
    logits = torch.randn((70, e + 1), generator=g, device=DEV).to(dt)
    bias = 0.1 * torch.randn(e, generator=g, device=DEV)
    for b in (bias, None):
        for sigmoid in (True, False):
            check_route(logits, k, oracle_mod, b, 1, sigmoid, groups, topk_groups)


def test_route_ties_go_to_the_lower_index(oracle_mod):
    """Equal logits (bf16 steps make many), equal groups, and biases that make unequal logits nearly equal."""
    flat = torch.zeros((3, 130), device=DEV)
    ids, w = check_route(flat, 5, oracle_mod)
    assert (ids == np.arange(5)).all() and np.allclose(w, 0.2)
    check_route(flat, 5, oracle_mod, torch.zeros(130, device=DEV), groups=13, topk_groups=2)
    g = torch.Generator(device=DEV).manual_seed(5)
    steps = torch.randint(-2, 3, (200, 256), generator=g, device=DEV).float()
    for bias in (None, torch.zeros(256, device=DEV), torch.randint(0, 2, (256,), generator=g, device=DEV).float()):
        for sigmoid in (True, False):
            check_route(steps, 8, oracle_mod, bias, sigmoid=sigmoid)
            check_route(steps, 8, oracle_mod, bias, sigmoid=sigmoid, groups=8, topk_groups=3)


def cancelling_bias(size, groups, per):
    """Each group's first expert at +size, the others at -size: its two largest values nearly cancel in its rating."""
    bias = torch.full((groups, per), -size, device=DEV)
    bias[:, 0] = size
    return bias.flatten()


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("size", [100.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("groups,per,kept", [(2, 2, 1), (8, 2, 4), (16, 4, 5), (32, 8, 8)])
def test_route_groups_whose_values_cancel(size, groups, per, kept, sigmoid, oracle_mod):
    """A rating near zero from values far from it: what rounds is the values. At 1e4 and 1e6 the fp32 ratings put
    groups of tens of these tokens in another order than the 64-bit ones."""
    g = torch.Generator(device=DEV).manual_seed(int(size) + groups)
    logits = torch.randn((400, groups * per), generator=g, device=DEV)
    check_route(logits, min(6, kept * per), oracle_mod, cancelling_bias(size, groups, per), 0, sigmoid, groups, kept)


def test_route_groups_whose_values_cancel_by_hand(oracle_mod):
    """Sigmoids 0.590492 + 0.698044 = 1.288536 below 0.647484 + 0.641067 = 1.288552. Beside +-1000 fp32 steps are
    6.1e-5, no value is within 7e-6 of a tie, and the first rating is the larger by one step."""
    logits = torch.tensor([[0.366, 0.838, 0.608, 0.58]], device=DEV)
    bias = torch.tensor([1000.0, -1000.0, 1000.0, -1000.0], device=DEV)
    ids, _ = check_route(logits, 2, oracle_mod, bias, 0, True, 2, 1)
    assert ids[0].tolist() == [2, 3]


@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_values_fp32_cannot_tell_apart(sigmoid, oracle_mod):
    """Biases that cancel the scores to within fp32's rounding, either way: the 64-bit order holds."""
    r = np.random.default_rng(6)
    n, e = 64, 64
    logits = torch.from_numpy(r.standard_normal((1, e)).astype(np.float32)).repeat(n, 1)
    l = logits[0].double().numpy()
    s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l) / np.exp(l).sum()
    bias = torch.from_numpy((1.0 - s).astype(np.float32))  # score + bias = 1 but for the bias' rounding
    # a row's logits moved by single steps, so that rows differ
    moved = torch.nextafter(logits, torch.full_like(logits, 9.0))
    logits = torch.where(torch.from_numpy(r.random((n, e)) < 0.5), moved, logits).to(DEV)
    check_route(logits, 8, oracle_mod, bias.to(DEV), sigmoid=sigmoid)
    check_route(logits, 8, oracle_mod, bias.to(DEV), sigmoid=sigmoid, groups=8, topk_groups=2)
    check_route(logits, 8, oracle_mod, 5.0 + bias.to(DEV), sigmoid=sigmoid)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("e,k", [(24, 4), (24, 24), (40, 31), (40, 32), (300, 6)])
def test_route_few_near_one_another(e, k, sigmoid, oracle_mod):
    """As above, with up to 24 experts near one another and the others far below, or all in pairs and threes."""
    r = np.random.default_rng(e + k)
    for size in (2, 3, 24):
        base = r.standard_normal(e).astype(np.float32)
        rows = np.repeat(base[None], 50, 0)
        steps = np.spacing(rows) * r.integers(-1, 2, rows.shape)
        rows = np.where(r.random(rows.shape) < 0.5, rows + steps.astype(np.float32), rows)
        l = base.astype(np.float64)
        s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l) / np.exp(l).sum()
        height = -0.25 * (np.arange(e) // size)  # sets of `size` experts at the same height
        bias = (height[r.permutation(e)] - s).astype(np.float32)
        check_route(torch.from_numpy(rows).to(DEV), k, oracle_mod, torch.from_numpy(bias).to(DEV), sigmoid=sigmoid)


@pytest.mark.parametrize("e,groups", [(30, 1), (256, 1), (256, 8), (1000, 1)])
@pytest.mark.parametrize("near", [3, 8, 40])
def test_route_ties_among_near_logits(e, groups, near, oracle_mod):
    """Equal logits at the edge of the choice with others a unit or two in the last place away; no bias, and
    a bias that is the same for all of them."""
    r = np.random.default_rng(e + near)
    rows = r.standard_normal((60, e)).astype(np.float32)
    for row in rows:
        at = r.permutation(e)[:near]
        level = np.sort(row)[-6]
        row[at] = level + np.spacing(level) * r.integers(-1, 2, at.size).astype(np.float32)
    logits = torch.from_numpy(rows).to(DEV)
    for bias in (None, torch.full((e,), 0.125, device=DEV)):
        for sigmoid in (True, False):
            check_route(logits, 6, oracle_mod, bias, 0, sigmoid, groups, (groups + 1) // 2)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_masks(sigmoid, oracle_mod):
    """-inf, the types' lowest values, NaN and +inf; rows with fewer experts than slots, and with none."""
    inf, nan, low = float("inf"), float("nan"), torch.finfo(F32).min
    g = torch.Generator(device=DEV).manual_seed(7)
    logits = torch.randn((8, 42), generator=g, device=DEV)
    logits[0, 3:40] = -inf           # three experts left
    logits[1, :] = -inf              # none, and no shared one
    logits[2, :40] = nan             # only the shared ones
    logits[3, 40] = -inf             # a masked shared expert
    logits[4, 5:] = low              # masked by the lowest value: still chosen when nothing else is left
    logits[5, ::2] = -inf
    logits[6, :] = low
    bias = 0.1 * torch.randn(40, generator=g, device=DEV)
    for b in (None, bias):
        for groups, kept in ((1, 1), (8, 3)):
            for renorm in (True, False):
                ids, w = check_route(logits, 6, oracle_mod, b, 2, sigmoid, groups, kept, renorm)
                assert (ids[1] == -1).all() and (w[1] == 0).all()
                assert np.isfinite(w).all()
    ids, _ = run_route(logits, 6, None, 2, scoring=int(sigmoid))
    assert ids[0].tolist()[3:6] == [-1, -1, -1] and ids[2].tolist() == [-1] * 6 + [40, 41]
    hot = logits.clone()
    hot[7, 9] = inf                  # counts as the largest finite value
    ids, w = run_route(hot, 6, None, 2, scoring=int(sigmoid))
    assert ids[7, 0] == 9 and np.isfinite(w[7]).all()
    if not sigmoid:
        assert w[7, 0] == 1.0 and (w[7, 1:] == 0).all()


@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_bias_without_a_value(sigmoid, oracle_mod):
    """NaN and -inf in the bias keep an expert out, +inf puts it first (several by index)."""
    g = torch.Generator(device=DEV).manual_seed(9)
    logits = torch.randn((20, 48), generator=g, device=DEV)
    bias = 0.1 * torch.randn(48, generator=g, device=DEV)
    bias[3] = bias[17] = float("nan")
    bias[20:30] = -float("inf")
    bias[40] = bias[12] = float("inf")
    for groups, kept in ((1, 1), (6, 4)):
        ids, _ = check_route(logits, 5, oracle_mod, bias, 0, sigmoid, groups, kept)
        assert (ids[:, :2] == [12, 40]).all()
    bias[:] = float("nan")
    ids, w = check_route(logits, 5, oracle_mod, bias, 0, sigmoid)
    assert (ids == -1).all() and (w == 0).all()


@pytest.mark.parametrize("k,shared", [(1, 31), (31, 1), (32, 0), (12, 0)])
def test_route_all_slots(k, shared, oracle_mod):
    g = torch.Generator(device=DEV).manual_seed(10)
    logits = torch.randn((40, 64 + shared), generator=g, device=DEV)
    check_route(logits, k, oracle_mod, 0.1 * torch.randn(64, generator=g, device=DEV), shared)


def test_no_rows_on_the_gpu():
    e = lambda *shape, dtype=F32: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    dmel.dmel_add_rmsnorm(e(0, 64), e(64), e(0, 64), residual=e(0, 64))
    dmel.dmel_route(e(0, 8), e(0, 2, dtype=torch.int32), e(0, 2))
    assert dmel.dmel_experts_workspace_size(0, 2, 4, 64, 32) == 0
    dmel.dmel_experts(e(0, 64, dtype=BF16), e(0, 2, dtype=torch.int32), e(0, 2), e(4, 64, 64, dtype=BF16),
                      e(4, 32, 64, dtype=BF16), e(0, 64, dtype=BF16), None)
    assert dmel.dmel_last_launch_count() == 0


def test_route_small_scores_keep_their_ratios(oracle_mod):
    """Sigmoids far below fp32's range: the renormalised weights are those of the formula."""
    logits = torch.tensor([[-200.0, -201.0, -203.0, -260.0], [-90.0, -89.0, -95.0, -88.5]], device=DEV)
    check_route(logits, 3, oracle_mod)
    ids, w = run_route(logits, 2, None, 0)
    assert abs(w[0, 0] - 1 / (1 + np.exp(-1.0))) < 1e-6


def test_route_many_tokens_and_rows_behind(oracle_mod):
    n = 148 * 64 * 4 * 2 + 3
    g = torch.Generator(device=DEV).manual_seed(8)
    logits = torch.randn((n, 9), generator=g, device=DEV)
    ids = torch.full((n + 2, 3), -7, dtype=torch.int32, device=DEV)
    w = torch.full((n + 2, 3), 9.0, device=DEV)
    dmel.dmel_route(logits, ids[:n], w[:n], n_shared=1, renormalise=False)
    top = torch.topk(logits[:, :8], 2, dim=1)
    assert torch.equal(ids[:n, :2].long(), top.indices) and (ids[:n, 2] == 8).all()
    ref = torch.sigmoid(torch.cat([top.values, logits[:, 8:]], 1).double())
    assert ((w[:n].double() - ref).abs() <= 16 * 2.0 ** -24 * ref).all()
    assert (ids[n:] == -7).all() and (w[n:] == 9.0).all()


@pytest.mark.parametrize("e,groups,kept", [(64, 1, 1), (64, 8, 3), (300, 1, 1)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_second_tokens_of_a_warp(e, groups, kept, sigmoid, oracle_mod):
    """More tokens than warps: 500 rows, each at many places of a prompt, have their ids and weights wherever they
    stand. A third of them has values that only fp64 tells apart, a third groups that cancel."""
    g = torch.Generator(device=DEV).manual_seed(e + groups)
    base = torch.randn((500, e), generator=g, device=DEV)
    n = 148 * 64 * 4 * 2 + 777
    at = torch.randint(0, 500, (n,), generator=g, device=DEV)
    plain = 0.1 * torch.randn(e, generator=g, device=DEV)
    row = base[0].double()
    score = torch.sigmoid(row) if sigmoid else torch.softmax(row, 0)
    near = (1.0 - score).float()
    base[100:250] = torch.where(torch.rand((150, e), generator=g, device=DEV) < 0.5, base[0],
                                torch.nextafter(base[0], torch.full_like(base[0], 9.0)))
    for bias in (plain, near, cancelling_bias(1e4, groups, e // groups)):
        rid, rw = oracle_mod.route(f64(base), 0, 6, sigmoid, f64(bias), groups, kept)
        ids, w = run_route(base[at], 6, bias, scoring=int(sigmoid), n_groups=groups, topk_groups=kept)
        where = at.cpu().numpy()
        np.testing.assert_array_equal(ids, rid[where])
        spread = float(base.max() - base.min())
        assert (np.abs(w - rw[where]) <= (2 * spread + 28) * 2.0 ** -24 * rw[where]).all()


# ------------------------------------------------------------------------------ experts

def expert_inputs(seed, n, slots, e, d, h, empty=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, d), generator=g, device=DEV).to(BF16)
    w_in = (torch.randn((e, d, 2 * h), generator=g, device=DEV) / d ** 0.5).to(BF16)
    w_out = (torch.randn((e, h, d), generator=g, device=DEV) / h ** 0.5).to(BF16)
    ids = torch.randint(0, e, (n, slots), generator=g, device=DEV, dtype=torch.int32)
    if empty:
        ids[torch.rand((n, slots), generator=g, device=DEV) < empty] = -1
    w = torch.randn((n, slots), generator=g, device=DEV)
    return x, ids, w, w_in, w_out


def run_experts(x, ids, w, w_in, w_out, stream=None, workspace=None):
    e, h, d = w_out.shape
    n, slots = ids.shape
    if workspace is None:
        # the scratch's old contents do not matter
        workspace = torch.full((dmel.dmel_experts_workspace_size(n, slots, e, d, h),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((n, d), 5.0, dtype=BF16, device=DEV)
    dmel.dmel_experts(x, ids, w, w_in, w_out, out, workspace, stream=stream)
    return out


def check_experts(x, ids, w, w_in, w_out, oracle_mod):
    out = run_experts(x, ids, w, w_in, w_out)
    assert dmel.dmel_last_launch_count() >= 1
    masked = torch.where(ids >= 0, w, torch.zeros_like(w))
    ref, _, spread, slots_size = oracle_mod.experts(f64(x), ids.cpu().numpy(), f64(masked), f64(w_in), f64(w_out))
    got = f64(out)
    assert np.isfinite(got).all()
    # no element beyond what the roundings can do together (a slot's row to 11 bits among them), and the
    # whole as far off as independent roundings are: each uniform within half a step, 2^-8 / sqrt 3 of the
    # value at most, for the gated row and the output (and an eighth of that for the slots' rows)
    sums = ids.shape[1] * 2.0 ** -23 * np.abs(ref) + 2.0 ** -11 * slots_size
    assert (np.abs(got - ref) <= 2.0 ** -8 * 1.01 * np.abs(ref) + 1.01 * spread + sums + 1e-37).all()
    if ref.size >= 2000:
        assert np.linalg.norm(got - ref) <= 1.25 * 2 ** 0.5 * 2.0 ** -8 / 3 ** 0.5 * np.linalg.norm(ref)
    assert dmel.dmel_get_device_error(clear=True) == 0
    return out


@pytest.mark.parametrize("n,slots,e,d,h", [
    (1, 1, 1, 8, 8), (1, 6, 32, 512, 128), (2, 3, 4, 72, 40), (5, 2, 3, 200, 264), (40, 2, 2, 136, 72),
    (300, 2, 3, 264, 136), (257, 1, 1, 64, 64), (700, 3, 7, 328, 200), (64, 8, 96, 128, 64), (33, 64, 5, 64, 24),
    (1100, 4, 2, 64, 520), (3, 2, 1024, 24, 16), (171, 3, 40, 72, 40), (64, 1, 1, 64, 264), (65, 1, 1, 64, 72),
    (16, 4, 33, 520, 136), (32, 2, 3, 264, 72), (13, 5, 9, 520, 136),
    # the first product's K in parts: 2, 4, 4, 2, 3
    (5, 2, 3, 2056, 72), (40, 2, 2, 4104, 136), (1, 1, 2, 4096, 64), (700, 1, 1, 2200, 200), (130, 3, 5, 3080, 264),
    # the widest
    (3, 2, 2, 65536, 8), (3, 2, 2, 8, 65536)])
def test_experts(n, slots, e, d, h, oracle_mod):
    check_experts(*expert_inputs(n + d, n, slots, e, d, h), oracle_mod)


@pytest.mark.parametrize("n,slots,e,d,h", [(30000, 5, 3, 16, 8), (20000, 6, 32, 16, 8), (1500, 1, 1000, 16, 8),
                                           (14000, 2, 5, 2056, 600)])
def test_experts_many_slots(n, slots, e, d, h):
    """Plans of several blocks and batches, tiles of twice the columns: against the formula in fp64, expert by expert."""
    x, ids, w, w_in, w_out = expert_inputs(n, n, slots, e, d, h, empty=0.1)
    out = run_experts(x, ids, w, w_in, w_out)
    ref = torch.zeros((n, d), dtype=torch.float64, device=DEV)
    for i in range(e):
        t, j = torch.nonzero(ids == i, as_tuple=True)
        a = x[t].double() @ w_in[i].double()
        y = torch.nn.functional.silu(a[:, :h]) * a[:, h:] @ w_out[i].double()
        ref.index_add_(0, t, y * w[t, j].double()[:, None])
    # the roundings of the gated row and the output, as in check_experts
    assert (out.double() - ref).norm() <= 1.25 * 2 ** 0.5 * 2.0 ** -8 / 3 ** 0.5 * ref.norm()
    assert (out[(ids < 0).all(1)] == 0).all()


@pytest.mark.parametrize("slots,e,d,h,most", [(6, 32, 1032, 136, 18), (1, 2, 4096, 264, 2048), (2, 3, 2056, 72, 300)])
def test_experts_workspace_of_the_largest_batch(slots, e, d, h, most):
    """One workspace, sized for the largest batch, for every smaller one: the bits of a workspace of the call's own."""
    x, ids, w, w_in, w_out = expert_inputs(65, most, slots, e, d, h)
    size = dmel.dmel_experts_workspace_size(most, slots, e, d, h)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    for n in sorted({1, 2, 5, 10, 11, 16, 17, 64 // slots, 64 // slots + 1, most // 2, most - 1, most}):
        args = x[:n].contiguous(), ids[:n].contiguous(), w[:n].contiguous(), w_in, w_out
        assert torch.equal(run_experts(*args, workspace=ws), run_experts(*args)), n
    assert dmel.dmel_get_device_error(clear=True) == 0


def test_experts_model_width(oracle_mod):
    """6144 columns, 1,024 hidden: one token's six experts, and a step of 20 tokens."""
    x, ids, w, w_in, w_out = expert_inputs(50, 20, 6, 8, 6144, 1024)
    a = check_experts(x, ids, w, w_in, w_out, oracle_mod)
    b = check_experts(x[:1].clone(), ids[:1].clone(), w[:1].clone(), w_in, w_out, oracle_mod)
    assert (a[0].float() - b[0].float()).norm() <= 2.0 ** -7 * b[0].float().norm()


def test_experts_exact_on_integers():
    """One-hot tokens, gates of 64 (silu(64) is 64 in fp32) and small integers elsewhere: every product and
    sum is exact, so each output is the exact value rounded once."""
    for n, slots, e, d, h in ((3, 2, 4, 80, 56), (500, 3, 5, 344, 216), (90, 2, 64, 136, 72)):
        g = torch.Generator(device=DEV).manual_seed(n)
        at = torch.randint(0, d, (n,), generator=g, device=DEV)
        x = torch.nn.functional.one_hot(at, d).to(BF16)
        w_in = torch.randint(-1, 2, (e, d, 2 * h), generator=g, device=DEV).to(BF16)
        w_in[:, :, :h] = 64.0
        w_out = torch.randint(-1, 2, (e, h, d), generator=g, device=DEV).to(BF16)
        ids = torch.randint(0, e, (n, slots), generator=g, device=DEV, dtype=torch.int32)
        w = 2.0 ** torch.randint(-1, 2, (n, slots), generator=g, device=DEV)
        up = w_in[ids.long(), at[:, None], h:].double()              # [n, slots, h]
        ref = torch.zeros((n, d), dtype=torch.float64, device=DEV)
        for j in range(slots):
            ref += w[:, j:j + 1].double() * torch.bmm(64 * up[:, j:j + 1], w_out[ids[:, j].long()].double())[:, 0]
        assert torch.equal(run_experts(x, ids, w, w_in, w_out), ref.float().to(BF16))


def check_experts_on_device(x, ids, w, w_in, w_out):
    """As check_experts, the formula in fp64 on the device, expert by expert."""
    out = run_experts(x, ids, w, w_in, w_out)
    (n, d), (e, h, _) = x.shape, w_out.shape
    ref, spread, size = (torch.zeros((n, d), dtype=torch.float64, device=DEV) for _ in range(3))
    for i in range(e):
        t, j = torch.nonzero(ids == i, as_tuple=True)
        if t.numel() == 0:
            continue
        xi, wi, wo, wt = x[t].double(), w_in[i].double(), w_out[i].double(), w[t, j].double()[:, None]
        a, b = xi @ wi, xi.abs() @ wi.abs()
        g, u = a[:, :h], a[:, h:]
        hid = g * torch.sigmoid(g) * u
        y = wt * (hid @ wo)
        sums = (d / 16 + 16) * 2.0 ** -23
        dh = 2.0 ** -8 * hid.abs() + sums * (1.1 * b[:, :h] * u.abs() + g.abs() * b[:, h:])
        ref.index_add_(0, t, y)
        size.index_add_(0, t, y.abs())
        spread.index_add_(0, t, wt.abs() * ((dh + (h / 16 + 16) * 2.0 ** -23 * hid.abs()) @ wo.abs()))
    off = (out.double() - ref).abs()
    sums = ids.shape[1] * 2.0 ** -23 * ref.abs() + 2.0 ** -11 * size
    assert (off <= 2.0 ** -8 * 1.01 * ref.abs() + 1.01 * spread + sums + 1e-37).all()
    assert off.norm() <= 1.25 * 2 ** 0.5 * 2.0 ** -8 / 3 ** 0.5 * ref.norm()
    assert (out[(ids < 0).all(1)] == 0).all()
    assert dmel.dmel_get_device_error(clear=True) == 0
    return out


@pytest.mark.parametrize("n,slots,e,d,h", [
    (14000, 2, 5, 2056, 600), (19000, 1, 1, 2048, 520),   # tiles of twice the columns, with a remainder of columns
    (30000, 5, 3, 72, 40), (20000, 6, 32, 136, 72), (1500, 1, 1000, 16, 8)])  # plans of several blocks and batches
def test_experts_many_slots_value_by_value(n, slots, e, d, h):
    check_experts_on_device(*expert_inputs(n, n, slots, e, d, h, empty=0.1))


@pytest.mark.parametrize("n,slots,e,d,h", [(14000, 2, 5, 2056, 600), (30000, 5, 3, 72, 40), (20000, 6, 32, 136, 72),
                                           (4000, 17, 300, 80, 56)])
def test_experts_many_slots_exact_on_integers(n, slots, e, d, h):
    """As test_experts_exact_on_integers, at tiles of twice the columns and plans of several blocks and batches: a slot's
    values are 64 times whole numbers up to 600, which 11 bits hold."""
    g = torch.Generator(device=DEV).manual_seed(n)
    at = torch.randint(0, d, (n,), generator=g, device=DEV)
    x = torch.nn.functional.one_hot(at, d).to(BF16)
    w_in = torch.randint(-1, 2, (e, d, 2 * h), generator=g, device=DEV).to(BF16)
    w_in[:, :, :h] = 64.0
    w_out = torch.randint(-1, 2, (e, h, d), generator=g, device=DEV).to(BF16)
    ids = torch.randint(-1, e, (n, slots), generator=g, device=DEV, dtype=torch.int32)
    w = 2.0 ** torch.randint(-1, 2, (n, slots), generator=g, device=DEV)
    ref = torch.zeros((n, d), dtype=torch.float64, device=DEV)
    for i in range(e):
        t, j = torch.nonzero(ids == i, as_tuple=True)
        ref.index_add_(0, t, w[t, j].double()[:, None] * (64 * w_in[i, at[t], h:].double() @ w_out[i].double()))
    assert torch.equal(run_experts(x, ids, w, w_in, w_out), ref.float().to(BF16))


@pytest.mark.parametrize("n", [1, 8, 64, 600])
def test_experts_as_the_router_feeds_them(n):
    """256 routed experts, 6 chosen, and 2 shared ones that every token takes, 6144 columns and 1,024 hidden: tiles of
    many tokens beside tiles of one or two."""
    e, d, h = 258, 6144, 1024
    g = torch.Generator(device=DEV).manual_seed(n)
    weight = lambda *shape: torch.empty(shape, dtype=BF16, device=DEV).normal_(0.0, shape[1] ** -0.5, generator=g)  # noqa: E731
    w_in, w_out = weight(e, d, 2 * h), weight(e, h, d)
    x = torch.randn((n, d), generator=g, device=DEV).to(BF16)
    ids = torch.empty((n, 8), dtype=torch.int32, device=DEV)
    w = torch.empty((n, 8), device=DEV)
    logits = torch.randn((n, e), generator=g, device=DEV)
    dmel.dmel_route(logits, ids, w, n_shared=2, bias=0.05 * torch.randn(e - 2, generator=g, device=DEV))
    assert (ids[:, 6:] == torch.tensor([256, 257], device=DEV)).all()
    check_experts_on_device(x, ids, w, w_in, w_out)


def test_experts_empty_slots_and_bad_ids(oracle_mod):
    x, ids, w, w_in, w_out = expert_inputs(60, 90, 3, 6, 136, 72, empty=0.4)
    ids[5] = -1                      # a token without an expert: zeros
    w[ids < 0] = float("nan")        # weights of empty slots are not read
    out = check_experts(x, ids, w, w_in, w_out, oracle_mod)
    assert (out[5] == 0).all()
    assert (run_experts(x, torch.full_like(ids, -1), w, w_in, w_out) == 0).all()
    bad = torch.where(ids < 0, 6, ids)
    bad[7, 0] = -2
    ref = torch.where((bad == 6) | (bad == -2), -1, bad)
    wz = torch.nan_to_num(w)
    assert torch.equal(run_experts(x, bad, wz, w_in, w_out), run_experts(x, ref, wz, w_in, w_out))
    assert dmel.dmel_get_device_error(clear=True) & dmel.DMEL_DEVERR_EXPERT


def test_experts_one_expert_for_all_and_twice_in_a_token(oracle_mod):
    x, ids, w, w_in, w_out = expert_inputs(61, 290, 2, 9, 72, 40)
    ids[:] = 4
    out = check_experts(x, ids, w, w_in, w_out, oracle_mod)
    # two slots of one expert add their weights
    both = run_experts(x, ids[:, :1].contiguous(), w.sum(1, keepdim=True), w_in, w_out)
    assert ((out.float() - both.float()).abs() <= 2.0 ** -6 * both.float().abs() + 1e-3).all()


def test_experts_nan_stays_with_its_token():
    x, ids, w, w_in, w_out = expert_inputs(62, 200, 2, 3, 200, 72)
    clean = run_experts(x, ids, w, w_in, w_out)
    x[77, 3] = float("nan")
    x[78, 5] = float("inf")
    out = run_experts(x, ids, w, w_in, w_out)
    assert out[77].isnan().all()
    rest = torch.ones(200, dtype=torch.bool, device=DEV)
    rest[77:79] = False
    assert torch.equal(out[rest], clean[rest])


def test_experts_infinity_stays_in_its_column():
    """Columns whose products overflow, beside columns far above fp16's range and far below it."""
    x, ids, w, w_in, w_out = expert_inputs(64, 90, 2, 3, 200, 72)
    x = x.abs() + 1.0
    w_in[:, :, 0] = w_in[:, :, 72] = 1e8  # gate and up sums of 2e10 and more: a hidden value above 4e20 ...
    w_out[:, 0] = 0.0                     # ... which no column reads
    w_out[:, :, 20:40] *= 1e7
    w_out[:, :, 130:150] *= 1e-7
    clean = run_experts(x, ids, w, w_in, w_out)
    assert clean.isfinite().all()
    w_out[:, 0, 5] = w_out[:, 0, 140] = 1e30  # two that do
    out = run_experts(x, ids, w, w_in, w_out)
    assert not out[:, [5, 140]].isfinite().any()
    others = [c for c in range(200) if c not in (5, 140)]
    assert torch.equal(out[:, others], clean[:, others])


def test_experts_same_bits_every_time_and_rows_behind():
    x, ids, w, w_in, w_out = expert_inputs(63, 600, 4, 7, 264, 136)
    first = run_experts(x, ids, w, w_in, w_out)
    big = torch.full((603, 264), 7.0, dtype=BF16, device=DEV)
    ws = torch.zeros(dmel.dmel_experts_workspace_size(600, 4, 7, 264, 136), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        dmel.dmel_experts(x, ids, w, w_in, w_out, big[:600], ws)
        assert torch.equal(big[:600], first) and (big[600:] == 7.0).all()


# ------------------------------------------------------------------------------ together, streams, graphs

def block_step(s, x, state, ws, stream=None):
    """One pass through the block: ShortConv, residual + norm, router, experts, residual + norm in 8 bits."""
    kw = dict(stream=stream)
    dmel.dmel_shortconv(x, s["off"], s["conv"], s["y"], state=state, state_out=state, **kw)
    dmel.dmel_add_rmsnorm(s["y"], s["g1"], s["n1"], residual=s["stream"], residual_out=s["stream"], **kw)
    logits = torch.matmul(s["n1"], s["router"]).float()
    dmel.dmel_route(logits, s["ids"], s["wts"], n_shared=2, bias=s["bias"], **kw)
    dmel.dmel_experts(s["n1"], s["ids"], s["wts"], s["w_in"], s["w_out"], s["moe"], ws, **kw)
    dmel.dmel_add_rmsnorm(s["moe"], s["g2"], s["n2"], residual=s["stream"], residual_out=s["stream"], scales=s["sc"],
                          scale_block=128, **kw)
    return logits


def block_state(seed, n, d=264, h=72, e=16, k=3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *shape, scale=1.0: scale * torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    return dict(off=torch.arange(n + 1, dtype=torch.int64, device=DEV), conv=rn(d, 4, scale=0.3), y=torch.empty((n, d), dtype=BF16, device=DEV),
                g1=(1 + rn(d, scale=0.1)).to(BF16), g2=(1 + rn(d, scale=0.1)).to(BF16), n1=torch.empty((n, d), dtype=BF16, device=DEV),
                stream=rn(n, d).to(BF16), router=rn(d, e + 2, scale=d ** -0.5).to(BF16), bias=rn(e, scale=0.05),
                ids=torch.empty((n, k + 2), dtype=torch.int32, device=DEV), wts=torch.empty((n, k + 2), device=DEV),
                w_in=rn(e + 2, d, 2 * h, scale=d ** -0.5).to(BF16), w_out=rn(e + 2, h, d, scale=h ** -0.5).to(BF16),
                moe=torch.empty((n, d), dtype=BF16, device=DEV), n2=torch.empty((n, d), dtype=E4M3, device=DEV),
                sc=torch.empty((n, -(-d // 128)), device=DEV)), rn(n, d).to(BF16), rn(n, 3, d).to(BF16)


def workspace_for(s):
    e, h, d = s["w_out"].shape
    n, slots = s["ids"].shape
    return torch.empty(dmel.dmel_experts_workspace_size(n, slots, e, d, h), dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("n", [1, 5, 150])
def test_block_against_the_oracle(n, oracle_mod):
    """The run of calls a decoder layer makes, each against the oracle on what it was given."""
    s, x, state = block_state(70 + n, n)
    before, stream0 = state.clone(), s["stream"].clone()
    # keep what the first norm leaves in the stream
    dmel.dmel_shortconv(x, s["off"], s["conv"], s["y"], state=state.clone())
    mid = torch.empty_like(stream0)
    dmel.dmel_add_rmsnorm(s["y"], s["g1"], s["n1"], residual=stream0, residual_out=mid)
    logits = block_step(s, x, state, workspace_for(s))
    ry, _ = oracle_mod.shortconv(f64(x), s["off"].cpu().numpy(), f64(s["conv"]), f64(before))
    assert (np.abs(f64(s["y"]) - ry) <= 2.0 ** -7 * (np.abs(ry) + 0.1)).all()
    r1, y1 = oracle_mod.add_rmsnorm(f64(s["y"]), f64(stream0), f64(s["g1"]), 1e-6)
    assert (np.abs(f64(mid) - r1) <= 2.0 ** -8 * 1.01 * np.abs(r1)).all()
    assert (np.abs(f64(s["n1"]) - y1) <= (2.0 ** -8 * 1.01 + norm_bound(264)) * np.abs(y1)).all()
    ids, _ = oracle_mod.route(f64(logits), 2, 3, True, f64(s["bias"]))
    np.testing.assert_array_equal(s["ids"].cpu().numpy(), ids)
    assert (s["ids"][:, 3:] == torch.tensor([16, 17], device=DEV)).all()
    ref, _, spread, size = oracle_mod.experts(f64(s["n1"]), ids, f64(s["wts"]), f64(s["w_in"]), f64(s["w_out"]))
    assert (np.abs(f64(s["moe"]) - ref) <= 2.0 ** -8 * 1.01 * np.abs(ref) + 1.01 * spread + 2.0 ** -11 * size + 1e-6 * np.abs(ref)).all()
    r2, y2, sc2 = oracle_mod.add_rmsnorm(f64(s["moe"]), f64(mid), f64(s["g2"]), 1e-6, 128)
    assert (np.abs(f64(s["stream"]) - r2) <= 2.0 ** -8 * 1.01 * np.abs(r2)).all()
    each = np.repeat(sc2, 128, axis=1)[:, :264]
    q = y2 / each
    assert (np.abs(f64(s["n2"].float()) - q) <= (2.0 ** -4 + 1e-5) * np.abs(q) + 2.0 ** -10).all()
    assert dmel.dmel_get_device_error(clear=True) == 0


@pytest.mark.parametrize("n", [3, 20, 400])
def test_calls_that_follow_at_once(n):
    """Each call reads what the one before wrote and reuses its workspace: a chain of calls without a pause
    gives the bits of the same calls one at a time."""
    s, x, state = block_state(90 + n, n)
    ws = workspace_for(s)
    names = ("y", "n1", "stream", "ids", "wts", "moe", "n2", "sc")

    def chain(sync):
        kept, st = [], state.clone()
        inp = x.clone()
        for _ in range(12):
            block_step(s, inp, st, ws) if not sync else stepwise(inp, st)
            kept.append([s[k].clone() for k in names])
            inp.copy_(s["moe"])
        torch.cuda.synchronize()
        return kept

    def stepwise(inp, st):
        old = {f: getattr(dmel, f) for f in ("dmel_shortconv", "dmel_add_rmsnorm", "dmel_route", "dmel_experts")}
        for f, call in old.items():
            setattr(dmel, f, lambda *a, _call=call, **kw: (torch.cuda.synchronize(), _call(*a, **kw), torch.cuda.synchronize()))
        try:
            block_step(s, inp, st, ws)
        finally:
            for f, call in old.items():
                setattr(dmel, f, call)

    start = {k: s[k].clone() for k in names}
    runs = []
    for sync in (True, False, False):
        for k in names:
            s[k].copy_(start[k])
        runs.append(chain(sync))
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            for k, p, q in zip(names, a, b):
                assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), k
    # without anything between: the residual stream through 40 norms, and one expert call after another
    w, r = s["g1"], start["stream"].clone()
    for _ in range(40):
        dmel.dmel_add_rmsnorm(r, w, r, residual=start["stream"])
    one = start["stream"].clone()
    for _ in range(40):
        dmel.dmel_add_rmsnorm(one, w, one, residual=start["stream"])
        torch.cuda.synchronize()
    assert torch.equal(r, one)
    outs = [torch.empty_like(s["moe"]) for _ in range(8)]
    xs = [torch.roll(x, i, 0).contiguous() for i in range(8)]
    for a, b in zip(xs, outs):
        dmel.dmel_experts(a, s["ids"], s["wts"], s["w_in"], s["w_out"], b, ws)
    for a, b in zip(xs, outs):
        alone = torch.empty_like(b)
        torch.cuda.synchronize()
        dmel.dmel_experts(a, s["ids"], s["wts"], s["w_in"], s["w_out"], alone, ws)
        assert torch.equal(alone, b)
    assert dmel.dmel_get_device_error(clear=True) == 0


def test_block_in_graphs_and_on_other_streams():
    """Captured and replayed with new inputs, two graphs with a workspace each replayed at the same time on
    two streams, and calls on a stream that is not the current one: the same bits as eager calls."""
    runs = []
    for seed in (80, 81):
        s, x, state = block_state(seed, 37)
        ws = workspace_for(s)
        x2 = torch.roll(x, 1, 0)
        want = []
        first = {k: v.clone() for k, v in dict(stream=s["stream"], state=state).items()}
        for xi in (x, x2):
            block_step(s, xi, state, ws)
            want.append({k: s[k].clone() for k in ("y", "n1", "ids", "wts", "moe", "stream", "sc")} | {"n2": s["n2"].view(torch.uint8).clone()})
        s["stream"].copy_(first["stream"]); state.copy_(first["state"])
        buf = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block_step(s, buf, state, ws, stream=torch.cuda.current_stream())
        s["stream"].copy_(first["stream"]); state.copy_(first["state"])
        runs.append((s, state, buf, (x, x2), want, graph, first, ws))

    def same(s, w):
        got = {k: s[k] for k in w if k != "n2"} | {"n2": s["n2"].view(torch.uint8)}
        return all(torch.equal(got[k], w[k]) for k in w)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(2):
        for (s, state, buf, xs, want, graph, first, ws), st in zip(runs, streams):
            with torch.cuda.stream(st):
                buf.copy_(xs[i])
                graph.replay()
        torch.cuda.synchronize()
        for s, state, buf, xs, want, graph, first, ws in runs:
            assert same(s, want[i]), i
    # eager on the side streams, given by argument for the library's calls
    for s, state, buf, xs, want, graph, first, ws in runs:
        s["stream"].copy_(first["stream"]); state.copy_(first["state"])
    torch.cuda.synchronize()
    for i in range(2):
        for (s, state, buf, xs, want, graph, first, ws), st in zip(runs, streams):
            with torch.cuda.stream(st):  # (torch.matmul of the step goes by the current stream)
                block_step(s, xs[i], state, ws, stream=st)
        torch.cuda.synchronize()
        for s, state, buf, xs, want, graph, first, ws in runs:
            assert same(s, want[i]), i
    del runs


def test_block_captured_behind_a_join_of_streams():
    """Calls captured right behind a copy and behind the join of another stream, where a launch has several
    predecessors of several kinds: the same bits as eager calls, for new inputs too."""
    s, x, state = block_state(82, 29)
    ws = workspace_for(s)
    buf, other = x.clone(), torch.empty_like(s["stream"])
    side = torch.cuda.Stream()
    first = s["stream"].clone()

    def calls(main):
        # the norm behind the join of a copy on the side and the stream's own copy
        side.wait_stream(main)
        with torch.cuda.stream(side):
            other.copy_(first)
            other.mul_(2)
        s["y"].copy_(buf)
        main.wait_stream(side)
        dmel.dmel_add_rmsnorm(s["y"], s["g1"], s["n1"], residual=other, residual_out=s["stream"])
        # the router on the side, the experts behind its join
        logits = torch.matmul(s["n1"], s["router"]).float()
        side.wait_stream(main)
        dmel.dmel_route(logits, s["ids"], s["wts"], n_shared=2, bias=s["bias"], stream=side)
        s["moe"].zero_()
        main.wait_stream(side)
        dmel.dmel_experts(s["n1"], s["ids"], s["wts"], s["w_in"], s["w_out"], s["moe"], ws)
        dmel.dmel_add_rmsnorm(s["moe"], s["g2"], s["n2"], residual=s["stream"], residual_out=s["stream"], scales=s["sc"],
                              scale_block=128)
        return logits  # (kept: the side stream reads it)

    names = ("n1", "stream", "ids", "wts", "moe", "n2", "sc")
    want, inputs = [], (x, torch.roll(x, 1, 0), torch.roll(x, 2, 0))
    for xi in inputs:
        buf.copy_(xi)
        keep = calls(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append([s[k].clone() for k in names])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        keep = calls(torch.cuda.current_stream())  # noqa: F841
    for _ in range(2):
        for xi, old in zip(inputs, want):
            buf.copy_(xi)
            graph.replay()
            torch.cuda.synchronize()
            for k, v in zip(names, old):
                assert torch.equal(s[k].view(torch.uint8), v.view(torch.uint8)), k
    assert dmel.dmel_get_device_error(clear=True) == 0
