"""CPU tests of the decoder-block operators (residual addition with RMSNorm, routing, experts): what the
ABI and the binding refuse, workspace sizes, and pins of the fp64 oracle they are compared with."""
import ctypes

import numpy as np
import pytest
import torch

from encoder_free_audio_b200 import build, dmel

INVALID = dmel.DMEL_ERR_INVALID_ARG
VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dmel.library()


def at(i):
    """Address number i of buffers far apart (never dereferenced: the call fails its checks first)."""
    return (i + 1) << 40


# ------------------------------------------------------------------------------ the C ABI refuses

NORM = dict(x=at(0), residual=at(1), n=4, dim=64, dtype=dmel.DMEL_BF16, w=at(2), eps=1e-6, residual_out=at(3), out=at(4),
            out_dtype=dmel.DMEL_BF16, scales=None, block=0)


def norm(lib, **kw):
    a = {**NORM, **kw}
    return lib.dmel_add_rmsnorm(a["x"], a["residual"], a["n"], a["dim"], a["dtype"], a["w"], a["eps"], a["residual_out"],
                                a["out"], a["out_dtype"], a["scales"], a["block"], None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(dim=0), dict(dim=60), dict(dim=-8), dict(dim=16392), dict(dtype=dmel.DMEL_E4M3), dict(dtype=7),
    dict(out_dtype=3), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=None), dict(w=None), dict(out=None), dict(x=at(0) + 2), dict(w=at(2) + 8), dict(out=at(4) + 8),
    dict(residual=at(1) + 4), dict(residual_out=at(3) + 4),
    dict(scales=at(5)), dict(block=128),                                     # not an e4m3 output
    dict(out_dtype=dmel.DMEL_E4M3), dict(out_dtype=dmel.DMEL_E4M3, scales=at(5) + 2),
    dict(out_dtype=dmel.DMEL_E4M3, scales=at(5), out=at(4) + 4), dict(out_dtype=dmel.DMEL_E4M3, scales=at(5), block=48),
    dict(out_dtype=dmel.DMEL_E4M3, scales=at(5), block=-32),
    dict(out=at(0) + 16), dict(out=at(0), out_dtype=dmel.DMEL_F32), dict(residual_out=at(1) + 64),
    dict(out=at(3)), dict(out=at(2)), dict(residual_out=at(2)),
    dict(out_dtype=dmel.DMEL_E4M3, scales=at(4) + 16), dict(out_dtype=dmel.DMEL_E4M3, scales=at(0)),
])
def test_add_rmsnorm_refuses(lib, bad):
    assert norm(lib, **bad) == INVALID


def test_add_rmsnorm_no_rows_is_a_no_op(lib):
    assert norm(lib, n=0, x=None, w=None, out=None) == dmel.DMEL_OK
    assert dmel.dmel_last_launch_count() == 0


ROUTER = dict(n_experts=16, n_shared=2, top_k=4, n_groups=4, topk_groups=2, scoring=dmel.DMEL_ROUTE_SIGMOID, renormalise=1,
              scale=1.0)


def route(lib, router=None, logits=at(0), n=4, dtype=dmel.DMEL_F32, bias=at(1), ids=at(2), weights=at(3)):
    return lib.dmel_route(logits, n, dtype, bias, None if router is None else dmel.Router(**router), ids, weights, None)


@pytest.mark.parametrize("bad", [
    dict(n_experts=0), dict(n_experts=1028), dict(n_shared=-1), dict(top_k=0), dict(top_k=9), dict(n_groups=0),
    dict(n_groups=3), dict(n_groups=33, n_experts=66), dict(topk_groups=0), dict(topk_groups=5), dict(scoring=2),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(n_experts=64, top_k=31), dict(n_shared=40),
])
def test_route_refuses_settings(lib, bad):
    assert route(lib, {**ROUTER, **bad}) == INVALID


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(dtype=dmel.DMEL_E4M3), dict(logits=None), dict(ids=None), dict(weights=None), dict(logits=at(0) + 2),
    dict(bias=at(1) + 2), dict(ids=at(2) + 2), dict(weights=at(3) + 1), dict(ids=at(3)), dict(ids=at(0) + 32),
    dict(weights=at(1)),
])
def test_route_refuses_buffers(lib, bad):
    assert route(lib, ROUTER, **bad) == INVALID
    assert route(lib, None) == INVALID
    assert route(lib, ROUTER, n=0, logits=None, ids=None, weights=None) == dmel.DMEL_OK


EXPERTS = dict(n_experts=8, dim=64, hidden=32, w_in=at(5), w_out=at(6))


def experts(lib, w=EXPERTS, x=at(0), n=4, ids=at(1), weights=at(2), slots=2, out=at(3), workspace=at(4), size=None):
    ws = None if w is None else dmel.ExpertWeights(**w)
    if size is None:
        size = lib.dmel_experts_workspace_size(max(n, 0), slots, ws) if ws is not None else 0
    return lib.dmel_experts(x, n, ids, weights, slots, ws, out, workspace, size, None)


@pytest.mark.parametrize("bad", [
    dict(n_experts=0), dict(n_experts=1025), dict(dim=0), dict(dim=60), dict(dim=65544), dict(hidden=0), dict(hidden=4),
    dict(hidden=65544), dict(w_in=None), dict(w_out=None), dict(w_in=at(5) + 8), dict(w_out=at(6) + 2), dict(w_in=at(3)),
])
def test_experts_refuses_weights(lib, bad):
    assert experts(lib, {**EXPERTS, **bad}, size=1 << 30) == INVALID


@pytest.mark.parametrize("bad", [
    dict(w=None, size=1 << 30), dict(n=-1), dict(slots=0), dict(slots=65), dict(n=1 << 30, size=1 << 62), dict(x=None),
    dict(ids=None), dict(weights=None), dict(out=None), dict(workspace=None), dict(workspace=at(4) + 128),
    dict(x=at(0) + 2), dict(ids=at(1) + 2), dict(weights=at(2) + 2), dict(out=at(3) + 8), dict(out=at(0)),
    dict(out=at(4) + 256), dict(workspace=at(5)), dict(size=16),
])
def test_experts_refuses(lib, bad):
    assert experts(lib, **bad) == INVALID


def test_experts_no_tokens_is_a_no_op(lib):
    assert experts(lib, n=0, x=None, out=None, workspace=None) == dmel.DMEL_OK


def test_experts_workspace_size(lib):
    size = dmel.dmel_experts_workspace_size
    assert size(0, 6, 32, 6144, 1024) == 0 and size(5, 0, 32, 6144, 1024) == 0 and size(5, 6, 0, 6144, 1024) == 0
    rows = 4096 * 6
    # the gated rows in bf16, the outputs per slot in 16 bits with a scale per 128 columns, and the plan: rows and tokens of the slots,
    # tiles of 256 tokens and one more per expert
    need = rows * (1024 * 2 + 6144 * 2 + 48 * 4) + rows * 8 + (rows // 256 + 32) * 16
    assert need <= size(4096, 6, 32, 6144, 1024) <= need + 6 * 256 + 256


# (slots, experts, dim, hidden) and the largest batch: rows in fp32 up to 64 slots; K in parts, in the small calls, in
# tiles of 32, 128 and 256 tokens; neither
BATCHES = [(6, 32, 6144, 1024, 300), (1, 2, 4096, 512, 2200), (2, 3, 2056, 72, 700), (3, 7, 2056, 520, 800),
           (64, 5, 64, 24, 40), (1, 1, 65536, 8, 10000), (8, 258, 6144, 64, 700), (1, 1024, 24, 16, 3000)]


@pytest.mark.parametrize("slots,e,d,h,most", BATCHES)
def test_experts_workspace_of_a_batch_serves_smaller_ones(lib, slots, e, d, h, most):
    sizes = [dmel.dmel_experts_workspace_size(t, slots, e, d, h) for t in range(most + 1)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    w = dict(n_experts=e, dim=d, hidden=h, w_in=at(5), w_out=at(6))
    fits = lambda t, size: experts(lib, w, n=t, slots=slots, workspace=at(4), size=size) != INVALID  # noqa: E731
    assert all(fits(t, sizes[most]) for t in range(1, most + 1))
    assert all(fits(t, sizes[t]) for t in range(1, most + 1))
    # no more than the neediest of the batches
    assert not all(fits(t, sizes[most] - 1) for t in range(1, most + 1))


def test_experts_workspace_size_of_the_largest_calls(lib):
    size = dmel.dmel_experts_workspace_size
    assert size(1 << 30, 1, 1024, 65536, 65536) > (1 << 30) * 65536 * 4
    assert size((1 << 30) // 64, 64, 1, 8, 8) > size(1 << 20, 64, 1, 8, 8)


# ------------------------------------------------------------------------------ the binding refuses

def test_route_settings_held_in_tensors_are_read_at_each_call(monkeypatch):
    """A scale or a count that the caller keeps in a tensor and changes there."""
    seen = []
    monkeypatch.setattr(dmel, "_run_on", lambda device, stream, where, entry, *args: seen.append(args[4]))
    scale, groups = torch.tensor(2.5), torch.tensor(2)
    for s, k in ((2.5, 2), (7.0, 4)):
        scale.fill_(s)
        groups.fill_(k)
        dmel.dmel_route(torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), scale=scale,
                        n_groups=groups, topk_groups=groups)
        assert (seen[-1].scale, seen[-1].n_groups, seen[-1].topk_groups) == (s, k, k)
    for bad in (dict(n_groups=2.0), dict(n_shared=0.5), dict(scoring="1"), dict(scale=None)):
        with pytest.raises(TypeError):
            dmel.dmel_route(torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), **bad)



def test_binding_refuses_what_c_cannot_see(lib):
    f, b = torch.float32, torch.bfloat16
    x, w = torch.zeros(4, 64), torch.ones(64)
    for what, call in {
        "rows, dim": lambda: dmel.dmel_add_rmsnorm(x[0], w, x[0].clone()),
        "strides": lambda: dmel.dmel_add_rmsnorm(torch.zeros(64, 4).t(), w, torch.zeros(4, 64)),
        "rms_weight": lambda: dmel.dmel_add_rmsnorm(x, w.to(b), torch.zeros(4, 64)),
        "out:": lambda: dmel.dmel_add_rmsnorm(x, w, torch.zeros(4, 72)),
        "residual:": lambda: dmel.dmel_add_rmsnorm(x, w, torch.zeros(4, 64), residual=torch.zeros(3, 64)),
        "residual_out": lambda: dmel.dmel_add_rmsnorm(x, w, torch.zeros(4, 64), residual_out=torch.zeros(4, 64, dtype=b)),
        "scales": lambda: dmel.dmel_add_rmsnorm(x, w, torch.zeros(4, 64).to(torch.float8_e4m3fn), scales=torch.zeros(4, 3),
                                                scale_block=32),
        "want a CUDA device": lambda: dmel.dmel_add_rmsnorm(x, w, torch.zeros(4, 64)),
        "ids:": lambda: dmel.dmel_route(x, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)),
        "weights:": lambda: dmel.dmel_route(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 3)),
        "bias:": lambda: dmel.dmel_route(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), bias=torch.zeros(63)),
        "two dimensions": lambda: dmel.dmel_route(x, torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2)),
    }.items():
        with pytest.raises(dmel.DmelError, match=what) as e:
            call()
        assert e.value.status == INVALID
    with pytest.raises(TypeError):
        dmel.dmel_add_rmsnorm(x.half(), w.half(), torch.zeros(4, 64))
    xb, ids, wt = torch.zeros(4, 64, dtype=b), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w_in, w_out, ws = torch.zeros(8, 64, 64, dtype=b), torch.zeros(8, 32, 64, dtype=b), torch.zeros(1 << 16, dtype=torch.uint8)
    for what, a in {
        "x:": (x, ids, wt, w_in, w_out, xb.clone(), ws), "w_in": (xb, ids, wt, w_in[:, :, :32], w_out, xb.clone(), ws),
        "out:": (xb, ids, wt, w_in, w_out, x, ws), "ids:": (xb, ids.long(), wt, w_in, w_out, xb.clone(), ws),
        "weights:": (xb, ids, wt.to(b), w_in, w_out, xb.clone(), ws), "dimensions": (xb, ids, wt, w_in, w_out[0], xb, ws),
        "workspace": (xb, ids, wt, w_in, w_out, xb.clone(), torch.zeros(1 << 16, dtype=f)),
        "want a CUDA device": (xb, ids, wt, w_in, w_out, xb.clone(), ws),
    }.items():
        with pytest.raises(dmel.DmelError, match=what):
            dmel.dmel_experts(*a)


def test_binding_runs_on_the_tensors_device(monkeypatch):
    """A call on device 1 while device 0 is current: made with device 1 current, on its current stream or on a
    stream of its own, never on another device's."""
    import contextlib
    current = [0]

    @contextlib.contextmanager
    def on(index):
        current.append(index)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    calls = []

    def entry(*args):
        calls.append((current[-1], args))
        return dmel.DMEL_OK

    dmel._run_on(1, None, "call", entry, 5)
    dmel._run_on(0, None, "call", entry, 6)

    class Stream:
        device_index, device, cuda_stream = 1, "cuda:1", 77

    dmel._run_on(1, Stream, "call", entry, 7)
    assert calls == [(1, (5, 1001)), (0, (6, 1000)), (1, (7, 77))] and current == [0]
    with pytest.raises(dmel.DmelError, match="a stream of cuda:1"):
        dmel._run_on(0, Stream, "call", entry, 8)


# ------------------------------------------------------------------------------ pins of the oracle

def test_oracle_add_rmsnorm_closed_form(oracle_mod):
    """Equal values c give w_j sign(c) (eps small); torch's rms_norm in fp64; scales of known blocks."""
    w = np.linspace(0.5, 2.0, 72)
    s, y, sc = oracle_mod.add_rmsnorm(np.full((1, 72), -3.0), np.full((1, 72), 1.0), w, 1e-300, 32)
    np.testing.assert_allclose(s, -2.0)
    np.testing.assert_allclose(y[0], -w, rtol=1e-14)
    np.testing.assert_allclose(sc[0], [w[31] / 448, w[63] / 448, w[71] / 448], rtol=1e-14)
    r = np.random.default_rng(1)
    x, z = r.standard_normal((5, 40)), r.standard_normal((5, 40))
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x + z), (40,), torch.from_numpy(w[:40]), 1e-6)
    np.testing.assert_allclose(oracle_mod.add_rmsnorm(x, z, w[:40], 1e-6)[1], ref.numpy(), rtol=1e-12)


def test_oracle_route_by_hand(oracle_mod):
    l = np.array([[0.0, 2.0, 2.0, -1.0, 0.0, np.nan, -np.inf, 1.0, 0.5]])  # 8 experts, 1 shared
    ids, w = oracle_mod.route(l, 1, 4, True)
    assert ids.tolist() == [[1, 2, 7, 0, 8]]
    sg = 1 / (1 + np.exp(-np.array([2.0, 2.0, 1.0, 0.0, 0.5])))
    np.testing.assert_allclose(w[0], sg / sg.sum(), rtol=1e-14)
    # groups of two rate 0.5 + 0.88, 0.88 + 0.27, 0.5 (its other expert is masked), 0.73 (likewise)
    ids, _ = oracle_mod.route(l, 1, 2, True, bias=np.zeros(8), n_groups=4, topk_groups=1)
    assert ids.tolist() == [[1, 0, 8]]
    ids, _ = oracle_mod.route(l, 1, 4, True, bias=np.zeros(8), n_groups=4, topk_groups=3)
    assert ids.tolist() == [[1, 2, 7, 0, 8]]
    # fewer experts than slots
    m = np.full((1, 5), -np.inf)
    m[0, 3] = 0.25
    ids, w = oracle_mod.route(m, 1, 3, False)
    assert ids.tolist() == [[3, -1, -1, -1]] and w.tolist() == [[1.0, 0.0, 0.0, 0.0]]
    ids, w = oracle_mod.route(np.full((1, 4), -np.inf), 0, 2, False)
    assert ids.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]


def test_oracle_experts_by_hand(oracle_mod):
    """A gate of 64 (silu(64) = 64 in fp64 to 1e-28) and identity-like products."""
    x = np.array([[1.0, 0.0]])
    w_in = np.zeros((2, 2, 4))
    w_in[1, 0] = [64.0, 64.0, 2.0, -3.0]
    w_out = np.zeros((2, 2, 3))
    w_out[1] = [[1.0, 0.0, 2.0], [0.0, 1.0, 1.0]]
    out, h, _, size = oracle_mod.experts(x, np.array([[1, -1]]), np.array([[0.5, 9.0]]), w_in, w_out)
    np.testing.assert_allclose(h[0, 0], [128.0, -192.0], rtol=1e-14)
    np.testing.assert_allclose(out[0], [64.0, -96.0, 32.0], rtol=1e-14)
    np.testing.assert_allclose(size[0], [64.0, 96.0, 32.0], rtol=1e-14)
