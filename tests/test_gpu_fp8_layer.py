"""The FP8 operators together, as they are used: a layer's forward pass (routing, quantiser, gate/up
product with SwiGLU and requantisation, down product, finalize), a training step of an expert
projection beside the router's balance term, on other streams and in replayed HIP graphs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_02_amd as moe
from tests import fp8_ref as ref
from tests.fp8_ref import U16, U32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    yield
    torch.cuda.synchronize()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *s, scale=1.0, dt=torch.bfloat16):
    return (scale * torch.randn(*s, generator=g, device="cuda")).to(dt)


def _rows(t):
    return ref.rows_value(t.q.cpu().numpy(), t.sf.cpu().numpy())


def _tiles(t):
    return ref.weights_value(t.q.cpu().numpy(), t.sf.cpu().numpy())


def _weights(g, E, H, I):
    return (moe.quantize_fp8_weights_alloc(_randn(g, E, 2 * I, H, scale=0.05)),
            moe.quantize_fp8_weights_alloc(_randn(g, E, H, I, scale=0.05)))


LAYERS = {"one token": (1, 16, 4, 512, 128), "few tokens": (9, 8, 2, 272, 256), "many tokens": (700, 12, 3, 400, 128),
          "large tiles": (1300, 16, 4, 1040, 1024)}


@pytest.mark.parametrize("layer", LAYERS)
def test_layer_forward(layer):
    """Each stage against 64 bits on what the stage before it gave (a code of the requantised act
    next to a border may fall either way, so the stages are held one by one)."""
    T, E, k, H, I = LAYERS[layer]
    g = _gen(T + E)
    W1, W2 = _weights(g, E, H, I)
    logits, x = _randn(g, T, E, dt=torch.float32), _randn(g, T, H)
    plan = moe.MoEFP8LayerPlan(T, E, k, H, I, W1, W2)
    out = plan.forward(logits, x).double().cpu().numpy()
    ids, w, off, src, tsr = (t.cpu().numpy() for t in (plan.ids, plan.w, plan.off, plan.row_src, plan.tsr))
    assert np.array_equal(np.sort(ids, 1), np.sort(logits.topk(k, 1).indices.cpu().numpy(), 1))
    assert np.array_equal(off[1:] - off[:-1], np.bincount(ids.ravel(), minlength=E))
    q, s = ref.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(plan.xq.q.cpu().numpy(), q) and np.array_equal(plan.xq.sf.cpu().numpy(), s)
    y, mag = ref.product(ref.rows_value(q, s), _tiles(W1), off, src)
    gate, up, e = y[:, :I], y[:, I:], ref.core_error(H) * mag
    act = ref.swiglu(y)
    silu = gate / (1 + np.exp(-gate))
    tol = 1.1 * np.abs(up) * e[:, :I] + (np.abs(silu) + e[:, :I]) * e[:, I:] + (8 + 2 * np.abs(gate)) * 2 * U32 * np.abs(act)
    aq = _rows(plan.actq)
    sf = np.repeat(plan.actq.sf.cpu().numpy().astype(np.float64), 128, 1)
    assert (np.abs(aq - act) <= (np.abs(act) + tol) * 2.0 ** -4 + sf * 2.0 ** -10 + tol + 4 * U32 * np.abs(act)).all()
    Y, mag = ref.product(aq, _tiles(W2), off)
    got = plan.Y.double().cpu().numpy()
    assert (np.abs(got - Y) <= U16 * np.abs(Y) + (1 + U16) * ref.core_error(I) * mag).all()
    terms = w[:, :, None].astype(np.float64) * got[tsr.reshape(T, k)]
    want, mag = terms.sum(1), np.abs(terms).sum(1)
    assert (np.abs(out - want) <= U16 * np.abs(want) + 2 * k * U32 * mag).all()


def _training_step(x, w, dy, logits, ids, off, src, R, topk_w, d_topk_w, grad):
    """What a training loop calls for one expert projection and the router."""
    W, Wt = moe.quantize_fp8_weights_alloc(w, transposed=True)
    xq, dyq = moe.quantize_fp8_alloc(x), moe.quantize_fp8_alloc(dy)
    y = moe.grouped_gemm_fp8_alloc(xq, W, off, R, A_rows=src)
    dx = moe.grouped_gemm_fp8_alloc(dyq, Wt, off, R)
    Yt, Xt = moe.quantize_fp8_tokens_alloc(dy, off, R), moe.quantize_fp8_tokens_alloc(x, off, R, rows=src)
    dw = moe.grouped_wgrad_fp8_alloc(Yt, Xt, off, R)
    loss, counts, coef = moe.balance_loss_alloc(logits, ids)
    dl = torch.empty_like(logits)
    moe.moe_balance_loss_backward(logits, coef, grad, dl, None, None, ids, topk_w, d_topk_w)
    return dict(y=y, dx=dx, dw=dw, loss=loss, counts=counts, dl=dl), (W, xq, dyq, Yt, Xt)


def _training_inputs(seed, T=150, E=6, k=2, N=272, K=400):
    g = _gen(seed)
    logits = _randn(g, T, E, dt=torch.float32)
    ids, w, off, src, _ = moe.route_permute_alloc(logits, k)
    R = T * k
    return dict(x=_randn(g, T, K), w=_randn(g, E, N, K, scale=0.05), dy=_randn(g, R, N, scale=1e-3), logits=logits, ids=ids, off=off,
                src=src, R=R, topk_w=w, d_topk_w=_randn(g, T, k, dt=torch.float32), grad=torch.full((1,), 0.01, device="cuda"))


def test_training_step():
    a = _training_inputs(3)
    got, (W, xq, dyq, Yt, Xt) = _training_step(**a)
    off, src = a["off"].cpu().numpy(), a["src"].cpu().numpy()
    wv = _tiles(W)
    for key, av, wm, rows in (("y", _rows(xq), wv, src), ("dx", _rows(dyq), wv.transpose(0, 2, 1), None)):
        want, mag = ref.product(av, wm, off, rows)
        err = np.abs(got[key].double().cpu().numpy() - want)
        assert (err <= U16 * np.abs(want) + (1 + U16) * ref.core_error(wm.shape[2]) * mag).all(), key
    n = sum(-(-int(s) // 128) for s in np.diff(off))
    want, mag = ref.wgrad(ref.tokens_value(Yt.q[:n].cpu().numpy(), Yt.sf[:n].cpu().numpy()),
                          ref.tokens_value(Xt.q[:n].cpu().numpy(), Xt.sf[:n].cpu().numpy()), off)
    assert (np.abs(got["dw"].double().cpu().numpy() - want) <= U32 * np.abs(want) + ref.sum_error(a["R"]) * mag).all()
    # against the gradients of the unquantised product: FP8 keeps 2^-4 per operand at worst, whose
    # errors add up at random over the contraction, so 2^-4 of the 2-norm is far outside
    x, w, dy = a["x"].double().cpu()[src.astype(np.int64)], a["w"].double().cpu(), a["dy"].double().cpu()
    for e in range(len(off) - 1):
        s = slice(off[e], off[e + 1])
        for key, want in (("y", x[s] @ w[e].T), ("dx", dy[s] @ w[e])):
            assert (got[key][s].double().cpu() - want).norm() <= 2.0 ** -4 * want.norm()
        want = dy[s].T @ x[s]
        assert (got["dw"][e].double().cpu() - want).norm() <= 2.0 ** -4 * want.norm()
    assert torch.equal(got["counts"][0], a["off"][1:] - a["off"][:-1])


def test_work_on_another_stream():
    """Inputs made, operators called and results read on a side stream, with the default stream busy."""
    a = _training_inputs(5)
    want, _ = _training_step(**a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.randn(2048, 2048, device="cuda")
    for _ in range(20):
        busy = busy @ busy * 1e-3
    with torch.cuda.stream(side):
        a = {k: v.clone() if torch.is_tensor(v) else v for k, v in a.items()}
        got, _ = _training_step(**a)
    side.synchronize()
    for key in want:
        assert torch.equal(want[key].view(torch.uint8), got[key].view(torch.uint8)), key
    torch.cuda.synchronize()


def test_stream_argument():
    """The allocating helpers given a stream: what they allocate belongs to that stream, so memory that
    the current stream's queued work still holds is not written."""
    a = _training_inputs(6)
    want, _ = _training_step(**a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        junk = [torch.randn(1 << 20, device="cuda") for _ in range(8)]
        held = [(j * 2).sum() for j in junk]
        del junk
        W = moe.quantize_fp8_weights_alloc(a["w"], stream=side)
        y = moe.grouped_gemm_fp8_alloc(moe.quantize_fp8_alloc(a["x"], side), W, a["off"], a["R"], A_rows=a["src"], stream=side)
        loss, counts, coef = moe.balance_loss_alloc(a["logits"], a["ids"], stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want["y"].view(torch.int16))
        assert torch.equal(loss, want["loss"]) and torch.equal(counts, want["counts"])
        del held


def test_token_gradient_is_finalize_with_unit_weights():
    """A token's rows of dx, summed by moe_finalize with weights of one."""
    a = _training_inputs(9)
    T, k, H = a["x"].shape[0], 2, a["x"].shape[1]
    *_, tsr = moe.route_permute_alloc(a["logits"], k)
    dx = _training_step(**a)[0]["dx"]
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_finalize(dx, torch.ones(T, k, device="cuda"), tsr, out)
    rows = dx.double()[tsr.view(T, k).long()]
    assert ((out.double() - rows.sum(1)).abs() <= U16 * rows.sum(1).abs() + 2 * k * U32 * rows.abs().sum(1)).all()


def test_two_streams_at_once():
    """Two independent steps on two streams do not touch each other (each has its own workspace)."""
    ins = [_training_inputs(s, T=400) for s in (7, 8)]
    want = [_training_step(**a)[0] for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] = _training_step(**ins[i])[0]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for key in w:
                assert torch.equal(w[key].view(torch.uint8), g[key].view(torch.uint8)), key


def test_graph_replays_match_eager():
    """The training step and the layer's forward pass captured; every replay, with other inputs copied
    in, eager work and synchronisations between, gives the eager bytes."""
    ins = [_training_inputs(s) for s in (20, 21)]
    refs = [{k: v.clone() for k, v in _training_step(**a)[0].items()} for a in ins]
    static = {k: v.clone() if torch.is_tensor(v) else v for k, v in ins[0].items()}
    _training_step(**static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, _ = _training_step(**static)
    for r in range(4):
        which = r % 2
        for k, v in static.items():
            if torch.is_tensor(v):
                v.copy_(ins[which][k])
        for v in outs.values():
            v.view(torch.uint8).fill_(0xA5 - r)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for key, want in refs[which].items():
            assert torch.equal(outs[key].view(torch.uint8), want.view(torch.uint8)), (r, key)
        _training_step(**ins[1 - which])
        torch.cuda.synchronize()


def test_layer_graph_replays_match_eager():
    T, E, k, H, I = 64, 12, 3, 400, 128
    g = _gen(30)
    W1, W2 = _weights(g, E, H, I)
    eager, graphed = (moe.MoEFP8LayerPlan(T, E, k, H, I, W1, W2) for _ in range(2))
    ins = [(_randn(g, T, E, dt=torch.float32), _randn(g, T, H)) for _ in range(2)]
    refs = [eager.forward(*i).clone() for i in ins]
    logits, x = ins[0][0].clone(), ins[0][1].clone()
    graph = graphed.graph(logits, x)
    for r in range(4):
        logits.copy_(ins[r % 2][0])
        x.copy_(ins[r % 2][1])
        graphed.out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphed.out.view(torch.int16), refs[r % 2].view(torch.int16)), r
        eager.forward(*ins[1 - r % 2])
        torch.cuda.synchronize()


def test_binding_refuses_mixed_devices_and_host_tensors():
    g = _gen(1)
    x = _randn(g, 4, 32)
    q, sf = torch.empty(4, 32, dtype=torch.uint8, device="cuda"), torch.empty(4, 1, device="cuda")
    for bad in ((x.cpu(), q, sf), (x, q.cpu(), sf), (x, q, sf.cpu()), (x.cpu(), q.cpu(), sf.cpu())):
        with pytest.raises(moe.MoeError):
            moe.moe_quantize_fp8(*bad)


def test_binding_refuses_a_stream_of_another_device():
    class Elsewhere:
        device_index, cuda_stream = 1, 0
    a = _training_inputs(3)
    X, W = moe.quantize_fp8_alloc(a["x"]), moe.quantize_fp8_weights_alloc(a["w"])
    D = torch.empty(a["R"], a["w"].shape[1], dtype=torch.bfloat16, device="cuda")
    args = moe.make_gemm_fp8_args(X.q, X.sf, W.q, W.sf, a["off"], a["R"], moe.MOE_EPI_NONE, D, A_rows=a["src"])
    calls = [lambda s: moe.moe_grouped_gemm_fp8(args, s), lambda s: moe.moe_quantize_fp8(a["x"], X.q, X.sf, s),
             lambda s: moe.moe_quantize_fp8_weights(a["w"], W.q, W.sf, stream=s)]
    for call in calls:
        with pytest.raises(moe.MoeError):
            call(Elsewhere())
        call(torch.cuda.current_stream())


def test_layer_refuses_other_shapes():
    T, E, k, H, I = 20, 32, 2, 272, 128
    g = _gen(31)
    plan = moe.MoEFP8LayerPlan(T, E, k, H, I, *_weights(g, E, H, I))
    logits, x = _randn(g, T, E, dt=torch.float32), _randn(g, T, H)
    want = plan.forward(logits, x).clone()
    for l, y in ((logits[:-1], x), (logits, x[:-1]), (logits[:, :-16].contiguous(), x), (logits.double(), x), (logits.T, x)):
        with pytest.raises(moe.MoeError):
            plan.forward(l, y)
    assert torch.equal(plan.forward(logits, x).view(torch.int16), want.view(torch.int16))
